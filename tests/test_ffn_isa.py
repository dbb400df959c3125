"""Checks on the gfx950 assembly of the feed-forward products (CPU only): the
matrix instruction of their type, no scratch or memory wait of the compiler's
in a K loop, the wait states of the inline-assembly loads."""
from __future__ import annotations

import re
import subprocess

import pytest

import test_isa as isa


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    from implicit_gemm_convolution_amd import build

    text = open(build.ffn_assembly(str(tmp_path_factory.mktemp("ffn_asm")))).read()
    kernels = {}
    for name in sorted(set(re.findall(r"^\s+\.amdhsa_kernel (\S+)", text, re.M))):
        body = text[re.search(r"^" + re.escape(name) + r":", text, re.M).end():].split(".Lfunc_end", 1)[0]
        meta = text.split(".amdhsa_kernel " + name, 1)[1].split(".end_amdhsa_kernel", 1)[0]
        kernels[subprocess.run(["c++filt", name], capture_output=True, text=True).stdout.strip()] = (body, meta)
    assert kernels
    return kernels


@pytest.fixture(scope="module")
def tiles(asm):
    found = {k: v for k, v in asm.items() if "gemm_tile_kernel<" in k}
    assert found
    return found


def _lines(body):
    out = [l.split(";")[0].strip() for l in body.splitlines()]
    return [l for l in out if l and not l.startswith(".")]


def test_matrix_instruction_of_the_type(asm):
    for name, (body, _) in asm.items():
        m = re.search(r"gemm_(?:any|tile|skinny)_kernel<(true|false)", name)
        if not m:
            continue
        kinds = set(re.findall(r"v_mfma_\w+", body))
        assert kinds == {"v_mfma_f32_16x16x32_bf16" if m.group(1) == "true" else "v_mfma_f32_16x16x32_f16"}, name


def test_no_scratch_in_k_loops_and_lds_within_limit(asm):
    for name, (body, meta) in asm.items():
        lines = _lines(body)
        mf = [i for i, l in enumerate(lines) if l.startswith("v_mfma")]
        if mf:
            assert not any(l.startswith("scratch_") for l in lines[mf[0]:mf[-1] + 1]), name
        assert int(re.search(r"\.amdhsa_group_segment_fixed_size (\d+)", meta).group(1)) <= 160 * 1024, name
        assert int(re.search(r"\.amdhsa_private_segment_fixed_size (\d+)", meta).group(1)) <= 16, name


def test_k_loops_of_the_direct_kernels_have_only_their_own_memory_waits(tiles):
    for name, (body, _) in tiles.items():
        lines = _lines(body)
        mf = [i for i, l in enumerate(lines) if l.startswith("v_mfma")]
        stray = [l for l in lines[mf[0]:mf[-1]] if l.startswith("s_waitcnt") and "vmcnt" in l and "lgkmcnt(0)" not in l]
        assert not stray, (name, stray[:2])


def test_no_packed_fp32(asm):
    for name, (body, _) in asm.items():
        assert not re.search(r"v_pk_(add|mul|fma)_f32", body), name


def test_direct_to_lds_loads_respect_sgpr_hazards(asm):
    isa.test_direct_to_lds_loads_respect_sgpr_hazards(asm)


def test_wide_stores_keep_their_data(asm):
    """As for the other kernels; code after a jump or the program's end does not follow the store."""
    def cut(body):
        return re.sub(r"^(\s*s_(endpgm|branch|setpc_b64)\b.*)$", r"\1\n s_nop 7", body, flags=re.M)

    isa.test_no_vector_write_of_a_wide_store_s_data_right_after_it({k: (cut(b), m) for k, (b, m) in asm.items()})


def test_no_atomics(asm):
    """Results do not depend on the order in which workgroups finish."""
    for name, (body, _) in asm.items():
        assert "atomic" not in body, name

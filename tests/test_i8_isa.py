"""Checks on the gfx950 assembly of the products in 8 bits (CPU only), as for the
16-bit products."""
from __future__ import annotations

import re
import subprocess

import pytest

import test_ffn_isa as ffn


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    from implicit_gemm_convolution_amd import build

    text = open(build.i8_assembly(str(tmp_path_factory.mktemp("i8_asm")))).read()
    kernels = {}
    for name in sorted(set(re.findall(r"^\s+\.amdhsa_kernel (\S+)", text, re.M))):
        body = text[re.search(r"^" + re.escape(name) + r":", text, re.M).end():].split(".Lfunc_end", 1)[0]
        meta = text.split(".amdhsa_kernel " + name, 1)[1].split(".end_amdhsa_kernel", 1)[0]
        kernels[subprocess.run(["c++filt", name], capture_output=True, text=True).stdout.strip()] = (body, meta)
    assert kernels
    return kernels


def test_matrix_instruction_of_the_type(asm):
    found = [n for n in asm if re.search(r"i8_(?:tile|skinny)_kernel<", n)]
    assert found
    for name in found:
        assert set(re.findall(r"v_mfma_\w+", asm[name][0])) == {"v_mfma_i32_16x16x64_i8"}, name


def test_k_loops_of_the_direct_kernels_have_only_their_own_memory_waits(asm):
    ffn.test_k_loops_of_the_direct_kernels_have_only_their_own_memory_waits({k: v for k, v in asm.items() if "i8_tile_kernel<" in k})


def test_no_scratch_in_k_loops_and_lds_within_limit(asm):
    ffn.test_no_scratch_in_k_loops_and_lds_within_limit(asm)


def test_no_packed_fp32(asm):
    ffn.test_no_packed_fp32(asm)


def test_direct_to_lds_loads_respect_sgpr_hazards(asm):
    ffn.test_direct_to_lds_loads_respect_sgpr_hazards(asm)


def test_wide_stores_keep_their_data(asm):
    ffn.test_wide_stores_keep_their_data(asm)


def test_no_atomics(asm):
    ffn.test_no_atomics(asm)

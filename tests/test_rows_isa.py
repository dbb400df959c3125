"""Checks on the gfx950 assembly of the row operators (CPU only): registers hold
their rows, no packed fp32, no atomics."""
from __future__ import annotations

import re
import subprocess

import pytest

import test_ffn_isa as ffn


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    from implicit_gemm_convolution_amd import build

    text = open(build.rows_assembly(str(tmp_path_factory.mktemp("rows_asm")))).read()
    kernels = {}
    for name in sorted(set(re.findall(r"^\s+\.amdhsa_kernel (\S+)", text, re.M))):
        body = text[re.search(r"^" + re.escape(name) + r":", text, re.M).end():].split(".Lfunc_end", 1)[0]
        meta = text.split(".amdhsa_kernel " + name, 1)[1].split(".end_amdhsa_kernel", 1)[0]
        kernels[subprocess.run(["c++filt", name], capture_output=True, text=True).stdout.strip()] = (body, meta)
    assert any("row_kernel<" in k for k in kernels) and any("dropout_kernel<" in k for k in kernels)
    return kernels


def test_rows_stay_in_registers(asm):
    for name, (body, meta) in asm.items():
        assert int(re.search(r"\.amdhsa_private_segment_fixed_size (\d+)", meta).group(1)) == 0, name
        assert "scratch_" not in body, name


def test_no_packed_fp32(asm):
    ffn.test_no_packed_fp32(asm)


def test_no_atomics(asm):
    ffn.test_no_atomics(asm)


def test_wide_stores_keep_their_data(asm):
    ffn.test_wide_stores_keep_their_data(asm)


def test_generator_uses_wide_products(asm):
    """Ten rounds of two 32 x 32 bit products for each of a chunk's two calls."""
    for name, (body, _) in asm.items():
        if "dropout_kernel<" in name:
            assert len(re.findall(r"v_mad_u64_u32|v_mul_hi_u32", body)) >= 38, name

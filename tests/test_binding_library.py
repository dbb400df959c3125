"""The binding's calls go to the library that is loaded."""
from __future__ import annotations

import shutil

import pytest

from test_ffn_abi import P, igc  # noqa: F401


@pytest.mark.parametrize("native", [True, False], ids=["marshal", "ctypes"])
def test_calls_follow_the_library(igc, monkeypatch, tmp_path, native):  # noqa: F811
    b = igc.binding
    if not native:
        monkeypatch.setattr(b, "_native", False)
    bad = dict(M=1, N=6, X=P, ldx=6, Y=P, ldy=6, p=0.5, seed=1, stream=0, check=False)
    first = b.load()
    assert igc.dropout(**{**bad, "ldy": 5}) == igc.IGC_EINVAL and b"5 of Y" in first.igc_last_error()
    monkeypatch.setattr(b, "LIB_PATH", str(shutil.copy(b.LIB_PATH, tmp_path / "libigc.so")))
    monkeypatch.setattr(b, "_lib", None)
    assert igc.dropout(**{**bad, "p": 2.0}) == igc.IGC_EINVAL
    second = b.load()
    assert second is not first and b"p must" in second.igc_last_error() and b"5 of Y" in first.igc_last_error()
    monkeypatch.setattr(b, "_lib", first)
    assert igc.dropout(**{**bad, "ldx": 5}) == igc.IGC_EINVAL
    assert b"5 of X" in first.igc_last_error() and b"p must" in second.igc_last_error()

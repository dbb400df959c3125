"""The kernel of products in 8 bits on rows of any alignment, in the gfx950 assembly (CPU only)."""
from __future__ import annotations

import re

from test_i8_isa import asm  # noqa: F401


def _steady_loop(lines):
    """The shortest stretch that ends in a jump to its beginning and has matrix instructions."""
    at, best = {}, None
    for i, l in enumerate(lines):
        m = re.match(r"(\.LBB\w+):", l)
        if m:
            at[m.group(1)] = i
    for i, l in enumerate(lines):
        m = re.match(r"s_c?branch\w*\s+(\.LBB\w+)", l)
        if m and at.get(m.group(1), i) < i:
            loop = lines[at[m.group(1)] + 1:i]
            if any(x.startswith("v_mfma") for x in loop) and (best is None or len(loop) < len(best)):
                best = loop
    return best


def test_matrix_instruction_of_the_type(asm):  # noqa: F811
    found = [n for n in asm if "i8_any_kernel<" in n]
    assert len(found) == 4
    for name in found:
        assert set(re.findall(r"v_mfma_\w+", asm[name][0])) == {"v_mfma_i32_16x16x64_i8"}, name


def test_loads_of_later_tiles_stay_on_their_way(asm):  # noqa: F811
    """The loop takes four K tiles a turn without a branch, and no wait in it is for the youngest tile's loads."""
    for name, (body, _) in asm.items():
        if "i8_any_kernel<" not in name:
            continue
        lines = [l.split(";")[0].strip() for l in body.splitlines()]
        loop = _steady_loop([l for l in lines if l])
        loads = [l for l in loop if l.startswith(("global_load", "buffer_load"))]
        glu = ", 5, 4>" in name
        assert len(loads) == 4 * (6 if glu else 4), name              # 64 rows of A and 64 (or twice 64) of B, 16 bytes a lane
        assert sum(l.startswith("v_mfma") for l in loop) == 4 * (16 if glu else 8), name
        assert not any(l.startswith(("s_cbranch", "s_branch", "scratch_")) for l in loop), name
        waits = [int(n) for l in loop for n in re.findall(r"vmcnt\((\d+)\)", l)]
        assert waits and min(waits) >= len(loads) // 4, (name, waits)

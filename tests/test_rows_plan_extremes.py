"""Plans of the norm's backward pass over very many rows, on the CPU (rows_plan_main.hip)."""
from __future__ import annotations

import pytest

from test_rows_plan import _back, host  # noqa: F401

MOST_ROWS = 4096  # that a thread adds one after the other


@pytest.mark.parametrize("N", [1, 128, 200, 4096, 8192])
@pytest.mark.parametrize("M", [8192, 10 ** 6, 10 ** 8, 2 ** 31 - 4096])
def test_rows_of_a_thread_in_registers(host, M, N):  # noqa: F811
    """One workgroup a compute unit as long as that leaves a thread no more rows than it may add."""
    status, query, need, _, launches = host("layer_norm_backward", **_back(M, N))
    assert status == query == 0
    threads = 16
    while threads * 8 < N:
        threads *= 2
    rows, blocks = 1024 // threads, launches[0][1]
    assert -(-M // (rows * blocks)) <= MOST_ROWS
    assert blocks == max(min(256, -(-M // rows)), -(-M // (rows * MOST_ROWS)))
    assert need >= blocks * 2 * N * 4


@pytest.mark.parametrize("N", [8193, 20000, 10 ** 6])
@pytest.mark.parametrize("M", [1, 5000, 10 ** 6, 2 ** 31 - 4096])
def test_rows_of_a_thread_by_columns(host, M, N):  # noqa: F811
    """Four waves share a block's rows."""
    status, query, need, _, launches = host("layer_norm_backward", **_back(M, N))
    assert status == query == 0
    groups = launches[1][1]
    blocks = groups // -(-N // 512)
    assert groups <= 0x7fffff and need >= 8 * M + blocks * 2 * N * 4
    if blocks < 0x7fffff // -(-N // 512):  # (else the launch has no room for more)
        assert -(-M // blocks) <= 4 * MOST_ROWS

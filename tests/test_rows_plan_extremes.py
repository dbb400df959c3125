"""The row operators at the ends of their sizes on the CPU (rows_plan_main.hip): plans of very many rows, matrices of nothing."""
from __future__ import annotations

import pytest

from test_rows_plan import P, _back, _norm, host  # noqa: F401

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


def test_matrices_of_nothing_may_be_null(host):  # noqa: F811
    """As torch gives them: rows without elements, no rows."""
    for M, N in ((5, 0), (0, 6), (0, 0)):
        assert host("layer_norm_forward", **_norm(M, N, X=0, Y=0))[0] == 0
        assert host("layer_norm_forward", **_norm(M, N, X=0, Y=0, scale=P))[0] == 0
        status, query, need, _, _ = host("layer_norm_backward", **_back(M, N, dY=0, X=0, dX=0, dgamma=0, dbeta=0, workspace=0))
        assert status == query == need == 0
    assert host("layer_norm_forward", **_norm(5, 6, Y=0))[0] == -1
    assert host("layer_norm_backward", **_back(5, 6, dX=0, dgamma=0, dbeta=0))[0] == -1

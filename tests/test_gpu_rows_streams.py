"""The row operators and the products in 8 bits on a stream of their own beside
a busy default stream, captured into graphs that share a workspace, and two at
once on two streams: the results are those of a call on the default stream."""
from __future__ import annotations

import threading

import pytest

from test_gpu_ffn import igc, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def _calls(torch, igc, kind, seed=0):  # noqa: F811
    """(name, outputs, inputs, function of stream and workspace) of each entry point; odd lengths and whole chunks."""
    M, N, K = 200, 1001, 1040
    gen = torch.Generator(device="cuda")
    gen.manual_seed(12 + seed)
    t = torch.float16 if kind == igc.IGC_F16 else torch.bfloat16
    normal = lambda r, c: torch.randn(r, c, generator=gen, device="cuda").to(t)  # noqa: E731
    new = lambda r, c: torch.empty(r, c, dtype=t, device="cuda")  # noqa: E731
    byte = lambda r, c: torch.randint(-127, 128, (r, c), generator=gen, device="cuda", dtype=torch.int8)  # noqa: E731
    vec = lambda n: torch.rand(n, generator=gen, device="cuda") + 0.5  # noqa: E731
    X, dY, R, g, b = normal(M, N), normal(M, N), normal(M, N), vec(N), vec(N)
    Y, dX, D = new(M, N), new(M, N), new(M, N)
    mean, rstd, dg, db, s, sn = (torch.empty(n, device="cuda") for n in (M, M, N, N, M, M))
    m0, r0 = X.float().mean(1), 1 / X.float().std(1)
    step = torch.full((1,), 5, dtype=torch.int64, device="cuda")
    Q, Qn = torch.empty(M, N, dtype=torch.int8, device="cuda"), torch.empty(M, N, dtype=torch.int8, device="cuda")
    q, W, V, xs, sw, sv = byte(M, K), byte(N, K), byte(N, K), vec(M) * 0.01, vec(N) * 0.01, vec(N) * 0.01
    qo, Wo = byte(M, K - 3), byte(N, K - 3)
    L, H, Lo = new(M, N), new(M, N), new(M, N)
    kw = dict(type=kind)

    def no_ws(f):
        return lambda workspace=None, **s: f(**s)

    return [
        ("layer_norm_forward", [Y, mean, rstd, Qn, sn], [X], no_ws(lambda **k: igc.layer_norm_forward(
            M, N, X, N, Y, N, gamma=g, beta=b, mean=mean, rstd=rstd, Q=Qn, ldq=N, scale=sn, **kw, **k))),
        ("layer_norm_backward", [dX, dg, db], [dY], lambda **k: igc.layer_norm_backward(
            M, N, dY, N, X, N, m0, r0, gamma=g, R=R, ldr=N, dX=dX, lddx=N, dgamma=dg, dbeta=db, **kw, **k)),
        ("dropout", [D], [X], no_ws(lambda **k: igc.dropout(M, N, X, N, D, N, 0.3, 77, 2, step=step, R=R, ldr=N, **kw, **k))),
        ("quantize_rows", [Q, s], [X], no_ws(lambda **k: igc.quantize_rows(M, N, X, N, Q, N, s, **kw, **k))),
        ("linear_i8", [L], [q], lambda **k: igc.linear_i8(M, N, K, q, K, xs, W, K, sw, L, N, y_type=kind, bias=b, R=R, ldr=N, **k)),
        ("linear_i8_odd", [Lo], [qo], lambda **k: igc.linear_i8(M, N, K - 3, qo, K - 3, xs, Wo, K - 3, sw, Lo, N, y_type=kind, **k)),
        ("glu_i8", [H], [q], lambda **k: igc.glu_i8(M, N, K, q, K, xs, W, K, sw, V, K, sv, H, N, bias_g=b, **kw, **k)),
    ]


def _fill(torch, outs):  # noqa: F811
    for t in outs:
        t.fill_(-128 if t.dtype == torch.int8 else float("nan"))


@pytest.mark.parametrize("given", [True, False], ids=["argument", "current"])
@pytest.mark.parametrize("kind", ["IGC_F16", "IGC_BF16"])
def test_every_call_on_a_stream_of_its_own(torch, igc, kind, given):  # noqa: F811
    ws, own = (torch.empty(32 << 20, dtype=torch.uint8, device="cuda") for _ in range(2))
    big = torch.zeros(8192, 8192, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(big)
    s = torch.cuda.Stream()
    for name, outs, _, call in _calls(torch, igc, getattr(igc, kind)):
        call(workspace=ws)
        want = [t.clone() for t in outs]
        _fill(torch, outs)
        s.wait_stream(torch.cuda.current_stream())  # inputs and fills
        for _ in range(60):  # about 40 ms: a call that went to the default stream would not be done when its copy is made
            torch.mm(big, big, out=out)
        if given:
            call(stream=s, workspace=own)
        with torch.cuda.stream(s):
            if not given:
                call(workspace=own)
            got = [t.to("cpu", non_blocking=False) for t in outs]  # waits for this stream alone
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w.cpu()), name


def test_graphs_that_share_a_workspace(torch, igc):  # noqa: F811
    """Two captured runs of every call, replayed in turn on changing inputs with eager calls between them."""
    ws = torch.full((32 << 20,), 255, dtype=torch.uint8, device="cuda")
    runs = [_calls(torch, igc, igc.IGC_BF16, seed) for seed in (0, 1)]
    graphs = []
    for calls in runs:
        for _, _, _, call in calls:
            call(workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _, _, _, call in calls:
                call(workspace=ws)
        graphs.append(graph)
    for i in range(5):
        calls, graph = runs[i % 2], graphs[i % 2]
        for _, outs, ins, _ in calls:
            for t in ins:
                t.copy_(t.roll(1, 0))
            _fill(torch, outs)
        ws[:1 << 20].fill_(i)  # what it holds does not matter
        graph.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in outs] for _, outs, _, _ in calls]
        for (name, outs, _, call), kept in zip(calls, got):
            _fill(torch, outs)
            call(workspace=ws)
            torch.cuda.synchronize()
            for a, b in zip(outs, kept):
                assert torch.equal(a, b), name


def test_two_calls_at_once(torch, igc):  # noqa: F811
    """From two threads, on two streams, each with its own workspace."""
    runs = [_calls(torch, igc, igc.IGC_F16, seed) for seed in (0, 1)]
    spaces = [torch.empty(32 << 20, dtype=torch.uint8, device="cuda") for _ in runs]
    want = []
    for calls, ws in zip(runs, spaces):
        for _, outs, _, call in calls:
            call(workspace=ws)
        torch.cuda.synchronize()
        want.append([[t.clone() for t in outs] for _, outs, _, _ in calls])
        for _, outs, _, _ in calls:
            _fill(torch, outs)
    torch.cuda.synchronize()
    errors = []

    def work(calls, ws, stream):
        try:
            for _ in range(20):
                for _, _, _, call in calls:
                    call(workspace=ws, stream=stream)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c, w, torch.cuda.Stream())) for c, w in zip(runs, spaces)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for calls, kept in zip(runs, want):
        for (name, outs, _, _), k in zip(calls, kept):
            for a, b in zip(outs, k):
                assert torch.equal(a, b), name

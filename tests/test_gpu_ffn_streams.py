"""Every feed-forward entry point on a stream of its own, while the default
stream is still busy with earlier work: the results are those of a call on the
default stream, and they are there when the call's own stream has ended."""
from __future__ import annotations

import pytest

from test_gpu_ffn import igc, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def _calls(torch, igc, kind):  # noqa: F811
    """(name, outputs, function of stream and workspace) of each entry point; odd lengths, so that rows are padded too."""
    M, N, K = 130, 1001, 2057
    gen = torch.Generator(device="cuda")
    gen.manual_seed(12)
    t = torch.float16 if kind == igc.IGC_F16 else torch.bfloat16
    normal = lambda r, c, std=1.0: (torch.randn(r, c, generator=gen, device="cuda") * std).to(t)  # noqa: E731
    new = lambda r, c: torch.empty(r, c, dtype=t, device="cuda")  # noqa: E731
    X, W, V, R, dY, Z = normal(M, K), normal(N, K, K ** -0.5), normal(N, K, K ** -0.5), normal(M, N), normal(M, N), normal(M, N)
    b, db, norm = torch.randn(N, generator=gen, device="cuda"), torch.empty(N, device="cuda"), torch.empty(1, device="cuda")
    Y, H, dX, dW, dV = new(M, N), new(M, N), new(M, K), new(N, K), new(N, K)
    clipped = [torch.empty_like(g) for g in (X, W, b)]
    kw = dict(type=kind, act=igc.IGC_ACT_SILU)
    return [
        ("linear_forward", [Y], lambda **s: igc.linear_forward(M, N, K, X, K, W, K, Y, N, bias=b, R=R, ldr=N, **kw, **s)),
        ("linear_backward", [dX, dW, db], lambda **s: igc.linear_backward(M, N, K, dY, N, Z=Z, ldz=N, X=X, ldx=K, W=W, ldw=K, dX=dX, lddx=K,
                                                                          dW=dW, lddw=K, dbias=db, **kw, **s)),
        ("glu_forward", [H], lambda **s: igc.glu_forward(M, N, K, X, K, W, K, V, K, H, N, bias_g=b, **kw, **s)),
        ("glu_backward", [dX, dW, dV], lambda **s: igc.glu_backward(M, N, K, dY, N, Z, N, R, N, X=X, ldx=K, Wg=W, ldwg=K, Wu=V, ldwu=K,
                                                                    dX=dX, lddx=K, dWg=dW, lddwg=K, dWu=dV, lddwu=K, **kw, **s)),
        ("grad_clip", [*clipped, norm], lambda **s: igc.grad_clip([X, W, b], 1.0, norm, out=clipped, **s)),
    ]


@pytest.mark.parametrize("given", [True, False], ids=["argument", "current"])
@pytest.mark.parametrize("kind", ["IGC_F16", "IGC_BF16"])
def test_every_call_on_a_stream_of_its_own(torch, igc, kind, given):  # noqa: F811
    ws, own = (torch.empty(96 << 20, dtype=torch.uint8, device="cuda") for _ in range(2))
    big = torch.zeros(8192, 8192, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(big)
    s = torch.cuda.Stream()
    for name, outs, call in _calls(torch, igc, getattr(igc, kind)):
        call(workspace=ws)
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(float("nan"))
        s.wait_stream(torch.cuda.current_stream())  # inputs and fills
        for _ in range(100):  # about 60 ms: a call that went to the default stream would not be done when its copy is made
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

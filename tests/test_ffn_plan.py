"""Plans, workspace sizes and refusals of the feed-forward entry points on the
CPU: their host side with the launches replaced by lines (ffn_plan_main.hip)."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
P, WS = 1 << 20, 1 << 40  # addresses that are never read


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    from implicit_gemm_convolution_amd import build

    out = str(tmp_path_factory.mktemp("plan") / "ffn_plan")
    subprocess.check_call([build.HIPCC, "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-ffp-contract=off", "-Wno-everything",
                           "-I", os.path.join(build.ROOT, "include"), os.path.join(HERE, "ffn_plan_main.hip"), "-o", out])

    def run(entry, **fields):
        """(status, workspace bytes, the products' plans, the other launches) of one call."""
        fields.setdefault("workspace", WS)
        fields.setdefault("ws_bytes", 1 << 50)
        text = subprocess.run([out], input=entry + " " + " ".join("%s=%d" % i for i in fields.items()) + "\n", capture_output=True,
                              text=True, check=True).stdout
        end = re.search(r"^status (-?\d+) query (-?\d+) need (\d+)", text, re.M)
        assert end, text
        pairs = lambda l: {k: int(v) for k, v in re.findall(r"(\w+)=(-?\d+)", l)}  # noqa: E731
        products = [pairs(l) for l in text.splitlines() if l.startswith(("product", "joint"))]
        launches = [l.split(" groups=")[0][7:] for l in text.splitlines() if l.startswith("launch")]
        assert end[1] == end[2], text
        return int(end[1]), int(end[3]), products, launches

    return run


def test_largest_extents_keep_their_sizes(host):
    """At the largest extents that are taken no size has wrapped; past them the call is refused and nothing is launched."""
    n = 2 ** 30 - 2048
    glu = dict(M=2, N=n, K=8, type=1, act=4, dH=P, lddh=n, G=P, ldg=n, U=P, ldu=n, Wg=P, ldwg=8, Wu=P, ldwu=8, dX=P, lddx=8)
    status, need, products, _ = host("glu_backward", **glu)
    assert status == 0 and [p["R"] for p in products] == [2 * n] and need >= 2 * 2 * n * 2
    assert host("glu_backward", **{**glu, "N": 2 ** 30, "lddh": 2 ** 30, "ldg": 2 ** 30, "ldu": 2 ** 30}) == (-2, 0, [], [])
    n = 2 ** 31 - 4096
    lin = dict(M=1, N=n, K=8, type=1, act=4, dY=P, lddy=n, Z=P, ldz=n, W=P, ldw=8, dX=P, lddx=8)
    status, need, products, _ = host("linear_backward", **lin)
    assert status == 0 and [p["R"] for p in products] == [n] and need >= 2 * n
    m = 2 ** 31 - 1
    assert host("linear_backward", **{**lin, "N": m, "lddy": m, "ldz": m}) == (-2, 0, [], [])


@pytest.mark.parametrize("entry", ["linear_forward", "glu_forward"])
@pytest.mark.parametrize("M", [1, 16, 64])
def test_padded_rows_take_the_kernel_of_aligned_rows(host, entry, M):
    """X at an odd 2-byte offset and a wide aligned weight: X is copied into aligned rows, and the product loads those."""
    N, K = 16384, 4096
    odd, good = P + 2, P
    weights = dict(W=good, ldw=K, Y=P, ldy=N, y_type=1) if entry == "linear_forward" else dict(Wg=good, ldwg=K, Wu=good, ldwu=K, H=P, ldh=N)
    _, _, (aligned,), _ = host(entry, M=M, N=N, K=K, type=1, X=good, ldx=K, **weights)
    status, _, (p,), launches = host(entry, M=M, N=N, K=K, type=1, X=odd, ldx=K, **weights)
    assert status == 0 and launches == ["(igc_ffn::pad_kernel<0>)"]
    assert p == aligned and p["odd"] == 0
    # without a workspace nothing is padded
    status, _, (p,), launches = host(entry, M=M, N=N, K=K, type=1, X=odd, ldx=K, workspace=0, **weights)
    assert status == 0 and not launches and p["odd"] == 1

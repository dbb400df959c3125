"""Plans, workspace sizes and refusals of the products in 8 bits and of the norm's
backward pass on the CPU: their host side with the launches replaced by lines
(rows_plan_main.hip)."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
P, WS = 1 << 20, 1 << 40  # addresses that are never read
BYTES = 8                 # the variant that takes rows of any alignment as they lie
TILES, FEW = (0, 1, 2, 3), (6, 7)


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    from implicit_gemm_convolution_amd import build

    out = str(tmp_path_factory.mktemp("plan") / "rows_plan")
    subprocess.check_call([build.HIPCC, "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-ffp-contract=off", "-Wno-everything",
                           "-I", os.path.join(build.ROOT, "include"), os.path.join(HERE, "rows_plan_main.hip"), "-o", out])

    def run(entry, **fields):
        """(status, workspace bytes, the products, the other launches) of one call."""
        fields.setdefault("workspace", WS)
        fields.setdefault("ws_bytes", 1 << 50)
        text = subprocess.run([out], input=entry + " " + " ".join("%s=%d" % i for i in fields.items()) + "\n", capture_output=True,
                              text=True, check=True).stdout
        end = re.search(r"^status (-?\d+) query (-?\d+) need (\d+)", text, re.M)
        assert end, text
        products = [{k: int(v) for k, v in re.findall(r"(\w+)=(-?\d+)", l)} for l in text.splitlines() if l.startswith("product")]
        launches = [re.fullmatch(r"launch (.*) groups=(\d+) threads=(\d+)", l).groups() for l in text.splitlines() if l.startswith("launch")]
        return int(end[1]), int(end[2]), int(end[3]), products, [(a, int(b), int(c)) for a, b, c in launches]

    return run


def _linear(M, N, K, **more):
    f = dict(M=M, N=N, K=K, y_type=1, X=P, ldx=K, x_scale=P, W=P, ldw=K, w_scale=P, Y=P, ldy=N)
    f.update(more)
    return f


def _glu(M, N, K, **more):
    f = dict(M=M, N=N, K=K, type=1, act=4, X=P, ldx=K, x_scale=P, Wg=P, ldwg=K, wg_scale=P, Wu=P, ldwu=K, wu_scale=P, H=P, ldh=N)
    f.update(more)
    return f


def test_aligned_operands_are_never_copied(host):
    for M in (1, 16, 64, 65, 300, 4096):
        for entry, f in (("linear_i8", _linear(M, 4096, 4096)), ("glu_i8", _glu(M, 4096, 4096))):
            status, query, need, (p,), launches = host(entry, **f)
            assert status == query == 0 and not launches and p["variant"] in TILES + FEW and p["a"] == p["b"] == P
            assert p["R"] == 4096 and need == p["part"]


@pytest.mark.parametrize("M", [1, 40, 100, 1000, 8000])
@pytest.mark.parametrize("K", [1, 15, 17, 130, 2049, 8001])
def test_every_other_alignment_has_a_plan(host, M, K):
    """Copies come with a workspace that holds them; everything else needs none; K, rows and addresses are those of what is read."""
    for entry, f in (("linear_i8", _linear(M, 1001, K, X=P + 1, W=P + 3)), ("glu_i8", _glu(M, 1001, K, X=P + 1, Wg=P + 3, Wu=P + 2))):
        status, query, need, (p,), launches = host(entry, **f)
        assert status == query == 0
        if launches:
            whole = -(-K // 16) * 16
            assert [l[0] for l in launches] == ["(igc_ffn::pad_bytes_kernel<0>)"] and p["variant"] in TILES
            assert p["R"] == p["lda"] == p["ldb"] == whole and p["a"] >= WS and p["b"] >= WS + M * whole
            assert need >= (M + 1001 * (2 if entry == "glu_i8" else 1)) * whole
            assert host(entry, **{**f, "ws_bytes": need - 1})[0] == -1
            assert host(entry, **{**f, "workspace": 0})[0] == -1
            assert host(entry, **{**f, "workspace": WS + 128})[0] == -1
        else:
            assert need == 0 and p["variant"] in FEW + (BYTES,) and p["R"] == K and p["a"] == P + 1 and p["b"] == P + 3
            assert p["odd"] == 1 or p["variant"] == BYTES
            assert host(entry, **{**f, "workspace": 0})[0] == 0


def test_only_what_needs_it_is_copied(host):
    _, _, need, (p,), launches = host("linear_i8", **_linear(4096, 8192, 4096, X=P + 4))
    assert launches and p["b"] == P and p["ldb"] == 4096 and p["a"] == WS
    _, _, need, (p,), launches = host("linear_i8", **_linear(4096, 8192, 4096, ldw=4097))
    assert launches and p["a"] == P and p["b"] == WS and p["ldb"] == 4096


def test_too_many_rows_to_copy(host):
    """Copies are numbered in 32 bits: past that rows are taken as they lie."""
    status, _, need, (p,), launches = host("linear_i8", **_linear(2 ** 31 - 4096, 1, 17))
    assert status == 0 and need == 0 and not launches and p["variant"] == BYTES
    assert host("linear_i8", **_linear(2 ** 31 - 4095, 1, 17))[0] == -2


def test_k_past_int32_sums(host):
    assert host("linear_i8", **_linear(4, 4, 131072))[:2] == (-3, -3)
    assert host("glu_i8", **_glu(4, 4, 131072))[:2] == (-3, -3)
    assert host("linear_i8", **_linear(200, 4, 131071))[0] == 0


def _back(M, N, **more):
    f = dict(M=M, N=N, type=1, x_type=1, dY=P, lddy=N, X=P, ldx=N, mean=P, rstd=P, gamma=P, dX=P, lddx=N, dgamma=P, dbeta=P)
    f.update(more)
    return f


@pytest.mark.parametrize("N", [1, 100, 4096, 8192, 8193, 100000, 2 ** 31 - 4096])
@pytest.mark.parametrize("M", [0, 1, 777, 100000])
def test_norm_backward_sizes(host, M, N):
    """The partial sums of every block fit, without a wrap at the largest sizes; a byte less is refused."""
    status, query, need, _, launches = host("layer_norm_backward", **_back(M, N))
    assert status == query == 0
    width = -(-N // 64) * 64
    if M == 0:
        assert need == 0 and len(launches) == 1
        return
    in_registers = N <= 8192
    assert len(launches) == (2 if in_registers else 3)
    blocks = launches[-2][1] // (1 if in_registers else -(-N // 512))
    assert need >= blocks * 2 * width * 4 + (0 if in_registers else 8 * M) and blocks <= max(256, 4 * 256)
    assert host("layer_norm_backward", **_back(M, N, ws_bytes=need - 1))[0] == -1
    # without the vectors there is less to keep, without dX no means
    status, _, less, _, launches = host("layer_norm_backward", **_back(M, N, dgamma=0, dbeta=0))
    assert status == 0 and less == (0 if in_registers else -(-8 * M // 256) * 256)
    status, _, sums, _, launches = host("layer_norm_backward", **_back(M, N, dX=0))
    assert status == 0 and len(launches) == 2 and sums == need - less


def _norm(M, N, **more):
    f = dict(M=M, N=N, type=1, x_type=1, X=P, ldx=N, Y=P, ldy=N)
    f.update(more)
    return f


def test_long_rows_share_the_caches(host):
    """Workgroups that read their rows again: two to each of 256 compute units, one where two rows are too much for its share of a cache."""
    for N, x_type, groups in ((20000, 1, 512), (32768, 1, 512), (32769, 1, 256), (65536, 1, 256), (65537, 1, 512), (16385, 2, 256), (32769, 2, 512),
                              (2 ** 31 - 4096, 2, 512)):
        status, _, _, _, launches = host("layer_norm_forward", **_norm(100000, N, x_type=x_type))
        assert status == 0 and [l[1:] for l in launches] == [(groups, 1024)]
    for M, groups in ((1, 1), (300, 300), (511, 511), (512, 256)):
        assert [l[1:] for l in host("layer_norm_forward", **_norm(M, 40000))[4]] == [(groups, 1024)]

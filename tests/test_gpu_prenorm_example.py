"""The pre-norm example: a run of the operators together.  Its step in a graph
does what it does eagerly, its gradients are those of the network in 64 bits, and
its blocks in 8 bits give what their formulas give."""
from __future__ import annotations

import importlib.util
import os

import pytest

from philox import border, words

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "prenorm_block.py")
SMALL = dict(blocks=2, width=200, hidden=520, batch=96)


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("prenorm_block_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_captured_step_is_the_eager_one(example):
    more = dict(steps=8, report=lambda s: None, **SMALL)
    net, _, losses = example.train(**more)
    eager, _, same = example.train(graph=False, **more)
    assert losses == same and len(set(losses)) == len(losses)  # every kernel adds in a fixed order; masks and weights change with the step
    assert int(net.step_number) == int(eager.step_number) == 8 * 2


def test_gradients(example):
    """Against autograd of the same network in 64 bits, with the masks from the tests' own generator."""
    import torch

    net = example.Network(seed=5, p=0.2, **SMALL)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    for b in net.blocks:
        for t in b.weights()[3:]:
            t.add_(0.2 * torch.randn(t.shape, generator=gen, device="cuda"))
    M, K = SMALL["batch"], SMALL["width"]
    x = torch.randn(M, K, generator=gen, device="cuda").to(example.KIND)
    target = torch.randn(M, K, generator=gen, device="cuda")
    net.step_number.fill_(7)
    dx = net.gradients(x, target)
    T = border(0.2)
    xs = x.double().requires_grad_()
    params = [[w.double().requires_grad_() for w in b.weights()] for b in net.blocks]
    h = xs
    for i, (Wg, Wu, W3, bg, bu, b3, gamma, beta) in enumerate(params):
        d = h - h.mean(1, keepdim=True)
        n = d / ((d * d).mean(1, keepdim=True) + 1e-5).sqrt() * gamma + beta
        g, u = n @ Wg.T + bg, n @ Wu.T + bu
        o = (g * torch.sigmoid(g) * u) @ W3.T + b3
        keep = torch.from_numpy(words(M, K, example.SEED, 7 + i) >= T).cuda()
        h = torch.where(keep, o * (2.0 ** 32 / (2 ** 32 - T)), torch.zeros_like(o)) + h
    ((h - target.double()) ** 2).mean().backward()
    got = [dx] + [g for b in net.blocks for g in b.grads]
    want = [xs.grad] + [w.grad for block in params for w in block]
    for i, (a, b) in enumerate(zip(got, want)):
        # each value between the operators is rounded to bf16 (2^-9 rms of its size at most), about ten of them one after the
        # other on every path through the two blocks, independently: sqrt(10) of that, with as much again in the sums that
        # cancel: 2^-9 * 3.2 * 2 = 1.3e-2 of the gradient's size
        off = float((a.double() - b).square().mean().sqrt() / b.square().mean().sqrt())
        assert off <= 1.3e-2, (i, off)


def test_serving_in_8_bits(example):
    """Each step of the chain from its own inputs; rows alone and in a batch."""
    import torch

    net = example.Network(seed=6, p=0.0, **SMALL)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    x = torch.randn(SMALL["batch"], SMALL["width"], generator=gen, device="cuda").to(example.KIND)
    served = example.Served(net)
    got = served(x)

    def rows(v):
        top = v.abs().amax(1, keepdim=True)
        return (127 * v / top).round(), (top / 127)

    h = x.double()
    for b in net.blocks:
        d = h - h.mean(1, keepdim=True)
        n = (d / ((d * d).mean(1, keepdim=True) + 1e-5).sqrt() * b.gamma.double() + b.beta.double()).to(example.KIND).double()
        q, s = rows(n)
        (wg, sg), (wu, su), (w3, s3) = (rows(w.double()) for w in (b.Wg, b.Wu, b.W3))
        g, u = (q @ wg.T) * s * sg.T + b.bg.double(), (q @ wu.T) * s * su.T + b.bu.double()
        m = (g * torch.sigmoid(g) * u).to(example.KIND).double()
        q, s = rows(m)
        h = ((q @ w3.T) * s * s3.T + b.b3.double() + h).to(example.KIND).double()
    # values next to a border between two bf16 values go either way, and with them a step of 1/127 of a row's largest of a few of
    # the values behind each output, twice a block: a few of the outputs by some of their own steps, 2^-8, and none by more than 4
    size = h.square().mean().sqrt()
    assert float((got.double() - h).abs().max() / size) <= 4 * 2.0 ** -8 * float(h.abs().max() / size)
    assert float((got.double() - h).square().mean().sqrt() / size) <= 2.0 ** -9
    for n in (1, 7, 70):
        alone = served(x[:n])
        assert float((alone.double() - got[:n].double()).square().mean().sqrt() / size) <= 2.0 ** -9

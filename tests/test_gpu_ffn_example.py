"""The feed-forward example: its training step in a graph does what it does
eagerly, the loss falls, and a token served alone gets its batch's outputs."""
from __future__ import annotations

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("feed_forward_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_training_and_serving(example):
    small = dict(steps=24, blocks=2, width=256, hidden=680, outputs=48, batch=96, report=lambda s: None)
    net, x, losses = example.train(**small)
    _, _, eager = example.train(graph=False, **small)
    assert losses == eager  # every kernel adds in a fixed order
    # gradient descent from a random start against a teacher of the same size
    assert losses[-1] < 0.8 * losses[0], losses
    together = net.forward(x).clone()
    scale = float(together.square().mean().sqrt())
    for rows in (1, 7):
        alone = net.serve(x[:rows])
        # bf16 sums kept between the layers may round the other way where the
        # fp32 sums are added in another order: one step (2^-7) of a few of the
        # values behind each output, 2 blocks deep
        assert float((alone - together[:rows]).abs().max()) <= 4 * 2.0 ** -7 * scale

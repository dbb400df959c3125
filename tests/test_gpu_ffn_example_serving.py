"""The feed-forward example serves batches whose calls ask for more workspace than its training step."""
from __future__ import annotations

import pytest

from test_gpu_ffn_example import example  # noqa: F401

pytestmark = pytest.mark.gpu


def test_serving_fewer_rows_than_the_batch(example):  # noqa: F811
    import torch

    net = example.Network(blocks=1, width=4096, hidden=8200, outputs=8, batch=384, seed=1)
    x = torch.randn(384, 4096, device="cuda").bfloat16()
    together = net.forward(x).clone()
    scale = float(together.square().mean().sqrt())
    for rows in (193, 200, 384, 1):
        alone = net.serve(x[:rows])
        # as in the training test, one block deep: sums added in another order
        assert float((alone - together[:rows]).abs().max()) <= 4 * 2.0 ** -7 * scale

"""A small network of gated feed-forward blocks, trained and then served.

Each block is x + W3 (silu(x Wg^T + bg) * (x Wu^T + bu)) + b3: glu_forward, then
linear_forward with the block's input as its residual; a last linear_forward
maps the width to the outputs.  A training step runs the two backward passes of
every block, clips all gradients by their global norm with grad_clip and takes
a plain gradient step.  After the first, eager step the step is captured into
a HIP graph and replayed.  At the end single tokens are served.

    python examples/feed_forward.py [--steps 60] [--blocks 2] [--eager]

The data is made here: noisy outputs of a random network of the same form.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import implicit_gemm_convolution_amd as igc  # noqa: E402

KIND, TYPE = torch.bfloat16, igc.IGC_BF16


class Block:
    """One gated block: its weights, their gradients and the sums it keeps for the backward pass."""

    def __init__(self, width, hidden, batch, gen):
        new = lambda *s: torch.empty(*s, dtype=KIND, device="cuda")  # noqa: E731
        normal = lambda r, c: (torch.randn(r, c, generator=gen, device="cuda") * c ** -0.5).to(KIND)  # noqa: E731
        self.width, self.hidden, self.batch = width, hidden, batch
        self.Wg, self.Wu, self.W3 = normal(hidden, width), normal(hidden, width), normal(width, hidden)
        self.bg, self.bu, self.b3 = (torch.zeros(n, device="cuda") for n in (hidden, hidden, width))
        self.grads = [torch.empty_like(t) for t in self.weights()]
        self.G, self.U, self.H, self.dH = (new(batch, hidden) for _ in range(4))
        self.out, self.dX = new(batch, width), new(batch, width)

    def weights(self):
        return [self.Wg, self.Wu, self.W3, self.bg, self.bu, self.b3]

    def forward(self, x, ws, keep=True, H=None, out=None):
        M, K, N = x.shape[0], self.width, self.hidden
        H, out = (self.H, self.out) if H is None else (H, out)
        igc.glu_forward(M, N, K, x, K, self.Wg, K, self.Wu, K, H, N, bias_g=self.bg, bias_u=self.bu,
                        G=self.G if keep else None, ldg=N, U=self.U if keep else None, ldu=N, type=TYPE, workspace=ws)
        igc.linear_forward(M, K, N, H, N, self.W3, N, out, K, bias=self.b3, R=x, ldr=K, type=TYPE, workspace=ws)
        return out

    def backward(self, x, dout, ws):
        """The gradients of the weights, and of x, given that of the output."""
        M, K, N = self.batch, self.width, self.hidden
        dWg, dWu, dW3, dbg, dbu, db3 = self.grads
        igc.linear_backward(M, K, N, dout, K, X=self.H, ldx=N, W=self.W3, ldw=N, dX=self.dH, lddx=N, dW=dW3, lddw=N, dbias=db3,
                            type=TYPE, workspace=ws)
        igc.glu_backward(M, N, K, self.dH, N, self.G, N, self.U, N, X=x, ldx=K, Wg=self.Wg, ldwg=K, Wu=self.Wu, ldwu=K,
                         dX=self.dX, lddx=K, dWg=dWg, lddwg=K, dWu=dWu, lddwu=K, dbias_g=dbg, dbias_u=dbu, type=TYPE, workspace=ws)
        self.dX.add_(dout)  # the residual's share
        return self.dX


class Network:
    def __init__(self, blocks, width, hidden, outputs, batch, seed):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.blocks = [Block(width, hidden, batch, gen) for _ in range(blocks)]
        self.width, self.hidden, self.outputs, self.batch = width, hidden, outputs, batch
        self.W = (torch.randn(outputs, width, generator=gen, device="cuda") * width ** -0.5).to(KIND)
        self.b = torch.zeros(outputs, device="cuda")
        self.dW, self.db = torch.empty_like(self.W), torch.empty_like(self.b)
        self.y = torch.empty(batch, outputs, device="cuda")  # fp32
        self.dy = torch.empty(batch, outputs, dtype=KIND, device="cuda")
        self.dx = torch.empty(batch, width, dtype=KIND, device="cuda")
        self.norm, self.error = torch.empty(1, device="cuda"), torch.empty_like(self.y)
        self.ws = torch.empty(self._workspace(), dtype=torch.uint8, device="cuda")

    def weights(self):
        return [t for b in self.blocks for t in b.weights()] + [self.W, self.b]

    def grads(self):
        return [t for b in self.blocks for t in b.grads] + [self.dW, self.db]

    def _forward_workspace(self, M):
        """The most that one forward call of M rows asks for (fewer rows may ask for more: their reductions are split)."""
        K, N, C, b = self.width, self.hidden, self.outputs, self.blocks[0]
        return max(
            igc.glu_forward_workspace_size(M, N, K, b.out, K, b.Wg, K, b.Wu, K, b.H, N, G=b.G, ldg=N, U=b.U, ldu=N, type=TYPE),
            igc.linear_forward_workspace_size(M, K, N, b.H, N, b.W3, N, b.out, K, R=b.out, ldr=K, type=TYPE),
            igc.linear_forward_workspace_size(M, C, K, b.out, K, self.W, K, self.y, C, type=TYPE, y_type=igc.IGC_F32))

    def _workspace(self):
        """The most that one call of a step asks for."""
        M, K, N, C, b = self.batch, self.width, self.hidden, self.outputs, self.blocks[0]
        return max(
            self._forward_workspace(M),
            igc.linear_backward_workspace_size(M, C, K, self.dy, C, X=b.out, ldx=K, W=self.W, ldw=K, dX=self.dx, lddx=K, dW=self.dW,
                                               lddw=K, dbias=self.db, type=TYPE),
            igc.linear_backward_workspace_size(M, K, N, b.out, K, X=b.H, ldx=N, W=b.W3, ldw=N, dX=b.dH, lddx=N, dW=b.grads[2],
                                               lddw=N, dbias=b.grads[5], type=TYPE),
            igc.glu_backward_workspace_size(M, N, K, b.dH, N, b.G, N, b.U, N, X=b.out, ldx=K, Wg=b.Wg, ldwg=K, Wu=b.Wu, ldwu=K,
                                            dX=b.dX, lddx=K, dWg=b.grads[0], lddwg=K, dWu=b.grads[1], lddwu=K, dbias_g=b.grads[3],
                                            dbias_u=b.grads[4], type=TYPE),
            igc.grad_clip_workspace_size(self.grads(), 1.0, self.norm), 256)

    def head(self, x, y, ws):
        K, C = self.width, self.outputs
        igc.linear_forward(x.shape[0], C, K, x, K, self.W, K, y, C, y_type=igc.IGC_F32, bias=self.b, type=TYPE, workspace=ws)
        return y

    def forward(self, x):
        for b in self.blocks:
            x = b.forward(x, self.ws)
        return self.head(x, self.y, self.ws)

    def step(self, x, target, rate, max_norm):
        """One step of gradient descent on the mean squared error."""
        M, K, C = self.batch, self.width, self.outputs
        torch.sub(self.forward(x), target, out=self.error)
        self.dy.copy_(self.error * (2.0 / self.error.numel()))
        last = self.blocks[-1].out
        igc.linear_backward(M, C, K, self.dy, C, X=last, ldx=K, W=self.W, ldw=K, dX=self.dx, lddx=K, dW=self.dW, lddw=K,
                            dbias=self.db, type=TYPE, workspace=self.ws)
        d = self.dx
        for i in reversed(range(len(self.blocks))):
            d = self.blocks[i].backward(self.blocks[i - 1].out if i else x, d, self.ws)
        grads = self.grads()
        igc.grad_clip(grads, max_norm, self.norm, workspace=self.ws)
        for w, g in zip(self.weights(), grads):
            w.sub_(g.to(w.dtype), alpha=rate)

    def loss(self):
        return float(self.error.square().mean())

    def serve(self, x):
        """The outputs of a few tokens (any number of rows up to the batch)."""
        M = x.shape[0]
        need = self._forward_workspace(M)
        # (not in the step's place: a captured step still writes there)
        ws = self.ws if need <= self.ws.numel() else torch.empty(need, dtype=torch.uint8, device="cuda")
        H = torch.empty(M, self.hidden, dtype=KIND, device="cuda")
        for b in self.blocks:
            x = b.forward(x, ws, keep=False, H=H, out=torch.empty(M, self.width, dtype=KIND, device="cuda"))
        return self.head(x, torch.empty(M, self.outputs, device="cuda"), ws)


def train(steps=60, blocks=2, width=512, hidden=1368, outputs=96, batch=384, rate=0.3, max_norm=0.5, graph=True, report=print):
    """Trains a network; returns it, its inputs and the losses of every step."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    teacher, net = Network(blocks, width, hidden, outputs, batch, 2), Network(blocks, width, hidden, outputs, batch, 3)
    x = torch.randn(batch, width, generator=gen, device="cuda").to(KIND)
    target = teacher.forward(x) + 0.05 * torch.randn(batch, outputs, generator=gen, device="cuda")
    losses = []
    net.step(x, target, rate, max_norm)
    losses.append(net.loss())
    run = lambda: net.step(x, target, rate, max_norm)  # noqa: E731
    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            net.step(x, target, rate, max_norm)
        run = captured.replay
    for i in range(1, steps):
        run()
        losses.append(net.loss())
        if i % 10 == 0 or i == steps - 1:
            report("step %3d  loss %.4f  gradient norm %.4f" % (i, losses[-1], float(net.norm)))
    return net, x, losses


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--eager", action="store_true", help="do not capture the step into a graph")
    a = ap.parse_args()
    net, x, losses = train(a.steps, a.blocks, graph=not a.eager)
    together = net.forward(x)
    alone = net.serve(x[:1])
    off = float((alone - together[:1]).abs().max()) / math.sqrt(float(together.square().mean()))
    print("loss %.4f -> %.4f; one token alone and in its batch differ by %.1e of the outputs' size" % (losses[0], losses[-1], off))


if __name__ == "__main__":
    main()

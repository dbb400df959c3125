"""Pre-norm gated blocks with dropout, trained in a HIP graph and served in 8 bits.

Each block is x + drop(W3 (silu(n Wg^T + bg) * (n Wu^T + bu)) + b3) with
n = norm(x): layer_norm_forward, glu_forward, linear_forward, dropout with the
residual.  A training step runs their backward passes (dropout is its own: the
same call on the gradient), clips with grad_clip and takes a plain gradient step;
the step's number lies on the device, where dropout reads it, so a replayed graph
draws new masks.  For serving, the weights are put into 8 bits once, with a scale
for each channel (quantize_rows does it), and a token's rows by
layer_norm_forward and quantize_rows: glu_i8, then linear_i8 with the residual.

    python examples/prenorm_block.py [--steps 60] [--blocks 2] [--eager]

The data is made here: noisy outputs of a random network of the same form.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import implicit_gemm_convolution_amd as igc  # noqa: E402

KIND, TYPE = torch.bfloat16, igc.IGC_BF16
SEED = 1234


class Block:
    """One block: its weights, their gradients and what it keeps for the backward pass."""

    def __init__(self, width, hidden, batch, gen, place, p):
        new = lambda *s: torch.empty(*s, dtype=KIND, device="cuda")  # noqa: E731
        normal = lambda r, c: (torch.randn(r, c, generator=gen, device="cuda") * c ** -0.5).to(KIND)  # noqa: E731
        vec = lambda n, v=0.0: torch.full((n,), v, device="cuda")  # noqa: E731
        self.width, self.hidden, self.batch, self.place, self.p = width, hidden, batch, place, p
        self.Wg, self.Wu, self.W3 = normal(hidden, width), normal(hidden, width), normal(width, hidden)
        self.bg, self.bu, self.b3, self.gamma, self.beta = vec(hidden), vec(hidden), vec(width), vec(width, 1.0), vec(width)
        self.grads = [torch.empty_like(t) for t in self.weights()]
        self.N, self.O, self.out, self.dN, self.dO, self.dX = (new(batch, width) for _ in range(6))
        self.G, self.U, self.H, self.dH = (new(batch, hidden) for _ in range(4))
        self.mean, self.rstd = vec(batch), vec(batch)

    def weights(self):
        return [self.Wg, self.Wu, self.W3, self.bg, self.bu, self.b3, self.gamma, self.beta]

    def forward(self, x, step, ws):
        M, K, N = x.shape[0], self.width, self.hidden
        igc.layer_norm_forward(M, K, x, K, self.N, K, gamma=self.gamma, beta=self.beta, mean=self.mean, rstd=self.rstd, type=TYPE)
        igc.glu_forward(M, N, K, self.N, K, self.Wg, K, self.Wu, K, self.H, N, bias_g=self.bg, bias_u=self.bu, G=self.G, ldg=N, U=self.U,
                        ldu=N, type=TYPE, workspace=ws)
        igc.linear_forward(M, K, N, self.H, N, self.W3, N, self.O, K, bias=self.b3, type=TYPE, workspace=ws)
        igc.dropout(M, K, self.O, K, self.out, K, self.p, SEED, self.place, step=step, R=x, ldr=K, type=TYPE)
        return self.out

    def backward(self, x, dout, step, ws):
        """The gradients of the weights, and of x, given that of the output."""
        M, K, N = self.batch, self.width, self.hidden
        dWg, dWu, dW3, dbg, dbu, db3, dgamma, dbeta = self.grads
        igc.dropout(M, K, dout, K, self.dO, K, self.p, SEED, self.place, step=step, type=TYPE)
        igc.linear_backward(M, K, N, self.dO, K, X=self.H, ldx=N, W=self.W3, ldw=N, dX=self.dH, lddx=N, dW=dW3, lddw=N, dbias=db3, type=TYPE,
                            workspace=ws)
        igc.glu_backward(M, N, K, self.dH, N, self.G, N, self.U, N, X=self.N, ldx=K, Wg=self.Wg, ldwg=K, Wu=self.Wu, ldwu=K, dX=self.dN,
                         lddx=K, dWg=dWg, lddwg=K, dWu=dWu, lddwu=K, dbias_g=dbg, dbias_u=dbu, type=TYPE, workspace=ws)
        igc.layer_norm_backward(M, K, self.dN, K, x, K, self.mean, self.rstd, gamma=self.gamma, R=dout, ldr=K, dX=self.dX, lddx=K,
                                dgamma=dgamma, dbeta=dbeta, type=TYPE, workspace=ws)
        return self.dX

    def workspace(self):
        """The most that one call of a step asks for."""
        M, K, N = self.batch, self.width, self.hidden
        g = self.grads
        return max(
            igc.glu_forward_workspace_size(M, N, K, self.N, K, self.Wg, K, self.Wu, K, self.H, N, G=self.G, ldg=N, U=self.U, ldu=N, type=TYPE),
            igc.linear_forward_workspace_size(M, K, N, self.H, N, self.W3, N, self.O, K, type=TYPE),
            igc.linear_backward_workspace_size(M, K, N, self.dO, K, X=self.H, ldx=N, W=self.W3, ldw=N, dX=self.dH, lddx=N, dW=g[2], lddw=N,
                                               dbias=g[5], type=TYPE),
            igc.glu_backward_workspace_size(M, N, K, self.dH, N, self.G, N, self.U, N, X=self.N, ldx=K, Wg=self.Wg, ldwg=K, Wu=self.Wu, ldwu=K,
                                            dX=self.dN, lddx=K, dWg=g[0], lddwg=K, dWu=g[1], lddwu=K, dbias_g=g[3], dbias_u=g[4], type=TYPE),
            igc.layer_norm_backward_workspace_size(M, K, self.dN, K, self.N, K, self.mean, self.rstd, R=self.dO, ldr=K, dX=self.dX, lddx=K,
                                                   dgamma=g[6], dbeta=g[7], type=TYPE))


class Network:
    def __init__(self, blocks, width, hidden, batch, seed, p):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.blocks = [Block(width, hidden, batch, gen, i, p) for i in range(blocks)]
        self.width, self.batch = width, batch
        self.step_number = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.norm, self.error = torch.empty(1, device="cuda"), torch.empty(batch, width, device="cuda")
        self.dy = torch.empty(batch, width, dtype=KIND, device="cuda")
        need = max(*(b.workspace() for b in self.blocks), igc.grad_clip_workspace_size(self.grads(), 1.0, self.norm), 256)
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def weights(self):
        return [t for b in self.blocks for t in b.weights()]

    def grads(self):
        return [t for b in self.blocks for t in b.grads]

    def forward(self, x):
        for b in self.blocks:
            x = b.forward(x, self.step_number, self.ws)
        return x

    def gradients(self, x, target):
        """Those of the mean squared error, unclipped; of x too."""
        torch.sub(self.forward(x).float(), target, out=self.error)
        self.dy.copy_(self.error * (2.0 / self.error.numel()))
        d = self.dy
        for i in reversed(range(len(self.blocks))):
            d = self.blocks[i].backward(self.blocks[i - 1].out if i else x, d, self.step_number, self.ws)
        return d

    def step(self, x, target, rate, max_norm):
        """One step of gradient descent; the next one draws other masks."""
        self.gradients(x, target)
        grads = self.grads()
        igc.grad_clip(grads, max_norm, self.norm, workspace=self.ws)
        for w, g in zip(self.weights(), grads):
            w.sub_(g.to(w.dtype), alpha=rate)
        self.step_number.add_(len(self.blocks))

    def loss(self):
        return float(self.error.square().mean())


class Served:
    """A network's blocks with their weights in 8 bits, for rows of any number."""

    def __init__(self, net):
        self.width, self.blocks = net.width, []
        for b in net.blocks:
            weights = []
            for w in (b.Wg, b.Wu, b.W3):
                rows, cols = w.shape
                q, s = torch.empty(rows, cols, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
                igc.quantize_rows(rows, cols, w, cols, q, cols, s, type=TYPE)
                weights += [q, s]
            self.blocks.append((b, weights))

    def __call__(self, x):
        M, K = x.shape
        N = self.blocks[0][0].hidden
        q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        h, hq, hs = torch.empty(M, N, dtype=KIND, device="cuda"), torch.empty(M, N, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        b, (wg, sg, wu, su, w3, s3) = self.blocks[0]
        need = max(igc.glu_i8_workspace_size(M, N, K, q, K, s, wg, K, sg, wu, K, su, h, N, type=TYPE),
                   igc.linear_i8_workspace_size(M, K, N, hq, N, hs, w3, N, s3, x, K, R=x, ldr=K, y_type=TYPE), 256)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        for b, (wg, sg, wu, su, w3, s3) in self.blocks:
            out = torch.empty_like(x)
            igc.layer_norm_forward(M, K, x, K, None, K, gamma=b.gamma, beta=b.beta, Q=q, ldq=K, scale=s, type=TYPE)
            igc.glu_i8(M, N, K, q, K, s, wg, K, sg, wu, K, su, h, N, bias_g=b.bg, bias_u=b.bu, type=TYPE, workspace=ws)
            igc.quantize_rows(M, N, h, N, hq, N, hs, type=TYPE)
            igc.linear_i8(M, K, N, hq, N, hs, w3, N, s3, out, K, bias=b.b3, R=x, ldr=K, y_type=TYPE, workspace=ws)
            x = out
        return x


def train(steps=60, blocks=2, width=512, hidden=1376, batch=384, p=0.1, rate=0.3, max_norm=0.5, graph=True, report=print):
    """Trains a network; returns it, its inputs and the losses of every step."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    teacher, net = Network(blocks, width, hidden, batch, 2, 0.0), Network(blocks, width, hidden, batch, 3, p)
    x = torch.randn(batch, width, generator=gen, device="cuda").to(KIND)
    target = teacher.forward(x).float() + 0.05 * torch.randn(batch, width, generator=gen, device="cuda")
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
    for b in net.blocks:
        b.p = 0.0  # (serving drops nothing)
    full, served = net.forward(x).float(), Served(net)
    eight, alone = served(x).float(), served(x[:1]).float()
    size = float(full.square().mean().sqrt())
    print("loss %.4f -> %.4f; in 8 bits off by %.1e of the outputs' size (rms), one token alone and in its batch by %.1e" %
          (losses[0], losses[-1], float((eight - full).square().mean().sqrt()) / size, float((alone - eight[:1]).abs().max()) / size))


if __name__ == "__main__":
    main()

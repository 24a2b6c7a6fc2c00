"""Trains a small sequence model through the factor, and runs it step by step.

``python -m differentiable_cholesky_gb300.train_steps --steps 30`` draws packed
sequences of uneven lengths from a noisy linear process and fits a recurrent
model of the next observation: blocks of norm, gates and values from one
projection, gated linear recurrence and output projection on a residual stream,
and a Gaussian whose covariance is learned through its Cholesky factor.  Every
step uses the library's operators together: ``rms_norm``, ``linrec``,
``cholesky`` and the solve with the factor, their adjoints, and ``AdamW``, which
skips a step where the covariance was not positive definite.  Afterwards the
model walks one sequence token by token with ``linrec_step`` and compares its
predictions with the whole pass.  The projections are torch products.
"""
from __future__ import annotations

import argparse

import torch

from . import binding, learn


class SolveWithFactor(torch.autograd.Function):
    """``A^-1 B`` with ``A = L L^T``: the library's solve and its reverse mode."""

    @staticmethod
    def forward(ctx, L, B, status):
        X = binding.chol_solve(L, B, status=status)
        ctx.save_for_backward(L, X, status)
        return X

    @staticmethod
    def backward(ctx, adj_X):
        L, X, status = ctx.saved_tensors
        adj_B, adj_L = binding.chol_solve_adj(L, X, adj_X.contiguous(), status=status)
        return adj_L, adj_B, None


class Model:
    """Next-observation model of sequences of ``size`` numbers: ``width``
    channels, ``depth`` blocks, parameters of type ``dtype`` and a float64
    square root of the covariance."""

    def __init__(self, size: int, width: int, depth: int, dtype=torch.float32, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def draw(*shape, scale):
            x = torch.randn(shape, generator=gen, device="cuda") * scale
            return x.to(dtype).requires_grad_(True)

        def ones(n):
            return torch.ones(n, dtype=dtype, device="cuda", requires_grad=True)

        self.size, self.width = size, width
        self.enter = draw(size, width, scale=size ** -0.5)
        self.blocks = [dict(norm=ones(width), gates=draw(width, 2 * width, scale=width ** -0.5),
                            out=draw(width, width, scale=0.5 * width ** -0.5)) for _ in range(depth)]
        self.norm, self.leave = ones(width), draw(width, size, scale=0.1 * width ** -0.5)
        self.root = torch.eye(size, dtype=torch.float64, device="cuda").requires_grad_(True)

    def parameters(self):
        return [self.enter, *[p for b in self.blocks for p in b.values()], self.norm, self.leave,
                self.root]

    def _block(self, block, x, stream, recurrence):
        """One block: ``x`` joins the residual stream, and what comes out is
        the next ``x``."""
        y, stream = learn.rms_norm(x, block["norm"], stream)
        both = y @ block["gates"]
        h = recurrence(both[..., :self.width], both[..., self.width:])
        return h @ block["out"], stream

    def _forward(self, inputs, recurrences):
        x = inputs.to(self.enter.dtype) @ self.enter
        stream = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
        for block, recurrence in zip(self.blocks, recurrences):
            x, stream = self._block(block, x, stream, recurrence)
        y, _ = learn.rms_norm(x, self.norm, stream)
        return y @ self.leave

    def predict(self, inputs, offsets):
        """Means of the next observations for packed ``[T, size]`` inputs."""
        def whole(gate, x):
            return learn.linrec(gate, x, None, offsets)[0]
        return self._forward(inputs, [whole] * len(self.blocks))

    def step(self, inputs, states):
        """The same for one observation of each sequence (``[B, size]``);
        ``states`` (a float32 ``[B, width]`` for each block) are advanced."""
        def one(state):
            return lambda gate, x: learn.linrec_step(gate, x, state)
        with torch.no_grad():
            return self._forward(inputs, [one(s) for s in states])

    def loss(self, inputs, targets, offsets):
        """Mean negative log-likelihood (up to a constant), and the factor's status."""
        off = (targets - self.predict(inputs, offsets)).double()
        n = off.shape[0]
        cov = self.root @ self.root.t() + 1e-3 * torch.eye(self.size, dtype=torch.float64, device="cuda")
        L, status = binding.cholesky(cov[None])
        X = SolveWithFactor.apply(L, off.t().contiguous()[None], status)
        half_log_det = torch.diagonal(L[0]).log().sum()
        return 0.5 * (X[0] * off.t()).sum() / n + half_log_det, status


def draw_sequences(lengths, size: int, seed: int):
    """Packed observations of a stable linear process with correlated noise."""
    gen = torch.Generator().manual_seed(seed)
    A = torch.linalg.qr(torch.randn(size, size, generator=gen))[0] * 0.9
    mix = torch.randn(size, size, generator=gen) * 0.3
    rows = []
    for n in lengths:
        y = torch.randn(size, generator=gen)
        for _ in range(n):
            y = A @ y + mix @ torch.randn(size, generator=gen)
            rows.append(y)
    return torch.stack(rows).cuda()


def train(steps: int = 30, size: int = 8, width: int = 128, depth: int = 2, state_bits: int = 32,
          lr: float = 3e-3, seed: int = 0, log=print):
    """Runs the steps; returns the model and the losses."""
    lengths = [200, 1, 37, 512, 64, 2, 128, 80]
    data = draw_sequences([n + 1 for n in lengths], size, seed + 1)
    # inputs and targets: each sequence without its last, and without its first
    at, keep = 0, []
    for n in lengths:
        keep += range(at, at + n)
        at += n + 1
    keep = torch.tensor(keep, device="cuda")
    inputs, targets = data[keep], data[keep + 1]
    offsets = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], device="cuda")
    model = Model(size, width, depth, seed=seed)
    params = model.parameters()
    optimiser = learn.AdamW(params, lr=lr, betas=(0.9, 0.95), state_bits=state_bits,
                            weight_decay=[0.0 if p.dim() < 2 or p is model.root else 0.01 for p in params])
    losses = []
    for k in range(steps):
        loss, status = model.loss(inputs, targets, offsets)
        for p in params:
            p.grad = None
        loss.backward()
        norm = torch.stack([p.grad.float().norm() for p in params]).norm()
        clip = (1.0 / norm.clamp(min=1.0)).float()
        optimiser.step(grad_scale=clip, status=status)
        losses.append(loss.detach())
        if k % 10 == 0 or k == steps - 1:
            log(f"step {k}: loss {losses[-1].item():.4f}, gradient {norm.item():.3f}")
    return model, [x.item() for x in losses], inputs[:lengths[0]]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--size", type=int, default=8)
    ap.add_argument("--width", type=int, default=128)
    ap.add_argument("--depth", type=int, default=2)
    ap.add_argument("--state-bits", type=int, default=32, choices=[32, 8])
    ap.add_argument("--lr", type=float, default=3e-3)
    args = ap.parse_args()
    model, _, sequence = train(args.steps, args.size, args.width, args.depth, args.state_bits, args.lr)
    with torch.no_grad():
        whole = model.predict(sequence, torch.tensor([0, len(sequence)], device="cuda"))
    states = [torch.zeros((1, args.width), device="cuda") for _ in model.blocks]
    steps = torch.cat([model.step(y[None], states) for y in sequence])
    off = ((steps - whole).norm() / whole.norm()).item()
    print(f"{len(sequence)} steps one by one: {off:.2e} from the whole pass")


if __name__ == "__main__":
    main()

"""The vocabulary cross entropy and its gradients in 64 bits where the tensors are (so that large cases are quick),
with bounds that tell the target's value of d from the others."""
from __future__ import annotations

import torch

BF16 = torch.bfloat16
REST_TOKENS = 128           # up to these, dW takes what all values of d lose to rounding


def seeded(tokens, vocab, dim, seed, pads=True, hot=False, spread=2.0):
    """(h, W, targets, dloss) on the GPU; hot: every other token has one of three targets."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.randn(tokens, dim, generator=g, device="cuda").to(BF16)
    W = (torch.randn(vocab, dim, generator=g, device="cuda") * (spread / dim ** 0.5)).to(BF16)
    t = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    if hot:
        t[::2] = torch.tensor([0, vocab // 2, vocab - 1], device="cuda")[torch.arange(tokens, device="cuda")[::2] % 3]
    if pads and tokens > 2:
        t[1::5] = -100
        t[2] = vocab
        t[0] = vocab - 1
    dloss = (torch.rand(tokens, generator=g, device="cuda") + 0.5) / tokens
    dloss[::3] *= -1
    return h, W, t, dloss


class Vocabulary64:
    """loss, lse, dh and dW in 64 bits, and bounds of what fp32 sums and d in bf16 may be off by.

    z sums dim products, each step within 2^-23 of the magnitudes summed (the matrix cores may truncate): zerr.  lse:
    zerr, exp (its argument within 2^-23 |z - max|, the function within 2^-22), at most 256 sums in sequence and its own
    rounding.  A value of d is off by its argument's error; but for the target's it is rounded to bf16 (2^-8, half of
    eps) for both products, for dW of up to REST_TOKENS tokens to two bf16 (2^-16).  What the target's value loses is
    kept in fp32 and rounded to bf16 at most once more: 2^-16.  The products sum vocab (tokens) terms within 2^-23 each,
    and the results are rounded to bf16."""

    def __init__(self, h, W, targets, dloss):
        tokens, vocab, dim = h.shape[0], W.shape[0], h.shape[1]
        h, W, t = h.double(), W.double(), targets.long()
        ok = (t >= 0) & (t < vocab)
        at = torch.where(ok, t, 0)
        z = h @ W.t()
        self.lse = torch.logsumexp(z, dim=1)
        self.loss = torch.where(ok, self.lse - z.gather(1, at[:, None]).squeeze(1), 0.0)
        p = torch.softmax(z, dim=1)
        zerr = (dim + 8) * 2.0 ** -23 * (h.abs() @ W.abs().t()).amax(dim=1)
        top = z.amax(dim=1)
        spread = (p * (top[:, None] - z)).sum(dim=1)
        self.lse_tol = zerr + (256 + 2 * spread + 4) * 2.0 ** -23 + 2.0 ** -23 * self.lse.abs()
        self.loss_tol = self.lse_tol + zerr + 2.0 ** -23 * (self.loss.abs() + z.abs().amax(dim=1))
        del z
        g = torch.where(ok, dloss.double(), 0.0)[:, None]
        target = torch.zeros_like(p, dtype=torch.bool).scatter_(1, at[:, None], ok[:, None])
        d = (p - target.double()) * g
        argument = g.abs() * p * (1.01 * (zerr + self.lse_tol)[:, None] + 2.0 ** -20) + \
            g.abs() * target * 2.0 ** -22
        del p
        kept = torch.where(target, 2.0 ** -16, 2.0 ** -8)
        self.dh, self.dW = d @ W, d.t() @ h
        err = argument + kept * d.abs()
        self.dh_tol = 1.01 * (err @ W.abs() + (vocab + 8) * 2.0 ** -23 * (d.abs() @ W.abs()) +
                              2.0 ** -8 * self.dh.abs())
        if tokens <= REST_TOKENS:
            err = argument + 2.0 ** -16 * d.abs()
        self.dW_tol = 1.01 * (err.t() @ h.abs() + (tokens + 8) * 2.0 ** -23 * (d.abs().t() @ h.abs()) +
                              2.0 ** -8 * self.dW.abs())
        # in the 2-norm: the results' own rounding, and that of the values of d that are not a target's, which act
        # on rows of W and h that have nothing to do with them
        lost = torch.where(target, 0.0, d.float().to(BF16).double() - d).square()
        self.dh_off = float(((self.dh.float().to(BF16).double() - self.dh).square().sum() +
                             (lost @ W.square().sum(dim=1)).sum()).sqrt())
        if tokens <= REST_TOKENS:
            lost.zero_()
        self.dW_off = float(((self.dW.float().to(BF16).double() - self.dW).square().sum() +
                             (lost.t() @ h.square().sum(dim=1)).sum()).sqrt())


def within(got, ref, tol):
    """Whether every element is within its tolerance (NaN is not)."""
    return bool(((got.double() - ref).abs() <= tol).all())

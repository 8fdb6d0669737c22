"""The operators on decoded tensors in 64 bits, and seeded inputs for their tests."""
from __future__ import annotations

import torch


def q4_case(rows, cols, group, zeros, seed, device="cuda"):
    """(codes, scales, zeros or None, the matrix in 64 bits)."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 16, (rows, cols), generator=g)
    groups = -(-cols // group)
    scales = (torch.rand(rows, groups, generator=g) + 0.5).mul_(0.02).to(torch.bfloat16)
    scales[torch.rand(rows, groups, generator=g) < 0.25] *= -1
    z = torch.randint(0, 16, (rows, groups), generator=g) if zeros else None
    at = torch.arange(cols) // group
    w = scales.double()[:, at] * (q.double() - (8.0 if z is None else z.double()[:, at]))
    codes = (q[:, 0::2] | (q[:, 1::2] << 4)).to(torch.uint8).contiguous()
    return (codes.to(device), scales.to(device), None if z is None else z.to(torch.uint8).to(device), w)


def q4_tolerance(w, x):
    """Bound of |y - y64| for fp32 sums over exact products of codes and x.

    Every product of a code less its zero point with x, and every sum of a
    group's, is exact or rounded within 24 sequential fp32 operations of the
    products' magnitudes (8 products, the group's scale, the join of lanes and
    waves); groups follow each other, one step per 128 columns at most.  x may
    be held relative to a larger |x| near it: in f16, scaled for the largest of
    at most 512 columns, it is off by less than 2^-39 of that one, for which
    2^-30 of the largest of its own 128 columns stands.  w: rows x cols, x: vecs x cols, both 64-bit."""
    cols = w.shape[1]
    pad = -cols % 128
    xm = torch.nn.functional.pad(x.abs(), (0, pad)).reshape(x.shape[0], -1, 128).amax(dim=2)
    xm = xm.repeat_interleave(128, dim=1)[:, :cols]
    return (cols / 128 + 24) * 2.0 ** -24 * (x.abs() @ w.abs().t()) + 2.0 ** -30 * (xm @ w.abs().t())


def embed_grad_ref(dout, ids, vocab, scale):
    """(gradient, sum of magnitudes, largest number of tokens of a row), all 64-bit."""
    total = torch.zeros(vocab, dout.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(total)
    ids = ids.cpu().long()
    ok = (ids >= 0) & (ids < vocab)
    d = dout.cpu().double()[ok]
    total.index_add_(0, ids[ok], d)
    mag.index_add_(0, ids[ok], d.abs())
    most = int(torch.bincount(ids[ok], minlength=1).max()) if bool(ok.any()) else 0
    return scale * total, abs(scale) * mag, most


class CrossEntropy64:
    """loss, lse, dh and dW in 64 bits, with bounds on what fp32 sums and bf16 d may be off by.

    z is a sum of dim products, each step within 2^-23 of the magnitudes summed
    (the matrix cores may truncate): zerr = (dim + 8) 2^-23 max_v sum |h W|.
    lse: zerr, plus exp (arguments rounded within 2^-23 |z - max|, the function
    within 2^-22), plus at most 256 sequential fp32 sums and joins, plus its own
    rounding.  d is off by its argument's error and rounded to bf16 (2^-8 of
    |d|, half of eps); the products sum vocab (tokens) terms within 2^-23 each;
    dh and dW are rounded once more (2^-8)."""

    def __init__(self, h, W, targets, dloss=None):
        h, W = h.cpu().double(), W.cpu().double()
        t = targets.cpu().long()
        vocab = W.shape[0]
        ok = (t >= 0) & (t < vocab)
        at = torch.where(ok, t, 0)
        z = h @ W.t()
        self.lse = torch.logsumexp(z, dim=1)
        self.loss = torch.where(ok, self.lse - z.gather(1, at[:, None]).squeeze(1), 0.0)
        p = torch.softmax(z, dim=1)
        zerr = (W.shape[1] + 8) * 2.0 ** -23 * (h.abs() @ W.abs().t()).amax(dim=1)
        spread = (p * (z.amax(dim=1, keepdim=True) - z)).sum(dim=1)
        self.lse_tol = zerr + (256 + 2 * spread + 4) * 2.0 ** -23 + 2.0 ** -23 * self.lse.abs()
        self.loss_tol = self.lse_tol + zerr + 2.0 ** -23 * (self.loss.abs() + z.abs().amax(dim=1))
        if dloss is None:
            return
        g = torch.where(ok, dloss.cpu().double(), 0.0)[:, None]
        onehot = torch.zeros_like(p).scatter_(1, at[:, None], 1.0)
        d = (p - onehot) * g
        derr = d.abs() * 2.0 ** -8 + g.abs() * p * (1.01 * (zerr + self.lse_tol)[:, None] + 2.0 ** -20) + \
            g.abs() * onehot * 2.0 ** -22
        self.dh = d @ W
        self.dW = d.t() @ h
        self.dh_tol = derr @ W.abs() + (vocab + 8) * 2.0 ** -23 * (d.abs() @ W.abs()) + 2.0 ** -8 * self.dh.abs()
        self.dW_tol = derr.t() @ h.abs() + (len(t) + 8) * 2.0 ** -23 * (d.abs().t() @ h.abs()) + \
            2.0 ** -8 * self.dW.abs()
        # the rounding of dh (dW) acts on the computed value, not on the exact one
        self.dh_tol *= 1.01
        self.dW_tol *= 1.01


def within(got, ref, tol):
    """Whether every element is within its tolerance (NaN is not)."""
    return bool((((got.cpu().double() - ref).abs() <= tol) | (got.cpu().double() == ref)).all())

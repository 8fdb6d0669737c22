"""e4m3 codes with scales per block of 128, norms and clipping in 64 bits, and bounds on what fp32 sums may be off by."""
from __future__ import annotations

import torch

BLOCK = 128
U32 = 2.0 ** -24          # half a step of fp32, relative
UBF16 = 2.0 ** -8
TINY = 2.0 ** -126        # fp32's smallest normal value


def blocks(n):
    return -(-n // BLOCK)


def code_values():
    """What each of the 256 codes stands for, from the format's definition (4 exponent bits with bias 7, 3 of mantissa)."""
    v = torch.empty(256, dtype=torch.float64)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = float("nan") if e == 15 and m == 7 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = -x if c & 128 else x
    return v


VALUES = code_values()


def values_of(codes):
    """Codes (bytes or float8) to their values, on the host."""
    return VALUES[codes.cpu().view(torch.uint8).long()]


def per_column(scales, cols):
    return scales.double().cpu().repeat_interleave(BLOCK, dim=1)[:, :cols]


def block_max(y):
    """Largest magnitude of each row's blocks (NaN where one holds a NaN)."""
    rows, cols = y.shape
    padded = torch.nn.functional.pad(y, (0, blocks(cols) * BLOCK - cols))
    return padded.abs().reshape(rows, -1, BLOCK).amax(dim=2)


def check_codes(codes, scales, y, yerr):
    """Codes and scales of a matrix y (64-bit), which the kernel has within yerr of it.

    The scale is the largest magnitude over 448, with 1 / 448 rounded and the product rounded: 2^-23.  A code is the
    quotient by the scale rounded to e4m3, half a step: 2^-4 of the value, or half of the smallest step, 2^-10 of the
    scale, and the quotient is within 2^-22 (the reciprocal within 2^-23, and one product)."""
    cols = y.shape[1]
    codes, scales = codes.cpu(), scales.cpu().double()
    top, topmost = block_max(y), block_max(y.abs() + yerr)
    want = torch.clamp(top, min=2.0 ** -100) / 448
    slack = (topmost - top) / 448 + 2.0 ** -23 * want
    assert bool(((scales - want).abs() <= slack * 1.001).all()), "scales"
    wide = per_column(scales, cols)
    got = values_of(codes) * wide
    half = torch.maximum(y.abs() * 2.0 ** -4, wide * 2.0 ** -10)
    assert bool(((got - y).abs() <= half * 1.0001 + yerr + 2.0 ** -22 * y.abs()).all()), "codes"
    # and they are the nearest: a code's neighbours are no nearer
    q = y / wide
    grid = VALUES[:127]
    at = torch.bucketize(q.abs(), grid)
    lower, upper = grid[(at - 1).clamp(0)], grid[at.clamp(max=126)]
    near = torch.minimum((q.abs() - lower).abs(), (q.abs() - upper).abs())
    off = (values_of(codes) - q).abs() - near
    assert bool((off <= (yerr / wide) * 2 + 2.0 ** -21 * q.abs() + 1e-30).all()), "not the nearest codes"


def quantised(y):
    """Codes and scales of a matrix (any float type), made on the host for tests' inputs."""
    scales = (block_max(y.double()).clamp_min(2.0 ** -100) / 448).float()
    return (y.double() / per_column(scales, y.shape[1])).float().to(torch.float8_e4m3fn), scales


def matrix_codes(w):
    """e4m3 codes of a matrix with scales per 128 x 128, and the matrix they stand for in 64 bits."""
    rows, cols = w.shape
    top = torch.nn.functional.pad(block_max(w.double()), (0, 0, 0, blocks(rows) * BLOCK - rows))
    scales = (top.reshape(blocks(rows), BLOCK, -1).amax(dim=1).clamp_min(1e-30) / 448).float()
    wide = per_column(scales, cols).repeat_interleave(BLOCK, dim=0)[:rows]
    codes = (w.double() / wide).float().to(torch.float8_e4m3fn)
    return codes, scales, values_of(codes) * wide


def eights(t):
    """Largest magnitude of each row's groups of 8 columns."""
    rows, cols = t.shape
    return torch.nn.functional.pad(t.abs(), (0, -cols % 8)).reshape(rows, -1, 8)


def _largest_of_eights(x, w):
    """Sum over groups of 8 columns of the largest |product| there, for each row of x and of w."""
    device = "cuda" if torch.cuda.is_available() else "cpu"
    xe, we = eights(x).to(device), eights(w).to(device)
    total = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device=device)
    for t0 in range(0, x.shape[0], 512):
        for k in range(xe.shape[1]):
            total[t0:t0 + 512] += (xe[t0:t0 + 512, None, k] * we[None, :, k]).amax(dim=2)
    return total.cpu()


def gemm_tolerance(x, w, out_bf16, y):
    """Bound of |y - y64| for fp32 sums of the products of codes.

    Results in bf16 may come of 8-bit matrix instructions, which sum 8 neighbouring products at a time and drop what
    lies below 2^-14 of the largest: 8 times 2^-14 of it per group of eight at most.

    A block's 128 products are exact in fp32 and summed in any order, each step within 2^-23 of the magnitudes summed
    (the matrix cores may truncate); times the product of the scales, itself rounded, and added to the other blocks'
    in order or split by split: blocks + splits + 4 further roundings.  Below fp32's normal range, absolute steps."""
    cols = x.shape[1]
    steps = min(cols, BLOCK) + 2 * blocks(cols) + 4
    tol = steps * 2.0 ** -23 * (x.abs() @ w.abs().t()) + 1e-40
    if out_bf16:
        tol = tol + 2.0 ** -11 * _largest_of_eights(x, w)
    return tol + (UBF16 * (y.abs() + tol) if out_bf16 else 0.0)


def norm_error(dim, rounds=8):
    """Relative error of rstd: a lane adds 8 rounds squares, then 10 joins of lanes and waves; half of that in the root,
    which with the mean's product, the sum with eps, the root and the quotient adds 4 roundings (the root and the
    quotient within two steps each)."""
    return (8 * rounds + 10) / 2 * U32 + 8 * U32


class Norm64:
    """h, rstd and y in 64 bits, and how far fp32 may be off y before its last rounding."""

    def __init__(self, x, weight, eps, residual=None):
        x = x.cpu()
        self.h = x if residual is None else (x.float() + residual.cpu().float()).to(torch.bfloat16)
        h = self.h.double()
        self.w = weight.cpu().double()
        self.rstd = 1.0 / torch.sqrt((h * h).sum(dim=1) / x.shape[1] + eps)
        self.u = h * self.rstd[:, None]
        self.y = self.u * self.w
        self.err = norm_error(x.shape[1])
        self.yerr = (self.err + 2 * U32) * self.y.abs() + 1e-40

    def grad(self, dy, dsum=None):
        """(dh, its bound, dweight, its bound).  In fp32 u is within err, du = dy u within err + 2 roundings, the mean
        of g u adds a lane's 64 terms and 10 joins; dweight adds n terms of one column in some order."""
        n, dim = self.h.shape
        dy = dy.cpu().double()
        g = dy * self.w
        gu = g * self.u
        along = gu.sum(dim=1, keepdim=True) / dim
        add = torch.zeros_like(g) if dsum is None else dsum.cpu().double()
        dh = add + self.rstd[:, None] * (g - self.u * along)
        off = (self.err + (8 * 8 + 16) * U32) * gu.abs().sum(dim=1, keepdim=True) / dim
        tol = self.rstd[:, None] * ((self.err + 4 * U32) * g.abs() + self.u.abs() * (off + (2 * self.err + 4 * U32) *
                                                                                     along.abs()))
        tol = tol + 2 * U32 * (dh.abs() + add.abs()) + 1e-40
        mag = (dy * self.u).abs().sum(dim=0)
        return (dh, tol + UBF16 * (dh.abs() + tol), (dy * self.u).sum(dim=0), (self.err + (n + 40) * U32) * mag + 1e-40)


def within(got, want, tol):
    got = got.cpu().double()
    off = (got - want).abs() - tol
    bad = ~(off <= 0)
    if bool(bad.any()):
        i = int(torch.nonzero(bad.flatten())[0])
        print(f"{int(bad.sum())} of {bad.numel()} off, the first at {i}: {got.flatten()[i]:.9g}, not "
              f"{want.flatten()[i]:.9g}; worst {float(off.max()):.3g} past its bound", flush=True)
        return False
    return True

"""GPU tests of the norm, the codes and clipping where tensors are so large that they are read and written past the caches:
the same bits as calls on a part of the rows at a time, which are not, and 64-bit sums for what is summed over all rows."""
import math

import pytest
import torch

from e4m3_ref import U32, blocks, norm_error, within
from gpu_util import log

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
CACHE = 256 << 20
EPS = 1e-5


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    yield mod
    torch.cuda.empty_cache()


def _normal(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF16)


def _parts(n):
    """Four parts of the rows, each below the caches."""
    cuts = [n * k // 4 for k in range(5)]
    return [slice(a, b) for a, b in zip(cuts, cuts[1:])]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dim", [136, 28680])
def test_codes(wc, dim, gated):
    per = 5 if gated else 3
    n = CACHE // (per * dim) + 3
    assert n * dim * per > CACHE
    x = _normal(dim, n, dim * (2 if gated else 1))
    log(f"case: quant_fp8 {n}x{dim} gated {gated}, past the caches")
    codes = torch.empty(n, dim, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n, blocks(dim), device="cuda")
    wc.quant_fp8_async(x, n, dim, codes, scales, gated=gated)
    for at in _parts(n):
        some = x[at]
        c, s = torch.empty_like(codes[at]), torch.empty_like(scales[at])
        wc.quant_fp8_async(some, len(some), dim, c, s, gated=gated)
        assert torch.equal(codes[at], c) and torch.equal(scales[at], s)


@pytest.mark.parametrize("dim", [504, 4104, 20008, 40008])   # 1, 2, 4 and 8 rounds of a row
def test_norm(wc, dim):
    n = CACHE // (6 * dim) + 5                               # read x and the residual, written the sum: 6 bytes, and more
    x, r, w = _normal(1, n, dim), _normal(2, n, dim, scale=2.0), _normal(3, dim)
    log(f"case: rms_norm {n}x{dim}, past the caches")

    def call(x, r, bf16, codes):
        m = len(x)
        out = dict(sum_dev=torch.empty_like(x), rstd_dev=torch.empty(m, device="cuda"))
        if bf16:
            out["y_dev"] = torch.empty_like(x)
        if codes:
            out["codes_dev"] = torch.empty(m, dim, dtype=torch.uint8, device="cuda")
            out["scales_dev"] = torch.empty(m, blocks(dim), device="cuda")
        wc.rms_norm_async(x, w, m, dim, EPS, residual_dev=r, **out)
        return out

    for bf16, codes in ((True, False), (False, True)):
        whole = call(x, r, bf16, codes)
        for at in _parts(n):
            part = call(x[at], r[at], bf16, codes)
            for k, t in part.items():
                assert torch.equal(whole[k][at], t), k


@pytest.mark.parametrize("dsum", [False, True])
@pytest.mark.parametrize("dim", [504, 4104, 20008, 40008])
def test_gradient(wc, dim, dsum):
    n = CACHE // (6 * dim) + 5                               # read dy and h, written dh: 6 bytes, and those of dsum
    h, w, dy = _normal(1, n, dim), _normal(3, dim), _normal(4, n, dim, scale=0.05)
    ds = _normal(5, n, dim, scale=0.05) if dsum else None
    y, rstd = torch.empty_like(h), torch.empty(n, device="cuda")
    wc.rms_norm_async(h, w, n, dim, EPS, y_dev=y, rstd_dev=rstd)
    log(f"case: rms_norm gradient {n}x{dim} dsum {dsum}, past the caches")
    dh, dw = torch.empty_like(h), torch.empty(dim, device="cuda")
    need = wc.rms_norm_grad_work_bytes(n, dim)
    work = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    wc.rms_norm_grad_async(dy, h, w, rstd, n, dim, dh, dw, work, need, dsum_dev=ds)
    for at in _parts(n):
        part = torch.empty_like(dh[at])
        wc.rms_norm_grad_async(dy[at], h[at], w, rstd[at], len(part), dim, part, None, None, 0,
                               dsum_dev=None if ds is None else ds[at])
        assert torch.equal(dh[at], part)
    want, mag = torch.zeros(dim, dtype=torch.float64, device="cuda"), torch.zeros(dim, dtype=torch.float64, device="cuda")
    for at in (slice(k, k + 512) for k in range(0, n, 512)):
        wide = h[at].double()
        du = dy[at].double() * wide / torch.sqrt((wide * wide).mean(dim=1, keepdim=True) + EPS)
        want += du.sum(dim=0)
        mag += du.abs().sum(dim=0)
    # u is off by rstd's error, du by two more roundings, and n terms are added in some order
    assert within(dw, want.cpu(), ((norm_error(dim) + (n + 40) * U32) * mag + 1e-40).cpu())
    before = torch.randn(dim, device="cuda")
    more = before.clone()
    into = dy.clone()                                        # in place, and added to what is there: the same bits
    wc.rms_norm_grad_async(into, h, w, rstd, n, dim, into, more, work, need, dsum_dev=ds, accumulate=True)
    assert torch.equal(into, dh) and torch.equal(more, before + dw)
    assert bool((work[need:] == 0xFF).all())


@pytest.mark.parametrize("kind", [F32, BF16, None], ids=["f32", "bf16", "mixed"])
@pytest.mark.parametrize("count", [5, 60])                  # in one batch of few tensors, or of many
def test_clipping(wc, count, kind):
    per = (80 << 20) // 2 // count
    kinds = [kind or (F32, BF16)[i % 2] for i in range(count)]
    sizes = [per + 1 + i % 7 for i in range(count)]
    log(f"case: clip_grads of {count} tensors of {per} elements, past the caches")
    grads = [_normal(i, n, scale=0.01).to(k) for i, (n, k) in enumerate(zip(sizes, kinds))]
    outs = [torch.empty_like(t) for t in grads]
    handle, norm = wc.GradList(grads, outs), torch.empty(1, device="cuda")
    work = torch.empty(wc.clip_grads_work_bytes(handle), dtype=torch.uint8, device="cuda")
    want = math.sqrt(sum(float((t.double() ** 2).sum()) for t in grads))
    for bound in (1.0, 1e9):
        wc.clip_grads_async(handle, bound, norm, work, work.numel())
        assert abs(float(norm) - want) <= (U32 + 1e-12) * want
        for g, out in zip(grads, outs):
            if bound > want:
                assert torch.equal(g, out)
                continue
            exact = g.double() * (bound / want)             # the factor is rounded, the product, and its type
            tol = (2.0 ** -23 + (2.0 ** -8 if g.dtype == BF16 else 0.0) + 1e-9) * exact.abs() + 1e-38
            assert bool(((out.double() - exact).abs() <= tol).all())

"""GPU tests of the root-mean-square norm with the residual's addition, and of its gradient."""
import pytest
import torch

from e4m3_ref import Norm64, U32, UBF16, blocks, check_codes, within
from gpu_util import log

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn
EPS = 1e-5
GUARD = 64


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


def _guarded(n, dtype, fill):
    return torch.full((n + GUARD,), fill, dtype=dtype, device="cuda")


def _kept(t, n, fill):
    return bool((t[n:].float() == fill).all())


def _inputs(n, dim, seed, residual):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, dim, generator=g).to(BF16)
    r = (torch.randn(n, dim, generator=g) * 3).to(BF16) if residual else None
    w = (torch.randn(dim, generator=g) * 0.3 + 1).to(BF16)
    return x, r, w, g


def _dev(t):
    return None if t is None else t.cuda()


SHAPES = [(1, 8), (3, 16), (2, 128), (5, 136), (4, 512), (9, 520), (515, 1160), (2, 2048), (130, 4096), (3, 4104),
          (7, 8192), (2, 16392), (1, 28672), (2, 65536), (2050, 264)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("n,dim", SHAPES)
def test_norm(wc, n, dim, residual):
    x, r, w, _ = _inputs(n, dim, n + dim, residual)
    log(f"case: rms_norm {n}x{dim} residual {residual}")
    y, total = _guarded(n * dim, BF16, 7.0), _guarded(n * dim, BF16, 7.0)
    codes, scales = _guarded(n * dim, torch.uint8, 90), _guarded(n * blocks(dim), torch.float32, -7.0)
    rstd = _guarded(n, torch.float32, -7.0)
    args = dict(residual_dev=_dev(r), sum_dev=total if residual else None)
    wc.rms_norm_async(x.cuda(), w.cuda(), n, dim, EPS, y_dev=y, codes_dev=codes, scales_dev=scales, rstd_dev=rstd, **args)
    torch.cuda.synchronize()
    assert (_kept(y, n * dim, 7.0) and _kept(total, n * dim, 7.0) and _kept(codes, n * dim, 90) and
            _kept(scales, n * blocks(dim), -7.0) and _kept(rstd, n, -7.0)), "wrote past the end"
    ref = Norm64(x, w, EPS, r)
    if residual:
        assert torch.equal(total[:n * dim].cpu().reshape(n, dim), ref.h)
    assert within(rstd[:n], ref.rstd, ref.err * ref.rstd)
    got = y[:n * dim].reshape(n, dim)
    assert within(got, ref.y, ref.yerr + UBF16 * (ref.y.abs() + ref.yerr))
    check_codes(codes[:n * dim].reshape(n, dim), scales[:n * blocks(dim)].reshape(n, -1), ref.y, ref.yerr)
    # one output at a time: the same bits
    alone, codes2 = torch.empty(n, dim, dtype=BF16, device="cuda"), torch.empty(n, dim, dtype=F8, device="cuda")
    scales2 = torch.empty(n, blocks(dim), device="cuda")
    wc.rms_norm_async(x.cuda(), w.cuda(), n, dim, EPS, y_dev=alone, **args)
    wc.rms_norm_async(x.cuda(), w.cuda(), n, dim, EPS, codes_dev=codes2, scales_dev=scales2, **args)
    assert torch.equal(alone, got)
    assert torch.equal(codes2.view(torch.uint8).flatten(), codes[:n * dim])
    assert torch.equal(scales2.flatten(), scales[:n * blocks(dim)])


@pytest.mark.parametrize("dim", [136, 4096, 8200])
def test_in_place(wc, dim):
    n = 21
    x, r, w, _ = _inputs(n, dim, dim, True)
    log(f"case: rms_norm in place, {n}x{dim}")
    want_h, want_y = torch.empty(n, dim, dtype=BF16, device="cuda"), torch.empty(n, dim, dtype=BF16, device="cuda")
    wc.rms_norm_async(x.cuda(), w.cuda(), n, dim, EPS, y_dev=want_y, residual_dev=r.cuda(), sum_dev=want_h)
    res, into = r.cuda(), x.cuda()
    wc.rms_norm_async(into, w.cuda(), n, dim, EPS, y_dev=into, residual_dev=res, sum_dev=res)
    assert torch.equal(res, want_h) and torch.equal(into, want_y)
    first = x.cuda()
    wc.rms_norm_async(first, w.cuda(), n, dim, EPS, y_dev=want_y, residual_dev=r.cuda(), sum_dev=first)
    assert torch.equal(first, want_h) and torch.equal(into, want_y)
    plain, own = torch.empty_like(want_y), x.cuda()
    wc.rms_norm_async(x.cuda(), w.cuda(), n, dim, EPS, y_dev=plain)
    wc.rms_norm_async(own, w.cuda(), n, dim, EPS, y_dev=own)
    assert torch.equal(own, plain)


@pytest.mark.parametrize("dim", [24, 4096, 16384])
def test_rows_of_zeros_and_no_numbers(wc, dim):
    """A row of zeros is zero (eps 0: no number); a row with an infinity or NaN stays among itself."""
    x, _, w, _ = _inputs(6, dim, 2, False)
    x[1] = 0
    x[2, 3] = float("nan")
    x[4, 5] = float("inf")
    log(f"case: rms_norm rows of zeros and no numbers, dim {dim}")
    y = torch.empty(6, dim, dtype=BF16, device="cuda")
    codes, scales = torch.empty(6, dim, dtype=F8, device="cuda"), torch.empty(6, blocks(dim), device="cuda")
    wc.rms_norm_async(x.cuda(), w.cuda(), 6, dim, EPS, y_dev=y, codes_dev=codes, scales_dev=scales)
    y = y.cpu()
    assert bool((y[1] == 0).all()) and bool((codes[1].float() == 0).all())
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(scales[2]).all())
    assert bool(torch.isnan(y[4, 5])) and bool(torch.isnan(scales[4, 0]))
    ref = Norm64(x[[0, 3, 5]], w, EPS)
    assert within(y[[0, 3, 5]], ref.y, ref.yerr + UBF16 * (ref.y.abs() + ref.yerr))
    wc.rms_norm_async(torch.zeros(1, dim, dtype=BF16, device="cuda"), w.cuda(), 1, dim, 0.0,
                      y_dev=(z := torch.empty(1, dim, dtype=BF16, device="cuda")))
    assert bool(torch.isnan(z).all())


def _grad(wc, dy, h, w, rstd, n, dim, dsum, accumulate=None, want=("dh", "dw"), **kw):
    dh = _guarded(n * dim, BF16, 7.0) if "dh" in want else None
    dw = _guarded(dim, torch.float32, -7.0) if "dw" in want else None
    if accumulate is not None:
        dw[:dim] = accumulate
    need = wc.rms_norm_grad_work_bytes(n, dim)
    work = torch.full((need + GUARD,), 0xFF, dtype=torch.uint8, device="cuda")
    wc.rms_norm_grad_async(dy, h, w, rstd, n, dim, dh, dw, work, need, dsum_dev=dsum, accumulate=accumulate is not None,
                           **kw)
    torch.cuda.synchronize()
    assert bool((work[need:] == 0xFF).all()), "wrote past the workspace"
    assert dh is None or _kept(dh, n * dim, 7.0)
    assert dw is None or _kept(dw, dim, -7.0)
    return None if dh is None else dh[:n * dim].reshape(n, dim), None if dw is None else dw[:dim]


@pytest.mark.parametrize("dsum", [False, True])
@pytest.mark.parametrize("n,dim", SHAPES + [(4100, 136), (2600, 2048)])
def test_gradient(wc, n, dim, dsum):
    x, _, w, g = _inputs(n, dim, n * 3 + dim, False)
    dy = (torch.randn(n, dim, generator=g) * 0.05).to(BF16)
    ds = (torch.randn(n, dim, generator=g) * 0.05).to(BF16) if dsum else None
    log(f"case: rms_norm gradient {n}x{dim} dsum {dsum}")
    y, rstd = torch.empty(n, dim, dtype=BF16, device="cuda"), torch.empty(n, device="cuda")
    xd, wd, dyd, dsd = x.cuda(), w.cuda(), dy.cuda(), _dev(ds)
    wc.rms_norm_async(xd, wd, n, dim, EPS, y_dev=y, rstd_dev=rstd)
    dh, dw = _grad(wc, dyd, xd, wd, rstd, n, dim, dsd)
    want, tol, want_dw, tol_dw = Norm64(x, w, EPS).grad(dy, ds)
    assert within(dh, want, tol) and within(dw, want_dw, tol_dw)
    # each alone, in place, and added to what is there: the same bits
    alone, none = _grad(wc, dyd, xd, wd, rstd, n, dim, dsd, want=("dh",))
    assert none is None and torch.equal(alone, dh)
    none, alone = _grad(wc, dyd, xd, wd, rstd, n, dim, dsd, want=("dw",))
    assert none is None and torch.equal(alone, dw)
    before = torch.randn(dim, generator=g).cuda()
    assert torch.equal(_grad(wc, dyd, xd, wd, rstd, n, dim, dsd, accumulate=before)[1], before + dw)
    work = torch.empty(wc.rms_norm_grad_work_bytes(n, dim), dtype=torch.uint8, device="cuda")
    for into in (dyd.clone(), xd.clone()) + ((dsd.clone(),) if dsum else ()):
        names = dict(dy=dyd, h=xd, ds=dsd)
        for k, t in names.items():
            if t is not None and torch.equal(into, t):
                names[k] = into
        wc.rms_norm_grad_async(names["dy"], names["h"], wd, rstd, n, dim, into, dw, work, work.numel(),
                               dsum_dev=names["ds"])
        assert torch.equal(into, dh)
        assert within(dw, want_dw, tol_dw)


def test_gradient_by_differences(wc):
    """dh and dweight against central differences of the formula in 64 bits, along random directions.

    With step d the differences are off by d^2 / 6 of the third derivative (here below 1e-7 of the sums' magnitudes)."""
    n, dim = 5, 136
    x, _, w, g = _inputs(n, dim, 77, False)
    dy = torch.randn(n, dim, generator=g).to(BF16)
    log("case: rms_norm gradient against differences")
    rstd, y = torch.empty(n, device="cuda"), torch.empty(n, dim, dtype=BF16, device="cuda")
    wc.rms_norm_async(x.cuda(), w.cuda(), n, dim, EPS, y_dev=y, rstd_dev=rstd)
    dh, dw = _grad(wc, dy.cuda(), x.cuda(), w.cuda(), rstd, n, dim, None)
    _, tol, _, tol_dw = Norm64(x, w, EPS).grad(dy)

    def loss(h, weight):
        return float((dy.double() * h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS) * weight).sum())

    step = 1e-4
    for k in range(8):
        along = torch.randn(n, dim, generator=g).double()
        h, weight = x.double(), w.double()
        diff = (loss(h + step * along, weight) - loss(h - step * along, weight)) / (2 * step)
        mag = float((dy.double().abs() * along.abs()).sum())
        assert abs(float((dh.cpu().double() * along).sum()) - diff) <= float((tol * along.abs()).sum()) + 1e-6 * mag
        a = torch.randn(dim, generator=g).double()
        diff = (loss(h, weight + step * a) - loss(h, weight - step * a)) / (2 * step)
        assert abs(float((dw.cpu().double() * a).sum()) - diff) <= float((tol_dw * a.abs()).sum()) + 1e-6 * mag


def test_gradient_of_no_tokens(wc):
    e = torch.empty(0, device="cuda")
    dw = torch.full((64,), 3.0, device="cuda")
    log("case: rms_norm gradient of no tokens")
    args = (e.to(BF16), e.to(BF16), torch.ones(64, dtype=BF16, device="cuda"), e, 0, 64)
    assert wc.rms_norm_grad_work_bytes(0, 64) == 0
    wc.rms_norm_grad_async(*args, e.to(BF16), dw, None, 0, accumulate=True)
    assert bool((dw == 3.0).all())
    wc.rms_norm_grad_async(*args, e.to(BF16), dw, None, 0)
    assert bool((dw == 0.0).all())
    wc.rms_norm_grad_async(*args, e.to(BF16), None, None, 0)
    wc.rms_norm_async(args[0], args[2], 0, 64, EPS, y_dev=args[0])


def test_streams_and_graph(wc):
    """Two calls at once on streams and workspaces of their own, and a captured step that is replayed."""
    n, dim = 300, 1160
    x, r, w, g = _inputs(n, dim, 5, True)
    x, r, w = x.cuda(), r.cuda(), w.cuda()
    dy = torch.randn(n, dim, generator=g).to(BF16).cuda()

    def state():
        return dict(sum=torch.empty_like(x), y=torch.empty_like(x), rstd=torch.empty(n, device="cuda"),
                    dh=torch.empty_like(x), dw=torch.empty(dim, device="cuda"),
                    work=torch.empty(wc.rms_norm_grad_work_bytes(n, dim), dtype=torch.uint8, device="cuda"))

    def step(s, stream=None):
        wc.rms_norm_async(x, w, n, dim, EPS, y_dev=s["y"], residual_dev=r, sum_dev=s["sum"], rstd_dev=s["rstd"],
                          stream=stream)
        wc.rms_norm_grad_async(dy, s["sum"], w, s["rstd"], n, dim, s["dh"], s["dw"], s["work"], s["work"].numel(),
                               dsum_dev=s["y"], stream=stream)

    def same(a, b):
        return all(torch.equal(a[k], b[k]) for k in ("sum", "y", "rstd", "dh", "dw"))

    log("case: rms_norm on two streams and captured")
    want, a, b = state(), state(), state()
    step(want)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    step(a, one)
    step(b, two)
    torch.cuda.synchronize()
    assert same(a, want) and same(b, want)
    s = state()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s)
    for seed in range(3):
        x.copy_(torch.randn(n, dim, generator=torch.Generator().manual_seed(seed)))
        step(want)
        graph.replay()
        torch.cuda.synchronize()
        assert same(s, want)


def test_error_of_rstd_is_counted(wc):
    """The bound that the other tests use for rstd, on sums of many equal squares (where roundings all go one way)."""
    for dim in (64, 4096, 65536):
        x = torch.full((1, dim), 1.0 + 2.0 ** -7).to(BF16)
        y, rstd = torch.empty(1, dim, dtype=BF16, device="cuda"), torch.empty(1, device="cuda")
        wc.rms_norm_async(x.cuda(), torch.ones(dim, dtype=BF16, device="cuda"), 1, dim, 0.0, y_dev=y, rstd_dev=rstd)
        want = 1.0 / (1.0 + 2.0 ** -7)
        assert abs(float(rstd) - want) <= ((8 * 8 + 10) / 2 + 8) * U32 * want

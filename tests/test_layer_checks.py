"""Refusals of the norm, e4m3 and clipping operators, on the CPU: sizes, alignment and types are checked before any
launch, by the library and, for tensors, by the Python binding."""
import ctypes
import math

import pytest
import torch

from test_operator_checks import DevTensor, ReachedC, _check_tensors, _status

P = 1 << 24
INV = -1


@pytest.fixture(scope="module")
def wc():
    from lossless_entropy_coded_amd import wc as mod
    return mod


@pytest.fixture()
def device0(wc, monkeypatch):
    monkeypatch.setattr(wc, "_current_device", lambda: 0)
    real = wc._lib

    class Lib:
        def __getattr__(self, name):
            if name in ("wc_fp8_check", "wc_gemm_fp8_work_bytes", "wc_status_str"):
                return getattr(real, name)
            return lambda *a: (_ for _ in ()).throw(ReachedC())

    monkeypatch.setattr(wc, "_lib", Lib())
    return wc


def _calls(entry, order, ok):
    def call(**kw):
        a = dict(ok, **kw)
        return entry(*[a[k] for k in order], None)
    return call


def test_quant_refusals(wc):
    call = _calls(wc._lib.wc_quant_fp8_async, ("x", "n", "dim", "gated", "codes", "scales"),
                  dict(x=P, n=4, dim=64, gated=0, codes=P, scales=P))
    for bad in (dict(x=0), dict(x=P + 8), dict(codes=0), dict(codes=P + 8), dict(scales=0), dict(scales=P + 2),
                dict(dim=0), dict(dim=12), dict(dim=(1 << 16) + 8), dict(n=(1 << 20) + 1)):
        assert call(**bad) == INV, bad
        assert call(**dict({"gated": 1}, **bad)) == INV, bad
    assert call(n=0, x=0, codes=0, scales=0) == wc.WC_OK


def test_norm_refusals(wc):
    order = ("x", "residual", "weight", "n", "dim", "eps", "sum", "y", "codes", "scales", "rstd")
    call = _calls(wc._lib.wc_rms_norm_async, order, dict(x=P, residual=P, weight=P, n=4, dim=64, eps=1e-5, sum=P, y=P,
                                                         codes=P, scales=P, rstd=P))
    for bad in (dict(x=0), dict(x=P + 8), dict(weight=0), dict(weight=P + 2), dict(residual=P + 8), dict(sum=P + 8),
                dict(residual=0), dict(sum=0), dict(y=P + 8), dict(codes=P + 8), dict(scales=P + 2), dict(rstd=P + 2),
                dict(codes=0), dict(scales=0), dict(y=0, codes=0, scales=0), dict(eps=-1e-9), dict(eps=math.nan),
                dict(dim=0), dict(dim=20), dict(dim=(1 << 16) + 8), dict(n=(1 << 20) + 1)):
        assert call(**bad) == INV, bad
    assert call(n=0, x=0, residual=0, weight=0, sum=0) == wc.WC_OK
    order = ("dy", "h", "weight", "rstd", "dsum", "n", "dim", "dh", "dw", "acc", "work", "work_bytes")
    need = wc.rms_norm_grad_work_bytes(100, 64)
    assert need > 0
    call = _calls(wc._lib.wc_rms_norm_grad_async, order, dict(dy=P, h=P, weight=P, rstd=P, dsum=P, n=100, dim=64, dh=P,
                                                              dw=P, acc=0, work=P, work_bytes=need))
    for bad in (dict(dy=0), dict(dy=P + 8), dict(h=0), dict(h=P + 8), dict(weight=0), dict(weight=P + 8), dict(rstd=0),
                dict(rstd=P + 2), dict(dsum=P + 8), dict(dh=P + 8), dict(dw=P + 2), dict(dh=0, dw=0), dict(work=0),
                dict(work=P + 128), dict(work_bytes=need - 1), dict(dim=0), dict(dim=12), dict(dim=(1 << 16) + 8),
                dict(n=(1 << 20) + 1)):
        assert call(**bad) == INV, bad
    assert call(n=0, dw=0, dy=0, h=0, weight=0, rstd=0, work=0) == wc.WC_OK
    for bad in ((1, 0), (1, 12), (1, (1 << 16) + 8), ((1 << 20) + 1, 8)):
        with pytest.raises(wc.WCError):
            wc.rms_norm_grad_work_bytes(*bad)


def _fp8(wc, codes=P, scales=P, rows=300, cols=64):
    return ctypes.byref(wc._Fp8(codes, scales, rows, cols))


BAD_FP8 = [dict(codes=0), dict(scales=0), dict(codes=P + 8), dict(scales=P + 2), dict(cols=0), dict(cols=8),
           dict(cols=40), dict(cols=(1 << 16) + 16), dict(rows=(1 << 22) + 1)]


def test_gemm_refusals(wc):
    lib, b = wc._lib, ctypes.c_uint64(0)
    for good in ({}, dict(cols=16), dict(cols=1 << 16), dict(rows=1 << 22), dict(rows=0, codes=0, scales=0)):
        assert lib.wc_fp8_check(_fp8(wc, **good)) == wc.WC_OK, good
    for bad in BAD_FP8:
        assert lib.wc_fp8_check(_fp8(wc, **bad)) == INV, bad
        assert lib.wc_gemm_fp8_work_bytes(_fp8(wc, **bad), 4, ctypes.byref(b)) == INV, bad
        assert lib.wc_gemm_fp8_async(_fp8(wc, **bad), P, P, 4, P, 0, P, 1 << 40, None) == INV, bad
    assert lib.wc_fp8_check(None) == INV
    assert lib.wc_gemm_fp8_work_bytes(None, 4, ctypes.byref(b)) == INV
    assert lib.wc_gemm_fp8_work_bytes(_fp8(wc), 4, None) == INV
    wide = dict(rows=4096, cols=1 << 16)
    assert lib.wc_gemm_fp8_work_bytes(_fp8(wc, **wide), 3, ctypes.byref(b)) == wc.WC_OK
    call = _calls(lib.wc_gemm_fp8_async, ("W", "x", "xs", "n", "y", "kind", "work", "work_bytes"),
                  dict(W=_fp8(wc, **wide), x=P, xs=P, n=3, y=P, kind=0, work=P, work_bytes=b.value))
    bad = [dict(W=None), dict(x=0), dict(x=P + 8), dict(xs=0), dict(xs=P + 2), dict(y=0), dict(y=P + 8), dict(kind=2),
           dict(n=(1 << 20) + 1), dict(W=_fp8(wc, rows=1 << 19), n=(1 << 19) + 1)]
    if b.value:
        bad += [dict(work=0), dict(work=P + 128), dict(work_bytes=b.value - 1)]
    for kw in bad:
        assert call(**kw) == INV, kw
    assert call(n=0, x=0, xs=0, y=0, work=0) == wc.WC_OK
    assert call(W=_fp8(wc, rows=0, codes=0, scales=0), x=0, xs=0, y=0, work=0) == wc.WC_OK


def test_gemm_workspaces_are_bounded(wc):
    """Split sums never need more than a few times what the output and the matrix hold."""
    b = ctypes.c_uint64(0)
    for rows in (1, 100, 1024, 5000, 28672, 1 << 22):
        for cols in (16, 128, 4096, 28672, 1 << 16):
            for tokens in (1, 2, 16, 17, 64, 200, 1000, 60000):
                assert wc._lib.wc_gemm_fp8_work_bytes(_fp8(wc, rows=rows, cols=cols), tokens, ctypes.byref(b)) == wc.WC_OK
                assert b.value <= 4 * rows * tokens * -(-cols // 128) and b.value < 1 << 32, (rows, cols, tokens)


def _grads(wc, *items):
    array = (wc._Grad * max(len(items), 1))()
    for i, it in enumerate(items):
        array[i] = wc._Grad(*it)
    return array


def test_clip_refusals(wc):
    lib, b = wc._lib, ctypes.c_uint64(0)
    good = _grads(wc, (P, P, 100, 0), (P + 2, P + 6, 7, 1), (0, 0, 0, 0))
    assert lib.wc_clip_grads_work_bytes(good, 3, ctypes.byref(b)) == wc.WC_OK and b.value > 0
    need = b.value
    for bad in ((0, P, 1, 0), (P, 0, 1, 0), (P + 2, P, 1, 0), (P, P + 2, 1, 0), (P + 1, P, 1, 1), (P, P, 1, 2),
                (P, P, wc.MAX_GRAD_NUMEL + 1, 0)):
        assert lib.wc_clip_grads_work_bytes(_grads(wc, bad), 1, ctypes.byref(b)) == INV, bad
        assert lib.wc_clip_grads_async(_grads(wc, bad), 1, 1.0, P, P, 1 << 40, None) == INV, bad
    assert lib.wc_clip_grads_work_bytes(good, 3, None) == INV
    assert lib.wc_clip_grads_work_bytes(None, 1, ctypes.byref(b)) == INV
    assert lib.wc_clip_grads_work_bytes(good, (1 << 20) + 1, ctypes.byref(b)) == INV
    call = _calls(lib.wc_clip_grads_async, ("grads", "n", "max", "norm", "work", "work_bytes"),
                  dict(grads=good, n=3, max=1.0, norm=P, work=P, work_bytes=need))
    for bad in (dict(max=-1.0), dict(max=math.nan), dict(norm=0), dict(norm=P + 2), dict(work=0), dict(work=P + 128),
                dict(work_bytes=need - 1)):
        assert call(**bad) == INV, bad
    most = _grads(wc, *[(P, P, wc.MAX_GRAD_NUMEL, 0)] * 200)
    assert lib.wc_clip_grads_work_bytes(most, 200, ctypes.byref(b)) == wc.WC_OK and b.value < 1 << 24


# ---- the binding's checks of tensors -----------------------------------------------

def test_binding_norm(device0):
    wc = device0
    call = lambda x, w, r, s, y, c, k, d: wc.rms_norm_async(  # noqa: E731
        x, w, 3, 136, 1e-5, y_dev=y, codes_dev=c, scales_dev=k, residual_dev=r, sum_dev=s, rstd_dev=d, stream=0)
    wide = 2 * 3 * 136
    _check_tensors(wc, call, (wide, 272, wide, wide, wide, 3 * 136, 3 * 2 * 4, 12))
    grad = lambda a, h, w, r, s, d, g, k: wc.rms_norm_grad_async(  # noqa: E731
        a, h, w, r, 3, 136, d, g, k, 4096, dsum_dev=s, stream=0)
    _check_tensors(wc, grad, (wide, wide, 272, 12, wide, wide, 544, 4096))
    t = DevTensor(1 << 20)
    for n, dim in ((-1, 136), (3, -8), (1 << 32, 136), (3, 1 << 32)):
        assert _status(lambda: wc.rms_norm_async(t, t, n, dim, 1e-5, y_dev=t, stream=0)) == INV
        assert _status(lambda: wc.rms_norm_grad_async(t, t, t, t, n, dim, t, t, t, 4096, stream=0)) == INV
        assert _status(lambda: wc.rms_norm_grad_work_bytes(n, dim)) == INV
    wrong = DevTensor(wide, dtype="torch.float16")
    assert _status(lambda: wc.rms_norm_async(wrong, t, 3, 136, 1e-5, y_dev=t, stream=0)) == INV
    assert _status(lambda: wc.rms_norm_grad_async(t, t, t, t, 3, 136, t, t, None, 8, stream=0)) == INV
    assert _status(lambda: wc.rms_norm_grad_async(t, t, t, t, 3, 136, t, None, None, 0, stream=0)) == "reached C"


def test_binding_quant_and_gemm(device0):
    wc = device0
    _check_tensors(wc, lambda x, c, s: wc.quant_fp8_async(x, 3, 136, c, s, stream=0), (816, 408, 24))
    _check_tensors(wc, lambda x, c, s: wc.quant_fp8_async(x, 3, 136, c, s, gated=True, stream=0), (1632, 408, 24))
    for dtype, want in (("torch.float8_e4m3fn", "reached C"), ("torch.uint8", "reached C"), ("torch.int8", "reached C"),
                        ("torch.float8_e5m2", INV), ("torch.float8_e4m3fnuz", INV), ("torch.bfloat16", INV)):
        codes = DevTensor(408, dtype=dtype)
        assert _status(lambda: wc.quant_fp8_async(DevTensor(816), 3, 136, codes, DevTensor(24), stream=0)) == want, dtype
    for i, n in enumerate((130 * 144, 2 * 2 * 4)):
        for t in (DevTensor(n - 1), DevTensor(n, cuda=False), DevTensor(n, index=1), DevTensor(n, contiguous=False)):
            parts = [DevTensor(130 * 144), DevTensor(16)]
            parts[i] = t
            assert _status(lambda: wc.Fp8Matrix(*parts, 130, 144)) == INV, i
    big = DevTensor(1 << 40)
    for rows, cols in ((130, 40), (130, 0), (-1, 144), (1 << 32, 144), ((1 << 22) + 1, 16), (130, (1 << 16) + 16)):
        assert _status(lambda: wc.Fp8Matrix(big, big, rows, cols)) == INV, (rows, cols)
    m = wc.Fp8Matrix(DevTensor(130 * 144), DevTensor(16), 130, 144)
    _check_tensors(wc, lambda x, s, y, w: wc.gemm_fp8_async(m, x, s, 5, y, w, 4096, stream=0),
                   (5 * 144, 5 * 8, 5 * 260, 4096))
    _check_tensors(wc, lambda x, s, y, w: wc.gemm_fp8_async(m, x, s, 5, y, w, 4096, out="f32", stream=0),
                   (5 * 144, 5 * 8, 5 * 520, 4096))
    t = DevTensor(1 << 20)
    assert _status(lambda: wc.gemm_fp8_async(m, t, t, 5, t, None, 0, stream=0)) == "reached C"
    assert _status(lambda: wc.gemm_fp8_async(m, t, t, 5, t, None, 64, stream=0)) == INV
    assert _status(lambda: wc.gemm_fp8_async(m, t, t, 5, t, t, 64, out="f16", stream=0)) == INV
    for tokens in (-1, 1 << 32):
        assert _status(lambda: wc.gemm_fp8_async(m, t, t, tokens, t, t, 64, stream=0)) == INV
        assert _status(lambda: wc.gemm_fp8_work_bytes(m, tokens)) == INV
    m.device = 1
    assert _status(lambda: wc.gemm_fp8_async(m, t, t, 5, t, t, 64, stream=0)) == INV


def test_binding_clip(device0):
    wc = device0

    class Grad(DevTensor):
        next_at = 1 << 24

        def __init__(self, n, dtype="torch.float32", at=None, **kw):
            super().__init__(n * (4 if dtype == "torch.float32" else 2), dtype=dtype, **kw)
            self._n, self._at = n, at or Grad.next_at
            Grad.next_at += 1 << 12

        def data_ptr(self):
            return self._at

        def numel(self):
            return self._n

        def element_size(self):
            return self.nbytes // max(self._n, 1)

    good = [Grad(10), Grad(4, "torch.bfloat16"), Grad(0)]
    handle = wc.GradList(good)
    t = DevTensor(4096)
    assert _status(lambda: wc.clip_grads_async(handle, 1.0, t, t, 4096, stream=0)) == "reached C"
    assert _status(lambda: wc.clip_grads_async(handle, 1.0, DevTensor(3), t, 4096, stream=0)) == INV
    assert _status(lambda: wc.clip_grads_async(handle, 1.0, t, DevTensor(4095), 4096, stream=0)) == INV
    assert _status(lambda: wc.clip_grads_async(handle, 1.0, t, None, 8, stream=0)) == INV
    for grads, outs in (([Grad(10)], []), ([Grad(10)], [Grad(9)]), ([Grad(10)], [Grad(10, "torch.bfloat16")]),
                        ([Grad(10, "torch.float16")], None), ([Grad(10, "torch.int32")], None),
                        ([Grad(10, index=1)], None), ([Grad(10, cuda=False)], None),
                        ([Grad(10, contiguous=False)], None), ([Grad(10)], [Grad(10, contiguous=False)])):
        assert _status(lambda: wc.GradList(grads, outs)) == INV
    handle.device = 1
    assert _status(lambda: wc.clip_grads_async(handle, 1.0, t, t, 4096, stream=0)) == INV

    def g(at, n=10):
        return Grad(n, at=at)

    a = 1 << 20
    for grads, outs in (([g(a), g(a)], None),                            # the same tensor twice, in place
                        ([g(a), g(a + 36)], None),                       # the last element of one is the other's first
                        ([g(a), g(a + 400)], [g(a + 800), g(a + 836)]),  # outputs that overlap
                        ([g(a), g(a + 400)], [g(a + 400), g(a + 800)]),  # an output that is another's gradient
                        ([g(a), g(a + 40)], [g(a + 4), g(a + 400)])):    # an output that is part of its own gradient
        assert _status(lambda: wc.GradList(grads, outs)) == INV
    for grads, outs in (([g(a), g(a + 40)], None), ([g(a), g(a)], [g(a + 400), g(a + 440)]),
                        ([g(a), g(a + 400)], [g(a), g(a + 800)]), ([g(a, 0), g(a), g(a, 0)], None)):
        assert len(wc.GradList(grads, outs)._tensors[0]) == len(grads)


def test_operators_fail_without_a_device(wc):
    """Host tensors never reach a kernel."""
    if torch.cuda.is_available():
        pytest.skip("a device is there")
    t = torch.zeros(4096, dtype=torch.uint8)
    assert _status(lambda: wc.quant_fp8_async(t, 4, 64, t, t, stream=0)) == INV
    assert _status(lambda: wc.rms_norm_async(t, t, 4, 64, 1e-5, y_dev=t, stream=0)) == INV
    assert _status(lambda: wc.Fp8Matrix(t, t, 4, 64)) == INV
    assert _status(lambda: wc.GradList([torch.zeros(4)])) == INV

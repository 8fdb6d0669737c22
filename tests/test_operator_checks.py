"""Refusals of the operators on decoded tensors, on the CPU: sizes, alignment and types are checked before any launch,
by the library (through its C entry points) and, for tensors, by the Python binding."""
import ctypes
import types

import pytest
import torch

P = 1 << 24                 # a well-aligned stand-in for a device pointer (never dereferenced: every call is refused)
INV = -1


@pytest.fixture(scope="module")
def wc():
    from lossless_entropy_coded_amd import wc as mod
    return mod


def _q4(wc, codes=P, scales=P, zeros=0, rows=16, cols=64, group=32):
    return wc._Q4(codes, scales, zeros, rows, cols, group)


BAD_Q4 = [dict(codes=0), dict(scales=0), dict(codes=P + 8), dict(scales=P + 1), dict(cols=0), dict(cols=60),
          dict(cols=4), dict(cols=(1 << 16) + 8), dict(group=0), dict(group=16), dict(group=48),
          dict(rows=(1 << 22) + 1)]


def test_q4_check(wc):
    for good in ({}, dict(zeros=P + 3), dict(cols=8), dict(group=1 << 20), dict(rows=0, codes=0, scales=0),
                 dict(rows=1 << 22), dict(cols=1 << 16)):
        assert wc._lib.wc_q4_check(ctypes.byref(_q4(wc, **good))) == wc.WC_OK, good
    for bad in BAD_Q4:
        assert wc._lib.wc_q4_check(ctypes.byref(_q4(wc, **bad))) == INV, bad
    assert wc._lib.wc_q4_check(None) == INV


def test_gemv_q4_refusals(wc):
    call = wc._lib.wc_gemv_q4_async
    for bad in BAD_Q4:
        assert call(ctypes.byref(_q4(wc, **bad)), P, 1, P, None) == INV, bad
    m = ctypes.byref(_q4(wc))
    assert call(None, P, 1, P, None) == INV
    assert call(m, P, 17, P, None) == INV
    assert call(m, None, 1, P, None) == INV
    assert call(m, P, 1, None, None) == INV
    assert call(m, P + 8, 1, P, None) == INV
    assert call(m, P, 1, P + 2, None) == INV
    assert call(m, None, 0, None, None) == wc.WC_OK
    assert call(ctypes.byref(_q4(wc, rows=0)), None, 4, None, None) == wc.WC_OK


def test_lookup_refusals(wc):
    ok = dict(table=P, vocab=10, dim=64, ids=P, id_bytes=8, n=4, scale=1.0, out=P)

    def call(**kw):
        a = dict(ok, **kw)
        return wc._lib.wc_embed_async(a["table"], a["vocab"], a["dim"], a["ids"], a["id_bytes"], a["n"], a["scale"],
                                      a["out"], None)

    for bad in (dict(table=0), dict(table=P + 8), dict(ids=0), dict(ids=P + 4), dict(ids=P + 2, id_bytes=4),
                dict(id_bytes=2), dict(id_bytes=0), dict(out=0), dict(out=P + 4), dict(dim=0), dict(dim=12),
                dict(dim=(1 << 16) + 8), dict(vocab=(1 << 22) + 1), dict(n=(1 << 20) + 1)):
        assert call(**bad) == INV, bad
    assert call(n=0, ids=0, out=0, table=0) == wc.WC_OK
    q4 = wc._lib.wc_embed_q4_async
    for bad in BAD_Q4:
        assert q4(ctypes.byref(_q4(wc, **bad)), P, 8, 4, 1.0, P, None) == INV, bad
    m = ctypes.byref(_q4(wc))
    for args in ((0, 8, 4, 1.0, P), (P + 4, 8, 4, 1.0, P), (P, 3, 4, 1.0, P), (P, 8, 4, 1.0, 0),
                 (P, 8, 4, 1.0, P + 8), (P, 8, (1 << 20) + 1, 1.0, P)):
        assert q4(m, *args, None) == INV, args
    assert q4(m, None, 8, 0, 1.0, None, None) == wc.WC_OK


def test_gradient_refusals(wc):
    need = wc.embed_grad_work_bytes(100, 64)
    ok = dict(dout=P, ids=P, id_bytes=8, n=100, dtable=P, kind=0, vocab=10, dim=64, acc=0, work=P, work_bytes=need)

    def call(**kw):
        a = dict(ok, **kw)
        return wc._lib.wc_embed_grad_async(a["dout"], a["ids"], a["id_bytes"], a["n"], 1.0, a["dtable"], a["kind"],
                                           a["vocab"], a["dim"], a["acc"], a["work"], a["work_bytes"], None)

    for bad in (dict(dout=0), dict(dout=P + 8), dict(ids=0), dict(ids=P + 4), dict(id_bytes=16), dict(dtable=0),
                dict(dtable=P + 8), dict(kind=2), dict(vocab=(1 << 22) + 1), dict(dim=0), dict(dim=20),
                dict(dim=(1 << 16) + 8), dict(n=(1 << 20) + 1), dict(work=0), dict(work=P + 128),
                dict(work_bytes=need - 1)):
        assert call(**bad) == INV, bad
    assert call(vocab=0, dtable=0) == wc.WC_OK
    assert call(n=0, acc=1, dtable=0, work=0) == wc.WC_OK
    assert wc.embed_grad_work_bytes(0, 8) == 0
    for bad in ((1, 0), (1, 12), (1, (1 << 16) + 8), ((1 << 20) + 1, 8)):
        with pytest.raises(wc.WCError):
            wc.embed_grad_work_bytes(*bad)


def test_cross_entropy_refusals(wc):
    tokens, vocab, dim = 100, 1000, 64
    need_loss = wc.ce_work_bytes(tokens, vocab, dim, grad=False)
    need = wc.ce_work_bytes(tokens, vocab, dim, grad=True)
    assert need >= need_loss > 0
    ok = dict(h=P, W=P, t=P, tb=8, tokens=tokens, vocab=vocab, dim=dim, loss=P, lse=P, dloss=P, dh=P, dW=P, work=P,
              work_bytes=need)

    def loss(**kw):
        a = dict(ok, **dict({"work_bytes": need_loss}, **kw))
        return wc._lib.wc_ce_loss_async(a["h"], a["W"], a["t"], a["tb"], a["tokens"], a["vocab"], a["dim"], a["loss"],
                                        a["lse"], a["work"], a["work_bytes"], None)

    def grad(**kw):
        a = dict(ok, **kw)
        return wc._lib.wc_ce_grad_async(a["h"], a["W"], a["t"], a["tb"], a["tokens"], a["vocab"], a["dim"], a["lse"],
                                        a["dloss"], a["dh"], a["dW"], a["work"], a["work_bytes"], None)

    both = (dict(h=0), dict(h=P + 8), dict(W=0), dict(W=P + 8), dict(t=0), dict(t=P + 4), dict(tb=2), dict(vocab=0),
            dict(vocab=(1 << 22) + 1), dict(dim=0), dict(dim=36), dict(dim=(1 << 16) + 8), dict(tokens=(1 << 20) + 1),
            dict(lse=0), dict(lse=P + 2), dict(work=0), dict(work=P + 128))
    for bad in both + (dict(loss=0), dict(loss=P + 1), dict(work_bytes=need_loss - 1)):
        assert loss(**bad) == INV, bad
    for bad in both + (dict(dloss=0), dict(dloss=P + 2), dict(dh=0, dW=0), dict(dh=P + 8), dict(dW=P + 8),
                       dict(work_bytes=need - 1)):
        assert grad(**bad) == INV, bad
    assert loss(tokens=0, h=0, t=0, loss=0, lse=0, work=0) == wc.WC_OK
    assert grad(tokens=0, h=0, t=0, dloss=0, lse=0, work=0, dW=0) == wc.WC_OK
    assert wc.ce_work_bytes(0, 10, 8) == 0
    for bad in ((1, 0, 8), (1, 8, 0), (1, 8, 12), ((1 << 20) + 1, 8, 8)):
        with pytest.raises(wc.WCError):
            wc.ce_work_bytes(*bad)


def test_cross_entropy_calls_hold_in_a_launch(wc):
    """A tile of z is a workgroup: a call has tiles for fewer than 2^32 threads, or is refused."""
    most = wc.MAX_LOGITS
    for tokens, vocab, more in ((1 << 20, most >> 20, (0, 1)), (most >> 22, 1 << 22, (1, 0))):
        assert wc.ce_work_bytes(tokens, vocab, 64) > 0
        tokens, vocab = tokens + more[0], vocab + more[1]
        with pytest.raises(wc.WCError):
            wc.ce_work_bytes(tokens, vocab, 64)
        args, work = (P, P, P, 8, tokens, vocab, 64), 1 << 60
        assert wc._lib.wc_ce_loss_async(*args, P, P, P, work, None) == INV
        assert wc._lib.wc_ce_grad_async(*args, P, P, P, P, P, work, None) == INV


# ---- the binding's checks of tensors -----------------------------------------------


class DevTensor:
    """A device tensor as the binding's checks see it (never dereferenced)."""

    def __init__(self, nbytes, cuda=True, index=0, contiguous=True, dtype="torch.int64"):
        self.is_cuda, self.dtype = cuda, dtype
        self.device = types.SimpleNamespace(index=index)
        self.nbytes, self._contiguous = nbytes, contiguous

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 1 << 24

    def is_contiguous(self):
        return self._contiguous

    def numel(self):
        return self.nbytes

    def element_size(self):
        return 1


@pytest.fixture()
def device0(wc, monkeypatch):
    """The binding as on a machine whose current device is 0, with calls that get past its checks reported."""
    monkeypatch.setattr(wc, "_current_device", lambda: 0)

    class Lib:
        def __getattr__(self, name):
            if name in ("wc_q4_check", "wc_status_str"):
                return getattr(real, name)
            return lambda *a: (_ for _ in ()).throw(ReachedC())

    real = wc._lib
    monkeypatch.setattr(wc, "_lib", Lib())
    return wc


class ReachedC(Exception):
    pass


def _status(fn):
    try:
        fn()
    except ReachedC:
        return "reached C"
    except Exception as e:  # noqa: BLE001
        return getattr(e, "status", repr(e))
    return "returned"


def _variants(n, dtype="torch.int64"):
    """Stand-ins that the binding must refuse where n bytes are needed on device 0."""
    return {"short": DevTensor(n - 1, dtype=dtype), "on the host": DevTensor(n, cuda=False, dtype=dtype),
            "on another device": DevTensor(n, index=1, dtype=dtype),
            "strided": DevTensor(n, contiguous=False, dtype=dtype)}


def _check_tensors(wc, call, sizes):
    """call(*tensors) reaches C with tensors of the sizes given, and is refused with any one of them unfit."""
    good = [DevTensor(n) for n in sizes]
    assert _status(lambda: call(*good)) == "reached C"
    for i, n in enumerate(sizes):
        for what, t in _variants(n).items():
            assert _status(lambda: call(*good[:i], t, *good[i + 1:])) == wc.WC_ERR_INVALID_ARG, (i, what)


def test_binding_gemv_q4(device0):
    wc = device0
    for i in range(3):
        for what, t in _variants((16 * 32, 2 * 16 * 2, 16 * 2)[i]).items():
            parts = [DevTensor(16 * 32), DevTensor(2 * 16 * 2), DevTensor(16 * 2)]
            parts[i] = t
            assert _status(lambda: wc.Q4Matrix(parts[0], parts[1], 16, 64, 32, zeros=parts[2])) == \
                wc.WC_ERR_INVALID_ARG, (i, what)
    for bad in ((16, 60, 32), (16, 64, 0), (16, 64, 33), (-1, 64, 32), (1 << 32, 64, 32)):
        assert _status(lambda: wc.Q4Matrix(DevTensor(1 << 40), DevTensor(1 << 40), *bad)) == wc.WC_ERR_INVALID_ARG, bad
    m = wc.Q4Matrix(DevTensor(16 * 32), DevTensor(64), 16, 64, 32)
    _check_tensors(wc, lambda x, y: wc.gemv_q4_async(m, x, 3, y, stream=0), (3 * 128, 3 * 64))
    assert _status(lambda: wc.gemv_q4_async(m, DevTensor(1), -1, DevTensor(1), stream=0)) == wc.WC_ERR_INVALID_ARG
    m.device = 1
    assert _status(lambda: wc.gemv_q4_async(m, DevTensor(384), 3, DevTensor(192), stream=0)) == wc.WC_ERR_INVALID_ARG


def test_binding_embed(device0):
    wc = device0
    _check_tensors(wc, lambda t, i, o: wc.embed_async(t, 10, 64, i, 5, o, stream=0), (1280, 40, 640))
    m = wc.Q4Matrix(DevTensor(10 * 32), DevTensor(40), 10, 64, 32)
    _check_tensors(wc, lambda i, o: wc.embed_q4_async(m, i, 5, o, stream=0), (40, 640))
    ids32 = DevTensor(20, dtype="torch.int32")
    assert _status(lambda: wc.embed_async(DevTensor(1280), 10, 64, ids32, 5, DevTensor(640), stream=0)) == "reached C"
    for bad in ("torch.float32", "torch.int16", "torch.uint8"):
        ids = DevTensor(40, dtype=bad)
        assert _status(lambda: wc.embed_async(DevTensor(1280), 10, 64, ids, 5, DevTensor(640), stream=0)) == \
            wc.WC_ERR_INVALID_ARG
    call = lambda d, i, t, w: wc.embed_grad_async(d, i, 5, t, 10, 64, w, 4096, stream=0)  # noqa: E731
    _check_tensors(wc, call, (640, 40, 2560, 4096))
    half = lambda d, i, t, w: wc.embed_grad_async(d, i, 5, t, 10, 64, w, 4096, out="bf16", stream=0)  # noqa: E731
    _check_tensors(wc, half, (640, 40, 1280, 4096))
    assert _status(lambda: wc.embed_grad_async(DevTensor(640), DevTensor(40), 5, DevTensor(2560), 10, 64,
                                               DevTensor(4096), 4096, out="f16", stream=0)) == wc.WC_ERR_INVALID_ARG


def test_binding_cross_entropy(device0):
    wc = device0
    _check_tensors(wc, lambda h, W, t, a, b, w: wc.ce_loss_async(h, W, t, 5, 10, 64, a, b, w, 4096, stream=0),
                   (640, 1280, 40, 20, 20, 4096))
    _check_tensors(wc, lambda h, W, t, e, g, a, b, w: wc.ce_grad_async(h, W, t, 5, 10, 64, e, g, a, b, w, 4096,
                                                                      stream=0),
                   (640, 1280, 40, 20, 20, 640, 1280, 4096))
    good = [DevTensor(n) for n in (640, 1280, 40, 20, 20)]
    args = lambda dh, dW: (good[0], good[1], good[2], 5, 10, 64, good[3], good[4], dh, dW,  # noqa: E731
                           DevTensor(4096), 4096)
    assert _status(lambda: wc.ce_grad_async(*args(None, DevTensor(1280)), stream=0)) == "reached C"
    assert _status(lambda: wc.ce_grad_async(*args(DevTensor(640), None), stream=0)) == "reached C"


def test_operators_fail_without_a_device(wc):
    """Host tensors never reach a kernel."""
    if torch.cuda.is_available():
        pytest.skip("a device is there")
    t = torch.zeros(4096, dtype=torch.uint8)
    ids = torch.zeros(8, dtype=torch.int64)
    assert _status(lambda: wc.Q4Matrix(t, t, 4, 64, 32)) == wc.WC_ERR_INVALID_ARG
    assert _status(lambda: wc.embed_async(t, 4, 64, ids, 8, t, stream=0)) == wc.WC_ERR_INVALID_ARG
    assert _status(lambda: wc.ce_loss_async(t, t, ids, 8, 4, 64, t, t, t, 1, stream=0)) == wc.WC_ERR_INVALID_ARG

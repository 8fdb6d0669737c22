"""Tensors of another floating type than an operator reads are refused before any call, on the CPU.  (Tensors of whole
numbers are taken as the words that they hold: a decoded plane of bf16 may be int16.)"""
import pytest

from test_operator_checks import DevTensor, _status, device0, wc  # noqa: F401  (fixtures)

BIG = 1 << 40
OPERANDS = {   # call: (its operands, the type of each; None: not checked here)
    "gemv_q4": ("bf16", "f32"),
    "embed": ("bf16", None, "bf16"),
    "embed_q4": (None, "bf16"),
    "embed_grad f32": ("bf16", None, "f32", None),
    "embed_grad bf16": ("bf16", None, "bf16", None),
    "ce_loss": ("bf16", "bf16", None, "f32", "f32", None),
    "ce_grad": ("bf16", "bf16", None, "f32", "f32", "bf16", "bf16", None),
}
FLOATS = {"bf16": "torch.bfloat16", "f32": "torch.float32"}
WRONG = ("torch.float16", "torch.float64", "torch.float8_e4m3fn", "torch.complex64")


def _call(wc, name):  # noqa: F811
    m = wc.Q4Matrix(DevTensor(BIG, dtype="torch.uint8"), DevTensor(BIG, dtype="torch.bfloat16"), 16, 64, 32)
    return {
        "gemv_q4": lambda x, y: wc.gemv_q4_async(m, x, 3, y, stream=0),
        "embed": lambda t, i, o: wc.embed_async(t, 10, 64, i, 5, o, stream=0),
        "embed_q4": lambda i, o: wc.embed_q4_async(m, i, 5, o, stream=0),
        "embed_grad f32": lambda d, i, t, w: wc.embed_grad_async(d, i, 5, t, 10, 64, w, 4096, stream=0),
        "embed_grad bf16": lambda d, i, t, w: wc.embed_grad_async(d, i, 5, t, 10, 64, w, 4096, out="bf16", stream=0),
        "ce_loss": lambda h, W, t, a, b, w: wc.ce_loss_async(h, W, t, 5, 10, 64, a, b, w, 4096, stream=0),
        "ce_grad": lambda h, W, t, e, g, a, b, w: wc.ce_grad_async(h, W, t, 5, 10, 64, e, g, a, b, w, 4096, stream=0),
    }[name]


@pytest.mark.parametrize("name", OPERANDS)
def test_floating_types(device0, name):  # noqa: F811
    kinds = OPERANDS[name]
    good = [DevTensor(BIG, dtype=FLOATS.get(k, "torch.int64")) for k in kinds]
    call = _call(device0, name)
    for _ in range(2):          # (types seen before are looked up)
        assert _status(lambda: call(*good)) == "reached C"
        for i, kind in enumerate(kinds):
            if kind is None:
                continue
            for wrong in WRONG + tuple(f for k, f in FLOATS.items() if k != kind):
                bad = [*good[:i], DevTensor(BIG, dtype=wrong), *good[i + 1:]]
                assert _status(lambda: call(*bad)) == device0.WC_ERR_INVALID_ARG, (i, wrong)
            words = [*good[:i], DevTensor(BIG, dtype="torch.int16"), *good[i + 1:]]
            assert _status(lambda: call(*words)) == "reached C"


def test_floating_types_of_a_matrix(device0):  # noqa: F811
    wc = device0  # noqa: F811
    good = dict(codes="torch.uint8", scales="torch.bfloat16", zeros="torch.uint8")
    make = lambda types: wc.Q4Matrix(DevTensor(BIG, dtype=types["codes"]), DevTensor(BIG, dtype=types["scales"]),  # noqa: E731
                                     16, 64, 32, zeros=DevTensor(BIG, dtype=types["zeros"]))
    assert _status(lambda: make(good)) == "returned"
    assert _status(lambda: make(dict(good, codes="torch.int8", scales="torch.int16"))) == "returned"
    for what in good:
        for wrong in WRONG + ("torch.float32",) + (() if what == "scales" else ("torch.bfloat16",)):
            assert _status(lambda: make(dict(good, **{what: wrong}))) == wc.WC_ERR_INVALID_ARG, (what, wrong)


def test_pointers_are_not_checked(device0):  # noqa: F811
    P = 1 << 24
    for name, kinds in OPERANDS.items():
        assert _status(lambda: _call(device0, name)(*[P] * len(kinds))) == "reached C", name

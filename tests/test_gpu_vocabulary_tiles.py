"""GPU tests of the vocabulary cross entropy on the tiles that large vocabularies and large batches take.

Which kernel a size takes is the library's choice; CHOICES names what it is meant to be for each shape here, and
choices() repeats the library's rules (csrc/cross_entropy.hip: takes_thin, takes_big, dh_plan, dw_takes_big, layout) so
that a shape that leaves the kernel which it is here for is seen.  Whoever changes the rules changes both."""
import pytest
import torch

from gpu_util import log
from vocabulary_ref import Vocabulary64, seeded, within

pytestmark = pytest.mark.gpu

CUS, DIES, UNIT = 256, 8, 64


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


def _big(m, n):
    if m <= 128 or n <= 128:
        return False
    big, mid = -(-m // 256) * -(-n // 256), -(-m // 128) * -(-n // 128)
    return 3 * -(-big // CUS) < 2 * -(-mid // (2 * CUS))


def _z(tokens, vocab):
    if tokens <= 64 and -(-vocab // 256) >= CUS // 2:
        return "thin"
    return "big" if _big(vocab, tokens) else "mid"


def _dh(tokens, dim, piece):
    best = (1e30, "", 0)
    for name, m, slots, us in (("big", 256, CUS, 1.1), ("mid", 128, 2 * CUS, 0.8)):
        tiles, s = -(-dim // m) * -(-tokens // m), 1
        while s <= 16 * DIES and (s == 1 or (piece >= s * UNIT and tiles * s <= 4 * slots)):
            time = -(-tiles * s // slots) * (6.0 + -(-piece // s) / UNIT * us) + s * tokens * dim * 8 / 4e6
            if time < best[0]:
                best = (time, name, s)
            s = DIES if s == 1 else s + DIES
    return best[1:]


def choices(tokens, vocab, dim):
    """(loss's tile, pieces, d's tiles, dh's tile and splits, dW's tiles)"""
    rows = tokens * (2 if tokens <= 128 else 1)
    piece = min(max((256 << 20) // (2 * rows) // 1024 * 1024, 1024), -(-vocab // 256) * 256)
    lengths = [min(piece, vocab - v) for v in range(0, vocab, piece)]
    return (_z(tokens, vocab), len(lengths), {_z(tokens, n) for n in lengths}, _dh(tokens, dim, piece),
            {"big" if tokens >= 1024 and _big(dim, n) else "mid" for n in lengths})


CHOICES = {   # tokens, vocab, dim: as choices() gives them
    (1, 33000, 8): ("thin", 1, {"thin"}, ("mid", 128), {"mid"}),
    (16, 32768, 64): ("thin", 1, {"thin"}, ("mid", 128), {"mid"}),
    (33, 32769, 136): ("thin", 1, {"thin"}, ("mid", 128), {"mid"}),
    (64, 40001, 264): ("thin", 1, {"thin"}, ("mid", 120), {"mid"}),
    (200, 100001, 200): ("big", 1, {"big"}, ("mid", 128), {"mid"}),
    (2500, 3000, 520): ("mid", 1, {"mid"}, ("big", 8), {"mid"}),
    (1030, 4000, 1160): ("mid", 1, {"mid"}, ("big", 8), {"mid"}),
    (1100, 9000, 1032): ("big", 1, {"big"}, ("big", 8), {"big"}),
    (1025, 12000, 2056): ("big", 1, {"big"}, ("big", 8), {"big"}),
    (3000, 5000, 2056): ("big", 1, {"big"}, ("mid", 1), {"big"}),
    (9000, 32003, 2056): ("big", 3, {"big"}, ("big", 1), {"mid", "big"}),
}


def test_shapes_take_the_kernels_that_they_are_here_for():
    for shape, what in CHOICES.items():
        assert choices(*shape) == what, shape


def _loss(wc, h, W, t):
    (tokens, dim), vocab = h.shape, W.shape[0]
    loss = torch.full((tokens + 64,), 77.0, device="cuda")
    lse = torch.full((tokens + 64,), 77.0, device="cuda")
    work = torch.full((wc.ce_work_bytes(tokens, vocab, dim, grad=False),), 255, dtype=torch.uint8, device="cuda")
    wc.ce_loss_async(h, W, t, tokens, vocab, dim, loss, lse, work, work.numel())
    torch.cuda.synchronize()
    assert bool((loss[tokens:] == 77.0).all()) and bool((lse[tokens:] == 77.0).all())
    return loss[:tokens], lse[:tokens]


def _grad(wc, h, W, t, lse, dloss, want="hW"):
    (tokens, dim), vocab = h.shape, W.shape[0]
    sizes = {"h": (tokens, dim), "W": (vocab, dim)}
    out = {k: torch.full((a * b + 64,), 77.0, dtype=torch.bfloat16, device="cuda") if k in want else None
           for k, (a, b) in sizes.items()}
    work = torch.full((wc.ce_work_bytes(tokens, vocab, dim),), 255, dtype=torch.uint8, device="cuda")
    wc.ce_grad_async(h, W, t, tokens, vocab, dim, lse, dloss, out["h"], out["W"], work, work.numel())
    torch.cuda.synchronize()
    for k, (a, b) in sizes.items():
        assert out[k] is None or bool((out[k][a * b:] == 77.0).all()), "wrote past a gradient"
    return [None if out[k] is None else out[k][:a * b].reshape(a, b) for k, (a, b) in sizes.items()]


@pytest.mark.parametrize("tokens,vocab,dim", CHOICES)
def test_loss_and_gradients(wc, tokens, vocab, dim):
    h, W, t, dloss = seeded(tokens, vocab, dim, tokens + dim, hot=tokens > 4000)
    if tokens % 2:
        t = t.to(torch.int32)
    ref = Vocabulary64(h, W, t, dloss)
    log(f"case: ce_loss tokens {tokens} vocab {vocab} dim {dim}")
    loss, lse = _loss(wc, h, W, t)
    assert within(lse, ref.lse, ref.lse_tol)
    assert within(loss, ref.loss, ref.loss_tol)
    log(f"case: ce_grad tokens {tokens} vocab {vocab} dim {dim}")
    dh, dW = _grad(wc, h, W, t, lse, dloss)
    assert within(dh, ref.dh, ref.dh_tol)
    assert within(dW, ref.dW, ref.dW_tol)
    # the same bits again, and one gradient without the other
    again = _loss(wc, h, W, t)
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])
    assert torch.equal(_grad(wc, h, W, t, lse, dloss, "h")[0], dh)
    assert torch.equal(_grad(wc, h, W, t, lse, dloss, "W")[1], dW)


@pytest.mark.parametrize("tokens,vocab,dim", [(33, 32769, 136), (1100, 9000, 1032)])
def test_tokens_without_a_loss_hold_anything(wc, tokens, vocab, dim):
    """Infinities and NaNs in h, lse and dloss of tokens without a target leave every gradient's bits as they were."""
    h, W, t, dloss = seeded(tokens, vocab, dim, 4)
    off = (t < 0) | (t >= vocab)
    log(f"case: ce {tokens}x{vocab}x{dim}, tokens without a target not finite")
    loss, lse = _loss(wc, h, W, t)
    dh, dW = _grad(wc, h, W, t, lse, dloss)
    h[off] = float("nan")
    h[off.nonzero()[0], ::2] = float("inf")
    dloss[off] = float("nan")
    loss2, lse2 = _loss(wc, h, W, t)
    assert torch.equal(loss2, loss) and torch.equal(lse2[~off], lse[~off])
    dh2, dW2 = _grad(wc, h, W, t, lse2, dloss)
    assert torch.equal(dh2, dh) and torch.equal(dW2, dW)


@pytest.mark.parametrize("tokens,vocab,dim", [(40, 33001, 72), (1100, 9000, 1032)])
def test_entries_that_are_left_out(wc, tokens, vocab, dim):
    """Vocabulary rows at -inf for positive h leave those entries out of the loss; a NaN in h gives that token NaN, no
    other."""
    h, W, t, dloss = seeded(tokens, vocab, dim, 6, pads=False)
    h[:, 0] = h[:, 0].abs() + 0.5
    out = torch.tensor([0, 300, vocab - 1], device="cuda")
    W[out, 0] = float("-inf")
    t[torch.isin(t, out)] = 1
    keep = torch.ones(vocab, dtype=torch.bool, device="cuda")
    keep[out] = False
    ref = Vocabulary64(h, W[keep], (torch.cumsum(keep, 0) - 1)[t], dloss)
    log(f"case: ce {tokens}x{vocab}x{dim} with entries at -inf")
    loss, lse = _loss(wc, h, W, t)
    assert within(lse, ref.lse, ref.lse_tol) and within(loss, ref.loss, ref.loss_tol)
    h[7, 3] = float("nan")
    loss2, lse2 = _loss(wc, h, W, t)
    rest = torch.arange(tokens, device="cuda") != 7
    assert bool(torch.isnan(loss2[7])) and bool(torch.isnan(lse2[7]))
    assert torch.equal(loss2[rest], loss[rest]) and torch.equal(lse2[rest], lse[rest])

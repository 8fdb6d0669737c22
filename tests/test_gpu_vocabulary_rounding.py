"""GPU tests of what the vocabulary gradients lose to rounding, the rows of targets above all: the largest value of a
token's d goes into dh and dW with more than the eight bits of bf16."""
import pytest
import torch

from gpu_util import log
from vocabulary_ref import Vocabulary64, seeded, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


def _gradients(wc, h, W, t, dloss):
    (tokens, dim), vocab = h.shape, W.shape[0]
    loss, lse = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
    dh, dW = torch.empty_like(h), torch.empty_like(W)
    work = torch.full((wc.ce_work_bytes(tokens, vocab, dim),), 255, dtype=torch.uint8, device="cuda")
    wc.ce_loss_async(h, W, t, tokens, vocab, dim, loss, lse, work, work.numel())
    wc.ce_grad_async(h, W, t, tokens, vocab, dim, lse, dloss, dh, dW, work, work.numel())
    torch.cuda.synchronize()
    return dh, dW


# tokens around 128 (up to which all of d is kept), and more than are looked through at a time (2048, 4096 with the
# large tiles of 9000 x 1032); few entries with many tokens each, and many with few
@pytest.mark.parametrize("tokens,vocab,dim,hot", [(20, 300, 72, False), (128, 2000, 520, True), (129, 2000, 520, False),
                                                  (129, 7, 72, False), (600, 1500, 264, True), (2049, 700, 136, True),
                                                  (5000, 130, 64, False), (1100, 9000, 1032, False),
                                                  (4300, 9000, 1032, True)])
def test_target_rows(wc, tokens, vocab, dim, hot):
    h, W, t, dloss = seeded(tokens, vocab, dim, tokens, hot=hot)
    if tokens % 2:
        t = t.to(torch.int32)
    ref = Vocabulary64(h, W, t, dloss)
    log(f"case: ce_grad roundings, tokens {tokens} vocab {vocab} dim {dim} hot {hot}")
    dh, dW = _gradients(wc, h, W, t, dloss)
    assert within(dh, ref.dh, ref.dh_tol)
    assert within(dW, ref.dW, ref.dW_tol)
    # both norms are over thousands of independent roundings: a tenth is many times their spread
    assert float((dh.double() - ref.dh).norm()) <= 1.1 * ref.dh_off
    assert float((dW.double() - ref.dW).norm()) <= 1.1 * ref.dW_off
    again = _gradients(wc, h, W, t, dloss)
    assert torch.equal(dh, again[0]) and torch.equal(dW, again[1])


@pytest.mark.parametrize("tokens,vocab,dim", [(20, 300, 72), (200, 300, 72), (1100, 9000, 1032)])
def test_infinite_upstream_gradient(wc, tokens, vocab, dim):
    """An infinite dloss makes its token's d infinite and dW with it, of the sign that the formula gives: what an
    infinity loses to rounding is nothing."""
    h, W, t, dloss = seeded(tokens, vocab, dim, 8, pads=False)
    at = tokens // 2
    h[at] = torch.where(h[at] == 0, 1.0, h[at].float()).to(torch.bfloat16)
    for value in (float("inf"), float("-inf")):
        dloss[at] = value
        log(f"case: ce_grad {tokens}x{vocab}x{dim}, dloss {value}")
        dh, dW = _gradients(wc, h, W, t, dloss)
        rows = torch.arange(vocab, device="cuda")
        sign = torch.where(rows == t[at], -1.0, 1.0)[:, None] * h[at].float().sign()[None] * value
        assert torch.equal(dW.float(), sign)
        rest = torch.arange(tokens, device="cuda") != at
        assert bool(torch.isfinite(dh[rest]).all()) and not bool(torch.isfinite(dh[at]).any())

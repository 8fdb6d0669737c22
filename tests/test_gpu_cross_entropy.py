"""GPU tests of the vocabulary product's softmax cross entropy and its gradients."""
import pytest
import torch

from gpu_util import log
from operator_ref import CrossEntropy64, within

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
GUARD = 64


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


def _inputs(tokens, vocab, dim, seed, pads=True, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(tokens, dim, generator=g).to(BF16)
    W = (torch.randn(vocab, dim, generator=g) * (spread / dim ** 0.5)).to(BF16)
    t = torch.randint(0, vocab, (tokens,), generator=g)
    if pads and tokens > 2:
        t[1::5] = -100
        t[2] = vocab
        t[0] = vocab - 1
    dloss = (torch.rand(tokens, generator=g) + 0.5) / tokens
    dloss[::3] *= -1
    return h, W, t, dloss


def _padded(n, dtype, fill):
    return torch.full((n + GUARD,), fill, dtype=dtype, device="cuda")


def _loss(wc, h, W, t, stream=None):
    tokens, dim = h.shape
    vocab = W.shape[0]
    loss, lse = _padded(tokens, torch.float32, 77.0), _padded(tokens, torch.float32, 77.0)
    work = torch.full((max(wc.ce_work_bytes(tokens, vocab, dim, grad=False), 1),), 255, dtype=torch.uint8,
                      device="cuda")
    wc.ce_loss_async(h, W, t, tokens, vocab, dim, loss, lse, work, work.numel(), stream=stream)
    torch.cuda.synchronize()
    assert bool((loss[tokens:] == 77.0).all()) and bool((lse[tokens:] == 77.0).all())
    return loss[:tokens], lse[:tokens]


def _grad(wc, h, W, t, lse, dloss, want="hW"):
    tokens, dim = h.shape
    vocab = W.shape[0]
    dh = _padded(tokens * dim, BF16, 77.0) if "h" in want else None
    dW = _padded(vocab * dim, BF16, 77.0) if "W" in want else None
    work = torch.full((max(wc.ce_work_bytes(tokens, vocab, dim), 1),), 255, dtype=torch.uint8, device="cuda")
    wc.ce_grad_async(h, W, t, tokens, vocab, dim, lse, dloss, dh, dW, work, work.numel())
    torch.cuda.synchronize()
    for b, n in ((dh, tokens * dim), (dW, vocab * dim)):
        assert b is None or bool((b[n:] == 77.0).all()), "wrote past a gradient"
    return (None if dh is None else dh[:tokens * dim].reshape(tokens, dim),
            None if dW is None else dW[:vocab * dim].reshape(vocab, dim))


SHAPES = [(1, 1, 8), (1, 8, 8), (2, 5, 24), (5, 131, 40), (16, 1000, 64), (17, 257, 72), (31, 129, 128),
          (33, 2049, 136), (64, 300, 256), (65, 1024, 264), (127, 515, 64), (128, 128, 64), (130, 700, 200),
          (255, 260, 96), (257, 511, 328), (300, 3000, 64), (515, 1003, 1160), (40, 9000, 64), (700, 2300, 128)]


@pytest.mark.parametrize("tokens,vocab,dim", SHAPES)
def test_loss_and_gradients(wc, tokens, vocab, dim):
    h, W, t, dloss = _inputs(tokens, vocab, dim, tokens + vocab)
    ref = CrossEntropy64(h, W, t, dloss)
    if tokens % 2:
        t = t.to(torch.int32)
    hd, Wd, td, gd = h.cuda(), W.cuda(), t.cuda(), dloss.cuda()
    log(f"case: ce_loss tokens {tokens} vocab {vocab} dim {dim}")
    loss, lse = _loss(wc, hd, Wd, td)
    assert within(lse, ref.lse, ref.lse_tol)
    assert within(loss, ref.loss, ref.loss_tol)
    log(f"case: ce_grad tokens {tokens} vocab {vocab} dim {dim}")
    dh, dW = _grad(wc, hd, Wd, td, lse, gd)
    assert within(dh, ref.dh, ref.dh_tol)
    assert within(dW, ref.dW, ref.dW_tol)
    # the same bits again, and one gradient without the other
    loss2, lse2 = _loss(wc, hd, Wd, td)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    assert torch.equal(_grad(wc, hd, Wd, td, lse, gd, "h")[0], dh)
    assert torch.equal(_grad(wc, hd, Wd, td, lse, gd, "W")[1], dW)


def test_several_pieces(wc):
    """More vocabulary than one piece of the gradient's workspace holds: d spans several pieces."""
    tokens, vocab, dim = 9000, 32000, 64
    h, W, t, dloss = _inputs(tokens, vocab, dim, 3)
    hd, Wd, td, gd = h.cuda(), W.cuda(), t.cuda(), dloss.cuda()
    log("case: ce over several vocabulary pieces")
    loss, lse = _loss(wc, hd, Wd, td)
    dh, dW = _grad(wc, hd, Wd, td, lse, gd)
    # rows of dh (and the loss) do not depend on other tokens: a sample of them against the formula
    at = torch.arange(0, tokens, 97)
    ref = CrossEntropy64(h[at], W, t[at], dloss[at])
    assert within(lse[at.cuda()], ref.lse, ref.lse_tol) and within(loss[at.cuda()], ref.loss, ref.loss_tol)
    assert within(dh[at.cuda()], ref.dh, ref.dh_tol)
    # dW in 64 bits on the GPU, piece by piece
    h64, ok = hd.double(), (td >= 0) & (td < vocab)
    for v0 in range(0, vocab, 8000):
        z = h64 @ Wd[v0:v0 + 8000].double().t()
        d = torch.exp(z - torch.logsumexp(h64 @ Wd.double().t(), dim=1)[:, None])
        inside = ok & (td >= v0) & (td < v0 + 8000)
        d[inside, td[inside] - v0] -= 1
        d *= torch.where(ok, gd.double(), 0.0)[:, None]
        want = d.t() @ h64
        # the bound of the class above with zerr of these sizes (dim 64): d's rounding and the result's
        mag = d.abs().t() @ h64.abs()
        zerr = (dim + 8) * 2.0 ** -23 * 64.0
        tol = mag * (2.0 ** -8 + 4 * zerr + (tokens + 8) * 2.0 ** -23) * 1.01 + 2.0 ** -8 * 1.01 * want.abs()
        assert within(dW[v0:v0 + 8000], want.cpu(), tol.cpu())


def test_peaked_and_flat_rows(wc):
    """A token whose target holds nearly all the mass (d next to zero), one whose logits are all equal, large logits."""
    tokens, vocab, dim = 6, 600, 64
    h, W, t, dloss = _inputs(tokens, vocab, dim, 5, pads=False)
    h[0] = W[int(t[0])] * 30
    h[1] = 0
    h[2] *= 50
    ref = CrossEntropy64(h, W, t, dloss)
    hd, Wd, td = h.cuda(), W.cuda(), t.cuda()
    log("case: ce peaked, flat and large rows")
    loss, lse = _loss(wc, hd, Wd, td)
    assert within(lse, ref.lse, ref.lse_tol) and within(loss, ref.loss, ref.loss_tol)
    dh, dW = _grad(wc, hd, Wd, td, lse, dloss.cuda())
    assert within(dh, ref.dh, ref.dh_tol) and within(dW, ref.dW, ref.dW_tol)


def test_all_tokens_masked(wc):
    """No token has a target: zero loss and gradients, whatever dloss holds; lse is still written."""
    h, W, t, dloss = _inputs(20, 300, 64, 6)
    t[:] = -1
    dloss[:] = float("nan")
    hd, Wd, td = h.cuda(), W.cuda(), t.cuda()
    log("case: ce with every token masked")
    loss, lse = _loss(wc, hd, Wd, td)
    ref = CrossEntropy64(h, W, t)
    assert bool((loss == 0).all()) and within(lse, ref.lse, ref.lse_tol)
    dh, dW = _grad(wc, hd, Wd, td, lse, dloss.cuda())
    assert bool((dh == 0).all()) and bool((dW == 0).all())


def test_non_finite_logits(wc):
    """A vocabulary row at -inf for positive h leaves that entry out; a NaN in h gives that token NaN, no other."""
    tokens, vocab, dim = 40, 700, 64
    h, W, t, _ = _inputs(tokens, vocab, dim, 7, pads=False)
    h[:, 0] = h[:, 0].abs() + 0.5
    W[300, 0] = float("-inf")
    t[t == 300] = 0
    keep = torch.arange(vocab) != 300
    shifted = torch.where(t > 300, t - 1, t)
    ref = CrossEntropy64(h, W[keep], shifted)
    log("case: ce with a vocabulary entry at -inf")
    loss, lse = _loss(wc, h.cuda(), W.cuda(), t.cuda())
    assert within(lse, ref.lse, ref.lse_tol) and within(loss, ref.loss, ref.loss_tol)
    h[7, 3] = float("nan")
    loss2, lse2 = _loss(wc, h.cuda(), W.cuda(), t.cuda())
    rest = torch.arange(tokens) != 7
    assert bool(torch.isnan(loss2[7])) and bool(torch.isnan(lse2[7]))
    assert torch.equal(loss2[rest.cuda()], loss[rest.cuda()])


@pytest.mark.parametrize("tokens,vocab,dim", [(9, 300, 72), (150, 2000, 264), (700, 2300, 128)])
def test_tokens_without_a_loss_hold_anything(wc, tokens, vocab, dim):
    """Infinities and NaNs in h, lse and dloss of tokens without a target leave every gradient's bits as they were."""
    h, W, t, dloss = _inputs(tokens, vocab, dim, 11)
    Wd, td = W.cuda(), t.cuda()
    off = (t < 0) | (t >= vocab)
    log(f"case: ce {tokens}x{vocab}x{dim}, tokens without a target not finite")
    loss, lse = _loss(wc, h.cuda(), Wd, td)
    dh, dW = _grad(wc, h.cuda(), Wd, td, lse, dloss.cuda())
    where = off.nonzero().flatten()
    h[where] = float("nan")
    h[where[0], ::2] = float("inf")
    dloss[where] = float("nan")
    loss2, lse2 = _loss(wc, h.cuda(), Wd, td)
    assert torch.equal(loss2, loss) and torch.equal(lse2[~off.cuda()], lse[~off.cuda()])
    dh2, dW2 = _grad(wc, h.cuda(), Wd, td, lse2, dloss.cuda())
    assert torch.equal(dh2, dh) and torch.equal(dW2, dW)


def test_no_tokens(wc):
    """No tokens: nothing but a zero dW."""
    W = torch.randn(50, 16).to(BF16).cuda()
    h = torch.zeros(0, 16, dtype=BF16, device="cuda")
    z = torch.zeros(0, device="cuda")
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    assert wc.ce_work_bytes(0, 50, 16) == 0
    log("case: ce of no tokens")
    _loss(wc, h, W, t)
    _, dW = _grad(wc, h, W, t, z, z)
    assert bool((dW == 0).all())


def test_gradient_against_differences(wc):
    """dh and dW against central differences of the 64-bit loss along random directions."""
    tokens, vocab, dim = 50, 400, 72
    h, W, t, dloss = _inputs(tokens, vocab, dim, 9)
    hd, Wd, td = h.cuda(), W.cuda(), t.cuda()
    _, lse = _loss(wc, hd, Wd, td)
    dh, dW = _grad(wc, hd, Wd, td, lse, dloss.cuda())
    ref = CrossEntropy64(h, W, t, dloss)
    g = torch.Generator().manual_seed(1)
    sh = torch.randn(tokens, dim, generator=g, dtype=torch.float64)
    sW = torch.randn(vocab, dim, generator=g, dtype=torch.float64)
    total = lambda a, b: float((CrossEntropy64(a, b, t).loss * dloss.double()).sum())  # noqa: E731
    e = 1e-4
    slope_h = (total(h.double() + e * sh, W.double()) - total(h.double() - e * sh, W.double())) / (2 * e)
    slope_W = (total(h.double(), W.double() + e * sW) - total(h.double(), W.double() - e * sW)) / (2 * e)
    # differences: e^2 / 6 of the third derivative, below 1e-5 here; the kernel: its bound along the direction
    assert abs(float((dh.cpu().double() * sh).sum()) - slope_h) <= float((ref.dh_tol * sh.abs()).sum()) + 1e-5
    assert abs(float((dW.cpu().double() * sW).sum()) - slope_W) <= float((ref.dW_tol * sW.abs()).sum()) + 1e-5


def test_side_stream_and_graph(wc):
    """Loss and gradients captured in one graph, replayed on new inputs, against eager calls on the current stream."""
    tokens, vocab, dim = 150, 1500, 128
    sets = [_inputs(tokens, vocab, dim, s) for s in (1, 2, 3)]
    h, W, t, g = (x.cuda() for x in sets[0])
    loss, lse = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
    dh, dW = torch.empty_like(h), torch.empty_like(W)
    work = torch.empty(wc.ce_work_bytes(tokens, vocab, dim), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wc.ce_loss_async(h, W, t, tokens, vocab, dim, loss, lse, work, work.numel())
        wc.ce_grad_async(h, W, t, tokens, vocab, dim, lse, g, dh, dW, work, work.numel())
    side = torch.cuda.Stream()
    for i in (1, 2, 0, 1):
        log(f"case: ce captured, inputs {i}")
        for dst, src in zip((h, W, t, g), sets[i]):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        loss2, lse2 = _loss(wc, h, W, t, stream=side)
        dh2, dW2 = _grad(wc, h, W, t, lse2, g)
        assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
        assert torch.equal(dh, dh2) and torch.equal(dW, dW2)


def _relative(got, ref):
    return float((got.cpu().double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("tokens,vocab,dim", [(1, 700, 64), (7, 3000, 136), (64, 5000, 256), (128, 2000, 520),
                                              (129, 2000, 520), (600, 1500, 264)])
def test_gradients_lose_little_to_rounding(wc, tokens, vocab, dim):
    """In the 2-norm, which averages roundings: dh and dW are off by their own rounding to bf16 and little more; from
    129 tokens on dW takes d rounded to bf16 too, as much again and independent of it."""
    h, W, t, dloss = _inputs(tokens, vocab, dim, 21, pads=False)
    ref = CrossEntropy64(h, W, t, dloss)
    hd, Wd, td = h.cuda(), W.cuda(), t.cuda()
    log(f"case: ce_grad roundings, tokens {tokens} vocab {vocab} dim {dim}")
    _, lse = _loss(wc, hd, Wd, td)
    dh, dW = _grad(wc, hd, Wd, td, lse, dloss.cuda())
    alone = [_relative(r.to(BF16), r) for r in (ref.dh, ref.dW)]
    # dh: d's non-target values, at most 1 / (1 - p) of the target's in sum, lose 2^-8 of themselves at most
    assert _relative(dh, ref.dh) <= 1.5 * alone[0]
    assert _relative(dW, ref.dW) <= (1.1 if tokens <= 128 else 1.6) * alone[1]

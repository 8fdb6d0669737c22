"""GPU tests of the embedding lookup (bf16 and 4-bit tables) and its gradient."""
import pytest
import torch

from gpu_util import log
from operator_ref import embed_grad_ref, q4_case, within

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


def _ids(vocab, n, seed, dtype=torch.int64, pads=True):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, vocab, (n,), generator=g)
    if pads and n > 3:
        ids[::7] = -1
        ids[3::11] = vocab
        ids[2] = -2 ** 31 if dtype == torch.int32 else -2 ** 62
        ids[-1] = vocab - 1
        ids[0] = 0
    return ids.to(dtype)


def _guarded(n, dim):
    buf = torch.full((n * dim + 64,), 123.0, dtype=BF16, device="cuda")
    return buf, buf[:n * dim].reshape(n, dim)


LOOKUPS = [(1, 8, 1), (5, 8, 3), (7, 24, 33), (100, 256, 70), (50, 1160, 19), (33, 2048, 300), (20, 4096, 1),
           (9, 8200, 40), (1000, 264, 1000)]


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("vocab,dim,n", LOOKUPS)
def test_lookup(wc, vocab, dim, n, dtype):
    table = torch.randn(vocab, dim, generator=torch.Generator().manual_seed(dim)).to(BF16)
    ids = _ids(vocab, n, n, dtype)
    ok = (ids >= 0) & (ids < vocab)
    rows = table[torch.where(ok, ids, 0).long()]
    rows[~ok] = 0
    for scale in (1.0, 11.5):
        log(f"case: embed {vocab}x{dim} n {n} {dtype} scale {scale}")
        buf, out = _guarded(n, dim)
        wc.embed_async(table.cuda(), vocab, dim, ids.cuda(), n, out, scale=scale)
        torch.cuda.synchronize()
        assert bool((buf[n * dim:] == 123.0).all()), "wrote past out"
        if scale == 1.0:
            assert torch.equal(out.cpu().view(torch.int16), rows.view(torch.int16))
        else:
            ref = rows.double() * scale
            # one fp32 product (2^-24) rounded to bf16 (2^-8 at most)
            assert within(out, ref, ref.abs() * (2.0 ** -8 + 2.0 ** -23))


def test_lookup_keeps_special_words(wc):
    """Scale 1 copies bits: NaN payloads, infinities, -0, subnormals."""
    words = torch.tensor([0x7FC1, 0x7F80, -0x80, -0x8000, 0x0001, 0x7F81, 0x3F80, 0x0000], dtype=torch.int16)
    table = words.reshape(1, 8).view(BF16).cuda()
    out = torch.empty(2, 8, dtype=BF16, device="cuda")
    wc.embed_async(table, 1, 8, torch.zeros(2, dtype=torch.int64, device="cuda"), 2, out)
    assert torch.equal(out.cpu().view(torch.int16), words.repeat(2, 1))


@pytest.mark.parametrize("vocab,dim,n,group,zeros", [(1, 8, 1, 32, False), (6, 24, 9, 32, True), (40, 256, 70, 64, True),
                                                     (50, 1160, 33, 96, True), (33, 4096, 100, 128, False),
                                                     (9, 8200, 40, 65536, True)])
def test_lookup_q4(wc, vocab, dim, n, group, zeros):
    codes, scales, z, w = q4_case(vocab, dim, group, zeros, dim)
    ids = _ids(vocab, n, n)
    ok = (ids >= 0) & (ids < vocab)
    matrix = wc.Q4Matrix(codes, scales, vocab, dim, group, zeros=z)
    for scale in (1.0, 45.25):
        log(f"case: embed_q4 {vocab}x{dim} n {n} group {group} zeros {zeros} scale {scale}")
        buf, out = _guarded(n, dim)
        wc.embed_q4_async(matrix, ids.cuda(), n, out, scale=scale)
        torch.cuda.synchronize()
        assert bool((buf[n * dim:] == 123.0).all()), "wrote past out"
        ref = w[torch.where(ok, ids, 0)] * scale
        ref[~ok] = 0
        # scale * (code - zero point) is exact in fp32; one product and the rounding to bf16 follow
        assert within(out, ref, ref.abs() * (2.0 ** -8 + 2.0 ** -23))


GRADS = [(1, 8, 1), (3, 8, 5), (10, 24, 31), (10, 24, 32), (10, 24, 33), (4, 264, 200), (300, 1160, 97),
         (1, 2056, 1000), (5000, 64, 4095), (70, 64, 4096), (5000, 64, 4097), (50, 40, 9000), (3, 32, 20000)]


def _grad(wc, dout, ids, vocab, out, scale, accumulate=False, start=None):
    n, dim = dout.shape
    t = torch.float32 if out == "f32" else BF16
    buf = torch.full((vocab * dim + 64,), 7.0, dtype=t, device="cuda")
    if start is not None:
        buf[:vocab * dim] = start.reshape(-1).cuda()
    work = torch.full((wc.embed_grad_work_bytes(n, dim),), 255, dtype=torch.uint8, device="cuda")
    wc.embed_grad_async(dout.cuda(), ids.cuda(), n, buf, vocab, dim, work, work.numel(), out=out, scale=scale,
                        accumulate=accumulate)
    torch.cuda.synchronize()
    assert bool((buf[vocab * dim:] == 7.0).all()), "wrote past dtable"
    return buf[:vocab * dim].reshape(vocab, dim)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("vocab,dim,n", GRADS)
def test_gradient(wc, vocab, dim, n, out):
    g = torch.Generator().manual_seed(n)
    dout = torch.randn(n, dim, generator=g).to(BF16)
    for what, ids in (("spread", _ids(vocab, n, n, torch.int32)), ("spread, no pads", _ids(vocab, n, n, pads=False)),
                      ("half on one row", torch.where(torch.rand(n, generator=g) < 0.5, vocab // 2,
                                                      _ids(vocab, n, n + 1)))):
        log(f"case: embed_grad {vocab}x{dim} n {n} {out} {what}")
        ref, mag, most = embed_grad_ref(dout, ids, vocab, 11.5)
        got = _grad(wc, dout, ids, vocab, out, 11.5)
        # at most `most` fp32 sums and the product with the scale; bf16: rounded once
        tol = (most + 2) * 2.0 ** -24 * mag * 1.01 + (2.0 ** -8 * 1.01 * ref.abs() if out == "bf16" else 0)
        assert within(got, ref, tol), what
        again = _grad(wc, dout, ids, vocab, out, 11.5)
        assert torch.equal(got, again), "two runs differ"


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_gradient_accumulates(wc, out):
    """Sums go on top of the table's values; rows without tokens keep theirs, bit for bit."""
    vocab, dim, n = 40, 136, 500
    g = torch.Generator().manual_seed(8)
    dout = torch.randn(n, dim, generator=g).to(BF16)
    ids = torch.randint(0, 20, (n,), generator=g) * 2
    start = torch.randn(vocab, dim, generator=g).to(torch.float32 if out == "f32" else BF16)
    log(f"case: embed_grad accumulate {out}")
    ref, mag, most = embed_grad_ref(dout, ids, vocab, 0.5)
    got = _grad(wc, dout, ids, vocab, out, 0.5, accumulate=True, start=start)
    assert torch.equal(got[1::2].cpu(), start[1::2])
    ref = ref + start.double()
    tol = (most + 3) * 2.0 ** -24 * (mag + start.double().abs()) * 1.01
    if out == "bf16":
        tol = tol + 2.0 ** -8 * 1.01 * ref.abs()
    assert within(got, ref, tol)


def test_gradient_without_tokens(wc):
    """No tokens, and none inside the vocabulary: a table of zeros, or one left as it was."""
    dout = torch.randn(50, 16).to(BF16)
    start = torch.randn(9, 16)
    for n, ids in ((0, torch.zeros(0, dtype=torch.int64)), (50, torch.full((50,), -1))):
        log(f"case: embed_grad of {n} tokens, none valid")
        assert bool((_grad(wc, dout[:n], ids, 9, "f32", 1.0) == 0).all())
        assert bool((_grad(wc, dout[:n], ids, 9, "bf16", 1.0) == 0).all())
        assert torch.equal(_grad(wc, dout[:n], ids, 9, "f32", 1.0, accumulate=True, start=start).cpu(), start)


def test_gradient_against_differences(wc):
    """The gradient of L = sum(out * v) by central differences of L in 64 bits along a random direction."""
    vocab, dim, n, scale = 30, 64, 90, 3.0
    g = torch.Generator().manual_seed(1)
    ids = _ids(vocab, n, 4)
    v = torch.randn(n, dim, generator=g).to(BF16)
    table = torch.randn(vocab, dim, generator=g, dtype=torch.float64)
    step = torch.randn(vocab, dim, generator=g, dtype=torch.float64)
    ok = (ids >= 0) & (ids < vocab)
    loss = lambda t: float((torch.where(ok[:, None], t[torch.where(ok, ids, 0)], 0.0) * scale * v.double()).sum())
    slope = (loss(table + 1e-3 * step) - loss(table - 1e-3 * step)) / 2e-3
    got = _grad(wc, v, ids, vocab, "f32", scale).cpu().double()
    ref, mag, most = embed_grad_ref(v, ids, vocab, scale)
    assert abs(float((got * step).sum()) - slope) <= float(((most + 2) * 2.0 ** -24 * mag * step.abs()).sum()) + \
        1e-9 * abs(slope) + 1e-9 * float((mag * step.abs()).sum())


def test_side_stream_and_graph(wc):
    """Lookup and gradient captured in one graph and replayed on new ids, against eager calls."""
    vocab, dim, n = 500, 128, 5000
    g = torch.Generator().manual_seed(2)
    table = torch.randn(vocab, dim, generator=g).to(BF16).cuda()
    dout = torch.randn(n, dim, generator=g).to(BF16)
    batches = [_ids(vocab, n, s) for s in (1, 2, 3)]
    ids = batches[0].cuda()
    out = torch.empty(n, dim, dtype=BF16, device="cuda")
    grad = torch.empty(vocab, dim, device="cuda")
    work = torch.empty(wc.embed_grad_work_bytes(n, dim), dtype=torch.uint8, device="cuda")
    d = dout.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wc.embed_async(table, vocab, dim, ids, n, out, scale=2.0)
        wc.embed_grad_async(d, ids, n, grad, vocab, dim, work, work.numel(), scale=2.0)
    side = torch.cuda.Stream()
    for i in (1, 2, 0, 1):
        log(f"case: embed and embed_grad captured, batch {i}")
        ids.copy_(batches[i])
        out.zero_(), grad.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        want = _grad(wc, dout, batches[i], vocab, "f32", 2.0)
        rows = torch.empty_like(out)
        torch.cuda.synchronize()
        wc.embed_async(table, vocab, dim, ids, n, rows, scale=2.0, stream=side)
        side.synchronize()
        assert torch.equal(out, rows) and torch.equal(grad, want)


def _large_table(wc, vocab, dim, n, out):
    if torch.cuda.mem_get_info()[0] < vocab * dim * (4 if out == "f32" else 2) * 5 // 4:
        pytest.skip("needs more device memory")
    g = torch.Generator().manual_seed(8)
    ids = torch.randint(0, vocab, (n,), generator=g)
    ids[0], ids[1], ids[2] = 0, vocab - 1, -1
    dout = torch.randn(n, dim, generator=g).to(BF16)
    log(f"case: embed_grad {vocab}x{dim} {out}, {n} tokens")
    table = torch.full((vocab, dim), 1.0, dtype=torch.float32 if out == "f32" else BF16, device="cuda")
    work = torch.empty(wc.embed_grad_work_bytes(n, dim), dtype=torch.uint8, device="cuda")
    wc.embed_grad_async(dout.cuda(), ids.cuda(), n, table, vocab, dim, work, work.numel(), out=out)
    torch.cuda.synchronize()
    rows, where = ids[ids >= 0].unique(return_inverse=True)
    d = dout[ids >= 0].double()
    want = torch.zeros(len(rows), dim, dtype=torch.float64).index_add_(0, where, d)
    mag = torch.zeros(len(rows), dim, dtype=torch.float64).index_add_(0, where, d.abs())
    got = table[rows.cuda()]
    # fewer than n sums within 2^-24 each, then one rounding to the output's type
    tol = mag * n * 2.0 ** -24 + (want.abs() * 2.0 ** -8 if out == "bf16" else 0)
    assert bool(((got.cpu().double() - want).abs() <= tol).all())
    table[rows.cuda()] = 0
    for part in table.view(torch.int16).split(1 << 17):
        assert int(part.count_nonzero()) == 0, "a row without tokens was not written"


def test_gradient_of_a_table_beyond_a_launch(wc):
    """More 16-byte pieces than a launch has threads: every row is written all the same."""
    _large_table(wc, 1 << 22, 8256, 100, "bf16")
    torch.cuda.empty_cache()


@pytest.mark.parametrize("vocab,dim,n,out", [(70000, 1024, 5000, "f32"), (70001, 1032, 4097, "bf16"),
                                             (40000, 2056, 12000, "f32"), (300000, 392, 9000, "bf16"),
                                             (9000, 8200, 6000, "f32"), (1 << 21, 64, 700, "f32"),
                                             (50, 72, 1024, "f32"), (50, 72, 1025, "f32"), (1, 8, 8192, "f32"),
                                             (7000, 64, 8191, "bf16"), (7000, 64, 8193, "bf16"), (1, 8, 8193, "f32"),
                                             (1 << 22, 8, 9001, "f32"), (1 << 20, 64, 12345, "bf16")])
def test_gradient_of_tables_written_by_several_launches(wc, vocab, dim, n, out):
    """Tables whose rows are set beside the sort, beside the ranking and by the summing launch; sizes where the way of
    sorting changes."""
    _large_table(wc, vocab, dim, n, out)

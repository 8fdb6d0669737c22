"""GPU tests that NaN stays where it belongs, and that views, streams and graphs do, on the tiles of products with e4m3
matrices in bf16."""
import pytest
import torch

from e4m3_ref import blocks, quantised
from gpu_util import log
from test_gpu_gemm_fp8 import _case, _run

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


# a size of each tile in bf16, those of 256 x 256 with whole and with odd rows, and two in fp32
NAN = [(256, 512, 1, "bf16"), (256, 512, 20, "bf16"), (300, 400, 200, "bf16"), (4138, 400, 49, "bf16"), (4110, 272, 70, "bf16"),
       (16645, 400, 171, "bf16"), (1027, 4016, 454, "bf16"), (2051, 1040, 515, "bf16"), (4100, 656, 1030, "bf16"),
       (4352, 272, 4100, "bf16"), (4097, 272, 4097, "bf16"), (1027, 4016, 454, "f32"), (261, 656, 33100, "f32")]


@pytest.mark.parametrize("rows,cols,tokens,out", NAN)
def test_no_numbers_stay_among_themselves(wc, rows, cols, tokens, out):
    """A NaN code or scale reaches its own row, or the rows of its block, or its own token alone, and nothing else changes."""
    codes, scales, _, xc, xs, _ = _case(rows, cols, tokens, 9)
    log(f"case: gemm_fp8 NaN, {rows}x{cols}, {tokens} tokens, {out}")
    codes, scales, xc, xs = codes.view(torch.uint8).cuda(), scales.cuda(), xc.view(torch.uint8).cuda(), xs.cuda()
    want = _run(wc, wc.Fp8Matrix(codes, scales, rows, cols), xc, xs, tokens, out)
    assert bool(torch.isfinite(want).all())

    def check(bad_rows, bad_tokens, codes=codes, scales=scales, xc=xc, xs=xs):
        y = _run(wc, wc.Fp8Matrix(codes, scales, rows, cols), xc, xs, tokens, out)
        bad = torch.zeros(tokens, rows, dtype=torch.bool, device="cuda")
        bad[:, bad_rows] = True
        bad[bad_tokens] = True
        assert bool(torch.isnan(y[bad]).all()) and torch.equal(y[~bad], want[~bad])

    none = slice(0, 0)
    for r in (0, rows // 2, rows - 1):
        c = codes.clone()
        c[r, cols - 1 if r else 0] = 0x7F
        check(r, none, codes=c)
    s = scales.clone()
    s[-1, 0] = float("nan")
    check(slice((rows - 1) // 128 * 128, rows), none, scales=s)
    for t in (0, tokens // 2, tokens - 1):
        c, s = xc.clone(), xs.clone()
        c[t, cols // 2] = 0xFF
        check(none, t, xc=c)
        s[t, blocks(cols) - 1] = float("nan")
        check(none, t, xs=s)


@pytest.mark.parametrize("rows,cols,tokens", [(520, 1296, 7), (520, 1296, 150), (1001, 4112, 333), (2051, 1040, 515),
                                              (8387, 5456, 65), (4097, 272, 4097), (4352, 272, 4100)])
def test_views_streams_and_graph_in_bf16(wc, rows, cols, tokens):
    """Operands that lie inside larger tensors whose neighbours are NaN, two streams at once, and a captured call that is
    replayed with other activations."""
    codes, scales, w, xc, xs, x = _case(rows, cols, tokens, tokens + 3)
    log(f"case: gemm_fp8 views, streams and graph, {rows}x{cols}, {tokens} tokens, bf16")

    def inside(t, fill, pad):
        big = torch.full((t.numel() + 2 * pad,), fill, dtype=t.dtype, device="cuda")
        view = big[pad:pad + t.numel()]
        view.copy_(t.flatten())
        return view

    wv, xv = inside(codes.view(torch.uint8), 0x7F, 4096), inside(xc.view(torch.uint8), 0x7F, 4096)
    sv, xsv = inside(scales, float("nan"), 64), inside(xs, float("nan"), 64)
    W = wc.Fp8Matrix(wv, sv, rows, cols)
    y = _run(wc, W, xv, xsv, tokens, "bf16")
    whole = wc.Fp8Matrix(codes.cuda(), scales.cuda(), rows, cols)
    assert bool(torch.isfinite(y).all()) and torch.equal(y, _run(wc, whole, xc.cuda(), xs.cuda(), tokens, "bf16"))
    need = wc.gemm_fp8_work_bytes(W, tokens)
    calls = [(torch.cuda.Stream(), torch.empty(tokens, rows, dtype=BF16, device="cuda"),
              torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    for stream, into, work in calls:
        wc.gemm_fp8_async(W, xv, xsv, tokens, into, work, need, out="bf16", stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(into, y) for _, into, _ in calls)
    into, work = calls[0][1:]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wc.gemm_fp8_async(W, xv, xsv, tokens, into, work, need, out="bf16")
    for seed in range(3):
        other, others = quantised(torch.randn(tokens, cols, generator=torch.Generator().manual_seed(seed)))
        xv.copy_(other.view(torch.uint8).flatten())
        xsv.copy_(others.flatten())
        eager = _run(wc, W, xv, xsv, tokens, "bf16")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(into, eager)

"""The norm, e4m3 and clipping operators together, as a program uses them: a gated layer whose matrices are decoded from
containers of e4m3 planes, and a training step from the embedding to the clipped gradients."""
import pytest
import torch

from e4m3_ref import (BLOCK, Norm64, UBF16, blocks, check_codes, gemm_tolerance, matrix_codes, per_column, values_of,
                      within)
from gpu_util import log, to_device_aligned
from operator_ref import CrossEntropy64, embed_grad_ref
from operator_ref import within as close

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn
EPS = 1e-5


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


@pytest.mark.parametrize("dim,ffn,tokens", [(256, 640, 1), (272, 400, 19), (512, 1296, 200)])
def test_layer(wc, dim, ffn, tokens):
    """Norm with the residual into codes, gate and up products, their gated codes, the down product, and the next norm:
    each step within its own bound, given what the step before it wrote."""
    g = torch.Generator().manual_seed(dim)
    up_codes, up_scales, up = matrix_codes(torch.randn(2 * ffn, dim, generator=g) * 0.05)
    down_codes, down_scales, down = matrix_codes(torch.randn(dim, ffn, generator=g) * 0.05)
    x, r = torch.randn(tokens, dim, generator=g).to(BF16), torch.randn(tokens, dim, generator=g).to(BF16)
    weight = (torch.randn(dim, generator=g) * 0.2 + 1).to(BF16)
    log(f"case: layer {dim} x {ffn}, {tokens} tokens")
    blob = wc.encode_u8_host([up_codes.view(torch.uint8), down_codes.view(torch.uint8)])
    with wc.Plan(blob) as plan:
        _, dblob = to_device_aligned(blob)
        plane = torch.empty(plan.n_elems, dtype=torch.uint8, device="cuda")
        wc.decode_u8_async(plan, dblob, plane)
        at, n = plan.tensor_offsets, plan.tensor_numels
        W_up = wc.Fp8Matrix(plane[at[0]:at[0] + n[0]], up_scales.cuda(), 2 * ffn, dim)
        W_down = wc.Fp8Matrix(plane[at[1]:at[1] + n[1]], down_scales.cuda(), dim, ffn)
        xd, rd, wd = x.cuda(), r.cuda(), weight.cuda()
        codes, scales = torch.empty(tokens, dim, dtype=F8, device="cuda"), torch.empty(tokens, blocks(dim), device="cuda")
        mid, mids = torch.empty(tokens, ffn, dtype=F8, device="cuda"), torch.empty(tokens, blocks(ffn), device="cuda")
        both, y = torch.empty(tokens, 2 * ffn, dtype=BF16, device="cuda"), torch.empty_like(xd)
        last = torch.empty_like(xd)
        need = max(wc.gemm_fp8_work_bytes(W_up, tokens), wc.gemm_fp8_work_bytes(W_down, tokens))
        work = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
        wc.rms_norm_async(xd, wd, tokens, dim, EPS, codes_dev=codes, scales_dev=scales, residual_dev=rd, sum_dev=rd)
        wc.gemm_fp8_async(W_up, codes, scales, tokens, both, work, work.numel())
        wc.quant_fp8_async(both, tokens, ffn, mid, mids, gated=True)
        wc.gemm_fp8_async(W_down, mid, mids, tokens, y, work, work.numel())
        first = rd.clone()
        wc.rms_norm_async(y, wd, tokens, dim, EPS, y_dev=last, residual_dev=rd, sum_dev=rd)
        torch.cuda.synchronize()
    ref = Norm64(x, weight, EPS, r)
    assert torch.equal(first.cpu(), ref.h)
    check_codes(codes, scales, ref.y, ref.yerr)
    a = values_of(codes) * per_column(scales, dim)
    want = a @ up.t()
    assert within(both, want, gemm_tolerance(a, up, True, want))
    gate, lift = both.cpu().double().split(ffn, dim=1)
    act = gate * torch.sigmoid(gate) * lift
    check_codes(mid, mids, act, (3 * gate.abs() + 12) * 2.0 ** -24 * act.abs() + 1e-37 * lift.abs())
    b = values_of(mid) * per_column(mids, ffn)
    want = b @ down.t()
    assert within(y, want, gemm_tolerance(b, down, True, want))
    ref = Norm64(y, weight, EPS, first)
    assert torch.equal(rd.cpu(), ref.h)
    assert within(last, ref.y, ref.yerr + UBF16 * (ref.y.abs() + ref.yerr))


@pytest.mark.parametrize("vocab,dim,tokens", [(600, 64, 11), (1003, 136, 40), (2000, 256, 130)])
def test_training_step(wc, vocab, dim, tokens):
    """Embedding, two norms in a row with a residual, the loss, all gradients, and their clipping."""
    g = torch.Generator().manual_seed(vocab)
    table = (torch.randn(vocab, dim, generator=g)).to(BF16).cuda()
    head = (torch.randn(vocab, dim, generator=g) * 0.1).to(BF16).cuda()
    w1 = (torch.randn(dim, generator=g) * 0.2 + 1).to(BF16).cuda()
    w2 = (torch.randn(dim, generator=g) * 0.2 + 1).to(BF16).cuda()
    ids = torch.randint(0, vocab, (tokens,), generator=g).cuda()
    targets = torch.roll(ids, -1)
    log(f"case: training step {vocab}x{dim}, {tokens} tokens")

    def new():
        return torch.empty(tokens, dim, dtype=BF16, device="cuda")

    rows, y1, h2, y2, dy2, dh2, drows = (new() for _ in range(7))
    r1, r2, loss, lse = (torch.empty(tokens, device="cuda") for _ in range(4))
    dw1, dw2 = torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")
    dhead, dtable = torch.empty_like(head), torch.empty(vocab, dim, device="cuda")
    dloss = torch.full((tokens,), 1.0 / tokens, device="cuda")
    work = torch.empty(max(wc.ce_work_bytes(tokens, vocab, dim), wc.embed_grad_work_bytes(tokens, dim),
                           wc.rms_norm_grad_work_bytes(tokens, dim)), dtype=torch.uint8, device="cuda")
    size = work.numel()
    wc.embed_async(table, vocab, dim, ids, tokens, rows)
    wc.rms_norm_async(rows, w1, tokens, dim, EPS, y_dev=y1, rstd_dev=r1)
    wc.rms_norm_async(y1, w2, tokens, dim, EPS, y_dev=y2, residual_dev=rows, sum_dev=h2, rstd_dev=r2)
    wc.ce_loss_async(y2, head, targets, tokens, vocab, dim, loss, lse, work, size)
    wc.ce_grad_async(y2, head, targets, tokens, vocab, dim, lse, dloss, dy2, dhead, work, size)
    wc.rms_norm_grad_async(dy2, h2, w2, r2, tokens, dim, dh2, dw2, work, size)
    # h2 = rows + y1: its gradient goes to y1 and to rows
    wc.rms_norm_grad_async(dh2, rows, w1, r1, tokens, dim, drows, dw1, work, size, dsum_dev=dh2)
    wc.embed_grad_async(drows, ids, tokens, dtable, vocab, dim, work, size)
    grads = [dtable, dhead, dw1, dw2]
    outs = [torch.empty_like(t) for t in grads]
    handle = wc.GradList(grads, outs)
    norm, clip_work = torch.empty(1, device="cuda"), torch.empty(wc.clip_grads_work_bytes(handle), dtype=torch.uint8,
                                                                 device="cuda")
    wc.clip_grads_async(handle, 0.01, norm, clip_work, clip_work.numel())
    torch.cuda.synchronize()

    assert torch.equal(rows, table[ids])
    one = Norm64(rows, w1, EPS)
    assert within(y1, one.y, one.yerr + UBF16 * (one.y.abs() + one.yerr))
    two = Norm64(y1, w2, EPS, rows)
    assert torch.equal(h2.cpu(), two.h) and within(y2, two.y, two.yerr + UBF16 * (two.y.abs() + two.yerr))
    ce = CrossEntropy64(y2, head.cpu(), targets.cpu(), dloss)
    assert close(loss, ce.loss, ce.loss_tol) and close(dy2, ce.dh, ce.dh_tol) and close(dhead, ce.dW, ce.dW_tol)
    dh, tol, dw, dw_tol = two.grad(dy2)
    assert within(dh2, dh, tol) and within(dw2, dw, dw_tol)
    dh, tol, dw, dw_tol = one.grad(dh2, dh2)
    assert within(drows, dh, tol) and within(dw1, dw, dw_tol)
    want, mag, most = embed_grad_ref(drows, ids, vocab, 1.0)
    assert within(dtable, want, (most + 3) * 2.0 ** -24 * mag + 1e-40)
    total = sum(float(t.double().square().sum()) for t in grads) ** 0.5
    assert abs(float(norm) - total) <= 2.0 ** -23 * total and total > 0.01
    for t, out in zip(grads, outs):
        exact = t.cpu().double() * (0.01 / total)
        assert within(out, exact, exact.abs() * (2.0 ** -22 + (UBF16 if t.dtype == BF16 else 0.0)) + 1e-40)
    assert BLOCK == wc.FP8_BLOCK

"""The operators on decoded tensors together, as a program uses them: a container's vocabulary matrix is decoded, its
rows are looked up, a 4-bit layer from a decoded code plane is applied token by token, the loss is taken against the
same matrix, and the gradients of the tied matrix are added up."""
import numpy as np
import pytest
import torch

from gpu_util import log, to_device_aligned
from operator_ref import CrossEntropy64, embed_grad_ref, q4_tolerance, within

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


@pytest.mark.parametrize("vocab,dim,tokens", [(600, 64, 11), (1003, 136, 40), (2000, 256, 130)])
def test_step(wc, vocab, dim, tokens):
    g = torch.Generator().manual_seed(vocab)
    table = (torch.randn(vocab, dim, generator=g) * 0.1).to(BF16)
    plane = torch.randint(0, 256, (dim, dim // 2), generator=g, dtype=torch.uint8)
    scales = (torch.rand(dim, -(-dim // 32), generator=g) * 0.05).to(BF16)
    ids = torch.randint(0, vocab, (tokens,), generator=g)
    ids[tokens // 2] = -1                                            # a padded place
    targets = torch.roll(ids, -1)
    log(f"case: decode, look up, 4-bit layer, loss and gradients: {vocab}x{dim}, {tokens} tokens")

    blob, codes_blob = wc.encode_host([table]), wc.encode_u8_host([plane])
    with wc.Plan(blob) as plan, wc.Plan(codes_blob) as codes_plan:
        _, dblob = to_device_aligned(blob)
        _, dcodes = to_device_aligned(codes_blob)
        W = torch.empty(vocab, dim, dtype=BF16, device="cuda")
        codes = torch.empty(dim, dim // 2, dtype=torch.uint8, device="cuda")
        wc.decode_async(plan, dblob, W)
        wc.decode_u8_async(codes_plan, dcodes, codes)
        matrix = wc.Q4Matrix(codes, scales.cuda(), dim, dim, 32)
        ids_d, targets_d = ids.cuda(), targets.cuda()
        rows = torch.empty(tokens, dim, dtype=BF16, device="cuda")
        wc.embed_async(W, vocab, dim, ids_d, tokens, rows, scale=8.0)
        y = torch.empty(tokens, dim, device="cuda")
        for t0 in range(0, tokens, wc.GEMV_Q4_MAX_VECS):
            n = min(wc.GEMV_Q4_MAX_VECS, tokens - t0)
            wc.gemv_q4_async(matrix, rows[t0:t0 + n], n, y[t0:t0 + n])
        h = y.to(BF16)
        loss, lse = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
        dloss = torch.full((tokens,), 1.0 / tokens, device="cuda")
        dh, dW = torch.empty_like(h), torch.empty_like(W)
        work = torch.empty(max(wc.ce_work_bytes(tokens, vocab, dim), wc.embed_grad_work_bytes(tokens, dim)),
                           dtype=torch.uint8, device="cuda")
        wc.ce_loss_async(h, W, targets_d, tokens, vocab, dim, loss, lse, work, work.numel())
        wc.ce_grad_async(h, W, targets_d, tokens, vocab, dim, lse, dloss, dh, dW, work, work.numel())
        head = dW.clone()
        # the layer's own gradient is not the library's: rows' gradient stands in as dh
        wc.embed_grad_async(dh, ids_d, tokens, dW, vocab, dim, work, work.numel(), out="bf16", scale=8.0,
                            accumulate=True)
        torch.cuda.synchronize()

    assert torch.equal(W.cpu().view(torch.int16), table.view(torch.int16))
    assert np.array_equal(codes.cpu().numpy(), plane.numpy())
    ok = ids >= 0
    want = torch.where(ok[:, None], table[torch.where(ok, ids, 0)].float() * 8.0, 0.0).to(BF16)
    assert torch.equal(rows.cpu(), want)                              # a power of two: exact
    q = torch.stack((plane & 15, plane >> 4), dim=2).reshape(dim, dim).double() - 8
    w = q * scales.double().repeat_interleave(32, dim=1)[:, :dim]
    assert within(y, want.double() @ w.t(), q4_tolerance(w, want.double()))
    ref = CrossEntropy64(h, table, targets, dloss)
    assert within(loss, ref.loss, ref.loss_tol) and within(lse, ref.lse, ref.lse_tol)
    assert within(dh, ref.dh, ref.dh_tol) and within(head, ref.dW, ref.dW_tol)
    more, mag, most = embed_grad_ref(dh, ids, vocab, 8.0)
    total = head.cpu().double() + more
    tol = (most + 3) * 2.0 ** -24 * (mag + head.cpu().double().abs()) * 1.01 + 2.0 ** -8 * 1.01 * total.abs()
    assert within(dW, total, tol)

"""Matrices of e4m3 values whose products, in every group of eight, are two of 2^16 that cancel and six of 1 or -1: all sums
are whole numbers below 2^24 in any order, so fp32 sums are exact, and sums that drop what is far below the largest of
eight are not."""
import torch


def codes_of(values):
    """Values that e4m3 holds, as bytes."""
    codes = values.to(torch.float8_e4m3fn)
    assert torch.equal(codes.double(), values.double())
    return codes.view(torch.uint8)


def cancelling(rows, cols, tokens):
    """(w, x, x w^T): in every group of eight columns 256, -256 and signs by 256, 256 and ones."""
    assert cols % 8 == 0 and 2 * 65536 + cols < 1 << 24
    g = torch.Generator().manual_seed(rows + cols + tokens)
    w = torch.randint(0, 2, (rows, cols), generator=g).float() * 2 - 1
    x = torch.ones(tokens, cols)
    w[:, 0::8], w[:, 1::8], x[:, 0::8], x[:, 1::8] = 256.0, -256.0, 256.0, 256.0
    one = (torch.arange(cols) % 8 >= 2).double()
    return w, x, (w.double() @ one)[None].expand(tokens, rows).contiguous()


def dropping(w, x):
    """x w^T as 8-bit matrix instructions sum it: of each eight products, the bits below 2^-14 of the largest's power of two
    are dropped."""
    total = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64)
    for k in range(0, w.shape[1], 8):
        p = x[:, None, k:k + 8].double() * w[None, :, k:k + 8].double()
        step = torch.exp2(torch.floor(torch.log2(p.abs().amax(dim=2, keepdim=True))) - 14)
        total += (torch.trunc(p / step) * step).sum(dim=2)
    return total

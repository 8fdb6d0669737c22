"""What tests/cancelling.py gives tells sums that keep every product from those of 8-bit matrix instructions."""
import torch

from cancelling import cancelling, codes_of, dropping


def test_dropped_products_are_seen():
    """The sums that the GPU tests call exact are not those that 8-bit matrix instructions give, in either type."""
    w, x, want = cancelling(60, 400, 3)
    codes_of(w), codes_of(x)
    assert torch.equal(x.double() @ w.double().t(), want) and float(want.abs().max()) >= 16
    got = dropping(w, x)
    wrong = got != want
    assert bool(wrong[want != 0].all()) and bool((got.to(torch.bfloat16) != want.to(torch.bfloat16))[want != 0].all())

"""Sizes of workspaces that C's 64-bit type would take for other ones are refused before any call, on the CPU."""
import pytest

from test_operator_checks import DevTensor, _status, device0, wc  # noqa: F401  (fixtures)


@pytest.mark.parametrize("size", [-1, -4096, 1 << 64, (1 << 64) + 4096])
def test_sizes_that_would_wrap_round(device0, size):  # noqa: F811
    """-1 would reach C as 2^64 - 1, larger than any workspace that the call needs, and the kernels would write past it."""
    wc = device0  # noqa: F811
    t = DevTensor(1 << 70)          # holds any number of bytes, so that no other check refuses the call
    calls = {
        "embed_grad": lambda b: wc.embed_grad_async(t, t, 5, t, 10, 64, t, b, stream=0),
        "ce_loss": lambda b: wc.ce_loss_async(t, t, t, 5, 10, 64, t, t, t, b, stream=0),
        "ce_grad": lambda b: wc.ce_grad_async(t, t, t, 5, 10, 64, t, t, t, t, t, b, stream=0),
    }
    for what, call in calls.items():
        assert _status(lambda: call(4096)) == "reached C", what
        assert _status(lambda: call(size)) == wc.WC_ERR_INVALID_ARG, what

"""Outputs of the norm that would overwrite each other are refused by the binding, on the CPU."""
import pytest

from test_layer_checks import device0, wc  # noqa: F401  (fixtures)
from test_operator_checks import DevTensor, _status


@pytest.mark.parametrize("codes", [False, True])
def test_sum_and_y_in_one_tensor(device0, codes):  # noqa: F811
    wc = device0   # noqa: F811
    wide = 2 * 3 * 136
    x, r, w, other = DevTensor(wide), DevTensor(wide), DevTensor(272), DevTensor(wide)
    more = dict(codes_dev=DevTensor(3 * 136), scales_dev=DevTensor(24)) if codes else {}

    def call(y, total):
        return _status(lambda: wc.rms_norm_async(x, w, 3, 136, 1e-5, y_dev=y, residual_dev=r, sum_dev=total, stream=0, **more))

    for t in (x, r, other):
        assert call(t, t) == wc.WC_ERR_INVALID_ARG
    for y, total in ((x, r), (x, other), (other, x), (other, r)):
        assert call(y, total) == "reached C"

"""8-bit rows over the whole range of bfloat16, against exact arithmetic.

mla_quantize_i8 promises the codes of exact arithmetic for every finite row.
"""

import numpy as np
import pytest
import torch

from tests.test_gpu_layer import F32, M, _codes64  # noqa: F401

pytestmark = pytest.mark.gpu

SMALLEST = 2.0 ** -149     # float32's smallest step


def _pairs(top):
    """Rows whose maximum is every mantissa at exponent `top`, and every mantissa up to eight exponents below it."""
    m = torch.arange(128, 256).double()
    rows = []
    for gap in range(0, 9):
        r = torch.zeros(128, 144, dtype=torch.float64)
        r[:, 0] = m * 2.0 ** (top - 7)
        r[:, 1:129] = (m * 2.0 ** (top - 7 - gap))[None, :].minimum(r[:, :1])
        r[:, 1:129:3] *= -1
        rows.append(r)
    return torch.cat(rows).float().bfloat16()


@pytest.mark.parametrize("top", [127, 126, 125, 124, 123, 122, 121, 120, 119, 100, 64, -64, -100, -118, -119, -120, -121, -122,
                                 -124, -126, -128, -130, -132])
def test_quantize_every_mantissa_pair_over_the_exponents(M, top):  # noqa: F811
    x = _pairs(top)
    assert torch.isfinite(x.float()).all()
    x8 = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    s = torch.empty(x.shape[0], device="cuda")
    M.mla_quantize_i8(x.cuda(), x.shape[1], x.shape[0], x.shape[1], x8, s)
    want, scale = _codes64(x)
    np.testing.assert_array_equal(x8.cpu().numpy(), want)
    assert np.all(np.abs(s.double().cpu().numpy() - scale) <= F32 * scale + SMALLEST / 2)

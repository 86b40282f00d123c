"""8-bit rows over the whole range of bfloat16, against exact arithmetic.

mla_quantize_i8 promises the codes of exact arithmetic for every finite row;
mla_block_norm's int8 output follows the same rule on float32 values.
"""

import numpy as np
import pytest
import torch

from tests.test_gpu_layer import BF, EPS, F32, M, _codes64  # noqa: F401

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


@pytest.mark.parametrize("d", [16, 512, 2064, 8208])     # a warp per row, a block per row with two and four vectors a thread
@pytest.mark.parametrize("both", [False, True])
def test_block_norm_int8_over_the_exponents(M, d, both):  # noqa: F811
    """Rows from the smallest bfloat16 numbers up, zeros among them: codes round(127 r w / max), whatever max is."""
    tops = list(range(-132, -110)) + [-100, -99, -64, -20, 0, 20, 40]
    g = torch.Generator()
    g.manual_seed(d)
    v = torch.randint(-127, 128, (len(tops), d), generator=g).double()
    v[:, 3] = 127
    v[:, 1::7] = 0
    u = (v * 2.0 ** (torch.tensor(tops).double()[:, None] - 6)).float().bfloat16().cuda()
    u[0, :] = 0
    u[0, 5] = 2.0 ** -133
    n = len(tops)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    out8 = torch.full((n, d), 99, dtype=torch.int8, device="cuda")
    s = torch.empty(n, device="cuda")
    out = torch.empty(n, d, dtype=torch.bfloat16, device="cuda") if both else None
    M.mla_block_norm(u, d, None, None, 0, 1.0, None, None, w, EPS, n, d, out, out8, s)
    r = u.double()
    top = r.abs().amax(1, keepdim=True)
    q = 127.0 * r / top
    # the factor 127 / max and its product with r round to float32 (2^-24 each), then to the nearest integer
    assert ((out8.double() - q).abs() <= 0.5 + 127 * 4 * F32).all()
    assert (out8.abs().amax(1) == 127).all()
    rstd = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    # max * rstd / 127: the mean's tree and a handful of roundings, and float32's smallest step at the bottom
    want = top * rstd / 127
    assert ((s.double()[:, None] - want).abs() <= 64 * F32 * want + SMALLEST).all()
    if both:
        y = r * rstd
        # one rounding to bf16 (its smallest step is 2^-133)
        assert ((out.double() - y).abs() <= (BF + 64 * F32) * y.abs() + 2.0 ** -133).all()

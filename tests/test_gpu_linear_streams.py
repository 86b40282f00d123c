"""Int8 products on two streams at once, at shapes whose blocks share SMs."""

import pytest
import torch

from tests.test_gpu_layer import M, _check_linear, _gen, _i8  # noqa: F401

pytestmark = pytest.mark.gpu

PAIRS = [((129, 2048, 2176), (144, 2048, 2176)), ((140, 1024, 2304), (65, 512, 4096)), ((257, 1024, 2304), (1, 5120, 2112)),
         ((129, 2048, 2176), (2048, 512, 6144))]


@pytest.mark.parametrize("pair", PAIRS)
def test_two_products_at_once(M, pair):  # noqa: F811
    jobs = []
    for n, d_in, d_out in pair:
        g = _gen(n + d_in + d_out)
        x8, w8 = _i8(g, n, d_in), _i8(g, d_out, d_in)
        sx = torch.rand(n, generator=g, device="cuda") + 0.01
        sw = torch.rand(d_out, generator=g, device="cuda") * 1e-3 + 1e-5
        out = torch.empty(n, d_out, dtype=torch.bfloat16, device="cuda")
        jobs.append((torch.cuda.Stream(), x8, sx, w8, sw, out, torch.zeros(1, dtype=torch.int32, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(50):
        for stream, x8, sx, w8, sw, out, status in jobs:
            M.mla_linear_i8(x8, x8.shape[1], sx, w8, sw, out, *x8.shape, w8.shape[0], status, stream)
    torch.cuda.synchronize()
    for _, x8, sx, w8, sw, out, status in jobs:
        assert M.mla_read_status(status) == 0
        _check_linear(out, x8, sx, w8, sw)

"""The int8 product's bounded waits, exercised without a GPU fault.

mla_test_arm_linear_timeout makes the next product withhold one load (a
barrier that nothing completes) and bounds its waits by a few milliseconds.
The call has to return, report MLA_STATUS_TIMEOUT, write nothing behind its
output and leave the context usable: the same call right after it is exact.
"""

import pytest
import torch

from tests.test_gpu_layer import M, _check_linear, _gen, _i8, _linear  # noqa: F401

pytestmark = pytest.mark.gpu

# split kernel: one CTA, clusters of several, several token tiles; wide kernel: one round, several
SIZES = [(1, 16, 8), (32, 2048, 264), (1, 5120, 2112), (129, 1552, 392), (300, 272, 7696), (2048, 1536, 6144)]


@pytest.mark.parametrize("n,d_in,d_out", SIZES)
def test_withheld_load_times_out_and_the_next_call_is_exact(M, n, d_in, d_out):  # noqa: F811
    g = _gen(n + d_in + d_out)
    x8, w8 = _i8(g, n, d_in), _i8(g, d_out, d_in)
    sx = torch.rand(n, generator=g, device="cuda") + 0.01
    sw = torch.rand(d_out, generator=g, device="cuda") * 1e-3 + 1e-5
    out = torch.full((n + 1, d_out), 5.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    M.mla_test_arm_linear_timeout(5_000_000)    # 5 ms per wait
    M.mla_linear_i8(x8, d_in, sx, w8, sw, out, n, d_in, d_out, status)
    torch.cuda.synchronize()                    # the call returned: nothing hangs
    assert M.mla_read_status(status) == M.MLA_STATUS_TIMEOUT
    assert (out[n] == 5.0).all()
    for _ in range(2):
        _check_linear(_linear(M, x8, sx, w8, sw), x8, sx, w8, sw)


def test_sizes_reach_both_kernels(M):  # noqa: F811
    kinds = {M.mla_linear_i8_shape(*s)[1] == 512 for s in SIZES}
    assert kinds == {False, True}


def test_arm_rejects_out_of_range_limits(M):  # noqa: F811
    for bad in (0, 3_000_000_000):
        with pytest.raises(M.MlaError) as e:
            M.mla_test_arm_linear_timeout(bad)
        assert e.value.code == -3

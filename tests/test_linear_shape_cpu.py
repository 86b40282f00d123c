"""Tensor memory of the int8 product's kernels, from the host's launch shapes.

A CTA that asks for tensor memory waits, without a bound, until its SM has
that many columns free, and the CTAs of a cluster wait for each other.  So the
blocks that fit one SM by their shared memory must fit its 512 columns too, in
any mix of launches: then an SM never holds a CTA that waits for another.
"""

import ctypes
import random

import pytest

from mla_latent_kv_38_b200 import build

SM_SMEM, BLOCK_RESERVED, COLUMNS, MOST = 228 * 1024, 1024, 512, 227 * 1024


@pytest.fixture(scope="module")
def M():
    build.build()
    from mla_latent_kv_38_b200 import binding
    return binding


def _sizes():
    rng = random.Random(5)
    for n in list(range(1, 300)) + [511, 512, 513, 897, 1025, 4096, 65536]:
        for d_in in (16, 128, 144, 256, 272, 512, 1024, 1040, 2048, 4096, 16384, 65536):
            for d_out in (8, 128, 136, 2112, 2176, 2304, 5120, 24576):
                yield n, d_in, d_out
    for _ in range(20000):
        yield rng.randint(1, 2000), 16 * rng.randint(1, 600), 8 * rng.randint(1, 2000)


def test_blocks_that_share_an_sm_share_its_tensor_memory(M):
    seen = set()
    for sizes in _sizes():
        cluster, cols, smem = M.mla_linear_i8_shape(*sizes)
        assert 1 <= cluster <= 8 and cols in (32, 64, 128, 256, 512) and 0 < smem <= MOST, sizes
        # a block's share of the SM's columns is at most its share of the shared memory
        assert cols * SM_SMEM <= COLUMNS * (smem + BLOCK_RESERVED), (sizes, cols, smem)
        seen.add((cluster, cols))
    assert {c for _, c in seen} == {32, 64, 128, 256, 512} and {k for k, _ in seen} == {1, 2, 4, 8}


def test_shape_refusals(M):
    p = [ctypes.c_int(0), ctypes.c_int(0), ctypes.c_size_t(0)]
    call = lambda n, i, o, *q: M.raw_call("mla_linear_i8_shape", n, i, o, *q)  # noqa: E731
    refs = [ctypes.byref(x) for x in p]
    for k in range(3):
        assert call(4, 512, 128, *[None if j == k else r for j, r in enumerate(refs)]) == -1
    for bad in ((0, 512, 128), (65537, 512, 128), (4, 8, 128), (4, 520, 128), (4, 65552, 128), (4, 512, 12), (4, 512, 131080)):
        assert call(*bad, *refs) == -3, bad

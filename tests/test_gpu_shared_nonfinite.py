"""Infinities and NaN among the keys that a row of mla_decode_shared sees.

A score that is NaN or +inf leaves neither a weight nor a log-sum-exp: the
row's latent and lse are NaN, whichever key range they were computed in.
mla_decode on the same cache gives the same.
"""

import math

import pytest
import torch

from tests.test_gpu_shared import M, V2, Case  # noqa: F401

pytestmark = pytest.mark.gpu

COL = 9      # the latent column that takes the value


def _put(c, b, j, value):
    """Key j of sequence b (j < 64 n_shared: a shared key, of every sequence)."""
    page = int(c.shared[j // 64]) if j < 64 * c.n_shared else int(c.table[b, j // 64])
    c.pool[page, j % 64, COL] = value


def _rows(c):
    n = c.B * c.T_q
    return c.latent[:n].view(c.B, c.T_q, c.n_h, -1), c.lse[:n].view(c.B, c.T_q, c.n_h)


def _run(c):
    c.run()
    torch.cuda.synchronize()
    assert c.status() == 0
    return _rows(c)


SEEN = [   # n_h, T_q, n_shared, own keys: with and without units of the shared pages, in one and in many parts
    (16, 1, 40, [70, 900, 500] * 4),
    (128, 1, 24, [70, 700, 300]),
    (128, 2, 5, [2, 130]),
    (16, 4, 4, [4, 67, 300]),
    (16, 3, 0, [300, 3]),
    (1, 1, 1, [1, 1]),
]


@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("impl", [0, 1])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("shape", SEEN)
def test_a_seen_score_without_a_weight_makes_the_row_nan(M, shape, value, impl, splits):  # noqa: F811
    n_h, T_q, n_shared, own = shape
    make = lambda: Case(M, n_h, *V2, T_q, n_shared, own, impl, splits)  # noqa: E731
    clean = make()
    clean.q_abs[:, :, COL] = 1.0      # +inf keys score +inf
    lat0, lse0 = (x.clone() for x in _run(clean))
    if n_shared:
        c = make()
        c.q_abs[:, :, COL] = 1.0
        _put(c, 0, 64 * (n_shared - 1) + 5, value)
        lat, lse = _run(c)
        assert torch.isnan(lat).all() and torch.isnan(lse).all()
    c = make()
    c.q_abs[:, :, COL] = 1.0
    b = 1
    _put(c, b, 64 * n_shared, value)
    lat, lse = _run(c)
    assert torch.isnan(lat[b]).all() and torch.isnan(lse[b]).all()
    for o in range(len(own)):
        if o != b:
            assert torch.equal(lat[o], lat0[o]) and torch.equal(lse[o], lse0[o])


def test_mla_decode_agrees_on_nan_rows(M):  # noqa: F811
    for splits in (0, 1, 3):
        c = Case(M, 128, *V2, 2, 6, [2, 77, 1500, 513], 0, splits)
        _put(c, 2, 64 * 6 + 1000, math.nan)
        lat, lse = _run(c)
        full = c.table.clone()
        full[:, :6] = c.shared
        ws = torch.zeros(M.mla_decode_workspace_bytes(c.cfg, c.B, 2, splits), dtype=torch.uint8, device="cuda")
        lat1, lse1 = torch.empty_like(c.latent), torch.empty_like(c.lse)
        M.mla_decode(c.cfg, c.q_abs, c.q_r, c.pool, c.blocks, full, c.mb, c.lens, c.B, 2, splits, ws, ws.numel(), lat1, lse1)
        torch.cuda.synchronize()
        n = c.B * 2
        assert torch.equal(torch.isnan(lat1[:n]).view_as(lat), torch.isnan(lat))
        assert torch.equal(torch.isnan(lse1[:n]).view_as(lse), torch.isnan(lse))
        assert torch.isnan(lat[2]).all() and torch.isnan(lse[2]).all() and torch.isfinite(lat[:2].float()).all()

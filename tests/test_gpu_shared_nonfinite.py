"""Infinities and NaN among the keys that a row of mla_decode_shared sees.

A score that is NaN or +inf leaves neither a weight nor a log-sum-exp: the
row's latent and lse are NaN, whichever key range they were computed in.  A
score of -inf is a weight of zero; times the infinity in the key's latent that
made it, it is NaN in that column (0 inf), and the other columns and the lse
are those of the keys without it.  mla_decode on the same cache gives the same.
Bounds of finite values as in test_gpu_shared.py.
"""

import math

import pytest
import torch

from tests.test_gpu_shared import BF, M, SCORE, V2, Case  # noqa: F401

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


MINUS = [  # n_h, T_q, n_shared, own keys, the key's place before the sequence's end
    (16, 4, 3, [4, 66, 131, 259], 2), (1, 70, 3, [70, 130, 200], 35), (128, 3, 3, [3, 66, 257], 1), (40, 3, 3, [64], 2),
    (16, 4, 20, [70, 66, 131, 259], 66), (24, 9, 6, [9, 70, 64], 9), (16, 2, 0, [65, 200], 1), (16, 1, 9, [65, 200] * 6, 30)]


@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("impl", [0, 1])
@pytest.mark.parametrize("n_h,T_q,n_shared,own,back", MINUS)
def test_a_score_of_minus_infinity(M, impl, n_h, T_q, n_shared, own, back, splits):  # noqa: F811
    """An infinity in one latent column of one key, against a negative query: NaN in that column of the rows that see
    the key, whatever else shares their unit of work; the rest as if the key were not there."""
    make = lambda: Case(M, n_h, *V2, T_q, n_shared, own, impl, splits)  # noqa: E731
    clean = make()
    clean.q_abs[:, :, COL] = -0.5
    lat0, lse0 = (x.clone() for x in _run(clean))
    c = make()
    c.q_abs[:, :, COL] = -0.5
    at = [64 * n_shared + k - back for k in own]
    for b in range(len(own)):
        _put(c, b, at[b], math.inf)
    lat, lse = _run(c)
    prefix = c.pool[c.shared.long()].reshape(-1, 576)
    scale = 1.0 / math.sqrt(192)
    for b, k in enumerate(own):
        ids = c.table[b, n_shared:(64 * n_shared + k + 63) // 64].long()
        keys = torch.cat([prefix, c.pool[ids].reshape(-1, 576)[:k]]).double()
        for t in range(T_q):
            last = 64 * n_shared + k - T_q + t
            # keys at infinity that this row sees: its sequence's own, and those of the others put among shared keys
            hit = ~torch.isfinite(keys[:last + 1, COL])
            if not hit.any():
                assert torch.equal(lat[b, t], lat0[b, t]) and torch.equal(lse[b, t], lse0[b, t]), (b, t)
                continue
            assert torch.isnan(lat[b, t, :, COL]).all(), (b, t)
            see = keys[:last + 1][~hit]
            n = b * T_q + t
            s = torch.cat([c.q_abs[n], c.q_r[n]], 1).double() @ see.T * scale
            want = torch.logsumexp(s, 1)
            p = torch.exp(s - want[:, None])
            o, mag = p @ see[:, :512], p @ see[:, :512].abs()
            rest = torch.arange(512, device="cuda") != COL
            err = (lat[b, t].double() - o).abs()
            assert (err <= (BF + SCORE) * mag + BF * o.abs())[:, rest].all(), (b, t)
            assert ((lse[b, t].double() - want).abs() <= SCORE).all(), (b, t)

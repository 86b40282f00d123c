"""mla_decode_shared with a prompt chunk behind the shared pages: hundreds of
tokens a sequence, up to unit counts past the decode's own schedule."""

import pytest
import torch

from tests.test_gpu_shared import BF, M, SCORE, V2, Case  # noqa: F401

pytestmark = pytest.mark.gpu

CHUNKS = [   # n_h, T_q, n_shared, own keys, impl
    (128, 300, 5, [300, 437], 0),
    (128, 129, 33, [129, 130, 400], 0),
    (256, 520, 3, [520, 583], 0),          # 2,080 units
    (16, 500, 9, [500, 565, 700], 0),      # units of eight whole tokens
    (40, 257, 2, [257, 321], 0),
    (8, 333, 60, [333, 334, 500], 0),
    (12, 150, 4, [150, 200], 1),
]


@pytest.mark.parametrize("case", CHUNKS)
def test_a_chunk_behind_shared_pages(M, case):  # noqa: F811
    n_h, T_q, n_shared, own, impl = case
    c = Case(M, n_h, *V2, T_q, n_shared, own, impl)
    c.run()
    torch.cuda.synchronize()
    assert c.status() == 0
    c.check()


def test_a_chunk_in_a_padded_batch(M):  # noqa: F811
    """A sequence without room for the chunk is flagged and zeroed; the others are as without it."""
    c = Case(M, 128, *V2, 200, 4, [200, 0, 263], 0)
    c.lens[1] = 64 * 4 + 199
    c.run()
    torch.cuda.synchronize()
    assert c.status() == M.MLA_STATUS_BAD_SEQ_LEN
    c.check()


@pytest.mark.parametrize("n_h,T_q", [(128, 200), (256, 64)])
def test_a_chunk_matches_mla_decode(M, n_h, T_q):  # noqa: F811
    c = Case(M, n_h, *V2, T_q, 6, [T_q, T_q + 77, T_q + 513], 0)
    c.run()
    full = c.table.clone()
    full[:, :6] = c.shared
    ws = torch.zeros(M.mla_decode_workspace_bytes(c.cfg, c.B, T_q, 0), dtype=torch.uint8, device="cuda")
    lat, lse = torch.empty_like(c.latent), torch.empty_like(c.lse)
    M.mla_decode(c.cfg, c.q_abs, c.q_r, c.pool, c.blocks, full, c.mb, c.lens, c.B, T_q, 0, ws, ws.numel(), lat, lse)
    torch.cuda.synchronize()
    n = c.B * T_q
    # each side rounds its weights and its result to bf16
    assert ((lat[:n].float() - c.latent[:n].float()).abs() <= 4 * BF * lat[:n].float().abs().clamp(min=0.25)).all()
    assert ((lse[:n] - c.lse[:n]).abs() <= 2 * SCORE).all()


@pytest.mark.parametrize("n_h,B", [(8, 111), (8, 112), (7, 127), (16, 74), (127, 7)])
def test_row_counts_around_the_merges_two_forms(M, n_h, B):  # noqa: F811
    c = Case(M, n_h, *V2, 1, 6, [1 + (37 * b) % 130 for b in range(B)], 0)
    c.run()
    torch.cuda.synchronize()
    assert c.status() == 0
    c.check()


@pytest.mark.parametrize("impl", [0, 1])
@pytest.mark.parametrize("n_h,B", [(16, 12), (128, 2)])
def test_a_table_without_room_behind_the_shared_pages(M, n_h, B, impl):  # noqa: F811
    """n_shared = max_blocks_per_seq: no sequence has a valid length, with and without units of the shared pages."""
    c = Case(M, n_h, *V2, 1, 8, [0] * B, impl, spare=-1)
    assert c.mb == 8
    c.lens.fill_(64 * 8)
    c.run()
    torch.cuda.synchronize()
    assert c.status() == M.MLA_STATUS_BAD_SEQ_LEN
    c.check()

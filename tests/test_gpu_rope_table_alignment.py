"""mla_rope_append with a RoPE table that has a float's alignment and no more."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_38_b200 import build
    build.build()
    from mla_latent_kv_38_b200 import binding
    return binding


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("offset", [1, 2, 3])
def test_append_does_not_depend_on_the_tables_alignment(M, cache, offset):
    n_h, d_c, d_h, d_r, B, T_q, max_pos = 5, 64, 16, 24, 3, 4, 200
    cfg = M.MlaConfig(n_h, d_c, d_h, d_r)
    g = torch.Generator(device="cuda")
    g.manual_seed(offset)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, c = n(B * T_q, n_h, d_r), n(B * T_q, d_r), n(B * T_q, d_c)
    pos = torch.tensor([7, 8, 9, 10, 62, 63, 64, 65, 196, 197, 198, 199], dtype=torch.int32, device="cuda")
    table = torch.randperm(12, generator=g, device="cuda").int().view(B, 4)
    rope = M.mla_rope_table(d_r, 10000.0, max_pos).cuda()
    wide = torch.empty(rope.numel() + 4, device="cuda")
    odd = wide[offset:offset + rope.numel()]
    odd.copy_(rope.view(-1))
    assert rope.data_ptr() % 16 == 0 and odd.data_ptr() % 16 == 4 * offset
    row = d_c + d_r if cache == "bf16" else M.mla_e4m3_row_bytes(d_c, d_r)
    dtype = torch.bfloat16 if cache == "bf16" else torch.uint8
    call = M.mla_rope_append if cache == "bf16" else M.mla_rope_append_e4m3
    got = []
    for tab in (rope, odd):
        q_r, pool = q.clone(), torch.zeros(12, 64, row, dtype=dtype, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(cfg, q_r, k, c, pos, tab, max_pos, table, 4, pool, 12, B, T_q, status)
        torch.cuda.synchronize()
        assert M.mla_read_status(status) == 0
        got.append((q_r, pool))
    assert torch.equal(got[0][0].view(torch.int16), got[1][0].view(torch.int16)) and torch.equal(got[0][1], got[1][1])

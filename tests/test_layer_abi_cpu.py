"""Host-side argument checks of the operators around the decode: every refusal
happens before a device is touched, so these calls are safe without a GPU."""

import ctypes

import pytest

from mla_latent_kv_38_b200 import build

FAKE = 0x10000  # 256-byte aligned non-null value; never dereferenced by these calls
P = ctypes.c_void_p(FAKE)
ODD16 = ctypes.c_void_p(FAKE + 8)
ODD4 = ctypes.c_void_p(FAKE + 2)
NULL, CONFIG, SIZE, WORKSPACE, ALIGN = -1, -2, -3, -4, -7


@pytest.fixture(scope="module")
def M():
    build.build()
    from mla_latent_kv_38_b200 import binding
    return binding


def _cfg(M, **kw):
    base = dict(n_h=128, d_c=512, d_h=128, d_r=64)
    base.update(kw)
    return M.MlaConfig(**base)


def test_decode_shared_refusals(M):
    def call(c=None, q_abs=P, q_r=P, pool=P, num_blocks=2048, shared=P, n_shared=8, bt=P, mbps=64, lens=P, B=32, T_q=1,
             splits=0, ws=P, ws_bytes=1 << 34, out=P, lse=P):
        return M.raw_call("mla_decode_shared", ctypes.byref(c or _cfg(M)), q_abs, q_r, pool, num_blocks, shared, n_shared,
                          bt, mbps, lens, B, T_q, splits, ws, ctypes.c_size_t(ws_bytes), out, lse, None)

    assert call(c=_cfg(M, block_size=32)) == CONFIG
    assert call(c=_cfg(M, d_c=256, impl=2)) == CONFIG                 # tcgen05: 512 + 64 columns only
    for name in ("q_abs", "q_r", "pool", "shared", "bt", "lens", "ws", "out", "lse"):
        assert call(**{name: None}) == NULL, name
    for name in ("q_abs", "q_r", "pool", "out"):
        assert call(**{name: ODD16}) == ALIGN, name
    for name in ("shared", "bt", "lens", "lse"):
        assert call(**{name: ODD4}) == ALIGN, name
    for bad in (dict(B=0), dict(T_q=0), dict(B=65536), dict(num_blocks=0), dict(mbps=0), dict(splits=-1),
                dict(n_shared=-1), dict(n_shared=65), dict(mbps=(1 << 24) + 1)):
        assert call(**bad) == SIZE, bad
    # pages of all units together are counted in 32 bits
    assert call(mbps=1 << 24) == SIZE and call(c=_cfg(M, n_h=129), B=64, mbps=1 << 22) == SIZE
    assert call(ws=ctypes.c_void_p(FAKE + 16)) == WORKSPACE
    need = M.mla_decode_shared_workspace_bytes(_cfg(M), 32, 1, 0)
    assert need > 0 and need % 256 == 0
    assert call(ws_bytes=need - 1) == WORKSPACE
    for bad in ((0, 1, 0), (1, 0, 0), (65536, 1, 0), (32, 1, -1)):
        assert M.mla_decode_shared_workspace_bytes(_cfg(M), *bad) == 0, bad
    assert M.mla_decode_shared_workspace_bytes(_cfg(M, block_size=32), 32, 1, 0) == 0
    assert M.mla_decode_shared_workspace_bytes(_cfg(M, d_c=256, impl=2), 32, 1, 0) == 0


def test_quantize_refusals(M):
    def call(x=P, ld=512, rows=4, d=512, x8=P, scale=P):
        return M.raw_call("mla_quantize_i8", x, ctypes.c_int64(ld), rows, d, x8, scale, None)

    for name in ("x", "x8", "scale"):
        assert call(**{name: None}) == NULL, name
    assert call(x=ODD16) == ALIGN and call(x8=ODD16) == ALIGN and call(scale=ODD4) == ALIGN
    for bad in (dict(rows=0), dict(rows=(1 << 24) + 1), dict(d=0), dict(d=8), dict(d=24, ld=24), dict(d=65552, ld=65552),
                dict(ld=504), dict(ld=516), dict(ld=(1 << 31) + 8)):
        assert call(**bad) == SIZE, bad


def test_linear_refusals(M):
    def call(x8=P, ld=512, sx=P, w8=P, sw=P, out=P, n_tok=4, d_in=512, d_out=128, status=None):
        return M.raw_call("mla_linear_i8", x8, ctypes.c_int64(ld), sx, w8, sw, out, n_tok, d_in, d_out, status, None)

    for name in ("x8", "sx", "w8", "sw", "out"):
        assert call(**{name: None}) == NULL, name
    for name in ("x8", "w8", "out"):
        assert call(**{name: ODD16}) == ALIGN, name
    for name in ("sx", "sw", "status"):
        assert call(**{name: ODD4}) == ALIGN, name
    for bad in (dict(n_tok=0), dict(n_tok=65537), dict(d_in=0), dict(d_in=8), dict(d_in=520, ld=528),
                dict(d_in=65552, ld=65552), dict(d_out=0), dict(d_out=12), dict(d_out=131080), dict(ld=496),
                dict(ld=520), dict(ld=(1 << 31) + 16)):
        assert call(**bad) == SIZE, bad


def test_block_norm_refusals(M):
    f = ctypes.c_float

    def call(u=P, ld_u=512, w_post=P, gate=P, ld_gate=512, alpha=1.0, res=P, res_out=P, w_pre=P, eps=1e-6, n_tok=4,
             d=512, out=P, out8=None, scale=None):
        return M.raw_call("mla_block_norm", u, ctypes.c_int64(ld_u), w_post, gate, ctypes.c_int64(ld_gate), f(alpha), res,
                          res_out, w_pre, f(eps), n_tok, d, out, out8, scale, None)

    assert call(u=None) == NULL
    assert call(res_out=None, out=None, w_pre=None) == NULL          # no output
    assert call(res=None) == NULL                                    # residual_out without residual
    assert call(w_pre=None) == NULL                                  # out without w_pre
    assert call(out=None) == NULL                                    # w_pre without out or out8
    assert call(out8=P) == NULL and call(scale=P) == NULL            # codes and scales only together
    for name in ("u", "w_post", "gate", "res", "res_out", "w_pre", "out"):
        assert call(**{name: ODD16}) == ALIGN, name
    assert call(out8=ODD16, scale=P) == ALIGN and call(out8=P, scale=ODD4) == ALIGN
    for bad in (dict(n_tok=0), dict(n_tok=(1 << 24) + 1), dict(d=0), dict(d=12), dict(d=16392, ld_u=16392, ld_gate=0),
                dict(ld_u=504), dict(ld_u=516), dict(ld_gate=504), dict(ld_gate=516), dict(ld_gate=-512), dict(eps=0.0),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(alpha=float("inf")),
                dict(alpha=float("nan")), dict(ld_u=(1 << 31) + 8),
                dict(d=520, ld_u=520, ld_gate=0, out8=P, scale=P)):  # int8 rows: a multiple of 16
        assert call(**bad) == SIZE, bad


@pytest.mark.parametrize("name", ["mla_norm_rope_append", "mla_norm_rope_append_e4m3"])
def test_norm_rope_append_refusals(M, name):
    f = ctypes.c_float

    def call(c=None, q=P, kv=P, ld_kv=576, w=P, eps=1e-6, pos=P, table=P, max_pos=4096, bt=P, mbps=64, pool=P,
             num_blocks=2048, B=32, T_q=1, q_c=P, q_r=P, status=None):
        return M.raw_call(name, ctypes.byref(c or _cfg(M)), q, kv, ctypes.c_int64(ld_kv), w, f(eps), pos, table, max_pos,
                          bt, mbps, pool, num_blocks, B, T_q, q_c, q_r, status, None)

    assert call(c=_cfg(M, block_size=16)) == CONFIG
    if name.endswith("e4m3"):
        assert call(c=_cfg(M, d_c=96)) == CONFIG
    for k in ("kv", "w", "pos", "table", "bt", "pool", "q", "q_c", "q_r"):   # the three query tensors only together
        assert call(**{k: None}) == NULL, k
    for k in ("q", "kv", "w", "table", "pool", "q_c", "q_r"):
        assert call(**{k: ODD16}) == ALIGN, k
    for k in ("pos", "bt", "status"):
        assert call(**{k: ODD4}) == ALIGN, k
    for bad in (dict(B=0), dict(T_q=0), dict(B=1 << 13, T_q=1 << 12), dict(max_pos=0), dict(mbps=0), dict(num_blocks=0),
                dict(ld_kv=568), dict(ld_kv=580), dict(ld_kv=(1 << 31) + 8), dict(eps=0.0), dict(eps=float("nan"))):
        assert call(**bad) == SIZE, bad

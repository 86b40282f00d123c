"""The operators around the decode against plain implementations in 64 bits.

mla_quantize_i8, mla_linear_i8, mla_block_norm, mla_norm_rope_append (and its
e4m3 form).  Bounds: a bf16 rounding is off by at most 2^-8 of the value, a
float32 operation by 2^-24; sums of d float32 terms in any order by at most
d 2^-24 of the sum of magnitudes, of which the kernels' trees reach far less.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = 2.0 ** -8, 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_38_b200 import build
    build.build()
    from mla_latent_kv_38_b200 import binding
    return binding


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _n(g, *s):
    return torch.randn(*s, generator=g, device="cuda").bfloat16()


def _i8(g, *s):
    return torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)


# ---- quantisation ----------------------------------------------------------

def _codes64(x):
    """Codes and scales in exact arithmetic (numpy rounds halves to even)."""
    v = x.double().cpu().numpy()
    amax = np.abs(v).max(1, keepdims=True)
    q = np.divide(127.0 * v, amax, out=np.zeros_like(v), where=amax > 0)
    return np.rint(q).astype(np.int8), (amax / 127.0)[:, 0]


@pytest.mark.parametrize("rows,d,ld", [(1, 16, 16), (3, 48, 56), (7, 512, 576), (5, 1536, 2112), (33, 5120, 5120),
                                       (2, 16384, 16384), (3, 16400, 16400), (2, 65536, 65536), (4000, 64, 64)])
def test_quantize_codes_are_exact(M, rows, d, ld):
    g = _gen(d + rows)
    buf = _n(g, rows, ld)
    x = buf[:, :d]
    x[0, :] = 0.0                                         # a row of zeros
    if rows > 1:
        x[1, 1::2] = x[1, 0] / 2                          # exact halves of a code step when x[1, 0] is the maximum
        x[1, ::2] = x[1, 0]
    x8 = torch.full((rows + 1, d), 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 1,), 7.0, device="cuda")
    M.mla_quantize_i8(x, ld, rows, d, x8, s)
    want, scale = _codes64(x)
    np.testing.assert_array_equal(x8[:rows].cpu().numpy(), want)
    assert (x8[rows] == 99).all() and s[rows] == 7.0      # rows behind the last one untouched
    got = s[:rows].double().cpu().numpy()
    assert np.all(np.abs(got - scale) <= F32 * scale)


def test_quantize_every_mantissa_pair(M):
    """All pairs of 8-bit mantissas and the exponent gaps of a code step, ties included."""
    m = torch.arange(128, 256, device="cuda").double()
    rows = []
    for gap in range(0, 9):
        r = torch.zeros(128, 144, dtype=torch.float64, device="cuda")
        r[:, 0] = m * 2.0 ** 9                             # the row's maximum
        r[:, 1:129] = (m * 2.0 ** (9 - gap))[None, :].minimum(r[:, :1])
        rows.append(r)
    x = torch.cat(rows).bfloat16()
    x8 = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    s = torch.empty(x.shape[0], device="cuda")
    M.mla_quantize_i8(x, x.shape[1], x.shape[0], x.shape[1], x8, s)
    np.testing.assert_array_equal(x8.cpu().numpy(), _codes64(x)[0])


# ---- the int8 product -------------------------------------------------------

SHAPES = [(1, 16, 8), (1, 5120, 2112), (2, 48, 24), (15, 128, 128), (16, 144, 136), (17, 1536, 200), (32, 2048, 264),
          (33, 272, 1000), (64, 640, 72), (100, 512, 640), (129, 1552, 392), (255, 96, 128), (256, 256, 256),
          (257, 1040, 520), (300, 512, 2112), (513, 208, 1032), (1030, 400, 776), (32, 16384, 5120), (2048, 1536, 1024),
          (7, 65536, 16), (3, 32, 131072)]


def _linear(M, x8, sx, w8, sw, ld=None, out=None):
    n, d_in = x8.shape
    out = torch.full((n + 1, w8.shape[0]), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.mla_linear_i8(x8, ld or d_in, sx, w8, sw, out, n, d_in, w8.shape[0], status)
    torch.cuda.synchronize()
    assert M.mla_read_status(status) == 0
    assert torch.isnan(out[n:].float()).all()              # rows behind the last one untouched
    return out[:n]


def _check_linear(out, x8, sx, w8, sw):
    acc = x8.double() @ w8.double().T                      # exact: below 2^53
    ref = acc * sx.double()[:, None] * sw.double()[None, :]
    err = (out.double() - ref).abs()
    # the sum to float32, two products, one rounding to bf16 (scales keep every product normal)
    assert (err <= ref.abs() * (BF + 4 * F32)).all(), err.max()


@pytest.mark.parametrize("n,d_in,d_out", SHAPES)
def test_linear_matches_the_exact_sum(M, n, d_in, d_out):
    g = _gen(n * 7 + d_in + d_out)
    x8, w8 = _i8(g, n, d_in), _i8(g, d_out, d_in)
    sx = torch.rand(n, generator=g, device="cuda") + 0.01
    sw = torch.rand(d_out, generator=g, device="cuda") * 1e-3 + 1e-5
    _check_linear(_linear(M, x8, sx, w8, sw), x8, sx, w8, sw)


@pytest.mark.parametrize("n", [1, 40, 300])
def test_linear_strided_rows_and_extreme_sums(M, n):
    """Rows of a wider matrix; all codes at the ends of the range (-128 included), so sums reach 2^30."""
    g = _gen(n)
    wide = torch.full((n, 65536 + 64), 5, dtype=torch.int8, device="cuda")
    x8 = wide[:, 64:]
    x8[:] = -128
    w8 = torch.full((24, 65536), -128, dtype=torch.int8, device="cuda")
    w8[1] = 127
    w8[2, ::2] = 127
    sx = torch.rand(n, generator=g, device="cuda") + 0.5
    sw = torch.rand(24, generator=g, device="cuda") + 0.5
    _check_linear(_linear(M, x8, sx, w8, sw, ld=65536 + 64), x8, sx, w8, sw)


def test_linear_scales_beyond_float32_products(M):
    """Scales whose own product leaves the float32 range, with sums that bring the result back; and zero scales."""
    x8 = torch.full((4, 64), 127, dtype=torch.int8, device="cuda")
    w8 = torch.full((16, 64), 127, dtype=torch.int8, device="cuda")
    sx = torch.tensor([1e-20, 1e20, 0.0, 1.0], device="cuda")
    sw = torch.full((16,), 1e-16, device="cuda")
    sw[1] = 0.0
    _check_linear(_linear(M, x8, sx, w8, sw), x8, sx, w8, sw)


@pytest.mark.parametrize("n,d_in,d_out", [(129, 144, 15368), (300, 272, 7696), (1030, 144, 3336), (5000, 64, 1032),
                                          (256, 2064, 15360), (2048, 16, 2056), (514, 272, 6328), (1000, 144, 6648),
                                          (514, 1040, 6400), (16384, 64, 8), (1300, 2320, 8000)])
def test_linear_many_tokens(M, n, d_in, d_out):
    """Enough output tiles for the many-token kernel, whole and ragged ones."""
    g = _gen(n + d_in * 3 + d_out)
    x8, w8 = _i8(g, n, d_in), _i8(g, d_out, d_in)
    sx = torch.rand(n, generator=g, device="cuda") + 0.01
    sw = torch.rand(d_out, generator=g, device="cuda") * 1e-3 + 1e-5
    _check_linear(_linear(M, x8, sx, w8, sw), x8, sx, w8, sw)


def test_linear_many_tokens_strided_and_extreme(M):
    n, d_in = 300, 1040
    wide = torch.full((n, d_in + 48), 5, dtype=torch.int8, device="cuda")
    x8 = wide[:, 16:16 + d_in]
    x8[:] = -128
    w8 = torch.full((7696, d_in), -128, dtype=torch.int8, device="cuda")
    w8[1::3] = 127
    sx = torch.rand(n, generator=_gen(1), device="cuda") + 0.5
    sw = torch.rand(7697, generator=_gen(2), device="cuda")[1:] + 0.5     # 4-byte aligned only
    sw = torch.cat([sw[:1], sw])[1:]
    assert sw.data_ptr() % 16 == 4
    _check_linear(_linear(M, x8, sx, w8, sw, ld=d_in + 48), x8, sx, w8, sw)


def test_quantize_smallest_and_largest_rows(M):
    """Rows whose 127 / max overflows float32, and rows at the top of the range."""
    tiny = 2.0 ** -133
    x = torch.zeros(4, 32, dtype=torch.float64, device="cuda")
    x[0, :20] = torch.arange(-10, 10, device="cuda") * tiny
    x[1, 3] = tiny
    x[2, :] = torch.linspace(-1, 1, 32, device="cuda", dtype=torch.float64) * 2.0 ** -126
    x[3, :] = torch.linspace(-1, 1, 32, device="cuda", dtype=torch.float64) * 3e38
    x = x.bfloat16()
    x8 = torch.empty(4, 32, dtype=torch.int8, device="cuda")
    s = torch.empty(4, device="cuda")
    M.mla_quantize_i8(x, 32, 4, 32, x8, s)
    np.testing.assert_array_equal(x8.cpu().numpy(), _codes64(x)[0])


@pytest.mark.parametrize("rows,d", [(700, 16), (3000, 1536), (2500, 2048), (700, 2056 + 8)])
def test_quantize_many_rows(M, rows, d):
    x = _n(_gen(rows + d), rows, d)
    x8 = torch.empty(rows, d, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    M.mla_quantize_i8(x, d, rows, d, x8, s)
    want, scale = _codes64(x)
    np.testing.assert_array_equal(x8.cpu().numpy(), want)
    assert np.all(np.abs(s.double().cpu().numpy() - scale) <= F32 * scale)


# ---- norms and residual -----------------------------------------------------

NORMS = [  # n_tok, d, w_post, gate, residual, stride padding of u
    (1, 8, True, "", True, 0), (3, 72, False, "rows", True, 8), (9, 256, True, "vector", False, 0),
    (10, 264, True, "rows", True, 16), (33, 512, False, "", False, 64), (32, 1536, False, "", False, 576),
    (5, 2056, True, "vector", True, 0), (37, 5120, True, "rows", True, 0), (2, 8192, False, "vector", True, 0),
    (3, 8200, True, "", True, 8), (4, 16384, True, "rows", True, 0), (1500, 520, True, "vector", True, 0),
    (6000, 64, True, "rows", True, 0), (5000, 5120, False, "", True, 0)]


def _norm64(u, w_post, gate, alpha, res, w_pre):
    x = u.double()
    if w_post is not None:
        x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * w_post.double()
    if gate is not None:
        x = x * gate.double()
    mag = x.abs()
    r = x
    if res is not None:
        mag = res.double().abs() + abs(alpha) * mag
        r = res.double() + alpha * x
    rstd = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    return r, r * rstd * w_pre.double(), mag, mag * rstd * w_pre.double().abs()


@pytest.mark.parametrize("n_tok,d,post,gate,residual,pad", NORMS)
@pytest.mark.parametrize("to", ["bf16", "int8", "both"])
def test_block_norm(M, n_tok, d, post, gate, residual, pad, to):
    if to != "bf16" and d % 16:
        d += 8
    g = _gen(n_tok + d)
    u = _n(g, n_tok, d + pad)[:, :d]
    res = _n(g, n_tok, d) * 3 if residual else None
    w_post = 1 + 0.2 * _n(g, d) if post else None
    w_pre = 1 + 0.2 * _n(g, d)
    gt = {"": None, "vector": _n(g, d), "rows": _n(g, n_tok, d + pad)}[gate]
    alpha = 0.37
    res_out = torch.full((n_tok + 1, d), 5.0, dtype=torch.bfloat16, device="cuda") if residual else None
    out = torch.full((n_tok + 1, d), 5.0, dtype=torch.bfloat16, device="cuda") if to != "int8" else None
    out8 = torch.full((n_tok + 1, d), 99, dtype=torch.int8, device="cuda") if to != "bf16" else None
    scale = torch.full((n_tok + 1,), 7.0, device="cuda") if to != "bf16" else None
    M.mla_block_norm(u, d + pad, w_post, gt, d + pad if gate == "rows" else 0, alpha, res, res_out, w_pre, EPS, n_tok, d,
                     out, out8, scale)
    torch.cuda.synchronize()
    r, y, r_mag, y_mag = _norm64(u, w_post, gt if gate != "rows" else gt[:, :d], alpha, res, w_pre)
    # a handful of float32 operations on each term, and the mean's tree of at most 32 levels
    slop = 64 * F32
    if residual:
        assert ((res_out[:n_tok].double() - r).abs() <= BF * r.abs() + slop * r_mag).all()
        assert (res_out[n_tok] == 5.0).all()
    if out is not None:
        assert ((out[:n_tok].double() - y).abs() <= BF * y.abs() + slop * y_mag).all()
        assert (out[n_tok] == 5.0).all()
    if out8 is not None:
        s = scale[:n_tok].double()[:, None]
        amax = y.abs().amax(1, keepdim=True)
        assert ((s - amax / 127).abs() <= slop * y_mag.amax(1, keepdim=True) / 127).all()
        # half a step, and the rounding of what is divided
        assert ((out8[:n_tok].double() * s - y).abs() <= 0.5 * s + 2 * slop * y_mag.amax(1, keepdim=True)).all()
        assert (out8[:n_tok].abs().amax(1) == 127).all()
        assert (out8[n_tok] == 99).all() and scale[n_tok] == 7.0


def test_block_norm_in_place_residual_only_and_zero_rows(M):
    g = _gen(5)
    u, res = _n(g, 9, 640), _n(g, 9, 640)
    u[3] = 0
    res[3] = 0
    w = 1 + 0.2 * _n(g, 640)
    r, y, r_mag, _ = _norm64(u, None, None, -2.0, res, w)
    inplace = res.clone()
    M.mla_block_norm(u, 640, None, None, 0, -2.0, inplace, inplace, None, EPS, 9, 640)      # the residual add alone
    torch.cuda.synchronize()
    assert ((inplace.double() - r).abs() <= BF * r.abs() + 8 * F32 * r_mag).all()
    inplace = res.clone()
    out, out8, s = torch.empty_like(u), torch.empty(9, 640, dtype=torch.int8, device="cuda"), torch.empty(9, device="cuda")
    M.mla_block_norm(u, 640, None, None, 0, -2.0, inplace, inplace, w, EPS, 9, 640, out, out8, s)
    torch.cuda.synchronize()
    assert (out[3] == 0).all() and (out8[3] == 0).all() and s[3] == 0 and torch.isfinite(out.float()).all()
    assert ((inplace.double() - r).abs() <= BF * r.abs() + 8 * F32 * r_mag).all()
    # residual not written back: the norm of the sum alone
    keep = res.clone()
    again = torch.empty_like(u)
    M.mla_block_norm(u, 640, None, None, 0, -2.0, keep, None, w, EPS, 9, 640, again)
    torch.cuda.synchronize()
    assert torch.equal(keep, res) and torch.equal(again, out)


# ---- append from the projections' rows --------------------------------------

APPENDS = [  # n_h, d_c, d_h, d_r, B, T_q, row stride of kv
    (4, 64, 32, 16, 1, 1, 80), (1, 8, 8, 8, 3, 2, 32), (12, 136, 24, 24, 5, 3, 160), (16, 320, 256, 40, 2, 70, 360),
    (128, 512, 128, 64, 32, 1, 2112), (128, 512, 128, 64, 2, 131, 576)]


def _append_case(M, n_h, d_c, d_h, d_r, B, T_q, ld, seed):
    g = _gen(seed)
    n = B * T_q
    wide = _n(g, n, ld) * 2
    kv = wide[:, ld - d_c - d_r:]
    lens = torch.randint(T_q, T_q + 200, (B,), generator=g, device="cuda").tolist()
    mb = (max(lens) + 63) // 64 + 1
    table = torch.randperm(B * mb + 3, generator=g, device="cuda")[:B * mb].int().view(B, mb)
    pos = torch.tensor([L - T_q + t for L in lens for t in range(T_q)], dtype=torch.int32, device="cuda")
    return dict(q=_n(g, n, n_h, d_h + d_r), kv=kv, w=1 + 0.2 * _n(g, d_c), pos=pos, table=table, mb=mb,
                blocks=B * mb + 3, rope=M.mla_rope_table(d_r, 10000.0, max(lens)).cuda(), max_pos=max(lens),
                q_c=torch.full((n, n_h, d_h), 9.0, dtype=torch.bfloat16, device="cuda"),
                q_r=torch.full((n, n_h, d_r), 9.0, dtype=torch.bfloat16, device="cuda"))


def _rope_bits(x, pos, rope):
    """Float32 model of the rotation without fused multiply-add, as the cache append's."""
    h = x.shape[-1] // 2
    v, tab = x.float().cpu().numpy(), rope.cpu().numpy()[pos.cpu().numpy()]
    shape = (len(tab),) + (1,) * (v.ndim - 2) + (h,)
    c, s = tab[:, :h].reshape(shape), tab[:, h:].reshape(shape)
    a, b = v[..., :h], v[..., h:]
    y = np.concatenate([a * c - b * s, b * c + a * s], -1).astype(np.float32)
    return torch.from_numpy(y).bfloat16()


@pytest.mark.parametrize("shape", APPENDS)
def test_norm_rope_append(M, shape):
    n_h, d_c, d_h, d_r, B, T_q, ld = shape
    k = _append_case(M, *shape, seed=sum(shape))
    cfg = M.MlaConfig(n_h, d_c, d_h, d_r)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool = torch.full((k["blocks"], 64, d_c + d_r), float("nan"), dtype=torch.bfloat16, device="cuda")
    M.mla_norm_rope_append(cfg, k["q"], k["kv"], ld, k["w"], EPS, k["pos"], k["rope"], k["max_pos"], k["table"], k["mb"],
                           pool, k["blocks"], B, T_q, k["q_c"], k["q_r"], status)
    torch.cuda.synchronize()
    assert M.mla_read_status(status) == 0
    n = B * T_q
    seq = torch.arange(n, device="cuda") // T_q
    p = k["pos"].long()
    slot = k["table"][seq, p // 64].long() * 64 + p % 64
    rows = pool.view(-1, d_c + d_r)
    c = k["kv"][:, :d_c].double()
    want = c * torch.rsqrt((c * c).mean(1, keepdim=True) + EPS) * k["w"].double()
    got = rows[slot]
    assert ((got[:, :d_c].double() - want).abs() <= want.abs() * (BF + 64 * F32)).all()
    assert torch.equal(got[:, d_c:].cpu(), _rope_bits(k["kv"][:, d_c:], k["pos"], k["rope"]))
    rest = torch.ones(rows.shape[0], dtype=torch.bool, device="cuda")
    rest[slot] = False
    assert torch.isnan(rows[rest].float()).all()            # every other row as it was
    assert torch.equal(k["q_c"], k["q"][:, :, :d_h])
    assert torch.equal(k["q_r"].cpu(), _rope_bits(k["q"][:, :, d_h:], k["pos"], k["rope"]))
    # a cache fill without queries writes the same rows
    fill = torch.full_like(pool, float("nan"))
    M.mla_norm_rope_append(cfg, None, k["kv"], ld, k["w"], EPS, k["pos"], k["rope"], k["max_pos"], k["table"], k["mb"],
                           fill, k["blocks"], B, T_q)
    torch.cuda.synchronize()
    assert torch.equal(fill.view(torch.int16), pool.view(torch.int16))


@pytest.mark.parametrize("shape", [s for s in APPENDS if s[1] % 64 == 0])
def test_norm_rope_append_e4m3_is_the_two_steps(M, shape):
    """The low-bit form quantises exactly the bf16 rows that the bf16 form appends."""
    n_h, d_c, d_h, d_r, B, T_q, ld = shape
    k = _append_case(M, *shape, seed=sum(shape))
    cfg = M.MlaConfig(n_h, d_c, d_h, d_r)
    pool = torch.zeros((k["blocks"], 64, d_c + d_r), dtype=torch.bfloat16, device="cuda")
    low = torch.full((k["blocks"], 64, M.mla_e4m3_row_bytes(d_c, d_r)), 0x7F, dtype=torch.uint8, device="cuda")
    args = (k["q"], k["kv"], ld, k["w"], EPS, k["pos"], k["rope"], k["max_pos"], k["table"], k["mb"])
    M.mla_norm_rope_append(cfg, *args, pool, k["blocks"], B, T_q, k["q_c"], k["q_r"])
    q_c, q_r = k["q_c"].clone(), k["q_r"].clone()
    M.mla_norm_rope_append_e4m3(cfg, *args, low, k["blocks"], B, T_q, k["q_c"], k["q_r"])
    want = torch.full_like(low, 0x7F)
    n = B * T_q
    seq = torch.arange(n, device="cuda") // T_q
    p = k["pos"].long()
    slot = k["table"][seq, p // 64].long() * 64 + p % 64
    normed = pool.view(-1, d_c + d_r)[slot][:, :d_c].contiguous()
    keys = k["kv"][:, d_c:].contiguous()
    M.mla_rope_append_e4m3(cfg, None, keys, normed, k["pos"], k["rope"], k["max_pos"], k["table"], k["mb"], want,
                           k["blocks"], B, T_q)
    torch.cuda.synchronize()
    assert torch.equal(low, want) and torch.equal(k["q_c"], q_c) and torch.equal(k["q_r"], q_r)


def test_norm_rope_append_skips_invalid_tokens(M):
    """Padded tokens (position -1), positions past the table or the pages, and bad blocks: flagged and left alone."""
    shape = (4, 64, 32, 16, 6, 1, 80)
    k = _append_case(M, *shape, seed=3)
    cfg = M.MlaConfig(4, 64, 32, 16)
    k["pos"][1], k["pos"][2] = -1, k["max_pos"]
    k["table"][4, :] = k["blocks"]
    k["table"][5, :] = -1
    for e4m3 in (False, True):
        call = M.mla_norm_rope_append_e4m3 if e4m3 else M.mla_norm_rope_append
        width = M.mla_e4m3_row_bytes(64, 16) if e4m3 else 80
        pool = torch.full((k["blocks"], 64, width), 3, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_c, q_r = k["q_c"].clone(), k["q_r"].clone()
        call(cfg, k["q"], k["kv"], 80, k["w"], EPS, k["pos"], k["rope"], k["max_pos"], k["table"], k["mb"], pool,
             k["blocks"], 6, 1, q_c, q_r, status)
        torch.cuda.synchronize()
        assert M.mla_read_status(status) == M.MLA_STATUS_BAD_POSITION | M.MLA_STATUS_BAD_BLOCK
        written = (pool != 3).any(-1).view(-1).nonzero().view(-1).tolist()
        p = k["pos"].tolist()
        assert sorted(written) == sorted(int(k["table"][b, p[b] // 64]) * 64 + p[b] % 64 for b in (0, 3))
        for b in range(6):
            if b in (1, 2):
                assert (q_c[b] == 9.0).all() and (q_r[b] == 9.0).all()
            else:
                assert torch.equal(q_c[b], k["q"][b, :, :32])



# ---- a layer's step: the operators one after the other ------------------------

class Layer:
    """One attention layer's serving step of a batch behind shared pages, every projection around the per-head ones
    in 8-bit integers: norm, down projections, norm of the query latent, W^UQ, append, absorb_q, decode, up_v, W^O, and
    the residual add with the next block's norm."""

    D, CQ, DC, DR, DH = 1024, 256, 512, 64, 128

    def __init__(self, M, n_h, B, T_q, n_shared, own):
        g = _gen(n_h + B)
        self.M, self.cfg, self.B, self.T_q, self.n_h, self.n = M, M.MlaConfig(n_h, self.DC, self.DH, self.DR), B, T_q, n_h, B * T_q
        n, D = self.n, self.D
        pages = n_shared + max((k + 63) // 64 for k in own)
        self.mb, self.n_shared = pages, n_shared
        blocks = n_shared + B * (pages - n_shared)
        perm = torch.randperm(blocks, generator=g, device="cuda").int()
        self.shared = perm[:n_shared].contiguous()
        self.table = torch.full((B, pages), -1, dtype=torch.int32, device="cuda")
        self.table[:, n_shared:] = perm[n_shared:].view(B, -1)
        self.table[:, :n_shared] = self.shared                    # the append reads the whole row
        self.pool = _n(g, blocks, 64, self.DC + self.DR)
        lens = torch.tensor([64 * n_shared + k for k in own], device="cuda")
        self.lens = lens.int()
        self.pos = (lens[:, None] - T_q + torch.arange(T_q, device="cuda")).int().reshape(-1)
        self.rope = M.mla_rope_table(self.DR, 10000.0, 64 * pages).cuda()
        self.x, self.res = _n(g, n, D), _n(g, n, D) * 2
        self.w_in, self.w_cq, self.w_kv, self.w_next = (1 + 0.1 * _n(g, k) for k in (D, self.CQ, self.DC, D))

        def weight(o, i):
            w = (_n(g, o, i).float() / i ** 0.5).bfloat16()
            w8, sw = torch.empty(o, i, dtype=torch.int8, device="cuda"), torch.empty(o, device="cuda")
            M.mla_quantize_i8(w, i, o, i, w8, sw)
            return w8, sw
        self.w_down = weight(self.CQ + self.DC + self.DR, D)
        self.w_uq = weight(n_h * (self.DH + self.DR), self.CQ)
        self.w_o = weight(D, n_h * self.DH)
        self.w_uk, self.w_uv = ((_n(g, n_h, self.DH, self.DC).float() / self.DC ** 0.5).bfloat16() for _ in range(2))
        bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        i8 = lambda *s: torch.zeros(*s, dtype=torch.int8, device="cuda")  # noqa: E731
        f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        self.r = dict(res1=bf(n, D), h8=i8(n, D), sh=f(n), down=bf(n, self.CQ + self.DC + self.DR), cq8=i8(n, self.CQ), scq=f(n),
                      q=bf(n, n_h, self.DH + self.DR), q_c=bf(n, n_h, self.DH), q_r=bf(n, n_h, self.DR),
                      q_abs=bf(n, n_h, self.DC), latent=bf(n, n_h, self.DC), lse=f(n, n_h), o=bf(n, n_h * self.DH),
                      o8=i8(n, n_h * self.DH), so=f(n), u=bf(n, D), res2=bf(n, D), y=bf(n, D))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.zeros(M.mla_decode_shared_workspace_bytes(self.cfg, B, T_q), dtype=torch.uint8, device="cuda")

    def step(self, between=lambda: None):
        M, r, n, D, CQ, n_h = self.M, self.r, self.n, self.D, self.CQ, self.n_h
        W = CQ + self.DC + self.DR
        calls = [
            lambda: M.mla_block_norm(self.x, D, None, None, 0, 1.0, self.res, r["res1"], self.w_in, EPS, n, D, None, r["h8"], r["sh"]),
            lambda: M.mla_linear_i8(r["h8"], D, r["sh"], *self.w_down, r["down"], n, D, W, self.status),
            lambda: M.mla_block_norm(r["down"], W, None, None, 0, 1.0, None, None, self.w_cq, EPS, n, CQ, None, r["cq8"], r["scq"]),
            lambda: M.mla_linear_i8(r["cq8"], CQ, r["scq"], *self.w_uq, r["q"], n, CQ, n_h * (self.DH + self.DR), self.status),
            lambda: M.mla_norm_rope_append(self.cfg, r["q"], r["down"][:, CQ:], W, self.w_kv, EPS, self.pos, self.rope,
                                           self.rope.shape[0], self.table, self.mb, self.pool, self.pool.shape[0], self.B,
                                           self.T_q, r["q_c"], r["q_r"], self.status),
            lambda: M.mla_absorb_q(self.cfg, r["q_c"], self.w_uk, r["q_abs"], n),
            lambda: M.mla_decode_shared(self.cfg, r["q_abs"], r["q_r"], self.pool, self.pool.shape[0], self.shared, self.n_shared,
                                        self.table, self.mb, self.lens, self.B, self.T_q, 0, self.ws, self.ws.numel(),
                                        r["latent"], r["lse"]),
            lambda: M.mla_up_v(self.cfg, r["latent"], self.w_uv, r["o"], n),
            lambda: M.mla_quantize_i8(r["o"], n_h * self.DH, n, n_h * self.DH, r["o8"], r["so"]),
            lambda: M.mla_linear_i8(r["o8"], n_h * self.DH, r["so"], *self.w_o, r["u"], n, n_h * self.DH, D, self.status),
            lambda: M.mla_block_norm(r["u"], D, None, None, 0, 0.5, r["res1"], r["res2"], self.w_next, EPS, n, D, r["y"]),
        ]
        for call in calls:
            call()
            between()

    def results(self):
        torch.cuda.synchronize()
        assert self.M.mla_read_status(self.status) == 0 and self.M.mla_read_status(self.ws) == 0
        return {k: v.clone() for k, v in self.r.items()} | {"pool": self.pool.clone()}


@pytest.mark.parametrize("n_h,B,T_q,n_shared,own", [(16, 6, 2, 5, [2, 70, 130, 64, 3, 200]), (128, 3, 1, 9, [1, 64, 300]),
                                                    (16, 40, 4, 3, [4, 67, 100, 150] * 10)])
def test_a_layers_step(M, n_h, B, T_q, n_shared, own):
    a = Layer(M, n_h, B, T_q, n_shared, own)
    a.step(torch.cuda.synchronize)                # one call at a time
    want = a.results()
    # each projection and norm against its own inputs in 64 bits (the decode has its own tests)
    r = want
    rr, y, r_mag, y_mag = _norm64(a.x, None, None, 1.0, a.res, a.w_in)
    assert ((r["res1"].double() - rr).abs() <= BF * rr.abs() + 64 * F32 * r_mag).all()
    # codes of a float32 value a few roundings away from y may fall one step apart, next to a half
    assert ((r["h8"].double() - 127 * y / y.abs().amax(1, keepdim=True)).abs() <= 0.5 + 127 * 64 * F32 * (y_mag / y.abs().amax(1, keepdim=True))).all()
    _check_linear(r["down"], r["h8"], r["sh"], *a.w_down)
    _check_linear(r["q"].view(a.n, -1), r["cq8"], r["scq"], *a.w_uq)
    _check_linear(r["u"], r["o8"], r["so"], *a.w_o)
    assert torch.equal(r["q_c"], r["q"][:, :, :a.DH])
    # the decode's output against the keys that the append wrote
    keys = torch.cat([a.pool[a.shared.long()].reshape(-1, 576), a.pool[a.table[0, n_shared:].long()].reshape(-1, 576)]).double()
    see = keys[:64 * n_shared + own[0]]           # sequence 0, its last token
    q = torch.cat([r["q_abs"][T_q - 1], r["q_r"][T_q - 1]], 1).double()
    s = q @ see.T / 192 ** 0.5
    p = torch.softmax(s, 1)
    err = (577 * F32 * (q.abs() @ see.abs().T) / 192 ** 0.5 + 4 * F32 * s.abs()).amax(1)[:, None]   # of a weight, through its score
    o, mag = p @ see[:, :512], p @ see[:, :512].abs()
    assert ((r["latent"][T_q - 1].double() - o).abs() <= (BF + 2 * err + 1e-4) * mag + BF * o.abs()).all()
    rr, y, r_mag, y_mag = _norm64(r["u"], None, None, 0.5, r["res1"], a.w_next)
    assert ((r["res2"].double() - rr).abs() <= BF * rr.abs() + 64 * F32 * r_mag).all()
    assert ((r["y"].double() - y).abs() <= BF * y.abs() + 64 * F32 * y_mag).all()

    def same(got):
        for k, v in want.items():
            assert torch.equal(v.view(torch.uint8) if v.dtype != torch.int8 else v, got[k].view(torch.uint8) if v.dtype != torch.int8 else got[k]), k
    # back to back, and captured: the same bits, whatever overlaps
    for v in a.r.values():
        v.zero_()
    a.step()
    same(a.results())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
        a.step()
    for v in a.r.values():
        v.zero_()
    for _ in range(3):
        graph.replay()
    same(a.results())

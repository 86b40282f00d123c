"""mla_decode_shared: the decode of a batch behind shared cache pages, against a
plain softmax over each row's whole key list in 64 bits.

Bounds, per output element o = sum_j p_j c_j (A = sum_j p_j |c_j|): the tensor
cores take the weights as bf16 (off by 2^-8 of each at most) and the result is
rounded to bf16; scores are float32 sums of 576 exact products, off by at most
576 2^-24 of the sum of their magnitudes, which moves each weight by as much
(and the lse too): with |q_i k_i| summing to at most about 400 at these inputs
and the scale 1/sqrt(d_h + d_r) that is below 2e-3 at the very worst; the
kernels' sums stay a hundred times below it.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8
SCORE = 1e-4     # relative error of a weight from its score


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_38_b200 import build
    build.build()
    from mla_latent_kv_38_b200 import binding
    return binding


class Case:
    """A batch behind n_shared pages; own[b] keys of sequence b behind them (this step's tokens included; negative: a
    length that the call has to flag)."""

    def __init__(self, M, n_h, d_c, d_h, d_r, T_q, n_shared, own, impl, splits=0, seed=0, spare=1):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 1000 * n_h + n_shared)
        self.M, self.cfg = M, M.MlaConfig(n_h, d_c, d_h, d_r, impl=impl)
        self.n_h, self.d_c, self.d_h, self.d_r, self.T_q, self.n_shared, self.own = n_h, d_c, d_h, d_r, T_q, n_shared, own
        self.splits = splits
        B = self.B = len(own)
        D = d_c + d_r
        pages = [(max(k, 0) + 63) // 64 for k in own]
        self.mb = n_shared + max(max(pages), 1) + spare
        self.blocks = n_shared + sum(pages) + 2
        perm = torch.randperm(self.blocks, generator=g, device="cuda").int()
        # rows behind a sequence's end and unused pages hold NaN; so do table entries that must not be read
        self.pool = torch.full((self.blocks, 64, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.shared = perm[:n_shared].contiguous()
        self.table = torch.full((B, self.mb), -7, dtype=torch.int32, device="cuda")
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.pool[self.shared.long()] = rnd(n_shared, 64, D)
        at = n_shared
        for b, k in enumerate(own):
            ids = perm[at:at + pages[b]]
            at += pages[b]
            self.table[b, n_shared:n_shared + pages[b]] = ids
            rows = rnd(64 * pages[b], D)
            rows[max(k, 0):] = float("nan")
            self.pool[ids.long()] = rows.view(-1, 64, D)
        self.lens = torch.tensor([64 * n_shared + k if k > 0 else k for k in own], dtype=torch.int32, device="cuda")
        n = B * T_q
        self.q_abs, self.q_r = (rnd(n, n_h, d_c) * 0.5), rnd(n, n_h, d_r)
        self.latent = torch.full((n + 1, n_h, d_c), 77.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((n + 1, n_h), 77.0, device="cuda")
        self.ws = torch.zeros(M.mla_decode_shared_workspace_bytes(self.cfg, B, T_q, splits), dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        self.M.mla_decode_shared(self.cfg, self.q_abs, self.q_r, self.pool, self.blocks,
                                 self.shared if self.n_shared else None, self.n_shared, self.table, self.mb, self.lens,
                                 self.B, self.T_q, self.splits, self.ws, self.ws.numel(), self.latent, self.lse, stream)

    def status(self):
        return self.M.mla_read_status(self.ws)

    def valid(self, b):
        return 64 * self.n_shared + self.T_q <= int(self.lens[b]) <= 64 * self.mb

    def check(self):
        P, T_q = 64 * self.n_shared, self.T_q
        prefix = self.pool[self.shared.long()].reshape(-1, self.d_c + self.d_r)
        scale = 1.0 / math.sqrt(self.d_h + self.d_r)
        for b, k in enumerate(self.own):
            rows = slice(b * T_q, (b + 1) * T_q)
            got, lse = self.latent[rows].double(), self.lse[rows].double()
            if not self.valid(b):
                assert (got == 0).all() and (lse == -math.inf).all(), b
                continue
            ids = self.table[b, self.n_shared:(P + k + 63) // 64].long()
            keys = torch.cat([prefix, self.pool[ids].reshape(-1, self.d_c + self.d_r)[:k]]).double()
            for t in range(T_q):
                n = b * T_q + t
                see = keys[:P + k - T_q + t + 1]
                s = (self.q_abs[n].double() @ see[:, :self.d_c].T + self.q_r[n].double() @ see[:, self.d_c:].T) * scale
                want_lse = torch.logsumexp(s, 1)
                p = torch.exp(s - want_lse[:, None])
                o, mag = p @ see[:, :self.d_c], p @ see[:, :self.d_c].abs()
                err = (got[t] - o).abs()
                assert (err <= (BF + SCORE) * mag + BF * o.abs()).all(), (b, t, (err / mag).max().item())
                assert ((lse[t] - want_lse).abs() <= SCORE).all(), (b, t)
        assert (self.latent[self.B * T_q:] == 77.0).all() and (self.lse[self.B * T_q:] == 77.0).all()


V2 = (512, 128, 64)
PORTABLE = [   # n_h, (d_c, d_h, d_r), T_q, n_shared, own keys
    (4, (64, 32, 16), 1, 2, [128]),
    (12, (136, 24, 8), 2, 1, [2, 3, 64, 65, 70]),
    (1, (8, 8, 8), 1, 3, [1, 200]),
    (33, (256, 64, 64), 3, 0, [3, 190]),
    (128, V2, 1, 5, [1, 63, 64, 65, 130]),
    (16, V2, 4, 4, [4, 5, 67, 300]),
]


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("case", PORTABLE)
def test_portable_kernels(M, case, splits):
    n_h, (d_c, d_h, d_r), T_q, n_shared, own = case
    c = Case(M, n_h, d_c, d_h, d_r, T_q, n_shared, own, M.IMPL_SIMT, splits)
    c.run()
    torch.cuda.synchronize()
    assert c.status() == 0
    c.check()


SHAPES = [     # n_h, T_q, n_shared, own keys (the 512 + 64 column row)
    (1, 1, 1, [1]),
    (3, 2, 2, [2, 9, 64]),
    (16, 1, 4, [1, 70, 33]),
    (16, 3, 37, [3, 64, 65, 128, 129, 300, 257] * 3),
    (40, 5, 8, [5, 61, 200]),
    (127, 1, 3, [1, 500]),
    (128, 1, 56, [1, 17, 63, 64, 65, 255, 256, 257, 512, 300] * 3),
    (128, 4, 9, [4, 700, 64]),
    (129, 2, 5, [2, 130]),
    (200, 1, 4, [90, 1]),
    (256, 2, 4, [2, 90]),
    (1024, 1, 2, [3]),
    (128, 1, 0, [1, 200, 513]),
    (16, 2, 0, [2, 200]),
    (8, 1, 1000, [1, 5]),
]


@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("case", SHAPES)
def test_cache_row_of_576(M, case, splits):
    n_h, T_q, n_shared, own = case
    c = Case(M, n_h, *V2, T_q, n_shared, own, M.IMPL_AUTO, splits)
    c.run()
    torch.cuda.synchronize()
    assert c.status() == 0
    c.check()


@pytest.mark.parametrize("impl", [0, 1])
def test_invalid_lengths_are_flagged_and_leave_the_others(M, impl):
    """A padded batch: lengths of zero, inside the shared pages, and beyond the table."""
    c = Case(M, 16, *V2, 2, 3, [0, 70, -5, 2, 0, 130], impl)
    c.lens[4] = 64 * 3 + 1            # one token short of T_q behind the shared pages
    c.lens[0] = 64 * c.mb + 1
    c.own = [0, 70, 0, 2, 0, 130]
    c.run()
    torch.cuda.synchronize()
    assert c.status() == M.MLA_STATUS_BAD_SEQ_LEN
    c.check()


@pytest.mark.parametrize("impl", [0, 1])
def test_lengths_at_the_ends_of_int32(M, impl):
    c = Case(M, 16, *V2, 1, 3, [0, 70, 0, 130], impl)
    c.lens[0], c.lens[2] = -2 ** 31, 2 ** 31 - 1
    c.run()
    torch.cuda.synchronize()
    assert c.status() == M.MLA_STATUS_BAD_SEQ_LEN
    c.check()


@pytest.mark.parametrize("impl", [0, 1])
def test_bad_blocks_are_flagged(M, impl):
    """Entries outside the pool, shared and own, are flagged; nothing is read out of bounds."""
    for where in ("shared", "own"):
        c = Case(M, 16, *V2, 1, 3, [70, 130], impl)
        c.pool.nan_to_num_(0.0)
        if where == "shared":
            c.shared[1] = c.blocks
        else:
            c.table[1, 4] = -1
        c.run()
        torch.cuda.synchronize()
        assert c.status() == M.MLA_STATUS_BAD_BLOCK, where
        assert torch.isfinite(c.latent.float()).all() and torch.isfinite(c.lse).all()


def test_matches_mla_decode_on_the_same_table(M):
    """The plain decode with the shared blocks written into every table row computes the same rows."""
    c = Case(M, 128, *V2, 2, 6, [2, 77, 300, 513], 0)
    c.run()
    full = c.table.clone()
    full[:, :6] = c.shared
    ws = torch.zeros(M.mla_decode_workspace_bytes(c.cfg, c.B, 2, 0), dtype=torch.uint8, device="cuda")
    lat, lse = torch.empty_like(c.latent), torch.empty_like(c.lse)
    M.mla_decode(c.cfg, c.q_abs, c.q_r, c.pool, c.blocks, full, c.mb, c.lens, c.B, 2, 0, ws, ws.numel(), lat, lse)
    torch.cuda.synchronize()
    n = c.B * 2
    # each side rounds its weights and its result to bf16
    assert ((lat[:n].float() - c.latent[:n].float()).abs() <= 4 * BF * lat[:n].float().abs().clamp(min=0.25)).all()
    assert ((lse[:n] - c.lse[:n]).abs() <= 2 * SCORE).all()


@pytest.mark.parametrize("impl", [0, 1])
def test_streams_and_graphs(M, impl):
    """Two batches with their own workspaces on two streams, then captured and replayed on changed inputs."""
    a, b = (Case(M, 32, *V2, 1, 5, own, impl, seed=s) for s, own in ((1, [5, 200, 64]), (2, [90, 1])))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a.run(s1)
        b.run(s2)
    torch.cuda.synchronize()
    a.check()
    b.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
        b.run()
    for c in (a, b):
        c.q_abs.copy_(c.q_abs.flip(0))
        c.latent.fill_(77.0)
        c.lse.fill_(77.0)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert a.status() == 0 and b.status() == 0
    a.check()
    b.check()


MANY_TOKENS = [  # units of many whole tokens, whose last keys only some of their rows see; unit counts past one block's scan
    (1, 100, 2, [100, 150, 228]),
    (2, 70, 3, [70, 71, 133, 200]),
    (24, 9, 6, [9, 70, 64]),
    (48, 4, 21, [4, 66, 130]),
    (65, 3, 5, [3, 190]),
    (128, 2, 3, [2, 3, 65, 70] * 300),
    (16, 1, 40, [1, 2, 66] * 800),
]


@pytest.mark.parametrize("case", MANY_TOKENS)
def test_units_of_many_tokens_and_many_units(M, case):
    n_h, T_q, n_shared, own = case
    c = Case(M, n_h, *V2, T_q, n_shared, own, M.IMPL_AUTO)
    c.run()
    torch.cuda.synchronize()
    assert c.status() == 0
    c.check()


@pytest.mark.parametrize("impl", [0, 1])
@pytest.mark.parametrize("n_h,T_q,own", [(16, 4, [4, 66, 131, 259]), (1, 70, [70, 130, 200]), (128, 3, [3, 66, 257]), (40, 3, [64])])
def test_non_finite_keys_of_later_tokens(M, impl, n_h, T_q, own):
    """Infinities and NaN in the rows that only a step's last tokens see leave the tokens before them as they are."""
    c = Case(M, n_h, *V2, T_q, 3, own, impl)
    hide = max(1, T_q // 2)                    # the last `hide` tokens of each sequence
    for b, k in enumerate(own):
        for j in range(k - hide, k):
            page = int(c.table[b, (64 * 3 + j) // 64])
            c.pool[page, j % 64, ::3] = float("nan")
            c.pool[page, j % 64, 1::3] = float("inf")
    c.run()
    torch.cuda.synchronize()
    assert c.status() == 0
    got, lse = c.latent[:c.B * T_q].view(c.B, T_q, n_h, -1), c.lse[:c.B * T_q].view(c.B, T_q, n_h)
    clean = Case(M, n_h, *V2, T_q, 3, own, impl)
    clean.run()
    torch.cuda.synchronize()
    clean.check()
    first = slice(0, T_q - hide)
    assert torch.equal(got[:, first], clean.latent[:c.B * T_q].view(c.B, T_q, n_h, -1)[:, first])
    assert torch.equal(lse[:, first], clean.lse[:c.B * T_q].view(c.B, T_q, n_h)[:, first])


@pytest.mark.parametrize("n_h,T_q,n_shared,own", [(128, 1, 24, [70, 700, 300]), (128, 2, 70, [900, 1500]), (16, 2, 40, [70, 900, 500] * 4)])
def test_growing_maxima(M, n_h, T_q, n_shared, own):
    """Keys that grow along the sequence, so that the running maximum is passed by far again and again."""
    c = Case(M, n_h, *V2, T_q, n_shared, own, 0)
    P = 64 * n_shared
    ramp = lambda pos: 0.25 + 6.0 * (pos / (P + max(own)))  # noqa: E731
    for j in range(n_shared):
        c.pool[c.shared[j].long()] *= ramp(64 * j)
    for b, k in enumerate(own):
        for j in range((k + 63) // 64):
            c.pool[c.table[b, n_shared + j].long()] *= ramp(P + 64 * j)
    c.run()
    torch.cuda.synchronize()
    assert c.status() == 0
    prefix = c.pool[c.shared.long()].reshape(-1, 576)
    scale = 1.0 / math.sqrt(192)
    for b, k in enumerate(own):
        ids = c.table[b, n_shared:(P + k + 63) // 64].long()
        keys = torch.cat([prefix, c.pool[ids].reshape(-1, 576)[:k]]).double()
        for t in range(T_q):
            n = b * T_q + t
            see = keys[:P + k - T_q + t + 1]
            q = torch.cat([c.q_abs[n], c.q_r[n]], 1).double()
            s = q @ see.T * scale
            want = torch.logsumexp(s, 1)
            p = torch.exp(s - want[:, None])
            o, mag = p @ see[:, :512], p @ see[:, :512].abs()
            # a float32 sum of 576 products is off by at most 576 2^-24 of their magnitudes, and a weight (and
            # the lse) by as much again through the scaled score and its exponent
            err = (577 * 2.0 ** -24 * (q.abs() @ see.abs().T) * scale + 2.0 ** -22 * s.abs()).amax(1)
            got, lse = c.latent[n].double(), c.lse[n].double()
            assert ((got - o).abs() <= (BF + 2 * err[:, None] + SCORE) * mag + BF * o.abs()).all(), (b, t)
            assert ((lse - want).abs() <= err + SCORE).all(), (b, t)

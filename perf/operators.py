"""Cases, plain forms and exact values of the operators around the latent-cache decode.

Four operators of one attention layer in serving, each reached through
``mla_latent_kv_38_b200.binding``:

  shared   mla_decode_shared: attention of a batch whose sequences share their
           first cache pages, the shared pages computed once for all rows
  linear   mla_quantize_i8 + mla_linear_i8: a projection in 8-bit integers with
           one scale per token and per output channel
  norm     mla_block_norm: a block's output normed, gated, scaled and added to
           the residual stream, and the norm in front of the next block (its
           output in bf16, or in 8-bit integers straight into mla_linear_i8)
  append   mla_norm_rope_append: the down projection's rows normed, rotated and
           appended to the paged cache, the query rows split and rotated

``own`` selects between the plain forms (elementary torch operations in
float32) and the library's kernels.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
D_C, D_R, D_H = 512, 64, 128          # latent columns, RoPE columns, head width
D_MODEL, D_CQ = 5120, 1536            # model width, query latent
PAGE = 64
SCALE = 1.0 / math.sqrt(D_H + D_R)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # three chats of one tensor-parallel shard (16 of 128 heads) behind a short system prompt: latency
        dict(name="shared shard small", op="shared", B=3, T_q=1, n_h=16, pages=4, own_max=70),
        # the decode workload's batch and length with the chunk workload's prefix of 56 pages shared
        dict(name="shared decode", op="shared", B=32, T_q=1, n_h=128, pages=56, own_max=512),
        # a large batch on one shard, two tokens a step (one drafted), a prompt with few-shot examples
        dict(name="shared shard large", op="shared", B=128, T_q=2, n_h=16, pages=129, own_max=1500),
        # the multi-token workload (64 sequences, 4 tokens) with 8,192 shared keys: the largest
        dict(name="shared multi token", op="shared", B=64, T_q=4, n_h=128, pages=128, own_max=900),
        # one token through the down projections (query latent and cache row side by side)
        dict(name="linear one token", op="linear", n_tok=1, d_in=D_MODEL, d_out=D_CQ + D_C + D_R),
        # the output projection at the decode batch
        dict(name="linear output", op="linear", n_tok=32, d_in=128 * D_H, d_out=D_MODEL),
        # the query up-projection of a prefill of 2,048 tokens
        dict(name="linear prefill", op="linear", n_tok=2048, d_in=D_CQ, d_out=128 * (D_H + D_R)),
        # between two blocks at the decode batch
        dict(name="norm decode", op="norm", n_tok=32, d=D_MODEL, post=True, gate="vector", residual=True, to="bf16"),
        # between two blocks in a prefill, the gate computed per token
        dict(name="norm prefill", op="norm", n_tok=4096, d=D_MODEL, post=True, gate="rows", residual=True, to="bf16"),
        # the residual add and norm in front of the down projections, into 8-bit integers and their product
        dict(name="norm into linear", op="norm", n_tok=37, d=D_MODEL, post=False, gate="", residual=True, to="linear"),
        # the decode batch's new rows
        dict(name="append decode", op="append", B=32, T_q=1, n_h=128, start=4000),
        # a chunk of the chunked prefill, at odd positions
        dict(name="append chunk", op="append", B=4, T_q=509, n_h=128, start=3500),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "linear", "norm", "append"])
    if op == "shared":
        n_h = rng.choice([8, 16, 32, 64, 128])
        T_q = rng.choice([1, 1, 2, 3, 4])
        B = _log(rng, 1, min(128, 64 * 4 * 128 // (n_h * T_q)))
        own_max = max(T_q, _log(rng, 1, 900))
        return dict(op=op, B=B, T_q=T_q, n_h=n_h, pages=_log(rng, 1, 128), own_max=own_max)
    if op == "linear":
        d_in = 16 * _log(rng, 4, 1024)
        d_out = 8 * _log(rng, 8, 3200)
        most = 2048 * D_CQ * 128 * (D_H + D_R) // (d_in * d_out)
        return dict(op=op, n_tok=_log(rng, 1, max(1, min(4096, most))), d_in=d_in, d_out=d_out)
    if op == "norm":
        to = rng.choice(["bf16", "bf16", "linear"])
        d = (16 * _log(rng, 8, 512)) if to == "linear" else (8 * _log(rng, 16, 1024))
        return dict(op=op, n_tok=_log(rng, 1, max(1, 4096 * D_MODEL // max(d, D_CQ))), d=d, post=rng.random() < 0.5,
                    gate=rng.choice(["", "vector", "rows"]), residual=rng.random() < 0.7, to=to)
    n_h = rng.choice([4, 16, 128])
    B = _log(rng, 1, 64)
    return dict(op=op, B=B, T_q=_log(rng, 1, max(1, 2036 // B)), n_h=n_h, start=rng.randrange(0, 4000))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _rope_table(max_pos):
    m = torch.arange(D_R // 2, dtype=torch.float64)
    th = torch.arange(max_pos, dtype=torch.float64)[:, None] * (10000.0 ** (-2.0 * m / D_R))
    return torch.cat([th.cos(), th.sin()], 1).float().to(DEV)


def _weight_i8(g, d_out, d_in):
    """A bf16 weight of deviation 1/sqrt(d_in) as int8 rows with a scale each: laid out once, kept by the program."""
    w = (torch.randn(d_out, d_in, generator=g, device=DEV) / math.sqrt(d_in)).bfloat16().float()
    amax = w.abs().amax(1, keepdim=True)
    return torch.round(w * 127.0 / amax).to(torch.int8), (amax / 127.0).squeeze(1)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    n = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()  # noqa: E731
    bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    s = dict(case)
    if case["op"] == "shared":
        B, T_q, n_h, pages = case["B"], case["T_q"], case["n_h"], case["pages"]
        lens = torch.randint(T_q, case["own_max"] + 1, (B,), generator=g, device=DEV)   # own keys, this step's included
        own_pages = (case["own_max"] + PAGE - 1) // PAGE
        blocks = pages + B * own_pages
        perm = torch.randperm(blocks, generator=g, device=DEV).int()
        table = torch.full((B, pages + own_pages), -1, dtype=torch.int32, device=DEV)
        table[:, :pages] = perm[:pages]
        table[:, pages:] = perm[pages:].view(B, own_pages)
        # stale rows of earlier sequences behind each sequence's last one
        s.update(pool=n(blocks, PAGE, D_C + D_R), table=table, shared=perm[:pages].contiguous(),
                 lens=(lens + PAGE * pages).int(), max_len=PAGE * pages + case["own_max"],
                 q_abs=n(B * T_q, n_h, D_C) * 0.5, q_r=n(B * T_q, n_h, D_R),
                 latent=bf(B * T_q, n_h, D_C), lse=torch.empty(B * T_q, n_h, device=DEV))
    elif case["op"] == "linear":
        w8, sw = _weight_i8(g, case["d_out"], case["d_in"])
        n_tok = case["n_tok"]
        s.update(x=n(n_tok, case["d_in"]), w8=w8, sw=sw, out=bf(n_tok, case["d_out"]),
                 x8=torch.empty(n_tok, case["d_in"], dtype=torch.int8, device=DEV), sx=torch.empty(n_tok, device=DEV))
    elif case["op"] == "norm":
        n_tok, d = case["n_tok"], case["d"]
        s.update(u=n(n_tok, d), res=n(n_tok, d) * 4.0, w_pre=1.0 + 0.1 * n(d), w_post=1.0 + 0.1 * n(d),
                 gate={"": None, "vector": n(d), "rows": n(n_tok, d)}[case["gate"]], alpha=0.22, res_out=bf(n_tok, d), y=bf(n_tok, d))
        if case["to"] == "linear":
            s["w8"], s["sw"] = _weight_i8(g, D_CQ + D_C + D_R, d)
            s.update(y8=torch.empty(n_tok, d, dtype=torch.int8, device=DEV), sy=torch.empty(n_tok, device=DEV),
                     out=bf(n_tok, D_CQ + D_C + D_R))
    else:
        B, T_q, n_h = case["B"], case["T_q"], case["n_h"]
        n_tok = B * T_q
        last = case["start"] + T_q + B                            # sequences start one position apart
        per = (last + PAGE - 1) // PAGE
        first = case["start"] // PAGE                             # only the pages that this step touches exist
        used = per - first
        perm = torch.randperm(B * used, generator=g, device=DEV).int().view(B, used)
        table = torch.full((B, per), -1, dtype=torch.int32, device=DEV)
        table[:, first:] = perm
        pos = (case["start"] + torch.arange(B, device=DEV)[:, None] + torch.arange(T_q, device=DEV)).int().reshape(-1)
        down = n(n_tok, D_CQ + D_C + D_R)                         # the down projection's rows: query latent, then cache row
        s.update(q=n(n_tok, n_h, D_H + D_R), kv=down[:, D_CQ:], w=1.0 + 0.1 * n(D_C), pos=pos, rope=_rope_table(last),
                 table=table, pool=n(B * used, PAGE, D_C + D_R), q_c=bf(n_tok, n_h, D_H), q_r=bf(n_tok, n_h, D_R))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _OWN[s["op"]](s)
    return _PLAIN[s["op"]](s)


def _plain_shared(s):
    B, T_q, n_h, pages = s["B"], s["T_q"], s["n_h"], s["pages"]
    q = torch.cat([s["q_abs"], s["q_r"]], -1).float() * SCALE                    # (n_tok, n_h, 576)
    prefix = s["pool"][s["shared"].long()].reshape(-1, D_C + D_R).float()
    table = s["table"][:, pages:].long()
    rows = s["pool"][table].reshape(B, -1, D_C + D_R).float()                    # each sequence's own rows, with stale ones
    a = q.reshape(-1, D_C + D_R) @ prefix.T                                      # every row against the shared keys
    b = torch.bmm(q.reshape(B, T_q * n_h, D_C + D_R), rows.transpose(1, 2)).view(B, T_q, n_h, -1)
    limit = s["lens"].long()[:, None] - PAGE * pages - T_q + torch.arange(T_q, device=DEV)   # last own key each token sees
    seen = torch.arange(rows.shape[1], device=DEV) <= limit[:, :, None]
    b = b.masked_fill(~seen[:, :, None, :], float("-inf")).view(a.shape[0], -1)
    top = torch.maximum(a.amax(1), b.amax(1))[:, None]
    a, b = torch.exp(a - top), torch.exp(b - top)
    total = a.sum(1, keepdim=True) + b.sum(1, keepdim=True)
    o = a @ prefix[:, :D_C] + torch.bmm(b.view(B, T_q * n_h, -1), rows[:, :, :D_C]).view(a.shape[0], D_C)
    lse = (top + torch.log(total)).view(B * T_q, n_h)
    return {"latent": (o / total).view(B * T_q, n_h, D_C).bfloat16(), "lse": lse}


def _plain_quantize(y):
    """Codes and scale of each row: round(127 y / amax), amax / 127."""
    amax = y.abs().amax(1, keepdim=True)
    codes = torch.where(amax > 0, torch.round(127.0 * y / amax), torch.zeros_like(y))
    return codes, amax / 127.0


def _plain_product(codes, scale, w8, sw):
    return ((codes @ w8.float().T) * scale * sw).bfloat16()


def _plain_linear(s):
    return {"out": _plain_product(*_plain_quantize(s["x"].float()), s["w8"], s["sw"])}


def _plain_norm(s):
    x = s["u"].float()
    if s["post"]:
        x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * s["w_post"].float()
    if s["gate"] is not None:
        x = x * s["gate"].float()
    if s["residual"]:
        x = s["res"].float() + s["alpha"] * x
    y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * s["w_pre"].float()
    got = {"res": x.bfloat16()} if s["residual"] else {}
    if s["to"] == "bf16":
        got["y"] = y.bfloat16()
    else:
        got["out"] = _plain_product(*_plain_quantize(y), s["w8"], s["sw"])
    return got


def _plain_append(s):
    n_tok = s["B"] * s["T_q"]
    kv = s["kv"].float()
    c, k = kv[:, :D_C], kv[:, D_C:]
    c = c * torch.rsqrt((c * c).mean(1, keepdim=True) + EPS) * s["w"].float()
    pos = s["pos"].long()
    h = D_R // 2
    cos, sin = s["rope"][pos, :h], s["rope"][pos, h:]
    turn = lambda x, co, si: torch.cat([x[..., :h] * co - x[..., h:] * si, x[..., h:] * co + x[..., :h] * si], -1)  # noqa: E731
    row = torch.cat([c, turn(k, cos, sin)], 1).bfloat16()
    seq = torch.arange(n_tok, device=DEV) // s["T_q"]
    block = s["table"][seq, pos // PAGE].long()
    s["pool"].view(-1, D_C + D_R)[block * PAGE + pos % PAGE] = row
    q = s["q"].float()
    return {"pool": s["pool"], "q_c": q[:, :, :D_H].bfloat16(),
            "q_r": turn(q[:, :, D_H:], cos[:, None], sin[:, None]).bfloat16()}


_PLAIN = {"shared": _plain_shared, "linear": _plain_linear, "norm": _plain_norm, "append": _plain_append}


def _own_shared(s):
    from mla_latent_kv_38_b200 import binding as M
    if "ws" not in s:   # kept by the program from step to step
        s["cfg"] = M.MlaConfig(s["n_h"], D_C, D_H, D_R)
        s["ws"] = torch.empty(M.mla_decode_shared_workspace_bytes(s["cfg"], s["B"], s["T_q"]), dtype=torch.uint8, device=DEV)
    pool, table = s["pool"], s["table"]
    M.mla_decode_shared(s["cfg"], s["q_abs"], s["q_r"], pool, pool.shape[0], s["shared"], s["pages"], table, table.shape[1],
                        s["lens"], s["B"], s["T_q"], 0, s["ws"], s["ws"].numel(), s["latent"], s["lse"])
    return {"latent": s["latent"], "lse": s["lse"]}


def _own_linear(s):
    from mla_latent_kv_38_b200 import binding as M
    n_tok, d_in, d_out = s["n_tok"], s["d_in"], s["d_out"]
    M.mla_quantize_i8(s["x"], d_in, n_tok, d_in, s["x8"], s["sx"])
    M.mla_linear_i8(s["x8"], d_in, s["sx"], s["w8"], s["sw"], s["out"], n_tok, d_in, d_out)
    return {"out": s["out"]}


def _own_norm(s):
    from mla_latent_kv_38_b200 import binding as M
    d, bf16 = s["d"], s["to"] == "bf16"
    M.mla_block_norm(s["u"], d, s["w_post"] if s["post"] else None, s["gate"],
                     d if s["gate"] is not None and s["gate"].dim() == 2 else 0, s["alpha"], s["res"] if s["residual"] else None,
                     s["res_out"] if s["residual"] else None, s["w_pre"], EPS, s["n_tok"], d,
                     s["y"] if bf16 else None, None if bf16 else s["y8"], None if bf16 else s["sy"])
    got = {"res": s["res_out"]} if s["residual"] else {}
    if bf16:
        got["y"] = s["y"]
    else:
        M.mla_linear_i8(s["y8"], d, s["sy"], s["w8"], s["sw"], s["out"], s["n_tok"], d, D_CQ + D_C + D_R)
        got["out"] = s["out"]
    return got


def _own_append(s):
    from mla_latent_kv_38_b200 import binding as M
    if "cfg" not in s:
        s["cfg"] = M.MlaConfig(s["n_h"], D_C, D_H, D_R)
    pool, table = s["pool"], s["table"]
    M.mla_norm_rope_append(s["cfg"], s["q"], s["kv"], s["kv"].stride(0), s["w"], EPS, s["pos"], s["rope"], s["rope"].shape[0],
                           table, table.shape[1], pool, pool.shape[0], s["B"], s["T_q"], s["q_c"], s["q_r"])
    return {"pool": pool, "q_c": s["q_c"], "q_r": s["q_r"]}


_OWN = {"shared": _own_shared, "linear": _own_linear, "norm": _own_norm, "append": _own_append}


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its values in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    """Each input read once, each output written once; a multiplication and an addition per product term."""
    op = case["op"]
    if op == "shared":
        n, P = case["B"] * case["T_q"], PAGE * case["pages"]
        own_keys = case["B"] * (case["T_q"] + case["own_max"]) / 2.0         # the lengths' mean: they are drawn evenly
        rows = n * case["n_h"]
        seen = rows * (P + own_keys / case["B"] - (case["T_q"] - 1) / 2.0)
        return {"bytes": (P + own_keys) * 2 * (D_C + D_R) + rows * (2 * (D_C + D_R) + 2 * D_C + 4),
                "flops": seen * (2 * (D_C + D_R) + 2 * D_C)}
    if op == "linear":
        n, i, o = case["n_tok"], case["d_in"], case["d_out"]
        return {"bytes": 2 * n * i + i * o + 4 * o + 2 * n * o, "flops": 2 * n * i * o + 2 * n * i}
    if op == "norm":
        n, d = case["n_tok"], case["d"]
        rows = 1 + (2 if case["residual"] else 0) + (1 if case["gate"] == "rows" else 0) + (1 if case["to"] == "bf16" else 0)
        vectors = 1 + (1 if case["post"] else 0) + (1 if case["gate"] == "vector" else 0)
        w = {"bytes": 2 * n * d * rows + 2 * d * vectors, "flops": 12 * n * d}
        if case["to"] == "linear":
            o = D_CQ + D_C + D_R
            w = {"bytes": w["bytes"] + d * o + 4 * o + 2 * n * o, "flops": w["flops"] + 2 * n * d * o}
        return w
    n = case["B"] * case["T_q"]
    row, query = D_C + D_R, case["n_h"] * (D_H + D_R)
    return {"bytes": 4 * n * (row + query) + n * (4 + 4 * D_R + 4) + 2 * D_C, "flops": n * (5 * D_C + 3 * D_R + 3 * case["n_h"] * D_R)}


def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s)


def _exact_shared(s):
    """Sequence by sequence: all its keys in order, the shared ones in front, then one softmax."""
    T_q, n_h, pages = s["T_q"], s["n_h"], s["pages"]
    latent = torch.empty(s["B"], T_q, n_h, D_C, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["B"], T_q, n_h, dtype=torch.float64, device=DEV)
    lens = s["lens"].tolist()
    for b in range(s["B"]):
        blocks = s["table"][b, :(lens[b] + PAGE - 1) // PAGE].long()
        keys = s["pool"][blocks].double().reshape(-1, D_C + D_R)[:lens[b]]
        qa = s["q_abs"].view(s["B"], T_q, n_h, D_C)[b].double()
        qr = s["q_r"].view(s["B"], T_q, n_h, D_R)[b].double()
        for t in range(T_q):
            see = keys[:lens[b] - T_q + t + 1]
            score = (qa[t] @ see[:, :D_C].T + qr[t] @ see[:, D_C:].T) / math.sqrt(D_H + D_R)
            lse[b, t] = torch.logsumexp(score, 1)
            latent[b, t] = torch.exp(score - lse[b, t][:, None]) @ see[:, :D_C]
    return {"latent": latent.view(-1, n_h, D_C), "lse": lse.view(-1, n_h)}


def _exact_quantized(y):
    peak = y.abs().max(1, keepdim=True).values
    return torch.round(y * 127 / peak.clamp(min=1e-300)) * peak / 127


def _exact_product(y, w8, sw):
    return _exact_quantized(y) @ (w8.double() * sw.double()[:, None]).T


def _exact_linear(s):
    return {"out": _exact_product(s["x"].double(), s["w8"], s["sw"])}


def _exact_norm(s):
    unit = lambda v: v / torch.sqrt(torch.sum(v * v, 1, keepdim=True) / v.shape[1] + EPS)  # noqa: E731
    v = s["u"].double()
    if s["post"]:
        v = unit(v) * s["w_post"].double()
    if s["gate"] is not None:
        v = s["gate"].double() * v
    got = {}
    if s["residual"]:
        v = s["alpha"] * v + s["res"].double()
        got["res"] = v
    v = unit(v) * s["w_pre"].double()
    got["y" if s["to"] == "bf16" else "out"] = v if s["to"] == "bf16" else _exact_product(v, s["w8"], s["sw"])
    return got


def _exact_append(s):
    """Each token's key turned as a complex number by its position's angle."""
    tab = s["rope"].double()[s["pos"].long()]
    turn = torch.complex(tab[:, :D_R // 2], tab[:, D_R // 2:])

    def rotated(x, by):
        z = torch.complex(x[..., :D_R // 2].contiguous(), x[..., D_R // 2:].contiguous()) * by
        return torch.cat([z.real, z.imag], -1)

    kv = s["kv"].double()
    c = kv[:, :D_C]
    c = c * s["w"].double() / torch.sqrt((c ** 2).sum(1, keepdim=True) / D_C + EPS)
    pool = s["pool"].double()
    at, table, T_q = s["pos"].tolist(), s["table"].tolist(), s["T_q"]
    block = torch.tensor([table[i // T_q][p // PAGE] for i, p in enumerate(at)], device=DEV)
    slot = torch.tensor([p % PAGE for p in at], device=DEV)
    pool[block, slot] = torch.cat([c, rotated(kv[:, D_C:], turn)], 1)
    q = s["q"].double()
    return {"pool": pool, "q_c": q[..., :D_H], "q_r": rotated(q[..., D_H:], turn[:, None])}


_EXACT = {"shared": _exact_shared, "linear": _exact_linear, "norm": _exact_norm, "append": _exact_append}

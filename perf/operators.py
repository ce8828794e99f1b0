"""The attention operators of a serving step, as measurable cases.

Two operators that a layer runs between its query/key/value projection and its experts:

  append  norms of queries and keys per head, the rotation by position, and keys and values written into a
          paged cache, from the rows of the fused projection;
  attend  causal attention of a ragged batch of new tokens (one per sequence, a few, or a chunk) over that
          paged cache, grouped heads, with the log-sum-exp of every row.

A token of sequence b with q_len[b] new tokens and kv_len[b] tokens in all (the new ones among them) sits at
position kv_len[b] - q_len[b] + i; position p of sequence b is row p % page of page block_table[b][p // page].
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one request, one token: the shortest call there is; pairs next to each other, the whole head rotated
        dict(name="append_t1", op="append", dtype="fp16", seqs=1, chunks=0, chunk=0, dec=1, ctx=500, ragged=False, idle=0,
             hq=32, hkv=8, d=128, page=16, order="token", rot=128, inter=True, norm=False, mix=1),
        # four concurrent requests, the decode batch of the 2048-wide layer: head norms, a quarter of the head rotated
        dict(name="append_t4", op="append", dtype="bf16", seqs=4, chunks=0, chunk=0, dec=1, ctx=4096, ragged=True, idle=0,
             hq=16, hkv=2, d=256, page=64, order="token", rot=64, inter=False, norm=True, mix=2),
        # two odd chunks of a 4096-wide layer next to decoding requests, head-major pages
        dict(name="append_t2048_mixed", op="append", dtype="fp16", seqs=16, chunks=2, chunk=1017, dec=1, ctx=2000, ragged=True, idle=0,
             hq=32, hkv=8, d=128, page=16, order="head", rot=128, inter=True, norm=False, mix=3),
        # the prefill chunk of the 2048-wide layer
        dict(name="append_t8192", op="append", dtype="bf16", seqs=1, chunks=1, chunk=8192, dec=1, ctx=8192, ragged=False, idle=0,
             hq=16, hkv=2, d=256, page=64, order="token", rot=64, inter=False, norm=True, mix=4),
        # one request with a short context: latency alone
        dict(name="attend_t1", op="attend", dtype="bf16", seqs=1, chunks=0, chunk=0, dec=1, ctx=500, ragged=False, idle=0,
             hq=32, hkv=8, d=128, page=16, order="token", window=0, mix=5),
        # four concurrent requests of the 2048-wide layer
        dict(name="attend_t4", op="attend", dtype="bf16", seqs=4, chunks=0, chunk=0, dec=1, ctx=4096, ragged=True, idle=0,
             hq=16, hkv=2, d=256, page=64, order="token", window=0, mix=6),
        # four requests with two draft tokens each to verify
        dict(name="attend_verify_t12", op="attend", dtype="bf16", seqs=4, chunks=0, chunk=0, dec=3, ctx=16384, ragged=True, idle=0,
             hq=16, hkv=2, d=256, page=64, order="token", window=0, mix=7),
        # a full decode batch with contexts from a few tokens to 16384, three of its slots idle (no context at all)
        dict(name="attend_decode_b64", op="attend", dtype="fp16", seqs=64, chunks=0, chunk=0, dec=1, ctx=16384, ragged=True, idle=3,
             hq=32, hkv=8, d=128, page=32, order="head", window=0, mix=8),
        # one request with a long context: the work of a few rows has to fill the GPU
        dict(name="attend_decode_131072", op="attend", dtype="bf16", seqs=1, chunks=0, chunk=0, dec=1, ctx=131071, ragged=False, idle=0,
             hq=32, hkv=8, d=128, page=16, order="token", window=0, mix=9),
        # a chunk of a prompt at 8000 tokens, with decoding requests in the same call
        dict(name="attend_chunk_mixed", op="attend", dtype="bf16", seqs=9, chunks=1, chunk=509, dec=1, ctx=8192, ragged=False, idle=0,
             hq=32, hkv=8, d=128, page=16, order="token", window=0, mix=10),
        # two prompts of odd lengths through a layer with a sliding window and small heads
        dict(name="attend_window_2x1999", op="attend", dtype="fp16", seqs=2, chunks=2, chunk=1999, dec=1, ctx=1999, ragged=True, idle=0,
             hq=16, hkv=4, d=64, page=32, order="head", window=1000, mix=11),
        # the prefill chunk of the 2048-wide layer
        dict(name="attend_prefill_t8192", op="attend", dtype="bf16", seqs=1, chunks=1, chunk=8192, dec=1, ctx=8192, ragged=False, idle=0,
             hq=16, hkv=2, d=256, page=64, order="token", window=0, mix=12),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8, 16])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), hq=hkv * group, hkv=hkv, d=rng.choice([64, 96, 128, 256]),
             page=rng.choice([8, 16, 24, 32, 64, 128]), order=rng.choice(["token", "head"]), ragged=rng.random() < 0.7, idle=0,
             mix=rng.randrange(1 << 20))
    if c["hq"] > 40:
        c["hq"] = 5 * hkv
    kind = rng.choice(["decode", "decode", "verify", "chunk", "mixed"])
    if kind in ("decode", "verify"):
        c.update(seqs=log_int(rng, 1, 64), chunks=0, chunk=0, dec=1 if kind == "decode" else rng.randint(2, 8))
        c["idle"] = 1 if c["seqs"] > 3 and rng.random() < 0.5 else 0
        c["ctx"] = log_int(rng, 16, min(131072, max(16, 500_000 // c["seqs"])))
    else:
        c.update(seqs=log_int(rng, 1, 4), chunk=log_int(rng, 9, 4096), dec=1)
        c["chunks"] = c["seqs"]
        if kind == "mixed":
            c["seqs"] += log_int(rng, 1, 8)
        # the plain form holds every row's scores: its room bounds the context
        room = int(6e8 / (c["seqs"] * c["chunk"] * c["hq"]))
        if room < c["chunk"]:
            c["chunk"] = max(9, int(math.sqrt(6e8 / (c["seqs"] * c["hq"]))))
            room = c["chunk"]
        c["ctx"] = log_int(rng, c["chunk"], max(c["chunk"], min(32768, room)))
    if op == "append":
        c["rot"] = rng.choice([c["d"], c["d"] // 2, c["d"] // 4])
        c.update(inter=rng.random() < 0.5, norm=rng.random() < 0.5)
    else:
        c["window"] = rng.choice([0, 0, log_int(rng, 16, 4096)])
    return c


def lengths(c):
    """(q_len, kv_len) of every sequence: of the case alone."""
    rng = random.Random(c["mix"])
    q, kv = [], []
    for b in range(c["seqs"]):
        n = c["chunk"] if b < c["chunks"] else c["dec"]
        if c["ragged"] and b and b < c["chunks"]:
            n = max(1, n - rng.randrange(1 + n // 3))
        total = max(n, c["ctx"])
        if c["ragged"]:
            total = max(n, log_int(rng, max(n, 1 + total // 16), total))
        q.append(n)
        kv.append(total)
    for b in rng.sample(range(c["seqs"]), c["idle"]):
        kv[b] = 0
    return q, kv


def visible(c):
    """Query-key pairs of one head, and the cache rows that they touch."""
    pairs = rows = 0
    for n, total in zip(*lengths(c)):
        w = c.get("window") or 1 << 40
        first = None
        for i in range(n):
            p = total - n + i
            if p >= 0:
                pairs += min(p + 1, w)
                first = max(0, p + 1 - w) if first is None else first
        rows += 0 if first is None else total - first
    return pairs, rows


def work(c):
    q, kv = lengths(c)
    tokens, heads = sum(q), c["hq"] + 2 * c["hkv"]
    if c["op"] == "append":
        moved = 2 * tokens * heads * c["d"] * 2 + tokens * c["rot"] * 4
        return {"bytes": moved, "flops": tokens * (heads * c["d"] * (4 if c["norm"] else 0) + (c["hq"] + c["hkv"]) * c["rot"] * 3)}
    pairs, rows = visible(c)
    return {"bytes": rows * c["hkv"] * c["d"] * 4 + tokens * c["hq"] * (c["d"] * 4 + 4), "flops": 4 * pairs * c["hq"] * c["d"]}


# ------------------------------------------------------------------------------------------------ inputs
def inputs(c, seed):
    """What both operators share: the batch, its pages in no order, and a cache that holds the context already."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + c["mix"])
    dt = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dt)

    q_len, kv_len = lengths(c)
    page = c["page"]
    width = max(1, -(-max(kv_len) // page)) + 1  # room to grow by a page
    pages = sum(-(-n // page) for n in kv_len) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(c["seqs"], width, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(kv_len):
        need = -(-n // page)
        table[b, :need] = order[at:at + need]
        at += need

    def cache():
        if c["order"] == "token":
            return normal(pages, page, c["hkv"], c["d"])
        return normal(pages, c["hkv"], page, c["d"]).permute(0, 2, 1, 3)

    start = [0]
    for n in q_len:
        start.append(start[-1] + n)
    s = dict(c=c, k_cache=cache(), v_cache=cache(), table=table, max_q=max(q_len),
             q_start=torch.tensor(start, dtype=torch.int32, device=DEV), kv_len=torch.tensor(kv_len, dtype=torch.int32, device=DEV))
    tokens = start[-1]
    if c["op"] == "append":
        # the rows of the fused projection: queries, keys and values side by side
        qkv = normal(tokens, c["hq"] + 2 * c["hkv"], c["d"])
        s["q"], s["k"], s["v"] = qkv.split([c["hq"], c["hkv"], c["hkv"]], dim=1)
        inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        angle = torch.arange(width * page, device=DEV, dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()  # [positions, rot]: cosines, then sines
        if c["norm"]:  # weights around one, held as their distance from it
            s["q_weight"], s["k_weight"] = (torch.randn(c["d"], generator=g, device=DEV) * 0.1 for _ in range(2))
        s["q_out"] = torch.empty(tokens, c["hq"], c["d"], dtype=dt, device=DEV)
    else:
        # queries and keys have unit size for each component: some rows attend widely, some to a few places
        s["q"] = (normal(tokens, c["hq"], c["d"]).float() * (0.5 + 2.5 * torch.rand(1, c["hq"], 1, generator=g, device=DEV))).to(dt)
        s["scale"] = c["d"] ** -0.5
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(tokens, c["hq"], dtype=torch.float32, device=DEV)
    return s


def prepare(case, seed):
    s = inputs(case, seed)
    if own:  # the handle of the cache and its batch, and the workspace that goes with it
        from bit_moe_expert_router_gb300 import attention
        s["attention"] = attention
        s["batch"] = attention.KVBatch(s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["kv_len"], n_q_heads=case["hq"],
                                       max_q_len=s["max_q"])
        if case["op"] == "append":
            s["prep"] = attention.HeadPrep(s["cos_sin"], interleaved=case["inter"], q_weight=s.get("q_weight"),
                                           k_weight=s.get("k_weight"), eps=EPS, weight_offset=1.0)
        else:
            s["workspace"] = s["batch"].alloc_workspace()
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        attention = s["attention"]
        if s["c"]["op"] == "append":
            attention.moe_w4a8_kv_append(s["batch"], s["prep"], s["q"], s["k"], s["v"], s["q_out"])
            return [s["q_out"], s["k_cache"], s["v_cache"]]
        attention.moe_w4a8_paged_attention(s["batch"], s["q"], s["out"], s["lse"], scale=s["scale"], window=s["c"]["window"],
                                           workspace=s["workspace"])
        return [s["out"], s["lse"]]
    return plain_append(s) if s["c"]["op"] == "append" else plain_attend(s)


def plain_heads(x, weight, cos, sin, inter):
    """x [tokens, heads, d] in 32 bits: the norm of each head, then the rotation of its first part."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (weight + 1.0)
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if inter else (x[..., :half], x[..., half:2 * half])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y, z], dim=-1).flatten(-2) if inter else torch.cat([y, z], dim=-1)
    return torch.cat([turned, x[..., 2 * half:]], dim=-1)


def plain_append(s):
    c, dt = s["c"], s["q"].dtype
    token = torch.arange(s["q"].shape[0], device=DEV)
    seq = (token[:, None] >= s["q_start"][None, 1:]).sum(1)
    pos = (s["kv_len"][seq] - s["q_start"][seq + 1] + token).long()
    kept = pos >= 0
    at = pos.clamp_min(0)
    cs = s["cos_sin"][at][:, None, :]
    cos, sin = cs[..., :c["rot"] // 2], cs[..., c["rot"] // 2:]
    q = plain_heads(s["q"].float(), s.get("q_weight"), cos, sin, c["inter"])
    k = plain_heads(s["k"].float(), s.get("k_weight"), cos, sin, c["inter"])
    q = torch.where(kept[:, None, None], q, torch.zeros_like(q)).to(dt)
    page, row = s["table"][seq, at // c["page"]].long(), at % c["page"]
    page = torch.where(kept, page, s["k_cache"].shape[0] - 1)
    keep = kept[:, None, None]
    s["k_cache"][page, row] = torch.where(keep, k.to(dt), s["k_cache"][page, row])
    s["v_cache"][page, row] = torch.where(keep, s["v"], s["v_cache"][page, row])
    return [q, s["k_cache"], s["v_cache"]]


def plain_attend(s):
    c, dt = s["c"], s["q"].dtype
    b, hkv, g, d = c["seqs"], c["hkv"], c["hq"] // c["hkv"], c["d"]
    pages = s["table"].long()
    k = s["k_cache"][pages].reshape(b, -1, hkv, d).float()
    v = s["v_cache"][pages].reshape(b, -1, hkv, d).float()
    step = torch.arange(s["max_q"], device=DEV)
    q_len = s["q_start"][1:] - s["q_start"][:-1]
    live = step[None] < q_len[:, None]
    token = (s["q_start"][:-1, None] + step).clamp_max(s["q"].shape[0] - 1).long()
    q = s["q"][token].float().reshape(b, -1, hkv, g, d)
    pos = (s["kv_len"] - q_len)[:, None] + step
    key = torch.arange(k.shape[1], device=DEV)
    seen = key <= pos[..., None]
    if c["window"]:
        seen = seen & (key > pos[..., None] - c["window"])
    x = torch.matmul(q.permute(0, 2, 3, 1, 4), k.permute(0, 2, 3, 1)[:, :, None]) * s["scale"]  # [b, hkv, g, q, key]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    y = torch.matmul(x, v.permute(0, 2, 1, 3)[:, :, None]) / torch.where(total == 0, torch.ones_like(total), total)
    lse = torch.log(total) + top
    y, lse = y.permute(0, 3, 1, 2, 4).reshape(b, -1, c["hq"], d), lse.permute(0, 3, 1, 2, 4).reshape(b, -1, c["hq"])
    return [y[live].to(dt), lse[live]]


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    c, s = case, inputs(case, seed)
    q_len, kv_len = lengths(c)
    page, group, start = c["page"], c["hq"] // c["hkv"], 0
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    table = s["table"].tolist()
    q_all = s["q"].double()
    if c["op"] == "append":
        q_out = torch.zeros(sum(q_len), c["hq"], c["d"], dtype=torch.float64, device=DEV)
        half = c["rot"] // 2
        # the angles as complex numbers of the stored cosines and sines
        turn = torch.complex(s["cos_sin"][:, :half].double(), s["cos_sin"][:, half:].double())

        def head(x, weight, where):
            if weight is not None:
                size = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / c["d"]
                x = x / torch.sqrt(size + EPS) * (1.0 + weight.double())
            x = x.clone()
            part = x[..., :c["rot"]].unflatten(-1, (half, 2) if c["inter"] else (2, half)).movedim(-1 if c["inter"] else -2, 0)
            z = torch.complex(part[0].contiguous(), part[1].contiguous()) * turn[where][:, None]
            if c["inter"]:
                x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2] = z.real, z.imag
            else:
                x[..., :half], x[..., half:c["rot"]] = z.real, z.imag
            return x

        for b, (n, total) in enumerate(zip(q_len, kv_len)):
            skip = max(0, n - total)  # tokens before position zero
            rows = slice(start + skip, start + n)
            start += n
            if skip == n:
                continue
            where = torch.arange(total - n + skip, total, device=DEV)
            q_out[rows] = head(q_all[rows], s.get("q_weight"), where)
            pages = torch.tensor([table[b][p // page] for p in where.tolist()], device=DEV)
            k_cache[pages, where % page] = head(s["k"][rows].double(), s.get("k_weight"), where)
            v_cache[pages, where % page] = s["v"][rows].double()
        return [q_out, k_cache, v_cache]
    out = torch.zeros(sum(q_len), c["hq"], c["d"], dtype=torch.float64, device=DEV)
    lse = torch.full((sum(q_len), c["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    for b, (n, total) in enumerate(zip(q_len, kv_len)):
        first, start = start, start + n
        if total == 0:
            continue
        ids = torch.tensor(table[b][:-(-total // page)], device=DEV)
        keys = k_cache[ids].flatten(0, 1)[:total]
        values = v_cache[ids].flatten(0, 1)[:total]
        for h in range(c["hq"]):
            kh, vh = keys[:, h // group].T.contiguous(), values[:, h // group].contiguous()
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                at = total - n + i + torch.arange(m, device=DEV)[:, None]
                hi = min(total, total - n + i + m)
                lo = max(0, total - n + i + 1 - c["window"]) if c["window"] else 0
                if hi <= lo:
                    continue
                key = torch.arange(lo, hi, device=DEV)[None]
                hidden = key > at
                if c["window"]:
                    hidden |= at - key >= c["window"]
                x = (q_all[first + i:first + i + m, h] @ kh[:, lo:hi]) * s["scale"]
                x[hidden] = -math.inf
                z = torch.logsumexp(x, dim=1)
                lse[first + i:first + i + m, h] = z
                out[first + i:first + i + m, h] = torch.nan_to_num(torch.exp(x - z[:, None])) @ vh[lo:hi]
    return [out, lse]

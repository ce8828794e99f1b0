"""The operators of a serving layer with latent attention and scored routing, as measurable cases.

Three operators that such a layer runs between its projections and its experts:

  append  the norm of a token's latent vector, the rotation by position of the key part that all heads share and of every
          head's query part, and latent and key part written as one row of a paged cache;
  attend  causal attention of a ragged batch of new tokens over that paged cache in the absorbed form: every head's query
          is as wide as a row, a row is the key of all heads and its latent part is their value; with the log-sum-exp;
  route   scores of the experts (softmax or sigmoid of the router's logits), a bias that moves the choice but not the
          weights, groups of experts of which some are kept, the best experts with their weights.

A token of sequence b with q_len[b] new tokens and kv_len[b] tokens in all (the new ones among them) sits at
position kv_len[b] - q_len[b] + i; position p of sequence b is row p % page of page block_table[b][p // page].
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
NOPE = 128  # components of a projected query head that are not rotated: the rows that the rotated parts are taken from


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one request, one token of a layer of few heads: the shortest call there is; neighbours rotated
        dict(name="append_t1", op="append", dtype="fp16", seqs=1, chunks=0, chunk=0, dec=1, ctx=500, ragged=False, idle=0,
             h=16, dc=512, rot=64, page=16, inter=True, norm=True, mix=1),
        # a full decode batch of a layer of many heads, some of its slots idle
        dict(name="append_t64", op="append", dtype="bf16", seqs=64, chunks=0, chunk=0, dec=1, ctx=2048, ragged=True, idle=3,
             h=128, dc=512, rot=64, page=64, inter=True, norm=True, mix=2),
        # two odd chunks of prompts next to decoding requests; halves rotated, a smaller latent, no norm
        dict(name="append_t2042_mixed", op="append", dtype="fp16", seqs=10, chunks=2, chunk=1017, dec=1, ctx=2000, ragged=False, idle=0,
             h=32, dc=256, rot=32, page=32, inter=False, norm=False, mix=3),
        # the prefill chunk
        dict(name="append_t8192", op="append", dtype="bf16", seqs=1, chunks=1, chunk=8192, dec=1, ctx=8192, ragged=False, idle=0,
             h=16, dc=512, rot=64, page=64, inter=True, norm=True, mix=4),
        # one request with a short context: latency alone
        dict(name="attend_t1", op="attend", dtype="bf16", seqs=1, chunks=0, chunk=0, dec=1, ctx=500, ragged=False, idle=0,
             h=16, dc=512, rot=64, page=16, mix=5),
        # four requests with two draft tokens each to verify
        dict(name="attend_verify_t12", op="attend", dtype="fp16", seqs=4, chunks=0, chunk=0, dec=3, ctx=16384, ragged=True, idle=0,
             h=16, dc=512, rot=64, page=32, mix=6),
        # a full decode batch of many heads with contexts from a few tokens to 16384, three of its slots idle (no context at all)
        dict(name="attend_decode_b64", op="attend", dtype="bf16", seqs=64, chunks=0, chunk=0, dec=1, ctx=16384, ragged=True, idle=3,
             h=128, dc=512, rot=64, page=64, mix=7),
        # one request with a long context: the work of a few rows has to fill the GPU
        dict(name="attend_decode_131072", op="attend", dtype="bf16", seqs=1, chunks=0, chunk=0, dec=1, ctx=131071, ragged=False, idle=0,
             h=32, dc=512, rot=64, page=64, mix=8),
        # an odd chunk of a prompt at 8000 tokens, with decoding requests in the same call
        dict(name="attend_chunk_mixed", op="attend", dtype="bf16", seqs=9, chunks=1, chunk=509, dec=1, ctx=8192, ragged=False, idle=0,
             h=32, dc=512, rot=64, page=64, mix=9),
        # four requests' next token among 512 experts, ten of them picked
        dict(name="route_t4", op="route", dtype="fp32", t=4, e=512, k=10, score="sigmoid", bias=True, groups=1, kept=1, top=1, renorm=True,
             scale=1.0, mix=10),
        # a decode batch whose router leaves 16-bit logits: softmax scores, groups by their best expert, weights as they are
        dict(name="route_t64", op="route", dtype="bf16", t=64, e=160, k=6, score="softmax", bias=False, groups=8, kept=3, top=1, renorm=False,
             scale=16.0, mix=11),
        # the prefill chunk: sigmoid scores, a bias, groups by the sum of their two best experts
        dict(name="route_t8192", op="route", dtype="fp32", t=8192, e=256, k=8, score="sigmoid", bias=True, groups=8, kept=4, top=2, renorm=True,
             scale=2.5, mix=12),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "route"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        e = groups * max(4, log_int(rng, 16, 512) // groups)
        kept = groups if groups == 1 else rng.randint(1, groups)
        c = dict(op=op, dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]), t=log_int(rng, 1, 8192), e=e, k=rng.randint(1, min(10, kept * (e // groups))),
                 score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, groups=groups, kept=kept, top=rng.choice([1, 2]),
                 renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5, 16.0]), mix=rng.randrange(1 << 20))
        return c
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), h=rng.choice([1, 5, 8, 16, 20, 32, 48, 64, 128]), dc=rng.choice([128, 256, 384, 448, 512]),
             rot=rng.choice([32, 64]), page=rng.choice([8, 16, 24, 32, 64, 128]), ragged=rng.random() < 0.7, idle=0, mix=rng.randrange(1 << 20))
    kind = rng.choice(["decode", "decode", "verify", "chunk", "mixed"])
    if kind in ("decode", "verify"):
        c.update(seqs=log_int(rng, 1, 64), chunks=0, chunk=0, dec=1 if kind == "decode" else rng.randint(2, 8))
        c["idle"] = 1 if c["seqs"] > 3 and rng.random() < 0.5 else 0
        c["ctx"] = log_int(rng, 16, min(131072, 400_000 // c["seqs"], max(16, int(4e7 / (c["seqs"] * c["dec"] * c["h"])))))
    else:
        c.update(seqs=log_int(rng, 1, 4), chunk=log_int(rng, 9, 2048), dec=1)
        c["chunks"] = c["seqs"]
        if kind == "mixed":
            c["seqs"] += log_int(rng, 1, 8)
        # the plain form holds every row's scores: its room bounds the context
        room = int(1.2e8 / (c["seqs"] * c["chunk"] * c["h"]))
        if room < c["chunk"]:
            c["chunk"] = max(9, int(math.sqrt(1.2e8 / (c["seqs"] * c["h"]))))
            room = c["chunk"]
        c["ctx"] = log_int(rng, c["chunk"], max(c["chunk"], min(32768, room)))
    if op == "append":
        c.update(inter=rng.random() < 0.5, norm=rng.random() < 0.7)
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
        if total:
            pairs += sum(max(0, total - n + i + 1) for i in range(n))
            rows += total
    return pairs, rows


def work(c):
    if c["op"] == "route":
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": c["t"] * (c["e"] * size + c["k"] * 8) + (c["e"] * 4 if c["bias"] else 0), "flops": c["t"] * c["e"] * 8}
    tokens, row = sum(lengths(c)[0]), c["dc"] + c["rot"]
    if c["op"] == "append":
        moved = tokens * (row + c["h"] * c["rot"]) * 2 * 2 + tokens * c["rot"] * 4
        return {"bytes": moved, "flops": tokens * (c["dc"] * (4 if c["norm"] else 0) + (c["h"] + 1) * c["rot"] * 3)}
    pairs, rows = visible(c)
    return {"bytes": rows * row * 2 + tokens * c["h"] * ((row + c["dc"]) * 2 + 4), "flops": 2 * pairs * c["h"] * (row + c["dc"])}


# ------------------------------------------------------------------------------------------------ inputs
def inputs(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + c["mix"])
    dt = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)

    if c["op"] == "route":
        s = dict(c=c, logits=(normal(c["t"], c["e"]) * 1.5).to(dt), ids=torch.empty(c["t"], c["k"], dtype=torch.int32, device=DEV),
                 w=torch.empty(c["t"], c["k"], dtype=torch.float32, device=DEV))
        # a bias of the size that balancing steps leave behind
        s["bias"] = normal(c["e"]) * (0.05 if c["score"] == "sigmoid" else 0.2 / c["e"]) if c["bias"] else None
        return s
    q_len, kv_len = lengths(c)
    page, row = c["page"], c["dc"] + c["rot"]
    width = max(1, -(-max(kv_len) // page)) + 1  # room to grow by a page
    pages = sum(-(-n // page) for n in kv_len) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)  # pages in no order
    table = torch.zeros(c["seqs"], width, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(kv_len):
        need = -(-n // page)
        table[b, :need] = order[at:at + need]
        at += need
    start = [0]
    for n in q_len:
        start.append(start[-1] + n)
    s = dict(c=c, cache=normal(pages, page, row).to(dt), table=table, max_q=max(q_len),
             q_start=torch.tensor(start, dtype=torch.int32, device=DEV), kv_len=torch.tensor(kv_len, dtype=torch.int32, device=DEV))
    tokens = start[-1]
    if c["op"] == "append":
        # rows of two projections: latent and key part side by side, every query head's rotated part behind the other
        s["latent"], s["k_rot"] = (normal(tokens, row) * 2.0).to(dt).split([c["dc"], c["rot"]], dim=1)
        s["q_rot"] = normal(tokens, c["h"], NOPE + c["rot"]).to(dt)[..., NOPE:]
        inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        angle = torch.arange(width * page, device=DEV, dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()  # [positions, rot]: cosines, then sines
        s["weight"] = 1.0 + normal(c["dc"]) * 0.1 if c["norm"] else None
        # the attention's queries, whose other part is a product's: the rotated part goes into its place there
        s["q_out"] = torch.zeros(tokens, c["h"], row, dtype=dt, device=DEV)[..., c["dc"]:]
    else:
        # queries and rows have unit size for each component: some heads attend widely, some to a few places
        s["q"] = (normal(tokens, c["h"], row) * (0.5 + 2.5 * torch.rand(1, c["h"], 1, generator=g, device=DEV))).to(dt)
        s["scale"] = row ** -0.5
        s["out"] = torch.empty(tokens, c["h"], c["dc"], dtype=dt, device=DEV)
        s["lse"] = torch.empty(tokens, c["h"], dtype=torch.float32, device=DEV)
    return s


def prepare(case, seed):
    s = inputs(case, seed)
    if own:  # the rule of the router, or the handle of the cache and its batch with the workspace that goes with it
        import bit_moe_expert_router_gb300 as moe
        s["moe"] = moe
        if case["op"] == "route":
            s["rule"] = moe.RouteRule(case["e"], case["k"], score=case["score"], n_groups=case["groups"], topk_groups=case["kept"],
                                      group_top=case["top"], renormalise=case["renorm"], scale=case["scale"])
            return s
        s["batch"] = moe.LatentBatch(s["cache"], s["table"], s["q_start"], s["kv_len"], n_heads=case["h"], latent_dim=case["dc"], max_q_len=s["max_q"])
        if case["op"] == "append":
            s["prep"] = moe.HeadPrep(s["cos_sin"], interleaved=case["inter"], k_weight=s["weight"], eps=EPS)
        else:
            s["workspace"] = s["batch"].alloc_workspace()
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["c"]["op"]
    if own:
        moe = s["moe"]
        if op == "route":
            moe.moe_w4a8_route_scored(s["logits"], s["rule"], s["ids"], s["w"], bias=s["bias"])
            return [s["ids"], s["w"]]
        if op == "append":
            moe.moe_w4a8_latent_append(s["batch"], s["prep"], s["latent"], s["k_rot"], s["q_rot"], s["q_out"])
            return [s["q_out"], s["cache"]]
        moe.moe_w4a8_latent_attention(s["batch"], s["q"], s["out"], s["lse"], scale=s["scale"], workspace=s["workspace"])
        return [s["out"], s["lse"]]
    return {"route": plain_route, "append": plain_append, "attend": plain_attend}[op](s)


def plain_turn(x, cos, sin, inter):
    """The rotation of the last dimension, in 32 bits."""
    half = cos.shape[-1]
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :half], x[..., half:])
    y, z = a * cos - b * sin, b * cos + a * sin
    return torch.stack([y, z], dim=-1).flatten(-2) if inter else torch.cat([y, z], dim=-1)


def plain_append(s):
    c, dt = s["c"], s["cache"].dtype
    token = torch.arange(s["q_rot"].shape[0], device=DEV)
    seq = (token[:, None] >= s["q_start"][None, 1:]).sum(1)
    pos = (s["kv_len"][seq] - s["q_start"][seq + 1] + token).long()
    kept = pos >= 0
    at = pos.clamp_min(0)
    cos, sin = s["cos_sin"][at].split(c["rot"] // 2, dim=1)
    x = s["latent"].float()
    if c["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"]
    row = torch.cat([x, plain_turn(s["k_rot"].float(), cos, sin, c["inter"])], dim=1).to(dt)
    q = plain_turn(s["q_rot"].float(), cos[:, None], sin[:, None], c["inter"])
    q = torch.where(kept[:, None, None], q, torch.zeros_like(q)).to(dt)
    page, line = s["table"][seq, at // c["page"]].long(), at % c["page"]
    page = torch.where(kept, page, s["cache"].shape[0] - 1)
    s["cache"][page, line] = torch.where(kept[:, None], row, s["cache"][page, line])
    return [q, s["cache"]]


def plain_attend(s):
    c, dt = s["c"], s["q"].dtype
    b, h, d = c["seqs"], c["h"], c["dc"] + c["rot"]
    x = s["cache"][s["table"].long()].reshape(b, -1, d).float()  # every sequence's rows, one after another
    step = torch.arange(s["max_q"], device=DEV)
    q_len = s["q_start"][1:] - s["q_start"][:-1]
    live = step[None] < q_len[:, None]
    token = (s["q_start"][:-1, None] + step).clamp_max(s["q"].shape[0] - 1).long()
    q = s["q"][token].float().reshape(b, -1, d)  # [b, token and head, d]
    pos = (s["kv_len"] - q_len)[:, None] + step
    hidden = (torch.arange(x.shape[1], device=DEV) > pos[..., None]).repeat_interleave(h, dim=1)
    y = torch.matmul(q, x.transpose(1, 2)) * s["scale"]
    y = y.masked_fill(hidden, -math.inf)
    top = y.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    y = torch.exp(y - top)
    total = y.sum(-1, keepdim=True)
    o = torch.matmul(y, x[..., :c["dc"]]) / torch.where(total == 0, torch.ones_like(total), total)
    lse = torch.log(total) + top
    o, lse = o.reshape(b, -1, h, c["dc"]), lse.reshape(b, -1, h)
    return [o[live].to(dt), lse[live]]


def plain_route(s):
    # in 64 bits: two experts' scores can lie closer together than 32 bits tell
    c = s["c"]
    logits = s["logits"].double()
    if c["score"] == "softmax":
        score = torch.exp(logits - logits.amax(-1, keepdim=True))
        score = score / score.sum(-1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
    choice = score if s["bias"] is None else score + s["bias"].double()
    parts = choice.unflatten(1, (c["groups"], -1))
    best = parts.sort(dim=-1, descending=True).values[..., :c["top"]].sum(-1)
    order = best.sort(dim=-1, descending=True, stable=True).indices[:, :c["kept"]]
    kept = torch.zeros_like(best, dtype=torch.bool).scatter_(1, order, True)
    choice = torch.where(kept[..., None], parts, torch.full_like(parts, -math.inf)).flatten(1)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return [ids.to(torch.int32), (w * c["scale"]).float()]


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    return {"route": exact_route, "append": exact_append, "attend": exact_attend}[case["op"]](case, inputs(case, seed))


def exact_append(c, s):
    q_len, kv_len = lengths(c)
    cache, table, start, half = s["cache"].double(), s["table"].tolist(), 0, c["rot"] // 2
    q_out = torch.zeros(sum(q_len), c["h"], c["rot"], dtype=torch.float64, device=DEV)
    # the angles as complex numbers of the stored cosines and sines
    turn = torch.complex(s["cos_sin"][:, :half].double(), s["cos_sin"][:, half:].double())

    def turned(x, by):
        x = x.double().unflatten(-1, (half, 2) if c["inter"] else (2, half)).movedim(-1 if c["inter"] else -2, 0)
        z = torch.complex(x[0].contiguous(), x[1].contiguous()) * by
        return torch.stack([z.real, z.imag], dim=-1 if c["inter"] else -2).flatten(-2)

    for b, (n, total) in enumerate(zip(q_len, kv_len)):
        skip = max(0, n - total)  # tokens before position zero
        rows = slice(start + skip, start + n)
        start += n
        if skip == n:
            continue
        where = torch.arange(total - n + skip, total, device=DEV)
        x = s["latent"][rows].double()
        if c["norm"]:
            x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / c["dc"] + EPS) * s["weight"].double()
        pages = torch.tensor([table[b][p // c["page"]] for p in where.tolist()], device=DEV)
        cache[pages, where % c["page"], :c["dc"]] = x
        cache[pages, where % c["page"], c["dc"]:] = turned(s["k_rot"][rows], turn[where])
        q_out[rows] = turned(s["q_rot"][rows], turn[where][:, None])
    return [q_out, cache]


def exact_attend(c, s):
    q_len, kv_len = lengths(c)
    table, start = s["table"].tolist(), 0
    out = torch.zeros(sum(q_len), c["h"], c["dc"], dtype=torch.float64, device=DEV)
    lse = torch.full((sum(q_len), c["h"]), -math.inf, dtype=torch.float64, device=DEV)
    for b, (n, total) in enumerate(zip(q_len, kv_len)):
        first, start = start, start + n
        if total == 0:
            continue
        ids = torch.tensor(table[b][:-(-total // c["page"])], device=DEV)
        rows = s["cache"][ids].flatten(0, 1)[:total].double()
        per = max(1, (1 << 26) // (total * c["h"]))  # tokens at a time
        for i in range(max(0, n - total), n, per):
            m = min(per, n - i)
            hi = total - n + i + m
            at = hi - m + torch.arange(m, device=DEV)[:, None, None]
            q = s["q"][first + i:first + i + m].double()
            x = torch.einsum("qhd,kd->qhk", q, rows[:hi]) * s["scale"]
            x = torch.where(torch.arange(hi, device=DEV) <= at, x, -math.inf)
            z = torch.logsumexp(x, dim=-1)
            lse[first + i:first + i + m] = z
            out[first + i:first + i + m] = torch.einsum("qhk,kd->qhd", torch.exp(x - z[..., None]), rows[:hi, :c["dc"]])
    return [out, lse]


def exact_route(c, s):
    x = s["logits"].double()
    log_s = torch.log_softmax(x, -1) if c["score"] == "softmax" else -torch.logaddexp(torch.zeros_like(x), -x)
    value = torch.exp(log_s)
    r = value if s["bias"] is None else value + s["bias"].double()
    size = c["e"] // c["groups"]
    if c["groups"] > 1:
        group = torch.stack([r[:, i * size:(i + 1) * size].topk(c["top"], dim=1).values.sum(1) for i in range(c["groups"])], dim=1)
        # a group's place: how many are better, or as good and before it
        before = torch.arange(c["groups"], device=DEV)
        better = (group[:, None, :] > group[:, :, None]) | ((group[:, None, :] == group[:, :, None]) & (before[None, None, :] < before[None, :, None]))
        out_of = (better.sum(-1) >= c["kept"]).repeat_interleave(size, dim=1)
        r = r.masked_fill(out_of, -math.inf)
    ids = torch.empty(c["t"], c["k"], dtype=torch.int64, device=DEV)
    at = torch.arange(c["e"], device=DEV)
    for j in range(c["k"]):  # the largest that is left, the first of equals
        best = r.amax(1, keepdim=True)
        ids[:, j] = torch.where(r == best, at, c["e"]).amin(1)
        r = r.masked_fill(at == ids[:, j:j + 1], -math.inf)
    picked = log_s.gather(1, ids)
    w = torch.softmax(picked, -1) if c["renorm"] else torch.exp(picked)
    return [ids.to(torch.int32), w * c["scale"]]

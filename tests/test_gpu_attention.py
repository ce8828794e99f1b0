"""The attention operators on the GPU against their definitions in 64 bits.

Tolerances.  u is the element type's unit roundoff, the most that rounding to nearest moves a value (half of the type's
eps: 2^-8 for bf16, 2^-11 for fp16), e = 2^-24 that of fp32.

append: a norm and a rotation in fp32, one rounding at the end.  A component is a sum of two products of values of at
most `big` = the head's largest normed component, with a few fp32 roundings each: |err| <= u |ref| + 32 e big.

attend: a score is an fp32 sum of D products, off by at most d = (D + 8) e sum_i |q_i k_i| scale; a weight p = exp(s - m) is
then off by a factor of 1 + d (and 4 e from the exponential), and rounded to the element type as the second product's
operand, by a factor of 1 + u and below the smallest normal fp16 by 2^-25 absolute (the weights are at least 1 where the
reference is the row's maximum).  With A = sum p |v| / sum p and n keys: |err| <= u |ref| + (u + 2 d + 8 e) A + n 2^-25 max |v| +
n e A, where the last term is the fp32 sum's.  lse: |err| <= d + (n + 64) e + 2^-22 |ref|.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = {name: (dt, torch.finfo(dt).eps / 2) for name, dt in (("bf16", torch.bfloat16), ("fp16", torch.float16))}
E = 2.0 ** -24
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from bit_moe_expert_router_gb300 import attention
    attention._load()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


class Case:
    """A ragged batch with its pages in no order; what the cache holds outside of the sequences is `junk`."""

    def __init__(self, q_len, kv_len, hq, hkv, d, page, dtype="bf16", order="token", seed=0, junk=math.nan, spare=2, pad_tokens=0):
        from bit_moe_expert_router_gb300 import attention
        self.q_len, self.kv_len, self.hq, self.hkv, self.d, self.page = q_len, kv_len, hq, hkv, d, page
        self.dt, self.u = DTYPES[dtype]
        self.g = gen(seed)
        b = len(q_len)
        need = [-(-n // page) for n in kv_len]
        width = max(1, max(need))
        pages = sum(need) + spare
        perm = torch.randperm(pages, generator=self.g, device=DEV).tolist()
        self.table = torch.full((b, width), -7, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
            at += n
        shape = (pages, page, hkv, d) if order == "token" else (pages, hkv, page, d)

        def cache():
            t = torch.full(shape, junk, dtype=self.dt, device=DEV)
            return t if order == "token" else t.permute(0, 2, 1, 3)
        self.k_cache, self.v_cache = cache(), cache()
        self.keys, self.values = [], []  # of each sequence, [kv_len, hkv, d]
        for i, n in enumerate(kv_len):
            k, v = (self.normal(n, hkv, d) for _ in range(2))
            self.keys.append(k)
            self.values.append(v)
            pos = torch.arange(n)
            pg, row = self.table[i][pos // page].long().to(DEV), (pos % page).to(DEV)
            self.k_cache[pg, row], self.v_cache[pg, row] = k, v
        start = [0]
        for n in q_len:
            start.append(start[-1] + n)
        self.start, self.tokens = start, start[-1] + pad_tokens
        self.q = self.normal(self.tokens, hq, d)
        i32 = dict(dtype=torch.int32, device=DEV)
        self.q_start, self.lens = torch.tensor(start, **i32), torch.tensor(kv_len, **i32)
        self.table_dev = self.table.to(DEV)
        self.batch = attention.KVBatch(self.k_cache, self.v_cache, self.table_dev, self.q_start, self.lens, n_q_heads=hq,
                                       max_q_len=max(max(q_len), 1))

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device=DEV).to(self.dt)

    def attend(self, window=0, scale=None, q=None, out=None, lse=True, batch=None):
        from bit_moe_expert_router_gb300 import attention
        batch = batch or self.batch
        q = self.q if q is None else q
        out = torch.full_like(q, 77.0) if out is None else out
        lse_t = torch.full((q.shape[0], self.hq), 77.0, device=DEV) if lse else None
        ws = batch.alloc_workspace()
        ws.fill_(255)
        attention.moe_w4a8_paged_attention(batch, q, out, lse_t, scale=scale, window=window, workspace=ws)
        from bit_moe_expert_router_gb300 import binding
        assert binding.moe_w4a8_device_status(ws) == 0
        return out, lse_t

    def reference(self, window=0, scale=None):
        """(out, lse, out's bound, lse's bound) in 64 bits, straight from the definition."""
        scale = self.d ** -0.5 if scale is None else scale
        out = torch.zeros(self.tokens, self.hq, self.d, dtype=torch.float64, device=DEV)
        lse = torch.full((self.tokens, self.hq), -math.inf, dtype=torch.float64, device=DEV)
        tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
        grp = self.hq // self.hkv
        for i, (n, total) in enumerate(zip(self.q_len, self.kv_len)):
            k, v = self.keys[i].double(), self.values[i].double()
            for j in range(n):
                p = total - n + j
                lo = max(0, p + 1 - window) if window else 0
                if p < lo:
                    continue
                t = self.start[i] + j
                qt = self.q[t].double().reshape(self.hkv, grp, self.d)
                kk, vv = k[lo:p + 1].permute(1, 2, 0), v[lo:p + 1].permute(1, 0, 2)  # [hkv, d, n], [hkv, n, d]
                s = qt @ kk * scale
                z = torch.logsumexp(s, -1, keepdim=True)
                w = torch.exp(s - z)
                o = w @ vv
                dlt = (self.d + 8) * E * (qt.abs() @ kk.abs() * scale).amax(-1, keepdim=True)
                a = w @ vv.abs()
                m = p + 1 - lo
                out[t], lse[t] = o.reshape(self.hq, self.d), z.reshape(self.hq)
                bound = self.u * o.abs() + (self.u + 2 * dlt + (8 + m) * E) * a + m * 2.0 ** -25 * vv.abs().amax()
                tol[t] = bound.reshape(self.hq, self.d)
                ltol[t] = (dlt + (m + 64) * E + z.abs() * 2.0 ** -22).reshape(self.hq)
        return out, lse, tol, ltol

    def check(self, window=0, scale=None, **kw):
        out, lse = self.attend(window, scale, **kw)
        ref, rl, tol, ltol = self.reference(window, scale)
        assert not out.isnan().any()
        worst = ((out.double() - ref).abs() - tol).max().item() if self.tokens else 0.0
        assert worst <= 0, f"out is {worst:.3e} beyond its bound"
        seen = rl > -math.inf
        assert torch.equal(lse > -math.inf, seen)
        if seen.any():
            assert ((lse.double() - rl).abs() - ltol)[seen].max().item() <= 0, "lse is beyond its bound"
        return out, lse


# ------------------------------------------------------------------------------------------------ attend
LENGTHS = {
    "one": ([1], [1]),
    "empty": ([1, 1, 0, 1], [0, 5, 9, 1]),                     # no context, no new token
    "before_zero": ([4, 3], [2, 0]),                           # more new tokens than positions
    "edges": ([1] * 9, [15, 16, 17, 63, 64, 65, 127, 128, 129]),
    "long": ([1, 1], [1500, 2311]),                            # cut into pieces
    "verify": ([3, 2, 5], [40, 700, 1027]),
    "chunk": ([70, 33, 1], [70, 200, 310]),
    "prompt": ([300, 129], [300, 650]),
    "mixed": ([1, 260, 1, 2], [900, 420, 0, 77]),
}
HEADS = {"plain": (2, 2), "grouped": (8, 2), "odd": (10, 2), "wide": (32, 2), "many": (48, 1)}


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_lengths(lengths, d):
    Case(*LENGTHS[lengths], 8, 2, d, 16, seed=1).check()


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lengths", ["edges", "verify", "mixed"])
def test_head_groups(lengths, heads):
    Case(*LENGTHS[lengths], *HEADS[heads], 64, 16, "fp16", "head", seed=2).check()


@pytest.mark.parametrize("d", [8, 40, 72, 96, 136, 192, 248])
@pytest.mark.parametrize("lengths", ["long", "chunk"])
def test_head_sizes(lengths, d):
    Case(*LENGTHS[lengths], 4, 2, d, 16, "fp16", seed=3).check()


@pytest.mark.parametrize("page", [1, 5, 8, 12, 24, 48, 80, 256])
@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("lengths", ["verify", "mixed"])
def test_pages(lengths, order, page):
    Case(*LENGTHS[lengths], 8, 2, 128, page, "bf16", order, seed=4).check()


@pytest.mark.parametrize("window", [1, 15, 100, 128, 1000, 10 ** 6])
@pytest.mark.parametrize("lengths", ["empty", "long", "prompt", "mixed"])
def test_windows(lengths, window):
    for d in (64, 128):
        Case(*LENGTHS[lengths], 8, 2, d, 32, "fp16", seed=5).check(window=window)


@pytest.mark.parametrize("lengths", ["long", "prompt"])
def test_sharp_and_flat_scores(lengths):
    """A scale that leaves one key, one that leaves them all, and scores that grow along the sequence (the reference
    maximum moves at every tile)."""
    for scale in (4.0, 1e-4):
        Case(*LENGTHS[lengths], 8, 2, 64, 16, "bf16", seed=6).check(scale=scale)
    c = Case(*LENGTHS[lengths], 8, 2, 64, 16, "bf16", seed=7)
    c.q.fill_(0.25)
    for i, n in enumerate(c.kv_len):
        k = (torch.arange(n, device=DEV)[:, None, None] * 0.02 + torch.zeros_like(c.keys[i], dtype=torch.float32)).to(c.dt)
        c.keys[i] = k
        pos = torch.arange(n)
        c.k_cache[c.table[i][pos // c.page].long().to(DEV), (pos % c.page).to(DEV)] = k
    c.check(scale=1.0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_hidden_places_stay_out(d):
    """Infinities and NaN at positions that a row does not see (later tokens of the chunk, places before its window)
    do not reach it; the rows that see them do get them."""
    for q_len, kv_len, window in (([40, 3], [200, 150], 0), ([1, 1], [700, 90], 50)):
        c = Case(q_len, kv_len, 8, 2, d, 16, seed=8)
        clean, clean_lse = c.attend(window)
        last = kv_len[0] - 1
        bad = [last] if not window else [last - window]  # seen by the last token alone, or by none
        for p in bad:
            pg, row = int(c.table[0][p // 16]), p % 16
            c.v_cache[pg, row] = math.nan
            c.v_cache[pg, row, :, 0] = math.inf
            c.k_cache[pg, row, 0] = math.nan
        out, lse = c.attend(window)
        t = q_len[0] - 1
        others = [i for i in range(c.tokens) if i != t or window]
        ref, rl, tol, ltol = c.reference(window)
        assert ((out.double() - ref).abs() <= tol)[others].all()
        assert ((lse.double() - rl).abs() <= ltol)[others].all()
        if not window:
            assert out[t].isnan().any() and lse[t, :4].isnan().all()
        assert clean.isfinite().all() and clean_lse.isfinite().all()


def test_page_ids_out_of_range_read_zeros():
    for q_len in (1, 50):
        c = Case([q_len], [200], 4, 2, 64, 16, "fp16", seed=9, junk=1.0)
        for bad, col in ((-1, 3), (10 ** 9, 5)):
            c.table_dev[0, col] = bad
            c.keys[0][16 * col:16 * col + 16] = 0
            c.values[0][16 * col:16 * col + 16] = 0
        c.check()


def test_positions_past_the_table_do_not_exist():
    """kv_len beyond what a row of the table holds: rows keep their positions, the keys end with the table."""
    for q_len in (1, 40):
        c = Case([q_len], [96], 4, 2, 64, 16, seed=10)
        ref = c.attend()[0]
        c.lens.fill_(96 + 500)
        out = c.attend()[0]
        assert out.isfinite().all()
        # the last token sees all 96 keys either way
        assert torch.allclose(out[-1].float(), ref[-1].float(), atol=2e-2)


@pytest.mark.parametrize("lengths", ["edges", "prompt"])
def test_strides_and_missing_lse(lengths):
    c = Case(*LENGTHS[lengths], 8, 2, 64, 16, seed=11)
    wide = torch.randn(c.tokens, 3, 8, 128, generator=c.g, device=DEV).to(c.dt)
    q = wide[:, 1, :, :64]
    q.copy_(c.q)
    out = torch.full((8, c.tokens, 72), 5.0, dtype=c.dt, device=DEV)
    got, _ = c.attend(q=q, out=out.permute(1, 0, 2)[:, :, :64], lse=False)
    plain, _ = c.attend()
    assert torch.equal(got, plain)
    assert (out[:, :, 64:] == 5.0).all()


def test_tokens_of_no_sequence_are_cleared():
    for q_len, kv_len in (([1, 2], [5, 9]), ([60, 1], [60, 9])):
        c = Case(q_len, kv_len, 4, 2, 64, 16, seed=12, pad_tokens=5)
        out, lse = c.check()
        assert (out[c.start[-1]:] == 0).all() and (lse[c.start[-1]:] == -math.inf).all()


@pytest.mark.parametrize("lengths", ["long", "prompt", "mixed"])
def test_two_runs_give_the_same_bits(lengths):
    for d in (64, 128, 256):
        c = Case(*LENGTHS[lengths], 16, 4, d, 16, seed=13)
        a, la = c.attend()
        b, lb = c.attend()
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_bounds_on_lengths_are_hints_only():
    """max_q_len and max_kv_len below the batch's own: the same values from another kernel."""
    from bit_moe_expert_router_gb300 import attention
    for lengths in ("long", "prompt", "mixed"):
        c = Case(*LENGTHS[lengths], 8, 2, 128, 16, seed=14)
        low = attention.KVBatch(c.k_cache, c.v_cache, c.table_dev, c.q_start, c.lens, n_q_heads=8, max_q_len=1, max_kv_len=1)
        c.check(batch=low)
        high = attention.KVBatch(c.k_cache, c.v_cache, c.table_dev, c.q_start, c.lens, n_q_heads=8, max_q_len=4096)
        c.check(batch=high)


def test_another_stream_and_a_graph():
    c = Case(*LENGTHS["mixed"], 8, 2, 128, 16, seed=15)
    from bit_moe_expert_router_gb300 import attention
    ref, _ = c.attend()
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    ws, out = c.batch.alloc_workspace(), torch.zeros_like(c.q)
    with torch.cuda.stream(side):
        attention.moe_w4a8_paged_attention(c.batch, c.q, out, workspace=ws)
    torch.cuda.current_stream(DEV).wait_stream(side)
    assert torch.equal(out, ref)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attention.moe_w4a8_paged_attention(c.batch, c.q, out, workspace=ws)
    for step in range(3):  # new queries and lengths, the same graph
        c.q.copy_(c.normal(*c.q.shape))
        c.lens[0] -= step
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c.attend()[0])


def test_a_cache_of_more_than_two_to_the_31_elements():
    pages, page, hkv, d = (1 << 31) // (64 * 2 * 256) + 40, 64, 2, 256
    from bit_moe_expert_router_gb300 import attention
    k, v = (torch.zeros(pages, page, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    assert k.numel() > 1 << 31
    for q_len in (1, 80):
        c = Case([q_len], [300], 4, 2, 256, 64, seed=16)
        table = torch.tensor([[pages - 1, 3, pages - 9, 0, pages - 30]], dtype=torch.int32, device=DEV)
        for x, id in enumerate(table[0].tolist()):
            m = min(64, 300 - 64 * x)
            k[id, :m], v[id, :m] = c.keys[0][64 * x:64 * x + m], c.values[0][64 * x:64 * x + m]
        c.check(batch=attention.KVBatch(k, v, table, c.q_start, c.lens, n_q_heads=4, max_q_len=q_len))


def test_many_sequences():
    n = 700
    lens = [(37 * i) % 90 for i in range(n)]
    Case([1] * n, lens, 4, 2, 64, 16, "fp16", seed=17).check()


def test_refusals_on_the_device():
    from bit_moe_expert_router_gb300 import attention
    c = Case([1, 1], [5, 9], 4, 2, 64, 16)
    ws = c.batch.alloc_workspace()
    out = torch.empty_like(c.q)
    with pytest.raises(TypeError, match="dtype"):
        attention.moe_w4a8_paged_attention(c.batch, c.q.half(), out, workspace=ws)
    with pytest.raises(ValueError, match="shape"):
        attention.moe_w4a8_paged_attention(c.batch, c.q, out[:1], workspace=ws)
    with pytest.raises(ValueError, match="contiguous"):
        attention.moe_w4a8_paged_attention(c.batch, c.q.transpose(1, 2).contiguous().transpose(1, 2), out, workspace=ws)
    with pytest.raises(ValueError, match="lse"):
        attention.moe_w4a8_paged_attention(c.batch, c.q, out, torch.zeros(2, 5, device=DEV), workspace=ws)
    with pytest.raises(ValueError, match="on cpu"):
        attention.moe_w4a8_paged_attention(c.batch, c.q.cpu(), out, workspace=ws)
    with pytest.raises(attention.MoeError) as err:
        attention.moe_w4a8_paged_attention(c.batch, c.q, out, workspace=ws[:1024])
    assert err.value.status == 3
    odd = torch.empty(2, 4, 68, dtype=c.dt, device=DEV)[:, :, :64]  # rows of 136 bytes
    with pytest.raises(attention.MoeError) as err:
        attention.moe_w4a8_paged_attention(c.batch, odd, out, workspace=ws)
    assert err.value.status == 1
    with pytest.raises(ValueError, match="shape"):
        attention.KVBatch(c.k_cache, c.v_cache, c.table_dev, c.q_start[:2], c.lens, n_q_heads=4, max_q_len=1)
    with pytest.raises(attention.MoeError):
        attention.KVBatch(c.k_cache, c.v_cache, c.table_dev, c.q_start, c.lens, n_q_heads=3, max_q_len=1)


# ------------------------------------------------------------------------------------------------ append
def prep_reference(x, weight, offset, eps, table, rows, rot, inter):
    """[n, heads, d] in 64 bits -> (normed and turned, the largest normed component of each head)."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (weight.double() + offset)
    big = x.abs().amax(-1, keepdim=True)
    if rot:
        cs = table[rows].double()[:, None]
        c, s = cs[..., :rot // 2], cs[..., rot // 2:]
        x = x.clone()
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
        p, q = x[..., a].clone(), x[..., b].clone()
        x[..., a], x[..., b] = p * c - q * s, q * c + p * s
    return x, big


def run_append(c, rot, inter, norm, offset=1.0, fused=True, in_place=False, positions=None, table=None, eps=1e-6):
    from bit_moe_expert_router_gb300 import attention
    if fused:
        qkv = c.normal(c.tokens, c.hq + 2 * c.hkv, c.d)
        q, k, v = qkv.split([c.hq, c.hkv, c.hkv], dim=1)
    else:  # head-major
        q, k, v = (c.normal(h, c.tokens, c.d).transpose(0, 1) for h in (c.hq, c.hkv, c.hkv))
    rows = c.table.shape[1] * c.page
    if table is None and rot:
        table = attention.rope_table(rows, rot, device=DEV)
    qw, kw = (torch.randn(c.d, generator=c.g, device=DEV) * 0.2 for _ in range(2)) if norm else (None, None)
    prep = attention.HeadPrep(table, inter, qw, kw, eps=eps, weight_offset=offset, positions=positions)
    out = q if in_place else torch.full((c.tokens, c.hq, c.d), 9.0, dtype=c.dt, device=DEV)
    q0, k0, v0, kc0, vc0 = q.clone(), k.clone(), v.clone(), c.k_cache.clone(), c.v_cache.clone()
    attention.moe_w4a8_kv_append(c.batch, prep, q, k, v, out)
    torch.cuda.synchronize()
    want_k, want_v, want_q = kc0.double(), vc0.double(), torch.zeros(c.tokens, c.hq, c.d, dtype=torch.float64, device=DEV)
    big_q, big_k = torch.zeros(c.tokens, c.hq, 1, dtype=torch.float64, device=DEV), torch.zeros_like(want_k[..., :1])
    table_ids = c.table_dev.cpu()
    for i, (n, total) in enumerate(zip(c.q_len, c.kv_len)):
        for j in range(n):
            t, p = c.start[i] + j, total - n + j
            turn = p if positions is None else int(positions[t])
            if p < 0 or (rot and not 0 <= turn < table.shape[0]):
                continue
            at = torch.tensor([turn], device=DEV)
            want_q[t], big_q[t] = (y[0] for y in prep_reference(q0[t:t + 1], qw, offset, eps, table, at, rot, inter))
            pg = int(table_ids[i, p // c.page]) if p // c.page < table_ids.shape[1] else -1
            if not 0 <= pg < c.k_cache.shape[0]:
                continue
            want_k[pg, p % c.page], big_k[pg, p % c.page] = (y[0] for y in prep_reference(k0[t:t + 1], kw, offset, eps, table, at, rot, inter))
            want_v[pg, p % c.page] = v0[t].double()
    for got, want, big in ((out, want_q, big_q), (c.k_cache, want_k, big_k), (c.v_cache, want_v, torch.zeros_like(big_k))):
        same_nan = torch.equal(got.isnan(), want.isnan())
        assert same_nan, "written where nothing was to be, or not written"
        err = (got.double() - want).abs() - (c.u * want.abs() + 32 * E * big)
        assert torch.nan_to_num(err, nan=0.0).max().item() <= 0
    if not in_place:
        assert torch.equal(q, q0) and torch.equal(k, k0) and torch.equal(v, v0)


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 24), (64, 6), (128, 128), (128, 64), (96, 24), (96, 96), (40, 40), (256, 64), (256, 128),
                                   (256, 256), (256, 160), (192, 192), (8, 2), (128, 0)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_append_heads(d, rot, inter, norm):
    run_append(Case([1, 3, 1], [20, 33, 1], 6, 2, d, 16, "bf16" if norm else "fp16", seed=20), rot, inter, norm)


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("order", ["token", "head"])
def test_append_lengths(lengths, order):
    run_append(Case(*LENGTHS[lengths], 5, 1, 64, 16, "fp16", order, seed=21, pad_tokens=3), 32, False, True)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (16, 2, 256), (3, 3, 64), (7, 1, 96)])
def test_append_of_many_tokens(hq, hkv, d):
    """Enough tokens for the kernel's other shape (many heads of a token to a warp)."""
    c = Case([700, 1, 611], [700, 50, 900], hq, hkv, d, 24, "bf16", seed=22)
    run_append(c, d // 2, True, True)
    run_append(c, d // 2 // 16 * 16, False, False)


def test_append_in_place_and_strided():
    for rot, inter in ((64, False), (24, False), (24, True)):
        run_append(Case([2, 1], [9, 30], 4, 2, 64, 8, seed=23), rot, inter, True, fused=False)
        run_append(Case([2, 1], [9, 30], 4, 2, 64, 8, seed=24), rot, inter, True, in_place=True)


def test_append_positions_of_the_callers():
    from bit_moe_expert_router_gb300 import attention
    c = Case([3, 1], [9, 30], 4, 2, 64, 8, seed=25)
    table = attention.rope_table(1000, 64, device=DEV, scaling="yarn", factor=4.0, original=250)
    pos = torch.tensor([900, 0, -1, 1000], dtype=torch.int32, device=DEV)  # the last two are outside of the table: padding
    run_append(c, 64, False, False, positions=pos, table=table)


def test_append_skips_pages_that_are_not_there():
    c = Case([4, 2], [20, 10], 4, 2, 64, 8, seed=26)
    c.table_dev[0, 2], c.table_dev[1, 1] = 10 ** 6, -3
    run_append(c, 64, True, True)


def test_append_then_attend_is_attention_of_the_whole():
    """A prompt in one piece, in two chunks, and token by token leave the same cache and give the same rows."""
    from bit_moe_expert_router_gb300 import attention
    n, hq, hkv, d, page = 90, 8, 2, 64, 16
    g = gen(27)
    qkv = torch.randn(n, hq + 2 * hkv, d, generator=g, device=DEV).bfloat16()
    prep = attention.HeadPrep(attention.rope_table(n, d, device=DEV))

    def serve(cuts):
        k, v = (torch.zeros(8, page, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        table = torch.tensor([[5, 2, 7, 0, 1, 3]], dtype=torch.int32, device=DEV)
        q_start, lens = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        batch = attention.KVBatch(k, v, table, q_start, lens, n_q_heads=hq, max_q_len=n)
        ws, rows, at = batch.alloc_workspace(), [], 0
        for m in cuts:
            q, kk, vv = qkv[at:at + m].split([hq, hkv, hkv], dim=1)
            at += m
            q_start[1], lens[0] = m, at
            out, qr = (torch.empty(m, hq, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
            attention.moe_w4a8_kv_append(batch, prep, q, kk, vv, qr)
            attention.moe_w4a8_paged_attention(batch, qr, out, workspace=ws)
            rows.append(out)
        return k, v, torch.cat(rows)

    k, v, rows = serve([n])
    for cuts in ([33, 57], [50] + [1] * 40, [89, 1]):
        k2, v2, rows2 = serve(cuts)
        assert torch.equal(k, k2) and torch.equal(v, v2)
        # the same weights rounded at other references: within two units of the row's largest value
        assert (rows.float() - rows2.float()).abs().max() <= 2 * torch.finfo(torch.bfloat16).eps * rows.float().abs().max()

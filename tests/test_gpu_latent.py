"""Latent attention on the GPU against its definition in 64 bits.

Tolerances.  u is the element type's unit roundoff (half of its eps: 2^-8 for bf16, 2^-11 for fp16), e = 2^-24 that of fp32.

append: the norm's factor, weight and product, then a sum of two products of values of at most `big` = the row's (or the
head's) largest component before the turn, each with a few fp32 roundings, and one rounding at the end:
|err| <= u |ref| + 32 e big; fp16 results below its smallest normal number are rounded to multiples of 2^-24, off by 2^-25.

attend: a score is an fp32 sum of D products, off by at most d = (D + 8) e sum_i |q_i x_i| scale; a weight p = exp(s - m) is
then off by a factor of 1 + d (and 4 e from the exponential), and rounded to the element type as the second product's
operand, by a factor of 1 + u and below the smallest normal fp16 by 2^-25 absolute (the weights are at least 1 where the
reference is the row's maximum, and that lags behind by a factor of 2^8 at most, to the better).  With A = sum p |x| / sum p and n
keys: |err| <= u |ref| + (u + 2 d + 8 e) A + n 2^-25 max |x| + n e A, where the last term is the fp32 sum's.
lse: |err| <= d + (n + 64) e + 2^-22 |ref|.
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
    from bit_moe_expert_router_gb300 import latent
    latent._load()


class Case:
    """A ragged batch with its pages in no order; what the cache holds outside of the sequences is `junk`."""

    def __init__(self, q_len, kv_len, h, dc, rot, page, dtype="bf16", seed=0, junk=math.nan, spare=2, pad_tokens=0, row_pad=0):
        from bit_moe_expert_router_gb300 import latent
        self.q_len, self.kv_len, self.h, self.dc, self.rot, self.page, self.d = q_len, kv_len, h, dc, rot, page, dc + rot
        self.dt, self.u = DTYPES[dtype]
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)
        need = [-(-n // page) for n in kv_len]
        pages = sum(need) + spare
        perm = torch.randperm(pages, generator=self.g, device=DEV).tolist()
        self.table = torch.full((len(q_len), max(1, max(need))), -7, dtype=torch.int32)
        self.cache = torch.full((pages, page, self.d + row_pad), junk, dtype=self.dt, device=DEV)[..., :self.d]
        self.rows, at = [], 0  # the rows of each sequence, [kv_len, d]
        for i, n in enumerate(need):
            self.table[i, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
            at += n
            x = self.normal(kv_len[i], self.d)
            self.rows.append(x)
            self.cache[self.where(i)] = x
        start = [0]
        for n in q_len:
            start.append(start[-1] + n)
        self.start, self.tokens = start, start[-1] + pad_tokens
        self.q = self.normal(self.tokens, h, self.d)
        i32 = dict(dtype=torch.int32, device=DEV)
        self.q_start, self.lens, self.table_dev = torch.tensor(start, **i32), torch.tensor(kv_len, **i32), self.table.to(DEV)
        self.batch = latent.LatentBatch(self.cache, self.table_dev, self.q_start, self.lens, n_heads=h, latent_dim=dc,
                                        max_q_len=max(max(q_len), 1))

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device=DEV).to(self.dt)

    def where(self, i, pos=None):
        """(pages, rows) of positions of sequence i."""
        pos = torch.arange(self.kv_len[i]) if pos is None else torch.as_tensor(pos)
        return self.table[i][pos // self.page].long().to(DEV), (pos % self.page).to(DEV)

    def attend(self, scale=None, q=None, out=None, lse=True, batch=None):
        from bit_moe_expert_router_gb300 import binding, latent
        batch = batch or self.batch
        q = self.q if q is None else q
        out = torch.full((q.shape[0], self.h, self.dc), 77.0, dtype=self.dt, device=DEV) if out is None else out
        lse_t = torch.full((q.shape[0], self.h), 77.0, device=DEV) if lse else None
        ws = batch.alloc_workspace()
        ws.fill_(255)
        latent.moe_w4a8_latent_attention(batch, q, out, lse_t, scale=scale, workspace=ws)
        assert binding.moe_w4a8_device_status(ws) == 0
        return out, lse_t

    def reference(self, scale=None):
        """(out, lse, out's bound, lse's bound) in 64 bits, straight from the definition; rows' values may be non-finite."""
        scale = self.d ** -0.5 if scale is None else scale
        f64 = dict(dtype=torch.float64, device=DEV)
        out, lse = torch.zeros(self.tokens, self.h, self.dc, **f64), torch.full((self.tokens, self.h), -math.inf, **f64)
        tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
        for i, (n, total) in enumerate(zip(self.q_len, self.kv_len)):
            for j in range(max(0, n - total), n):
                p, t = total - n + j, self.start[i] + j
                x, q = self.rows[i][:p + 1].double(), self.q[t].double()
                v = x[:, :self.dc]
                s = q @ x.T * scale
                z = torch.logsumexp(s, -1, keepdim=True)
                w = torch.exp(s - z)
                a = w @ v.abs()
                dlt = (self.d + 8) * E * (q.abs() @ x.abs().T * scale).amax(-1, keepdim=True)
                out[t], lse[t] = w @ v, z[:, 0]
                tol[t] = self.u * out[t].abs() + (self.u + 2 * dlt + (9 + p) * E) * a + (p + 1) * 2.0 ** -25 * v.abs().amax()
                ltol[t] = (dlt + (p + 65) * E + z.abs() * 2.0 ** -22)[:, 0]
        return out, lse, tol, ltol

    def check(self, scale=None, **kw):
        out, lse = self.attend(scale, **kw)
        ref, ref_lse, tol, ltol = self.reference(scale)
        for what, got, want, bound in (("out", out, ref, tol), ("lse", lse, ref_lse, ltol)):
            odd = ~want.isfinite()
            same = torch.where(want.isnan(), got.isnan(), got.double() == want)
            assert bool(same[odd].all()), f"{what}: {int((~same & odd).sum())} values that are not finite differ"
            err = ((got.double() - want).abs() - bound)[~odd]
            assert not err.isnan().any(), f"{what}: {int(err.isnan().sum())} values are NaN where they should not be"
            assert err.numel() == 0 or err.max().item() <= 0, f"{what} is {err.max().item():.3e} beyond its bound"
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
    "mixed": ([1, 130, 1, 2], [900, 320, 0, 77]),
}


@pytest.mark.parametrize("h", [1, 5, 16, 20, 32, 48, 64, 128])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_lengths_and_heads(lengths, h):
    Case(*LENGTHS[lengths], h, 512, 64, 16, seed=1).check()


@pytest.mark.parametrize("dc,rot", [(8, 0), (64, 8), (64, 64), (72, 24), (128, 0), (128, 64), (192, 32), (248, 8), (256, 64), (384, 64), (448, 64),
                                    (504, 40), (512, 0), (512, 8)])
@pytest.mark.parametrize("lengths", ["long", "chunk"])
def test_sizes(lengths, dc, rot):
    Case(*LENGTHS[lengths], 12, dc, rot, 16, "fp16", seed=2).check()


@pytest.mark.parametrize("page", [8, 16, 24, 32, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("h", [16, 128])
def test_pages(h, page):
    for lengths in ("verify", "mixed"):
        Case(*LENGTHS[lengths], h, 512, 64, page, seed=3).check()


def test_a_thousand_heads_and_a_prompt_of_many_tiles():
    Case([2, 1], [130, 70], 1000, 512, 64, 64, seed=4).check()
    Case([700], [900], 8, 256, 64, 32, "fp16", seed=5).check()


@pytest.mark.parametrize("h", [16, 32, 64, 128])
def test_a_long_context(h):
    """One sequence that fills the GPU by its keys alone: a piece of many units for each CTA or pair, every tile cut."""
    Case([1], [131071], h, 512, 64, 64, seed=31).check()


@pytest.mark.parametrize("lengths", ["long", "chunk"])
def test_sharp_and_flat_scores(lengths):
    """A scale that leaves one key, one that leaves them all, and scores that grow along the sequence (the reference
    maximum moves at every tile)."""
    for scale in (4.0, 1e-4):
        Case(*LENGTHS[lengths], 16, 128, 64, 16, seed=6).check(scale=scale)
    for h in (16, 128):
        c = Case(*LENGTHS[lengths], h, 128, 64, 16, seed=7)
        c.q.fill_(0.25)
        for i, n in enumerate(c.kv_len):
            c.rows[i] = (torch.arange(n, device=DEV)[:, None] * 0.02 + torch.zeros(n, c.d, device=DEV)).to(c.dt)
            c.cache[c.where(i)] = c.rows[i]
        c.check(scale=1.0)


@pytest.mark.parametrize("h", [4, 16, 40, 128])
def test_hidden_places_stay_out(h):
    """A NaN or an infinity at a position reaches the rows that see it and no others, in whole tiles and in pieces."""
    for q_len, kv_len in (([40, 3], [200, 150]), ([9, 2], [1700, 900]), ([5], [64])):
        for part, value in ((slice(None), math.nan), (3, math.inf), (slice(512, 576), math.nan), (511, -math.inf)):
            c = Case(q_len, kv_len, h, 512, 64, 16, seed=8)
            for back in (1, 3):
                p = kv_len[0] - back
                c.rows[0][p, part] = value
                c.cache[c.where(0, [p])] = c.rows[0][p:p + 1]
            c.check()


def test_page_ids_out_of_range_read_zeros():
    for h, q_len in ((16, 1), (4, 50), (128, 1)):
        c = Case([q_len], [200], h, 512, 64, 16, "fp16", seed=9, junk=1.0)
        for bad, col in ((-1, 3), (10 ** 9, 5)):
            c.table_dev[0, col] = bad
            c.rows[0][16 * col:16 * col + 16] = 0
        c.check()


def test_positions_past_the_table_do_not_exist():
    """kv_len beyond what a row of the table holds: rows keep their positions, the keys end with the table."""
    for q_len in (1, 40):
        c = Case([q_len], [96], 16, 512, 64, 16, seed=10)
        ref = c.attend()[0]
        c.lens.fill_(96 + 500)
        out = c.attend()[0]
        assert out.isfinite().all()
        # the last token sees all 96 keys either way: the same weights, rounded at references that may differ
        assert (out[-1].float() - ref[-1].float()).abs().max() <= 4 * c.u * c.rows[0].float().abs().max()


@pytest.mark.parametrize("lengths", ["edges", "chunk"])
@pytest.mark.parametrize("h", [16, 128])
def test_strides_and_missing_lse(lengths, h):
    c = Case(*LENGTHS[lengths], h, 512, 64, 16, seed=11, row_pad=64)
    wide = torch.randn(c.tokens, 2, h, 640, generator=c.g, device=DEV).to(c.dt)
    q = wide[:, 1, :, :576]
    q.copy_(c.q)
    out = torch.full((h, c.tokens, 520), 5.0, dtype=c.dt, device=DEV)
    got, _ = c.attend(q=q, out=out.permute(1, 0, 2)[:, :, :512], lse=False)
    plain, _ = c.check()
    assert torch.equal(got, plain)
    assert (out[:, :, 512:] == 5.0).all()


def test_pages_side_by_side():
    """A cache whose pages lie row by row beside one another (page stride below row stride)."""
    from bit_moe_expert_router_gb300 import latent
    for h in (16, 128):
        c = Case([1, 9], [300, 70], h, 512, 64, 16, seed=12)
        beside = c.cache.permute(1, 0, 2).contiguous().permute(1, 0, 2)
        assert beside.stride(0) < beside.stride(1)
        c.check(batch=latent.LatentBatch(beside, c.table_dev, c.q_start, c.lens, n_heads=h, latent_dim=512, max_q_len=9))


def test_tokens_of_no_sequence_are_cleared():
    for h, q_len, kv_len in ((16, [1, 2], [5, 9]), (128, [60, 1], [60, 9])):
        c = Case(q_len, kv_len, h, 512, 64, 16, seed=12, pad_tokens=5)
        out, lse = c.check()
        assert (out[c.start[-1]:] == 0).all() and (lse[c.start[-1]:] == -math.inf).all()


@pytest.mark.parametrize("lengths", ["long", "chunk", "mixed"])
def test_two_runs_give_the_same_bits(lengths):
    for h in (16, 64, 128):
        c = Case(*LENGTHS[lengths], h, 512, 64, 16, seed=13)
        a, la = c.attend()
        b, lb = c.attend()
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_bounds_on_lengths_are_hints_only():
    """max_q_len and max_kv_len below or above the batch's own: the same values from another kernel or launch."""
    from bit_moe_expert_router_gb300 import latent
    for lengths in ("long", "chunk", "mixed"):
        for h in (16, 48):
            c = Case(*LENGTHS[lengths], h, 512, 64, 16, seed=14)
            for q_hint, kv_hint in ((1, 1), (1, None), (2, None), (4096, None), (4096, 1)):
                c.check(batch=latent.LatentBatch(c.cache, c.table_dev, c.q_start, c.lens, n_heads=h, latent_dim=512, max_q_len=q_hint, max_kv_len=kv_hint))


def test_another_stream_and_a_graph():
    from bit_moe_expert_router_gb300 import latent
    for h in (16, 128):
        c = Case(*LENGTHS["mixed"], h, 512, 64, 16, seed=15)
        ref, _ = c.attend()
        side = torch.cuda.Stream(DEV)
        side.wait_stream(torch.cuda.current_stream(DEV))
        ws, out = c.batch.alloc_workspace(), torch.zeros_like(ref)
        with torch.cuda.stream(side):
            latent.moe_w4a8_latent_attention(c.batch, c.q, out, workspace=ws)
        torch.cuda.current_stream(DEV).wait_stream(side)
        assert torch.equal(out, ref)
        out.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            latent.moe_w4a8_latent_attention(c.batch, c.q, out, workspace=ws)
        for step in range(3):  # new queries and lengths, the same graph
            c.q.copy_(c.normal(*c.q.shape))
            c.lens[0] -= step
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, c.attend()[0])


def test_one_workspace_for_calls_and_graphs_of_every_kind():
    """What a call leaves in a workspace (pieces, their records) never reaches the next one, eager or replayed."""
    from bit_moe_expert_router_gb300 import latent
    cases = [Case(*LENGTHS[k], h, 512, 64, 16, seed=30) for k, h in (("mixed", 128), ("long", 16), ("one", 128), ("edges", 32), ("chunk", 48), ("empty", 16), ("long", 128))]
    refs = [c.attend()[0] for c in cases]
    ws, outs = cases[0].batch.alloc_workspace(), [torch.empty_like(r) for r in refs]
    ws.fill_(255)

    def attend(i):
        latent.moe_w4a8_latent_attention(cases[i].batch, cases[i].q, outs[i], workspace=ws)
    graphs = [torch.cuda.CUDAGraph() for _ in cases]
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            attend(i)
    for turn in range(3):
        for out in outs:
            out.fill_(77.0)
        for i in range(len(cases)):
            j = (3 * i + turn) % len(cases)
            graphs[j].replay() if (i + turn) % 2 else attend(j)
        torch.cuda.synchronize()
        for i, (out, ref) in enumerate(zip(outs, refs)):
            assert torch.equal(out, ref), (turn, i)


def test_two_calls_at_once():
    """Calls on two streams with a workspace each, over one cache."""
    from bit_moe_expert_router_gb300 import latent
    c = Case([1, 1, 3], [3000, 2000, 900], 16, 512, 64, 16, seed=16)
    ref = c.attend()[0]
    streams, spaces = [torch.cuda.Stream(DEV) for _ in range(2)], [c.batch.alloc_workspace() for _ in range(2)]
    outs = [torch.zeros_like(ref) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, ws, out in zip(streams, spaces, outs):
            with torch.cuda.stream(s):
                latent.moe_w4a8_latent_attention(c.batch, c.q, out, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(out, ref) for out in outs)


def test_a_cache_of_more_than_two_to_the_31_elements():
    from bit_moe_expert_router_gb300 import latent
    pages = (1 << 31) // (64 * 576) + 40
    cache = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device=DEV)
    for h, q_len in ((16, 1), (128, 3)):
        c = Case([q_len], [300], h, 512, 64, 64, seed=17)
        table = torch.tensor([[pages - 1, 3, pages - 9, 0, pages - 30]], dtype=torch.int32, device=DEV)
        for x, id in enumerate(table[0].tolist()):
            m = min(64, 300 - 64 * x)
            cache[id, :m] = c.rows[0][64 * x:64 * x + m]
        c.check(batch=latent.LatentBatch(cache, table, c.q_start, c.lens, n_heads=h, latent_dim=512, max_q_len=q_len))


def test_many_sequences():
    n = 700
    Case([1] * n, [(37 * i) % 90 for i in range(n)], 16, 128, 64, 16, "fp16", seed=18).check()


def test_refusals_on_the_device():
    from bit_moe_expert_router_gb300 import latent
    c = Case([1, 1], [5, 9], 4, 128, 64, 16)
    ws, out = c.batch.alloc_workspace(), torch.empty(2, 4, 128, dtype=c.dt, device=DEV)

    def attend(q=c.q, out=out, lse=None, ws=ws, **kw):
        latent.moe_w4a8_latent_attention(c.batch, q, out, lse, workspace=ws, **kw)
    for error, match, kw in ((TypeError, "dtype", dict(q=c.q.half())), (ValueError, "shape", dict(out=out[:1])),
                             (ValueError, "shape", dict(q=c.q[..., :128])), (ValueError, "contiguous", dict(q=c.q.transpose(1, 2).contiguous().transpose(1, 2))),
                             (ValueError, "lse", dict(lse=torch.zeros(2, 5, device=DEV))), (ValueError, "on cpu", dict(q=c.q.cpu()))):
        with pytest.raises(error, match=match):
            attend(**kw)
    odd = torch.empty(2, 4, 196, dtype=c.dt, device=DEV)[:, :, :192]  # rows of 392 bytes
    for status, kw in ((3, dict(ws=ws[:1024])), (1, dict(q=odd)), (1, dict(scale=0.0)), (1, dict(scale=math.inf))):
        with pytest.raises(latent.MoeError) as err:
            attend(**kw)
        assert err.value.status == status
    for kw in (dict(n_heads=0), dict(n_heads=1025), dict(max_q_len=0), dict(latent_dim=100)):
        with pytest.raises(latent.MoeError):
            latent.LatentBatch(c.cache, c.table_dev, c.q_start, c.lens, **{**dict(n_heads=4, latent_dim=128, max_q_len=1), **kw})
    with pytest.raises(latent.MoeError):  # pages of a size that is not a multiple of 8
        latent.LatentBatch(c.cache[:, :12], c.table_dev, c.q_start, c.lens, n_heads=4, latent_dim=128, max_q_len=1)
    with pytest.raises(ValueError, match="shape"):
        latent.LatentBatch(c.cache, c.table_dev, c.q_start[:2], c.lens, n_heads=4, latent_dim=128, max_q_len=1)
    with pytest.raises(ValueError, match="latent_dim"):
        latent.LatentBatch(c.cache, c.table_dev, c.q_start, c.lens, n_heads=4, latent_dim=200, max_q_len=1)


# ------------------------------------------------------------------------------------------------ append
def turned(x, cs, inter):
    half = cs.shape[-1] // 2
    c, s = cs[..., :half], cs[..., half:]
    y = x.clone()
    a, b = (slice(0, None, 2), slice(1, None, 2)) if inter else (slice(0, half), slice(half, None))
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def run_append(c, inter, norm, offset=0.0, in_place=False, positions=None, table=None, eps=1e-6):
    from bit_moe_expert_router_gb300 import attention, latent
    rot = c.rot
    kv = c.normal(c.tokens, c.d + 8) * 3  # latent and key part side by side in a projection's rows, with something behind
    x, k = kv[:, :c.dc], kv[:, c.dc:c.d]
    q = c.normal(c.tokens, c.h, 24 + rot)[..., 24:]
    if table is None and rot:
        table = attention.rope_table(c.table.shape[1] * c.page, rot, device=DEV)
    w = 1.0 + 0.2 * torch.randn(c.dc, generator=c.g, device=DEV) if norm else None
    prep = attention.HeadPrep(table, inter, None, w, eps=eps, weight_offset=offset, positions=positions)
    wide = torch.full((c.tokens, c.h, 2 * rot + 8), 9.0, dtype=c.dt, device=DEV)
    out = q if in_place else wide[..., :rot]
    q0, before = q.clone(), c.cache.clone()
    if rot:
        got = latent.moe_w4a8_latent_append(c.batch, prep, x, k, q, out)
        assert got is out
    else:
        latent.moe_w4a8_latent_append(c.batch, prep, x)
    torch.cuda.synchronize()
    want, want_q = before.double(), torch.zeros(c.tokens, c.h, rot, dtype=torch.float64, device=DEV)
    big, big_q = torch.zeros_like(want[..., :1]), torch.zeros_like(want_q[..., :1])
    ids = c.table_dev.cpu()
    for i, (n, total) in enumerate(zip(c.q_len, c.kv_len)):
        for j in range(n):
            t, p = c.start[i] + j, total - n + j
            at = p if positions is None else int(positions[t])
            if p < 0 or (rot and not 0 <= at < table.shape[0]):
                continue
            y, kk = x[t].double(), k[t].double()
            if norm:
                y = y / torch.sqrt((y * y).mean() + eps) * (w.double() + offset)
            if rot:
                want_q[t], kk = turned(q0[t].double(), table[at].double(), inter), turned(kk, table[at].double(), inter)
                big_q[t] = q0[t].double().abs().amax(-1, keepdim=True)
            pg = int(ids[i, p // c.page]) if p // c.page < ids.shape[1] else -1
            if 0 <= pg < c.cache.shape[0]:
                want[pg, p % c.page] = torch.cat([y, kk])
                big[pg, p % c.page] = torch.cat([y, k[t].double()]).abs().max()
    for got, ref, b in ((out, want_q, big_q), (c.cache, want, big)) if rot else ((c.cache, want, big),):
        assert torch.equal(got.isnan(), ref.isnan()), "written where nothing was to be, or not written"
        err = (got.double() - ref).abs() - (c.u * ref.abs() + 32 * E * b + 2.0 ** -25)
        assert torch.nan_to_num(err, nan=0.0).max().item() <= 0
    assert (wide[..., rot:] == 9.0).all()
    if not in_place:
        assert torch.equal(q, q0)


@pytest.mark.parametrize("dc,rot", [(512, 64), (256, 32), (8, 8), (72, 24), (512, 0), (128, 16), (504, 56), (64, 40), (384, 48)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_append_sizes(dc, rot, inter, norm):
    run_append(Case([1, 3, 1], [20, 33, 1], 6, dc, rot, 16, "bf16" if norm else "fp16", seed=20), inter, norm, offset=float(inter))


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("h", [1, 5, 128])
def test_append_lengths(lengths, h):
    run_append(Case(*LENGTHS[lengths], h, 512, 64, 16, "fp16", seed=21, pad_tokens=3), False, True)
    run_append(Case(*LENGTHS[lengths], h, 512, 64, 16, "fp16", seed=21, pad_tokens=3), True, True)


@pytest.mark.parametrize("h,rot", [(16, 64), (128, 64), (33, 32), (3, 8)])
def test_append_of_many_tokens(h, rot):
    """Enough tokens for the kernel's other shape (several rounds of heads to a warp)."""
    c = Case([700, 1, 611], [700, 50, 900], h, 128, rot, 24, seed=22)
    run_append(c, True, True)
    run_append(c, False, False)


def test_append_in_place_and_a_padded_cache():
    for rot, inter in ((64, False), (24, False), (24, True)):
        run_append(Case([2, 1], [9, 30], 5, 64, rot, 8, seed=23, row_pad=16), inter, True, in_place=True)


def test_append_positions_of_the_callers():
    from bit_moe_expert_router_gb300 import attention
    c = Case([3, 1], [9, 30], 4, 128, 64, 8, seed=25)
    table = attention.rope_table(1000, 64, device=DEV, scaling="yarn", factor=4.0, original=250)
    pos = torch.tensor([900, 0, -1, 1000], dtype=torch.int32, device=DEV)  # the last two are outside of the table: padding
    run_append(c, False, True, positions=pos, table=table)


def test_append_skips_pages_that_are_not_there():
    c = Case([4, 2], [20, 10], 4, 128, 64, 8, seed=26)
    c.table_dev[0, 2], c.table_dev[1, 1] = 10 ** 6, -3
    run_append(c, True, True)


def test_append_refusals():
    from bit_moe_expert_router_gb300 import attention, latent
    c = Case([1, 1], [5, 9], 4, 128, 64, 16)
    table = attention.rope_table(32, 64, device=DEV)
    x, k, q = c.normal(2, 128), c.normal(2, 64), c.normal(2, 4, 64)
    for match, prep in (("q_weight", attention.HeadPrep(table, q_weight=torch.ones(128, device=DEV))), ("norm weight", attention.HeadPrep(table, k_weight=torch.ones(64, device=DEV))),
                        ("wide", attention.HeadPrep(attention.rope_table(32, 32, device=DEV))), ("wide", attention.HeadPrep()),
                        ("positions", attention.HeadPrep(table, positions=torch.zeros(3, dtype=torch.int32, device=DEV)))):
        with pytest.raises(ValueError, match=match):
            latent.moe_w4a8_latent_append(c.batch, prep, x, k, q, q)
    prep = attention.HeadPrep(table)
    for error, args in ((ValueError, (x, None, q, q)), (ValueError, (x, k, q[:, :3], q)), (TypeError, (x.half(), k, q, q)), (ValueError, (x[:, :64], k, q, q)),
                        (ValueError, (x, k, q, None))):
        with pytest.raises(error):
            latent.moe_w4a8_latent_append(c.batch, prep, *args)


def test_append_then_attend_is_attention_of_the_whole():
    """A prompt in one piece, in two chunks, and token by token leave the same cache and give the same rows."""
    from bit_moe_expert_router_gb300 import attention, latent
    n, h, dc, rot, page = 90, 16, 512, 64, 16
    g = torch.Generator(device=DEV)
    g.manual_seed(27)
    kv = torch.randn(n, dc + rot, generator=g, device=DEV).bfloat16()
    q_all = torch.randn(n, h, dc + rot, generator=g, device=DEV).bfloat16()
    prep = attention.HeadPrep(attention.rope_table(n, rot, device=DEV), True, k_weight=torch.ones(dc, device=DEV))

    def serve(cuts):
        cache = torch.zeros(8, page, dc + rot, dtype=torch.bfloat16, device=DEV)
        table = torch.tensor([[5, 2, 7, 0, 1, 3]], dtype=torch.int32, device=DEV)
        q_start, lens = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        batch = latent.LatentBatch(cache, table, q_start, lens, n_heads=h, latent_dim=dc, max_q_len=n)
        ws, rows, at = batch.alloc_workspace(), [], 0
        for m in cuts:
            x, k = kv[at:at + m].split([dc, rot], dim=1)
            q = q_all[at:at + m].clone()
            at += m
            q_start[1], lens[0] = m, at
            out = torch.empty(m, h, dc, dtype=torch.bfloat16, device=DEV)
            latent.moe_w4a8_latent_append(batch, prep, x, k, q[..., dc:], q[..., dc:])
            latent.moe_w4a8_latent_attention(batch, q, out, workspace=ws)
            rows.append(out)
        return cache, torch.cat(rows)

    cache, rows = serve([n])
    for cuts in ([33, 57], [50] + [1] * 40, [89, 1]):
        cache2, rows2 = serve(cuts)
        assert torch.equal(cache, cache2)
        # the same weights rounded at other references: within two units of the row's largest value
        assert (rows.float() - rows2.float()).abs().max() <= 2 * torch.finfo(torch.bfloat16).eps * rows.float().abs().max()

"""A decoder layer's serving step: attention over the paged cache, then the routed experts.

``ServingLayer`` strings the operators together as a serving program does: a norm, the fused query/key/value
projection, ``moe_w4a8_kv_append``, ``moe_w4a8_paged_attention``, the output projection, a norm, the router's logits
and ``moe_w4a8_forward_bf16`` on the packed expert bank.  The four dense projections are torch matrix products; nothing
in a step reads anything back to the host.

``LatentServingLayer`` is the same for layers that cache one latent vector per token for all heads and choose their
experts by scores: ``moe_w4a8_latent_append``, ``moe_w4a8_latent_attention`` with the expansion of the latent vector
absorbed into the queries and the output, ``moe_w4a8_route_scored`` and ``moe_w4a8_forward_bf16_routed``.

    python -m bit_moe_expert_router_gb300.serve [latent]

runs a synthetic layer on cuda:0 (seeded random weights): a prompt in two chunks beside a decoding request, then some
decoding steps of both, and prints the time of each kind of step.
"""
from __future__ import annotations

import torch

from . import attention, binding, latent


def rms_norm(x, weight, eps=1e-6):
    y = x.float()
    return (y * torch.rsqrt((y * y).mean(-1, keepdim=True) + eps) * weight).to(x.dtype)


class ServingLayer:
    """One layer with its paged cache, for up to `seqs` sequences of up to `pages_per_seq` pages.

    w: dict of torch CUDA tensors -- norm1, norm2 [H] and q_norm, k_norm [D] float32; wqkv [H, (Hq + 2 Hkv) D], wo [Hq D, H],
    router [H, E] bf16; w13, s13, w2, s2: the expert bank (see the C header).
    """

    def __init__(self, w, n_q_heads, n_kv_heads, head_dim, top_k, n_shared, group, seqs, pages_per_seq, page_size=64, rot_dim=None,
                 base=10000.0):
        self.w, dev = w, w["wqkv"].device
        self.hq, self.hkv, self.d = n_q_heads, n_kv_heads, head_dim
        self.top_k, self.n_shared, self.group = top_k, n_shared, group
        cache = (seqs * pages_per_seq, page_size, n_kv_heads, head_dim)
        i32 = dict(dtype=torch.int32, device=dev)
        # a serving program's allocator hands out pages as sequences grow; here each sequence has its own
        self.block_table = torch.arange(seqs * pages_per_seq, **i32).reshape(seqs, pages_per_seq)
        self.q_start, self.kv_len = torch.zeros(seqs + 1, **i32), torch.zeros(seqs, **i32)
        self.k_cache, self.v_cache = (torch.empty(cache, dtype=torch.bfloat16, device=dev) for _ in range(2))
        self.prep = attention.HeadPrep(attention.rope_table(pages_per_seq * page_size, rot_dim or head_dim, base, device=dev),
                                       q_weight=w["q_norm"], k_weight=w["k_norm"])
        self._batch = attention.KVBatch(self.k_cache, self.v_cache, self.block_table, self.q_start, self.kv_len, n_q_heads=self.hq, max_q_len=1)
        self._attend_workspace, self._moe_workspaces = self._batch.alloc_workspace(), {}

    def batch(self, max_q_len: int) -> attention.KVBatch:
        """The layer's one handle, set for a step of at most max_q_len new tokens per sequence."""
        self._batch.max_q_len = max_q_len
        return self._batch

    def dims(self, tokens: int) -> binding.Dims:
        w13, w2 = self.w["w13"], self.w["w2"]
        return binding.Dims(tokens, w2.shape[1], w13.shape[1] // 2, w13.shape[0] - self.n_shared, self.n_shared, self.top_k, self.group)

    def workspaces(self, tokens: int, batch):
        """(attention's, the experts') for a step of `tokens`.  Attention's does not depend on them.  The experts' is that of
        the next power of two, so all of them together are less than four times what the largest step needs; they are kept, because
        a captured graph holds their addresses."""
        size = 1 << (tokens - 1).bit_length()
        if size not in self._moe_workspaces:
            need = binding.moe_w4a8_forward_bf16_workspace_size(self.dims(size))
            self._moe_workspaces[size] = binding.alloc_workspace(need, self.k_cache.device)
        return self._attend_workspace, self._moe_workspaces[size]

    def forward(self, x, max_q_len: int):
        """x [tokens, H] bf16, the new tokens of all sequences in order; q_start and kv_len hold the step's lengths."""
        w, n = self.w, x.shape[0]
        batch = self.batch(max_q_len)
        ws_attend, ws_moe = self.workspaces(n, batch)
        qkv = (rms_norm(x, w["norm1"]) @ w["wqkv"]).unflatten(1, (self.hq + 2 * self.hkv, self.d))
        q, k, v = qkv.split([self.hq, self.hkv, self.hkv], dim=1)
        attention.moe_w4a8_kv_append(batch, self.prep, q, k, v, q)
        out = torch.empty(n, self.hq, self.d, dtype=x.dtype, device=x.device)
        attention.moe_w4a8_paged_attention(batch, q, out, workspace=ws_attend)
        x = x + out.flatten(1) @ w["wo"]
        y = rms_norm(x, w["norm2"])
        logits = (y @ w["router"]).float()
        moe = torch.empty(n, x.shape[1], dtype=torch.float32, device=x.device)
        binding.moe_w4a8_forward_bf16(y, logits, w["w13"], w["s13"], w["w2"], w["s2"], self.dims(n), moe, ws_moe)
        return (x.float() + moe).to(x.dtype)


class LatentServingLayer:
    """One layer of latent attention with its paged cache, for up to `seqs` sequences of up to `pages_per_seq` pages.

    w: dict of torch CUDA tensors -- norm1, norm2 [H] and latent_norm [Dc] float32; wq [H, heads (Dn + R)] (a head's Dn components
    without a position, then its R rotated ones), wkv [H, Dc + R] (the latent vector, then the key part), wk [heads, Dn, Dc] and wv
    [heads, Dc, Dv] (the latent vector's expansion to a head's keys and values), wo [heads Dv, H], router [H, E] bf16; router_bias
    [E] float32 or None; w13, s13, w2, s2: the expert bank (see the C header).  rule: how the experts are chosen.
    """

    def __init__(self, w, rule: binding.RouteRule, n_shared, group, seqs, pages_per_seq, page_size=64, base=10000.0):
        self.w, self.rule, dev = w, rule, w["wq"].device
        self.heads, self.dn, self.dc = w["wk"].shape
        self.rot = w["wkv"].shape[1] - self.dc
        self.n_shared, self.group = n_shared, group
        self.scale = (self.dn + self.rot) ** -0.5  # of the heads before the absorption
        i32 = dict(dtype=torch.int32, device=dev)
        # a serving program's allocator hands out pages as sequences grow; here each sequence has its own
        self.block_table = torch.arange(seqs * pages_per_seq, **i32).reshape(seqs, pages_per_seq)
        self.q_start, self.kv_len = torch.zeros(seqs + 1, **i32), torch.zeros(seqs, **i32)
        self.cache = torch.empty(seqs * pages_per_seq, page_size, self.dc + self.rot, dtype=torch.bfloat16, device=dev)
        self.prep = attention.HeadPrep(attention.rope_table(pages_per_seq * page_size, self.rot, base, device=dev), interleaved=True,
                                       k_weight=w["latent_norm"])
        self.batch = latent.LatentBatch(self.cache, self.block_table, self.q_start, self.kv_len, n_heads=self.heads, latent_dim=self.dc, max_q_len=1)
        self._attend_workspace, self._moe_workspaces = self.batch.alloc_workspace(), {}

    def dims(self, tokens: int) -> binding.Dims:
        w13, w2 = self.w["w13"], self.w["w2"]
        return binding.Dims(tokens, w2.shape[1], w13.shape[1] // 2, w13.shape[0] - self.n_shared, self.n_shared, self.rule.top_k, self.group)

    def moe_workspace(self, tokens: int):
        """The experts' workspace of the next power of two of tokens, kept: a captured graph holds its address."""
        size = 1 << (tokens - 1).bit_length()
        if size not in self._moe_workspaces:
            need = binding.moe_w4a8_forward_bf16_workspace_size(self.dims(size))
            self._moe_workspaces[size] = binding.alloc_workspace(need, self.cache.device)
        return self._moe_workspaces[size]

    def forward(self, x, max_q_len: int):
        """x [tokens, H] bf16, the new tokens of all sequences in order; q_start and kv_len hold the step's lengths."""
        w, n, dev = self.w, x.shape[0], x.device
        self.batch.max_q_len = max_q_len
        y = rms_norm(x, w["norm1"])
        q_nope, q_rot = (y @ w["wq"]).unflatten(1, (self.heads, self.dn + self.rot)).split([self.dn, self.rot], dim=2)
        c, k_rot = (y @ w["wkv"]).split([self.dc, self.rot], dim=1)
        # a head's query against the latent vectors themselves, its rotated part behind
        q = torch.empty(n, self.heads, self.dc + self.rot, dtype=x.dtype, device=dev)
        q[..., :self.dc] = torch.bmm(q_nope.transpose(0, 1), w["wk"]).transpose(0, 1)
        latent.moe_w4a8_latent_append(self.batch, self.prep, c, k_rot, q_rot, q[..., self.dc:])
        o = torch.empty(n, self.heads, self.dc, dtype=x.dtype, device=dev)
        latent.moe_w4a8_latent_attention(self.batch, q, o, scale=self.scale, workspace=self._attend_workspace)
        x = x + torch.bmm(o.transpose(0, 1), w["wv"]).transpose(0, 1).flatten(1) @ w["wo"]
        y = rms_norm(x, w["norm2"])
        ids = torch.empty(n, self.rule.top_k, dtype=torch.int32, device=dev)
        weights = torch.empty(n, self.rule.top_k, dtype=torch.float32, device=dev)
        logits = torch.mm(y, w["router"], out_dtype=torch.float32)  # (rounded to 16 bits, close experts would change places)
        binding.moe_w4a8_route_scored(logits, self.rule, ids, weights, bias=w["router_bias"])
        moe = torch.empty(n, x.shape[1], dtype=torch.float32, device=dev)
        binding.moe_w4a8_forward_bf16_routed(y, ids, weights, w["w13"], w["s13"], w["w2"], w["s2"], self.dims(n), moe, self.moe_workspace(n))
        return (x.float() + moe).to(x.dtype)


def synthetic_latent_layer(workload, rule, heads, nope, latent_dim, rot_dim, v_dim, seqs, pages_per_seq, device="cuda:0", seed=0, **kw) -> LatentServingLayer:
    """A layer of latent attention with the workload's expert bank and random dense weights."""
    from . import synth
    bank = synth.make_bank(workload)
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    h = workload.H

    def dense(*shape, rows):
        return (torch.randn(*shape, generator=g, device=device) * rows ** -0.5).bfloat16()

    def norm(n):
        return 1.0 + 0.1 * torch.randn(n, generator=g, device=device)

    w = dict(norm1=norm(h), norm2=norm(h), latent_norm=norm(latent_dim), wq=dense(h, heads * (nope + rot_dim), rows=h),
             wkv=dense(h, latent_dim + rot_dim, rows=h), wk=dense(heads, nope, latent_dim, rows=latent_dim), wv=dense(heads, latent_dim, v_dim, rows=latent_dim),
             wo=dense(heads * v_dim, h, rows=heads * v_dim), router=dense(h, workload.E, rows=h),
             router_bias=0.05 * torch.randn(workload.E, generator=g, device=device))
    w.update({name: torch.from_numpy(getattr(bank, name)).to(device) for name in ("w13", "s13", "w2", "s2")})
    return LatentServingLayer(w, rule, workload.S, workload.group, seqs, pages_per_seq, **kw)


def synthetic_layer(workload, n_q_heads, n_kv_heads, head_dim, seqs, pages_per_seq, device="cuda:0", seed=0, **kw) -> ServingLayer:
    """A layer with the workload's expert bank and random dense weights."""
    from . import synth
    bank = synth.make_bank(workload)
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    h = workload.H

    def dense(rows, cols):
        return (torch.randn(rows, cols, generator=g, device=device) * rows ** -0.5).bfloat16()

    def norm(n):
        return 1.0 + 0.1 * torch.randn(n, generator=g, device=device)

    w = dict(norm1=norm(h), norm2=norm(h), q_norm=norm(head_dim), k_norm=norm(head_dim),
             wqkv=dense(h, (n_q_heads + 2 * n_kv_heads) * head_dim), wo=dense(n_q_heads * head_dim, h), router=dense(h, workload.E))
    w.update({name: torch.from_numpy(getattr(bank, name)).to(device) for name in ("w13", "s13", "w2", "s2")})
    return ServingLayer(w, n_q_heads, n_kv_heads, head_dim, workload.top_k, workload.S, workload.group, seqs, pages_per_seq, **kw)


def main(kind: str = "grouped") -> None:
    from . import synth
    w = synth.Workload("serve", T=4, H=2048, I=512, E=64, S=1, top_k=8, group=128)
    if kind == "latent":
        rule = binding.RouteRule(w.E, w.top_k, "sigmoid", n_groups=8, topk_groups=4, group_top=2, scale=2.5)
        layer = synthetic_latent_layer(w, rule, 16, 128, 512, 64, 128, seqs=2, pages_per_seq=64)
    else:
        layer = synthetic_layer(w, 16, 2, 256, seqs=2, pages_per_seq=64, rot_dim=64)
    g = torch.Generator(device="cuda:0")
    g.manual_seed(1)
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    # (new tokens of the sequences) step by step: the second sequence decodes while the first one's prompt comes in chunks
    steps = [(0, 40)] + [(1000, 1), (700, 1)] + [(1, 1)] * 20
    lens = [0, 0]
    for i, q in enumerate(steps):
        lens = [a + b for a, b in zip(lens, q)]
        layer.q_start.copy_(torch.tensor([0, q[0], sum(q)], dtype=torch.int32))
        layer.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        x = torch.randn(sum(q), w.H, generator=g, device="cuda:0").bfloat16()
        start.record()
        y = layer.forward(x, max(q))
        stop.record()
        torch.cuda.synchronize()
        if i < 4 or i == len(steps) - 1:
            print(f"step {i}: new tokens {q}, positions {tuple(lens)}, {start.elapsed_time(stop) * 1e3:.0f} us, rms {y.float().square().mean().sqrt():.3f}")


if __name__ == "__main__":
    import sys
    main(*sys.argv[1:2])

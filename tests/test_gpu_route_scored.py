"""Routing by scores on the GPU against its definition in 64 bits: the chosen experts are the same, in the same order.

Weights.  With e = 2^-24: a sigmoid is expf (2 e) and a sum and a quotient rounded correctly, off by 6 e at most; a softmax
score has a quotient of two exponentials whose arguments |x - max| are rounded (e each) and whose sum is taken of fast
exponentials: off by (16 + E / 8 + 4 |x - max|) e.  Weights divided by their sum are off by three times that and (k + 4) e for the
sum and the quotient; the scale adds e.
"""
import ctypes
import math

import pytest
import torch

E24 = 2.0 ** -24
DEV = "cuda:0"
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def scores(x, score):
    x = x.double()
    if score == "softmax":
        return torch.where(x.isnan(), x, torch.softmax(torch.where(x.isnan(), -math.inf, x), -1))  # (a NaN is left out of the others' sum)
    return torch.where(x >= 0, 1 / (1 + torch.exp(-x.abs())), torch.exp(-x.abs()) / (1 + torch.exp(-x.abs())))


def reference(x, k, score, bias, groups, kept, top, renorm, scale):
    s = scores(x, score)
    r = s if bias is None else s + bias.double()
    choice = x.double() if bias is None else r
    choice = torch.where(choice.isnan(), -1e300, choice.clamp_min(-1e200))  # a NaN behind all numbers
    t, e = x.shape
    if kept < groups:
        by = r if bias is not None or top == 2 else x.double()
        by = torch.where(by.isnan(), -math.inf, by).unflatten(1, (groups, -1))
        value = by.sort(dim=-1, descending=True).values[..., :top].sum(-1)
        order = value.sort(dim=-1, descending=True, stable=True).indices[:, :kept]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, order, True)
        choice = torch.where(keep[..., None], choice.unflatten(1, (groups, -1)), -math.inf).flatten(1)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, ids)
    if renorm:
        log_s = torch.where(x.isnan(), math.nan, x.double()) if score == "softmax" else -torch.logaddexp(torch.zeros_like(s), -x.double())
        w = torch.softmax(log_s.gather(1, ids), -1)
    rel = (16 + e / 8 + 4 * (x.double().amax(-1, keepdim=True) - x.double().gather(1, ids)).nan_to_num(0, 0, 0).abs()) * E24 if score == "softmax" else 6 * E24
    tol = ((3 * rel + (k + 4) * E24 if renorm else rel) + E24) * w.abs() * abs(scale)
    return ids.int(), w * scale, tol + 1e-37


def run(x, k, score="softmax", bias=None, groups=1, kept=1, top=1, renorm=True, scale=1.0):
    from bit_moe_expert_router_gb300 import binding
    rule = binding.RouteRule(x.shape[1], k, score, groups, kept, top, renorm, scale)
    ids = torch.full((x.shape[0], k), -5, dtype=torch.int32, device=DEV)
    w = torch.full((x.shape[0], k), 55.0, device=DEV)
    binding.moe_w4a8_route_scored(x, rule, ids, w, bias=bias)
    return ids, w


def check(x, k, score="softmax", bias=None, groups=1, kept=1, top=1, renorm=True, scale=1.0):
    ids, w = run(x, k, score, bias, groups, kept, top, renorm, scale)
    ref, want, tol = reference(x, k, score, bias, groups, kept, top, renorm, scale)
    wrong = (ids != ref).any(-1)
    assert not wrong.any(), f"{int(wrong.sum())} tokens choose other experts, the first {int(wrong.nonzero()[0])}: {ids[wrong][0].tolist()} for {ref[wrong][0].tolist()}"
    assert torch.equal(w.isnan(), want.isnan())
    err = torch.nan_to_num((w.double() - want).abs() - tol, nan=0.0)
    assert err.max() <= 0, f"weights are {err.max().item():.3e} beyond their bound"
    return ids, w


def logits(t, e, dtype="fp32", seed=0, size=1.5):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(t, e, generator=g, device=DEV) * size).to(DTYPES[dtype]), g


GROUPS = [(1, 1, 1), (8, 4, 2), (8, 3, 1), (4, 1, 2), (2, 2, 1), (32, 9, 1), (16, 5, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("groups,kept,top", GROUPS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_groups_scores_and_biases(cuda_lib, groups, kept, top, score, biased):
    for e, k, dtype in ((64, 2, "fp32"), (160, 5, "bf16"), (256, 8, "fp32"), (512, 10, "fp16"), (1024, 32, "fp32"), (96, 3, "fp16")):
        x, g = logits(300, e, dtype, seed=e + groups)
        size = 0.05 if score == "sigmoid" else 0.3 / e
        bias = torch.randn(e, generator=g, device=DEV) * size if biased else None
        check(x, min(k, kept * (e // groups)), score, bias, groups, kept, top, renorm=k % 2 == 0, scale=2.5)


@pytest.mark.gpu
@pytest.mark.parametrize("e", [1, 2, 3, 5, 31, 32, 33, 63, 100, 257, 384, 1000])
def test_sizes(cuda_lib, e):
    for k in sorted({1, min(e, 7), min(e, 31), min(e, 32)}):
        for dtype in DTYPES:
            x, g = logits(5, e, dtype, seed=k)
            for score in ("softmax", "sigmoid"):
                for bias in (None, torch.randn(e, generator=g, device=DEV)):
                    check(x, k, score, bias, renorm=bool(k % 2))


@pytest.mark.gpu
def test_many_tokens(cuda_lib):
    """Among 60000 tokens some hundred have candidates closer together than fp32 can tell apart."""
    x, g = logits(60000, 256, seed=1)
    bias = torch.randn(256, generator=g, device=DEV) * 0.05
    check(x, 8, "sigmoid", bias, 8, 4, 2, True, 2.5)
    check(x, 8, "softmax", bias / 64, 8, 4, 2, True, 1.0)
    check(x, 8, "softmax", None, 8, 4, 2, False, 1.0)


@pytest.mark.gpu
def test_equal_and_nearly_equal_candidates(cuda_lib):
    x = torch.zeros(9, 96, device=DEV)
    for bias in (None, torch.zeros(96, device=DEV)):
        for groups, kept in ((1, 1), (8, 3)):
            ids, _ = check(x, 12, "sigmoid", bias, groups, kept)
            assert torch.equal(ids[0], torch.arange(12, dtype=torch.int32, device=DEV))
    # few different values, so that many are the same, also across the border of the list
    for dtype in DTYPES:
        x, g = logits(400, 256, dtype, seed=2)
        x = (x * 2).round() / 2
        some = torch.randint(0, 2, (256,), generator=g, device=DEV).float() * 0.25
        for bias in (None, torch.zeros(256, device=DEV), some):
            for groups, kept, top in ((1, 1, 1), (8, 4, 2), (4, 2, 1)):
                if bias is some or top == 2:
                    continue  # (sums of different scores that come out the same are no business of a test)
                check(x, 8, "sigmoid", bias, groups, kept, top)
                check(x, 8, "softmax", bias, groups, kept, top)
    # neighbours in fp32: the keys' low bits decide
    base = torch.randn(400, 1, generator=g, device=DEV)
    steps = torch.randint(0, 12, (400, 128), generator=g, device=DEV)
    for x in ((base.view(torch.int32) + steps.int()).view(torch.float32),
              (base.view(torch.int32) + steps).view(torch.float32)):  # (the halves of 64-bit numbers: zeros and NaN among them)
        check(x, 8)
        check(x, 32, "sigmoid", None, 4, 2)
    # scores that the bias brings together to within 1e-9 and less
    x, g = logits(400, 64, seed=3)
    bias = (0.5 - scores(x[:1], "sigmoid")[0]).float()
    x = x[:1] + torch.randn(400, 64, generator=g, device=DEV) * 1e-8
    check(x, 8, "sigmoid", bias)
    check(x, 8, "sigmoid", bias, 8, 4, 2)
    check(x, 32, "sigmoid", bias)


@pytest.mark.gpu
def test_far_logits(cuda_lib):
    """Scores that vanish in fp32, infinities and NaN."""
    x, g = logits(64, 128, seed=4)
    check(x * 40, 8, "sigmoid")
    check(x * 40, 8, "softmax", renorm=True)
    check(x - 150, 8, "sigmoid", renorm=True)
    check(x + 150, 8, "sigmoid", renorm=True)
    check(x - 150, 8, "sigmoid", torch.randn(128, generator=g, device=DEV), renorm=False)
    y = x.clone()
    y[:, ::3] = -math.inf
    y[0] = -math.inf
    y[0, 5:20] = 1.0
    for bias in (None, torch.randn(128, generator=g, device=DEV)):
        check(y, 8, "sigmoid", bias)
        check(y, 8, "softmax", bias, renorm=False)
        check(y, 8, "sigmoid", bias, 8, 4, 2)
    z = x.clone()
    z[:, 7] = math.nan
    z[3] = math.nan
    z[4, 8:] = math.nan
    for bias in (None, torch.randn(128, generator=g, device=DEV)):
        check(z, 8, "sigmoid", bias)
        check(z, 8, "sigmoid", bias, 8, 2, 1)
    check(z, 8, "softmax")


@pytest.mark.gpu
def test_strides_streams_and_graphs(cuda_lib):
    from bit_moe_expert_router_gb300 import binding
    for e, pad in ((256, 64), (256, 3), (160, 7)):
        wide, g = logits(70, e + pad, seed=5)
        bias = torch.randn(e, generator=g, device=DEV) * 0.05
        ids, w = check(wide[:, :e], 8, "sigmoid", bias, 8, 4, 2)
        rule = binding.RouteRule(e, 8, "sigmoid", 8, 4, 2)
        ids2, w2 = torch.zeros_like(ids), torch.zeros_like(w)
        side = torch.cuda.Stream(DEV)
        side.wait_stream(torch.cuda.current_stream(DEV))
        with torch.cuda.stream(side):
            binding.moe_w4a8_route_scored(wide[:, :e], rule, ids2, w2, bias=bias)
        torch.cuda.current_stream(DEV).wait_stream(side)
        assert torch.equal(ids, ids2) and torch.equal(w, w2)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            binding.moe_w4a8_route_scored(wide[:, :e], rule, ids2, w2, bias=bias)
        wide.copy_(torch.randn(wide.shape, generator=g, device=DEV))
        graph.replay()
        ids, w = check(wide[:, :e], 8, "sigmoid", bias, 8, 4, 2)
        assert torch.equal(ids, ids2) and torch.equal(w, w2)
    empty = torch.empty(0, 64, device=DEV)
    run(empty, 4)


@pytest.mark.gpu
def test_softmax_without_groups_is_the_routers_choice(cuda_lib):
    """The rule that moe_w4a8_route has: the same experts, and weights to the last bits."""
    from bit_moe_expert_router_gb300 import binding
    x, _ = logits(513, 512, seed=6)
    d = binding.dims_of(513, 128, 64, 512, 0, 10, 32)
    i32 = dict(dtype=torch.int32, device=DEV)
    ids, w = torch.empty(513, 10, **i32), torch.empty(513, 10, device=DEV)
    n = 513 * 10
    binding.moe_w4a8_route(x, d, ids, w, torch.empty(512, **i32), torch.empty(513, **i32), torch.empty(n, **i32), torch.empty(n, **i32),
                           binding.alloc_workspace(binding.moe_w4a8_workspace_size(d), DEV))
    got, gw = run(x, 10)
    assert torch.equal(ids, got)
    assert (gw - w).abs().max() <= 16 * E24


@pytest.mark.gpu
def test_the_experts_take_the_choice(cuda_lib):
    """forward_bf16_routed with the chosen experts is forward_routed on the quantised activations, on every engine."""
    import _gpu_helpers as gh
    from bit_moe_expert_router_gb300 import binding, synth
    for w in (synth.Workload("rs_dec", T=4, H=2048, I=512, E=16, S=1, top_k=4, group=128), synth.Workload("rs_tc", T=300, H=256, I=128, E=8, S=1, top_k=2, group=128),
              synth.WORKLOADS["tiny"]):
        d, bank = gh.dims(w), gh.device_bank(w)
        x, g = logits(w.T, w.H, "bf16", seed=7)
        r, _ = logits(w.T, w.E, seed=8)
        ids, wt = run(r, w.top_k, "sigmoid", torch.randn(w.E, generator=g, device=DEV) * 0.1, renorm=True, scale=2.5)
        out, ref = (torch.full((w.T, w.H), math.nan, device=DEV) for _ in range(2))
        binding.moe_w4a8_forward_bf16_routed(x, ids, wt, *bank, d, out, binding.alloc_workspace(binding.moe_w4a8_forward_bf16_workspace_size(d), DEV))
        xs = x.float().abs().amax(-1) / torch.full((w.T,), 127.0, device=DEV)  # (by a number it would be a product)
        xq = (x.float() / xs[:, None]).round().clamp(-127, 127).to(torch.int8)
        binding.moe_w4a8_forward_routed(xq, xs, ids, wt, *bank, d, ref, binding.alloc_workspace(binding.moe_w4a8_workspace_size(d), DEV))
        assert out.isfinite().all() and torch.equal(out, ref)


# ------------------------------------------------------------------------------------------------ refusals
FAKE = 0x100000  # never dereferenced: every call below is refused, or has no tokens
GOOD = dict(n_experts=64, top_k=4, score=1, n_groups=8, topk_groups=4, group_top=2, renormalise=1, scale=2.5)


def _route(lib, n=2, logits=FAKE, stride=64, dtype=0, bias=FAKE, ids=FAKE, w=FAKE, rule=True, **kw):
    from bit_moe_expert_router_gb300 import binding
    r = binding._RouteRule(**{**GOOD, **kw})
    return lib.moe_w4a8_route_scored(ctypes.byref(r) if rule else None, n, logits, stride, dtype, bias, ids, w, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n_experts=0), 1), (dict(top_k=0), 1), (dict(top_k=65), 1), (dict(score=2), 1), (dict(score=-1), 1), (dict(n_groups=0), 1), (dict(n_groups=7), 1),
    (dict(topk_groups=0), 1), (dict(topk_groups=9), 1), (dict(group_top=0), 1), (dict(group_top=3), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1),
    (dict(top_k=9, topk_groups=1), 1), (dict(n_groups=64), 1), (dict(stride=63), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(n=-1), 1),
    (dict(logits=None), 1), (dict(logits=FAKE + 4), 1), (dict(bias=FAKE + 8), 1), (dict(ids=None), 1), (dict(w=FAKE + 4), 1), (dict(rule=False), 1),
    (dict(n_experts=2048, stride=2048), 2), (dict(top_k=33, topk_groups=8), 2), (dict(n_experts=60, n_groups=6, topk_groups=4), 2),
    (dict(n_experts=128, n_groups=64, stride=128), 2), (dict(n=(1 << 24) + 1), 2), (dict(n=0), 0), (dict(n=0, logits=None, ids=None, w=None, bias=None), 0)])
def test_refusals(cuda_lib, kw, status):
    from bit_moe_expert_router_gb300 import binding
    assert _route(binding._load(), **kw) == status


def test_the_binding_refuses(cuda_lib):
    from bit_moe_expert_router_gb300 import binding
    with pytest.raises(ValueError, match="score"):
        binding.RouteRule(64, 4, "tanh")
    for kw in (dict(top_k=65), dict(n_groups=3), dict(n_groups=8, topk_groups=9), dict(group_top=3), dict(scale=math.nan)):
        with pytest.raises(binding.MoeError):
            binding.RouteRule(64, **{**dict(top_k=4), **kw})
    rule = binding.RouteRule(64, 4)
    ids, w = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 4)
    with pytest.raises(TypeError, match="dtype"):
        binding.moe_w4a8_route_scored(torch.zeros(2, 64, dtype=torch.float64), rule, ids, w)
    with pytest.raises(ValueError, match="CUDA"):
        binding.moe_w4a8_route_scored(torch.zeros(2, 64), rule, ids, w)


@pytest.mark.gpu
def test_the_binding_refuses_on_the_device(cuda_lib):
    from bit_moe_expert_router_gb300 import binding
    rule = binding.RouteRule(64, 4)
    x, ids, w = torch.zeros(2, 64, device=DEV), torch.zeros(2, 4, dtype=torch.int32, device=DEV), torch.zeros(2, 4, device=DEV)
    for error, args, kw in ((ValueError, (x[:, :32], rule, ids, w), {}), (ValueError, (x.t().contiguous().t(), rule, ids, w), {}), (TypeError, (x, rule, ids.long(), w), {}),
                            (ValueError, (x, rule, ids[:1], w), {}), (ValueError, (x, rule, ids, w.cpu()), {}), (ValueError, (x, rule, ids, w), dict(bias=torch.zeros(63, device=DEV))),
                            (TypeError, (x, rule, ids, w), dict(bias=torch.zeros(64, device=DEV).half())), (ValueError, (x, rule, None, w), {})):
        with pytest.raises(error):
            binding.moe_w4a8_route_scored(*args, **kw)

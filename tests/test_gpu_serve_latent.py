"""The serving layer of latent attention: append, attention, scored routing and the routed experts in one step."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")


def _layer():
    from bit_moe_expert_router_gb300 import binding, serve, synth
    w = synth.Workload("serve_latent_test", T=4, H=256, I=128, E=16, S=1, top_k=3, group=128)
    rule = binding.RouteRule(16, 3, "sigmoid", n_groups=4, topk_groups=2, group_top=2, scale=2.5)
    return serve.synthetic_latent_layer(w, rule, 8, 32, 128, 32, 48, seqs=2, pages_per_seq=6, page_size=16)


def _set(layer, q, lens):
    layer.q_start.copy_(torch.tensor([0, q[0], q[0] + q[1]], dtype=torch.int32))
    layer.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))


def _plain(layer, x):
    """The layer on one whole sequence with attention in the expanded form, in fp32 from the same weights; the experts through the
    library's own layer call, with the experts that the plain formula picks."""
    from bit_moe_expert_router_gb300 import attention, binding, serve
    n, p = x.shape[0], layer.w
    y = serve.rms_norm(x, p["norm1"])
    q = (y @ p["wq"]).unflatten(1, (8, 64)).float()
    kv = (y @ p["wkv"]).float()
    table = attention.rope_table(n, 32, device=x.device)
    cos, sin = table[:, :16], table[:, 16:]

    def turn(t, c, s):
        a, b = t[..., 0::2], t[..., 1::2]
        return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2).bfloat16().float()

    latent = kv[:, :128]
    latent = (latent * torch.rsqrt((latent * latent).mean(-1, keepdim=True) + 1e-6) * p["latent_norm"]).bfloat16().float()
    k_nope = torch.einsum("kc,hnc->khn", latent, p["wk"].float())
    v = torch.einsum("kc,hcv->khv", latent, p["wv"].float())
    k_rot = turn(kv[:, 128:], cos, sin)
    s = torch.einsum("qhn,khn->hqk", q[..., :32], k_nope) + torch.einsum("qhr,kr->hqk", turn(q[..., 32:], cos[:, None], sin[:, None]), k_rot)
    s = (s / 8).masked_fill(torch.ones(n, n, device=x.device).triu(1).bool(), float("-inf"))
    o = torch.einsum("hqk,khv->qhv", s.softmax(-1), v).bfloat16()
    x = x + o.flatten(1) @ p["wo"]
    y = serve.rms_norm(x, p["norm2"])
    score = (y @ p["router"]).double().sigmoid()
    r = (score + p["router_bias"].double()).unflatten(1, (4, 4))
    keep = torch.zeros(n, 4, dtype=torch.bool, device=x.device).scatter_(1, r.topk(2, dim=-1).values.sum(-1).topk(2, dim=1).indices, True)
    ids = r.masked_fill(~keep[..., None], -1e9).flatten(1).topk(3, dim=1).indices
    w = score.gather(1, ids)
    w = (w / w.sum(-1, keepdim=True) * 2.5).float()
    d = layer.dims(n)
    out = torch.empty(n, 256, device=x.device)
    binding.moe_w4a8_forward_bf16_routed(y, ids.int().contiguous(), w, p["w13"], p["s13"], p["w2"], p["s2"], d, out,
                                         binding.alloc_workspace(binding.moe_w4a8_forward_bf16_workspace_size(d), x.device))
    return (x.float() + out).bfloat16()


def test_prompt_in_chunks_and_decoding_is_the_whole():
    """Two sequences, chunks and single tokens beside one another, in the absorbed form: each row as from its whole sequence at
    once in the expanded form.  The two round the rows differently (bf16), which can move a token's routing; most rows stay within
    a few roundings, as the median and the 90th percentile show."""
    layer = _layer()
    g = torch.Generator(device="cuda:0")
    g.manual_seed(3)
    xs = [torch.randn(n, 256, generator=g, device="cuda:0").bfloat16() for n in (70, 41)]
    got, at = [[], []], [0, 0]
    for q in [(30, 1), (0, 20), (39, 1)] + [(0, 1)] * 18 + [(1, 1)]:
        rows = [x[a:a + n] for x, a, n in zip(xs, at, q)]
        at = [a + n for a, n in zip(at, q)]
        _set(layer, q, at)
        y = layer.forward(torch.cat(rows), max(q))
        got[0].append(y[:q[0]])
        got[1].append(y[q[0]:])
    assert at == [70, 41]
    for x, parts in zip(xs, got):
        ref = _plain(layer, x).float()
        err = (torch.cat(parts).float() - ref).abs().amax(-1) / ref.abs().amax(-1)
        assert err.isfinite().all()
        assert err.median() <= 2.0 ** -6 and err.quantile(0.9) <= 2.0 ** -4


def test_a_decoding_step_is_captured_and_replayed():
    layer = _layer()
    g = torch.Generator(device="cuda:0")
    g.manual_seed(4)
    _set(layer, (20, 9), (20, 9))
    layer.forward(torch.randn(29, 256, generator=g, device="cuda:0").bfloat16(), 20)
    x = torch.randn(2, 256, generator=g, device="cuda:0").bfloat16()
    _set(layer, (1, 1), (21, 10))
    layer.forward(x, 1)  # (warm-up: workspaces)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.forward(x, 1)
    for step in range(3):
        x.copy_(torch.randn(2, 256, generator=g, device="cuda:0").bfloat16())
        _set(layer, (1, 1), (21 + step, 10 + step))
        graph.replay()
        got = out.clone()
        assert torch.equal(got, layer.forward(x, 1))


def test_the_command_runs(capsys):
    from bit_moe_expert_router_gb300 import serve
    serve.main("latent")
    out = capsys.readouterr().out
    assert out.count("step") == 5 and "nan" not in out

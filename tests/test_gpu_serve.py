"""The serving layer: the attention operators and the routed experts in one step, as a program runs them."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")


def _layer():
    from bit_moe_expert_router_gb300 import serve, synth
    w = synth.Workload("serve_test", T=4, H=256, I=128, E=8, S=1, top_k=2, group=128)
    return w, serve.synthetic_layer(w, 8, 2, 64, seqs=2, pages_per_seq=6, page_size=16, rot_dim=32)


def _set(layer, q, lens):
    layer.q_start.copy_(torch.tensor([0, q[0], q[0] + q[1]], dtype=torch.int32))
    layer.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))


def _plain(layer, w, x):
    """The layer in fp32 on one whole sequence, from the same weights: attention by its formula, the experts through
    the library's own layer call (its parity is tested elsewhere)."""
    from bit_moe_expert_router_gb300 import attention, binding, serve
    n, p = x.shape[0], layer.w
    qkv = (serve.rms_norm(x, p["norm1"]) @ p["wqkv"]).unflatten(1, (12, 64)).float()
    q, k, v = qkv.split([8, 2, 2], dim=1)
    table = attention.rope_table(n, 32, device=x.device)
    c, s = table[:, None, :16], table[:, None, 16:]

    def head(y, weight):
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight
        a, b = y[..., :16], y[..., 16:32]
        return torch.cat([a * c - b * s, b * c + a * s, y[..., 32:]], -1).bfloat16().float()

    q, k = head(q, p["q_norm"]), head(k, p["k_norm"])
    k, v = (t.repeat_interleave(4, dim=1) for t in (k, v))
    sc = torch.einsum("qhd,khd->hqk", q, k) / 8
    sc = sc.masked_fill(torch.ones(n, n, device=x.device).triu(1).bool(), float("-inf"))
    o = torch.einsum("hqk,khd->qhd", sc.softmax(-1), v).bfloat16()
    x = x + o.flatten(1) @ p["wo"]
    y = serve.rms_norm(x, p["norm2"])
    d = layer.dims(n)
    out = torch.empty(n, 256, device=x.device)
    binding.moe_w4a8_forward_bf16(y, (y @ p["router"]).float(), p["w13"], p["s13"], p["w2"], p["s2"], d, out,
                                  binding.alloc_workspace(binding.moe_w4a8_forward_bf16_workspace_size(d), x.device))
    return (x.float() + out).bfloat16()


def test_prompt_in_chunks_and_decoding_is_the_whole():
    """Two sequences, chunks and single tokens beside one another: each row as from its whole sequence at once.  The two
    paths round attention's rows differently (bf16), which can move a token's routing; most rows stay within a few
    roundings, as the median and the 90th percentile show."""
    w, layer = _layer()
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
        ref = _plain(layer, w, x).float()
        err = (torch.cat(parts).float() - ref).abs().amax(-1) / ref.abs().amax(-1)
        assert err.isfinite().all()
        assert err.median() <= 2.0 ** -6 and err.quantile(0.9) <= 2.0 ** -4


def test_the_command_runs(capsys):
    from bit_moe_expert_router_gb300 import serve
    serve.main()
    out = capsys.readouterr().out
    assert out.count("step") == 5 and "nan" not in out

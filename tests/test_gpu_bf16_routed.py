"""moe_w4a8_forward_bf16_routed with every routing that its description allows: an expert twice in a token, ids outside the bank, weights of any
sign, a captured and replayed call, a token count of zero and one; on each engine equal to moe_w4a8_forward_routed on the quantised activations."""
import pytest
import torch

import _gpu_helpers as gh
from bit_moe_expert_router_gb300 import binding, synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LAYERS = {"decode": (synth.Workload("br_dec", T=4, H=2048, I=512, E=16, S=1, top_k=4, group=128), 1),
          "tcgen05": (synth.Workload("br_tc", T=300, H=256, I=128, E=8, S=1, top_k=2, group=128), 2),
          "grouped": (synth.WORKLOADS["tiny"], 0)}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")


def _quantised(x):
    scale = x.float().abs().amax(-1) / torch.full((x.shape[0],), 127.0, device=DEV)  # (by a number it would be a product)
    return (x.float() / scale[:, None]).round().clamp(-127, 127).to(torch.int8), scale


@pytest.mark.parametrize("name", LAYERS)
def test_routings_of_every_kind(name):
    w, engine = LAYERS[name]
    d, bank = gh.dims(w), gh.device_bank(w)
    assert binding.moe_w4a8_engine_for(d) == engine
    g = torch.Generator(device=DEV)
    g.manual_seed(80)
    x = torch.randn(w.T, w.H, generator=g, device=DEV).bfloat16()
    xq, xs = _quantised(x)
    wt = torch.randn(w.T, w.top_k, generator=g, device=DEV)
    ids = torch.stack([torch.randperm(w.E, generator=g, device=DEV)[:w.top_k] for _ in range(w.T)]).int()
    twice, outside = ids.clone(), ids.clone()
    twice[:, 1] = twice[:, 0]
    outside[0, 0], outside[-1, -1], outside[w.T // 2, 0] = -1, w.E, 2 ** 31 - 1
    workspace = binding.alloc_workspace(binding.moe_w4a8_forward_bf16_workspace_size(d), DEV)
    out, ref = (torch.empty(w.T, w.H, device=DEV) for _ in range(2))
    given = torch.empty_like(ids)

    def call():
        binding.moe_w4a8_forward_bf16_routed(x, given, wt, *bank, d, out, workspace)

    given.copy_(ids)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for routing, clamped in ((ids, ids), (twice, twice), (torch.full_like(ids, 3), torch.full_like(ids, 3)), (outside, outside.clamp(0, w.E - 1))):
        binding.moe_w4a8_forward_routed(xq, xs, clamped, wt, *bank, d, ref, binding.alloc_workspace(binding.moe_w4a8_workspace_size(d), DEV))
        assert ref.isfinite().all()
        given.copy_(routing)
        for run in (call, graph.replay):
            out.fill_(float("nan"))
            run()
            assert binding.moe_w4a8_device_status(workspace) == 0
            assert torch.equal(out, ref)


@pytest.mark.parametrize("name", LAYERS)
def test_no_token_and_one(name):
    w, _ = LAYERS[name]
    bank = gh.device_bank(w)
    g = torch.Generator(device=DEV)
    g.manual_seed(81)
    for n in (0, 1):
        d = binding.Dims(n, w.H, w.I, w.E, w.S, w.top_k, w.group)
        x = torch.randn(n, w.H, generator=g, device=DEV).bfloat16()
        ids, wt = torch.arange(w.top_k, dtype=torch.int32, device=DEV).expand(n, -1).contiguous(), torch.ones(n, w.top_k, device=DEV)
        out, ref = (torch.zeros(n, w.H, device=DEV) for _ in range(2))
        binding.moe_w4a8_forward_bf16_routed(x, ids, wt, *bank, d, out, binding.alloc_workspace(binding.moe_w4a8_forward_bf16_workspace_size(d), DEV))
        if n:
            binding.moe_w4a8_forward_routed(*_quantised(x), ids, wt, *bank, d, ref, binding.alloc_workspace(binding.moe_w4a8_workspace_size(d), DEV))
        assert torch.equal(out, ref)

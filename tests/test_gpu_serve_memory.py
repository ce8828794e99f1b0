"""What a serving layer holds on the device does not grow with the number of different steps that it has run."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")


def test_many_token_counts_and_lengths_hold_no_more_than_the_largest():
    from bit_moe_expert_router_gb300 import binding, serve, synth
    w = synth.Workload("serve_memory", T=4, H=256, I=128, E=8, S=1, top_k=2, group=128)
    layer = serve.synthetic_layer(w, 8, 2, 64, seqs=2, pages_per_seq=8, page_size=16, rot_dim=32)

    def step(n, m):  # n tokens of the first sequence's prompt, m of the second's
        layer.q_start.copy_(torch.tensor([0, n, n + m], dtype=torch.int32))
        layer.kv_len.copy_(torch.tensor([n, m], dtype=torch.int32))
        x = torch.ones(n + m, 256, dtype=torch.bfloat16, device="cuda:0")
        assert layer.forward(x, max(n, m)).isfinite().all()

    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for n in range(1, 97):
        step(n, 1 + n % 32)
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated() - before
    attend = layer.batch(1).workspace_size()
    experts = binding.moe_w4a8_forward_bf16_workspace_size(layer.dims(128))
    matmul = 128 << 20  # what torch's products keep for themselves
    assert held <= attend + 4 * experts + matmul, f"{held >> 20} MiB held, of which attention needs {attend >> 20} and the experts {experts >> 20}"
    assert 96 * attend > 2 * (attend + 4 * experts + matmul)  # (one for each count would not have passed)


def test_the_bound_on_new_tokens_can_be_set():
    from test_gpu_attention import Case
    c = Case([300, 129], [300, 650], 8, 2, 64, 16, seed=70)
    for n in (1, 7, 4096):
        c.batch.max_q_len = n
        assert c.batch.max_q_len == n
        c.check()
    with pytest.raises(ValueError, match="max_q_len"):
        c.batch.max_q_len = 0

"""Which kernels a call launches: those that some sequence of the batch can need, and no others."""
import pytest
import torch
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from bit_moe_expert_router_gb300 import attention
    attention._load()


def launches(c):
    """How many kernels a call launches: the nodes of its captured graph."""
    import ctypes

    from bit_moe_expert_router_gb300 import attention
    ws, out = c.batch.alloc_workspace(), torch.zeros_like(c.q)
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        attention.moe_w4a8_paged_attention(c.batch, c.q, out, workspace=ws)
    n = ctypes.c_size_t(0)
    runtime = ctypes.CDLL(f"libcudart.so.{torch.version.cuda.split('.')[0]}")
    assert runtime.cudaGraphGetNodes(ctypes.c_void_p(graph.raw_cuda_graph()), None, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("hq,kernels", [(8, 4), (32, 4), (34, 2), (64, 2)])
def test_a_ragged_batch_launches_the_split_engine_where_a_sequence_can_have_so_few_rows(hq, kernels):
    """Each engine has a kernel and a join; with more than 16 heads to a group no sequence has 16 rows or fewer."""
    c = Case([120, 1, 90, 30], [200, 700, 90, 400], hq, 2, 64, 16, "fp16", seed=80)
    c.check()
    assert launches(c) == kernels

"""What is written to the batch's arrays just before a call, in the stream and without a wait on the host, is what the call
reads, also where two kernels share the batch and the second begins beside the first."""
import pytest
import torch
from _attention_reference import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from bit_moe_expert_router_gb300 import attention
    attention._load()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_lengths_pages_and_rows_written_just_before(d):
    from bit_moe_expert_router_gb300 import attention
    # two batches of the same shape over one cache: decoding requests beside chunks, in another order and with other lengths
    a = Batch([1, 200, 1, 1, 90], [700, 640, 30, 1500, 90], 8, 2, d, 16, seed=60)
    b = Batch([90, 1, 1, 200, 1], [300, 900, 1, 300, 1200], 8, 2, d, 16, seed=61)
    width = max(a.table_dev.shape[1], b.table_dev.shape[1])
    tables = [torch.nn.functional.pad(c.table_dev, (0, width - c.table_dev.shape[1]), value=-1) + at
              for c, at in ((a, 0), (b, a.k_cache.shape[0]))]
    sides = list(zip((a, b), tables))
    pages = a.k_cache.shape[0] + b.k_cache.shape[0]
    k, v = (torch.zeros(pages, 16, 2, d, dtype=a.dt, device=a.q.device) for _ in range(2))
    table, start, lens, q = torch.empty_like(tables[0]), torch.empty_like(a.q_start), torch.empty_like(a.lens), torch.empty_like(a.q)
    batch = attention.KVBatch(k, v, table, start, lens, n_q_heads=8, max_q_len=200)
    ws = batch.alloc_workspace()

    def step(i, out):
        c, ids = sides[i % 2]
        k.zero_(), v.zero_()  # (another step's rows are gone)
        first = 0 if c is a else a.k_cache.shape[0]
        k[first:first + c.k_cache.shape[0]].copy_(c.k_cache)
        v[first:first + c.v_cache.shape[0]].copy_(c.v_cache)
        table.copy_(ids), start.copy_(c.q_start), lens.copy_(c.lens), q.copy_(c.q)
        attention.moe_w4a8_paged_attention(batch, q, out, workspace=ws)

    outs = [torch.zeros_like(q) for _ in range(12)]
    for i, out in enumerate(outs):
        step(i, out)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        ref, _, tol, _ = sides[i % 2][0].reference()
        assert ((out.double() - ref).abs() <= tol).all(), f"step {i}"

"""How a batch's work is dealt over the GPU: batches at and above the 32 sequences that one warp deals, sequences of many row tiles
among short ones, on both engines, up to the most sequences that a call takes."""
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


def lengths(n, long):
    """n sequences of up to 90 new tokens and 500 positions (some empty), `long` of them of 1100 to 1500 new tokens."""
    q = [(37 * i + 5) % 91 for i in range(n)]
    kv = [m + (113 * i) % 410 if i % 7 else (13 * i) % 40 for i, m in enumerate(q)]
    for x in range(long):
        i = (x * n) // long + 2
        q[i] = 1100 + 190 * x
        kv[i] = q[i] + 77 * x
    return q, kv


@pytest.mark.parametrize("n,long", [(32, 2), (33, 1), (40, 3), (100, 0)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_chunks_of_many_sequences(n, long, d):
    Batch(*lengths(n, long), 8, 2, d, 16, seed=90).check()


@pytest.mark.parametrize("window", [0, 100])
def test_long_and_short_sequences_with_a_window(window):
    Batch(*lengths(48, 2), 8, 2, 64, 32, "fp16", "head", seed=91).check(window=window)


@pytest.mark.parametrize("n,long", [(32, 1), (45, 2)])
@pytest.mark.parametrize("d", [64, 256])
def test_chunks_from_pages_that_boxes_do_not_divide(n, long, d):
    """Odd pages: every row tile goes to the split engine, hundreds of them to a long sequence."""
    Batch(*lengths(n, long), 4, 2, d, 5, seed=92).check()


@pytest.mark.parametrize("q", [1, 5])
def test_the_most_sequences(q):
    n = 2048
    Batch([q if i % 5 else 0 for i in range(n)], [(7 * i) % 60 for i in range(n)], 8, 2, 64, 16, "fp16", seed=93).check()

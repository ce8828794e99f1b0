"""Windows so large that positions less a window leave 32 bits, with tokens before position zero: no window at all."""
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


@pytest.mark.parametrize("window", [2 ** 31 - 2, 2 ** 31 - 1, 2 ** 31, 1 << 40, 2 ** 62, 2 ** 63 - 1])
@pytest.mark.parametrize("lengths", [([4, 3], [2, 0]), ([8], [5]), ([60, 9], [50, 4]), ([300, 1], [280, 1000])])
@pytest.mark.parametrize("d", [64, 128])
def test_windows_beyond_32_bits(lengths, window, d):
    c = Batch(*lengths, 8, 2, d, 16, seed=50)
    out, lse = c.check(window=window)
    plain, plain_lse = c.attend()
    assert torch.equal(out, plain) and torch.equal(lse, plain_lse)


@pytest.mark.parametrize("window", [1, 7, 64, 1000])
def test_windows_with_tokens_before_position_zero(window):
    for lengths in (([4, 3], [2, 0]), ([300, 40], [280, 11])):
        Batch(*lengths, 8, 2, 64, 16, "fp16", seed=51).check(window=window)

"""Attention of batches in which some queries, keys or values are not finite: the rows that see them get them, every
other row keeps its value, and the kernel goes on (the status word stays clear: Case.attend checks it)."""
import math

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


# 8 / 2 heads: 128 tokens are 512 rows of a key/value head (at up to 128 components two row tiles of a CTA pair), 40 are 160
# (one tile, which takes the S buffers in turn), 700 positions six tiles of keys; 120 sequences: several tiles to a CTA pair.
PAIRS = ([128, 40] * 60, [600, 700] * 60)


@pytest.mark.parametrize("d", [64, 72, 128, 256])
def test_one_row_tile_after_two(d):
    Batch(*PAIRS, 8, 2, d, 16, seed=40).check()


@pytest.mark.parametrize("d", [64, 72, 128, 256])
def test_one_row_tile_after_two_with_queries_that_are_not_finite(d):
    """The second row tile of the first kind of sequence has nothing but NaN rows."""
    c = Batch(*PAIRS, 8, 2, d, 16, seed=41)
    for i in range(0, 120, 2):
        c.q[c.start[i] + 64:c.start[i] + 128] = math.nan
    c.check()


@pytest.mark.parametrize("d", [64, 72, 128, 256])
def test_one_row_tile_after_two_with_values_that_one_token_sees(d):
    """A value of the last position of every sequence: its last token's, hidden from all the others of its row tile."""
    c = Batch(*PAIRS, 8, 2, d, 16, "fp16", seed=42)
    for i, n in enumerate(c.kv_len):
        c.spoil_value(i, n - 1, math.nan if i % 4 < 2 else math.inf, comp=i % d)
    c.check()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lengths", [([200] * 90, [200] * 90), ([300, 20, 1], [2000, 1500, 1700])])
def test_values_that_later_tokens_see(lengths, d):
    """Whole row tiles, several to a CTA, and tiles in pieces: rows before the place keep their values, rows after it have NaN (or
    the infinity) in that component alone."""
    c = Batch(*lengths, 8, 2, d, 16, seed=43)
    for i, (n, total) in enumerate(zip(*lengths)):
        c.spoil_value(i, total - n + (2 * n) // 3, (math.nan, math.inf, -math.inf)[i % 3], head=i % 2, comp=(7 * i) % d)
    c.check()

"""Latent attention with queries of every layout: rows of one stride, whole heads or tokens to a tile, and neither of these (heads that do
not divide a tile in a wider array, one query for all heads or all tokens), against the definition in 64 bits.

The rows past a sequence's last and the components past a row's last hold NaN where there is memory for them, so that a place read from
beyond shows."""
import math

import pytest
import torch

from test_gpu_latent import DEV, LENGTHS, Case, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


def _wide(c):
    """The queries as parts of a wider array, tokens apart by more than their heads, NaN between them."""
    wide = torch.full((c.tokens, 2, c.h, c.d + 24), math.nan, dtype=c.dt, device=DEV)
    q = wide[:, 1, :, 8:8 + c.d]
    q.copy_(c.q)
    return q


# rows of a CTA by the heads and new tokens of a call: 16 (5 heads, 1 token), 32 (20 heads, 1), 64
@pytest.mark.parametrize("h", [3, 5, 12, 20, 33, 48, 100])
@pytest.mark.parametrize("lengths", ["empty", "before_zero", "edges", "long", "verify", "chunk", "mixed"])
@pytest.mark.parametrize("dc,rot,dtype", [(512, 64, "bf16"), (72, 24, "fp16")])
def test_heads_that_do_not_divide_a_tile(h, lengths, dc, rot, dtype):
    c = Case(*LENGTHS[lengths], h, dc, rot, 16, dtype, seed=41, pad_tokens=2)
    q = _wide(c)
    assert q.stride(0) != h * q.stride(1)
    c.check(q=q)


@pytest.mark.parametrize("dc,rot", [(8, 0), (64, 8), (128, 0), (200, 40), (504, 64), (512, 8)])
def test_sizes_of_such_rows(dc, rot):
    for lengths in ("long", "chunk"):
        c = Case(*LENGTHS[lengths], 20, dc, rot, 16, seed=42)
        c.check(q=_wide(c))


@pytest.mark.parametrize("h", [1, 5, 16, 20, 48, 64, 128])
@pytest.mark.parametrize("lengths", ["edges", "long", "chunk"])
@pytest.mark.parametrize("over", ["heads", "tokens", "both"])
def test_one_query_for_many(h, lengths, over):
    """A query broadcast over heads, over tokens, or both (strides of zero)."""
    c = Case(*LENGTHS[lengths], h, 512, 64, 16, seed=43)
    q = c.q[:, :1] if over == "heads" else c.q[:1] if over == "tokens" else c.q[:1, :1]
    q = q.expand(c.tokens, h, c.d)
    c.q = q.contiguous()
    c.check(q=q)


@pytest.mark.parametrize("h", [5, 20, 48])
def test_heads_behind_one_another(h):
    """Heads further apart than tokens: the array is [heads][tokens][D]."""
    for lengths in ("edges", "long", "chunk"):
        c = Case(*LENGTHS[lengths], h, 512, 64, 16, "fp16", seed=44)
        c.check(q=c.q.transpose(0, 1).contiguous().transpose(0, 1))

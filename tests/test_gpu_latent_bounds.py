"""Latent attention against bounds that are close: a long context.

With the terms of test_gpu_latent.  bf16 has the exponents of fp32, so a weight is rounded by a factor of 1 + u and never to a fixed
grid.  The sums: an accumulator takes 16 keys at a time, and what their products, the rescalings and the join of pieces add is a
chain of n / 16 + 64 + (pieces) steps, each off by 2 e of at most A (the tensor unit truncates); the sum of the weights is one of
n / 8 + 64 + (pieces) additions, each off by e; a GPU has fewer than 200 pieces, so with A = sum p |x| / sum p
|err| <= u |ref| + (u + 2 d + 8 e + 4 (n / 16 + 264) e) A."""
import math

import pytest
import torch

from test_gpu_latent import DEV, E, Case, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [20000, 131071])
def test_a_long_context_closely(h, n):
    c = Case([1], [n], h, 512, 64, 64, seed=51)
    out, lse = c.attend()
    scale = c.d ** -0.5
    x, q = c.rows[0].double(), c.q[0].double()
    v = x[:, :c.dc]
    s = q @ x.T * scale
    z = torch.logsumexp(s, -1, keepdim=True)
    w = torch.exp(s - z)
    ref, a = w @ v, w @ v.abs()
    d = (c.d + 8) * E * (q.abs() @ x.abs().T * scale).amax(-1, keepdim=True)
    tol = c.u * ref.abs() + (c.u + 2 * d + 8 * E + 4 * (n / 16 + 264) * E) * a
    err = (out[0].double() - ref).abs()
    assert (err - tol).max().item() <= 0
    assert ((lse[0].double() - z[:, 0]).abs() <= d[:, 0] + (n / 16 + 328) * 2 * E + z[:, 0].abs() * 2.0 ** -22).all()
    # what the bound would let through: it is small beside the outputs, so one that is wrong by half is not
    assert tol.max() < 0.25 * ref.std()
    assert ((0.5 * ref).abs() > tol).double().mean() > 0.5

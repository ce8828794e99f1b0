"""Latent attention in fp16: weights far below the largest.

The second product's operands are fp16, which rounds what lies below 2^-14 to multiples of 2^-24, so by 2^-25 at most.  The
kernel's weights are 2^7 exp(s - m) with a reference m that is never above the row's maximum, so the largest is 2^7 at least, and
relative to it that rounding is off by 2^-32 a key: with n keys of values of at most 1, by n 2^-32 in the output.  The other terms are those of
test_gpu_latent: u |ref| + (u + 2 d + (9 + n) e) sum p |x| / sum p."""
import math

import pytest
import torch

from test_gpu_latent import DEV, E, Case, _lib  # noqa: F401

pytestmark = pytest.mark.gpu
LN2 = math.log(2.0)


def _check(c, scores_of):
    """Sequence 0 with the scores (natural logarithms) that the first component of a row holds, q = (1, 0, ..); values of 0 and 1."""
    n = c.kv_len[0]
    x = torch.zeros(n, c.d, dtype=c.dt, device=DEV)
    x[:, 0] = torch.as_tensor(scores_of, dtype=torch.float64, device=DEV).to(c.dt)
    x[:, 1] = (x[:, 0] < x[:, 0].max()).to(c.dt)       # the flat tail's part
    x[:, 2] = 1.0
    c.rows[0] = x
    c.cache[c.where(0)] = x
    c.q.zero_()
    c.q[..., 0] = 1.0
    out, lse = c.attend(scale=1.0)
    ref, ref_lse, _, ltol = c.reference(scale=1.0)
    d = (c.d + 8) * E * x[:, 0].double().abs().max()
    w = torch.softmax(x[:, 0].double(), 0)
    tol = c.u * ref.abs() + (c.u + 2 * d + (9 + n) * E) * (w @ x[:, :c.dc].double().abs()) + n * 2.0 ** -32
    tol = tol + 2.0 ** -25  # fp16 outputs below its smallest normal number
    assert ((out.double() - ref).abs()[..., 1:] <= tol[..., 1:]).all()
    assert ((lse.double() - ref_lse).abs() <= ltol).all()
    return ref[-1, 0, 1].item(), tol[-1, 0, 1].item()


@pytest.mark.parametrize("h", [5, 20, 64])
@pytest.mark.parametrize("n", [100, 1000, 20000])
@pytest.mark.parametrize("at", [0.0, 0.4, 1.0])
def test_a_sharp_key_and_a_flat_tail(h, n, at):
    """One key 2^26 times the weight of each other: the others' part of the output is n 2^-26, and is there."""
    c = Case([1], [n], h, 128, 64, 16, "fp16", seed=1)
    s = torch.zeros(n)
    s[min(int(at * n), n - 1)] = 26 * LN2
    tail, tol = _check(c, s)
    assert tail > 8 * tol or n == 100


@pytest.mark.parametrize("h", [5, 64])
def test_references_that_lag(h):
    """Scores that stay just below what raises the reference (2^8 over it): the weights are 2^15 then, and do not overflow."""
    c = Case([1], [3000], h, 128, 64, 16, "fp16", seed=2)
    s = torch.full((3000,), 7.95 * LN2)
    s[::32] = 0.0
    s[:32] = 0.0
    _check(c, s)
    s[1500:] += 7.9 * LN2
    _check(c, s)

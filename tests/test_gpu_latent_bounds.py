"""Latent attention against bounds that are close: a long context, and rows that see infinities.

With the terms of test_gpu_latent.  bf16 has the exponents of fp32, so a weight is rounded by a factor of 1 + u and never to a fixed
grid.  The sums: an accumulator takes 16 keys at a time, and what their products, the rescalings and the join of pieces add is a
chain of n / 16 + 64 + (pieces) steps, each off by 2 e of at most A (the tensor unit truncates); the sum of the weights is one of
n / 8 + 64 + (pieces) additions, each off by e; a GPU has fewer than 200 pieces, so with A = sum p |x| / sum p
|err| <= u |ref| + (u + 2 d + 8 e + 4 (n / 16 + 264) e) A.  A row that is taken again key by key has n steps in either sum, and weights of
32 bits."""
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


@pytest.mark.parametrize("h", [4, 16, 40, 128])
@pytest.mark.parametrize("q_len,kv_len", [([40, 3], [200, 150]), ([9, 2], [1700, 900]), ([5], [64]), ([1], [6000])])
def test_rows_that_see_an_infinity(h, q_len, kv_len):
    """An infinity in a cache row: heads whose score there is -inf have no weight for it, so all their components but the infinite one are
    the finite positions' alone, and are compared with finite bounds."""
    compared = 0
    for part, value in ((3, math.inf), (511, -math.inf), (540, math.inf)):
        c = Case(q_len, kv_len, h, 512, 64, 16, seed=52)
        seen = [kv_len[0] - 1, kv_len[0] // 2] if q_len[0] > 1 else [kv_len[0] // 2]
        for p in seen:
            c.rows[0][p, part] = value
            c.cache[c.where(0, [p])] = c.rows[0][p:p + 1]
        out, lse = c.attend()
        scale = c.d ** -0.5
        for i, (n, total) in enumerate(zip(q_len, kv_len)):
            for j in range(max(0, n - total), n):
                p, t = total - n + j, c.start[i] + j
                x, q = c.rows[i][:p + 1].double(), c.q[t].double()
                s = q @ x.T * scale
                plus = (s == math.inf).any(-1)            # these heads have no finite output
                got = out[t].double()
                assert got[plus].isnan().all() and (lse[t][plus] == math.inf).all()
                finite = s.isfinite()
                s = s.masked_fill(~finite, -math.inf)
                z = torch.logsumexp(s, -1, keepdim=True)
                w = torch.exp(s - z)
                v = x[:, :c.dc]
                inf = v.isinf()
                v = v.masked_fill(inf, 0.0)
                ref, a = w @ v, w @ v.abs()
                xa = x.abs().masked_fill(x.isinf(), 0.0)
                d = (c.d + 8) * E * (q.abs() @ xa.T * scale).amax(-1, keepdim=True)
                tol = c.u * ref.abs() + (c.u + 2 * d + (9 + 2 * p) * E) * a
                assert tol.isfinite().all()
                bad = inf.any(0)[None].expand_as(ref)     # 0 x inf: a NaN by the formula
                rows = ~plus
                assert got[rows][bad[rows]].isnan().all()
                ok = rows[:, None] & ~bad
                assert got[ok].isfinite().all()
                assert ((got - ref).abs() <= tol)[ok].all()
                err = (lse[t].double() - z[:, 0]).abs()
                assert (err <= d[:, 0] + (p + 65) * E + z[:, 0].abs() * 2.0 ** -22)[rows].all()
                compared += int((ok & ~finite.all(-1)[:, None]).sum())
    assert compared > 0


@pytest.mark.parametrize("h,dc", [(16, 512), (5, 384), (64, 512)])
def test_a_row_of_few_pieces_is_taken_again_whole(h, dc):
    """A row with a NaN in one component, its keys cut into fewer than nine pieces: all its components come from one walk over the
    keys, which has weights of 32 bits, so the finite ones have no rounding of weights to bf16 in them.  (Few keys and scores close to one
    another, so that the bound of what is left is below that rounding.)"""
    n = 40
    c = Case([1] * n, [200 + i for i in range(n)], h, dc, 64, 16, seed=53)
    for i in range(n):
        p = 60 + i
        c.rows[i][p, 3] = math.inf
        c.cache[c.where(i, [p])] = c.rows[i][p:p + 1]
    scale, compared = 3e-4, 0
    out, lse = c.attend(scale)
    for i in range(n):
        x, q, got = c.rows[i].double(), c.q[i].double(), out[i].double()
        minus = q[:, 3] < 0  # the others' scores there are +inf
        assert got[~minus].isnan().all() and got[minus][:, 3].isnan().all()
        x[60 + i, 3] = 0.0
        s = (q @ x.T * scale)
        s[:, 60 + i] = -math.inf
        w, v, p = torch.softmax(s, -1), x[:, :dc], c.kv_len[i]
        ref, a = w @ v, w @ v.abs()
        d = (c.d + 8) * E * (q.abs() @ x.abs().T * scale).amax(-1, keepdim=True)
        tol = c.u * ref.abs() + (2 * d + (9 + 2 * p) * E) * a
        keep = minus[:, None] & (torch.arange(dc, device=DEV) != 3)
        assert ((got - ref).abs() <= tol)[keep].all()
        compared += int(keep.sum())
    assert compared > 0


@pytest.mark.parametrize("h", [4, 40, 128])
@pytest.mark.parametrize("kv_len", [1, 90, 3000])
@pytest.mark.parametrize("part", [3, 540])
def test_a_row_whose_scores_are_all_minus_infinity(h, kv_len, part):
    """Every position it sees has an infinity against its query: weights of zero, so zeros, a NaN in a component that is infinite, and lse -inf."""
    c = Case([1, 1], [kv_len, kv_len], h, 512, 64, 16, seed=54)
    c.rows[0][:, part] = math.inf
    c.cache[c.where(0)] = c.rows[0]
    minus = c.q[0, :, part] < 0
    out, lse = c.attend()
    assert minus.any() or h == 4
    assert (lse[0] == torch.where(minus, -math.inf, math.inf)).all()
    other = torch.arange(512, device=DEV) != part
    assert (out[0][minus][:, other] == 0).all() and out[0][~minus].isnan().all()
    if part < 512:
        assert out[0][minus][:, part].isnan().all()
    ref, ref_lse, tol, ltol = c.reference()
    assert ((out[1].double() - ref[1]).abs() <= tol[1]).all() and ((lse[1].double() - ref_lse[1]).abs() <= ltol[1]).all()

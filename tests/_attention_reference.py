"""The attention operator's definition in 64 bits, a sequence at a time, for batches with non-finite values in them.

The bounds are those derived in test_gpu_attention.py; a value that is not finite reaches the rows that see it and no
others.
"""
import math

import torch
from test_gpu_attention import DEV, E, Case


class Batch(Case):
    """A Case whose sequences' keys, values and queries can be spoiled in single places."""

    def spoil_value(self, seq, pos, value, head=slice(None), comp=slice(None)):
        self.values[seq][pos, head, comp] = value
        self.v_cache[int(self.table[seq][pos // self.page]), pos % self.page, head, comp] = value

    def spoil_key(self, seq, pos, value, head=slice(None), comp=slice(None)):
        self.keys[seq][pos, head, comp] = value
        self.k_cache[int(self.table[seq][pos // self.page]), pos % self.page, head, comp] = value

    def reference(self, window=0, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        shape, grp = (self.tokens, self.hq), self.hq // self.hkv
        f64 = dict(dtype=torch.float64, device=DEV)
        out, lse, tol, ltol = torch.zeros(*shape, self.d, **f64), torch.full(shape, -math.inf, **f64), torch.zeros(*shape, self.d, **f64), torch.zeros(shape, **f64)
        for i, (n, total) in enumerate(zip(self.q_len, self.kv_len)):
            if n == 0 or total == 0:
                continue
            rows = slice(self.start[i], self.start[i] + n)
            pos = torch.arange(total - n, total, device=DEV)[:, None]
            key = torch.arange(total, device=DEV)[None]
            seen = (key <= pos) & (pos - key < window if window else True)
            q = self.q[rows].double().reshape(n, self.hkv, grp, self.d).permute(1, 2, 0, 3)  # [hkv, grp, n, d]
            k, v = (t.double().permute(1, 0, 2) for t in (self.keys[i], self.values[i]))     # [hkv, total, d]
            sound = torch.where(v.isfinite(), v, 0.0)
            s = (q @ k.transpose(1, 2)[:, None] * scale).masked_fill(~seen, -math.inf)
            none = ~seen.any(-1)
            z = torch.logsumexp(s, -1, keepdim=True)
            w = torch.where(seen, torch.exp(s - z), 0.0)
            o, a = w @ sound[:, None], w @ sound.abs()[:, None]
            # the values that are not finite: their sum over the rows that see them
            odd = torch.where(v.isfinite(), 0.0, v)
            for p in (~v.isfinite()).any(-1).any(0).nonzero().flatten().tolist():
                o = torch.where(seen[:, p][:, None], o + odd[:, p][:, None, None], o)
            m = seen.sum(-1)[:, None]
            dlt = (self.d + 8) * E * (q.abs() @ k.abs().transpose(1, 2)[:, None] * scale).masked_fill(~seen, 0.0).amax(-1, keepdim=True)
            bound = self.u * o.abs() + (self.u + 2 * dlt + (8 + m) * E) * a + m * 2.0 ** -25 * sound.abs().amax()
            lbound = dlt + (m + 64) * E + z.abs() * 2.0 ** -22
            o[:, :, none] = 0.0
            z[:, :, none] = -math.inf

            def back(x):
                return x.permute(2, 0, 1, 3).reshape(n, self.hq, -1)
            out[rows], lse[rows], tol[rows], ltol[rows] = back(o), back(z)[..., 0], back(bound), back(lbound)[..., 0]
        return out, lse, tol, ltol

    def check(self, window=0, scale=None, **kw):
        """As Case.check, where the reference may hold values that are not finite: they have to be the same."""
        out, lse = self.attend(window, scale, **kw)
        ref, ref_lse, tol, lse_tol = self.reference(window, scale)
        for what, got, want, bound in (("out", out, ref, tol), ("lse", lse, ref_lse, lse_tol)):
            odd = ~want.isfinite()
            same = torch.where(want.isnan(), got.isnan(), got.double() == want)
            assert bool(same[odd].all()), f"{what}: {int((~same & odd).sum())} values that are not finite differ"
            err = ((got.double() - want).abs() - bound)[~odd]
            assert not err.isnan().any(), f"{what}: {int(err.isnan().sum())} values are NaN where they should not be"
            assert err.numel() == 0 or err.max().item() <= 0, f"{what} is {err.max().item():.3e} beyond its bound"
        return out, lse

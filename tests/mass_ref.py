"""Row masses in 64 bits, the inputs of their tests and how far a correct result may be from them."""
from __future__ import annotations

import math

import numpy as np
import torch


class Case:
    """Queries, their log-sum-exps and a paged cache of several sequences. Rows outside the sequences hold NaN or an
    infinity, the table names blocks that do not exist for pages without a row, and query rows behind the last
    sequence are NaN. decode: one query a sequence."""

    def __init__(self, seed, dtype, heads, width, page, kv, q=None, tail=0, spread=1.0, scale=None, pad=0, offset=0, extra=1,
                 layers=1):
        r = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.decode = q is None
        self.q_lens = [1] * len(kv) if q is None else list(q)
        self.kv, self.page, self.heads, self.width = list(kv), page, heads, width
        self.scale = 1 / math.sqrt(192) if scale is None else scale
        per = max(1, max(-(-n // page) for n in kv)) + extra
        blocks = len(kv) * per
        table = r.permutation(blocks).reshape(len(kv), per).astype(np.int32)
        whole = torch.full((offset + blocks * layers * page * (width + pad),), math.nan, dtype=dtype, device="cuda")
        cache = whole[offset:].view(blocks, layers, page, width + pad)[:, layers - 1, :, :width]
        cache[::2] = math.inf
        for b, n in enumerate(kv):
            t = np.arange(n)
            at = torch.from_numpy(table[b, t // page].astype(np.int64)).cuda(), torch.from_numpy(t % page).cuda()
            cache[at] = (torch.randn(n, width, generator=g, device="cuda") * spread).to(dtype)
            table[b, -(-n // page):] = r.choice([-1, blocks + 7, 2 ** 31 - 1, -(2 ** 31)], per + (-n // page))
        self.cache, self.table_np, self.table = cache, table, torch.from_numpy(table).cuda()
        self.tokens = sum(self.q_lens) + tail
        qs = torch.full((offset + self.tokens * heads * (width + pad),), math.nan, dtype=dtype, device="cuda")
        self.q = qs[offset:].view(self.tokens, heads, width + pad)[..., :width]
        live = sum(self.q_lens)
        self.q[:live] = (torch.randn(live, heads, width, generator=g, device="cuda") * spread).to(dtype)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(self.q_lens)]), dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(self.kv, dtype=torch.int32, device="cuda")
        self.lse = torch.full((self.tokens, heads), math.nan, device="cuda")
        self.rows = per * page
        self.mass = torch.rand(len(kv), self.rows, generator=g, device="cuda")
        self._scores()

    def _scores(self):
        self.parts, at = [], 0
        for b, (n, k) in enumerate(zip(self.kv, self.q_lens)):
            t = np.arange(n)
            keys = self.cache[torch.from_numpy(self.table_np[b, t // self.page].astype(np.int64)).cuda(),
                              torch.from_numpy(t % self.page).cuda()].double()
            x = self.q[at:at + k].double()
            s = torch.einsum("ihe,te->iht", x, keys) * self.scale
            big = torch.einsum("ihe,te->iht", x.abs(), keys.abs()) * abs(self.scale)
            seen = torch.arange(n, device="cuda") <= torch.arange(n - k, n, device="cuda")[:, None]
            s = torch.where(seen[:, None], s, -math.inf)
            self.lse[at:at + k] = torch.logsumexp(s, -1).float() if n else -math.inf
            self.parts.append((s, big, at, n, k))
            at += k

    def want(self, decay):
        """Masses after the call and their bounds."""
        want, tol = self.mass.double(), torch.zeros_like(self.mass, dtype=torch.float64)
        for b, (s, big, at, n, k) in enumerate(self.parts):
            if n == 0 or k == 0:
                continue
            lse = self.lse[at:at + k].double()[..., None]
            w = torch.where(lse == -math.inf, 0.0, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)))
            # a logit: width + 24 roundings of float32 partial sums no larger than `big`, then a product, a
            # difference and an exponential; the sums: one rounding a term
            d = (self.width + 24) * 2.0 ** -23 * big + (torch.nan_to_num(s, neginf=0).abs() + torch.nan_to_num(lse, neginf=0).abs()) * 2.0 ** -22 + 2.0 ** -21
            total = w.sum((0, 1))
            old = torch.zeros(n, dtype=torch.float64, device="cuda") if decay == 0 else want[b, :n] * decay
            want[b, :n] = old + total
            tol[b, :n] = (w * d).sum((0, 1)) * 1.01 + (k * self.heads + 8) * 2.0 ** -24 * total + (old.abs() + total) * 2.0 ** -23 + 1e-37
        return want, tol

    def run(self, mla, decay=1.0, mass=None, **more):
        mass = self.mass.clone() if mass is None else mass
        if self.decode:
            mla.mla_decode_mass(mass, self.q, self.cache, self.table, self.lens, self.lse, self.scale, decay=decay, **more)
        else:
            mla.mla_prefill_mass(mass, self.q, self.cache, self.table, self.cu, self.lens, self.lse, self.scale, decay=decay, **more)
        return mass

    def check(self, got, decay=1.0):
        want, tol = self.want(decay)
        off = (got.double() - want).abs() - tol
        assert not torch.isnan(off).any(), "NaN"
        assert off.max() <= 0, f"{off.max():.3e} beyond its bound at {np.unravel_index(int(off.argmax()), off.shape)}"
        for b, n in enumerate(self.kv):      # behind the rows: left as they were
            assert torch.equal(got[b, n:], self.mass[b, n:])

"""A plain 64-bit implementation of attention limited to a window and sinks, the inputs of its tests
and how far a correct result may be from it."""
from __future__ import annotations

import math

import numpy as np
import torch


def rows_seen(p: int, window: int, sinks: int):
    """Rows that a query at position p attends."""
    return [t for t in range(p + 1) if t < sinks or t > p - window]


def attend(q, rows, latent: int, scale: float):
    """o [H, latent], lse [H] of q [H, E] over rows [n, E] (float64), and the bounds' terms: the mean
    of |value| under the weights [H, latent], and the largest sum of |q_e * k_e| * scale of a row [H]."""
    heads = q.shape[0]
    if rows.shape[0] == 0:
        return (np.zeros((heads, latent)), np.full(heads, -np.inf), np.zeros((heads, latent)), np.zeros(heads))
    s = (q @ rows.T) * scale
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(1, keepdims=True)
    p = p / total
    v = rows[:, :latent]
    big = (np.abs(q) @ np.abs(rows).T).max(1) * scale
    return p @ v, (m + np.log(total))[:, 0], p @ np.abs(v), big


class Case:
    """Queries and a paged cache of several sequences. Every row that no query attends holds NaN or an
    infinity, and the table names blocks that do not exist for pages without an attended row."""

    def __init__(self, *, seed, dtype, heads, latent, rope, page, kv, q, window, sinks, tail=0, spread=1.0,
                 scale=None, q_pad=0, cache_pad=0):
        r = np.random.default_rng(seed)
        width = latent + rope
        self.dt = torch.float32 if dtype == "f32" else torch.bfloat16
        self.dtype, self.latent, self.rope, self.window, self.sinks = dtype, latent, rope, window, sinks
        self.scale = 1 / math.sqrt(192) if scale is None else scale
        self.kv, self.q_lens = list(kv), list(q)
        tokens = sum(q) + tail
        blocks_per = max(1, max(-(-n // page) for n in kv) + 1)
        used = len(kv) * blocks_per
        order = r.permutation(used)
        table = order.reshape(len(kv), blocks_per).astype(np.int32)
        real = r.standard_normal((used, page, width)) * spread
        cache = np.full((used, page, width), np.nan)
        cache[::2] = np.inf
        cache[1::4] = -np.inf
        for b, (n, k) in enumerate(zip(kv, q)):
            seen = sorted({t for p in range(max(0, n - k), n) for t in rows_seen(p, window, sinks)})
            pages = {t // page for t in seen}
            for t in seen:
                cache[table[b, t // page], t % page] = real[table[b, t // page], t % page]
            for i in range(blocks_per):
                if i not in pages:
                    table[b, i] = [-1, used + 7, 2 ** 31 - 1, -(2 ** 31)][r.integers(4)]
        self.table_np = table
        full = torch.zeros((used, page, width + cache_pad), dtype=self.dt)
        full[..., :width] = torch.from_numpy(cache).to(self.dt)
        full[..., width:] = float("nan")
        self.cache = full
        self.width = width
        qs = torch.zeros((tokens, heads, width + q_pad), dtype=self.dt)
        qs[..., :width] = torch.from_numpy(r.standard_normal((tokens, heads, width)) * spread).to(self.dt)
        self.qs = qs
        self.page = page

    def dev(self):
        """cache, q, table, lengths and cumulated query lengths on the GPU."""
        cu = np.concatenate([[0], np.cumsum(self.q_lens)]).astype(np.int32)
        return (self.cache.cuda()[..., :self.width], self.qs.cuda()[..., :self.width],
                torch.from_numpy(self.table_np).cuda(), torch.tensor(self.kv, dtype=torch.int32).cuda(),
                torch.from_numpy(cu).cuda())

    def want(self):
        """o, lse and how far a result may be from them, per element."""
        rows64 = self.cache[..., :self.width].double().numpy()
        q64 = self.qs[..., :self.width].double().numpy()
        tokens, heads = q64.shape[:2]
        o, lse = np.zeros((tokens, heads, self.latent)), np.zeros((tokens, heads))
        tol_o, tol_lse = np.zeros_like(o), np.zeros_like(lse)
        at = 0
        for b, (n, k) in enumerate(zip(self.kv, self.q_lens)):
            for i in range(k):
                seen = np.array(rows_seen(n - k + i, self.window, self.sinks), dtype=np.int64)
                rows = rows64[self.table_np[b, seen // self.page], seen % self.page] if len(seen) else \
                    np.zeros((0, self.width))
                o[at], lse[at], mean, big = attend(q64[at], rows, self.latent, self.scale)
                # logits: at most width + 24 roundings of float32 partial sums no larger than `big`; the
                # weights move by that, the sums over n rows by n roundings; on the tensor cores each
                # weight is rounded to bf16 once (2^-8 of it), and the result once more (2^-8 of it)
                d = (self.width + 24) * 2.0 ** -23 * big + len(seen) * 2.0 ** -23 + 2.0 ** -20
                tol_lse[at] = d + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse[at]), lse[at], 0))
                tol_o[at] = 2 * d[:, None] * mean + 2.0 ** -23
                if self.dtype == "bf16":
                    tol_o[at] += 2.0 ** -8 * (mean + np.abs(o[at])) * 1.01
                at += 1
        return o, lse, tol_o, tol_lse


def check(got_o, got_lse, want, rows: int):
    """The first `rows` rows of the outputs against want()."""
    o, lse, tol_o, tol_lse = (w[:rows] for w in want)
    g = got_o[:rows].double().cpu().numpy()
    assert np.isfinite(g).all(), "non-finite output"
    off = np.abs(g - o) - tol_o
    assert off.max(initial=-1) <= 0, f"o: {off.max():.3e} beyond its bound at {np.unravel_index(off.argmax(), off.shape)}"
    if got_lse is not None:
        gl = got_lse[:rows].double().cpu().numpy()
        empty = ~np.isfinite(lse)
        assert np.array_equal(gl[empty], lse[empty])
        off = np.abs(gl[~empty] - lse[~empty]) - tol_lse[~empty]
        assert off.max(initial=-1) <= 0, f"lse: {off.max():.3e} beyond its bound"

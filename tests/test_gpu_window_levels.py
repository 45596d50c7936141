"""Windowed attention with logits far apart, exact in float32: the running maximum raised little by little and at
once, weights that vanish and count all the same. Logits are whole multiples of ln 2, so weights are powers of
two, which bf16 holds, and values are as large as their weights are small: every part of a row counts alike."""
import math

import numpy as np
import pytest
import torch

import window_ref as wr
from test_gpu_window import decode_case, outputs, prefill_case

pytestmark = pytest.mark.gpu

LN2 = float(np.float32(math.log(2)))
# what a run of 50 rows adds to the level of the run before, over and over. A tile is 128 rows on the tensor
# cores, where the maximum is raised by more than 8, and 32 on the CUDA cores
STEPS = {"up little": [1, 2, 0, 3], "up by 8 and 9": [8, 0, 9, -8, 8, -9], "up at once": [0, 0, 40, 0, 0, 35, 0],
         "down": [0, -3, -9, -1], "zigzag": [25, -24, 9, -9, 30, -31, 7, 1], "level": [0]}


def level_case(which, geometry, steps, kv, window, sinks, seed):
    make = decode_case if which == "decode" else lambda g, n, w, s, **more: \
        prefill_case(g, n, [min(3, k) for k in n], w, s, **more)
    c = make(geometry, kv, window, sinks, seed=seed, scale=LN2)
    r = np.random.default_rng(seed)
    c.qs[:] = 0
    heads = c.qs.shape[1]
    for h in range(heads):
        c.qs[:, h, 512 + h % 64] = 1      # head h takes its levels from rope column h % 64
    for b, n in enumerate(kv):
        runs = np.cumsum([steps[i % len(steps)] for i in range(n // 50 + 1)])
        runs = np.clip(runs - runs.max(initial=0), -80, 0) + 90
        for t in range(n):
            block = c.table_np[b, t // c.page]
            if not 0 <= block < c.cache.shape[0] or not torch.isfinite(c.cache[block, t % c.page, 0]):
                continue                  # a row that nothing attends
            level = int(runs[t // 50])
            row = c.cache[block, t % c.page]
            row[:512] = torch.from_numpy(r.standard_normal(512) + 1.0).to(c.dt) * 2.0 ** (90 - level)
            row[512:576] = level - torch.from_numpy(r.integers(0, 3, 64)).to(c.dt)
    return c


def check(c, o, l):
    """Against 64 bits. Logits: the product with the scale and that with log2 e, of levels up to 90, 2^-16 in
    all; the exponential 2 + 1.2 x 63 units in the last place (its fast form), once more for merged pieces: 2^-16
    each; the sums a unit a row. Twice each, in the numerator and the sum: 2^-13. And the result's rounding."""
    rows64 = c.cache[..., :c.width].double().numpy()
    got_o, got_l = o.double().cpu().numpy(), l.double().cpu().numpy()
    at = 0
    for b, (n, k) in enumerate(zip(c.kv, c.q_lens)):
        for i in range(k):
            seen = np.array(wr.rows_seen(n - k + i, c.window, c.sinks), dtype=np.int64)
            rows = rows64[c.table_np[b, seen // c.page], seen % c.page] if len(seen) else np.zeros((0, c.width))
            want, lse, mean, _ = wr.attend(c.qs[at, :, :c.width].double().numpy(), rows, 512, c.scale)
            rel = 2.0 ** -13 + len(seen) * 2.0 ** -23
            out = (2.0 ** -8 if c.dtype == "bf16" else 2.0 ** -24) * 1.01
            off = np.abs(got_o[at] - want) - (rel * mean + out * np.abs(want))
            assert off.max() <= 0, f"token {at}: {off.max():.3e} beyond its bound, of {np.abs(want).mean():.3e}"
            if len(seen):
                assert (np.abs(got_l[at] - lse) <= rel + 2.0 ** -22 * np.abs(lse)).all()
            else:
                assert np.isneginf(got_l[at]).all()
            at += 1


@pytest.mark.parametrize("steps", STEPS)
@pytest.mark.parametrize("geometry", ["v3", "h20", "lite_f32"])
@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("window,sinks", [(500, 4), (1500, 70)])
def test_levels(mla, which, geometry, steps, window, sinks):
    # whole row tiles, and (the longer window) pieces of them that are merged
    c = level_case(which, geometry, STEPS[steps], [1700, 130, 0, 1001], window, sinks, seed=101)
    cache, q, table, kv, cu = c.dev()
    o, l = outputs(c)
    if which == "decode":
        mla.mla_decode_window(o, q, cache, table, kv, 512, 64, c.scale, window, sinks=sinks, lse_out=l)
    else:
        mla.mla_prefill_window(o, q, cache, table, cu, kv, 512, 64, c.scale, window, sinks=sinks, lse_out=l)
    mla.mla_device_error()
    check(c, o, l)


@pytest.mark.parametrize("splits", [1, 2, 5, 40])
@pytest.mark.parametrize("geometry", ["v3", "lite_f32"])
def test_levels_of_pieces(mla, geometry, splits):
    c = level_case("decode", geometry, STEPS["zigzag"], [1700, 1100], 1600, 0, seed=102)
    cache, q, table, kv, _ = c.dev()
    o, l = outputs(c)
    mla.mla_decode_window(o, q, cache, table, kv, 512, 64, c.scale, 1600, lse_out=l, num_splits=splits)
    mla.mla_device_error()
    check(c, o, l)

"""How far masses are from 64 bits on the whole. The bounds of mass_ref are those of the worst inputs; a systematic error far
below them shows in the mean over many rows, and a random one in the norm.

A weight e^x is off by e^x times the error of x, its exponent. By arithmetic, of what a score's float32 partial sums p lose:
  tensor cores  a step of 16 columns adds to a partial sum and drops what lies below its last place: toward zero, half
                a place of p on average and one at most. A score's first half of 64-column chunks (rounded up) is one
                chain, the others another; the two are added to the nearest.
  CUDA cores    each product is added to the nearest: half a place at most, of either sign.
Then scale (on the tensor cores times log2 e, rounded once: known, and part of the 64-bit value below), lse (the same, once a
query and head), their sum and the exponential, each to the nearest but the last, off by 2^-22 at most; then sums of weights
to the nearest. What is rounded to the nearest counts by its square, with six standard deviations: half a place is 1 / sqrt 3
times as much as one standard deviation of a rounding's error."""
import math

import pytest
import torch

from mass_ref import Case

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LOG2E = torch.tensor(1.4426950408889634, dtype=F32)


def place(x):
    """The last place of float32 values: 2^(exponent - 23)."""
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -100))) - 23)


def expected(c, tensor_cores, chains=2):
    """Of every row that a query attends: its mass in 64 bits, what it loses toward zero on average, and the variance of the rest."""
    got = []
    at = 0
    scale = torch.tensor(c.scale, dtype=F32)
    for b, (n, k) in enumerate(zip(c.kv, c.q_lens)):
        t = torch.arange(n, device="cuda")
        keys = c.cache[c.table[b].long()[t // c.page], t % c.page].double()
        mass, loss, var = (torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(3))
        for i in range(k):
            q, lse = c.q[at + i].double(), c.lse[at + i]
            seen = t <= n - k + i
            step = 16 if tensor_cores else 1
            parts = (q[:, None] * keys[None]).unflatten(-1, (-1, step)).sum(-1)               # [heads, rows, steps]
            s = parts.sum(-1)
            if tensor_cores:
                chunks = c.width // 64
                cut = (chunks + 1) // 2 * 4 if chains == 2 else chunks * 4
                chain = torch.cat([parts[..., :cut].cumsum(-1), parts[..., cut:].cumsum(-1)], -1)
                by = (scale * LOG2E).double().item() * math.log(2)
                l = (lse * LOG2E.cuda()).double() * math.log(2)
                # toward zero: a positive sum's exponent is smaller by it
                lost = (place(chain) * chain.sign()).sum(-1) / 2 * abs(by) * math.copysign(1, by)
                dev = ((place(chain).square().sum(-1) + place(s).square()) / 12) * by ** 2
            else:
                by, l, lost = scale.double().item(), lse.double(), 0.0
                dev = place(parts.cumsum(-1)).square().sum(-1) / 12 * by ** 2
            w = torch.exp(s * by - l[:, None]) * seen
            x = (s * by - l[:, None]).abs() + l.abs()[:, None]
            mass += w.sum(0)
            loss += (w * lost).sum(0)
            var += (w.square() * (dev + (x * 2.0 ** -23).square() / 12 + 2.0 ** -44)).sum(0)
        var += (mass * 2.0 ** -23).square() / 12 * (8 + math.log2(max(2, k * c.heads)))        # sums of weights
        got.append((mass, loss, var))
        at += k
    return got


def shares(c, got, want):
    """Means over the rows that hold mass: of the relative error, of the expected loss, of six deviations of the mean; and the
    same three as norms."""
    e = torch.cat([(g[:n].double() - m) / m for g, n, (m, _, _) in zip(got, c.kv, want)])
    loss = torch.cat([lo / m for m, lo, _ in want])
    var = torch.cat([v / m.square() for m, _, v in want])
    fine = torch.cat([m for m, _, _ in want]) > 0
    e, loss, var = e[fine], loss[fine], var[fine]
    return e.mean().item(), loss.mean().item(), 6 * (var.sum().sqrt() / var.numel()).item(), \
        (e.square().mean().sqrt().item(), loss.square().mean().sqrt().item(), var.mean().sqrt().item())


# tensor cores: a decode, a prefill of whole tiles, one whose rows are cut over the units; CUDA cores: both types
CASES = [(BF16, 128, 576, 64, [700, 900], None), (BF16, 16, 576, 64, [300, 700], [40, 9]), (BF16, 128, 512, 64, [3000], [6]),
         (BF16, 128, 64, 64, [500], None), (F32, 16, 576, 64, [300, 200], None), (F32, 16, 576, 64, [300], [5]), (BF16, 16, 576, 5, [300], None)]


@pytest.mark.parametrize("dtype,heads,width,page,kv,q", CASES)
@pytest.mark.parametrize("positive", [False, True])
def test_no_more_is_lost_than_roundings_do(mla, dtype, heads, width, page, kv, q, positive):
    # positive: values of one sign, whose partial sums grow all the way
    tc = dtype == BF16 and page == 64
    c = Case(61, dtype, heads, width, page, kv, q, scale=8 / (width * 2 / math.pi) if positive else None)
    if positive:
        c.q.abs_()
        c.cache.copy_(c.cache.abs())
        c._scores()
    got = c.run(mla, 0.0)
    mean, lost, random, norms = shares(c, got, expected(c, tc))
    # toward zero, at most twice the average of half a place; the exponential may be off to one side by 2^-22
    assert -2 * max(lost, 0) - random - 2.0 ** -22 <= mean <= 2 * max(-lost, 0) + random + 2.0 ** -22, (mean, lost, random)
    assert norms[0] <= 2 * norms[1] + 3 * norms[2] + 2.0 ** -22, norms


@pytest.mark.parametrize("heads,kv,q", [(128, [900], None), (128, [3000], [4]), (16, [600], [33])])
def test_two_chains_lose_half_of_what_one_does(mla, heads, kv, q):
    c = Case(67, BF16, heads, 576, 64, kv, q, scale=8 / (576 * 2 / math.pi))
    c.q.abs_()
    c.cache.copy_(c.cache.abs())
    c._scores()
    mean, lost, random, _ = shares(c, c.run(mla, 0.0), expected(c, True))
    _, one, _, _ = shares(c, c.run(mla, 0.0), expected(c, True, chains=1))
    # half a place on average, with a quarter more for what a step's own products lose before they are added
    most = 1.25 * lost + random + 2.0 ** -22
    assert 0.9 * one > most              # a single chain would not pass
    assert -mean <= most, (mean, lost, one, random)

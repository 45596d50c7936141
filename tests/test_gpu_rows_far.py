"""Caches whose offsets pass 32 bits, and tables far longer than their sequences."""
import math

import pytest
import torch

import norm_rope_ref as ref
from mass_ref import Case

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def far():
    """A bf16 cache of 2.6e9 values; its last blocks are used."""
    cache = torch.empty(70000, 64, 576, dtype=BF16, device="cuda")
    cache[-40:] = 0
    yield cache
    del cache
    torch.cuda.empty_cache()


def test_rows_written_far(mla, far):
    g = torch.Generator().manual_seed(1)
    kv, w = torch.randn(100, 576, generator=g).to(BF16), (1 + torch.randn(512, generator=g) / 4).to(BF16)
    pos, cs = torch.arange(100), ref.table(100, 64)
    slots = 69990 * 64 + torch.randperm(640, generator=g)[:100]
    mla.mla_norm_rope_cache_write(far, kv.cuda(), w.cuda(), pos.cuda(), cs.cuda(), slots.cuda())
    mla.mla_device_error()
    want, err = ref.rows(kv, w, cs[pos], True, 1e-6)
    ref.check(far.view(-1, 576)[slots.cuda()], want, err, BF16, "rows")


def test_slots_beyond_31_bits(mla):
    # more than 2^31 rows of 16 codes
    cache = torch.empty((1 << 24) + 2, 128, 16, dtype=torch.uint8, device="cuda")
    cache[-2:] = 0
    x = torch.randn(50, 16, generator=torch.Generator().manual_seed(2)).to(BF16)
    w, scale = torch.ones(16, dtype=BF16), 0.01
    slots = (1 << 31) + torch.randperm(256, generator=torch.Generator().manual_seed(3))[:50]
    none = torch.zeros(50, dtype=torch.int64, device="cuda")
    mla.mla_norm_rope_cache_write_fp8(cache, x.cuda(), w.cuda(), none, torch.zeros(1, 0, device="cuda"), slots.cuda(),
                                      torch.tensor([scale], device="cuda"))
    mla.mla_device_error()
    y, rel = ref.normed(x, w, 1e-6)
    y = y / torch.tensor(scale).double()
    ref.check_codes(cache.view(-1, 16)[slots.cuda()], y, y.abs() * (rel + 2.0 ** -23), "codes")
    del cache
    torch.cuda.empty_cache()


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("simt", [False, True])
def test_masses_of_far_rows(mla, far, prefill, simt):
    c = Case(5, BF16, 16, 576, 64, [300, 190], [7, 190] if prefill else None, pad=1 if simt else 0)
    base = 69960
    far[base:base + c.cache.shape[0]] = c.cache
    near = c.run(mla)
    c.cache, c.table = far, torch.where((c.table >= 0) & (c.table < c.cache.shape[0]), c.table + base, c.table)
    got = c.run(mla)
    mla.mla_device_error()
    assert torch.equal(got, near)


@pytest.mark.parametrize("other", [False, True])
def test_rows_moved_far(mla, far, other):
    g = torch.Generator(device="cuda").manual_seed(7)
    n, budget, base = 500, 130, 69960
    far[base:base + 16] = torch.randn(16, 64, 576, generator=g, device="cuda").to(BF16)
    before = far[base:base + 16].clone()
    table = (base + torch.randperm(8, generator=torch.Generator().manual_seed(1))).to(torch.int32).view(1, 8).cuda()
    dst = (table + 8) if other else table
    mass = torch.rand(1, 512, generator=g, device="cuda")
    lens, out, kept = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), \
        torch.zeros(1, budget, dtype=torch.int32, device="cuda")
    mla.mla_cache_evict(far, mass.clone(), table, lens, budget, out, sinks=4, recent=20, block_table_out=dst, kept_out=kept)
    mla.mla_device_error()
    t = kept[0].long()
    want = torch.cat([torch.arange(4), 4 + mass[0, 4:480].cpu().sort(descending=True, stable=True).indices[:106], torch.arange(480, 500)])
    assert torch.equal(t.cpu(), want.sort().values) and out.item() == budget
    j = torch.arange(budget, device="cuda")
    moved = far[dst[0, j // 64].long(), j % 64]
    assert torch.equal(moved, before[table[0, t // 64].long() - base, t % 64])


@pytest.mark.parametrize("dtype,heads", [(BF16, 128), (F32, 16), (F32, 40)])
def test_tables_far_longer_than_their_sequences(mla, dtype, heads):
    # room for 131072 rows each, and a sequence that takes more blocks of the CUDA cores than it is given at once
    for kv in ([20, 0, 130], [5000]):
        c = Case(heads, dtype, heads, 64, 64, kv, extra=2048 - (-(-max(kv) // 64)))
        c.check(c.run(mla))
        mla.mla_device_error()
    q = [3, 0, 100]
    c = Case(heads + 1, dtype, heads, 64, 64, [300, 50, 100], q, extra=2040)
    c.check(c.run(mla))
    lens, kept = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, 40, dtype=torch.int32, device="cuda")
    mla.mla_cache_evict(c.cache, c.mass, c.table, c.lens, 40, lens, recent=5, kept_out=kept)
    mla.mla_device_error()
    assert lens.tolist() == [40, 40, 40]


def test_a_mass_that_overflows_is_infinite(mla):
    # log-sum-exps far too small: the weights leave float32's range, in no other row and to no NaN
    c = Case(9, BF16, 16, 576, 64, [100, 90])
    c.lse[0] = -1000.0
    got = c.run(mla)
    assert torch.isinf(got[0, :100]).all() and (got[0, :100] > 0).all() and torch.isfinite(got[1]).all()
    c.lse[0] = 1000.0
    assert torch.equal(c.run(mla)[0], c.mass[0])
    assert math.isfinite(c.run(mla)[1].sum().item())

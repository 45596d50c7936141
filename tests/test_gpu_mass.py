"""Row masses against 64 bits, with derived bounds."""
import math

import pytest
import torch

from mass_ref import Case

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LENS = [0, 1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700]


@pytest.mark.parametrize("decay", [1.0, 0.75])
@pytest.mark.parametrize("dtype,heads,width,page", [
    (BF16, 128, 576, 64), (BF16, 64, 512, 64), (BF16, 16, 576, 16), (BF16, 20, 576, 8), (BF16, 1, 64, 32), (BF16, 65, 128, 128),
    (BF16, 33, 320, 192), (F32, 16, 576, 64), (BF16, 130, 576, 64), (BF16, 16, 576, 5), (F32, 3, 20, 7), (BF16, 5, 100, 1)])
def test_decode(mla, dtype, heads, width, page, decay):
    c = Case(heads + page, dtype, heads, width, page, LENS)
    c.check(c.run(mla, decay), decay)
    mla.mla_device_error()


@pytest.mark.parametrize("dtype,heads,width,page", [
    (BF16, 128, 576, 64), (BF16, 64, 512, 64), (BF16, 16, 576, 16), (BF16, 20, 576, 8), (BF16, 1, 64, 32), (BF16, 65, 128, 128),
    (BF16, 33, 320, 192), (BF16, 100, 576, 64), (F32, 16, 576, 64), (BF16, 130, 64, 64), (BF16, 16, 576, 5), (F32, 3, 20, 7)])
@pytest.mark.parametrize("kv,q", [
    ([700], [1]), ([700], [33]), ([257, 1, 129, 300], [257, 1, 2, 0]), ([0, 5, 256, 130, 512], [3, 9, 256, 131, 17]), ([1024], [300])])
def test_prefill(mla, dtype, heads, width, page, kv, q):
    # among them more queries than rows (the first ones attend nothing) and sequences without queries or rows
    c = Case(heads + len(kv), dtype, heads, width, page, kv, q, tail=3)
    c.check(c.run(mla))
    mla.mla_device_error()


@pytest.mark.parametrize("heads,width", [(128, 576), (64, 512), (20, 576)])
@pytest.mark.parametrize("kv,q", [([9000], [40]), ([3000, 4000, 70], [200, 20, 70]), ([2500], [1000])])
def test_prefill_cut_over_the_units(mla, heads, width, kv, q):
    # a tile of rows has more queries than a work unit takes: its sums come in pieces
    c = Case(heads, BF16, heads, width, 64, kv, q)
    got = c.run(mla, 0.5)
    c.check(got, 0.5)
    assert torch.equal(got, c.run(mla, 0.5))        # and always in the same order


def test_decode_long_and_many(mla):
    kv = [16384, 1, 0, 9999] + [int(x) for x in torch.randint(0, 1500, (150,), generator=torch.Generator().manual_seed(1))]
    c = Case(7, BF16, 128, 576, 64, kv)
    got = c.run(mla)
    c.check(got)
    assert torch.equal(got, c.run(mla))


@pytest.mark.parametrize("dtype,page", [(BF16, 64), (F32, 64), (BF16, 3)])
@pytest.mark.parametrize("prefill", [False, True])
def test_decay_zero_reads_nothing(mla, dtype, page, prefill):
    c = Case(3, dtype, 16, 576, page, [300, 0, 65], [4, 2, 65] if prefill else None)
    c.mass[:] = math.nan
    got = c.run(mla, 0.0)
    c.mass[:] = 0
    for b, n in enumerate(c.kv):
        assert torch.isnan(got[b, n:]).all()
        got[b, n:] = 0
    c.check(got, 0.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_masses_of_a_query_sum_to_its_heads(mla, dtype):
    c = Case(5, dtype, 128, 576, 64, [500, 1000], [7, 9])
    got = c.run(mla, 0.0, mass=torch.zeros_like(c.mass))
    assert (got.sum(1).cpu() - torch.tensor([7 * 128.0, 9 * 128.0])).abs().max() < 0.05


@pytest.mark.parametrize("dtype,heads,width,page,pad,offset,layers", [
    (BF16, 128, 576, 64, 8, 0, 3), (BF16, 16, 576, 64, 64, 8, 1), (BF16, 16, 576, 64, 1, 0, 1), (BF16, 16, 576, 64, 0, 1, 1),
    (F32, 16, 576, 16, 3, 1, 2)])
@pytest.mark.parametrize("prefill", [False, True])
def test_strides_and_offsets(mla, dtype, heads, width, page, pad, offset, layers, prefill):
    c = Case(11, dtype, heads, width, page, [333, 64, 700], [5, 64, 0] if prefill else None, pad=pad, offset=offset, layers=layers)
    c.check(c.run(mla))
    mla.mla_device_error()


@pytest.mark.parametrize("spread,scale", [(3.0, None), (1.0, 0.0), (1.0, -0.07), (0.01, 5.0)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scales(mla, spread, scale, dtype):
    # peaked and even weights, a scale of zero, a negative one
    for q in (None, [9, 40]):
        c = Case(13, dtype, 128, 576, 64, [300, 90], q, spread=spread, scale=scale)
        c.check(c.run(mla))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("prefill", [False, True])
def test_queries_that_attended_nothing_give_nothing(mla, dtype, prefill):
    c = Case(17, dtype, 16, 576, 64, [300, 90], [5, 6] if prefill else None)
    c.lse[0, 3] = -math.inf
    c.lse[1, :] = -math.inf
    c.lse[0, 5] = math.inf
    got = c.run(mla)
    c.check(got)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("prefill", [False, True])
def test_a_poisoned_sequence_does_not_reach_another(mla, dtype, prefill):
    # queries and rows of NaN in sequence 1: its own masses become NaN, the others' do not change
    c = Case(19, dtype, 16, 576, 64, [300, 90, 70], [5, 6, 33] if prefill else None)
    clean = c.run(mla)
    at = 5 if prefill else 1
    c.q[at] = math.nan
    n = c.cache[c.table[1, 0].long()].clone()
    n[3] = math.inf
    c.cache[c.table[1, 0].long()] = n
    got = c.run(mla)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])
    assert torch.isnan(got[1, :90 - 5]).all()


@pytest.mark.parametrize("dtype,page", [(BF16, 64), (BF16, 16), (F32, 64)])
@pytest.mark.parametrize("prefill", [False, True])
def test_bad_blocks_are_reported_and_left(mla, dtype, page, prefill):
    c = Case(23, dtype, 16, 576, page, [300, 200], [5, 6] if prefill else None)
    c.table[0, 1] = 10 ** 6
    got = c.run(mla)
    with pytest.raises(mla.MlaError) as e:
        mla.mla_device_error()
    assert e.value.status == mla.MLA_ERR_DEVICE_DATA
    assert torch.equal(got[0, page:2 * page], c.mass[0, page:2 * page])
    want, tol = c.want(1.0)
    off = (got.double() - want).abs() - tol
    off[0, page:2 * page] = 0
    assert off.max() <= 0
    mla.mla_device_error()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bad_lengths(mla, dtype):
    c = Case(29, dtype, 16, 576, 64, [300, 200, 90], [5, 6, 7])
    c.lens[1] = -4
    c.cu[3] = 10 ** 6              # beyond the queries
    got = c.run(mla)
    with pytest.raises(mla.MlaError):
        mla.mla_device_error()
    assert torch.equal(got[1:], c.mass[1:])
    want, tol = c.want(1.0)
    assert ((got[0].double() - want[0]).abs() - tol[0]).max() <= 0


def test_no_queries(mla):
    c = Case(31, BF16, 16, 576, 64, [300])
    mla.mla_decode_mass(c.mass[:0], c.q[:0], c.cache, c.table[:0], c.lens[:0], c.lse[:0], c.scale)
    before = c.mass.clone()
    mla.mla_prefill_mass(c.mass, c.q[:0], c.cache, c.table, torch.zeros(2, dtype=torch.int32, device="cuda"), c.lens, c.lse[:0], c.scale)
    assert torch.equal(c.mass, before)
    mla.mla_device_error()


@pytest.mark.parametrize("prefill", [False, True])
def test_captured_and_on_another_stream(mla, prefill):
    c = Case(37, BF16, 128, 576, 64, [3000, 90, 700], [40, 6, 300] if prefill else None)
    want = c.run(mla, 0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = c.mass.clone()
    side.wait_stream(torch.cuda.current_stream())
    c.run(mla, 0.5, mass=other, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, want)
    graph, mass = torch.cuda.CUDAGraph(), c.mass.clone()
    with torch.cuda.graph(graph):
        c.run(mla, 0.5, mass=mass)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(mass, want)


@pytest.mark.parametrize("prefill", [False, True])
def test_more_sequences_than_a_block_has_threads(mla, prefill):
    kv = [int(x) for x in torch.randint(0, 400, (300,), generator=torch.Generator().manual_seed(3))]
    q = [min(n, i % 7) for i, n in enumerate(kv)] if prefill else None
    c = Case(41, BF16, 16, 576, 64, kv, q)
    got = c.run(mla, 0.5)
    c.check(got, 0.5)
    assert torch.equal(got, c.run(mla, 0.5))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("prefill", [False, True])
def test_masses_in_a_wider_buffer(mla, dtype, prefill):
    c = Case(43, dtype, 16, 576, 64, [300, 90, 0, 129], [5, 6, 0, 129] if prefill else None)
    wide = torch.full((4, c.rows + 9), 7.0, device="cuda")
    mass = wide[:, 3:3 + c.rows]
    mass.copy_(c.mass)
    got = c.run(mla, 0.5, mass=mass)
    c.check(got.contiguous(), 0.5)
    assert (wide[:, :3] == 7).all() and (wide[:, 3 + c.rows:] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_rows_than_masses(mla, dtype):
    # a length beyond the masses counts as the largest that they hold, and is reported
    c = Case(47, dtype, 16, 576, 64, [300, 90])
    whole = c.run(mla)
    got = c.run(mla, mass=c.mass[:, :200].clone())
    with pytest.raises(mla.MlaError):
        mla.mla_device_error()
    assert torch.equal(got, whole[:, :200])


@pytest.mark.parametrize("dtype,page,pad", [(F32, 64, 0), (BF16, 48, 0), (F32, 16, 1), (BF16, 5, 4)])
@pytest.mark.parametrize("heads,width", [(16, 576), (20, 100), (64, 330), (128, 576), (7, 33)])
@pytest.mark.parametrize("prefill", [False, True])
def test_wide_tiles_on_the_cuda_cores(mla, dtype, page, pad, heads, width, prefill):
    # enough rows for tiles of 128, with 16 to 128 queries each; widths that end inside a step or a word, rows that
    # are not 16-byte aligned
    r = torch.Generator().manual_seed(heads + page)
    kv = [0, 1, 127, 128, 129] + [int(x) for x in torch.randint(0, 600, (40,), generator=r)]
    q = [min(n + 1, 1 + i % 3) for i, n in enumerate(kv)] if prefill else None
    c = Case(heads + width, dtype, heads, width, page, kv, q, pad=pad)
    got = c.run(mla, 0.5)
    c.check(got, 0.5)
    assert torch.equal(got, c.run(mla, 0.5))
    mla.mla_device_error()


@pytest.mark.parametrize("dtype,heads", [(F32, 16), (F32, 128), (BF16, 130)])
@pytest.mark.parametrize("kv,q", [([700], [300]), ([130, 0, 400, 65], [130, 2, 37, 1]), ([5000, 3], [20, 3])])
def test_queries_over_the_blocks_of_a_cluster(mla, dtype, heads, kv, q):
    c = Case(heads, dtype, heads, 192, 64, kv, q, tail=1)
    got = c.run(mla, 0.5)
    c.check(got, 0.5)
    assert torch.equal(got, c.run(mla, 0.5))
    mla.mla_device_error()


@pytest.mark.parametrize("batch", [385, 900])
@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_more_sequences_than_a_block_has_threads(mla, batch, prefill, dtype):
    r = torch.Generator().manual_seed(batch)
    kv = [int(x) for x in torch.randint(0, 300, (batch,), generator=r)]
    kv[:330] = [n if i % 3 == 0 else 0 for i, n in enumerate(kv[:330])]   # long runs of sequences without rows
    kv[40:200] = [0] * 160
    q = [min(n, i % 5) for i, n in enumerate(kv)] if prefill else None
    c = Case(batch, dtype, 16, 128, 64, kv, q)
    got = c.run(mla, 0.5)
    c.check(got, 0.5)
    assert torch.equal(got, c.run(mla, 0.5))
    mla.mla_device_error()


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype,heads,page", [(BF16, 16, 64), (BF16, 128, 64), (BF16, 70, 16), (F32, 16, 64), (BF16, 16, 5)])
@pytest.mark.parametrize("kv,q", [([300, 90], None), ([300, 90], [5, 6]), ([700, 40], [300, 64]), ([9000], [40])])
def test_whatever_a_query_without_attention_holds(mla, value, dtype, heads, page, kv, q):
    # lse -inf: a padded query, say, of values that nobody wrote; on the tensor cores and on the CUDA cores
    c = Case(53, dtype, heads, 576, page, kv, q)
    r = torch.Generator().manual_seed(heads)
    off = (torch.rand(c.tokens, heads, generator=r) < 0.3).cuda()
    off[-1, :] = True
    c.lse[off] = -math.inf
    want = c.want(0.5)
    zeros, poisoned = c.q.clone(), c.q.clone()
    zeros[off] = 0
    poisoned[off] = value
    c.q = zeros
    clean = c.run(mla, 0.5)
    c.q = poisoned
    got = c.run(mla, 0.5)
    mla.mla_device_error()
    assert torch.equal(got, clean)
    off = (got.double() - want[0]).abs() - want[1]
    assert not torch.isnan(off).any() and off.max() <= 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("prefill", [False, True])
def test_log_sum_exps_of_any_size(mla, dtype, prefill):
    # weights beyond float32 are infinite, those of +inf nothing, of NaN NaN: each for the rows that its query attends
    for lse, want in ((-3e38, math.inf), (-1e30, math.inf), (3e38, 0.0), (math.inf, 0.0), (math.nan, math.nan)):
        c = Case(59, dtype, 16, 576, 64, [300, 90], [5, 6] if prefill else None)
        clean = c.run(mla, 0.0)
        c.lse[1 if not prefill else 7, 3] = lse     # in sequence 1: its only query, or the third of six
        got = c.run(mla, 0.0)
        n = 90 if not prefill else 87
        assert torch.equal(got[0], clean[0]) and torch.equal(got[1, n:], clean[1, n:])
        seen = got[1, :n]
        if want == 0.0:
            assert torch.isfinite(seen).all() and (seen <= clean[1, :n]).all()
        else:
            assert (torch.isnan(seen) if math.isnan(want) else torch.isinf(seen)).all()

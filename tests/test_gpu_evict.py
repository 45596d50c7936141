"""Eviction against its definition: whole numbers and bits, so every comparison is exact."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def stays(mass, n, budget, sinks, recent):
    """Rows of n that stay, in order: NaN before everything, then the heaviest, then the lowest."""
    if n <= budget:
        return list(range(n))
    held = [t for t in range(n) if t < sinks or t >= n - recent]
    free = sorted(range(sinks, n - recent), key=lambda t: (0 if np.isnan(mass[t]) else 1, 0 if np.isnan(mass[t]) else -float(mass[t]), t))
    return sorted(held + free[:budget - len(held)])


class Case:
    def __init__(self, seed, lens, page, width, dtype, masses="spread", layers=1, pad=0, other=False, offset=0, extra=0):
        r = np.random.default_rng(seed)
        batch, self.page, self.lens = len(lens), page, lens
        most = max(1, -(-max(lens) // page)) + extra
        blocks = batch * most
        order = r.permutation(2 * blocks).astype(np.int32)
        self.table, self.other = order[:blocks].reshape(batch, most), order[blocks:].reshape(batch, most)
        # the codes of any type: bytes
        size = torch.empty(0, dtype=dtype).element_size()
        row = (width + pad) * size
        flat = torch.from_numpy(r.integers(0, 256, 2 * blocks * layers * page * row + offset * size, dtype=np.uint8)).cuda()
        self.whole = flat[offset * size:].view(dtype).view(2 * blocks, layers, page, width + pad)
        self.cache = self.whole[:, layers // 2, :, :width]
        rows = max(max(lens), 1) + extra
        m = np.exp(3 * r.standard_normal((batch, rows)))
        if masses == "few":
            m = r.integers(0, 3, (batch, rows)) / 4
        elif masses == "signs":
            m = r.standard_normal((batch, rows)) * 10.0 ** r.integers(-40, 30, (batch, rows))
            m[:, ::7] = -0.0
            m[:, 3::7] = 0.0
        elif masses == "odd":
            m = r.choice([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 1.0, 3e38], (batch, rows))
        elif masses == "same":
            m = np.full((batch, rows), 0.25)
        self.mass = torch.from_numpy(m.astype(np.float32))
        self.dst = self.other if other else self.table

    def want(self, budget, sinks, recent, mass_out, kept):
        """Bytes of the whole buffer, masses, lengths and kept rows."""
        whole = self.whole.clone()
        layer, width = self.whole.shape[1] // 2, self.cache.shape[2]
        lens_out, page = [], self.page
        for b, n in enumerate(self.lens):
            rows = stays(self.mass[b].numpy(), n, budget, sinks, recent)
            t, j = np.array(rows, dtype=np.int64), np.arange(len(rows))
            src = self.whole[self.table[b, t // page], layer, t % page, :width]
            whole[self.dst[b, j // page], layer, j % page, :width] = src
            kept[b] = -1
            kept[b, :len(rows)] = torch.from_numpy(t.astype(np.int32))
            out = torch.zeros(n)
            out[:len(rows)] = self.mass[b][t]
            upto = min(n, mass_out.shape[1])
            mass_out[b, :upto] = out[:upto]
            lens_out.append(len(rows))
        return whole, mass_out, lens_out, kept


def bits(t):
    return t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16 if t.element_size() == 2 else torch.uint8).cpu()


def run(mla, c, budget, sinks, recent, in_place=True, out_rows=None, stride=0, check=True):
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    batch, rows = c.mass.shape
    wide = torch.full((batch, rows + stride), 9.0, device="cuda")
    mass = wide[:, :rows]
    mass.copy_(c.mass)
    out_rows = rows if out_rows is None else out_rows
    mass_out = None if in_place else torch.full((batch, out_rows), 7.0, device="cuda")
    kept = torch.full((batch, budget), 5, dtype=torch.int32, device="cuda")
    want = c.want(budget, sinks, recent, c.mass.clone() if in_place else torch.full((batch, out_rows), 7.0), kept.cpu().clone())
    table = torch.from_numpy(c.table).cuda()
    dst = table if c.dst is c.table else torch.from_numpy(c.dst).cuda()
    lens_out = torch.zeros_like(lens)
    mla.mla_cache_evict(c.cache, mass, table, lens, budget, lens_out, sinks=sinks, recent=recent, block_table_out=dst,
                        mass_out=mass_out, kept_out=kept)
    if not check:
        return
    mla.mla_device_error()
    whole, m, l, k = want
    assert lens_out.tolist() == l
    assert torch.equal(kept.cpu(), k)
    assert torch.equal(bits(mass if in_place else mass_out), bits(m))
    assert torch.equal(bits(c.whole), bits(whole))
    assert stride == 0 or (wide[:, rows:] == 9).all()


@pytest.mark.parametrize("masses", ["spread", "few", "signs", "odd", "same"])
@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,budget,sinks,recent", [
    ([0, 1, 2, 3, 50, 129], 2, 0, 0), ([100, 64, 65, 63, 0], 64, 4, 16), ([300, 299, 1], 256, 256, 0), ([300, 17], 256, 0, 256),
    ([33], 1, 0, 1), ([1500, 1025, 1024, 1023], 1024, 1, 1000), ([700], 700, 3, 5), ([5], 900, 0, 2)])
def test_rows_that_stay(mla, masses, other, in_place, lens, budget, sinks, recent):
    run(mla, Case(len(lens) + budget, lens, 16, 64, torch.bfloat16, masses, other=other), budget, sinks, recent, in_place)


@pytest.mark.parametrize("n,budget", [(16384, 4096), (16385, 16384), (16385, 5000), (40000, 333), (70001, 40000)])
@pytest.mark.parametrize("masses", ["spread", "few", "odd"])
@pytest.mark.parametrize("in_place", [False, True])
def test_long_sequences(mla, n, budget, masses, in_place):
    # more rows than a block holds in registers
    run(mla, Case(n, [n, n // 3], 64, 8, torch.bfloat16, masses), budget, 3, 65, in_place)


@pytest.mark.parametrize("dtype,width,page,layers,pad,offset", [
    (torch.bfloat16, 576, 64, 3, 0, 0), (torch.bfloat16, 576, 64, 1, 8, 0), (torch.float32, 576, 16, 1, 0, 0),
    (torch.uint8, 656, 64, 2, 0, 0), (torch.uint8, 576, 16, 1, 0, 0), (torch.uint8, 577, 5, 1, 0, 0), (torch.bfloat16, 20, 3, 1, 0, 1),
    (torch.bfloat16, 22, 7, 1, 0, 0), (torch.float32, 3, 1, 1, 0, 0), (torch.uint8, 16, 128, 1, 0, 0), (torch.float32, 5, 8, 1, 0, 1)])
@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("lens", [[700], [333, 0, 90, 801] * 5])
def test_types_and_strides(mla, dtype, width, page, layers, pad, offset, other, lens):
    run(mla, Case(width + page, lens, page, width, dtype, layers=layers, pad=pad, other=other, offset=offset), 300, 4, 33)


def test_many_sequences(mla):
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 400, 200)]
    run(mla, Case(5, lens, 16, 576, torch.bfloat16), 128, 4, 16)


@pytest.mark.parametrize("out_rows", [100, 256, 700])
def test_masses_of_other_widths(mla, out_rows):
    run(mla, Case(9, [500, 90, 256], 16, 64, torch.bfloat16, extra=17), 256, 2, 8, in_place=False, out_rows=out_rows, stride=5)


def test_partly_moved_tables(mla):
    # the first pages stay where they are (shared with nobody), the others go to new ones
    c = Case(11, [200, 130], 16, 64, torch.bfloat16)
    c.dst = c.other.copy()
    c.dst[:, :3] = c.table[:, :3]
    run(mla, c, 100, 4, 8)


def test_lengths_in_place_and_no_kept(mla):
    c = Case(13, [300, 10], 16, 64, torch.bfloat16)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    want = c.want(64, 2, 8, c.mass.clone(), torch.zeros(2, 64, dtype=torch.int32))
    mass = c.mass.cuda()
    mla.mla_cache_evict(c.cache, mass, torch.from_numpy(c.table).cuda(), lens, 64, lens, sinks=2, recent=8)
    mla.mla_device_error()
    assert lens.tolist() == want[2] and torch.equal(mass.cpu(), want[1]) and torch.equal(bits(c.whole), bits(want[0]))


@pytest.mark.parametrize("which", ["old", "new", "negative"])
def test_bad_blocks_are_reported_and_left(mla, which):
    c = Case(17, [200, 200], 16, 64, torch.bfloat16, "same", other=which == "new")
    before = c.whole.clone()
    rows = stays(c.mass[1].numpy(), 200, 100, 4, 8)
    bad = 1 if which == "new" else 12          # of sequence 1: a page that rows move to, or from
    (c.dst if which == "new" else c.table)[1, bad] = -3 if which == "negative" else 10 ** 6
    good = c.table.copy(), c.dst.copy()
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    lens_out = torch.zeros_like(lens)
    table = torch.from_numpy(c.table).cuda()
    mla.mla_cache_evict(c.cache, c.mass.cuda(), table, lens, 100, lens_out, sinks=4, recent=8,
                        block_table_out=None if c.dst is c.table else torch.from_numpy(c.dst).cuda())
    with pytest.raises(mla.MlaError) as e:
        mla.mla_device_error()
    assert e.value.status == mla.MLA_ERR_DEVICE_DATA
    assert lens_out.tolist() == [100, 100]
    want = before.clone()
    for b in range(2):
        for j, t in enumerate(rows):
            if b == 1 and bad == (j if which == "new" else t) // 16:
                continue
            want[good[1][b, j // 16], 0, j % 16] = before[good[0][b, t // 16], 0, t % 16]
    assert torch.equal(bits(c.whole), bits(want))
    mla.mla_device_error()


def test_lengths_beyond_the_table(mla):
    c = Case(19, [160, 90], 16, 64, torch.bfloat16)
    want = c.want(100, 0, 10, c.mass.clone(), torch.zeros(2, 100, dtype=torch.int32))
    mass, lens_out = c.mass.cuda(), torch.zeros(2, dtype=torch.int32, device="cuda")
    lens = torch.tensor([10 ** 9, -5], dtype=torch.int32, device="cuda")
    mla.mla_cache_evict(c.cache, mass, torch.from_numpy(c.table).cuda(), lens, 100, lens_out, recent=10)
    with pytest.raises(mla.MlaError):
        mla.mla_device_error()
    assert lens_out.tolist() == [100, 0]
    assert torch.equal(mass[0].cpu(), want[1][0]) and torch.equal(mass[1].cpu(), c.mass[1])


def test_captured_graphs_and_streams(mla):
    # two graphs with workspaces of their own, replayed twice on two streams; the masses stay, so every replay
    # moves the same rows
    cases = [Case(s, [500, 90, 400], 16, 64, torch.bfloat16, other=True) for s in (21, 22)]
    graphs, outs = [], []
    for c in cases:
        args = (c.cache, c.mass.cuda(), torch.from_numpy(c.table).cuda(), torch.tensor(c.lens, dtype=torch.int32, device="cuda"))
        out, lens_out = torch.full_like(c.mass, 7.0).cuda(), torch.zeros(3, dtype=torch.int32, device="cuda")
        dst, ws = torch.from_numpy(c.dst).cuda(), torch.empty(mla.mla_cache_evict_workspace_size(3, c.mass.shape[1], 200),
                                                              dtype=torch.uint8, device="cuda")
        want = c.want(200, 4, 9, torch.full_like(c.mass, 7.0), torch.zeros(3, 200, dtype=torch.int32))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mla.mla_cache_evict(*args, 200, lens_out, sinks=4, recent=9, block_table_out=dst, mass_out=out, workspace=ws)
        graphs.append((g, args, dst, ws))
        outs.append((c, want, out, lens_out))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(2):
        for s, (g, *_) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, want, out, lens_out in outs:
        assert lens_out.tolist() == want[2] and torch.equal(out.cpu(), want[1]) and torch.equal(bits(c.whole), bits(want[0]))


@pytest.mark.parametrize("lens,budget", [([140001], 70000), ([131073, 0, 1, 5, 9001], 131000), ([20000, 700, 16385, 8192, 2], 600)])
@pytest.mark.parametrize("masses", ["spread", "few", "odd", "same"])
@pytest.mark.parametrize("in_place", [False, True])
def test_several_blocks_a_sequence(mla, lens, budget, masses, in_place):
    # sequences of all lengths in calls whose tables have room for long ones; the first more than eight blocks hold
    run(mla, Case(len(lens) + budget, lens, 64, 24, torch.bfloat16, masses, extra=3), budget, 3, 65, in_place)


def test_several_blocks_a_slice(mla):
    # wide rows, one to nine sequences: a slice's rows are dealt over eight blocks down to one
    for lens in ([5000], [4000, 3000], [2500] * 3 + [17], [1500, 2600] * 4 + [900]):
        for dtype, width in ((torch.bfloat16, 576), (torch.float32, 576), (torch.uint8, 656)):
            run(mla, Case(len(lens) + width, lens, 64, width, dtype), 1300, 4, 64)


def test_very_wide_rows(mla):
    # more slices of columns than a grid has rows
    run(mla, Case(31, [5, 9], 2, 300001, torch.uint8), 4, 1, 1)


@pytest.mark.parametrize("several", [False, True])
def test_clusters_captured_with_lengths_in_place(mla, several):
    # one long sequence beside short ones, captured once and replayed twice: the second replay finds nothing to drop
    lens = [20000, 3, 0, 12000] if several else [20000]
    c = Case(41, lens, 64, 64, torch.bfloat16)
    mass, table = c.mass.cuda(), torch.from_numpy(c.table).cuda()
    budget, n = 5000, torch.tensor(lens, dtype=torch.int32, device="cuda")
    kept = torch.full((len(lens), budget), 5, dtype=torch.int32, device="cuda")
    want = c.want(budget, 4, 64, c.mass.clone(), kept.cpu().clone())
    before = c.whole.clone(), c.mass.clone(), n.clone()
    ws = torch.empty(mla.mla_cache_evict_workspace_size(len(lens), mass.shape[1], budget), dtype=torch.uint8, device="cuda")

    def call():
        mla.mla_cache_evict(c.cache, mass, table, n, budget, n, sinks=4, recent=64, block_table_out=table, kept_out=kept, workspace=ws)

    call()
    torch.cuda.synchronize()
    c.whole.copy_(before[0])
    mass.copy_(before[1])
    n.copy_(before[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    torch.cuda.synchronize()
    assert n.tolist() == want[2] and torch.equal(kept.cpu(), want[3])
    assert torch.equal(bits(mass), bits(want[1])) and torch.equal(bits(c.whole), bits(want[0]))
    graph.replay()
    mla.mla_device_error()
    assert n.tolist() == want[2]
    assert torch.equal(kept.cpu(), torch.where(torch.arange(budget) < torch.tensor(want[2])[:, None], torch.arange(budget), -1).int())
    assert torch.equal(bits(mass), bits(want[1])) and torch.equal(bits(c.whole), bits(want[0]))


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_rows_that_do_not_move_need_no_block(mla, bad):
    # a copy of the table as block_table_out: rows whose place does not change are not looked at, as in place
    c = Case(61, [200, 90, 130], 16, 64, torch.bfloat16, other=False)
    c.mass[:, :40] = 1e6                      # the first pages' rows stay where they are
    want = c.want(100, 0, 4, c.mass.clone(), torch.zeros(3, 100, dtype=torch.int32))
    c.table[:, :2] = bad                      # 32 rows without blocks; of sequence 1 (90 rows) every row stays in place
    c.table[1] = bad
    for copy in (False, True):
        table = torch.from_numpy(c.table).cuda()
        whole, mass = c.whole.clone(), c.mass.cuda()
        n = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
        mla.mla_cache_evict(whole[:, 0], mass, table, n, 100, n, recent=4, block_table_out=table.clone() if copy else None)
        mla.mla_device_error()
        assert n.tolist() == want[2] and torch.equal(mass.cpu(), want[1]) and torch.equal(bits(whole), bits(want[0]))
    # a row whose new page lies outside the new table is one that cannot move
    short = table[:, :4].clone()
    mla.mla_cache_evict(c.whole[:, 0], c.mass.cuda(), table, torch.tensor(c.lens, dtype=torch.int32, device="cuda"), 100,
                        torch.zeros(3, dtype=torch.int32, device="cuda"), recent=4, block_table_out=short)
    with pytest.raises(mla.MlaError):
        mla.mla_device_error()

"""The ds_mla write and the read-backs with so many rows that a warp takes several, at every remainder, exactly."""
import pytest
import torch

from test_gpu_cache_io import entry_of, latents, read, read_case, same

pytestmark = pytest.mark.gpu


def many():
    """Rows from which on a warp takes four: 32 an SM."""
    return 32 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("more", [-1, 0, 1, 2, 3])
@pytest.mark.parametrize("first", [0, 3])
def test_write_of_many_rows(mla, dtype, more, first):
    # padding, slots past the cache and good ones side by side; first 3: source rows off 16 bytes
    tokens, page = many() + more, 64
    kv_c, k_pe = latents(tokens, 90 + more, dtype)
    kv_c[5, 17], kv_c[6, 300], kv_c[7], kv_c[8, 511] = float("nan"), float("inf"), 0.0, -0.0
    wide = torch.zeros(tokens, 700, dtype=dtype, device="cuda")
    wide[:, first:first + 512], wide[:, 600 + first:664 + first] = kv_c.cuda(), k_pe.cuda()
    blocks = -(-tokens // page) + 1
    g = torch.Generator().manual_seed(91)
    slots = torch.randperm(blocks * page, generator=g)[:tokens]
    kind = torch.randint(0, 10, (tokens,), generator=g)
    slots[kind == 2] += blocks * page
    slots[kind == 0], slots[kind == 1], slots[-2] = -1, -2 ** 40, -1
    whole = torch.randint(0, 256, (blocks, 2, page, 656), dtype=torch.uint8, device="cuda")
    want = whole.clone()
    mla.mla_cache_write_ds_mla(whole[:, 1], wide[:, first:first + 512], wide[:, 600 + first:664 + first], slots.cuda())
    with pytest.raises(mla.MlaError) as e:
        mla.mla_device_error()
    assert e.value.status == mla.MLA_ERR_DEVICE_DATA
    keep = ((slots >= 0) & (slots < blocks * page)).nonzero()[:, 0]
    want[(slots[keep] // page).cuda(), 1, (slots[keep] % page).cuda()] = entry_of(kv_c, k_pe)[keep].cuda()
    off = (whole != want).nonzero()
    assert not len(off), f"{len(off)} bytes differ, the first at {off[0].tolist()}"


FORMATS = [("plain", 576), ("plain", 512), ("plain", 37), ("plain", 1000), ("e4m3", 576), ("e4m3", 45), ("e4m3", 1544),
           ("ds_mla", 576)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,width", FORMATS)
@pytest.mark.parametrize("more", [0, 1, 2, 3])
@pytest.mark.parametrize("first", [0, 1])
def test_read_of_many_rows(mla, dtype, fmt, width, more, first):
    # sequences of 0 to 17 rows: their borders fall everywhere within a warp's four. Bad block ids, and rows of
    # no sequence, beside good ones; first 1: rows of out off 16 bytes. Widths of 1000 and 1544 take several
    # rounds of chunks
    rows, page, tail = many() + more, 16, 5
    kv = []
    while sum(kv) < rows:
        kv.append(min(7 * len(kv) % 18, rows - sum(kv)))
    starts = [5 * i % 23 for i in range(len(kv))]
    cache, scale, table, cu, st, want = read_case(fmt, dtype, width, page, kv, starts, layers=2)
    table, at = table.clone(), cu.tolist()
    bad = torch.zeros(rows, dtype=torch.bool)
    for b in (11, 300, len(kv) - 1):
        table[b, 0] = -1 if b == 11 else 2 ** 31 - 1
        bad[at[b]:at[b] + max(0, min(kv[b], page - starts[b]))] = True
    st[200] = -100                                      # before the sequence's first row
    bad[at[200]:at[201]] = True
    assert bad.sum() > 20
    out = torch.full((rows + tail, width + 8), 5.0, dtype=dtype, device="cuda")
    read(mla, fmt, out[:, first:first + width], cache, table, cu, st, scale)
    with pytest.raises(mla.MlaError) as e:
        mla.mla_device_error()
    assert e.value.status == mla.MLA_ERR_DEVICE_DATA
    got = out[:, first:first + width]
    assert same(got[:rows][~bad.cuda()], want[~bad])
    assert (got[:rows][bad.cuda()] == 5).all() and (got[rows:] == 5).all()
    assert (out[:, :first] == 5).all() and (out[:, first + width:] == 5).all()


@pytest.mark.parametrize("fmt,width", [("plain", 576), ("e4m3", 576), ("ds_mla", 576)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_read_of_many_whole_rows(mla, dtype, fmt, width):
    # the form a user's buffers have: contiguous rows, 16-byte aligned
    rows = 4 * many() + 2
    kv, starts = [rows // 3, 0, rows - rows // 3 - 1, 1], [0, 9, 70, 3]
    cache, scale, table, cu, st, want = read_case(fmt, dtype, width, 16, kv, starts)
    out = torch.full((rows + 1, width), 5.0, dtype=dtype, device="cuda")
    read(mla, fmt, out, cache, table, cu, st, scale)
    mla.mla_device_error()
    assert same(out[:rows], want) and (out[rows:] == 5).all()

"""The ds_mla cache write and the read-backs against their definitions, value by value."""
import numpy as np
import pytest
import torch

import window_ref as wr

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def entry_of(kv_c, k_pe):
    """The 656 bytes of each row, from the definition, on the CPU: the quotient in 64 bits, rounded once."""
    x = kv_c.float().cpu().view(-1, 4, 128)
    top = torch.where(x.isnan(), torch.zeros_like(x), x).abs().amax(-1).clamp_max(torch.finfo(torch.float32).max)
    scale = (top / 448).clamp_min(2.0 ** -126)
    y = (x.double() / scale.double()[..., None]).clamp(-448, 448)                # clamp keeps a NaN
    # e4m3: steps of 2^(exponent - 3), no exponent below -6; torch.round takes halves to even
    step = torch.exp2(y.abs().clamp_min(2.0 ** -20).log2().floor().clamp_min(-6) - 3)
    codes = (torch.round(y / step) * step).float().to(E4M3).view(-1, 512)
    pe = k_pe.cpu().to(torch.bfloat16)
    return torch.cat([codes.view(torch.uint8), scale.view(torch.uint8), pe.contiguous().view(torch.uint8)], 1)


def latents(tokens, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    spread = torch.exp(2 * torch.randn(tokens, 4, 1, generator=g))
    x = (torch.randn(tokens, 4, 128, generator=g) * spread).view(tokens, 512).to(dtype)
    return x, torch.randn(tokens, 64, generator=g).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,page,layers", [(1, 64, 1), (64, 64, 3), (77, 16, 1), (130, 1, 2), (2049, 100, 1)])
def test_write_ds_mla(mla, dtype, tokens, page, layers):
    kv_c, k_pe = latents(tokens, tokens, dtype)
    if tokens > 20:
        kv_c[3] = 0                                  # a group of zeros
        kv_c[4, :128] = 1e-38                        # below the smallest scale's reach
        kv_c[5, 130] = float("inf")
        kv_c[6, 140] = float("nan")
        kv_c[7, 256:384] = -float("inf")
        kv_c[8, 384:] = float("nan")
        kv_c[9, 5] = 3e38
    blocks = -(-tokens // page) + 2
    order = np.random.default_rng(tokens).permutation(blocks * page)[:tokens].astype(np.int64)
    order[::7] = -1
    whole = torch.randint(0, 256, (blocks, layers, page, 656), dtype=torch.uint8, device="cuda")
    before = whole.clone()
    cache = whole[:, layers - 1]
    mla.mla_cache_write_ds_mla(cache, kv_c.cuda(), k_pe.cuda(), torch.from_numpy(order).cuda())
    mla.mla_device_error()
    want = before.clone()
    rows = torch.from_numpy(order)
    keep = (rows >= 0).nonzero()[:, 0]
    want[rows[keep].cuda() // page, layers - 1, rows[keep].cuda() % page] = entry_of(kv_c, k_pe)[keep].cuda()
    # a NaN of the rope may change its payload; every other byte is the definition's
    assert torch.equal(whole, want)


def test_write_ds_mla_rounds_a_quotient_once(mla):
    # short values and short maxima: many quotients near the middle of two codes, some of them where
    # float32's nearest to the quotient is the middle itself (the last lines before the call show it)
    m = torch.arange(128, 256)
    x = torch.zeros(128, 4, 128)
    for g in range(4):
        x[:, g] = (torch.arange(128) + 128 * (g & 1)) * 2.0 ** -(g + 1)
        x[:, g, 0] = m * 2.0 ** -(g // 2)
    kv_c = x.view(128, 512).to(torch.bfloat16)
    assert torch.equal(kv_c.float(), x.view(128, 512))
    k_pe = torch.zeros(128, 64, dtype=torch.bfloat16)
    want = entry_of(kv_c, k_pe)
    top = x.abs().amax(-1, keepdim=True) / 448
    assert not torch.equal((x / top).to(E4M3).view(128, 512).view(torch.uint8), want[:, :512])
    cache = torch.zeros(2, 64, 656, dtype=torch.uint8, device="cuda")
    mla.mla_cache_write_ds_mla(cache, kv_c.cuda(), k_pe.cuda(), torch.arange(128, device="cuda"))
    mla.mla_device_error()
    assert torch.equal(cache.view(128, 656).cpu(), want)


def test_write_ds_mla_strided_rows_and_views(mla):
    # source rows inside wider rows, not 16-byte aligned; a [.., 1, 656] cache
    kv_c, k_pe = latents(50, 3, torch.bfloat16)
    wide = torch.zeros(50, 700, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:515], wide[:, 601:665] = kv_c.cuda(), k_pe.cuda()
    cache = torch.zeros(4, 16, 1, 656, dtype=torch.uint8, device="cuda")
    mla.mla_cache_write_ds_mla(cache, wide[:, 3:515], wide[:, 601:665], torch.arange(50, device="cuda"))
    mla.mla_device_error()
    assert torch.equal(cache.view(64, 656)[:50].cpu(), entry_of(kv_c, k_pe))
    assert (cache.view(64, 656)[50:] == 0).all()


def test_write_ds_mla_slots_past_the_cache(mla):
    kv_c, k_pe = latents(3, 4, torch.float32)
    cache = torch.zeros(2, 8, 656, dtype=torch.uint8, device="cuda")
    mla.mla_cache_write_ds_mla(cache, kv_c.cuda(), k_pe.cuda(), torch.tensor([16, 2, 2 ** 40], device="cuda"))
    with pytest.raises(mla.MlaError) as e:
        mla.mla_device_error()
    assert e.value.status == mla.MLA_ERR_DEVICE_DATA
    assert torch.equal(cache.view(16, 656)[2].cpu(), entry_of(kv_c, k_pe)[1])
    assert int((cache != 0).any(-1).sum()) == 1


def test_written_values_are_near(mla):
    # half an e4m3 step of the value (2^-4 of it), half the smallest step below the normal codes
    # (2^-10 of the scale), and the scale's own rounding
    kv_c, k_pe = latents(500, 5, torch.float32)
    cache = torch.zeros(8, 64, 656, dtype=torch.uint8, device="cuda")
    mla.mla_cache_write_ds_mla(cache, kv_c.cuda(), k_pe.cuda(), torch.arange(500, device="cuda"))
    out = torch.zeros(500, 576, device="cuda")
    mla.mla_cache_read_ds_mla(out, cache, torch.arange(8, dtype=torch.int32, device="cuda")[None],
                              torch.tensor([0, 500], dtype=torch.int32, device="cuda"))
    mla.mla_device_error()
    x = kv_c.double().view(500, 4, 128)
    scale = x.abs().amax(-1, keepdim=True) / 448
    off = (out[:, :512].cpu().double().view(500, 4, 128) - x).abs()
    assert (off <= x.abs() * (2.0 ** -4 + 2.0 ** -20) + scale * 2.0 ** -10 * 1.0001).all()
    assert torch.equal(out[:, 512:].cpu(), k_pe.to(torch.bfloat16).float())


def read_case(fmt, dtype, width, page, kv, starts, seed=0, layers=1):
    """A cache of the format, its rows' values [blocks, page, width] in dtype, table, cu and starts."""
    g = torch.Generator().manual_seed(seed)
    per = max(1, max(-(-(a + b) // page) for a, b in zip(kv, starts)))
    blocks = per * len(kv) + 1
    table = torch.randperm(blocks - 1, generator=g).to(torch.int32).view(len(kv), per)
    if fmt == "plain":
        cache = torch.randn(blocks, layers, page, width, generator=g).to(dtype)
        cache[0, :, 0, :3] = torch.tensor([float("nan"), -0.0, float("inf")])
        values, scale = cache[:, layers - 1], None
    elif fmt == "e4m3":
        codes = torch.randint(0, 256, (blocks, layers, page, width), generator=g, dtype=torch.uint8)
        cache, scale = codes.view(E4M3), torch.tensor([0.0371])
        values = (cache[:, layers - 1].float() * scale).to(dtype)
    else:
        codes = torch.randint(0, 256, (blocks, layers, page, 512), generator=g, dtype=torch.uint8)
        scales = torch.exp(3 * torch.randn(blocks, layers, page, 4, generator=g))
        pe = torch.randn(blocks, layers, page, 64, generator=g).to(torch.bfloat16)
        cache, scale = torch.cat([codes, scales.view(torch.uint8), pe.view(torch.uint8)], -1), None
        lat = (codes.view(E4M3).float().view(*codes.shape[:3], 4, 128) * scales[..., None]).flatten(-2)
        values = torch.cat([lat, pe.float()], -1)[:, layers - 1].to(dtype)
    cu = torch.tensor([0, *np.cumsum(kv)], dtype=torch.int32)
    want = torch.cat([values[table[b].long()[(s + torch.arange(n)) // page], (s + torch.arange(n)) % page]
                      for b, (n, s) in enumerate(zip(kv, starts))])
    dev = cache.cuda()[:, layers - 1]
    return dev, scale, table.cuda(), cu.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), want


def read(mla, fmt, out, cache, table, cu, starts, scale):
    if fmt == "plain":
        mla.mla_cache_read(out, cache, table, cu, seq_starts=starts)
    elif fmt == "e4m3":
        mla.mla_cache_read_fp8(out, cache, table, cu, scale.cuda(), seq_starts=starts)
    else:
        mla.mla_cache_read_ds_mla(out, cache, table, cu, seq_starts=starts)


def same(got, want):
    """Equal values, NaN where NaN is expected."""
    got, want = got.cpu(), want.cpu()
    return bool((((got == want) & (got.signbit() == want.signbit())) | (got.isnan() & want.isnan())).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,width", [("plain", 576), ("plain", 512), ("plain", 37), ("e4m3", 576), ("e4m3", 512),
                                       ("e4m3", 45), ("ds_mla", 576)])
@pytest.mark.parametrize("page,layers,kv,starts", [
    (64, 1, [1], [0]), (64, 3, [130, 0, 64, 7], [0, 5, 64, 1000]), (1, 1, [3, 9], [2, 0]), (100, 2, [0, 0, 250], [0, 9, 1])])
def test_read(mla, dtype, fmt, width, page, layers, kv, starts):
    cache, scale, table, cu, st, want = read_case(fmt, dtype, width, page, kv, starts, layers=layers)
    rows = sum(kv)
    out = torch.full((rows + 3, width), 5.0, dtype=dtype, device="cuda")
    read(mla, fmt, out, cache, table, cu, st, scale)
    mla.mla_device_error()
    assert same(out[:rows], want)
    assert (out[rows:] == 5).all()


@pytest.mark.parametrize("fmt", ["plain", "e4m3", "ds_mla"])
def test_read_into_strided_rows(mla, fmt):
    # an out whose rows are not 16-byte aligned, and one of aligned wider rows
    cache, scale, table, cu, st, want = read_case(fmt, torch.bfloat16, 576, 16, [40, 41], [3, 0])
    for first, wide in ((1, 601), (8, 640)):
        whole = torch.full((81, wide), 5.0, dtype=torch.bfloat16, device="cuda")
        read(mla, fmt, whole[:, first:first + 576], cache, table, cu, st, scale)
        mla.mla_device_error()
        assert same(whole[:, first:first + 576], want)
        assert (whole[:, :first] == 5).all() and (whole[:, first + 576:] == 5).all()


@pytest.mark.parametrize("fmt", ["plain", "e4m3", "ds_mla"])
def test_read_leaves_bad_rows(mla, fmt):
    # a bad block id, a negative start, a start beyond the table: those rows stay, the others are read
    cache, scale, table, cu, st, want = read_case(fmt, torch.bfloat16, 576, 16, [40, 20, 10, 8], [0, 0, 0, 0])
    table, st = table.clone(), st.clone()
    table[0, 1] = 10 ** 7
    st[1] = -3
    st[2] = 16 * table.shape[1] - 4
    out = torch.full((78, 576), 5.0, dtype=torch.bfloat16, device="cuda")
    read(mla, fmt, out, cache, table, cu, st, scale)
    with pytest.raises(mla.MlaError) as e:
        mla.mla_device_error()
    assert e.value.status == mla.MLA_ERR_DEVICE_DATA
    assert same(out[:16], want[:16]) and same(out[32:40], want[32:40]) and same(out[70:], want[70:])
    assert (out[16:32] == 5).all() and (out[40:43] == 5).all() and (out[64:70] == 5).all()


def test_read_offsets_beyond_32_bits(mla):
    stride = 2 ** 32 + 4096
    far = torch.empty(stride + 64 * 656, dtype=torch.uint8, device="cuda").as_strided((2, 64, 656), (stride, 656, 1))
    cache, scale, table, cu, st, want = read_case("ds_mla", torch.bfloat16, 576, 64, [100], [0])
    far[0].copy_(cache[table[0, 0]])
    far[1].copy_(cache[table[0, 1]])
    out = torch.zeros(100, 576, dtype=torch.bfloat16, device="cuda")
    mla.mla_cache_read_ds_mla(out, far, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), cu)
    mla.mla_device_error()
    assert same(out, want)


def test_write_read_attend_together(mla):
    """A chunk over a quantised prefix, then a single token: rows written as ds_mla entries are attended
    sparsely where they lie, and read back as a cache for the windowed prefill and decode."""
    heads, kv, new, window, sinks = 128, 300, 7, 120, 4
    kv_c, k_pe = latents(kv, 8, torch.bfloat16)
    kv_c = kv_c / kv_c.float().std()
    page = 64
    blocks = 5
    order = torch.randperm(blocks, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    at = torch.arange(kv)
    slots = (order.long()[at // page] * page + at % page).cuda()
    entries = torch.zeros(blocks, page, 656, dtype=torch.uint8, device="cuda")
    mla.mla_cache_write_ds_mla(entries, kv_c.cuda(), k_pe.cuda(), slots)
    cu = torch.tensor([0, kv], dtype=torch.int32, device="cuda")
    rows = torch.zeros(blocks * page, 576, dtype=torch.bfloat16, device="cuda")
    mla.mla_cache_read_ds_mla(rows, entries, order.cuda()[None], cu)
    q = torch.randn(new, heads, 576, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    scale = 192 ** -0.5
    o = torch.zeros(new, heads, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(new, heads, device="cuda")
    straight = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
    mla.mla_prefill_window(o, q, rows.view(blocks, page, 576), straight,
                           torch.tensor([0, new], dtype=torch.int32, device="cuda"),
                           torch.tensor([kv], dtype=torch.int32, device="cuda"), 512, 64, scale, window, sinks=sinks,
                           lse_out=lse)
    last, last_lse = torch.zeros_like(o[:1]), torch.zeros_like(lse[:1])
    mla.mla_decode_window(last, q[-1:], rows.view(blocks, page, 576), straight,
                          torch.tensor([kv], dtype=torch.int32, device="cuda"), 512, 64, scale, window, sinks=sinks,
                          lse_out=last_lse)
    # the same rows of the last token as a list of slots over the entries themselves
    seen = [slots[t].item() for t in wr.rows_seen(kv - 1, window, sinks)]
    sparse, sparse_lse = torch.zeros_like(o[:1]), torch.zeros_like(lse[:1])
    mla.mla_decode_sparse_fp8(sparse, q[-1:], entries, torch.tensor([seen], dtype=torch.int32, device="cuda"), scale,
                              lse_out=sparse_lse)
    mla.mla_device_error()
    rows64 = rows.double().cpu().numpy()
    for i in range(new):
        seen = wr.rows_seen(kv - new + i, window, sinks)
        want, want_lse, mean, big = wr.attend(q[i].double().cpu().numpy(), rows64[seen], 512, scale)
        d = 600 * 2.0 ** -23 * big + len(seen) * 2.0 ** -23 + 2.0 ** -20
        tol = 2.0 ** -8 * (mean + np.abs(want)) * 1.01 + 2 * d[:, None] * mean
        assert (np.abs(o[i].double().cpu().numpy() - want) <= tol).all()
        assert (np.abs(lse[i].double().cpu().numpy() - want_lse) <= d + 1e-5).all()
    assert (np.abs(last[0].double().cpu().numpy() - want) <= tol).all()
    # the sparse decode rounds each weight three times (2^-8 each), and values once
    assert (np.abs(sparse[0].double().cpu().numpy() - want) <= 4 * tol).all()
    assert (sparse_lse - last_lse).abs().max() < 1.2e-2


def test_refusals_of_the_binding(mla):
    cache = torch.zeros(2, 8, 656, dtype=torch.uint8, device="cuda")
    kv_c, k_pe = torch.zeros(3, 512, device="cuda"), torch.zeros(3, 64, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    for args in ((cache, kv_c, k_pe, slots.int()), (cache.float(), kv_c, k_pe, slots), (cache, kv_c.half(), k_pe.half(), slots),
                 (cache, kv_c, k_pe.bfloat16(), slots), (cache, kv_c[:, :256], k_pe, slots), (cache, kv_c, k_pe, slots[:2]),
                 (cache, kv_c.cpu(), k_pe, slots), (cache[:, :, :640], kv_c, k_pe, slots),
                 (cache[:, :, 1:], kv_c, k_pe, slots)):
        with pytest.raises(mla.MlaError):
            mla.mla_cache_write_ds_mla(*args)
    out = torch.zeros(4, 576, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for args in ((out[:, :512], cache, table, cu), (out, cache, table, cu[:1]), (out, cache, table.long(), cu),
                 (out, cache, table, cu.long()), (out.half(), cache, table, cu), (out, cache.cpu(), table, cu),
                 (out.t(), cache, table, cu), (out, cache, table[0], cu), (out, cache, table[0, 0], cu),
                 (out, cache, table, cu[0]), (out, cache[0], table, cu), (out[0], cache, table, cu)):
        with pytest.raises(mla.MlaError):
            mla.mla_cache_read_ds_mla(*args)
    with pytest.raises(mla.MlaError):
        mla.mla_cache_read(out, torch.zeros(1, 8, 512, device="cuda"), table, cu)
    with pytest.raises(mla.MlaError):
        mla.mla_cache_read(out, torch.zeros(1, 8, 576, device="cuda").bfloat16(), table, cu)
    with pytest.raises(mla.MlaError):
        mla.mla_cache_read_fp8(out, torch.zeros(1, 8, 576, dtype=torch.uint8, device="cuda"), table, cu, torch.ones(1))
    assert (out == 0).all() and (cache == 0).all()

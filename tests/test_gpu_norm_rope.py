"""Norms and rotations of query heads and of cache rows against 64 bits, with derived bounds."""
import pytest
import torch

import norm_rope_ref as ref

pytestmark = pytest.mark.gpu

EPS = 1e-6
BF16, F32 = torch.bfloat16, torch.float32
POSITIONS = 300

# heads, nope, rope, latent
V3, LITE, NOPE, ODD, WIDE = (128, 128, 64, 512), (16, 128, 64, 512), (64, 256, 0, 512), (3, 7, 6, 20), (5, 1000, 64, 1000)


def inputs(seed, tokens, dims, dtype, per_head=True, pad=0):
    heads, nope, rope, latent = dims
    g = torch.Generator().manual_seed(seed)

    def draw(*shape):
        return torch.randn(*shape, generator=g)

    width = nope + rope
    q = (draw(tokens, heads, width + pad) * torch.exp(draw(tokens, heads, 1))).to(dtype)
    kv = (draw(tokens, latent + rope + pad) * torch.exp(2 * draw(tokens, 1))).to(dtype)
    qw = (1 + draw(heads, width) / 4).to(dtype) if per_head else (1 + draw(width) / 4).to(dtype)
    kw = (1 + draw(latent) / 4).to(dtype)
    pos = torch.randint(0, POSITIONS, (tokens,), generator=g)
    return q[..., :width], kv[:, :latent + rope], qw, kw, pos, ref.table(POSITIONS, rope)


def slots_of(seed, tokens, rows):
    order = torch.randperm(rows, generator=torch.Generator().manual_seed(seed))[:tokens]
    order[::5] = -1
    return order


def gpu(t, offset):
    """t on the GPU, its data `offset` elements behind an aligned address, its padded strides kept."""
    flat = torch.full((t.untyped_storage().nbytes() // t.element_size() + offset,), float("nan"), dtype=t.dtype, device="cuda")
    whole = flat[offset:].as_strided(t.shape, t.stride())
    whole.copy_(t)
    return whole


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dims,tokens,offset,pad", [(V3, 1, 0, 0), (V3, 19, 0, 8), (LITE, 37, 0, 0), (NOPE, 9, 0, 0), (ODD, 5, 0, 0),
                                                    (ODD, 33, 1, 3), (LITE, 6, 1, 0), (LITE, 7, 0, 1), (WIDE, 3, 0, 0)])
@pytest.mark.parametrize("norm", ["none", "all", "per head"])
def test_queries(mla, interleaved, dtype, dims, tokens, offset, pad, norm):
    q, _, w, _, pos, cs = inputs(tokens, tokens, dims, dtype, norm == "per head", pad)
    w = None if norm == "none" else w
    heads, nope, rope, latent = dims
    nope_out = torch.full((tokens, heads, nope), float("nan"), dtype=dtype, device="cuda")
    q_cat = torch.full((tokens, heads, latent + rope), float("nan"), dtype=dtype, device="cuda")
    dq, dw = gpu(q, offset), None if w is None else w.cuda()
    mla.mla_norm_rope_q(nope_out, q_cat[..., latent:], dq, dw, pos.cuda(), cs.cuda(), eps=EPS, interleaved=interleaved)
    mla.mla_device_error()
    (n, en), (r, er) = ref.queries(q, w, nope, cs[pos], interleaved, EPS)
    ref.check(nope_out, n, en, dtype, "nope")
    ref.check(q_cat[..., latent:], r, er, dtype, "rope")
    assert torch.isnan(q_cat[..., :latent]).all()
    if norm == "none":
        assert torch.equal(nope_out.cpu(), q[..., :nope])
    # in place: the same bits
    n2, r2 = dq[..., :nope], dq[..., nope:]
    mla.mla_norm_rope_q(n2, r2, dq, dw, pos.cuda(), cs.cuda(), eps=EPS, interleaved=interleaved)
    assert torch.equal(n2, nope_out) and torch.equal(r2, q_cat[..., latent:])


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dims,tokens,offset,pad,page,layers", [
    (V3, 1, 0, 0, 64, 1), (V3, 77, 0, 8, 16, 3), (NOPE, 30, 0, 0, 64, 1), (ODD, 41, 1, 3, 5, 2), (LITE, 11, 1, 0, 64, 1),
    (LITE, 12, 0, 1, 1, 1), (WIDE, 9, 0, 0, 8, 1)])
def test_rows(mla, interleaved, dtype, dims, tokens, offset, pad, page, layers):
    _, kv, _, w, pos, cs = inputs(tokens, tokens, dims, dtype, pad=pad)
    latent, rope = dims[3], dims[2]
    blocks = -(-tokens // page) + 2
    whole = torch.full((blocks, layers, page, latent + rope), 7.0, dtype=dtype, device="cuda")
    slots = slots_of(tokens, tokens, blocks * page)
    mla.mla_norm_rope_cache_write(whole[:, layers - 1], gpu(kv, offset), w.cuda(), pos.cuda(), cs.cuda(), slots.cuda(),
                                  eps=EPS, interleaved=interleaved)
    mla.mla_device_error()
    want, err = ref.rows(kv, w, cs[pos], interleaved, EPS)
    real = slots >= 0
    got = whole[:, layers - 1].reshape(blocks * page, -1).cpu()
    ref.check(got[slots[real]], want[real], err[real], dtype, "rows")
    left = torch.ones(blocks * page, dtype=torch.bool)
    left[slots[real]] = False
    assert (got[left] == 7).all() and (layers == 1 or (whole[:, :layers - 1] == 7).all())


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dims,tokens,offset,pad", [(V3, 1, 0, 0), (V3, 70, 0, 8), (NOPE, 30, 0, 0), (ODD, 41, 1, 3),
                                                    (LITE, 11, 1, 0), (WIDE, 9, 0, 0)])
def test_rows_e4m3(mla, interleaved, dtype, dims, tokens, offset, pad):
    _, kv, _, w, pos, cs = inputs(tokens + 1, tokens, dims, dtype, pad=pad)
    latent, rope, page = dims[3], dims[2], 16
    blocks = -(-tokens // page) + 2
    cache = torch.full((blocks, page, latent + rope), 0x55, dtype=torch.uint8, device="cuda")
    slots, scale = slots_of(tokens, tokens, blocks * page), 0.0171
    mla.mla_norm_rope_cache_write_fp8(cache, gpu(kv, offset), w.cuda(), pos.cuda(), cs.cuda(), slots.cuda(),
                                      torch.tensor([scale], device="cuda"), eps=EPS, interleaved=interleaved)
    mla.mla_device_error()
    want, err = ref.rows(kv, w, cs[pos], interleaved, EPS)
    y = want / torch.tensor(scale).double()
    # the quotient is rounded to float32 before it becomes a code
    err = err / scale + (y.abs() + err / scale) * 2.0 ** -24
    real = slots >= 0
    got = cache.view(blocks * page, -1).cpu()
    ref.check_codes(got[slots[real]], y[real], err[real], "codes")
    left = torch.ones(blocks * page, dtype=torch.bool)
    left[slots[real]] = False
    assert (got[left] == 0x55).all()


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,offset,pad,layers", [(1, 0, 0, 1), (130, 0, 8, 3), (9, 1, 0, 1), (10, 0, 1, 2)])
def test_rows_ds_mla(mla, interleaved, dtype, tokens, offset, pad, layers):
    _, kv, _, w, pos, cs = inputs(tokens + 2, tokens, V3, dtype, pad=pad)
    if tokens > 9:
        kv[3, :512] = 0                       # a row of zeros
        kv[4, :512] = 0
        kv[4, 5] = -1                         # one value in a row: three groups of zeros
        kv[6, 128:256] = 2.0 ** -100          # next to nothing beside the rest
    blocks, page = -(-tokens // 16) + 1, 16
    whole = torch.full((blocks, layers, page, 656), 0x55, dtype=torch.uint8, device="cuda")
    slots = slots_of(tokens, tokens, blocks * page)
    mla.mla_norm_rope_cache_write_ds_mla(whole[:, layers - 1], gpu(kv, offset), w.cuda(), pos.cuda(), cs.cuda(), slots.cuda(),
                                         eps=EPS, interleaved=interleaved)
    mla.mla_device_error()
    want, err = ref.rows(kv, w, cs[pos], interleaved, EPS)
    real = slots >= 0
    got = whole[:, layers - 1].reshape(blocks * page, 656).cpu()
    e, want, err = got[slots[real]], want[real], err[real]
    c, ec = want[:, :512].view(-1, 4, 128), err[:, :512].view(-1, 4, 128)
    scale = (c.abs().amax(-1) / 448).clamp_min(2.0 ** -126)
    es = ec.amax(-1) / 448 + scale * 2.0 ** -23
    scales = e[:, 512:528].contiguous().view(F32).double()
    assert ((scales - scale).abs() <= es).all(), "scales"
    # codes by the scale as it is stored
    y, ey = (c / scales[..., None]).flatten(1), (ec / scales[..., None]).flatten(1)
    ref.check_codes(e[:, :512], y, ey + y.abs() * 2.0 ** -50, "codes")
    ref.check(e[:, 528:].contiguous().view(BF16), want[:, 512:], err[:, 512:], BF16, "rope")
    left = torch.ones(blocks * page, dtype=torch.bool)
    left[slots[real]] = False
    assert (got[left] == 0x55).all() and (layers == 1 or (whole[:, :layers - 1] == 0x55).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dims,tokens,offset", [(V3, 1, 0), (V3, 65, 0), (NOPE, 5, 0), (ODD, 12, 0), (LITE, 4, 1)])
@pytest.mark.parametrize("norm", [True, False])
def test_both_in_one_launch(mla, dtype, dims, tokens, offset, norm):
    # the two calls' results, bit for bit; without a norm the nope columns stay where they are
    q, kv, qw, kw, pos, cs = inputs(tokens + 3, tokens, dims, dtype)
    heads, nope, rope, latent = dims
    q, kv, qw, kw, pos, cs = gpu(q, offset), gpu(kv, offset), qw.cuda() if norm else None, kw.cuda(), pos.cuda(), cs.cuda()
    blocks, page = -(-tokens // 16) + 1, 16
    slots = slots_of(tokens, tokens, blocks * page).cuda()
    got = []
    for together in (False, True):
        nope_out = torch.zeros(tokens, heads, nope, dtype=dtype, device="cuda") if norm else q[..., :nope]
        q_cat = torch.zeros(tokens, heads, latent + rope, dtype=dtype, device="cuda")
        cache = torch.zeros(blocks, page, latent + rope, dtype=dtype, device="cuda")
        if together:
            mla.mla_norm_rope_q_cache_write(nope_out, q_cat[..., latent:], q, qw, cache, kv, kw, pos, cs, slots, eps=EPS)
        else:
            mla.mla_norm_rope_q(nope_out, q_cat[..., latent:], q, qw, pos, cs, eps=EPS)
            mla.mla_norm_rope_cache_write(cache, kv, kw, pos, cs, slots, eps=EPS)
        got.append((nope_out, q_cat, cache))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_positions_outside_the_table(mla):
    q, kv, qw, kw, pos, cs = inputs(4, 6, LITE, BF16)
    pos[1], pos[4] = POSITIONS, -1
    nope = torch.full((6, 16, 128), 7.0, dtype=BF16, device="cuda")
    pe, cache = nope[..., :64].clone(), torch.full((1, 8, 576), 7.0, dtype=BF16, device="cuda")
    mla.mla_norm_rope_q_cache_write(nope, pe, q.cuda(), qw.cuda(), cache, kv.cuda(), kw.cuda(), pos.cuda(), cs.cuda(),
                                    torch.tensor([0, 1, 2, 8, 4, 5], device="cuda"), eps=EPS)
    with pytest.raises(mla.MlaError) as e:
        mla.mla_device_error()
    assert e.value.status == mla.MLA_ERR_DEVICE_DATA
    good = [0, 2, 3, 5]
    (n, en), (r, er) = ref.queries(q[good], qw, 128, cs[pos[good]], True, EPS)
    ref.check(nope[good], n, en, BF16, "nope")
    ref.check(pe[good], r, er, BF16, "rope")
    assert (nope[[1, 4]] == 7).all() and (pe[[1, 4]] == 7).all()
    want, err = ref.rows(kv, kw, cs[pos.clamp(0, POSITIONS - 1)], True, EPS)
    ref.check(cache[0, [0, 2, 5]], want[[0, 2, 5]], err[[0, 2, 5]], BF16, "rows")
    assert (cache[0, [1, 3, 4, 6, 7]] == 7).all()       # 1, 4: bad positions, 3: its slot lies outside
    mla.mla_device_error()


def test_no_tokens(mla):
    z = torch.zeros
    cs, none = ref.table(4, 64).cuda(), z(0, dtype=torch.int64, device="cuda")
    q, kv = z(0, 16, 192, device="cuda"), z(0, 576, device="cuda")
    mla.mla_norm_rope_q_cache_write(q[..., :128], q[..., 128:], q, None, z(1, 8, 576, device="cuda"), kv, z(512, device="cuda"),
                                    none, cs, none)
    mla.mla_device_error()


def test_captured_and_on_another_stream(mla):
    q, kv, qw, kw, pos, cs = (t.cuda() for t in inputs(5, 33, V3, BF16))
    slots = torch.arange(33, device="cuda")
    outs = [[torch.zeros(33, 128, 128, dtype=BF16, device="cuda"), torch.zeros(33, 128, 64, dtype=BF16, device="cuda"),
             torch.zeros(1, 64, 576, dtype=BF16, device="cuda")] for _ in range(3)]

    def call(o, **more):
        mla.mla_norm_rope_q_cache_write(o[0], o[1], q, qw, o[2], kv, kw, pos, cs, slots, **more)

    call(outs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(outs[1], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs[2])
    graph.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        for a, b in zip(outs[0], o):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dims", [(16, 0, 64, 512), (16, 64, 0, 512), (2, 0, 2, 3), (4, 64, 512, 64), (4, 8, 24, 40)])
def test_heads_of_rope_alone_and_of_none(mla, dtype, dims):
    heads, nope, rope, latent = dims
    for norm in (False, True):
        for interleaved in (False, True):
            q, kv, w, kw, pos, cs = inputs(7, 9, dims, dtype)
            w = w if norm else None
            n, r = torch.zeros(9, heads, nope, dtype=dtype, device="cuda"), torch.zeros(9, heads, rope, dtype=dtype, device="cuda")
            cache, slots = torch.zeros(2, 8, latent + rope, dtype=dtype, device="cuda"), torch.arange(9)
            mla.mla_norm_rope_q_cache_write(n, r, q.cuda(), None if w is None else w.cuda(), cache, kv.cuda(), kw.cuda(), pos.cuda(),
                                            cs.cuda(), slots.cuda(), eps=EPS, interleaved=interleaved)
            mla.mla_device_error()
            (wn, en), (wr, er) = ref.queries(q, w, nope, cs[pos], interleaved, EPS)
            ref.check(n, wn, en, dtype, "nope")
            ref.check(r, wr, er, dtype, "rope")
            want, err = ref.rows(kv, kw, cs[pos], interleaved, EPS)
            ref.check(cache.view(16, -1)[:9], want, err, dtype, "rows")


@pytest.mark.parametrize("form", ["", "_fp8", "_ds_mla"])
@pytest.mark.parametrize("offset,pad", [(0, 4), (1, 0), (0, 3), (2, 2)])
def test_tables_of_other_strides(mla, form, offset, pad):
    # a table cut from a wider one, its rows on any 4-byte boundary: the results do not change
    _, kv, _, w, pos, cs = inputs(9, 20, LITE, BF16)
    wide = torch.full((POSITIONS * (64 + pad) + offset,), float("nan"), device="cuda")
    other = wide[offset:].view(POSITIONS, 64 + pad)[:, :64]
    other.copy_(cs)
    got = []
    for table in (cs.cuda(), other):
        cache = torch.zeros(3, 8, 656 if form == "_ds_mla" else 576, dtype=torch.uint8 if form else BF16, device="cuda")
        more = [torch.tensor([0.01], device="cuda")] if form == "_fp8" else []
        for interleaved in (False, True):
            getattr(mla, "mla_norm_rope_cache_write" + form)(cache, kv.cuda(), w.cuda(), pos.cuda(), table, torch.arange(20).cuda(), *more,
                                                             eps=EPS, interleaved=interleaved)
            got.append(cache.clone())
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [0.0171, 1.0, 2.0 ** -70, 3e25, 1e-30, 2.0 ** 60, -0.5])
def test_e4m3_quotients_are_the_cache_writes(mla, dtype, scale):
    # at position 0 the rotation leaves every value as it is, so the rope columns' codes are those that
    # mla_cache_write_fp8 gives the same values: infinities, NaN, zeros of both signs and values near the middle of codes too
    g = torch.Generator().manual_seed(5)
    rows, rope, latent = 300, 256, 16
    x = torch.randn(rows, rope, generator=g) * torch.exp(6 * torch.randn(rows, 1, generator=g)) * abs(scale)
    x[:20] = (torch.arange(20 * rope).view(20, rope) % 2048 - 1024) / 8 * scale          # codes, middles of codes
    x[20:24] = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 3e38, -3e38, 1e-45]).repeat(4, rope // 8)
    x = x.to(dtype).cuda()
    kv = torch.cat([torch.ones(rows, latent, dtype=dtype, device="cuda"), x], 1)
    cs = torch.cat([torch.ones(1, rope // 2), torch.zeros(1, rope // 2)], 1).cuda()
    slots, zero = torch.arange(rows, device="cuda"), torch.zeros(rows, dtype=torch.int64, device="cuda")
    s = torch.tensor([scale], device="cuda")
    a, b = (torch.zeros(5, 64, latent + rope, dtype=torch.uint8, device="cuda") for _ in range(2))
    finite = torch.isfinite(x).all(1).cpu()
    for interleaved in (False, True):
        mla.mla_norm_rope_cache_write_fp8(a, kv, torch.ones(latent, dtype=dtype, device="cuda"), zero, cs, slots, s, interleaved=interleaved)
        mla.mla_cache_write_fp8(b, kv[:, :latent], x, slots, s)
        mla.mla_device_error()
        u, v = (t.view(320, -1)[:rows, latent:].cpu()[finite] for t in (a, b))
        # x c - y 0 and y c + x 0 are x and y, but for the sign of a zero
        zero_sign = (u ^ v) == 0x80
        assert ((u == v) | (zero_sign & (u & 0x7F == 0))).all()


def test_many_rows_one_behind_the_other(mla):
    # more rows than warps run at once, so that a warp takes several
    for form, dtype in (("", BF16), ("", F32), ("_fp8", BF16), ("_ds_mla", F32), ("_ds_mla", BF16)):
        _, kv, _, w, pos, cs = inputs(17, 9001, LITE, dtype)
        slots = slots_of(3, 9001, 9100)
        cache = torch.zeros(91, 100, 656 if form == "_ds_mla" else 576, dtype=torch.uint8 if form else dtype, device="cuda")
        one = torch.zeros_like(cache)
        more = [torch.tensor([0.01], device="cuda")] if form == "_fp8" else []
        call = getattr(mla, "mla_norm_rope_cache_write" + form)
        kv, w, pos, cs, slots = kv.cuda(), w.cuda(), pos.cuda(), cs.cuda(), slots.cuda()
        call(cache, kv, w, pos, cs, slots, *more, eps=EPS)
        for i in range(0, 9001, 1500):                # few enough for a warp each
            call(one, kv[i:i + 1500], w, pos[i:i + 1500], cs, slots[i:i + 1500], *more, eps=EPS)
        assert torch.equal(cache, one)


@pytest.mark.parametrize("form", ["", "_fp8"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("rope,latent,pad", [(64, 512, 0), (64, 512, 4), (0, 640, 0), (128, 512, 0), (256, 16, 0), (64, 264, 0), (16, 8, 0), (64, 640, 0)])
def test_many_rows_side_by_side(mla, form, interleaved, rope, latent, pad):
    # two rows a warp: rows that are padding, lie outside the cache or have no angles beside rows that are written,
    # entries of 4-byte alignment (pad), and the same bits as in calls of few rows
    T = 7001
    _, kv, _, w, pos, cs = inputs(23, T, (1, 8, rope, latent), BF16)
    slots = slots_of(4, T, 7200)
    slots[7::10] = 7200 + 5
    if rope:
        pos[3::11], pos[9::17] = POSITIONS, -1
    kind = torch.uint8 if form else BF16
    step = pad if form else 2 * pad
    whole, other = (torch.full((72, 100, latent + rope + step), 7, dtype=kind, device="cuda") for _ in range(2))
    cache, one = whole[..., :latent + rope], other[..., :latent + rope]
    more = [torch.tensor([0.01], device="cuda")] if form else []
    call = getattr(mla, "mla_norm_rope_cache_write" + form)
    kv, w, pos, cs, slots = kv.cuda(), w.cuda(), pos.cuda(), cs.cuda(), slots.cuda()
    call(cache, kv, w, pos, cs, slots, *more, eps=EPS, interleaved=interleaved)
    with pytest.raises(mla.MlaError):
        mla.mla_device_error()
    for i in range(0, T, 1000):
        call(one, kv[i:i + 1000], w, pos[i:i + 1000], cs, slots[i:i + 1000], *more, eps=EPS, interleaved=interleaved)
    with pytest.raises(mla.MlaError):
        mla.mla_device_error()
    assert torch.equal(whole, other)
    fine = (slots >= 0) & (slots < 7200) & (((pos >= 0) & (pos < POSITIONS)) | (rope == 0))
    written = torch.zeros(7200, dtype=torch.bool, device="cuda")
    written[slots[fine]] = True
    flat = whole.view(7200, -1)
    assert (flat[~written] == 7).all() and (flat[:, latent + rope:] == 7).all()
    assert (flat[written] != 7).any(1).all()


BIG = [1e20, float("inf"), float("-inf"), float("nan")]


def by_nothing(x):
    """A row's values by the factor 0 of a sum of squares beyond float32 (of NaN: NaN)."""
    x = x.double().cpu()
    return x * float("nan") if torch.isnan(x).any() else x * 0.0


def same(a, b):
    return torch.equal(torch.nan_to_num(a.double().cpu(), nan=7e77), torch.nan_to_num(b.double().cpu(), nan=7e77))


@pytest.mark.parametrize("big", BIG)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dims,offset", [(LITE, 0), (NOPE, 0), ((4, 448, 64, 512), 0), ((2, 960, 64, 512), 0), (ODD, 0), (LITE, 1)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_heads_whose_squares_overflow(mla, big, dtype, dims, offset, interleaved):
    # the factor is 0: finite columns become 0, an infinite one NaN; the heads beside it do not change
    heads, nope, rope, latent = dims
    q, _, w, _, pos, cs = inputs(11, 5, dims, dtype)
    loud = q.clone()
    loud[1, 1, 3], loud[3, 0, nope + rope - 1] = big, big
    got = []
    for x in (q, loud):
        n, r = (torch.full((5, heads, c), 7.0, dtype=dtype, device="cuda") for c in (nope, rope))
        mla.mla_norm_rope_q(n, r, gpu(x, offset), w.cuda(), pos.cuda(), cs.cuda(), eps=EPS, interleaved=interleaved)
        got.append(torch.cat([n, r], 2).cpu())
    mla.mla_device_error()
    for t, h in ((1, 1), (3, 0)):
        x = by_nothing(loud[t, h])
        pe = ref.rotated(x[None, nope:], cs[pos[t]][None], interleaved, 0.0)[0][0]
        assert same(got[1][t, h], torch.cat([x[:nope], pe]))
        got[1][t, h] = got[0][t, h]
    assert torch.equal(*got)


@pytest.mark.parametrize("big", BIG)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("form", ["", "_fp8", "_ds_mla"])
@pytest.mark.parametrize("tokens,offset", [(6, 0), (6, 1), (7001, 0)])
def test_rows_whose_squares_overflow(mla, big, dtype, form, tokens, offset):
    _, kv, _, w, pos, cs = inputs(12, tokens, LITE, dtype)
    loud = kv.clone()
    rows = (2, 5)
    loud[rows[0], 7], loud[rows[1], 511] = big, big
    more = [torch.tensor([0.01], device="cuda")] if form == "_fp8" else []
    got = []
    for x in (kv, loud):
        cache = torch.zeros(1, tokens, 656 if form == "_ds_mla" else 576, dtype=torch.uint8 if form else dtype, device="cuda")
        getattr(mla, "mla_norm_rope_cache_write" + form)(cache, gpu(x, offset), w.cuda(), pos.cuda(), cs.cuda(),
                                                         torch.arange(tokens, device="cuda"), *more, eps=EPS)
        got.append(cache[0].cpu())
    mla.mla_device_error()
    for t in rows:
        latents = got[1][t, :512]
        if form:
            latents = latents.view(ref.E4M3)
        assert same(latents.float(), by_nothing(loud[t, :512]))
        if form == "_ds_mla":       # groups of zeros (a NaN does not count)
            assert (got[1][t, 512:528].view(F32) == 2.0 ** -126).all()
            got[1][t, :528] = got[0][t, :528]
        got[1][t, :512] = got[0][t, :512]
    assert torch.equal(*got)


# scales of either side of where the quotients' short form ends, and ordinary ones
QUOTIENTS = [0.0171, 1.0, -0.5, 2.0 ** -60, 1.0001 * 2.0 ** -60, 0.9999 * 2.0 ** 60, 2.0 ** 60, -1.37 * 2.0 ** 59, 1.7 * 2.0 ** -59]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", QUOTIENTS)
@pytest.mark.parametrize("rows", [300, 6000])
@pytest.mark.parametrize("rope", [64, 128])
def test_e4m3_quotients_value_by_value(mla, dtype, scale, rows, rope):
    # ropes that the kernel of whole words takes, in rows of a warp and of half a warp; at position 0 the rotation leaves
    # a value as it is where its partner is finite: all of those have mla_cache_write_fp8's codes
    g = torch.Generator().manual_seed(6)
    latent = 16
    s = torch.tensor([scale])
    x = torch.randn(rows, rope, generator=g) * torch.exp(6 * torch.randn(rows, 1, generator=g)) * abs(scale)
    x[:20] = (torch.arange(20 * rope).view(20, rope) % 2048 - 1024) / 8 * s              # codes, middles of codes
    x[20:60] = torch.nextafter(x[:20].repeat(2, 1), torch.tensor([1e38, -1e38])[:, None, None].expand(2, 20, rope).reshape(40, rope))
    x[60:64] = torch.tensor([0.0, -0.0, 3.3e38, -3.3e38, 1e-45, -1e-45, 2.0 ** -126, 2.0 ** -120]).repeat(4, rope // 8)
    odd = torch.tensor([float("inf"), -float("inf"), float("nan")])
    x[64:128:2, 5] = odd.repeat(11)[:32]
    x[65:128:2, rope // 2 + 8] = odd.repeat(11)[:32]
    x = x.to(dtype)
    kv = torch.cat([torch.ones(rows, latent, dtype=dtype), x], 1).cuda()
    cs = torch.cat([torch.ones(1, rope // 2), torch.zeros(1, rope // 2)], 1).cuda()
    slots, zero = torch.arange(rows, device="cuda"), torch.zeros(rows, dtype=torch.int64, device="cuda")
    a, b = (torch.zeros(1, rows, latent + rope, dtype=torch.uint8, device="cuda") for _ in range(2))
    for interleaved in (False, True):
        mla.mla_norm_rope_cache_write_fp8(a, kv, torch.ones(latent, dtype=dtype, device="cuda"), zero, cs, slots, s.cuda(),
                                          interleaved=interleaved)
        mla.mla_cache_write_fp8(b, kv[:, :latent], kv[:, latent:], slots, s.cuda())
        mla.mla_device_error()
        u, v = (t[0, :, latent:].cpu() for t in (a, b))
        partner = torch.arange(rope) ^ 1 if interleaved else (torch.arange(rope) + rope // 2) % rope
        fine = torch.isfinite(x)[:, partner]
        assert fine.sum() == rows * rope - 64 and (~torch.isfinite(x) & fine).sum() == 64
        # x c - y 0 and y c + x 0 are x and y, but for the sign of a zero; a NaN has either sign
        low = u & 0x7F
        assert ((u == v) | (low == (v & 0x7F)) & ((low == 0) | (low == 0x7F)) | ~fine).all()

"""Windowed decode and prefill (sliding window and sinks) against a plain 64-bit implementation."""
import pytest
import torch

import window_ref as wr

pytestmark = pytest.mark.gpu

GEOMETRIES = {
    "v3": dict(dtype="bf16", heads=128, latent=512, rope=64),
    "nope64": dict(dtype="bf16", heads=64, latent=512, rope=0),
    "h64": dict(dtype="bf16", heads=64, latent=512, rope=64),
    "h16": dict(dtype="bf16", heads=16, latent=512, rope=64),
    "h20": dict(dtype="bf16", heads=20, latent=512, rope=64),
    "h96": dict(dtype="bf16", heads=96, latent=512, rope=0),
    "h1": dict(dtype="bf16", heads=1, latent=512, rope=64),
    "h130": dict(dtype="bf16", heads=130, latent=512, rope=64),
    "lite_f32": dict(dtype="f32", heads=16, latent=512, rope=64),
    "small_bf16": dict(dtype="bf16", heads=5, latent=40, rope=6),
    "small_f32": dict(dtype="f32", heads=3, latent=24, rope=0),
}


def outputs(c):
    tokens, heads = c.qs.shape[:2]
    return (torch.full((tokens, heads, c.latent), 7.0, dtype=c.dt, device="cuda"),
            torch.full((tokens, heads), 7.0, dtype=torch.float32, device="cuda"))


def decode(mla, c, lse=True, **more):
    cache, q, table, kv, _ = c.dev()
    o, l = outputs(c)
    mla.mla_decode_window(o, q, cache, table, kv, c.latent, c.rope, c.scale, c.window, sinks=c.sinks,
                          lse_out=l if lse else None, **more)
    mla.mla_device_error()
    return o, l if lse else None


def prefill(mla, c, lse=True, **more):
    cache, q, table, kv, cu = c.dev()
    o, l = outputs(c)
    mla.mla_prefill_window(o, q, cache, table, cu, kv, c.latent, c.rope, c.scale, c.window, sinks=c.sinks,
                           lse_out=l if lse else None, **more)
    mla.mla_device_error()
    return o, l if lse else None


def decode_case(geometry, kv, window, sinks, page=64, seed=1, **more):
    return wr.Case(seed=seed, **GEOMETRIES[geometry], page=page, kv=kv, q=[1] * len(kv), window=window, sinks=sinks,
                   **more)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (63, 0), (64, 4), (65, 64), (128, 70), (500, 1),
                                          (2 ** 31 - 1, 0), (100, 2 ** 31 - 1), (200, 129)])
def test_decode_windows_and_sinks(mla, window, sinks):
    c = decode_case("v3", [0, 1, 2, 63, 64, 65, 127, 128, 129, 300, 641], window, sinks)
    wr.check(*decode(mla, c), c.want(), len(c.kv))


@pytest.mark.parametrize("geometry", GEOMETRIES)
@pytest.mark.parametrize("page", [64, 16, 128, 8, 1, 100])
def test_decode_geometries_and_pages(mla, geometry, page):
    c = decode_case(geometry, [1, 77, 0, 513], 150, 5, page=page, seed=3)
    wr.check(*decode(mla, c), c.want(), 4)


@pytest.mark.parametrize("splits", [0, 1, 2, 7, 300])
def test_decode_splits(mla, splits):
    c = decode_case("v3", [2000, 3, 0, 900, 1500], 1200, 70, seed=4)
    wr.check(*decode(mla, c, num_splits=splits), c.want(), 5)


def test_decode_without_lse_and_many_sequences(mla):
    c = decode_case("h16", [(37 * i) % 200 for i in range(700)], 50, 3, seed=5)
    wr.check(*decode(mla, c, lse=False), c.want(), 700)


@pytest.mark.parametrize("geometry", ["v3", "lite_f32"])
def test_decode_wide_logits(mla, geometry):
    # products of a thousand: every row's weight is nearly all on one key
    c = decode_case(geometry, [700, 64], 400, 4, seed=6, spread=6.0, scale=0.25)
    wr.check(*decode(mla, c), c.want(), 2)


def test_decode_strided_views(mla):
    # rows of q and of the cache inside wider rows, o inside a wider buffer
    c = decode_case("v3", [300, 65], 128, 4, seed=7, q_pad=64, cache_pad=32)
    cache, q, table, kv, _ = c.dev()
    big = torch.full((2, 2, 128, 512), 7.0, dtype=c.dt, device="cuda")
    wide = torch.full((2, 9), -5, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    mla.mla_decode_window(big[:, 1], q, cache, wide[:, :table.shape[1]], kv, 512, 64, c.scale, 128, sinks=4)
    mla.mla_device_error()
    wr.check(big[:, 1], None, c.want(), 2)
    assert (big[:, 0] == 7).all()


def test_decode_equals_mla_decode_where_the_window_holds_all(mla):
    c = decode_case("v3", [500, 64, 1], 500, 0, seed=8)
    cache, q, table, kv, _ = c.dev()
    o, l = decode(mla, c)
    full, full_l = outputs(c)
    mla.mla_decode(full, q, cache, table, kv, 512, 64, c.scale, lse_out=full_l)
    mla.mla_device_error()
    want = c.want()
    wr.check(o, l, want, 3)
    assert (full_l - l).abs().max() < 1.2e-2


def prefill_case(geometry, kv, q, window, sinks, page=64, seed=11, **more):
    return wr.Case(seed=seed, **GEOMETRIES[geometry], page=page, kv=kv, q=q, window=window, sinks=sinks, **more)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (64, 4), (65, 64), (130, 70), (2 ** 31 - 1, 0),
                                          (50, 2 ** 31 - 1)])
@pytest.mark.parametrize("geometry", ["v3", "nope64", "h20"])
def test_prefill_windows_and_sinks(mla, geometry, window, sinks):
    c = prefill_case(geometry, [1, 40, 300, 0, 129], [1, 40, 33, 0, 129], window, sinks)
    wr.check(*prefill(mla, c), c.want(), sum(c.q_lens))


@pytest.mark.parametrize("geometry", GEOMETRIES)
@pytest.mark.parametrize("page", [64, 16, 128, 1, 100])
def test_prefill_geometries_and_pages(mla, geometry, page):
    c = prefill_case(geometry, [70, 200], [21, 9], 60, 5, page=page)
    wr.check(*prefill(mla, c), c.want(), 30)


@pytest.mark.parametrize("geometry", ["v3", "h16", "lite_f32"])
def test_prefill_rows_of_no_sequence_and_negative_positions(mla, geometry):
    # five rows behind the last sequence; a chunk longer than its cache
    c = prefill_case(geometry, [3, 20, 1], [8, 0, 4], 2, 1, tail=5)
    o, l = prefill(mla, c)
    wr.check(o, l, c.want(), 12)
    assert (o[12:] == 7).all() and (l[12:] == 7).all()
    assert (o[:5] == 0).all() and torch.isneginf(l[:5]).all()


def test_prefill_few_tokens_over_a_long_axis(mla):
    c = prefill_case("v3", [5001], [3], 4500, 16, seed=13)
    wr.check(*prefill(mla, c), c.want(), 3)


def test_prefill_many_short_sequences(mla):
    n = 400
    c = prefill_case("h16", [5 + i % 90 for i in range(n)], [i % 6 for i in range(n)], 40, 2, seed=14)
    wr.check(*prefill(mla, c), c.want(), sum(c.q_lens))


@pytest.mark.parametrize("geometry", ["v3", "nope64"])
def test_prefill_many_row_tiles(mla, geometry):
    # more row tiles than the split schedule takes (whole tiles are dealt out then)
    c = prefill_case(geometry, [1100, 30], [1100, 17], 3, 1, seed=15) if geometry == "v3" else \
        prefill_case(geometry, [2300, 30], [2300, 17], 3, 1, seed=15)
    wr.check(*prefill(mla, c), c.want(), sum(c.q_lens))


def test_prefill_is_the_decode_of_each_token(mla):
    c = prefill_case("v3", [200], [6], 90, 4, seed=16)
    cache, q, table, kv, cu = c.dev()
    o, l = prefill(mla, c)
    want = c.want()
    lens = torch.arange(195, 201, dtype=torch.int32, device="cuda")
    od, ld = outputs(c)
    mla.mla_decode_window(od, q, cache, table.expand(6, -1).contiguous(), lens, 512, 64, c.scale, 90, sinks=4,
                          lse_out=ld)
    mla.mla_device_error()
    wr.check(o, l, want, 6)
    wr.check(od, ld, want, 6)


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_bad_table_entries_and_lengths_are_reported(mla, which):
    c = prefill_case("v3", [100, 130], [1, 1], 80, 0, seed=17)
    want = c.want()
    call = decode if which == "decode" else prefill
    # the second sequence's attended page 1 names a block that does not exist
    c.table_np = c.table_np.copy()
    c.table_np[1, 1] = 10 ** 6
    cache, q, table, kv, cu = c.dev()
    o, l = outputs(c)
    if which == "decode":
        mla.mla_decode_window(o, q, cache, table, kv, 512, 64, c.scale, 80, lse_out=l)
    else:
        mla.mla_prefill_window(o, q, cache, table, cu, kv, 512, 64, c.scale, 80, lse_out=l)
    with pytest.raises(mla.MlaError) as e:
        mla.mla_device_error()
    assert e.value.status == mla.MLA_ERR_DEVICE_DATA
    wr.check(o, l, want, 1)     # the first sequence is right
    assert torch.isfinite(o).all()


def test_a_length_beyond_the_table_is_reported(mla):
    c = decode_case("v3", [60, 60], 2 ** 31 - 1, 0, seed=18)
    cache, q, table, kv, _ = c.dev()
    o, l = outputs(c)
    mla.mla_decode_window(o, q, cache, table[:, :1].contiguous(), torch.tensor([60, 99], dtype=torch.int32, device="cuda"),
                          512, 64, c.scale, 60, lse_out=l)
    with pytest.raises(mla.MlaError):
        mla.mla_device_error()
    wr.check(o, l, c.want(), 1)


def test_captured_and_replayed_with_new_inputs(mla):
    a = decode_case("v3", [900, 333, 64], 256, 4, seed=19)
    b = decode_case("v3", [100, 700, 901], 256, 4, seed=20)
    cache, q, table, kv, _ = a.dev()
    o, l = outputs(a)
    ws = torch.empty(mla.mla_decode_window_workspace_size(3, 128, 512), dtype=torch.uint8, device="cuda")

    def call():
        mla.mla_decode_window(o, q, cache, table, kv, 512, 64, a.scale, 256, sinks=4, lse_out=l, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    mla.mla_device_error()
    wr.check(o, l, a.want(), 3)
    cache_b, q_b, table_b, kv_b, _ = b.dev()
    if cache_b.shape == cache.shape and table_b.shape == table.shape:
        cache.copy_(cache_b)
        table.copy_(table_b)
    else:   # the same buffers hold the other case's pages
        pytest.fail("the two cases need pages of one shape")
    q.copy_(q_b)
    kv.copy_(kv_b)
    graph.replay()
    mla.mla_device_error()
    wr.check(o, l, b.want(), 3)


def test_two_streams_at_once(mla):
    cases = [decode_case("v3", [900, 333, 64], 256, 4, seed=21), prefill_case("v3", [300, 90], [20, 9], 77, 3, seed=22)]
    state = []
    for c in cases:
        state.append((c, c.dev(), outputs(c)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for (c, (cache, q, table, kv, cu), (o, l)), s, which in zip(state, streams, ["decode", "prefill"]):
            if which == "decode":
                mla.mla_decode_window(o, q, cache, table, kv, 512, 64, c.scale, c.window, sinks=c.sinks, lse_out=l,
                                      stream=s)
            else:
                mla.mla_prefill_window(o, q, cache, table, cu, kv, 512, 64, c.scale, c.window, sinks=c.sinks,
                                       lse_out=l, stream=s)
    torch.cuda.synchronize()
    mla.mla_device_error()
    for c, _, (o, l) in state:
        wr.check(o, l, c.want(), sum(c.q_lens))


def test_runs_repeat_bit_for_bit(mla):
    c = decode_case("v3", [3000, 700, 1999], 2500, 4, seed=23)
    first = decode(mla, c)
    for _ in range(3):
        again = decode(mla, c)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_offsets_beyond_32_bits(mla):
    # a block stride of 2^31 + 64 elements: the third block lies 8 GB into the buffer
    c = decode_case("v3", [150], 120, 4, seed=24)
    cache, q, _, kv, _ = c.dev()
    stride = 2 ** 31 + 64
    buffer = torch.empty(2 * stride + 64 * 576, dtype=torch.bfloat16, device="cuda")
    far = buffer.as_strided((3, 64, 576), (stride, 576, 1))
    for i in range(3):
        far[i].copy_(cache[c.table_np[0, i]])
    table = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    o, l = outputs(c)
    mla.mla_decode_window(o, q, far, table, kv, 512, 64, c.scale, 120, sinks=4, lse_out=l)
    mla.mla_device_error()
    wr.check(o, l, c.want(), 1)


@pytest.mark.parametrize("tokens,bounds", [(12, [0, 5, 3, 12]), (12, [0, 12, 0, 12]), (12, [-1, 4, 8, 12]),
                                           (12, [0, 4, 8, 13]), (12, [0, 2 ** 31 - 1, 4, 12]),
                                           (1100, [0, 1100, 0, 1100]), (1100, [0, 400, 300, 1101])])
@pytest.mark.parametrize("geometry", ["v3", "lite_f32"])
def test_bounds_that_decrease_or_leave_the_tokens_are_reported(mla, geometry, tokens, bounds):
    c = prefill_case(geometry, [70, 70, 70], [tokens, 0, 0], 9, 0, seed=26)
    cache, q, table, kv, _ = c.dev()
    o, l = outputs(c)
    cache = torch.zeros_like(cache)
    table = torch.zeros_like(table)
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    mla.mla_prefill_window(o, q, cache, table, cu, kv, 512, 64, c.scale, 9, lse_out=l)
    with pytest.raises(mla.MlaError) as e:
        mla.mla_device_error()
    assert e.value.status == mla.MLA_ERR_DEVICE_DATA
    assert (o == 7).all() and (l == 7).all()
    # and the next call is right
    c = prefill_case(geometry, [70, 33], [3, 2], 9, 0, seed=27)
    wr.check(*prefill(mla, c), c.want(), 5)


@pytest.mark.parametrize("geometry", ["h16", "lite_f32"])
def test_decode_of_more_sequences_than_a_block_has_threads(mla, geometry):
    c = decode_case(geometry, [(53 * i) % 90 for i in range(1100)], 40, 2, seed=28)
    wr.check(*decode(mla, c), c.want(), 1100)


@pytest.mark.parametrize("page", [32, 24, 192, 320])
@pytest.mark.parametrize("geometry", ["v3", "h64"])
def test_more_page_sizes(mla, geometry, page):
    c = prefill_case(geometry, [420, 31], [4, 3], 170, 33, page=page, seed=29)
    wr.check(*prefill(mla, c), c.want(), 7)


def test_output_rows_on_16_byte_boundaries(mla):
    c = prefill_case("h64", [300, 40], [5, 4], 100, 4, seed=30)
    cache, q, table, kv, cu = c.dev()
    wide = torch.full((9, 64, 536), 7.0, dtype=c.dt, device="cuda")
    o = wide[..., 8:520]
    assert o.data_ptr() % 32 == 16
    mla.mla_prefill_window(o, q, cache, table, cu, kv, 512, 64, c.scale, 100, sinks=4)
    mla.mla_device_error()
    wr.check(o, None, c.want(), 9)
    assert (wide[..., :8] == 7).all() and (wide[..., 520:] == 7).all()


@pytest.mark.parametrize("geometry", ["v3", "lite_f32"])
@pytest.mark.parametrize("scale", [0.0, -0.05])
def test_scales_that_are_not_positive(mla, geometry, scale):
    c = decode_case(geometry, [100, 0, 300], 120, 4, seed=31, scale=abs(scale))
    want = c.want()
    # the queries negated and the scale too: the same scores
    if scale < 0:
        c.qs, c.scale = -c.qs, scale
    wr.check(*decode(mla, c), want, 3)


def test_inputs_of_one_row_or_head_repeated(mla):
    # strides of zero: every head, and every sequence, has the same query
    c = decode_case("v3", [200, 90], 120, 4, seed=32)
    c.qs = c.qs[:1, :1].expand(2, 128, -1)
    cache, _, table, kv, _ = c.dev()
    q = c.qs[:1, :1].contiguous().cuda().expand(2, 128, -1)
    assert q.stride() == (0, 0, 1)
    o, l = outputs(c)
    mla.mla_decode_window(o, q, cache, table, kv, 512, 64, c.scale, 120, sinks=4, lse_out=l)
    mla.mla_device_error()
    wr.check(o, l, c.want(), 2)


@pytest.mark.parametrize("geometry", ["v3", "h64", "lite_f32"])
def test_a_nan_of_one_query_stays_in_its_row(mla, geometry):
    c = prefill_case(geometry, [90, 700], [4, 1], 640, 4, seed=33)
    want = c.want()
    c.qs[1, 3, 7] = float("nan")
    c.qs[4, 5, 9] = float("nan")     # a row that is cut over units and merged
    o, l = prefill(mla, c)
    for t, h in ((1, 3), (4, 5)):
        assert o[t, h].isnan().all() and l[t, h].isnan()
        o[t, h] = torch.from_numpy(want[0][t, h]).to(o)
        l[t, h] = float(want[1][t, h])
    # rounding `want` itself is within its bound
    wr.check(o, l, want, 5)


def test_more_splits_than_there_is_work(mla):
    c = decode_case("lite_f32", [2000, 3, 0], 2000, 0, seed=34)
    wr.check(*decode(mla, c, num_splits=2 ** 31 - 1), c.want(), 3)
    assert mla.mla_decode_window_workspace_size(3, 16, 512, 2 ** 31 - 1) == \
        mla.mla_decode_window_workspace_size(3, 16, 512, 4096)


def test_two_graphs_share_a_workspace(mla):
    cases = [prefill_case("v3", [700, 64], [9, 5], 500, 4, seed=35), prefill_case("h20", [100, 300], [40, 30], 77, 3, seed=36)]
    need = max(mla.mla_prefill_window_workspace_size(sum(c.q_lens), len(c.kv), c.qs.shape[1], 512) for c in cases)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs = []
    for c in cases:
        cache, q, table, kv, cu = c.dev()
        o, l = outputs(c)

        def call():
            mla.mla_prefill_window(o, q, cache, table, cu, kv, 512, 64, c.scale, c.window, sinks=c.sinks, lse_out=l,
                                   workspace=ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((g, c, o, l, (cache, q, table, kv, cu)))
    for _ in range(3):
        for g, _, o, l, _ in graphs:
            o.zero_()
            l.zero_()
            g.replay()
    mla.mla_device_error()
    for _, c, o, l, _ in graphs:
        wr.check(o, l, c.want(), sum(c.q_lens))


def test_results_are_there_for_the_next_kernel(mla):
    # two sequences a unit (of 76), none cut: the merge has nothing to do, and what follows on the stream waits
    # for the whole call all the same
    c = decode_case("v3", [200] * 152, 200, 0, seed=37)
    cache, q, table, kv, _ = c.dev()
    want, _ = decode(mla, c)
    o, _ = outputs(c)
    wr.check(want, None, c.want(), 152)
    for _ in range(50):
        o.fill_(7.0)
        mla.mla_decode_window(o, q, cache, table, kv, 512, 64, c.scale, 200)
        copy = o.clone()
        assert torch.equal(copy, want)


def test_the_default_stream_by_number(mla):
    c = decode_case("v3", [70, 200], 100, 4, seed=38)
    wr.check(*decode(mla, c, stream=0), c.want(), 2)


@pytest.mark.parametrize("dtype,heads,latent,rope,batch", [("f32", 16, 501, 3, 90), ("f32", 16, 500, 8, 90),
                                                           ("bf16", 3, 30, 5, 2), ("bf16", 7, 129, 0, 4),
                                                           ("f32", 9, 512, 64, 3), ("bf16", 130, 512, 64, 12)])
def test_cut_rows_of_odd_widths(mla, dtype, heads, latent, rope, batch):
    # rows cut over work units and merged: whole rows or parts of them a warp, widths of any remainder
    kv = [150 + (97 * i) % 300 for i in range(batch)]
    c = wr.Case(seed=39, dtype=dtype, heads=heads, latent=latent, rope=rope, page=16, kv=kv, q=[1] * batch, window=400,
                sinks=2)
    wr.check(*decode(mla, c), c.want(), batch)


@pytest.mark.parametrize("kv,window", [([8000], 8000), ([2000] * 24, 2000), ([1500, 20, 1100, 640, 0, 2], 1400)])
@pytest.mark.parametrize("geometry", ["v3", "h16"])
def test_cut_rows_of_few_and_many_pieces(mla, geometry, kv, window):
    if geometry == "v3" and len(kv) > 10:
        kv = kv[:20]
    c = decode_case(geometry, kv, window, 4, seed=40)
    wr.check(*decode(mla, c), c.want(), len(kv))


@pytest.mark.parametrize("splits", [1, 2, 3, 300])
def test_decode_splits_of_a_short_window(mla, splits):
    c = decode_case("v3", [2000, 3, 0, 900, 1500], 90, 2, seed=42)
    wr.check(*decode(mla, c, num_splits=splits), c.want(), 5)


@pytest.mark.parametrize("heads", [600, 2500])
def test_more_heads_than_blocks_run_at_once(mla, heads):
    c = wr.Case(seed=43, dtype="f32", heads=heads, latent=16, rope=2, page=16, kv=[100, 0, 40, 333], q=[1] * 4, window=60,
                sinks=3)
    wr.check(*decode(mla, c), c.want(), 4)


@pytest.mark.parametrize("geometry", ["v3", "h16", "h20", "nope64"])
@pytest.mark.parametrize("batch", [1, 31, 33])
def test_prompts_of_few_tokens_and_short_windows(mla, geometry, batch):
    # row tiles described by the units themselves up to 32 sequences, scheduled beyond; some prompts are empty
    q = [(5 * i) % 3 if batch > 1 else 7 for i in range(batch)]
    kv = [max(k, (61 * i) % 400) for i, k in enumerate(q)]
    c = prefill_case(geometry, kv, q, 120, 5, seed=44, tail=2)
    wr.check(*prefill(mla, c), c.want(), sum(q))


def test_a_padded_batch_of_prompts(mla):
    # many more rows of q than tokens, as a captured call pads them; long rows, so that the few there are get cut
    c = prefill_case("v3", [2000, 900, 0], [3, 2, 0], 1900, 4, seed=41, tail=400)
    o, l = prefill(mla, c)
    wr.check(o, l, c.want(), 5)
    assert (o[5:] == 7).all() and (l[5:] == 7).all()


def test_refusals_of_the_binding(mla):
    c = decode_case("v3", [70], 20, 0, seed=25)
    cache, q, table, kv, cu = c.dev()
    o, l = outputs(c)

    def refused(**change):
        a = dict(o=o, q=q, cache=cache, table=table, kv=kv, window=20, sinks=0, lse=l) | change
        with pytest.raises(mla.MlaError) as e:
            mla.mla_decode_window(a["o"], a["q"], a["cache"], a["table"], a["kv"], 512, 64, 0.1, a["window"],
                                  sinks=a["sinks"], lse_out=a["lse"])
        assert e.value.status in (mla.MLA_ERR_INVALID_ARG, mla.MLA_ERR_UNSUPPORTED)
    refused(window=0)
    refused(window=-3)
    refused(sinks=-1)
    refused(kv=kv.long())
    refused(kv=torch.cat([kv, kv]))
    refused(table=table.expand(2, -1).contiguous())
    refused(lse=l.double())
    refused(lse=l[:, :3])
    refused(q=q.float())
    refused(o=o.cpu())
    refused(o=o.transpose(1, 2))
    refused(table=table[:, :0])
    refused(table=table[0])
    refused(table=table[0, 0])
    refused(q=q[0])
    refused(q=q[0, 0, 0])
    refused(kv=kv[0])
    refused(cache=cache[0])
    assert (o == 7).all() and (l == 7).all()

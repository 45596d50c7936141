"""The cache read-backs, the ds_mla write and the windowed attention as seen from the host, without a
GPU: malformed arguments are rejected before anything touches the device."""
import pytest

from test_abi import _contig, _view, mla  # noqa: F401  (the module's library fixture)

P = 0x10000


def decode(lib, *, dtype=1, o=None, q=None, cache=None, table=P, stride=4, blocks=4, lens=P, L=512, R=64, scale=0.1,
           window=8, sinks=2, splits=0, ws=P, ws_bytes=1 << 40):
    return lib.mla_decode_window(dtype, o or _contig([2, 16, 512]), None, q or _contig([2, 16, 576]),
                                 cache or _contig([4, 64, 576]), table, stride, blocks, lens, L, R, scale, window,
                                 sinks, splits, ws, ws_bytes, None)


def prefill(lib, *, dtype=1, o=None, q=None, cache=None, table=P, stride=4, blocks=4, cu=P, lens=P, batch=2, L=512,
            R=64, scale=0.1, window=8, sinks=2, ws=P, ws_bytes=1 << 40):
    return lib.mla_prefill_window(dtype, o or _contig([5, 16, 512]), None, q or _contig([5, 16, 576]),
                                  cache or _contig([4, 64, 576]), table, stride, blocks, cu, lens, batch, L, R, scale,
                                  window, sinks, ws, ws_bytes, None)


COMMON = [dict(window=0), dict(window=-1), dict(sinks=-1), dict(dtype=9), dict(table=None), dict(lens=None),
          dict(blocks=0), dict(stride=3), dict(L=0), dict(R=-1), dict(L=500), dict(ws=None), dict(ws_bytes=100),
          dict(ws=P + 8), dict(cache=_contig([4, 64, 512])), dict(cache=_contig([0, 64, 576])),
          dict(cache=_view([4, 64, 576], [64 * 576 * 2, 576 * 2, 2]))]


@pytest.mark.parametrize("change", COMMON + [dict(splits=-1), dict(o=_contig([2, 16, 576])), dict(q=_contig([2, 576]))])
def test_decode_window_rejects(mla, change):  # noqa: F811
    assert decode(mla.lib(), **change) == mla.MLA_ERR_INVALID_ARG
    assert mla.lib().mla_last_error()


@pytest.mark.parametrize("change", COMMON + [dict(batch=-1), dict(cu=None), dict(o=_contig([5, 16, 576]))])
def test_prefill_window_rejects(mla, change):  # noqa: F811
    assert prefill(mla.lib(), **change) == mla.MLA_ERR_INVALID_ARG
    assert mla.lib().mla_last_error()


def test_window_empty_and_unsupported(mla):  # noqa: F811
    lib = mla.lib()
    assert decode(lib, o=_contig([0, 16, 512]), q=_contig([0, 16, 576])) == mla.MLA_OK
    assert prefill(lib, o=_contig([0, 16, 512]), q=_contig([0, 16, 576])) == mla.MLA_OK
    assert prefill(lib, batch=0) == mla.MLA_OK
    assert decode(lib, L=576, R=0, o=_contig([2, 16, 576])) == mla.MLA_ERR_UNSUPPORTED
    assert lib.mla_decode_window_workspace_size(-1, 2, 3, 0) == 0
    assert lib.mla_prefill_window_workspace_size(1, -1, 2, 3) == 0
    assert lib.mla_decode_window_workspace_size(64, 128, 512, 0) > 0
    assert lib.mla_prefill_window_workspace_size(64, 1, 128, 512) > 0


def write(lib, *, dtype=1, cache=None, kv_c=None, k_pe=None, slots=P, n=3):
    return lib.mla_cache_write_ds_mla(dtype, cache or _contig([2, 8, 656]), kv_c or _contig([3, 512]),
                                      k_pe or _contig([3, 64]), slots, n, None)


@pytest.mark.parametrize("change", [
    dict(dtype=5), dict(cache=_contig([2, 8, 576])), dict(cache=_contig([2, 8, 656], data=P + 8)),
    dict(cache=_view([2, 8, 656], [8 * 664, 664, 1])), dict(kv_c=_contig([3, 256])), dict(k_pe=_contig([3, 32])),
    dict(kv_c=_contig([4, 512])), dict(slots=None), dict(n=-1), dict(kv_c=_view([3, 512], [1024, 2]))])
def test_write_ds_mla_rejects(mla, change):  # noqa: F811
    assert write(mla.lib(), **change) == mla.MLA_ERR_INVALID_ARG
    assert mla.lib().mla_last_error()


def test_write_ds_mla_empty(mla):  # noqa: F811
    assert write(mla.lib(), kv_c=_contig([0, 512]), k_pe=_contig([0, 64]), n=0, slots=None) == mla.MLA_OK


def reads(lib, fmt, *, dtype=1, out=None, cache=None, table=P, stride=4, blocks=4, cu=P, batch=2, scale=P):
    width = 656 if fmt == "ds_mla" else 576
    args = (dtype, out or _contig([9, 576]), cache or _contig([4, 8, width]), table, stride, blocks, cu, None, batch)
    if fmt == "plain":
        return lib.mla_cache_read(*args, None)
    if fmt == "fp8":
        return lib.mla_cache_read_fp8(*args, scale, None)
    return lib.mla_cache_read_ds_mla(*args, None)


@pytest.mark.parametrize("fmt", ["plain", "fp8", "ds_mla"])
@pytest.mark.parametrize("change", [dict(dtype=4), dict(out=_contig([9, 500])), dict(out=_contig([9, 2, 288])),
                                    dict(table=None), dict(cu=None), dict(batch=-1), dict(blocks=0), dict(stride=2),
                                    dict(cache=_contig([4, 8, 512])), dict(out=_view([9, 576], [1152, 2]))])
def test_read_rejects(mla, fmt, change):  # noqa: F811
    assert reads(mla.lib(), fmt, **change) == mla.MLA_ERR_INVALID_ARG
    assert mla.lib().mla_last_error()


@pytest.mark.parametrize("fmt", ["plain", "fp8", "ds_mla"])
def test_read_empty(mla, fmt):  # noqa: F811
    assert reads(mla.lib(), fmt, out=_contig([0, 576])) == mla.MLA_OK
    assert reads(mla.lib(), fmt, batch=0, table=None, cu=None) == mla.MLA_OK
    if fmt == "fp8":
        assert reads(mla.lib(), fmt, scale=None) == mla.MLA_ERR_INVALID_ARG

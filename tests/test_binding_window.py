"""Refusals of the binding's newer calls that need no GPU: tensors that do not lie on one."""
import pytest
import torch


@pytest.fixture(scope="module")
def mla():
    from mla_latent_kv_11_gb300 import build
    build.build()
    import mla_latent_kv_11_gb300 as m
    return m


def calls(mla, **more):
    z = torch.zeros
    i32 = dict(dtype=torch.int32)
    entries, rows, table, cu = z(2, 8, 656, dtype=torch.uint8), z(4, 576), z(1, 1, **i32), torch.tensor([0, 4], **i32)
    q, o, cache, lens = z(1, 2, 576), z(1, 2, 512), z(1, 64, 576), z(1, **i32)
    window = dict(window=8, sinks=1) | more
    return [lambda: mla.mla_cache_write_ds_mla(entries, z(3, 512), z(3, 64), z(3, dtype=torch.int64)),
            lambda: mla.mla_cache_read(rows, z(1, 8, 576), table, cu),
            lambda: mla.mla_cache_read_fp8(rows, z(1, 8, 576, dtype=torch.uint8), table, cu, torch.ones(1)),
            lambda: mla.mla_cache_read_ds_mla(rows, entries, table, cu),
            lambda: mla.mla_decode_window(o, q, cache, table, lens, 512, 64, 0.1, **window),
            lambda: mla.mla_prefill_window(o, q, cache, table, torch.tensor([0, 1], **i32), lens, 512, 64, 0.1, **window)]


@pytest.mark.parametrize("which", range(6))
def test_host_tensors_are_refused(mla, which):
    with pytest.raises(mla.MlaError) as e:
        calls(mla)[which]()
    assert e.value.status == mla.MLA_ERR_INVALID_ARG and "device" in str(e.value)


def test_the_stream_without_the_direct_question(mla, monkeypatch):
    # a torch release without the private call: the public stream object serves
    class Stream:
        cuda_stream = 77
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream)
    assert mla._stream_on(None, 0) == 77 and mla._stream_on(5, 0) == 5


@pytest.mark.parametrize("more", [dict(window=2 ** 32 + 5), dict(window=2 ** 31), dict(window=2 ** 63 - 1),
                                  dict(sinks=2 ** 32), dict(sinks=-2 ** 32 + 3)])
@pytest.mark.parametrize("which", [4, 5])
def test_counts_beyond_32_bits_are_refused(mla, which, more):
    # passed on they would lose their upper bits: a window of 2^32 + 5 rows would be one of 5
    with pytest.raises(mla.MlaError) as e:
        calls(mla, **more)[which]()
    assert e.value.status == mla.MLA_ERR_INVALID_ARG and next(iter(more)) in str(e.value)


def test_splits_beyond_32_bits_are_refused(mla):
    with pytest.raises(mla.MlaError) as e:
        calls(mla, num_splits=2 ** 32 + 1)[4]()
    assert "num_splits" in str(e.value)

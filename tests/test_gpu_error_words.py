"""mla_device_error over all of the library's parts: each reports, and one call reads and clears them all."""
import pytest
import torch

from test_gpu_window import decode_case, outputs

pytestmark = pytest.mark.gpu


def bad_write(mla):
    cache = torch.zeros(2, 8, 576, device="cuda")
    mla.mla_cache_write(cache, torch.zeros(1, 512, device="cuda"), torch.zeros(1, 64, device="cuda"),
                        torch.tensor([16], device="cuda"))


def bad_ds_mla_write(mla):
    cache = torch.zeros(2, 8, 656, dtype=torch.uint8, device="cuda")
    mla.mla_cache_write_ds_mla(cache, torch.zeros(1, 512, device="cuda"), torch.zeros(1, 64, device="cuda"),
                               torch.tensor([16], device="cuda"))


def bad_window_decode(mla, geometry, rows):
    # a page that the cache does not hold; `rows` of a window decide whether a schedule is made
    c = decode_case(geometry, [rows], rows, 0, seed=61)
    cache, q, table, kv, _ = c.dev()
    table[0, 1] = 10 ** 6
    o, l = outputs(c)
    mla.mla_decode_window(o, q, cache, table, kv, 512, 64, c.scale, rows, lse_out=l)


def bad_window_length(mla):
    # a length beyond the table, found by the schedule
    c = decode_case("lite_f32", [2000], 2000, 0, seed=62)
    cache, q, table, kv, _ = c.dev()
    o, l = outputs(c)
    mla.mla_decode_window(o, q, cache, table, kv + 1000, 512, 64, c.scale, 1000, lse_out=l)


def bad_decode(mla, geometry):
    c = decode_case(geometry, [300], 300, 0, seed=63)
    cache, q, table, kv, _ = c.dev()
    table[0, 1] = 10 ** 6
    o, _ = outputs(c)
    mla.mla_decode(o, q, cache, table, kv, 512, 64, c.scale)


PARTS = [bad_write, bad_ds_mla_write, lambda m: bad_window_decode(m, "v3", 300), lambda m: bad_window_decode(m, "v3", 3000),
         lambda m: bad_window_decode(m, "lite_f32", 300), bad_window_length, lambda m: bad_decode(m, "v3"),
         lambda m: bad_decode(m, "lite_f32")]


@pytest.mark.parametrize("which", range(len(PARTS)))
def test_every_part_reports_once(mla, which):
    mla.mla_device_error()
    PARTS[which](mla)
    with pytest.raises(mla.MlaError) as e:
        mla.mla_device_error()
    assert e.value.status == mla.MLA_ERR_DEVICE_DATA
    mla.mla_device_error()


def test_one_call_reads_and_clears_them_all(mla):
    for part in PARTS:
        part(mla)
    with pytest.raises(mla.MlaError) as e:
        mla.mla_device_error()
    assert e.value.status == mla.MLA_ERR_DEVICE_DATA
    mla.mla_device_error()


def test_errors_of_another_stream(mla):
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for part in PARTS:
            part(mla)
        with pytest.raises(mla.MlaError):
            mla.mla_device_error()
    mla.mla_device_error()


def test_a_wait_that_runs_out_goes_before_bad_data(mla):
    bad_ds_mla_write(mla)
    mla.mla_check_bounded_wait(2000)
    with pytest.raises(mla.MlaError) as e:
        mla.mla_device_error()
    assert e.value.status == mla.MLA_ERR_TIMEOUT
    mla.mla_device_error()

"""Codes of the ds_mla cache write for every value a group can hold, byte for byte."""
import pytest
import torch

from test_gpu_cache_io import entry_of

pytestmark = pytest.mark.gpu


def rows_of(values, top):
    """Rows [T, 512] whose groups of 128 hold `top` and 127 of the values no larger in magnitude."""
    v = values[values.float().abs() <= top]
    v = torch.cat([v, torch.zeros(-len(v) % (4 * 127), dtype=v.dtype)]).view(-1, 4, 127)
    return torch.cat([torch.full((*v.shape[:2], 1), top, dtype=v.dtype), v], -1).view(-1, 512)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("top", [448.0, 1.0, 2.0 ** -7, 1.9921875, 3e38, 2.0 ** -120, 2.0 ** -133, 0.0])
def test_every_value_of_a_group(mla, dtype, top):
    # bf16: every bit pattern, so both zeros and the values below the normal ones too; float32: patterns of
    # every sign and exponent, and many below the normal ones
    top = float(torch.tensor(top).to(torch.bfloat16))
    if dtype == torch.bfloat16:
        values = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    else:
        values = torch.randint(-2 ** 31, 2 ** 31, (100000,), generator=torch.Generator().manual_seed(1)).to(torch.int32)
        values[:2] = torch.tensor([0, -2 ** 31])
        values[2:20000] >>= torch.arange(2, 20000) % 24      # the sign and few other bits: below the normal ones
        values[2:20000] &= -(2 ** 31) | 2 ** 23 - 1
        values = values.view(torch.float32)
    kv_c = rows_of(values, top)
    n = len(kv_c)
    cache = torch.zeros(n, 1, 656, dtype=torch.uint8, device="cuda")
    mla.mla_cache_write_ds_mla(cache, kv_c.cuda(), torch.zeros(n, 64, dtype=dtype, device="cuda"),
                               torch.arange(n, device="cuda"))
    mla.mla_device_error()
    want = entry_of(kv_c, torch.zeros(n, 64, dtype=dtype))
    got = cache.view(n, 656).cpu()
    off = (got != want).nonzero()
    assert not len(off), f"{len(off)} bytes differ, the first at {off[0].tolist()}: {got[tuple(off[0])]} for " \
                         f"{want[tuple(off[0])]}"

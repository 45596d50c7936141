"""The two CTAs of a tensor-core row tile hold half of its rows each, and the first issues the products of
both: every tile has to read the second CTA's weights and cleared rows as they were written."""
import pytest
import torch

import window_ref as wr
from test_gpu_window import decode_case, outputs, prefill_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_both_halves_of_every_tile_under_other_traffic(mla, which):
    # 10 to 50 tiles a row tile, weights that differ from tile to tile, rows to clear at both ends of each
    # window, and another stream that keeps memory and shared memory busy: 50 times the same bits, and those
    # within the bound of 64 bits
    if which == "decode":
        c = decode_case("v3", [6000, 3001, 2999, 1500, 4097, 1300], 2900, 70, seed=51, spread=1.5)
    else:
        c = prefill_case("h64", [2500, 1400], [9, 6], 1333, 5, seed=52, spread=1.5)
    cache, q, table, kv, cu = c.dev()
    o, l = outputs(c)
    first = None
    source, sink = (torch.zeros(64 << 20, dtype=torch.uint8, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(50):
        with torch.cuda.stream(side):
            sink.copy_(source)
        if which == "decode":
            mla.mla_decode_window(o, q, cache, table, kv, 512, 64, c.scale, c.window, sinks=c.sinks, lse_out=l)
        else:
            mla.mla_prefill_window(o, q, cache, table, cu, kv, 512, 64, c.scale, c.window, sinks=c.sinks, lse_out=l)
        if first is None:
            first = o.clone(), l.clone()
        else:
            assert torch.equal(o, first[0]) and torch.equal(l, first[1])
    torch.cuda.synchronize()
    mla.mla_device_error()
    wr.check(*first, c.want(), sum(c.q_lens))

"""Norms with rotations, row masses and eviction as seen from the host, without a GPU: malformed arguments are rejected
before anything touches the device."""
import os
import subprocess
import sys

import pytest
import torch

from test_abi import _contig, _view, mla  # noqa: F401  (the module's library fixture)
from mla_latent_kv_11_gb300 import MlaTensor

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000
NONE = MlaTensor()


def norm_q(lib, *, dtype=1, nope=None, pe=None, q=None, w=None, eps=1e-6, pos=P, cs=P, stride=64, count=9):
    return lib.mla_norm_rope_q(dtype, nope or _contig([3, 4, 128]), pe or _contig([3, 4, 64]), q or _contig([3, 4, 192]),
                               w or NONE, eps, pos, cs, stride, count, 1, None)


@pytest.mark.parametrize("change", [
    dict(dtype=7), dict(nope=_contig([3, 4, 120])), dict(nope=_contig([3, 5, 128])), dict(pe=_contig([2, 4, 64])),
    dict(q=_contig([3, 4, 192], data=0)), dict(q=_contig([12, 192])), dict(q=_view([3, 4, 192], [4 * 384, 384, 2])),
    dict(w=_contig([3, 192])), dict(w=_contig([4, 128])), dict(w=_contig([192])), dict(eps=-1.0), dict(eps=float("nan")),
    dict(pos=None), dict(cs=None), dict(stride=63), dict(count=0), dict(count=-1),
    dict(pe=_contig([3, 4, 63]), nope=_contig([3, 4, 129]))])
def test_norm_q_rejects(mla, change):  # noqa: F811
    assert norm_q(mla.lib(), **change) == mla.MLA_ERR_INVALID_ARG
    assert mla.lib().mla_last_error()


def rows(lib, form="", *, dtype=1, cache=None, kv=None, w=None, eps=1e-6, pos=P, cs=P, stride=64, count=9, slots=P, n=3, scale=P):
    more = [scale] if form == "_fp8" else []
    entry = 656 if form == "_ds_mla" else 576
    return getattr(lib, "mla_norm_rope_cache_write" + form)(
        dtype, cache or _contig([2, 8, entry]), kv or _contig([3, 576]), w or _contig([512]), eps, pos, cs, stride, count, 0, slots, n,
        *more, None)


ROWS = [dict(dtype=-1), dict(kv=_contig([2, 576])), dict(kv=_contig([3, 500])), dict(w=_contig([577])), dict(w=_contig([0])),
        dict(w=_contig([1, 512])), dict(n=-1), dict(n=4), dict(slots=None), dict(pos=None), dict(cs=None), dict(stride=10),
        dict(count=0), dict(eps=-0.5), dict(w=_contig([511])), dict(cache=_contig([0, 8, 576])), dict(cache=_contig([2, 8, 570])),
        dict(w=_contig([512], data=0))]


@pytest.mark.parametrize("form", ["", "_fp8", "_ds_mla"])
@pytest.mark.parametrize("change", ROWS)
def test_norm_rows_reject(mla, form, change):  # noqa: F811
    assert rows(mla.lib(), form, **change) == mla.MLA_ERR_INVALID_ARG
    assert mla.lib().mla_last_error()


def test_norm_rows_of_formats(mla):  # noqa: F811
    lib = mla.lib()
    assert rows(lib, "_fp8", scale=None) == mla.MLA_ERR_INVALID_ARG
    assert rows(lib, "_ds_mla", cache=_contig([2, 8, 656], data=P + 8)) == mla.MLA_ERR_INVALID_ARG
    assert rows(lib, "_ds_mla", w=_contig([448])) == mla.MLA_ERR_INVALID_ARG
    for form in ("", "_fp8", "_ds_mla"):
        assert rows(lib, form, n=0, kv=_contig([0, 576]), pos=None, cs=None, slots=None) == mla.MLA_OK


def both(lib, *, nope=None, pe=None, q=None, qw=NONE, cache=None, kv=None, kw=None, n=3):
    return lib.mla_norm_rope_q_cache_write(1, nope or _contig([3, 4, 128]), pe or _contig([3, 4, 64]), q or _contig([3, 4, 192]), qw,
                                           cache or _contig([2, 8, 576]), kv or _contig([3, 576]), kw or _contig([512]), 1e-6, P, P,
                                           64, 9, 1, P, n, None)


@pytest.mark.parametrize("change", [dict(n=2), dict(kv=_contig([3, 544]), cache=_contig([2, 8, 544])), dict(qw=_contig([5, 192])),
                                    dict(q=_contig([2, 4, 192]), nope=_contig([2, 4, 128]), pe=_contig([2, 4, 64])),
                                    dict(nope=_contig([3, 4, 64])), dict(kw=_contig([600]))])
def test_both_reject(mla, change):  # noqa: F811
    assert both(mla.lib(), **change) == mla.MLA_ERR_INVALID_ARG
    assert mla.lib().mla_last_error()


def test_norm_of_nothing_and_of_too_much(mla):  # noqa: F811
    lib = mla.lib()
    assert norm_q(lib, nope=_contig([0, 4, 128]), pe=_contig([0, 4, 64]), q=_contig([0, 4, 192]), pos=None, cs=None) == mla.MLA_OK
    n = 2 ** 20
    assert norm_q(lib, nope=_contig([n, n, 128]), pe=_contig([n, n, 64]), q=_contig([n, n, 192])) == mla.MLA_ERR_UNSUPPORTED


def decode_mass(lib, *, dtype=1, mass=P, stride=256, rows=256, q=None, cache=None, table=P, bt=4, blocks=4, lens=P, lse=P, scale=0.1,
                decay=1.0):
    return lib.mla_decode_mass(dtype, mass, stride, rows, q or _contig([2, 16, 576]), cache or _contig([4, 64, 576]), table, bt,
                               blocks, lens, lse, scale, decay, None)


def prefill_mass(lib, *, dtype=1, mass=P, stride=256, rows=256, q=None, cache=None, table=P, bt=4, blocks=4, cu=P, lens=P, batch=2,
                 lse=P, scale=0.1, decay=1.0, ws=P, ws_bytes=1 << 30):
    return lib.mla_prefill_mass(dtype, mass, stride, rows, q or _contig([5, 16, 576]), cache or _contig([4, 64, 576]), table, bt,
                                blocks, cu, lens, batch, lse, scale, decay, ws, ws_bytes, None)


MASS = [dict(dtype=3), dict(mass=None), dict(lse=None), dict(table=None), dict(lens=None), dict(blocks=0), dict(bt=3), dict(rows=0),
        dict(stride=255), dict(scale=float("nan")), dict(scale=float("inf")), dict(decay=float("nan")), dict(decay=-float("inf")),
        dict(cache=_contig([4, 64, 512])), dict(cache=_contig([0, 64, 576])), dict(q=_contig([2, 576])),
        dict(q=_contig([2, 16, 0]), cache=_contig([4, 64, 0])), dict(cache=_view([4, 64, 576], [64 * 1152, 1152, 2]))]


@pytest.mark.parametrize("change", MASS)
def test_decode_mass_rejects(mla, change):  # noqa: F811
    assert decode_mass(mla.lib(), **change) == mla.MLA_ERR_INVALID_ARG
    assert mla.lib().mla_last_error()


@pytest.mark.parametrize("change", MASS + [dict(cu=None), dict(batch=-1), dict(ws=None), dict(ws_bytes=16), dict(ws=P + 16)])
def test_prefill_mass_rejects(mla, change):  # noqa: F811
    assert prefill_mass(mla.lib(), **change) == mla.MLA_ERR_INVALID_ARG
    assert mla.lib().mla_last_error()


def test_mass_of_nothing_and_of_too_much(mla):  # noqa: F811
    lib = mla.lib()
    assert decode_mass(lib, q=_contig([0, 16, 576])) == mla.MLA_OK
    assert prefill_mass(lib, q=_contig([0, 16, 576])) == mla.MLA_OK
    assert prefill_mass(lib, batch=0) == mla.MLA_OK
    for wide in (dict(q=_contig([2, 16, 1025]), cache=_contig([4, 64, 1025])), dict(q=_contig([2, 5000, 64]), cache=_contig([4, 64, 64])),
                 dict(q=_contig([70000, 2, 64]), cache=_contig([4, 64, 64]))):
        assert decode_mass(lib, **wide) == mla.MLA_ERR_UNSUPPORTED
    assert prefill_mass(lib, batch=70000) == mla.MLA_ERR_UNSUPPORTED
    assert lib.mla_prefill_mass_workspace_size() > 0


def evict(lib, *, size=2, cache=None, mass=P, ms=256, mr=256, table=P, bt=4, blocks=4, lens=P, batch=2, budget=100, sinks=4,
          recent=8, table_out=None, bto=0, blocks_out=0, mass_out=None, mos=0, mor=0, lens_out=P, kept=None, ws=P, ws_bytes=1 << 30):
    return lib.mla_cache_evict(size, cache or _contig([4, 64, 576]), mass, ms, mr, table, bt, blocks, lens, batch, budget, sinks, recent,
                               table_out, bto, blocks_out, mass_out, mos, mor, lens_out, kept, ws, ws_bytes, None)


@pytest.mark.parametrize("change", [
    dict(size=0), dict(size=8), dict(cache=_contig([4, 64])), dict(cache=_contig([4, 0, 576])), dict(budget=0), dict(budget=-3),
    dict(sinks=-1), dict(recent=-1), dict(sinks=60, recent=41), dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), dict(batch=-1),
    dict(mass=None), dict(table=None), dict(lens=None), dict(lens_out=None), dict(blocks=0), dict(bt=3), dict(mr=0), dict(ms=255),
    dict(table_out=P, bto=3, blocks_out=4), dict(table_out=P, bto=4, blocks_out=0), dict(mass_out=P, mos=9, mor=10),
    dict(mass_out=P, mos=9, mor=0), dict(ws=None), dict(ws_bytes=64), dict(ws=P + 128),
    dict(cache=_view([4, 64, 576], [64 * 1152, 1152, 2]))])
def test_evict_rejects(mla, change):  # noqa: F811
    assert evict(mla.lib(), **change) == mla.MLA_ERR_INVALID_ARG
    assert mla.lib().mla_last_error()


def test_evict_of_nothing_and_of_too_much(mla):  # noqa: F811
    lib = mla.lib()
    assert evict(lib, batch=0) == mla.MLA_OK
    assert evict(lib, batch=70000) == mla.MLA_ERR_UNSUPPORTED
    assert lib.mla_cache_evict_workspace_size(-1, 2, 3) == 0
    # the lists of rows that stay are no longer than the sequences
    assert lib.mla_cache_evict_workspace_size(4, 100, 10 ** 6) == lib.mla_cache_evict_workspace_size(4, 100, 100) > 0


def calls(m):
    z, i32, i64 = torch.zeros, dict(dtype=torch.int32), dict(dtype=torch.int64)
    q, kv, cs, pos, slots = z(3, 4, 192), z(3, 576), z(9, 64), z(3, **i64), z(3, **i64)
    cache, entries, w = z(2, 8, 576), z(2, 8, 656, dtype=torch.uint8), z(512)
    table, lens, cu, mass = z(1, 2, **i32), z(1, **i32), torch.tensor([0, 3], **i32), z(1, 16)
    return [lambda: m.mla_norm_rope_q(q[..., :128], q[..., 128:], q, None, pos, cs),
            lambda: m.mla_norm_rope_cache_write(cache, kv, w, pos, cs, slots),
            lambda: m.mla_norm_rope_cache_write_fp8(cache.to(torch.uint8), kv, w, pos, cs, slots, torch.ones(1)),
            lambda: m.mla_norm_rope_cache_write_ds_mla(entries, kv, w, pos, cs, slots),
            lambda: m.mla_norm_rope_q_cache_write(q[..., :128], q[..., 128:], q, None, cache, kv, w, pos, cs, slots),
            lambda: m.mla_decode_mass(mass, z(1, 4, 576), cache, table, lens, z(1, 4), 0.1),
            lambda: m.mla_prefill_mass(mass, z(3, 4, 576), cache, table, cu, lens, z(3, 4), 0.1),
            lambda: m.mla_cache_evict(cache, mass, table, lens, 4, lens)]


@pytest.mark.parametrize("which", range(8))
def test_host_tensors_are_refused(mla, which):  # noqa: F811
    with pytest.raises(mla.MlaError) as e:
        calls(mla)[which]()
    assert e.value.status == mla.MLA_ERR_INVALID_ARG and "device" in str(e.value)


BAD = [lambda m, z: m.mla_norm_rope_q(z(3, 4, 128), z(3, 4, 64), z(3, 4, 192), None, z(3), z(9, 64)),
       lambda m, z: m.mla_norm_rope_q(z(3, 4, 128), z(3, 4, 64), z(3, 4, 192), None, z(2, dtype=torch.int64), z(9, 64)),
       lambda m, z: m.mla_norm_rope_q(z(3, 4, 128), z(3, 4, 64), z(3, 4, 192), None, z(3, dtype=torch.int64), z(9, 32)),
       lambda m, z: m.mla_norm_rope_q(z(3, 4, 128), z(3, 4, 64), z(12, 192), None, z(12, dtype=torch.int64), z(9, 64)),
       lambda m, z: m.mla_norm_rope_cache_write(z(2, 8, 576), z(3, 576), z(512), z(3, dtype=torch.int64), z(9, 64).double(),
                                                z(3, dtype=torch.int64)),
       lambda m, z: m.mla_norm_rope_cache_write(z(2, 8, 576), z(3, 576), z(512), z(3, dtype=torch.int64), z(64, 9).T,
                                                z(3, dtype=torch.int64)),
       lambda m, z: m.mla_norm_rope_cache_write(z(2, 8, 576), z(3, 576), z(512), z(3, dtype=torch.int64), z(9, 64), z(3)),
       lambda m, z: m.mla_norm_rope_cache_write_fp8(z(2, 8, 576), z(3, 576), z(512), z(3, dtype=torch.int64), z(9, 64),
                                                    z(3, dtype=torch.int64), z(1)),
       lambda m, z: m.mla_decode_mass(z(2, 16), z(1, 4, 576), z(2, 8, 576), z(1, 2, dtype=torch.int32), z(1, dtype=torch.int32),
                                      z(1, 4), 0.1),
       lambda m, z: m.mla_decode_mass(z(1, 16).double(), z(1, 4, 576), z(2, 8, 576), z(1, 2, dtype=torch.int32),
                                      z(1, dtype=torch.int32), z(1, 4), 0.1),
       lambda m, z: m.mla_decode_mass(z(1, 16), z(1, 4, 576), z(2, 8, 576), z(1, 2, dtype=torch.int32), z(1, dtype=torch.int32),
                                      z(1, 5), 0.1),
       lambda m, z: m.mla_prefill_mass(z(1, 16), z(3, 4, 576), z(2, 8, 576), z(1, 2, dtype=torch.int32), z(3, dtype=torch.int32),
                                       z(1, dtype=torch.int32), z(3, 4), 0.1),
       lambda m, z: m.mla_cache_evict(z(2, 8, 576), z(1, 16), z(1, 2, dtype=torch.int32), z(1, dtype=torch.int32), 2 ** 32 + 4,
                                      z(1, dtype=torch.int32)),
       lambda m, z: m.mla_cache_evict(z(2, 8, 576), z(1, 16), z(1, 2, dtype=torch.int32), z(1, dtype=torch.int32), 4,
                                      z(1, dtype=torch.int64)),
       lambda m, z: m.mla_cache_evict(z(2, 8, 576), z(1, 16), z(1, 2, dtype=torch.int32), z(1, dtype=torch.int32), 4,
                                      z(1, dtype=torch.int32), kept_out=z(1, 5, dtype=torch.int32)),
       lambda m, z: m.mla_cache_evict(z(2, 8, 576), z(1, 16), z(2, 2, dtype=torch.int32), z(1, dtype=torch.int32), 4,
                                      z(1, dtype=torch.int32))]


@pytest.mark.parametrize("which", range(len(BAD)))
def test_the_binding_refuses(mla, which):  # noqa: F811
    with pytest.raises(mla.MlaError) as e:
        BAD[which](mla, torch.zeros)
    assert e.value.status == mla.MLA_ERR_INVALID_ARG and "on one CUDA device" not in str(e.value)


def test_a_refused_lse_is_named(mla):  # noqa: F811
    for which in (9 + 1, None):
        with pytest.raises(mla.MlaError) as e:
            if which is not None:
                BAD[which](mla, torch.zeros)
            else:
                z, i32 = torch.zeros, dict(dtype=torch.int32)
                mla.mla_prefill_mass(z(1, 16), z(3, 4, 576), z(2, 8, 576), z(1, 2, **i32), z(2, **i32), z(1, **i32), z(3, 4).double(), 0.1)
        assert "lse must" in str(e.value)


def test_widths_beyond_32_bits_are_refused(mla):  # noqa: F811
    # passed on they would lose their upper bits: masses of 2^32 + 8 rows would be those of 8
    z, i32 = torch.zeros, dict(dtype=torch.int32)
    wide, table = (torch.empty(1, 2 ** 32 + 8, dtype=t, device="meta") for t in (torch.float32, torch.int32))
    for mass, tab in ((wide, z(1, 2, **i32)), (z(1, 16), table)):
        for call in (lambda: mla.mla_decode_mass(mass, z(1, 4, 576), z(2, 8, 576), tab, z(1, **i32), z(1, 4), 0.1),
                     lambda: mla.mla_prefill_mass(mass, z(3, 4, 576), z(2, 8, 576), tab, z(2, **i32), z(1, **i32), z(3, 4), 0.1),
                     lambda: mla.mla_cache_evict(z(2, 8, 576), mass, tab, z(1, **i32), 4, z(1, **i32))):
            with pytest.raises(mla.MlaError) as e:
                call()
            assert e.value.status == mla.MLA_ERR_INVALID_ARG and "32 bits" in str(e.value)


def test_importing_the_package_does_not_import_torch():
    # a build, or a ctypes user of the library, needs none
    code = ("import sys, mla_latent_kv_11_gb300 as m; assert 'torch' not in sys.modules; "
            "m.lib(); assert 'torch' not in sys.modules; import torch; "
            "\ntry: m.mla_norm_rope_q(*[torch.zeros(1, 1, 2)] * 4, torch.zeros(1), torch.zeros(1, 2))"
            "\nexcept m.MlaError as e: print(e)")
    got = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "positions must be" in got.stdout, got.stderr

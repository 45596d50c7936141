"""Windowed calls that make a schedule and merge cut row tiles: captured, on several streams, with one
workspace for several calls, and with a merge that has nothing to join. Each test shows by the workspace that
its calls are such (short windows on the tensor cores need neither)."""
import pytest
import torch

import window_ref as wr
from test_gpu_window import decode_case, outputs, prefill_case

pytestmark = pytest.mark.gpu

# more tiles than go without a schedule (8 of 128 rows on the tensor cores; none on the CUDA cores)
LONG = {"v3": 1900, "h20": 1700, "lite_f32": 700}


def size_of(mla, c, which, **more):
    tokens, heads = c.qs.shape[:2]
    return mla.mla_decode_window_workspace_size(tokens, heads, c.latent, **more) if which == "decode" else \
        mla.mla_prefill_window_workspace_size(tokens, len(c.kv), heads, c.latent)


class Call:
    """A windowed call of a case, with its buffers on the GPU."""

    def __init__(self, mla, which, c, workspace=None, **more):
        self.mla, self.which, self.c, self.more = mla, which, c, more
        self.inputs, (self.o, self.l) = c.dev(), outputs(c)
        self.workspace = workspace

    def __call__(self, stream=None):
        c, (cache, q, table, kv, cu) = self.c, self.inputs
        more = dict(sinks=c.sinks, lse_out=self.l, workspace=self.workspace, stream=stream, **self.more)
        if self.which == "decode":
            self.mla.mla_decode_window(self.o, q, cache, table, kv, c.latent, c.rope, c.scale, c.window, **more)
        else:
            self.mla.mla_prefill_window(self.o, q, cache, table, cu, kv, c.latent, c.rope, c.scale, c.window, **more)

    def parts_written(self):
        """Bytes that one call changes in its workspace: (schedule or more, pieces too)."""
        keep = self.workspace
        self.workspace = torch.full((size_of(self.mla, self.c, self.which, **self.more),), 0xA5, dtype=torch.uint8,
                                    device="cuda")
        self()
        changed = int((self.workspace != 0xA5).sum())
        self.workspace = keep
        # the schedule of the few row tiles here takes less than 64 KB; a piece is a row of `latent` float32
        # values a head, most of whose bytes change
        return changed > 0, changed > 64 << 10

    def wipe(self):
        self.o.fill_(7.0)
        self.l.fill_(7.0)

    def check(self):
        wr.check(self.o, self.l, self.c.want(), sum(self.c.q_lens))

    def load(self, c):
        """Another case of the same shapes into the same buffers."""
        for mine, new in zip(self.inputs, c.dev()):
            assert mine.shape == new.shape
            mine.copy_(new)
        self.c = c


def cut_case(which, geometry, seed, kv=(2100, 333, 1500)):
    n = LONG[geometry]
    kv = [min(k, 2100 * n // 1900) for k in kv]
    if which == "decode":
        return decode_case(geometry, kv, n, 4, seed=seed)
    return prefill_case(geometry, kv, [min(k, 3) for k in kv], n, 4, seed=seed)


@pytest.mark.parametrize("geometry", LONG)
@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_captured_and_replayed_with_new_inputs(mla, which, geometry):
    a, b = cut_case(which, geometry, 71), cut_case(which, geometry, 72, kv=(700, 2100, 1999))
    call = Call(mla, which, a)
    assert call.parts_written() == (True, True)
    call.workspace = torch.empty(size_of(mla, a, which), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()      # twice, so that a schedule follows a merge in the same workspace
    for c in (a, b, a):
        if call.c is not c:
            call.load(c)
        call.wipe()
        graph.replay()
        mla.mla_device_error()
        call.check()


@pytest.mark.parametrize("geometry", LONG)
def test_two_graphs_share_a_workspace(mla, geometry):
    cases = [("decode", cut_case("decode", geometry, 73)), ("prefill", cut_case("prefill", geometry, 74, kv=(2100, 70, 900)))]
    workspace = torch.empty(max(size_of(mla, c, w) for w, c in cases), dtype=torch.uint8, device="cuda")
    calls, graphs = [Call(mla, w, c, workspace) for w, c in cases], []
    for call in calls:
        assert call.parts_written() == (True, True)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append(graph)
    for call in calls:
        call.wipe()
    for _ in range(20):
        for graph in graphs:
            graph.replay()
    mla.mla_device_error()
    for call in calls:
        call.check()


@pytest.mark.parametrize("geometry", LONG)
def test_one_after_the_other_in_one_workspace(mla, geometry):
    # each call's schedule is written while the one before may still merge, but for the order of the stream
    cases = [("decode", cut_case("decode", geometry, 75)), ("prefill", cut_case("prefill", geometry, 76, kv=(64, 2100, 900))),
             ("decode", cut_case("decode", geometry, 77, kv=(1, 0, 2100)))]
    workspace = torch.empty(max(size_of(mla, c, w) for w, c in cases), dtype=torch.uint8, device="cuda")
    calls = [Call(mla, w, c, workspace) for w, c in cases]
    for call in calls:
        assert call.parts_written() == (True, True)
        call.wipe()
    for _ in range(30):
        for call in calls:
            call()
    mla.mla_device_error()
    for call in calls:
        call.check()


@pytest.mark.parametrize("geometry", LONG)
def test_two_streams_at_once(mla, geometry):
    calls = [Call(mla, "decode", cut_case("decode", geometry, 78)),
             Call(mla, "prefill", cut_case("prefill", geometry, 79, kv=(2100, 90, 1000)))]
    for call in calls:
        assert call.parts_written() == (True, True)
        call.wipe()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        for call, stream in zip(calls, streams):
            call(stream)        # a workspace of its own each time
    torch.cuda.synchronize()
    mla.mla_device_error()
    for call in calls:
        call.check()


@pytest.mark.parametrize("geometry,batch,splits", [("v3", 60, 60), ("v3", 120, 60), ("lite_f32", 24, 24),
                                                   ("lite_f32", 40, 20)])
def test_a_merge_with_nothing_to_join(mla, geometry, batch, splits):
    # equal sequences over as many units, or half as many: whole row tiles, so that the merge has nothing to do
    # and what follows on the stream waits for the attention through it alone
    c = decode_case(geometry, [1270] * batch, 1200, 0, seed=80)
    call = Call(mla, "decode", c, num_splits=splits)
    assert call.parts_written() == (True, False)
    call.workspace = torch.empty(size_of(mla, c, "decode", num_splits=splits), dtype=torch.uint8, device="cuda")
    call.wipe()
    call()
    mla.mla_device_error()
    call.check()
    want = call.o.clone()
    for _ in range(50):
        call.wipe()
        call()
        copy = call.o.clone()
        assert torch.equal(copy, want)


@pytest.mark.parametrize("batch,splits", [(60, 0), (5, 60)])
def test_the_kernel_behind_a_merge_sees_the_outputs(mla, batch, splits):
    # the library's own next kernel may be launched before the merge ends: it waits for it
    c = decode_case("v3", [1270] * batch, 1200, 0, seed=81)
    call = Call(mla, "decode", c, num_splits=splits)
    assert call.parts_written()[0]
    call.workspace = torch.empty(size_of(mla, c, "decode", num_splits=splits), dtype=torch.uint8, device="cuda")
    call()
    want = call.o.clone()
    copy = torch.zeros(batch, 128, 512 + 64, dtype=torch.bfloat16, device="cuda")
    rope = torch.zeros(batch, 128, 64, dtype=torch.bfloat16, device="cuda")
    for _ in range(50):
        call.wipe()
        call()
        mla.mla_concat_q(copy, call.o, rope)
        assert torch.equal(copy[..., :512], want)
    mla.mla_device_error()
    call.check()

"""Cases of four operators of the paged latent cache, each in a plain form and as the library's call.

  write_ds_mla   rows [c_kv | k_pe] quantised into 656-byte fp8 ds_mla entries as they are written
  read           rows of a paged cache (plain, e4m3 or ds_mla) gathered and dequantised into contiguous rows
  decode_window  one query token a sequence over the latest `window` rows of its cache and its first `sinks` rows
  prefill_window a chunk of query tokens a sequence, causal, with the same window and sinks

`own` false: elementary torch operations in 32 bits. `own` true: the library's calls.
"""
import math
import random

import torch

own = False

LATENT, ROPE, ENTRY, GROUP = 512, 64, 656, 128
E4M3_MAX = 448.0
TINY = 2.0 ** -126          # the smallest scale of a group


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one sequence enters the cache of a decode step: latency
        dict(name="write ds_mla 1 token", op="write_ds_mla", dtype="bf16", tokens=1, pad=0, page=64, layers=1),
        # a decode step of 64 sequences, one layer of a block-major buffer of three
        dict(name="write ds_mla 64 tokens of 3 layers", op="write_ds_mla", dtype="bf16", tokens=64, pad=0, page=64,
             layers=3),
        # a long prompt's rows, with padding slots, from float32 activations, an odd count
        dict(name="write ds_mla 40961 tokens f32", op="write_ds_mla", dtype="f32", tokens=40961, pad=257, page=64,
             layers=1),
        # a prefix of a few sequences read back before a chunk is prefilled over it
        dict(name="read ds_mla 4 x 16K", op="read", cache="ds_mla", dtype="bf16", batch=4, kv_min=16384, kv_max=16384,
             start_max=0, page=64, rope=64, tail=0, lens=1),
        # an e4m3 cache, ragged parts that begin inside the sequences, odd lengths, rows left over at the end
        dict(name="read e4m3 ragged", op="read", cache="e4m3", dtype="f32", batch=37, kv_min=0, kv_max=1999,
             start_max=333, page=16, rope=64, tail=5, lens=2),
        # a plain cache without a rope part, one short sequence
        dict(name="read bf16 77 rows", op="read", cache="plain", dtype="bf16", batch=1, kv_min=77, kv_max=77,
             start_max=0, page=64, rope=0, tail=0, lens=3),
        # one sequence of a chat: latency
        dict(name="decode window 1 x 700", op="decode_window", dtype="bf16", heads=128, rope=64, batch=1, kv_min=700,
             kv_max=700, empty=False, window=512, sinks=4, page=64, lens=4),
        # 64 sequences of 1K to 16K rows, a window of 4096 and four sinks
        dict(name="decode window 64 x 1K-16K", op="decode_window", dtype="bf16", heads=128, rope=64, batch=64,
             kv_min=1024, kv_max=16384, empty=False, window=4096, sinks=4, page=64, lens=5),
        # float32 with 16 heads, an empty sequence, odd window
        dict(name="decode window f32 5 x 256", op="decode_window", dtype="f32", heads=16, rope=64, batch=5, kv_min=1,
             kv_max=256, empty=True, window=101, sinks=1, page=64, lens=6),
        # four prompts' chunks of 1024 tokens over 1K to 8K rows
        dict(name="prefill window 4 x 1024", op="prefill_window", dtype="bf16", heads=128, rope=64, batch=4, q_min=1024,
             q_max=1024, kv_min=1024, kv_max=8192, tail=0, window=2048, sinks=4, page=64, lens=7),
        # no rope part, 64 heads, ragged prompts from their first token, many sinks
        dict(name="prefill window nope ragged", op="prefill_window", dtype="bf16", heads=64, rope=0, batch=5, q_min=1,
             q_max=1999, kv_min=1, kv_max=1999, tail=3, window=777, sinks=70, page=64, lens=8),
        # seven new tokens over one long cache (drafted tokens to verify): few rows, a long axis
        dict(name="prefill window 7 over 16K", op="prefill_window", dtype="bf16", heads=128, rope=64, batch=1, q_min=7,
             q_max=7, kv_min=16001, kv_max=16001, tail=0, window=16384, sinks=16, page=64, lens=9),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _drawn(rng):
    op = rng.choice(["write_ds_mla", "read", "decode_window", "prefill_window"])
    page = rng.choice([16, 32, 64, 64, 128])
    if op == "write_ds_mla":
        tokens = _log(rng, 1, 40961)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), tokens=tokens, pad=rng.randint(0, tokens // 8),
                    page=page, layers=rng.choice([1, 1, 3]))
    lens = rng.randint(10, 1 << 30)
    if op == "read":
        kv = _log(rng, 1, 16384)
        cache = rng.choice(["ds_mla", "e4m3", "plain"])
        return dict(op=op, cache=cache, dtype=rng.choice(["bf16", "f32"]), batch=_log(rng, 1, 64),
                    kv_min=rng.randint(0, kv), kv_max=kv, start_max=rng.choice([0, 0, 100, 1000]), page=page,
                    rope=64 if cache == "ds_mla" else rng.choice([64, 0]), tail=rng.randint(0, 3), lens=lens)
    heads, rope = rng.choice([(128, 64), (128, 64), (64, 64), (64, 0), (16, 64), (20, 64)])
    window, sinks = _log(rng, 1, 16384), rng.choice([0, 1, 4, 4, 64, _log(rng, 1, 300)])
    if op == "decode_window":
        if rng.random() < 0.15:
            kv = _log(rng, 1, 512)
            return dict(op=op, dtype="f32", heads=16, rope=64, batch=_log(rng, 1, 8), kv_min=rng.randint(1, kv),
                        kv_max=kv, empty=rng.random() < 0.5, window=_log(rng, 1, 512), sinks=sinks, page=page, lens=lens)
        kv = _log(rng, 1, 16384)
        return dict(op=op, dtype="bf16", heads=heads, rope=rope, batch=_log(rng, 1, 96), kv_min=rng.randint(1, kv),
                    kv_max=kv, empty=rng.random() < 0.2, window=window, sinks=sinks, page=page, lens=lens)
    q = _log(rng, 1, 2048)
    kv = max(q, _log(rng, 1, 16384))
    return dict(op=op, dtype="bf16", heads=heads, rope=rope, batch=_log(rng, 1, 8), q_min=rng.randint(1, q), q_max=q,
                kv_min=q, kv_max=kv, tail=rng.choice([0, 0, 2]), window=window, sinks=sinks, page=page, lens=lens)


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = [max(a, b) for a, b in zip(most.get(c["op"], [0, 0, 0]), [w["bytes"], w["flops"], _plain_size(c)])]
    while True:
        c = _drawn(rng)
        w = work(c)
        if all(a <= b for a, b in zip([w["bytes"], w["flops"], _plain_size(c)], most[c["op"]])):
            return c


def _lengths(case):
    """(rows in the cache, query tokens or first row) of every sequence of a case."""
    r = random.Random(case["lens"])
    kv = [r.randint(case["kv_min"], case["kv_max"]) for _ in range(case["batch"])]
    if case["op"] == "read":
        return kv, [r.randint(0, case["start_max"]) for _ in kv]
    if case["op"] == "decode_window":
        if case["empty"]:
            kv[0] = 0
        return kv, [min(1, n) for n in kv]
    return kv, [min(n, r.randint(case["q_min"], case["q_max"])) for n in kv]


def _plain_size(case):
    """Scores of the plain form (its largest intermediate); 0 where there are none."""
    if case["op"] not in ("decode_window", "prefill_window"):
        return 0
    kv, q = _lengths(case)
    return case["batch"] * case["heads"] * max(q + [1]) * (_span(case, kv, q) + case["sinks"])


def _span(case, kv, q):
    return max(1, min(max(kv), max(q) + case["window"] - 1))


def _size(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    op = case["op"]
    if op == "write_ds_mla":
        rows = case["tokens"] - case["pad"]
        return {"bytes": rows * (576 * _size(case["dtype"]) + ENTRY) + 8 * case["tokens"], "flops": rows * 2 * LATENT}
    kv, other = _lengths(case)
    if op == "read":
        rows, width = sum(kv), LATENT + case["rope"]
        stored = {"ds_mla": ENTRY, "e4m3": width, "plain": width * _size(case["dtype"])}[case["cache"]]
        pages = sum(-(-n // case["page"]) for n in kv)
        return {"bytes": rows * (stored + width * _size(case["dtype"])) + 4 * pages, "flops": rows * width}
    window, sinks, heads, width = case["window"], case["sinks"], case["heads"], LATENT + case["rope"]
    pairs = rows = 0
    for n, q in zip(kv, other):
        for p in range(n - q, n):
            pairs += min(p + 1, window) + min(sinks, max(0, p + 1 - window))
        if q:
            first = max(0, n - q - window + 1)
            rows += n - first + min(sinks, first)
    tokens, size = sum(other), _size(case["dtype"])
    return {"bytes": rows * width * size + tokens * heads * ((width + LATENT) * size + 4) + 4 * rows // case["page"],
            "flops": pairs * heads * 2 * (width + LATENT)}


# ----------------------------------------------------------------------------- inputs
def _torch_dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _randn(shape, gen, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _table(kv, page, gen):
    """A block table over a random order of the pages, and how many there are."""
    most = max(1, max(-(-n // page) for n in kv))
    blocks = len(kv) * most
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    return order.view(len(kv), most), blocks


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _cumulated(v):
    got = [0]
    for n in v:
        got.append(got[-1] + n)
    return got


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, page = case["op"], case["page"]
    st = {"op": op, "page": page}
    if op == "write_ds_mla":
        tokens, dtype = case["tokens"], _torch_dtype(case["dtype"])
        blocks = -(-tokens // page) + 3
        buffer = torch.zeros(blocks, case["layers"], page, ENTRY, dtype=torch.uint8, device="cuda")
        # latents after their norm, each group of columns with a spread of its own
        spread = torch.exp(torch.randn(tokens, 4, 1, generator=gen, device="cuda"))
        st["kv_c"] = (torch.randn(tokens, 4, GROUP, generator=gen, device="cuda") * spread).view(tokens, LATENT).to(dtype)
        st["k_pe"] = _randn((tokens, ROPE), gen, dtype)
        slots = torch.randperm(blocks * page, generator=gen, device="cuda")[:tokens].to(torch.int64)
        slots[torch.randperm(tokens, generator=gen, device="cuda")[:case["pad"]]] = -1
        return st | {"cache": buffer[:, case["layers"] // 2], "slots": slots}
    kv, other = _lengths(case)
    if op == "read":
        rope, dtype = case["rope"], _torch_dtype(case["dtype"])
        ends = [a + b for a, b in zip(kv, other)]
        st["table"], blocks = _table(ends, page, gen)
        st["format"], width = case["cache"], LATENT + rope
        if case["cache"] == "plain":
            st["cache"] = _randn((blocks, page, width), gen, dtype)
        elif case["cache"] == "e4m3":
            st["cache"] = _randn((blocks, page, width), gen, torch.float32, 32.0).to(torch.float8_e4m3fn)
            st["scale"] = _ints([1 / 32 + 1 / 999], torch.float32)
        else:
            codes = _randn((blocks, page, LATENT), gen, torch.float32, 100.0).clamp(-448, 448).to(torch.float8_e4m3fn)
            scales = torch.rand(blocks, page, 4, generator=gen, device="cuda") / 64 + 1 / 128
            pe = _randn((blocks, page, ROPE), gen, torch.bfloat16)
            st["cache"] = torch.cat([codes.view(torch.uint8), scales.view(torch.uint8), pe.view(torch.uint8)], -1)
        st["out"] = torch.zeros(sum(kv) + case["tail"], width, dtype=dtype, device="cuda")
        return st | {"cu": _ints(_cumulated(kv)), "starts": _ints(other)}
    dtype, heads, rope = _torch_dtype(case["dtype"]), case["heads"], case["rope"]
    width = LATENT + rope
    st["table"], blocks = _table(kv, page, gen)
    tokens = case["batch"] if op == "decode_window" else sum(other) + case["tail"]
    st |= {"cache": _randn((blocks, page, width), gen, dtype), "q": _randn((tokens, heads, width), gen, dtype),
           "kv": _ints(kv), "rope": rope, "scale": 1 / math.sqrt(192), "window": case["window"], "sinks": case["sinks"],
           "span": _span(case, kv, other), "max_q": max(other + [1])}
    st["o"] = torch.zeros(tokens, heads, LATENT, dtype=dtype, device="cuda")
    st["lse"] = torch.zeros(tokens, heads, dtype=torch.float32, device="cuda")
    if op == "prefill_window":
        st["cu"] = _ints(_cumulated(other))
    return st


# ----------------------------------------------------------------------------- one pass
def run(st):
    if own:
        return _own(st)
    return {"write_ds_mla": _write_plain, "read": _read_plain, "decode_window": _decode_plain,
            "prefill_window": _prefill_plain}[st["op"]](st)


def _own(st):
    import mla_latent_kv_11_gb300 as mla
    op = st["op"]
    if op == "write_ds_mla":
        mla.mla_cache_write_ds_mla(st["cache"], st["kv_c"], st["k_pe"], st["slots"])
        return _entries(st["cache"])
    if op == "read":
        if st["format"] == "plain":
            mla.mla_cache_read(st["out"], st["cache"], st["table"], st["cu"], seq_starts=st["starts"])
        elif st["format"] == "e4m3":
            mla.mla_cache_read_fp8(st["out"], st["cache"], st["table"], st["cu"], st["scale"], seq_starts=st["starts"])
        else:
            mla.mla_cache_read_ds_mla(st["out"], st["cache"], st["table"], st["cu"], seq_starts=st["starts"])
        return st["out"]
    if "workspace" not in st:    # kept from the first pass on, as a serving loop keeps it
        tokens, heads = st["q"].shape[:2]
        need = mla.mla_decode_window_workspace_size(tokens, heads, LATENT) if op == "decode_window" else \
            mla.mla_prefill_window_workspace_size(tokens, st["kv"].numel(), heads, LATENT)
        st["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    if op == "decode_window":
        mla.mla_decode_window(st["o"], st["q"], st["cache"], st["table"], st["kv"], LATENT, st["rope"], st["scale"],
                              st["window"], sinks=st["sinks"], lse_out=st["lse"], workspace=st["workspace"])
    else:
        mla.mla_prefill_window(st["o"], st["q"], st["cache"], st["table"], st["cu"], st["kv"], LATENT, st["rope"],
                               st["scale"], st["window"], sinks=st["sinks"], lse_out=st["lse"],
                               workspace=st["workspace"])
    return st["o"], st["lse"]


def _entries(cache):
    """A ds_mla cache as the values it stands for: codes, scales, rope."""
    return {"codes": cache[..., :LATENT].view(torch.float8_e4m3fn),
            "scales": cache[..., LATENT:LATENT + 16].view(torch.float32),
            "rope": cache[..., LATENT + 16:].view(torch.bfloat16)}


def _write_plain(st):
    x = st["kv_c"].float().view(-1, 4, GROUP)
    scale = (x.abs().amax(-1) / E4M3_MAX).clamp_min(TINY)
    codes = (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(-1, LATENT)
    entry = torch.cat([codes.view(torch.uint8), scale.view(torch.uint8), st["k_pe"].to(torch.bfloat16).view(torch.uint8)], -1)
    real = st["slots"] >= 0
    slots = st["slots"][real]
    st["cache"][slots // st["page"], slots % st["page"]] = entry[real]
    return _entries(st["cache"])


def _owner(cu, rows):
    """The sequence of each of `rows` rows, its place in it, and whether it has one."""
    i = torch.arange(rows, device=cu.device, dtype=torch.int32)
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True).clamp_max(cu.numel() - 2)
    return b, i - cu[b], i < cu[-1]


def _read_plain(st):
    out, cache, page = st["out"], st["cache"], st["page"]
    b, i, real = _owner(st["cu"], out.shape[0])
    p = (st["starts"][b] + i).long()
    p = torch.where(real, p, torch.zeros_like(p))
    entry = cache[st["table"][b, p // page].long(), p % page] if st["format"] == "plain" else \
        cache.view(torch.uint8)[st["table"][b, p // page].long(), p % page]
    if st["format"] == "plain":
        rows = entry
    elif st["format"] == "e4m3":
        rows = entry.view(torch.float8_e4m3fn).float() * st["scale"]
    else:
        e = _entries(entry)
        rows = torch.cat([(e["codes"].float().view(-1, 4, GROUP) * e["scales"][..., None]).view(-1, LATENT),
                          e["rope"].float()], -1)
    out.copy_(torch.where(real[:, None], rows.to(out.dtype), out))
    return out


def _attend(q, keys, visible, scale):
    """o [B, N, LATENT] and lse [B, N] of queries q [B, N, E] over keys [B, n, E]; visible [B, N or broadcast, n]."""
    keys = keys.float()
    s = torch.bmm(q.float(), keys.transpose(1, 2)).mul_(scale).masked_fill_(~visible, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p, keys[..., :LATENT]) / torch.where(total == 0, torch.ones_like(total), total)
    return o, (m + total.log())[..., 0]


def _keys(st, first, n):
    """Positions [B, sinks + n] of the first `sinks` rows and of `n` rows from `first`, and the rows there."""
    dev = first.device
    b = first.numel()
    at = torch.cat([torch.arange(st["sinks"], device=dev).expand(b, -1),
                    first[:, None] + torch.arange(n, device=dev)], 1)
    inside = at.clamp_max(st["table"].shape[1] * st["page"] - 1)
    blocks = st["table"].gather(1, inside // st["page"]).long()
    return at, st["cache"][blocks, inside % st["page"]]


def _decode_plain(st):
    kv = st["kv"].long()
    first = (kv - st["window"]).clamp_min(st["sinks"])
    at, keys = _keys(st, first, st["span"])
    visible = (at < kv[:, None])[:, None]
    o, lse = _attend(st["q"], keys, visible, st["scale"])
    st["o"].copy_(o)
    st["lse"].copy_(lse)
    return st["o"], st["lse"]


def _prefill_plain(st):
    cu, kv, heads, max_q = st["cu"].long(), st["kv"].long(), st["q"].shape[1], st["max_q"]
    lens = cu[1:] - cu[:-1]
    first = (kv - lens - st["window"] + 1).clamp_min(st["sinks"])
    at, keys = _keys(st, first, st["span"])
    i = torch.arange(max_q, device=cu.device)
    q = st["q"][(cu[:-1, None] + i).clamp_max(st["q"].shape[0] - 1)]
    p = (kv - lens)[:, None, None] + i[:, None]
    k = at[:, None]
    visible = (k <= p) & ((k < st["sinks"]) | (k > p - st["window"])) & (k < kv[:, None, None])
    visible = visible[:, :, None].expand(-1, -1, heads, -1).reshape(len(kv), max_q * heads, -1)
    o, lse = _attend(q.reshape(len(kv), max_q * heads, -1), keys, visible, st["scale"])
    b, place, real = _owner(st["cu"], st["q"].shape[0])
    place = place.clamp_max(max_q - 1)
    o = o.view(len(kv), max_q, heads, LATENT)[b, place]
    lse = lse.view(len(kv), max_q, heads)[b, place]
    st["o"].copy_(torch.where(real[:, None, None], o.to(st["o"].dtype), st["o"]))
    st["lse"].copy_(torch.where(real[:, None], lse, st["lse"]))
    return st["o"], st["lse"]


# ----------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op, page = case["op"], case["page"]
    if op == "write_ds_mla":
        return _write_exact(st)
    kv, other = _lengths(case)
    if op == "read":
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        at = 0
        for b, (n, start) in enumerate(zip(kv, other)):
            rows = torch.arange(start, start + n, device="cuda")
            out[at:at + n] = _values64(st, st["table"][b].long()[rows // page] * page + rows % page)
            at += n
        return out
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    if op == "decode_window":
        lse[[b for b, n in enumerate(kv) if n == 0]] = -math.inf
    rows64 = st["cache"].view(-1, st["cache"].shape[-1])
    at = 0
    for b, (n, q) in enumerate(zip(kv, other)):
        base = b if op == "decode_window" else at
        at += q
        step = max(1, 16384 // case["heads"])
        for t in range(0, q, step):
            tokens = range(t, min(q, t + step))
            lo, hi = n - q + tokens[0], n - q + tokens[-1]     # positions of the first and last query
            low = max(0, lo - case["window"] + 1)
            rows = torch.tensor([*range(min(case["sinks"], low)), *range(low, hi + 1)], device="cuda")
            k = rows64[st["table"][b].long()[rows // page] * page + rows % page].double()
            pos = torch.arange(lo, hi + 1, device="cuda")[:, None]
            seen = (rows <= pos) & ((rows > pos - case["window"]) | (rows < case["sinks"]))
            x = st["q"][base + t:base + tokens[-1] + 1].double()
            s = torch.einsum("the,ne->thn", x, k) * st["scale"]
            s = torch.where(seen[:, None], s, -math.inf)
            lse[base + t:base + tokens[-1] + 1] = torch.logsumexp(s, -1)
            o[base + t:base + tokens[-1] + 1] = torch.einsum("thn,nl->thl", torch.softmax(s, -1), k[:, :LATENT])
    return o, lse


def _values64(st, at):
    if st["format"] == "plain":
        return st["cache"].view(-1, st["cache"].shape[-1])[at].double()
    raw = st["cache"].view(torch.uint8).view(-1, st["cache"].shape[-1])[at]
    codes = raw[:, :LATENT] if st["format"] == "ds_mla" else raw
    sign = 1.0 - 2.0 * (codes >> 7).double()
    power, part = ((codes >> 3) & 15).double(), (codes & 7).double()
    v = sign * torch.where(power == 0, part / 8 * 2.0 ** -6, (1 + part / 8) * torch.exp2(power - 7))
    if st["format"] == "e4m3":
        return v * st["scale"].double()
    scales = raw[:, LATENT:LATENT + 16].contiguous().view(torch.float32).double().repeat_interleave(GROUP, 1)
    return torch.cat([v * scales, raw[:, LATENT + 16:].contiguous().view(torch.bfloat16).double()], 1)


def _write_exact(st):
    rows = st["cache"].shape[0] * st["page"]
    codes = torch.zeros(rows, LATENT, dtype=torch.float64, device="cuda")
    scales = torch.zeros(rows, 4, dtype=torch.float64, device="cuda")
    rope = torch.zeros(rows, ROPE, dtype=torch.float64, device="cuda")
    keep = (st["slots"] >= 0).nonzero()[:, 0]
    slots, x = st["slots"][keep], st["kv_c"][keep].double().unflatten(1, (4, GROUP))
    scale = torch.clamp(torch.linalg.vector_norm(x, math.inf, -1) / E4M3_MAX, min=TINY)
    y = x / scale.float().double()[..., None]     # by the scale as it is stored
    # e4m3: steps of 2^(exponent - 3), no exponent below -6, halves to even
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(y.abs(), min=2.0 ** -20))), min=-6) - 3)
    codes[slots] = torch.clamp(torch.round(y / step) * step, -E4M3_MAX, E4M3_MAX).flatten(1)
    scales[slots], rope[slots] = scale, st["k_pe"][keep].double()
    n = st["cache"].shape[0]
    return {"codes": codes.view(n, st["page"], -1), "scales": scales.view(n, st["page"], -1),
            "rope": rope.view(n, st["page"], -1)}

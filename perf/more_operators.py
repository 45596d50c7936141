"""Cases of the operators at both ends of a cache row's life, each in a plain form and as the library's call.

  norm_rope      per-head norms and the position rotation of new queries, and of new rows as they enter the cache
  mass_decode    what one query token a sequence gives each cached row, summed over heads, added to the row's mass
  mass_prefill   the same for a chunk of causal query tokens a sequence
  evict          the heaviest rows of each sequence kept and moved together, the rest dropped

`own` false: elementary torch operations in 32 bits. `own` true: the library's calls.
"""
import math
import random

import torch

own = False

ENTRY, GROUP = 656, 128
E4M3_MAX = 448.0
TINY = 2.0 ** -126          # the smallest scale of a group
EPS = 1e-6


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one sequence in a decode step, queries without a norm of their own: latency
        dict(name="norm rope 1 token", op="norm_rope", part="both", format="plain", dtype="bf16", tokens=1, pad=0, heads=128,
             nope=128, rope=64, latent=512, q_norm=False, per_head=False, interleaved=True, page=64, layers=1),
        # a decode step of 64 sequences, norms of the queries' heads, halves rotated, one layer of a buffer of three
        dict(name="norm rope 64 tokens", op="norm_rope", part="both", format="plain", dtype="bf16", tokens=64, pad=0,
             heads=128, nope=128, rope=64, latent=512, q_norm=True, per_head=False, interleaved=False, page=64, layers=3),
        # a chunk of prompts: queries and rows
        dict(name="norm rope 4096 tokens", op="norm_rope", part="both", format="plain", dtype="bf16", tokens=4096, pad=0,
             heads=128, nope=128, rope=64, latent=512, q_norm=True, per_head=True, interleaved=True, page=64, layers=1),
        # a long prompt's rows into an fp8 ds_mla cache from float32 activations, an odd count with padding slots
        dict(name="norm rope ds_mla 20011 f32", op="norm_rope", part="write", format="ds_mla", dtype="f32", tokens=20011,
             pad=111, heads=0, nope=0, rope=64, latent=512, q_norm=False, per_head=False, interleaved=True, page=64,
             layers=1),
        # one sequence of a chat: latency
        dict(name="mass decode 1 x 700", op="mass_decode", dtype="bf16", heads=128, latent=512, rope=64, batch=1, kv_min=700,
             kv_max=700, empty=False, decay=1.0, page=64, lens=1),
        # 64 sequences of 1K to 16K rows
        dict(name="mass decode 64 x 1K-16K", op="mass_decode", dtype="bf16", heads=128, latent=512, rope=64, batch=64,
             kv_min=1024, kv_max=16384, empty=False, decay=1.0, page=64, lens=2),
        # float32 with 16 heads, an empty sequence, a mass that fades
        dict(name="mass decode f32 5 x 256", op="mass_decode", dtype="f32", heads=16, latent=512, rope=64, batch=5, kv_min=1,
             kv_max=256, empty=True, decay=0.9375, page=64, lens=3),
        # four prompts' chunks of 512 tokens over 1K to 8K rows
        dict(name="mass prefill 4 x 512", op="mass_prefill", dtype="bf16", heads=128, latent=512, rope=64, batch=4, q_min=512,
             q_max=512, kv_min=1024, kv_max=8192, tail=0, decay=1.0, page=64, lens=4),
        # the last 32 tokens of one long prompt weigh all of its rows before most are dropped; no rope part
        dict(name="mass prefill 32 over 16K", op="mass_prefill", dtype="bf16", heads=64, latent=512, rope=0, batch=1,
             q_min=32, q_max=32, kv_min=16001, kv_max=16001, tail=3, decay=0.0, page=64, lens=5),
        # one short sequence cut to 512 rows, in its own pages: latency
        dict(name="evict 1 x 700", op="evict", format="plain", dtype="bf16", width=576, batch=1, kv_min=700, kv_max=700,
             budget=512, sinks=4, recent=64, page=64, place="same", lens=6),
        # 64 sequences of 1K to 8K rows cut to 2K rows, in their own pages
        dict(name="evict 64 x 1K-8K", op="evict", format="plain", dtype="bf16", width=576, batch=64, kv_min=1024, kv_max=8192,
             budget=2048, sinks=4, recent=256, page=64, place="same", lens=7),
        # ragged sequences of an fp8 ds_mla cache, some shorter than the budget, into other pages (theirs are shared)
        dict(name="evict ds_mla ragged", op="evict", format="ds_mla", dtype="bf16", width=ENTRY, batch=37, kv_min=0,
             kv_max=1999, budget=777, sinks=1, recent=33, page=16, place="other", lens=8),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _drawn(rng):
    op = rng.choice(["norm_rope", "mass_decode", "mass_prefill", "evict"])
    page, lens = rng.choice([16, 32, 64, 64, 128]), rng.randint(10, 1 << 30)
    if op == "norm_rope":
        form = rng.choice(["plain", "plain", "e4m3", "ds_mla"])
        part = rng.choice(["both", "both", "q", "write"]) if form == "plain" else "write"
        tokens = _log(rng, 1, 40000) if part == "write" else _log(rng, 1, 4096)
        heads, nope, rope = rng.choice([(128, 128, 64), (64, 128, 64), (64, 256, 0), (16, 128, 64), (20, 128, 64)])
        return dict(op=op, part=part, format=form, dtype=rng.choice(["bf16", "bf16", "f32"]), tokens=tokens,
                    pad=rng.randint(0, tokens // 8), heads=heads, nope=nope, rope=64 if form == "ds_mla" else rope,
                    latent=512, q_norm=rope == 0 or rng.random() < 0.6, per_head=rng.random() < 0.3,
                    interleaved=rng.random() < 0.5, page=page, layers=rng.choice([1, 1, 3]))
    if op == "evict":
        form, kv = rng.choice(["plain", "plain", "e4m3", "ds_mla"]), _log(rng, 1, 16384)
        dtype = rng.choice(["bf16", "bf16", "f32"]) if form == "plain" else "bf16"
        budget = _log(rng, 1, kv)
        sinks = rng.randint(0, min(64, budget))
        return dict(op=op, format=form, dtype=dtype, width=ENTRY if form == "ds_mla" else rng.choice([576, 512]),
                    batch=_log(rng, 1, 64), kv_min=rng.randint(0, kv), kv_max=kv, budget=budget, sinks=sinks,
                    recent=rng.randint(0, budget - sinks), page=page, place=rng.choice(["same", "other"]), lens=lens)
    heads, rope = rng.choice([(128, 64), (128, 64), (64, 64), (64, 0), (16, 64), (20, 64)])
    decay = rng.choice([1.0, 1.0, 0.0, 0.9375, rng.random()])
    if op == "mass_decode":
        if rng.random() < 0.15:
            kv = _log(rng, 1, 512)
            return dict(op=op, dtype="f32", heads=16, latent=512, rope=64, batch=_log(rng, 1, 8), kv_min=rng.randint(1, kv),
                        kv_max=kv, empty=rng.random() < 0.5, decay=decay, page=page, lens=lens)
        kv = _log(rng, 1, 16384)
        return dict(op=op, dtype="bf16", heads=heads, latent=512, rope=rope, batch=_log(rng, 1, 96),
                    kv_min=rng.randint(1, kv), kv_max=kv, empty=rng.random() < 0.2, decay=decay, page=page, lens=lens)
    q = _log(rng, 1, 1024)
    kv = max(q, _log(rng, 1, 16384))
    return dict(op=op, dtype="bf16", heads=heads, latent=512, rope=rope, batch=_log(rng, 1, 8), q_min=rng.randint(1, q),
                q_max=q, kv_min=q, kv_max=kv, tail=rng.choice([0, 0, 2]), decay=decay, page=page, lens=lens)


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
    """(rows in the cache, query tokens) of every sequence of a case."""
    r = random.Random(case["lens"])
    kv = [r.randint(case["kv_min"], case["kv_max"]) for _ in range(case["batch"])]
    if case["op"] == "mass_prefill":
        return kv, [min(n, r.randint(case["q_min"], case["q_max"])) for n in kv]
    if case.get("empty"):
        kv[0] = 0
    return kv, [min(1, n) for n in kv]


def _plain_size(case):
    """Values of the plain form's largest intermediate."""
    if case["op"] == "norm_rope":
        return case["tokens"] * (case["heads"] * (case["nope"] + case["rope"]) + case["latent"] + case["rope"])
    kv, q = _lengths(case)
    if case["op"] == "evict":
        return case["batch"] * max(kv + [1]) * case["width"]
    return case["batch"] * case["heads"] * max(q + [1]) * max(kv + [1])


def _size(dtype):
    return 4 if dtype == "f32" else 2


def _row_bytes(case):
    if case["format"] == "ds_mla":
        return ENTRY
    width = case["width"] if case["op"] == "evict" else case["latent"] + case["rope"]
    return width * (1 if case["format"] == "e4m3" else _size(case["dtype"]))


def work(case):
    op = case["op"]
    if op == "norm_rope":
        size, tokens, nope, rope = _size(case["dtype"]), case["tokens"], case["nope"], case["rope"]
        total, flops = tokens * (8 + 4 * rope), 0
        if case["part"] != "write":     # without a norm only the rotated columns are read and written
            cols = tokens * case["heads"] * ((nope + rope) if case["q_norm"] else rope)
            total, flops = total + 2 * cols * size, 4 * cols
        if case["part"] != "q":
            rows = tokens - case["pad"]
            total += rows * ((case["latent"] + rope) * size + _row_bytes(case)) + 8 * tokens
            flops += rows * 4 * (case["latent"] + rope)
        return {"bytes": total, "flops": flops}
    kv, q = _lengths(case)
    if op == "evict":
        moved = sum(min(n, case["budget"]) - min(n, case["sinks"]) for n in kv
                    if n > case["budget"] or case["place"] == "other")
        return {"bytes": 2 * moved * _row_bytes(case) + 8 * sum(kv) + 4 * case["batch"] * (case["budget"] + 2), "flops": 0}
    width, heads, size = case["latent"] + case["rope"], case["heads"], _size(case["dtype"])
    pairs = sum(k * (n - k) + k * (k + 1) // 2 for n, k in zip(kv, q))
    rows, tokens = sum(n for n, k in zip(kv, q) if k), sum(q)
    return {"bytes": rows * (width * size + (4 if case["decay"] == 0 else 8)) + tokens * heads * (width * size + 4) +
            4 * rows // case["page"], "flops": pairs * heads * 2 * width}


# ----------------------------------------------------------------------------- inputs
def _torch_dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _randn(shape, gen, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _cumulated(v):
    got = [0]
    for n in v:
        got.append(got[-1] + n)
    return got


def _rows(form, shape, width, dtype, gen):
    """A cache of `shape` rows in its format."""
    if form == "plain":
        return _randn((*shape, width), gen, dtype)
    if form == "e4m3":
        return _randn((*shape, width), gen, torch.float32, 32.0).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = _randn((*shape, 512), gen, torch.float32, 100.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = torch.rand(*shape, 4, generator=gen, device="cuda") / 64 + 1 / 128
    return torch.cat([codes.view(torch.uint8), scales.view(torch.uint8),
                      _randn((*shape, 64), gen, torch.bfloat16).view(torch.uint8)], -1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, page = case["op"], case["page"]
    st = {"op": op, "page": page}
    if op == "norm_rope":
        return st | _prepare_norm_rope(case, gen)
    kv, q = _lengths(case)
    most = max(1, max(-(-n // page) for n in kv))
    batch, blocks = case["batch"], case["batch"] * most
    # block tables over a random order of the pages
    order = torch.randperm(2 * blocks if op == "evict" else blocks, generator=gen, device="cuda").to(torch.int32)
    st |= {"table": order[:blocks].view(batch, most), "kv": _ints(kv), "most": max(kv + [1])}
    dtype = _torch_dtype(case["dtype"])
    if op == "evict":
        # masses of many sizes, as attention gives them; rows just written have none yet
        mass = torch.exp(3 * torch.randn(batch, st["most"], generator=gen, device="cuda"))
        mass[torch.rand(batch, st["most"], generator=gen, device="cuda") < 0.1] = 0
        st |= {"budget": case["budget"], "sinks": case["sinks"], "recent": case["recent"], "format": case["format"],
               "cache": _rows(case["format"], (2 * blocks, page), case["width"], dtype, gen), "mass": mass,
               "table_out": order[blocks:].view(batch, most) if case["place"] == "other" else st["table"],
               "mass_out": torch.zeros_like(mass), "kv_out": torch.zeros_like(st["kv"]),
               "kept": torch.zeros(batch, case["budget"], dtype=torch.int32, device="cuda")}
        return st
    width, tokens = case["latent"] + case["rope"], batch if op == "mass_decode" else sum(q) + case["tail"]
    st |= {"cache": _rows("plain", (blocks, page), width, dtype, gen), "q": _randn((tokens, case["heads"], width), gen, dtype),
           "scale": 1 / math.sqrt(192), "decay": case["decay"], "max_q": max(q + [1]),
           "mass": torch.rand(batch, st["most"], generator=gen, device="cuda") * 4}
    if op == "mass_prefill":
        st["cu"] = _ints(_cumulated(q))
    # the log-sum-exp of each query's row, as the attention before it leaves it
    s = _scores(st)
    lse = torch.logsumexp(s, -1)
    st["lse"] = lse if op == "mass_decode" else _by_token(st, lse, math.inf)
    return st


def _prepare_norm_rope(case, gen):
    dtype, tokens, page = _torch_dtype(case["dtype"]), case["tokens"], case["page"]
    heads, nope, rope, latent = case["heads"], case["nope"], case["rope"], case["latent"]
    st = {"part": case["part"], "format": case["format"], "interleaved": case["interleaved"], "latent": latent, "rope": rope,
          "nope": nope, "q_weight": None}
    # positions anywhere in a context of 128K; the table's angles in 64 bits
    st["positions"] = torch.randint(0, 1 << 17, (tokens,), generator=gen, device="cuda")
    st["cos_sin"] = _cos_sin(1 << 17, rope)
    if case["part"] != "write":
        # heads of different loudness
        loud = torch.exp(torch.randn(tokens, heads, 1, generator=gen, device="cuda") / 2)
        st["q"] = (_randn((tokens, heads, nope + rope), gen, torch.float32) * loud).to(dtype)
        if case["q_norm"]:
            shape = (heads, nope + rope) if case["per_head"] else (nope + rope,)
            st["q_weight"] = (1 + _randn(shape, gen, torch.float32, 0.2)).to(dtype)
            st["q_nope"] = torch.zeros(tokens, heads, nope, dtype=dtype, device="cuda")
        else:
            st["q_nope"] = st["q"][..., :nope]      # nothing to do there
        st["q_cat"] = torch.zeros(tokens, heads, latent + rope, dtype=dtype, device="cuda")
    if case["part"] != "q":
        blocks = -(-tokens // page) + 3
        spread = torch.exp(torch.randn(tokens, 1, generator=gen, device="cuda"))
        st["kv"] = (_randn((tokens, latent + rope), gen, torch.float32) * spread).to(dtype)
        st["kv_weight"] = (1 + _randn((latent,), gen, torch.float32, 0.2)).to(dtype)
        kind, width = (dtype, latent + rope) if case["format"] == "plain" else \
            (torch.uint8, ENTRY if case["format"] == "ds_mla" else latent + rope)
        st["cache"] = torch.zeros(blocks, case["layers"], page, width, dtype=kind, device="cuda")[:, case["layers"] // 2]
        slots = torch.randperm(blocks * page, generator=gen, device="cuda")[:tokens].to(torch.int64)
        slots[torch.randperm(tokens, generator=gen, device="cuda")[:case["pad"]]] = -1
        st["slots"] = slots
        st["scale"] = _ints([1 / 64 + 1 / 999], torch.float32)
    return st


def _cos_sin(positions, rope):
    i = torch.arange(rope // 2, dtype=torch.float64, device="cuda")
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2 * i / max(1, rope))
    return torch.cat([angle.cos(), angle.sin()], -1).float()


# ----------------------------------------------------------------------------- one pass
def run(st):
    if own:
        return _own(st)
    return {"norm_rope": _norm_rope_plain, "evict": _evict_plain}.get(st["op"], _mass_plain)(st)


def _own(st):
    import mla_latent_kv_11_gb300 as mla
    op = st["op"]
    if op == "norm_rope":
        common = dict(eps=EPS, interleaved=st["interleaved"])
        if st["part"] == "q":
            mla.mla_norm_rope_q(st["q_nope"], st["q_cat"][..., st["latent"]:], st["q"], st["q_weight"], st["positions"],
                                st["cos_sin"], **common)
        elif st["part"] == "both":
            mla.mla_norm_rope_q_cache_write(st["q_nope"], st["q_cat"][..., st["latent"]:], st["q"], st["q_weight"], st["cache"],
                                            st["kv"], st["kv_weight"], st["positions"], st["cos_sin"], st["slots"], **common)
        elif st["format"] == "plain":
            mla.mla_norm_rope_cache_write(st["cache"], st["kv"], st["kv_weight"], st["positions"], st["cos_sin"],
                                          st["slots"], **common)
        elif st["format"] == "e4m3":
            mla.mla_norm_rope_cache_write_fp8(st["cache"], st["kv"], st["kv_weight"], st["positions"], st["cos_sin"],
                                              st["slots"], st["scale"], **common)
        else:
            mla.mla_norm_rope_cache_write_ds_mla(st["cache"], st["kv"], st["kv_weight"], st["positions"], st["cos_sin"],
                                                 st["slots"], **common)
        return _norm_rope_outputs(st)
    if "workspace" not in st:    # kept from the first pass on, as a serving loop keeps it
        need = {"mass_decode": lambda: 0, "mass_prefill": lambda: mla.mla_prefill_mass_workspace_size(),
                "evict": lambda: mla.mla_cache_evict_workspace_size(st["kv"].numel(), st["mass"].shape[1], st["budget"])}[op]()
        st["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    if op == "mass_decode":
        mla.mla_decode_mass(st["mass"], st["q"], st["cache"], st["table"], st["kv"], st["lse"], st["scale"],
                            decay=st["decay"])
        return st["mass"]
    if op == "mass_prefill":
        mla.mla_prefill_mass(st["mass"], st["q"], st["cache"], st["table"], st["cu"], st["kv"], st["lse"], st["scale"],
                             decay=st["decay"], workspace=st["workspace"])
        return st["mass"]
    mla.mla_cache_evict(st["cache"], st["mass"], st["table"], st["kv"], st["budget"], st["kv_out"], sinks=st["sinks"],
                        recent=st["recent"], block_table_out=st["table_out"], mass_out=st["mass_out"], kept_out=st["kept"],
                        workspace=st["workspace"])
    return _evict_outputs(st)


def _values(cache, form):
    """A cache as the values it stands for."""
    if form == "plain":
        return cache
    if form == "e4m3":
        return cache.view(torch.float8_e4m3fn)
    return {"codes": cache[..., :512].view(torch.float8_e4m3fn), "scales": cache[..., 512:528].view(torch.float32),
            "rope": cache[..., 528:].view(torch.bfloat16)}


def _norm_rope_outputs(st):
    got = []
    if st["part"] != "write":
        got += [st["q_nope"], st["q_cat"][..., st["latent"]:]] if st["q_weight"] is not None else [st["q_cat"][..., st["latent"]:]]
    if st["part"] != "q":
        got.append(_values(st["cache"], st["format"]))
    return got


def _norm(x, weight):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _rotate(x, cos_sin, interleaved):
    """x [T, ..., R] rotated by its token's angles cos_sin [T, R]."""
    if x.shape[-1] == 0:
        return x
    half = x.shape[-1] // 2
    cos_sin = cos_sin.view(x.shape[0], *[1] * (x.dim() - 2), 2 * half)
    c, s = cos_sin[..., :half], cos_sin[..., half:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    a, b = a * c - b * s, b * c + a * s
    return torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)


def _norm_rope_plain(st):
    angles, nope, latent = st["cos_sin"][st["positions"]], st["nope"], st["latent"]
    if st["part"] != "write":
        if st["q_weight"] is not None:
            x = _norm(st["q"].float(), st["q_weight"])
            st["q_nope"].copy_(x[..., :nope])
            pe = x[..., nope:]
        else:
            pe = st["q"][..., nope:].float()
        st["q_cat"][..., latent:] = _rotate(pe, angles, st["interleaved"]).to(st["q_cat"].dtype)
    if st["part"] != "q":
        x = st["kv"].float()
        c_kv, k_pe = _norm(x[:, :latent], st["kv_weight"]), _rotate(x[:, latent:], angles, st["interleaved"])
        if st["format"] == "plain":
            rows = torch.cat([c_kv, k_pe], -1).to(st["cache"].dtype)
        elif st["format"] == "e4m3":
            rows = (torch.cat([c_kv, k_pe], -1) / st["scale"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            x = c_kv.view(-1, 4, GROUP)
            scale = (x.abs().amax(-1) / E4M3_MAX).clamp_min(TINY)
            codes = (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(-1, latent)
            rows = torch.cat([codes.view(torch.uint8), scale.view(torch.uint8), k_pe.to(torch.bfloat16).view(torch.uint8)], -1)
        real = st["slots"] >= 0
        slots = st["slots"][real]
        st["cache"][slots // st["page"], slots % st["page"]] = rows[real]
    return _norm_rope_outputs(st)


def _scores(st):
    """Scaled scores [B, query rows, rows] of every sequence's queries, -inf where a row is not attended."""
    kv, most, page = st["kv"].long(), st["most"], st["page"]
    at = torch.arange(most, device=kv.device)
    keys = st["cache"][st["table"][:, at // page].long(), at % page].float()
    if st["op"] == "mass_decode":
        q, visible = st["q"].float(), (at < kv[:, None])[:, None]
    else:
        cu, heads, max_q = st["cu"].long(), st["q"].shape[1], st["max_q"]
        lens, i = cu[1:] - cu[:-1], torch.arange(max_q, device=kv.device)
        q = st["q"][(cu[:-1, None] + i).clamp_max(st["q"].shape[0] - 1)].flatten(1, 2).float()
        p = (kv - lens)[:, None] + i
        visible = (at <= p[..., None]) & (i < lens[:, None])[..., None]
        visible = visible[:, :, None].expand(-1, -1, heads, -1).flatten(1, 2)
    return torch.bmm(q, keys.transpose(1, 2)).mul_(st["scale"]).masked_fill_(~visible, -math.inf)


def _by_token(st, x, fill):
    """[B, max_q * H] of a prefill as [tokens, H]; `fill` behind the last sequence."""
    cu, tokens = st["cu"].long(), st["q"].shape[0]
    i = torch.arange(tokens, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True).clamp_max(cu.numel() - 2)
    x = x.view(cu.numel() - 1, st["max_q"], -1)[b, (i - cu[b]).clamp(0, st["max_q"] - 1)]
    return torch.where((i < cu[-1])[:, None], x, fill)


def _mass_plain(st):
    s, mass, kv = _scores(st), st["mass"], st["kv"]
    has = kv > 0
    if st["op"] == "mass_prefill":
        cu, lens = st["cu"].long(), st["cu"][1:] - st["cu"][:-1]
        lse = st["lse"][(cu[:-1, None] + torch.arange(st["max_q"], device=kv.device)).clamp_max(st["q"].shape[0] - 1)].flatten(1)
        has = has & (lens > 0)
    else:
        lse = st["lse"]
    lse = torch.where(lse == -math.inf, math.inf, lse)      # a query that attends nothing gives nothing
    got = s.sub_(lse[..., None]).exp_().sum(1)
    new = got if st["decay"] == 0 else mass * st["decay"] + got
    rows = (torch.arange(st["most"], device=kv.device) < kv[:, None]) & has[:, None]
    mass.copy_(torch.where(rows, new, mass))
    return mass


def _evict_outputs(st):
    return {"cache": _values(st["cache"], st["format"]), "mass": st["mass_out"], "kv": st["kv_out"], "kept": st["kept"]}


def _evict_plain(st):
    mass, kv, budget, page = st["mass"], st["kv"].long()[:, None], st["budget"], st["page"]
    at = torch.arange(st["most"], device=mass.device)[None]
    held = (at < st["sinks"]) | (at >= kv - st["recent"])
    rank = torch.where(held, math.inf, mass).masked_fill(at >= kv, -math.inf)
    first = torch.sort(rank, dim=1, descending=True, stable=True).indices      # ties: the lowest row first
    keep = torch.zeros_like(held).scatter_(1, first[:, :budget], True) & (at < kv)
    left = kv.clamp_max(budget)
    rows = torch.sort((~keep).to(torch.uint8), dim=1, stable=True).indices[:, :budget]      # the kept rows in order
    j = torch.arange(rows.shape[1], device=mass.device)[None]
    real = j < left
    st["kept"].fill_(-1)
    st["kept"][:, :rows.shape[1]] = torch.where(real, rows, -1).to(torch.int32)
    st["kv_out"].copy_(left[:, 0])
    out = torch.where(at < kv, 0.0, st["mass_out"])
    out[:, :rows.shape[1]] = torch.where(real, mass.gather(1, rows), out[:, :rows.shape[1]])
    st["mass_out"].copy_(out)
    src = st["cache"][st["table"].gather(1, rows // page).long(), rows % page][real]
    to = st["table_out"].gather(1, (j // page).expand_as(rows)).long()
    st["cache"][to[real], (j % page).expand_as(rows)[real]] = src
    return _evict_outputs(st)


# ----------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm_rope":
        return _norm_rope_exact(st)
    kv, q = _lengths(case)
    if case["op"] == "evict":
        return _evict_exact(st, kv)
    rows64 = st["cache"].view(-1, st["cache"].shape[-1])
    mass, page, heads, at = st["mass"].double(), st["page"], case["heads"], 0
    for b, (n, k) in enumerate(zip(kv, q)):
        base = b if case["op"] == "mass_decode" else at
        at += k
        if n == 0 or k == 0:
            continue
        pos = torch.arange(n, device="cuda")
        keys = rows64[st["table"][b].long()[pos // page] * page + pos % page].double()
        total = torch.zeros(n, dtype=torch.float64, device="cuda")
        step = max(1, 16384 // heads)
        for t in range(0, k, step):
            m = min(step, k - t)
            x = st["q"][base + t:base + t + m].double().flatten(0, 1) @ keys.T * st["scale"]
            w = torch.exp(x - st["lse"][base + t:base + t + m].double().flatten()[:, None]).view(m, heads, n).sum(1)
            seen = pos <= torch.arange(n - k + t, n - k + t + m, device="cuda")[:, None]
            total += (w * seen).sum(0)
        mass[b, :n] = total if case["decay"] == 0 else mass[b, :n] * case["decay"] + total
    return mass


def _evict_exact(st, kv):
    page, budget = st["page"], st["budget"]
    form, cache, table, other = st["format"], st["cache"].clone(), st["table"].tolist(), st["table_out"].tolist()
    flat, mass_out = cache.view(-1, cache.shape[-1]), st["mass_out"].double()
    left, kept_all = [], []
    for b, n in enumerate(kv):
        mass = st["mass"][b].tolist()
        kept = list(range(n))
        if n > budget:
            held = [t for t in kept if t < st["sinks"] or t >= n - st["recent"]]
            free = sorted((t for t in kept if st["sinks"] <= t < n - st["recent"]), key=lambda t: (-mass[t], t))
            kept = sorted(held + free[:budget - len(held)])
        left.append(len(kept))
        kept_all.append(kept + [-1] * (budget - len(kept)))
        mass_out[b, :n] = 0
        if kept:
            mass_out[b, :len(kept)] = torch.tensor([mass[t] for t in kept], dtype=torch.float64)
            src = _ints([table[b][t // page] * page + t % page for t in kept], torch.int64)
            to = _ints([other[b][j // page] * page + j % page for j in range(len(kept))], torch.int64)
            flat[to] = flat[src]
    if form == "plain":
        values = cache.double()
    elif form == "e4m3":
        values = _e4m3_values(cache)
    else:
        values = {"codes": _e4m3_values(cache[..., :512]), "scales": cache[..., 512:528].contiguous().view(torch.float32).double(),
                  "rope": cache[..., 528:].contiguous().view(torch.bfloat16).double()}
    return {"cache": values, "mass": mass_out, "kv": _ints(left), "kept": _ints(kept_all)}


def _e4m3_values(codes):
    sign = 1.0 - 2.0 * (codes >> 7).double()
    power, part = ((codes >> 3) & 15).double(), (codes & 7).double()
    return sign * torch.where(power == 0, part / 8 * 2.0 ** -6, (1 + part / 8) * torch.exp2(power - 7))


def _e4m3_nearest(y):
    """y rounded to the nearest e4m3 value: steps of 2^(exponent - 3), no exponent below -6, halves to even."""
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(y.abs(), min=2.0 ** -20))), min=-6) - 3)
    return torch.clamp(torch.round(y / step) * step, -E4M3_MAX, E4M3_MAX)


def _turned(x, angles, interleaved):
    """Pairs of x as complex numbers, times the unit numbers of their angles."""
    half = x.shape[-1] // 2
    if half == 0:
        return x
    turn = torch.complex(angles[:, :half].double(), angles[:, half:].double())
    turn = turn if x.dim() == 2 else turn[:, None]
    if interleaved:
        return torch.view_as_real(torch.view_as_complex(x.double().unflatten(-1, (half, 2)).contiguous()) * turn).flatten(-2)
    z = torch.complex(x[..., :half].double().contiguous(), x[..., half:].double().contiguous()) * turn
    return torch.cat([z.real, z.imag], -1)


def _norm_rope_exact(st):
    got, angles, latent, nope = [], st["cos_sin"].index_select(0, st["positions"]), st["latent"], st["nope"]
    if st["part"] != "write":
        x = st["q"].double()
        if st["q_weight"] is not None:
            x = x * st["q_weight"].double() / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
            got.append(x[..., :nope])
        got.append(_turned(x[..., nope:], angles, st["interleaved"]))
    if st["part"] != "q":
        keep = (st["slots"] >= 0).nonzero()[:, 0]
        slots, x = st["slots"][keep], st["kv"][keep].double()
        c = x[:, :latent]
        c = c * st["kv_weight"].double() / torch.sqrt((c * c).sum(-1, keepdim=True) / latent + EPS)
        pe = _turned(x[:, latent:], angles[keep], st["interleaved"])
        blocks, page = st["cache"].shape[:2]

        def placed(v):
            full = torch.zeros(blocks * page, v.shape[-1], dtype=torch.float64, device="cuda")
            full[slots] = v
            return full.view(blocks, page, -1)

        if st["format"] == "plain":
            got.append(placed(torch.cat([c, pe], -1)))
        elif st["format"] == "e4m3":
            got.append(placed(_e4m3_nearest(torch.cat([c, pe], -1) / st["scale"].double())))
        else:
            g = c.unflatten(1, (4, GROUP))
            scale = torch.clamp(torch.linalg.vector_norm(g, math.inf, -1) / E4M3_MAX, min=TINY)
            got.append({"codes": placed(_e4m3_nearest(g / scale.float().double()[..., None]).flatten(1)),
                        "scales": placed(scale), "rope": placed(pe)})
    return got

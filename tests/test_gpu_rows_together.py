"""The operators around the attention together, as a serving loop runs them: new rows and queries normalised and rotated,
absorbed, written, attended; the rows weighed; the lightest dropped when the cache passes its budget; and on."""
import math

import pytest
import torch

import mass_ref
import norm_rope_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
POSITIONS = 400


def attend(q, rows, latent, scale):
    """o [H, latent] and lse [H] of one query over rows, in 64 bits; the sum of |weight * value|."""
    s = q.double() @ rows.double().T * scale
    p = torch.softmax(s, -1)
    return p @ rows[:, :latent].double(), torch.logsumexp(s, -1), p @ rows[:, :latent].double().abs()


@pytest.mark.parametrize("dtype,heads,graph", [(BF16, 128, False), (BF16, 128, True), (BF16, 16, False), (F32, 16, False)])
def test_a_serving_loop(mla, dtype, heads, graph):
    nope, rope, latent, page, batch, budget, sinks, recent = 128, 64, 512, 16, 3, 48, 4, 8
    scale, width = 1 / math.sqrt(nope + rope), latent + rope
    g = torch.Generator(device="cuda").manual_seed(heads)

    def draw(*shape, by=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * by).to(dtype)

    w_uk, kw, qw = draw(heads, nope, latent, by=1 / math.sqrt(nope)), (1 + draw(latent, by=0.2)).to(dtype), (1 + draw(nope + rope, by=0.2)).to(dtype)
    cs = ref.table(POSITIONS, rope).cuda()
    pages = -(-(budget + 40) // page)
    table = torch.randperm(batch * pages, generator=torch.Generator().manual_seed(1)).view(batch, pages).to(torch.int32).cuda()
    cache = torch.zeros(batch * pages, page, width, dtype=dtype, device="cuda")
    mass = torch.zeros(batch, pages * page, device="cuda")
    prompt = [30, 7, 1]
    lens = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    held = list(prompt)                               # rows of each sequence, on the host
    seen = list(prompt)                               # tokens of each sequence: the position of its next

    def slots_of(b, rows):
        rows = torch.tensor(rows, device="cuda")
        return table[b, rows // page].long() * page + rows % page

    def rows_of(b):
        return cache.view(-1, width)[slots_of(b, range(held[b]))]

    # ---- prompts: a prefill, whose queries weigh the rows
    tokens = sum(prompt)
    q, kv = draw(tokens, heads, nope + rope), draw(tokens, width)
    pos = torch.cat([torch.arange(n) for n in prompt]).cuda()
    slots = torch.cat([slots_of(b, range(n)) for b, n in enumerate(prompt)])
    q_nope, q_cat = torch.empty_like(q[..., :nope]), torch.zeros(tokens, heads, width, dtype=dtype, device="cuda")
    mla.mla_norm_rope_q_cache_write(q_nope, q_cat[..., latent:], q, qw, cache, kv, kw, pos, cs, slots)
    mla.mla_absorb_q(q_cat[..., :latent].transpose(0, 1), q_nope.transpose(0, 1), w_uk)
    cu = torch.tensor([0] + [sum(prompt[:i + 1]) for i in range(batch)], dtype=torch.int32, device="cuda")
    o, lse = torch.zeros(tokens, heads, latent, dtype=dtype, device="cuda"), torch.zeros(tokens, heads, device="cuda")
    mla.mla_prefill(o, q_cat, cache, table, cu, lens, max(prompt), latent, rope, scale, lse_out=lse)
    mla.mla_prefill_mass(mass, q_cat, cache, table, cu, lens, lse, scale)
    mla.mla_device_error()
    want, err = ref.rows(kv.cpu(), kw.cpu(), cs[pos].cpu(), True, 1e-6)
    ref.check(cache.view(-1, width)[slots], want, err, dtype, "prompt rows")
    for b, n in enumerate(prompt):
        total = mass[b, :n].sum().item()
        assert abs(total - n * heads) < 2e-2 * n * heads          # each query's weights sum to 1 a head
        assert (mass[b, n:] == 0).all()

    # ---- steps of one token a sequence
    q, kv = torch.empty(batch, heads, nope + rope, dtype=dtype, device="cuda"), torch.empty(batch, width, dtype=dtype, device="cuda")
    q_nope, q_cat = torch.empty_like(q[..., :nope]), torch.zeros(batch, heads, width, dtype=dtype, device="cuda")
    pos, slots = torch.zeros(batch, dtype=torch.int64, device="cuda"), torch.zeros(batch, dtype=torch.int64, device="cuda")
    o, lse = torch.zeros(batch, heads, latent, dtype=dtype, device="cuda"), torch.zeros(batch, heads, device="cuda")
    ws = torch.empty(mla.mla_decode_workspace_size(batch, heads, latent), dtype=torch.uint8, device="cuda")
    ews = torch.empty(mla.mla_cache_evict_workspace_size(batch, mass.shape[1], budget), dtype=torch.uint8, device="cuda")
    kept = torch.zeros(batch, budget, dtype=torch.int32, device="cuda")

    def step():
        mla.mla_norm_rope_q_cache_write(q_nope, q_cat[..., latent:], q, qw, cache, kv, kw, pos, cs, slots)
        mla.mla_absorb_q(q_cat[..., :latent].transpose(0, 1), q_nope.transpose(0, 1), w_uk)
        mla.mla_decode(o, q_cat, cache, table, lens, latent, rope, scale, lse_out=lse, workspace=ws)
        mla.mla_decode_mass(mass, q_cat, cache, table, lens, lse, scale)

    replay = None
    evictions = 0
    for i in range(30):
        q.copy_(draw(batch, heads, nope + rope))
        kv.copy_(draw(batch, width))
        pos.copy_(torch.tensor(seen))
        slots.copy_(torch.cat([slots_of(b, [held[b]]) for b in range(batch)]))
        lens += 1
        held, seen = [n + 1 for n in held], [n + 1 for n in seen]
        before = mass.clone()
        if graph and replay is None:
            step()                                    # a first pass outside the capture
            mass.copy_(before)
            replay = torch.cuda.CUDAGraph()
            with torch.cuda.graph(replay):
                step()
        if graph:
            replay.replay()
        else:
            step()
        mla.mla_device_error()
        for b in range(batch):
            rows = rows_of(b)
            want, err = ref.rows(kv[b:b + 1].cpu(), kw.cpu(), cs[pos[b:b + 1]].cpu(), True, 1e-6)
            ref.check(rows[-1:], want, err, dtype, "new row")
            want_o, want_lse, mean = attend(q_cat[b], rows, latent, scale)
            # the decode's own bounds: 2^-8 for its weights' and its output's rounding on the bf16 path (three roundings
            # of a weight) and float32 sums on the other
            tol = (5 * 2.0 ** -8 if dtype == BF16 else 1e-5) * (mean + want_o.abs()) + 1e-6
            assert ((o[b].double() - want_o).abs() <= tol).all()
            assert (lse[b] - want_lse).abs().max() <= (1.2e-2 if dtype == BF16 else 1e-3)
            w = torch.exp(q_cat[b].double() @ rows.double().T * scale - lse[b].double()[:, None]).sum(0)
            got = mass[b, :held[b]].double() - before[b, :held[b]].double()
            assert (got - w).abs().max() <= 1e-4 * (1 + before[b].max().item() / 16), "mass"
        if max(held) > budget:
            evictions += 1
            cut, m = [rows_of(b).clone() for b in range(batch)], mass.clone()
            mla.mla_cache_evict(cache, mass, table, lens, budget - 8, lens, sinks=sinks, recent=recent, kept_out=kept[:, :budget - 8].contiguous(),
                                workspace=ews)
            mla.mla_device_error()
            held = [min(n, budget - 8) for n in held]
            assert lens.tolist() == held
            for b in range(batch):
                n = cut[b].shape[0]
                t = list(range(n))
                if n > budget - 8:
                    free = sorted(range(sinks, n - recent), key=lambda x: (-m[b, x].item(), x))[:budget - 8 - sinks - recent]
                    t = sorted(list(range(sinks)) + free + list(range(n - recent, n)))
                assert torch.equal(rows_of(b), cut[b][t]) and torch.equal(mass[b, :len(t)], m[b, t])
                assert (mass[b, len(t):n] == 0).all()
    assert evictions >= 2


def test_the_masses_choose_the_rows_that_matter(mla):
    # one row that every query turns to, far from both ends: it stays, whatever else goes
    c = mass_ref.Case(3, BF16, 16, 576, 64, [500], [40])
    hot = 237
    q = c.q[:40].float()
    c.cache[c.table[0, hot // 64].long(), hot % 64] = (q.mean((0, 1)) * 40).to(BF16)
    c.lse[:] = math.inf
    s = torch.einsum("ihe,te->iht", q.double(), c.cache[c.table[0, :8].long()].flatten(0, 1)[:500].double()) * c.scale
    seen = torch.arange(500, device="cuda") <= torch.arange(460, 500, device="cuda")[:, None]
    c.lse[:40] = torch.logsumexp(torch.where(seen[:, None], s, -math.inf), -1).float()
    mass = c.run(mla, 0.0)
    kept, lens = torch.zeros(1, 100, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_cache_evict(c.cache, mass, c.table, c.lens, 100, lens, sinks=4, recent=16, kept_out=kept)
    mla.mla_device_error()
    assert hot in kept[0].tolist() and lens.tolist() == [100]

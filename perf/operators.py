"""The attention operators over a cache whose rows are not the queries' own positions, as cases to measure.

cross     pa_cross_attention: any number of query tokens per sequence attend to an encoder's states in a paged pool
mass      pa_decode_mass: one decode step that also adds every cached token's attention weight to its running mass
select    pa_evict_select: the tokens of each (sequence, kv head) that stay, by recency and mass
compact   pa_evict_compact: the kept rows moved into fresh blocks

With `own` false, run() computes the plain form in elementary torch operations, in 32 bits; with `own` true it calls
the library. Lengths follow from the case alone (spread over [lo, hi]); values, block tables and order from the seed.
"""
import math

import torch

own = False

BS = 16  # tokens per block


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decoder token attends to one utterance's encoder states: pure latency
        dict(name="cross_one_token", op="cross", kv="bf16", n_h=32, n_kv=8, d_h=128, num_seqs=1, q_lo=1, q_hi=1,
             ctx_lo=1500, ctx_hi=1500),
        # a step of a mixed batch: some sequences add one token, some a short forced prompt
        dict(name="cross_mixed", op="cross", kv="bf16", n_h=32, n_kv=8, d_h=128, num_seqs=48, q_lo=1, q_hi=61,
             ctx_lo=200, ctx_hi=4096),
        # decoder prompts over long documents: bound by the tensor cores
        dict(name="cross_prompt", op="cross", kv="bf16", n_h=32, n_kv=8, d_h=128, num_seqs=8, q_lo=512, q_hi=1024,
             ctx_lo=4096, ctx_hi=8192),
        # one head per kv head and 64 wide, odd prompts over encoder windows of up to 1500 states
        dict(name="cross_d64", op="cross", kv="bf16", n_h=16, n_kv=16, d_h=64, num_seqs=32, q_lo=33, q_hi=447,
             ctx_lo=701, ctx_hi=1500),
        # INT8 states, short prompts
        dict(name="cross_int8", op="cross", kv="int8", n_h=32, n_kv=32, d_h=128, num_seqs=16, q_lo=16, q_hi=256,
             ctx_lo=512, ctx_hi=4096),
        # the smallest geometry of the repository, two short sequences
        dict(name="mass_tiny", op="mass", kv="bf16", n_h=4, n_kv=2, d_h=64, num_seqs=2, ctx_lo=5, ctx_hi=37),
        # a serving batch of the Llama-3-8B layer
        dict(name="mass_batch", op="mass", kv="bf16", n_h=32, n_kv=8, d_h=128, num_seqs=64, ctx_lo=512, ctx_hi=4096),
        # few long contexts, INT8 cache
        dict(name="mass_long_int8", op="mass", kv="int8", n_h=32, n_kv=8, d_h=128, num_seqs=4, ctx_lo=32768,
             ctx_hi=131072),
        # the serving batch is cut to 1024 tokens a sequence
        dict(name="select_batch", op="select", n_kv=8, num_seqs=64, ctx_lo=900, ctx_hi=4096, budget=1024, recent=256),
        # long contexts cut to an eighth
        dict(name="select_long", op="select", n_kv=8, num_seqs=4, ctx_lo=32768, ctx_hi=131072, budget=16384,
             recent=2048),
        dict(name="compact_batch", op="compact", kv="bf16", n_kv=8, d_h=128, num_seqs=64, ctx_lo=900, ctx_hi=4096,
             budget=1024, recent=256),
        dict(name="compact_long_int8", op="compact", kv="int8", n_kv=8, d_h=128, num_seqs=4, ctx_lo=32768,
             ctx_hi=131072, budget=16384, recent=2048),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cross", "cross", "mass", "select", "compact"])
    kv = rng.choice(["bf16", "int8", "int4"])
    g = rng.choice([1, 2, 4, 8, 16])
    n_kv = rng.choice([1, 2, 3, 4, 8])
    d_h = rng.choice([64, 128])
    if op == "cross":
        ctx_hi, q_hi = _log_int(rng, 64, 16384), _log_int(rng, 1, 1024)
        q_hi = max(1, min(q_hi, int(9.6e8 / (g * n_kv * ctx_hi))))  # fewer products than the largest listed case
        most = max(1, int(9.6e8 / (g * n_kv * ctx_hi * q_hi)))
        return dict(op=op, kv=kv, n_h=g * n_kv, n_kv=n_kv, d_h=d_h, num_seqs=min(most, _log_int(rng, 1, 64)),
                    q_lo=_log_int(rng, 1, q_hi), q_hi=q_hi, ctx_lo=_log_int(rng, 1, ctx_hi), ctx_hi=ctx_hi)
    ctx_hi = _log_int(rng, 32, 131072)
    num_seqs = min(max(1, 200000 // ctx_hi), _log_int(rng, 1, 96))
    ctx_lo = _log_int(rng, max(1, ctx_hi // 8), ctx_hi)
    if op == "mass":
        return dict(op=op, kv=kv, n_h=g * n_kv, n_kv=n_kv, d_h=d_h, num_seqs=num_seqs, ctx_lo=ctx_lo, ctx_hi=ctx_hi)
    budget = _log_int(rng, 16, ctx_hi)
    cut = dict(num_seqs=num_seqs, n_kv=n_kv, ctx_lo=ctx_lo, ctx_hi=ctx_hi, budget=budget,
               recent=rng.randint(0, budget // 2))
    return dict(op=op, **cut) if op == "select" else dict(op=op, kv=kv, d_h=d_h, **cut)


def _spread(n, lo, hi):
    """n lengths over [lo, hi], both ends among them, in no order."""
    if n == 1:
        return [hi]
    got = [lo + (hi - lo) * i // (n - 1) for i in range(n)]
    step = next(s for s in range(max(1, int(0.618 * n)), n + 1) if math.gcd(s, n) == 1)
    return [got[i * step % n] for i in range(n)]


def _lengths(case):
    ctx = _spread(case["num_seqs"], case["ctx_lo"], case["ctx_hi"])
    q = _spread(case["num_seqs"], case["q_lo"], case["q_hi"])[::-1] if case["op"] == "cross" else None
    return ctx, q


def _row_bytes(case):
    return {"bf16": 2 * case["d_h"], "int8": case["d_h"] + 4, "int4": case["d_h"] // 2 + 4}[case["kv"]]


def work(case):
    ctx, q = _lengths(case)
    blocks = sum(-(-n // BS) for n in ctx)
    if case["op"] == "cross":
        pairs = sum(a * b for a, b in zip(ctx, q))
        return {"bytes": 4 * sum(q) * case["n_h"] * case["d_h"] + 2 * sum(ctx) * case["n_kv"] * _row_bytes(case) + 4 * blocks,
                "flops": 4 * case["d_h"] * case["n_h"] * pairs}
    if case["op"] == "mass":
        return {"bytes": 4 * len(ctx) * case["n_h"] * case["d_h"] + 2 * sum(ctx) * case["n_kv"] * _row_bytes(case)
                + 8 * sum(ctx) * case["n_kv"] + 4 * blocks,
                "flops": 4 * case["d_h"] * case["n_h"] * sum(ctx)}
    kept = sum(min(n, case["budget"]) for n in ctx)
    units = len(ctx) * case["n_kv"]
    if case["op"] == "select":
        return {"bytes": 4 * sum(ctx) * case["n_kv"] + 4 * units * case["budget"] + 8 * len(ctx), "flops": 0}
    room = -(-case["budget"] // BS) * BS
    return {"bytes": 4 * kept * case["n_kv"] * _row_bytes(case) + 8 * kept * case["n_kv"] + 4 * units * room, "flops": 0}


# ------------------------------------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, gen, dtype=torch.float32, scale=1.0):
    """N(0, scale^2) rounded to dtype, made in pieces."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        n = min(1 << 27, flat.numel() - i)
        x = torch.randn(n, generator=gen, device="cuda") * scale
        flat[i:i + n] = x if dtype != torch.int8 else x.round_().clamp_(-127, 127)
    return out


def _pool(case, num_blocks, gen):
    """K or V rows of a pool (codes and scales): rows of about N(0, 1) values."""
    shape = (num_blocks, case["n_kv"], BS, case["d_h"])
    if case["kv"] == "bf16":
        return _randn(shape, gen, torch.bfloat16), None
    scale = torch.exp(0.25 * torch.randn(shape[:3], generator=gen, device="cuda"))
    if case["kv"] == "int8":
        return _randn(shape, gen, torch.int8, 40.0), scale / 40
    codes = _randn(shape, gen, torch.int8, 2.3).clamp_(-7, 7)
    return (codes[..., 0::2] & 15 | codes[..., 1::2] << 4).view(torch.uint8), scale / 2.3


def prepare(case, seed):
    gen = _generator(seed)
    ctx, q = _lengths(case)
    B, n_kv = case["num_seqs"], case["n_kv"]
    s = dict(case=case, ctx=ctx, context_lens=torch.tensor(ctx, dtype=torch.int32, device="cuda"))
    max_blocks = -(-max(ctx) // BS)
    if case["op"] == "select":
        s["mass"] = _masses(B, n_kv, max_blocks * BS, gen)
        return s
    blocks = [-(-n // BS) for n in ctx]
    fresh = -(-case["budget"] // BS) if case["op"] == "compact" else 0
    num_blocks = int(1.05 * sum(blocks)) + 1 + B * fresh
    order = torch.randperm(num_blocks, generator=gen, device="cuda").to(torch.int32)
    at = torch.tensor([0] + blocks[:-1], device="cuda").cumsum(0)
    slot = at[:, None] + torch.arange(max_blocks, device="cuda")
    used = torch.arange(max_blocks, device="cuda") < torch.tensor(blocks, device="cuda")[:, None]
    s["block_tables"] = torch.where(used, order[torch.where(used, slot, 0)], -1).to(torch.int32).contiguous()
    s["k_cache"], s["k_scale"] = _pool(case, num_blocks, gen)
    s["v_cache"], s["v_scale"] = _pool(case, num_blocks, gen)
    if case["op"] == "compact":
        s["new_tables"] = order[sum(blocks):sum(blocks) + B * fresh].view(B, fresh).contiguous()
        s["mass"] = _masses(B, n_kv, max_blocks * BS, gen)
        s["mass_out"] = torch.zeros(B, n_kv, fresh * BS, device="cuda")
        s["keep"], s["keep_lens"] = _plain_select(s["mass"], s["context_lens"], case["budget"], case["recent"])
        return s
    s["scale"] = 1 / math.sqrt(case["d_h"])
    if case["op"] == "cross":
        s["cu_q"] = torch.tensor([0] + q, device="cuda").cumsum(0).to(torch.int32)
        s["max_q"] = max(q)
        s["q"] = _randn((sum(q), case["n_h"], case["d_h"]), gen, torch.bfloat16, 2.0)
    else:
        s["q"] = _randn((B, case["n_h"], case["d_h"]), gen, torch.bfloat16, 2.0)
        s["mass"] = _masses(B, n_kv, max_blocks * BS, gen) * (
            torch.arange(max_blocks * BS, device="cuda") < s["context_lens"][:, None, None])
        s["mass_out"] = s["mass"].clone()
    return s


def _masses(B, n_kv, tokens, gen):
    """Heavy-tailed sums of weights; a twentieth of the tokens were never attended."""
    m = torch.exp(2 * torch.randn((B, n_kv, tokens), generator=gen, device="cuda") - 4)
    return m * (torch.rand((B, n_kv, tokens), generator=gen, device="cuda") > 0.05)


# ------------------------------------------------------------------------------------------------ plain forms
def _rows(s, which):
    """The cached rows of every sequence, [B, n_kv, max_ctx, d_h] in 32 bits."""
    pool, scale = s[which + "_cache"], s[which + "_scale"]
    table = s["block_tables"].clamp(min=0).long()
    x = pool[table]
    if pool.dtype == torch.uint8:
        lo, hi = (x & 15).to(torch.int8), (x >> 4).to(torch.int8)
        x = torch.stack([(lo ^ 8) - 8, (hi ^ 8) - 8], dim=-1).flatten(-2)
    x = x.float()
    if scale is not None:
        x = x * scale[table][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_weights(s, q, rows):
    """softmax(scale q K^T) of q [B, n_kv, rows, d_h] over each sequence's tokens."""
    k = _rows(s, "k")
    score = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    seen = torch.arange(k.shape[2], device="cuda") < s["context_lens"][:, None, None, None]
    score = score.masked_fill_(~seen, -math.inf)
    e = torch.exp(score.sub_(score.amax(-1, keepdim=True)))
    return e.div_(e.sum(-1, keepdim=True))


def _plain_cross(s):
    q, cu = s["q"], s["cu_q"].long()
    (T, n_h, d), B, Q = q.shape, cu.shape[0] - 1, s["max_q"]
    n_kv = s["k_cache"].shape[1]
    g = n_h // n_kv
    i = torch.arange(Q, device="cuda")
    token = torch.where(i < (cu[1:] - cu[:-1])[:, None], cu[:-1, None] + i, 0)
    x = q.float()[token].view(B, Q, n_kv, g, d).permute(0, 2, 1, 3, 4).reshape(B, n_kv, Q * g, d)
    o = torch.matmul(_plain_weights(s, x, Q * g), _rows(s, "v"))
    o = o.view(B, n_kv, Q, g, d).transpose(1, 2).reshape(B, Q, n_h, d)
    t = torch.arange(T, device="cuda")
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    return o[b, t - cu[b]].to(q.dtype)


def _plain_mass(s):
    q = s["q"]
    B, n_h, d = q.shape
    n_kv = s["k_cache"].shape[1]
    w = _plain_weights(s, q.float().view(B, n_kv, n_h // n_kv, d), n_h // n_kv)
    s["mass_out"].copy_(s["mass"] + w.sum(2))
    return torch.matmul(w, _rows(s, "v")).view(B, n_h, d).to(q.dtype), s["mass_out"]


def _plain_select(mass, context_lens, budget, recent):
    j = torch.arange(mass.shape[2], device=mass.device)
    n = context_lens.long()[:, None, None]
    k = n.clamp(max=budget)
    key = torch.where(j >= n - k.clamp(max=recent), math.inf, mass)
    key = torch.where(j < n, key, -math.inf)
    by = torch.sort(key, dim=2, descending=True, stable=True).indices
    by = by[:, :, :budget] if by.shape[2] >= budget else torch.nn.functional.pad(by, (0, budget - by.shape[2]))
    live = torch.arange(budget, device=mass.device) < k
    kept = torch.sort(torch.where(live, by, mass.shape[2]), dim=2).values
    return torch.where(live, kept, -1).to(torch.int32), k[:, 0, 0].to(torch.int32)


def _plain_compact(s):
    keep, lens = s["keep"].long(), s["keep_lens"].long()[:, None, None]
    B, n_kv, budget = keep.shape
    # entries behind the last kept one repeat it
    i = torch.minimum(torch.arange(budget, device="cuda"), lens - 1).expand(B, n_kv, budget)
    j = torch.gather(keep, 2, i)
    b = torch.arange(B, device="cuda")[:, None, None]
    h = torch.arange(n_kv, device="cuda")[None, :, None]
    src = s["block_tables"].long()[b, j // BS]
    dst = s["new_tables"].long()[b, i // BS]
    for pool in (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]):
        if pool is not None:
            pool[dst, h, i % BS] = pool[src, h, j % BS]
    live = torch.arange(s["mass_out"].shape[2], device="cuda") < lens
    moved = torch.gather(s["mass"], 2, j)
    moved = torch.nn.functional.pad(moved, (0, s["mass_out"].shape[2] - budget))
    s["mass_out"].copy_(torch.where(live, moved, 0))
    return _moved(s)


def _moved(s):
    """The pools (codes as the whole numbers that they are, with their scales) and the masses."""
    return [s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["mass_out"]]


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        if op == "select":
            return _plain_select(s["mass"], s["context_lens"], case["budget"], case["recent"])
        return {"cross": _plain_cross, "mass": _plain_mass, "compact": _plain_compact}[op](s)
    import paged_kv_cache_94_gb300 as pa
    if op == "cross":
        return pa.pa_cross_attention(s["q"], s["cu_q"], s["k_cache"], s["v_cache"], s["block_tables"],
                                     s["context_lens"], s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if op == "mass":
        return pa.pa_decode_mass(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"], s["scale"],
                                 s["mass"], mass_out=s["mass_out"], k_scale=s["k_scale"],
                                 v_scale=s["v_scale"]), s["mass_out"]
    if op == "select":
        return pa.pa_evict_select(s["mass"], s["context_lens"], case["budget"], case["recent"])
    pa.pa_evict_compact(s["k_cache"], s["v_cache"], s["block_tables"], s["keep"], s["keep_lens"], s["new_tables"],
                        mass=s["mass"], mass_out=s["mass_out"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return _moved(s)


# ------------------------------------------------------------------------------------------------ in 64 bits
def _values(pool, scale, table, n, head):
    """Rows 0 .. n-1 of one kv head through one block table, in 64 bits."""
    blocks = table[:(n + BS - 1) // BS].long()
    x = pool[blocks, head].reshape(-1, pool.shape[-1])[:n]
    if pool.dtype == torch.uint8:
        full = torch.empty(n, 2 * x.shape[1], dtype=torch.float64, device=x.device)
        for part, code in ((0, x % 16), (1, torch.div(x, 16, rounding_mode="floor"))):
            code = code.double()
            full[:, part::2] = torch.where(code > 7, code - 16, code)
        x = full
    x = x.double()
    return x if scale is None else x * scale[blocks, head].reshape(-1)[:n, None].double()


def exact(case, seed):
    s = prepare(case, seed)
    ctx, q_len = _lengths(case)
    n_kv = case["n_kv"]
    if case["op"] in ("cross", "mass"):
        q = s["q"].double()
        g = q.shape[1] // n_kv
        out = torch.zeros_like(q)
        mass = s["mass"].double() if case["op"] == "mass" else None
        first = 0
        for b, n in enumerate(ctx):
            last = first + (q_len[b] if q_len else 1)
            for h in range(n_kv):
                k = _values(s["k_cache"], s["k_scale"], s["block_tables"][b], n, h)
                v = _values(s["v_cache"], s["v_scale"], s["block_tables"][b], n, h)
                for m in range(h * g, h * g + g):
                    w = torch.softmax(q[first:last, m] @ k.T / math.sqrt(case["d_h"]), dim=1)
                    out[first:last, m] = w @ v
                    if mass is not None:
                        mass[b, h, :n] += w[0]
            first = last
        return out if mass is None else (out, mass)
    if case["op"] == "select":
        return _exact_select(s, case, ctx)
    for b, n in enumerate(ctx):
        kept = min(n, case["budget"])
        i = torch.arange(kept, device="cuda")
        to = s["new_tables"][b].long()[i // BS]
        s["mass_out"][b] = 0
        for h in range(n_kv):
            j = s["keep"][b, h, :kept].long()
            fro = s["block_tables"][b].long()[j // BS]
            for pool in (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]):
                if pool is not None:
                    pool[to, h, i % BS] = pool[fro, h, j % BS]
            s["mass_out"][b, h, :kept] = s["mass"][b, h, j]
    return [None if x is None else x.double() if x.is_floating_point() else x for x in _moved(s)]


def _exact_select(s, case, ctx):
    import numpy as np
    mass = s["mass"].cpu().numpy().astype(np.float64)
    keep = np.full((len(ctx), case["n_kv"], case["budget"]), -1, np.int32)
    for b, n in enumerate(ctx):
        k = min(n, case["budget"])
        r = min(case["recent"], k)
        for h in range(case["n_kv"]):
            heavy = np.lexsort((np.arange(n - r), -mass[b, h, :n - r]))[:k - r]
            keep[b, h, :k] = np.concatenate([np.sort(heavy), np.arange(n - r, n)])
    return torch.from_numpy(keep), torch.tensor([min(n, case["budget"]) for n in ctx], dtype=torch.int32)

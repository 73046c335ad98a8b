"""A step with rotary positions and a window that keeps its first tokens, as cases to measure.

rope      pa_rope_write: queries and keys turned by positions on one or several axes (time, height, width), keys and
          values appended to the paged pool, in one call
attend    pa_window_attention: any number of new tokens per sequence (a prompt, a chunk of one, a draft to verify) attend
          causally within a sliding window, and to the sequence's first tokens
decode    pa_window_decode: the same for one new token per sequence

With `own` false, run() computes the plain form in elementary torch operations, in 32 bits (angles in 64); with `own`
true it calls the library. Lengths follow from the case alone (spread over [lo, hi]); values, block tables and order
from the seed. window = 0 is none.
"""
import math

import torch

own = False

BS = 16  # tokens per block


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the new tokens of a serving batch of the Llama-3-8B layer: pure latency
        dict(name="rope_step", op="rope", kv="bf16", n_h=32, n_kv=8, d_h=128, tokens=64, far=4096, axes=1, dims=128,
             pairs="halves", fused=False),
        # a prompt of images and video: three axes, q, k and v as views of one projection's output
        dict(name="rope_prompt", op="rope", kv="bf16", n_h=32, n_kv=8, d_h=128, tokens=8192, far=131072, axes=3,
             dims=128, pairs="halves", fused=True),
        # an odd chunk into an INT8 pool, half of each head turned, adjacent values as pairs
        dict(name="rope_chunk_int8", op="rope", kv="int8", n_h=16, n_kv=16, d_h=64, tokens=4111, far=8192, axes=2,
             dims=32, pairs="adjacent", fused=True),
        # one to eight draft tokens of each sequence are verified
        dict(name="attend_verify", op="attend", kv="bf16", n_h=32, n_kv=8, d_h=128, num_seqs=48, q_lo=1, q_hi=8,
             ctx_lo=200, ctx_hi=8192, window=4096, n_first=4),
        # a step of chunked prompts with the Mistral-7B window
        dict(name="attend_chunks", op="attend", kv="bf16", n_h=32, n_kv=8, d_h=128, num_seqs=8, q_lo=512, q_hi=2048,
             ctx_lo=2048, ctx_hi=8192, window=4096, n_first=4),
        # one long prompt without a window, bound by the tensor cores
        dict(name="attend_prompt", op="attend", kv="bf16", n_h=32, n_kv=8, d_h=128, num_seqs=1, q_lo=16384, q_hi=16384,
             ctx_lo=16384, ctx_hi=16384, window=0, n_first=0),
        # one head per kv head and 64 wide, whole odd prompts, a window that is no multiple of anything
        dict(name="attend_d64", op="attend", kv="bf16", n_h=16, n_kv=16, d_h=64, num_seqs=24, q_lo=33, q_hi=1999,
             ctx_lo=33, ctx_hi=1999, window=333, n_first=5),
        # short chunks over long contexts of an INT8 pool
        dict(name="attend_int8", op="attend", kv="int8", n_h=32, n_kv=32, d_h=128, num_seqs=16, q_lo=16, q_hi=256,
             ctx_lo=512, ctx_hi=8192, window=2000, n_first=17),
        # one sequence alone: pure latency
        dict(name="decode_one", op="decode", kv="bf16", n_h=32, n_kv=8, d_h=128, num_seqs=1, ctx_lo=5000, ctx_hi=5000,
             window=1024, n_first=4),
        # a serving batch with the Mistral-7B window
        dict(name="decode_batch", op="decode", kv="bf16", n_h=32, n_kv=8, d_h=128, num_seqs=64, ctx_lo=512,
             ctx_hi=16384, window=4096, n_first=4),
        # few long contexts of an INT8 pool, a wide window and a whole instruction kept in front
        dict(name="decode_long_int8", op="decode", kv="int8", n_h=32, n_kv=8, d_h=128, num_seqs=4, ctx_lo=32768,
             ctx_hi=131072, window=65536, n_first=500),
        # many short sequences of an INT4 pool, one head per kv head and 64 wide
        dict(name="decode_int4", op="decode", kv="int4", n_h=16, n_kv=16, d_h=64, num_seqs=96, ctx_lo=1, ctx_hi=3001,
             window=1001, n_first=20),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "decode"])
    g = rng.choice([1, 2, 4, 8, 16])
    n_kv = rng.choice([1, 2, 3, 4, 8])
    heads = dict(op=op, n_h=g * n_kv, n_kv=n_kv, d_h=rng.choice([64, 128]))
    if op == "rope":
        return dict(kv=rng.choice(["bf16", "int8"]), **heads, tokens=_log_int(rng, 1, 4096),
                    far=_log_int(rng, 16, 1 << 20), axes=rng.choice([1, 2, 3, 4]),
                    dims=heads["d_h"] // rng.choice([1, 1, 2]), pairs=rng.choice(["halves", "adjacent"]),
                    fused=rng.choice([False, True]))
    kv = rng.choice(["bf16", "int8", "int4"])
    n_first = rng.choice([0, 1, 4, 17, 64, 200])
    if op == "attend":
        ctx_hi, q_hi = _log_int(rng, 64, 16384), _log_int(rng, 1, 1024)
        q_hi = max(1, min(q_hi, ctx_hi, int(4.0e9 / (g * n_kv * ctx_hi))))
        most = max(1, int(4.0e9 / (g * n_kv * ctx_hi * q_hi)))
        window = rng.choice([0, _log_int(rng, 1, ctx_hi)])
        return dict(kv=kv, **heads, num_seqs=min(most, _log_int(rng, 1, 64)), q_lo=_log_int(rng, 1, q_hi), q_hi=q_hi,
                    ctx_lo=_log_int(rng, 1, ctx_hi), ctx_hi=ctx_hi, window=window, n_first=n_first)
    ctx_hi = _log_int(rng, 32, 131072)
    num_seqs = min(max(1, 200000 // ctx_hi), _log_int(rng, 1, 96))
    return dict(kv=kv, **heads, num_seqs=num_seqs, ctx_lo=_log_int(rng, max(1, ctx_hi // 16), ctx_hi), ctx_hi=ctx_hi,
                window=_log_int(rng, 1, ctx_hi), n_first=n_first)


def _spread(n, lo, hi):
    """n lengths over [lo, hi], both ends among them, in no order."""
    if n == 1:
        return [hi]
    got = [lo + (hi - lo) * i // (n - 1) for i in range(n)]
    step = next(s for s in range(max(1, int(0.618 * n)), n + 1) if math.gcd(s, n) == 1)
    return [got[i * step % n] for i in range(n)]


def _lengths(case):
    """Context and new tokens of each sequence; a sequence has at most its context as new tokens."""
    ctx = _spread(case["num_seqs"], case["ctx_lo"], case["ctx_hi"])
    if case["op"] == "decode":
        return ctx, [1] * len(ctx)
    q = _spread(case["num_seqs"], case["q_lo"], case["q_hi"])
    return ctx, [min(a, b) for a, b in zip(ctx, q)]


def _row_bytes(case):
    return {"bf16": 2 * case["d_h"], "int8": case["d_h"] + 4, "int4": case["d_h"] // 2 + 4}[case["kv"]]


def work(case):
    n_h, n_kv, d = case["n_h"], case["n_kv"], case["d_h"]
    if case["op"] == "rope":
        row = 4 * n_h * d + 4 * n_kv * d + 2 * n_kv * _row_bytes(case) + 4 * case["axes"] + 8
        return {"bytes": case["tokens"] * row, "flops": case["tokens"] * (n_h + n_kv) * 3 * case["dims"]}
    ctx, q = _lengths(case)
    w, first = case["window"], case["n_first"]
    pairs = rows = 0
    for n, new in zip(ctx, q):
        lo = max(0, n - new + 1 - w) if w else 0  # the first key in some token's window
        rows += n - lo + min(lo, first)
        pairs += sum(min(p, w or p) + min(first, max(0, p - (w or p))) for p in range(n - new + 1, n + 1))
    return {"bytes": 4 * sum(q) * n_h * d + 2 * rows * n_kv * _row_bytes(case) + 4 * (rows // BS) + 8 * len(ctx),
            "flops": 4 * d * n_h * pairs}


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
    return _prepare_rope(case, gen) if case["op"] == "rope" else _prepare_attention(case, gen)


def _prepare_rope(case, gen):
    T, n_h, n_kv, d = case["tokens"], case["n_h"], case["n_kv"], case["d_h"]
    pairs, axes = case["dims"] // 2, case["axes"]
    i = torch.arange(pairs, device="cuda")
    s = dict(case=case, inv_freq=500000.0 ** (-i.double() / pairs))
    s["axis"] = (i * axes // pairs).to(torch.int32)  # a run of pairs for each axis
    if case["fused"]:
        qkv = _randn((T, (n_h + 2 * n_kv) * d), gen, torch.bfloat16)
        s["q"] = qkv[:, :n_h * d].view(T, n_h, d)
        s["k"] = qkv[:, n_h * d:(n_h + n_kv) * d].view(T, n_kv, d)
        s["v"] = qkv[:, (n_h + n_kv) * d:].view(T, n_kv, d)
    else:
        s["q"] = _randn((T, n_h, d), gen, torch.bfloat16)
        s["k"] = _randn((T, n_kv, d), gen, torch.bfloat16)
        s["v"] = _randn((T, n_kv, d), gen, torch.bfloat16)
    # the first axis goes on with the tokens, the others run over rows and columns of a grid
    t = torch.arange(T, device="cuda") + torch.randint(0, case["far"], (1,), generator=gen, device="cuda")
    grid = torch.randint(0, 64, (max(1, axes - 1), T), generator=gen, device="cuda")
    s["positions"] = torch.cat([t[None], grid[:axes - 1]]).to(torch.int32).contiguous()
    num_blocks = -(-T * 9 // (8 * BS)) + 1  # a ninth of the slots stay as they are
    s["slots"] = torch.randperm(num_blocks * BS, generator=gen, device="cuda")[:T].contiguous()
    s["k_cache"], s["k_scale"] = _pool(case, num_blocks, gen)
    s["v_cache"], s["v_scale"] = _pool(case, num_blocks, gen)
    return s


def _prepare_attention(case, gen):
    ctx, q = _lengths(case)
    B = case["num_seqs"]
    s = dict(case=case, context_lens=torch.tensor(ctx, dtype=torch.int32, device="cuda"))
    max_blocks = -(-max(ctx) // BS)
    blocks = torch.tensor([-(-n // BS) for n in ctx], device="cuda")
    num_blocks = int(1.05 * int(blocks.sum())) + 1
    order = torch.randperm(num_blocks, generator=gen, device="cuda").to(torch.int32)
    block = torch.arange(max_blocks, device="cuda")
    used = block < blocks[:, None]
    table = order[torch.where(used, (blocks.cumsum(0) - blocks)[:, None] + block, 0)]
    if case["window"]:  # blocks that no token sees any more have been given back
        lo = s["context_lens"].long() - torch.tensor(q, device="cuda") + 1 - case["window"]
        used &= (block < -(-case["n_first"] // BS)) | (block >= lo.clamp(min=0)[:, None] // BS)
    s["block_tables"] = torch.where(used, table, -1).to(torch.int32).contiguous()
    s["k_cache"], s["k_scale"] = _pool(case, num_blocks, gen)
    s["v_cache"], s["v_scale"] = _pool(case, num_blocks, gen)
    s["scale"] = 1 / math.sqrt(case["d_h"])
    s["cu_q"] = torch.tensor([0] + q, device="cuda").cumsum(0).to(torch.int32)
    s["max_q"] = max(q)
    s["q"] = _randn((sum(q), case["n_h"], case["d_h"]), gen, torch.bfloat16, 2.0)
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _turn(x, cos, sin, adjacent):
    """The leading 2 * pairs values of each head turned, pair by pair: (a, b) -> (a cos - b sin, b cos + a sin)."""
    n = 2 * cos.shape[1]
    x, rest = x.float()[..., :n], x.float()[..., n:]
    a, b = (x[..., 0::2], x[..., 1::2]) if adjacent else (x[..., :n // 2], x[..., n // 2:])
    cos, sin = cos[:, None], sin[:, None]
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, dim=-1).flatten(-2) if adjacent else torch.cat(y, dim=-1)
    return torch.cat([y, rest], dim=-1)


def _stored(s):
    """What a call has written: a bf16 pool itself; of codes the new rows' values, and the scales."""
    if s["k_scale"] is None:
        return [s["k_cache"], s["v_cache"]]
    at = s["slots"] // BS, slice(None), s["slots"] % BS
    return [(s[c + "_cache"][at] * s[c + "_scale"][at][..., None]).to(torch.bfloat16) for c in "kv"] + \
           [s["k_scale"], s["v_scale"]]


def _plain_rope(s):
    case = s["case"]
    angle = s["positions"][s["axis"].long()].T.double() * s["inv_freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    adjacent = case["pairs"] == "adjacent"
    q = _turn(s["q"], cos, sin, adjacent).to(torch.bfloat16)
    at = s["slots"] // BS, slice(None), s["slots"] % BS
    _append(s, "k", _turn(s["k"], cos, sin, adjacent), at)
    _append(s, "v", s["v"].float(), at)
    return [q] + _stored(s)


def _append(s, which, x, at):
    if s[which + "_scale"] is None:
        s[which + "_cache"][at] = x.to(torch.bfloat16)
        return
    scale = x.abs().amax(-1) / 127
    s[which + "_cache"][at] = (x / scale[..., None]).nan_to_num(0.0).round().clamp(-128, 127).to(torch.int8)
    s[which + "_scale"][at] = scale


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


def _plain_attention(s):
    """Queries padded to the longest sequence's, all keys scored, what a token does not see masked."""
    q, cu, case = s["q"], s["cu_q"].long(), s["case"]
    (T, n_h, d), B, Q = q.shape, cu.shape[0] - 1, s["max_q"]
    n_kv = s["k_cache"].shape[1]
    g = n_h // n_kv
    new = cu[1:] - cu[:-1]
    i = torch.arange(Q, device="cuda")
    token = torch.where(i < new[:, None], cu[:-1, None] + i, 0)
    x = q.float()[token].view(B, Q, n_kv, g, d).permute(0, 2, 3, 1, 4).reshape(B, n_kv, g * Q, d)
    k = _rows(s, "k")
    score = torch.matmul(x, k.transpose(2, 3)).mul_(s["scale"]).view(B, n_kv, g, Q, -1)
    j = torch.arange(k.shape[2], device="cuda")
    p = ((s["context_lens"] - new)[:, None] + i)[:, :, None]
    seen = j <= p
    if case["window"]:
        seen &= (j > p - case["window"]) | (j < case["n_first"])
    score.masked_fill_(~seen[:, None, None], -math.inf)
    e = score.sub_(score.amax(-1, keepdim=True)).exp_()
    e.div_(e.sum(-1, keepdim=True))
    o = torch.matmul(e.view(B, n_kv, g * Q, -1), _rows(s, "v"))
    o = o.view(B, n_kv, g, Q, d).permute(0, 3, 1, 2, 4).reshape(B, Q, n_h, d)
    t = torch.arange(T, device="cuda")
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    return o[b, t - cu[b]].to(q.dtype)


def run(state):
    s, case = state, state["case"]
    if not own:
        return _plain_rope(s) if case["op"] == "rope" else _plain_attention(s)
    import paged_kv_cache_94_gb300 as pa
    if case["op"] == "rope":
        q = pa.pa_rope_write(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"], s["k_cache"],
                             s["v_cache"], axis=s["axis"], adjacent=case["pairs"] == "adjacent",
                             k_scale=s["k_scale"], v_scale=s["v_scale"])
        return [q] + _stored(s)
    pool = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], window=case["window"], n_first=case["n_first"])
    if case["op"] == "attend":
        return pa.pa_window_attention(s["q"], s["cu_q"], s["k_cache"], s["v_cache"], s["block_tables"],
                                      s["context_lens"], s["scale"], **pool)
    return pa.pa_window_decode(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"], s["scale"],
                               **pool)


# ------------------------------------------------------------------------------------------------ in 64 bits
def _values(pool, scale, table, keep, head):
    """The rows `keep` (positions) of one kv head through one block table, in 64 bits."""
    block, row = table[keep // BS].long(), keep % BS
    x = pool[block, head, row]
    if pool.dtype == torch.uint8:
        full = torch.empty(len(keep), 2 * x.shape[1], dtype=torch.float64, device=x.device)
        for part, code in ((0, x % 16), (1, torch.div(x, 16, rounding_mode="floor"))):
            code = code.double()
            full[:, part::2] = torch.where(code > 7, code - 16, code)
        x = full
    x = x.double()
    return x if scale is None else x * scale[block, head, row, None].double()


def _exact_rope(s, case):
    import numpy as np
    T, pairs = case["tokens"], case["dims"] // 2
    pos = s["positions"].cpu().numpy().astype(np.float64)
    freq, axis = s["inv_freq"].cpu().numpy(), s["axis"].cpu().numpy()
    out = {}
    for name in "qkv":
        x = s[name].double().cpu().numpy().copy()
        for i in range(pairs if name != "v" else 0):
            turn = np.exp(1j * pos[axis[i]] * freq[i])[:, None]
            a, b = (2 * i, 2 * i + 1) if case["pairs"] == "adjacent" else (i, i + pairs)
            z = (x[:, :, a] + 1j * x[:, :, b]) * turn
            x[:, :, a], x[:, :, b] = z.real, z.imag
        out[name] = torch.from_numpy(x).cuda()
    block, row = s["slots"] // BS, s["slots"] % BS
    stored, scales = [], []
    for name in "kv":
        x, pool = out[name], s[name + "_cache"]
        if case["kv"] == "bf16":
            pool = pool.double()
            for h in range(case["n_kv"]):
                pool[block, h, row] = x[:, h]
            stored.append(pool)
            continue
        step = x.abs().max(dim=2).values / 127
        stored.append(torch.round(x / step[:, :, None]) * step[:, :, None])
        scale = s[name + "_scale"].double()
        for h in range(case["n_kv"]):
            scale[block, h, row] = step[:, h]
        scales.append(scale)
    return [out["q"]] + stored + scales


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s, case)
    ctx, new = _lengths(case)
    n_kv, w = case["n_kv"], case["window"]
    q = s["q"].double()
    g = q.shape[1] // n_kv
    out = torch.zeros_like(q)
    first = 0
    for b, (n, m) in enumerate(zip(ctx, new)):
        j = torch.arange(n, device="cuda")
        oldest = n - m  # position of the first new token
        j = j[(j < case["n_first"]) | (j + w > oldest)] if w else j
        p = torch.arange(oldest, n, device="cuda")[:, None]
        hidden = j[None] > p
        if w:
            hidden |= (j[None] + w <= p) & (j[None] >= case["n_first"])
        for h in range(n_kv):
            k = _values(s["k_cache"], s["k_scale"], s["block_tables"][b], j, h)
            v = _values(s["v_cache"], s["v_scale"], s["block_tables"][b], j, h)
            for head in range(h * g, h * g + g):
                score = q[first:first + m, head] @ k.T / math.sqrt(case["d_h"])
                score[hidden] = -math.inf
                out[first:first + m, head] = torch.softmax(score, dim=1) @ v
        first += m
    return out

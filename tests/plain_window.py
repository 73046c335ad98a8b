"""Plain forms, in 64 bits on the CPU, of rotary positions with the append, and of causal
attention within a window and to a sequence's first tokens.

Error bounds (each counts roundings, none is fitted):
  attention   a weight as in plain_attention.attend: e; a weight enters the products in two
              bf16 parts, 2^-16 (codes in the decode: as one fp16 value, 2^-11, or 2^-25 of
              the largest |v| each where it is subnormal); each 16 keys' products are added
              with one fp32 rounding or truncation, 2^-23 of the sum so far, in two parts;
              merges of records 2^-18 in all; the output is rounded once, 2^-8 |out|.
  rotary      an angle below pi / 4 rounded to fp32 and its sine and cosine within two
              units in the last place: 2^-22 of each term, the rotation's three roundings
              2^-22; bf16 results are rounded once, 2^-8 |result|.
"""
import numpy as np
import torch

from tests.plain_attention import gather_rows


def seen_keys(n_new, ctx, window, n_first):
    """[n_new, ctx] truth values: which of the context's keys each of its last n_new tokens
    attends to."""
    p = torch.arange(ctx - n_new, ctx)[:, None]
    j = torch.arange(ctx)[None]
    if window == 0:
        return j <= p
    return (j <= p) & ((j > p - window) | (j < n_first))


def attend_seen(q, k, v, scale, seen, first_part=2.0 ** -16, v_top=0.0):
    """q [rows, d], k, v [n, d] (float64, finite where seen), seen [rows, n] -> the output
    (zero rows where nothing is seen) and its tolerance without the final rounding."""
    n, d = k.shape
    if n == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    used = seen.any(0)[:, None]
    k, v = torch.where(used, k, 0.0), torch.where(used, v, 0.0)
    s = (q @ k.T * scale).masked_fill(~seen, -torch.inf)
    top = s.amax(1, keepdim=True).clamp(min=-1e300)
    w = torch.exp(s - top)
    w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    e = (d + 8) * 2.0 ** -23 * float((q.abs() @ k.abs().T).max()) * abs(scale)
    e = 2 * e + 64 * 2.0 ** -23 + first_part + 2.0 ** -18 + (n / 8 + 16) * 2.0 ** -23
    return w @ v, e * (w @ v.abs()) + n * 2.0 ** -25 * v_top


def check_window(out, q, cu, pool, bt, ctx, scale, window, n_first, seqs=None, first_part=2.0 ** -16,
                 codes_in_16=False, rows_of=None):
    """out [T, n_h, d] against the plain form; sequence b's new tokens are rows cu[b] ..
    cu[b + 1] - 1 of q. rows_of(b, h) -> its K and V rows (default: through the pool)."""
    kc, vc, ks, vs = [None if t is None else t.cpu() for t in pool]
    q, out = q.cpu().double(), out.cpu().double()
    n_kv = kc.shape[1]
    g = q.shape[1] // n_kv
    bt = bt.cpu()
    for b in range(len(ctx)) if seqs is None else seqs:
        lo, hi = int(cu[b]), int(cu[b + 1])
        n = hi - lo
        if n == 0:
            continue
        # (an entry that no token sees may be anything: read block 0 there)
        t = torch.where((bt[b] >= 0) & (bt[b] < kc.shape[0]), bt[b], 0)
        early = max(0, n - ctx[b])
        seen = seen_keys(n - early, ctx[b], window, n_first)
        seen = torch.cat([torch.zeros(early, ctx[b], dtype=torch.bool), seen])
        for h in range(n_kv):
            k, v = rows_of(b, h) if rows_of else (gather_rows(kc, ks, t, ctx[b], h),
                                                  gather_rows(vc, vs, t, ctx[b], h))
            heads = slice(h * g, (h + 1) * g)
            x = q[lo:hi, heads].reshape(n * g, -1)
            got = out[lo:hi, heads].reshape(n * g, -1)
            some = seen.repeat_interleave(g, 0)
            top = float(torch.where(seen.any(0)[:, None], v, 0.0).abs().max()) if ctx[b] else 0.0
            o, tol = attend_seen(x, k, v, scale, some, first_part, 128 * top if codes_in_16 else 0.0)
            tol = tol + 2.0 ** -8 * (o.abs() + tol) + 1e-30
            bad = ~((got - o).abs() <= tol)
            assert not bad.any(), (b, h, int(bad.sum()), float((got - o).abs().max()),
                                   bad.nonzero()[:4].tolist())
            assert (got[~some.any(1)] == 0).all()


def turned(x, positions, inv_freq, axis, adjacent, amplitude):
    """x [T, heads, d] (float64) turned by positions [axes, T], and the tolerance without the
    final rounding."""
    x = x.clone()
    tol = torch.zeros_like(x)
    pairs = len(inv_freq)
    # (an angle in 64 bits is off by 2^-53 of itself: too much for positions far out only)
    wide = np.longdouble if int(positions.abs().max() if positions.numel() else 0) > 1 << 21 or \
        int(positions.min() if positions.numel() else 0) < -(1 << 21) else np.float64
    at = positions.numpy().astype(wide)[np.asarray([int(a) for a in axis])]
    angle = (at * np.asarray([float(f) for f in inv_freq], dtype=wide)[:, None]).T  # [T, pairs]
    cos = torch.from_numpy(np.cos(angle).astype(np.float64))[:, None] * amplitude
    sin = torch.from_numpy(np.sin(angle).astype(np.float64))[:, None] * amplitude
    a, b = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if adjacent else \
        (slice(0, pairs), slice(pairs, 2 * pairs))
    u, w = x[..., a].clone(), x[..., b].clone()
    x[..., a], x[..., b] = u * cos - w * sin, w * cos + u * sin
    tol[..., a] = tol[..., b] = 2.0 ** -21 * (u.abs() + w.abs()) * abs(amplitude)
    return x, tol

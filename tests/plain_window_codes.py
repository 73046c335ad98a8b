"""Plain form, in 64 bits on the CPU, and tolerance of pa_window_decode over INT8 and INT4 pools.

What the kernel rounds besides what tests/plain_attention.py and tests/plain_window.py count (each
bound counts roundings, none is fitted): a weight times its V scale, w s, is one fp16 value against
the exact codes, off by 2^-11 of itself, or two where an item of two blocks holds a value that may
pass 8 in magnitude (its scale times 128, INT4: times 8), off by 2^-22 and the second's own 2^-11.
An fp16 value below 2^-14 is off by up to 2^-25 instead: of the largest scale, whose weights count
from 1, so 2^-25 times the largest scale times its largest code for each key."""
import torch

from tests.plain_attention import gather_rows
from tests.plain_window import seen_keys


def attend_codes(q, k, v, v_scale, top_code, scale, seen):
    """q [rows, d], k, v [n, d], v_scale [n] (float64, finite where seen), seen [rows, n] -> the
    output (zero rows where nothing is seen) and its tolerance without the final rounding."""
    n, d = k.shape
    if n == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    used = seen.any(0)
    k, v = (torch.where(used[:, None], x, 0.0) for x in (k, v))
    top = torch.where(used, v_scale, 0.0).abs() * top_code  # what the scale lets a value be
    s = (q @ k.T * scale).masked_fill(~seen, -torch.inf)
    w = torch.exp(s - s.amax(1, keepdim=True).clamp(min=-1e300))
    w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    e = (d + 8) * 2.0 ** -23 * float((q.abs() @ k.abs().T).max()) * abs(scale)
    e = 2 * e + 64 * 2.0 ** -23 + 2.0 ** -21 + 2.0 ** -18 + (n / 8 + 16) * 2.0 ** -23
    one = torch.where(top <= 8.0, 2.0 ** -11, 0.0)[:, None]
    return w @ v, w @ ((e + one) * v.abs()) + int(used.sum()) * 2.0 ** -25 * float(top.max())


def check_codes(out, q, pool, bt, ctx, scale, window, n_first, seqs=None):
    """out [B, n_h, d] of one token a sequence against the plain form."""
    kc, vc, ks, vs = [t.cpu() for t in pool]
    q, out, bt = q.cpu().double(), out.cpu().double(), bt.cpu()
    n_kv = kc.shape[1]
    g = q.shape[1] // n_kv
    top_code = 128 if kc.dtype == torch.int8 else 8
    for b in range(len(ctx)) if seqs is None else seqs:
        # (an entry that the token does not see may be anything: read block 0 there)
        t = torch.where((bt[b] >= 0) & (bt[b] < kc.shape[0]), bt[b], 0)
        n = ctx[b]
        for h in range(n_kv):
            heads = slice(h * g, (h + 1) * g)
            if n == 0:
                assert (out[b, heads] == 0).all()
                continue
            seen = seen_keys(1, n, window, n_first).expand(g, n)
            k, v = (gather_rows(p, s, t, n, h) for p, s in ((kc, ks), (vc, vs)))
            v_scale = vs[t[:-(-n // 16)].long(), h].reshape(-1)[:n].double()
            o, tol = attend_codes(q[b, heads], k, v, v_scale, top_code, scale, seen)
            tol = tol + 2.0 ** -8 * (o.abs() + tol) + 1e-30
            bad = ~((out[b, heads] - o).abs() <= tol)
            assert not bad.any(), (b, h, int(bad.sum()),
                                   float((out[b, heads] - o).abs().max()), bad.nonzero()[:4].tolist())

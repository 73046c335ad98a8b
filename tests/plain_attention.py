"""Plain forms, in 64 bits on the CPU, of the operators over a cache whose rows are
not the queries' own positions: attention of any query over a sequence's cached
rows with its weights, the choice of the tokens that stay, and their move.

Error bounds for comparisons (each counts roundings, none is fitted):
  scores   a dot product of d exact products, summed in fp32 in any order and with
           truncation at worst, is off by (d + 8) 2^-23 sum |q_i k_i| scale, the
           scale and code multiplications included;
  weights  2^x of a score off by e is off by the factor 1 + e; numerator and
           denominator both: 2 max e, plus the exponential's and the sums'
           roundings, 64 2^-23 in all.
"""
import numpy as np
import torch


def cached_rows(pool, scale, table, n, head):
    """Rows 0 .. n-1 (float64 [n, d]) of one kv head through one block table (CPU tensors)."""
    rows = []
    for j in range(n):
        blk = int(table[j // 16])
        x = pool[blk, head, j % 16]
        if pool.dtype == torch.uint8:
            b = x.numpy().astype(np.int64)
            x = torch.from_numpy(np.stack([b & 15, b >> 4], -1).reshape(-1))
            x = torch.where(x > 7, x - 16, x)
        x = x.double()
        rows.append(x if scale is None else x * float(scale[blk, head, j % 16]))
    return torch.stack(rows) if rows else torch.zeros(0, 1, dtype=torch.float64)


def attend(q, k, v, scale):
    """q [rows, d], k and v [n, d] (float64) -> out [rows, d], weights [rows, n], and the
    relative error a weight may have."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.zeros(q.shape[0], 0, dtype=torch.float64), 0.0
    w = torch.softmax(q @ k.T * scale, dim=1)
    e = (q.shape[1] + 8) * 2.0 ** -23 * float((q.abs() @ k.abs().T).max()) * abs(scale)
    return w @ v, w, 2 * e + 64 * 2.0 ** -23


def choose(mass, n, budget, recent):
    """Kept tokens of one (sequence, kv head), written out: the last `recent`, and the
    heaviest others, ties to the lowest index, NaN below everything."""
    k = min(n, budget)
    r = min(recent, k)
    rest = sorted(range(n - r), key=lambda j: (-np.inf if np.isnan(mass[j]) else mass[j]) * -1.0)
    # (sorted is stable: equal masses stay in index order; NaN among -inf is put last)
    nan_last = [j for j in rest if not np.isnan(mass[j])] + [j for j in rest if np.isnan(mass[j])]
    return sorted(nan_last[:k - r]) + list(range(n - r, n))


def gather_rows(pool, scale, table, n, head):
    """cached_rows in one gather, for long contexts."""
    blocks = table[:-(-n // 16)].long()
    x = pool[blocks, head].reshape(-1, pool.shape[-1])[:n]
    if pool.dtype == torch.uint8:
        x = torch.stack([x & 15, x >> 4], -1).flatten(1).to(torch.int16)
        x = torch.where(x > 7, x - 16, x)
    x = x.double()
    return x if scale is None else x * scale[blocks, head].reshape(-1)[:n, None].double()

"""K that is not finite where a token looks, in pa_window_attention and pa_window_decode: the row
is what softmax gives. A score of minus infinity has weight 0; plus infinity, NaN, and a row of
minus infinities alone make the row NaN; rows of zeros mean that nothing is seen."""
import pytest
import torch

import paged_kv_cache_94_gb300 as pa
from tests.plain_attention import gather_rows
from tests.plain_window import attend_seen, seen_keys
from tests.test_gpu_window_attention import attend
from tests.test_gpu_window_decode import case, decode

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = 64


def pool_and_queries(kv, g, new, n):
    """Queries and K of which value 0 alone decides the sign of a score: q[0] = 1, k >= 0
    elsewhere 0, so that K rows of value x at 0 score x."""
    q, cu, pool, bt = case(kv, D, g, 1, [new], [n], seed=60 + new)
    q.zero_()
    q[..., 0] = 1.0
    kc, _, ks, _ = pool
    kc.zero_()
    if kv == "bf16":
        kc[..., 0] = torch.randn(kc.shape[:3], generator=torch.Generator().manual_seed(1)).to(kc)
    else:
        kc[..., 0] = 1  # (INT4: the low nibble)
        ks.copy_(torch.randn(ks.shape, generator=torch.Generator().manual_seed(1)).abs())
    return q, cu, pool, bt


def put(pool, bt, kv, keys, x):
    kc, _, ks, _ = pool
    for j in keys:
        if kv == "bf16":
            kc[int(bt[0, j // 16]), 0, j % 16, 0] = x
        else:
            ks[int(bt[0, j // 16]), 0, j % 16] = x


CASES = {
    "one_minus": (lambda n: [n - 30], float("-inf")),
    "one_plus": (lambda n: [n - 30], float("inf")),
    "one_nan": (lambda n: [n - 30], float("nan")),
    "a_stretch_of_nan": (lambda n: range(n - 90, n - 20), float("nan")),
    "all_minus": (lambda n: range(n), float("-inf")),
    "all_nan": (lambda n: range(n), float("nan")),
    "late_minus": (lambda n: range(n - 60, n), float("-inf")),
}


@pytest.mark.parametrize("what", CASES)
@pytest.mark.parametrize("window,n_first", [(0, 0), (40, 0), (40, 20)])
@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_k_that_is_not_finite(kv, window, n_first, what):
    n = 700
    keys, x = CASES[what][0](n), CASES[what][1]
    for g, new in ((1, 1), (8, 1), (1, 200), (4, 40), (2, 90)):
        q, cu, pool, bt = pool_and_queries(kv, g, new, n)
        put(pool, bt, kv, keys, x)
        seen = seen_keys(new, n, window, n_first)
        t = torch.zeros(n, dtype=torch.bool)
        t[list(keys)] = True
        bad = seen & t
        if x == float("-inf"):
            nan = bad.sum(1) == seen.sum(1)
        else:
            nan = bad.any(1)
        host = [None if y is None else y.cpu() for y in pool]
        k, v = (gather_rows(host[i], host[2 + i], bt[0], n, 0) for i in (0, 1))
        few = (seen & ~t).repeat_interleave(g, 0)
        codes = kv != "bf16" and new == 1  # (the decode: weights in one fp16 part)
        ref, tol = attend_seen(q.cpu().double().flatten(0, 1), k, v, 0.5, few,
                               2.0 ** -11 if codes else 2.0 ** -16, float(v.abs().max()))
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
        ref, tol = ref.view(new, g, D), tol.view(new, g, D)
        for num_ctas in (0, 1, 9):
            outs = [attend(q, cu, pool, bt, [n], 0.5, window, n_first, num_ctas=num_ctas)]
            if new == 1:
                outs.append(decode(q, pool, bt, [n], 0.5, window, n_first, num_ctas=num_ctas))
            for i, (out, st) in enumerate(outs):
                assert st == 0
                out = out.cpu()
                assert torch.isnan(out[nan]).all(), (g, new, num_ctas, i)
                assert torch.isfinite(out[~nan]).all(), (g, new, num_ctas, i)
                if x == float("-inf"):  # as if those keys were not there
                    got = out[~nan].double().flatten(0, 1)
                    assert ((got - ref[~nan].flatten(0, 1)).abs() <= tol[~nan].flatten(0, 1)).all()


@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_rows_that_see_nothing_stay_zero(kv):
    """Bad blocks alone, or no position at all: zeros, whatever the pool holds."""
    n = 80
    for g, new in ((1, 1), (2, 1), (1, 70), (4, 90)):
        q, cu, pool, bt = pool_and_queries(kv, g, new, n)
        put(pool, bt, kv, range(n), float("nan"))
        bt = torch.full_like(bt, -3)
        for num_ctas in (0, 1, 9):
            out, st = attend(q, cu, pool, bt, [n], 0.5, 30, 5, num_ctas=num_ctas)
            assert st == pa.PA_DEV_BAD_BLOCK and (out == 0).all()
            if new == 1:
                out, st = decode(q, pool, bt, [n], 0.5, 30, 5, num_ctas=num_ctas)
                assert st == pa.PA_DEV_BAD_BLOCK and (out == 0).all()


@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_minus_infinity_next_to_bad_blocks(kv):
    """Of what a row sees one block is bad and the rest scores minus infinity: NaN; where the rest
    is bad too: zeros."""
    n, new, window = 96, 96, 20
    q, cu, pool, bt = pool_and_queries(kv, 2, new, n)
    put(pool, bt, kv, range(n), float("-inf"))
    gone = [0, 1, 4]  # blocks
    bt[0, gone] = pool[0].shape[0] + 5
    good = torch.ones(n, dtype=torch.bool)
    for i in gone:
        good[16 * i:16 * i + 16] = False
    sees = (seen_keys(new, n, window, 3) & good).any(1)
    assert 0 < int(sees.sum()) < new
    for num_ctas in (0, 1, 9):
        out, st = attend(q, cu, pool, bt, [n], 0.5, window, 3, num_ctas=num_ctas)
        out = out.cpu()
        assert st == pa.PA_DEV_BAD_BLOCK
        assert torch.isnan(out[sees]).all() and (out[~sees] == 0).all()
    out, st = decode(q[-1:], pool, bt, [n], 0.5, window, 3)
    assert st == pa.PA_DEV_BAD_BLOCK and torch.isnan(out).all()

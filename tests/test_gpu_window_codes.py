"""pa_window_decode over INT8 and INT4 pools at the tolerance of every operator here,
|d| <= 1e-2 (1 + |ref|) per element, over the dynamic ranges that real K/V reach
(workloads.PROFILES), and at the tolerance of its own arithmetic (tests/plain_window_codes.py),
which a block left out does not pass."""
import math

import pytest
import torch

import paged_kv_cache_94_gb300 as pa
from tests.gpu_helpers import assert_close, gpu_pool
from tests.plain_attention import gather_rows
from tests.plain_window import attend_seen, seen_keys
from tests.plain_window_codes import check_codes
from tests.range_cases import HEAD_DIMS, PROFILES, workload
from tests.test_gpu_evict import poison
from tests.test_gpu_window_decode import case, decode, give_back

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("d_h", HEAD_DIMS)
@pytest.mark.parametrize("kv", ["int8", "int4"])
def test_dynamic_range(kv, d_h, profile):
    for g in (1, 8):
        w = workload("window_range", 7100 + g, kv, d_h, g, profile, "plain")
        pool = gpu_pool(w, DEV, fill_nan=True)
        host = [t.cpu() for t in pool]
        table, ctx = torch.from_numpy(w.block_tables), w.context_lens.tolist()
        q = w.q()
        for window, n_first in ((0, 0), (300, 17), (300, 0), (40, 5)):
            ref = torch.zeros(q.shape, dtype=torch.float64)
            for b, n in enumerate(ctx):
                seen = seen_keys(1, n, window, n_first).expand(g, n)
                for h in range(w.geom.n_kv):
                    heads = slice(h * g, (h + 1) * g)
                    k, v = (gather_rows(host[i], host[2 + i], table[b], n, h) for i in (0, 1))
                    ref[b, heads], _ = attend_seen(q[b, heads].double(), k, v, w.scale, seen)
            for num_ctas in (0, 1, 300):
                out, st = decode(q.to(DEV), pool, table, ctx, w.scale, window, n_first, num_ctas=num_ctas)
                assert st == 0
                what = f"g{g} window{window}+{n_first} ctas{num_ctas}"
                assert_close(out.float().cpu().numpy(), ref.numpy(), what)
                check_codes(out, q, pool, table, ctx, w.scale, window, n_first)


@pytest.mark.parametrize("window,n_first", [(0, 0), (1, 4), (130, 0), (200, 150), (64, 5000), (48, 33)])
@pytest.mark.parametrize("g", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", ["int8", "int4"])
def test_ragged_contexts(kv, d, g, window, n_first):
    """Values of an ordinary size, and V scales 40 and 1000 times that here and there: items of
    one part, of two, and runs that change from one to the other."""
    ctx = [1, 0, 17, 33, 64, 65, 130, 500, 3001, 16, 48, 49]
    q, _, pool, bt = case(kv, d, g, 2, [1] * len(ctx), ctx, seed=50 + g)
    poison(pool, bt, ctx)
    bt = give_back(bt, ctx, [1] * len(ctx), window, n_first)
    scale = 1 / math.sqrt(d)
    gen = torch.Generator().manual_seed(51)
    plain = pool[3].clone()
    for factors in ((1.0,), (1.0, 1.0, 40.0), (1.0, 0.01, 1000.0)):
        pick = torch.randint(0, len(factors), plain.shape[:2], generator=gen)
        pool[3] = plain * torch.tensor(factors)[pick].to(DEV)[..., None]
        for num_ctas in (0, 1, 7):
            out, st = decode(q, pool, bt, ctx, scale, window, n_first, num_ctas=num_ctas)
            assert st == 0
            check_codes(out, q, pool, bt, ctx, scale, window, n_first)


@pytest.mark.parametrize("kv", ["int8", "int4"])
def test_long_contexts(kv):
    ctx = [40000, 9001, 20016]
    q, _, pool, bt = case(kv, 128, 4, 2, [1] * 3, ctx, seed=52)
    for window, n_first in ((0, 0), (16000, 500)):
        for num_ctas in (0, 3):
            out, st = decode(q, pool, bt, ctx, 0.09, window, n_first, num_ctas=num_ctas)
            assert st == 0
            check_codes(out, q, pool, bt, ctx, 0.09, window, n_first)


@pytest.mark.parametrize("kv", ["int8", "int4"])
def test_without_a_window_large_values_stay_close_to_pa_decode(kv):
    """Where V is large the two differ by what pa_decode rounds, no more: 2^-11 of the weighted
    magnitudes, and the rounding of both outputs."""
    ctx = [700, 33, 4100, 128, 5]
    q, _, pool, bt = case(kv, 128, 4, 2, [1] * 5, ctx, seed=53)
    pool[3] = pool[3] * 300
    cl = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    want = pa.pa_decode(q, pool[0], pool[1], bt.to(DEV), cl, 0.09, k_scale=pool[2], v_scale=pool[3],
                        num_ctas=50).double()
    out, _ = decode(q, pool, bt, ctx, 0.09, 0, 0, num_ctas=50)
    top = float(pool[3].max()) * (128 if kv == "int8" else 8)
    tol = 2 * 2.0 ** -11 * top + 2.0 ** -7 * want.abs()
    assert ((out.double() - want).abs() <= tol).all()

"""pa_window_decode over INT8 and INT4 pools at the tolerance of every operator here,
|d| <= 1e-2 (1 + |ref|) per element, over the dynamic ranges that real K/V reach
(workloads.PROFILES)."""
import pytest
import torch

import paged_kv_cache_94_gb300 as pa
from tests.gpu_helpers import assert_close, gpu_pool
from tests.plain_attention import gather_rows
from tests.plain_window import attend_seen, seen_keys
from tests.range_cases import HEAD_DIMS, PROFILES, workload
from tests.test_gpu_window_decode import case, decode

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

"""pa_window_attention and pa_window_decode over the dynamic ranges that real K/V reach
(workloads.PROFILES), at the tolerance that every decode of these pools meets: |d| <=
1e-2 (1 + |ref|) per element, with V rows whose magnitudes span 1e-3 .. 1e3 and cancel among
them. 40 new tokens per sequence (40 packed rows of a kv head with g = 1, 320 with g = 8),
and one; no window, and windows with first tokens.

The decode of INT8 and INT4 pools is held to its own arithmetic instead (tests/plain_window.py):
a weight times its V scale is one fp16 value, off by up to 2^-11, and a window of 300 tokens
leaves rows of weights over |v| of up to 1e3 whose sum, sum_j w_j |v_j|, passes 250: 2^-11 of
that is 0.12, more than 1e-2 (1 + |ref|) where the terms cancel to an |ref| below 11."""
import pytest
import torch

import paged_kv_cache_94_gb300 as pa
from tests.gpu_helpers import assert_close, gpu_pool
from tests.plain_attention import gather_rows
from tests.plain_window import attend_seen, seen_keys
from tests.range_cases import HEAD_DIMS, POOLS, PROFILES, workload

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("d_h", HEAD_DIMS)
@pytest.mark.parametrize("kv_dtype", POOLS)
def test_window_dynamic_range(kv_dtype, d_h, profile):
    for g in (1, 8):
        w = workload("window_range", 7100 + g, kv_dtype, d_h, g, profile, "plain")
        pool = gpu_pool(w, DEV, fill_nan=True)
        host = [None if t is None else t.cpu() for t in pool]
        table = torch.from_numpy(w.block_tables)
        ctx = torch.from_numpy(w.context_lens)
        for nq, window, n_first in ((40, 0, 0), (40, 200, 5), (1, 0, 0), (1, 300, 17)):
            f = torch.linspace(1.0, 0.5, nq)[None, :, None, None]
            q = (w.q().float()[:, None] * f).to(torch.bfloat16)
            ref = torch.zeros(q.shape, dtype=torch.float64)
            own = torch.zeros(q.shape, dtype=torch.float64)
            for b in range(w.B):
                n = int(w.context_lens[b])
                early = max(0, nq - n)
                if early == nq:
                    continue
                seen = seen_keys(nq - early, n, window, n_first).repeat_interleave(g, 0)
                for h in range(w.geom.n_kv):
                    heads = slice(h * g, (h + 1) * g)
                    k = gather_rows(host[0], host[2], table[b], n, h)
                    v = gather_rows(host[1], host[3], table[b], n, h)
                    x = q[b, early:, heads].double().reshape(-1, d_h)
                    used = torch.where(seen.any(0)[:, None], v, 0.0)
                    o, tol = attend_seen(x, k, v, w.scale, seen, 2.0 ** -11,
                                         128 * float(used.abs().max()))
                    ref[b, early:, heads] = o.view(-1, g, d_h)
                    own[b, early:, heads] = (tol + 2.0 ** -8 * (o.abs() + tol)).view(-1, g, d_h)
            cu = (torch.arange(w.B + 1, dtype=torch.int32) * nq).to(DEV)
            for num_ctas in (0, 1, 300):
                status = torch.zeros(1, dtype=torch.int32, device=DEV)
                kw = dict(window=window, n_first=n_first, k_scale=pool[2], v_scale=pool[3],
                          dev_status=status, num_ctas=num_ctas)
                args = (pool[0], pool[1], table.to(DEV), ctx.to(DEV), w.scale)
                what = f"g{g} nq{nq} window{window} ctas{num_ctas}"
                out = pa.pa_window_attention(q.flatten(0, 1).to(DEV), cu, *args, **kw)
                assert_close(out.float().cpu().numpy(), ref.flatten(0, 1).numpy(), what)
                if nq == 1:
                    out = pa.pa_window_decode(q[:, 0].contiguous().to(DEV), *args, **kw)
                    if kv_dtype == "bf16":
                        assert_close(out.float().cpu().numpy(), ref[:, 0].numpy(), what)
                    else:
                        assert ((out.cpu().double() - ref[:, 0]).abs() <= own[:, 0] + 1e-30).all(), what
                torch.cuda.synchronize()
                assert int(status.item()) == 0

"""pa_cross_attention over the dynamic ranges that real K/V reach (workloads.PROFILES),
at the tolerance that every decode of these pools meets: |d| <= 1e-2 (1 + |ref|) per
element, with V rows whose magnitudes span 1e-3 .. 1e3 and cancel among them. A weight
may then be off by no more than about 2^-14 relative, so one rounding of it to bf16
(2^-8) is too much.

One query per sequence (a unit of one half, few live rows), and 40 per sequence: 40 packed
rows of a kv head with g = 1 (one half), 320 with g = 8 (two halves, then one)."""
import pytest
import torch

import paged_kv_cache_94_gb300 as pa
from tests.gpu_helpers import assert_close, gpu_pool
from tests.plain_attention import attend, gather_rows
from tests.range_cases import HEAD_DIMS, POOLS, PROFILES, workload

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("d_h", HEAD_DIMS)
@pytest.mark.parametrize("kv_dtype", POOLS)
def test_cross_attention_dynamic_range(kv_dtype, d_h, profile):
    for g in (1, 8):
        w = workload("cross_range", 7000 + g, kv_dtype, d_h, g, profile, "plain")
        pool = gpu_pool(w, DEV, fill_nan=True)
        host = [None if t is None else t.cpu() for t in pool]
        table = torch.from_numpy(w.block_tables)
        for nq in (1, 40):
            # token t of a sequence: its query, shrunk a little more at every token
            f = torch.linspace(1.0, 0.5, nq)[None, :, None, None]
            q = (w.q().float()[:, None] * f).to(torch.bfloat16)
            ref = torch.empty(q.shape, dtype=torch.float64)
            for b in range(w.B):
                n = int(w.context_lens[b])
                for h in range(w.geom.n_kv):
                    heads = slice(h * g, (h + 1) * g)
                    k = gather_rows(host[0], host[2], table[b], n, h)
                    v = gather_rows(host[1], host[3], table[b], n, h)
                    o, _, _ = attend(q[b, :, heads].double().reshape(-1, d_h), k, v, w.scale)
                    ref[b, :, heads] = o.view(nq, g, d_h)
            cu = (torch.arange(w.B + 1, dtype=torch.int32) * nq).to(DEV)
            for num_ctas in (0, 1, 300):
                status = torch.zeros(1, dtype=torch.int32, device=DEV)
                out = pa.pa_cross_attention(
                    q.flatten(0, 1).to(DEV), cu, pool[0], pool[1], table.to(DEV),
                    torch.from_numpy(w.context_lens).to(DEV), w.scale, k_scale=pool[2],
                    v_scale=pool[3], dev_status=status, num_ctas=num_ctas)
                torch.cuda.synchronize()
                assert int(status.item()) == 0
                assert_close(out.float().cpu().numpy(), ref.flatten(0, 1).numpy(),
                             f"g{g} nq{nq} ctas{num_ctas}")

"""pa_window_decode on the GPU against the plain form in 64 bits (tests/plain_window.py has
the tolerances): windows and first tokens of every kind over ragged contexts, pool types and
head layouts, forced splits, blocks given back, values that are not finite where a token
does not look, reports, streams and graphs."""
import math

import pytest
import torch

import paged_kv_cache_94_gb300 as pa
from tests.plain_window import check_window, seen_keys
from tests.test_gpu_evict import make_pool, make_tables, poison

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MASKS = [(0, 0), (1, 0), (1, 4), (33, 17), (130, 0), (200, 150), (64, 5000), (100000, 3)]


def case(kv, d, g, n_kv, q_lens, ctx, seed=0, lead=0, pad=0, extra=1):
    gen = torch.Generator().manual_seed(seed)
    bt, total, _ = make_tables(gen, ctx, extra=extra)
    pool = make_pool(gen, total, n_kv, d, kv)
    cu = torch.tensor([lead] + q_lens).cumsum(0).to(torch.int32)
    q = (2 * torch.randn(int(cu[-1]) + pad, n_kv * g, d, generator=gen)).to(torch.bfloat16)
    return q.to(DEV), cu, pool, bt


def give_back(bt, ctx, q_lens, window, n_first):
    """Table entries of blocks that no new token sees become junk."""
    bt = bt.clone()
    if window == 0:
        return bt
    for b, (n, new) in enumerate(zip(ctx, q_lens)):
        seen = seen_keys(min(n, new), n, window, n_first).any(0)
        for i in range(-(-n // 16)):
            if not seen[16 * i:16 * i + 16].any():
                bt[b, i] = (-7, 1 << 30)[i % 2]
    return bt


def decode(q, pool, bt, ctx, scale, window, n_first, **kw):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pa.pa_window_decode(q, pool[0], pool[1], bt.to(DEV),
                              torch.tensor(ctx, dtype=torch.int32, device=DEV), scale,
                              window=window, n_first=n_first, k_scale=pool[2], v_scale=pool[3],
                              dev_status=status, **kw)
    torch.cuda.synchronize()
    return out, int(status.item())


def check_decode(out, q, pool, bt, ctx, scale, window, n_first, **kw):
    codes = pool[0].dtype != torch.bfloat16
    check_window(out, q, range(len(ctx) + 1), pool, bt, ctx, scale, window, n_first,
                 first_part=2.0 ** -11 if codes else 2.0 ** -16, codes_in_16=codes, **kw)


@pytest.mark.parametrize("window,n_first", MASKS + [(16, 16), (17, 15), (48, 33), (2, 1)])
@pytest.mark.parametrize("g", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_ragged_contexts(kv, d, g, window, n_first):
    ctx = [1, 0, 17, 33, 64, 65, 130, 500, 3001, 16, 48, 49]
    q, _, pool, bt = case(kv, d, g, 2, [1] * len(ctx), ctx, seed=20 + g)
    poison(pool, bt, ctx)
    bt = give_back(bt, ctx, [1] * len(ctx), window, n_first)
    scale = 1 / math.sqrt(d)
    for num_ctas in (0, 1, 7):
        out, st = decode(q, pool, bt, ctx, scale, window, n_first, num_ctas=num_ctas)
        assert st == 0
        check_decode(out, q, pool, bt, ctx, scale, window, n_first)


@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_what_it_does_not_see_may_be_anything(kv):
    """Every position outside the window and the first tokens holds NaN (or a NaN scale)."""
    ctx, window, n_first, d = [700, 90, 41], 37, 5, 128
    q, _, pool, bt = case(kv, d, 4, 2, [1] * 3, ctx, seed=21)
    want, _ = decode(q, pool, bt, ctx, 0.1, window, n_first)
    check_decode(want, q, pool, bt, ctx, 0.1, window, n_first)
    for b, n in enumerate(ctx):
        for j in (~seen_keys(1, n, window, n_first)[0]).nonzero().flatten().tolist():
            for t in (pool[2:] if kv != "bf16" else pool[:2]):
                t[int(bt[b, j // 16]), :, j % 16] = float("nan")
    out, st = decode(q, pool, bt, ctx, 0.1, window, n_first)
    assert st == 0 and torch.equal(out, want)


def test_without_a_window_it_is_pa_decode():
    """Bit for bit on the same grid: window 0 or longer than every context, all tokens first;
    and without first tokens it is pa_decode's window."""
    ctx = [700, 33, 4100, 128, 5]
    for kv in ("bf16", "int8", "int4"):
        q, _, pool, bt = case(kv, 128, 4, 2, [1] * 5, ctx, seed=22)
        cl = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        want = pa.pa_decode(q, pool[0], pool[1], bt.to(DEV), cl, 0.09, k_scale=pool[2],
                            v_scale=pool[3], num_ctas=50)
        for window, n_first in ((0, 0), (0, 7), (5000, 0), (5000, 40), (10, 4100)):
            out, _ = decode(q, pool, bt, ctx, 0.09, window, n_first, num_ctas=50)
            assert torch.equal(out, want), (kv, window, n_first)
        want = pa.pa_decode(q, pool[0], pool[1], bt.to(DEV), cl, 0.09, k_scale=pool[2],
                            v_scale=pool[3], num_ctas=50, window=200)
        out, _ = decode(q, pool, bt, ctx, 0.09, 200, 0, num_ctas=50)
        assert torch.equal(out, want), kv


def test_reports():
    ctx = [100, 300, 64, 50]
    q, _, pool, bt = case("bf16", 128, 2, 2, [1] * 4, ctx, seed=23, extra=0)
    want, _ = decode(q, pool, bt, ctx, 0.1, 40, 20)
    bt2 = bt.clone()
    bt2[1, 18], bt2[1, 7] = -7, 1 << 30  # the second is not seen
    ctx2 = [100, 300, bt.shape[1] * 16 + 1, -1]
    out, st = decode(q, pool, bt2, ctx2, 0.1, 40, 20)
    assert st == pa.PA_DEV_BAD_BLOCK | pa.PA_DEV_BAD_CONTEXT
    assert torch.equal(out[0], want[0]) and (out[2:] == 0).all()
    assert torch.isfinite(out[1]).all()


def test_eight_thousand_sequences():
    B = 8192
    gen = torch.Generator().manual_seed(11)
    ctx = torch.randint(0, 60, (B,), generator=gen).tolist()
    q, _, pool, bt = case("bf16", 64, 2, 1, [1] * B, ctx, seed=11)
    out, st = decode(q, pool, bt, ctx, 0.125, 20, 3)
    assert st == 0
    check_decode(out, q, pool, bt, ctx, 0.125, 20, 3,
                 seqs=list(range(0, 60)) + list(range(B - 60, B)))


def test_two_graphs_and_two_streams_at_once():
    """Captured twice and replayed together, then called on two streams at once: every call
    has a workspace of its own."""
    ctx, runs = [5000, 900], []
    for i in range(2):
        q, _, pool, bt = case("bf16", 128, 4, 2, [1, 1], ctx, seed=30 + i)
        args = (q, pool[0], pool[1], bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV),
                0.1, 3000, 4)
        want = pa.pa_window_decode(*args)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = pa.pa_window_decode(*args)
        runs.append((graph, s, out, want, args))
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, s, *_ in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for graph, s, out, want, args in runs:
        assert torch.equal(out, want)
    got = []
    for _ in range(10):
        for graph, s, out, want, args in runs:
            got.append((pa.pa_window_decode(*args, stream=s), want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)
    calls = [(pa.pa_window_decode(*r[4], prepare=True), r[3]) for r in runs]
    for call, want in calls * 2:
        assert torch.equal(call(), want)

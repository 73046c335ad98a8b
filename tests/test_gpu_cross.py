"""pa_cross_attention on the GPU against the plain form in 64 bits: ragged queries
and contexts, every pool type and head layout, forced splits, value ranges,
reports, streams and graphs.

Tolerance per element: a weight is off by its own error e (plain_attention) and one
rounding to bf16 (2^-8 relative), so the sum by (2^-8 + e) sum_j w_j |v_j|; fp32 sums
and the merge add 2^-18 of that; the output is rounded once more, 2^-8 |out|."""
import math

import pytest
import torch

import paged_kv_cache_94_gb300 as pa
from tests.plain_attention import attend, cached_rows, gather_rows
from tests.test_gpu_evict import make_pool, make_tables, poison

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def check(out, q, cu, pool, bt, ctx, scale, seqs=None, skip=()):
    """out against the plain form, for the sequences `seqs` (default all)."""
    kc, vc, ks, vs = [None if t is None else t.cpu() for t in pool]
    q, out = q.cpu().double(), out.cpu()
    n_kv = kc.shape[1]
    g = q.shape[1] // n_kv
    for b in range(len(ctx)) if seqs is None else seqs:
        lo, hi = int(cu[b]), int(cu[b + 1])
        if lo == hi or b in skip:
            continue
        for h in range(n_kv):
            k, v = gather_rows(kc, ks, bt[b], ctx[b], h), gather_rows(vc, vs, bt[b], ctx[b], h)
            heads = slice(h * g, (h + 1) * g)
            x = q[lo:hi, heads].reshape(-1, q.shape[2])
            got = out[lo:hi, heads].reshape(-1, q.shape[2]).double()
            o, w, e = attend(x, k, v, scale)
            if ctx[b] == 0:
                assert (got == 0).all()
                continue
            tol = (2.0 ** -8 + 2.0 ** -18 + e) * (w @ v.abs()) + 2.0 ** -8 * o.abs() * 1.01
            bad = ~((got - o).abs() <= tol + 1e-30)
            assert not bad.any(), (b, h, int(bad.sum()), float((got - o).abs().max()),
                                   bad.nonzero()[:4].tolist())


def case(kv, d, g, n_kv, q_lens, ctx, seed=0, lead=0, pad=0, q_scale=2.0, extra=1):
    gen = torch.Generator().manual_seed(seed)
    bt, total, _ = make_tables(gen, ctx, extra=extra)
    pool = make_pool(gen, total, n_kv, d, kv)
    cu = torch.tensor([lead] + q_lens).cumsum(0).to(torch.int32)
    q = (q_scale * torch.randn(int(cu[-1]) + pad, n_kv * g, d, generator=gen)).to(torch.bfloat16)
    return q.to(DEV), cu, pool, bt


def run(q, cu, pool, bt, ctx, scale, **kw):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pa.pa_cross_attention(q, cu.to(DEV), pool[0], pool[1], bt.to(DEV),
                                torch.tensor(ctx, dtype=torch.int32, device=DEV), scale,
                                k_scale=pool[2], v_scale=pool[3], dev_status=status, **kw)
    torch.cuda.synchronize()
    return out, int(status.item())


def test_gathered_rows_are_the_cached_rows():
    gen = torch.Generator().manual_seed(0)
    bt, total, _ = make_tables(gen, [37])
    for kv in ("bf16", "int8", "int4"):
        pool = [None if t is None else t.cpu() for t in make_pool(gen, total, 2, 64, kv)]
        assert torch.equal(gather_rows(pool[0], pool[2], bt[0], 37, 1),
                           cached_rows(pool[0], pool[2], bt[0], 37, 1))


@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("d", [128, 64])
def test_one_token_one_tile(d, kv):
    q, cu, pool, bt = case(kv, d, 1, 1, [1], [16])
    out, st = run(q, cu, pool, bt, [16], 1 / math.sqrt(d))
    assert st == 0
    check(out, q, cu, pool, bt, [16], 1 / math.sqrt(d))


Q_LENS = [1, 0, 3, 17, 130, 2, 300, 64, 5]
CTX = [5, 40, 0, 127, 129, 1, 257, 128, 1000]


@pytest.mark.parametrize("num_ctas", [0, 1, 7])
@pytest.mark.parametrize("g", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_ragged_queries_over_ragged_contexts(kv, d, g, num_ctas):
    q, cu, pool, bt = case(kv, d, g, 2, Q_LENS, CTX, seed=g, lead=3, pad=9)
    poison(pool, bt, CTX)
    out = torch.full_like(q, 5.0)
    scale = 1 / math.sqrt(d)
    _, st = run(q, cu, pool, bt, CTX, scale, out=out, num_ctas=num_ctas)
    assert st == 0
    assert (out[:3] == 5.0).all() and (out[-9:] == 5.0).all()  # no sequence's rows
    check(out, q, cu, pool, bt, CTX, scale)


@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("d,g,n_kv", [(128, 4, 2), (64, 1, 3)])
def test_prompts_over_long_contexts(d, g, n_kv, kv):
    q_lens, ctx = [700, 65, 1], [3001, 2048, 4999]
    q, cu, pool, bt = case(kv, d, g, n_kv, q_lens, ctx, seed=3)
    out, st = run(q, cu, pool, bt, ctx, 1 / math.sqrt(d))
    again, _ = run(q, cu, pool, bt, ctx, 1 / math.sqrt(d))
    assert st == 0 and torch.equal(out, again)
    check(out, q, cu, pool, bt, ctx, 1 / math.sqrt(d))


@pytest.mark.parametrize("num_ctas", [0, 2, 3, 40, 300])
@pytest.mark.parametrize("kv", ["bf16", "int4"])
def test_one_long_context_is_split_and_merged(kv, num_ctas):
    """Few query rows over long contexts: many CTAs a unit, one merge."""
    q_lens, ctx = [1, 2], [20000, 7777]
    q, cu, pool, bt = case(kv, 128, 4, 1, q_lens, ctx, seed=4)
    for _ in range(3):  # the counters are left zero
        out, st = run(q, cu, pool, bt, ctx, 0.1, num_ctas=num_ctas)
    assert st == 0
    check(out, q, cu, pool, bt, ctx, 0.1)


@pytest.mark.parametrize("kind", ["rising", "falling", "big", "flat", "negative", "v_range"])
@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_value_ranges(kv, kind):
    """Scores that climb tile after tile (the softmax base moves), fall, are huge, all
    equal, or negated; V rows over six decades."""
    n, d = 1500, 128
    q, cu, pool, bt = case(kv, d, 2, 1, [150], [n], seed=5)
    scale = 1 / math.sqrt(d)
    if kind in ("rising", "falling"):
        q = q.abs()
        steps = torch.linspace(0.05, 3.0, n)
        if kind == "falling":
            steps = steps.flip(0)
        for j in range(n):
            at = (bt[0, j // 16].long(), slice(None), j % 16)
            if kv == "bf16":
                pool[0][at] = pool[0][at].abs() * float(steps[j])
            else:
                pool[0][at] = pool[0][at].abs()
                pool[2][at] *= float(steps[j])
    elif kind == "big":
        q = q * 40
    elif kind == "flat":
        scale = 0.0
    elif kind == "negative":
        scale = -scale
    else:
        gen = torch.Generator().manual_seed(6)
        f = 10 ** (6 * torch.rand(pool[1].shape[:3], generator=gen) - 3).to(DEV)
        if kv == "bf16":
            pool[1] = (pool[1].float() * f[..., None]).to(torch.bfloat16)
        else:
            pool[3] = pool[3] * f
    for num_ctas in (0, 1):
        out, st = run(q, cu, pool, bt, [n], scale, num_ctas=num_ctas)
        assert st == 0
        check(out, q, cu, pool, bt, [n], scale)


@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_many_short_segments_per_cta(kv):
    """Units of one or two key tiles, many to a CTA: the stages hand over at every tile."""
    gen = torch.Generator().manual_seed(12)
    q_lens = torch.randint(1, 300, (60,), generator=gen).tolist()
    ctx = torch.randint(1, 400, (60,), generator=gen).tolist()
    q, cu, pool, bt = case(kv, 128, 1, 4, q_lens, ctx, seed=12)
    for num_ctas in (0, 5):
        out, st = run(q, cu, pool, bt, ctx, 0.09, num_ctas=num_ctas)
        assert st == 0
        check(out, q, cu, pool, bt, ctx, 0.09)


def test_single_queries_agree_with_the_decode():
    ctx = [700, 33, 4100, 128]
    q, cu, pool, bt = case("bf16", 128, 4, 2, [1] * 4, ctx, seed=7)
    out, _ = run(q, cu, pool, bt, ctx, 0.09)
    dec = pa.pa_decode(q, pool[0], pool[1], bt.to(DEV),
                       torch.tensor(ctx, dtype=torch.int32, device=DEV), 0.09)
    check(out, q, cu, pool, bt, ctx, 0.09)
    check(dec, q, cu, pool, bt, ctx, 0.09)


def test_non_finite_rows_stay_their_own():
    """A query of NaN or infinities changes no other row's result."""
    ctx = [300]
    q, cu, pool, bt = case("bf16", 64, 1, 1, [200], ctx, seed=8)
    want, _ = run(q, cu, pool, bt, ctx, 0.1)
    q[7] = float("nan")
    q[130] = float("inf")
    out, st = run(q, cu, pool, bt, ctx, 0.1)
    assert st == 0 and torch.isnan(out[7]).all() and torch.isnan(out[130]).all()
    rest = [i for i in range(200) if i not in (7, 130)]
    assert torch.equal(out[rest], want[rest])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_non_finite_rows_stay_their_own_in_every_pool(kv, d):
    """Each row of a group of four that lie eight apart (a thread of the quantised softmax has
    them) and its neighbours, in a unit of one half (90 rows) and in one of two (250)."""
    ctx = [700, 333]
    q, cu, pool, bt = case(kv, d, 1, 1, [90, 250], ctx, seed=13)
    want = {c: run(q, cu, pool, bt, ctx, 0.1, num_ctas=c)[0] for c in (0, 1)}
    for odd, value in (((3, 13, 49, 90 + 5, 90 + 140), float("nan")),
                       ((11, 27, 60, 90 + 21, 90 + 200), float("inf")),
                       ((19, 34, 89, 90, 90 + 249), -float("inf"))):
        x = q.clone()
        x[list(odd)] = value
        for num_ctas in (0, 1):
            out, st = run(x, cu, pool, bt, ctx, 0.1, num_ctas=num_ctas)
            assert st == 0 and torch.isnan(out[list(odd)]).all()
            rest = [i for i in range(340) if i not in odd]
            assert torch.equal(out[rest], want[num_ctas][rest])


@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_reports(kv):
    ctx = [100, 300, 64, 50, 20]
    q_lens = [3, 40, 2, 4, 5]
    q, cu, pool, bt = case(kv, 128, 2, 2, q_lens, ctx, seed=9, extra=0)
    want, _ = run(q, cu, pool, bt, ctx, 0.1)
    bt2 = bt.clone()
    bt2[1, 5], bt2[1, 18] = -7, pool[0].shape[0]       # tokens 80 .. 95 and 288 .. 299
    ctx2 = [100, 300, bt.shape[1] * 16 + 1, -1, 20]
    out, st = run(q, cu, pool, bt2, ctx2, 0.1, out=torch.full_like(q, 5.0))
    assert st == pa.PA_DEV_BAD_BLOCK | pa.PA_DEV_BAD_CONTEXT
    assert torch.equal(out[:3], want[:3]) and torch.equal(out[49:], want[49:])
    assert (out[43:49] == 0).all()
    # sequence 1 without the bad blocks' tokens
    keep = [j for j in range(300) if j // 16 not in (5, 18)]
    kc, vc, ks, vs = [None if t is None else t.cpu() for t in pool]
    for h in range(2):
        k, v = (gather_rows(p, s, bt[1], 300, h)[keep] for p, s in ((kc, ks), (vc, vs)))
        x = q[3:43, 2 * h:2 * h + 2].cpu().double().reshape(-1, 128)
        o, w, e = attend(x, k, v, 0.1)
        got = out[3:43, 2 * h:2 * h + 2].cpu().double().reshape(-1, 128)
        tol = (2.0 ** -8 + 2.0 ** -18 + e) * (w @ v.abs()) + 2.0 ** -8 * o.abs() * 1.01
        assert ((got - o).abs() <= tol).all()
    # offsets that decrease, or leave the tokens
    for i, bad in ((2, 2), (5, 1000), (0, -4)):
        cu2 = cu.clone()
        cu2[i] = bad
        out, st = run(q, cu2, pool, bt, ctx, 0.1, out=torch.full_like(q, 5.0))
        assert st == pa.PA_DEV_BAD_CONTEXT
        for b in range(5):
            lo, hi = int(cu2[b]), int(cu2[b + 1])
            if 0 <= lo <= hi <= q.shape[0] and (lo, hi) == (int(cu[b]), int(cu[b + 1])):
                # (with decreasing offsets the next sequence claims some of these rows too)
                rows = [t for t in range(lo, hi)
                        if not any(c != b and int(cu2[c]) <= t < int(cu2[c + 1]) for c in range(5))]
                assert torch.equal(out[rows], want[rows]), (i, b)


def test_nothing_to_do():
    q, cu, pool, bt = case("bf16", 128, 4, 2, [0, 0], [30, 40], seed=10, pad=4)
    out, st = run(q, cu, pool, bt, [30, 40], 0.1, out=torch.full_like(q, 5.0))
    assert st == 0 and (out == 5.0).all()
    empty = pa.pa_cross_attention(q[:0], cu.to(DEV), pool[0], pool[1], bt.to(DEV),
                                  torch.tensor([30, 40], dtype=torch.int32, device=DEV), 0.1)
    assert empty.shape == (0, 8, 128)


def test_eight_thousand_sequences():
    B = 8192
    gen = torch.Generator().manual_seed(11)
    ctx = torch.randint(0, 40, (B,), generator=gen).tolist()
    q_lens = torch.randint(0, 4, (B,), generator=gen).tolist()
    q, cu, pool, bt = case("bf16", 64, 2, 1, q_lens, ctx, seed=11)
    out, st = run(q, cu, pool, bt, ctx, 0.125)
    assert st == 0
    check(out, q, cu, pool, bt, ctx, 0.125, seqs=list(range(0, 60)) + list(range(B - 60, B)))


def test_two_graphs_and_two_streams_at_once():
    """Captured twice and replayed together, then called on two streams at once: every
    call has a workspace of its own."""
    ctx, q_lens = [5000, 900], [1, 30]
    scale = 0.1
    runs = []
    for i in range(2):
        q, cu, pool, bt = case("bf16", 128, 4, 2, q_lens, ctx, seed=20 + i)
        args = (q, cu.to(DEV), pool[0], pool[1], bt.to(DEV),
                torch.tensor(ctx, dtype=torch.int32, device=DEV), scale)
        want = pa.pa_cross_attention(*args)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = pa.pa_cross_attention(*args)
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
            got.append((pa.pa_cross_attention(*args, stream=s), want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)
    calls = [(pa.pa_cross_attention(*r[4], prepare=True), r[3]) for r in runs]
    for call, want in calls * 2:
        assert torch.equal(call(), want)


def test_over_what_an_eviction_kept():
    """Encoder states: their masses from decode steps, cut to the heaviest, then a prompt
    attends to what is left."""
    gen = torch.Generator().manual_seed(30)
    B, n_kv, g, d, n, budget = 3, 2, 4, 128, 500, 96
    bt, total, rest = make_tables(gen, [n] * B, spare=B * 6)
    pool = make_pool(gen, total, n_kv, d, "bf16")
    cl = torch.full((B,), n, dtype=torch.int32, device=DEV)
    btd = bt.to(DEV)
    mass = torch.zeros(B, n_kv, bt.shape[1] * 16, device=DEV)
    for _ in range(4):
        q = (2 * torch.randn(B, n_kv * g, d, generator=gen)).to(torch.bfloat16).to(DEV)
        pa.pa_decode_mass(q, pool[0], pool[1], btd, cl, 0.1, mass)
    keep, lens = pa.pa_evict_select(mass, cl, budget)
    new = rest[:B * 6].view(B, 6).to(DEV)
    pa.pa_evict_compact(pool[0], pool[1], btd, keep, lens, new)
    q_lens = [40, 1, 77]
    cu = torch.tensor([0] + q_lens).cumsum(0).to(torch.int32)
    q = torch.randn(int(cu[-1]), n_kv * g, d, generator=gen).to(torch.bfloat16).to(DEV)
    out = pa.pa_cross_attention(q, cu.to(DEV), pool[0], pool[1], new, lens, 0.1)
    kc, vc = pool[0].cpu(), pool[1].cpu()
    for b in range(B):
        for h in range(n_kv):
            j = keep[b, h].cpu().long()
            k = kc[bt[b].long()[j // 16], h, j % 16].double()
            v = vc[bt[b].long()[j // 16], h, j % 16].double()
            heads = slice(h * g, (h + 1) * g)
            x = q[cu[b]:cu[b + 1], heads].cpu().double().reshape(-1, d)
            o, w, e = attend(x, k, v, 0.1)
            got = out[cu[b]:cu[b + 1], heads].cpu().double().reshape(-1, d)
            tol = (2.0 ** -8 + 2.0 ** -18 + e) * (w @ v.abs()) + 2.0 ** -8 * o.abs() * 1.01
            assert ((got - o).abs() <= tol).all()

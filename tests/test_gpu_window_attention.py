"""pa_window_attention on the GPU against the plain form in 64 bits (tests/plain_window.py has
the tolerances): ragged tokens and contexts, windows and first tokens of every kind, pool
types and head layouts, forced splits, blocks given back, values that are not finite where a
token does not look, reports, streams and graphs, and a whole run of rotary append, prompt
and single tokens."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_94_gb300 as pa
from tests.plain_attention import gather_rows
from tests.plain_window import attend_seen, check_window, seen_keys, turned
from tests.test_gpu_evict import make_pool, poison
from tests.test_gpu_window_decode import MASKS, case, check_decode, decode, give_back

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
Q_LENS = [1, 0, 3, 17, 130, 2, 300, 64, 5, 9]
CTX = [5, 40, 0, 127, 131, 1, 457, 128, 1000, 6]  # some sequences have more tokens than context


def attend(q, cu, pool, bt, ctx, scale, window, n_first, **kw):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pa.pa_window_attention(q, cu.to(DEV), pool[0], pool[1], bt.to(DEV),
                                 torch.tensor(ctx, dtype=torch.int32, device=DEV), scale,
                                 window=window, n_first=n_first, k_scale=pool[2],
                                 v_scale=pool[3], dev_status=status, **kw)
    torch.cuda.synchronize()
    return out, int(status.item())


@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("d", [128, 64])
def test_one_token_one_tile(d, kv):
    q, cu, pool, bt = case(kv, d, 1, 1, [1], [16])
    out, st = attend(q, cu, pool, bt, [16], 1 / math.sqrt(d), 0, 0)
    assert st == 0
    check_window(out, q, cu, pool, bt, [16], 1 / math.sqrt(d), 0, 0)


@pytest.mark.parametrize("window,n_first", MASKS)
@pytest.mark.parametrize("g", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_ragged_tokens_over_ragged_contexts(kv, d, g, window, n_first):
    q, cu, pool, bt = case(kv, d, g, 2, Q_LENS, CTX, seed=g, lead=3, pad=9)
    poison(pool, bt, CTX)
    bt = give_back(bt, CTX, Q_LENS, window, n_first)
    scale = 1 / math.sqrt(d)
    for num_ctas in (0, 1, 7):
        out = torch.full_like(q, 5.0)
        _, st = attend(q, cu, pool, bt, CTX, scale, window, n_first, out=out, num_ctas=num_ctas)
        assert st == 0
        assert (out[:3] == 5.0).all() and (out[-9:] == 5.0).all()  # no sequence's rows
        check_window(out, q, cu, pool, bt, CTX, scale, window, n_first)


@pytest.mark.parametrize("window,n_first", [(0, 0), (700, 4), (1024, 129)])
@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("d,g,n_kv", [(128, 4, 2), (64, 1, 3)])
def test_prompts_over_long_contexts(d, g, n_kv, kv, window, n_first):
    q_lens, ctx = [1500, 65, 1, 2048], [3001, 2048, 4999, 2048]
    q, cu, pool, bt = case(kv, d, g, n_kv, q_lens, ctx, seed=3)
    scale = 1 / math.sqrt(d)
    bt = give_back(bt, ctx, q_lens, window, n_first)
    out, st = attend(q, cu, pool, bt, ctx, scale, window, n_first)
    again, _ = attend(q, cu, pool, bt, ctx, scale, window, n_first)
    assert st == 0 and torch.equal(out, again)
    check_window(out, q, cu, pool, bt, ctx, scale, window, n_first)


@pytest.mark.parametrize("num_ctas", [0, 2, 3, 40, 300])
@pytest.mark.parametrize("kv", ["bf16", "int4"])
def test_few_tokens_over_long_contexts_are_split_and_merged(kv, num_ctas):
    q_lens, ctx = [1, 2, 40], [20000, 7777, 9000]
    q, cu, pool, bt = case(kv, 128, 4, 1, q_lens, ctx, seed=4)
    for window, n_first in ((0, 0), (6000, 20)):
        for _ in range(3):  # the counters are left zero
            out, st = attend(q, cu, pool, bt, ctx, 0.1, window, n_first, num_ctas=num_ctas)
        assert st == 0
        check_window(out, q, cu, pool, bt, ctx, 0.1, window, n_first)


@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_many_short_segments_per_cta(kv):
    gen = torch.Generator().manual_seed(12)
    ctx = torch.randint(1, 700, (60,), generator=gen).tolist()
    q_lens = [min(n, int(torch.randint(1, 600, (1,), generator=gen))) for n in ctx]
    q, cu, pool, bt = case(kv, 128, 1, 4, q_lens, ctx, seed=12)
    for window, n_first in ((0, 0), (90, 2)):
        for num_ctas in (0, 5):
            out, st = attend(q, cu, pool, bt, ctx, 0.09, window, n_first, num_ctas=num_ctas)
            assert st == 0
            check_window(out, q, cu, pool, bt, ctx, 0.09, window, n_first)


@pytest.mark.parametrize("kind", ["rising", "falling", "big", "flat", "negative", "v_range"])
@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_value_ranges(kv, kind):
    """Scores that climb tile after tile, fall, are huge, all equal, or negated; V rows over
    six decades."""
    n, d, new = 1500, 128, 900
    q, cu, pool, bt = case(kv, d, 2, 1, [new], [n], seed=5)
    scale = 1 / math.sqrt(d)
    if kind in ("rising", "falling"):
        q = q.abs()
        steps = torch.linspace(0.05, 3.0, n)
        if kind == "falling":
            steps = steps.flip(0)
        for j in range(n):
            at = (bt[0, j // 16].long(), slice(None), j % 16)
            pool[0][at] = pool[0][at].abs() * (float(steps[j]) if kv == "bf16" else 1)
            if kv != "bf16":
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
    for window, n_first in ((0, 0), (400, 5)):
        for num_ctas in (0, 1):
            out, st = attend(q, cu, pool, bt, [n], scale, window, n_first, num_ctas=num_ctas)
            assert st == 0
            check_window(out, q, cu, pool, bt, [n], scale, window, n_first)


@pytest.mark.parametrize("new", [40, 500])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_what_a_token_does_not_see_may_be_anything(kv, d, new):
    """K and V that are not finite at some positions: rows that do not see them come out as if
    they were not there, rows that do are not finite (V: in its own columns)."""
    n, window, n_first, g = 800, 150, 9, 2
    q, cu, pool, bt = case(kv, d, g, 1, [new], [n], seed=14)
    kc, vc, ks, vs = pool
    slot = lambda j: (int(bt[0, j // 16]), 0, j % 16)  # noqa: E731
    inf, nan = float("inf"), float("nan")
    bad_v = {n - 3: inf, n - 130: nan, n - 131: -inf, n - 200: inf, 8: nan, 300: inf}
    bad_k = {n - 20: nan, n - 170: inf, n - 260: -inf}
    clean = [None if t is None else t.clone() for t in pool]
    for j, x in bad_v.items():
        if kv == "bf16":
            vc[slot(j)][j % d] = x
        else:
            vs[slot(j)] = x
    for j, x in bad_k.items():
        if kv == "bf16":
            kc[slot(j)][j % d] = x
        else:
            ks[slot(j)] = x
    seen = seen_keys(new, n, window, n_first)
    for num_ctas in (0, 1, 9):
        want, _ = attend(q, cu, clean, bt, [n], 0.1, window, n_first, num_ctas=num_ctas)
        out, st = attend(q, cu, pool, bt, [n], 0.1, window, n_first, num_ctas=num_ctas)
        assert st == 0
        check_window(want, q, cu, clean, bt, [n], 0.1, window, n_first)
        hit = torch.zeros(new, d, dtype=torch.bool)  # what may not be finite
        for j in bad_v:
            if kv == "bf16":
                hit[seen[:, j], j % d] = True
            else:
                hit |= seen[:, j][:, None]
        for j in bad_k:
            hit |= seen[:, j][:, None]
        hit = hit[:, None].expand(new, g, d)
        out, want = out.cpu(), want.cpu()
        assert torch.isfinite(out[~hit]).all()
        # (the softmax base may have been another key's: not bit for bit)
        tol = 2.0 ** -7 * want.abs() + 2.0 ** -12
        rows = ~hit.any(2)
        assert ((out - want).abs() <= tol)[rows].all()
        v_only = torch.zeros(new, dtype=torch.bool)
        for j in bad_v:
            v_only |= seen[:, j]
        for j in bad_k:
            v_only &= ~seen[:, j]
        if kv == "bf16":
            assert not torch.isfinite(out[v_only][hit[v_only]]).any()
            assert ((out - want).abs() <= tol)[v_only][~hit[v_only]].all()


def test_one_infinite_value():
    """One infinite V entry among finite ones: the rows that see it are not finite there, in
    tiles that some row does not see whole and in others, cut or not."""
    n, new, d = 600, 300, 128
    for j, sign in ((n - 5, 1), (n - 120, -1), (310, 1), (10, -1)):
        q, cu, pool, bt = case("bf16", d, 2, 1, [new], [n], seed=15)
        pool[1][int(bt[0, j // 16]), 0, j % 16, 7] = sign * float("inf")
        seen = seen_keys(new, n, 0, 0)[:, j]
        for num_ctas in (0, 1):
            out, _ = attend(q, cu, pool, bt, [n], 0.01, 0, 0, num_ctas=num_ctas)
            assert not torch.isfinite(out[seen][..., 7]).any()
            assert torch.isfinite(out[~seen]).all() and torch.isfinite(out[..., 8:]).all()


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_non_finite_queries_stay_their_own(kv):
    ctx = [700, 333]
    q, cu, pool, bt = case(kv, 128, 1, 1, [90, 250], ctx, seed=13)
    want = {c: attend(q, cu, pool, bt, ctx, 0.1, 100, 3, num_ctas=c)[0] for c in (0, 1)}
    odd = (3, 13, 49, 90 + 5, 90 + 140)
    q[list(odd)] = float("nan")
    for num_ctas in (0, 1):
        out, st = attend(q, cu, pool, bt, ctx, 0.1, 100, 3, num_ctas=num_ctas)
        assert st == 0 and torch.isnan(out[list(odd)]).all()
        rest = [i for i in range(340) if i not in odd]
        assert torch.equal(out[rest], want[num_ctas][rest])


@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_reports(kv):
    ctx = [100, 300, 64, 50, 20]
    q_lens = [3, 40, 2, 4, 5]
    window, n_first = 120, 20
    q, cu, pool, bt = case(kv, 128, 2, 2, q_lens, ctx, seed=9, extra=0)
    want, _ = attend(q, cu, pool, bt, ctx, 0.1, window, n_first)
    bt2 = bt.clone()
    bt2[1, 1], bt2[1, 12], bt2[1, 18] = -7, pool[0].shape[0], 1 << 30  # 16 .., 192 .., 288 ..
    ctx2 = [100, 300, bt.shape[1] * 16 + 1, -1, 20]
    out, st = attend(q, cu, pool, bt2, ctx2, 0.1, window, n_first, out=torch.full_like(q, 5.0))
    assert st == pa.PA_DEV_BAD_BLOCK | pa.PA_DEV_BAD_CONTEXT
    assert torch.equal(out[:3], want[:3]) and torch.equal(out[49:], want[49:])
    assert (out[43:49] == 0).all()
    # sequence 1 without the bad blocks' tokens
    kc, vc, ks, vs = [None if t is None else t.cpu() for t in pool]
    seen = seen_keys(40, 300, window, n_first)
    for i in (1, 12, 18):
        seen[:, 16 * i:16 * i + 16] = False
    for h in range(2):
        k, v = (gather_rows(p, s, bt[1], 300, h) for p, s in ((kc, ks), (vc, vs)))
        x = q[3:43, 2 * h:2 * h + 2].cpu().double().reshape(-1, 128)
        got = out[3:43, 2 * h:2 * h + 2].cpu().double().reshape(-1, 128)
        o, tol = attend_seen(x, k, v, 0.1, seen.repeat_interleave(2, 0))
        assert ((got - o).abs() <= tol + 2.0 ** -8 * (o.abs() + tol)).all()
    for i, bad in ((2, 2), (5, 1000), (0, -4)):  # offsets that decrease, or leave the tokens
        cu2 = cu.clone()
        cu2[i] = bad
        out, st = attend(q, cu2, pool, bt, ctx, 0.1, window, n_first, out=torch.full_like(q, 5.0))
        assert st == pa.PA_DEV_BAD_CONTEXT


def test_nothing_to_do():
    q, cu, pool, bt = case("bf16", 128, 4, 2, [0, 0], [30, 40], seed=10, pad=4)
    out, st = attend(q, cu, pool, bt, [30, 40], 0.1, 5, 1, out=torch.full_like(q, 5.0))
    assert st == 0 and (out == 5.0).all()
    assert attend(q[:0], cu, pool, bt, [30, 40], 0.1, 5, 1)[0].shape == (0, 8, 128)


def test_eight_thousand_sequences():
    B = 8192
    gen = torch.Generator().manual_seed(11)
    ctx = torch.randint(0, 60, (B,), generator=gen).tolist()
    q_lens = torch.randint(0, 4, (B,), generator=gen).tolist()
    q, cu, pool, bt = case("bf16", 64, 2, 1, q_lens, ctx, seed=11)
    out, st = attend(q, cu, pool, bt, ctx, 0.125, 20, 3)
    assert st == 0
    check_window(out, q, cu, pool, bt, ctx, 0.125, 20, 3,
                 seqs=list(range(0, 60)) + list(range(B - 60, B)))


@pytest.mark.parametrize("seed", range(24))
def test_random_cases(seed):
    gen = torch.Generator().manual_seed(1000 + seed)
    pick = lambda xs: xs[int(torch.randint(0, len(xs), (1,), generator=gen))]  # noqa: E731
    kv, d, g, n_kv = pick(["bf16", "int8", "int4"]), pick([64, 128]), pick([1, 2, 4, 8, 16]), pick([1, 3])
    B = pick([1, 3, 9])
    top = pick([40, 300, 2500])
    ctx = torch.randint(0, top, (B,), generator=gen).tolist()
    q_lens = [int(torch.randint(0, n + 3, (1,), generator=gen)) for n in ctx]
    window = pick([0, int(torch.randint(1, top + 1, (1,), generator=gen))])
    n_first = pick([0, 1, 16, 31, 77, 300])
    q, cu, pool, bt = case(kv, d, g, n_kv, q_lens, ctx, seed=seed, pad=1)
    poison(pool, bt, ctx)
    back = give_back(bt, ctx, q_lens, window, n_first)
    scale = 1 / math.sqrt(d)
    for num_ctas in (0, pick([1, 2, 5, 33, 500])):
        out, st = attend(q, cu, pool, back, ctx, scale, window, n_first, num_ctas=num_ctas)
        assert st == 0
        check_window(out, q, cu, pool, back, ctx, scale, window, n_first)
    one = (2 * torch.randn(B, n_kv * g, d, generator=gen)).to(torch.bfloat16).to(DEV)
    back = give_back(bt, ctx, [1] * B, window, n_first)
    for num_ctas in (0, pick([1, 2, 5, 33, 500])):
        out, st = decode(one, pool, back, ctx, scale, window, n_first, num_ctas=num_ctas)
        assert st == 0
        check_decode(out, one, pool, back, ctx, scale, window, n_first)


def test_one_token_of_each_sequence_both_ways():
    ctx = [700, 33, 4100, 128]
    for kv in ("bf16", "int8", "int4"):
        q, cu, pool, bt = case(kv, 128, 4, 2, [1] * 4, ctx, seed=24)
        for window, n_first in ((0, 0), (64, 4), (333, 100)):
            a, _ = attend(q, cu, pool, bt, ctx, 0.09, window, n_first)
            b, _ = decode(q, pool, bt, ctx, 0.09, window, n_first)
            check_window(a, q, cu, pool, bt, ctx, 0.09, window, n_first)
            check_decode(b, q, pool, bt, ctx, 0.09, window, n_first)


def test_two_graphs_and_two_streams_at_once():
    """Captured twice and replayed together, then called on two streams at once: every call
    has a workspace of its own."""
    ctx, runs = [5000, 900], []
    for i in range(2):
        q, cu, pool, bt = case("bf16", 128, 4, 2, [1, 30], ctx, seed=30 + i)
        args = (q, cu.to(DEV), pool[0], pool[1], bt.to(DEV),
                torch.tensor(ctx, dtype=torch.int32, device=DEV), 0.1, 3000, 4)
        want = pa.pa_window_attention(*args)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = pa.pa_window_attention(*args)
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
            got.append((pa.pa_window_attention(*args, stream=s), want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)
    calls = [(pa.pa_window_attention(*r[4], prepare=True), r[3]) for r in runs]
    for call, want in calls * 2:
        assert torch.equal(call(), want)


@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_a_run_of_prompt_chunks_and_single_tokens(kv):
    """What a serving loop does: blocks from the allocator, rotary append of a prompt chunk by
    chunk, attention of each chunk, then single tokens; blocks that leave the window go back
    to the allocator and are written by others. Every output against the plain form of the
    whole history."""
    gen = torch.Generator().manual_seed(40)
    n_kv, g, d, window, n_first, pairs = 2, 4, 128, 100, 20, 64
    scale = 1 / math.sqrt(d)
    lens = [230, 77, 161]
    B, steps, cap = len(lens), 40, 32
    alloc = pa.BlockAllocator(60)
    pool = make_pool(gen, 60, n_kv, d, kv)
    freq = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    table = torch.full((B, cap), -1, dtype=torch.int32)
    held = [0] * B
    k_all = [torch.zeros(n_kv, 0, d, dtype=torch.float64) for _ in range(B)]
    v_all = [torch.zeros(n_kv, 0, d, dtype=torch.float64) for _ in range(B)]
    done = [0] * B

    def step(new):
        """new[b] more tokens of every sequence, as one ragged batch."""
        for b in range(B):
            need = -(-(done[b] + new[b]) // 16) - held[b]
            if need > 0:
                fresh = torch.from_numpy(alloc.allocate_private(16 * need))
                table[b, held[b]:held[b] + need] = fresh
                held[b] += need
        T = sum(new)
        q, k, v = (torch.randn(T, h, d, generator=gen).to(torch.bfloat16) for h in (n_kv * g, n_kv, n_kv))
        pos = torch.cat([torch.arange(done[b], done[b] + new[b]) for b in range(B)])
        seq = torch.cat([torch.full((new[b],), b) for b in range(B)])
        slots = table[seq, pos // 16].long() * 16 + pos % 16
        pos3 = torch.stack([pos, pos // 7, pos % 7]).to(torch.int32)
        axis = torch.arange(pairs, dtype=torch.int32) % 3
        qr = pa.pa_rope_write(q.to(DEV), k.to(DEV), v.to(DEV), pos3.to(DEV), freq.to(DEV),
                              slots.to(DEV), pool[0], pool[1], axis=axis.to(DEV),
                              k_scale=pool[2], v_scale=pool[3])
        want, tol = turned(q.double(), pos3, freq, axis, False, 1.0)
        assert ((qr.cpu().double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()
        cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
        host = [None if t is None else t.cpu() for t in pool]
        for b in range(B):  # the rows as they were stored, kept here for good
            at = torch.arange(done[b], done[b] + new[b])
            for which, kept in ((0, k_all), (1, v_all)):
                rows = []
                for h in range(n_kv):
                    t = torch.where(table[b] >= 0, table[b], 0)
                    rows.append(gather_rows(host[which], host[2 + which], t, done[b] + new[b], h)[at])
                kept[b] = torch.cat([kept[b], torch.stack(rows)], dim=1)
            done[b] += new[b]
        ctx = torch.tensor(done, dtype=torch.int32, device=DEV)
        args = (pool[0], pool[1], table.to(DEV), ctx, scale, window, n_first)
        sc = dict(k_scale=pool[2], v_scale=pool[3])
        one = max(new) == 1
        out = (pa.pa_window_decode(qr, *args, **sc) if one else
               pa.pa_window_attention(qr, cu.to(DEV), *args, **sc))
        codes = one and kv != "bf16"
        check_window(out, qr, cu, pool, table, list(done), scale, window, n_first,
                     first_part=2.0 ** -11 if codes else 2.0 ** -16, codes_in_16=codes,
                     rows_of=lambda b, h: (k_all[b][h], v_all[b][h]))
        # what no later token sees goes back
        for b in range(B):
            for i in range(-(-n_first // 16), max(0, done[b] + 1 - window) // 16):
                if table[b, i] >= 0:
                    alloc.free(np.array([int(table[b, i])], np.int32))
                    table[b, i] = -1

    at = [0] * B
    while any(x < n for x, n in zip(at, lens)):
        new = [min(90, n - x) for x, n in zip(at, lens)]
        step(new)
        at = [x + y for x, y in zip(at, new)]
    for _ in range(steps):
        step([1] * B)

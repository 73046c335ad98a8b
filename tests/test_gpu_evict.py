"""pa_decode_mass, pa_evict_select and pa_evict_compact on the GPU against their
plain forms in 64 bits, apart and as one eviction step after another."""
import math
import threading

import numpy as np
import pytest
import torch

import paged_kv_cache_94_gb300 as pa
from tests.gpu_helpers import assert_close
from tests.plain_attention import attend, cached_rows, choose

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make_pool(gen, num_blocks, n_kv, d, kv):
    """Random pool on the device: (k, v, k_scale, v_scale)."""
    if kv == "bf16":
        return [torch.randn(num_blocks, n_kv, 16, d, generator=gen).to(torch.bfloat16).to(DEV)
                for _ in range(2)] + [None, None]
    if kv == "int8":
        c = [torch.randint(-127, 128, (num_blocks, n_kv, 16, d), generator=gen,
                           dtype=torch.int8).to(DEV) for _ in range(2)]
        step = 1 / 50
    else:
        c = [torch.randint(0, 256, (num_blocks, n_kv, 16, d // 2), generator=gen,
                           dtype=torch.uint8).to(DEV) for _ in range(2)]
        step = 1 / 3
    s = [((0.5 + torch.rand(num_blocks, n_kv, 16, generator=gen)) * step).to(DEV)
         for _ in range(2)]
    return c + s


def make_tables(gen, ctx, spare=0, extra=0):
    """Block tables [B, max_blocks + extra] of scattered blocks (-1 behind), pool size."""
    nblk = [-(-max(n, 0) // 16) for n in ctx]
    total = sum(nblk) + 1 + spare
    order = torch.randperm(total, generator=gen).to(torch.int32)
    bt = torch.full((len(ctx), max(max(nblk), 1) + extra), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(nblk):
        bt[b, :n] = order[at:at + n]
        at += n
    return bt, total, order[at:]


def poison(pool, bt, ctx):
    """NaN (or NaN scales) in every slot no sequence holds."""
    kc, vc, ks, vs = pool
    used = torch.zeros(kc.shape[0], 16, dtype=torch.bool)
    for b, n in enumerate(ctx):
        for j in range(n):
            used[bt[b, j // 16], j % 16] = True
    free = ~used[:, None, :].expand(kc.shape[:3]).to(DEV)
    for t in ((ks, vs) if ks is not None else (kc, vc)):
        t[free] = float("nan")


def plain_step(q, pool, bt, ctx, scale):
    """(out, weights per (b, kv head) summed over its heads, allowed relative error)."""
    kc, vc, ks, vs = [None if t is None else t.cpu() for t in pool]
    n_kv = kc.shape[1]
    B, n_h, d = q.shape
    g = n_h // n_kv
    out, w = torch.zeros(B, n_h, d, dtype=torch.float64), {}
    for b, n in enumerate(ctx):
        for h in range(n_kv):
            k, v = cached_rows(kc, ks, bt[b], n, h), cached_rows(vc, vs, bt[b], n, h)
            o, wt, e = attend(q[b, h * g:(h + 1) * g].cpu().double(), k, v, scale)
            out[b, h * g:(h + 1) * g] = o
            w[b, h] = (wt.sum(0), e)
    return out, w


CTX = [0, 1, 15, 16, 17, 33, 100, 257]


@pytest.mark.parametrize("num_ctas", [0, 1, 7, 300])
@pytest.mark.parametrize("g", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_mass_matches_the_plain_form(kv, d, g, num_ctas):
    gen = torch.Generator().manual_seed(17 * g + d)
    n_kv, scale = 2, 1 / math.sqrt(d)
    bt, total, _ = make_tables(gen, CTX, extra=1)
    pool = make_pool(gen, total, n_kv, d, kv)
    poison(pool, bt, CTX)
    q = (2 * torch.randn(len(CTX), n_kv * g, d, generator=gen)).to(torch.bfloat16).to(DEV)
    cap = bt.shape[1] * 16
    mass = torch.rand(len(CTX), n_kv, cap, generator=gen).to(DEV)
    for b, n in enumerate(CTX):
        mass[b, :, n:] = float("nan")
    args = (q, pool[0], pool[1], bt.to(DEV), torch.tensor(CTX, dtype=torch.int32, device=DEV),
            scale)
    kw = dict(k_scale=pool[2], v_scale=pool[3], num_ctas=num_ctas)
    before = mass.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    other = torch.full_like(mass, 7.0)
    out = pa.pa_decode_mass(*args, mass, mass_out=other, dev_status=status, **kw)
    plain_out = pa.pa_decode(*args, **kw)
    out2 = pa.pa_decode_mass(*args, mass, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(out, plain_out) and torch.equal(out2, plain_out)
    ref, w = plain_step(q, pool, bt, CTX, scale)
    assert_close(out.float().cpu().numpy(), ref.numpy())
    for b, n in enumerate(CTX):
        assert (other[b, :, n:] == 7.0).all() and torch.isnan(mass[b, :, n:]).all()
        for h in range(n_kv):
            wt, e = w[b, h]
            want = before[b, h, :n].cpu().double() + wt
            tol = wt * e + 2.0 ** -23 * want + 1e-37
            assert ((mass[b, h, :n].cpu().double() - want).abs() <= tol).all(), (b, h)
            assert torch.equal(mass[b, h, :n], other[b, h, :n])


@pytest.mark.parametrize("g", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_output_is_the_decode_s_bit_for_bit_over_long_contexts(kv, d, g):
    """Both calls on their default grids, with more key blocks than either has warps: every
    unit is cut, at the same places in both only if the grids are equal."""
    gen = torch.Generator().manual_seed(40 + g)
    ctx, n_kv = [30000, 4097, 9001], 2
    bt, total, _ = make_tables(gen, ctx)
    pool = make_pool(gen, total, n_kv, d, kv)
    q = torch.randn(len(ctx), n_kv * g, d, generator=gen).to(torch.bfloat16).to(DEV)
    args = (q, pool[0], pool[1], bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV),
            0.1)
    mass = torch.zeros(len(ctx), n_kv, bt.shape[1] * 16, device=DEV)
    kw = dict(k_scale=pool[2], v_scale=pool[3])
    out = pa.pa_decode_mass(*args, mass, **kw)
    assert torch.equal(out, pa.pa_decode(*args, **kw))


@pytest.mark.parametrize("num_ctas", [1, 40])
@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_mass_of_a_row_with_a_score_that_is_not_a_number(kv, num_ctas):
    """One NaN among a kv head's scores makes all the weights of its rows NaN; the other kv
    head's masses are untouched by it. Whole units (one CTA) and cut ones."""
    gen = torch.Generator().manual_seed(12)
    ctx, n_kv, g, d = [300, 1, 77], 2, 4, 128
    bt, total, _ = make_tables(gen, ctx)
    pool = make_pool(gen, total, n_kv, d, kv)
    q = torch.randn(3, n_kv * g, d, generator=gen).to(torch.bfloat16).to(DEV)
    cl = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    kw = dict(k_scale=pool[2], v_scale=pool[3], num_ctas=num_ctas)
    clean = torch.zeros(3, n_kv, bt.shape[1] * 16, device=DEV)
    pa.pa_decode_mass(q, pool[0], pool[1], bt.to(DEV), cl, 0.1, clean, **kw)
    keys = pool[0] if kv == "bf16" else pool[2]      # a K row, or its scale
    for b, j in ((0, 140), (1, 0)):
        keys[int(bt[b, j // 16]), 1, j % 16] = float("nan")
    mass = torch.zeros_like(clean)
    pa.pa_decode_mass(q, pool[0], pool[1], bt.to(DEV), cl, 0.1, mass, **kw)
    assert torch.isnan(mass[0, 1, :300]).all() and torch.isnan(mass[1, 1, :1]).all()
    assert torch.equal(mass[:, 0], clean[:, 0]) and torch.equal(mass[2], clean[2])
    assert (mass[0, 1, 300:] == 0).all() and (mass[1, 1, 1:] == 0).all()


def test_two_threads_on_one_stream():
    """Calls of different batch sizes share the stream's workspace, one after another."""
    gen = torch.Generator().manual_seed(30)
    n_kv, g, d = 8, 4, 128

    def setting(B):
        ctx = [1 + (37 * b) % 90 for b in range(B)]
        bt, total, _ = make_tables(gen, ctx)
        pool = make_pool(gen, total, n_kv, d, "bf16")
        q = torch.randn(B, n_kv * g, d, generator=gen).to(torch.bfloat16).to(DEV)
        args = (q, pool[0], pool[1], bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV))
        mass = torch.zeros(B, n_kv, bt.shape[1] * 16, device=DEV)
        want = torch.empty_like(mass)
        out = pa.pa_decode_mass(*args, 0.1, mass, mass_out=want, num_ctas=64)
        return args, mass, want, out

    cases = [setting(200), setting(3)]
    torch.cuda.synchronize()
    wrong = []

    def run(args, mass, want, out):
        got = torch.empty_like(mass)
        for _ in range(100):
            o = pa.pa_decode_mass(*args, 0.1, mass, mass_out=got, num_ctas=64)
        torch.cuda.synchronize()
        for b, n in enumerate(args[4].tolist()):
            if not torch.equal(got[b, :, :n], want[b, :, :n]):
                wrong.append(b)
        if not torch.equal(o, out):
            wrong.append("out")

    threads = [threading.Thread(target=run, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_a_stream_s_larger_workspace_replaces_the_smaller_one():
    """A wider table needs a larger workspace: both are never held at once."""
    gen = torch.Generator().manual_seed(50)
    ctx, n_kv, g, d = [100] * 8, 4, 4, 64
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        args = []
        for extra in (1000, 2000):
            bt, total, _ = make_tables(gen, ctx, extra=extra)
            pool = make_pool(gen, total, n_kv, d, "bf16")
            q = torch.randn(8, n_kv * g, d, generator=gen).to(torch.bfloat16).to(DEV)
            args.append((q, pool[0], pool[1], bt.to(DEV),
                         torch.tensor(ctx, dtype=torch.int32, device=DEV), 0.1,
                         torch.zeros(8, n_kv, bt.shape[1] * 16, device=DEV)))
        out = [torch.empty_like(a[0]) for a in args]
        pa.pa_decode_mass(*args[0], out=out[0])
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        pa.pa_decode_mass(*args[1], out=out[1])
        torch.cuda.synchronize()
        larger = 4 * 8 * n_kv * g * (2000 + 7) * 16
        assert torch.cuda.max_memory_allocated() - before < larger
        assert torch.cuda.memory_allocated() - before > larger // 4


def test_numbers_beyond_32_bits_are_refused():
    """Cut to their low bits they would be another budget, or another CTA count."""
    mass = torch.rand(1, 1, 64, device=DEV)
    cl = torch.tensor([64], dtype=torch.int32, device=DEV)
    for kw in (dict(budget=(1 << 32) + 5), dict(budget=5, recent=1 << 32)):
        with pytest.raises(ValueError, match="32 bits"):
            pa.pa_evict_select(mass, cl, **kw)
    gen = torch.Generator().manual_seed(60)
    bt, total, _ = make_tables(gen, [64])
    pool = make_pool(gen, total, 1, 64, "bf16")
    q = torch.randn(1, 1, 64, generator=gen).to(torch.bfloat16).to(DEV)
    with pytest.raises(ValueError, match="32 bits"):
        pa.pa_decode_mass(q, pool[0], pool[1], bt.to(DEV), cl, 0.1, mass,
                          num_ctas=(1 << 32) + 1)
    cu = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="32 bits"):
        pa.pa_cross_attention(q, cu, pool[0], pool[1], bt.to(DEV), cl, 0.1,
                              num_ctas=(1 << 32) + 1)


def test_mass_of_shared_blocks_bad_blocks_and_bad_lengths():
    gen = torch.Generator().manual_seed(3)
    ctx = [40, 40, 100, 64, 30]
    bt, total, _ = make_tables(gen, ctx)
    bt[1] = bt[0]                                   # two sequences on the same blocks
    pool = make_pool(gen, total, 2, 128, "bf16")
    q = torch.randn(5, 8, 128, generator=gen).to(torch.bfloat16).to(DEV)
    good = plain_step(q, pool, bt, [40, 40, 100, 0, 30], 0.1)[1]
    bad = bt.clone()
    bad[2, 3] = total + 5                           # tokens 48 .. 63 of sequence 2
    bad_ctx = torch.tensor([40, 40, 100, bt.shape[1] * 16 + 1, 30], dtype=torch.int32, device=DEV)
    for num_ctas in (0, 3):
        mass = torch.zeros(5, 2, bt.shape[1] * 16, device=DEV)
        mass[3] = 5.0
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = pa.pa_decode_mass(q, pool[0], pool[1], bad.to(DEV), bad_ctx, 0.1, mass,
                                dev_status=status, num_ctas=num_ctas)
        torch.cuda.synchronize()
        assert int(status.item()) == pa.PA_DEV_BAD_BLOCK | pa.PA_DEV_BAD_CONTEXT
        assert (mass[3] == 5.0).all() and (out[3] == 0).all()
        assert torch.equal(mass[0, :, :40] > 0, mass[1, :, :40] > 0)
        assert (mass[2, :, 48:64] == 0).all()
        # what the bad block leaves sums to one weight per query head
        assert torch.allclose(mass[2].sum(1), torch.full((2,), 4.0, device=DEV), rtol=1e-4)
        for b in (0, 1, 4):
            for h in range(2):
                wt, e = good[b, h]
                assert ((mass[b, h, :ctx[b]].cpu().double() - wt).abs() <=
                        wt * (e + 2.0 ** -22)).all()


def test_mass_captured_twice_and_replayed_at_once():
    """Two graphs on two streams, each with its own scratch, add in place at every replay."""
    gen = torch.Generator().manual_seed(4)
    ctx = [700, 1300, 90]
    bt, total, _ = make_tables(gen, ctx)
    pool = make_pool(gen, total, 2, 128, "bf16")
    cl = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    btd = bt.to(DEV)
    runs = []
    for i in range(2):
        q = torch.randn(3, 8, 128, generator=gen).to(torch.bfloat16).to(DEV)
        one = torch.zeros(3, 2, bt.shape[1] * 16, device=DEV)
        want = pa.pa_decode_mass(q, pool[0], pool[1], btd, cl, 0.1, one).clone()
        mass = torch.zeros_like(one)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = pa.pa_decode_mass(q, pool[0], pool[1], btd, cl, 0.1, mass)
        runs.append((graph, s, out, want, mass, one, q))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, s, *_ in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for graph, s, out, want, mass, one, q in runs:
        assert torch.equal(out, want)
        # 20 sums in fp32, each rounded once
        assert ((mass.double() - 20 * one.double()).abs() <= 20 * 2.0 ** -24 * 20 * one).all()


def test_mass_prepared_and_on_another_stream():
    gen = torch.Generator().manual_seed(5)
    ctx = [300, 20]
    bt, total, _ = make_tables(gen, ctx)
    pool = make_pool(gen, total, 2, 64, "int8")
    q = torch.randn(2, 4, 64, generator=gen).to(torch.bfloat16).to(DEV)
    args = (q, pool[0], pool[1], bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV), 0.1)
    kw = dict(k_scale=pool[2], v_scale=pool[3])
    a, b = (torch.zeros(2, 2, bt.shape[1] * 16, device=DEV) for _ in range(2))
    want = pa.pa_decode_mass(*args, a, **kw)
    call = pa.pa_decode_mass(*args, b, prepare=True, **kw)
    # a smaller and a larger batch between the preparation and the call
    pa.pa_decode_mass(q[:1], pool[0], pool[1], args[3][:1], args[4][:1], 0.1, a[:1].clone(), **kw)
    big = 40
    pa.pa_decode_mass(q.repeat(big, 1, 1), pool[0], pool[1], args[3].repeat(big, 1),
                      args[4].repeat(big), 0.1, a.repeat(big, 1, 1), **kw)
    assert torch.equal(call(), want) and torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = torch.zeros_like(a)
    s.wait_stream(torch.cuda.current_stream())
    got = pa.pa_decode_mass(*args, c, stream=s, **kw)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(a, c)


# ------------------------------------------------------------------------------------------ select
def check_select(mass, ctx, budget, recent):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    keep, lens = pa.pa_evict_select(mass.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV),
                                    budget, recent, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    m = mass.numpy()
    for b, n in enumerate(ctx):
        assert int(lens[b]) == min(n, budget)
        for h in range(mass.shape[1]):
            want = choose(m[b, h], n, budget, recent)
            want += [-1] * (budget - len(want))
            assert keep[b, h].tolist() == want, (b, h, n, budget, recent)


@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (7, 3), (64, 64), (64, 0), (100, 17),
                                           (5000, 100)])
@pytest.mark.parametrize("tokens", [1, 31, 515, 4097])
def test_select_matches_the_plain_choice(tokens, budget, recent):
    gen = torch.Generator().manual_seed(tokens + budget)
    ctx = sorted({0, 1, min(33, tokens), tokens // 2, tokens - 1, tokens})
    mass = torch.exp(2 * torch.randn(len(ctx), 3, tokens, generator=gen))
    for b, n in enumerate(ctx):
        mass[b, :, n:] = float("nan")
    check_select(mass, ctx, budget, recent)


def test_select_with_a_budget_near_2_31():
    """The unused tail of one row is 8.6 GB long; its indices stay below 2^31."""
    n, budget = 5000, 2 ** 31 - 1
    keep, lens = pa.pa_evict_select(torch.rand(1, 1, n, device=DEV),
                                    torch.tensor([n], dtype=torch.int32, device=DEV), budget, 3)
    assert lens.tolist() == [n]
    assert torch.equal(keep[0, 0, :n], torch.arange(n, dtype=torch.int32, device=DEV))
    for part in keep[0, 0, n:].split(1 << 28):
        assert int(part.min()) == int(part.max()) == -1


@pytest.mark.parametrize("tokens,budget", [(20000, 900), (60001, 30000), (140003, 16384),
                                           (200003, 70000)])
def test_select_of_long_rows(tokens, budget):
    """Rows over a cluster of CTAs, the longest too long to be kept between the sweeps."""
    gen = torch.Generator().manual_seed(tokens)
    check_select(torch.exp(torch.randn(2, 1, tokens, generator=gen)), [tokens, tokens - 777],
                 budget, 100)


def test_select_of_many_long_rows():
    """More rows than SMs and too long to be kept: one CTA a row, read again."""
    gen = torch.Generator().manual_seed(9)
    check_select(torch.rand(80, 4, 24600, generator=gen), [24600 - b for b in range(80)], 50, 5)


@pytest.mark.parametrize("case", ["equal", "zeros", "steps", "signs", "special"])
@pytest.mark.parametrize("tokens", [700, 9000])
def test_select_ties_and_special_values(case, tokens):
    gen = torch.Generator().manual_seed(1)
    shape = (2, 2, tokens)
    if case == "equal":
        mass = torch.full(shape, 0.37)
    elif case == "zeros":
        mass = torch.where(torch.rand(shape, generator=gen) < 0.9, 0.0, -0.0)
        mass[:, :, 5::97] = 1e-30
    elif case == "steps":
        mass = torch.randint(0, 4, shape, generator=gen).float()
    elif case == "signs":
        mass = torch.randn(shape, generator=gen)
    else:
        mass = torch.randn(shape, generator=gen)
        mass[:, :, ::7] = float("nan")
        mass[:, :, 3::11] = float("inf")
        mass[:, :, 4::13] = float("-inf")
        mass[:, :, 5::17] = 1e-42  # subnormal
    for budget, recent in ((1, 0), (99, 10), (tokens - 3, 2), (tokens, 0)):
        check_select(mass, [tokens, tokens - 5], budget, recent)


def test_select_reports_bad_lengths():
    mass = torch.rand(3, 2, 50, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ctx = torch.tensor([-1, 51, 20], dtype=torch.int32, device=DEV)
    keep, lens = pa.pa_evict_select(mass, ctx, 8, 2, dev_status=status)
    assert int(status.item()) == pa.PA_DEV_BAD_CONTEXT
    assert lens.tolist() == [0, 0, 8] and (keep[:2] == -1).all() and (keep[2] >= 0).all()


# ----------------------------------------------------------------------------------------- compact
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("with_mass", [False, True])
def test_compact_moves_rows_and_nothing_else(kv, d, with_mass):
    gen = torch.Generator().manual_seed(d)
    ctx, n_kv, budget = [0, 1, 16, 47, 700, 1111], 3, 600
    bt, total, rest = make_tables(gen, ctx, spare=6 * 38 + 4)
    bt[4, :2] = bt[5, :2]                            # shared old blocks
    new = rest[:6 * 38].view(6, 38).clone()
    pool = make_pool(gen, total, n_kv, d, kv)
    before = [None if t is None else t.clone() for t in pool]
    lens = [min(n, budget) - (n == 47) for n in ctx]
    keep = torch.full((6, n_kv, budget), -1, dtype=torch.int32)
    for b, n in enumerate(ctx):
        for h in range(n_kv):
            keep[b, h, :lens[b]] = torch.randperm(n, generator=gen)[:lens[b]].sort().values
    mass = torch.rand(6, n_kv, bt.shape[1] * 16, generator=gen).to(DEV)
    mass_out = torch.full((6, n_kv, 38 * 16), 9.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_evict_compact(pool[0], pool[1], bt.to(DEV), keep.to(DEV),
                        torch.tensor(lens, dtype=torch.int32, device=DEV), new.to(DEV),
                        mass=mass if with_mass else None, mass_out=mass_out if with_mass else None,
                        k_scale=pool[2], v_scale=pool[3], dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for b in range(6):
        for h in range(n_kv):
            i = torch.arange(lens[b])
            j = keep[b, h, :lens[b]].long()
            src, dst = bt[b].long()[j // 16], new[b].long()[i // 16]
            for t in before:
                if t is not None:
                    t[dst, h, i % 16] = t[src, h, j % 16]
            if with_mass:
                assert torch.equal(mass_out[b, h, :lens[b]], mass[b, h, j])
                assert (mass_out[b, h, lens[b]:] == 0).all()
    for t, want in zip(pool, before):
        assert t is None or torch.equal(t, want)


def test_compact_reports_what_it_cannot_move():
    gen = torch.Generator().manual_seed(8)
    ctx = [64, 64, 64, 64]
    bt, total, rest = make_tables(gen, ctx, spare=12)
    new = rest[:8].view(4, 2).clone()
    pool = make_pool(gen, total, 1, 128, "bf16")
    before = [t.clone() for t in pool[:2]]
    keep = torch.arange(0, 40, 2, dtype=torch.int32).repeat(4, 1, 1)  # 20 rows, a table of 32
    keep[0, 0, 3], keep[0, 0, 4] = 64, -5            # outside the old table
    bt2, new2 = bt.clone(), new.clone()
    bt2[1, 0] = total                                # old rows 0 .. 15
    new2[2, 1] = -1                                  # new rows 16 .. 31
    lens = torch.tensor([20, 20, 20, 21], dtype=torch.int32, device=DEV)  # 21 > budget
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mass = torch.rand(4, 1, 64, device=DEV)
    mass_out = torch.full((4, 1, 32), 9.0, device=DEV)
    pa.pa_evict_compact(pool[0], pool[1], bt2.to(DEV), keep.to(DEV), lens, new2.to(DEV), mass=mass,
                        mass_out=mass_out, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == pa.PA_DEV_BAD_BLOCK | pa.PA_DEV_BAD_CONTEXT
    for b in range(3):
        for i in range(20):
            j = int(keep[b, 0, i])
            if (b == 0 and i in (3, 4)) or (b == 1 and j < 16) or (b == 2 and i >= 16):
                assert mass_out[b, 0, i] == 0
                continue
            assert mass_out[b, 0, i] == mass[b, 0, j]
            for t in before:
                t[new[b, i // 16].long(), 0, i % 16] = t[bt[b, j // 16].long(), 0, j % 16]
    assert (mass_out[3] == 0).all() and (mass_out[:, 0, 20:] == 0).all()
    for t, want in zip(pool, before):
        assert torch.equal(t, want)


# ------------------------------------------------------------------------------- the steps together
@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_serving_loop_with_eviction(kv):
    """Sequences grow token by token; every 24 tokens each is cut to its budget. A
    plain simulation keeps each kv head's own list of rows."""
    gen = torch.Generator().manual_seed(21)
    B, n_kv, g, d, budget, recent, mb = 3, 2, 4, 64, 40, 12, 6
    alloc = pa.BlockAllocator(48)
    kc, vc, ks, vs = pa.allocate_pool(48, n_kv, d, kv, DEV)
    tables = np.full((B, mb), -1, np.int32)
    nblk = np.zeros(B, np.int32)
    ctx = np.zeros(B, np.int64)
    mass = torch.zeros(B, n_kv, mb * 16, device=DEV)
    # the simulation's rows: where each kept row sits is checked through the pool's values
    tokens = [[[] for _ in range(n_kv)] for _ in range(B)]
    sim_mass = [[np.zeros(0) for _ in range(n_kv)] for _ in range(B)]
    slack = [[np.zeros(0) for _ in range(n_kv)] for _ in range(B)]
    rows_k, rows_v = {}, {}
    for step in range(80):
        k = torch.randn(B, n_kv, d, generator=gen).to(torch.bfloat16).to(DEV)
        v = torch.randn(B, n_kv, d, generator=gen).to(torch.bfloat16).to(DEV)
        q = (2 * torch.randn(B, n_kv * g, d, generator=gen)).to(torch.bfloat16).to(DEV)
        slots, cow = alloc.append_slots(tables, nblk, [step] * B)
        assert len(cow) == 0
        pa.pa_cache_write(k, v, torch.from_numpy(slots).to(DEV), kc, vc, ks, vs)
        ctx += 1
        bt = torch.from_numpy(tables).to(DEV)
        cl = torch.from_numpy(ctx.astype(np.int32)).to(DEV)
        out = pa.pa_decode_mass(q, kc, vc, bt, cl, 0.125, mass, k_scale=ks, v_scale=vs)
        pools = [None if t is None else t.cpu() for t in (kc, vc, ks, vs)]
        for b in range(B):
            for h in range(n_kv):
                n = int(ctx[b])
                at = torch.from_numpy(tables[b])
                rk = cached_rows(pools[0], pools[2], at, n, h)
                rv = cached_rows(pools[1], pools[3], at, n, h)
                tokens[b][h].append(step)
                rows_k[b, h, step], rows_v[b, h, step] = rk[-1], rv[-1]
                # the cache holds exactly the simulation's rows, in order
                assert torch.equal(rk, torch.stack([rows_k[b, h, t] for t in tokens[b][h]]))
                assert torch.equal(rv, torch.stack([rows_v[b, h, t] for t in tokens[b][h]]))
                o, w, e = attend(q[b, h * g:(h + 1) * g].cpu().double(), rk, rv, 0.125)
                assert_close(out[b, h * g:(h + 1) * g].float().cpu().numpy(), o.numpy())
                w = w.sum(0).numpy()
                sim_mass[b][h] = np.append(sim_mass[b][h], 0.0) + w
                slack[b][h] = np.append(slack[b][h], 0.0) + w * e + 2.0 ** -23 * sim_mass[b][h]
                got = mass[b, h, :n].double().cpu().numpy()
                assert (np.abs(got - sim_mass[b][h]) <= slack[b][h] + 1e-37).all()
                assert (mass[b, h, n:] == 0).all()
        if step % 24 == 23:
            keep, lens = pa.pa_evict_select(mass, cl, budget, recent)
            new = np.full((B, mb), -1, np.int32)
            for b in range(B):
                fresh = alloc.allocate_private(min(int(ctx[b]), budget))
                new[b, :len(fresh)] = fresh
            moved = torch.empty_like(mass)
            pa.pa_evict_compact(kc, vc, bt, keep, lens, torch.from_numpy(new).to(DEV), mass=mass,
                                mass_out=moved, k_scale=ks, v_scale=vs)
            m = mass.cpu().numpy()
            for b in range(B):
                alloc.free(tables[b, :nblk[b]])
                for h in range(n_kv):
                    chosen = choose(m[b, h], int(ctx[b]), budget, recent)
                    assert keep[b, h, :len(chosen)].tolist() == chosen
                    tokens[b][h] = [tokens[b][h][j] for j in chosen]
                    sim_mass[b][h], slack[b][h] = sim_mass[b][h][chosen], slack[b][h][chosen]
            mass, tables = moved, new
            ctx = np.minimum(ctx, budget)
            nblk = ((ctx + 15) // 16).astype(np.int32)
            assert lens.tolist() == ctx.tolist()

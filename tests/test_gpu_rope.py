"""pa_rope_write on the GPU against the plain form in 64 bits (tests/plain_window.py has the
tolerances): pool types, head layouts, pair layouts, axes, far and negative positions,
strides, slots, reports, streams."""
import pytest
import torch

import paged_kv_cache_94_gb300 as pa
from tests.plain_window import turned
from tests.test_gpu_evict import make_pool

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def inputs(T, n_h, n_kv, d, axes, pairs, seed, lo=0, hi=5000, fused=True):
    gen = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, (n_h + 2 * n_kv) * d, generator=gen).to(torch.bfloat16).to(DEV)
    q = qkv[:, :n_h * d].view(T, n_h, d)
    k = qkv[:, n_h * d:(n_h + n_kv) * d].view(T, n_kv, d)
    v = qkv[:, (n_h + n_kv) * d:].view(T, n_kv, d)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(lo, hi, (axes, T), generator=gen, dtype=torch.int64).to(torch.int32)
    freq = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    axis = torch.randint(0, axes, (pairs,), generator=gen, dtype=torch.int32)
    return gen, q, k, v, pos, freq, axis


def near(got, want, tol, rounding=2.0 ** -8):
    """got was rounded once, by `rounding` relative; want is right within tol before that."""
    got, want, tol = got.cpu().double(), want.cpu(), tol.cpu()
    bad = ~((got - want).abs() <= tol + rounding * (want.abs() + tol) + 1e-30)
    assert not bad.any(), (int(bad.sum()), float((got - want).abs().max()), bad.nonzero()[:4].tolist())


def slots_of(gen, T, num_blocks):
    return torch.randperm(num_blocks * 16, generator=gen)[:T]


def stored_near(pool, which, slots, want, tol, kv):
    """The pool's rows at `slots` are what the quantiser makes of `want`, within tol."""
    codes, scale = pool[which], pool[2 + which]
    blk, off = (slots // 16).to(DEV), (slots % 16).to(DEV)
    rows = codes[blk, :, off].cpu()
    if kv == "bf16":
        return near(rows, want, tol)
    top = 127 if kv == "int8" else 7
    if kv == "int4":
        rows = torch.stack([rows & 15, rows >> 4], -1).flatten(-2).to(torch.int16)
        rows = torch.where(rows > 7, rows - 16, rows)
    step = scale[blk, :, off].cpu().double()
    worst = want.abs().amax(-1)
    assert ((step - worst / top).abs() <= (tol.amax(-1) + 2.0 ** -23 * worst) / top + 1e-30).all()
    # |x / step - code| <= 1/2, but for x's error and the division's rounding
    x = want / step.clamp(min=1e-300)[..., None]
    off_by = (x - rows.double()).abs() - 0.5 - tol / step.clamp(min=1e-300)[..., None] - 2.0 ** -22 * top
    assert (off_by[step > 0] <= 0).all(), float(off_by.max())
    assert (rows[step == 0] == 0).all()


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("d,pairs", [(64, 32), (64, 8), (128, 64), (128, 24)])
@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_against_the_plain_form(kv, d, pairs, adjacent):
    for T, n_h, n_kv, axes, fused in ((1, 4, 1, 1, False), (5, 16, 2, 3, True), (33, 8, 8, 2, True),
                                      (1000, 32, 8, 4, True), (777, 2, 1, 1, False),
                                      (3001, 8, 4, 3, True), (20011, 2, 2, 2, False)):
        gen, q, k, v, pos, freq, axis = inputs(T, n_h, n_kv, d, axes, pairs, T, fused=fused)
        blocks = T // 16 + 3
        pool = make_pool(gen, blocks, n_kv, d, kv)
        before = [None if t is None else t.clone() for t in pool]
        plain = [None if t is None else t.clone() for t in pool]
        slots = slots_of(gen, T, blocks)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = pa.pa_rope_write(q, k, v, pos.to(DEV), freq.to(DEV), slots.to(DEV), pool[0], pool[1],
                               axis=axis.to(DEV), adjacent=adjacent, amplitude=1.25,
                               k_scale=pool[2], v_scale=pool[3], dev_status=status)
        assert int(status.item()) == 0
        near(out, *turned(q.cpu().double(), pos, freq, axis, adjacent, 1.25))
        stored_near(pool, 0, slots, *turned(k.cpu().double(), pos, freq, axis, adjacent, 1.25), kv)
        # V is pa_cache_write's, bit for bit, and nothing else in the pool has changed
        pa.pa_cache_write(v.contiguous(), v.contiguous(), slots.to(DEV), plain[0], plain[1],
                          plain[2], plain[3])
        assert torch.equal(pool[1], plain[1])
        assert kv == "bf16" or torch.equal(pool[3], plain[3])
        free = torch.ones(blocks, 16, dtype=torch.bool)
        free[slots // 16, slots % 16] = False
        free = free[:, None].expand(blocks, n_kv, 16).to(DEV)
        assert torch.equal(pool[0][free], before[0][free])
        assert kv == "bf16" or torch.equal(pool[2][free], before[2][free])


@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
def test_position_zero_is_the_plain_append(kv):
    gen, q, k, v, pos, freq, axis = inputs(70, 8, 2, 128, 2, 64, 1)
    a = make_pool(gen, 8, 2, 128, kv)
    b = [None if t is None else t.clone() for t in a]
    slots = slots_of(gen, 70, 8).to(DEV)
    out = pa.pa_rope_write(q, k, v, torch.zeros_like(pos).to(DEV), freq.to(DEV), slots, a[0], a[1],
                           axis=axis.to(DEV), k_scale=a[2], v_scale=a[3])
    pa.pa_cache_write(k.contiguous(), v.contiguous(), slots, b[0], b[1], b[2], b[3])
    assert torch.equal(out, q)
    assert all(x is None or torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("lo,hi", [(0, 1 << 20), ((1 << 31) - 3000, (1 << 31) - 1),
                                   (-(1 << 31), -(1 << 31) + 3000), (-50, 50)])
def test_far_and_negative_positions(lo, hi):
    """The angle of every int32 position: an angle in fp32 would be off by whole turns. (An
    inv_freq counts as a 64-bit fraction of a turn: 2^31 of them are off by 2^-32 turns.)"""
    gen, q, k, v, pos, freq, axis = inputs(64, 4, 2, 128, 2, 64, 2, lo, hi)
    pool = make_pool(gen, 8, 2, 128, "bf16")
    out = pa.pa_rope_write(q, k, v, pos.to(DEV), freq.to(DEV), slots_of(gen, 64, 8).to(DEV), pool[0],
                           pool[1], axis=axis.to(DEV))
    want, tol = turned(q.cpu().double(), pos, freq, axis, False, 1.0)
    near(out, want, tol)


def test_one_axis_without_a_list():
    gen, q, k, v, pos, freq, _ = inputs(40, 4, 2, 64, 1, 16, 3)
    pool = make_pool(gen, 4, 2, 64, "bf16")
    out = pa.pa_rope_write(q, k, v, pos[0].to(DEV), freq.to(DEV), slots_of(gen, 40, 4).to(DEV), pool[0],
                           pool[1])
    near(out, *turned(q.cpu().double(), pos, freq, [0] * 16, False, 1.0))


def test_in_place_and_again():
    gen, q, k, v, pos, freq, axis = inputs(300, 8, 2, 128, 3, 64, 4, fused=False)
    pool = make_pool(gen, 20, 2, 128, "bf16")
    args = (pos.to(DEV), freq.to(DEV), slots_of(gen, 300, 20).to(DEV), pool[0], pool[1])
    want = pa.pa_rope_write(q, k, v, *args, axis=axis.to(DEV))
    mine = q.clone()
    got = pa.pa_rope_write(mine, k, v, *args, axis=axis.to(DEV), out=mine)
    assert got.data_ptr() == mine.data_ptr() and torch.equal(mine, want)
    # (half of q, or k: refused before anything runs)
    both = torch.cat([q, q])
    for x, y, out in ((both[:300], k, both[150:450]), (q[:, :2].contiguous(), k, k)):
        with pytest.raises(pa.PAError):
            pa.pa_rope_write(x, y, v, *args, axis=axis.to(DEV), out=out)


def test_slots_that_are_skipped_or_bad():
    gen, q, k, v, pos, freq, axis = inputs(50, 4, 2, 128, 1, 64, 5)
    for kv in ("bf16", "int8"):
        pool = make_pool(gen, 5, 2, 128, kv)
        want = [None if t is None else t.clone() for t in pool]
        slots = slots_of(gen, 50, 5)
        call = lambda s, p, **kw: pa.pa_rope_write(  # noqa: E731
            q, k, v, pos.to(DEV), freq.to(DEV), s.to(DEV), p[0], p[1], axis=axis.to(DEV),
            k_scale=p[2], v_scale=p[3], **kw)
        full = call(slots, want)
        bad = slots.clone()
        bad[3], bad[20], bad[49] = -1, -5, 80  # a pool of 80 slots
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        before = [None if t is None else t.clone() for t in pool]
        out = call(bad, pool, dev_status=status)
        assert int(status.item()) == pa.PA_DEV_BAD_SLOT and torch.equal(out, full)
        for a, b, c in zip(pool, want, before):
            if a is None:
                continue
            for t in range(50):
                blk, off = int(slots[t]) // 16, int(slots[t]) % 16
                assert torch.equal(a[blk, :, off], (c if t in (3, 20, 49) else b)[blk, :, off])


def test_axis_that_is_not_there_and_frequency_that_is_no_number():
    gen, q, k, v, pos, freq, axis = inputs(20, 4, 2, 128, 2, 64, 6)
    pool = make_pool(gen, 3, 2, 128, "bf16")
    slots = slots_of(gen, 20, 3).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    odd = axis.clone()
    odd[5], odd[9] = 2, -1
    out = pa.pa_rope_write(q, k, v, pos.to(DEV), freq.to(DEV), slots, pool[0], pool[1],
                           axis=odd.to(DEV), dev_status=status)
    assert int(status.item()) == pa.PA_DEV_BAD_CONTEXT
    for i in (5, 9):
        assert torch.equal(out[..., [i, i + 64]], q[..., [i, i + 64]])
    freq[7], freq[8] = float("nan"), float("inf")
    out = pa.pa_rope_write(q, k, v, pos.to(DEV), freq.to(DEV), slots, pool[0], pool[1],
                           axis=axis.to(DEV))
    nan = torch.isnan(out).all(0).all(0).cpu()
    assert nan.nonzero().flatten().tolist() == [7, 8, 71, 72] and not torch.isnan(out[..., 9]).any()


@pytest.mark.parametrize("kv", ["int8", "int4"])
def test_rows_of_zeros(kv):
    gen, q, k, v, pos, freq, axis = inputs(20, 4, 2, 64, 1, 32, 7)
    k[3] = 0
    v[4] = 0
    pool = make_pool(gen, 3, 2, 64, kv)
    slots = slots_of(gen, 20, 3)
    pa.pa_rope_write(q, k, v, pos.to(DEV), freq.to(DEV), slots.to(DEV), pool[0], pool[1],
                     axis=axis.to(DEV), k_scale=pool[2], v_scale=pool[3])
    for t, which in ((3, 0), (4, 1)):
        blk, off = int(slots[t]) // 16, int(slots[t]) % 16
        assert (pool[which][blk, :, off] == 0).all() and (pool[2 + which][blk, :, off] == 0).all()


def test_streams_graphs_and_prepared_calls():
    gen, q, k, v, pos, freq, axis = inputs(64, 32, 8, 128, 3, 64, 8)
    pools = [make_pool(gen, 6, 8, 128, "bf16") for _ in range(3)]
    for p in pools[1:]:
        for a, b in zip(p[:2], pools[0]):
            a.copy_(b)
    args = (q, k, v, pos.to(DEV), freq.to(DEV), slots_of(gen, 64, 6).to(DEV))
    want = pa.pa_rope_write(*args, *pools[0][:2], axis=axis.to(DEV))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    ax = axis.to(DEV)
    with torch.cuda.graph(graph, stream=s):
        out = pa.pa_rope_write(*args, *pools[1][:2], axis=ax)
    graph.replay()
    torch.cuda.synchronize()
    other = pa.pa_rope_write(*args, *pools[2][:2], axis=ax, stream=s)
    torch.cuda.synchronize()
    call = pa.pa_rope_write(*args, *pools[2][:2], axis=ax, prepare=True)
    assert torch.equal(out, want) and torch.equal(other, want) and torch.equal(call(), want)
    for p in pools[1:]:
        assert torch.equal(p[0], pools[0][0]) and torch.equal(p[1], pools[0][1])


def test_nothing_to_do():
    gen, q, k, v, pos, freq, axis = inputs(4, 4, 2, 64, 1, 32, 9)
    pool = make_pool(gen, 3, 2, 64, "bf16")
    out = pa.pa_rope_write(q[:0], k[:0], v[:0], pos[:, :0].to(DEV).contiguous(), freq.to(DEV),
                           torch.zeros(0, dtype=torch.int64, device=DEV), pool[0], pool[1])
    assert out.shape == (0, 4, 64)

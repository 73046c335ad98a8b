"""Host-side checks of pa_window_attention and pa_window_decode: arguments refused before any CUDA call."""
import ctypes

import pytest
import torch

import paged_kv_cache_94_gb300 as pa
from paged_kv_cache_94_gb300 import build as pa_build

FAKE = ctypes.c_void_p(256)  # never dereferenced: the calls return before any launch
FAR = ctypes.c_void_p(1 << 30)
ODD = ctypes.c_void_p(258)


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.library()


def _geom(**kw):
    base = dict(num_blocks=100, n_h=32, n_kv=8, d_h=128, block_size=16, kv_dtype=0, reserved=0)
    base.update(kw)
    return pa.pa_geom(**base)


def test_decode_argument_checks(lib):
    def call(q=FAKE, kc=FAKE, ks=None, bt=FAKE, mb=16, ctx=FAKE, B=4, window=64, first=4, out=FAR,
             ws=FAKE, g=None, grid=0):
        return lib.pa_window_decode(q, kc, FAKE, ks, ks, bt, mb, ctx, B, 0.1, window, first, out, ws,
                                    1 << 20, g or _geom(), None, None, grid)
    assert call(B=0) == 0
    for kw in (dict(B=-1), dict(B=8193), dict(mb=0), dict(grid=-1), dict(window=-1), dict(first=-1)):
        assert call(**kw) == -2, kw
    assert call(mb=1 << 30) == -4
    for kw in (dict(q=None), dict(kc=None), dict(bt=None), dict(ctx=None), dict(out=None)):
        assert call(**kw) == -1, kw
    assert call(ws=None) == -7
    for kw in (dict(q=ODD), dict(kc=ODD), dict(out=ODD), dict(ws=ctypes.c_void_p(272))):
        assert call(**kw) == -11, kw
    assert call(ks=FAKE) == -2 and call(g=_geom(kv_dtype=1)) == -1
    assert call(out=FAKE) == -2 and call(out=ctypes.c_void_p(256 + 8192)) == -2  # meets q
    assert call(g=_geom(d_h=96)) == -4 and call(g=_geom(n_h=30)) == -2


def test_decode_workspace_size(lib):
    # counters, and a record for each CTA and unit
    assert lib.pa_window_decode_workspace_size(_geom(), 4, 10) == 256 + (10 + 32) * 4 * 130 * 4
    assert lib.pa_window_decode_workspace_size(_geom(d_h=96), 4, 10) == 0
    assert lib.pa_window_decode_workspace_size(_geom(), -1, 10) == 0


def test_decode_binding_refuses():
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_window_decode(q, kc, kc, i, i[0], 0.1, 4, 1)


def test_attention_argument_checks(lib):
    def call(q=FAKE, T=64, cu=FAKE, kc=FAKE, ks=None, bt=FAKE, mb=16, ctx=FAKE, B=4, window=64,
             first=4, out=FAR, ws=FAKE, g=None, grid=0):
        return lib.pa_window_attention(q, T, cu, kc, FAKE, ks, ks, bt, mb, ctx, B, 0.1, window, first,
                                       out, ws, 1 << 20, g or _geom(), None, None, grid)
    assert call(B=0) == 0 and call(T=0) == 0
    for kw in (dict(T=-1), dict(B=-1), dict(B=8193), dict(mb=0), dict(grid=-1), dict(grid=8193),
               dict(window=-1), dict(first=-1)):
        assert call(**kw) == -2, kw
    assert call(T=1 << 26) == -4 and call(mb=1 << 30) == -4
    for kw in (dict(q=None), dict(cu=None), dict(kc=None), dict(bt=None), dict(ctx=None),
               dict(out=None)):
        assert call(**kw) == -1, kw
    assert call(ws=None) == -7
    for kw in (dict(q=ODD), dict(cu=ODD), dict(kc=ODD), dict(out=ODD), dict(bt=ODD),
               dict(ctx=ODD), dict(ws=ctypes.c_void_p(272))):
        assert call(**kw) == -11, kw
    assert call(ks=FAKE) == -2 and call(g=_geom(kv_dtype=1)) == -1
    assert call(out=FAKE) == -2 and call(out=ctypes.c_void_p(256 + 8192)) == -2  # meets q
    assert call(g=_geom(d_h=96)) == -4 and call(g=_geom(n_h=30)) == -2


def test_attention_workspace_size_and_binding(lib):
    assert lib.pa_window_attention_workspace_size(_geom(), 100) == 512 + 100 * 2 * 256 * 130 * 4
    assert lib.pa_window_attention_workspace_size(_geom(d_h=96), 4) == 0
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_window_attention(q, torch.zeros(2, dtype=torch.int32), kc, kc, i, i[0], 0.1, 4, 1)
    with pytest.raises(ValueError, match="32 bits"):
        pa.pa_window_attention(q, torch.zeros(2, dtype=torch.int32), kc, kc, i, i[0], 0.1, 1 << 40)


def test_blocks_behind_the_window_go_back(lib):
    """A sequence gives the blocks between its first tokens' and its window's back
    (pa_allocator_free on those table entries) and goes on appending; the pool hands them out
    again, and the sequence's own end releases the rest."""
    import numpy as np
    window, n_first, total = 40, 20, 12
    alloc = pa.BlockAllocator(total)
    table, _ = alloc.allocate_prompt(np.arange(100, dtype=np.int32))
    tables = np.full((1, 64), -1, np.int32)
    tables[0, :len(table)] = table
    n = np.array([len(table)], np.int32)
    gone = set()
    for i in range(300):  # far more tokens than the pool has room for at once
        slots, cow = alloc.append_slots(tables, n, np.array([i], np.int32))
        ctx = 101 + i
        assert len(cow) == 0 and slots[0] // 16 == tables[0, n[0] - 1] and slots[0] % 16 == (ctx - 1) % 16
        for j in range(-(-n_first // 16), max(0, ctx + 1 - window) // 16):
            if tables[0, j] >= 0:
                alloc.free(tables[0, j:j + 1].copy())
                gone.add(int(tables[0, j]))
                tables[0, j] = -1
        held = [int(b) for b in tables[0, :n[0]] if b >= 0]
        assert len(held) == len(set(held)) and alloc.num_free() == total - len(held)
    assert any(b in gone for b in held)  # the pool has handed some out again
    alloc.free(np.array(held, np.int32))
    assert alloc.num_free() == total

"""Host-side checks of the attention-mass and eviction entry points: argument
checks that return before any CUDA call, and the allocator's private blocks."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_94_gb300 as pa
from paged_kv_cache_94_gb300 import build as pa_build

FAKE = ctypes.c_void_p(256)  # never dereferenced: the calls return before any launch
OTHER = ctypes.c_void_p(512)
ODD = ctypes.c_void_p(258)


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.library()


def _geom(**kw):
    base = dict(num_blocks=100, n_h=32, n_kv=8, d_h=128, block_size=16, kv_dtype=0, reserved=0)
    base.update(kw)
    return pa.pa_geom(**base)


def test_decode_mass_argument_checks(lib):
    def call(mass=FAKE, mass_out=FAKE, B=4, mb=16, ws=FAKE, g=None, grid=0, q=FAKE, ks=None):
        return lib.pa_decode_mass(q, FAKE, FAKE, ks, ks, FAKE, mb, FAKE, B, 0.1, FAKE, mass,
                                  mass_out, ws, 1 << 20, g or _geom(), None, None, grid)
    assert call(B=0) == 0
    assert call(B=-1) == -2 and call(B=9000) == -2 and call(mb=0) == -2 and call(grid=-1) == -2
    assert call(mass=None) == -1 and call(mass_out=None) == -1 and call(q=None) == -1
    assert call(ws=None) == -7
    assert call(mass=ctypes.c_void_p(264)) == -11 and call(mass_out=ODD) == -11
    assert call(ks=FAKE) == -2                       # bf16 pools take no scales
    assert call(g=_geom(kv_dtype=1)) == -1
    assert call(g=_geom(d_h=96)) == -4


def test_decode_mass_workspace_holds_the_scores(lib):
    g = _geom()
    a = lib.pa_decode_mass_workspace_size(g, 4, 10, 100)
    b = lib.pa_decode_mass_workspace_size(g, 4, 11, 100)
    assert b - a == 4 * 32 * 16 * 4                  # one block of scores a query head
    assert a > lib.pa_decode_workspace_size(g, 4, 100) + 4 * 32 * 160 * 4
    for bad in (dict(n_h=30), dict(d_h=96)):
        assert lib.pa_decode_mass_workspace_size(_geom(**bad), 4, 10, 100) == 0
    assert lib.pa_decode_mass_workspace_size(g, -1, 10, 100) == 0
    assert lib.pa_decode_mass_workspace_size(g, 4, 0, 100) == 0
    assert lib.pa_decode_mass_workspace_size(g, 8192, 1 << 20, 100) == 0


def test_evict_select_argument_checks(lib):
    def call(mass=FAKE, S=64, ctx=FAKE, B=4, n_kv=8, budget=16, recent=4, keep=FAKE, lens=FAKE):
        return lib.pa_evict_select(mass, S, ctx, B, n_kv, budget, recent, keep, lens, None, None)
    assert call(B=0) == 0
    for kw in (dict(B=-1), dict(B=8193), dict(n_kv=0), dict(S=0), dict(S=1 << 31), dict(budget=0),
               dict(budget=-3), dict(recent=-1), dict(recent=17)):
        assert call(**kw) == -2, kw
    for kw in (dict(mass=None), dict(ctx=None), dict(keep=None), dict(lens=None)):
        assert call(**kw) == -1, kw
    assert call(mass=ODD) == -11 and call(keep=ODD) == -11
    assert call(n_kv=1 << 26) == -4


def test_evict_compact_argument_checks(lib):
    def call(kc=FAKE, ks=None, bt=FAKE, mb=16, keep=FAKE, budget=16, lens=FAKE, nt=OTHER, nb=4,
             B=4, mass=None, mo=None, g=None):
        return lib.pa_evict_compact(kc, FAKE, ks, ks, bt, mb, keep, budget, lens, nt, nb, B, mass,
                                    mo, g or _geom(), None, None)
    assert call(B=0) == 0
    for kw in (dict(B=-1), dict(mb=0), dict(nb=0), dict(budget=0)):
        assert call(**kw) == -2, kw
    assert call(nt=FAKE) == -2                       # in place
    assert call(mass=FAKE, mo=FAKE) == -2
    assert call(mass=FAKE) == -1 and call(mo=FAKE) == -1
    for kw in (dict(kc=None), dict(bt=None), dict(keep=None), dict(lens=None), dict(nt=None)):
        assert call(**kw) == -1, kw
    assert call(kc=ODD) == -11 and call(keep=ODD) == -11
    assert call(ks=FAKE) == -2 and call(g=_geom(kv_dtype=2)) == -1
    assert call(mb=1 << 30) == -4


def test_select_refuses_to_write_the_lengths_it_reads(lib):
    assert lib.pa_evict_select(FAKE, 64, FAKE, 4, 8, 16, 4, OTHER, FAKE, None, None) == -2


def test_compact_refuses_tables_of_more_rows_than_32_bits_count(lib):
    """2^27 blocks of 16 rows for one sequence."""
    assert lib.pa_evict_compact(FAKE, FAKE, None, None, FAKE, 16, FAKE, 16, FAKE, OTHER, 1 << 27, 1,
                                FAKE, OTHER, _geom(), None, None) == -4


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    m = torch.zeros(1, 2, 16)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_decode_mass(q, kc, kc, i, i[0], 0.1, m)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_evict_select(m, i[0], 4)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_evict_compact(kc, kc, i, torch.zeros(1, 2, 4, dtype=torch.int32), i[0], i)


def test_private_blocks(lib):
    a = pa.BlockAllocator(8)
    prompt, _ = a.allocate_prompt(list(range(40)))            # 3 blocks
    t = a.allocate_private(37)
    assert len(t) == 3 and not set(t) & set(prompt)
    assert [a.block_info(b) for b in t] == [(1, 16, None), (1, 16, None), (1, 5, None)]
    assert a.num_free() == 2
    # a prompt of the private blocks' token ids hits none of them
    again, cached = a.allocate_prompt([0] * 16)
    assert cached == 0 and again[0] not in t
    # appending goes on behind the last row
    tables = np.full((1, 4), -1, np.int32)
    tables[0, :3] = t
    n = np.array([3], np.int32)
    slots, cow = a.append_slots(tables, n, [7])
    assert slots[0] == t[2] * 16 + 5 and len(cow) == 0 and n[0] == 3
    free = a.num_free()
    with pytest.raises(pa.PAError) as e:
        a.allocate_private(16 * (free + 1))
    assert e.value.status == pa.PA_ERR_OUT_OF_BLOCKS and a.num_free() == free
    assert len(a.allocate_private(0)) == 0
    with pytest.raises(pa.PAError):
        a.allocate_private(-1)
    a.free(t)
    assert a.num_free() == free + 3
    n_blocks = ctypes.c_int32()
    table = np.empty(4, np.int32)
    p = ctypes.c_void_p(table.ctypes.data)
    assert lib.pa_allocator_allocate_private(a._h, 40, p, 2, ctypes.byref(n_blocks)) == -2
    assert lib.pa_allocator_allocate_private(a._h, 40, None, 4, ctypes.byref(n_blocks)) == -1
    assert lib.pa_allocator_allocate_private(None, 40, p, 4, ctypes.byref(n_blocks)) == -1


def test_private_blocks_of_more_tokens_than_32_bits_count():
    """2^32 + 16 tokens are not 16."""
    a = pa.BlockAllocator(8)
    with pytest.raises(ValueError, match="32 bits"):
        a.allocate_private((1 << 32) + 16)
    assert a.num_free() == 8

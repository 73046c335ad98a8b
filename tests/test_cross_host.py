"""Host-side checks of pa_cross_attention: arguments refused before any CUDA call."""
import ctypes

import pytest
import torch

import paged_kv_cache_94_gb300 as pa
from paged_kv_cache_94_gb300 import build as pa_build

FAKE = ctypes.c_void_p(256)  # never dereferenced: the calls return before any launch
ODD = ctypes.c_void_p(258)


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.library()


def _geom(**kw):
    base = dict(num_blocks=100, n_h=32, n_kv=8, d_h=128, block_size=16, kv_dtype=0, reserved=0)
    base.update(kw)
    return pa.pa_geom(**base)


def test_argument_checks(lib):
    def call(q=FAKE, T=64, cu=FAKE, kc=FAKE, ks=None, bt=FAKE, mb=16, ctx=FAKE, B=4, out=FAKE,
             ws=FAKE, g=None, grid=0):
        return lib.pa_cross_attention(q, T, cu, kc, FAKE, ks, ks, bt, mb, ctx, B, 0.1, out, ws,
                                      1 << 20, g or _geom(), None, None, grid)
    assert call(B=0) == 0 and call(T=0) == 0
    for kw in (dict(T=-1), dict(B=-1), dict(B=8193), dict(mb=0), dict(grid=-1), dict(grid=8193)):
        assert call(**kw) == -2, kw
    assert call(T=1 << 26) == -4 and call(mb=1 << 30) == -4
    for kw in (dict(q=None), dict(cu=None), dict(kc=None), dict(bt=None), dict(ctx=None),
               dict(out=None)):
        assert call(**kw) == -1, kw
    assert call(ws=None) == -7
    for kw in (dict(q=ODD), dict(cu=ODD), dict(kc=ODD), dict(out=ODD), dict(bt=ODD),
               dict(ctx=ODD), dict(ws=ctypes.c_void_p(272))):
        assert call(**kw) == -11, kw
    assert call(g=_geom(kv_dtype=1), ks=ctypes.c_void_p(264)) == -11
    assert call(ks=FAKE) == -2 and call(g=_geom(kv_dtype=1)) == -1
    assert call(g=_geom(d_h=96)) == -4 and call(g=_geom(n_h=30)) == -2
    assert call(g=_geom(kv_dtype=9)) == -3


def test_workspace_size(lib):
    assert lib.pa_cross_workspace_size(_geom(), 100) == 512 + 100 * 2 * 256 * 130 * 4
    assert lib.pa_cross_workspace_size(_geom(d_h=64), 1) == 256 + 2 * 256 * 66 * 4
    assert lib.pa_cross_workspace_size(_geom(d_h=96), 4) == 0
    assert lib.pa_cross_workspace_size(_geom(), -1) == 0
    assert lib.pa_cross_workspace_size(_geom(), 8193) == 0


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_cross_attention(q, torch.zeros(2, dtype=torch.int32), kc, kc, i, i[0], 0.1)

"""Host-side checks of pa_rope_write: arguments refused before any CUDA call."""
import ctypes

import pytest
import torch

import paged_kv_cache_94_gb300 as pa
from paged_kv_cache_94_gb300 import build as pa_build

FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: the calls return before any launch
FAR = ctypes.c_void_p(1 << 30)
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.library()


def _geom(**kw):
    base = dict(num_blocks=100, n_h=32, n_kv=8, d_h=128, block_size=16, kv_dtype=0, reserved=0)
    base.update(kw)
    return pa.pa_geom(**base)


def test_argument_checks(lib):
    def call(q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, T=64, pos=FAKE, axes=1, freq=FAKE,
             axis=None, pairs=64, adjacent=0, slots=FAKE, out=FAR, kc=FAR, scales=None, g=None):
        return lib.pa_rope_write(q, qs, k, ks, v, vs, T, pos, axes, freq, axis, pairs, adjacent, 1.0,
                                 slots, out, kc, FAR, scales, scales, g or _geom(), None, None)
    assert call(T=0) == 0
    for kw in (dict(T=-1), dict(axes=0), dict(axes=5), dict(pairs=0), dict(pairs=72),
               dict(adjacent=2), dict(qs=4088), dict(ks=1016), dict(vs=0)):
        assert call(**kw) == -2, kw
    for kw in (dict(pairs=12), dict(T=1 << 31), dict(g=_geom(n_h=65536, n_kv=4096))):
        assert call(**kw) == -4, kw
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(pos=None), dict(freq=None),
               dict(slots=None), dict(out=None), dict(kc=None)):
        assert call(**kw) == -1, kw
    for kw in (dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(pos=ODD), dict(freq=ODD), dict(axis=ODD),
               dict(slots=ODD), dict(out=ODD), dict(kc=ODD), dict(qs=4100), dict(ks=1028),
               dict(vs=1028)):
        assert call(**kw) == -11, kw
    assert call(scales=FAKE) == -2 and call(g=_geom(kv_dtype=1)) == -1
    assert call(g=_geom(kv_dtype=2), scales=ODD) == -11
    assert call(g=_geom(d_h=96)) == -4 and call(g=_geom(n_h=30)) == -2
    # out meets part of what is read: a token's queries further on, or the keys
    assert call(out=ctypes.c_void_p((1 << 20) + 8192)) == -2
    assert call(out=FAKE, q=FAR) == -2
    assert call(out=FAKE, qs=8192, k=FAR, v=FAR) == -2  # q in place, but not dense


def test_binding_refuses_cpu_tensors():
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_rope_write(x, x, x, torch.zeros(1, dtype=torch.int32), torch.zeros(32).double(),
                         torch.zeros(1, dtype=torch.int64), kc, kc)

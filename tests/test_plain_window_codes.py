"""The plain form of the window decode over codes, and that its tolerance can tell (CPU)."""
import pytest
import torch

from tests.plain_window import attend_seen
from tests.plain_window_codes import attend_codes


def rows(n, d, g, spread, bits):
    """Queries and dequantised K and V of n tokens; V rows over `spread` decades."""
    gen = torch.Generator().manual_seed(n)
    top = 127 if bits == 8 else 7
    q = torch.randn(g, d, generator=gen, dtype=torch.float64)
    k, v = (torch.randn(n, d, generator=gen, dtype=torch.float64) for _ in range(2))
    v = v * 10 ** (spread * (torch.rand(n, 1, generator=gen, dtype=torch.float64) - 0.5))
    out = []
    for x in (k, v):
        s = x.abs().amax(1) / top
        out += [torch.round(x / s[:, None]) * s[:, None], s]
    return q, out[0], out[2], out[3]


@pytest.mark.parametrize("n,spread,bits", [(17, 0, 8), (300, 6, 4), (300, 6, 8)])
def test_it_is_the_plain_form(n, spread, bits):
    q, k, v, s = rows(n, 64, 4, spread, bits)
    seen = torch.rand(4, n, generator=torch.Generator().manual_seed(1)) < 0.7
    seen[2] = False
    o, tol = attend_codes(q, k, v, s, 1 << (bits - 1), 0.125, seen)
    want, _ = attend_seen(q, k, v, 0.125, seen)
    assert torch.equal(o, want) and (o[2] == 0).all() and torch.isfinite(tol).all()


@pytest.mark.parametrize("n,spread,bits", [(3001, 0, 8), (3001, 0, 4), (1201, 6, 8), (1201, 6, 4)])
def test_a_block_left_out_is_seen(n, spread, bits):
    """An output without one of the blocks is outside the tolerance for many of its elements."""
    q, k, v, s = rows(n, 128, 16, spread, bits)
    seen = torch.ones(16, n, dtype=torch.bool)
    o, tol = attend_codes(q, k, v, s, 1 << (bits - 1), 128 ** -0.5, seen)
    tol = tol + 2.0 ** -8 * (o.abs() + tol)
    for block in (0, 33, 70):
        less = seen.clone()
        less[:, 16 * block:16 * block + 16] = False
        other, _ = attend_codes(q, k, v, s, 1 << (bits - 1), 128 ** -0.5, less)
        assert ((other - o).abs() > tol).double().mean() > 0.25

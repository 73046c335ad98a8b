"""The plain forms of window attention and rotary positions against the definitions written
out key by key (CPU)."""
import math

import pytest
import torch

from tests.plain_window import attend_seen, seen_keys, turned


@pytest.mark.parametrize("window,n_first", [(0, 0), (0, 5), (1, 0), (3, 2), (100, 1), (4, 100)])
def test_seen_keys(window, n_first):
    for ctx, new in ((1, 1), (9, 9), (20, 3)):
        got = seen_keys(new, ctx, window, n_first)
        for i in range(new):
            p = ctx - new + i
            want = [j <= p and (window == 0 or p - j < window or j < n_first) for j in range(ctx)]
            assert got[i].tolist() == want


def test_attend_seen_row_by_row():
    gen = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(n, 8, generator=gen, dtype=torch.float64) for n in (3, 5, 5))
    seen = torch.tensor([[1, 0, 0, 1, 0], [0, 0, 0, 0, 0], [1, 1, 1, 1, 0]], dtype=torch.bool)
    k[4] = v[4] = float("nan")  # nobody sees it
    o, tol = attend_seen(q, k, v, 0.7, seen)
    for r in (0, 2):
        e = [math.exp(0.7 * float(q[r] @ k[j])) if seen[r, j] else 0.0 for j in range(5)]
        want = sum(e[j] * v[j] for j in range(5) if seen[r, j]) / sum(e)
        assert torch.allclose(o[r], want, rtol=1e-12, atol=1e-12)
    assert (o[1] == 0).all() and torch.isfinite(tol).all()


@pytest.mark.parametrize("adjacent", [False, True])
def test_turned_is_a_rotation_of_each_pair(adjacent):
    x = torch.zeros(2, 1, 8, dtype=torch.float64)
    x[:, 0, 2 if adjacent else 1] = 1.0   # the first value of pair 1
    x[:, 0, 6] = 5.0                      # behind three pairs: stays
    freq = torch.tensor([1.0, math.pi / 2, 0.1])
    pos = torch.tensor([[7, 9], [1, 3]])
    y, _ = turned(x, pos, freq, [0, 1, 0], adjacent, 2.0)
    first, second = (2, 3) if adjacent else (1, 4)
    assert torch.allclose(y[:, 0, first], torch.tensor([0.0, 0.0], dtype=torch.float64), atol=1e-6)
    assert torch.allclose(y[:, 0, second], torch.tensor([2.0, -2.0], dtype=torch.float64))
    assert (y[:, 0, 6] == 5.0).all()

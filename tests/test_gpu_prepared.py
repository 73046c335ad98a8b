"""Prepared calls of cross attention and of the decode with masses, issued on another stream
than the one that prepared them: their hidden counters are zero and their memory is
theirs, whatever the preparing stream still has to run."""
import pytest
import torch

import paged_kv_cache_94_gb300 as pa
from tests.test_gpu_evict import make_pool, make_tables

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SLEEP = 200_000_000  # cycles: about a tenth of a second of a stream


def setting(op):
    """call(**kw) of an operator whose units are cut (a cut unit needs its counter), the bytes
    of its workspace, and the tensors that a run writes."""
    gen = torch.Generator().manual_seed(1)
    ctx, n_kv, g, d = [5000, 900], 2, 4, 128
    bt, total, _ = make_tables(gen, ctx)
    pool = make_pool(gen, total, n_kv, d, "bf16")
    btd, cl = bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV)
    geom = pa.geometry(pool[0], n_kv * g)
    q = torch.randn(2, n_kv * g, d, generator=gen).to(torch.bfloat16).to(DEV)
    if op == "cross":
        cu = torch.arange(3, dtype=torch.int32, device=DEV)

        def call(**kw):
            return pa.pa_cross_attention(q, cu, pool[0], pool[1], btd, cl, 0.1, **kw)
        nbytes = pa.library().pa_cross_workspace_size(geom, 0)
    else:
        mass = torch.zeros(2, n_kv, bt.shape[1] * 16, device=DEV)
        mass_out = torch.empty_like(mass)

        def call(**kw):
            return pa.pa_decode_mass(q, pool[0], pool[1], btd, cl, 0.1, mass, mass_out=mass_out,
                                     **kw)
        nbytes = pa.library().pa_decode_mass_workspace_size(geom, 2, bt.shape[1], 0)
    want = call().clone()
    torch.cuda.synchronize()
    return call, nbytes, want


def soil(nbytes, stream):
    """Blocks of the stream's allocator, of a workspace's size, left full of ones."""
    with torch.cuda.stream(stream):
        junk = [torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]
        del junk


@pytest.mark.parametrize("op", ["cross", "mass"])
def test_prepared_on_a_busy_stream_and_issued_on_another(op):
    call, nbytes, want = setting(op)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    soil(nbytes, a)
    with torch.cuda.stream(a):
        torch.cuda._sleep(SLEEP)
        prepared = call(prepare=True)
    with torch.cuda.stream(b):
        for _ in range(3):
            out = prepared()
    b.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("op", ["cross", "mass"])
def test_memory_of_a_dropped_call_is_not_reused_under_it(op):
    call, nbytes, want = setting(op)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        prepared = call(prepare=True)
    with torch.cuda.stream(b):
        torch.cuda._sleep(SLEEP)
        out = prepared()
    del prepared
    soil(nbytes, a)
    with torch.cuda.stream(a):
        others = [call(prepare=True) for _ in range(4)]
        soil(nbytes, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for other in others:
        assert torch.equal(other(), want)
        torch.cuda.synchronize()


@pytest.mark.parametrize("op", ["cross", "mass"])
def test_prepared_inside_a_capture_or_captured_later(op):
    call, nbytes, want = setting(op)
    soil(nbytes, torch.cuda.current_stream())
    before = call(prepare=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        inside = call(prepare=True)
        out = inside()
        out_before = before()
    torch.cuda.synchronize()
    for _ in range(3):
        out.zero_()
        out_before.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out_before, want)
    out.zero_()
    inside()  # and outside the graph
    torch.cuda.synchronize()
    assert torch.equal(out, want)

"""pa_prefill launches that run at the same time share nothing: captured calls
replayed on two streams at once, and more eager calls in flight than a table
of launches would hold."""
import numpy as np
import pytest

from paged_kv_cache_120_gb300 import binding, workloads

from test_gpu_cross import dev  # noqa: F401
from test_gpu_nonfinite import Poisoned

pytestmark = pytest.mark.gpu


def make(dev, k, dtype, fp8):
    """Many work units, ragged; the two have different unit counts."""
    rng = np.random.default_rng(30 + k)
    n = (60, 41)[k]
    qlen = rng.integers(0, 150, n)
    qlen[0] = 300
    c = Poisoned(dev, dtype, *((8, 8, 64), (16, 4, 64))[k], qlen, qlen + rng.integers(0, 200, n), fp8=fp8, seed=40 + k)
    c.causal = True
    c.reference()
    return c


def call(c, out, stream=None):
    total = int(c.cu[-1])
    a = (out[:total], c.q[:total], c.pool, c.bt_d, c.cu_d, c.kv_d, c.scale, c.max_q)
    if c.fp8:
        binding.pa_prefill_fp8(*a, workloads.FP8_K_SCALE, workloads.FP8_V_SCALE, None, stream)
    else:
        binding.pa_prefill(*a, None, stream)


@pytest.mark.parametrize("dtype,fp8", [(workloads.F16, False), (workloads.BF16, True)], ids=["f16", "bf16-fp8"])
def test_two_graphs_at_once_share_nothing(dev, dtype, fp8):
    import torch
    cases = [make(dev, k, dtype, fp8) for k in range(2)]
    outs = [torch.full_like(c.q, float("nan")) for c in cases]
    graphs, streams = [torch.cuda.CUDAGraph() for _ in cases], [torch.cuda.Stream() for _ in cases]
    for c, o in zip(cases, outs):
        call(c, o)
    torch.cuda.synchronize()
    for c, o, g in zip(cases, outs, graphs):
        with torch.cuda.graph(g, capture_error_mode="relaxed"):
            for _ in range(40):
                call(c, o)
    for _ in range(4):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for c, o in zip(cases, outs):
            c.check(o)


def test_a_graph_beside_eager_calls(dev):
    """200 eager calls on one stream while a graph of them replays on another."""
    import torch
    a, b = (make(dev, k, workloads.F16, False) for k in range(2))
    oa, ob = (torch.full_like(c.q, float("nan")) for c in (a, b))
    call(a, oa)
    call(b, ob)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        for _ in range(70):
            call(a, oa)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for o in (oa, ob):
        o.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side[0]):
            g.replay()
        for _ in range(70):
            call(b, ob, side[1])
    torch.cuda.synchronize()
    a.check(oa)
    b.check(ob)


@pytest.mark.parametrize("most", [1000, 4096, 2 ** 31 - 1])
def test_a_loose_query_bound(dev, most):
    """Units beyond the chunks are claimed and skipped; a bound above all the queries says no more than their number."""
    import torch
    c = make(dev, 1, workloads.F16, False)
    out = torch.full_like(c.q, float("nan"))
    c.max_q = most
    call(c, out)
    c.check(out)

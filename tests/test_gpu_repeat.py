"""The same bits again: cross attention repeats itself whatever ran before it,
and a sequence's rows do not depend on its neighbours' queries."""
import numpy as np
import pytest

from paged_kv_cache_120_gb300 import workloads

from test_gpu_cross import CrossCase, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def bits(t):
    import torch
    return t.view(torch.int16)


@pytest.mark.parametrize("split", [False, True], ids=["whole", "split"])
@pytest.mark.parametrize("heads,qlen", [((7, 1, 64), [10, 16, 40]), ((6, 2, 128), [25, 40, 9]), ((4, 4, 64), [100, 70]),
                                        ((5, 1, 128), [24, 10])],
                         ids=lambda x: "x".join(map(str, x)))
def test_rows_do_not_depend_on_the_neighbours_queries(dev, heads, qlen, split):
    """The first sequence's rows, with ordinary and with huge queries behind them (a query tile's rows past the sequence
    hold the next one's)."""
    import torch
    c = CrossCase(dev, workloads.F16, *heads, qlen, [700] * len(qlen), seed=1, extra_width=250)
    c.pool *= 9
    first = c.run(c.workspace() if split else None).clone()
    n = int(c.cu[1])
    c.q[n:int(c.cu[-1])] = 60000
    again = c.run(c.workspace() if split else None)
    torch.cuda.synchronize()
    assert torch.isfinite(first[:n]).all()
    assert torch.equal(bits(first[:n]), bits(again[:n]))


@pytest.mark.parametrize("split", [False, True], ids=["whole", "split"])
@pytest.mark.parametrize("heads,qlen", [((7, 1, 64), [16, 32]), ((6, 2, 128), [40, 80]), ((20, 4, 64), [24] * 9),
                                        ((15, 1, 128), [8] * 5)],
                         ids=lambda x: "x".join(map(str, x)))
def test_rows_do_not_depend_on_what_ran_before(dev, heads, qlen, split):
    """A group of heads that leaves rows of the query tile unfilled: they hold what the last kernel left in shared memory,
    here its queries, ordinary or huge."""
    import torch
    c = CrossCase(dev, workloads.F16, *heads, qlen, [700] * len(qlen), seed=2, extra_width=250)
    c.pool *= 9
    # Fills both query tiles of every SM, at the victim's head size.
    filler = CrossCase(dev, workloads.F16, 4, 4, heads[2], [256] * 100, [16] * 100, seed=3)
    results = []
    for value in (0.0, 60000.0, -60000.0):
        filler.q.fill_(value)
        ws = c.workspace() if split else None
        torch.cuda.synchronize()
        filler.run()
        results.append(c.run(ws).clone())
    torch.cuda.synchronize()
    total = int(c.cu[-1])
    for r in results[1:]:
        assert torch.equal(bits(results[0][:total]), bits(r[:total]))


@pytest.mark.parametrize("dtype,fp8", [(workloads.F16, False), (workloads.BF16, True)], ids=["f16", "bf16-fp8"])
@pytest.mark.parametrize("heads,qmax,kvmax,n", [((20, 20, 64), 1, 1500, 64), ((32, 8, 128), 4, 3000, 20),
                                                ((32, 8, 128), 600, 2000, 4), ((20, 20, 64), 224, 1500, 40)],
                         ids=["decode", "candidates", "chunks", "prompts"])
def test_twenty_calls_give_the_same_bits(dev, heads, qmax, kvmax, n, dtype, fp8):
    import torch
    rng = np.random.default_rng(5)
    c = CrossCase(dev, dtype, *heads, rng.integers(0, qmax + 1, n) if qmax > 1 else [1] * n, rng.integers(0, kvmax + 1, n),
                  fp8=fp8, seed=4)
    for ws in (c.workspace(), None):
        first = c.run(ws).clone()
        c.check(first)
        total = int(c.cu[-1])
        for _ in range(20):
            again = c.run(ws)
            assert torch.equal(bits(again[:total]), bits(first[:total]))

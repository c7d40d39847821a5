"""Tree attention of one query tile: a row's threads read the output only behind the last P V of their unit, however far apart the
threads of a unit are. Bounds as in test_gpu_tree_attention.py."""
import numpy as np
import pytest

import test_gpu_tree_attention as single
from test_gpu_tree_attention import Batch, dev  # noqa: F401

from paged_kv_cache_120_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [True, False], ids=["fp8", "16"])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", [(16, 2, 128), (12, 2, 64), (40, 8, 128)])
def test_many_units_repeat(dev, hq, hkv, d, kind, fp8):  # noqa: F811
    """Units of two to four K/V tiles, some of whose rows wait for V elements to be cleared: forty runs, one result."""
    rng = np.random.default_rng(d + hq)
    seqs = 170
    counts, context = rng.integers(3, 17, seqs), rng.integers(100, 420, seqs)
    b = Batch(dev, 4, counts.tolist(), context.tolist(), hq, hkv, d, kind, fp8, 16)
    out = b.run()
    b.check(out)
    for s in range(0, seqs, 3):  # the tree's last node holds NaN in V: its own row, and no other
        b.flat[1, b.slots[s][-1]] = 0x7F if fp8 else float("nan")
    first = b.run()
    seen_by = [set(np.flatnonzero(b.seen[s][:, -1])) for s in range(seqs)]
    for s in range(seqs):
        clean = [i for i in range(counts[s]) if s % 3 or i not in seen_by[s]]
        rows = [int(b.cu[s]) + i for i in clean]
        assert (first[rows] == out[rows]).all(), s
    for _ in range(40):
        again = b.run()
        assert ((again == first) | (again.isnan() & first.isnan())).all(), "two runs differ"
    assert binding.pa_get_device_error() == 0


@pytest.mark.parametrize("turn", range(6))
@pytest.mark.parametrize("fp8", [True, False], ids=["fp8", "16"])
def test_nonfinite_nodes_of_ragged_trees(dev, fp8, turn):  # noqa: F811
    rng = np.random.default_rng(turn)
    single.test_nonfinite_nodes_reach_only_who_sees_them(dev, rng.integers(2, 10, 150).tolist(), rng.integers(0, 400, 150).tolist(), 16, 2,
                                                         128, "bf16", fp8)

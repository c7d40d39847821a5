"""Tree attention of two query tiles in large batches of ragged trees: a CTA works on one unit after another, and most units' second
tile has no queries. The bounds are those of test_gpu_tree_attention.py."""
import numpy as np
import pytest

import test_gpu_tree_attention as single
from test_gpu_tree_attention import Batch, dev  # noqa: F401

from paged_kv_cache_120_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [True, False], ids=["fp8", "16"])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seqs,hq,hkv", [(64, 32, 8), (110, 16, 2), (130, 12, 2)])
def test_ragged_trees_of_up_to_two_tiles(dev, seqs, hq, hkv, d, kind, fp8):  # noqa: F811
    """Whole units (no workspace), and a table wide enough that the units' K/V tiles are shared out."""
    rng = np.random.default_rng(seqs + d)
    most = 64 if hkv == 8 else 32
    counts = rng.integers(1, most + 1, seqs)
    counts[rng.random(seqs) < 0.6] = rng.integers(1, 9)  # of one tile
    counts[5], counts[7] = most, 0
    b = Batch(dev, seqs, counts.tolist(), rng.integers(0, 300, seqs).tolist(), hq, hkv, d, kind, fp8, 16)
    want = b.want()
    out = b.run()
    b.check(out, want)
    for _ in range(4):
        assert (b.run() == out).all(), "two runs differ"
    b.tables = np.concatenate([b.tables, np.full((seqs, 4096), -1, np.int32)], 1)
    ws = b.workspace()
    out = b.run(ws)
    b.check(out, want)
    assert (b.run(ws) == out).all(), "two runs differ"
    assert binding.pa_get_device_error() == 0


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_second_tiles_that_come_and_go(dev, kind):  # noqa: F811
    """FP8 cache: long contexts beside short ones, so that the two tiles' threads are far apart; every other tree has one tile."""
    rng = np.random.default_rng(3)
    seqs = 96
    counts = [int(rng.integers(33, 65)) if s % 2 else int(rng.integers(1, 33)) for s in range(seqs)]
    context = [int(rng.integers(1500, 2000)) if s % 8 == 0 else int(rng.integers(0, 60)) for s in range(seqs)]
    b = Batch(dev, 9, counts, context, 32, 8, 128, kind, True, 32)
    want = b.want()
    out = b.run()
    b.check(out, want)
    for _ in range(8):
        assert (b.run() == out).all(), "two runs differ"
    assert binding.pa_get_device_error() == 0


@pytest.mark.parametrize("fp8", [True, False], ids=["fp8", "16"])
@pytest.mark.parametrize("hq,hkv,d", [(16, 2, 128), (12, 2, 64), (32, 8, 128)])
def test_nonfinite_nodes_in_warps_of_uneven_rows(dev, hq, hkv, d, fp8):  # noqa: F811
    """The rows of a warp see different numbers of nodes whose V is not finite, and some rows are nobody's: lanes part while those
    are added, and the warp meets again before its next read of tensor memory."""
    rng = np.random.default_rng(hq + d)
    for most in (9, 45):  # one query tile, and two
        counts = rng.integers(2, most + 1, 80)
        single.test_nonfinite_nodes_reach_only_who_sees_them(dev, counts.tolist(), rng.integers(0, 150, 80).tolist(), hq, hkv, d, "bf16", fp8)

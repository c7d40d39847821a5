"""Tree attention's form for few rows in large batches: a warp takes many sequences one after another through one ring of tiles."""
import numpy as np
import pytest

import test_gpu_tree_attention as single
from test_gpu_tree_attention import dev  # noqa: F401

from paged_kv_cache_120_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True], ids=["16", "fp8"])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 128), (32, 8, 64)])
def test_nonfinite_nodes_in_tiles_whose_place_is_used_again(dev, hq, hkv, d, kind, fp8):  # noqa: F811
    """Elements of V that are not finite are taken out of a tile in shared memory, where later tiles land after it."""
    rng = np.random.default_rng(hq + d)
    counts = rng.integers(2, 5, 500)
    context = rng.integers(0, 300, 500)
    single.test_nonfinite_nodes_reach_only_who_sees_them(dev, counts.tolist(), context.tolist(), hq, hkv, d, kind, fp8)


@pytest.mark.parametrize("fp8", [False, True], ids=["16", "fp8"])
@pytest.mark.parametrize("context", [700, 6000])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (2, 2)])
def test_idle_rows_change_no_bits(dev, hq, hkv, context, fp8):  # noqa: F811
    """A sequence's share-out goes by the sequences that have nodes: idle rows before and behind it leave its bits as they are."""
    alone = single.Batch(dev, 6, [3], [context], hq, hkv, 128, "bf16", fp8, 16)
    out = alone.run(alone.workspace())
    alone.check(out)
    for before, behind in ((1, 0), (0, 1), (1, 2)):
        b = single.Batch(dev, 6, [3], [context], hq, hkv, 128, "bf16", fp8, 16)
        idle = lambda n, value: np.full(n, value, np.int32)  # noqa: E731
        b.cu = np.concatenate([idle(before, 0), b.cu, idle(behind, b.cu[-1])])
        b.lens = np.concatenate([idle(before, 900), b.lens, idle(behind, 0)])
        b.lens = np.minimum(b.lens, b.width * 16)
        b.tables = np.concatenate([np.zeros((before, b.width), np.int32), b.tables, np.full((behind, b.width), -1, np.int32)])
        ws = binding.tree_attention_workspace(b.query, b.pool, 1 + before + behind, b.maxq)
        assert (b.run(ws) == out).all(), (before, behind)
    assert binding.pa_get_device_error() == 0

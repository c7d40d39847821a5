"""Tree attention's form for few rows in large batches: a warp takes many sequences one after another through one ring of tiles."""
import numpy as np
import pytest

import test_gpu_tree_attention as single
from test_gpu_tree_attention import dev  # noqa: F401

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

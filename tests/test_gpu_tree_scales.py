"""Tree attention with scores that a scale of zero or below makes: every form, both cache types, masks of all kinds, units whole and
shared out."""
import numpy as np
import pytest

from test_gpu_tree_attention import Batch, dev, wild  # noqa: F401

from paged_kv_cache_120_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [True, False], ids=["fp8", "16"])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.11, 0.3])
@pytest.mark.parametrize("counts,context,hq,hkv,d", [([4, 2, 4], [0, 300, 20], 4, 4, 128), ([4, 4, 1], [150, 16, 0], 8, 2, 64),
                                                     ([16, 9, 12], [0, 260, 130], 8, 2, 128), ([20, 3], [0, 400], 6, 6, 64),
                                                     ([64, 40, 7], [0, 300, 90], 16, 2, 128), ([150, 130], [0, 200], 2, 2, 64)])
def test_scales(dev, counts, context, hq, hkv, d, scale, kind, fp8):  # noqa: F811
    b = Batch(dev, 77, counts, context, hq, hkv, d, kind, fp8, 16, masks=wild)
    b.scale = scale
    want = b.want()
    b.check(b.run(), want)
    # A table so wide that units are shared out.
    b.tables = np.concatenate([b.tables, np.full((len(counts), 2048), -1, np.int32)], 1)
    b.check(b.run(b.workspace()), want)
    assert binding.pa_get_device_error() == 0

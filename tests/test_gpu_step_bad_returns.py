"""pa_build_step: block ids outside the pool in a finished row's table are
flagged when they are returned, whether or not the step hands them out again."""
import numpy as np
import pytest

from paged_kv_cache_120_gb300 import binding

from step_reference import build_step
from test_gpu_step_maps import StepCase, dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [-1, 8, 2 ** 31 - 1])
@pytest.mark.parametrize("taken", [0, 1, 2])
def test_bad_ids_of_a_finished_row(dev, bad, taken):
    """Its blocks are bad, 5: 0, 1 or both are taken by the row behind it; they stay as they are on the list."""
    tables = np.array([[bad, 5, -1], [-1, -1, -1]], np.int32)
    free = np.array([1, 2, -1, -1, -1, -1, -1, -1], np.int32)
    query = np.array([-1, 16 * taken])
    c = StepCase(dev, tables, [20, 0], query, free, 2, 40, 16)
    c.run()
    with np.errstate(over="ignore"):
        want = build_step(tables, [20, 0], query, free, 2, 40, 16)
    want["slots"][:16 * min(taken, 1)] = -1  # the last block returned, the first logical one, is the first taken
    c.check(want, error=binding.PA_DEVERR_BLOCK_ID)

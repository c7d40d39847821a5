"""pa_verify_draft, children drawn from the drafter's rows: entries of those rows that are not above 0 weigh nothing."""
import numpy as np
import pytest

import tree_reference as ref
from test_gpu_tree_ops import check_verify, dev, offsets, rows, run_verify  # noqa: F401

from paged_kv_cache_120_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("counts,fan,vocab,pad,shift", [([9] * 20, 3, 1001, 5, 3), ([12, 1, 13], 4, 32000, 0, 0), ([5] * 60, 2, 64, 0, 1)])
def test_negative_and_nan_entries(dev, counts, fan, vocab, pad, shift, kind):  # noqa: F811
    import torch
    rng = np.random.default_rng(vocab)
    kind = getattr(torch, kind)
    cu, total = offsets(counts), int(sum(counts))
    parents = np.concatenate([ref.random_parents(rng, n, fan) for n in counts]).astype(np.int32)
    target, p = rows(rng, total, vocab, kind, 3.0)
    p[rng.random(p.shape) < 0.2] = 0.0  # no weight: such a child is never accepted
    target = torch.from_numpy(p).to(kind)
    q = target.double().numpy()[:, ::-1].copy() + p
    kinds = rng.random(q.shape)
    q[kinds < 0.25] *= -1.0
    q[kinds > 0.9] = np.nan
    draft = torch.from_numpy(q).to(kind)
    q = draft.double().numpy()
    # Children: half of them entries that weigh nothing, the others likely ones.
    tokens = np.zeros(total, np.int32)
    for s in range(len(counts)):
        for i in range(cu[s], cu[s + 1]):
            a = cu[s] + max(parents[i], 0)
            none = np.flatnonzero(~(q[a] > 0))
            tokens[i] = rng.choice(none) if rng.random() < 0.5 else np.argsort(-p[a])[rng.integers(0, 3)]
    uniforms = rng.random((total, 2)).astype(np.float32)
    got = run_verify(dev, parents, tokens, cu, target, draft, uniforms, pad, shift)
    check_verify(got, parents, tokens, cu, target.double().numpy(), q, uniforms)
    assert binding.pa_get_device_error() == 0


def test_a_child_without_weight_is_refused(dev):  # noqa: F811
    """A child to which the target gives 0 and the drafter a negative entry is no accepted token; refusing it takes nothing away."""
    import torch
    target = torch.tensor([[0.0, 0.5, 0.25, 0.25]] * 2)
    for entry in (-0.5, float("nan")):
        draft = torch.tensor([[entry, 0.5, entry, 0.0]] * 2)
        for u, want in ((0.1, 2), (0.45, 2), (0.55, 3), (0.95, 3)):  # left: (0, 0, 0.25, 0.25)
            got = run_verify(dev, np.array([-1, 0]), np.array([0, 0]), np.array([0, 2]), target, draft,
                             np.array([[0.0, u], [0.5, 0.0]], np.float32))
            assert got[0].tolist() == [1] and got[2].tolist() == [want, -1], (entry, u)

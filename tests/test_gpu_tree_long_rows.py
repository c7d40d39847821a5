"""pa_verify_draft on rows so long that a warp's part of one is more than 64 tiles of 512 bytes: it keeps the sums of groups of tiles
then, and a draw walks through a group's tiles again."""
import numpy as np
import pytest

import tree_reference as ref
from test_gpu_tree_ops import check_verify, dev, offsets, run_verify  # noqa: F401

from paged_kv_cache_120_gb300 import binding

pytestmark = pytest.mark.gpu


def aimed(p, at):
    """A fp32 number whose draw from the rows p (one each) falls into entry `at`, or next to it where 24 bits do not resolve it."""
    sums = np.cumsum(np.maximum(p, 0), -1)
    i = np.arange(len(at))
    return (((sums[i, at] + np.where(at > 0, sums[i, np.maximum(at - 1, 0)], 0)) / 2) / sums[:, -1]).astype(np.float32)


@pytest.mark.parametrize("mode", ["sample", "draft"])
@pytest.mark.parametrize("seqs,live,vocab,kind,pad,shift", [
    (320, 48, 131075, "float32", 1, 3), (320, 40, 300001, "bfloat16", 0, 5), (320, 30, 262144, "float16", 0, 0),  # a CTA a sequence
    (3, 3, 700001, "float32", 2, 1), (2, 2, 1100000, "bfloat16", 0, 0)])                                          # clusters of 8
def test_groups_of_tiles(dev, seqs, live, vocab, kind, pad, shift, mode):  # noqa: F811
    """Draws that fall into the first, middle and last tiles of groups and parts, and onto the row's ends."""
    import torch
    rng = np.random.default_rng(vocab)
    kind = getattr(torch, kind)
    counts = np.zeros(seqs, int)
    counts[rng.permutation(seqs)[:live]] = 2
    cu, total = offsets(counts), 2 * live
    # Few rows, each used several times: a row's sums in 64 bits take long. Whole numbers over a power of two, so that those are exact.
    base = [torch.from_numpy(rng.integers(0, 200, vocab) * (rng.random(vocab) < 0.7) / 2.0 ** 24).to(kind) for _ in range(2)]
    target = torch.stack([base[(i // 2) % 2] for i in range(total)])
    p = target.double().numpy()
    vec = 16 // target.element_size()
    tile = 32 * vec  # entries
    places = np.concatenate([np.arange(0, vocab, 8 * tile), np.arange(0, vocab, 8 * tile) + 8 * tile - 1, np.arange(0, vocab, tile * 3) + 7,
                             [0, 1, vocab - 1, vocab - 2]])
    places = places[places < vocab]
    uniforms = np.stack([rng.random(total).astype(np.float32), aimed(p, rng.choice(places, total))], 1)
    uniforms[1, 1], uniforms[3, 1] = 0.0, 1 - 2.0 ** -24
    tokens, draft, q = rng.integers(0, vocab, total), None, None
    parents = np.tile([-1, 0], live)
    if mode == "draft":
        # Children that are refused (the drafter gives them all it has) and, at some roots, accepted ones.
        hot = torch.from_numpy(rng.integers(0, 200, vocab) / 2.0 ** 25).to(kind)
        draft = torch.stack([hot] * total)
        q = draft.double().numpy()
        tokens[1::2] = np.argsort(-(q[0] - p[0]))[:live]
        # The draw behind a refusal is from what is left.
        left = np.maximum(p - q, 0)
        uniforms[::2, 1] = aimed(left[::2], rng.choice(places, live))
        uniforms[1::4, 0] = np.float32(1 - 2.0 ** -24)
    got = run_verify(dev, parents, tokens, cu, target, draft, uniforms, pad, shift)
    check_verify(got, parents, tokens, cu, p, q, uniforms)
    assert binding.pa_get_device_error() == 0


@pytest.mark.parametrize("back", [False, True], ids=["behind", "around"])
@pytest.mark.parametrize("entry", [0, 5, 14])
@pytest.mark.parametrize("seed", range(3))
def test_draws_at_the_end_of_a_group(dev, seed, entry, back):  # noqa: F811
    """u = 1/2 and rows whose first entries, up to the end of a group of tiles, hold half of the sum but for a few steps of 2^-45: a
    sum in another order may fall on the other side of u times the whole. Sums are held to about 46 bits (2^-43 of the row's is
    allowed here), so the token is one at the border, never one far behind it. Whole numbers of 2^-40 throughout: int64 sums are exact."""
    import torch
    vocab, live, seqs = 131072, 96, 320
    rng = np.random.default_rng(seed)
    step = 2.0 ** -40
    x = np.exp(2.0 * rng.standard_normal(vocab)).astype(np.float32)
    part, group = vocab // 8, 1024  # entries: of a warp, of a group of 8 tiles
    border = 3 * part + (entry + 1) * group
    x[border:] *= np.float32(0.25 * border / (vocab - border))
    x = (np.round(np.minimum(x, 1e4).astype(np.float64) / step) * step).astype(np.float32)
    x = np.maximum(x, np.float32(step))
    x[-4:] = 0
    whole = lambda a: np.round(np.asarray(a, np.float64) / step).astype(np.int64)  # noqa: E731
    assert np.array_equal(whole(x) * step, x.astype(np.float64))
    gap = int(whole(x[:border]).sum()) - int(whole(x[border:]).sum())
    assert gap > 0
    if back:  # u times the sum moves across the border
        gap -= int(whole(x).sum()) >> 43
    for k in (-4, -3, -2):  # three entries make up for the gap, each as much of it as fp32 holds
        x[k] = np.nextafter(np.float32(gap * step), np.float32(0)) if gap * step > 2.0 ** -16 else np.float32(gap * step)
        gap -= int(whole(x[k]))
    assert 0 <= gap < 2 ** 16
    rows = np.repeat(x[None], live, 0)
    z = int(whole(x).sum())
    shift = np.linspace(-1, 1, live) * z * 2.0 ** -44
    rows[:, -1] = ((shift - shift[0] + gap) * step).astype(np.float32)  # from the border's far side to this one
    counts = np.zeros(seqs, int)
    counts[rng.permutation(seqs)[:live]] = 1
    uniforms = np.full((live, 2), 0.5, np.float32)
    got = run_verify(dev, np.full(live, -1), np.zeros(live), offsets(counts), torch.from_numpy(rows), None, uniforms)
    drawn = got[2]
    for i in range(live):
        sums = np.cumsum(whole(rows[i]))
        half, near = int(sums[-1]) // 2, int(sums[-1]) >> 43
        t = int(drawn[i])
        assert sums[t] + near > half and sums[t] - int(whole(rows[i, t])) - near <= half, (i, t, border)
    assert binding.pa_get_device_error() == 0

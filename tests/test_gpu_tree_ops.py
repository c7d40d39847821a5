"""The speculative step's maps, verification and commit against plain forms in 64 bits: every result is a whole number or a bit
copy, so everything is compared for equality."""
import numpy as np
import pytest

from paged_kv_cache_120_gb300 import binding, build

import tree_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    binding.lib()
    assert binding.pa_get_device_error() == 0
    return torch.device("cuda:0")


def gpu(a, dev, dtype=np.int32):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).to(dev)


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


# ---------------------------------------------------------------- pa_build_tree

@pytest.mark.parametrize("counts,fan,words", [
    ([1], 1, 1), ([2, 0, 3], 1, 1), ([32, 33, 31], 1, 2), ([64] * 9, 8, 2), ([1024], 1, 32), ([1000, 5, 1024], 2, 32),
    ([257, 256], 1000, 9), ([7] * 300, 3, 3), ([100, 0, 0, 17], 4, 32)])
def test_build_tree(dev, counts, fan, words):
    rng = np.random.default_rng(sum(counts))
    cu, total = offsets(counts), int(sum(counts))
    parents = np.concatenate([ref.random_parents(rng, n, fan, 0.2) if n else np.zeros(0, np.int32) for n in counts])
    lens = np.array(counts, np.int32) + rng.integers(0, 5000, len(counts)).astype(np.int32)
    spare = 3  # rows behind the last sequence
    want_m, want_p = np.full((total + spare, words), 77, np.int32), np.full(total + spare, 77, np.int32)
    for s, n in enumerate(counts):
        seen, depth = ref.closure(parents[cu[s]:cu[s + 1]])
        want_m[cu[s]:cu[s + 1]] = ref.pack(seen, words)
        want_p[cu[s]:cu[s + 1]] = lens[s] - n + depth
    masks, pos = gpu(np.full((total + spare, words), 77), dev), gpu(np.full(total + spare, 77), dev)
    args = gpu(np.concatenate([parents, np.full(spare, -1)]), dev), gpu(cu, dev), gpu(lens, dev)
    binding.pa_build_tree(*args, pos, masks)
    assert np.array_equal(masks.cpu().numpy(), want_m)
    assert np.array_equal(pos.cpu().numpy(), want_p)
    masks.fill_(77)
    binding.pa_build_tree(*args, None, masks)
    assert np.array_equal(masks.cpu().numpy(), want_m)
    assert binding.pa_get_device_error() == 0


def test_build_tree_flags(dev):
    """Bad parents count as none; inconsistent sequences are left alone."""
    masks, pos = gpu(np.full((8, 1), 77), dev), gpu(np.full(8, 77), dev)
    binding.pa_build_tree(gpu([-1, 0, 2, 9, -2, -1, 0, 1], dev), gpu([0, 5, 8], dev), gpu([5, 2], dev), pos, masks)
    assert binding.pa_get_device_error() == binding.PA_DEVERR_TREE | binding.PA_DEVERR_SEQ_LEN
    assert masks.flatten().tolist() == [1, 3, 4, 8, 16, 77, 77, 77] and pos.tolist() == [0, 1, 0, 0, 0, 77, 77, 77]
    masks, pos = gpu(np.full((40, 1), 77), dev), gpu(np.full(40, 77), dev)
    for cu in ([0, 40], [-3, 4], [0, 41], [5, 3]):  # 33 nodes and more need two words
        binding.pa_build_tree(gpu(np.full(40, -1), dev), gpu(cu, dev), gpu([100], dev), pos, masks)
        assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN
        assert (masks == 77).all() and (pos == 77).all()


# -------------------------------------------------------------- pa_verify_draft

def rows(rng, total, vocab, kind, peak):
    """Rows of probabilities as the element type holds them (a torch CPU tensor), and as float64."""
    import torch
    z = rng.standard_normal((total, vocab)) * peak
    p = np.exp(z - z.max(-1, keepdims=True))
    t = torch.from_numpy(p / p.sum(-1, keepdims=True)).to(kind)
    return t, t.double().numpy()


def run_verify(dev, parents, tokens, cu, target, draft, uniforms, pad=0, shift=0):
    """The kernel's (count, path, tokens); rows `pad` entries further apart than they are long, `shift` entries off alignment."""
    import torch
    total, vocab = target.shape

    def place(t):
        if t is None:
            return None
        wide = torch.full((total * (vocab + pad) + shift + 8,), float("nan"), dtype=t.dtype, device=dev)
        view = wide[shift:shift + total * (vocab + pad)].view(total, vocab + pad)[:, :vocab]
        view.copy_(t)
        return view
    out = lambda n: torch.full((n,), 77, dtype=torch.int32, device=dev)  # noqa: E731
    count, path, new = out(len(cu) - 1), out(total), out(total)
    u = None if uniforms is None else gpu(uniforms, dev, np.float32)
    binding.pa_verify_draft(count, path, new, gpu(tokens, dev), gpu(parents, dev), gpu(cu, dev), place(target), place(draft), u)
    return count.cpu().numpy(), path.cpu().numpy(), new.cpu().numpy()


def check_verify(got, parents, tokens, cu, target, draft, uniforms):
    count, path, new = got
    for s in range(len(cu) - 1):
        a, b = cu[s], cu[s + 1]
        if a == b:
            assert count[s] == 0
            continue
        want_path, want_new = ref.verify(parents[a:b], tokens[a:b], target[a:b], None if draft is None else draft[a:b],
                                         None if uniforms is None else uniforms[a:b].astype(np.float64))
        n = len(want_path)
        assert count[s] == n and path[a:b].tolist() == want_path + [-1] * (b - a - n), s
        assert new[a:b].tolist() == want_new + [-1] * (b - a - n), s


CASES = [  # counts, fan, vocab, peak, pad, shift
    ([1], 1, 1, 1.0, 0, 0), ([5, 0, 1, 3], 2, 7, 1.0, 0, 0), ([6] * 40, 1, 1000, 2.0, 0, 0), ([9] * 20, 3, 1001, 2.0, 5, 3),
    ([24, 1, 13], 3, 32000, 4.0, 0, 0), ([8, 8], 2, 100003, 4.0, 0, 1), ([16], 4, 131072, 4.0, 0, 0), ([7] * 400, 2, 130, 1.0, 2, 0),
    ([33, 40], 8, 4099, 3.0, 1, 2)]


@pytest.mark.parametrize("mode", ["greedy", "sample", "draft"])
@pytest.mark.parametrize("kind", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_verify(dev, case, kind, mode):
    import torch
    counts, fan, vocab, peak, pad, shift = CASES[case]
    rng = np.random.default_rng(case)
    kind = getattr(torch, kind)
    cu, total = offsets(counts), int(sum(counts))
    parents = np.concatenate([ref.random_parents(rng, n, fan, 0.1) if n else np.zeros(0, np.int32) for n in counts]).astype(np.int32)
    target, p = rows(rng, total, vocab, kind, peak)
    # A drafter near the target, so that nodes deep down are reached.
    near = torch.from_numpy(p * np.exp(0.7 * rng.standard_normal(p.shape)))
    draft = (near / near.sum(-1, keepdim=True)).to(kind)
    q = draft.double().numpy()
    tokens = np.zeros(total, np.int32)
    for s in range(len(counts)):
        for i in range(cu[s], cu[s + 1]):
            a = cu[s] + max(parents[i], 0)
            if mode == "draft":
                tokens[i] = min(vocab - 1, np.searchsorted(np.cumsum(q[a]), rng.random() * q[a].sum(), side="right"))
            else:
                best = np.argsort(-q[a])[:fan + 1]
                tokens[i] = best[rng.integers(0, len(best))]
    tokens[rng.random(total) < 0.05] = vocab + 3  # no token of the vocabulary
    tokens[rng.random(total) < 0.02] = -1
    uniforms = None if mode == "greedy" else rng.random((total, 2)).astype(np.float32)
    use = draft if mode == "draft" else None
    got = run_verify(dev, parents, tokens, cu, target, use, uniforms, pad, shift)
    check_verify(got, parents, tokens, cu, p, q if mode == "draft" else None, uniforms)
    again = run_verify(dev, parents, tokens, cu, target, use, uniforms, pad, shift)
    assert all(np.array_equal(a, b) for a, b in zip(got, again))
    assert binding.pa_get_device_error() == 0


@pytest.mark.parametrize("pads", [(0, 3), (1, 0), (4, 4)])
def test_verify_rows_that_lie_differently(dev, pads):
    """Target and drafter rows with other strides, so that their alignments differ."""
    import torch
    rng = np.random.default_rng(3)
    counts, vocab = [4] * 30, 517
    cu, total = offsets(counts), 120
    parents = np.concatenate([ref.random_parents(rng, 4, 2) for _ in counts])
    (target, p), (draft, q) = rows(rng, total, vocab, torch.float32, 2.0), rows(rng, total, vocab, torch.float32, 2.0)
    tokens = np.array([rng.choice(vocab, p=q[cu[i // 4] + max(parents[i], 0)] / q[cu[i // 4] + max(parents[i], 0)].sum())
                       for i in range(total)])
    u = rng.random((total, 2)).astype(np.float32)
    wide = [torch.zeros(total, vocab + pad, device=dev)[:, :vocab] for pad in pads]
    wide[0].copy_(target)
    wide[1].copy_(draft)
    out = lambda n: torch.zeros(n, dtype=torch.int32, device=dev)  # noqa: E731
    count, path, new = out(30), out(total), out(total)
    binding.pa_verify_draft(count, path, new, gpu(tokens, dev), gpu(parents, dev), gpu(cu, dev), wide[0], wide[1],
                            gpu(u, dev, np.float32))
    check_verify((count.cpu().numpy(), path.cpu().numpy(), new.cpu().numpy()), parents, tokens, cu, p, q, u)


def test_verify_borders(dev):
    """Rows where a rule decides: equal rows (every child accepted), a drafter that covers the target (nothing left: the
    target's own row), one-hot rows, ties, zeros in front and behind, u = 0 and the largest u below 1, infinities in logits."""
    import torch
    vocab = 300
    one = np.float32(1 - 2 ** -24)
    flat = np.full(vocab, 1 / 512, np.float32)
    hot = np.zeros(vocab, np.float32)
    hot[123] = 1
    middle = np.zeros(vocab, np.float32)
    middle[100:103] = [0.5, 0.25, 0.25]
    runs = [  # target row, drafter row, tokens of two children, uniforms of root and children
        (flat, flat, (5, 6), (0.5, 0.5, 0.5)), (flat, 2 * flat, (5, 6), (0.3, 0.75, 0.9)), (hot, flat, (7, 123), (0.0, 0.9, 0.9)),
        (hot, flat, (7, 8), (one, one, one)), (middle, hot, (123, 123), (0.0, 0.0, 0.0)), (middle, hot, (123, 123), (one, 0.2, 0.2)),
        (middle, middle, (100, 102), (0.5, one, one)), (middle, flat, (0, 299), (0.75, 0.0, 0.0)),
        (middle, flat, (299, 0), (0.4999999, 0.5, 0.5))]
    total = 3 * len(runs)
    parents = np.array([-1, 0, 0] * len(runs))
    cu = np.arange(0, total + 1, 3)
    tokens = np.concatenate([[0, *t] for _, _, t, _ in runs])
    target = np.stack([r[0] for r in runs for _ in range(3)])
    draft = np.stack([r[1] for r in runs for _ in range(3)])
    u = np.array([[[r[3][0], r[3][0]], [r[3][1], r[3][1]], [r[3][2], r[3][2]]] for r in runs], np.float32).reshape(-1, 2)
    for use in (draft, None):
        got = run_verify(dev, parents, tokens, cu, torch.from_numpy(target), None if use is None else torch.from_numpy(use), u)
        check_verify(got, parents, tokens, cu, target.astype(np.float64), None if use is None else use.astype(np.float64), u)
    assert binding.pa_get_device_error() == 0
    logits = np.stack([np.full(vocab, -np.inf), flat, np.where(np.arange(vocab) == 40, np.inf, -1), np.full(vocab, np.nan),
                       np.where(np.arange(vocab) < 200, np.nan, -5.0), np.full(vocab, -0.0), -flat]).astype(np.float32)
    logits[5, 77] = 0.0  # equals -0
    n = len(logits)
    got = run_verify(dev, np.full(n, -1), np.zeros(n), np.arange(n + 1), torch.from_numpy(logits), None, None)
    assert got[2].tolist() == [0, 0, 40, 0, 200, 0, 0] and got[0].tolist() == [1] * n
    assert binding.pa_get_device_error() == 0


def test_verify_flags(dev):
    """Rows without a positive finite sum give token 0 and a flag; entries that are negative or NaN weigh nothing."""
    import torch
    vocab = 50
    target = torch.zeros(4, vocab)
    target[1] = float("nan")
    target[1, 30] = 0.5
    target[2, 3] = float("inf")
    target[3] = -1.0
    u = np.full((4, 2), 0.5, np.float32)
    got = run_verify(dev, np.full(4, -1), np.zeros(4), np.arange(5), target, None, u)
    assert binding.pa_get_device_error() == binding.PA_DEVERR_TREE
    assert got[2].tolist() == [0, 30, 0, 0] and got[0].tolist() == [1] * 4
    got = run_verify(dev, np.array([-1, 5, 0, -1]), np.zeros(4), np.array([0, 4]), target[[1, 1, 1, 1]], None, u)
    assert binding.pa_get_device_error() == binding.PA_DEVERR_TREE and got[2].tolist() == [30, -1, -1, -1]
    for cu in ([0, 5], [-1, 3], [3, 1]):
        got = run_verify(dev, np.full(4, -1), np.zeros(4), np.array(cu), target, None, u)
        assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN and got[0].tolist() == [0] and (got[2] == 77).all()


def test_verify_many_sequences_keep_the_law(dev):
    """4096 sequences over one row, two children each drawn from another one: the first new token's counts are within 5 standard
    deviations of the target's."""
    import torch
    rng = np.random.default_rng(11)
    p, q = rng.dirichlet(np.ones(7)), rng.dirichlet(np.ones(7))
    S = 4096
    parents = np.tile([-1, 0, 0], S)
    tokens = rng.choice(7, 3 * S, p=q)
    target, draft = torch.from_numpy(np.tile(p, (3 * S, 1))).float(), torch.from_numpy(np.tile(q, (3 * S, 1))).float()
    u = rng.random((3 * S, 2)).astype(np.float32)
    cu = np.arange(0, 3 * S + 1, 3)
    got = run_verify(dev, parents, tokens, cu, target, draft, u)
    check_verify(got, parents, tokens, cu, target.double().numpy(), draft.double().numpy(), u)
    counts = np.bincount(got[2][::3], minlength=7)
    assert np.all(np.abs(counts - S * p) <= 5 * np.sqrt(S * p * (1 - p)))


# -------------------------------------------------------------- pa_commit_draft

def make_commit(rng, counts, kept, context, block, width, blocks):
    """Tables, lengths and ascending paths."""
    lens = np.array([c + n for c, n in zip(context, counts)], np.int32)
    held = -(-lens // block)
    perm = rng.permutation(blocks)
    tables, at = np.full((len(counts), width), -1, np.int32), 0
    for s, h in enumerate(held):
        tables[s, :h] = perm[at:at + h]
        at += h
    path = np.full(int(sum(counts)), -1, np.int32)
    cu = offsets(counts)
    for s, (n, k) in enumerate(zip(counts, kept)):
        path[cu[s]:cu[s] + k] = np.sort(rng.permutation(n)[:k])
    return tables, lens, path, cu, perm[at:]


@pytest.mark.parametrize("code", ["f16", "bf16", "fp8"])
@pytest.mark.parametrize("counts,kept,context,block,hkv,d,layers", [
    ([8, 0, 5], [3, 0, 5], [0, 7, 30], 16, 2, 64, 1), ([64, 64], [40, 1], [100, 15], 16, 8, 128, 3), ([300], [300], [1], 32, 1, 64, 2),
    ([1000, 3], [17, 0], [9, 64], 48, 3, 32, 5), ([16] * 70, [5, 9] * 35, list(range(70)), 16, 1, 16, 2), ([33], [20], [0], 16, 40, 128, 40)])
def test_commit(dev, code, counts, kept, context, block, hkv, d, layers):
    import torch
    rng = np.random.default_rng(len(counts) + d)
    width = max(-(-(c + n) // block) for c, n in zip(context, counts)) + 2
    used = sum(-(-(c + n) // block) for c, n in zip(context, counts))
    blocks = used + 9
    tables, lens, path, cu, free = make_commit(rng, counts, kept, context, block, width, blocks)
    kind = np.uint8 if code == "fp8" else np.int16
    td = {"f16": torch.float16, "bf16": torch.bfloat16, "fp8": torch.uint8}[code]
    shape = (2, blocks, block, hkv, d)
    host = [rng.integers(0, 255, shape).astype(kind) for _ in range(layers)]
    for in_place in (False, True):
        pools = [torch.from_numpy(h.copy()).to(dev).view(td) for h in host]
        lens_d, cu_d = gpu(lens, dev), gpu(cu, dev)
        stack = np.full(blocks, -7, np.int32)
        stack[:len(free)] = free
        free_d, n_d = gpu(stack, dev), gpu([len(free)], dev)
        out, n_out = (lens_d, n_d) if in_place else (torch.empty_like(lens_d), torch.empty_like(n_d))
        binding.pa_commit_draft(pools, gpu(tables, dev), cu_d, lens_d, gpu(kept, dev), gpu(path, dev), out, free_d, n_d, n_out)
        want = [h.copy() for h in host]
        after, back = ref.commit(want, tables, cu, lens.tolist(), kept, path, free.tolist(), block)
        for pool, w in zip(pools, want):
            assert np.array_equal(pool.cpu().view(torch.uint8 if code == "fp8" else torch.int16).numpy(), w)
        assert out.tolist() == after and n_out.item() == len(back)
        assert free_d[:len(back)].tolist() == back and (free_d[len(back):] == -7).all()
        # Without a free list nothing is returned.
        pools = [torch.from_numpy(h.copy()).to(dev).view(td) for h in host]
        out = torch.empty_like(lens_d)
        binding.pa_commit_draft(pools, gpu(tables, dev), cu_d, gpu(lens, dev), gpu(kept, dev), gpu(path, dev), out)
        assert out.tolist() == after
        for pool, w in zip(pools, want):
            assert np.array_equal(pool.cpu().view(torch.uint8 if code == "fp8" else torch.int16).numpy(), w)
    assert binding.pa_get_device_error() == 0


def test_commit_bad_sequences_stay(dev):
    """Counts, paths and lengths that are inconsistent leave their sequence as it was; the others are served."""
    import torch
    rng = np.random.default_rng(1)
    block, blocks, counts = 16, 40, [6] * 6
    tables, lens, path, cu, free = make_commit(rng, counts, [3] * 6, [20] * 6, block, 3, blocks)
    kept = [3, 7, -1, 3, 3, 3]
    path[cu[3]:cu[3] + 3] = [0, 4, 4]
    path[cu[4]:cu[4] + 3] = [0, 2, 6]
    path[cu[5]:cu[5] + 3] = [0, 2, 5]
    host = rng.integers(0, 255, (2, blocks, block, 1, 16)).astype(np.int16)
    pool = torch.from_numpy(host.copy()).to(dev).view(torch.float16)
    stack = np.concatenate([free, np.full(blocks - len(free), -7)])
    free_d, n_d, lens_d = gpu(stack, dev), gpu([len(free)], dev), gpu(lens, dev)
    binding.pa_commit_draft([pool], gpu(tables, dev), gpu(cu, dev), lens_d, gpu(kept, dev), gpu(path, dev), lens_d, free_d, n_d, n_d)
    assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN | binding.PA_DEVERR_TREE
    good = [s for s in (0, 5)]
    want, sub = host.copy(), [kept[s] if s in good else 0 for s in range(6)]
    cut = [cu[s + 1] - cu[s] if s in good else 0 for s in range(6)]
    assert lens_d.tolist() == [23 if s in good else 26 for s in range(6)]
    for s in good:
        w = ref.commit([want], tables[s:s + 1], [0, 6], [26], [sub[s]], path[cu[s]:cu[s + 1]], [], block)
        assert w[0] == [23] and cut[s] == 6
    assert np.array_equal(pool.cpu().view(torch.int16).numpy(), want)
    assert n_d.item() == len(free)  # 26 and 23 tokens hold two blocks each


def test_commit_bad_blocks_and_counts(dev):
    """A block id outside the pool: its token stays, the others move. A free list that would overflow keeps what fits."""
    import torch
    block, blocks = 16, 6
    host = np.arange(2 * blocks * block * 8, dtype=np.int16).reshape(2, blocks, block, 1, 8)
    tables = np.array([[0, 1, 99, 2]], np.int32)
    path = np.zeros(40, np.int32)
    path[:4] = [0, 3, 30, 39]
    pool = torch.from_numpy(host.copy()).to(dev).view(torch.bfloat16)
    lens_d, n_d, free_d = gpu([50], dev), gpu([5], dev), gpu([3, 4, 5, 3, 4, -7], dev)
    binding.pa_commit_draft([pool], gpu(tables, dev), gpu([0, 40], dev), lens_d, gpu([4], dev), gpu(path, dev), lens_d, free_d, n_d, n_d)
    assert binding.pa_get_device_error() == binding.PA_DEVERR_BLOCK_ID
    want = host.reshape(2, -1, 8).copy()
    flat = want.copy()
    flat[:, 11] = want[:, 13]           # node 3 (position 13) to 11
    flat[:, 13] = want[:, 2 * 16 + 1]   # node 39 (position 49) to 13; node 30 (position 40) lies in block 99
    assert np.array_equal(pool.cpu().view(torch.int16).numpy().reshape(2, -1, 8), flat)
    assert lens_d.item() == 14 and n_d.item() == 6 and free_d.tolist() == [3, 4, 5, 3, 4, 2]
    lens_d, n_d = gpu([50], dev), gpu([7], dev)
    binding.pa_commit_draft([pool], gpu(tables, dev), gpu([0, 40], dev), lens_d, gpu([40], dev), gpu(np.arange(40), dev), lens_d, free_d,
                            n_d, n_d)
    assert binding.pa_get_device_error() == binding.PA_DEVERR_BLOCK_ID and n_d.item() == 6 and lens_d.item() == 50


def test_binding_refuses(dev):
    """Tensors of another type, shape or device than the call documents."""
    import torch
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    f = lambda *s: torch.zeros(*s, device=dev)  # noqa: E731
    E = binding.PAError
    with pytest.raises(E):
        binding.pa_build_tree(i(4).long(), i(2), i(1), i(4), i(4, 1))
    with pytest.raises(E):
        binding.pa_build_tree(i(4), i(3), i(1), i(4), i(4, 1))
    with pytest.raises(E):
        binding.pa_build_tree(i(4), i(2), i(1), i(4), i(4))
    with pytest.raises(E):
        binding.pa_verify_draft(i(1), i(4), i(4), i(4), i(4), i(2), f(4, 9), f(4, 8), f(4, 2))
    with pytest.raises(E):
        binding.pa_verify_draft(i(1), i(4), i(4), i(4), i(4), i(2), f(4, 9), f(4, 9).half(), f(4, 2))
    with pytest.raises(E):
        binding.pa_verify_draft(i(1), i(4), i(4), i(4), i(4), i(2), f(9, 4).t(), None, f(4, 2))
    with pytest.raises(E):
        binding.pa_verify_draft(i(1), i(4), i(4), i(4), i(4), i(2), f(4, 9), f(4, 9))
    with pytest.raises(E):
        binding.pa_verify_draft(i(1), i(4), i(4), i(4).cpu(), i(4), i(2), f(4, 9))
    pool = torch.zeros(2, 4, 16, 1, 8, dtype=torch.float16, device=dev)
    with pytest.raises(E):
        binding.pa_commit_draft([pool, pool.bfloat16()], i(1, 2), i(2), i(1), i(1), i(4), i(1))
    with pytest.raises(E):
        binding.pa_commit_draft([pool], i(1, 2), i(2), i(1), i(1), i(4), i(1), i(3), i(1), i(1))
    with pytest.raises(E):
        binding.pa_commit_draft([pool], i(1, 2), i(2), i(1), i(1), i(4), i(1), i(4))

"""pa_tree_attention and pa_tree_attention_fp8 against attention under masks in 64 bits.

Bounds, per element of the output o of weights w over values v: half a step of the output's type, |o| e_out / 2; each weight is
rounded once (relative e_p / 2, e_p of the type the weights are multiplied in: fp16 over an FP8 cache) and the sum that divides
them holds the same rounded weights, which moves o by at most e_p / 2 (sum w |v| + |o|); weights below the least normal fp16 are
off by 2^-25 of the largest instead, 2^-25 L max |v| for L tokens; fp32 scores of D products of magnitude |q||k| and the exponential
leave the weights off by less than 2^-16 relative, 2^-16 (sum w |v| + |o|).
"""
import numpy as np
import pytest

from paged_kv_cache_120_gb300 import binding, build, workloads

import tree_reference as ref

pytestmark = pytest.mark.gpu

E_OUT = {"f16": 2.0 ** -10, "bf16": 2.0 ** -7}
KS, VS = 0.0125, 0.01


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    binding.lib()
    assert binding.pa_get_device_error() == 0
    return torch.device("cuda:0")


def gpu(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)


class Batch:
    """Trees over a pool whose unused slots hold NaN; tables of blocks in random places."""

    def __init__(self, dev, seed, counts, context, hq, hkv, d, kind, fp8, block, fan=4, words=None, masks=None, spare=2):
        import torch
        self.rng = rng = np.random.default_rng(seed)
        self.dev, self.hq, self.hkv, self.d, self.kind, self.fp8, self.block = dev, hq, hkv, d, kind, fp8, block
        self.counts, self.context = list(counts), list(context)
        self.lens = np.array([c + n for c, n in zip(context, counts)], np.int32)
        self.cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.total = int(self.cu[-1])
        self.maxq = max(1, max(counts))
        self.words = words or -(-self.maxq // 32)
        held = -(-self.lens // block)
        self.width = max(1, int(held.max())) + 1
        self.blocks = int(held.sum()) + 2
        perm = rng.permutation(self.blocks)
        self.tables, at = np.full((len(counts), self.width), -1, np.int32), 0
        for s, h in enumerate(held):
            self.tables[s, :h] = perm[at:at + h]
            at += h
        td = {"f16": torch.float16, "bf16": torch.bfloat16}[kind]
        g = torch.Generator(device=dev).manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
        self.query = normal(self.total + spare, hq, d).to(td)  # rows behind the last sequence
        pool = normal(2, self.blocks, block, hkv, d)
        if fp8:
            pool[0] /= KS
            pool[1] /= VS
            self.pool = pool.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            self.pool = pool.to(td)
        used = torch.zeros(self.blocks * block, dtype=torch.bool, device=dev)
        self.slots = [np.array([self.tables[s, t // block] * block + t % block for t in range(L)], np.int64)
                      for s, L in enumerate(self.lens)]
        for at in self.slots:
            used[torch.from_numpy(at).to(dev)] = True
        self.flat = self.pool.view(2, -1, hkv, d)
        self.flat[:, ~used] = 0x7F if fp8 else float("nan")
        self.seen = []
        for s, n in enumerate(counts):
            if masks is None:
                seen, _ = ref.closure(ref.random_parents(rng, n, fan, 0.1)) if n else (np.zeros((0, 0), bool), None)
            else:
                seen = masks(rng, n)
            self.seen.append(seen)
        bits = np.concatenate([ref.pack(m, self.words) for m in self.seen if len(m)] + [np.zeros((spare, self.words), np.int32)])
        # Bits behind a sequence's nodes count for nothing: some are set.
        at = 0
        for m in self.seen:
            n = len(m)
            for w in range(self.words):
                extra = 0 if 32 * (w + 1) <= n else (0xFFFFFFFF << max(0, n - 32 * w)) & 0xFFFFFFFF
                bits[at:at + n, w] |= np.uint32(extra).view(np.int32) if rng.random() < 0.7 else 0
            at += n
        self.masks = bits
        self.scale = d ** -0.5

    def values(self, s):
        import torch
        at = torch.from_numpy(self.slots[s]).to(self.dev)
        rows = self.flat[:, at]
        if self.fp8:
            rows = rows.view(torch.float8_e4m3fn).float()
            rows = torch.stack([rows[0] * KS, rows[1] * VS])
        return rows.double().cpu().numpy()

    def seen_of(self, s):
        return np.concatenate([np.ones((self.counts[s], self.context[s]), bool), self.seen[s]], 1)

    def want(self):
        """(out, bound) in 64 bits."""
        out, bound = np.zeros((self.total, self.hq, self.d)), np.zeros((self.total, self.hq, self.d))
        q = self.query.double().cpu().numpy()
        ep = E_OUT["f16" if self.fp8 else self.kind]
        for s, n in enumerate(self.counts):
            if n == 0:
                continue
            a, b = self.cu[s], self.cu[s + 1]
            k, v = self.values(s)
            o, mean = ref.attend(q[a:b], k, v, self.seen_of(s), self.scale)
            out[a:b] = o
            top = np.abs(np.where(np.isfinite(v), v, 0)).max()
            tiny = 2.0 ** -25 * len(k) * top if ep == E_OUT["f16"] else 0.0
            bound[a:b] = E_OUT[self.kind] / 2 * np.abs(o) + (ep / 2 + 2.0 ** -16) * (mean + np.abs(o)) + tiny + 2.0 ** -25
        return out, bound

    def workspace(self):
        return binding.tree_attention_workspace(self.query, self.pool, len(self.counts), self.maxq)

    def run(self, workspace=None, maxq=None, flags=0, out=None):
        import torch
        if out is None:
            out = torch.full_like(self.query, 55.0)
        args = (out, self.query, self.pool, gpu(self.tables, self.dev), gpu(self.cu, self.dev), gpu(self.lens, self.dev),
                gpu(self.masks, self.dev), self.scale, maxq or self.maxq)
        if self.fp8:
            binding.pa_tree_attention_fp8(*args, KS, VS, workspace, flags)
        else:
            binding.pa_tree_attention(*args, workspace, flags)
        return out

    def check(self, out, want=None):
        o, bound = want or self.want()
        got = out.double().cpu().numpy()
        assert (got[self.total:] == 55.0).all(), "rows behind the last sequence were written"
        got = got[:self.total]
        assert np.isfinite(got).all()
        worst = np.max(np.abs(got - o) / bound) if self.total else 0.0
        assert worst <= 1.0, f"error {worst:.2f} of the bound"


SHAPES = [  # counts, contexts, hq, hkv, d, block
    ([4, 1, 0, 3], [30, 0, 5, 17], 4, 4, 128, 16),                  # few rows, 8 columns
    ([4, 2, 4], [200, 31, 0], 8, 2, 64, 16),                       # few rows, 16 columns
    ([5] * 3 + [0, 2], [1000, 3, 128, 9, 256], 16, 8, 128, 32),
    ([8, 7, 1], [100, 127, 128], 40, 8, 128, 16),                  # one tile of 40 rows
    ([25, 1, 0, 13], [250, 1500, 7, 0], 6, 6, 64, 32),
    ([64, 64, 33], [64, 0, 700], 4, 1, 128, 16),                   # two tiles
    ([128, 100], [29, 300], 2, 2, 64, 48),
    ([300, 17, 129], [111, 40, 0], 16, 2, 128, 16),                # many tiles of 16 nodes
    ([700], [2000], 2, 1, 64, 16),
    ([1024], [5], 1, 1, 128, 64),
    ([33], [9000], 8, 2, 128, 16),                                 # shared out over the SMs
    ([12] * 40, [3 * i for i in range(40)], 12, 2, 128, 16),
    ([3] * 60, list(range(1, 61)), 16, 1, 128, 16),
    ([2, 6], [50, 20], 32, 1, 64, 16),                             # a group of 32 heads
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_tree_attention(dev, shape, kind, fp8):
    counts, context, hq, hkv, d, block = SHAPES[shape]
    b = Batch(dev, shape, counts, context, hq, hkv, d, kind, fp8, block)
    want = b.want()
    ws = b.workspace()
    for workspace in {id(ws): ws, id(None): None}.values():
        out = b.run(workspace)
        b.check(out, want)
        assert (b.run(workspace) == out).all(), "two runs differ"
    b.check(b.run(ws, flags=binding.PA_DECODE_SHARED_BLOCKS), want)
    assert binding.pa_get_device_error() == 0


@pytest.mark.parametrize("maxq", [7, 16, 90, 1000])
def test_looser_bounds(dev, maxq):
    """A bound above the most nodes chooses other kernels and the same results within the bounds; more mask words than needed."""
    b = Batch(dev, 3, [7, 2, 5], [130, 0, 45], 8, 4, 128, "bf16", False, 16, words=32)
    b.maxq = maxq
    want = b.want()
    b.check(b.run(b.workspace()), want)
    b.check(b.run(None), want)


def wild(rng, n):
    """Masks that are no tree's: any bits, some rows without any."""
    seen = rng.random((n, n)) < 0.3
    seen[rng.random(n) < 0.3] = False
    return seen


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("counts,context,hq,hkv,d", [([4, 3, 4], [0, 0, 20], 4, 4, 128), ([4, 4, 2], [0, 16, 0], 8, 2, 64),
                                                     ([40, 9, 64], [0, 0, 100], 8, 8, 64), ([60, 200], [0, 0], 8, 2, 128)])
def test_any_masks_and_empty_rows(dev, counts, context, hq, hkv, d, fp8):
    """Without a context a row whose mask is empty is zeros, exactly."""
    b = Batch(dev, 17, counts, context, hq, hkv, d, "f16", fp8, 16, masks=wild)
    want = b.want()
    assert any(not b.seen_of(s).any(1).all() for s in range(len(counts)))
    for ws in (b.workspace(), None):
        out = b.run(ws)
        b.check(out, want)
        for s in range(len(counts)):
            empty = ~b.seen_of(s).any(1)
            assert (out[b.cu[s]:b.cu[s + 1]].cpu().numpy()[empty] == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("counts,context,hq,hkv,d", [([4, 3], [37, 14], 4, 4, 128), ([4, 4], [37, 0], 8, 2, 64), ([16, 9], [300, 121], 8, 4, 128),
                                                     ([70, 64], [90, 64], 8, 2, 128), ([200], [50], 4, 4, 64)])
def test_nonfinite_nodes_reach_only_who_sees_them(dev, counts, context, hq, hkv, d, kind, fp8):
    """Half of the nodes hold NaN in K, or NaN and infinities in V. Rows that do not see them are as exact as ever; rows that see
    such a V have it in those dimensions; rows that see a NaN score are NaN."""
    import torch
    b = Batch(dev, 23, counts, context, hq, hkv, d, kind, fp8, 16, fan=3)
    bad_k, bad_v = [], []
    for s, n in enumerate(counts):
        leaf = [i for i in range(n) if b.seen[s][:, i].sum() == 1]
        some = b.rng.permutation(leaf)[:max(1, len(leaf) // 2)]
        bad_k.append(set(some[::2].tolist()))
        bad_v.append(set(some[1::2].tolist()))
    clean = b.want()  # of the finite values
    nan, inf = (0x7F, None) if fp8 else (float("nan"), float("inf"))
    dims = [3, d - 1]
    for s in range(len(counts)):
        for i in bad_k[s]:
            b.flat[0, b.slots[s][context[s] + i]] = nan
        for i in bad_v[s]:
            at = b.slots[s][context[s] + i]
            b.flat[1, at, :, dims[0]] = nan
            b.flat[1, at, :, dims[1]] = nan if inf is None else inf
    for ws in (b.workspace(), None):
        out = b.run(ws).double().cpu().numpy()[:b.total]
        for s, n in enumerate(counts):
            for i in range(n):
                row, o, bound = out[b.cu[s] + i], clean[0][b.cu[s] + i], clean[1][b.cu[s] + i]
                sees = set(np.flatnonzero(b.seen[s][i]).tolist())
                if sees & bad_k[s]:
                    assert np.isnan(row).all(), (s, i)
                elif sees & bad_v[s]:
                    rest = np.setdiff1d(np.arange(d), dims)
                    assert np.all(np.abs(row[:, rest] - o[:, rest]) <= bound[:, rest]), (s, i)
                    assert np.isnan(row[:, dims[0]]).all()
                    assert np.isnan(row[:, dims[1]]).all() if fp8 else (row[:, dims[1]] == np.inf).all()
                else:
                    assert np.all(np.abs(row - o) <= bound), (s, i)
    assert binding.pa_get_device_error() == 0


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_scale_zero_and_negative(dev, scale):
    for counts, context, hq, hkv in (([4, 3], [5, 0], 4, 4), ([64, 30], [0, 100], 4, 1), ([20], [200], 2, 2)):
        b = Batch(dev, 5, counts, context, hq, hkv, 64, "bf16", False, 16)
        b.scale = scale
        want = b.want()
        for ws in (b.workspace(), None):
            b.check(b.run(ws), want)


def test_where_blocks_lie_does_not_matter(dev):
    """The same tokens in other blocks: the same bits."""
    import torch
    for counts, context, hq, hkv in (([4, 3], [500, 40], 4, 4), ([33, 9], [300, 1000], 8, 2)):
        b = Batch(dev, 31, counts, context, hq, hkv, 128, "bf16", False, 16)
        ws = b.workspace()
        out = b.run(ws)
        perm = b.rng.permutation(b.blocks)
        pool = torch.empty_like(b.pool)
        pool[:, torch.from_numpy(perm).to(dev)] = b.pool
        b.pool = pool
        b.tables = np.where(b.tables >= 0, perm[np.maximum(b.tables, 0)], -1)
        assert (b.run(ws) == out).all()


@pytest.mark.parametrize("counts,hq,hkv", [([4, 4, 4], 4, 4), ([30, 30, 30], 4, 4), ([64, 64, 64], 8, 2)])
def test_bad_rows_are_left_and_flagged(dev, counts, hq, hkv):
    """A length below its nodes or above the table, offsets past the rows: not written, flagged; the others as ever. A block id
    outside the pool reads as zeros."""
    b = Batch(dev, 8, counts, [40, 50, 60], hq, hkv, 64, "f16", False, 16)
    want = b.want()
    keep = b.lens.copy()
    for bad in (counts[1] - 1, b.width * 16 + 1, -1):
        b.lens = keep.copy()
        b.lens[1] = bad
        for ws in (b.workspace(), None):
            out = b.run(ws).double().cpu().numpy()
            assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN
            a, z = b.cu[1], b.cu[2]
            assert (out[a:z] == 55.0).all()
            for r in (slice(0, a), slice(z, b.total)):
                assert np.all(np.abs(out[r] - want[0][r]) <= want[1][r])
    b.lens = keep
    b.tables[1, 1] = b.blocks + 5
    b.slots[1] = np.array([t if not 16 <= i < 32 else 0 for i, t in enumerate(b.slots[1])])
    values = b.values

    def zeroed(s):
        kv = values(s)
        if s == 1:
            kv[:, 16:32] = 0
        return kv
    b.values = zeroed
    want = b.want()
    for ws in (b.workspace(), None):
        b.check(b.run(ws), want)
        assert binding.pa_get_device_error() == binding.PA_DEVERR_BLOCK_ID


@pytest.mark.parametrize("counts,context,hq,hkv", [([4, 4], [300, 20], 4, 4), ([33, 20], [700, 20], 8, 2)])
def test_captured_and_on_another_stream(dev, counts, context, hq, hkv):
    """A captured call replays on new lengths and masks; two captured calls share a workspace on one stream."""
    import torch
    b = Batch(dev, 12, counts, context, hq, hkv, 128, "bf16", False, 16)
    ws = b.workspace()
    b.run(ws)  # attributes and tensor maps
    args = [gpu(b.tables, dev), gpu(b.cu, dev), gpu(b.lens, dev), gpu(b.masks, dev)]
    outs = [torch.full_like(b.query, 55.0) for _ in range(2)]
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream, capture_error_mode="relaxed"):
            for out in outs:
                binding.pa_tree_attention(out, b.query, b.pool, *args, b.scale, b.maxq, ws)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            b.check(out)
            out.fill_(55.0)
        # Other trees, and one sequence's context cut short: the graph reads them anew.
        b.seen = [ref.closure(ref.random_parents(b.rng, n, 2))[0] for n in counts]
        b.masks = np.concatenate([ref.pack(m, b.words) for m in b.seen] + [np.zeros((2, b.words), np.int32)])
        b.context[0] = context[0] - 37
        b.lens[0] = b.context[0] + counts[0]
        b.slots[0] = b.slots[0][:b.lens[0]]
        args[2].copy_(gpu(b.lens, dev))
        args[3].copy_(gpu(b.masks, dev))


def test_binding_refuses(dev):
    b = Batch(dev, 1, [4], [9], 4, 4, 64, "f16", False, 16)
    E = binding.PAError
    good = dict(out=b.query.clone(), query=b.query, kv_cache=b.pool, block_tables=gpu(b.tables, dev), cu_seqlens_q=gpu(b.cu, dev),
                seq_lens=gpu(b.lens, dev), tree_masks=gpu(b.masks, dev), scale=0.1, max_seqlen_q=4)
    binding.pa_tree_attention(**good)
    for name, value in (("out", b.query.float()), ("kv_cache", b.pool.bfloat16()), ("tree_masks", gpu(b.masks, dev)[:-1]),
                        ("tree_masks", gpu(b.masks, dev).flatten()), ("seq_lens", gpu([1, 2], dev)), ("max_seqlen_q", 33),
                        ("block_tables", gpu(b.tables, dev).long()), ("kv_cache", b.pool[:1])):
        with pytest.raises((E, TypeError)):
            binding.pa_tree_attention(**dict(good, **{name: value}))
    with pytest.raises((E, TypeError)):
        binding.pa_tree_attention_fp8(**good, k_scale=1.0, v_scale=1.0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("counts,context,hq,hkv,d", [([4, 2], [37, 0], 4, 4, 128), ([16, 9], [300, 121], 8, 4, 128), ([25], [500], 6, 6, 64),
                                                     ([70, 64], [90, 64], 8, 2, 128)])
def test_queries_that_are_not_finite(dev, counts, context, hq, hkv, d, kind, fp8):
    """A NaN or an infinity in a query makes that head's row of that node NaN; every other row keeps its bits."""
    b = Batch(dev, 41, counts, context, hq, hkv, d, kind, fp8, 16)
    for ws in (b.workspace(), None):
        clean, query = b.run(ws), b.query
        b.query = query.clone()
        bad = {(0, 1): float("nan"), (1, 0): float("inf"), (b.total - 1, hq - 1): -float("inf"), (2, 2): float("nan")}
        for (node, head), value in bad.items():
            b.query[node, head, 5] = value
        out = b.run(ws)
        b.query = query
        for (node, head) in bad:
            assert out[node, head].isnan().all(), (node, head)
            out[node, head] = clean[node, head]
        assert (out == clean).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind,peak", [("f16", 60.0), ("bf16", 3e4)])
def test_large_scores(dev, kind, peak, fp8):
    """Scores of hundreds to 2^20 and more: one token takes the row (its neighbours are many units of the exponent away), in every
    form of the kernels. The bound is that of rounding the output and V alone, for rows whose runner-up weighs less than 2^-40."""
    import torch
    for counts, context, hq, hkv, d in (([4], [60], 4, 4, 128), ([20], [300], 4, 4, 128), ([20], [300], 4, 4, 64), ([80], [300], 4, 2, 128)):
        b = Batch(dev, 51, counts, context, hq, hkv, d, kind, fp8, 16)
        b.query *= peak
        q = b.query.double().cpu().numpy()
        k, v = b.values(0)
        seen = b.seen_of(0)
        g = hq // hkv
        for ws in (b.workspace(), None):
            out = b.run(ws).double().cpu().numpy()
            assert np.isfinite(out[:b.total]).all()
            for i in range(b.total):
                for h in range(hq):
                    at = np.flatnonzero(seen[i])
                    s = k[at, h // g] @ q[i, h] * b.scale * np.log2(np.e)
                    top = np.argsort(-s)[:2]
                    # fp32 scores of |q||k| D are off by 2^-24 of their terms' sum, and 8-bit terms of the queries by 2^-18 of
                    # the largest element's.
                    off = np.abs(k[at, h // g]).sum(1).max() * np.abs(q[i, h]).max() * b.scale * 2.0 ** (-17 if fp8 else -22)
                    if s[top[0]] - s[top[1]] > 40 + 2 * off:
                        want = v[at[top[0]], h // g]
                        assert np.all(np.abs(out[i, h] - want) <= np.abs(want) * 2 * E_OUT[kind] + 2.0 ** -24), (i, h)


def test_workspace_that_is_too_small(dev):
    for counts, context, hq, hkv in (([4], [300], 4, 4), ([33], [9000], 8, 2)):
        b = Batch(dev, 2, counts, context, hq, hkv, 128, "bf16", False, 16)
        ws = b.workspace()
        with pytest.raises(binding.PAError) as e:
            b.run(ws[:ws.numel() - 256])
        assert e.value.code == binding.PA_ERR_WORKSPACE
        with pytest.raises(binding.PAError) as e:
            b.run(ws[16:])
        assert e.value.code in (binding.PA_ERR_WORKSPACE, binding.PA_ERR_INVALID_ARG)


@pytest.mark.parametrize("seqs", [33, 128, 129])
@pytest.mark.parametrize("values", [(7,), (0, 5, 130, 131, 290)])
def test_many_sequences_of_equal_and_unequal_lengths(dev, seqs, values):
    """Whole units are taken longest sequence first, up to 128 of them; every row is there once."""
    rng = np.random.default_rng(seqs)
    counts, context = rng.integers(0, 12, seqs), rng.choice(values, seqs)
    b = Batch(dev, seqs, counts.tolist(), context.tolist(), 4, 2, 64, "f16", False, 16)
    b.check(b.run())


@pytest.mark.parametrize("seqs, longest", [(1, 0), (1, 500), (1, 7000), (3, 1100), (9, 60), (40, 1500)])
@pytest.mark.parametrize("fp8", [False, True], ids=["16", "fp8"])
def test_few_rows_shared_out_by_length(dev, seqs, longest, fp8):
    """Few rows: a warp's share grows with the segments' lengths."""
    rng = np.random.default_rng(longest + seqs)
    counts = rng.integers(1, 5, seqs)
    context = rng.integers(longest // 2, longest + 1, seqs)
    b = Batch(dev, seqs, counts.tolist(), context.tolist(), 8, 2, 128, "bf16", fp8, 16)
    b.check(b.run(b.workspace()))

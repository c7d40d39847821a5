"""pa_cross_attention and its FP8 form against the definition in 64 bits.

Tolerance per element, with o = sum w v the exact result, A = sum w |v|, u the
half step of the type P is rounded to (the query's; fp16 over an FP8 cache)
and u_o that of the output: rounding P moves numerator and denominator by at
most u A and u |o|; the output's rounding adds u_o |o|. fp32 scores of D <= 128
products of N(0, 1) draws are off by at most D 2^-24 sum |q k| scale < 1e-4 and
their exponentials by about as much, 3e-4 A in all. Weights below fp16's
normal range round by at most 2^-25 of the largest: + L 2^-25 max |v|.
"""
import math

import numpy as np
import pytest

from paged_kv_cache_120_gb300 import binding, build, workloads

from step_reference import ceil_div, cross_attention

pytestmark = pytest.mark.gpu

HALF = {workloads.F16: 2.0 ** -11, workloads.BF16: 2.0 ** -8}
KS, VS = workloads.FP8_K_SCALE, workloads.FP8_V_SCALE


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    binding.lib()
    assert binding.pa_get_device_error() == 0
    return torch.device("cuda:0")


class CrossCase:
    """Sequences with qlen[s] queries and kv[s] cached states; every slot that belongs to no state holds NaN."""

    def __init__(self, dev, dtype, hq, hkv, D, qlen, kv, B=16, fp8=False, seed=0, behind=3, scale=None, extra_width=1):
        import torch
        rng = np.random.default_rng(seed)
        self.dev, self.dtype, self.hq, self.hkv, self.D, self.B, self.fp8 = dev, dtype, hq, hkv, D, B, fp8
        self.qlen, self.kv = np.asarray(qlen), np.asarray(kv, np.int32)
        self.scale = 1 / math.sqrt(D) if scale is None else scale
        held = -(-self.kv // B)
        self.nb = int(held.sum()) + 3
        perm = rng.permutation(self.nb).astype(np.int32)
        self.bt = np.full((len(kv), max(1, int(held.max())) + extra_width), -1, np.int32)
        at = 0
        for s, n in enumerate(held):
            self.bt[s, :n] = perm[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(qlen)]).astype(np.int32)
        total = int(self.cu[-1])
        shape = (2, self.nb, B, hkv, D)
        if fp8:
            self.pool = workloads.fp8_codes(shape, 1.0, seed + 1, dev)
            self.pool[0], self.pool[1] = (workloads.fp8_codes(shape[1:], s, seed + 1 + k, dev) for k, s in enumerate((KS, VS)))
        else:
            self.pool = workloads.normal_values(shape, dtype, seed + 1, dev)
        used = np.zeros(self.nb * B, bool)
        for s, L in enumerate(self.kv):
            i = np.arange(L)
            used[self.bt[s, i // B] * B + i % B] = True
        unused = torch.from_numpy(np.nonzero(~used)[0]).to(dev)
        self.pool.view(2, -1, hkv, D)[:, unused] = 0x7F if fp8 else float("nan")
        # Rows behind the last sequence: in the buffers, not the call's to write.
        self.q = workloads.normal_values((total + behind, hq, D), dtype, seed + 2, dev)
        self.q[total:] = float("nan")
        self.bt_d, self.cu_d, self.kv_d = (torch.from_numpy(a).to(dev) for a in (self.bt, self.cu, self.kv))
        self.max_q = max(1, int(self.qlen.max()))

    def workspace(self):
        ws = binding.cross_attention_workspace(self.q, self.pool, len(self.kv), self.max_q)
        return None if ws is None else ws.fill_(0xFF)

    def run(self, workspace=None, flags=0, stream=None, out=None, max_q=None):
        import torch
        out = torch.full_like(self.q, float("nan")) if out is None else out
        a = (out, self.q, self.pool, self.bt_d, self.cu_d, self.kv_d, self.scale, max_q or self.max_q)
        if self.fp8:
            binding.pa_cross_attention_fp8(*a, KS, VS, workspace, flags, stream)
        else:
            binding.pa_cross_attention(*a, workspace, flags, stream)
        return out

    def reference(self):
        import torch
        pool = self.pool
        if self.fp8:
            pool = pool.view(torch.float8_e4m3fn).double()
            pool[0] *= KS
            pool[1] *= VS
        self.want, self.size = cross_attention(self.q.double(), pool.double(), self.bt, self.cu, self.kv, self.scale, self.B)
        vmax = 0.0
        for s, L in enumerate(self.kv):
            i = np.arange(L)
            at = torch.from_numpy((self.bt[s, i // self.B] * self.B + i % self.B).astype(np.int64)).to(self.dev)
            if L:
                vmax = max(vmax, float(pool.reshape(2, -1, self.hkv, self.D)[1, at].double().abs().max()))
        u = HALF[workloads.F16] if self.fp8 else HALF[self.dtype]
        self.tol = (u * (self.size + self.want.abs()) + HALF[self.dtype] * self.want.abs() + 3e-4 * self.size
                    + int(self.kv.max()) * 2.0 ** -25 * vmax)
        return self

    def check(self, out):
        import torch
        torch.cuda.synchronize()
        if not hasattr(self, "want"):
            self.reference()
        total = int(self.cu[-1])
        assert binding.pa_get_device_error() == 0
        assert torch.isnan(out[total:]).all(), "rows behind the last sequence were written"
        assert torch.isfinite(out[:total]).all()
        over = (out[:total].double() - self.want[:total]).abs() - self.tol[:total]
        assert float(over.max() if total else 0) <= 0, f"{float(over.max())} past the bound"

    def both(self, **kw):
        """With the workspace (where the shape has one) and without."""
        ws = self.workspace()
        if ws is not None:
            self.check(self.run(ws, **kw))
        self.check(self.run(None, **kw))
        return self


HEADS = [(4, 4, 64), (8, 2, 128), (16, 1, 64), (32, 1, 128), (12, 2, 128), (40, 40, 128), (20, 20, 64), (64, 8, 128)]
# Queries and states of many lengths, either the longer: none, one, across 16-token boxes and 128-token tiles.
QLEN = [1, 5, 0, 130, 3, 17, 1, 300, 2]
KV = [200, 0, 40, 33, 1, 128, 517, 129, 16]


@pytest.mark.parametrize("fp8", [False, True], ids=["16bit", "fp8"])
@pytest.mark.parametrize("dtype", [workloads.F16, workloads.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "%dx%dx%d" % h)
def test_ragged_prompts(dev, heads, dtype, fp8):
    CrossCase(dev, dtype, *heads, QLEN, KV, fp8=fp8, seed=sum(heads)).both()


@pytest.mark.parametrize("fp8", [False, True], ids=["16bit", "fp8"])
@pytest.mark.parametrize("dtype", [workloads.F16, workloads.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "%dx%dx%d" % h)
@pytest.mark.parametrize("block", [16, 48])
def test_single_tokens(dev, heads, dtype, fp8, block):
    """The decode form: one query per sequence (none for one), long, short, empty states."""
    kv = [1500, 1, 0, 16, 700, 17, 333, 2000, 15, 64]
    CrossCase(dev, dtype, *heads, [1, 1, 1, 1, 1, 0, 1, 1, 1, 1], kv, B=block, fp8=fp8, seed=sum(heads) + block).both()


@pytest.mark.parametrize("fp8", [False, True], ids=["16bit", "fp8"])
@pytest.mark.parametrize("heads,most", [((4, 4, 64), 16), ((8, 2, 128), 4), ((8, 2, 128), 2), ((6, 2, 128), 5), ((20, 20, 64), 5),
                                        ((20, 20, 64), 8), ((40, 40, 128), 3), ((16, 1, 64), 1), ((14, 2, 64), 2), ((8, 2, 128), 5)])
def test_a_few_candidates_each(dev, heads, most, fp8):
    """0 .. most queries per sequence: the rows of one kv head's tile are (query, head) pairs of ragged count."""
    rng = np.random.default_rng(most)
    qlen = rng.integers(0, most + 1, 23)
    qlen[4] = most
    kv = rng.integers(0, 900, 23)
    CrossCase(dev, workloads.BF16, *heads, qlen, kv, fp8=fp8, seed=most).both()


@pytest.mark.parametrize("most", [700, 10 ** 6, 2 ** 31 - 1])
def test_a_bound_far_above_all_the_queries(dev, most):
    """It means no more than total_q: no unit is taken in vain, nothing overflows."""
    c = CrossCase(dev, workloads.F16, 8, 8, 64, [3, 1, 300, 0, 40, 2], [100, 300, 50, 9, 0, 700])
    for ws in (binding.cross_attention_workspace(c.q, c.pool, 6, most), None):
        c.check(c.run(ws, max_q=most))


def test_a_larger_bound_than_the_longest_chunk(dev):
    c = CrossCase(dev, workloads.F16, 8, 2, 128, [1, 2, 1], [100, 300, 50])
    for most in (2, 3, 4, 5, 40, 1000):
        c.check(c.run(None, max_q=most))
        ws = binding.cross_attention_workspace(c.q, c.pool, 3, most)
        c.check(c.run(ws, max_q=most))


@pytest.mark.parametrize("fp8", [False, True], ids=["16bit", "fp8"])
@pytest.mark.parametrize("dtype", [workloads.F16, workloads.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("heads,most", [((4, 4, 64), 128), ((8, 2, 128), 32), ((32, 1, 128), 8), ((12, 2, 128), 16), ((20, 20, 64), 127)],
                         ids=lambda x: "%dx%dx%d" % x if isinstance(x, tuple) else str(x))
def test_chunks_of_one_query_tile(dev, heads, most, dtype, fp8):
    """Chunks that fit one 128-row tile (up to exactly): its two halves of the tensor memory then take every other K/V
    tile. One tile, odd and even counts of them, ends inside a tile, none; one sequence and many."""
    kv = [1, 127, 128, 129, 256, 257, 384, 1000, 0, 1151, 5, 640]
    qlen = [most, 1, most, most - 1, 2, most, 0, most, most, 3, most, most // 2]
    CrossCase(dev, dtype, *heads, qlen, kv, fp8=fp8, seed=most + dtype).both()
    CrossCase(dev, dtype, *heads, [most], [3333], fp8=fp8, seed=most + 1).both()


@pytest.mark.parametrize("qlen", [[1], [7], [600]])
def test_one_long_sequence(dev, qlen):
    CrossCase(dev, workloads.F16, 8, 2, 128, qlen, [30011], seed=5).both()


def test_many_short_sequences(dev):
    rng = np.random.default_rng(6)
    CrossCase(dev, workloads.F16, 4, 2, 64, rng.integers(0, 4, 700), rng.integers(0, 60, 700), seed=6).both()
    CrossCase(dev, workloads.F16, 4, 2, 64, np.ones(4096, int), rng.integers(0, 30, 4096), seed=7).both()


@pytest.mark.parametrize("fp8", [False, True], ids=["16bit", "fp8"])
@pytest.mark.parametrize("heads,most", [((8, 2, 128), 2), ((8, 2, 128), 4), ((16, 1, 64), 1)])
def test_the_largest_batch_of_short_queries(dev, heads, most, fp8):
    """4096 sequences: their lengths, offsets and tile counts fill what the tiles leave of the shared memory."""
    rng = np.random.default_rng(most)
    qlen = rng.integers(0, most + 1, 4096)
    qlen[7] = most
    CrossCase(dev, workloads.BF16, *heads, qlen, rng.integers(0, 40, 4096), fp8=fp8, seed=most).both()


@pytest.mark.parametrize("fp8", [False, True], ids=["16bit", "fp8"])
@pytest.mark.parametrize("heads,qlen,kv", [
    ((8, 8, 128), [300] * 6, [4000, 1, 1, 129, 0, 256]),            # long and one-tile units in one share
    ((2, 1, 64), [40, 1, 7], [1, 5000, 1]),                         # shares that hold only the cost of a unit
    ((8, 8, 64), [1] * 18 + [200], [1] * 18 + [6000]),              # many one-tile units ahead of a long one
    ((8, 8, 128), [100] * 9, [6400, 0, 1, 6400, 1, 1, 1, 1, 130])])
def test_shares_of_units_of_one_tile_and_of_many(dev, heads, qlen, kv, fp8):
    """K/V ranges shared out by weight: cuts before, in and behind units of one tile."""
    CrossCase(dev, workloads.F16, *heads, qlen, kv, fp8=fp8, seed=len(kv)).both()
    for cut in range(1, 4):  # the cuts move with the total
        CrossCase(dev, workloads.F16, *heads, qlen, [max(0, n - 128 * cut) if n > 1000 else n for n in kv], fp8=fp8,
                  seed=cut).both()


@pytest.mark.parametrize("n", [1, 31, 33, 64, 127, 128, 129, 200])
def test_batches_taken_longest_first(dev, n):
    """Around the batch size up to which whole units go by length: equal lengths, zeros, one far longer than the rest."""
    rng = np.random.default_rng(n)
    kv = rng.choice([0, 7, 7, 40, 129, 300], n)
    kv[n // 2] = 2500
    qlen = rng.integers(0, 150, n)
    qlen[-1] = 140
    CrossCase(dev, workloads.F16, 8, 4, 64, qlen, kv, seed=n).both()


@pytest.mark.parametrize("qlen", [[1, 1, 1], [4, 3, 2], [150, 20, 9]])
def test_without_any_states(dev, qlen):
    CrossCase(dev, workloads.F16, 8, 2, 128, qlen, [0, 0, 0]).both()


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
@pytest.mark.parametrize("qlen", [[1, 2, 1], [30, 200, 1]])
def test_other_scales(dev, scale, qlen):
    """Zero (plain means), negative, and large (nearly one-hot weights: score errors grow with the scale)."""
    c = CrossCase(dev, workloads.F16, 8, 2, 64, qlen, [77, 300, 0], scale=scale).reference()
    # fp32 scores: 64 * 2^-24 * sum |q k| (< 64 * 0.64 * 2) * 3 = 9e-4, twice for the quotient.
    c.tol = c.tol + (2e-3 * c.size if scale == 3.0 else 0)
    c.both()


def test_shared_tables(dev):
    """Several sequences over the same states, with and without the hint."""
    c = CrossCase(dev, workloads.BF16, 32, 8, 128, [1] * 12, [500] + [0] * 11, seed=9)
    c.bt[:], c.kv[:] = c.bt[0], 500 - np.arange(12)
    c.bt_d.copy_(__import__("torch").from_numpy(c.bt))
    c.kv_d.copy_(__import__("torch").from_numpy(c.kv))
    c.check(c.run(c.workspace(), flags=binding.PA_DECODE_SHARED_BLOCKS))
    c.both()


@pytest.mark.parametrize("qlen", [[1, 1, 1, 1], [4, 1, 3, 2], [130, 7, 40, 3]])
def test_the_same_bits_whatever_the_workspace_held_and_wherever_blocks_lie(dev, qlen):
    import torch
    c = CrossCase(dev, workloads.F16, 8, 2, 128, qlen, [3000, 100, 777, 2048], seed=10)
    ws = c.workspace()
    first = c.run(ws)
    c.check(first)
    ws.zero_()
    again = c.run(ws)
    perm = np.random.default_rng(1).permutation(c.nb).astype(np.int32)
    pool = torch.empty_like(c.pool)
    pool[:, torch.from_numpy(perm).to(dev).long()] = c.pool
    c.pool = pool
    c.bt_d.copy_(torch.from_numpy(np.where(c.bt >= 0, perm[c.bt], -1)))
    moved = c.run(ws)
    n = int(c.cu[-1])
    torch.cuda.synchronize()
    for o in (again, moved):
        assert torch.equal(o[:n].view(torch.int16), first[:n].view(torch.int16))


@pytest.mark.parametrize("qlen", [[1, 1, 1], [3, 1, 2], [130, 7, 40]])
def test_replayed_from_a_graph_with_new_lengths(dev, qlen):
    """A captured call reads the lengths, offsets and tables of the replay."""
    import torch
    c = CrossCase(dev, workloads.BF16, 8, 2, 128, qlen, [600, 900, 300], seed=11)
    ws, out = c.workspace(), torch.full_like(c.q, float("nan"))
    c.check(c.run(ws, out=out))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        c.run(ws, out=out)
    for kv in ([600, 900, 300], [1, 899, 0], [555, 16, 299]):
        c.kv[:] = kv
        c.kv_d.copy_(torch.from_numpy(c.kv))
        out.fill_(float("nan"))
        g.replay()
        c.reference()
        c.check(out)


@pytest.mark.parametrize("qlen", [[1, 1, 1, 1], [2, 1, 2, 1], [130, 7, 40, 3]])
def test_bad_sequences_are_flagged_and_their_rows_left(dev, qlen):
    """A length below zero or past the table; the others are right, and so is the next call."""
    import torch
    c = CrossCase(dev, workloads.F16, 8, 2, 128, qlen, [200, 100, 300, 50], seed=12)
    good = [(ws, c.run(ws)) for ws in (c.workspace(), None)]
    for bad in (-1, c.bt.shape[1] * 16 + 1, 2 ** 31 - 1):
        for ws, before in good:
            c.kv_d[1] = bad
            out = c.run(ws)
            torch.cuda.synchronize()
            assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN
            a, b = int(c.cu[1]), int(c.cu[2])
            assert torch.isnan(out[a:b]).all()
            c.kv_d[1] = 100
            keep = out.clone()
            keep[a:b] = before[a:b]
            c.check(keep)
            c.check(c.run(ws))


@pytest.mark.parametrize("cu", [[0, 3, 2, 5], [-2, 1, 2, 4], [0, 1, 90, 91], [0, 2 ** 31 - 1, -5, 3],
                                [0, 2 ** 31 - 2, 2 ** 31 - 1, 3]])
@pytest.mark.parametrize("most", [2, 100])
def test_bad_offsets_are_flagged_and_never_followed(dev, cu, most):
    import torch
    c = CrossCase(dev, workloads.F16, 8, 2, 128, [2, 2, 2], [200, 100, 300], seed=13)
    c.cu_d.copy_(torch.tensor(cu, dtype=torch.int64).to(torch.int32))
    for ws in (binding.cross_attention_workspace(c.q, c.pool, 3, most), None):
        guard = torch.full((c.q.shape[0] + 64,) + c.q.shape[1:], float("nan"), dtype=c.q.dtype, device=dev)
        c.run(ws, out=guard[32:32 + c.q.shape[0]], max_q=most)
        torch.cuda.synchronize()
        assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN
        assert torch.isnan(guard[:32]).all() and torch.isnan(guard[-32:]).all()


@pytest.mark.parametrize("qlen", [[1, 1], [3, 2], [140, 20]])
def test_bad_blocks_read_as_zeros(dev, qlen):
    import torch
    c = CrossCase(dev, workloads.F16, 8, 2, 128, qlen, [200, 100], seed=14)
    for bad in (c.nb, -1, 2 ** 31 - 1):
        bt = c.bt.copy()
        bt[0, 3] = bad
        c.bt_d.copy_(torch.from_numpy(bt))
        out = c.run(c.workspace())
        torch.cuda.synchronize()
        assert binding.pa_get_device_error() == binding.PA_DEVERR_BLOCK_ID
        assert torch.isfinite(out[:int(c.cu[-1])]).all()


def test_equal_to_decode_over_the_same_lengths(dev):
    """One query per sequence is pa_decode's definition: both within the bound of the same exact result."""
    import torch
    c = CrossCase(dev, workloads.F16, 32, 8, 128, [1] * 6, [900, 3, 0, 64, 1000, 17], seed=15, behind=0)
    out = torch.empty_like(c.q)
    binding.pa_decode(out, c.q, c.pool, c.bt_d, c.kv_d, c.scale, binding.decode_workspace(c.q, c.pool))
    c.check(out)
    c.check(c.run(c.workspace()))


def test_two_calls_on_two_streams(dev):
    """Two calls at once, each with its own workspace."""
    import torch
    a = CrossCase(dev, workloads.F16, 8, 2, 128, [1] * 40, [2000] * 40, seed=16)
    b = CrossCase(dev, workloads.BF16, 20, 20, 64, [60, 3, 200], [1500, 700, 1], seed=17)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [torch.full_like(c.q, float("nan")) for c in (a, b)]
    ws = [c.workspace() for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, w, o in zip((a, b), streams, ws, outs):
            c.run(w, stream=s, out=o)
    torch.cuda.synchronize()
    a.check(outs[0])
    b.check(outs[1])


def test_a_pool_past_2_to_the_32_bytes(dev):
    import torch
    c = CrossCase(dev, workloads.F16, 8, 8, 128, [1, 3, 70], [100, 90, 200], seed=18)
    nb = (5 << 30) // (16 * 8 * 128 * 2)
    pool = torch.zeros((2, nb, 16, 8, 128), dtype=torch.float16, device=dev)
    move = torch.from_numpy(np.linspace(0, nb - 1, c.nb).astype(np.int64)).to(dev)
    pool[:, move] = c.pool
    c.reference()
    c.pool = pool
    c.bt_d.copy_(torch.from_numpy(np.where(c.bt >= 0, move.cpu().numpy()[c.bt], -1)))
    c.both()


def test_two_graphs_at_once_share_nothing(dev):
    """Two captured calls of many work units each, replayed on two streams at once, over and over: each takes only its
    own units."""
    import torch
    rng = np.random.default_rng(19)
    cases = [CrossCase(dev, workloads.F16, 8, 8, 64, rng.integers(100, 400, 60), rng.integers(1, 600, 60), seed=20 + k)
             for k in range(2)]
    outs = [torch.full_like(c.q, float("nan")) for c in cases]
    ws = [c.workspace() for c in cases]
    graphs, streams = [torch.cuda.CUDAGraph() for _ in cases], [torch.cuda.Stream() for _ in cases]
    for c, w, o in zip(cases, ws, outs):
        c.run(w, out=o)
    torch.cuda.synchronize()
    for c, w, o, g in zip(cases, ws, outs, graphs):
        with torch.cuda.graph(g, capture_error_mode="relaxed"):
            for _ in range(40):
                c.run(w, out=o)
    for o in outs:
        o.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check(o)


def test_workspace_rules(dev):
    """The size asked for serves; less, or a misaligned one, is refused, whichever form the shape takes."""
    import torch
    for qlen, kv in (([1, 1], [100, 200]), ([40, 30], [100, 200])):
        c = CrossCase(dev, workloads.F16, 8, 2, 64, qlen, kv, seed=25)
        n = binding.pa_cross_attention_workspace_size(len(qlen), c.max_q, c.hq, c.hkv, 64, 16, binding.PA_F16, binding.PA_F16)
        big = torch.empty(n + 512, dtype=torch.uint8, device=dev)
        c.check(c.run(big[:n]))
        c.check(c.run(big))
        for bad in (big[:n - 128], big[16:16 + n]):
            with pytest.raises(binding.PAError) as e:
                c.run(bad)
            assert e.value.code == binding.PA_ERR_WORKSPACE
    # Many work units: no workspace is wanted, one given all the same is left alone.
    c = CrossCase(dev, workloads.F16, 8, 8, 64, [400] * 130, [64] * 130, seed=25)
    assert c.workspace() is None
    other = torch.full((512,), 7, dtype=torch.uint8, device=dev)
    c.check(c.run(other))
    assert bool((other == 7).all())
    assert binding.pa_get_device_error() == 0

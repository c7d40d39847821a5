"""Infinities and NaN in attended states, in every attention call: the rows
that the 64-bit definition makes finite are finite and within the bound, and
the others are not finite.

By the definition a NaN or +inf score makes its row NaN, a score of -inf has
weight 0 (a row of nothing but such scores is 0 / 0 = NaN), and a value that
is not finite reaches its column whatever its weight, 0 included (0 * inf is
NaN). Windows of such states are laid over tiles of 16 and 128 tokens, so that
a warp's share, a query tile's share of the K/V tiles, or a piece of a split
range holds nothing else. The bound on finite rows is test_gpu_cross.py's.
"""
import numpy as np
import pytest

from paged_kv_cache_120_gb300 import binding, workloads

from step_reference import cross_attention
from test_gpu_cross import HALF, KS, VS, CrossCase, dev  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = [(workloads.F16, False), (workloads.BF16, False), (workloads.F16, True), (workloads.BF16, True)]
IDS = ["f16", "bf16", "f16-fp8", "bf16-fp8"]
NAN, INF = float("nan"), float("inf")


class Poisoned(CrossCase):
    """States of some tokens replaced; `causal`: query i of sequence s sees kv[s] - qlen[s] + i + 1 tokens."""

    causal = False

    def slots(self, s, tokens):
        import torch
        i = np.asarray(tokens)
        return torch.from_numpy((self.bt[s, i // self.B] * self.B + i % self.B).astype(np.int64)).to(self.dev)

    def put(self, which, s, tokens, value, dims=slice(0, 1)):
        """K (0) or V (1) of the tokens in the dimensions, in every head; an FP8 pool takes NaN codes for NaN."""
        flat = self.pool.view(2, -1, self.hkv, self.D)
        at = self.slots(s, tokens)
        rows = flat[which, at]
        if self.fp8:
            assert np.isnan(value)
            rows[..., dims] = 0x7F
        else:
            rows[..., dims] = value
        flat[which, at] = rows
        return self

    def sign_of_first(self, sign):
        """Every query's first element has the sign: the sign of its scores with an infinite first key element."""
        self.q[..., 0] = sign * (self.q[..., 0].abs() + 0.125)
        return self

    def reference(self):
        import torch
        pool = self.pool
        if self.fp8:
            pool = pool.view(torch.float8_e4m3fn).double()
            pool[0] *= KS
            pool[1] *= VS
        pool = pool.double()
        total = int(self.cu[-1])
        if not self.causal:
            self.want, self.size = cross_attention(self.q[:total].double(), pool, self.bt, self.cu, self.kv, self.scale, self.B)
            return
        rows = np.repeat(np.arange(len(self.kv)), self.qlen)
        seen = np.concatenate([L - n + 1 + np.arange(n) for L, n in zip(self.kv, self.qlen)])
        self.want, self.size = cross_attention(self.q[:total].double(), pool, self.bt[rows], np.arange(total + 1), seen,
                                               self.scale, self.B)

    def check(self, out):
        import torch
        torch.cuda.synchronize()
        assert binding.pa_get_device_error() == 0
        total = int(self.cu[-1])
        want, got = self.want[:total], out[:total].double()
        fin = torch.isfinite(want)
        assert torch.equal(torch.isfinite(got), fin), \
            f"{int((torch.isfinite(got) & ~fin).sum())} finite where not, {int((~torch.isfinite(got) & fin).sum())} not where finite"
        flat = self.pool.view(2, -1, self.hkv, self.D)[1]
        v = flat.view(torch.float8_e4m3fn).double() * VS if self.fp8 else flat.double()
        vmax = float(v.nan_to_num(0, 0, 0).abs().max())
        u = HALF[workloads.F16] if self.fp8 else HALF[self.dtype]
        tol = (u * (self.size + want.abs()) + HALF[self.dtype] * want.abs() + 3e-4 * self.size
               + int(self.kv.max()) * 2.0 ** -25 * vmax)
        over = ((got - want).abs() - tol)[fin]
        assert over.numel() == 0 or float(over.max()) <= 0, f"{float(over.max())} past the bound"

    def run_decode(self):
        import torch
        out = torch.full_like(self.q, NAN)
        n = len(self.kv)
        a = (out[:n], self.q[:n], self.pool, self.bt_d, self.kv_d, self.scale)
        if self.fp8:
            ws = binding.decode_fp8_workspace(self.q[:n], self.pool).fill_(0xFF)
            binding.pa_decode_fp8(*a, KS, VS, ws)
        else:
            binding.pa_decode(*a, binding.decode_workspace(self.q[:n], self.pool).fill_(0xFF))
        return out

    def run_prefill(self, split):
        import torch
        out = torch.full_like(self.q, NAN)
        total = int(self.cu[-1])
        a = (out[:total], self.q[:total], self.pool, self.bt_d, self.cu_d, self.kv_d, self.scale, self.max_q)
        ws = None
        if split:
            ws = binding.prefill_workspace(self.q, self.pool, len(self.kv), self.max_q).fill_(0xFF)
        if self.fp8:
            binding.pa_prefill_fp8(*a, KS, VS, ws)
        else:
            binding.pa_prefill(*a, ws)
        if split:
            torch.cuda.synchronize()
            assert bool((ws != 0xFF).any()), "the K/V ranges were not split"
        return out

    def run_cross(self, split):
        import torch
        ws = self.workspace() if split else None
        out = self.run(ws)
        if split:
            torch.cuda.synchronize()
            assert bool((ws != 0xFF).any()), "the K/V ranges were not split"
        return out


def windows(L, width, starts):
    return [np.arange(a, min(L, a + width)) for a in starts if a < L]


# ------------------------------------------------------- the decode kernels

@pytest.mark.parametrize("call", ["decode", "cross"])
@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 2, 128), (16, 1, 64), (16, 1, 128)], ids=lambda h: "%dx%dx%d" % h)
def test_decode_nan_keys_of_a_whole_share(dev, heads, dtype, fp8, call):
    """Windows of 16 to 256 NaN keys: some warp's share of the tiles holds nothing else. Short sequences, and one tile."""
    for width in (1, 16, 32, 128, 256):
        c = Poisoned(dev, dtype, *heads, [1] * 8, [3040, 3000, 2049, 2048, 17, 16, 1, 640], fp8=fp8, seed=width)
        for s, start in enumerate((512, 2992, 2048, 0, 16, 0, 0, 100000)):
            for w in windows(int(c.kv[s]), width, [start]):
                c.put(0, s, w, NAN)
        c.reference()
        c.check(c.run_decode() if call == "decode" else c.run_cross(True))


@pytest.mark.parametrize("call", ["decode", "cross"])
@pytest.mark.parametrize("value", [INF, -INF], ids=["+inf", "-inf"])
@pytest.mark.parametrize("sign", [1, -1, 0], ids=["positive", "negative", "mixed"])
@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 2, 128), (16, 1, 64)], ids=lambda h: "%dx%dx%d" % h)
@pytest.mark.parametrize("dtype", [workloads.F16, workloads.BF16], ids=["f16", "bf16"])
def test_decode_infinite_keys(dev, heads, value, sign, call, dtype):
    """Scores of -inf weigh nothing, also where a tile, a share or a sequence's first tiles hold nothing else."""
    for width in (1, 16, 128, 400):
        c = Poisoned(dev, dtype, *heads, [1] * 7, [3000, 2049, 2048, 17, 16, 1, 640], seed=width)
        if sign:
            c.sign_of_first(sign)
        for s, start in enumerate((512, 2048, 0, 16, 0, 0, 100000)):
            for w in windows(int(c.kv[s]), width, [start]):
                c.put(0, s, w, value)
        c.reference()
        c.check(c.run_decode() if call == "decode" else c.run_cross(True))


@pytest.mark.parametrize("call", ["decode", "cross"])
@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
def test_decode_values_that_are_not_finite(dev, dtype, fp8, call):
    """They reach their columns, whatever the weight."""
    for value in (NAN,) if fp8 else (NAN, INF):
        c = Poisoned(dev, dtype, 8, 2, 128, [1] * 4, [2000, 129, 16, 700], fp8=fp8, seed=3)
        for s, start in enumerate((512, 128, 3)):
            c.put(1, s, windows(int(c.kv[s]), 16, [start])[0], value, dims=slice(5, 9))
        c.reference()
        c.check(c.run_decode() if call == "decode" else c.run_cross(True))


def test_decode_a_few_candidates(dev):
    """Several queries a sequence, some with NaN or infinite elements of their own: only those rows are lost."""
    for dtype, fp8 in TYPES:
        c = Poisoned(dev, dtype, 8, 2, 128, [4, 1, 0, 3, 2], [1500, 300, 40, 2000, 17], fp8=fp8, seed=4)
        c.put(0, 3, np.arange(1024, 1152), NAN)
        c.q[1, 3, 7] = NAN
        c.q[4, 0, 100] = INF
        c.reference()
        c.check(c.run_cross(True))


# --------------------------------------------------------- the chunk kernel

CHUNKS = [((4, 4, 64), [100], "solo"), ((8, 2, 128), [30, 7, 32], "solo"), ((4, 4, 64), [300, 3], "pairs"),
          ((8, 2, 128), [200, 40], "pairs")]


@pytest.mark.parametrize("split", [False, True], ids=["whole", "split"])
@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("heads,qlen,kind", CHUNKS, ids=lambda x: str(x) if isinstance(x, str) else "x".join(map(str, x)))
def test_chunk_nan_keys_of_a_whole_share(dev, heads, qlen, kind, dtype, fp8, split):
    """One NaN state behind a full K/V tile, and whole tiles of them, at many places: they are all that a query tile or a
    piece of a split range sees."""
    n = len(qlen)
    for L, width, starts in ((129, 1, (128,)), (2048, 128, range(0, 2048, 384)), (2049, 1, (0, 1920, 2048)),
                             (2000, 256, (128, 1792))):
        if split and L < 2000:
            continue
        for start in starts:
            c = Poisoned(dev, dtype, *heads, qlen, [L] * n, fp8=fp8, seed=start + n, extra_width=60)
            for w in windows(L, width, [start]):
                c.put(0, n - 1, w, NAN)
            c.reference()
            c.check(c.run_cross(split))


@pytest.mark.parametrize("split", [False, True], ids=["whole", "split"])
@pytest.mark.parametrize("value", [INF, -INF], ids=["+inf", "-inf"])
@pytest.mark.parametrize("heads,qlen,kind", CHUNKS, ids=lambda x: str(x) if isinstance(x, str) else "x".join(map(str, x)))
def test_chunk_infinite_keys(dev, heads, qlen, kind, value, split):
    n = len(qlen)
    for dtype, sign, scale in ((workloads.F16, 1, None), (workloads.BF16, -1, None), (workloads.F16, 0, None),
                               (workloads.BF16, 0, -0.1)):
        for L, width, start in ((129, 1, 128), (2048, 128, 0), (2048, 128, 640), (2049, 1, 2048), (2000, 256, 1792)):
            if split and L < 2000:
                continue
            c = Poisoned(dev, dtype, *heads, qlen, [L] * n, seed=L + start, scale=scale, extra_width=60)
            if sign:
                c.sign_of_first(sign)
            c.put(0, n - 1, windows(L, width, [start])[0], value)
            c.reference()
            c.check(c.run_cross(split))


@pytest.mark.parametrize("split", [False, True], ids=["whole", "split"])
@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("heads,qlen,kind", CHUNKS, ids=lambda x: str(x) if isinstance(x, str) else "x".join(map(str, x)))
def test_chunk_values_that_are_not_finite(dev, heads, qlen, kind, dtype, fp8, split):
    """Also behind keys so far below the others that their weights are 0 (0 * NaN is NaN)."""
    n = len(qlen)
    for L, width, start in ((256, 128, 128), (2048, 128, 640), (2049, 1, 2048)):
        if split and L < 2000:
            continue
        c = Poisoned(dev, dtype, *heads, qlen, [L] * n, fp8=fp8, seed=L, extra_width=60)
        w = windows(L, width, [start])[0]
        c.put(1, n - 1, w, NAN, dims=slice(5, 9))
        if not fp8:
            c.sign_of_first(1)
            c.put(0, n - 1, w, -60000.0)  # scores of -60000 * 0.125 * scale and less
        c.reference()
        c.check(c.run_cross(split))


@pytest.mark.parametrize("split", [False, True], ids=["whole", "split"])
@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("heads,qlen,kind", CHUNKS, ids=lambda x: str(x) if isinstance(x, str) else "x".join(map(str, x)))
def test_chunk_queries_that_are_not_finite(dev, heads, qlen, kind, dtype, fp8, split):
    """Only their own rows are lost."""
    c = Poisoned(dev, dtype, *heads, qlen, [2000] * len(qlen), fp8=fp8, seed=8, extra_width=60)
    c.q[3, 0, 7] = NAN
    c.q[5, 1] = NAN
    c.q[6, 2, 11] = INF
    c.q[int(c.cu[-1]) - 1, 3, 0] = -INF
    c.reference()
    assert not bool(c.want.isfinite().all()) and bool(c.want[4].isfinite().all())
    c.check(c.run_cross(split))
    c.causal = True
    c.reference()
    c.check(c.run_prefill(split))


@pytest.mark.parametrize("split", [False, True], ids=["whole", "split"])
@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("heads,qlen", [((4, 4, 64), [300, 3]), ((8, 2, 128), [33, 70])], ids=["4x4x64", "8x2x128"])
def test_causal_keys_that_are_not_finite(dev, heads, qlen, dtype, fp8, split):
    """pa_prefill: rows before the state are untouched, those behind it follow the definition."""
    n = len(qlen)
    for value in (NAN,) if fp8 else (NAN, INF, -INF):
        for L, width, start in ((2048, 128, 0), (2048, 128, 640), (2049, 1, 2048), (2000, 256, 1664), (2000, 1, 1999 - 40)):
            c = Poisoned(dev, dtype, *heads, qlen, [L] * n, fp8=fp8, seed=L + start, extra_width=60)
            c.causal = True
            c.put(0, n - 1, windows(L, width, [start])[0], value)
            c.reference()
            c.check(c.run_prefill(split))


@pytest.mark.parametrize("split", [False, True], ids=["whole", "split"])
@pytest.mark.parametrize("qlen", [[100], [300]])
def test_rows_whose_every_score_is_minus_infinity(dev, qlen, split):
    """0 / 0: NaN, as the decode kernels give it."""
    c = Poisoned(dev, workloads.F16, 4, 4, 64, qlen, [2000], seed=6, extra_width=60).sign_of_first(1)
    c.put(0, 0, np.arange(2000), -INF)
    c.reference()
    assert bool(c.want.isnan().all())
    c.check(c.run_cross(split))
    c.causal = True
    c.reference()
    c.check(c.run_prefill(split))


@pytest.mark.parametrize("qlen", [[1, 1], [100, 3], [300, 3]])
def test_scale_zero_times_infinity(dev, qlen):
    """0 * inf and 0 * NaN are NaN, in a sequence's last, partly filled tile as in a full one."""
    for L in (40, 128, 200):
        for value in (NAN, INF):
            c = Poisoned(dev, workloads.F16, 8, 2, 64, qlen, [L, 90], seed=7, scale=0.0)
            c.put(0, 0, [L - 9], value)
            c.reference()
            c.check(c.run(None))
            ws = c.workspace()
            if ws is not None:
                c.check(c.run(ws))

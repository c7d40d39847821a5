"""pa_rope_and_cache and its FP8 form against the definition in 64 bits.

Tolerance of a turned element y = x1 c - x2 s: half a step of its type
relative to y (one rounding), plus |x1| + |x2| times the error of the sines
and of two fp32 operations: the angle is off by at most 2^-31 turns (3e-9)
and the rounding of the reduced angle to fp32 (2^-25 half turns, 1e-7),
sincospif by 2 ulp (2.4e-7 at most near 1), the product and sum by 2^-23
(1.2e-7): 4.7e-7, taken as 1e-6; plus half the smallest step of fp16 (2^-25). Elements that
pass, V, and everything that is not written are equal bit for bit.
"""
import numpy as np
import pytest

import oracle
from paged_kv_cache_120_gb300 import binding, build, workloads

from harness import u16
from step_reference import rotate

pytestmark = pytest.mark.gpu

HALF = {workloads.F16: 2.0 ** -11, workloads.BF16: 2.0 ** -8}
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


class RopeCase:
    def __init__(self, dev, dtype, T, hq, hkv, D, rot=None, axes=1, adjacent=False, fp8=False, fused=False, B=16, seed=0,
                 far=1 << 17, skip=0.1, base=10000.0, pair_axes=None, in_place=False, pad=0):
        import torch
        rng = np.random.default_rng(seed)
        self.dtype, self.T, self.hq, self.hkv, self.D, self.B, self.fp8, self.adjacent = dtype, T, hq, hkv, D, B, fp8, adjacent
        rot = D if rot is None else rot
        self.freq = base ** (-2.0 * np.arange(rot // 2) / rot)
        self.axes = rng.integers(0, axes, rot // 2) if pair_axes is None else np.asarray(pair_axes)
        self.pos = rng.integers(-5, far, (axes, T))
        self.nb = T // B + 3
        self.slots = rng.permutation(self.nb * B)[:T].astype(np.int32)
        self.slots[rng.random(T) < skip] = -1
        val = lambda *s, k: workloads.normal_values(s, dtype, seed * 100 + k, dev)  # noqa: E731
        if fused:  # slices of one projection's rows, with room between the rows
            qkv = val(T, hq + 2 * hkv, D, k=1)
            wide = torch.full((T, (hq + 2 * hkv) * D + pad), float("nan"), dtype=qkv.dtype, device=dev)
            wide[:, :(hq + 2 * hkv) * D] = qkv.reshape(T, -1)
            cut = lambda a, h: wide[:, a * D:(a + h) * D].unflatten(1, (h, D))  # noqa: E731
            self.q, self.k, self.v = cut(0, hq), cut(hq, hkv), cut(hq + hkv, hkv)
        else:
            self.q, self.k, self.v = val(T, hq, D, k=1), val(T, hkv, D, k=2), val(T, hkv, D, k=3)
        shape = (2, self.nb, B, hkv, D)
        self.pool = (workloads.fp8_codes(shape, KS, seed + 7, dev) if fp8 else workloads.normal_values(shape, dtype, seed + 7, dev))
        self.out = self.q if in_place else torch.full((T, hq, D), float("nan"), dtype=self.q.dtype, device=dev)
        self.positions = torch.from_numpy(self.pos.astype(np.int32)).to(dev)
        self.slots_d = torch.from_numpy(self.slots).to(dev)
        self.plan = binding.rope_plan(self.freq, self.axes, dev)
        f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
        self.q64, self.k64, self.v_bits = f64(self.q), f64(self.k), u16(self.v)
        self.q_bits, self.k_bits = u16(self.q), u16(self.k)
        self.pool_before = self.pool.cpu().clone()
        self.rot = rot

    def run(self, stream=None):
        a = (self.out, self.q, self.k, self.v, self.pool, self.slots_d,
             self.positions[0] if len(self.pos) == 1 else self.positions, self.plan)
        if self.fp8:
            binding.pa_rope_and_cache_fp8(*a, KS, VS, adjacent=self.adjacent, stream=stream)
        else:
            binding.pa_rope_and_cache(*a, adjacent=self.adjacent, stream=stream)
        return self

    def near(self, got, want, size):
        assert np.isfinite(got).all()
        tol = HALF[self.dtype] * np.abs(want) + 1e-6 * size + 2.0 ** -25 * (size > 0)
        worst = np.max(np.abs(got - want) - tol)
        assert worst <= 0, f"{worst} past the bound"
        assert np.array_equal(got[size == 0], want[size == 0])

    def check(self, error=0):
        import torch
        torch.cuda.synchronize()
        assert binding.pa_get_device_error() == error
        q, q_size = rotate(self.q64, self.pos, self.freq, self.axes, self.adjacent)
        self.near(self.out.double().cpu().numpy(), q, q_size)
        k, k_size = rotate(self.k64, self.pos, self.freq, self.axes, self.adjacent)
        live = (self.slots >= 0) & (self.slots < self.nb * self.B)
        at = self.slots[live]
        rows = lambda p: p.reshape(2, self.nb * self.B, self.hkv, self.D)  # noqa: E731
        others = np.setdiff1d(np.arange(self.nb * self.B), at)
        if not self.fp8:
            got, before = rows(self.pool.cpu()), rows(self.pool_before)
            self.near(got[0, at].double().numpy(), k[live], k_size[live])
            assert np.array_equal(u16(got[1, at]), self.v_bits[live])
            assert torch.equal(got[:, others].contiguous().view(torch.int16), before[:, others].contiguous().view(torch.int16))
            return
        got, want = rows(self.pool.cpu().numpy()), self.pool_before.numpy().copy()
        assert oracle.reshape_and_cache_fp8(self.k_bits, self.v_bits, want, self.slots, self.nb, self.B, self.hkv, self.D,
                                            self.dtype, KS, VS) == live.sum()
        want = rows(want)
        assert np.array_equal(got[1], want[1])
        assert np.array_equal(got[0, others], want[0, others])
        # A code is the E4M3 value nearest to y / scale: half a step (2^-4 of it, 2^-10 among the subnormals), and the
        # turned value's own error; elements that pass are the write path's codes.
        value = np.array([oracle.e4m3_to_double(c) for c in range(256)])[got[0, at]]
        exact = np.clip(k[live] / KS, -448, 448)
        tol = 2.0 ** -4 * np.abs(exact) + 2.0 ** -10 + (1e-6 * k_size[live] + 2.0 ** -23 * np.abs(k[live])) / KS
        assert np.max(np.abs(value - exact) - tol) <= 0
        passed = k_size[live] == 0
        assert np.array_equal(got[0, at][passed], want[0, at][passed])


@pytest.mark.parametrize("fp8", [False, True], ids=["16bit", "fp8"])
@pytest.mark.parametrize("dtype", [workloads.F16, workloads.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("T,hq,hkv,D,rot,axes,adjacent,fused", [
    (1, 4, 4, 64, 64, 1, False, False),
    (1, 1, 1, 16, 16, 1, True, False),
    (7, 8, 2, 128, 128, 3, False, True),
    (65, 16, 1, 128, 64, 2, False, True),
    (130, 5, 5, 64, 32, 1, True, False),
    (33, 12, 2, 96, 80, 4, True, True),
    (301, 40, 40, 128, 128, 1, False, False),
    (19, 3, 1, 256, 256, 3, False, False),
    (5, 2, 2, 24, 16, 1, False, True),
    (9, 2, 1, 512, 512, 2, True, False),
])
def test_every_layout_equals_the_definition(dev, dtype, fp8, T, hq, hkv, D, rot, axes, adjacent, fused):
    RopeCase(dev, dtype, T, hq, hkv, D, rot, axes, adjacent, fp8, fused, seed=T + hq + D).run().check()


@pytest.mark.parametrize("fp8", [False, True], ids=["16bit", "fp8"])
@pytest.mark.parametrize("T,hq,hkv,D,rot,axes,adjacent,fused", [
    (2500, 4, 1, 64, 64, 1, False, True),
    (10001, 16, 4, 64, 32, 3, False, False),
    (9990, 3, 1, 32, 16, 2, True, True),
    (12289, 1, 1, 16, 16, 1, False, False),
    (2600, 12, 2, 128, 64, 1, True, True),
    (3000, 40, 40, 128, 128, 1, False, True),
])
def test_many_tokens(dev, fp8, T, hq, hkv, D, rot, axes, adjacent, fused):
    """Enough tokens for every CTA's ring to go round many times, several short tokens a unit, odd counts at the end."""
    RopeCase(dev, workloads.BF16, T, hq, hkv, D, rot, axes, adjacent, fp8, fused, seed=T, far=1 << 14).run().check()


@pytest.mark.parametrize("adjacent", [False, True])
def test_far_positions(dev, adjacent):
    """Positions over the whole 32-bit range, both signs."""
    c = RopeCase(dev, workloads.F16, 64, 4, 2, 64, axes=2, adjacent=adjacent, seed=3)
    rng = np.random.default_rng(4)
    c.pos = rng.integers(-2 ** 31, 2 ** 31, c.pos.shape)
    c.pos[:, :4] = [[0, 2 ** 31 - 1, -2 ** 31, -1]] * 2
    c.positions.copy_(__import__("torch").from_numpy(c.pos.astype(np.int32)))
    c.run().check()


def test_frequencies_of_any_size_and_sign(dev):
    c = RopeCase(dev, workloads.BF16, 40, 4, 2, 64, seed=5)
    c.freq = np.array([0.0, 1.0, -1.0, 1e-9, -3e-7, 7.5, -123.4, 2 * np.pi, np.pi, 1e6] + [0.01] * 22)
    c.plan = binding.rope_plan(c.freq, c.axes, dev)
    c.run().check()


def test_one_axis_equals_three_equal_axes(dev):
    """A text token's axes all hold its position: the bits of the one-axis call."""
    import torch
    a = RopeCase(dev, workloads.BF16, 50, 8, 2, 128, axes=1, seed=6).run()
    b = RopeCase(dev, workloads.BF16, 50, 8, 2, 128, axes=3, seed=6, pair_axes=np.arange(64) % 3)
    b.slots_d.copy_(a.slots_d)
    b.positions.copy_(a.positions.expand(3, 50))
    b.run()
    assert torch.equal(a.out.view(torch.int16), b.out.view(torch.int16))
    assert torch.equal(a.pool.view(torch.int16), b.pool.view(torch.int16))


def test_position_zero_changes_nothing(dev):
    import torch
    c = RopeCase(dev, workloads.F16, 30, 4, 4, 128, seed=7)
    c.positions.zero_()
    c.run()
    assert torch.equal(c.out, c.q)


@pytest.mark.parametrize("adjacent", [False, True])
def test_in_place_on_slices_with_room_between_rows(dev, adjacent):
    """query_out = query in a fused projection's rows; the rows' other columns (K, V, the room) stay."""
    import torch
    c = RopeCase(dev, workloads.BF16, 77, 8, 2, 64, adjacent=adjacent, fused=True, in_place=True, seed=8, pad=16)
    before = c.q.as_strided((77, c.q.stride(0)), (c.q.stride(0), 1)).clone()
    c.run().check()
    after = c.q.as_strided((77, c.q.stride(0)), (c.q.stride(0), 1))
    assert torch.equal(after[:, 8 * 64:].view(torch.int16), before[:, 8 * 64:].view(torch.int16))


def test_positions_with_a_stride(dev):
    """A [3, T] view of a longer buffer (a step's buffers are sized to a capacity)."""
    import torch
    c = RopeCase(dev, workloads.F16, 45, 4, 2, 64, axes=3, seed=9)
    wide = torch.full((3, 100), 12345, dtype=torch.int32, device=dev)
    wide[:, :45] = c.positions
    c.positions = wide[:, :45]
    c.run().check()


def test_bad_slots_are_skipped_and_flagged(dev):
    c = RopeCase(dev, workloads.F16, 40, 4, 2, 64, seed=10)
    c.slots[3], c.slots[17], c.slots[20] = c.nb * c.B, 2 ** 31 - 1, -2 ** 31
    c.slots_d.copy_(__import__("torch").from_numpy(c.slots))
    c.run().check(error=binding.PA_DEVERR_SLOT)


def test_an_axis_beyond_the_positions_reads_the_last(dev):
    c = RopeCase(dev, workloads.F16, 20, 4, 2, 64, axes=2, seed=11, pair_axes=np.arange(32) % 4)
    c.axes = np.minimum(c.axes, 1)
    c.run().check()


def test_special_values_stay_with_their_pair(dev):
    """Inf and NaN in one pair of a query and of a key reach that pair alone."""
    import torch
    c = RopeCase(dev, workloads.F16, 4, 2, 2, 64, seed=12, skip=0.0)
    c.run()
    clean_q, clean_k = c.out.clone(), c.pool.clone()
    c.q[1, 0, 5] = float("nan")
    c.k[2, 1, 40] = float("inf")
    c.run()
    torch.cuda.synchronize()
    hit = torch.zeros_like(c.out, dtype=torch.bool)
    hit[1, 0, [5, 37]] = True
    assert torch.isnan(c.out[hit]).all() and torch.equal(c.out[~hit], clean_q[~hit])
    row = c.pool.view(2, -1, 2, 64)[0, int(c.slots[2]), 1]
    assert (~torch.isfinite(row[[8, 40]])).all()
    row[[8, 40]] = clean_k.view(2, -1, 2, 64)[0, int(c.slots[2]), 1][[8, 40]]
    assert torch.equal(c.pool, clean_k)


def test_replayed_from_a_graph_and_on_another_stream(dev):
    import torch
    c = RopeCase(dev, workloads.BF16, 70, 8, 2, 128, axes=3, seed=13).run()
    torch.cuda.synchronize()
    want, pool = c.out.clone(), c.pool.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        c.run()
    side = torch.cuda.Stream()
    for again in (g.replay, lambda: c.run(side)):
        c.out.fill_(float("nan"))
        c.pool.zero_()
        side.wait_stream(torch.cuda.current_stream())
        again()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want)
        at = torch.from_numpy(c.slots[c.slots >= 0]).to(dev).long()
        assert torch.equal(c.pool.view(2, -1, 2, 128)[:, at], pool.view(2, -1, 2, 128)[:, at])


def test_a_pool_past_2_to_the_32_bytes(dev):
    """Slots whose byte offsets pass 2^32, in the K half and (always) in the V half."""
    import torch
    T, hkv, D, B = 5, 8, 128, 16
    c = RopeCase(dev, workloads.F16, T, 8, hkv, D, B=B, seed=14, skip=0.0)
    nb = (5 << 30) // (B * hkv * D * 2)
    c.nb = nb
    c.pool = torch.zeros((2, nb, B, hkv, D), dtype=torch.float16, device=dev)
    c.slots = np.array([0, nb * B - 1, nb * B // 2, 2 ** 32 // (hkv * D * 2), 2 ** 32 // (hkv * D * 2) - 1], np.int32)
    c.slots_d.copy_(torch.from_numpy(c.slots))
    c.run()
    torch.cuda.synchronize()
    k, size = rotate(c.k64, c.pos, c.freq, c.axes, False)
    flat = c.pool.view(2, nb * B, hkv, D)
    at = torch.from_numpy(c.slots).to(dev).long()
    c.near(flat[0, at].double().cpu().numpy(), k, size)
    assert np.array_equal(u16(flat[1, at]), c.v_bits)
    flat[:, at] = 0
    assert int(torch.count_nonzero(c.pool[0, ::997])) == 0 and int(torch.count_nonzero(c.pool[1, ::997])) == 0
    assert binding.pa_get_device_error() == 0


@pytest.mark.parametrize("dtype", [workloads.F16, workloads.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("scale", [0.0125, 0.01, 1.0, 1 / 3, 448.0, 6.1e-5, 1e-19, 3.3e19, 1e-25, 7e30])
def test_codes_of_every_value_are_the_write_paths(dev, dtype, scale):
    """All 65536 bit patterns as V and (unturned, at position 0) as K: the codes of pa_reshape_and_cache_fp8, which
    divides; the last two scales are outside the range of the reciprocal."""
    import torch
    T, hkv, D = 64, 8, 128
    x = torch.arange(65536, device=dev).to(torch.int32).to(torch.int16).view(workloads.torch_dtype(dtype)).view(T, hkv, D)
    pools = [torch.zeros((2, 4, 16, hkv, D), dtype=torch.uint8, device=dev) for _ in range(2)]
    slots = torch.arange(T, dtype=torch.int32, device=dev)
    binding.pa_reshape_and_cache_fp8(x, x, pools[0], slots, scale, scale)
    binding.pa_rope_and_cache_fp8(torch.empty_like(x), x, x, x, pools[1], slots, torch.zeros_like(slots),
                                  binding.rope_plan(np.ones(8), None, dev), scale, scale)
    torch.cuda.synchronize()
    assert torch.equal(pools[0][1], pools[1][1])
    # A turned pair mixes NaN and Inf (x 1 - Inf 0): compare K where the pair is finite, and the dimensions that pass.
    pair = torch.isfinite(x[..., :8]) & torch.isfinite(x[..., 8:16])
    got, want = (p[0].view(T, hkv, D) for p in pools)
    assert torch.equal(got[..., 16:], want[..., 16:])
    for a in (slice(0, 8), slice(8, 16)):
        # -0 - Inf-free products can turn -0 into +0: the codes of both are equal values.
        same = (got[..., a] == want[..., a]) | (((got[..., a] | want[..., a]) & 0x7F) == 0)
        assert bool(same[pair].all())


def test_no_tokens(dev):
    import torch
    c = RopeCase(dev, workloads.F16, 4, 2, 2, 64, seed=15)
    e = lambda t: t[:0]  # noqa: E731
    binding.pa_rope_and_cache(e(c.out), e(c.q), e(c.k), e(c.v), c.pool, e(c.slots_d), c.positions[0, :0], c.plan)
    torch.cuda.synchronize()
    assert torch.equal(c.pool.cpu(), c.pool_before)

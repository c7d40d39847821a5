"""The serving-step operators together, as a server uses them: every step's
maps built on the GPU, rotary writes by those slots, causal attention of the
new tokens over the cache (pa_prefill, pa_decode), cross attention to cached
encoder states, and the blocks of finished sequences returned; eagerly and
replayed from one CUDA graph. The other side is plain: a growing list of keys
and values per sequence, attention in 64 bits, the host allocator's tables.
"""
import numpy as np
import pytest

from paged_kv_cache_120_gb300 import binding, build, workloads

from step_reference import build_step, rotate

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


def attend(q, k, v, scale, causal_from=None):
    """q [n, Hq, D], k / v [L, Hkv, D], float64 -> [n, Hq, D]; query i sees tokens below causal_from + i + 1."""
    n, hq, d = q.shape
    L, hkv, _ = k.shape
    s = np.einsum("qhgd,lhd->qhgl", q.reshape(n, hkv, hq // hkv, d), k) * scale
    if causal_from is not None:
        s = np.where((np.arange(L) <= causal_from + np.arange(n)[:, None])[:, None, None], s, -np.inf)
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    return np.einsum("qhgl,lhd->qhgd", w, v).reshape(n, hq, d)


class Server:
    """Rows of a running batch over one self-attention pool and one pool of encoder states."""

    ROWS, B, WIDTH, CAP, HQ, HKV, D, NB = 6, 16, 12, 96, 8, 2, 64, 40

    def __init__(self, dev, dtype, fp8, seed):
        import torch
        self.dev, self.dtype, self.fp8 = dev, dtype, fp8
        self.rng = np.random.default_rng(seed)
        self.scale = self.D ** -0.5
        self.ks, self.vs = (workloads.FP8_K_SCALE, workloads.FP8_V_SCALE) if fp8 else (1.0, 1.0)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
        self.tables, self.lens, self.query = i32(self.ROWS, self.WIDTH), i32(self.ROWS), i32(self.ROWS)
        order = self.rng.permutation(self.NB).astype(np.int32)
        self.free, self.n = torch.from_numpy(order).to(dev), torch.full((1,), self.NB, dtype=torch.int32, device=dev)
        self.cu, self.pos, self.slots, self.adm = i32(self.ROWS + 1), i32(self.CAP), i32(self.CAP), i32(1)
        td = workloads.torch_dtype(dtype)
        shape = (2, self.NB, self.B, self.HKV, self.D)
        # A fresh pool holds whatever memory held: NaN here.
        self.pool = (torch.full(shape, 0x7F, dtype=torch.uint8, device=dev) if fp8
                     else torch.full(shape, float("nan"), dtype=td, device=dev))
        self.freq = 10000.0 ** (-2.0 * np.arange(self.D // 2) / self.D)
        self.axes = np.arange(self.D // 2) % 3
        self.plan = binding.rope_plan(self.freq, self.axes, dev)
        self.pos3 = i32(3, self.CAP)
        # Encoder states of each row: another length, some none.
        self.enc = self.rng.integers(0, 150, self.ROWS).astype(np.int32)
        self.enc[2] = 0
        held = -(-self.enc // self.B)
        enb = int(held.sum()) + 1
        perm = self.rng.permutation(enb).astype(np.int32)
        self.ebt = np.full((self.ROWS, int(held.max())), -1, np.int32)
        at = 0
        for r, h in enumerate(held):
            self.ebt[r, :h] = perm[at:at + h]
            at += h
        self.ebt_d, self.enc_d = torch.from_numpy(self.ebt).to(dev), torch.from_numpy(self.enc).to(dev)
        self.epool = workloads.normal_values((2, enb, self.B, self.HKV, self.D), dtype, seed + 5, dev)
        self.qkv = torch.zeros(self.CAP, (self.HQ + 2 * self.HKV) * self.D, dtype=td, device=dev)
        cut = lambda a, h: self.qkv[:, a * self.D:(a + h) * self.D].unflatten(1, (h, self.D))  # noqa: E731
        self.q, self.k, self.v = cut(0, self.HQ), cut(self.HQ, self.HKV), cut(self.HQ + self.HKV, self.HKV)
        self.rot, self.out, self.cross = (torch.zeros(self.CAP, self.HQ, self.D, dtype=td, device=dev) for _ in range(3))
        self.ws = binding.prefill_workspace(self.rot, self.pool, self.ROWS, self.CAP)
        self.cws = binding.cross_attention_workspace(self.rot, self.epool, self.ROWS, self.CAP)
        self.model_k = [np.zeros((0, self.HKV, self.D)) for _ in range(self.ROWS)]
        self.model_v = [np.zeros((0, self.HKV, self.D)) for _ in range(self.ROWS)]
        self.graph = None

    def calls(self):
        """The step's calls: fixed buffers, fixed sizes, so that they can be captured."""
        binding.pa_build_step(self.tables, self.lens, self.query, self.free, self.n, self.lens, self.n, self.cu, self.pos,
                              self.slots, self.adm, self.B)
        a = (self.rot, self.q, self.k, self.v, self.pool, self.slots, self.pos3, self.plan)
        p = (self.out, self.rot, self.pool, self.tables, self.cu, self.lens, self.scale, self.CAP)
        if self.fp8:
            binding.pa_rope_and_cache_fp8(*a, self.ks, self.vs)
            binding.pa_prefill_fp8(*p, self.ks, self.vs, self.ws)
        else:
            binding.pa_rope_and_cache(*a)
            binding.pa_prefill(*p, self.ws)
        binding.pa_cross_attention(self.cross, self.rot, self.epool, self.ebt_d, self.cu, self.enc_d, self.scale, self.CAP,
                                   self.cws)

    def step(self, query, replay):
        import torch
        before = dict(tables=self.tables.cpu().numpy(), lens=self.lens.cpu().numpy(), free=self.free.cpu().numpy(),
                      n=int(self.n))
        want = build_step(before["tables"], before["lens"], query, before["free"], before["n"], self.CAP, self.B)
        total = int(want["cu"][-1])
        # Each token has a time (its place in the sequence) and a row and column of its own.
        pos3 = np.stack([want["positions"], self.rng.integers(0, 40, self.CAP), self.rng.integers(0, 60, self.CAP)])
        self.qkv.copy_(workloads.normal_values(self.qkv.shape, self.dtype, int(self.rng.integers(1 << 30)), self.dev))
        self.query.copy_(torch.from_numpy(query.astype(np.int32)))
        self.pos3.copy_(torch.from_numpy(pos3.astype(np.int32)))
        for o in (self.out, self.cross):
            o.fill_(float("nan"))
        if replay:
            if self.graph is None:
                torch.cuda.synchronize()
                self.graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(self.graph, capture_error_mode="relaxed"):
                    self.calls()
            self.graph.replay()
        else:
            self.calls()
        torch.cuda.synchronize()
        assert binding.pa_get_device_error() == 0
        for name, t in (("tables", self.tables), ("lens", self.lens), ("free_list", self.free), ("cu", self.cu),
                        ("positions", self.pos), ("slots", self.slots)):
            assert np.array_equal(t.cpu().numpy(), want[name]), name
        assert int(self.n) == want["num_free"] and int(self.adm) == want["admitted"]
        f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
        q, _ = rotate(f64(self.q), pos3, self.freq, self.axes, False)
        k, _ = rotate(f64(self.k), pos3, self.freq, self.axes, False)
        v, out, cross = f64(self.v), f64(self.out), f64(self.cross)
        ek, ev = f64(self.epool).reshape(2, -1, self.HKV, self.D)
        # Inputs of the attentions carry the step's own roundings (of q and k, and an FP8 cache's codes): a score of D
        # products moves by about sqrt(D) half steps, so values of order 1 by a few: 5e-3 / 3e-2 (16 bits), 0.25 (FP8, whose
        # V alone is off by 2^-4 of values up to 4).
        near = 0.25 if self.fp8 else {workloads.F16: 5e-3, workloads.BF16: 3e-2}[self.dtype]
        tol16 = {workloads.F16: 5e-3, workloads.BF16: 3e-2}[self.dtype]
        for r in range(self.ROWS):
            a, b = int(want["cu"][r]), int(want["cu"][r + 1])
            if query[r] < 0:
                self.model_k[r] = self.model_v[r] = np.zeros((0, self.HKV, self.D))
            if a == b:
                continue
            old = len(self.model_k[r])
            self.model_k[r] = np.concatenate([self.model_k[r], k[a:b]])
            self.model_v[r] = np.concatenate([self.model_v[r], v[a:b]])
            ref = attend(q[a:b], self.model_k[r], self.model_v[r], self.scale, old)
            assert np.max(np.abs(out[a:b] - ref)) <= near
            i = np.arange(self.enc[r])
            at = self.ebt[r, i // self.B] * self.B + i % self.B if len(i) else i
            ref = attend(q[a:b], ek[at], ev[at], self.scale) if len(i) else np.zeros_like(q[a:b])
            assert np.max(np.abs(cross[a:b] - ref)) <= tol16
        assert np.isnan(out[total:]).all() and np.isnan(cross[total:]).all()
        return want


@pytest.mark.parametrize("replay", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("dtype,fp8", [(workloads.F16, False), (workloads.BF16, False), (workloads.BF16, True)],
                         ids=["f16", "bf16", "fp8"])
def test_a_serving_loop(dev, dtype, fp8, replay):
    s = Server(dev, dtype, fp8, seed=21)
    returned = stopped = 0
    for step in range(16):
        lens = s.lens.cpu().numpy()
        query = np.zeros(s.ROWS, int)
        for r in range(s.ROWS):
            u = s.rng.random()
            if lens[r] == 0:
                query[r] = int(s.rng.integers(1, 50)) if u < 0.7 else 0  # a prompt
            elif u < 0.15 or lens[r] > s.WIDTH * s.B - 20:
                query[r] = -1
                returned += 1
            else:
                query[r] = 1 if u < 0.8 else int(s.rng.integers(2, 18))  # a token, or a prompt's next chunk
        want = s.step(query, replay)
        stopped += want["admitted"] < s.ROWS
    assert returned > 2


def test_decode_steps_follow(dev):
    """Single-token steps: maps, rotary write, pa_decode (which may start beside the write) and the single-token cross
    attention; 20 of them, with lengths in place."""
    import torch
    s = Server(dev, workloads.F16, False, seed=22)
    s.step(np.array([30, 16, 1, 15, 5, 20]), False)
    q, out, cross = s.rot[:s.ROWS], torch.zeros_like(s.rot[:s.ROWS]), torch.zeros_like(s.rot[:s.ROWS])
    ws, cws = binding.decode_workspace(q, s.pool), binding.cross_attention_workspace(q, s.epool, s.ROWS, 1)
    slots, pos = s.slots[:s.ROWS], s.pos[:s.ROWS]
    plan = binding.rope_plan(s.freq, None, dev)
    s.query.fill_(1)
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    for step in range(20):
        new = workloads.normal_values((s.ROWS, s.HQ + 2 * s.HKV, s.D), s.dtype, 500 + step, dev)
        out.fill_(float("nan"))
        cross.fill_(float("nan"))
        binding.pa_build_step(s.tables, s.lens, s.query, s.free, s.n, s.lens, s.n, s.cu, pos, slots, s.adm, s.B)
        binding.pa_rope_and_cache(q, new[:, :s.HQ], new[:, s.HQ:s.HQ + s.HKV], new[:, s.HQ + s.HKV:], s.pool, slots, pos, plan)
        binding.pa_decode(out, q, s.pool, s.tables, s.lens, s.scale, ws, binding.PA_DECODE_LENS_READY)
        binding.pa_cross_attention(cross, q, s.epool, s.ebt_d, s.cu, s.enc_d, s.scale, 1, cws)
        torch.cuda.synchronize()
        x = f64(new)
        p = np.array([[len(k) for k in s.model_k]])
        assert pos.tolist() == p[0].tolist()
        zero = np.zeros(s.D // 2, int)
        rq, _ = rotate(x[:, :s.HQ], p, s.freq, zero, False)
        rk, _ = rotate(x[:, s.HQ:s.HQ + s.HKV], p, s.freq, zero, False)
        ek, ev = f64(s.epool).reshape(2, -1, s.HKV, s.D)
        for r in range(s.ROWS):
            s.model_k[r] = np.concatenate([s.model_k[r], rk[r:r + 1]])
            s.model_v[r] = np.concatenate([s.model_v[r], x[r:r + 1, s.HQ + s.HKV:]])
            assert np.max(np.abs(f64(out[r:r + 1]) - attend(rq[r:r + 1], s.model_k[r], s.model_v[r], s.scale))) <= 5e-3
            i = np.arange(s.enc[r])
            at = s.ebt[r, i // s.B] * s.B + i % s.B if len(i) else i
            ref = attend(rq[r:r + 1], ek[at], ev[at], s.scale) if len(i) else np.zeros((1, s.HQ, s.D))
            assert np.max(np.abs(f64(cross[r:r + 1]) - ref)) <= 5e-3
    assert binding.pa_get_device_error() == 0

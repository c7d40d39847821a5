"""The speculative step's operators together, as a server uses them: blocks for drafted trees, their maps, rotary writes, tree
attention in every layer, verification and commit, eagerly and replayed from one CUDA graph; sequences come and go between steps.
The other side is plain: a growing list of keys and values per sequence and layer, attention and verification in 64 bits."""
import numpy as np
import pytest

from paged_kv_cache_120_gb300 import binding, build, step, workloads

import tree_reference as ref
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


class Server:
    S, B, WIDTH, HQ, HKV, D, NB, LAYERS, VOCAB = 5, 16, 10, 8, 2, 64, 44, 3, 61

    def __init__(self, dev, dtype, fp8, mode, nodes, seed):
        import torch
        self.dev, self.dtype, self.fp8, self.mode, self.nodes = dev, dtype, fp8, mode, nodes
        self.rng = np.random.default_rng(seed)
        self.ks, self.vs = (workloads.FP8_K_SCALE, workloads.FP8_V_SCALE) if fp8 else (1.0, 1.0)
        td = workloads.torch_dtype(dtype)
        shape = (2, self.NB, self.B, self.HKV, self.D)
        pools = [torch.full(shape, 0x7F, dtype=torch.uint8, device=dev) if fp8 else
                 torch.full(shape, float("nan"), dtype=td, device=dev) for _ in range(self.LAYERS)]
        i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)  # noqa: E731
        self.freq = 10000.0 ** (-2.0 * np.arange(self.D // 2) / self.D)
        self.step = step.SpeculativeStep(pools, i32(np.full((self.S, self.WIDTH), -1)), i32(np.zeros(self.S)),
                                         i32(self.rng.permutation(self.NB)), i32([self.NB]), self.HQ, nodes, self.VOCAB,
                                         binding.rope_plan(self.freq, None, dev), self.ks, self.vs, dtype, mode)
        self.k = [[np.zeros((0, self.HKV, self.D)) for _ in range(self.S)] for _ in range(self.LAYERS)]
        self.v = [[np.zeros((0, self.HKV, self.D)) for _ in range(self.S)] for _ in range(self.LAYERS)]

    def turn(self, nodes):
        """One step: nodes[s] drafted nodes (0: idle, -1: finished). Returns the accepted counts."""
        import torch
        st, rng, S = self.step, self.rng, self.S
        f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
        total = S * self.nodes
        lens = st.seq_lens.cpu().numpy().copy()
        before = build_step(st.tables.cpu().numpy(), lens, nodes, st.free_list.cpu().numpy(), int(st.num_free), total, self.B)
        cu = before["cu"]
        used = int(cu[-1])
        parents = np.full(total, -1, np.int32)
        at = np.concatenate([[0], np.cumsum(np.maximum(nodes, 0))])  # the caller's layout: a row that gets no blocks is cut off
        for s in range(S):
            if nodes[s] > 0:
                parents[at[s]:at[s] + nodes[s]] = ref.random_parents(rng, nodes[s], 3, 0.15)
        p = rng.dirichlet(np.full(self.VOCAB, 0.05), total).astype(np.float32)
        q = (0.7 * p + 0.3 * rng.dirichlet(np.full(self.VOCAB, 0.05), total)).astype(np.float32)
        tokens = np.zeros(total, np.int32)
        for s in range(S):
            for i in range(at[s], at[s] + max(0, nodes[s])):
                row = at[s] + max(parents[i], 0)
                tokens[i] = rng.choice(self.VOCAB, p=q[row].astype(np.float64) / q[row].astype(np.float64).sum()) \
                    if self.mode == "draft" else np.argsort(-p[row])[rng.integers(0, 2)]
        u = rng.random((total, 2)).astype(np.float32)
        put = lambda t, a: t.copy_(torch.from_numpy(np.ascontiguousarray(a)))  # noqa: E731
        st.qkv.copy_(workloads.normal_values(st.qkv.shape, self.dtype, int(rng.integers(1 << 30)), self.dev))
        put(st.tokens, tokens)
        put(st.parents, parents)
        put(st.target, p)
        if st.draft is not None:
            put(st.draft, q)
        if st.uniforms is not None:
            put(st.uniforms, u)
        put(st.query_lens, np.asarray(nodes, np.int32))
        st.run()
        torch.cuda.synchronize()
        assert binding.pa_get_device_error() == 0
        assert np.array_equal(st.cu.cpu().numpy(), cu)
        # The nodes' positions: the context's length and the depth.
        seen, pos = [], np.zeros(total, np.int64)
        for s in range(S):
            if nodes[s] < 0:
                lens[s] = 0
                for layer in range(self.LAYERS):
                    self.k[layer][s] = self.v[layer][s] = np.zeros((0, self.HKV, self.D))
            m, depth = ref.closure(parents[cu[s]:cu[s + 1]])
            seen.append(m)
            pos[cu[s]:cu[s + 1]] = lens[s] + depth
        assert np.array_equal(st.positions.cpu().numpy()[:used], pos[:used])
        x = f64(st.qkv)
        zero = np.zeros(self.D // 2, int)
        rq, _ = rotate(x[:, :self.HQ], pos[None], self.freq, zero, False)
        rk, _ = rotate(x[:, self.HQ:self.HQ + self.HKV], pos[None], self.freq, zero, False)
        v = x[:, self.HQ + self.HKV:]
        # As in the serving step's test: rounded q and k (and codes) move a score by a few half steps.
        near = 0.25 if self.fp8 else {workloads.F16: 5e-3, workloads.BF16: 3e-2}[self.dtype]
        counts, after, free = st.count.cpu().numpy(), [], before["free_list"][:before["num_free"]].tolist()
        path, new = st.path.cpu().numpy(), st.new_tokens.cpu().numpy()
        outs = [f64(o) for o in st.outs]
        for s in range(S):
            a, b = cu[s], cu[s + 1]
            if a == b:
                assert counts[s] == 0
                after.append(lens[s])
                continue
            for layer in range(self.LAYERS):
                kk, vv = np.concatenate([self.k[layer][s], rk[a:b]]), np.concatenate([self.v[layer][s], v[a:b]])
                o, _ = ref.attend(rq[a:b], kk, vv, np.concatenate([np.ones((b - a, lens[s]), bool), seen[s]], 1), self.D ** -0.5)
                assert np.max(np.abs(outs[layer][a:b] - o)) <= near, (s, layer)
            want_path, want_new = ref.verify(parents[a:b], tokens[a:b], p[a:b].astype(np.float64),
                                             q[a:b].astype(np.float64) if self.mode == "draft" else None,
                                             None if self.mode == "greedy" else u[a:b].astype(np.float64))
            n = len(want_path)
            assert counts[s] == n and path[a:a + n].tolist() == want_path and new[a:a + n].tolist() == want_new
            for layer in range(self.LAYERS):
                self.k[layer][s] = np.concatenate([self.k[layer][s], rk[a:b][want_path]])
                self.v[layer][s] = np.concatenate([self.v[layer][s], v[a:b][want_path]])
            after.append(lens[s] + n)
            t = before["tables"][s]
            free += [t[j] for j in range(-(-(lens[s] + b - a) // self.B) - 1, -(-after[-1] // self.B) - 1, -1)]
        assert st.seq_lens.tolist() == after
        assert int(st.num_free) == len(free) and st.free_list.tolist()[:len(free)] == free
        return counts

    def check_decode(self):
        """What the steps have left in the pools is what a decode step reads."""
        import torch
        st = self.step
        q = workloads.normal_values((self.S, self.HQ, self.D), self.dtype, 77, self.dev)
        out = torch.zeros_like(q)
        for layer, pool in enumerate(st.pools):
            if self.fp8:
                ws = binding.decode_fp8_workspace(q, pool)
                binding.pa_decode_fp8(out, q, pool, st.tables, st.seq_lens, self.D ** -0.5, self.ks, self.vs, ws)
            else:
                ws = binding.decode_workspace(q, pool)
                binding.pa_decode(out, q, pool, st.tables, st.seq_lens, self.D ** -0.5, ws)
            got, qq = out.double().cpu().numpy(), q.double().cpu().numpy()
            for s in range(self.S):
                L = len(self.k[layer][s])
                o, _ = ref.attend(qq[s:s + 1], self.k[layer][s], self.v[layer][s], np.ones((1, L), bool), self.D ** -0.5)
                near = 0.25 if self.fp8 else {workloads.F16: 5e-3, workloads.BF16: 3e-2}[self.dtype]
                assert np.max(np.abs(got[s] - o)) <= near, (layer, s)


@pytest.mark.parametrize("replay", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("dtype,fp8,mode,nodes", [(workloads.F16, False, "greedy", 7), (workloads.BF16, False, "draft", 20),
                                                  (workloads.BF16, True, "sample", 20), (workloads.F16, True, "draft", 4),
                                                  (workloads.BF16, False, "sample", 40)])
def test_speculative_steps(dev, dtype, fp8, mode, nodes, replay):
    s = Server(dev, dtype, fp8, mode, nodes, seed=nodes)
    if replay:
        s.step.capture()
    moved = 0
    for turn in range(14):
        lens = s.step.seq_lens.cpu().numpy()
        want = np.zeros(s.S, int)
        for r in range(s.S):
            if lens[r] > s.WIDTH * s.B - 2 * nodes or (lens[r] and s.rng.random() < 0.06):
                want[r] = -1
            elif s.rng.random() < 0.9:
                want[r] = int(s.rng.integers(1, nodes + 1))
        counts = s.turn(want)
        moved += int((counts > 1).sum())
    assert moved > 5
    s.check_decode()


def test_modes_are_checked():
    with pytest.raises(ValueError):
        step.SpeculativeStep([], None, None, None, None, 1, 1, 1, None, mode="none")

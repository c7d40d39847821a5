"""A model inside the speculative step: its projections of each layer come from the layer before's attention, and the target's rows
from the last layer's, eagerly and in a CUDA graph. Every layer's rotated projections, and its attention over the bits that were
cached, are held to the plain forms in 64 bits, the outcome to the target's rows that the model wrote.

Bounds: rotated values are off by half a step of their type and 2^-18 of the largest value (fp32 products, angles within 1e-7).
Attention as in test_gpu_tree_attention.py, but for the scores: D products summed in fp32 are off by at most D 2^-24 of the sum of
their magnitudes, taken from the inputs, and a weight by that much of itself and the exponential's 2^-16."""
import numpy as np
import pytest

from paged_kv_cache_120_gb300 import binding, build, step, workloads

import tree_reference as ref
from step_reference import rotate

pytestmark = pytest.mark.gpu

S, B, WIDTH, HQ, HKV, D, NB, LAYERS, VOCAB, HIDDEN, NODES = 4, 16, 8, 8, 2, 64, 40, 3, 97, 128, 12


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    binding.lib()
    assert binding.pa_get_device_error() == 0
    return torch.device("cuda:0")


class Model:
    """Embedding, layers of a projection and an output product, and a softmax over the vocabulary."""

    def __init__(self, dev, dtype, seed):
        import torch
        g = torch.Generator(device=dev).manual_seed(seed)
        mat = lambda *s: (torch.randn(*s, generator=g, device=dev) / s[0] ** 0.5).to(dtype)  # noqa: E731
        self.embed = torch.randn(VOCAB, HIDDEN, generator=g, device=dev).to(dtype)
        self.qkv = [mat(HIDDEN, (HQ + 2 * HKV) * D) for _ in range(LAYERS)]
        self.out = [mat(HQ * D, HIDDEN) for _ in range(LAYERS)]
        self.vocab = mat(HIDDEN, VOCAB)
        self.h, self.log = None, None

    def record(self, st):
        """What the layer before read: its projections, its rotated queries and the K and V rows that it cached."""
        if self.log is not None:
            used = int(st.cu[-1])
            flat = st.pools[len(self.log)].view(2, -1, HKV, D)[:, st.slots[:used].long()]
            self.log.append([x.double().cpu().numpy() for x in (st.qkv, st.rotated, flat)])

    def project(self, st, layer):
        if layer > 0:
            self.record(st)
        if layer == 0:
            self.h = self.embed[st.tokens.long()]
        else:
            self.h = self.h + st.outs[layer - 1].flatten(1) @ self.out[layer - 1]
        st.qkv.copy_((self.h @ self.qkv[layer]).view_as(st.qkv))

    def head(self, st):
        self.record(st)
        h = self.h + st.outs[-1].flatten(1) @ self.out[-1]
        st.target.copy_((3 * (h @ self.vocab).float()).softmax(-1))


def make(dev, dtype, mode, model):
    import torch
    td = workloads.torch_dtype(dtype)
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)  # noqa: E731
    freq = 10000.0 ** (-2.0 * np.arange(D // 2) / D)
    pools = [torch.zeros(2, NB, B, HKV, D, dtype=td, device=dev) for _ in range(LAYERS)]
    st = step.SpeculativeStep(pools, i32(np.full((S, WIDTH), -1)), i32(np.zeros(S)), i32(np.arange(NB)), i32([NB]), HQ, NODES, VOCAB,
                              binding.rope_plan(freq, None, dev), dtype=dtype, mode=mode, project=model.project, head=model.head)
    return st, freq


def fill(st, rng, turn):
    """Trees of drafted tokens, most of them the same token twice or likely ones."""
    import torch
    nodes = rng.integers(1, NODES + 1, S) if turn else np.full(S, NODES)
    nodes[rng.random(S) < 0.15] = 0
    total = int(nodes.sum())
    put = lambda t, a: t.copy_(torch.from_numpy(np.ascontiguousarray(a)))  # noqa: E731
    parents, tokens = np.full(S * NODES, -1, np.int32), np.zeros(S * NODES, np.int32)
    parents[:total] = np.concatenate([ref.random_parents(rng, n, 4) if n else np.zeros(0, np.int32) for n in nodes])
    tokens[:total] = rng.integers(0, VOCAB, total)
    u = rng.random((S * NODES, 2)).astype(np.float32)
    q = rng.dirichlet(np.full(VOCAB, 0.3), S * NODES).astype(np.float32)
    put(st.query_lens, nodes.astype(np.int32))
    put(st.parents, parents)
    put(st.tokens, tokens)
    if st.uniforms is not None:
        put(st.uniforms, u)
    if st.draft is not None:
        put(st.draft, q)
    return nodes, parents, tokens, u, q


@pytest.mark.parametrize("dtype,mode", [(workloads.F16, "draft"), (workloads.BF16, "sample"), (workloads.BF16, "greedy")])
def test_a_model_in_the_step(dev, dtype, mode):
    import torch
    td = workloads.torch_dtype(dtype)
    model = Model(dev, td, 3)
    st, freq = make(dev, dtype, mode, model)
    rng = np.random.default_rng(1)
    keys, vals = ([[np.zeros((0, HKV, D)) for _ in range(S)] for _ in range(LAYERS)] for _ in range(2))
    zero = np.zeros(D // 2, int)
    e = {workloads.F16: 2.0 ** -10, workloads.BF16: 2.0 ** -7}[dtype]
    differ = 0
    for turn in range(5):
        nodes, parents, tokens, u, q = fill(st, rng, turn)
        lens = st.seq_lens.cpu().numpy().copy()
        model.log = []
        st.run()
        torch.cuda.synchronize()
        assert binding.pa_get_device_error() == 0 and len(model.log) == LAYERS
        differ += sum(not np.array_equal(model.log[0][0], x[0]) for x in model.log[1:])
        cu = np.concatenate([[0], np.cumsum(nodes)])
        p = st.target.double().cpu().numpy()
        counts, path, new = st.count.tolist(), st.path.cpu().numpy(), st.new_tokens.cpu().numpy()
        for s in range(S):
            a, b = cu[s], cu[s + 1]
            if a == b:
                assert counts[s] == 0
                continue
            seen, depth = ref.closure(parents[a:b])
            see = np.concatenate([np.ones((b - a, lens[s]), bool), seen], 1)
            want_path, want_new = ref.verify(parents[a:b], tokens[a:b], p[a:b], q[a:b].astype(np.float64) if mode == "draft" else None,
                                             None if mode == "greedy" else u[a:b].astype(np.float64))
            n = len(want_path)
            assert counts[s] == n and path[a:a + n].tolist() == want_path and new[a:a + n].tolist() == want_new
            for layer in range(LAYERS):
                x, rotated, cached = [z[..., a:b, :, :] for z in model.log[layer]]
                rq, _ = rotate(x[:, :HQ], (lens[s] + depth)[None], freq, zero, False)
                rk, _ = rotate(x[:, HQ:HQ + HKV], (lens[s] + depth)[None], freq, zero, False)
                for got, want in ((rotated, rq), (cached[0], rk)):
                    assert np.all(np.abs(got - want) <= e / 2 * np.abs(want) + 2.0 ** -18 * np.abs(x).max()), (s, layer)
                assert np.array_equal(cached[1], x[:, HQ + HKV:])
                kk, vv = np.concatenate([keys[layer][s], cached[0]]), np.concatenate([vals[layer][s], cached[1]])
                size = np.einsum("nhgd,lhd->nhgl", np.abs(rotated).reshape(b - a, HKV, HQ // HKV, D), np.abs(kk)).max() * D ** -0.5
                off = 2.0 ** -16 + D * 2.0 ** -24 * size
                o, mean = ref.attend(rotated, kk, vv, see, D ** -0.5)
                bound = e / 2 * np.abs(o) + (e / 2 + off) * (mean + np.abs(o)) + 2.0 ** -25 * (1 + len(kk) * np.abs(vv).max())
                assert np.all(np.abs(st.outs[layer][a:b].double().cpu().numpy() - o) <= bound), (s, layer)
                keys[layer][s] = np.concatenate([keys[layer][s], cached[0][want_path]])
                vals[layer][s] = np.concatenate([vals[layer][s], cached[1][want_path]])
            assert st.seq_lens[s].item() == lens[s] + n
    assert differ == 5 * (LAYERS - 1)  # each layer had projections of its own


def test_a_captured_step_replays_the_model(dev):
    """The same steps eagerly and from a graph: the same bits in pools, outcomes and lengths."""
    import torch
    runs = []
    for captured in (False, True):
        model = Model(dev, torch.bfloat16, 5)
        st, _ = make(dev, workloads.BF16, "draft", model)
        if captured:
            st.capture()
        rng, log = np.random.default_rng(8), []
        for turn in range(5):
            nodes = fill(st, rng, turn)[0]
            used = int(nodes.sum())
            st.run()
            log.append([t.clone() for t in (st.count, st.path[:used], st.new_tokens[:used], st.seq_lens, st.num_free, st.target[:used],
                                            *[o[:used] for o in st.outs])])
        runs.append((log, [p.clone() for p in st.pools]))
    torch.cuda.synchronize()
    assert binding.pa_get_device_error() == 0
    for a, b in zip(*[r[0] for r in runs]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert all(torch.equal(x, y) for x, y in zip(runs[0][1], runs[1][1]))


def test_without_a_model_the_buffers_are_the_callers(dev):
    """qkv and target as the caller filled them: what a model that fills them with the same values gives."""
    import torch
    results = []
    for inside in (False, True):
        qkv = workloads.normal_values((S * NODES, HQ + 2 * HKV, D), workloads.F16, 5, dev)
        g = torch.Generator(device=dev).manual_seed(2)
        rows = torch.rand(S * NODES, VOCAB, generator=g, device=dev).softmax(-1)
        model = Model(dev, torch.float16, 1)
        st, _ = make(dev, workloads.F16, "sample", model)
        if inside:
            st.project, st.head = (lambda s, layer: s.qkv.copy_(qkv)), (lambda s: s.target.copy_(rows))
        else:
            st.project = st.head = None
            st.qkv.copy_(qkv)
            st.target.copy_(rows)
        fill(st, np.random.default_rng(4), 0)
        st.run()
        results.append([t.clone() for t in (st.count, st.path, st.new_tokens, st.seq_lens, *st.outs, *st.pools)])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*results))
    assert binding.pa_get_device_error() == 0

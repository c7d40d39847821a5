"""CPU checks of the speculative step's C ABI and of its plain forms: bad arguments are refused on the host, before any CUDA
call, with a status and a message; the verification's law is the target's."""
import ctypes

import numpy as np
import pytest

from paged_kv_cache_120_gb300 import binding, build

import tree_reference as ref

INVALID, UNSUPPORTED, WORKSPACE = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED, binding.PA_ERR_WORKSPACE
P = 1 << 20  # stands for a device pointer: never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def caller(fn, order, ok):
    return lambda **kw: fn(*[dict(ok, **kw)[k] for k in order], None)


def test_build_tree_refusals(lib):
    order = ("parents", "cu", "lens", "S", "T", "pos", "masks", "words")
    call = caller(lib.pa_build_tree, order, dict(parents=P, cu=P, lens=P, S=3, T=9, pos=P, masks=P, words=2))
    assert call(S=-1) == INVALID and "num_seqs" in binding.pa_last_error()
    assert call(S=4097) == INVALID
    assert call(T=-1) == INVALID
    for w in (0, 33, -1):
        assert call(words=w) == INVALID and "mask_words" in binding.pa_last_error()
    for name in ("parents", "cu", "lens", "masks"):
        assert call(**{name: None}) == INVALID and "null" in binding.pa_last_error(), name
        assert call(**{name: P + 2}) == INVALID and "misaligned" in binding.pa_last_error(), name
    assert call(pos=P + 1) == INVALID
    assert call(S=0) == 0 and call(T=0) == 0


ATTEND = ("out", "q", "kv", "bt", "width", "cu", "lens", "masks", "words", "S", "T", "maxq", "scale", "hq", "hkv", "d", "nb", "bs",
          "dt")
ATTEND_OK = dict(out=P, q=P, kv=P, bt=P, width=4, cu=P, lens=P, masks=P, words=2, S=3, T=9, maxq=33, scale=0.1, hq=8, hkv=2, d=64,
                 nb=16, bs=16, dt=0)


def test_tree_attention_refusals(lib):
    def call(ws=None, ws_bytes=0, flags=0, **kw):
        head = [dict(ATTEND_OK, **kw)[k] for k in ATTEND]
        a = lib.pa_tree_attention(*head, ws, ws_bytes, flags, None)
        b = lib.pa_tree_attention_fp8(*head, 0.5, 0.5, ws, ws_bytes, flags, None)
        assert a == b
        return a
    assert call(dt=2) == UNSUPPORTED
    assert call(d=96) == UNSUPPORTED
    assert call(hq=7) == INVALID
    assert call(hq=34) == UNSUPPORTED
    assert call(bs=24) == INVALID and call(bs=0) == INVALID
    for name in ("S", "T", "maxq"):
        assert call(**{name: -1}) == INVALID
    assert call(nb=0) == INVALID and call(width=0) == INVALID
    assert call(width=(1 << 26) + 1) == INVALID
    assert call(scale=float("inf")) == INVALID
    assert call(flags=2) == INVALID and "flags" in binding.pa_last_error()
    assert call(maxq=65) == INVALID and "mask words" in binding.pa_last_error()
    assert call(maxq=1025, words=40) == INVALID
    assert call(words=0) == INVALID
    for name in ("out", "q", "kv", "bt", "cu", "lens"):
        assert call(**{name: None}) == INVALID and "null" in binding.pa_last_error(), name
        assert call(**{name: P + 2}) == INVALID and "misaligned" in binding.pa_last_error(), name
    assert call(masks=None) == INVALID and call(masks=P + 2) == INVALID
    assert call(S=0) == 0 and call(T=0) == 0 and call(maxq=0) == 0
    assert call(maxq=2, ws=P + 128, ws_bytes=1 << 30) == WORKSPACE
    head = [ATTEND_OK[k] for k in ATTEND]
    for ks, vs in ((0.0, 1.0), (1.0, -1.0), (float("nan"), 1.0), (1.0, float("inf"))):
        assert lib.pa_tree_attention_fp8(*head, ks, vs, None, 0, 0, None) == INVALID


def test_tree_attention_workspace_refusals(lib):
    n = ctypes.c_size_t(0)
    size = lambda *a: lib.pa_tree_attention_workspace_size(*a, ctypes.byref(n))  # noqa: E731
    assert size(3, 33, 8, 2, 96, 16, 0, 0) == UNSUPPORTED
    assert size(3, 33, 8, 2, 64, 8, 0, 0) == INVALID
    assert size(3, 33, 8, 2, 64, 16, 3, 3) == UNSUPPORTED
    assert size(3, 33, 8, 2, 64, 16, 0, 1) == UNSUPPORTED
    assert size(-1, 33, 8, 2, 64, 16, 0, 0) == INVALID
    assert lib.pa_tree_attention_workspace_size(3, 33, 8, 2, 64, 16, 0, 0, None) == INVALID
    assert size(0, 33, 8, 2, 64, 16, 0, 0) == 0 and n.value == 0


def test_verify_refusals(lib):
    order = ("count", "path", "out", "tokens", "parents", "cu", "S", "T", "target", "ts", "draft", "ds", "vocab", "dt", "u")
    call = caller(lib.pa_verify_draft, order, dict(count=P, path=P, out=P, tokens=P, parents=P, cu=P, S=3, T=9, target=P, ts=100,
                                                   draft=P, ds=100, vocab=100, dt=3, u=P))
    for dt in (2, 4, -1):
        assert call(dt=dt) == UNSUPPORTED
    assert call(S=-1) == INVALID and call(S=4097) == INVALID and call(T=-1) == INVALID
    assert call(vocab=0) == INVALID and call(vocab=(1 << 30) + 1, ts=1 << 31, ds=1 << 31) == INVALID
    assert call(ts=99) == INVALID and call(ds=99) == INVALID
    assert call(u=None) == INVALID and "greedy" in binding.pa_last_error()
    for name in ("count", "path", "out", "tokens", "parents", "cu", "target"):
        assert call(**{name: None}) == INVALID and "null" in binding.pa_last_error(), name
        assert call(**{name: P + 2}) == INVALID and "misaligned" in binding.pa_last_error(), name
    assert call(draft=P + 2) == INVALID and call(u=P + 2) == INVALID
    assert call(target=P + 1, draft=None, dt=0) == INVALID
    assert call(S=0) == 0


def test_commit_refusals(lib):
    order = ("layers", "bt", "width", "cu", "lens", "count", "path", "S", "T", "out", "free", "n", "n_out", "nb", "bs", "h", "d", "dt")
    pools = (ctypes.c_void_p * 2)(P, P)
    ok = dict(layers=2, bt=P, width=4, cu=P, lens=P, count=P, path=P, S=3, T=9, out=P, free=P, n=P, n_out=P, nb=16, bs=16, h=2, d=64,
              dt=0)
    call = lambda pools=pools, **kw: lib.pa_commit_draft(pools, *[dict(ok, **kw)[k] for k in order], None)  # noqa: E731
    assert call(dt=3) == UNSUPPORTED
    for kw in (dict(S=-1), dict(S=4097), dict(T=-1), dict(layers=0), dict(layers=513), dict(nb=0), dict(width=0), dict(bs=24), dict(h=0),
               dict(d=0), dict(width=(1 << 26) + 1), dict(h=1, d=4), dict(h=1, d=8, dt=2)):
        assert call(**kw) == INVALID, kw
    for name in ("bt", "cu", "lens", "count", "path", "out"):
        assert call(**{name: None}) == INVALID and "null" in binding.pa_last_error(), name
        assert call(**{name: P + 2}) == INVALID and "misaligned" in binding.pa_last_error(), name
    assert call(n=None) == INVALID and call(n_out=None) == INVALID and call(free=P + 2) == INVALID
    assert call(pools=None) == INVALID
    assert call(pools=(ctypes.c_void_p * 2)(P, P + 8)) == INVALID and "layer 1" in binding.pa_last_error()
    assert call(S=0) == 0


def test_plain_verify_keeps_the_law():
    """The first new token's distribution is the target's, for one, two and three children drawn from another row (and for
    children that were chosen): 20000 trials, every count within 5 standard deviations."""
    rng = np.random.default_rng(5)
    p, q = rng.dirichlet(np.ones(6)), rng.dirichlet(np.ones(6))
    trials = 20000
    for kids in (1, 2, 3):
        parents = np.array([-1] + [0] * kids)
        for drawn in (True, False):
            counts = np.zeros(6)
            for _ in range(trials):
                tokens = np.concatenate([[0], rng.choice(6, kids, p=q) if drawn else np.arange(kids)])
                u = rng.random((kids + 1, 2))
                target = np.stack([p] * (kids + 1))
                _, out = ref.verify(parents, tokens, target, np.stack([q] * (kids + 1)) if drawn else None, u)
                counts[out[0]] += 1
            assert np.all(np.abs(counts - trials * p) <= 5 * np.sqrt(trials * p * (1 - p))), (kids, drawn)

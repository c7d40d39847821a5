"""CPU checks of the serving-step operators' C ABI and binding: bad arguments
are refused on the host, before any CUDA call, with a status and a message."""
import ctypes

import numpy as np
import pytest

from paged_kv_cache_120_gb300 import binding, build

INVALID, UNSUPPORTED = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED
P = 1 << 20  # stands for a device pointer: never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def test_build_step_refusals(lib):
    order = ("bt", "width", "lens", "query", "S", "free", "n", "lens_out", "n_out", "cu", "pos", "slots", "cap", "adm", "nb",
             "bs")
    ok = dict(bt=P, width=4, lens=P, query=P, S=3, free=P, n=P, lens_out=P, n_out=P, cu=P, pos=P, slots=P, cap=8, adm=P,
              nb=16, bs=16)

    def call(**kw):
        return lib.pa_build_step(*[dict(ok, **kw)[k] for k in order], None)
    assert call(S=-1) == INVALID and "num_seqs" in binding.pa_last_error()
    assert call(S=4097) == INVALID
    for bs in (0, 8, 24, -16):
        assert call(bs=bs) == INVALID and "block_size" in binding.pa_last_error()
    assert call(nb=0) == INVALID
    assert call(width=0) == INVALID
    assert call(cap=-1) == INVALID
    assert call(cap=(1 << 30) + 1) == INVALID
    assert call(width=(1 << 26) + 1) == INVALID
    assert call(nb=1 << 27) == INVALID and "slot" in binding.pa_last_error()
    for name in ("bt", "lens", "query", "free", "n", "lens_out", "n_out", "cu", "slots", "adm"):
        assert call(**{name: None}) == INVALID and "null" in binding.pa_last_error(), name
        assert call(**{name: P + 2}) == INVALID and "misaligned" in binding.pa_last_error(), name
    assert call(pos=P + 1) == INVALID


def rope_args(**kw):
    order = ("qo", "q", "k", "v", "kv", "slots", "pos", "axes", "pstride", "plan", "rot", "adj", "T", "qos", "qs", "ks", "vs",
             "hq", "hkv", "d", "nb", "bs", "dt")
    ok = dict(qo=P, q=2 * P, k=P, v=P, kv=P, slots=P, pos=P, axes=3, pstride=5, plan=P, rot=64, adj=0, T=5, qos=512, qs=768,
              ks=768, vs=768, hq=8, hkv=2, d=64, nb=16, bs=16, dt=0)
    return [dict(ok, **kw)[k] for k in order]


def test_rope_refusals(lib):
    def call(**kw):
        a = lib.pa_rope_and_cache(*rope_args(**kw), None)
        b = lib.pa_rope_and_cache_fp8(*rope_args(**kw), 0.5, 0.5, None)
        assert a == b
        return a
    assert call(dt=2) == UNSUPPORTED
    for d in (0, 20, -8, 1032):
        assert call(d=d) == UNSUPPORTED, d
    for rot in (0, 8, 24, 80, -16):
        assert call(rot=rot) == UNSUPPORTED, rot
    assert call(rot=528, d=528, qos=4224, qs=4224, ks=4224, vs=4224) == UNSUPPORTED
    for axes in (0, 5, -1):
        assert call(axes=axes) == INVALID, axes
    assert call(pstride=4) == INVALID
    for name in ("qos", "qs"):
        assert call(**{name: 504}) == INVALID and call(**{name: 772}) == INVALID, name
    for name in ("ks", "vs"):
        assert call(**{name: 120}) == INVALID and call(**{name: 132}) == INVALID, name
    assert call(T=-1) == INVALID
    assert call(hq=0) == INVALID and call(hkv=0) == INVALID
    assert call(bs=24) == INVALID and call(nb=0) == INVALID and call(nb=1 << 27) == INVALID
    for name in ("qo", "q", "k", "v", "kv", "slots", "pos", "plan"):
        assert call(**{name: None}) == INVALID and "null" in binding.pa_last_error(), name
    for name in ("qo", "q", "k", "v", "kv"):
        assert call(**{name: P + 8}) == INVALID and "misaligned" in binding.pa_last_error(), name
    assert call(slots=P + 2) == INVALID and call(pos=P + 2) == INVALID and call(plan=P + 4) == INVALID
    assert call(q=P) == INVALID and "in place" in binding.pa_last_error()
    assert call(T=0) == binding.PA_OK
    for ks, vs in ((0.0, 1.0), (1.0, -2.0), (float("inf"), 1.0), (1.0, float("nan"))):
        assert lib.pa_rope_and_cache_fp8(*rope_args(), ks, vs, None) == INVALID
        assert "k_scale" in binding.pa_last_error()


def test_rope_refuses_more_tokens_than_its_indexes_count(lib):
    """Unit, token and window indexes are 32-bit and run past the last token: 2^30 tokens at most."""
    for T in (2 ** 30 + 1, 2 ** 31 - 8, 2 ** 31 - 1):
        for axes in (1, 2):
            args = rope_args(T=T, pstride=T, axes=axes)
            assert lib.pa_rope_and_cache(*args, None) == UNSUPPORTED and "tokens" in binding.pa_last_error()
            assert lib.pa_rope_and_cache_fp8(*args, 0.5, 0.5, None) == UNSUPPORTED


def test_rope_plan_words(lib):
    """Turns per position as a fraction of 2^64 (to 2 units of its 62 bits), the axis in the low two bits."""
    from fractions import Fraction
    two_pi = Fraction(6283185307179586476925286766559005768394, 10 ** 39)
    f = np.array([1.0, 0.5, 1e-9, -1.0, 123.456, -1e6, 4294967296.0, 0.0, 1e-300, -1e-300, 2 * np.pi])
    axes = np.arange(len(f)) % 4
    words = binding.pa_rope_plan(f, axes).view(np.uint64)
    for x, axis, w in zip(f, axes, words.tolist()):
        assert w & 3 == axis
        turns = Fraction(float(x)) / two_pi
        off = Fraction(w & ~3, 1 << 64) - (turns - turns.__floor__())
        off -= round(off)  # modulo a whole turn
        assert abs(off) <= Fraction(2, 1 << 62), x
    assert binding.pa_rope_plan([]).size == 0
    assert (binding.pa_rope_plan([1.0, 2.0]).view(np.uint64) & 3 == 0).all()


def test_rope_plan_refusals(lib):
    for bad in (float("nan"), float("inf"), -float("inf"), 4.3e9):
        with pytest.raises(binding.PAError) as e:
            binding.pa_rope_plan([1.0, bad])
        assert e.value.code == INVALID
    for axes in ([0, 4], [-1, 0], [0]):
        with pytest.raises(binding.PAError) as e:
            binding.pa_rope_plan([1.0, 0.5], axes)
        assert e.value.code == INVALID
    assert lib.pa_rope_plan(None, None, 3, None) == INVALID
    assert lib.pa_rope_plan(None, None, -1, None) == INVALID


def cross_args(**kw):
    order = ("out", "q", "kv", "bt", "width", "cu", "lens", "S", "total", "maxq", "scale", "hq", "hkv", "d", "nb", "bs", "dt")
    ok = dict(out=P, q=P, kv=P, bt=P, width=4, cu=P, lens=P, S=2, total=10, maxq=8, scale=0.1, hq=8, hkv=2, d=128, nb=16, bs=16,
              dt=0)
    return [dict(ok, **kw)[k] for k in order]


def test_cross_attention_refusals(lib):
    def call(ws=None, ws_bytes=0, flags=0, **kw):
        a = lib.pa_cross_attention(*cross_args(**kw), ws, ws_bytes, flags, None)
        b = lib.pa_cross_attention_fp8(*cross_args(**kw), 0.5, 0.5, ws, ws_bytes, flags, None)
        assert a == b
        return a
    for maxq in (1, 2, 8, 1000):  # the few-row and the many-row form refuse the same
        assert call(maxq=maxq, d=96) == UNSUPPORTED
        assert call(maxq=maxq, dt=2) == UNSUPPORTED
        assert call(maxq=maxq, hq=40, hkv=2) == UNSUPPORTED      # group 20
        assert call(maxq=maxq, hkv=3) == INVALID
        assert call(maxq=maxq, bs=24) == INVALID
        assert call(maxq=maxq, scale=float("inf")) == INVALID
        assert call(maxq=maxq, scale=float("nan")) == INVALID
        assert call(maxq=maxq, nb=0) == INVALID and call(maxq=maxq, width=0) == INVALID
        assert call(maxq=maxq, S=-1) == INVALID and call(maxq=maxq, total=-1) == INVALID
        assert call(maxq=maxq, width=(1 << 26) + 1) == INVALID
        assert call(maxq=maxq, flags=2) == INVALID and "flags" in binding.pa_last_error()
        for name in ("out", "q", "kv", "bt", "cu", "lens"):
            assert call(maxq=maxq, **{name: None}) == INVALID and "null" in binding.pa_last_error(), name
        for name in ("out", "q", "kv"):
            assert call(maxq=maxq, **{name: P + 8}) == INVALID and "misaligned" in binding.pa_last_error(), name
        for name in ("bt", "cu", "lens"):
            assert call(maxq=maxq, **{name: P + 2}) == INVALID and "misaligned" in binding.pa_last_error(), name
        assert call(maxq=maxq, S=0) == binding.PA_OK and call(maxq=maxq, total=0) == binding.PA_OK
    assert call(maxq=0) == binding.PA_OK
    assert call(maxq=-1) == INVALID
    for ks, vs in ((0.0, 1.0), (1.0, -2.0), (float("inf"), 1.0), (1.0, float("nan"))):
        assert lib.pa_cross_attention_fp8(*cross_args(), ks, vs, None, 0, 0, None) == INVALID
        assert "k_scale" in binding.pa_last_error()


def test_cross_attention_workspace_refusals(lib):
    def size(S=2, maxq=64, hq=8, hkv=2, d=128, bs=16, dt=0, cache=0, out=True):
        n = ctypes.c_size_t(99)
        rc = lib.pa_cross_attention_workspace_size(S, maxq, hq, hkv, d, bs, dt, cache, ctypes.byref(n) if out else None)
        assert not out or rc != binding.PA_OK or n.value == 0
        return rc
    assert size(out=False) == INVALID
    assert size(d=96) == UNSUPPORTED and size(hkv=3) == INVALID and size(hq=40) == UNSUPPORTED
    assert size(dt=2) == UNSUPPORTED and size(dt=0, cache=1) == UNSUPPORTED and size(cache=3) == UNSUPPORTED
    assert size(bs=24) == INVALID and size(S=-1) == INVALID and size(maxq=-1) == INVALID
    assert size(S=0) == binding.PA_OK and size(maxq=0) == binding.PA_OK and size(S=0, cache=2) == binding.PA_OK


def test_binding_refuses_host_tensors_before_the_library():
    import torch
    i = torch.zeros(4, dtype=torch.int32)
    h = torch.zeros(4, 8, 64, dtype=torch.float16)
    pool = torch.zeros(2, 4, 16, 2, 64, dtype=torch.float16)
    for call in (lambda: binding.pa_build_step(i.view(2, 2), i[:2], i[:2], i, i[:1], i[:2], i[:1], i[:3], i, i, i[:1], 16),
                 lambda: binding.pa_rope_and_cache(h, h, h[:, :2], h[:, :2], pool, i, i, torch.zeros(32, dtype=torch.int64)),
                 lambda: binding.pa_cross_attention(h, h, pool, i.view(2, 2), i[:3], i[:2], 0.1, 2)):
        with pytest.raises((binding.PAError, RuntimeError, AssertionError)):
            call()

"""Cross attention whose K/V ranges are shared out over the SMs: every call here
is checked to have split them (a workspace of 0xFF bytes is written into).

The split is taken for few work units against tables of many tokens, so these
tables are wide; the sequences in them are short and long. The bound is
test_gpu_cross.py's.
"""
import numpy as np
import pytest

from paged_kv_cache_120_gb300 import binding, workloads

from test_gpu_cross import CrossCase, HEADS, KV, QLEN, dev  # noqa: F401

pytestmark = pytest.mark.gpu

WIDE = 250  # blocks of 16 behind the longest sequence's: 31 tiles
TYPES = [(workloads.F16, False), (workloads.BF16, False), (workloads.F16, True), (workloads.BF16, True)]
IDS = ["f16", "bf16", "f16-fp8", "bf16-fp8"]


class Split(CrossCase):
    def __init__(self, *a, extra_width=WIDE, **kw):
        super().__init__(*a, extra_width=extra_width, **kw)

    def run_split(self, max_q=None, **kw):
        import torch
        ws = binding.cross_attention_workspace(self.q, self.pool, len(self.kv), max_q or self.max_q).fill_(0xFF)
        torch.cuda.synchronize()
        out = self.run(ws, max_q=max_q, **kw)
        torch.cuda.synchronize()
        assert bool((ws != 0xFF).any()), "the K/V ranges were not split"
        return out


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "%dx%dx%d" % h)
def test_ragged_prompts(dev, heads, dtype, fp8):
    # At most four units an SM are shared out: shorter chunks where there are many heads.
    c = Split(dev, dtype, *heads, np.minimum(QLEN, 130 if heads[1] >= 8 else 300), KV, fp8=fp8, seed=sum(heads))
    c.check(c.run_split())


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("heads,most", [((4, 4, 64), 128), ((8, 2, 128), 32), ((32, 1, 128), 8), ((12, 2, 128), 16)],
                         ids=lambda x: "%dx%dx%d" % x if isinstance(x, tuple) else str(x))
def test_chunks_of_one_query_tile(dev, heads, most, dtype, fp8):
    kv = [1, 127, 128, 129, 256, 257, 384, 1000, 0, 1151, 5, 640]
    qlen = [most, 1, most, most - 1, 2, most, 0, most, most, 3, most, most // 2]
    c = Split(dev, dtype, *heads, qlen, kv, fp8=fp8, seed=most + dtype)
    c.check(c.run_split())


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("heads,qlen,kv", [
    ((8, 8, 128), [300] * 6, [4000, 1, 1, 129, 0, 256]), ((2, 1, 64), [40, 1, 7], [1, 5000, 1]),
    ((8, 8, 64), [1] * 18 + [200], [1] * 18 + [6000]), ((8, 8, 128), [100] * 9, [6400, 0, 1, 6400, 1, 1, 1, 1, 130]),
    ((4, 2, 128), [500, 60], [0, 3000])])
def test_shares_of_units_of_one_tile_and_of_many(dev, heads, qlen, kv, dtype, fp8):
    for cut in range(3):
        c = Split(dev, dtype, *heads, qlen, [max(0, n - 128 * cut) if n > 1000 else n for n in kv], fp8=fp8, seed=cut)
        c.check(c.run_split())


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("qlen", [[130, 7, 40, 3], [30, 32, 1, 9]], ids=["pairs", "solo"])
def test_bad_sequences_are_flagged_and_their_rows_left(dev, qlen, dtype, fp8):
    import torch
    c = Split(dev, dtype, 8, 2, 128, qlen, [200, 100, 300, 50], fp8=fp8, seed=12)
    before = c.run_split()
    a, b = int(c.cu[1]), int(c.cu[2])
    for bad in (-1, c.bt.shape[1] * 16 + 1, 2 ** 31 - 1):
        c.kv_d[1] = bad
        out = c.run_split()
        assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN
        assert torch.isnan(out[a:b]).all()
        c.kv_d[1] = 100
        out[a:b] = before[a:b]
        c.check(out)
        c.check(c.run_split())


@pytest.mark.parametrize("cu", [[0, 3, 2, 5], [-2, 1, 2, 4], [0, 1, 90, 91], [0, 2 ** 31 - 1, -5, 3],
                                [0, 2 ** 31 - 2, 2 ** 31 - 1, 3]])
@pytest.mark.parametrize("most", [30, 100])
def test_bad_offsets_are_flagged_and_never_followed(dev, cu, most):
    import torch
    c = Split(dev, workloads.F16, 8, 2, 128, [2, 2, 2], [200, 100, 300], seed=13)
    c.cu_d.copy_(torch.tensor(cu, dtype=torch.int64).to(torch.int32))
    guard = torch.full((c.q.shape[0] + 64,) + c.q.shape[1:], float("nan"), dtype=c.q.dtype, device=dev)
    c.run_split(out=guard[32:32 + c.q.shape[0]], max_q=most)
    assert binding.pa_get_device_error() == binding.PA_DEVERR_SEQ_LEN
    assert torch.isnan(guard[:32]).all() and torch.isnan(guard[-32:]).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["16bit", "fp8"])
@pytest.mark.parametrize("qlen", [[140, 20], [30, 5]], ids=["pairs", "solo"])
def test_bad_blocks_read_as_zeros(dev, qlen, fp8):
    import torch
    c = Split(dev, workloads.BF16, 8, 2, 128, qlen, [200, 100], fp8=fp8, seed=14)
    zeroed = c.pool.view(2, -1, 2, 128)
    slots = torch.from_numpy((int(c.bt[0, 3]) * 16 + np.arange(16)).astype(np.int64)).to(dev)
    keep = zeroed[:, slots].clone()
    zeroed[:, slots] = 0
    c.reference()
    zeroed[:, slots] = keep
    for bad in (c.nb, -1, 2 ** 31 - 1):
        bt = c.bt.copy()
        bt[0, 3] = bad
        c.bt_d.copy_(torch.from_numpy(bt))
        out = c.run_split()
        assert binding.pa_get_device_error() == binding.PA_DEVERR_BLOCK_ID
        c.check(out)


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("qlen", [[130, 7, 40], [30, 7, 32]], ids=["pairs", "solo"])
def test_replayed_from_a_graph_with_new_lengths(dev, qlen, dtype, fp8):
    import torch
    c = Split(dev, dtype, 8, 2, 128, qlen, [600, 900, 300], fp8=fp8, seed=11)
    ws, out = c.workspace(), torch.full_like(c.q, float("nan"))
    c.check(c.run_split(out=out))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        c.run(ws, out=out)
    for kv in ([600, 900, 300], [1, 899, 0], [555, 16, 299], [0, 0, 0], [128, 129, 127]):
        c.kv[:] = kv
        c.kv_d.copy_(torch.from_numpy(c.kv))
        out.fill_(float("nan"))
        ws.fill_(0xFF)
        g.replay()
        c.reference()
        c.check(out)
        assert bool((ws != 0xFF).any())


def test_two_calls_on_two_streams(dev):
    import torch
    a = Split(dev, workloads.F16, 8, 2, 128, [100, 3], [2000, 700], seed=16)
    b = Split(dev, workloads.BF16, 20, 20, 64, [60, 3, 200], [1500, 700, 1], seed=17)
    for c in (a, b):
        c.check(c.run_split())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.full_like(c.q, float("nan")) for c in (a, b)]
    ws = [c.workspace() for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, w, o in zip((a, b), streams, ws, outs):
            c.run(w, stream=s, out=o)
    torch.cuda.synchronize()
    a.check(outs[0])
    b.check(outs[1])

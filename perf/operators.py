"""Cases of the paged cache's step operators: what they read and compute, in plain form and through the library.

Three operators of one serving step on a paged KV cache:
  maps   block tables, lengths, positions and slots of a step, built on the GPU from the requests' lengths
  rope   rotary positions with one or more axes on Q and K, K and V written to the cache by slot
  cross  attention of decoder tokens to all of an encoder's cached states, through block tables
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
K_SCALE, V_SCALE = 0.0125, 0.01  # per-tensor scales of an FP8 cache


def listed():
    return [
        # A decode step of a busy server: one new token for each of 256 sequences.
        dict(name="maps-decode-256", op="maps", seqs=256, block=16, width=512, median=800, chunk=1, idle=0.0, prefill=0.0,
             retire=0.0, capacity=256, spare=1.0),
        # The largest batch, mixed: idle rows, single tokens, prompt chunks, finished rows; the pool runs short.
        dict(name="maps-mixed-4096", op="maps", seqs=4096, block=16, width=256, median=500, chunk=256, idle=0.2, prefill=0.1,
             retire=0.005, capacity=65536, spare=0.5),
        # A few long prompts admitted whole.
        dict(name="maps-prompts-16", op="maps", seqs=16, block=32, width=1024, median=0, chunk=20001, idle=0.0, prefill=1.0,
             retire=0.0, capacity=262144, spare=1.0),
        # One decode step of the 40-head layer: latency.
        dict(name="rope-decode-64", op="rope", tokens=64, hq=40, hkv=40, d=128, rot=128, axes=1, mix=False, adjacent=False,
             fused=False, cache="16", type="f16", block=16, skip=0.0),
        # The 40-head layer's prompt chunk.
        dict(name="rope-chunk-8192", op="rope", tokens=8192, hq=40, hkv=40, d=128, rot=128, axes=1, mix=False, adjacent=False,
             fused=False, cache="16", type="f16", block=16, skip=0.0),
        # Image and video tokens (time, height, width) out of a fused projection, grouped heads; an odd count, some padding.
        dict(name="rope-video-16383", op="rope", tokens=16383, hq=32, hkv=8, d=128, rot=128, axes=3, mix=False, adjacent=False,
             fused=True, cache="16", type="bf16", block=16, skip=0.05),
        # The same into an FP8 cache, axes interleaved over the pairs.
        dict(name="rope-video-fp8-5001", op="rope", tokens=5001, hq=32, hkv=8, d=128, rot=128, axes=3, mix=True, adjacent=False,
             fused=True, cache="fp8", type="bf16", block=16, skip=0.0),
        # Half of a small head rotated, adjacent pairs, one token more than a round number.
        dict(name="rope-partial-1025", op="rope", tokens=1025, hq=16, hkv=4, d=64, rot=32, axes=1, mix=False, adjacent=True,
             fused=True, cache="16", type="f16", block=32, skip=0.0),
        # Speech-like decode: a single token per sequence to 1500 encoder states, every head its own.
        dict(name="cross-decode-64", op="cross", seqs=64, hq=20, hkv=20, d=64, qmin=1, qmax=1, kvmin=1500, kvmax=1500,
             cache="16", type="f16", block=16),
        # Image-like decode of several candidates per request (grouped heads), ragged image lengths, none for some rows.
        dict(name="cross-beams-fp8-48", op="cross", seqs=48, hq=32, hkv=8, d=128, qmin=1, qmax=4, kvmin=0, kvmax=6404,
             cache="fp8", type="bf16", block=16),
        # Prompt chunks against image states: the matrix-bound end.
        dict(name="cross-chunk-8x1024", op="cross", seqs=8, hq=32, hkv=8, d=128, qmin=1024, qmax=1024, kvmin=6404, kvmax=6404,
             cache="16", type="bf16", block=16),
        # Short prompts of many requests, ragged on both sides, small heads.
        dict(name="cross-prompts-40", op="cross", seqs=40, hq=20, hkv=20, d=64, qmin=0, qmax=224, kvmin=1, kvmax=1500,
             cache="16", type="f16", block=32),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["maps", "rope", "cross"])
    if op == "maps":
        seqs = spread(rng, 1, 4096)
        chunk = spread(rng, 1, max(1, min(20001, 262144 // seqs)))
        block = rng.choice([16, 32, 64])
        median = spread(rng, 16, 1000)
        return dict(op="maps", seqs=seqs, block=block, width=(8192 + chunk) // block + 1, median=median, chunk=chunk,
                    idle=rng.choice([0.0, 0.1, 0.3]), prefill=rng.choice([0.0, 0.2, 1.0]), retire=rng.choice([0.0, 0.05, 0.2]),
                    capacity=min(262144, seqs * chunk), spare=rng.choice([0.7, 1.0, 1.0]))
    kind, cache = rng.choice(["f16", "bf16"]), rng.choice(["16", "16", "fp8"])
    hq, hkv, d = rng.choice([(40, 40, 128), (32, 8, 128), (20, 20, 64), (16, 4, 64), (12, 2, 128), (16, 1, 128), (64, 8, 128)])
    if op == "rope":
        axes = rng.choice([1, 1, 2, 3])
        rot = rng.choice([d, d, d // 2])
        most = 8192 * 240 * 128 // ((2 * hq + 4 * hkv) * d)
        return dict(op="rope", tokens=spread(rng, 1, most), hq=hq, hkv=hkv, d=d, rot=rot, axes=axes,
                    mix=axes > 1 and rng.random() < 0.5, adjacent=rng.random() < 0.3, fused=rng.random() < 0.5, cache=cache,
                    type=kind, block=rng.choice([16, 32, 64]), skip=rng.choice([0.0, 0.0, 0.1]))
    seqs, qmax = spread(rng, 1, 128), rng.choice([1, 1, spread(rng, 2, 16), spread(rng, 16, 1024)])
    room = 8 * 1024 * 6404 * 32 * 128 / (seqs * qmax * hq * d)
    memory = 4e9 / (seqs * hkv * d * 4)
    kvmax = spread(rng, 16, int(max(16, min(20000, room, memory))))
    return dict(op="cross", seqs=seqs, hq=hq, hkv=hkv, d=d, qmin=rng.choice([qmax, qmax, 0]), qmax=qmax,
                kvmin=rng.choice([kvmax, 1, 0]), kvmax=kvmax, cache=cache, type=kind, block=rng.choice([16, 32, 64]))


def work(case):
    c = dict(case)
    if c["op"] == "maps":
        tokens = min(c["capacity"], c["seqs"] * (1 - c["idle"] - c["retire"]) * (1 + c["prefill"] * (c["chunk"] - 1) / 2))
        released = c["seqs"] * c["retire"] * c["median"] / c["block"]
        return {"bytes": 16 * c["seqs"] + 8 * c["capacity"] + 8 * tokens / c["block"] + 4 * released, "flops": 10 * tokens}
    if c["op"] == "rope":
        in_cache = 2 if c["cache"] == "16" else 1
        row = 2 * c["hq"] * c["d"] * 2 + (1 - c["skip"]) * 2 * c["hkv"] * c["d"] * (2 + in_cache)
        return {"bytes": c["tokens"] * (row + 4 * c["axes"] + 4), "flops": 6 * c["tokens"] * (c["hq"] + c["hkv"]) * c["rot"] / 2}
    rows, kv = float(even(c["qmin"], c["qmax"], c["seqs"]).sum()), float(even(c["kvmin"], c["kvmax"], c["seqs"]).mean())
    elem = 2 if c["cache"] == "16" else 1
    return {"bytes": 2 * c["seqs"] * kv * c["hkv"] * c["d"] * elem + 4 * rows * c["hq"] * c["d"],
            "flops": 4 * rows * kv * c["hq"] * c["d"]}


def even(lo, hi, n):
    """n whole numbers spread evenly from hi down to lo: prepare() shuffles them, so that a batch's totals are the case's."""
    return np.linspace(hi, lo, n).round().astype(np.int64)


# ------------------------------------------------------------------ inputs

def generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def shuffled(g, values):
    """The given whole numbers in an order of the seed's, on the GPU."""
    return torch.from_numpy(np.asarray(values)).cuda()[torch.randperm(len(values), generator=g, device="cuda")].to(torch.int32)


def tables_of(blocks, width, perm):
    """Tables whose row s holds the next blocks[s] entries of perm, -1 behind them."""
    j = torch.arange(width, device="cuda")
    at = (torch.cumsum(blocks, 0) - blocks)[:, None] + j
    return torch.where(j < blocks[:, None], perm[at.clamp(max=perm.numel() - 1)], -1).to(torch.int32)


def prepare(case, seed):
    return {"maps": prepare_maps, "rope": prepare_rope, "cross": prepare_cross}[case["op"]](dict(case), generator(seed))


def prepare_maps(c, g):
    n, b, width = c["seqs"], c["block"], c["width"]
    # Cached lengths spread as requests' are: lognormal about the median, within the table and leaving room for the chunk.
    normal = torch.special.ndtri((torch.arange(n, dtype=torch.float64) + 0.5) / n).numpy()
    cached = np.clip(np.round(np.exp(normal) * c["median"]), 0, width * b - c["chunk"]).astype(np.int64)
    idle, gone = round(n * c["idle"]), round(n * c["retire"])
    prompts = round((n - idle - gone) * c["prefill"])
    new = np.concatenate([np.zeros(idle), np.full(gone, -1), even(1, c["chunk"], prompts), np.ones(n - idle - gone - prompts)]).astype(np.int64)
    lens, query = shuffled(g, cached), shuffled(g, new)
    held = (lens.long() + b - 1) // b
    need = ((lens + query.clamp(min=0)).long() + b - 1) // b - held
    used, free = int(held.sum()), max(1, int(c["spare"] * int(need.sum())))
    room = int((np.maximum(new, 0) // b + 1).sum()) + 1
    perm = torch.randperm(used + room, generator=g, device="cuda")
    free_list = torch.full((used + room,), -1, dtype=torch.int32, device="cuda")
    free_list[:free] = perm[used:used + free].to(torch.int32)
    out = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(case=c, tables=tables_of(held, width, perm), lens=lens, query=query, free_list=free_list,
                num_free=torch.tensor([free], dtype=torch.int32, device="cuda"), lens_out=out(n), free_out=out(1),
                cu=out(n + 1), positions=out(c["capacity"]), slots=out(c["capacity"]), admitted=out(1))


def pair_axes(c):
    """The axis of each rotary pair: blocks of pairs in turn (time the fewest), or interleaved."""
    pairs = c["rot"] // 2
    i = np.arange(pairs)
    if c["mix"]:
        return (i % c["axes"]).astype(np.int32)
    if c["axes"] == 3:
        return np.where(i < pairs // 4, 0, np.where(i < pairs // 4 + (pairs - pairs // 4) // 2, 1, 2)).astype(np.int32)
    return (i * c["axes"] // pairs).astype(np.int32)


def pool_of(c, blocks, g):
    """A layer's pool of N(0, 1) values; FP8: codes of them under the scales."""
    shape = (2, blocks, c["block"], c["hkv"], c["d"])
    if c["cache"] == "16":
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(DTYPES[c["type"]])
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    x[0] /= K_SCALE
    x[1] /= V_SCALE
    return x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare_rope(c, g):
    t, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["d"]
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32).to(DTYPES[c["type"]])  # noqa: E731
    if c["fused"]:
        qkv = normal(t, hq + 2 * hkv, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = normal(t, hq, d), normal(t, hkv, d), normal(t, hkv, d)
    # Text positions run on from a far start; the other axes walk a 36 x 64 patch grid.
    start = int(torch.randint(0, 130000, (1,), generator=g, device="cuda"))
    i = torch.arange(t, device="cuda")
    walk = [start + i // (1 if c["axes"] == 1 else 2304), start + (i // 64) % 36, start + i % 64]
    positions = torch.stack(walk[:c["axes"]]).to(torch.int32)
    blocks = t // c["block"] + 8
    slots = torch.randperm(blocks * c["block"], generator=g, device="cuda")[:t].to(torch.int32)
    slots = torch.where(torch.rand(t, generator=g, device="cuda") < c["skip"], -1, slots).to(torch.int32)
    freq = 10000.0 ** (-2.0 * np.arange(c["rot"] // 2) / c["rot"])
    return dict(case=c, q=q, k=k, v=v, positions=positions, slots=slots, freq=freq, axes=pair_axes(c),
                freq_gpu=torch.from_numpy(freq).cuda(), axes_gpu=torch.from_numpy(pair_axes(c)).cuda().long(),
                pool=pool_of(c, blocks, g), out=torch.empty(t, hq, d, dtype=DTYPES[c["type"]], device="cuda"))


def prepare_cross(c, g):
    n, d = c["seqs"], c["d"]
    rows, kv = shuffled(g, even(c["qmin"], c["qmax"], n)), shuffled(g, even(c["kvmin"], c["kvmax"], n))
    held = (kv.long() + c["block"] - 1) // c["block"]
    blocks = int(held.sum()) + 4
    perm = torch.randperm(blocks, generator=g, device="cuda")
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    cu[1:] = torch.cumsum(rows, 0)
    total = int(cu[-1])
    query = torch.randn(total, c["hq"], d, generator=g, device="cuda", dtype=torch.float32).to(DTYPES[c["type"]])
    width = max(1, -(-c["kvmax"] // c["block"]))
    return dict(case=c, query=query, cu=cu, kv=kv, tables=tables_of(held, width, perm), pool=pool_of(c, blocks, g),
                out=torch.empty_like(query), scale=d ** -0.5)


# ------------------------------------------------------------------ a pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"maps": own_maps, "rope": own_rope, "cross": own_cross}[op](state)
    return {"maps": plain_maps, "rope": plain_rope, "cross": plain_cross}[op](state)


def own_maps(s):
    from paged_kv_cache_120_gb300 import binding
    binding.pa_build_step(s["tables"], s["lens"], s["query"], s["free_list"], s["num_free"], s["lens_out"], s["free_out"],
                          s["cu"], s["positions"], s["slots"], s["admitted"], s["case"]["block"])
    return dict(tables=s["tables"], lens=s["lens_out"], free_list=s["free_list"], num_free=s["free_out"], cu=s["cu"],
                positions=s["positions"], slots=s["slots"], admitted=s["admitted"])


def plain_maps(s):
    c = s["case"]
    b, width, cap = c["block"], c["width"], c["capacity"]
    lens, query, table, free_list = s["lens"].long(), s["query"].long(), s["tables"].long(), s["free_list"].long()
    n = s["num_free"].long()
    held = (lens + b - 1) // b
    gone = torch.where(query < 0, held, 0)
    released, gone_at = gone.sum(), torch.cumsum(gone, 0) - gone
    want = query.clamp(min=0)
    need = (lens + want + b - 1) // b - held
    fits = (torch.cumsum(need, 0) <= n + released) & (torch.cumsum(want, 0) <= cap)
    want, need = torch.where(fits, want, 0), torch.where(fits, need, 0)
    cu = torch.nn.functional.pad(torch.cumsum(want, 0), (1, 0))
    first = torch.cumsum(need, 0) - need
    taken = need.sum()
    # The stack: the free blocks, then each finished row's in reverse order.
    j = torch.arange(width, device="cuda")
    at = torch.where(j < gone[:, None], n + gone_at[:, None] + gone[:, None] - 1 - j, free_list.numel())
    stack = torch.nn.functional.pad(free_list, (0, 1)).scatter(0, at.reshape(-1), table.reshape(-1))
    new = (j >= held[:, None]) & (j < (held + need)[:, None])
    pop = (n + released - 1 - (first[:, None] + j - held[:, None])).clamp(0, free_list.numel())
    table = torch.where(new, stack[pop], table)
    left = n + released - taken
    i = torch.arange(free_list.numel(), device="cuda")
    free_list = torch.where((i >= n) & (i < left), stack[:-1], free_list)
    t = torch.arange(cap, device="cuda")
    row = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=c["seqs"] - 1)
    live = t < cu[-1]
    pos = torch.where(live, lens[row] + t - cu[row], 0)
    slots = torch.where(live, table[row, (pos // b).clamp(max=width - 1)] * b + pos % b, -1)
    small = lambda x: x.to(torch.int32)  # noqa: E731
    return dict(tables=small(table), lens=small(torch.where(query < 0, 0, lens + want)), free_list=small(free_list),
                num_free=small(left), cu=small(cu), positions=small(pos), slots=small(slots), admitted=small(fits.sum().reshape(1)))


def own_rope(s):
    from paged_kv_cache_120_gb300 import binding
    c = s["case"]
    if "plan" not in s:  # a program makes it once per model
        s["plan"] = binding.rope_plan(s["freq"], s["axes"], device="cuda")
    if c["cache"] == "16":
        binding.pa_rope_and_cache(s["out"], s["q"], s["k"], s["v"], s["pool"], s["slots"], s["positions"], s["plan"],
                                  adjacent=c["adjacent"])
        return dict(query=s["out"], cache=s["pool"])
    binding.pa_rope_and_cache_fp8(s["out"], s["q"], s["k"], s["v"], s["pool"], s["slots"], s["positions"], s["plan"],
                                  K_SCALE, V_SCALE, adjacent=c["adjacent"])
    return dict(query=s["out"], cache=s["pool"].view(torch.float8_e4m3fn))


def turned(x, cos, sin, rot, adjacent):
    """The first rot of the last dimension turned pair by pair, in x's type."""
    a, rest = x[..., :rot], x[..., rot:]
    x1, x2 = (a[..., 0::2], a[..., 1::2]) if adjacent else (a[..., :rot // 2], a[..., rot // 2:])
    y1, y2 = x1 * cos - x2 * sin, x1 * sin + x2 * cos
    y = torch.stack([y1, y2], -1).flatten(-2) if adjacent else torch.cat([y1, y2], -1)
    return torch.cat([y, rest], -1)


def plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[s["axes_gpu"]].T * s["freq_gpu"]  # [tokens, pairs], far positions: 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q = turned(s["q"].float(), cos, sin, c["rot"], c["adjacent"]).to(s["q"].dtype)
    k, v = turned(s["k"].float(), cos, sin, c["rot"], c["adjacent"]), s["v"].float()
    pool = s["pool"]
    flat = pool.view(2, -1, c["hkv"], c["d"])
    if c["cache"] == "16":
        k, v = k.to(pool.dtype), v.to(pool.dtype)
    else:
        code = lambda x, scale: (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        k, v = code(k, K_SCALE), code(v, V_SCALE)
    live = (s["slots"] >= 0)[:, None, None]
    slots = s["slots"].long().clamp(min=0)
    spare = flat.shape[1]  # padded tokens go behind the pool
    slots = torch.where(live[:, 0, 0], slots, spare)
    wide = torch.cat([flat, flat[:, :1]], 1)
    wide[0].index_copy_(0, slots, k)
    wide[1].index_copy_(0, slots, v)
    cache = wide[:, :-1].reshape(pool.shape)
    return dict(query=q, cache=cache if c["cache"] == "16" else cache.view(torch.float8_e4m3fn))


def own_cross(s):
    from paged_kv_cache_120_gb300 import binding
    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = binding.cross_attention_workspace(s["query"], s["pool"], c["seqs"], c["qmax"])
    if c["cache"] == "16":
        binding.pa_cross_attention(s["out"], s["query"], s["pool"], s["tables"], s["cu"], s["kv"], s["scale"], c["qmax"],
                                   s["workspace"])
    else:
        binding.pa_cross_attention_fp8(s["out"], s["query"], s["pool"], s["tables"], s["cu"], s["kv"], s["scale"], c["qmax"],
                                       K_SCALE, V_SCALE, s["workspace"])
    return s["out"]


def plain_cross(s):
    c = s["case"]
    n, hq, hkv, d, b = c["seqs"], c["hq"], c["hkv"], c["d"], c["block"]
    group, query, total = hq // hkv, s["query"], s["query"].shape[0]
    i = torch.arange(max(1, c["kvmax"]), device="cuda")
    inside = i < s["kv"][:, None]
    slots = torch.where(inside, s["tables"].long()[:, i // b] * b + i % b, 0)
    flat = s["pool"].view(2, -1, hkv, d)
    flat = flat if c["cache"] == "16" else flat.view(torch.float8_e4m3fn)
    k = flat[0][slots].float().permute(0, 2, 3, 1)   # [n, hkv, d, kv]
    v = flat[1][slots].float().permute(0, 2, 1, 3)   # [n, hkv, kv, d]
    k, v = (k, v) if c["cache"] == "16" else (k * K_SCALE, v * V_SCALE)
    t = torch.arange(total, device="cuda")
    seq = torch.searchsorted(s["cu"], t.int(), right=True) - 1
    at = t - s["cu"].long()[seq]
    q = torch.zeros(n, c["qmax"], hq, d, device="cuda")
    q[seq, at] = query.float()
    q = q.view(n, c["qmax"], hkv, group, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * c["qmax"], d)
    p = torch.matmul(q, k).mul_(s["scale"]).masked_fill_(~inside[:, None, None], -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(n, hkv, group, c["qmax"], d).permute(0, 3, 1, 2, 4).reshape(n, c["qmax"], hq, d)
    return o[seq, at].to(query.dtype)


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "maps":
        return exact_maps(s, c)
    if c["op"] == "rope":
        return exact_rope(s, c)
    flat = s["pool"].view(2, -1, c["hkv"], c["d"])
    out = torch.zeros(s["query"].shape, dtype=torch.float64, device="cuda")
    cu, kv, tables = s["cu"].tolist(), s["kv"].tolist(), s["tables"].long()
    scales = (1.0, 1.0) if c["cache"] == "16" else (K_SCALE, V_SCALE)
    group = c["hq"] // c["hkv"]
    for n in range(c["seqs"]):
        if cu[n] == cu[n + 1] or kv[n] == 0:
            continue
        i = torch.arange(kv[n], device="cuda")
        rows = flat[:, tables[n, i // c["block"]] * c["block"] + i % c["block"]]
        rows = rows if c["cache"] == "16" else rows.view(torch.float8_e4m3fn).float()
        for h in range(c["hkv"]):
            k, v = rows[0, :, h].double() * scales[0], rows[1, :, h].double() * scales[1]
            heads = slice(h * group, (h + 1) * group)
            q = s["query"][cu[n]:cu[n + 1], heads].double()
            w = torch.softmax(torch.einsum("qgd,td->qgt", q, k) * s["scale"], -1)
            out[cu[n]:cu[n + 1], heads] = torch.einsum("qgt,td->qgd", w, v)
    return out


def exact_rope(s, c):
    freq, axes = s["freq"], s["axes"]
    position = s["positions"].cpu().numpy().astype(np.float64)
    turn = torch.polar(torch.ones(c["tokens"], c["rot"] // 2, dtype=torch.float64),
                       torch.from_numpy(position[axes].T * freq)).cuda()[:, None]

    def rotated(x):
        y = x.double().clone()
        half = c["rot"] // 2
        at = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["adjacent"] else (slice(0, half), slice(half, c["rot"]))
        z = torch.complex(y[..., at[0]], y[..., at[1]]) * turn
        y[..., at[0]], y[..., at[1]] = z.real, z.imag
        return y

    k, v, pool = rotated(s["k"]), s["v"].double(), s["pool"]
    if c["cache"] == "fp8":
        k, v, pool = (k / K_SCALE).clamp(-448, 448), (v / V_SCALE).clamp(-448, 448), pool.view(torch.float8_e4m3fn).float()
    cache = pool.double().view(2, -1, c["hkv"], c["d"]).clone()
    live = s["slots"] >= 0
    at = s["slots"][live].long()
    cache[0][at], cache[1][at] = k[live], v[live]
    return dict(query=rotated(s["q"]), cache=cache.view(pool.shape))


def exact_maps(s, c):
    b, cap = c["block"], c["capacity"]
    tables, lens = s["tables"].cpu().numpy().copy(), s["lens"].cpu().numpy().astype(np.int64)
    query, out = s["query"].cpu().numpy(), s["free_list"].cpu().numpy().copy()
    stack = out[:int(s["num_free"])].tolist()
    free = len(stack)
    for n in np.nonzero(query < 0)[0]:
        stack += tables[n, :-(-lens[n] // b)][::-1].tolist()
    cu, slots, positions = [0], np.full(cap, -1, np.int32), np.zeros(cap, np.int32)
    after, admitted = lens.copy(), c["seqs"]
    for n in range(c["seqs"]):
        want, held = max(0, int(query[n])), -(-int(lens[n]) // b)
        need = -(-(int(lens[n]) + want) // b) - held
        if admitted < c["seqs"] or need > len(stack) or cu[-1] + want > cap:
            admitted, want = min(admitted, n), 0
        if want:
            if need:
                tables[n, held:held + need] = stack[len(stack) - need:][::-1]
                del stack[len(stack) - need:]
            at = np.arange(lens[n], lens[n] + want)
            positions[cu[-1]:cu[-1] + want] = at
            slots[cu[-1]:cu[-1] + want] = tables[n, at // b] * b + at % b
        after[n] = 0 if query[n] < 0 else lens[n] + want
        cu.append(cu[-1] + want)
    if len(stack) > free:
        out[free:len(stack)] = stack[free:]
    small = lambda x: np.asarray(x, np.int32)  # noqa: E731
    return dict(tables=tables, lens=small(after), free_list=out, num_free=small([len(stack)]), cu=small(cu), positions=positions,
                slots=slots, admitted=small([admitted]))

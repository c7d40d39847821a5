"""Cases of the paged cache's speculative step: a tree of drafted tokens per sequence, in plain form and through the library.

Four operators of one step that checks drafted tokens against a model, over a paged KV cache:
  maps     positions and ancestor masks of the trees, from each node's parent
  attend   attention of the tree's tokens to the cached context and to their ancestors, through block tables
  verify   which drafted tokens the target's rows accept, and the token drawn behind them, from given random numbers
  commit   the accepted tokens' K and V moved into place in every layer, lengths cut, surplus blocks returned
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
K_SCALE, V_SCALE = 0.0125, 0.01  # per-tensor scales of an FP8 cache


def listed():
    return [
        # The trees of a busy server's step, some rows idle.
        dict(name="maps-trees-256", op="maps", seqs=256, qmin=0, qmax=64, fan=8, ctx=2000),
        # A few long single-file drafts and wide ones: the deepest and the widest masks.
        dict(name="maps-long-16", op="maps", seqs=16, qmin=500, qmax=1000, fan=2, ctx=30000),
        # Three drafted tokens behind the last one, in single file, over the 40-head layer.
        dict(name="attend-chain-64", op="attend", seqs=64, hq=40, hkv=40, d=128, qmin=4, qmax=4, fan=1, ctxmin=24, ctxmax=2048,
             cache="16", type="f16", block=16),
        # Full trees of a large batch, grouped heads: reading and matrix work weigh the same.
        dict(name="attend-trees-64", op="attend", seqs=64, hq=32, hkv=8, d=128, qmin=64, qmax=64, fan=8, ctxmin=4096, ctxmax=4096,
             cache="16", type="bf16", block=16),
        # Trees of uneven sizes and contexts, some of them empty, over an FP8 cache.
        dict(name="attend-fp8-48", op="attend", seqs=48, hq=32, hkv=8, d=128, qmin=0, qmax=25, fan=4, ctxmin=0, ctxmax=8191,
             cache="fp8", type="bf16", block=16),
        # One user with a long context: latency.
        dict(name="attend-one-33", op="attend", seqs=1, hq=32, hkv=8, d=128, qmin=33, qmax=33, fan=4, ctxmin=32001, ctxmax=32001,
             cache="16", type="bf16", block=16),
        # Small heads, every one its own, ragged.
        dict(name="attend-small-40", op="attend", seqs=40, hq=20, hkv=20, d=64, qmin=1, qmax=25, fan=3, ctxmin=1, ctxmax=1500,
             cache="16", type="f16", block=32),
        # One user, no randomness: the most likely token of each row of logits.
        dict(name="verify-greedy-1", op="verify", seqs=1, qmin=32, qmax=32, fan=4, vocab=131072, type="bf16", mode="greedy"),
        # Five drafted tokens per sequence, drawn from a smaller model whose rows are given.
        dict(name="verify-chain-256", op="verify", seqs=256, qmin=6, qmax=6, fan=1, vocab=32000, type="f32", mode="draft"),
        # Trees whose children are the drafter's most likely tokens; an odd vocabulary.
        dict(name="verify-trees-48", op="verify", seqs=48, qmin=1, qmax=24, fan=3, vocab=100003, type="f32", mode="sample"),
        # A batch's accepted tokens moved in all 40 layers of the 40-head model.
        dict(name="commit-40x64", op="commit", seqs=64, layers=40, hkv=40, d=128, qmin=32, qmax=32, amax=7, ctxmax=24,
             cache="16", type="f16", block=16),
        # One user's, grouped heads, FP8: latency.
        dict(name="commit-32x1", op="commit", seqs=1, layers=32, hkv=8, d=128, qmin=63, qmax=63, amax=5, ctxmax=500,
             cache="fp8", type="bf16", block=16),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(40, 40, 128), (32, 8, 128), (20, 20, 64), (16, 4, 64), (12, 2, 128), (16, 1, 128), (64, 8, 128)]


def draw(rng):
    op = rng.choice(["maps", "attend", "attend", "verify", "commit"])
    if op == "maps":
        qmax = spread(rng, 1, 1000)
        return dict(op="maps", seqs=spread(rng, 1, min(1024, max(1, 16 * 1000 * 1000 // (qmax * qmax)))), qmin=rng.choice([qmax, 1, 0]),
                    qmax=qmax, fan=rng.choice([1, 2, 4, 8, 1000]), ctx=spread(rng, 1, 30000))
    if op == "attend":
        hq, hkv, d = rng.choice(HEADS)
        qmax = rng.choice([spread(rng, 1, 16), spread(rng, 8, 64), spread(rng, 32, 256)])
        seqs = spread(rng, 1, min(128, 4096 // qmax))
        room = 64 * 64 * 4096 * 32 * 128 / (seqs * qmax * hq * d) - qmax
        memory = 2e9 / (seqs * hkv * d * 4)
        ctxmax = spread(rng, 16, int(max(16, min(32000, room, memory))))
        return dict(op="attend", seqs=seqs, hq=hq, hkv=hkv, d=d, qmin=rng.choice([qmax, 1, 0]), qmax=qmax,
                    fan=rng.choice([1, 2, 4, 8]), ctxmin=rng.choice([ctxmax, 1, 0]), ctxmax=ctxmax,
                    cache=rng.choice(["16", "16", "fp8"]), type=rng.choice(["f16", "bf16"]), block=rng.choice([16, 32, 64]))
    if op == "verify":
        mode = rng.choice(["greedy", "sample", "draft", "draft"])
        vocab = spread(rng, 500, 160000)
        most = min(256 * 6 * 32000 // vocab, 4096)  # rows
        qmax = spread(rng, 1, min(48, max(1, most)))
        fan = rng.choice([1, 2, 3, 4])
        return dict(op="verify", seqs=spread(rng, 1, max(1, min(512, most // qmax))), qmin=rng.choice([qmax, 1, 0]), qmax=qmax,
                    fan=fan, vocab=vocab, type=rng.choice(["f32", "f32", "bf16", "f16"]), mode=mode)
    cache = rng.choice(["16", "16", "fp8"])
    _, hkv, d = rng.choice(HEADS)
    qmax = spread(rng, 1, 64)
    layers = spread(rng, 1, 60)
    most = 40 * 64 * 40 * 128 * 60 / (layers * hkv * d * (qmax + 80))
    return dict(op="commit", seqs=spread(rng, 1, int(max(1, min(256, most)))), layers=layers, hkv=hkv, d=d,
                qmin=rng.choice([qmax, 1, 0]), qmax=qmax, amax=spread(rng, 1, min(9, qmax)), ctxmax=spread(rng, 1, 64), cache=cache,
                type=rng.choice(["f16", "bf16"]), block=rng.choice([16, 32, 64]))


def even(lo, hi, n):
    """n whole numbers spread evenly from hi down to lo: prepare() shuffles them, so that a batch's totals are the case's."""
    return np.linspace(hi, lo, n).round().astype(np.int64)


def work(case):
    c = dict(case)
    nodes = even(c["qmin"], c["qmax"], c["seqs"])
    total = float(nodes.sum())
    if c["op"] == "maps":
        words = -(-c["qmax"] // 32)
        return {"bytes": 4 * total * (2 + words) + 8 * c["seqs"], "flops": total}
    if c["op"] == "attend":
        kv = float(even(c["ctxmin"], c["ctxmax"], c["seqs"]).mean()) + total / c["seqs"]
        elem = 2 if c["cache"] == "16" else 1
        return {"bytes": 2 * c["seqs"] * kv * c["hkv"] * c["d"] * elem + 4 * total * c["hq"] * c["d"] + 4 * total,
                "flops": 4 * total * kv * c["hq"] * c["d"]}
    if c["op"] == "verify":
        # A row of the target for each accepted token, and the next token's; of both models where the drafter's are given,
        # but then only of the last one. About two drafted tokens are accepted where there are as many.
        elem = 4 if c["type"] == "f32" else 2
        rows = 2.0 if c["mode"] == "draft" else float(np.minimum(nodes, 3).mean())
        return {"bytes": c["seqs"] * rows * c["vocab"] * elem + 24 * total, "flops": 2 * c["seqs"] * rows * c["vocab"]}
    row = 2 * c["hkv"] * c["d"] * (2 if c["cache"] == "16" else 1)
    moved = float(accepted_of(c, nodes)[1].sum())
    return {"bytes": 2 * moved * row * c["layers"] + 8 * total + 12 * c["seqs"], "flops": 0}


def accepted_of(c, nodes):
    """(accepted nodes, moved tokens) of the sequences of commit, in the order of their nodes."""
    n = np.minimum(even(1, c["amax"], c["seqs"])[::-1], np.maximum(nodes - 1, np.minimum(nodes, 1)))
    return n, np.maximum(n - 1, 0)


# ------------------------------------------------------------------ inputs

def generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).cuda()


def tables_of(blocks, width, perm):
    """Tables whose row s holds the next blocks[s] entries of perm, -1 behind them."""
    j = np.arange(width)
    at = (np.cumsum(blocks) - blocks)[:, None] + j
    return np.where(j < blocks[:, None], perm[np.minimum(at, len(perm) - 1)], -1)


def trees(c, rng):
    """Node counts and parents [seqs, qmax] of random trees: a node hangs below one of the `fan` before it."""
    nodes = rng.permutation(even(c["qmin"], c["qmax"], c["seqs"]))
    i = np.arange(c["qmax"])
    parent = i - 1 - np.floor(rng.random((c["seqs"], c["qmax"])) * np.minimum(i, c["fan"])).astype(np.int64)
    return nodes, parent


def offsets(nodes):
    return np.concatenate([[0], np.cumsum(nodes)])


def ragged(a, nodes):
    """The first nodes[s] entries of each row s, laid end to end."""
    return a[np.arange(a.shape[1]) < nodes[:, None]]


def pool_of(c, blocks, g):
    """A layer's pool of N(0, 1) values; FP8: codes of them under the scales."""
    x = torch.randn((2, blocks, c["block"], c["hkv"], c["d"]), generator=g, device="cuda", dtype=torch.float32)
    if c["cache"] == "16":
        return x.to(DTYPES[c["type"]])
    x[0] /= K_SCALE
    x[1] /= V_SCALE
    return x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    c = dict(case)
    make = {"maps": prepare_maps, "attend": prepare_attend, "verify": prepare_verify, "commit": prepare_commit}[c["op"]]
    return dict(make(c, generator(seed), np.random.default_rng(seed)), case=c)


def prepare_maps(c, g, rng):
    nodes, parent = trees(c, rng)
    context = rng.integers(0, c["ctx"] + 1, c["seqs"])
    total, words = int(nodes.sum()), -(-c["qmax"] // 32)
    return dict(parents=ints(ragged(parent, nodes)), cu=ints(offsets(nodes)), lens=ints(context + nodes),
                positions=torch.empty(total, dtype=torch.int32, device="cuda"),
                masks=torch.empty(total, words, dtype=torch.int32, device="cuda"))


def prepare_attend(c, g, rng):
    nodes, parent = trees(c, rng)
    length = rng.permutation(even(c["ctxmin"], c["ctxmax"], c["seqs"])) + nodes
    held = -(-length // c["block"])
    blocks = int(held.sum()) + 4
    width = max(1, -(-(c["ctxmax"] + c["qmax"]) // c["block"]))
    total = int(nodes.sum())
    query = torch.randn(total, c["hq"], c["d"], generator=g, device="cuda", dtype=torch.float32).to(DTYPES[c["type"]])
    parents, cu = ints(ragged(parent, nodes)), ints(offsets(nodes))
    masks = packed(closure(padded(parents, cu, c["qmax"], -1)))
    seq, at = where_of(cu, total)
    return dict(query=query, cu=cu, lens=ints(length), tables=ints(tables_of(held, width, rng.permutation(blocks))),
                masks=masks[seq, at].contiguous(), pool=pool_of(c, blocks, g), out=torch.empty_like(query), scale=c["d"] ** -0.5)


def prepare_verify(c, g, rng):
    nodes, parent = trees(c, rng)
    total, v, kind = int(nodes.sum()), c["vocab"], DTYPES[c["type"]]
    flat, cu = ints(ragged(parent, nodes)), ints(offsets(nodes))
    seq, at = where_of(cu, total)
    parents = padded(flat, cu, c["qmax"], -1)
    above = cu.long()[seq] + flat.long().clamp(min=0)  # the parent's row
    rank = (parents[:, None] == parents[:, :, None]).tril(-1).sum(-1)[seq, at]  # elder siblings
    logits = torch.randn(total, v, generator=g, device="cuda") * 4
    guess = torch.randn(total, v, generator=g, device="cuda").mul_(0.7).add_(logits)  # the smaller model's logits
    tokens = torch.empty(total, dtype=torch.int32, device="cuda")
    for lo in range(0, total, 512):
        rows = guess[above[lo:lo + 512]]
        if c["mode"] == "draft":  # drawn from the drafter's row
            noise = torch.rand(rows.shape, generator=g, device="cuda").clamp_(1e-20, 1 - 1e-7)
            tokens[lo:lo + 512] = (rows - torch.log(-torch.log(noise))).argmax(-1)
        else:  # its most likely ones
            top = rows.topk(min(v, c["fan"]), -1).indices
            tokens[lo:lo + 512] = top.gather(1, rank[lo:lo + 512, None].clamp(max=top.shape[1] - 1))[:, 0]
    softmax = lambda x: torch.exp(x - x.amax(-1, keepdim=True)).div_(torch.exp(x - x.amax(-1, keepdim=True)).sum(-1, keepdim=True))  # noqa: E731
    target = (logits if c["mode"] == "greedy" else softmax(logits)).to(kind)
    draft = softmax(guess).to(kind) if c["mode"] == "draft" else None
    uniforms = torch.rand(total, 2, generator=g, device="cuda") if c["mode"] != "greedy" else None
    out = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(parents=flat, cu=cu, tokens=tokens, target=target, draft=draft, uniforms=uniforms, count=out(c["seqs"]),
                path=out(total), chosen=out(total))


def prepare_commit(c, g, rng):
    order = rng.permutation(c["seqs"])
    nodes = even(c["qmin"], c["qmax"], c["seqs"])
    accepted = accepted_of(c, nodes)[0][order]
    nodes = nodes[order]
    length = rng.integers(0, c["ctxmax"] + 1, c["seqs"]) + nodes
    held = -(-length // c["block"])
    used = int(held.sum())
    width = max(1, -(-(c["ctxmax"] + c["qmax"]) // c["block"]))
    blocks = c["seqs"] * width + 5
    perm = rng.permutation(blocks - 1)  # the last block is nobody's
    path = np.full((c["seqs"], max(1, c["qmax"])), -1)
    for s, k in enumerate(accepted):
        if k > 0:
            path[s, 0] = 0
        if k > 1:
            path[s, 1:k] = 2 + np.sort(rng.permutation(nodes[s] - 2)[:k - 1])
    free_list = np.full(blocks, -1)
    free_list[:blocks - 1 - used] = perm[used:]
    out = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(pools=[pool_of(c, blocks, g) for _ in range(c["layers"])], tables=ints(tables_of(held, width, perm)),
                cu=ints(offsets(nodes)), lens=ints(length), count=ints(accepted), path=ints(ragged(path, nodes)),
                free_list=ints(free_list), num_free=ints(np.array([blocks - 1 - used])), lens_out=out(c["seqs"]), free_out=out(1))


# ------------------------------------------------------------------ a pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"maps": own_maps, "attend": own_attend, "verify": own_verify, "commit": own_commit}[op](state)
    return {"maps": plain_maps, "attend": plain_attend, "verify": plain_verify, "commit": plain_commit}[op](state)


def where_of(cu, total):
    """The sequence of each node and its place there."""
    t = torch.arange(total, device="cuda")
    seq = torch.searchsorted(cu, t.int(), right=True) - 1
    return seq, t - cu.long()[seq]


def padded(flat, cu, width, fill):
    """Rows of the sequences' nodes, `fill` behind them."""
    j = torch.arange(max(1, width), device="cuda")
    at = cu.long()[:-1, None] + j
    inside = at < cu.long()[1:, None]
    return torch.where(inside, torch.nn.functional.pad(flat.long(), (0, 1))[torch.where(inside, at, flat.numel())], fill)


def closure(parents):
    """[S, Q, Q]: whether node j is node i or one of its ancestors, by doubling the way up."""
    s, q = parents.shape
    none = torch.full((s, 1), q, dtype=torch.int64, device="cuda")
    up = torch.cat([torch.where(parents < 0, q, parents), none], 1)  # node q: above every root
    seen = torch.zeros(s, q + 1, q, dtype=torch.bool, device="cuda")
    seen[:, :q] = torch.eye(q, dtype=torch.bool, device="cuda")
    for _ in range(max(1, q - 1).bit_length()):
        seen = seen | seen.gather(1, up[:, :, None].expand(-1, -1, q))
        up = up.gather(1, up)
    return seen[:, :q]


def packed(bits):
    """The truth values of the last dimension as words of 32, the first the lowest bit."""
    words = -(-bits.shape[-1] // 32)
    wide = torch.nn.functional.pad(bits.long(), (0, 32 * words - bits.shape[-1])).unflatten(-1, (words, 32))
    value = (wide << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(value >= 1 << 31, value - (1 << 32), value).to(torch.int32)


def unpacked(words, n):
    return ((words.long()[..., None] >> torch.arange(32, device="cuda")) & 1).bool().flatten(-2)[..., :n]


def own_maps(s):
    from paged_kv_cache_120_gb300 import binding
    binding.pa_build_tree(s["parents"], s["cu"], s["lens"], s["positions"], s["masks"])
    return dict(positions=s["positions"], masks=s["masks"])


def plain_maps(s):
    c, cu = s["case"], s["cu"]
    total = s["parents"].numel()
    seen = closure(padded(s["parents"], cu, c["qmax"], -1))
    seq, at = where_of(cu, total)
    depth = seen.sum(-1)[seq, at] - 1
    first = (s["lens"] - (cu[1:] - cu[:-1])).long()[seq]
    return dict(positions=(first + depth).to(torch.int32), masks=packed(seen)[seq, at])


def own_attend(s):
    from paged_kv_cache_120_gb300 import binding
    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = binding.tree_attention_workspace(s["query"], s["pool"], c["seqs"], c["qmax"])
    if c["cache"] == "16":
        binding.pa_tree_attention(s["out"], s["query"], s["pool"], s["tables"], s["cu"], s["lens"], s["masks"], s["scale"],
                                  c["qmax"], s["workspace"])
    else:
        binding.pa_tree_attention_fp8(s["out"], s["query"], s["pool"], s["tables"], s["cu"], s["lens"], s["masks"], s["scale"],
                                      c["qmax"], K_SCALE, V_SCALE, s["workspace"])
    return s["out"]


def plain_attend(s):
    c = s["case"]
    n, hq, hkv, d, b, query = c["seqs"], c["hq"], c["hkv"], c["d"], c["block"], s["query"]
    qmax, group, total = max(1, c["qmax"]), hq // hkv, query.shape[0]
    i = torch.arange(max(1, c["ctxmax"] + c["qmax"]), device="cuda")
    slots = torch.where(i < s["lens"][:, None], s["tables"].long()[:, i // b] * b + i % b, 0)
    flat = s["pool"].view(2, -1, hkv, d)
    flat = flat if c["cache"] == "16" else flat.view(torch.float8_e4m3fn)
    k = flat[0][slots].float().permute(0, 2, 3, 1)   # [n, hkv, d, kv]
    v = flat[1][slots].float().permute(0, 2, 1, 3)   # [n, hkv, kv, d]
    k, v = (k, v) if c["cache"] == "16" else (k * K_SCALE, v * V_SCALE)
    seq, at = where_of(s["cu"], total)
    q = torch.zeros(n, qmax, hq, d, device="cuda")
    q[seq, at] = query.float()
    q = q.view(n, qmax, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * qmax, d)
    # Token i of the sequence is node i - context of its tree.
    tree = torch.zeros(n, qmax, 32 * s["masks"].shape[1], dtype=torch.bool, device="cuda")
    tree[seq, at] = unpacked(s["masks"], tree.shape[-1])
    context = (s["lens"] - (s["cu"][1:] - s["cu"][:-1]))[:, None]
    node = (i - context).clamp(0, tree.shape[-1] - 1)[:, None].expand(-1, qmax, -1)
    seen = ((i < context)[:, None] | tree.gather(2, node)) & (i < s["lens"][:, None])[:, None]
    p = torch.matmul(q, k).mul_(s["scale"]).view(n, hkv, group, qmax, -1).masked_fill_(~seen[:, None, None], -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True).clamp(min=-3e38)).exp_().view(n, hkv, group * qmax, -1)
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(n, hkv, group, qmax, d).permute(0, 3, 1, 2, 4).reshape(n, qmax, hq, d)
    return o[seq, at].to(query.dtype)


def own_verify(s):
    from paged_kv_cache_120_gb300 import binding
    binding.pa_verify_draft(s["count"], s["path"], s["chosen"], s["tokens"], s["parents"], s["cu"], s["target"], s["draft"],
                            s["uniforms"])
    return dict(count=s["count"], path=s["path"], chosen=s["chosen"])


def plain_verify(s):
    """All sequences go down their trees in step; sums and comparisons in 64 bits, where a draw next to a border is decided."""
    c, cu = s["case"], s["cu"].long()
    n, width, total = c["seqs"], max(1, c["qmax"]), s["parents"].numel()
    if total == 0:
        return dict(count=torch.zeros(n, dtype=torch.int32, device="cuda"), path=s["path"], chosen=s["chosen"])
    parents, tokens = padded(s["parents"], s["cu"], width, -2), s["tokens"].long()
    rank = (parents[:, None] == parents[:, :, None]).tril(-1).sum(-1)
    seq, at = where_of(s["cu"], total)
    below = cu[seq] + s["parents"].long().clamp(min=0)
    # The rows of each node's children in order, -1 behind them.
    kids = torch.full((total + 1, width), -1, device="cuda")
    kids[torch.where(s["parents"] >= 0, below, total), rank[seq, at]] = torch.arange(total, device="cuda")
    row, live = cu[:-1].clamp(max=total - 1), cu[1:] > cu[:-1]
    count = torch.zeros(n, dtype=torch.int64, device="cuda")
    path, chosen = torch.full((n, width), -1, device="cuda"), torch.full((n, width), -1, device="cuda")
    pick = lambda x, i: x.gather(1, i[:, None])[:, 0]  # noqa: E731
    for step in range(width):
        path[:, step] = torch.where(live, row - cu[:-1], -1)
        count += live
        p, after = s["target"][row].double(), torch.full((n,), -1, device="cuda")
        if c["mode"] == "greedy":
            token = torch.where(p == p.amax(-1, keepdim=True), torch.arange(c["vocab"], device="cuda"), c["vocab"]).amin(-1)
        else:
            w, q = p, None
            if c["mode"] == "draft":
                q = s["draft"][row].double()
                gone, left = torch.zeros(n, dtype=torch.float64, device="cuda"), torch.ones(n, dtype=torch.float64, device="cuda")
                for j in range(min(width, c["fan"])):
                    kid = kids[row, j]
                    x = tokens[kid.clamp(min=0)]
                    waits = (kid >= 0) & (after < 0)
                    fits = s["uniforms"][kid.clamp(min=0), 0].double() * pick(q, x) * left < pick(w, x)
                    after = torch.where(waits & fits, kid, after)
                    refused = waits & ~fits
                    gone = torch.where(refused, gone + left, gone)
                    w = torch.where(refused[:, None], (p - gone[:, None] * q).clamp(min=0), w)
                    left = torch.where(refused, w.sum(-1), left)
                w = torch.where((w.sum(-1) > 0)[:, None], w, p)
            sums = torch.cumsum(w, -1)
            token = (sums <= (s["uniforms"][row, 1].double() * sums[:, -1])[:, None]).sum(-1).clamp(max=c["vocab"] - 1)
        if c["mode"] != "draft":
            for j in range(min(width, c["fan"])):
                kid = kids[row, j]
                after = torch.where((kid >= 0) & (after < 0) & (tokens[kid.clamp(min=0)] == token), kid, after)
        goes = live & (after >= 0)
        chosen[:, step] = torch.where(live, torch.where(goes, tokens[after.clamp(min=0)], token), -1)
        live, row = goes, torch.where(goes, after, row)
    small = lambda x: x.to(torch.int32)  # noqa: E731
    return dict(count=small(count), path=small(path[seq, at]), chosen=small(chosen[seq, at]))


def own_commit(s):
    from paged_kv_cache_120_gb300 import binding
    binding.pa_commit_draft(s["pools"], s["tables"], s["cu"], s["lens"], s["count"], s["path"], s["lens_out"], s["free_list"],
                            s["num_free"], s["free_out"])
    return dict(pools=values(s), lens=s["lens_out"], free_list=s["free_list"], num_free=s["free_out"])


def values(s):
    return s["pools"] if s["case"]["cache"] == "16" else [p.view(torch.float8_e4m3fn) for p in s["pools"]]


def plain_commit(s):
    c = s["case"]
    b, width, pools = c["block"], max(1, c["qmax"]), s["pools"]
    cu, lens, count, table = s["cu"].long(), s["lens"].long(), s["count"].long()[:, None], s["tables"].long()
    nodes = cu[1:] - cu[:-1]
    j = torch.arange(width, device="cuda")
    path = padded(s["path"], s["cu"], width, 0)
    first = (lens - nodes)[:, None]
    slot = lambda pos: table.gather(1, (pos // b).clamp(0, table.shape[1] - 1)) * b + pos % b  # noqa: E731
    inside = j < nodes[:, None]
    spare = pools[0].shape[1] * b - 1  # nobody's slot
    to = torch.where(inside, slot(first + j), spare).reshape(-1)
    source = torch.where(inside, slot(first + torch.where(j < count, path, j)), spare).reshape(-1)
    for pool in pools:
        flat = pool.view(2, -1, c["hkv"], c["d"])
        flat[:, to] = flat[:, source]
    # Blocks behind the new end go back, row by row, each row's last one first.
    after = lens - nodes + torch.where(nodes > 0, count[:, 0], 0)
    held, kept = (lens + b - 1) // b, (after + b - 1) // b
    gone = held - kept
    col = torch.arange(table.shape[1], device="cuda")
    place = s["num_free"].long() + (torch.cumsum(gone, 0) - gone)[:, None] + (held[:, None] - 1 - col)
    back = (col >= kept[:, None]) & (col < held[:, None])
    wide = torch.nn.functional.pad(s["free_list"].long(), (0, 1))
    wide.scatter_(0, torch.where(back, place, s["free_list"].numel()).reshape(-1), table.reshape(-1))
    small = lambda x: x.to(torch.int32)  # noqa: E731
    return dict(pools=values(s), lens=small(after), free_list=small(wide[:-1]), num_free=small(s["num_free"].long() + gone.sum()))


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"maps": exact_maps, "attend": exact_attend, "verify": exact_verify, "commit": exact_commit}[case["op"]](s, s["case"])


def exact_maps(s, c):
    parents, cu, lens = s["parents"].tolist(), s["cu"].tolist(), s["lens"].tolist()
    masks, positions = np.zeros(tuple(s["masks"].shape), np.uint32), np.zeros(len(parents), np.int32)
    for n in range(c["seqs"]):
        for i in range(cu[n], cu[n + 1]):
            j = parents[i]
            if j >= 0:
                masks[i] = masks[cu[n] + j]
                positions[i] = positions[cu[n] + j] + 1
            else:
                positions[i] = lens[n] - (cu[n + 1] - cu[n])
            at = i - cu[n]
            masks[i, at // 32] |= np.uint32(1 << (at % 32))
    return dict(positions=torch.from_numpy(positions).cuda(), masks=torch.from_numpy(masks.view(np.int32)).cuda())


def exact_attend(s, c):
    flat = s["pool"].view(2, -1, c["hkv"], c["d"])
    out = torch.zeros(s["query"].shape, dtype=torch.float64, device="cuda")
    cu, lens, tables, masks = s["cu"].tolist(), s["lens"].tolist(), s["tables"].long(), s["masks"].cpu().numpy().view(np.uint32)
    scales = (1.0, 1.0) if c["cache"] == "16" else (K_SCALE, V_SCALE)
    group = c["hq"] // c["hkv"]
    for n in range(c["seqs"]):
        nodes = cu[n + 1] - cu[n]
        if nodes == 0:
            continue
        i = torch.arange(lens[n], device="cuda")
        rows = flat[:, tables[n, i // c["block"]] * c["block"] + i % c["block"]]
        rows = rows if c["cache"] == "16" else rows.view(torch.float8_e4m3fn).float()
        bits = np.unpackbits(masks[cu[n]:cu[n + 1]].view(np.uint8), axis=1, bitorder="little")[:, :nodes]
        hidden = torch.zeros(nodes, lens[n], dtype=torch.bool, device="cuda")
        hidden[:, lens[n] - nodes:] = torch.from_numpy(bits == 0).cuda()
        for h in range(c["hkv"]):
            k, v = rows[0, :, h].double() * scales[0], rows[1, :, h].double() * scales[1]
            heads = slice(h * group, (h + 1) * group)
            q = s["query"][cu[n]:cu[n + 1], heads].double()
            score = torch.einsum("qgd,td->gqt", q, k) * s["scale"]
            w = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
            out[cu[n]:cu[n + 1], heads] = torch.einsum("gqt,td->qgd", w, v)
    return out


def exact_verify(s, c):
    cu, parents, tokens = s["cu"].tolist(), s["parents"].tolist(), s["tokens"].tolist()
    count, path, chosen = np.zeros(c["seqs"], np.int32), np.full(len(parents), -1, np.int32), np.full(len(parents), -1, np.int32)
    uniforms = None if s["uniforms"] is None else s["uniforms"].double().cpu().numpy()
    values_of = lambda t, r: t[r].double().cpu().numpy()  # noqa: E731
    for n in range(c["seqs"]):
        row, lo, hi = cu[n], cu[n], cu[n + 1]
        while lo < hi:
            path[lo + count[n]] = row - lo
            p, accepted = values_of(s["target"], row), None
            kids = [i for i in range(row + 1, hi) if parents[i] == row - lo]
            if c["mode"] == "greedy":
                token = int(np.argmax(p))
            else:
                if c["mode"] == "draft":
                    # p and what is left of it after each refused child, each scaled to sum 1.
                    now, q = p, values_of(s["draft"], row)
                    for i in kids:
                        if uniforms[i, 0] * q[tokens[i]] < now[tokens[i]]:
                            accepted = i
                            break
                        now = np.maximum(now - q, 0)
                        if now.sum() > 0:
                            now = now / now.sum()
                    p = now if now.sum() > 0 else p
                sums = np.cumsum(p)
                token = int(np.searchsorted(sums, uniforms[row, 1] * sums[-1], side="right"))
            if c["mode"] != "draft":
                accepted = next((i for i in kids if tokens[i] == token), None)
            chosen[lo + count[n]] = token if accepted is None else tokens[accepted]
            count[n] += 1
            if accepted is None:
                break
            row = accepted
    gpu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return dict(count=gpu(count), path=gpu(path), chosen=gpu(chosen))


def exact_commit(s, c):
    b = c["block"]
    cu, lens, count, path = s["cu"].tolist(), s["lens"].tolist(), s["count"].tolist(), s["path"].tolist()
    tables, free_list, free = s["tables"].cpu().numpy(), s["free_list"].cpu().numpy().copy(), int(s["num_free"])
    source, to, after = [], [], []
    for n in range(c["seqs"]):
        first, k = lens[n] - (cu[n + 1] - cu[n]), count[n] if cu[n + 1] > cu[n] else 0
        for j in range(k):
            a, z = first + path[cu[n] + j], first + j
            source.append(tables[n, a // b] * b + a % b)
            to.append(tables[n, z // b] * b + z % b)
        after.append(first + k)
        for j in range(-(-lens[n] // b) - 1, -(-(first + k) // b) - 1, -1):
            free_list[free] = tables[n, j]
            free += 1
    source, to = torch.tensor(source, dtype=torch.int64, device="cuda"), torch.tensor(to, dtype=torch.int64, device="cuda")
    pools = []
    for pool in values(s):
        new = pool.clone()
        new.view(2, -1, c["hkv"], c["d"]).view(torch.int8)[:, to] = pool.view(2, -1, c["hkv"], c["d"]).view(torch.int8)[:, source]
        pools.append(new)
    return dict(pools=pools, lens=ints(np.array(after)), free_list=ints(free_list), num_free=ints(np.array([free])))

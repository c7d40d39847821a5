"""Plain forms of the speculative step's operators, in 64 bits: trees, attention under masks, verification, commit."""
import numpy as np


def random_parents(rng, n, fan, unused=0.0):
    """Parents of a random tree of n nodes, some of them unused (-1), none below an unused one."""
    parents = np.full(n, -1, np.int32)
    used = [0]
    for i in range(1, n):
        if rng.random() < unused:
            continue
        parents[i] = used[-1 - int(rng.integers(0, min(len(used), fan)))]
        used.append(i)
    return parents


def closure(parents):
    """(whether node j is node i or an ancestor [n, n], depths [n])."""
    n = len(parents)
    seen, depth = np.eye(n, dtype=bool), np.zeros(n, np.int64)
    for i, a in enumerate(parents):
        if 0 <= a < i:
            seen[i] |= seen[a]
            depth[i] = depth[a] + 1
    return seen, depth


def pack(seen, words):
    """Rows of truth values as int32 words, the first the lowest bit."""
    n, m = seen.shape
    bits = np.zeros((n, 32 * words), np.uint8)
    bits[:, :m] = seen
    return np.packbits(bits, axis=1, bitorder="little").view(np.uint32).view(np.int32).reshape(n, words)


def attend(q, k, v, seen, scale):
    """q [n, Hq, D], k / v [L, Hkv, D], seen [n, L] -> (out, weights' mean |v|), both [n, Hq, D], in 64 bits.
    What a row does not see counts for nothing, whatever it holds; a row that sees nothing is zeros."""
    n, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    out, mean = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    for i in range(n):
        at = np.flatnonzero(seen[i])
        if not len(at):
            continue
        kk, vv = k[at], v[at]
        for h in range(hkv):
            s = q[i, h * g:(h + 1) * g] @ kk[:, h].T * scale
            w = np.exp(s - s.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            out[i, h * g:(h + 1) * g] = w @ vv[:, h]
            mean[i, h * g:(h + 1) * g] = w @ np.abs(vv[:, h])
    return out, mean


def verify(parents, tokens, target, draft, uniforms):
    """One sequence: (accepted nodes, new tokens). target / draft [n, V] float64, uniforms [n, 2] or None (greedy)."""
    n = len(parents)
    path, out, node = [], [], 0
    while True:
        path.append(node)
        p, accepted = target[node], None
        kids = [i for i in range(node + 1, n) if parents[i] == node]
        if draft is not None:
            r, z, q = p, 1.0, np.maximum(np.nan_to_num(draft[node]), 0)
            for i in kids:
                x = tokens[i]
                if 0 <= x < len(p) and uniforms[i, 0] * q[x] * z < r[x]:
                    accepted = i
                    break
                r = np.maximum(r - z * q, 0)
                z = r.sum()
            p = r if r.sum() > 0 else p
        if accepted is None:
            if uniforms is None:
                y = int(np.argmax(np.where(np.isnan(p), -np.inf, p)))
            else:
                w = np.where(p > 0, p, 0)
                sums = np.cumsum(w)
                hit = np.flatnonzero((sums > uniforms[node, 1] * sums[-1]) & (w > 0))
                y = int(hit[0]) if len(hit) else 0
            if draft is None:
                accepted = next((i for i in kids if tokens[i] == y), None)
        if accepted is None:
            out.append(y)
            return path, out
        out.append(int(tokens[accepted]))
        node = accepted


def commit(pools, tables, cu, lens, count, path, free, block):
    """pools: list of arrays (2, NB, B, ...), changed in place; free: list of the free blocks, the next one last. -> (new lengths,
    free)."""
    free, after = list(free), []
    for s, L in enumerate(lens):
        n = cu[s + 1] - cu[s]
        if n == 0:
            after.append(L)
            continue
        k, first = count[s], L - n
        for pool in pools:
            flat = pool.reshape(2, -1, *pool.shape[3:])
            src = [tables[s][(first + a) // block] * block + (first + a) % block for a in path[cu[s]:cu[s] + k]]
            dst = [tables[s][(first + a) // block] * block + (first + a) % block for a in range(k)]
            flat[:, dst] = flat[:, src]
        after.append(first + k)
        free += [tables[s][j] for j in range(-(-L // block) - 1, -(-(first + k) // block) - 1, -1)]
    return after, free

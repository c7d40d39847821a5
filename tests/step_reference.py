"""Plain references of the serving-step operators, in 64 bits: the step's
index maps (numpy), rotary positions and cross attention (float64)."""
from __future__ import annotations

import numpy as np


def ceil_div(a, b):
    return -(-int(a) // int(b))


def build_step(tables, lens, query, free_list, num_free, capacity, block_size):
    """The step's maps by the definition: finished rows return their blocks
    in row order, then rows are served in order while blocks and tokens last.
    -> dict of the call's outputs (tables and free_list after it)."""
    tables, out = tables.copy(), free_list.copy()
    stack = out[:num_free].tolist()
    for s in np.nonzero(query < 0)[0]:
        stack += tables[s, :ceil_div(lens[s], block_size)][::-1].tolist()
    n = len(lens)
    cu, after, admitted = [0], np.asarray(lens).copy(), n
    slots, positions = np.full(capacity, -1, np.int32), np.zeros(capacity, np.int32)
    for s in range(n):
        want, held = max(0, int(query[s])), ceil_div(lens[s], block_size)
        need = ceil_div(int(lens[s]) + want, block_size) - held
        if admitted < n or need > len(stack) or cu[-1] + want > capacity:
            admitted, want = min(admitted, s), 0
        for j in range(need if want else 0):
            tables[s, held + j] = stack.pop()
        for i in range(want):
            p = int(lens[s]) + i
            positions[cu[-1] + i] = p
            slots[cu[-1] + i] = tables[s, p // block_size] * block_size + p % block_size
        after[s] = 0 if query[s] < 0 else lens[s] + want
        cu.append(cu[-1] + want)
    if len(stack) > num_free:
        out[num_free:len(stack)] = stack[num_free:]
    return dict(tables=tables, free_list=out, num_free=len(stack), cu=np.array(cu, np.int32), lens=after.astype(np.int32),
                slots=slots, positions=positions, admitted=admitted)


def rotate(x, positions, inv_freq, axes, adjacent):
    """x [T, H, D] float64 with its first 2 * len(inv_freq) dimensions turned;
    positions [A, T] whole numbers, reduced exactly to a fraction of a turn."""
    from fractions import Fraction
    pairs = len(inv_freq)
    # inv_freq / (2 pi) to 40 digits, so that positions of 2^31 keep their turn.
    two_pi = Fraction(6283185307179586476925286766559005768394, 10 ** 39)
    frac = [Fraction(float(f)) / two_pi for f in inv_freq]
    t = x.shape[0]
    turn = np.empty((t, pairs))
    for i in range(pairs):
        num, den = frac[i].numerator, frac[i].denominator
        scaled = (num << 80) // den  # turns per position, 80 fractional bits
        col = positions[axes[i]]
        turn[:, i] = [((int(p) * scaled) & ((1 << 80) - 1)) / float(1 << 80) for p in col]
    c, s = np.cos(2 * np.pi * turn)[:, None], np.sin(2 * np.pi * turn)[:, None]
    y = x.copy()
    r = 2 * pairs
    a = slice(0, r, 2) if adjacent else slice(0, pairs)
    b = slice(1, r, 2) if adjacent else slice(pairs, r)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    size = np.abs(x).copy()  # |x1| + |x2| of each element's pair; 0 where it passes
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    size[..., r:] = 0
    return y, size


def cross_attention(query, pool, tables, cu, kv_lens, scale, block_size):
    """query [T, Hq, D] and pool (2, NB, B, Hkv, D) as float64 torch tensors ->
    (out, sum of weight * |v|), both float64: the definition, sequence by
    sequence; rows of a sequence without states are zero."""
    import torch
    t, hq, d = query.shape
    hkv = pool.shape[3]
    group = hq // hkv
    flat = pool.reshape(2, -1, hkv, d)
    out, size = torch.zeros_like(query), torch.zeros_like(query)
    for s in range(len(kv_lens)):
        a, b, L = int(cu[s]), int(cu[s + 1]), int(kv_lens[s])
        if a == b or L == 0:
            continue
        i = np.arange(L)
        at = torch.from_numpy(tables[s, i // block_size].astype(np.int64) * block_size + i % block_size).to(query.device)
        k, v = flat[0, at], flat[1, at]  # [L, Hkv, D]
        q = query[a:b].reshape(b - a, hkv, group, d)
        w = torch.softmax(torch.einsum("qhgd,lhd->qhgl", q, k) * scale, -1)
        out[a:b] = torch.einsum("qhgl,lhd->qhgd", w, v).reshape(b - a, hq, d)
        size[a:b] = torch.einsum("qhgl,lhd->qhgd", w, v.abs()).reshape(b - a, hq, d)
    return out, size

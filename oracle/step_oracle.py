"""64-bit CPU statement of a step's rotary positions and of the calls on the
pages of a cache. Plain numpy, one element after another where that is the definition."""
from __future__ import annotations

import math

import numpy as np


def rope_frequencies(dim, base=10000.0, scaling="none", factor=1.0, original=4096, beta_fast=32.0, beta_slow=1.0,
                     mscale=0.0, mscale_all_dim=0.0):
    """(radians per position of each pair, factor of cosine and sine)."""
    f = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    if scaling == "none":
        return np.array(f), 1.0
    if scaling == "linear":
        return np.array(f) / factor, 1.0
    # wavelength 2 pi / f: a pair makes original / wavelength turns over the original context
    pair = lambda beta: dim / 2 * math.log(original / (2 * math.pi * beta), base)
    low, high = max(0, math.floor(pair(beta_fast))), min(dim - 1, math.ceil(pair(beta_slow)))
    out = []
    for i, v in enumerate(f):
        r = min(1.0, max(0.0, (i - low) / (high - low if high != low else 0.001)))
        out.append((1 - r) * v + r * v / factor)
    g = lambda m: 1.0 if factor <= 1 else 1.0 + 0.1 * m * math.log(factor)
    return np.array(out), g(mscale) / g(mscale_all_dim)


def rotate(x, positions, freqs, factor, half):
    """x [T, ..., 64] turned by its token's position, as complex numbers."""
    d = 2 * len(freqs)
    x = np.asarray(x, np.float64)
    turn = factor * np.exp(1j * np.asarray(positions, np.float64)[:, None] * freqs)
    turn = turn.reshape(turn.shape[:1] + (1,) * (x.ndim - 2) + turn.shape[1:])
    a, b = (x[..., :d // 2], x[..., d // 2:d]) if half else (x[..., 0:d:2], x[..., 1:d:2])
    z = (a + 1j * b) * turn
    y = x.copy()
    if half:
        y[..., :d // 2], y[..., d // 2:d] = z.real, z.imag
    else:
        y[..., 0:d:2], y[..., 1:d:2] = z.real, z.imag
    return y


def fork(parent, child, lens, free, table, refs, rows, scales, block, group):
    """``rows [num_blocks, block, width]``, ``scales [num_blocks, block / group]`` or
    None. Returns (table, refs, rows, scales, taken)."""
    table, refs, rows = table.copy(), refs.copy(), rows.copy()
    scales = None if scales is None else scales.copy()
    n, cols = table.shape
    taken = 0
    for p, c, ln in zip(parent, child, lens):
        if not (0 <= p < n and 0 <= c < n):
            continue
        whole = min(ln // block, cols)
        for j in range(whole):
            table[c, j] = table[p, j]
            if table[p, j] >= 0:
                refs[table[p, j]] += 1
        rest = ln % block
        if whole == cols or rest == 0:
            continue
        old = table[p, whole]
        table[c, whole] = -1
        if old < 0:
            continue
        if taken < len(free):
            new = free[taken]
            table[c, whole] = new
            refs[new] = 1
            rows[new, :rest] = rows[old, :rest]
            if scales is not None:
                k = -(-rest // group)
                scales[new, :k] = scales[old, :k]
        taken += 1
    return table, refs, rows, scales, taken


def free(listed, lens, table, refs, block):
    """Returns (table, refs, blocks freed in ascending order)."""
    table, refs = table.copy(), refs.copy()
    gone = []
    for i, r in enumerate(listed):
        if not 0 <= r < table.shape[0]:
            continue
        cols = table.shape[1] if lens is None else min(-(-lens[i] // block), table.shape[1])
        for c in range(cols):
            b = table[r, c]
            table[r, c] = -1
            if 0 <= b < len(refs):
                refs[b] -= 1
                if refs[b] == 0:
                    gone.append(b)
    return table, refs, sorted(gone)


def compact(refs, table, rows, scales):
    """Returns (refs, table, rows, scales, blocks in use)."""
    used = [b for b in range(len(refs)) if refs[b] > 0]
    n = len(used)
    holes = [b for b in range(n) if refs[b] <= 0]
    move = dict(zip([b for b in used if b >= n], holes))
    new, rows, out = np.zeros_like(refs), rows.copy(), table.copy()
    scales = None if scales is None else scales.copy()
    for b in used:
        to = move.get(b, b)
        new[to] = refs[b]
        rows[to] = rows[b]
        if scales is not None:
            scales[to] = scales[b]
    for b, to in move.items():
        out[table == b] = to
    return new, out, rows, scales, n

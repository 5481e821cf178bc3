"""Plain CPU oracle of the serving step over an e4m3 cache with group scales:
block tables and slot maps, the append, and the attention in float64.

TEST INFRASTRUCTURE, like the rest of this package: no code is shared with the
CUDA library. A cache slot s holds 576 codes that stand for
``code * scales[s // group]``; ``group`` divides the block size. Every function
is written from that definition, one request, run or token at a time, and
pinned by tests/test_scaled_cache.py.
"""
from __future__ import annotations

import numpy as np

from .mla_oracle import HEAD_DIM, KV_LORA_RANK, attend, decode_e4m3fn, encode_e4m3fn

MIN_SCALE, MAX_SCALE = 2.0 ** -60, 2.0 ** 60


def block_tables(query_start_loc, seq_lens, free_blocks, table, block_size, num_tokens):
    """(table, slots, req_id, positions, taken) of one step. ``table`` is
    copied; cells outside the step's new columns keep their values."""
    qsl = [int(v) for v in query_start_loc]
    table = np.array(table, dtype=np.int64)
    cols = table.shape[1]
    slots = np.full(num_tokens, -1, dtype=np.int64)
    req = np.full(num_tokens, -1, dtype=np.int64)
    pos = np.full(num_tokens, -1, dtype=np.int64)
    taken = 0
    for r, n in enumerate(int(v) for v in seq_lens):
        ctx = n - (qsl[r + 1] - qsl[r])
        for col in range(-(-ctx // block_size), min(-(-n // block_size), cols)):
            table[r, col] = free_blocks[taken] if taken < len(free_blocks) else -1
            taken += 1
        for t in range(qsl[r], qsl[r + 1]):
            p = ctx + t - qsl[r]
            req[t], pos[t] = r, p
            if p // block_size < cols and table[r, p // block_size] >= 0:
                slots[t] = table[r, p // block_size] * block_size + p % block_size
    return table, slots, req, pos, taken


def group_scale(amax: float) -> float:
    """The least power of two s with amax <= 448 s, within [MIN_SCALE, MAX_SCALE]."""
    s = MIN_SCALE
    while amax > 448.0 * s and s < MAX_SCALE:
        s *= 2.0
    return s


def cache_append(rows, slot_mapping, codes, scales, group):
    """(codes, scales) after the append of ``rows [T, 576]`` (float64 of bf16
    values). ``codes [slots, 576]`` uint8 and ``scales`` are copied."""
    codes, scales = np.array(codes), np.array(scales, dtype=np.float64)
    slot = [int(s) if 0 <= int(s) < codes.shape[0] else -1 for s in slot_mapping]
    t = 0
    while t < len(slot):
        if slot[t] < 0:
            t += 1
            continue
        end = t + 1
        while end < len(slot) and slot[end] == slot[end - 1] + 1 and slot[end] % group != 0:
            end += 1
        run = np.asarray(rows[t:end], dtype=np.float64)
        first, n = slot[t], end - t
        start = first - first % group
        finite = np.abs(run[np.isfinite(run)])
        s = group_scale(float(finite.max()) if finite.size else 0.0)
        if first > start:
            old = float(scales[first // group])
            if s > old:
                codes[start:first] = _encode(decode_e4m3fn(codes[start:first]) * (old / s))
            s = max(s, old)
        codes[first:first + n] = _encode(run / s)
        scales[first // group] = s
        t = end
    return codes, scales


def _encode(x):
    x = np.asarray(x, dtype=np.float64)
    out = encode_e4m3fn(np.clip(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0), -448.0, 448.0))
    return np.where(np.isnan(x), np.uint8(0x7F), out).astype(np.uint8)


def row_slots(block_table_row, block_size, n):
    """Slots of a request's first n positions."""
    p = np.arange(n)
    return np.asarray(block_table_row, dtype=np.int64)[p // block_size] * block_size + p % block_size


def token_slots(block_table, seq_lens, block_size, qo_indptr=None):
    """The list of visible slots of every token, in token order."""
    lists = []
    for r, n in enumerate(int(v) for v in seq_lens):
        q = 1 if qo_indptr is None else int(qo_indptr[r + 1]) - int(qo_indptr[r])
        lists += [row_slots(block_table[r], block_size, max(0, n - q + j + 1)) for j in range(q)]
    return lists


def decode(q_codes, q_scale, codes, scales, group, lists, softmax_scale, sinks=None, bounds=False):
    """(out [T, H, 512], lse [T, H]) in float64; token t attends to the slots
    lists[t]. With ``bounds`` also how far a kernel's results may lie off (see
    ``_bounds``)."""
    q = decode_e4m3fn(q_codes) * q_scale
    codes = np.asarray(codes).reshape(-1, HEAD_DIM)
    T, H = q.shape[:2]
    out, lse = np.zeros((T, H, KV_LORA_RANK)), np.full((T, H), -np.inf)
    tol_o, tol_l = np.zeros_like(out), np.zeros_like(lse)
    for t, rows in enumerate(lists):
        rows = np.asarray(rows, dtype=np.int64)
        rows = rows[rows >= 0]
        s = np.asarray(scales, dtype=np.float64)[rows // group]
        c = decode_e4m3fn(codes[rows])
        out[t], lse[t] = attend(q[t], c * s[:, None], softmax_scale, sinks)
        if bounds and len(rows):
            tol_o[t], tol_l[t] = _bounds(q[t], c, s, softmax_scale, out[t], lse[t], sinks)
        elif bounds and sinks is not None:
            # no key: lse = ln 2 (sink log2 e) in fp32, two products of two
            # rounded constants: four half steps, 4 * 2^-24 of the sink
            tol_l[t] = np.abs(np.asarray(sinks, dtype=np.float64)) * 2.0 ** -22
    return (out, lse, tol_o, tol_l) if bounds else (out, lse)


def _bounds(q, c, s, softmax_scale, out, lse, sinks):
    """Largest error of a kernel that keeps scores, sums and accumulators in
    fp32, rounds each weight p'_j ~ w_j s_j (w the softmax weights, the row's
    largest kept at p' >= 2^4) to an e4m3 term and a rest in e5m2 or, 32 times
    itself, in e4m3, and the output to bf16:
      * a weight: half a step of e4m3 leaves a rest of 2^-4 of it at most, half
        a step of e5m2 2^-3 of that: 2^-7. The f16 that both are taken from
        adds 2^-11. Below 2^-6 the first term's half step is 2^-10 and 2^-3 of
        the rest at most 2^-13, 2^-17 of the largest weight, and at most 2^-3
        of the weight, as the rest is no larger than it. A rest below the
        second term's normal range is off by half its smallest step: 2^-17 in
        e5m2, 2^-10 / 32 in the other, 2^-19 of the largest weight, and at most
        the weight itself;
      * a score: 576 fp32 additions, each off by at most 2^-23 (truncated
        alignment in the matrix unit) of the sum of magnitudes;
      * the exponent: its argument t = score log2 e + log2 s rounded a few
        times at 2^-24 of its size, exp2 and log2 at 2^-22, and sums of n terms;
      * the output: half a bf16 step, 2^-8 of the value.
    """
    z = softmax_scale * (q @ (c * s[:, None]).T)                     # [H, n]
    w = np.exp(z - lse[:, None])
    mags = softmax_scale * (np.abs(q) @ (np.abs(c) * s[:, None]).T)
    t = np.abs(z) / np.log(2.0) + np.abs(np.log2(s))
    n = c.shape[0]
    gamma = 576 * 2.0 ** -23 * mags.max(1) + (t.max(1) + 8.0) * 2.0 ** -21 + n * 2.0 ** -25
    v = np.abs(c[:, :KV_LORA_RANK])
    ws = w * s
    top = ws.max(1)[:, None]
    err = (2.0 ** -7 + 2.0 ** -11) * ws
    err += np.minimum(2.0 ** -17 * top, 2.0 ** -3 * ws) + np.minimum(2.0 ** -19 * top, ws)
    tol_o = (err + 2.0 * gamma[:, None] * ws) @ v
    tol_o = tol_o * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(out)
    tol_l = gamma + np.abs(lse) * 2.0 ** -22
    if sinks is not None:
        tol_l = tol_l + np.abs(np.asarray(sinks, dtype=np.float64)) * 2.0 ** -22
    return tol_o, tol_l

"""Cases of serving many samples of one prompt over the paged latent cache.

Three operators: the rotary positions of a step's queries and keys; the pages
of requests that fork from one another (their tables, reference counts and
contents: forked, copied, freed, compacted); and the attention of a batch whose
requests share a long prefix, computed once for all of them. ``own`` selects
the library's kernels; without it every operator runs in its plain torch form,
in 32 bits.

Cache rows are 576 wide (512 latent columns, which are also the values, and 64
rope columns): bf16, or e4m3 codes with ``scales[slot // group]`` as the fp32
scale of a group of ``group`` consecutive slots of a block.
"""
import math

import numpy as np
import torch

own = False

DIM, RANK, ROPE = 576, 512, 64
SOFTMAX_SCALE = 1.0 / math.sqrt(192.0)
Q_SCALE = 2.0 ** -6           # static scale of e4m3 queries: 448 / 64 = 7 standard deviations
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _rope(name, tokens, heads, fp8, layout, scaling, dim, far, pad=0):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "fp8": fp8, "layout": layout,
            "scaling": scaling, "dim": dim, "far": far, "pad": pad}


def _pages(name, kind, fp8, block, group, prompts, samples, ctx_lo, ctx_hi, blocks=0, live=0.0):
    return {"name": name, "op": "pages", "kind": kind, "fp8": fp8, "block": block, "group": group,
            "prompts": prompts, "samples": samples, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "blocks": blocks,
            "live": live}


def _shared(name, fp8, heads, groups, reqs, prefix_lo, prefix_hi, own_lo, own_hi, block, group, qlen=1, sinks=False,
            alone=0):
    return {"name": name, "op": "shared", "fp8": fp8, "heads": heads, "groups": groups, "reqs": reqs,
            "prefix_lo": prefix_lo, "prefix_hi": prefix_hi, "own_lo": own_lo, "own_hi": own_hi, "block": block,
            "group": group, "qlen": qlen, "sinks": sinks, "alone": alone}


def listed():
    return [
        # one decode step of a full batch: e4m3 queries, adjacent pairs, frequencies blended for long contexts
        _rope("rope_decode_64", 64, 128, True, "interleaved", "yarn", 64, 131072, pad=3),
        # a chunk of prompts of odd length on a rank's 16 heads: bf16, split halves, linear interpolation
        _rope("rope_prompt_8191", 8191, 16, False, "half", "linear", 64, 1 << 20),
        # four samples of one short prompt: latency only
        _pages("fork_1x4", "fork", True, 64, 64, 1, 4, 700, 1000),
        # eight samples of each of 64 prompts, a partly filled page copied for each
        _pages("fork_64x8", "fork", True, 64, 16, 64, 8, 500, 12000),
        # samples that are forked, and given up again
        _pages("fork_free_32x16", "fork_free", False, 64, 64, 32, 16, 100, 6000),
        # whole pages copied within a bf16 cache
        _pages("copy_4000", "copy", False, 64, 64, 1, 1, 0, 0, blocks=9000, live=4000 / 9000),
        # a fragmented pool, its pages moved together
        _pages("compact_16384", "compact", True, 64, 64, 256, 1, 100, 4100, blocks=16384, live=0.6),
        # a handful of samples in small pages: the latency of one call
        _shared("shared_4x16h", True, 16, 1, 4, 200, 300, 1, 60, 16, 16),
        # a system prompt on an attention-parallel rank's 16 heads
        _shared("shared_64x16384_16h", True, 16, 1, 64, 16400, 16400, 64, 1024, 64, 64),
        # the same on all 128 heads with sinks, two padding requests outside the group: the largest call
        _shared("shared_64x8192_128h", True, 128, 1, 64, 8192, 8192, 128, 2048, 64, 64, sinks=True, alone=2),
        # samples of 7 prompts of odd lengths, one to three tokens each, a scale for each token
        _shared("shared_groups_mtp", True, 32, 7, 56, 1500, 9000, 3, 700, 64, 1, qlen=3, alone=1),
        # a bf16 cache, all heads
        _shared("shared_bf16_32x8192", False, 128, 1, 32, 8200, 8200, 50, 900, 64, 64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "pages", "pages", "shared", "shared"])
    block = rng.choice([16, 32, 48, 64, 64, 128])
    group = rng.choice([g for g in (1, 2, 4, 8, 16, 24, 32, 48, 64, 128) if block % g == 0])
    if op == "rope":
        heads = rng.choice([1, 8, 16, 17, 32, 64, 128, _log_int(rng, 1, 128)])
        tokens = _log_int(rng, 1, max(1, min(16384, 131072 // heads)))
        return {"op": op, "tokens": tokens, "heads": heads, "fp8": rng.random() < 0.5,
                "layout": rng.choice(["interleaved", "half"]), "scaling": rng.choice(["none", "linear", "yarn"]),
                "dim": rng.choice([64, 64, 32, 2 * rng.randint(1, 32)]), "far": _log_int(rng, 64, 1 << 21),
                "pad": rng.choice([0, 0, rng.randint(1, 9)])}
    if op == "pages":
        kind = rng.choice(["fork", "fork_free", "copy", "compact"])
        c = {"op": op, "kind": kind, "fp8": rng.random() < 0.6, "block": block, "group": group, "prompts": 1,
             "samples": 1, "ctx_lo": 0, "ctx_hi": 0, "blocks": 0, "live": 0.0}
        if kind == "copy":
            c.update(blocks=_log_int(rng, 4, 500000 // block), live=rng.uniform(0.05, 0.45))
            return c
        hi = _log_int(rng, 2, 16384)
        c.update(ctx_lo=rng.randint(1, hi), ctx_hi=hi)
        c["prompts"] = _log_int(rng, 1, max(1, min(256, 500000 // hi)))
        if kind == "compact":
            c.update(live=rng.uniform(0.2, 0.95))
            need = sum(-(-int(v) // block) for v in _spread(c["prompts"], c["ctx_lo"], c["ctx_hi"]))
            c["blocks"] = int(need / c["live"]) + 1
        else:
            c["samples"] = _log_int(rng, 1, 16)
        return c
    fp8 = rng.random() < 0.7
    if not fp8:
        block = rng.choice([64, 64, 128])
        group = block
    heads = rng.choice([1, 8, 16, 17, 32, 48, 64, 96, 128, _log_int(rng, 1, 128)])
    groups = rng.choice([1, 1, 1, rng.randint(2, 9)])
    reqs = groups * _log_int(rng, 1, max(1, 64 // groups))
    qlen = rng.choice([1, 1, 1, rng.randint(2, 4)])
    prefix = _log_int(rng, 16, 16384)
    while reqs * qlen * heads * prefix > 64 * 128 * 8192:
        prefix //= 2
    own_hi = _log_int(rng, 4, 2048)
    return {"op": op, "fp8": fp8, "heads": heads, "groups": groups, "reqs": reqs,
            "prefix_lo": rng.randint(max(1, prefix // 3), prefix), "prefix_hi": prefix, "own_lo": rng.randint(1, own_hi),
            "own_hi": own_hi, "block": block, "group": group, "qlen": qlen, "sinks": rng.random() < 0.3,
            "alone": rng.choice([0, 0, 1, 3])}


# ---------------------------------------------------------------------------
# layouts of a case (the same set of lengths for every seed, in another order)
# ---------------------------------------------------------------------------

def _spread(n, lo, hi):
    """n lengths, evenly from lo to hi."""
    return np.round(lo + (np.arange(n) + 0.5) / n * (hi - lo)).astype(np.int64)


def _shared_lens(c):
    """(prefix of each group, own length and new tokens of each request of a group, in order of size)."""
    prefix = _spread(c["groups"], c["prefix_lo"], c["prefix_hi"])
    q = 1 + np.arange(c["reqs"], dtype=np.int64) % c["qlen"]
    return prefix, np.maximum(_spread(c["reqs"], c["own_lo"], c["own_hi"]), q), q


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _rows(gen, n):
    """n latent rows as a model makes them: unit-variance columns, tokens of differing size, a larger rope part."""
    x = torch.randn((n, DIM), device="cuda", generator=gen)
    x *= torch.exp(0.3 * torch.randn((n, 1), device="cuda", generator=gen))
    x[:, RANK:] *= 1.5
    return x.bfloat16()


def _cache(gen, blocks, block, group, fp8):
    """A cache of `blocks` pages in use and its scales: powers of two that bring each group to 448 or below."""
    slots = blocks * block
    step = block * max(1, 65536 // block)
    if not fp8:
        rows = torch.empty((slots, DIM), dtype=torch.bfloat16, device="cuda")
        for a in range(0, slots, step):
            rows[a:a + step] = _rows(gen, min(step, slots - a))
        return rows.view(blocks, block, DIM), None
    codes = torch.empty((slots, DIM), dtype=torch.uint8, device="cuda")
    scales = torch.empty(slots // group, dtype=torch.float32, device="cuda")
    for a in range(0, slots, step):
        b = min(slots, a + step)
        x = _rows(gen, b - a).float().view(-1, group * DIM)
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax(1) / 448.0)))
        codes[a:b] = (x / s[:, None]).clamp(-448, 448).view(-1, DIM).to(E4M3).view(torch.uint8)
        scales[a // group:b // group] = s
    return codes.view(E4M3).view(blocks, block, DIM), scales


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    rng, gen = np.random.default_rng(int(seed)), _gen(seed)
    return {"rope": _prepare_rope, "pages": _prepare_pages, "shared": _prepare_shared}[case["op"]](case, rng, gen)


ROPE_BASE, ROPE_FACTOR, ROPE_ORIGINAL = 10000.0, 40.0, 4096   # frequencies, and their stretch to long contexts
ROPE_MSCALE, ROPE_MSCALE_ALL = 1.0, 0.707


def _prepare_rope(c, rng, gen):
    T, H = c["tokens"], c["heads"]
    # positions of a step: runs of consecutive tokens, requests at any depth; padding behind them
    n = max(1, T // 97)
    starts = np.sort(rng.choice(T, size=min(n, T), replace=False))
    starts[0] = 0
    pos = np.arange(T) - np.repeat(starts, np.diff(np.append(starts, T)))
    pos = pos + np.repeat(rng.integers(0, c["far"], len(starts)), np.diff(np.append(starts, T)))
    pos[T - min(c["pad"], T):] = -1
    # the absorbed queries as the batched product leaves them (heads outermost), the
    # rope parts as slices of the projections' rows
    nope = torch.randn((H, T, RANK), device="cuda", generator=gen).bfloat16().transpose(0, 1)
    full = torch.randn((T, H, 128 + ROPE), device="cuda", generator=gen).bfloat16()
    kv = _rows(gen, T)
    s = {"op": "rope", "dim": c["dim"], "half": c["layout"] == "half", "fp8": c["fp8"], "pos": _i32(pos),
         "nope": nope, "q_pe": full[..., 128:], "k_pe": kv[:, RANK:],
         "q": torch.zeros((T, H, DIM), dtype=torch.uint8 if c["fp8"] else torch.bfloat16, device="cuda"),
         "k": torch.zeros((T, ROPE), dtype=torch.bfloat16, device="cuda")}
    if c["fp8"]:
        s["q"] = s["q"].view(E4M3)
    if own:
        from paged_mla_decode_06_gb300 import binding as B
        s["rope"] = B.mla_rope_plan(dim=c["dim"], layout=c["layout"], base=ROPE_BASE, scaling=c["scaling"],
                                    factor=ROPE_FACTOR, original_max_position=ROPE_ORIGINAL, mscale=ROPE_MSCALE,
                                    mscale_all_dim=ROPE_MSCALE_ALL)
    else:
        s["freqs"], s["mscale"] = _plain_freqs(c["dim"], c["scaling"])
    return s


def _plain_freqs(dim, scaling):
    """The angle of each pair per position (64 bits, on the GPU) and the factor of cosine and sine."""
    i = torch.arange(dim // 2, dtype=torch.float64)
    f = ROPE_BASE ** (-2.0 * i / dim)
    if scaling == "linear":
        return (f / ROPE_FACTOR).cuda(), 1.0
    if scaling == "none":
        return f.cuda(), 1.0

    def turn(beta):  # the pair that makes beta turns over the original context
        return dim * math.log(ROPE_ORIGINAL / (beta * 2 * math.pi)) / (2 * math.log(ROPE_BASE))
    low, high = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), dim - 1)
    ramp = ((i - low) / (high - low if high != low else 0.001)).clamp(0, 1)
    m = (0.1 * ROPE_MSCALE * math.log(ROPE_FACTOR) + 1) / (0.1 * ROPE_MSCALE_ALL * math.log(ROPE_FACTOR) + 1)
    return (f / ROPE_FACTOR * ramp + f * (1 - ramp)).cuda(), m


def _prepare_pages(c, rng, gen):
    bs, kind = c["block"], c["kind"]
    s = {"op": "pages", "kind": kind, "block": bs, "group": c["group"]}
    if kind == "copy":
        n = max(1, int(c["blocks"] * c["live"]))
        ids = rng.permutation(c["blocks"])
        s["cache"], s["scales"] = _cache(gen, c["blocks"], bs, c["group"], c["fp8"])
        s.update(src=_i32(ids[:n]), dst=_i32(ids[n:2 * n]))
        return s
    ctx = rng.permutation(_spread(c["prompts"], c["ctx_lo"], c["ctx_hi"]))
    need = -(-ctx // bs)
    cols = int(need.max()) + 1
    P, S = c["prompts"], c["samples"]
    used = int(need.sum())
    if kind == "compact":
        N = c["blocks"]
        low = _stay(c)                                   # live pages that keep their place
        ids = np.concatenate([rng.permutation(used)[:low], used + rng.permutation(N - used)[:used - low]])
        ids = rng.permutation(ids)
    else:
        N = used + P * S + 3
        ids = rng.permutation(N)
        s["free"] = _i32(ids[used:])
    table = np.full((P + (P * S if kind != "compact" else 0), cols), -1, np.int32)
    table[:P][np.arange(cols)[None, :] < need[:, None]] = ids[:used]
    refs = np.zeros(N, np.int32)
    refs[ids[:used]] = 1
    s["cache"], s["scales"] = _cache(gen, N, bs, c["group"], c["fp8"])
    s.update(table=_i32(table), refs=_i32(refs))
    if kind == "compact":
        s.update(table_out=torch.empty_like(s["table"]), refs_out=torch.empty_like(s["refs"]),
                 count=torch.empty(1, dtype=torch.int32, device="cuda"))
        if own:
            from paged_mla_decode_06_gb300 import binding as B
            s["workspace"] = torch.zeros(B.mla_cache_workspace(N), dtype=torch.uint8, device="cuda")
        return s
    parent = np.repeat(np.arange(P), S)
    s.update(parent=_i32(parent), child=_i32(P + rng.permutation(P * S)), lens=_i32(ctx[parent]),
             taken=torch.empty(1, dtype=torch.int32, device="cuda"))
    if kind == "fork_free":
        s.update(freed=torch.full((P * S,), -1, dtype=torch.int32, device="cuda"),
                 count=torch.empty(1, dtype=torch.int32, device="cuda"))
        if own:
            from paged_mla_decode_06_gb300 import binding as B
            s["workspace"] = torch.zeros(B.mla_cache_workspace(N), dtype=torch.uint8, device="cuda")
    return s


def _stay(c):
    """Live pages of a compaction that lie low enough already: their share of the pool."""
    used = int((-(-_spread(c["prompts"], c["ctx_lo"], c["ctx_hi"]) // c["block"])).sum())
    return max(used - (c["blocks"] - used), round(used * used / c["blocks"]))


def _prepare_shared(c, rng, gen):
    bs, H = c["block"], c["heads"]
    prefix, own_len, q = _shared_lens(c)
    G, R = c["groups"], c["reqs"]
    order = rng.permutation(R)
    own_len, q = own_len[order], q[order]
    prefix = rng.permutation(prefix)
    edges = np.round(np.arange(G + 1) * R / G).astype(np.int64)
    of = np.repeat(np.arange(G), np.diff(edges))
    lens = np.concatenate([prefix[of] + own_len, np.zeros(c["alone"], np.int64)])
    q = np.concatenate([q, np.ones(c["alone"], np.int64)])
    count, common = -(-lens // bs), prefix // bs          # pages of each request, whole pages of each prefix
    cols = int(count.max()) + 1
    ids = rng.permutation(int(common.sum() + (count[:R] - common[of]).sum()) + 1)
    table = np.full((len(lens), cols), ids[-1], np.int32)
    at = 0
    for g in range(G):
        table[edges[g]:edges[g + 1], :common[g]] = ids[at:at + common[g]]
        at += common[g]
    for r in range(R):
        n = count[r] - common[of[r]]
        table[r, common[of[r]]:count[r]] = ids[at:at + n]
        at += n
    cache, scales = _cache(gen, len(ids), bs, c["group"], c["fp8"])
    qsl = np.concatenate([[0], np.cumsum(q)])
    T = int(qsl[-1])
    x = torch.randn((T, H, DIM), device="cuda", generator=gen)
    s = {"op": "shared", "block": bs, "group": c["group"], "cache": cache, "scales": scales,
         "q": (x / Q_SCALE).clamp(-448, 448).to(E4M3) if c["fp8"] else x.bfloat16(),
         "q_scale": Q_SCALE if c["fp8"] else 1.0, "table": _i32(table), "lens": _i32(lens),
         "qsl": _i32(qsl) if c["qlen"] > 1 else None, "prefix": _i32(prefix), "edges": _i32(edges),
         "sinks": torch.randn(H, device="cuda", generator=gen) if c["sinks"] else None, "max_q": int(q.max()),
         # what the scheduler knows on the host besides: sizes of the groups
         "host": [(int(common[g]) * bs, int(edges[g]), int(edges[g + 1]), int(qsl[edges[g]]), int(qsl[edges[g + 1]]))
                  for g in range(G)], "max_own": int((lens - np.append(common[of] * bs, np.zeros(c["alone"]))).max()),
         "out": torch.empty((T, H, RANK), dtype=torch.bfloat16, device="cuda"),
         "lse": torch.empty((T, H), dtype=torch.float32, device="cuda")}
    if own:
        from paged_mla_decode_06_gb300 import binding as B
        s["plan"] = B.mla_decode_shared_plan(B.make_problem(
            num_tokens=T, num_heads=H, block_size=bs, num_blocks=len(ids), num_reqs=len(lens), max_blocks_per_req=cols,
            max_seq_len=int(lens.max()), max_qlen=int(q.max()), dtype="fp8" if c["fp8"] else "bf16",
            has_sinks=c["sinks"]), num_groups=G)
        s["workspace"] = torch.zeros(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    if not own:
        return {"rope": _plain_rope, "pages": _plain_pages, "shared": _plain_shared}[s["op"]](s)
    from paged_mla_decode_06_gb300 import binding as B
    if s["op"] == "rope":
        B.mla_rope_qk(s["rope"], s["pos"], ql_nope=s["nope"], q_pe=s["q_pe"], q_out=s["q"],
                      q_scale=Q_SCALE if s["fp8"] else None, k_pe=s["k_pe"], k_out=s["k"])
        return {"q": s["q"], "k": s["k"]}
    if s["op"] == "shared":
        B.mla_decode_fwd_shared(s["plan"], s["q"], s["cache"], kv_scales=s["scales"],
                                scale_group=s["group"] if s["scales"] is not None else 0, block_table=s["table"],
                                seq_lens=s["lens"], qo_indptr=s["qsl"], prefix_lens=s["prefix"],
                                group_indptr=s["edges"], softmax_scale=SOFTMAX_SCALE, q_scale=s["q_scale"],
                                sinks=s["sinks"], workspace=s["workspace"], out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    group = s["group"] if s["scales"] is not None else 0
    if s["kind"] == "copy":
        B.mla_cache_copy_blocks(s["src"], s["dst"], s["cache"], s["scales"], scale_group=group)
    elif s["kind"] == "compact":
        B.mla_cache_compact(s["refs"], s["table"], s["cache"], s["scales"], scale_group=group, refs_out=s["refs_out"],
                            table_out=s["table_out"], num_live=s["count"], workspace=s["workspace"])
    else:
        B.mla_cache_fork(s["parent"], s["child"], s["lens"], s["free"], s["table"], s["refs"], s["cache"], s["scales"],
                         scale_group=group, taken=s["taken"])
        if s["kind"] == "fork_free":
            B.mla_cache_free(s["child"], s["table"], s["refs"], freed=s["freed"], num_freed=s["count"],
                             workspace=s["workspace"])
    return _pages_out(s)


def _pages_out(s):
    names = {"copy": [], "compact": ["table_out", "refs_out", "count"], "fork": ["table", "refs", "taken"],
             "fork_free": ["table", "refs", "taken", "freed", "count"]}[s["kind"]]
    out = {n: s[n] for n in names}
    out["cache"] = s["cache"]
    if s["scales"] is not None:
        out["scales"] = s["scales"]
    return out


def _plain_rope(s):
    d, live = s["dim"], (s["pos"] >= 0)
    a = s["pos"].double()[:, None] * s["freqs"]
    cos, sin = (a.cos() * s["mscale"]).float(), (a.sin() * s["mscale"]).float()

    def turned(x, cos, sin):
        y = x.clone()
        if s["half"]:
            lo, hi = slice(0, d // 2), slice(d // 2, d)
        else:
            lo, hi = slice(0, d, 2), slice(1, d, 2)
        y[..., lo] = x[..., lo] * cos - x[..., hi] * sin
        y[..., hi] = x[..., hi] * cos + x[..., lo] * sin
        return y
    q = torch.cat([s["nope"].float(), turned(s["q_pe"].float(), cos[:, None], sin[:, None])], 2)
    k = turned(s["k_pe"].float(), cos, sin).bfloat16()
    if s["fp8"]:
        q = (q / Q_SCALE).clamp(-448, 448).to(E4M3).view(torch.uint8)
        codes = s["q"].view(torch.uint8)
        codes.copy_(torch.where(live[:, None, None], q, codes))
    else:
        s["q"].copy_(torch.where(live[:, None, None], q.bfloat16(), s["q"]))
    s["k"].copy_(torch.where(live[:, None], k, s["k"]))
    return {"q": s["q"], "k": s["k"]}


def _plain_pages(s):
    cache = s["cache"].view(torch.uint8) if s["scales"] is not None else s["cache"]
    bs = s["block"]
    scales = s["scales"].view(-1, bs // s["group"]) if s["scales"] is not None else None
    if s["kind"] == "copy":
        src, dst = s["src"].long(), s["dst"].long()
        cache[dst] = cache[src]
        if scales is not None:
            scales[dst] = scales[src]
        return _pages_out(s)
    if s["kind"] == "compact":
        live = s["refs"] > 0
        n = int(live.sum())
        at = torch.arange(live.numel(), device=live.device)
        src = at[live & (at >= n)]
        dst = at[~live & (at < n)]
        to = at.clone()
        to[src] = dst
        cache[dst] = cache[src]
        if scales is not None:
            scales[dst] = scales[src]
        s["table_out"].copy_(torch.where(s["table"] >= 0, to[s["table"].long().clamp_min(0)].int(), s["table"]))
        s["refs_out"].zero_()
        s["refs_out"][:n] = s["refs"][:n].where(live[:n], torch.zeros((), dtype=torch.int32, device=live.device))
        s["refs_out"][dst] = s["refs"][src]
        s["count"].fill_(n)
        return _pages_out(s)
    table, refs = s["table"], s["refs"]
    lens, parent, child = s["lens"].long(), s["parent"].long(), s["child"].long()
    whole, rest = lens // bs, lens % bs
    new = (rest > 0).long()
    base = new.cumsum(0) - new
    col = torch.arange(table.shape[1], device=table.device)
    rows = table[parent]
    kept = col < whole[:, None]
    last = (col == whole[:, None]) & (rest > 0)[:, None]
    fresh = s["free"][base.clamp(max=s["free"].numel() - 1)]
    table[child] = torch.where(kept, rows, torch.where(last, fresh[:, None], table[child]))
    refs.index_add_(0, rows[kept].long(), torch.ones_like(rows[kept]))
    some = rest > 0
    refs[fresh[some].long()] = 1
    old = rows.gather(1, whole.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    off = torch.arange(bs, device=table.device)
    cell = (some[:, None] & (off < rest[:, None])).nonzero()
    cache[fresh[cell[:, 0]].long(), cell[:, 1]] = cache[old[cell[:, 0]].long(), cell[:, 1]]
    if scales is not None:
        first = cell[cell[:, 1] % s["group"] == 0]
        unit = first[:, 1] // s["group"]
        scales[fresh[first[:, 0]].long(), unit] = scales[old[first[:, 0]].long(), unit]
    s["taken"].copy_(new.sum())
    if s["kind"] == "fork_free":
        rows = table[child]
        held = rows[rows >= 0].long()
        refs.index_add_(0, held, torch.full_like(rows[rows >= 0], -1))
        gone = torch.zeros_like(refs, dtype=torch.bool)
        gone[held] = True
        gone = (gone & (refs == 0)).nonzero()[:, 0]
        s["freed"][:gone.numel()] = gone.int()
        s["count"].fill_(gone.numel())
        table[child] = -1
    return _pages_out(s)


def _keys(s, slot):
    """The rows of the slots in 32 bits, their scales applied."""
    if s["scales"] is None:
        return s["cache"].view(-1, DIM)[slot].float()
    k = s["cache"].view(torch.uint8).view(-1, DIM)[slot].view(E4M3).float()
    return k.mul_(s["scales"][slot // s["group"]][..., None])


def _part(q, k, hidden):
    """Largest score, sum and weighted values of a set of keys; hidden ones left out."""
    sc = torch.matmul(q, k.transpose(-1, -2))
    if hidden is not None:
        sc.masked_fill_(hidden, -math.inf)
    m = sc.amax(-1)
    m0 = m.where(m > -math.inf, torch.zeros((), device=m.device))
    p = sc.sub_(m0[..., None]).exp_()
    return m, p.sum(-1), torch.matmul(p, k[..., :RANK])


def _plain_shared(s):
    bs, table, lens = s["block"], s["table"], s["lens"].long()
    T, H = s["q"].shape[:2]
    R, Q, dev = lens.numel(), s["max_q"], lens.device
    q = s["q"].float() * (SOFTMAX_SCALE * s["q_scale"])
    m = torch.full((T, H), -math.inf, device=dev)
    den = torch.zeros((T, H), device=dev)
    acc = torch.zeros((T, H, RANK), device=dev)
    begin = torch.zeros(R, dtype=torch.long, device=dev)  # first own key of each request
    for length, r0, r1, t0, t1 in s["host"]:             # the prefix, once for the requests of its group
        begin[r0:r1] = length
        if length:
            pos = torch.arange(length, device=dev)
            k = _keys(s, table[r0, pos // bs].long() * bs + pos % bs)
            gm, gl, go = _part(q[t0:t1].reshape(-1, DIM), k, None)
            m[t0:t1], den[t0:t1], acc[t0:t1] = gm.view(-1, H), gl.view(-1, H), go.view(-1, H, RANK)
    pos = begin[:, None] + torch.arange(max(s["max_own"], 1), device=dev)
    there = pos < lens[:, None]
    slot = (table.gather(1, (pos // bs).clamp(max=table.shape[1] - 1)).long() * bs + pos % bs).where(there, 0)
    k = _keys(s, slot)
    k.masked_fill_(~there[..., None], 0.0)
    start = s["qsl"].long() if s["qsl"] is not None else torch.arange(R + 1, device=dev)
    j, n = torch.arange(Q, device=dev), start[1:] - start[:-1]
    tok = (start[:-1, None] + j).clamp(max=T - 1)
    hidden = ~(there[:, None] & (pos[:, None] < (lens - n + 1)[:, None, None] + j[:, None]))
    hidden = hidden[:, :, None].expand(-1, -1, H, -1).reshape(R, Q * H, -1)
    om, ol, oo = _part(q[tok].reshape(R, Q * H, DIM), k, hidden)
    use = (j < n[:, None]).nonzero()                      # (request, row) of every token, in token order
    pick = lambda x, *d: x.view(R, Q, H, *d)[use[:, 0], use[:, 1]]
    om, ol, oo = pick(om), pick(ol), pick(oo, RANK)
    top = torch.maximum(m, om)
    if s["sinks"] is not None:
        top = torch.maximum(top, s["sinks"])
    top = top.where(top > -math.inf, torch.zeros((), device=dev))
    a, b = torch.exp(m - top), torch.exp(om - top)
    den = a * den + b * ol
    out = a[..., None] * acc + b[..., None] * oo
    if s["sinks"] is not None:
        den = den + torch.exp(s["sinks"] - top)
    out = out / den.where(den > 0, torch.ones((), device=dev))[..., None]
    return {"out": out.bfloat16(), "lse": top + den.log()}


# ---------------------------------------------------------------------------
# the work of one pass, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "rope":
        T, H = max(c["tokens"] - c["pad"], 0), c["heads"]
        return {"bytes": T * H * DIM * (2 + (1 if c["fp8"] else 2)) + T * ROPE * 4 + 4 * c["tokens"],
                "flops": 3.0 * T * (H + 1) * c["dim"]}
    if c["op"] == "pages":
        bs = c["block"]
        row = DIM + 4.0 / c["group"] if c["fp8"] else 2 * DIM
        if c["kind"] == "copy":
            n = max(1, int(c["blocks"] * c["live"]))
            return {"bytes": n * (2 * bs * row + 8), "flops": 0}
        ctx = _spread(c["prompts"], c["ctx_lo"], c["ctx_hi"])
        used, cells = int((-(-ctx // bs)).sum()), int((ctx // bs).sum()) * c["samples"]
        if c["kind"] == "compact":
            moved = used - _stay(c)
            cols = int((-(-ctx // bs)).max()) + 1
            return {"bytes": moved * 2 * bs * row + 8 * c["blocks"] + 8 * c["prompts"] * cols, "flops": 0}
        copied = int((ctx % bs).sum()) * c["samples"]
        # a cell read, one written and a count raised for every page shared; the same way back
        return {"bytes": 2 * copied * row + 16 * cells * (2 if c["kind"] == "fork_free" else 1), "flops": 0}
    prefix, own_len, q = _shared_lens(c)
    G, H, T = c["groups"], c["heads"], int(q.sum()) + c["alone"]
    edges = np.round(np.arange(G + 1) * c["reqs"] / G).astype(np.int64)
    per = np.diff(edges)
    el = 1 if c["fp8"] else 2
    keys = int(prefix.sum()) + int(own_len.sum())
    tokens = q.sum() / c["reqs"]                          # the mean of a request (their order is the seed's)
    pairs = float((prefix * per).sum()) * tokens + float((own_len * q).sum())
    return {"bytes": keys * (DIM * el + (4.0 / c["group"] if c["fp8"] else 0)) + T * H * (DIM * el + 2 * RANK + 4),
            "flops": 2.0 * pairs * H * (DIM + RANK)}


def exact(case, seed):
    if case["op"] == "pages":
        return None  # moved, counted and listed, not computed
    s = prepare(case, seed)
    return _exact_rope(s, case) if s["op"] == "rope" else _exact_shared(s)


def _exact_rope(s, c):
    """Each pair as a complex number, turned by the angle of its position."""
    d = c["dim"]
    freq, size = [], 1.0
    for i in range(d // 2):
        f = math.exp(-2.0 * i / d * math.log(ROPE_BASE))
        if c["scaling"] == "linear":
            f /= ROPE_FACTOR
        elif c["scaling"] == "yarn":
            edge = [d / 2 * math.log(ROPE_ORIGINAL / (2 * math.pi * b), ROPE_BASE) for b in (32, 1)]
            lo, hi = max(0, math.floor(edge[0])), min(d - 1, math.ceil(edge[1]))
            w = min(1.0, max(0.0, (i - lo) / (hi - lo if hi != lo else 0.001)))
            f = f * (1 - w) + f * w / ROPE_FACTOR
        freq.append(f)
    if c["scaling"] == "yarn":
        size = (1 + 0.1 * ROPE_MSCALE * math.log(ROPE_FACTOR)) / (1 + 0.1 * ROPE_MSCALE_ALL * math.log(ROPE_FACTOR))
    angle = s["pos"].double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    unit = torch.polar(torch.full_like(angle, size), angle)

    def turn(x, unit):
        x = x.double()
        if s["half"]:
            z = torch.complex(x[..., :d // 2], x[..., d // 2:d]) * unit
            return torch.cat([z.real, z.imag, x[..., d:]], -1)
        z = torch.view_as_complex(x[..., :d].contiguous().view(*x.shape[:-1], d // 2, 2)) * unit
        return torch.cat([torch.view_as_real(z).flatten(-2), x[..., d:]], -1)
    live = s["pos"] >= 0
    q = torch.cat([s["nope"].double(), turn(s["q_pe"], unit[:, None])], -1)
    if s["fp8"]:
        q = (q / Q_SCALE).clamp(-448, 448)
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    return {"q": q.where(live[:, None, None], zero), "k": turn(s["k_pe"], unit).where(live[:, None], zero)}


def _exact_shared(s):
    """Token after token, each over all the keys that its own request's pages hold."""
    T, H = s["q"].shape[:2]
    table, lens = s["table"].cpu().numpy().astype(np.int64), s["lens"].cpu().numpy()
    edges = s["qsl"].cpu().numpy() if s["qsl"] is not None else np.arange(len(lens) + 1)
    out = torch.zeros((T, H, RANK), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    for r in range(len(lens)):
        slots = (table[r][:, None] * s["block"] + np.arange(s["block"])).reshape(-1)[:int(lens[r])]
        at = torch.from_numpy(slots).cuda()
        if s["scales"] is None:
            kv = s["cache"].view(-1, DIM)[at].double()
        else:
            kv = s["cache"].view(torch.uint8).view(-1, DIM)[at].view(E4M3).double()
            kv = kv * s["scales"].double()[at // s["group"]][:, None]
        n = int(edges[r + 1] - edges[r])
        for i in range(n):
            t, seen = int(edges[r]) + i, max(0, int(lens[r]) - n + 1 + i)
            z = [(s["q"][t].double() * (s["q_scale"] * SOFTMAX_SCALE)) @ kv[:seen].T] if seen else []
            if s["sinks"] is not None:
                z.append(s["sinks"].double()[:, None])
            if not z:
                continue
            z = torch.cat(z, 1)
            lse[t] = torch.logsumexp(z, 1)
            if seen:
                out[t] = torch.exp(z[:, :seen] - lse[t][:, None]) @ kv[:seen, :RANK]
    return {"out": out, "lse": lse}

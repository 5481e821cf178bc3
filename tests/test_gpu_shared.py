"""The decode of a batch that shares prefixes on the GPU, against the oracle's
attention of each token over all its keys, within bounds derived element by
element. Unused rows, scales and table cells hold NaN or point at blocks that do."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from oracle import scaled_oracle as S
from oracle import step_oracle as P
from paged_mla_decode_06_gb300 import binding as B
from paged_mla_decode_06_gb300 import build as BUILD
from paged_mla_decode_06_gb300 import inputs as I

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(192.0)
QS, KVS = 2.0 ** -6, 0.25


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    BUILD.build()
    B.load_library()


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def bf16(x):
    t = torch.from_numpy(np.asarray(x, np.float32)).bfloat16()
    return t.double().numpy(), t


def shared_case(seed, kind, heads, bs, g, groups, alone=(), qlens=None, sinks=False, pad=0, spread=1.0):
    """``groups``: [(prefix, own lengths of its requests)], ``alone``: lengths of
    requests of no group behind them. ``kind``: "scaled", "fp8" or "bf16"."""
    rng = np.random.default_rng(seed)
    lens, prefix, edges = [], [], [0]
    for p, own in groups:
        prefix.append(p)
        lens += [p + o for o in own]
        edges.append(len(lens))
    lens = np.array(lens + list(alone), np.int64)
    need = -(-lens // bs)
    cols = max(1, int(need.max())) + 2
    total = int(need.sum()) + 1
    ids = list(rng.permutation(total))
    trap = ids.pop()
    table = np.full((len(lens), cols), trap)
    for (p, own), a, b in zip(groups, edges, edges[1:]):
        common = [ids.pop() for _ in range(p // bs if own else 0)]
        for r in range(a, b):
            n = min(int(need[r]), len(common))
            table[r, :n] = common[:n]
            for c in range(n, int(need[r])):
                table[r, c] = ids.pop()
    for r in range(edges[-1], len(lens)):
        for c in range(int(need[r])):
            table[r, c] = ids.pop()
    live = np.zeros(total * bs, bool)
    for r in range(len(lens)):
        live[S.row_slots(table[r], bs, int(lens[r]))] = True
    n = total * bs
    rows = bf16(rng.standard_normal((n, 576)) * np.exp(0.5 * spread * rng.standard_normal((n, 1))))[0]
    q = np.ones(len(lens), np.int64) if qlens is None else np.asarray(qlens)
    qo = np.concatenate([[0], np.cumsum(q)])
    T = int(qo[-1]) + pad
    x = rng.standard_normal((T, heads, 576)).astype(np.float32)
    c = dict(kind=kind, lens=lens, table=table, qo=qo, has_qo=qlens is not None or pad > 0, T=T, H=heads, bs=bs, g=g,
             nb=total, prefix=np.array(prefix), edges=np.array(edges), max_qlen=int(q.max()), live=live, pad=pad,
             sinks=rng.standard_normal(heads).astype(np.float32) if sinks else None)
    if kind == "bf16":
        rows[~live] = np.nan
        c["values"], c["kv"] = bf16(rows)
        c["q64"], c["q"] = bf16(x)
        return c
    if kind == "scaled":
        codes, scales = S.cache_append(rows, np.arange(n), np.zeros((n, 576), np.uint8), np.zeros(n // g), g)
        scales = (scales * rng.uniform(0.6, 1.4, scales.shape)).astype(np.float32).astype(np.float64)
        scales[~live.reshape(-1, g).any(1)] = np.nan
    else:
        codes, scales = I.float32_to_e4m3_codes((rows / KVS).astype(np.float32)), np.full(n // g, KVS)
    codes[~live] = 0x7F
    c.update(codes=codes, scales=scales, q=I.float32_to_e4m3_codes(x / QS))
    return c


def plan_of(c, **kw):
    return B.mla_decode_shared_plan(B.make_problem(
        num_tokens=c["T"], num_heads=c["H"], block_size=c["bs"], num_blocks=c["nb"], num_reqs=len(c["lens"]),
        max_blocks_per_req=c["table"].shape[1], max_seq_len=int(c["lens"].max()), max_qlen=c["max_qlen"],
        dtype="bf16" if c["kind"] == "bf16" else "fp8", has_sinks=c["sinks"] is not None, **kw),
        num_groups=len(c["prefix"]))


def args_of(c, plan):
    scaled = c["kind"] == "scaled"
    if c["kind"] == "bf16":
        q, kv = c["q"].cuda(), c["kv"].cuda().view(c["nb"], c["bs"], 576)
    else:
        q, kv = dev(c["q"]), dev(c["codes"]).view(c["nb"], c["bs"], 576)
    return (plan, q, kv), dict(
        kv_scales=dev(c["scales"], np.float32) if scaled else None, scale_group=c["g"] if scaled else 0,
        block_table=dev(c["table"], np.int32), seq_lens=dev(c["lens"], np.int32),
        qo_indptr=dev(c["qo"], np.int32) if c["has_qo"] else None, prefix_lens=dev(c["prefix"], np.int32),
        group_indptr=dev(c["edges"], np.int32), softmax_scale=SCALE, q_scale=1.0 if c["kind"] == "bf16" else QS,
        kv_scale=KVS if c["kind"] == "fp8" else 1.0, sinks=None if c["sinks"] is None else dev(c["sinks"]),
        workspace=torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda"),
        out=torch.full((c["T"], c["H"], 512), 3.0, dtype=torch.bfloat16, device="cuda"),
        lse=torch.full((c["T"], c["H"]), 3.0, device="cuda"))


def run_case(c, **kw):
    plan = plan_of(c, **kw)
    args, named = args_of(c, plan)
    B.mla_decode_fwd_shared(*args, **named)
    torch.cuda.synchronize()
    assert B.mla_workspace_status(plan.plan, named["workspace"]) == 0
    return named["out"].double().cpu().numpy(), named["lse"].double().cpu().numpy(), (args, named)


def weight_terms(c, lists, out, tol):
    """What the bounds of ``S.decode`` leave out for a weight p' of which the first term
    is e5m2 and the rest e4m3 (the row's largest at p' >= 2^4 again). The first is off by
    2^-3 of p' at most and the rest by 2^-4 of that, as there; a rest below 2^-6 is
    off by half of e4m3's smallest step, 2^-10, 2^-14 of the largest weight, and by no
    more than itself, 2^-3 of the weight. (A first term below 2^-14 is off by 2^-17 at
    most, 2^-21 of the largest.) The output's own rounding multiplies that by 1 + 2^-8."""
    q = O.decode_e4m3fn(c["q"]) * QS
    for t, slots in enumerate(lists):
        slots = np.asarray(slots, np.int64)
        slots = slots[slots >= 0]
        if not len(slots):
            continue
        s, k = c["scales"][slots // c["g"]], O.decode_e4m3fn(c["codes"][slots])
        z = SCALE * (q[t] @ (k * s[:, None]).T)
        ws = np.exp(z - np.logaddexp.reduce(z, axis=1)[:, None]) * s
        err = np.minimum(2.0 ** -14 * ws.max(1)[:, None], 2.0 ** -3 * ws)
        tol[t] += err @ np.abs(k[:, :512]) * (1 + 2.0 ** -8)


def expected(c):
    lists = S.token_slots(c["table"], c["lens"], c["bs"], c["qo"])
    if c["kind"] != "bf16":
        out, lse, to, tl = S.decode(c["q"][:len(lists)], QS, c["codes"], c["scales"], c["g"], lists, SCALE, c["sinks"],
                                    bounds=True)
        weight_terms(c, lists, out, to)
        return out, lse, to, tl
    T, H = len(lists), c["H"]
    out, lse = np.zeros((T, H, 512)), np.full((T, H), -np.inf)
    to, tl = np.zeros_like(out), np.zeros_like(lse)
    for t, slots in enumerate(lists):
        slots = np.asarray(slots, np.int64)
        slots = slots[slots >= 0]
        kv = c["values"][slots]
        out[t], lse[t] = S.attend(c["q64"][t], kv, SCALE, c["sinks"])
        if not len(slots):
            tl[t] = 0.0 if c["sinks"] is None else np.abs(c["sinks"]) * 2.0 ** -22
            continue
        # scores: 576 additions at 2^-23 of the magnitudes; weights rounded to bf16, the output too
        z = SCALE * (c["q64"][t] @ kv.T)
        mags = SCALE * (np.abs(c["q64"][t]) @ np.abs(kv).T)
        gamma = 576 * 2.0 ** -23 * mags.max(1) + (np.abs(z).max(1) / np.log(2) + 8) * 2.0 ** -21 + len(slots) * 2.0 ** -25
        w = np.exp(z - lse[t][:, None])
        to[t] = ((2.0 ** -8 + 2 * gamma[:, None]) * w) @ np.abs(kv[:, :512]) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(out[t])
        tl[t] = gamma + np.abs(lse[t]) * 2.0 ** -22 + (0.0 if c["sinks"] is None else np.abs(c["sinks"]) * 2.0 ** -22)
    return out, lse, to, tl


def compare(c, out, lse):
    ro, rl, to, tl = expected(c)
    n = ro.shape[0]
    assert np.isfinite(out[:n]).all()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse[:n]), empty)
    d = np.abs(out[:n] - ro) - to
    assert d.max() <= 0, (np.unravel_index(d.argmax(), d.shape), d.max(), np.abs(out[:n] - ro).max())
    e = np.where(empty, 0.0, np.abs(lse[:n] - np.where(empty, 0.0, rl)) - tl)
    assert np.where(empty, -1.0, e).max() <= 0, e.max()
    assert (out[n:] == 3.0).all() and (lse[n:] == 3.0).all()


def check(c, **kw):
    out, lse, rest = run_case(c, **kw)
    compare(c, out, lse)
    return out, lse, rest


KINDS = [("scaled", 64, 64), ("scaled", 64, 1), ("scaled", 16, 16), ("scaled", 48, 24), ("scaled", 32, 8),
         ("scaled", 128, 32), ("fp8", 64, 64), ("fp8", 16, 16), ("bf16", 64, 64), ("bf16", 128, 128)]


@pytest.mark.parametrize("kind,bs,g", KINDS)
def test_one_group(kind, bs, g):
    check(shared_case(bs + g, kind, 16, bs, g, [(300, [1, 37, 64, 129])]))


@pytest.mark.parametrize("kind,bs,g", KINDS)
@pytest.mark.parametrize("heads", [1, 17, 128])
def test_heads_and_sinks(kind, bs, g, heads):
    check(shared_case(heads, kind, heads, bs, g, [(777, [5, 1, 200])], alone=[0, 90], sinks=True))


@pytest.mark.parametrize("kind,bs,g", KINDS)
def test_groups_of_several_tokens(kind, bs, g):
    """Two groups and lone requests, one to four tokens each, so that tiles mix tokens
    of requests, causal rows end inside a group of keys, and padding follows."""
    check(shared_case(3, kind, 33, bs, g, [(130, [4, 9, 300]), (1000, [3, 140])], alone=[2, 260],
                      qlens=[1, 3, 4, 2, 3, 2, 1], pad=3))


@pytest.mark.parametrize("kind,bs,g", [("scaled", 64, 64), ("scaled", 16, 2), ("fp8", 64, 64), ("bf16", 64, 64)])
@pytest.mark.parametrize("prefix,own", [
    (0, [5, 700]), (1, [1, 1]), (63, [64, 65]), (64, [1, 1]), (128, [128, 128, 256]), (4000, [1, 2, 3, 4, 5, 6, 7, 8]),
    (191, [500, 1]), (20000, [3, 2000])])
def test_lengths(kind, bs, g, prefix, own):
    check(shared_case(prefix, kind, 24, bs, g, [(prefix, own)]))


@pytest.mark.parametrize("kind", ["scaled", "bf16"])
def test_many_requests_and_one_long_own_part(kind):
    check(shared_case(8, kind, 8, 64, 64, [(600, [1 + (i * 37) % 300 for i in range(90)] + [9000])]))


@pytest.mark.parametrize("kind", ["scaled", "fp8", "bf16"])
def test_requests_too_short_for_their_prefix_are_decoded_on_their_own(kind):
    """Members that do not see all of the prefix (padding among them) take no part: their
    rows are right by their own tables; so is the only member that is left."""
    c = shared_case(11, kind, 20, 64, 64, [(640, [10, 20, 30, 40]), (256, [9, 7])], qlens=[1, 2, 3, 1, 1, 1])
    full = c["lens"].copy()
    for lens in ([650, 0, 3, 680, 265, 263], [650, 641, 642, 680, 265, 263], [10, 20, 30, 680, 265, 100], [1, 2, 3, 4, 5, 0]):
        c["lens"] = np.array(lens)
        # rows behind the new ends hold what the requests had there: right codes, not NaN
        out, lse, _ = run_case(c)
        compare(c, out, lse)
    c["lens"] = full
    check(c)


def test_first_member_takes_no_part():
    c = shared_case(12, "scaled", 16, 64, 16, [(320, [5, 6, 7])])
    c["lens"][0] = 0
    c["table"][0, :] = c["table"][0, -1]  # not even its table row is read
    check(c)


@pytest.mark.parametrize("kind", ["scaled", "fp8", "bf16"])
def test_groups_by_default_and_empty_groups(kind):
    c = shared_case(13, kind, 16, 64, 64, [(512, [3, 200, 70])])
    plan = plan_of(c)
    args, named = args_of(c, plan)
    named["group_indptr"] = None
    B.mla_decode_fwd_shared(*args, **named)
    torch.cuda.synchronize()
    compare(c, named["out"].double().cpu().numpy(), named["lse"].double().cpu().numpy())
    c = shared_case(14, kind, 16, 64, 64, [(512, []), (300, [3, 200]), (100, []), (64, [1, 2, 70]), (999, [])])
    check(c)


def test_more_groups_than_the_schedule_caches():
    groups = [(64 + 64 * (i % 3), [1 + i % 5, 2 + i % 70]) for i in range(300)]
    check(shared_case(15, "scaled", 4, 64, 64, groups))


@pytest.mark.parametrize("kind,bs", [("scaled", 16), ("bf16", 64)])
def test_more_requests_than_the_schedule_caches(kind, bs):
    groups = [(3 * bs + 200, [1 + (i * j) % 60 for i in range(370)]) for j in (3, 5, 7)]
    check(shared_case(27, kind, 2, bs, bs, groups, alone=[5, 300]))


def test_repeated_calls_leave_no_status():
    """Waits that are passed over, or that take another phase for theirs, show in some
    call of many."""
    c = shared_case(28, "scaled", 32, 64, 1, [(1500 + 700 * i, [3 + 97 * j % 700 for j in range(8)]) for i in range(6)],
                    qlens=[1 + i % 3 for i in range(48)])
    args, named = args_of(c, plan_of(c))
    for _ in range(1500):
        B.mla_decode_fwd_shared(*args, **named)
    torch.cuda.synchronize()
    assert B.mla_workspace_status(args[0].plan, named["workspace"]) == 0
    compare(c, named["out"].double().cpu().numpy(), named["lse"].double().cpu().numpy())


def test_uneven_scales_and_a_key_that_outweighs_the_rest():
    c = shared_case(16, "scaled", 20, 64, 1, [(1500, [3, 400, 64])])
    rng = np.random.default_rng(0)
    ok = ~np.isnan(c["scales"])
    c["scales"][ok] *= np.exp2(rng.integers(-12, 3, int(ok.sum())))
    check(c)
    c["scales"][c["table"][0, 2] * 64 + 5] *= 2.0 ** 12   # of the prefix
    check(c)
    c["scales"][c["table"][1, 25] * 64 + 7] *= 2.0 ** 13  # of one request
    check(c)


def test_nan_keys_reach_the_rows_that_see_them_and_no_others():
    for bs, g in ((64, 16), (16, 1)):
        c = shared_case(17, "scaled", 24, bs, g, [(256, [6, 5]), (320, [70, 4])], qlens=[4, 1, 3, 2])
        ro, rl, to, tl = expected(c)
        bad = [S.row_slots(c["table"][0], bs, 262)[261], S.row_slots(c["table"][2], bs, 390)[388],
               S.row_slots(c["table"][3], bs, 324)[7]]   # the last is in the second group's prefix
        for i, slot in enumerate(bad):
            codes = c["codes"].copy()
            codes[slot, 11] = 0x7F                        # a value column
            out, lse, _ = run_case(dict(c, codes=codes))
            seen = [slot in np.asarray(s) for s in S.token_slots(c["table"], c["lens"], bs, c["qo"])]
            assert any(seen) and not all(seen)
            for t, s in enumerate(seen):
                assert np.isnan(lse[t]).all() == s and np.isnan(lse[t]).any() == s, (i, t)
                assert np.isnan(out[t]).any() == s
                if not s:
                    assert np.all(np.abs(out[t] - ro[t]) <= to[t])


def test_nan_and_infinite_queries_stay_in_their_rows():
    c = shared_case(18, "scaled", 24, 64, 64, [(256, [6, 5, 9])])
    ro, rl, to, tl = expected(c)
    q = c["q"].copy()
    q[1, 3, 500] = 0x7F
    out, lse, _ = run_case(dict(c, q=q))
    odd = np.zeros(lse.shape, bool)
    odd[1, 3] = True
    assert np.array_equal(np.isnan(lse), odd) and np.isnan(out[1, 3]).all()
    assert np.all((np.abs(out - ro) <= to)[~odd])


def test_sinks_of_minus_infinity_and_nan():
    c = shared_case(19, "scaled", 16, 64, 64, [(256, [6, 5])], alone=[0, 70], sinks=True)
    c["sinks"][:] = -np.inf
    plain = dict(c, sinks=None)
    a, al, _ = run_case(c)
    b, bl, _ = run_case(plain)
    assert np.array_equal(a, b) and np.array_equal(al, bl)
    c["sinks"][:] = 0.5
    c["sinks"][4] = np.nan
    out, lse, _ = run_case(c)
    odd = np.zeros(lse.shape, bool)
    odd[:, 4] = True
    assert np.array_equal(np.isnan(lse), odd)
    # (a row without keys has an output of zeros, whatever its sink)
    assert np.isnan(out[[0, 1, 3]][:, 4]).all()


def test_missing_blocks_are_skipped():
    """Cells without a block, in the prefix and in the own part: their keys are left out."""
    for bs in (64, 16):
        c = shared_case(20, "scaled", 20, bs, 8, [(512, [300, 70, 9])])
        c["table"][:, 128 // bs] = -1
        c["table"][0, 600 // bs] = -1
        check(c)


@pytest.mark.parametrize("kind,bs,kw", [("scaled", 8, {}), ("fp8", 8, {}), ("bf16", 16, {}), ("bf16", 48, {}),
                                        ("scaled", 64, dict(num_segments=3)),
                                        ("scaled", 64, dict(kernel=B.MLA_KERNEL_WARP_MMA))])
def test_plans_that_share_nothing_run_as_the_plain_decode(kind, bs, kw):
    c = shared_case(21, kind, 16, bs, bs, [(300, [9, 70])], alone=[31])
    assert plan_of(c, **kw).max_items == 0
    check(c, **kw)


@pytest.mark.parametrize("kind", ["scaled", "fp8", "bf16"])
def test_same_bits_on_every_run_and_like_the_plain_decode(kind):
    c = shared_case(22, kind, 128, 64, 64, [(3000, [1 + 97 * i % 1500 for i in range(12)])], sinks=True)
    out, lse, (args, named) = check(c)
    for _ in range(3):
        named["out"].fill_(0), named["lse"].fill_(0)
        B.mla_decode_fwd_shared(*args, **named)
        torch.cuda.synchronize()
        assert np.array_equal(named["out"].double().cpu().numpy(), out)
        assert np.array_equal(named["lse"].double().cpu().numpy(), lse)


def test_captured_and_replayed_with_other_lengths():
    c = shared_case(23, "scaled", 16, 64, 64, [(640, [300, 200, 100]), (320, [64, 65])], pad=2)
    plan = plan_of(c)
    args, named = args_of(c, plan)
    call = lambda: B.mla_decode_fwd_shared(*args, **named)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    full = c["lens"].copy()
    for lens, prefix, edges in ((full, [640, 320], [0, 3, 5]), (full - [200, 5, 99, 60, 0], [640, 320], [0, 3, 5]),
                                (full, [64, 1], [0, 2, 5]), (full, [130, 320], [1, 3, 4]), (full, [0, 0], [0, 3, 5])):
        c["lens"] = np.array(lens)
        named["seq_lens"].copy_(dev(lens, np.int32))
        named["prefix_lens"].copy_(dev(prefix, np.int32))
        named["group_indptr"].copy_(dev(edges, np.int32))
        named["out"].fill_(3.0), named["lse"].fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        assert B.mla_workspace_status(plan.plan, named["workspace"]) == 0
        compare(c, named["out"].double().cpu().numpy(), named["lse"].double().cpu().numpy())


def test_two_streams_at_once():
    cases = [shared_case(24 + i, "scaled", 64, 64, 64, [(2000, [100, 200, 300, 400])]) for i in range(2)]
    runs = []
    for c in cases:
        args, named = args_of(c, plan_of(c))
        runs.append((c, args, named, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for c, args, named, s in runs:
            with torch.cuda.stream(s):
                B.mla_decode_fwd_shared(*args, **named)
    torch.cuda.synchronize()
    for c, _, named, _ in runs:
        compare(c, named["out"].double().cpu().numpy(), named["lse"].double().cpu().numpy())


@pytest.mark.parametrize("kind,heads", [("scaled", 128), ("scaled", 16), ("fp8", 128), ("bf16", 128)])
def test_bounded_wait_runs_out_and_is_reported(kind, heads):
    c = shared_case(26, kind, heads, 64, 64, [(4096, [700, 90, 300, 50])])
    plan = plan_of(c)
    args, named = args_of(c, plan)
    plan.plan.wait_limit_us = 1
    B.mla_decode_fwd_shared(*args, **named)     # gives up, and returns
    torch.cuda.synchronize()
    assert B.mla_workspace_status(plan.plan, named["workspace"], clear=True) != 0
    plan.plan.wait_limit_us = 0
    B.mla_decode_fwd_shared(*args, **named)
    torch.cuda.synchronize()
    assert B.mla_workspace_status(plan.plan, named["workspace"]) == 0
    compare(c, named["out"].double().cpu().numpy(), named["lse"].double().cpu().numpy())


# ---- prefixes long enough, and read by enough requests, to be shared
def shared_groups(c):
    """Of each group, whether its prefix is computed once: the tiles that its participants
    have fewer in common, times the prefix's groups of 128 keys, are at least 6 times theirs."""
    qlens, found = np.diff(c["qo"]), []
    tiles = lambda tokens: -(-int(tokens) * c["H"] // 128)
    for p, a, b in zip(c["prefix"], c["edges"], c["edges"][1:]):
        keys = int(p) // c["bs"] * c["bs"]
        own = sum(tiles(qlens[r]) for r in range(a, b) if qlens[r] > 0 and c["lens"][r] - qlens[r] >= keys)
        found.append(keys > 0 and own > 0 and (own - tiles(qlens[a:b].sum())) * -(-keys // 128) >= 6 * own)
    return found


@pytest.mark.parametrize("kind,bs,g,heads", [(*k, h) for k in KINDS for h in (7, 64)]
                         + [(*k, h) for k in (KINDS[0], KINDS[1], KINDS[-2]) for h in (1, 16, 33)])
def test_shared_tiles_of_many_requests(kind, bs, g, heads):
    """Two groups, one to four tokens a request, lone requests and padding behind them."""
    several = heads <= 16
    c = shared_case(heads, kind, heads, bs, g, [(1599, [1 + 53 * i % 400 + 3 for i in range(12)]), (1664, [4, 700] * 5)],
                    alone=[0, 1, 260], qlens=[1 + i % 4 if several else 1 for i in range(22)] + [1, 1, 2], sinks=heads in (7, 33),
                    pad=2)
    assert shared_groups(c) == [True, True]
    check(c)


@pytest.mark.parametrize("kind", ["scaled", "fp8", "bf16"])
@pytest.mark.parametrize("prefix", [832, 850, 896, 1023, 1024, 8192])
def test_shared_prefixes_of_any_length(kind, prefix):
    c = shared_case(prefix, kind, 8, 64, 64, [(prefix, [1, 64, 65, 127, 128, 129, 300, 2, 3, 4, 5, 6, 7, 1, 1, 900])])
    assert shared_groups(c) == [True]
    check(c)


@pytest.mark.parametrize("bs,g", [(64, 16), (16, 1), (48, 48)])
def test_nan_keys_of_a_shared_prefix_and_behind_it(bs, g):
    c = shared_case(40, "scaled", 24, bs, g, [(1536, [6, 5, 9, 70, 3, 140, 8, 8]), (2048, [70, 4, 4, 6, 9, 30, 7, 5])],
                    qlens=[4, 1, 3, 2, 1, 1, 1, 1] + [1, 2, 3, 1, 1, 4, 1, 1])
    assert shared_groups(c) == [True, True]
    ro, rl, to, tl = expected(c)
    for r, at in ((0, 1541), (3, 1604), (9, 7), (0, 1000), (13, 2060)):
        slot = S.row_slots(c["table"][r], bs, at + 1)[at]
        codes = c["codes"].copy()
        codes[slot, 11] = 0x7F                            # a value column
        out, lse, _ = run_case(dict(c, codes=codes))
        seen = [slot in np.asarray(s) for s in S.token_slots(c["table"], c["lens"], bs, c["qo"])]
        assert any(seen) and not all(seen)
        for t, s in enumerate(seen):
            assert np.isnan(lse[t]).all() == s and np.isnan(lse[t]).any() == s, (r, at, t)
            assert np.isnan(out[t]).any() == s
            if not s:
                assert np.all(np.abs(out[t] - ro[t]) <= to[t]) and np.all(np.abs(lse[t] - rl[t]) <= tl[t])


def test_odd_queries_and_sinks_over_a_shared_prefix():
    c = shared_case(41, "scaled", 24, 64, 64, [(1600, [6, 5, 9, 1, 2, 3, 80, 4])], sinks=True)
    assert shared_groups(c) == [True]
    ro, rl, to, tl = expected(c)
    odd = np.zeros(rl.shape, bool)
    q, sinks = c["q"].copy(), c["sinks"].copy()
    q[1, 3, 500], sinks[4] = 0x7F, np.nan
    odd[1, 3] = odd[:, 4] = True
    out, lse, _ = run_case(dict(c, q=q, sinks=sinks))
    assert np.array_equal(np.isnan(lse), odd) and np.isnan(out[odd]).all()
    assert np.all((np.abs(out - ro) <= to)[~odd]) and np.all((np.abs(lse - rl) <= tl)[~odd])
    sinks[:] = -np.inf
    a, al, _ = run_case(dict(c, sinks=sinks))
    b, bl, _ = run_case(dict(c, sinks=None))
    assert np.array_equal(a, b) and np.array_equal(al, bl)


@pytest.mark.parametrize("bs,g", [(64, 8), (16, 16), (32, 1)])
def test_missing_blocks_of_a_shared_prefix(bs, g):
    c = shared_case(42, "scaled", 20, bs, g, [(1664, [300, 70, 9, 33, 64, 1, 2, 3])])
    assert shared_groups(c) == [True]
    c["table"][:, 128 // bs] = -1
    c["table"][:, 1024 // bs:1152 // bs] = -1             # a whole chunk of keys
    c["table"][0, 1750 // bs] = -1
    check(c)
    c["table"][:, :1664 // bs] = -1                       # the whole prefix
    check(c)


@pytest.mark.parametrize("kind", ["scaled", "fp8", "bf16"])
def test_members_that_take_no_part_in_a_shared_prefix(kind):
    """Requests too short for their group's prefix are decoded on their own, the first of
    them too, whose table row is then not the prefix's."""
    c = shared_case(43, kind, 12, 64, 64, [(1280, [5 + 7 * i for i in range(14)]), (1408, [4] * 12)],
                    qlens=[1 + i % 3 for i in range(26)])
    full = c["lens"].copy()
    for cut in ({0: 0}, {0: 1, 5: 1280, 6: 0, 25: 1000}, {r: 1281 for r in range(0, 14, 3)}, {r: r for r in range(3, 26)}):
        c["lens"] = full.copy()
        for r, n in cut.items():
            c["lens"][r] = n
        out, lse, _ = run_case(c)
        compare(c, out, lse)
    c["lens"] = full.copy()
    c["lens"][0] = 0
    c["table"][0, :] = c["table"][0, -1]
    assert all(shared_groups(c))
    check(c)


@pytest.mark.parametrize("kind", ["scaled", "bf16"])
def test_shared_prefixes_captured_and_replayed_with_other_groups(kind):
    c = shared_case(44, kind, 16, 64, 64, [(1600, [300, 200, 100, 5, 6, 7, 8, 9]), (2000, [64, 65] * 4)], pad=2)
    plan = plan_of(c)
    args, named = args_of(c, plan)
    call = lambda: B.mla_decode_fwd_shared(*args, **named)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    full, found = c["lens"].copy(), set()
    for lens, prefix, edges in ((full, [1600, 2000], [0, 8, 16]), (full - 4, [1600, 2000], [0, 8, 16]),
                                (full, [64, 1999], [0, 8, 16]), (full, [1600, 0], [0, 3, 16]), (full, [1000, 1300], [1, 8, 12]), (full, [0, 0], [0, 8, 16]),
                                (full, [1600, 1216], [0, 8, 16]), (full * 0, [1600, 2000], [0, 8, 16]),
                                (full, [1600, 2000], [8, 0, 16]), (full, [1600, 1600], [0, 16, 8]),
                                (full, [1600, 2000], [-5, 8, 99]), (full, [10 ** 9, -7], [0, 8, 16])):
        c.update(lens=np.array(lens), prefix=np.array(prefix), edges=np.array(edges))
        found.add(tuple(shared_groups(c)) if edges == sorted(edges) and 0 <= edges[0] and edges[-1] <= 16 else None)
        named["seq_lens"].copy_(dev(lens, np.int32))
        named["prefix_lens"].copy_(dev(prefix, np.int32))
        named["group_indptr"].copy_(dev(edges, np.int32))
        named["out"].fill_(3.0), named["lse"].fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        assert B.mla_workspace_status(plan.plan, named["workspace"]) == 0
        compare(c, named["out"].double().cpu().numpy(), named["lse"].double().cpu().numpy())
    assert {(True, True), (False, False)} <= found


def test_empty_requests_in_a_row():
    """Requests without keys, many of them one after another among long ones: their rows
    are written, and no wait of the loads takes one's output for another's."""
    for seed, kind in ((46, "scaled"), (47, "fp8"), (48, "bf16")):
        c = shared_case(seed, kind, 16, 64, 64, [(1600, [5 + 40 * i for i in range(10)])],
                        alone=[0] * 90 + [700, 0, 0, 0, 300, 0, 5] + [0] * 60, sinks=seed == 46)
        check(c)
        c = shared_case(seed, kind, 128, 64, 64, [(1600, [5, 700])], alone=[0] * 40 + [900] + [0] * 41)
        check(c)


@pytest.mark.parametrize("kind", ["scaled", "bf16"])
@pytest.mark.parametrize("kw", [dict(num_sms=1), dict(num_sms=7), dict(num_sms=600), dict(max_qlen=9),
                                dict(max_seq_len=2048)])
def test_plans_for_other_bounds(kind, kw):
    """Fewer and more workers than the GPU has, looser bounds than the call's."""
    c = shared_case(49, kind, 16, 64, 64, [(1600, [5 + 40 * i for i in range(10)])], alone=[0, 700],
                    qlens=[1, 2, 3] * 4)
    assert shared_groups(c) == [True]
    p = B.make_problem(**dict(dict(
        num_tokens=c["T"], num_heads=16, block_size=64, num_blocks=c["nb"], num_reqs=len(c["lens"]),
        max_blocks_per_req=c["table"].shape[1], max_seq_len=int(c["lens"].max()), max_qlen=3,
        dtype="bf16" if kind == "bf16" else "fp8"), **kw))
    plan = B.mla_decode_shared_plan(p, num_groups=1)
    args, named = args_of(c, plan)
    B.mla_decode_fwd_shared(*args, **named)
    torch.cuda.synchronize()
    assert B.mla_workspace_status(plan.plan, named["workspace"]) == 0
    compare(c, named["out"].double().cpu().numpy(), named["lse"].double().cpu().numpy())


@pytest.mark.parametrize("kind", ["scaled", "bf16"])
def test_tokens_before_the_first_request_are_left(kind):
    c = shared_case(50, kind, 16, 64, 64, [(1600, [5 + 40 * i for i in range(10)])], qlens=[1, 2] * 5, pad=2)
    d = dict(c, qo=c["qo"] + 2, q=(torch.roll if kind == "bf16" else np.roll)(c["q"], 2, 0))
    out, lse, _ = run_case(d)
    assert (out[:2] == 3.0).all() and (lse[:2] == 3.0).all()
    n = len(out) - 2
    c["T"], c["pad"] = n, 0
    compare(c, out[2:], lse[2:])


@pytest.mark.parametrize("kind", ["scaled", "fp8", "bf16"])
def test_requests_of_several_tiles(kind):
    c = shared_case(51, kind, 128, 64, 64, [(1300, [4, 90, 300])], alone=[2, 500], qlens=[4, 1, 3, 2, 4], sinks=True)
    check(c)


@pytest.mark.parametrize("groups", [2, 300])
def test_groups_that_overlap_share_nothing(groups):
    """An entry of group_indptr below the one before it: every request on its own."""
    c = shared_case(45, "scaled", 8, 64, 64, [(1280, [5 + 7 * i for i in range(12)])])
    c["prefix"] = np.full(groups, 1280)
    c["edges"] = np.array(([0, 12] * groups)[:groups + 1])
    check(c)


@pytest.mark.parametrize("L", [333, 1400])
def test_fork_then_decode_over_the_shared_pages(L):
    """Samples of a prompt as a server makes them: fork, block tables, rotary
    positions, append, the shared decode; then losers freed and the pool compacted, and
    another step."""
    rng = np.random.default_rng(30)
    bs, g, H, n = 64, 16, 16, 5
    nb, cols, rows_n = 60, L // 64 + 7, n + 1
    codes, scales = np.zeros((nb * bs, 576), np.uint8), np.full(nb * bs // g, np.nan)
    prompt = bf16(rng.standard_normal((L, 576)))[0]
    ids = rng.permutation(nb)
    need = -(-L // bs)
    table = np.full((rows_n, cols), -1)
    table[0, :need] = ids[:need]
    slots = S.row_slots(table[0], bs, L)
    codes, scales = S.cache_append(prompt, slots, codes, scales, g)
    refs = np.zeros(nb, np.int64)
    refs[ids[:need]] = 1
    free = ids[need:]
    T_, R_ = dev(table, np.int32), dev(refs, np.int32)
    kv, sc = dev(codes).view(nb, bs, 576), dev(scales, np.float32)
    taken, count, live = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(3))
    B.mla_cache_fork(dev([0] * n, np.int32), dev(np.arange(1, n + 1), np.int32), dev([L] * n, np.int32), dev(free, np.int32),
                     T_, R_, kv, sc, scale_group=g, taken=taken)
    assert taken.item() == n
    table, refs, c3, s3, _ = P.fork([0] * n, range(1, n + 1), [L] * n, free, table, refs, codes.reshape(nb, bs, 576),
                                    scales.reshape(nb, -1), bs, g)
    codes, scales, free = c3.reshape(-1, 576), s3.reshape(-1), free[n:]
    rope = B.mla_rope_plan(scaling="yarn", factor=40.0, mscale=1.0, mscale_all_dim=1.0)
    freqs, m = P.rope_frequencies(64, scaling="yarn", factor=40.0, mscale=1.0, mscale_all_dim=1.0)
    lens = np.full(rows_n, L)
    ws = torch.zeros(B.mla_cache_workspace(nb), dtype=torch.uint8, device="cuda")
    freed = torch.zeros(nb, dtype=torch.int32, device="cuda")
    active = np.arange(1, n + 1)                             # the samples; row 0 waits as it is
    for step in range(3):
        R = len(active)
        lens[active] += 1
        sl = dev(lens[active], np.int32)
        sub = T_[1:1 + R]                                    # (the active rows are contiguous)
        slot, req, pos = (torch.zeros(R, dtype=torch.int32, device="cuda") for _ in range(3))
        B.mla_block_tables(dev(np.arange(R + 1), np.int32), sl, dev(free, np.int32), sub, block_size=bs, slot_mapping=slot,
                           req_id=req, positions=pos, taken=taken)
        new, want_slots, _, want_pos, k = S.block_tables(np.arange(R + 1), lens[active], free, table[active], bs, R)
        table[active] = new
        for b in free[:k]:
            refs[b] = 1
        R_.copy_(dev(refs, np.int32))
        free = free[k:]
        assert np.array_equal(slot.cpu().numpy(), want_slots) and taken.item() == k
        nope = torch.from_numpy(rng.standard_normal((R, H, 512))).bfloat16()
        qpe = torch.from_numpy(rng.standard_normal((R, H, 64))).bfloat16()
        kvr = torch.from_numpy(rng.standard_normal((R, 576))).bfloat16()
        q = torch.zeros((R, H, 576), dtype=torch.uint8, device="cuda")
        kpe = kvr[:, 512:].cuda()
        B.mla_rope_qk(rope, pos, ql_nope=nope.cuda(), q_pe=qpe.cuda(), q_out=q, q_scale=QS, k_pe=kpe, k_out=kpe)
        want_k = P.rotate(kvr[:, 512:].double().numpy(), want_pos, freqs, m, False)
        assert np.abs(kpe.double().cpu().numpy() - want_k).max() <= 2.0 ** -8 * np.abs(want_k).max() + 2.0 ** -18
        want_q = P.rotate(qpe.double().numpy(), want_pos, freqs, m, False) / QS
        got_q = O.decode_e4m3fn(q.cpu().numpy())[..., 512:]
        assert np.all(np.abs(got_q - want_q) <= np.maximum(2.0 ** -4 * np.abs(want_q), 2.0 ** -10) + 2.0 ** -10)
        B.mla_cache_append(kvr[:, :512].cuda(), kpe, slot, kv, sc, scale_group=g)
        x = np.concatenate([kvr[:, :512].double().numpy(), kpe.double().cpu().numpy()], 1)
        codes, scales = S.cache_append(x, want_slots, codes, scales, g)
        plan = B.mla_decode_shared_plan(B.make_problem(
            num_tokens=R, num_heads=H, block_size=bs, num_blocks=nb, num_reqs=R, max_blocks_per_req=cols,
            max_seq_len=int(lens.max()), dtype="fp8"))
        dws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        out, lse = torch.zeros((R, H, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((R, H), device="cuda")
        B.mla_decode_fwd_shared(plan, q, kv, kv_scales=sc, scale_group=g, block_table=sub, seq_lens=sl,
                                prefix_lens=dev([L], np.int32), softmax_scale=SCALE, q_scale=QS, workspace=dws, out=out, lse=lse)
        torch.cuda.synchronize()
        lists = S.token_slots(table[active], lens[active], bs)
        ro, rl, to, tl = S.decode(q.cpu().numpy(), QS, codes, scales, g, lists, SCALE, bounds=True)
        weight_terms(dict(q=q.cpu().numpy(), scales=scales, codes=codes, g=g), lists, ro, to)
        assert np.all(np.abs(out.double().cpu().numpy() - ro) <= to) and np.all(np.abs(lse.double().cpu().numpy() - rl) <= tl)
        # the last sample loses; the pool closes up
        B.mla_cache_free(dev(active[-1:], np.int32), T_, R_, freed=freed, num_freed=count, workspace=ws)
        table, refs, gone = P.free(active[-1:], None, table, refs, bs)
        assert freed[:count.item()].cpu().tolist() == gone
        active = active[:-1]
        B.mla_cache_compact(R_, T_, kv, sc, scale_group=g, num_live=live, workspace=ws)
        refs, table, c3, s3, k = P.compact(refs, table, codes.reshape(nb, bs, 576), scales.reshape(nb, -1))
        codes, scales = c3.reshape(-1, 576), s3.reshape(-1)
        free = np.arange(k, nb)
        assert live.item() == k and np.array_equal(T_.cpu().numpy(), table) and np.array_equal(R_.cpu().numpy(), refs)
        assert np.array_equal(kv.cpu().numpy().reshape(-1, 576), codes)


def test_binding_refuses_on_the_device():
    c = shared_case(31, "scaled", 16, 64, 64, [(256, [6, 5])])
    plan = plan_of(c)
    (_, q, kv), named = args_of(c, plan)
    for bad in (dict(prefix_lens=named["prefix_lens"].long()), dict(prefix_lens=dev([1, 2], np.int32)),
                dict(group_indptr=dev([0, 1, 2], np.int32)), dict(kv_scales=None), dict(scale_group=48),
                dict(kv_scales=named["kv_scales"][:-1]), dict(block_table=named["block_table"][:1]),
                dict(block_table=named["block_table"][:, :2]), dict(seq_lens=named["seq_lens"].cpu()),
                dict(out=named["out"].float()), dict(lse=named["lse"][:1]), dict(sinks=torch.zeros(16, device="cuda")),
                dict(kv_scale=0.5), dict(prefix_lens=None)):
        with pytest.raises(B.MLAError) as e:
            B.mla_decode_fwd_shared(plan, q, kv, **dict(named, **bad))
        assert e.value.status == B.MLA_ERR_INVALID_ARG, bad
    with pytest.raises(B.MLAError) as e:
        B.mla_decode_fwd_shared(plan, q, kv, **dict(named, workspace=named["workspace"][:-256]))
    assert e.value.status == B.MLA_ERR_WORKSPACE
    with pytest.raises(B.MLAError):
        B.mla_decode_fwd_shared(plan, q[:1], kv, **named)

"""The decode of a batch that shares prefixes, and the decodes beside it, at their edges:
calls without a split row in captured graphs, rows and keys that are no numbers, more groups
and requests than the schedule keeps, the same bits on every run."""
import functools

import numpy as np
import pytest
import torch

from oracle import scaled_oracle as S
from paged_mla_decode_06_gb300 import binding as B
from paged_mla_decode_06_gb300 import build as BUILD
from paged_mla_decode_06_gb300 import inputs as I
from tests.gpu_helpers import oracle_slots, run_gpu
from tests.test_gpu_shared import args_of, dev, expected, shared_case, shared_groups

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    BUILD.build()
    B.load_library()


def widened(c, bound):
    """The case with columns for requests of ``bound`` tokens."""
    table = c["table"]
    more = -(-bound // c["bs"]) - table.shape[1]
    return dict(c, table=np.concatenate([table, np.full((len(table), max(more, 0)), table[0, -1])], 1))


def problem_of(c, bound=None, **kw):
    return B.make_problem(**dict(dict(
        num_tokens=c["T"], num_heads=c["H"], block_size=c["bs"], num_blocks=c["nb"], num_reqs=len(c["lens"]),
        max_blocks_per_req=c["table"].shape[1], max_seq_len=int(c["lens"].max() if bound is None else bound),
        max_qlen=c["max_qlen"], dtype="bf16" if c["kind"] == "bf16" else "fp8", has_sinks=c["sinks"] is not None), **kw))


@pytest.mark.parametrize("kind,heads,most", [("scaled", 128, 600), ("fp8", 16, 600), ("bf16", 128, 256)])
def test_what_follows_a_shared_call_without_split_rows_reads_all_of_it(kind, heads, most):
    """Short requests of a plan for long ones, none shared or cut: the merge has no row.
    A copy right behind the call in a graph finds all of its output."""
    rng = np.random.default_rng(60)
    c = widened(shared_case(60, kind, heads, 64, 64, [(0, [most] * 40)]), 8192)
    plan = B.mla_decode_shared_plan(problem_of(c, 8192), num_groups=1)
    args, named = args_of(c, plan)
    up = lambda n: -(-n // 256) * 256
    n = plan.partial_rows
    parts = named["workspace"][plan.workspace_bytes - 2 * up(4 * n) - up(2048 * n):]
    replayed_like_eager(lambda: B.mla_decode_fwd_shared(*args, **named), plan, plan.plan, named, c, parts,
                        [rng.integers(1, most + 1, 40) for _ in range(2)])


@pytest.mark.parametrize("kind,heads", [("scaled", 16), ("scaled", 128), ("fp8", 16), ("bf16", 128)])
def test_what_follows_a_decode_without_split_rows_reads_all_of_it(kind, heads):
    c = widened(shared_case(61, kind, heads, 64, 64, [(0, [64] * 40)]), 8192)
    plan = B.mla_decode_plan(problem_of(c, 8192))
    assert plan.schedule == 1
    args, named = args_of(c, plan)
    for k in ("prefix_lens", "group_indptr"):
        del named[k]
    scales, group = named.pop("kv_scales"), named.pop("scale_group")
    if kind == "scaled":
        del named["kv_scale"]
        call = lambda: B.mla_decode_fwd_scaled(*args, scales, scale_group=group, **named)
    else:
        call = lambda: B.mla_decode_fwd(*args, **named)
    parts = named["workspace"][plan.segm_output_offset:]
    rng = np.random.default_rng(61)
    replayed_like_eager(call, plan, plan, named, c, parts, [rng.integers(1, 65, 40) for _ in range(2)])


def replayed_like_eager(call, plan, decode_plan, named, c, parts, lengths):
    out, lse, want = named["out"], named["lse"], []
    parts.fill_(0x5A)
    for lens in lengths:
        named["seq_lens"].copy_(dev(lens, np.int32))
        out.fill_(float("nan")), lse.fill_(float("nan"))
        call()
        torch.cuda.synchronize()
        want.append((out.clone(), lse.clone()))
        assert out.isfinite().all() and lse.isfinite().all()
    assert (parts == 0x5A).all()                          # no row went through the merge
    got, got_lse = torch.empty_like(out), torch.empty_like(lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        got.copy_(out)
        got_lse.copy_(lse)
        out.fill_(float("nan"))
        lse.fill_(float("nan"))
    wrong = torch.zeros(1, dtype=torch.int64, device="cuda")
    sets = [dev(lens, np.int32) for lens in lengths]
    for i in range(200):
        named["seq_lens"].copy_(sets[i % 2])
        g.replay()
        wrong += (got.view(torch.int16) != want[i % 2][0].view(torch.int16)).sum()
        wrong += (got_lse.view(torch.int32) != want[i % 2][1].view(torch.int32)).sum()
    assert wrong.item() == 0
    assert B.mla_workspace_status(decode_plan, named["workspace"]) == 0


# ---- rows and keys that are no numbers

def poisoned(c, keys=(), queries=(), value=float("nan")):
    """``keys``: (slot, column), ``queries``: (token, head, column) that hold ``value``
    (e4m3: NaN)."""
    if c["kind"] == "bf16":
        d = dict(c, kv=c["kv"].clone(), q=c["q"].clone())
        for slot, col in keys:
            d["kv"][slot, col] = value
        for t, h, col in queries:
            d["q"][t, h, col] = value
        return d
    d = dict(c, codes=c["codes"].copy(), q=c["q"].copy())
    for slot, col in keys:
        d["codes"][slot, col] = 0x7F
    for t, h, col in queries:
        d["q"][t, h, col] = 0xFF
    return d


def ran(c, plan):
    args, named = args_of(c, plan)
    B.mla_decode_fwd_shared(*args, **named)
    torch.cuda.synchronize()
    assert B.mla_workspace_status(plan.plan, named["workspace"]) == 0
    return named["out"].double().cpu().numpy(), named["lse"].double().cpu().numpy()


def right_but(c, odd, out, lse):
    """Every row outside ``odd`` [T, H] within its bounds, no number in it NaN."""
    ro, rl, to, tl = expected(c)
    n = len(ro)
    assert (out[n:] == 3.0).all() and (lse[n:] == 3.0).all()
    out, lse = out[:n], lse[:n]
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse)[~odd], empty[~odd])
    assert np.all((np.abs(out - ro) <= to)[~odd])
    assert np.all((np.abs(np.where(empty, 0, lse) - np.where(empty, 0, rl)) <= tl)[~odd & ~empty])


# (kind, block size, group, heads, keys of the prefix, what the plan asks for): shared
# prefixes, and the plain decode of plans that cannot share on each of its kernels, whole and
# in pieces
ROUTES = [("bf16", 64, 64, 24, 1536, {}), ("fp8", 64, 64, 24, 1536, {}), ("scaled", 64, 16, 24, 1536, {}),
          ("bf16", 64, 64, 128, 300, {}), ("bf16", 64, 64, 24, 1536, dict(num_segments=3)), ("bf16", 16, 16, 16, 300, {}),
          ("bf16", 16, 16, 33, 1536, dict(num_segments=3)), ("fp8", 64, 64, 16, 300, {}),
          ("fp8", 64, 64, 128, 1536, dict(num_segments=3)), ("fp8", 8, 8, 16, 300, {}),
          ("fp8", 8, 8, 33, 1536, dict(num_segments=3)),
          ("fp8", 64, 64, 24, 1536, dict(num_segments=2, kernel=B.MLA_KERNEL_TCGEN05))]


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("kind,bs,g,heads,prefix,kw", ROUTES)
def test_rows_that_see_a_nan_are_nan_on_every_route(kind, bs, g, heads, prefix, kw, sinks):
    """A NaN key of the prefix, of one request's own keys, of one head's query: the rows
    that see it are NaN in output and LSE, the others right."""
    c = shared_case(62, kind, heads, bs, g, [(prefix, [6, 5, 9, 70, 3, 140, 8, 8])], alone=[260, 0], sinks=sinks)
    plan = B.mla_decode_shared_plan(problem_of(c, **kw), num_groups=1)
    assert (plan.max_items > 0) == (prefix > 768 and not kw)
    assert plan.max_items == 0 or shared_groups(c) == [True]
    for keys, queries in (([(c["table"][0, 200 // bs] * bs + 200 % bs, 11)], []),
                          ([(c["table"][3, (prefix + 60) // bs] * bs + (prefix + 60) % bs, 575)], [(1, 3, 500), (8, 2, 7)])):
        odd = np.zeros((c["T"], heads), bool)
        for slot, _ in keys:
            odd[[slot in np.asarray(s) for s in S.token_slots(c["table"], c["lens"], bs, c["qo"])]] = True
        for t, h, _ in queries:
            odd[t, h] = True
        assert odd.any() and not odd.all()
        out, lse = ran(poisoned(c, keys, queries), plan)
        assert np.isnan(out[odd]).all() and np.isnan(lse[odd]).all()
        right_but(c, odd, out, lse)


@pytest.mark.parametrize("kind,bs,g,heads,prefix,kw", ROUTES)
def test_keys_that_later_tokens_see_do_not_reach_the_earlier_ones(kind, bs, g, heads, prefix, kw):
    """The last keys of requests of several tokens, NaN or infinite in their value columns:
    the tokens before them, in whose softmax they are masked, keep their results."""
    c = shared_case(63, kind, heads, bs, g, [(prefix, [6, 5, 9, 70, 3, 140, 8, 8])], alone=[260, 0],
                    qlens=[4, 1, 3, 2, 1, 1, 1, 1, 2, 1])
    plan = B.mla_decode_shared_plan(problem_of(c, **kw), num_groups=1)
    assert (plan.max_items > 0) == (prefix > 768 and not kw)
    assert plan.max_items == 0 or shared_groups(c) == [True]
    slots = [S.row_slots(c["table"][r], bs, int(c["lens"][r]))[at] for r, at in ((0, -1), (0, -2), (2, -1), (3, -1), (8, -1))]
    keys = [(s, col) for s in slots for col in (0, 11, 300, 511)]
    seen = [any(s in np.asarray(t) for s in slots) for t in S.token_slots(c["table"], c["lens"], bs, c["qo"])]
    odd = np.zeros((c["T"], heads), bool)
    odd[seen] = True
    assert [int(s) for s in seen] == [0, 0, 1, 1, 0, 0, 0, 1, 0, 1, 0, 0, 0, 0, 0, 1, 0]
    for value in (float("nan"), float("inf"), float("-inf")) if kind == "bf16" else (float("nan"),):
        out, lse = ran(poisoned(c, keys, value=value), plan)
        right_but(c, odd, out, lse)
        if value != value:
            assert np.isnan(out[odd]).all() and np.isnan(lse[odd]).all()


@pytest.mark.parametrize("kind,bs,g,heads,prefix,kw", ROUTES)
def test_sinks_of_minus_infinity_and_nan_on_every_route(kind, bs, g, heads, prefix, kw):
    """A sink of -inf is none, also for rows without a key; one that is NaN makes its head's
    rows NaN."""
    c = shared_case(64, kind, heads, bs, g, [(prefix, [6, 5, 9, 70, 3, 140, 8, 8])], alone=[260, 0, 70], sinks=True)
    plan = B.mla_decode_shared_plan(problem_of(c, **kw), num_groups=1)
    assert plan.max_items == 0 or shared_groups(c) == [True]
    odd = np.zeros((c["T"], heads), bool)
    c["sinks"][:] = -np.inf
    c["sinks"][3] = 0.5
    out, lse = ran(c, plan)
    plain = dict(c, sinks=None)
    pout, plse = ran(plain, B.mla_decode_shared_plan(problem_of(plain, **kw), num_groups=1))
    odd[:, 3] = True
    assert np.array_equal(out[~odd], pout[~odd]) and np.array_equal(lse[~odd], plse[~odd])
    c["sinks"][:] = 0.5
    c["sinks"][3] = np.nan
    out, lse = ran(c, plan)
    assert np.isnan(lse[:, 3]).all() and np.isnan(out[np.arange(len(out)) != 9, 3]).all()  # (without keys: unspecified)
    c["sinks"][3] = 0.5
    right_but(c, odd, out, lse)


# ---- batches beyond what the schedule keeps in shared memory (256 groups, 1024 requests)

def repeated(c, order):
    """Groups ``order`` of the case one after another, as many requests of each as its
    second number: their table rows, lengths and queries again and again. Returns the new
    case and the token of ``c`` that each of its tokens repeats."""
    reqs, prefix, edges = [], [], [0]
    for g, n in order:
        a, b = c["edges"][g], c["edges"][g + 1]
        reqs += [a + i % (b - a) for i in range(n)]
        prefix.append(c["prefix"][g])
        edges.append(len(reqs))
    reqs = np.array(reqs)
    qlens = np.diff(c["qo"])
    tokens = np.concatenate([np.arange(c["qo"][r], c["qo"][r + 1]) for r in reqs])
    d = dict(c, lens=c["lens"][reqs], table=c["table"][reqs], qo=np.concatenate([[0], np.cumsum(qlens[reqs])]),
             T=len(tokens), q=c["q"][tokens], prefix=np.array(prefix), edges=np.array(edges))
    return d, tokens


@functools.lru_cache(maxsize=None)
def groups_to_repeat(kind, bs, g, several):
    c = shared_case(65, kind, 2 if several else 3, bs, g, [(1216 + 64 * i, [4 + 19 * j % 90 for j in range(9)]) for i in range(4)],
                    qlens=[1 + i % 3 for i in range(36)] if several else None)
    return c, expected(c)


@pytest.mark.parametrize("kind,bs,g", [("scaled", 16, 16), ("fp8", 64, 64), ("bf16", 64, 64)])
@pytest.mark.parametrize("groups,each", [(300, 3), (3, 400), (300, 8), (257, 4)])
@pytest.mark.parametrize("several", [False, True])
def test_more_groups_and_requests_than_the_schedule_keeps(kind, bs, g, groups, each, several):
    base, (ro, rl, to, tl) = groups_to_repeat(kind, bs, g, several)
    c, of = repeated(base, [(i % 4, each + (i % 2 if groups == 257 else 0)) for i in range(groups)])
    plan = B.mla_decode_shared_plan(problem_of(c), num_groups=groups)
    assert plan.max_items > 0 and all(shared_groups(c))
    assert len(c["lens"]) > 1024 or groups > 256
    out, lse = ran(c, plan)
    assert np.all(np.abs(out - ro[of]) <= to[of]) and np.all(np.abs(lse - rl[of]) <= tl[of])


@pytest.mark.parametrize("kind,bs,g", [("scaled", 64, 16), ("scaled", 64, 1), ("fp8", 64, 64), ("bf16", 64, 64)])
def test_a_shared_prefix_gives_the_same_bits_on_every_run_and_agrees_with_the_plain_decode(kind, bs, g):
    """Whatever the workspace held, and with the plain calls' results over the same tables
    within the bounds of both."""
    c = shared_case(66, kind, 16, bs, g, [(3000, [1 + 97 * i % 900 for i in range(12)])], sinks=True)
    assert shared_groups(c) == [True]
    plan = B.mla_decode_shared_plan(problem_of(c), num_groups=1)
    assert plan.max_items > 0
    args, named = args_of(c, plan)
    first = None
    for fill in (0, 0xFF, 0x01, 0x7F):
        named["workspace"][256:].fill_(fill)
        named["out"].fill_(0), named["lse"].fill_(0)
        for _ in range(3):
            B.mla_decode_fwd_shared(*args, **named)
        torch.cuda.synchronize()
        assert B.mla_workspace_status(plan.plan, named["workspace"]) == 0
        got = named["out"].clone(), named["lse"].clone()
        first = first or got
        assert torch.equal(got[0].view(torch.int16), first[0].view(torch.int16)) and torch.equal(got[1], first[1])
    ro, rl, to, tl = expected(c)
    assert np.all(np.abs(first[0].double().cpu().numpy() - ro) <= to)
    assert np.all(np.abs(first[1].double().cpu().numpy() - rl) <= tl)
    plain = {k: v for k, v in named.items() if k not in ("prefix_lens", "group_indptr", "kv_scales", "scale_group")}
    if kind == "scaled":
        del plain["kv_scale"]
        B.mla_decode_fwd_scaled(plan.plan, *args[1:], named["kv_scales"], scale_group=g, **plain)
    else:
        B.mla_decode_fwd(plan.plan, *args[1:], **plain)
    torch.cuda.synchronize()
    assert np.all(np.abs(named["out"].double().cpu().numpy() - first[0].double().cpu().numpy()) <= 2 * to)
    assert np.all(np.abs(named["lse"].double().cpu().numpy() - first[1].double().cpu().numpy()) <= 2 * tl)


@pytest.mark.parametrize("kernel,ns", [(B.MLA_KERNEL_AUTO, None), (B.MLA_KERNEL_AUTO, 3), (B.MLA_KERNEL_WARP_MMA, None),
                                       (B.MLA_KERNEL_WARP_MMA, 3)])
def test_sparse_rows_that_list_a_nan_key_are_nan(kernel, ns):
    """Keys of a slot list with a NaN, in the rope and in the value columns: the tokens that
    list them are NaN in output and LSE, the others as without it."""
    w = I.sparse_topk(num_reqs=2, tokens_per_req=6, num_heads=32, cache_tokens=4096, topk=1024, interspersed_rows=1, max_pad=64)
    slots = oracle_slots(w)
    out, lse, _ = run_gpu(w, num_segments=ns, kernel=kernel)
    lists = [set(s[s >= 0].tolist()) for s in slots]
    counts = np.bincount(slots[slots >= 0])
    rare = [int(s) for s in np.flatnonzero(counts == 1)[[3, -7]]]      # of one token each
    seen = np.array([any(s in t for s in rare) for t in lists])
    assert 1 <= seen.sum() <= 2
    flat = w.cache.reshape(-1, 576)
    flat[rare[0], 570], flat[rare[1], 9] = I.BF16_NAN_BITS, I.BF16_NAN_BITS
    bad, bad_lse, _ = run_gpu(w, num_segments=ns, kernel=kernel)
    assert np.isnan(bad[seen]).all() and np.isnan(bad_lse[seen]).all()
    assert np.array_equal(bad[~seen], out[~seen]) and np.array_equal(bad_lse[~seen], lse[~seen])

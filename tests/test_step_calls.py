"""Rotary positions and the calls on a cache's pages: the rotary plan and the
oracle against closed forms, and the refusals of the C ABI and of the binding. No
GPU: every call here fails its checks before a launch."""
import ctypes
import math

import numpy as np
import pytest

from oracle import step_oracle as S
from paged_mla_decode_06_gb300 import binding as B
from paged_mla_decode_06_gb300 import build as BUILD


@pytest.fixture(scope="module", autouse=True)
def lib():
    BUILD.build()
    return B.load_library()


# ---------------------------------------------------------------- the rotary plan

@pytest.mark.parametrize("dim", [2, 6, 34, 64])
@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(scaling="linear", factor=8.0),
    dict(scaling="yarn", factor=40.0, mscale=1.0, mscale_all_dim=0.707),
    dict(scaling="yarn", factor=4.0, original=32768, base=1e6), dict(scaling="yarn", factor=0.5, mscale=1.0),
    dict(scaling="yarn", factor=16.0, original=40, beta_fast=2.0, beta_slow=2.0)])
def test_plan_matches_the_formulas(dim, kw):
    args = dict(kw)
    if "original" in args:
        args["original_max_position"] = args.pop("original")
    rope = B.mla_rope_plan(dim=dim, **args)
    f, m = S.rope_frequencies(dim, **kw)
    # a few operations in 64 bits on either side
    np.testing.assert_allclose(np.array(rope.turns[:dim // 2]) * 2 * math.pi, f, rtol=1e-13)
    assert not any(rope.turns[dim // 2:])
    assert rope.mscale == pytest.approx(m, rel=2.0 ** -23)


def test_yarn_keeps_the_fast_pairs_and_stretches_the_slow_ones():
    f, _ = S.rope_frequencies(64)
    y, m = S.rope_frequencies(64, scaling="yarn", factor=40.0, mscale=1.0, mscale_all_dim=1.0)
    assert np.array_equal(y[:10], f[:10]) and np.allclose(y[24:], f[24:] / 40, rtol=1e-15) and m == 1.0
    assert np.all((y[10:24] <= f[10:24]) & (y[10:24] >= f[10:24] / 40))


@pytest.mark.parametrize("half", [False, True])
def test_rotation_by_hand(half):
    x = np.arange(1.0, 65.0)[None]
    y = S.rotate(x, [1], np.array([math.pi / 2, math.pi]), 2.0, half)
    a, b = ((0, 2), (1, 3)) if half else ((0, 1), (2, 3))
    want = x.copy()
    want[0, a[0]], want[0, a[1]] = -2 * x[0, a[1]], 2 * x[0, a[0]]
    want[0, b[0]], want[0, b[1]] = -2 * x[0, b[0]], -2 * x[0, b[1]]
    np.testing.assert_allclose(y, want, atol=1e-13)


@pytest.mark.parametrize("kw", [dict(dim=0), dict(dim=63), dict(dim=66), dict(dim=-2), dict(base=1.0),
                                dict(base=math.nan), dict(base=math.inf), dict(scaling="linear", factor=0.0),
                                dict(scaling="linear", factor=math.inf), dict(scaling="yarn", factor=-1.0),
                                dict(scaling="yarn", factor=2.0, original_max_position=0),
                                dict(scaling="yarn", factor=2.0, beta_fast=0.5, beta_slow=1.0),
                                dict(scaling="yarn", factor=2.0, beta_slow=0.0),
                                dict(scaling="yarn", factor=2.0, mscale=-1.0), dict(layout="diagonal"),
                                dict(scaling="other")])
def test_plan_refusals(kw):
    with pytest.raises(B.MLAError) as e:
        B.mla_rope_plan(**kw)
    assert e.value.status == B.MLA_ERR_INVALID_ARG


P = 1 << 20  # a pointer that no call may reach


def _rope(lib, rope="default", pos=P, T=4, H=2, nope=P, nt=1024, nh=512, pe=P, pt=128, ph=64, dt=1, qs=1.0, out=P,
          k=P, ks=64, ko=P, kos=64):
    r = B.mla_rope_plan() if rope == "default" else rope
    return lib.mla_rope_qk(None if r is None else ctypes.byref(r), pos, T, H, nope, nt, nh, pe, pt, ph, dt,
                           ctypes.c_float(qs), out, k, ks, ko, kos, None)


@pytest.mark.parametrize("kw", [
    dict(rope=None), dict(T=-1), dict(H=-1), dict(pos=None), dict(pos=P + 2), dict(nope=None), dict(pe=None),
    dict(out=None), dict(nope=P + 8), dict(out=P + 8), dict(pe=P + 2), dict(nt=1028), dict(nh=516), dict(pt=129),
    dict(ph=65), dict(nt=-8), dict(dt=2), dict(qs=0.0), dict(qs=math.nan), dict(qs=math.inf), dict(qs=1e-45),
    dict(k=P + 2), dict(ko=None), dict(ko=P + 2), dict(ks=65), dict(kos=62), dict(kos=65), dict(ks=128), dict(H=0, k=None)])
def test_rope_refusals(lib, kw):
    assert _rope(lib, **kw) == B.MLA_ERR_INVALID_ARG


def test_rope_refuses_a_plan_that_was_not_made(lib):
    r = B.mla_rope_plan()
    r.prob.dim = 65
    assert _rope(lib, rope=r) == B.MLA_ERR_INVALID_ARG
    r = B.mla_rope_plan()
    r.mscale = math.nan
    assert _rope(lib, rope=r) == B.MLA_ERR_INVALID_ARG
    assert _rope(lib, T=0) == B.MLA_OK


# ---------------------------------------------------------------- pages

def test_pages_by_hand():
    block, group = 4, 2
    table = np.array([[3, 5, -1], [9, 9, 9], [8, 8, 8]])
    refs = np.array([0, 0, 0, 1, 0, 1, 0])
    rows = np.arange(7 * 4 * 2.0).reshape(7, 4, 2)
    scales = np.arange(14.0).reshape(7, 2)
    t, r, c, s, taken = S.fork([0, 0], [1, 2], [7, 4], [6, 2], table, refs, rows, scales, block, group)
    assert taken == 1 and t.tolist() == [[3, 5, -1], [3, 6, 9], [3, 8, 8]]
    assert r.tolist() == [0, 0, 0, 3, 0, 1, 1]
    assert np.array_equal(c[6, :3], rows[5, :3]) and np.array_equal(c[6, 3], rows[6, 3])
    assert np.array_equal(s[6], scales[5])
    t[:, 2] = -1
    t2, r2, gone = S.free([1, 1, 7], None, t, r, block)
    assert gone == [6] and r2.tolist() == [0, 0, 0, 2, 0, 1, 0] and t2[1].tolist() == [-1] * 3
    r3, t3, c3, s3, n = S.compact(r2, t2, c, s)
    assert n == 2 and r3.tolist() == [2, 1, 0, 0, 0, 0, 0] and t3[0].tolist() == [0, 1, -1]
    assert np.array_equal(c3[0], rows[3]) and np.array_equal(c3[1], rows[5]) and np.array_equal(s3[1], scales[5])


def test_workspace_size(lib):
    assert B.mla_cache_workspace(0) == 0 and B.mla_cache_workspace(-4) == 0
    for n in (1, 33, 1000, 1 << 20):
        assert B.mla_cache_workspace(n) >= 256 + n // 8 + 8 * n


CACHE = dict(nb=10, bs=64, dt=1, g=16, kv=P, sc=P)
BAD_CACHE = [dict(nb=0), dict(bs=0), dict(dt=2), dict(g=-1), dict(g=48), dict(g=0), dict(sc=None), dict(kv=None),
             dict(kv=P + 8), dict(sc=P + 2), dict(dt=0)]


def _copy(lib, src=P, dst=P, n=3, **kw):
    c = dict(CACHE, **kw)
    return lib.mla_cache_copy_blocks(src, dst, n, c["nb"], c["bs"], c["dt"], c["g"], c["kv"], c["sc"], None)


def _fork(lib, parent=P, child=P, lens=P, n=3, free=P, nf=4, bt=P, stride=8, rows=5, cols=8, refs=P, taken=P, **kw):
    c = dict(CACHE, **kw)
    return lib.mla_cache_fork(parent, child, lens, n, free, nf, bt, stride, rows, cols, refs, c["nb"], c["bs"], c["dt"],
                              c["g"], c["kv"], c["sc"], taken, None)


def _free(lib, rows=P, lens=None, n=3, bt=P, stride=8, nrows=5, cols=8, refs=P, nb=10, bs=64, freed=P, cap=10, count=P,
          ws=P, nbytes=1 << 30):
    return lib.mla_cache_free(rows, lens, n, bt, stride, nrows, cols, refs, nb, bs, freed, cap, count, ws, nbytes, None)


def _compact(lib, refs=P, ro=P, bt=P, stride=8, to=P, tos=8, rows=5, cols=8, count=P, ws=P, nbytes=1 << 30, **kw):
    c = dict(CACHE, **kw)
    return lib.mla_cache_compact(refs, ro, bt, stride, to, tos, rows, cols, c["nb"], c["bs"], c["dt"], c["g"], c["kv"],
                                 c["sc"], count, ws, nbytes, None)


@pytest.mark.parametrize("call,kw", [(_copy, k) for k in BAD_CACHE + [dict(n=-1), dict(src=None), dict(dst=P + 1)]] +
                         [(_fork, k) for k in BAD_CACHE + [
                             dict(n=-1), dict(nf=-1), dict(rows=-1), dict(rows=0), dict(cols=0), dict(stride=7),
                             dict(parent=None), dict(child=P + 2), dict(lens=None), dict(bt=None), dict(refs=None),
                             dict(refs=P + 2), dict(free=None), dict(taken=None), dict(taken=P + 1)]] +
                         [(_free, k) for k in [
                             dict(n=-1), dict(nrows=-1), dict(nrows=0), dict(cols=0), dict(nb=0), dict(bs=0), dict(cap=-1),
                             dict(stride=7), dict(rows=None), dict(bt=None), dict(refs=None), dict(freed=None),
                             dict(count=None), dict(lens=P + 2), dict(ws=P + 4)]] +
                         [(_compact, k) for k in BAD_CACHE + [
                             dict(rows=-1), dict(cols=0), dict(stride=7), dict(tos=7), dict(refs=None), dict(ro=None),
                             dict(bt=None), dict(to=None), dict(count=None), dict(ws=P + 4), dict(stride=9)]])
def test_page_refusals(lib, call, kw):
    assert call(lib, **kw) == B.MLA_ERR_INVALID_ARG


def test_page_workspaces_and_sizes(lib):
    for call in (_free, _compact):
        assert call(lib, ws=None) == B.MLA_ERR_WORKSPACE
        assert call(lib, nbytes=B.mla_cache_workspace(10) - 1) == B.MLA_ERR_WORKSPACE
    for call in (_copy, _fork, _compact):
        assert call(lib, nb=1 << 26) == B.MLA_ERR_UNSUPPORTED
    assert _copy(lib, n=0) == B.MLA_OK
    assert lib.mla_cache_free is not None


def test_a_call_that_frees_no_rows_checks_its_workspace_too(lib):
    assert _free(lib, n=0, ws=None) == B.MLA_ERR_WORKSPACE
    assert _free(lib, n=0, nbytes=B.mla_cache_workspace(10) - 1) == B.MLA_ERR_WORKSPACE
    assert _free(lib, n=0, ws=P + 4) == B.MLA_ERR_INVALID_ARG


# ---------------------------------------------------------------- the decode over shared prefixes

def _problem(dtype="fp8", block=64, **kw):
    base = dict(num_tokens=6, num_reqs=6, num_heads=16, block_size=block, num_blocks=100, max_blocks_per_req=40,
                max_seq_len=40 * block, num_sms=152, dtype=dtype)
    base.update(kw)
    return B.make_problem(**base)


def test_shared_plan():
    p = B.mla_decode_shared_plan(_problem(), num_groups=2)
    assert p.num_groups == 2 and p.workers == 76 and p.unit_tiles == 1 and p.prefix_tiles == 1 + 2
    assert p.max_items == 3 + 6 + 76 and p.partial_rows == (3 + 76) * 128 + 96
    assert p.workspace_bytes >= p.partial_rows * 2056 and p.workspace_bytes >= p.plan.workspace_bytes
    p = B.mla_decode_shared_plan(_problem(num_heads=128, max_qlen=3, num_tokens=18))
    assert p.unit_tiles == 3 and p.prefix_tiles == 18 + 1


@pytest.mark.parametrize("kw", [dict(block=8), dict(block=24), dict(dtype="bf16", block=32), dict(num_segments=2),
                                dict(kernel=B.MLA_KERNEL_TCGEN05), dict(max_seq_len=500)])
def test_shared_plans_that_run_as_the_plain_decode(kw):
    p = B.mla_decode_shared_plan(_problem(**kw))
    assert p.max_items == 0 and p.workspace_bytes == p.plan.workspace_bytes


def test_shared_plan_refusals(lib):
    out = B.SharedPlan()
    pr = _problem()
    assert lib.mla_decode_shared_plan(None, 1, ctypes.byref(out)) == B.MLA_ERR_INVALID_ARG
    assert lib.mla_decode_shared_plan(ctypes.byref(pr), 1, None) == B.MLA_ERR_INVALID_ARG
    for g, want in ((0, B.MLA_ERR_INVALID_ARG), (-1, B.MLA_ERR_INVALID_ARG), (65536, B.MLA_ERR_UNSUPPORTED)):
        assert lib.mla_decode_shared_plan(ctypes.byref(pr), g, ctypes.byref(out)) == want
    pr = _problem(num_reqs=0, topk=128, max_blocks_per_req=0, max_seq_len=0)
    assert lib.mla_decode_shared_plan(ctypes.byref(pr), 1, ctypes.byref(out)) == B.MLA_ERR_UNSUPPORTED
    pr = _problem(num_heads=0)
    assert lib.mla_decode_shared_plan(ctypes.byref(pr), 1, ctypes.byref(out)) == B.MLA_ERR_INVALID_ARG


def _shared(lib, plan, q=P, kv=P, sc=P, g=64, bt=P, stride=40, sl=P, qo=None, pre=P, gi=P, scale=1.0, qs=1.0, ks=1.0,
            sinks=None, ws=P, nbytes=1 << 40, out=P, lse=P):
    f = ctypes.c_float
    return lib.mla_decode_fwd_shared(None if plan is None else ctypes.byref(plan), q, kv, sc, g, bt, stride, sl, qo, pre, gi,
                                     f(scale), f(qs), f(ks), sinks, ws, nbytes, out, lse, None)


@pytest.mark.parametrize("kw,status", [
    (dict(plan=None), 1), (dict(q=None), 1), (dict(q=P + 8), 1), (dict(kv=None), 1), (dict(kv=P + 8), 1),
    (dict(sc=None), 1), (dict(g=0), 1), (dict(g=48), 1), (dict(g=-64), 1), (dict(sc=P + 2), 1), (dict(bt=None), 1),
    (dict(bt=P + 2), 1), (dict(stride=39), 1), (dict(sl=None), 1), (dict(sl=P + 1), 1), (dict(pre=None), 1),
    (dict(pre=P + 2), 1), (dict(gi=P + 2), 1), (dict(gi=None), 1), (dict(scale=0.0), 1), (dict(scale=math.nan), 1),
    (dict(qs=-1.0), 1), (dict(ks=2.0), 1), (dict(ks=math.inf), 1), (dict(sinks=P), 1), (dict(out=None), 1),
    (dict(out=P + 8), 1), (dict(lse=None), 1), (dict(lse=P + 2), 1), (dict(ws=None), 3), (dict(nbytes=1000), 3),
    (dict(ws=P + 128), 1)])
def test_shared_refusals(lib, kw, status):
    plan = B.mla_decode_shared_plan(_problem(), num_groups=2)
    assert _shared(lib, **dict(dict(plan=plan), **kw)) == status


def test_shared_refusals_of_other_plans(lib):
    plan = B.mla_decode_shared_plan(_problem(dtype="bf16"), num_groups=2)
    assert _shared(lib, plan) == B.MLA_ERR_UNSUPPORTED                      # group scales of a bf16 cache
    plan = B.mla_decode_shared_plan(_problem(has_sinks=True), num_groups=2)
    assert _shared(lib, plan) == B.MLA_ERR_INVALID_ARG                      # no sinks
    plan = B.mla_decode_shared_plan(_problem(max_qlen=2), num_groups=2)
    assert _shared(lib, plan) == B.MLA_ERR_INVALID_ARG                      # no token offsets
    plan = B.mla_decode_shared_plan(_problem(), num_groups=2)
    plan.workers = 0
    assert _shared(lib, plan) == B.MLA_ERR_INVALID_ARG
    plan = B.mla_decode_shared_plan(_problem(num_tokens=0, num_reqs=0), num_groups=2)
    assert _shared(lib, plan, q=None, kv=None) == B.MLA_OK                  # nothing to do


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 3, dtype=torch.int32)
    kv = torch.zeros(4, 64, 576, dtype=torch.uint8)
    sc = torch.zeros(4)
    with pytest.raises(B.MLAError, match="CUDA"):
        B.mla_rope_qk(B.mla_rope_plan(), i, k_pe=torch.zeros(2, 64, dtype=torch.bfloat16),
                      k_out=torch.zeros(2, 64, dtype=torch.bfloat16))
    with pytest.raises(B.MLAError, match="CUDA"):
        B.mla_cache_copy_blocks(i, i, kv, sc, scale_group=64)
    with pytest.raises(B.MLAError, match="CUDA"):
        B.mla_cache_fork(i, i, i, i, t, i, kv, sc, scale_group=64, taken=i[:1])
    with pytest.raises(B.MLAError, match="CUDA"):
        B.mla_cache_free(i, t, i, freed=i, num_freed=i[:1], workspace=kv)
    with pytest.raises(B.MLAError, match="CUDA"):
        B.mla_cache_compact(i, t, kv, sc, scale_group=64, num_live=i[:1], workspace=kv)


def test_binding_refuses_lengths_without_a_block_size():
    torch = pytest.importorskip("torch")
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(B.MLAError, match="block_size"):
        B.mla_cache_free(i, torch.zeros(2, 2, dtype=torch.int32), i, lens=i, freed=i, num_freed=i[:1],
                         workspace=torch.zeros(256, dtype=torch.uint8))

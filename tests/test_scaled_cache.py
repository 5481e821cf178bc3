"""Block tables, the append to a cache with group scales and the attention over
it: the oracle against closed forms, and the refusals of the C ABI and of the
binding. No GPU: every call here fails its checks before a launch."""
import ctypes

import numpy as np
import pytest

import oracle as O
from oracle import scaled_oracle as S
from paged_mla_decode_06_gb300 import binding as B
from paged_mla_decode_06_gb300 import build as BUILD


@pytest.fixture(scope="module")
def lib():
    BUILD.build()
    return B.load_library()


# ---------------------------------------------------------------- the oracle

def test_block_tables_by_hand():
    # block size 4: request 0 grows from 3 to 6 tokens (one new block), 1 is a
    # prompt of 9 (three), 2 has nothing, 3 stays inside its block
    table = np.array([[7, 50, 51], [50, 50, 50], [50, 50, 50], [9, 50, 50]])
    tab, slots, req, pos, taken = S.block_tables([0, 3, 12, 12, 13], [6, 9, 0, 2], [20, 21, 22, 23, 24], table, 4, 15)
    assert taken == 4
    assert tab.tolist() == [[7, 20, 51], [21, 22, 23], [50, 50, 50], [9, 50, 50]]
    assert slots.tolist() == [31, 80, 81, 84, 85, 86, 87, 88, 89, 90, 91, 92, 37, -1, -1]
    assert req.tolist() == [0] * 3 + [1] * 9 + [3, -1, -1]
    assert pos.tolist() == [3, 4, 5] + list(range(9)) + [1, -1, -1]


def test_block_tables_short_list_and_narrow_table():
    tab, slots, _, pos, taken = S.block_tables([0, 9, 11], [9, 2], [5], np.full((2, 2), 60), 4, 11)
    assert taken == 3 and tab.tolist() == [[5, -1], [-1, 60]]
    assert slots.tolist() == [20, 21, 22, 23] + [-1] * 7 and pos[8] == 8


@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8),
                                        (0.0, S.MIN_SCALE), (896.0, 2.0), (1.75, 2.0 ** -8), (1.76, 2.0 ** -7)])
def test_group_scale(amax, scale):
    assert S.group_scale(amax) == scale


def test_append_keeps_grows_and_requantises():
    g = 4
    codes = np.zeros((8, 576), np.uint8)
    scales = np.array([np.nan, np.nan])
    rows = np.zeros((3, 576))
    rows[0, 0], rows[1, 1], rows[2, 2] = 448.0, -100.0, 1.0
    codes, scales = S.cache_append(rows[:2], [0, 1], codes, scales, g)      # a new group: the old scale is not read
    assert scales[0] == 1.0 and np.isnan(scales[1])
    assert O.decode_e4m3fn(codes[0, 0]) == 448.0 and O.decode_e4m3fn(codes[1, 1]) == -96.0
    c2, s2 = S.cache_append(rows[2:], [2], codes, scales, g)                # a smaller row keeps the scale
    assert s2[0] == 1.0 and np.array_equal(c2[:2], codes[:2])
    c3, s3 = S.cache_append(rows[:1] * 4, [2], codes, scales, g)            # a larger one moves the rows before it
    assert s3[0] == 4.0
    assert O.decode_e4m3fn(c3[0, 0]) * 4 == 448.0 and O.decode_e4m3fn(c3[1, 1]) * 4 == -96.0
    assert O.decode_e4m3fn(c3[2, 0]) * 4 == 4 * 448.0 and np.array_equal(c3[3:], codes[3:])


def test_append_error_is_half_a_step():
    rng = np.random.default_rng(0)
    x = O.decode_bf16((rng.standard_normal((64, 576)).astype(np.float32)).view(np.uint32) >> 16)
    codes, scales = S.cache_append(x, np.arange(64), np.zeros((64, 576), np.uint8), np.zeros(4), 16)
    back = O.decode_e4m3fn(codes) * np.repeat(scales, 16)[:, None]
    # half a step: 2^-4 of the value, or half of e4m3's smallest step 2^-9 times the scale
    assert np.all(np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * np.repeat(scales, 16)[:, None]))


def test_decode_matches_the_tensor_scale_and_closed_forms():
    rng = np.random.default_rng(1)
    H, n, bs, g = 5, 37, 16, 4
    q = rng.integers(0, 0x7E, (1, H, 576)).astype(np.uint8)
    cache = rng.integers(0, 0x70, (4, bs, 576)).astype(np.uint8)
    table = np.array([[2, 0, 3]])
    lists = S.token_slots(table, [n], bs)
    sinks = rng.standard_normal(H).astype(np.float32)
    out, lse = S.decode(q, 0.01, cache, np.full(16, 0.125), g, lists, 0.05, sinks)
    ro, rl = O.mla_decode(q, "fp8", 0.01, cache, "fp8", 0.125, table, [n], 0.05, block_size=bs, sinks=sinks)
    np.testing.assert_allclose(out, ro, rtol=1e-12)
    np.testing.assert_allclose(lse, rl, rtol=1e-12)
    # one key: its scaled value row, and its score as the LSE
    sc = rng.uniform(0.5, 2.0, 16)
    out, lse = S.decode(q, 0.01, cache, sc, g, [[21]], 0.05)
    key = O.decode_e4m3fn(cache.reshape(-1, 576)[21]) * sc[5]
    np.testing.assert_allclose(out[0], np.tile(key[:512], (H, 1)), rtol=1e-12)
    np.testing.assert_allclose(lse[0], 0.05 * 0.01 * O.decode_e4m3fn(q[0]) @ key, rtol=1e-12)
    # no key
    out, lse = S.decode(q, 0.01, cache, sc, g, [[-1, -1]], 0.05)
    assert not out.any() and np.isneginf(lse).all()


# ---------------------------------------------------------------- refusals of the C ABI

def _plan(dtype="fp8", block=64, **kw):
    base = dict(num_tokens=4, num_reqs=4, num_heads=16, block_size=block, num_blocks=100, max_blocks_per_req=10,
                max_seq_len=10 * block, num_sms=152, dtype=dtype)
    base.update(kw)
    return B.mla_decode_plan(B.make_problem(**base))


P = 1 << 20  # a pointer that no call may reach


def _fwd(lib, plan, name="mla_decode_fwd_scaled", q=P, kv=P, sc=P, g=64, bt=P, stride=10, sl=P, qo=None, slots=None,
         scale=1.0, qs=1.0, sinks=None, ws=P, nbytes=1 << 40, out=P, lse=P):
    return getattr(lib, name)(None if plan is None else ctypes.byref(plan), q, kv, sc, g, bt, stride, sl, qo, slots,
                              None, scale, qs, sinks, ws, nbytes, out, lse, None)


@pytest.mark.parametrize("name", ["mla_decode_fwd_scaled", "mla_decode_items_scaled"])
@pytest.mark.parametrize("kw,status", [
    (dict(g=0), 1), (dict(g=-64), 1), (dict(g=48), 1), (dict(g=128), 1), (dict(sc=None), 1), (dict(sc=P + 2), 1),
    (dict(q=None), 1), (dict(q=P + 8), 1), (dict(kv=None), 1), (dict(kv=P + 1), 1), (dict(bt=None), 1),
    (dict(sl=None), 1), (dict(stride=9), 1), (dict(slots=P), 1), (dict(scale=0.0), 1), (dict(qs=float("nan")), 1),
    (dict(qs=float("inf")), 1), (dict(sinks=P), 1), (dict(out=None), 1), (dict(lse=None), 1), (dict(out=P + 4), 1),
    (dict(ws=None), 3), (dict(nbytes=8), 3), (dict(ws=P + 16), 1)])
def test_decode_scaled_refuses(lib, name, kw, status):
    plan = _plan()
    assert plan.schedule == 1
    assert _fwd(lib, plan, name, **kw) == status


def test_decode_scaled_refuses_plans(lib):
    assert _fwd(lib, None) == B.MLA_ERR_INVALID_ARG
    assert _fwd(lib, _plan(dtype="bf16")) == B.MLA_ERR_UNSUPPORTED
    assert _fwd(lib, _plan(num_segments=2), "mla_decode_items_scaled") == B.MLA_ERR_INVALID_ARG
    # no tokens: nothing to do, whatever the pointers
    empty = _plan(num_tokens=0, num_reqs=0)
    assert _fwd(lib, empty, q=None, kv=None, sc=None, bt=None, sl=None, ws=None, out=None, lse=None) == 0
    assert _fwd(lib, empty, g=3) == B.MLA_ERR_INVALID_ARG


def _tables(lib, qsl=P, sl=P, R=4, T=9, bs=64, free=P, F=5, bt=P, stride=10, cols=10, slots=P, req=P, pos=P, taken=P):
    return lib.mla_block_tables(qsl, sl, R, T, bs, free, F, bt, stride, cols, slots, req, pos, taken, None)


@pytest.mark.parametrize("kw", [
    dict(R=-1), dict(T=-1), dict(bs=0), dict(F=-1), dict(cols=0), dict(stride=9), dict(qsl=None), dict(qsl=P + 1),
    dict(taken=None), dict(taken=P + 2), dict(sl=None), dict(bt=None), dict(bt=P + 1), dict(free=None),
    dict(free=P + 3), dict(slots=None), dict(slots=P + 2), dict(req=P + 1), dict(pos=P + 1), dict(sl=P + 2)])
def test_block_tables_refuses(lib, kw):
    assert _tables(lib, **kw) == B.MLA_ERR_INVALID_ARG


def _append(lib, c=P, cs=576, k=P, ks=576, slots=P, T=3, nb=4, bs=64, g=16, cache=P, sc=P):
    return lib.mla_cache_append(c, cs, k, ks, slots, T, nb, bs, g, cache, sc, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(nb=0), 1), (dict(bs=0), 1), (dict(g=0), 1), (dict(g=24), 1), (dict(g=128), 1),
    (dict(nb=1 << 26), 2), (dict(c=None), 1), (dict(k=None), 1), (dict(slots=None), 1), (dict(cache=None), 1),
    (dict(sc=None), 1), (dict(cs=511), 1), (dict(cs=516), 1), (dict(ks=63), 1), (dict(ks=68), 1), (dict(c=P + 8), 1),
    (dict(k=P + 2), 1), (dict(cache=P + 4), 1), (dict(sc=P + 2), 1), (dict(slots=P + 1), 1),
    (dict(T=0, c=None, k=None, slots=None, cache=None, sc=None), 0)])
def test_cache_append_refuses(lib, kw, status):
    assert _append(lib, **kw) == status


# ---------------------------------------------------------------- refusals of the binding

def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    BUILD.build()
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(B.MLAError, match="CUDA device"):
        B.mla_block_tables(i, i[:1], i, i.view(1, 2), block_size=4, slot_mapping=i, taken=i[:1])
    cache, sc = torch.zeros((1, 4, 576), dtype=torch.uint8), torch.zeros(1)
    kv = torch.zeros((2, 576), dtype=torch.bfloat16)
    with pytest.raises(B.MLAError, match="CUDA device"):
        B.mla_cache_append(kv[:, :512], kv[:, 512:], i, cache, sc, scale_group=4)
    with pytest.raises(B.MLAError, match="CUDA device"):
        B.mla_decode_fwd_scaled(_plan(), torch.zeros((4, 16, 576), dtype=torch.uint8), cache, sc, scale_group=4,
                                softmax_scale=1.0, out=kv, lse=sc)


@pytest.mark.parametrize("amax,scale", [(448.0 * 2.0 ** 60, 2.0 ** 60), (449.0 * 2.0 ** 60, 2.0 ** 60), (3.38e38, 2.0 ** 60),
                                        (448.0 * 2.0 ** 59, 2.0 ** 59), (225.0 * 2.0 ** 60, 2.0 ** 60)])
def test_group_scale_stays_in_the_decodes_range(amax, scale):
    """Scales lie in [2^-60, 2^60]; what is beyond 448 * 2^60 saturates."""
    assert S.group_scale(amax) == scale
    codes, scales = S.cache_append(np.full((1, 576), amax), [0], np.zeros((2, 576), np.uint8), np.zeros(1), 2)
    assert scales[0] == scale
    assert O.decode_e4m3fn(codes[0, 0]) == O.decode_e4m3fn(O.encode_e4m3fn(np.array(min(amax / scale, 448.0))))


# ---------------------------------------------------------------- the kernel that a scaled call runs on

# plans of 152 SMs: 1-3 warp MMA, 5 rows as N, 6 the scaled calls' own
@pytest.mark.parametrize("heads,reqs,bound,kw,kernel", [
    (16, 52, 16384, {}, 5), (16, 1, 64, {}, 5), (17, 52, 16384, {}, 5), (32, 52, 16384, {}, 5), (64, 52, 16384, {}, 5),
    (65, 52, 16384, {}, 6), (128, 1, 64, {}, 6), (16, 8, 4096, dict(qlen=5), 6), (16, 64, 4096, dict(qlen=4), 5),
    (17, 1, 32768, {}, 6), (17, 1, 32832, {}, 5), (64, 8, 4096, {}, 6), (64, 9, 4096, {}, 5),        # few keys
    (64, 76, 512, {}, 6), (64, 77, 512, {}, 5), (64, 76, 576, {}, 5), (16, 76, 512, {}, 5),          # one wave, short
    (16, 9, 4096, dict(block=16), 6), (16, 9, 128, dict(block=16), 1), (17, 9, 128, dict(block=16), 6),
    (128, 9, 4096, dict(block=48), 6), (16, 9, 0, dict(topk=128), 1), (16, 9, 0, dict(topk=256), 6),
    (16, 9, 4096, dict(kernel=B.MLA_KERNEL_WARP_MMA), 1), (128, 9, 4096, dict(kernel=B.MLA_KERNEL_WARP_MMA), 3),
    (16, 9, 4096, dict(kernel=B.MLA_KERNEL_TCGEN05), 6), (64, 9, 512, dict(kernel=B.MLA_KERNEL_TCGEN05_ROWS_N), 5),
    (64, 9, 512, dict(num_segments=2), 5), (128, 9, 512, dict(num_segments=2), 6)])
def test_kernel_of_a_scaled_call(lib, heads, reqs, bound, kw, kernel):
    kw = dict(kw)
    qlen, block, topk = kw.pop("qlen", 1), kw.pop("block", 64), kw.get("topk", 0)
    plan = B.mla_decode_plan(B.make_problem(
        num_tokens=reqs * qlen, num_reqs=0 if topk else reqs, num_heads=heads, block_size=block, num_blocks=100,
        max_blocks_per_req=-(-bound // block), max_seq_len=bound, max_qlen=qlen, num_sms=152, dtype="fp8", **kw))
    assert B.mla_decode_scaled_kernel(plan) == kernel


def test_kernel_of_a_scaled_call_refuses(lib):
    k = ctypes.c_int32(0)
    assert lib.mla_decode_scaled_kernel(None, ctypes.byref(k)) == B.MLA_ERR_INVALID_ARG
    assert lib.mla_decode_scaled_kernel(ctypes.byref(_plan()), None) == B.MLA_ERR_INVALID_ARG
    with pytest.raises(B.MLAError) as e:
        B.mla_decode_scaled_kernel(_plan(dtype="bf16"))
    assert e.value.status == B.MLA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(sl=None), 1), (dict(sl=P + 2), 1), (dict(ws=None), 3), (dict(nbytes=8), 3), (dict(ws=P + 16), 1)])
def test_schedule_scaled_refuses(lib, kw, status):
    a = dict(sl=P, ws=P, nbytes=1 << 40)
    a.update(kw)
    call = lambda p: lib.mla_decode_schedule_scaled(p, a["sl"], None, None, a["ws"], a["nbytes"], None)
    assert call(ctypes.byref(_plan())) == status
    assert call(None) == B.MLA_ERR_INVALID_ARG
    assert call(ctypes.byref(_plan(num_segments=2))) == B.MLA_ERR_INVALID_ARG
    assert call(ctypes.byref(_plan(dtype="bf16"))) == B.MLA_ERR_UNSUPPORTED


@pytest.mark.parametrize("g,rise", [(8, 2.0), (64, 0.4)])
def test_groups_that_grow_keep_within_a_smallest_step(g, rise):
    """Rounded again at each growth: half a smallest step of every scale since,
    less than one of the last in all."""
    rng = np.random.default_rng(95)
    n = min(g, 40)
    x = rng.standard_normal((n, 576)) * np.exp2(rise * np.arange(n))[:, None]
    codes, scales = np.zeros((64, 576), np.uint8), np.zeros(64 // g)
    for i in range(n):
        codes, scales = S.cache_append(x[i:i + 1], [i], codes, scales, g)
    off = np.abs(O.decode_e4m3fn(codes[:n]) * scales[0] - x)
    assert (off <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -9 * scales[0])).all()
    assert (off[np.abs(x) < 2.0 ** -6 * scales[0]] > 2.0 ** -10 * scales[0]).any()   # (the case is met)

"""Rotary positions and the calls on a cache's pages on the GPU, against the
oracle: integers and moved bytes bit for bit, rotations within the roundings."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import step_oracle as S
from paged_mla_decode_06_gb300 import binding as B
from paged_mla_decode_06_gb300 import build as BUILD

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    BUILD.build()
    B.load_library()


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def i32(a):
    return dev(a, np.int32)


# ---------------------------------------------------------------- rotary positions

def rope_case(seed, T, H, far=1 << 31, pad=0):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    pos = rng.integers(0, far, T)
    pos[:min(T, 3)] = [0, 1, far - 1][:min(T, 3)]
    if pad:
        pos[-pad:] = -rng.integers(1, 100, pad)
    return (pos, torch.randn((H, T, 512), generator=g).bfloat16().cuda().transpose(0, 1),
            torch.randn((T, H, 200), generator=g).bfloat16().cuda()[..., 130:194],
            torch.randn((T, 600), generator=g).bfloat16().cuda()[:, 514:578])


def rope_check(rope, kw, dim, half, T, H, fp8, q_scale=2.0 ** -6, seed=0, pad=0, in_place=False, far=1 << 31):
    pos, nope, pe, k = rope_case(seed, T, H, far, pad)
    out = torch.full((T, H, 576), 0x55, dtype=torch.uint8, device="cuda") if fp8 else \
        torch.full((T, H, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    k0 = k.double().cpu().numpy()
    k_out = k if in_place else torch.full((T, 80), 7.0, dtype=torch.bfloat16, device="cuda")[:, :64]
    B.mla_rope_qk(rope, i32(pos), ql_nope=nope, q_pe=pe, q_out=out, q_scale=q_scale if fp8 else None, k_pe=k, k_out=k_out)
    f, m = S.rope_frequencies(dim, **kw)
    live = pos >= 0

    def bound(x, y, unit):
        # cosine, sine and their factor in 32 bits (two ulps each and half an ulp), two products and a sum
        a = np.abs(x).reshape(*x.shape[:-1], -1)
        d = np.zeros_like(a)
        half_d = dim // 2
        if half:
            d[..., :half_d] = d[..., half_d:dim] = a[..., :half_d] + a[..., half_d:dim]
        else:
            d[..., 0:dim:2] = d[..., 1:dim:2] = a[..., 0:dim:2] + a[..., 1:dim:2]
        e = d * m * 2.0 ** -20 * unit
        return e, np.abs(y) * unit
    want = S.rotate(k0, pos, f, m, half)
    e, mag = bound(k0, want, 1.0)
    got = k_out.double().cpu().numpy()
    assert np.all(np.abs(got - want)[live] <= (e + 2.0 ** -8 * (mag + e))[live])
    assert np.array_equal(got[~live], k0[~live] if in_place else np.full_like(got[~live], 7.0))
    x = pe.double().cpu().numpy()
    want = np.concatenate([nope.double().cpu().numpy(), S.rotate(x, pos, f, m, half)], -1)
    e, mag = bound(x, want[..., 512:], 1.0 / q_scale if fp8 else 1.0)
    err = np.zeros_like(want)
    err[..., 512:] = e
    if not fp8:
        got = out.double().cpu().numpy()
        assert np.array_equal(got[live][..., :512], want[live][..., :512])
        assert np.all(np.abs(got - want)[live] <= (err + 2.0 ** -8 * (np.abs(want) + err))[live])
        assert np.all(got[~live] == 7.0)
        return
    v = np.clip(want / q_scale, -448, 448)
    err = err + np.abs(v) * 2.0 ** -22  # the reciprocal and its product
    got = O.decode_e4m3fn(out.cpu().numpy())
    assert np.all(np.abs(got - v)[live] <= (err + np.maximum(2.0 ** -4 * (np.abs(v) + err), 2.0 ** -10))[live])
    assert np.all(out.cpu().numpy()[~live] == 0x55)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dim", [2, 34, 62, 64])
def test_rope(dim, half, fp8):
    kw = dict(scaling="yarn", factor=40.0, original=4096, mscale=1.0, mscale_all_dim=0.3)
    rope = B.mla_rope_plan(dim=dim, layout="half" if half else "interleaved", scaling="yarn", factor=40.0,
                           mscale=1.0, mscale_all_dim=0.3)
    rope_check(rope, kw, dim, half, 13, 5, fp8, seed=dim, pad=2)


@pytest.mark.parametrize("T,H", [(1, 1), (1, 128), (5, 16), (64, 17), (700, 128), (2, 9)])
@pytest.mark.parametrize("fp8", [False, True])
def test_rope_shapes(T, H, fp8):
    rope = B.mla_rope_plan(scaling="linear", factor=3.0)
    rope_check(rope, dict(scaling="linear", factor=3.0), 64, False, T, H, fp8, q_scale=0.013, seed=T + H)


def test_rope_in_place_keys_and_each_alone():
    rope = B.mla_rope_plan(layout="half")
    rope_check(rope, {}, 64, True, 33, 4, False, in_place=True, pad=1, seed=3)
    pos, nope, pe, k = rope_case(5, 21, 6)
    both_q, both_k = torch.empty((21, 6, 576), dtype=torch.bfloat16, device="cuda"), torch.empty_like(k)
    B.mla_rope_qk(rope, i32(pos), ql_nope=nope, q_pe=pe, q_out=both_q, k_pe=k, k_out=both_k)
    q, ko = torch.empty_like(both_q), torch.empty_like(both_k)
    B.mla_rope_qk(rope, i32(pos), ql_nope=nope, q_pe=pe, q_out=q)
    B.mla_rope_qk(rope, i32(pos), k_pe=k, k_out=ko)
    assert torch.equal(q, both_q) and torch.equal(ko, both_k)
    B.mla_rope_qk(rope, i32([]), k_pe=k[:0], k_out=ko[:0])


def test_rope_strides_of_single_elements_say_nothing():
    rope = B.mla_rope_plan()
    pos, nope, pe, k = rope_case(6, 3, 1)
    q, ko = torch.zeros((3, 1, 576), dtype=torch.bfloat16, device="cuda"), torch.zeros_like(k)
    B.mla_rope_qk(rope, i32(pos), ql_nope=nope, q_pe=pe, q_out=q, k_pe=k, k_out=ko)
    odd = lambda x, st: torch.as_strided(x.contiguous(), x.shape, st)
    for i in range(3):
        q1, k1 = torch.zeros_like(q[:1]), torch.zeros_like(ko[:1])
        B.mla_rope_qk(rope, i32(pos[i:i + 1]), ql_nope=odd(nope[i:i + 1], (3, 5, 1)), q_pe=odd(pe[i:i + 1], (3, 5, 1)),
                      q_out=q1, k_pe=odd(k[i:i + 1], (3, 1)), k_out=k1)
        assert torch.equal(q1, q[i:i + 1]) and torch.equal(k1, ko[i:i + 1])


def test_rope_position_zero_is_the_concatenation_and_non_finite_values_stay_in_their_pair():
    rope = B.mla_rope_plan(dim=32)
    _, nope, pe, _ = rope_case(8, 4, 16)
    pe = pe.clone()
    pe[1, 2, 3], pe[2, 3, 40], pe[3, 4, 0] = float("nan"), float("inf"), float("-inf")
    a, b = (torch.empty((4, 16, 576), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.mla_rope_qk(rope, i32([0] * 4), ql_nope=nope, q_pe=pe, q_out=a)
    B.mla_concat_quant_q(nope.contiguous(), pe, out=b)
    same = (a == b) | (a.isnan() & b.isnan())
    odd = (~same).nonzero().tolist()
    assert odd in ([[1, 2, 514]], [[1, 2, 514], [3, 4, 513]]) and same[2].all()  # 0 times NaN or infinity


def test_rope_captured_and_on_a_side_stream():
    rope = B.mla_rope_plan()
    pos, nope, pe, k = rope_case(11, 40, 32)
    p = i32(pos)
    q, ko = torch.zeros((40, 32, 576), dtype=torch.uint8, device="cuda"), torch.zeros_like(k)
    call = lambda: B.mla_rope_qk(rope, p, ql_nope=nope, q_pe=pe, q_out=q, q_scale=0.02, k_pe=k, k_out=ko)
    call()
    want = q.clone(), ko.clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    q.zero_(), ko.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(ko, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    p += 3
    g.replay()
    torch.cuda.synchronize()
    graphed = q.clone()
    call()
    assert torch.equal(q, graphed) and not torch.equal(q, want[0])


# ---------------------------------------------------------------- pages

def cache_of(rng, nb, bs, group, kind):
    """(host rows of bytes, host scales or None, device cache, device scales or None)"""
    width = 576 * (2 if kind == "bf16" else 1)
    rows = rng.integers(0, 256, (nb, bs, width), dtype=np.uint8)
    kv = dev(rows) if kind != "bf16" else dev(rows).view(torch.bfloat16)
    if kind != "scaled":
        return rows, None, kv, None
    sc = rng.random((nb, bs // group), dtype=np.float32)
    return rows, sc, kv, dev(sc).view(-1)


def bytes_of(kv):
    return kv.view(torch.uint8).cpu().numpy()


def check_cache(kv, sc, rows, scales):
    assert np.array_equal(bytes_of(kv), rows)
    if scales is not None:
        assert np.array_equal(sc.cpu().numpy().reshape(scales.shape), scales)


SHAPES = [("scaled", 64, 16), ("scaled", 64, 1), ("scaled", 48, 48), ("scaled", 3, 1), ("bf16", 16, 16), ("fp8", 1, 1),
          ("bf16", 130, 130)]


@pytest.mark.parametrize("kind,bs,group", SHAPES)
@pytest.mark.parametrize("n", [1, 7, 200])
def test_copy_blocks(kind, bs, group, n):
    rng = np.random.default_rng(n + bs)
    nb = 2 * n + 5
    rows, scales, kv, sc = cache_of(rng, nb, bs, group, kind)
    ids = rng.permutation(nb)
    src, dst = ids[:n].copy(), ids[n:2 * n].copy()
    if n > 1:  # passed over
        src[0], dst[1] = -1, nb
    B.mla_cache_copy_blocks(i32(src), i32(dst), kv, sc, scale_group=group if sc is not None else 0)
    for s, d in zip(src, dst):
        if s >= 0 and d < nb:
            rows[d] = rows[s]
            if scales is not None:
                scales[d] = scales[s]
    check_cache(kv, sc, rows, scales)


def pool(seed, prompts, spare_rows, ctx, bs, extra=9, cols=None):
    """A table of prompts and free rows behind them, with sentinels in unused cells."""
    rng = np.random.default_rng(seed)
    need = -(-np.asarray(ctx) // bs)
    cols = int(need.max()) + 2 if cols is None else cols
    used = int(need.sum())
    ids = rng.permutation(used + extra)
    table = rng.integers(-9, 0, (prompts + spare_rows, cols))
    table[:prompts][np.arange(cols)[None, :] < need[:, None]] = ids[:used]
    refs = np.zeros(used + extra, np.int64)
    refs[ids[:used]] = 1
    return rng, table, refs, ids[used:]


@pytest.mark.parametrize("kind,bs,group", SHAPES)
@pytest.mark.parametrize("short", [0, 3])
def test_fork_free_and_compact(kind, bs, group, short):
    ctx = np.array([1, bs, bs + 1, 5 * bs - 1, 7 * bs + bs // 2, 2])
    rng, table, refs, free = pool(bs, 6, 14, ctx, bs, extra=16 - short)
    rows, scales, kv, sc = cache_of(rng, len(refs), bs, group, kind)
    g = group if sc is not None else 0
    parent = np.array([0, 1, 2, 3, 4, 5, 0, 3, 3, 4, 2, 77, 1])
    child = np.array([6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16, 17, -1])
    lens = np.concatenate([ctx, ctx[[0, 3]], [2 * bs + 1, 0, ctx[2]], [5, 5]])
    T, R = i32(table), i32(refs)
    taken = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    B.mla_cache_fork(i32(parent), i32(child), i32(lens), i32(free), T, R, kv, sc, scale_group=g, taken=taken)
    table, refs, rows, scales, want = S.fork(parent, child, lens, free, table, refs, rows, scales, bs, group)
    assert taken.item() == want
    assert np.array_equal(T.cpu().numpy(), table) and np.array_equal(R.cpu().numpy(), refs)
    check_cache(kv, sc, rows, scales)

    listed = np.array([7, 9, 9, 3, 14, -2, 20, 10])           # row 9 twice, rows that do not exist
    full = np.array([bs, lens[3], lens[3], ctx[3], lens[8], 0, 0, lens[4]])
    ws = torch.zeros(B.mla_cache_workspace(len(refs)), dtype=torch.uint8, device="cuda")
    freed = torch.full((len(refs),), 77, dtype=torch.int32, device="cuda")
    count = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    for ln in (full, None):
        B.mla_cache_free(i32(listed), T, R, lens=None if ln is None else i32(ln), block_size=bs, freed=freed,
                         num_freed=count, workspace=ws)
        table, refs, gone = S.free(listed, ln, table, refs, bs)
        assert count.item() == len(gone) and freed[:len(gone)].cpu().tolist() == gone
        assert np.array_equal(T.cpu().numpy(), table) and np.array_equal(R.cpu().numpy(), refs)
        listed = np.array([0, 15])
    assert not ws.any()

    live = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    to, ro = torch.full_like(T, 99), torch.full_like(R, 99)
    kv2, sc2 = kv.clone(), None if sc is None else sc.clone()
    B.mla_cache_compact(R, T, kv2, sc2, scale_group=g, refs_out=ro, table_out=to, num_live=live, workspace=ws)
    nrefs, ntable, nrows, nscales, n = S.compact(refs, table, rows, scales)
    assert live.item() == n and np.array_equal(ro.cpu().numpy(), nrefs) and np.array_equal(to.cpu().numpy(), ntable)
    check_cache(kv2, sc2, nrows, nscales)
    assert np.array_equal(R.cpu().numpy(), refs) and np.array_equal(T.cpu().numpy(), table)
    B.mla_cache_compact(R, T, kv, sc, scale_group=g, num_live=live, workspace=ws)  # in place, twice
    assert np.array_equal(R.cpu().numpy(), nrefs) and np.array_equal(T.cpu().numpy(), ntable)
    B.mla_cache_compact(R, T, kv, sc, scale_group=g, num_live=live, workspace=ws)
    assert np.array_equal(R.cpu().numpy(), nrefs) and np.array_equal(T.cpu().numpy(), ntable)
    check_cache(kv, sc, nrows, nscales)


@pytest.mark.parametrize("nb,share", [(1, 1.0), (1, 0.0), (31, 0.5), (8192, 0.3), (20001, 0.9), (70000, 0.02),
                                      (70000, 1.0), (513, 0.0)])
def test_compact_pools(nb, share):
    rng = np.random.default_rng(nb)
    refs = (rng.random(nb) < share) * rng.integers(1, 5, nb)
    table = rng.integers(-3, nb + 3, (11, 37))
    rows, _, kv, _ = cache_of(rng, nb, 1, 1, "fp8")
    R, T = i32(refs), i32(np.pad(table, ((0, 0), (2, 5))))
    view = T[:, 2:39]
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(B.mla_cache_workspace(nb), dtype=torch.uint8, device="cuda")
    B.mla_cache_compact(R, view, kv, num_live=live, workspace=ws)
    want = S.compact(refs, table, rows, None)
    assert live.item() == want[4] and np.array_equal(R.cpu().numpy(), want[0])
    assert np.array_equal(view.cpu().numpy(), want[1])
    check_cache(kv, None, want[2], None)
    assert not T[:, :2].any() and not T[:, 39:].any()


@pytest.mark.parametrize("forks", [600, 3000])
def test_many_forks_of_few_prompts(forks):
    bs, ctx = 16, np.array([100, 64, 33])
    rng, table, refs, free = pool(1, 3, forks, ctx, bs, extra=forks)
    rows, scales, kv, sc = cache_of(rng, len(refs), bs, 4, "scaled")
    parent = rng.integers(0, 3, forks)
    child = 3 + rng.permutation(forks)
    lens = np.minimum(rng.integers(0, 101, forks), ctx[parent])
    T, R = i32(table), i32(refs)
    taken = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.mla_cache_fork(i32(parent), i32(child), i32(lens), i32(free), T, R, kv, sc, scale_group=4, taken=taken)
    table, refs, rows, scales, want = S.fork(parent, child, lens, free, table, refs, rows, scales, bs, 4)
    assert taken.item() == want and np.array_equal(T.cpu().numpy(), table) and np.array_equal(R.cpu().numpy(), refs)
    check_cache(kv, sc, rows, scales)
    ws = torch.zeros(B.mla_cache_workspace(len(refs)), dtype=torch.uint8, device="cuda")
    freed, count = torch.full((50,), 77, dtype=torch.int32, device="cuda"), torch.zeros_like(taken)
    B.mla_cache_free(i32(child), T, R, freed=freed, num_freed=count, workspace=ws)   # a list too short
    table, refs, gone = S.free(child, None, table, refs, bs)
    assert count.item() == len(gone) == want and freed.cpu().tolist() == gone[:50]
    assert np.array_equal(T.cpu().numpy(), table) and np.array_equal(R.cpu().numpy(), refs)


def test_pages_without_work():
    _, _, kv, sc = cache_of(np.random.default_rng(0), 3, 16, 4, "scaled")
    none = i32([])
    T, R, one = i32([[1, 2]]), i32([0, 1, 1]), torch.full((1,), 77, dtype=torch.int32, device="cuda")
    ws = torch.zeros(B.mla_cache_workspace(3), dtype=torch.uint8, device="cuda")
    B.mla_cache_fork(none, none, none, None, T, R, kv, sc, scale_group=4, taken=one)
    assert one.item() == 0
    one.fill_(77)
    B.mla_cache_free(none, T, R, freed=none, num_freed=one, workspace=ws)
    assert one.item() == 0
    B.mla_cache_copy_blocks(none, none, kv, sc, scale_group=4)
    # no free block at all
    T = i32([[1, 2], [-1, -1]])
    B.mla_cache_fork(i32([0]), i32([1]), i32([20]), None, T, R, kv, sc, scale_group=4, taken=one)
    assert one.item() == 1 and T.tolist() == [[1, 2], [1, -1]] and R.tolist() == [0, 2, 1]


def test_binding_refuses_wrong_tensors():
    _, _, kv, sc = cache_of(np.random.default_rng(0), 3, 16, 4, "scaled")
    a, T, R, one = i32([0]), i32([[1, 2]]), i32([0, 1, 1]), i32([0])
    ws = torch.zeros(B.mla_cache_workspace(3), dtype=torch.uint8, device="cuda")
    calls = [lambda: B.mla_cache_copy_blocks(a, i32([1, 2]), kv, sc, scale_group=4),
             lambda: B.mla_cache_copy_blocks(a.long(), a, kv, sc, scale_group=4),
             lambda: B.mla_cache_copy_blocks(a, a, kv, sc),
             lambda: B.mla_cache_copy_blocks(a, a, kv, sc[:-1], scale_group=4),
             lambda: B.mla_cache_copy_blocks(a, a, kv.transpose(0, 1), sc, scale_group=4),
             lambda: B.mla_cache_copy_blocks(a, a, kv, sc, scale_group=5),
             lambda: B.mla_cache_fork(a, a, a, a, T, R[:2], kv, sc, scale_group=4, taken=one),
             lambda: B.mla_cache_fork(a, a, a, a, T[0], R, kv, sc, scale_group=4, taken=one),
             lambda: B.mla_cache_free(a, T, R, freed=a.cpu(), num_freed=one, workspace=ws),
             lambda: B.mla_cache_free(a, T, R, freed=a, num_freed=one, workspace=ws.cpu()),
             lambda: B.mla_cache_compact(R, T, kv, sc, scale_group=4, table_out=i32([[1]]), num_live=one, workspace=ws),
             lambda: B.mla_cache_compact(R, i32([[1, 2], [0, 0]]).t(), kv, sc, scale_group=4, num_live=one, workspace=ws),
             lambda: B.mla_rope_qk(B.mla_rope_plan(), a, k_pe=torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda"),
                                   k_out=torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda")),
             lambda: B.mla_rope_qk(B.mla_rope_plan(), a, k_pe=torch.zeros(1, 64, device="cuda"),
                                   k_out=torch.zeros(1, 64, device="cuda")),
             lambda: B.mla_rope_qk(B.mla_rope_plan(), a),
             lambda: B.mla_rope_qk(B.mla_rope_plan(), a, k_pe=torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda"))]
    for call in calls:
        with pytest.raises(B.MLAError) as e:
            call()
        assert e.value.status == B.MLA_ERR_INVALID_ARG


def test_pages_captured_and_replayed():
    """A captured fork, free and compaction replayed on other tables and lengths."""
    bs, ctx = 16, np.array([40, 25, 90, 16])
    rng, table, refs, free = pool(3, 4, 6, ctx, bs, extra=40)
    rows, scales, kv, sc = cache_of(rng, len(refs), bs, 8, "scaled")
    T, R, P, C, L, F = i32(table), i32(refs), i32([0, 1, 2]), i32([4, 5, 6]), i32([40, 25, 90]), i32(free)
    ws = torch.zeros(B.mla_cache_workspace(len(refs)), dtype=torch.uint8, device="cuda")
    one, freed, count, live = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (1, len(refs), 1, 1))

    def step():
        B.mla_cache_fork(P, C, L, F, T, R, kv, sc, scale_group=8, taken=one)
        B.mla_cache_free(P, T, R, freed=freed, num_freed=count, workspace=ws)
        B.mla_cache_compact(R, T, kv, sc, scale_group=8, num_live=live, workspace=ws)
    before = [t.clone() for t in (T, R, kv, sc)]
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens, par in (([40, 25, 90], [0, 1, 2]), ([16, 3, 33], [3, 1, 2]), ([0, 1, 17], [0, 0, 2])):
        for t, b in zip((T, R, kv, sc), before):
            t.copy_(b)
        L.copy_(i32(lens)), P.copy_(i32(par))
        g.replay()
        t, r, c, s, n = S.fork(par, [4, 5, 6], lens, free, table, refs, rows, scales, bs, 8)
        t, r, gone = S.free(par, None, t, r, bs)
        assert one.item() == n and count.item() == len(gone) and freed[:len(gone)].cpu().tolist() == gone
        r, t, c, s, n = S.compact(r, t, c, s)
        assert live.item() == n and np.array_equal(T.cpu().numpy(), t) and np.array_equal(R.cpu().numpy(), r)
        check_cache(kv, sc, c, s)


def test_counts_of_a_steps_blocks_are_set_on_the_device():
    """Steps of a captured server: block tables, the counts of the blocks that they took by
    elementwise operations that read ``taken`` on the GPU, rows given up. No block goes below
    zero, and what is not in use is in the list."""
    bs, R, cols, nb = 16, 6, 40, 90
    rng = np.random.default_rng(91)
    T_, refs = i32(np.full((R, cols), -1)), i32(np.zeros(nb))
    lens, qsl, free = i32(np.ones(R)), i32(np.arange(R + 1)), i32(np.zeros(nb))
    num_free = torch.zeros(1, dtype=torch.int32, device="cuda")
    taken, count = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    slot = torch.zeros(R, dtype=torch.int32, device="cuda")
    gone, freed = i32(np.full(2, -1)), i32(np.zeros(nb))
    ws = torch.zeros(B.mla_cache_workspace(nb), dtype=torch.uint8, device="cuda")
    place = torch.arange(nb, device="cuda", dtype=torch.int32)

    def step():
        B.mla_block_tables(qsl, lens, free, T_, block_size=bs, slot_mapping=slot, taken=taken)
        refs.index_add_(0, free, (place < torch.minimum(taken, num_free)).int())
        B.mla_cache_free(gone, T_, refs, freed=freed, num_freed=count, workspace=ws)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    T_.fill_(-1), refs.zero_()
    table, want, ids = np.full((R, cols), -1), np.zeros(nb, np.int64), list(rng.permutation(nb))
    n = np.zeros(R, np.int64)
    for k in range(60):
        n += 1
        drop = [int(rng.integers(R))] if k % 9 == 8 else []
        lens.copy_(i32(n))
        # (the list has room for every entry; those behind its end name no block of their own)
        free.copy_(i32(ids + [0] * (nb - len(ids))))
        num_free.fill_(len(ids))
        gone.copy_(i32(drop + [-1] * (2 - len(drop))))
        g.replay()
        for r in range(R):
            if (n[r] - 1) % bs == 0:
                table[r, (n[r] - 1) // bs] = ids[0]
                want[ids.pop(0)] += 1
        table, want, back = S.free(drop, None, table, want, bs)
        ids += back
        for r in drop:
            n[r] = 0
        assert np.array_equal(T_.cpu().numpy(), table) and np.array_equal(refs.cpu().numpy(), want)
        assert freed[:count.item()].tolist() == back and want.min() >= 0
        assert sorted(ids) == np.flatnonzero(want == 0).tolist()

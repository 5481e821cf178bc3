"""Block tables, the append to a cache with group scales and the attention over
it on the GPU, against the oracle: integers bit for bit, codes and scales bit
for bit (scales are powers of two, so one rounding separates a code from its
definition), the attention within the bounds the oracle derives element by
element. Unused rows and scales hold NaN wherever they must not be read."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from oracle import scaled_oracle as S
from paged_mla_decode_06_gb300 import binding as B
from paged_mla_decode_06_gb300 import build as BUILD
from paged_mla_decode_06_gb300 import inputs as I

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(192.0)
QS = 2.0 ** -6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    BUILD.build()
    B.load_library()


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


# ---------------------------------------------------------------- block tables

def tables_case(seed, q, ctx, bs, cols=None, free=None, lead=0, tail=0, short=0):
    rng = np.random.default_rng(seed)
    q, ctx = np.asarray(q, dtype=np.int64), np.asarray(ctx, dtype=np.int64)
    lens = q + ctx
    old, need = -(-ctx // bs), -(-lens // bs)
    if cols is None:
        cols = max(1, int(need.max()) if len(q) else 1) + 1
    ids = rng.permutation(int(need.sum()) + 7)
    table = rng.integers(-5, -1, (len(q), cols))          # sentinels: cells that must keep their value
    k = 0
    for r in range(len(q)):
        m = min(int(old[r]), cols)
        table[r, :m] = ids[k:k + m]
        k += m
    free = ids[k:len(ids) - short] if free is None else free
    qsl = lead + np.concatenate([[0], np.cumsum(q)])
    return dict(qsl=qsl, lens=lens, free=free, table=table, bs=bs, T=int(qsl[-1]) + tail)


def run_tables(c, extra=True):
    table = dev(c["table"], np.int32)
    bufs = [torch.full((c["T"],), 77, dtype=torch.int32, device="cuda") for _ in range(3)]
    taken = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    B.mla_block_tables(dev(c["qsl"], np.int32), dev(c["lens"], np.int32), dev(c["free"], np.int32), table,
                       block_size=c["bs"], slot_mapping=bufs[0], req_id=bufs[1] if extra else None,
                       positions=bufs[2] if extra else None, taken=taken)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (table, *bufs, taken)]


def check_tables(c):
    tab, slots, req, pos, taken = S.block_tables(c["qsl"], c["lens"], c["free"], c["table"], c["bs"], c["T"])
    g = run_tables(c)
    assert np.array_equal(g[0], tab)
    assert np.array_equal(g[1], slots)
    assert np.array_equal(g[2], req)
    assert np.array_equal(g[3], pos)
    assert int(g[4][0]) == taken


@pytest.mark.parametrize("case", [
    dict(q=[1], ctx=[0], bs=16), dict(q=[1], ctx=[16], bs=16), dict(q=[1], ctx=[15], bs=16),
    dict(q=[], ctx=[], bs=64, tail=5), dict(q=[], ctx=[], bs=64), dict(q=[0, 0], ctx=[0, 40], bs=16),
    dict(q=[3, 9, 0, 1], ctx=[3, 0, 0, 1], bs=4, tail=2), dict(q=[2000], ctx=[37], bs=16, tail=30),
    dict(q=[511, 1, 1, 513], ctx=[1, 63, 64, 0], bs=64), dict(q=[512, 512], ctx=[0, 0], bs=1),
    dict(q=[5, 7], ctx=[2, 100], bs=48, lead=3, tail=600), dict(q=[40, 40], ctx=[10, 90], bs=16, cols=4),
    dict(q=[40, 40, 40], ctx=[10, 90, 0], bs=16, short=4), dict(q=[9, 9], ctx=[0, 0], bs=4, free=[]),
    dict(q=[1] * 509, ctx=list(range(509)), bs=16, tail=3), dict(q=[1, 0] * 700, ctx=list(range(1400)), bs=64),
    dict(q=[0] * 1500 + [3] + [0] * 1100 + [2000, 0], ctx=[5] * 2603, bs=16)],
    ids=lambda c: f"R{len(c['q'])}_bs{c['bs']}_T{sum(c['q'])}")
def test_block_tables(case):
    check_tables(tables_case(len(case["q"]) + case["bs"], **case))


@pytest.mark.parametrize("seed", range(8))
def test_block_tables_random(seed):
    rng = np.random.default_rng(seed)
    R = int(rng.integers(1, 3000 if seed % 2 else 40))
    q = rng.integers(0, 6 if R > 100 else 900, R) * (rng.random(R) < 0.8)
    check_tables(tables_case(seed, q, rng.integers(0, 3000, R), int(rng.choice([1, 7, 16, 48, 64])),
                             tail=int(rng.integers(0, 40)), short=int(rng.integers(0, 9))))


def test_block_tables_strided_rows_and_optional_outputs():
    c = tables_case(3, [5, 1, 70], [0, 31, 64], 16)
    want = S.block_tables(c["qsl"], c["lens"], c["free"], c["table"], 16, c["T"])
    g = run_tables(c, extra=False)
    assert np.array_equal(g[0], want[0]) and np.array_equal(g[1], want[1])
    wide = torch.full((3, c["table"].shape[1] + 5), 99, dtype=torch.int32, device="cuda")
    view = wide[:, :c["table"].shape[1]]
    view.copy_(dev(c["table"], np.int32))
    slots, taken = torch.empty(c["T"], dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    B.mla_block_tables(dev(c["qsl"], np.int32), dev(c["lens"], np.int32), dev(c["free"], np.int32), view, block_size=16,
                       slot_mapping=slots, taken=taken)
    torch.cuda.synchronize()
    assert np.array_equal(view.cpu().numpy(), want[0]) and (wide[:, view.shape[1]:] == 99).all()
    assert np.array_equal(slots.cpu().numpy(), want[1])


# ---------------------------------------------------------------- append

def bf16(x):
    """float64 values of x rounded to bf16, and the bf16 tensor."""
    t = torch.from_numpy(np.asarray(x, dtype=np.float32)).bfloat16()
    return t.double().numpy(), t.cuda()


def filled(rng, slots, g):
    """A cache in use: codes under power-of-two scales that differ by group."""
    codes = np.zeros((slots, 576), np.uint8)
    rows = rng.standard_normal((slots, 576)) * np.exp(rng.standard_normal((slots, 1)))
    codes, scales = S.cache_append(bf16(rows)[0], np.arange(slots), codes, np.zeros(slots // g), g)
    return codes, scales


def run_append(kv, slots, codes, scales, bs, g):
    cache = dev(codes).view(-1, bs, 576)
    sc = dev(scales, np.float32)
    B.mla_cache_append(kv[:, :512], kv[:, 512:], dev(slots, np.int32), cache, sc, scale_group=g)
    torch.cuda.synchronize()
    return cache.view(-1, 576).cpu().numpy(), sc.cpu().numpy()


def check_append(rows, slots, codes, scales, bs, g):
    x, kv = bf16(rows)
    with np.errstate(invalid="ignore"):
        want_c, want_s = S.cache_append(x, slots, codes, scales, g)
    got_c, got_s = run_append(kv, slots, codes, scales, bs, g)
    assert np.array_equal(got_s, want_s.astype(np.float32), equal_nan=True)
    # -0 and 0 are one value: a code that underflows keeps its sign
    nz = (got_c & 0x7F).astype(bool) | (want_c & 0x7F).astype(bool)
    nan = ((got_c & 0x7F) == 0x7F) & ((want_c & 0x7F) == 0x7F)
    assert np.array_equal(got_c[nz & ~nan], want_c[nz & ~nan])
    return got_c, got_s


def step_slots(rng, ctx, q, bs, spare=2):
    """Slots of requests with ctx tokens in the cache and q new ones; all blocks scattered."""
    need = -(-(np.asarray(ctx) + np.asarray(q)) // bs)
    ids = rng.permutation(int(need.sum()) + spare)
    out, k = [], 0
    for c, n, m in zip(ctx, q, need):
        p = np.arange(c, c + n)
        out.append(ids[k + p // bs] * bs + p % bs)
        k += int(m)
    return np.concatenate(out) if out else np.zeros(0, np.int64), len(ids)


@pytest.mark.parametrize("bs,g", [(16, 1), (16, 2), (64, 4), (64, 8), (48, 3), (48, 6), (48, 12), (16, 16), (48, 24),
                                  (64, 64), (128, 128), (512, 256), (512, 512), (40, 40), (7, 7), (1, 1)])
def test_append(bs, g):
    rng = np.random.default_rng(bs * 1000 + g)
    ctx = [0, 1, bs - 1, bs, 3 * bs + bs // 2, 5, 2 * bs, 0]
    q = [1, 1, 1, 1, 2 * bs + 3, bs, bs // 2 + 1, 3 * bs]
    slots, nb = step_slots(rng, ctx, q, bs)
    codes, scales = filled(rng, nb * bs, g)
    slots = np.concatenate([slots[:5], [-1], slots[5:], [-1, -1, nb * bs, -7]])
    # -1 inside a request parts its run; one group then has two runs, unless a
    # group starts there: keep the hole between requests
    assert q[0] + q[1] + q[2] + q[3] == 4
    slots = np.concatenate([slots[:4], [-1], slots[4:5], slots[6:]])
    rows = rng.standard_normal((len(slots), 576)) * np.exp(1.5 * rng.standard_normal((len(slots), 1)))
    check_append(rows, slots, codes, scales, bs, g)


@pytest.mark.parametrize("g", [1, 8, 64])
def test_append_special_values(g):
    rng = np.random.default_rng(g)
    bs = 64
    slots, nb = step_slots(rng, [0, 10, 0, 0, 0, 63], [3, 2, 70, 1, 1, 1], bs)
    codes, scales = filled(rng, nb * bs, g)
    rows = rng.standard_normal((len(slots), 576))
    rows[0] = 0.0                          # zeros
    rows[3, 5], rows[3, 515] = np.inf, -np.inf
    rows[4, 7] = np.nan
    rows[10:40] = 0.0
    rows[20, 0] = 1e-37                    # below the smallest scale's range
    rows[60, 3] = 3.0e38
    rows[75] = np.nan                      # nothing finite
    rows[76] = 448.0
    got_c, got_s = check_append(rows, slots, codes, scales, bs, g)
    flat = got_c[slots[3]]
    assert O.decode_e4m3fn(flat[5]) == 448.0 and O.decode_e4m3fn(flat[515]) == -448.0
    assert (got_c[slots[4], 7] & 0x7F) == 0x7F
    assert (got_c[slots[75]] & 0x7F == 0x7F).all()
    assert np.isfinite(got_s).all() and (got_s >= 2.0 ** -60).all()


def test_append_fresh_group_ignores_its_old_scale_and_leaves_the_rest():
    bs, g = 64, 32
    codes = np.full((2 * bs, 576), 0x7F, np.uint8)
    scales = np.full(4, np.nan)
    rows = np.random.default_rng(0).standard_normal((5, 576))
    c, s = check_append(rows, [64, 65, 66, 67, 68], codes, scales, bs, g)
    assert np.isnan(s[[0, 1, 3]]).all() and np.isfinite(s[2])
    assert (c[:64] == 0x7F).all() and (c[69:] == 0x7F).all()


def test_append_token_by_token_grows_without_loss():
    """Rows of rising size, one call each: every requantisation is exact but
    for underflow, so the group ends as if it had been written in one call."""
    bs = g = 64
    rng = np.random.default_rng(5)
    rows = rng.standard_normal((40, 576)) * np.exp2(np.arange(40) / 8.0)[:, None]
    x, kv = bf16(rows)
    cache, sc = torch.zeros((1, bs, 576), dtype=torch.uint8, device="cuda"), torch.zeros(1, device="cuda")
    for t in range(40):
        B.mla_cache_append(kv[t:t + 1, :512], kv[t:t + 1, 512:], dev([t], np.int32), cache, sc, scale_group=g)
    torch.cuda.synchronize()
    once_c, once_s = S.cache_append(x, np.arange(40), np.zeros((64, 576), np.uint8), np.zeros(1), g)
    assert float(sc[0]) == once_s[0]
    a = O.decode_e4m3fn(cache.view(-1, 576).cpu().numpy())
    b = O.decode_e4m3fn(once_c)
    # subnormal codes: one rounding at each of at most 6 growths, each half of the smallest step or less
    assert np.all(np.abs(a - b) <= np.where(np.abs(b) < 2.0 ** -5, 6 * 2.0 ** -10, 0.0))


def test_append_sizes_and_empty():
    rng = np.random.default_rng(9)
    for T, bs, g in ((0, 64, 64), (1, 64, 64), (2431, 64, 64), (2433, 16, 16), (4001, 64, 2)):
        slots, nb = step_slots(rng, [11], [T], bs)
        codes, scales = filled(rng, nb * bs, g)
        check_append(rng.standard_normal((T, 576)), slots, codes, scales, bs, g)


def test_append_separate_parts_with_wide_strides():
    rng = np.random.default_rng(10)
    T, bs, g = 9, 16, 8
    x, kv = bf16(rng.standard_normal((T, 576)))
    c = torch.full((T, 1024), float("nan"), dtype=torch.bfloat16, device="cuda")
    k = torch.full((T, 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    c[:, 8:520], k[:, :64] = kv[:, :512], kv[:, 512:]
    cache, sc = torch.zeros((1, bs, 576), dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(2, device="cuda")
    B.mla_cache_append(c[:, 8:520], k[:, :64], dev(np.arange(T), np.int32), cache, sc, scale_group=g)
    torch.cuda.synchronize()
    want_c, want_s = S.cache_append(x, np.arange(T), np.zeros((bs, 576), np.uint8), np.zeros(2), g)
    assert np.array_equal(cache.view(torch.uint8).view(-1, 576).cpu().numpy(), want_c)
    assert np.array_equal(sc.cpu().numpy(), want_s)


# ---------------------------------------------------------------- attention

def decode_case(seed, lens, heads, bs, g, qlens=None, sinks=False, spread=1.0, topk=0, scale_exp=None):
    """Random requests; unused blocks, the rows behind a request's last and the
    scales of groups without a live row are NaN."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, dtype=np.int64)
    need = -(-lens // bs)
    ids = rng.permutation(int(need.sum()) + 2)
    cols = max(1, int(need.max()) if len(lens) else 1) + 1
    table = np.full((len(lens), cols), ids[-1])
    live = np.zeros(len(ids) * bs, bool)
    k = 0
    for r, m in enumerate(int(v) for v in need):
        table[r, :m] = ids[k:k + m]
        k += m
        live[S.row_slots(table[r], bs, int(lens[r]))] = True
    n = len(live)
    rows = bf16(rng.standard_normal((n, 576)) * np.exp(0.5 * spread * rng.standard_normal((n, 1))))[0]
    codes, scales = S.cache_append(rows, np.arange(n), np.zeros((n, 576), np.uint8), np.zeros(n // g), g)
    if scale_exp is not None:
        scales = scales * np.exp2(rng.integers(scale_exp[0], scale_exp[1] + 1, scales.shape))
    else:
        scales = scales * rng.uniform(0.6, 1.4, scales.shape).astype(np.float32)  # any scale, not powers of two alone
    scales = scales.astype(np.float32).astype(np.float64)
    codes[~live] = 0x7F
    scales[~live.reshape(-1, g).any(1)] = np.nan
    q = np.ones(len(lens), np.int64) if qlens is None else np.asarray(qlens)
    qo = np.concatenate([[0], np.cumsum(q)])
    T = int(qo[-1])
    qc = I.float32_to_e4m3_codes(rng.standard_normal((T, heads, 576)).astype(np.float32) / QS)
    c = dict(lens=lens, table=table, codes=codes, scales=scales, q=qc, qo=None if qlens is None else qo, bs=bs, g=g,
             H=heads, T=T, nb=len(ids), max_qlen=int(q.max()) if len(q) else 1, topk=topk,
             sinks=rng.standard_normal(heads).astype(np.float32) if sinks else None)
    if topk:
        slots = np.full((T, topk), -1)
        for t in range(T):
            m = min(topk, int(lens[t]))
            m -= int(rng.integers(0, m // 4 + 1))
            at = rng.choice(topk, m, replace=False)       # holes anywhere
            slots[t, at] = S.row_slots(table[t], bs, int(lens[t]))[rng.choice(int(lens[t]), m, replace=False)]
        c["slots"] = slots
    return c


def run_decode(c, num_segments=0, kernel=B.MLA_KERNEL_AUTO, expect=None, stages=False):
    sparse = c["topk"] > 0
    plan = B.mla_decode_plan(B.make_problem(
        num_tokens=c["T"], num_heads=c["H"], block_size=c["bs"], num_blocks=c["nb"],
        num_reqs=0 if sparse else len(c["lens"]), max_blocks_per_req=c["table"].shape[1],
        max_seq_len=int(c["lens"].max()), max_qlen=1 if sparse else c["max_qlen"], topk=c["topk"], dtype="fp8",
        has_sinks=c["sinks"] is not None, num_segments=num_segments, kernel=kernel))
    if expect is not None:
        assert plan.kernel == expect, plan.kernel
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = torch.full((c["T"], c["H"], 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c["T"], c["H"]), float("nan"), device="cuda")
    seq = None if sparse else dev(c["lens"], np.int32)
    qo = None if c["qo"] is None else dev(c["qo"], np.int32)
    sinks = None if c["sinks"] is None else dev(c["sinks"])
    args = (plan, dev(c["q"]), dev(c["codes"]).view(c["nb"], c["bs"], 576), dev(c["scales"], np.float32))
    kw = dict(scale_group=c["g"], block_table=None if sparse else dev(c["table"], np.int32), seq_lens=seq, qo_indptr=qo,
              sparse_slots=dev(c["slots"], np.int32) if sparse else None, softmax_scale=SCALE, q_scale=QS, sinks=sinks,
              workspace=ws, out=out, lse=lse)
    if stages:
        B.mla_decode_schedule(plan, seq_lens=seq, qo_indptr=qo, workspace=ws)
        B.mla_decode_items_scaled(*args, **kw)
        B.mla_merge_items(plan, qo_indptr=qo, sinks=sinks, workspace=ws, out=out, lse=lse)
    else:
        B.mla_decode_fwd_scaled(*args, **kw)
    torch.cuda.synchronize()
    assert B.mla_workspace_status(plan, ws) == 0
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), (args, kw, plan)


def check_decode(c, **kw):
    out, lse, ran = run_decode(c, **kw)
    lists = list(c["slots"]) if c["topk"] else S.token_slots(c["table"], c["lens"], c["bs"], c["qo"])
    ro, rl, to, tl = S.decode(c["q"], QS, c["codes"], c["scales"], c["g"], lists, SCALE, c["sinks"], bounds=True)
    compare(out, lse, ro, rl, to, tl)
    return out, lse, ran


def compare(out, lse, ro, rl, to, tl):
    assert np.isfinite(out).all() and not np.isnan(lse).any()
    assert np.array_equal(np.isneginf(lse), np.isneginf(rl))
    bad = np.abs(out - ro) > to
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(out - ro)[bad][:4], to[bad][:4])
    fin = np.isfinite(rl)
    off = np.abs(lse[fin] - rl[fin])
    assert (off <= tl[fin]).all(), np.max(off / np.maximum(tl[fin], 1e-30))
    # all roundings at once: the output's to bf16 (2^-8 / sqrt 3 of the value on
    # the mean, or less) and the weights' (the same, or less, of the output's
    # spread); a key missed or counted twice is far above it
    if out.size:
        norm = np.linalg.norm(ro)
        assert np.linalg.norm(out - ro) <= 5e-3 * norm + 1e-30, np.linalg.norm(out - ro) / norm


LENS = [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 192, 700, 1025, 2300]


# kernel ids of the plan: 1-3 warp MMA (16, 32, 64 rows), 4 CTA pair, 5 rows as N
@pytest.mark.parametrize("heads,bs,g,expect", [
    (16, 64, 64, 5), (1, 64, 1, 5), (7, 64, 16, 5), (17, 128, 128, 5), (32, 64, 32, 5), (48, 64, 8, 5), (64, 64, 64, 5),
    (57, 64, 2, 5), (96, 64, 64, 5), (81, 128, 4, 5), (128, 64, 64, 5), (128, 192, 24, 5), (113, 64, 1, 5),
    (16, 16, 16, 1), (5, 48, 24, 1), (32, 16, 1, 2), (20, 80, 40, 2), (128, 16, 8, 3), (99, 7, 7, 3), (64, 1, 1, 3)])
@pytest.mark.parametrize("sinks", [False, True])
def test_decode_single_tokens(heads, bs, g, expect, sinks):
    check_decode(decode_case(heads * 100 + g, LENS if bs > 1 else LENS[:11], heads, bs, g, sinks=sinks), expect=expect)


@pytest.mark.parametrize("heads,bs,g,expect", [(16, 64, 64, 5), (32, 64, 1, 5), (48, 64, 16, 4), (128, 64, 64, 4),
                                               (128, 64, 1, 4), (100, 128, 32, 4), (16, 16, 4, 3), (128, 48, 48, 3)])
@pytest.mark.parametrize("sinks", [False, True])
def test_decode_multi_token(heads, bs, g, expect, sinks):
    lens = [3, 4, 64, 66, 129, 130, 900, 1500]
    q = [3, 1, 2, 3, 3, 1, 2, 3] if heads != 32 else [2, 1, 2, 1, 2, 2, 1, 2]
    check_decode(decode_case(heads * 10 + g, lens, heads, bs, g, qlens=q, sinks=sinks), expect=expect)


@pytest.mark.parametrize("kernel,bs,heads", [(B.MLA_KERNEL_WARP_MMA, 64, 16), (B.MLA_KERNEL_WARP_MMA, 64, 128),
                                             (B.MLA_KERNEL_TCGEN05, 64, 16), (B.MLA_KERNEL_TCGEN05, 128, 128),
                                             (B.MLA_KERNEL_TCGEN05_ROWS_N, 64, 128)])
@pytest.mark.parametrize("ns", [0, 1, 3])
def test_decode_every_kernel_and_partition(kernel, bs, heads, ns):
    check_decode(decode_case(heads + ns, LENS, heads, bs, 32, sinks=ns == 3), kernel=kernel, num_segments=ns)


@pytest.mark.parametrize("heads,topk,bs,g", [(16, 128, 64, 64), (128, 256, 64, 1), (40, 384, 16, 8), (128, 2048, 48, 24)])
def test_decode_sparse(heads, topk, bs, g):
    lens = [topk + 5, 3 * topk, 1, topk // 2, 700]
    c = decode_case(topk + heads, lens, heads, bs, g, topk=topk, sinks=heads == 40)
    c["slots"][3] = -1                                     # a token that selects nothing
    check_decode(c)
    check_decode(c, num_segments=2)


@pytest.mark.parametrize("heads,bs,qlens", [(16, 64, None), (128, 64, None), (128, 64, [2, 3, 1, 3]), (16, 16, None)])
@pytest.mark.parametrize("exps", [(-6, 6), (-40, -36), (10, 14), (-50, 3)])
def test_decode_scales_far_apart(heads, bs, qlens, exps):
    """Groups whose scales differ by many binades: the weights' range follows
    the scaled values, so that small groups with large softmax weights still
    count in the denominator."""
    c = decode_case(7, [5, 300, 1100, 64], heads, bs, 8, qlens=qlens, scale_exp=exps, sinks=exps[0] == -6)
    check_decode(c)


@pytest.mark.parametrize("heads,bs,qlens", [(16, 64, None), (64, 64, None), (128, 64, None), (128, 64, [2]), (16, 16, None)])
def test_decode_one_key_outweighs_a_long_context(heads, bs, qlens):
    """One key without a value weighs 2^16 times as much as each of 9000 others
    whose values agree in sign: together they are the result."""
    c = decode_case(17, [9000], heads, bs, 1, qlens=qlens)
    rng = np.random.default_rng(18)
    q = np.tile(rng.standard_normal(576) * 2.0 ** -8, (c["T"], heads, 1)).astype(np.float32) / QS
    c["q"] = I.float32_to_e4m3_codes(q)
    c["codes"] &= 0x7F                                     # (poisoned slots stay NaN)
    at = S.row_slots(c["table"][0], bs, 9000)
    c["codes"][at] = I.float32_to_e4m3_codes(np.abs(rng.standard_normal((9000, 576))).astype(np.float32))
    c["scales"][at] = 1.0
    first = int(at[4000])
    rope = O.decode_e4m3fn(c["q"])[0, 0, 512:] * QS
    c["codes"][first, :512] = 0                            # it has no value of its own
    c["codes"][first, 512:] = I.float32_to_e4m3_codes(448 * np.sign(rope).astype(np.float32))
    c["scales"][first] = np.float32(16 * np.log(2.0) / (448 * SCALE * np.abs(rope).sum()))
    check_decode(c)


def test_decode_zero_groups():
    """Rows of zeros, written by the append under the smallest scale, weigh
    e^0 in the softmax beside keys of ordinary and of very negative score."""
    for bs, heads in ((64, 16), (64, 128), (16, 16)):
        c = decode_case(11, [640, 200], heads, bs, bs)
        z = S.row_slots(c["table"][0], bs, 640)[64:192]
        c["codes"][z] = 0
        c["scales"][np.unique(z // bs)] = 2.0 ** -60
        c["codes"][S.row_slots(c["table"][1], bs, 192)] = 0   # nearly everything is zero
        c["scales"][np.unique(S.row_slots(c["table"][1], bs, 192) // bs)] = 2.0 ** -60
        check_decode(c)


def test_decode_sinks_large_and_small():
    c = decode_case(12, [0, 40, 300], 16, 64, 64, sinks=True)
    c["sinks"][:4] = [60.0, -60.0, 0.0, 12.0]
    check_decode(c)


def test_decode_a_sink_of_minus_infinity_is_none():
    """Also for rows without keys: the bits of the call without sinks."""
    for heads, bs, q, lens in ((16, 64, None, [0, 40, 300]), (128, 64, None, [0, 40, 6000]), (128, 64, [2, 3, 1], [0, 40, 300]),
                               (16, 16, None, [0, 40, 300])):
        c = decode_case(15, lens, heads, bs, 16, qlens=q, sinks=True)
        c["sinks"][:] = -np.inf
        a = run_decode(c)
        c["sinks"] = None
        b = run_decode(c)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_decode_split_rows_and_stages():
    """One long request among short ones: pieces merged from partials; the
    three stages give the bits of the whole call, and so does a second call."""
    for heads, q in ((16, None), (128, None), (128, [2, 1, 3])):
        c = decode_case(13, [6000, 3, 500], heads, 64, 64, qlens=q)
        a = check_decode(c)
        b = run_decode(c, stages=True)
        again = run_decode(c)
        for x in (b, again):
            assert np.array_equal(a[0], x[0]) and np.array_equal(a[1], x[1])


def test_decode_unit_scales_match_the_tensor_scale():
    for heads, q in ((16, None), (128, None), (128, [3, 2])):
        c = decode_case(14, [700, 130], heads, 64, 64, qlens=q)
        c["scales"][:] = 0.125
        out, lse, (args, kw, plan) = check_decode(c)
        o2, l2 = torch.empty_like(kw["out"]), torch.empty_like(kw["lse"])
        B.mla_decode_fwd(plan, args[1], args[2], block_table=kw["block_table"], seq_lens=kw["seq_lens"],
                         qo_indptr=kw["qo_indptr"], softmax_scale=SCALE, q_scale=QS, kv_scale=0.125,
                         workspace=kw["workspace"], out=o2, lse=l2)
        torch.cuda.synchronize()
        lists = S.token_slots(c["table"], c["lens"], c["bs"], c["qo"])
        r = S.decode(c["q"], QS, c["codes"], c["scales"], c["g"], lists, SCALE, bounds=True)
        compare(o2.double().cpu().numpy(), l2.double().cpu().numpy(), *r)


def test_padding_requests_leave_other_rows_alone():
    c = decode_case(15, [0, 0, 90, 0], 128, 64, 16)
    out, lse, _ = check_decode(c)
    assert not out[[0, 1, 3]].any() and np.isneginf(lse[[0, 1, 3]]).all()


def test_binding_refuses_on_the_device():
    c = decode_case(16, [90], 16, 64, 16)
    _, _, ((plan, q, cache, sc), kw, _) = run_decode(c)
    for bad in (dict(scale_group=24), dict(scale_group=32), dict(block_table=kw["block_table"].long()),
                dict(seq_lens=kw["seq_lens"].repeat(2)), dict(out=kw["out"].half()), dict(lse=kw["lse"][:, ::2])):
        with pytest.raises(B.MLAError):
            B.mla_decode_fwd_scaled(plan, q, cache, sc, **{**kw, **bad})
    for a in ((q.repeat(2, 1, 1), cache, sc), (q, cache[:1], sc), (q, cache, sc.double()), (q, cache, sc.cpu()),
              (q.transpose(0, 1), cache, sc)):
        with pytest.raises(B.MLAError):
            B.mla_decode_fwd_scaled(plan, *a, **kw)
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(B.MLAError):
        B.mla_block_tables(i, i[:3].long(), i, i.view(1, 4), block_size=4, slot_mapping=i, taken=i[:1])
    with pytest.raises(B.MLAError):
        B.mla_block_tables(i[:3], i[:3], i, i.view(1, 4), block_size=4, slot_mapping=i, taken=i[:1])
    kv = torch.zeros((4, 576), dtype=torch.float16, device="cuda")
    with pytest.raises(B.MLAError):
        B.mla_cache_append(kv[:, :512], kv[:, 512:], i, cache, sc, scale_group=16)


# ---------------------------------------------------------------- the step, together

@pytest.mark.parametrize("heads,bs,g", [(16, 64, 64), (128, 64, 16), (16, 16, 1)])
def test_serving_steps(heads, bs, g):
    """Prompts, then decode steps of one to three tokens with requests that
    pause: every step builds its slots on the device, appends and attends; the
    oracle runs the same steps on the host."""
    rng = np.random.default_rng(heads + bs + g)
    R, cols, nb = 5, 12, 64
    ids = rng.permutation(nb)
    lens = np.zeros(R, np.int64)
    table = np.full((R, cols), -1)
    codes, scales = np.full((nb * bs, 576), 0x7F, np.uint8), np.full(nb * bs // g, np.nan)
    d_table, d_cache, d_sc = dev(table, np.int32), dev(codes).view(nb, bs, 576), dev(scales, np.float32)
    used = 0
    for q in ([70, 1, 0, 2 * bs + 1, 33], [1, 1, 5, 1, 1], [1, 3, 1, 0, 2], [3, 3, 3, 3, 3], [1, 0, 0, 1, 1]):
        q = np.asarray(q)
        lens = lens + q
        qsl = np.concatenate([[0], np.cumsum(q)])
        T = int(qsl[-1]) + 3                                # padded, as a captured batch is
        rows = rng.standard_normal((T, 576)) * np.exp(rng.standard_normal((T, 1)))
        x, kv = bf16(rows)
        free = ids[used:]
        table, slots, _, _, taken = S.block_tables(qsl, lens, free, table, bs, T)
        codes, scales = S.cache_append(x, slots, codes, scales, g)
        d_qsl, d_lens = dev(qsl, np.int32), dev(lens, np.int32)
        d_slots, d_taken = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        B.mla_block_tables(d_qsl, d_lens, dev(free, np.int32), d_table, block_size=bs, slot_mapping=d_slots, taken=d_taken)
        B.mla_cache_append(kv[:, :512], kv[:, 512:], d_slots, d_cache, d_sc, scale_group=g)
        n = int(qsl[-1])
        plan = B.mla_decode_plan(B.make_problem(num_tokens=n, num_heads=heads, block_size=bs, num_blocks=nb, num_reqs=R,
                                                max_blocks_per_req=cols, max_seq_len=cols * bs,
                                                max_qlen=int(q.max()), dtype="fp8"))
        ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        qc = I.float32_to_e4m3_codes(rng.standard_normal((n, heads, 576)).astype(np.float32) / QS)
        out, lse = torch.empty((n, heads, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((n, heads), device="cuda")
        B.mla_decode_fwd_scaled(plan, dev(qc), d_cache, d_sc, scale_group=g, block_table=d_table, seq_lens=d_lens,
                                qo_indptr=d_qsl, softmax_scale=SCALE, q_scale=QS, workspace=ws, out=out, lse=lse)
        torch.cuda.synchronize()
        assert int(d_taken[0]) == taken
        used += taken
        assert np.array_equal(d_table.cpu().numpy(), table) and np.array_equal(d_slots.cpu().numpy(), slots)
        assert np.array_equal(d_sc.cpu().numpy(), scales.astype(np.float32), equal_nan=True)
        lists = S.token_slots(table, lens, bs, qsl)
        compare(out.double().cpu().numpy(), lse.double().cpu().numpy(),
                *S.decode(qc, QS, codes, scales, g, lists, SCALE, bounds=True))


@pytest.mark.parametrize("H", [16, 128])
def test_step_captured_and_replayed(H):
    """One decode step captured in a graph on a side stream and replayed with
    other lengths, rows and queries in the same buffers."""
    rng = np.random.default_rng(21)
    R, cols, nb, bs, g = 3, 8, 32, 64, 64
    codes0, scales0 = filled(rng, nb * bs, g)
    ids = rng.permutation(nb)
    buf = dict(qsl=dev(np.arange(R + 1), np.int32), lens=dev(np.ones(R), np.int32), free=dev(ids[20:], np.int32),
               table=dev(np.full((R, cols), -1), np.int32), slots=dev(np.zeros(R), np.int32), taken=dev([0], np.int32),
               kv=torch.zeros((R, 576), dtype=torch.bfloat16, device="cuda"), cache=dev(codes0).view(nb, bs, 576),
               sc=dev(scales0, np.float32), q=torch.zeros((R, H, 576), dtype=torch.uint8, device="cuda"))
    plan = B.mla_decode_plan(B.make_problem(num_tokens=R, num_heads=H, block_size=bs, num_blocks=nb, num_reqs=R,
                                            max_blocks_per_req=cols, max_seq_len=cols * bs, dtype="fp8"))
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty((R, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((R, H), device="cuda")

    def step():
        B.mla_block_tables(buf["qsl"], buf["lens"], buf["free"], buf["table"], block_size=bs, slot_mapping=buf["slots"],
                           taken=buf["taken"])
        B.mla_cache_append(buf["kv"][:, :512], buf["kv"][:, 512:], buf["slots"], buf["cache"], buf["sc"], scale_group=g)
        B.mla_decode_fwd_scaled(plan, buf["q"], buf["cache"], buf["sc"], scale_group=g, block_table=buf["table"],
                                seq_lens=buf["lens"], softmax_scale=SCALE, q_scale=QS, workspace=ws, out=out, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([65, 1, 400], [64, 129, 2]):
        ctx = np.asarray(lens) - 1
        old = -(-ctx // bs)
        table, k = np.full((R, cols), -1), 0
        for r in range(R):
            table[r, :old[r]] = ids[k:k + old[r]]
            k += int(old[r])
        x, kv = bf16(rng.standard_normal((R, 576)) * 9)
        qc = I.float32_to_e4m3_codes(rng.standard_normal((R, H, 576)).astype(np.float32) / QS)
        for name, v in (("lens", np.asarray(lens, np.int32)), ("table", table.astype(np.int32)), ("q", qc)):
            buf[name].copy_(dev(v))
        buf["kv"].copy_(kv)
        buf["cache"].copy_(dev(codes0).view(nb, bs, 576))
        buf["sc"].copy_(dev(scales0, np.float32))
        graph.replay()
        torch.cuda.synchronize()
        table, slots, _, _, taken = S.block_tables(np.arange(R + 1), lens, ids[20:], table, bs, R)
        codes, scales = S.cache_append(x, slots, codes0, scales0, g)
        assert int(buf["taken"][0]) == taken and np.array_equal(buf["table"].cpu().numpy(), table)
        compare(out.double().cpu().numpy(), lse.double().cpu().numpy(),
                *S.decode(qc, QS, codes, scales, g, S.token_slots(table, lens, bs), SCALE, bounds=True))


def test_cache_beyond_32_bit_offsets():
    """Slots whose byte offsets pass 2^32: the append and every dense kernel."""
    bs, g = 64, 64
    nb = (1 << 32) // (576 * bs) + 40
    cache = torch.zeros((nb, bs, 576), dtype=torch.uint8, device="cuda")
    sc = torch.full((nb,), 2.0 ** -60, device="cuda")
    rng = np.random.default_rng(31)
    n = 200
    x, kv = bf16(rng.standard_normal((n, 576)))
    blocks = np.array([nb - 1, 3, nb - 7, nb - 2])
    slots = S.row_slots(blocks, bs, n)
    B.mla_cache_append(kv[:, :512], kv[:, 512:], dev(slots, np.int32), cache, sc, scale_group=g)
    small_c, small_s = S.cache_append(x, S.row_slots(np.arange(4), bs, n), np.zeros((4 * bs, 576), np.uint8), np.zeros(4), g)
    torch.cuda.synchronize()
    at = dev(blocks, np.int64)
    assert np.array_equal(cache[at].view(-1, 576).cpu().numpy(), small_c)
    assert np.array_equal(sc[at].cpu().numpy(), small_s)
    for heads, q, kernel in ((16, 1, B.MLA_KERNEL_AUTO), (128, 2, B.MLA_KERNEL_AUTO), (16, 1, B.MLA_KERNEL_WARP_MMA)):
        qc = I.float32_to_e4m3_codes(rng.standard_normal((q, heads, 576)).astype(np.float32) / QS)
        plan = B.mla_decode_plan(B.make_problem(num_tokens=q, num_heads=heads, block_size=bs, num_blocks=nb, num_reqs=1,
                                                max_blocks_per_req=4, max_seq_len=n, max_qlen=q, dtype="fp8", kernel=kernel))
        ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty((q, heads, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((q, heads), device="cuda")
        B.mla_decode_fwd_scaled(plan, dev(qc), cache, sc, scale_group=g, block_table=dev(blocks[None], np.int32),
                                seq_lens=dev([n], np.int32), qo_indptr=dev([0, q], np.int32), softmax_scale=SCALE,
                                q_scale=QS, workspace=ws, out=out, lse=lse)
        torch.cuda.synchronize()
        lists = S.token_slots(np.arange(4)[None], [n], bs, [0, q])
        compare(out.double().cpu().numpy(), lse.double().cpu().numpy(),
                *S.decode(qc, QS, small_c, small_s, g, lists, SCALE, bounds=True))


@pytest.mark.parametrize("heads,g", [(1, 64), (128, 1), (100, 16)])
def test_decode_sparse_ragged_lists(heads, g):
    """Slot lists of their own lengths, with holes, a slot listed twice and a
    list without slots."""
    rng = np.random.default_rng(heads)
    bs, nb = 64, 24
    codes, scales = filled(rng, nb * bs, g)
    lists = []
    for n in (0, 1, 2, 127, 128, 129, 500, 512):
        s = rng.choice(nb * bs, n, replace=False)
        s[rng.random(n) < 0.1] = -1
        if n > 2:
            s[-1] = s[0] = 5
        lists.append(s)
    lists.append(np.full(40, -1))
    T, topk = len(lists), 512
    indptr = np.concatenate([[0], np.cumsum([len(s) for s in lists])])
    qc = I.float32_to_e4m3_codes(rng.standard_normal((T, heads, 576)).astype(np.float32) / QS)
    for ns in (0, 1, 4):
        plan = B.mla_decode_plan(B.make_problem(num_tokens=T, num_heads=heads, block_size=bs, num_blocks=nb, num_reqs=0,
                                                max_blocks_per_req=0, max_seq_len=0, topk=topk, dtype="fp8", num_segments=ns))
        ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty((T, heads, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((T, heads), device="cuda")
        B.mla_decode_fwd_scaled(plan, dev(qc), dev(codes).view(nb, bs, 576), dev(scales, np.float32), scale_group=g,
                                sparse_slots=dev(np.concatenate(lists), np.int32), sparse_indptr=dev(indptr, np.int32),
                                softmax_scale=SCALE, q_scale=QS, workspace=ws, out=out, lse=lse)
        torch.cuda.synchronize()
        assert B.mla_workspace_status(plan, ws) == 0
        compare(out.double().cpu().numpy(), lse.double().cpu().numpy(),
                *S.decode(qc, QS, codes, scales, g, lists, SCALE, bounds=True))


def test_sparse_beyond_32_bit_offsets():
    bs, g, heads, topk = 64, 1, 128, 256
    nb = (1 << 32) // (576 * bs) + 40
    rng = np.random.default_rng(32)
    rows = np.concatenate([rng.choice(nb * bs, 100, replace=False), np.arange(nb * bs - 100, nb * bs)])
    codes, scales = filled(rng, len(rows), g)
    cache = torch.zeros((nb, bs, 576), dtype=torch.uint8, device="cuda")
    sc = torch.full((nb * bs,), float("nan"), device="cuda")
    cache.view(-1, 576)[dev(rows, np.int64)] = dev(codes)
    sc[dev(rows, np.int64)] = dev(scales, np.float32)
    slots = np.full((1, topk), -1)
    slots[0, 30:230] = rows
    lists = [np.where(slots[0] >= 0, np.arange(topk) - 30, -1)]
    qc = I.float32_to_e4m3_codes(rng.standard_normal((1, heads, 576)).astype(np.float32) / QS)
    plan = B.mla_decode_plan(B.make_problem(num_tokens=1, num_heads=heads, block_size=bs, num_blocks=nb, num_reqs=0,
                                            max_blocks_per_req=0, max_seq_len=0, topk=topk, dtype="fp8"))
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty((1, heads, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((1, heads), device="cuda")
    B.mla_decode_fwd_scaled(plan, dev(qc), cache, sc, scale_group=g, sparse_slots=dev(slots, np.int32), softmax_scale=SCALE,
                            q_scale=QS, workspace=ws, out=out, lse=lse)
    torch.cuda.synchronize()
    compare(out.double().cpu().numpy(), lse.double().cpu().numpy(),
            *S.decode(qc, QS, codes, scales, g, lists, SCALE, bounds=True))


def test_two_streams_at_once():
    """Calls in flight on two streams, each with its workspace: the bits of
    the calls made alone."""
    cases = [decode_case(41, [3000, 70, 900], 128, 64, 16), decode_case(42, [2000, 1, 640], 16, 64, 64)]
    alone = [run_decode(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for _, _, (args, kw, _) in alone:
        kw["out"].fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(8):
        for s, (_, _, (args, kw, _)) in zip(streams, alone):
            B.mla_decode_fwd_scaled(*args, **kw, stream=s)
    torch.cuda.synchronize()
    for out, lse, (_, kw, _) in alone:
        assert np.array_equal(out, kw["out"].double().cpu().numpy())
        assert np.array_equal(lse, kw["lse"].double().cpu().numpy())


@pytest.mark.parametrize("heads,qlens,topk", [(128, None, 0), (128, [3, 2], 0), (128, None, 512), (16, None, 0)])
def test_bounded_wait_runs_out_and_is_reported(heads, qlens, topk):
    """With a limit of a microsecond the kernel's waits give up: it drains what
    it issued, exits and leaves a code; the next call is right."""
    c = decode_case(43, [2000, 900], heads, 64, 16, qlens=qlens, topk=topk)
    _, _, (args, kw, plan) = check_decode(c)
    plan.wait_limit_us = 1
    B.mla_decode_fwd_scaled(*args, **kw)
    torch.cuda.synchronize()
    code = B.mla_workspace_status(plan, kw["workspace"], clear=True)
    assert code != 0
    plan.wait_limit_us = 0
    B.mla_decode_fwd_scaled(*args, **kw)
    torch.cuda.synchronize()
    assert B.mla_workspace_status(plan, kw["workspace"]) == 0
    lists = list(c["slots"]) if topk else S.token_slots(c["table"], c["lens"], c["bs"], c["qo"])
    compare(kw["out"].double().cpu().numpy(), kw["lse"].double().cpu().numpy(),
            *S.decode(c["q"], QS, c["codes"], c["scales"], c["g"], lists, SCALE, c["sinks"], bounds=True))


@pytest.mark.parametrize("heads,qlens,longest", [(16, None, 512), (17, None, 512), (48, None, 511), (64, [1, 3, 0, 2, 1, 1, 1], 300),
                                                 (128, None, 512), (128, [2, 3, 0, 3, 1, 1, 2], 512), (128, None, 513)])
@pytest.mark.parametrize("sinks", [False, True])
def test_decode_short_requests(heads, qlens, longest, sinks):
    """Short requests, which a whole call does not split, and the three stages
    over the same ones, which do; also in so many requests that neither kernel
    takes them in one wave."""
    lens = [longest, 64, 5, 129, 300, 2, 256]
    c = decode_case(51, lens, heads, 64, 16, qlens=qlens, sinks=sinks)
    check_decode(c)
    check_decode(c, stages=True)
    check_decode(decode_case(52, [33] * 40 + [100] * 40 + [0] * 80, heads, 64, 64, sinks=sinks))


@pytest.mark.parametrize("heads,qlens", [(1, None), (16, None), (32, [2]), (128, None), (128, [3])])
def test_decode_one_long_request(heads, qlens):
    """A row of many partials: more than 40 pieces, merged by four warps a row."""
    check_decode(decode_case(61, [19999], heads, 64, 64, qlens=qlens, sinks=True))
    check_decode(decode_case(62, [9001, 1], heads, 16, 8, qlens=None if qlens is None else qlens + [1]), num_segments=40)

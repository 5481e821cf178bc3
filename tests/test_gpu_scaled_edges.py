"""The serving step over a cache with group scales at its edges: table cells
without a block, rows behind the last request, sinks and keys that are no
numbers, work lists shared between calls, and every kernel a scaled call can
run on, each against the oracle."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import scaled_oracle as S
from paged_mla_decode_06_gb300 import binding as B
from paged_mla_decode_06_gb300 import build as BUILD
from paged_mla_decode_06_gb300 import inputs as I
from tests.gpu_helpers import assert_close
from tests.test_gpu_scaled_cache import QS, SCALE, compare, decode_case, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    BUILD.build()
    B.load_library()


class Call:
    """A decode over the case's tensors. ``bound``: the host's bound of the
    lengths, where it is not the longest; ``ahead`` and ``behind``: rows of q,
    out and lse before the first request and past the last."""

    def __init__(self, c, bound=None, ahead=0, behind=0, num_segments=0, kernel=B.MLA_KERNEL_AUTO):
        self.c = c
        table = c["table"]
        if bound is not None:  # columns that no request fills
            cols = max(table.shape[1], -(-bound // c["bs"]))
            table = np.concatenate([table, np.full((len(table), cols - table.shape[1]), table[0, -1])], 1)
        T = ahead + c["T"] + behind
        self.plan = B.mla_decode_plan(B.make_problem(
            num_tokens=T, num_heads=c["H"], block_size=c["bs"], num_blocks=c["nb"], num_reqs=len(c["lens"]),
            max_blocks_per_req=table.shape[1], max_seq_len=int(bound if bound is not None else c["lens"].max()),
            max_qlen=c["max_qlen"], dtype="fp8", has_sinks=c["sinks"] is not None, num_segments=num_segments,
            kernel=kernel))
        q = np.concatenate([np.full((n, c["H"], 576), 0x7F, np.uint8) if x is None else x
                            for n, x in ((ahead, None), (0, c["q"]), (behind, None))])
        self.args = (self.plan, dev(q), dev(c["codes"]).view(c["nb"], c["bs"], 576))
        self.scales = dev(c["scales"], np.float32)
        self.seq = dev(c["lens"], np.int32)
        self.qo = None if c["qo"] is None else dev(c["qo"] + ahead, np.int32)
        self.sinks = None if c["sinks"] is None else dev(c["sinks"])
        self.ws = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        self.out = torch.empty((T, c["H"], 512), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.empty((T, c["H"]), device="cuda")
        self.kw = dict(block_table=dev(table, np.int32), seq_lens=self.seq, qo_indptr=self.qo, softmax_scale=SCALE,
                       q_scale=QS, sinks=self.sinks, workspace=self.ws, out=self.out, lse=self.lse)

    def clear(self):
        self.out.fill_(-7.0)
        self.lse.fill_(-7.0)

    def result(self):
        torch.cuda.synchronize()
        assert B.mla_workspace_status(self.plan, self.ws) == 0
        return self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()

    def schedule(self, of=None):
        (of or B.mla_decode_schedule)(self.plan, seq_lens=self.seq, qo_indptr=self.qo, workspace=self.ws)

    def merge(self):
        B.mla_merge_items(self.plan, qo_indptr=self.qo, sinks=self.sinks, workspace=self.ws, out=self.out, lse=self.lse)

    def fwd_scaled(self):
        self.clear()
        B.mla_decode_fwd_scaled(*self.args, self.scales, scale_group=self.c["g"], **self.kw)
        return self.result()

    def stages_scaled(self, of=None):
        self.clear()
        self.schedule(of)
        B.mla_decode_items_scaled(*self.args, self.scales, scale_group=self.c["g"], **self.kw)
        self.merge()
        return self.result()

    def items(self, kv_scale):
        """The unscaled decode over the list in the workspace, and its merge."""
        self.clear()
        B.mla_decode_items(*self.args, kv_scale=kv_scale, **self.kw)
        self.merge()
        return self.result()


def reference(c):
    lists = S.token_slots(c["table"], c["lens"], c["bs"], c["qo"])
    return S.decode(c["q"], QS, c["codes"], c["scales"], c["g"], lists, SCALE, c["sinks"], bounds=True)


# (heads, block size, group, tokens of the requests): the rows-as-N kernel at
# 16 rows, the value-split kernel with shared scales and with one a key, over
# blocks that boxes do not fit, and the warp-MMA kernel
SHAPES = [(16, 64, 64, None), (16, 128, 1, [2, 1, 3, 1, 2]), (48, 64, 16, None), (128, 64, 64, None), (128, 128, 1, None),
          (128, 64, 16, [2, 3, 1, 1, 2]), (128, 48, 24, None), (16, 16, 16, None)]


@pytest.mark.parametrize("heads,bs,g,qlens", SHAPES)
@pytest.mark.parametrize("bound", [None, 60000])
def test_keys_without_a_block_are_skipped(heads, bs, g, qlens, bound):
    """Cells below 0 in the middle, at either end and over all of a request's
    columns, as a free list that was too short leaves them: no key of theirs
    counts, and none of another request's is read in their place."""
    c = decode_case(71, [300, 2 * bs, 700, 5000, 65], heads, bs, g, qlens=qlens, sinks=heads == 48)
    t = c["table"]
    t[0, 1] = -1
    t[1, :2] = -1
    t[2, 0] = t[2, -(-700 // bs) - 1] = -1
    t[3, [3, 4, 5, 20]] = -1
    t[3, 7] = -5
    call = Call(c, bound=bound)
    compare(*call.fwd_scaled(), *reference(c))
    if call.plan.schedule == 1:
        compare(*call.stages_scaled(), *reference(c))


def test_a_step_on_a_short_free_list():
    """Tables, append and decode of one step on one stream, three blocks short:
    the tokens without a slot are not written and not attended to."""
    rng = np.random.default_rng(72)
    R, cols, nb, bs, g, H = 3, 8, 16, 64, 64, 128
    q = np.array([200, 150, 100])
    qsl, T = np.concatenate([[0], np.cumsum(q)]), int(q.sum())
    free = rng.permutation(nb)[:6]                          # of the nine that the step takes
    rows = torch.from_numpy(rng.standard_normal((T, 576)).astype(np.float32)).bfloat16()
    table, slots, _, _, taken = S.block_tables(qsl, q, free, np.full((R, cols), -1), bs, T)
    codes, scales = S.cache_append(rows.double().numpy(), slots, np.full((nb * bs, 576), 0x7F, np.uint8), np.full(nb, np.nan), g)
    kv, d_table = rows.cuda(), dev(np.full((R, cols), -1), np.int32)
    cache, sc = dev(np.full((nb, bs, 576), 0x7F, np.uint8)), dev(np.full(nb, np.nan), np.float32)
    d_qsl, d_lens = dev(qsl, np.int32), dev(q, np.int32)
    d_slots, d_taken = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    plan = B.mla_decode_plan(B.make_problem(num_tokens=T, num_heads=H, block_size=bs, num_blocks=nb, num_reqs=R,
                                            max_blocks_per_req=cols, max_seq_len=cols * bs, max_qlen=200, dtype="fp8"))
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    qc = I.float32_to_e4m3_codes(rng.standard_normal((T, H, 576)).astype(np.float32) / QS)
    out, lse = torch.empty((T, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((T, H), device="cuda")
    B.mla_block_tables(d_qsl, d_lens, dev(free, np.int32), d_table, block_size=bs, slot_mapping=d_slots, taken=d_taken)
    B.mla_cache_append(kv[:, :512], kv[:, 512:], d_slots, cache, sc, scale_group=g)
    B.mla_decode_fwd_scaled(plan, dev(qc), cache, sc, scale_group=g, block_table=d_table, seq_lens=d_lens, qo_indptr=d_qsl,
                            softmax_scale=SCALE, q_scale=QS, workspace=ws, out=out, lse=lse)
    torch.cuda.synchronize()
    assert int(d_taken[0]) == taken == 9 and np.array_equal(d_table.cpu().numpy(), table)
    pick = np.concatenate([np.arange(0, T, 37), [T - 1]])   # (the oracle at 450 tokens x 128 heads is slow)
    lists = S.token_slots(table, q, bs, qsl)
    compare(out.double().cpu().numpy()[pick], lse.double().cpu().numpy()[pick],
            *S.decode(qc[pick], QS, codes, scales, g, [lists[t] for t in pick], SCALE, bounds=True))


# ---------------------------------------------------------------- rows of no request

@pytest.mark.parametrize("heads,bs,ns,bound", [(16, 64, 0, None), (16, 64, 0, 60000), (128, 64, 0, None), (128, 64, 3, None),
                                               (16, 64, 3, None), (16, 16, 0, None), (128, 48, 2, None)])
@pytest.mark.parametrize("ahead", [0, 2])
def test_rows_of_no_request_stay_as_they_were(heads, bs, ns, bound, ahead):
    """A padded batch: the last request, split into pieces, has fewer tokens
    than the longest, and the tensors more rows than there are tokens."""
    c = decode_case(73, [9000, 900, 9000], heads, bs, 16, qlens=[1, 3, 1], sinks=True)
    call = Call(c, ahead=ahead, behind=4, num_segments=ns, bound=bound)
    mine = slice(ahead, ahead + c["T"])
    other = np.r_[0:ahead, ahead + c["T"]:ahead + c["T"] + 4]
    for run in (call.fwd_scaled,) + ((call.stages_scaled,) if call.plan.schedule == 1 else ()):
        out, lse = run()
        assert (out[other] == -7.0).all() and (lse[other] == -7.0).all()
        compare(out[mine], lse[mine], *reference(c))


# ---------------------------------------------------------------- a list in a shared workspace

@pytest.mark.parametrize("heads,qlens", [(48, None), (128, None), (16, [3, 2, 2, 3, 1]), (16, None)])
def test_the_unscaled_items_run_over_the_list_of_a_scaled_call(heads, qlens):
    """One list serves any number of calls: the one that a scaled whole call
    leaves in the workspace is as good for mla_decode_items as that of
    mla_decode_schedule, before it or not. Rows that are split and rows that
    are not; no partial of the scaled call is left."""
    c = decode_case(74, [1500, 6500, 100, 2500, 64], heads, 64, 64, qlens=qlens)
    c["scales"][:] = 2.0 ** -7                              # values of about unit variance, as assert_close has them
    ref = reference(c)
    seen = np.array([len(s) for s in S.token_slots(c["table"], c["lens"], c["bs"], c["qo"])])
    for scheduled in (False, True):
        call = Call(c)
        assert call.plan.schedule == 1 and call.plan.kernel == 5
        if scheduled:
            call.schedule()
        compare(*call.fwd_scaled(), *ref)
        call.ws[call.plan.segm_output_offset:] = 0xFF       # NaN
        assert_close(*call.items(2.0 ** -7), *ref[:2], "fp8", f"scheduled {scheduled}", keys=seen)


# ---------------------------------------------------------------- values that are no numbers

@pytest.mark.parametrize("heads,bs,lens", [(16, 64, [0, 40, 9000]), (128, 64, [0, 40, 9000]), (16, 16, [0, 40, 300])])
@pytest.mark.parametrize("scaled", [True, False])
def test_a_sink_that_is_no_number_is_not_dropped(heads, bs, lens, scaled):
    """Its head is NaN in every row, split or not; the other heads keep their
    bits."""
    c = decode_case(75, lens, heads, bs, 16, sinks=True)
    got = []
    for sink in (0.5, np.nan):
        c["sinks"][5] = sink
        call = Call(c)
        call.clear()
        if scaled:
            got.append(call.fwd_scaled())
        else:
            B.mla_decode_fwd(*call.args, kv_scale=0.125, **call.kw)
            got.append(call.result())
    (out0, lse0), (out, lse) = got
    assert np.isfinite(out0).all() and np.isfinite(lse0).all()
    assert np.isnan(lse[:, 5]).all()
    assert np.isnan(out[1:, 5]).all()                       # (0 x NaN where there is no key: unspecified)
    rest = np.arange(heads) != 5
    assert np.array_equal(out[:, rest], out0[:, rest]) and np.array_equal(lse[:, rest], lse0[:, rest])


@pytest.mark.parametrize("heads,bs,g,bound", [(16, 64, 64, None), (8, 64, 1, 60000), (128, 64, 16, None), (128, 64, 1, None),
                                              (128, 48, 48, None), (16, 16, 16, None), (5, 16, 1, None)])
@pytest.mark.parametrize("last", [65, 130, 3000])
def test_a_nan_key_reaches_only_the_tokens_that_see_it(heads, bs, g, bound, last):
    """The last token of a request left NaN in its row: the earlier tokens, in
    whose softmax the key is masked, keep their results."""
    c = decode_case(76, [last, 200], heads, bs, g, qlens=[3, 2])
    ref = reference(c)
    bad = S.row_slots(c["table"][0], bs, last)[-1]
    c["codes"][bad, 3::7] = 0x7F
    c["codes"][bad, 4::7] = 0xFF
    out, lse = Call(c, bound=bound).fwd_scaled()
    keep = np.array([0, 1, 3, 4])
    compare(out[keep], lse[keep], *(x[keep] for x in ref))


@pytest.mark.parametrize("heads,bs,g,bound", [(16, 64, 64, None), (16, 64, 1, 60000), (40, 64, 16, 60000), (64, 64, 64, 60000),
                                              (128, 64, 16, None), (128, 64, 1, None), (128, 48, 48, None), (16, 16, 16, None)])
@pytest.mark.parametrize("sinks", [False, True])
def test_rows_that_see_a_nan_are_nan_split_or_not(heads, bs, g, bound, sinks):
    """A key with a NaN, a query of one head with a NaN and an ordinary
    request, whole and in pieces: every row is NaN in its output and its LSE
    or right, wherever the NaN lies."""
    c = decode_case(77, [65, 8000, 300, 8000], heads, bs, g, sinks=sinks)
    ref = reference(c)
    c["codes"][S.row_slots(c["table"][0], bs, 65)[3], 511] = 0x7F
    c["codes"][S.row_slots(c["table"][1], bs, 8000)[4001], 530] = 0xFF
    c["q"][2:, 7, 100] = 0x7F
    bad = np.zeros((4, heads), bool)
    bad[:2] = bad[2:, 7] = True
    for ns in (0, 3):
        out, lse = Call(c, bound=bound, num_segments=ns).fwd_scaled()
        assert np.isnan(out[bad]).all() and np.isnan(lse[bad]).all()
        compare(out[~bad], lse[~bad], *(x[~bad] for x in ref))


@pytest.mark.parametrize("g", [1, 8, 64])
@pytest.mark.parametrize("heads,bs", [(16, 64), (128, 64)])
def test_the_largest_and_smallest_rows_an_append_takes(heads, bs, g):
    """Rows of bf16's largest values, of 448 * 2^60, just beyond, and of zeros,
    appended: the scales stay in the decode's range, what is beyond saturates,
    and the decode over that cache is right."""
    rng = np.random.default_rng(78)
    n = 5 * 64
    rows = np.exp2(rng.uniform(-3, 3, (n, 576))) * rng.choice([-1.0, 1.0], (n, 576))
    rows[0:64] = 0.0
    rows[64, 7], rows[65, 3] = 3.38e38, -3.0e38
    rows[128, 0] = 448.0 * 2.0 ** 60
    rows[192, 0] = 452.0 * 2.0 ** 60
    t = torch.from_numpy(rows.astype(np.float32)).bfloat16()
    cache, sc = torch.zeros((5, bs, 576), dtype=torch.uint8, device="cuda"), torch.zeros(n // g, device="cuda")
    kv = t.cuda()
    B.mla_cache_append(kv[:, :512], kv[:, 512:], dev(np.arange(n), np.int32), cache, sc, scale_group=g)
    torch.cuda.synchronize()
    got_s, codes = sc.double().cpu().numpy(), cache.view(-1, 576).cpu().numpy()
    assert (got_s >= 2.0 ** -60).all() and (got_s <= 2.0 ** 60).all()
    want_c, want_s = S.cache_append(t.double().numpy(), np.arange(n), np.zeros((n, 576), np.uint8), np.zeros(n // g), g)
    assert np.array_equal(got_s, want_s)
    assert np.array_equal(O.decode_e4m3fn(codes), O.decode_e4m3fn(want_c))
    assert O.decode_e4m3fn(codes[64, 7]) == 448.0 and O.decode_e4m3fn(codes[65, 3]) == -448.0
    # the queries are orthogonal to the columns that differ by many binades, so
    # that the softmax weighs all keys
    qc = I.float32_to_e4m3_codes(rng.standard_normal((1, heads, 576)).astype(np.float32) * 2.0 ** -6 / QS)
    qc[..., [0, 3, 7]] = 0
    plan = B.mla_decode_plan(B.make_problem(num_tokens=1, num_heads=heads, block_size=bs, num_blocks=5, num_reqs=1,
                                            max_blocks_per_req=5, max_seq_len=n, dtype="fp8"))
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty((1, heads, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((1, heads), device="cuda")
    table = np.arange(5)[None]
    B.mla_decode_fwd_scaled(plan, dev(qc), cache, sc, scale_group=g, block_table=dev(table, np.int32),
                            seq_lens=dev([n], np.int32), softmax_scale=SCALE, q_scale=QS, workspace=ws, out=out, lse=lse)
    torch.cuda.synchronize()
    compare(out.double().cpu().numpy(), lse.double().cpu().numpy(),
            *S.decode(qc, QS, codes, got_s, g, S.token_slots(table, [n], bs), SCALE, bounds=True))


# ---------------------------------------------------------------- the rows-as-N kernel at 17 to 64 rows

# (heads, tokens of the requests, group): 32, 48 and 64 rows a CTA, part filled or full
ROWS_N = [(17, None, 64), (32, None, 1), (48, None, 16), (57, None, 2), (64, None, 64), (64, None, 1),
          (8, [3, 1, 2, 3, 1, 2], 32), (16, [1, 3, 3, 2, 1, 3], 8), (21, [2, 3, 1, 3, 3, 1], 64), (16, [4, 2, 4, 1, 4, 3], 16)]


@pytest.mark.parametrize("heads,qlens,g", ROWS_N)
@pytest.mark.parametrize("sinks", [False, True])
def test_rows_as_n_over_long_contexts(heads, qlens, g, sinks):
    """Requests that are split among many workers, and short and empty ones; the
    stages apart give the bits of the whole call (one list for both)."""
    lens = [9001, 4, 129, 24000, 64, 777] if qlens else [9001, 0, 129, 24000, 1, 777]
    c = decode_case(81 + heads, lens, heads, 64, g, qlens=qlens, sinks=sinks)
    call = Call(c)
    assert B.mla_decode_scaled_kernel(call.plan) == 5 and call.plan.tile_rows in (32, 48, 64)
    a = call.fwd_scaled()
    compare(*a, *reference(c))
    b = call.stages_scaled()
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("heads,qlens,g", ROWS_N)
@pytest.mark.parametrize("ns", [1, 3])
def test_rows_as_n_with_a_fixed_partition(heads, qlens, g, ns):
    lens = [300, 4, 129, 1500, 64, 777] if qlens else [300, 0, 129, 1500, 1, 777]
    c = decode_case(82 + heads, lens, heads, 64, g, qlens=qlens, sinks=ns == 3)
    call = Call(c, num_segments=ns)
    assert B.mla_decode_scaled_kernel(call.plan) == 5
    compare(*call.fwd_scaled(), *reference(c))


@pytest.mark.parametrize("heads", [32, 48, 64])
@pytest.mark.parametrize("exps", [(-6, 6), (-40, -36), (10, 14), (-50, 3)])
def test_rows_as_n_with_scales_far_apart(heads, exps):
    c = decode_case(83, [5, 300, 1100, 64], heads, 64, 8, scale_exp=exps, sinks=exps[0] == -6)
    call = Call(c, bound=60000)
    assert B.mla_decode_scaled_kernel(call.plan) == 5
    compare(*call.fwd_scaled(), *reference(c))


@pytest.mark.parametrize("heads,qlens", [(16, None), (32, None), (48, None), (64, None), (20, [3])])
def test_rows_as_n_where_one_key_outweighs_a_long_context(heads, qlens):
    """One key without a value weighs 2^16 times as much as each of 9000 others
    whose values agree in sign: together they are the result."""
    c = decode_case(84, [9000], heads, 64, 1, qlens=qlens)
    rng = np.random.default_rng(85)
    q = np.tile(rng.standard_normal(576) * 2.0 ** -8, (c["T"], heads, 1)).astype(np.float32) / QS
    c["q"] = I.float32_to_e4m3_codes(q)
    at = S.row_slots(c["table"][0], 64, 9000)
    c["codes"][at] = I.float32_to_e4m3_codes(np.abs(rng.standard_normal((9000, 576))).astype(np.float32))
    c["scales"][at] = 1.0
    first = int(at[4000])
    rope = O.decode_e4m3fn(c["q"])[0, 0, 512:] * QS
    c["codes"][first, :512] = 0
    c["codes"][first, 512:] = I.float32_to_e4m3_codes(448 * np.sign(rope).astype(np.float32))
    c["scales"][first] = np.float32(16 * np.log(2.0) / (448 * SCALE * np.abs(rope).sum()))
    call = Call(c, bound=60000)
    assert B.mla_decode_scaled_kernel(call.plan) == 5
    compare(*call.fwd_scaled(), *reference(c))


@pytest.mark.parametrize("heads", [17, 48, 64])
def test_rows_as_n_over_more_short_requests_than_one_wave(heads):
    c = decode_case(86, [33] * 40 + [100] * 40 + [0] * 80, heads, 64, 64)
    call = Call(c, bound=512)
    assert B.mla_decode_scaled_kernel(call.plan) == 5
    compare(*call.fwd_scaled(), *reference(c))


# ---------------------------------------------------------------- whole calls and stages

@pytest.mark.parametrize("heads,lens,qlens", [
    (128, [40000, 3000, 17, 30000, 9000], None), (113, [9000, 20000, 1, 33000, 700, 23000], None),
    (128, [30000, 300, 9000], [2, 3, 1]), (64, [10000, 300, 2000], None), (32, [10000, 1, 900], None),
    (17, [5000, 5000, 0, 70, 6100], None), (16, [9000, 9000, 500], [2, 3, 1])])
def test_stages_and_whole_calls(heads, lens, qlens):
    """Rows of many pieces on the value-split kernel: the three stages give a
    whole call's bits; over the list of mla_decode_schedule, which is that of the
    plan's own kernel (a cut at every worker's share, slivers too), other bits,
    as right."""
    c = decode_case(91, lens, heads, 64, 64, qlens=qlens, sinks=heads == 64)
    call = Call(c)
    assert B.mla_decode_scaled_kernel(call.plan) == 6 and call.plan.schedule == 1
    ref = reference(c)
    a = call.fwd_scaled()
    compare(*a, *ref)
    b = call.stages_scaled(B.mla_decode_schedule_scaled)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    mine = call.ws[256:call.plan.segm_output_offset].clone()
    compare(*call.stages_scaled(), *ref)
    if call.plan.kernel == 5:
        assert not torch.equal(mine, call.ws[256:call.plan.segm_output_offset])


def test_a_list_serves_calls_until_another_replaces_it():
    """Stages over one list, twice, around an unsplit whole call, which leaves
    the list alone."""
    c = decode_case(92, [300, 5, 129, 512], 128, 64, 16)
    call = Call(c)
    a = call.stages_scaled()
    compare(*a, *reference(c))
    compare(*call.fwd_scaled(), *reference(c))
    call.clear()
    B.mla_decode_items_scaled(*call.args, call.scales, scale_group=c["g"], **call.kw)
    call.merge()
    b = call.result()
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


# ---------------------------------------------------------------- groups that grow

@pytest.mark.parametrize("g,rise", [(8, 0.5), (8, 2.0), (64, 0.125), (64, 0.4)])
def test_append_groups_that_grow_keep_within_a_smallest_step(g, rise):
    """Rows of rising size, one call each. A value that ends in the normal range
    was rounded once: 2^-4 of it. One that ends below was rounded to a grid of
    its own at first and then to the smallest step of each later scale, half a
    step each time, of steps that are different powers of two up to the last
    one's u: u/2 + u/4 + ... < u = 2^-9 of the scale."""
    rng = np.random.default_rng(95)
    n = min(g, 40)
    rows = rng.standard_normal((n, 576)) * np.exp2(rise * np.arange(n))[:, None]
    t = torch.from_numpy(rows.astype(np.float32)).bfloat16()
    x, kv = t.double().numpy(), t.cuda()
    cache, sc = torch.zeros((1, 64, 576), dtype=torch.uint8, device="cuda"), torch.zeros(64 // g, device="cuda")
    for i in range(n):
        B.mla_cache_append(kv[i:i + 1, :512], kv[i:i + 1, 512:], dev([i], np.int32), cache, sc, scale_group=g)
    torch.cuda.synchronize()
    s = float(sc[0])
    assert s >= np.abs(x).max() / 448.0
    off = np.abs(O.decode_e4m3fn(cache.view(-1, 576)[:n].cpu().numpy()) * s - x)
    assert (off <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -9 * s)).all()
    small = np.abs(x) < 2.0 ** -6 * s
    assert rise < 0.3 or (off[small] > 2.0 ** -10 * s).any()   # (more than one rounding leaves: the case is met)

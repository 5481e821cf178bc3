"""The decode of a batch that shares prefixes, and the decodes beside it, at their edges:
calls without a split row in captured graphs."""
import numpy as np
import pytest
import torch

from paged_mla_decode_06_gb300 import binding as B
from paged_mla_decode_06_gb300 import build as BUILD
from tests.test_gpu_shared import KVS, QS, SCALE, args_of, dev, shared_case

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

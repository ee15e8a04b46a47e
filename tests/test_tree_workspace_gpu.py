"""The workspace of the tree attention: one buffer serves every attention
operator in turn, whatever the one before left in it."""
import pytest
import torch

import decode_attention_static_gb300 as da
import paged_reference as R
from test_tree_attention_gpu import BOTH, Case

pytestmark = pytest.mark.gpu

COUNTERS = 4096  # bytes at the start of a workspace that are zero between calls


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    da.load_library()


def others():
    """Calls of the other attention operators, as functions of a workspace (None: one of their own)."""
    gen = torch.Generator(device="cuda").manual_seed(5)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)

    calls = {}
    for name, B, H, Hkv, rows in (("1 x 20000", 1, 32, 8, 20000), ("7 ragged", 7, 8, 2, 3000), ("40 short", 40, 16, 4, 900)):
        page = 64
        n = torch.tensor([rows - 11 * b for b in range(B)], dtype=torch.int32, device="cuda")
        most = -(-rows // page)
        table = torch.randperm(B * most, generator=torch.Generator().manual_seed(B)).view(B, most).to(torch.int32).cuda()
        q, k, v = randn(B, H, 128), randn(B * most, Hkv, page, 128), randn(B * most, Hkv, page, 128)
        calls["paged " + name] = lambda ws, q=q, k=k, v=v, table=table, n=n: da.decode_attn_paged_fwd(
            q, k, v, table, n, workspace=ws)
        kc, vc = randn(B, Hkv, rows, 128), randn(B, Hkv, rows, 128)
        calls["window " + name] = lambda ws, q=q, k=kc, v=vc, n=n: da.decode_attn_window_fwd(q, k, v, n, 700, 4, workspace=ws)
        calls["static " + name] = lambda ws, q=q, k=kc, v=vc, n=n: da.decode_attn_fwd(q, k, v, n, workspace=ws)
    return calls


@BOTH
def test_one_workspace_for_every_attention_operator(eight):
    """Tree calls whose units are divided (with a join by the last CTA alone, and with helpers), paged, window and static
    calls in turn on one buffer give what they give on buffers of their own, and leave its counters zero."""
    trees = [Case(lens, news, H, Hkv, 128, "bf16", 64, eight, seed=len(lens)).cuda()
             for lens, news, H, Hkv in (([9000], [64], 8, 2), ([2000, 900, 40], [20, 9, 40], 16, 4), ([5000], [3], 4, 2))]
    calls = others()
    big = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    own = {name: call(big if name.startswith("static") else None) for name, call in calls.items()}
    own_trees = [t.check() for t in trees]
    size = max(da.decode_attn_tree_workspace_size(16, 4, 128), da.decode_attn_paged_workspace_size(32, 8, 128),
               *(da.decode_attn_workspace_size(*s) for s in ((1, 32, 8, 128, 20000), (7, 8, 2, 128, 3000), (40, 16, 4, 128, 900))))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for again in range(2):
        for i, tree in enumerate(trees):
            for name, call in calls.items():
                assert torch.equal(R.bits(tree.check(f"{name}, tree {i}", workspace=ws)), R.bits(own_trees[i]))
                assert not ws[:COUNTERS].any(), f"a tree call left counters ({i})"
                assert torch.equal(R.bits(call(ws)), R.bits(own[name])), f"{name} behind tree {i}"
                assert not ws[:COUNTERS].any(), f"{name} left counters"


@BOTH
@pytest.mark.parametrize("lens,news", [([9000], [64]), ([5000], [3])], ids=["many rows", "few rows"])
def test_workspace_never_zero_filled(lens, news, eight):
    """Counters that are not zero: rows of units in parts become NaN with the error bit, none keeps what was in `out`;
    zero-filled again the buffer serves."""
    case = Case(lens, news, 8, 2, 128, "bf16", 64, eight, seed=3).cuda()
    clean = case.check()
    ws = torch.full((da.decode_attn_tree_workspace_size(8, 2, 128),), 1, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(case.q, 7.0)
        case.call(out=out, err_flag=err, workspace=ws)
        assert int(err.item()) == da.DA_DEVERR_WORKSPACE and out.isnan().all()
    da.workspace_init(ws)
    assert torch.equal(R.bits(case.check(workspace=ws)), R.bits(clean))


@BOTH
def test_units_of_one_cta_need_no_counters(eight):
    """Where no unit is divided the workspace's contents do not matter."""
    case = Case([100, 30, 60], [5, 9, 60], 8, 2, 64, "f16", 16, eight, seed=3).cuda()
    ws = torch.full((da.decode_attn_tree_workspace_size(8, 2, 64),), 1, dtype=torch.uint8, device="cuda")
    case.check(workspace=ws)

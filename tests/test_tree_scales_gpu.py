"""Tree attention over 8-bit pages whose V has scales of zero beside small ones:
pages of zero take their part of the softmax's sum, and nothing of the other
pages' precision."""
import pytest
import torch

import draft_reference as Q
import paged_reference as R
from test_tree_attention_gpu import Case

import decode_attention_static_gb300 as da

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    da.load_library()


def with_v_scales(lens, news, H, D, scale_of_page, heavy=False):
    """A case whose sequences' page j has V scale scale_of_page(j); heavy: keys of the pages of zero that take
    nearly all of the weight."""
    case = Case(lens, news, H, 2, D, "bf16", 16, True, kind="tree", seed=H + len(lens))
    for b, n in enumerate(lens):
        pages = case.table[b, :-(-n // 16)].long()
        case.vs[pages] = torch.tensor([scale_of_page(j) for j in range(len(pages))])[:, None].expand(-1, 2)
        zero = pages[case.vs[pages, 0] == 0]
        if heavy:
            case.ks[zero] *= 4.0
        rows = torch.arange(n)
        at = case.table[b].long()[rows // 16]
        k, v = (x.view(torch.uint8)[at, :, rows % 16].view(R.E4M3).double() * s[at].double()[..., None]
                for x, s in ((case.k, case.ks), (case.v, case.vs)))
        t, m = int(case.start[b]), news[b]
        case.ref[t:t + m], case.slack[t:t + m] = Q.attend_seen(
            case.q[t:t + m].double(), k.transpose(0, 1), v.transpose(0, 1), Q.seen_rows(n, m, case.masks[b]), case.scale,
            2.0 ** -11)
    return case


@pytest.mark.parametrize("heavy", [False, True], ids=["alike", "heavy zeros"])
@pytest.mark.parametrize("exponent", [-9, -20, -30, -60])
@pytest.mark.parametrize("lens,news,H,D", [([300, 47], [20, 7], 8, 128), ([3000], [64], 16, 64), ([3000, 90], [3, 90], 4, 128)])
def test_zero_scales_beside_small_ones(lens, news, H, D, exponent, heavy):
    """Every third page's V has scale 0, the others 2^exponent or half of it."""
    case = with_v_scales(lens, news, H, D, lambda j: 0.0 if j % 3 == 1 else 2.0 ** (exponent - j % 2), heavy)
    assert heavy or case.ref.abs().max() > 2.0 ** (exponent - 4)
    case.cuda().check(f"2^{exponent}")


@pytest.mark.parametrize("lens,news,H", [([300], [20], 8), ([5000], [64], 8), ([5000], [3], 4)])
def test_nothing_but_zero_scales(lens, news, H):
    """Zero rows, whatever is joined."""
    case = with_v_scales(lens, news, H, 128, lambda j: 0.0)
    case.q *= 40.0  # (scores far from zero)
    case.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert (case.call(err_flag=err) == 0).all() and int(err.item()) == 0


def test_zero_scales_first():
    """A sequence whose first tiles have scales of zero alone, the later ones not, over several CTAs."""
    case = with_v_scales([6000, 700], [40, 5], 8, 128, lambda j: 0.0 if j < 30 else 2.0 ** -12)
    case.cuda().check()


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("exponent", [-96, 96])
@pytest.mark.parametrize("lens,news", [([300, 47], [20, 7]), ([3000], [64])])
def test_values_and_scales_far_from_one(lens, news, exponent, eight):
    """V of 2^96 and 2^-96 and their like (bf16 pages), or under scales of that size: kv_len times |V| below 2^110."""
    case = Case(lens, news, 8, 2, 128, "bf16", 32, eight, seed=7)
    if eight:
        case.vs *= 2.0 ** exponent
    else:
        case.v = (case.v.float() * 2.0 ** exponent).to(torch.bfloat16)
    case.ref *= 2.0 ** exponent
    case.slack *= 2.0 ** exponent
    case.cuda().check(f"2^{exponent}")

"""Infinities among the visible rows of the paged and window attention: what
they may spoil, and that they spoil nothing else."""
import pytest
import torch

import decode_attention_static_gb300 as da
import paged_reference as R
import test_paged_attention_gpu as T

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    da.load_library()


def inputs(dtype, lens, H, Hkv, D, seed):
    """q, and static caches whose rows past the lengths are NaN."""
    gen, dt, capacity = torch.Generator().manual_seed(seed), TYPES[dtype], max(lens) + 3
    q = R.randn((len(lens), H, D), dt, gen)
    k, v = (R.randn((len(lens), Hkv, capacity, D), dt, gen) for _ in range(2))
    for b, n in enumerate(lens):
        k[b, :, n:], v[b, :, n:] = R.NAN, R.NAN
    return q, k, v


def attend(q, k, v, lens, static):
    """The kernel over static caches, or over the same rows in pages of 16."""
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if static:
        return da.decode_attn_window_fwd(q.cuda(), k.cuda(), v.cuda(), n, k.shape[2]).cpu()
    B, Hkv, rows, D = k.shape
    pages = -(-rows // 16)
    pools = []
    for x in (k, v):
        x = torch.cat([x, torch.full((B, Hkv, pages * 16 - rows, D), R.NAN, dtype=x.dtype)], dim=2)
        pools.append(x.view(B, Hkv, pages, 16, D).transpose(1, 2).reshape(B * pages, Hkv, 16, D).contiguous().cuda())
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    return da.decode_attn_paged_fwd(q.cuda(), *pools, table, n).cpu()


def reference(q, k, v, lens):
    return [R.attend(q[b].double(), k[b, :, :n].double(), v[b, :, :n].double(), q.shape[2] ** -0.5)
            for b, n in enumerate(lens)]


CASES = pytest.mark.parametrize("static", [False, True], ids=["pages", "static"])
TYPE = pytest.mark.parametrize("dtype", ["f16", "bf16"])


@CASES
@TYPE
@pytest.mark.parametrize("lens,H,Hkv,D", [([40, 700], 8, 2, 128), ([1], 4, 1, 64), ([90] * 60, 16, 4, 64)])
def test_infinite_values(lens, H, Hkv, D, dtype, static):
    """An infinite element of V leaves that element of its heads' outputs without
    a finite value, and every other element as it was."""
    q, k, v = inputs(dtype, lens, H, Hkv, D, len(lens))
    want, G = reference(q, k, v, lens), H // Hkv
    for b, n in enumerate(lens):
        v[b, 0, n // 2, 5], v[b, Hkv - 1, n - 1, D - 1] = float("inf"), -float("inf")
    got = attend(q, k, v, lens, static)
    spoilt = torch.zeros(H, D, dtype=torch.bool)
    spoilt[:G, 5] = spoilt[H - G:, D - 1] = True
    for b, (ref, slack) in enumerate(want):
        assert not got[b][spoilt].isfinite().any()
        R.assert_rows(torch.where(spoilt, torch.zeros_like(got[b]), got[b]), torch.where(spoilt, 0.0, ref), slack, f"{b}")


@CASES
@TYPE
@pytest.mark.parametrize("lens", [[40, 300], [90] * 160])
def test_infinite_scores(lens, dtype, static):
    """An infinite element of K makes its row's score infinite, with the query's
    sign: such a head has no softmax at plus infinity, and one row less at
    minus infinity."""
    H, Hkv, D, row, at = 8, 2, 64, 17, 9
    q, k, v = inputs(dtype, lens, H, Hkv, D, 7)
    plain = reference(q, k, v, lens)
    k[:, 1, row, at] = float("inf")
    got = attend(q, k, v, lens, static)
    up = q[:, :, at] > 0
    assert up[:, 4:].any() and not up[:, 4:].all()
    rest = torch.arange(max(lens)) != row
    for b, n in enumerate(lens):
        assert got[b, 4:][up[b, 4:]].isnan().all()
        R.assert_rows(got[b, :4], plain[b][0][:4], plain[b][1][:4], "the other KV head")
        ref, slack = R.attend(q[b].double(), k[b, :, :n][:, rest[:n]].double(), v[b, :, :n][:, rest[:n]].double(), D ** -0.5)
        down = ~up[b, 4:]
        R.assert_rows(got[b, 4:][down], ref[4:][down], slack[4:][down], "a weight of zero")


@CASES
@TYPE
def test_no_row_has_a_weight(dtype, static):
    """Scores of minus infinity alone: NaN, as 0 / 0 is."""
    lens, H, Hkv, D = [3, 50, 700], 4, 1, 64
    q, k, v = inputs(dtype, lens, H, Hkv, D, 8)
    q[..., 0], k[:, :, :, 0] = q[..., 0].abs() + 1, -float("inf")
    assert attend(q, k, v, lens, static).isnan().all()


@CASES
@pytest.mark.parametrize("lens", [[700, 33], [90] * 160])
def test_large_values_do_not_overflow(lens, static):
    """Values of 2^106 over 700 rows, with scores that spread over 2^30: every sum
    stays in range, whatever the running reference is."""
    q, k, v = inputs("bf16", lens, 8, 2, 64, 9)
    q, v = (q.float() * 4).bfloat16(), (v.double() * 2.0 ** 106).bfloat16()
    assert v.nan_to_num().abs().max().double() * max(lens) < 2.0 ** 120
    want, got = reference(q, k, v, lens), attend(q, k, v, lens, static)
    for b, (ref, slack) in enumerate(want):
        R.assert_rows(got[b], ref, slack, f"{b}")


@pytest.mark.parametrize("lens", [[700, 33], [90] * 160])
def test_large_scales_do_not_overflow(lens):
    """The same with 8-bit pages whose V scales are 2^98 to 2^101."""
    case = T.Case(lens, 8, 2, 64, "bf16", 16, True, seed=10, spread=4.0)
    up = 2.0 ** 106
    case.vs = (case.vs.double() * up).float()
    case.ref, case.slack = case.ref * up, case.slack * up
    T.check(case, "large scales")

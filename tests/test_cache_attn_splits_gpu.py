"""Every way in which a paged attention call is divided over the device: teams
of one, two and four warps, the same number of CTAs for each group, and uneven
shares that cut groups anywhere; with one scan over the lengths and with
several; for both row sizes of 16-bit and 8-bit pages."""
import pytest
import torch

import cache_attn_split as S
import decode_attention_static_gb300 as da
import paged_reference as R
import test_paged_attention_gpu as T


def ragged(n, low, high, seed):
    lens = torch.randint(low, high + 1, (n,), generator=torch.Generator().manual_seed(seed)).tolist()
    lens[n // 2] = high
    return lens


# name: lengths, heads, KV heads, window, sinks, (way, scans; 0: differs with the row size)
CASES = {
    "8 ragged to 8191": (ragged(8, 1000, 8191, 1), 8, 2, 0, 0, ("shares", 1)),
    "8 ragged to 3000": (ragged(8, 300, 3000, 1), 16, 8, 0, 0, ("shares", 1)),
    "24 ragged to 1500": (ragged(24, 150, 1500, 2), 8, 8, 0, 0, ("shares", 1)),
    "one long of 400": ([20] * 399 + [10000], 4, 1, 0, 0, ("shares", 2)),
    "one long before idle ones": ([40] * 200 + [6000] + [0] * 200, 4, 2, 0, 0, ("shares", 2)),
    "one long, window": ([20] * 399 + [10000], 4, 1, 9000, 100, ("shares", 2)),
    "152 of 100": ([100] * 152, 8, 8, 0, 0, ("teams 1", 1)),
    "152 ragged to 200": (ragged(152, 0, 200, 3), 16, 8, 0, 0, ("teams 1", 1)),
    "304 of 60": ([60] * 304, 8, 4, 0, 0, ("teams 1", 0)),
    "152 ragged, window": (ragged(152, 0, 900, 3), 8, 8, 150, 20, ("teams 1", 1)),
    "76 of 150": ([150] * 76, 16, 8, 0, 0, ("teams 2", 1)),
    "60 ragged to 400": (ragged(60, 50, 400, 4), 8, 8, 0, 0, ("teams 2", 1)),
    "38 of 300": ([300] * 38, 16, 8, 0, 0, ("teams 4", 1)),
    "40 ragged to 300": (ragged(40, 100, 300, 5), 8, 8, 0, 0, ("teams", 1)),
    "8 of 2500": ([2500] * 8, 8, 8, 0, 0, ("even 2", 1)),
    "16 of 130": ([130] * 16, 8, 8, 0, 0, ("even 1", 1)),
}
SIZES = [(D, eight) for D in (64, 128) for eight in (False, True)]
EVERY = pytest.mark.parametrize("name", CASES)
SIZE = pytest.mark.parametrize("D,eight", SIZES, ids=[f"{'e4m3' if e else '16bit'}-{D}" for D, e in SIZES])


@EVERY
@SIZE
def test_the_cases_go_their_ways(name, D, eight):
    """By the rule, on a device of 152 multiprocessors."""
    lens, _, Hkv, window, sinks, (way, scans) = CASES[name]
    (kind, number), took = S.ways(lens, Hkv, D, eight, window, sinks)
    assert way in (kind, f"{kind} {number}") and scans in (0, took)


@pytest.mark.gpu
@EVERY
@SIZE
def test_ways(name, D, eight):
    """The result, every counter back at zero, and the same bits again."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lens, H, Hkv, window, sinks, _ = CASES[name]
    dtype = "bf16" if len(name) % 2 else "f16"
    case = T.Case(lens, H, Hkv, D, dtype, 16 if len(lens) > 99 else 32, eight, window, sinks, seed=D + len(lens))
    ws = da.alloc_paged_workspace(H, Hkv, D)
    first = T.check(case, name, workspace=ws).clone()
    assert not ws[:4096].any()
    assert torch.equal(R.bits(case.call(workspace=ws)), R.bits(first))


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("name", ["152 of 100", "76 of 150", "38 of 300", "24 ragged to 1500", "one long of 400"])
def test_ways_with_bad_lengths_and_pages(name, eight):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lens, H, Hkv, _, _, _ = CASES[name]
    case = T.Case(lens, H, Hkv, 64, "f16", 16, eight, seed=5).cuda()
    n = len(lens)
    bad = [n // 8, n // 2 - 1, n // 3, n - 2]
    case.kv_len[bad[0]], case.kv_len[bad[1]] = -1, 1 << 20
    case.table[bad[2], 0], case.table[bad[3], 1] = case.k.shape[0], -(1 << 31)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = case.call(err_flag=err)
    assert int(err.item()) == da.DA_DEVERR_KV_LEN | da.DA_DEVERR_PAGE
    assert out[torch.tensor(bad, device="cuda")].isnan().all()
    good = torch.tensor([b for b in range(n) if b not in bad])
    R.assert_rows(out[good.cuda()], case.ref[good], case.slack[good])

"""How many bits of a softmax weight reach the output of the paged and window
attention: rows of nearly equal weight and opposite values, whose difference
an output shows that is itself rounded to 8 or 11 bits."""
import pytest
import torch

import decode_attention_static_gb300 as da
import paged_reference as R

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
# What a weight w = 2^x may be off by, relative: the base-2 exponential 2^-22,
# and the two roundings of x, |x| < 2, times ln 2; two pieces of fp16 leave 2^-23,
# three of bf16 nothing.
WEIGHT = {"bf16": 2.0 ** -22 + 0.7 * 2 * 2.0 ** -24, "f16": 2.0 ** -22 + 0.7 * 2 * 2.0 ** -24 + 2.0 ** -23}


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    da.load_library()


@pytest.mark.parametrize("static", [False, True], ids=["pages", "static"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_weights_of_rows_that_cancel(dtype, D, static):
    """Three rows: one of weight 1 and value 0, two of weights w and w (1 + d),
    d < 2^-11, and values 1 and -1, so the output is about w d / (1 + 2 w). Every
    product is exact, and so are the scores: an error of the weights or of the
    sums (one step of 2^-23 for each of the three matrix instructions) is all
    that the output can show beside its own rounding."""
    dt, B, H = TYPES[dtype], 48, 8
    gen = torch.Generator().manual_seed(D)
    q, k, v = torch.zeros(B, H, D), torch.zeros(B, 1, 16, D), torch.zeros(B, 1, 16, D)
    q[..., 0] = 1.0
    q[..., D // 2 + 1] = 2.0 ** -10 * (1 + torch.arange(H) / 8)
    k[:, 0, 1:3, 0] = -(0.25 + torch.arange(B) / 64)[:, None]
    k[:, 0, 2, D // 2 + 1] = torch.randint(64, 128, (B,), generator=gen) / 512
    v[:, 0, 1], v[:, 0, 2] = 1.0, -1.0
    q, k, v = q.to(dt), k.to(dt), v.to(dt)
    x = torch.einsum("bhd,bnd->bhn", q.double(), k[:, 0, :3].double())
    p = torch.softmax(x, -1)
    ref = torch.einsum("bhn,bnd->bhd", p, v[:, 0, :3].double())
    assert ref.abs().max() < 2.0 ** -12
    slack = ((p[..., 1] + p[..., 2]) * WEIGHT[dtype] + 3 * 2.0 ** -23 * p[..., 1])[..., None].expand(B, H, D)
    n = torch.full((B,), 3, dtype=torch.int32, device="cuda")
    if static:
        out = da.decode_attn_window_fwd(q.cuda(), k.cuda(), v.cuda(), n, 3, scale=1.0)
    else:
        table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
        out = da.decode_attn_paged_fwd(q.cuda(), k.cuda(), v.cuda(), table, n, scale=1.0)
    R.assert_rows(out, ref, slack, "rows that cancel")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_long_sums_that_cancel(dtype):
    """8192 rows in 512 tiles, the second half with the first one's keys (and so
    its weights, bit for bit) and the opposite values: the output is 0, and every
    error of the running sum stays in it. Rounded to nearest, the sum after k
    tiles errs by up to half a step of 2^-23 of what it holds, in either
    direction: independent errors, whose total stays within six standard
    deviations (truncated ones would all point towards zero and add up). Within a
    tile a sum may be truncated, by a step of it for each of its three matrix
    instructions. Every sequence reads the same pages, so that one warp goes
    through many tiles."""
    dt, B, Hkv, G, D, page, n = TYPES[dtype], 152, 8, 2, 128, 64, 8192
    gen = torch.Generator().manual_seed(1)
    a = (torch.randint(-128, 129, (Hkv, n // 2), generator=gen) / 256)
    order = torch.randperm(n // 2, generator=gen)
    key = torch.cat([a, a[:, order]], dim=1)  # [Hkv, n]
    k, v = (torch.zeros(n // page, Hkv, page, D) for _ in range(2))
    k[..., 3] = key.view(Hkv, n // page, page).transpose(0, 1)
    v[:n // page // 2], v[n // page // 2:] = 1.0, -1.0
    q = torch.zeros(B, Hkv * G, D)
    q[..., 3] = 1 + torch.arange(B * Hkv * G).view(B, -1) % 64 / 64
    table = torch.arange(n // page, dtype=torch.int32).repeat(B, 1)
    lens = torch.full((B,), n, dtype=torch.int32)
    out = da.decode_attn_paged_fwd(*(t.cuda() for t in (q.to(dt), k.to(dt), v.to(dt), table, lens)), scale=1.0)
    amplitude = q[..., 3].view(B, Hkv, G, 1).double()
    p = torch.softmax(amplitude * key.double()[None, :, None], -1).flatten(1, 2)  # [B, H, n]
    running = (p * v[:, 0, :, 0].reshape(-1).double()).view(B, Hkv * G, n // 16, 16).sum(-1).cumsum(-1)
    assert running[..., -1].abs().max() < 1e-12
    slack = 6 * (2.0 ** -46 * running.square() / 12).sum(-1).sqrt() + 3 * 2.0 ** -23
    slack = slack[..., None].expand(-1, -1, D)
    R.assert_rows(out, torch.zeros(B, Hkv * G, D).double(), slack, "sums that cancel")


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [2, 6, 40])
def test_rows_beside_a_sink_without_a_value(rows, dtype, eight):
    """One row takes nearly all of the weight, and its value is 0: the output is
    what the others have, of weights around 2^-24. A score below 2^5 errs by half
    a step of 2^-19 and by log2 e, which 32 bits hold to 2^-26, the base-2
    exponential by 2^-22; 16-bit pieces leave 2^-38 of the largest weight."""
    dt, B, H, D = TYPES[dtype], 24, 8, 64
    q, k, v = torch.zeros(B, H, D), torch.zeros(B, 1, 48, D), torch.zeros(B, 1, 48, D)
    q[..., 2] = (1 + torch.arange(B * H) / 512).view(B, H).to(dt).float()
    key = -torch.tensor([15.0, 16.0])[torch.randint(0, 2, (B, rows - 1), generator=torch.Generator().manual_seed(rows))]
    k[:, 0, 1:rows, 2], v[:, 0, 1:rows] = key, 1.0
    x = q[..., 2, None].double() * k[:, :, :rows, 2].double()
    p = torch.softmax(x, -1)
    ref = p[..., 1:].sum(-1, keepdim=True).expand(B, H, D)
    weight = 2.0 ** -22 + 0.7 * (2.0 ** -20 + 32 * 2.0 ** -26)
    slack = ref * (weight + (rows / 16 + 4) * 2.0 ** -23) + (rows - 1) * 2.0 ** -38
    store = R.E4M3 if eight else dt
    pools = [t.view(B, 1, 3, 16, D).transpose(1, 2).reshape(B * 3, 1, 16, D).contiguous().to(store).cuda() for t in (k, v)]
    assert torch.equal(pools[0].float().cpu().view(B, 48, D), k[:, 0])
    if eight:
        pools += [torch.ones(B * 3, 1, device="cuda") for _ in range(2)]
    table = torch.arange(B * 3, dtype=torch.int32, device="cuda").view(B, 3)
    n = torch.full((B,), rows, dtype=torch.int32, device="cuda")
    attend = da.decode_attn_paged_q8_fwd if eight else da.decode_attn_paged_fwd
    R.assert_rows(attend(q.to(dt).cuda(), *pools, table, n, scale=1.0), ref, slack, f"{rows} rows")

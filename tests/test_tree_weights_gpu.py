"""How many bits of a softmax weight reach the output of the tree attention."""
import pytest
import torch

import decode_attention_static_gb300 as da
import draft_reference as Q
import paged_reference as R

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
FORMS = pytest.mark.parametrize("dtype,eight", [("f16", False), ("bf16", False), ("f16", True), ("bf16", True)],
                                ids=["f16", "bf16", "f16-e4m3", "bf16-e4m3"])


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    da.load_library()


def attend(q, k, v, news, masks, eight, scale, page=16):
    """q [B * news, H, D], k and v [B, n, Hkv, D] (n a multiple of the page): every sequence's last `news` rows are its
    tokens'. 8 bits: keys and values are stored over a scale of 2^-4."""
    B, n, Hkv, D = k.shape
    store = R.E4M3 if eight else q.dtype
    pools = [(x * (16 if eight else 1)).view(B * n // page, page, Hkv, D).transpose(1, 2).contiguous().to(store) for x in (k, v)]
    back = [p.float().transpose(1, 2).reshape(B, n, Hkv, D) / (16 if eight else 1) for p in pools]
    assert torch.equal(back[0], k.float()) and torch.equal(back[1], v.float())
    args = [x.cuda() for x in pools]
    if eight:
        args += [torch.full(pools[0].shape[:2], 2.0 ** -4, device="cuda") for _ in range(2)]
    table = torch.arange(B * n // page, dtype=torch.int32, device="cuda").view(B, -1)
    start = torch.arange(B + 1, dtype=torch.int32, device="cuda") * news
    call = da.decode_attn_tree_q8_fwd if eight else da.decode_attn_tree_fwd
    return call(q.cuda(), *args, table, torch.full((B,), n, dtype=torch.int32, device="cuda"), token_start=start,
                tree_mask=Q.words_of(masks, 4).cuda(), scale=scale).cpu()


def values(shape, dtype, eight, gen):
    """Values that a page and the output hold exactly."""
    x = torch.randn(shape, generator=gen)
    return (x * 16).to(R.E4M3).float() / 16 if eight else x.to(TYPES[dtype]).float()


@FORMS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("m,G", [(256, 8), (64, 4), (32, 4), (16, 4), (16, 1)])
def test_the_only_row_seen(m, G, D, dtype, eight):
    """Tokens without a prefix that see one row each: a weight over itself is 1, so the output is the row's value, bit
    for bit (units of two query tiles, of one, and of rows that stand two and four times in it)."""
    gen = torch.Generator().manual_seed(m + G)
    B, Hkv = 3, 2
    k, v = values((B, m, Hkv, D), dtype, eight, gen), values((B, m, Hkv, D), dtype, eight, gen)
    q = R.randn((B * m, Hkv * G, D), TYPES[dtype], gen)
    row = torch.stack([torch.randperm(m, generator=gen) for _ in range(B)])
    out = attend(q, k, v, m, [1 << int(j) for j in row.flatten()], eight, D ** -0.5)
    want = torch.stack([v[b, row[b]] for b in range(B)]).view(B * m, Hkv, D).repeat_interleave(G, 1).to(TYPES[dtype])
    assert torch.equal(out, want)


@FORMS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,m,H", [(48, 16, 8), (2048, 32, 16), (2048, 3, 8)])
def test_a_sink_takes_all_weight(n, m, H, D, dtype, eight):
    """The first row's score lies 90 and more (2^129) above the others': the output is its value, bit for bit."""
    gen = torch.Generator().manual_seed(n + m)
    k, v = values((1, n, 2, D), dtype, eight, gen), values((1, n, 2, D), dtype, eight, gen)
    q = torch.zeros(m, H, D)
    q[..., 3] = 1 + (torch.arange(m * H) % 96 / 128).view(m, H)  # (7 bits behind the point)
    k[..., 3] = 0.0
    k[:, 0, :, 3] = 13.0
    chain = [(2 << i) - 1 for i in range(m)]
    out = attend(q.to(TYPES[dtype]), k, v, m, chain, eight, 7.3)
    assert torch.equal(out, v[0, 0].repeat_interleave(H // 2, 0).to(out.dtype).expand(m, H, D))


@pytest.mark.parametrize("m", [1, 2, 8, 16])
def test_two_pieces_of_rows_that_cancel(m):
    """bf16, head_dim 128, at most 128 query rows of a KV head: weights of 16 bits. Three rows: one of weight 1 and value
    0, two of weights w and w (1 + d), d < 2^-11, and values 1 and -1, so the output is about w d / (1 + 2 w). Every
    product is exact, and so are the scores. A weight may be off by 2^-17 (the second piece is half a step of 2^-8 of
    what the first one leaves, 2^-9 of its power of two), by the base-2 exponential 2^-22 and by the two roundings of
    its argument, below 2; the sums by a step of 2^-23 for each product and for the joins of groups and copies."""
    B, H, D, n = 48, 8, 128, 32
    gen = torch.Generator().manual_seed(m)
    q, k, v = torch.zeros(B, m, H, D), torch.zeros(B, n, 1, D), torch.zeros(B, n, 1, D)
    base = n - m
    q[..., 0] = 1.0
    q[..., D // 2 + 1] = 2.0 ** -10 * (1 + torch.arange(H) / 8)
    q[..., 5] = 8.0
    k[:, :, 0, 5] = -64.0  # (rows of the prefix that take no weight)
    k[:, :3, 0, 5] = 0.0
    k[:, 1:3, 0, 0] = -(0.25 + torch.arange(B) / 64)[:, None]
    k[:, 2, 0, D // 2 + 1] = torch.randint(64, 128, (B,), generator=gen) / 512
    v[:, 1], v[:, 2] = 1.0, -1.0
    dt = torch.bfloat16
    q, k, v = q.to(dt), k.to(dt).float(), v.to(dt).float()
    x = torch.einsum("bmhd,bnd->bmhn", q.double(), k[:, :base, 0].double())
    p = torch.softmax(x, -1)
    ref = torch.einsum("bmhn,bnd->bmhd", p, v[:, :base, 0].double()).view(B * m, H, D)
    assert 2.0 ** -16 < ref.abs().max() < 2.0 ** -12
    weight = 2.0 ** -17 + 2.0 ** -22 + 0.7 * 2 * 2.0 ** -24
    slack = ((p[..., 1] + p[..., 2]) * weight + 8 * 2.0 ** -23 * p[..., 1]).view(B * m, H, 1).expand(-1, -1, D)
    out = attend(q.view(B * m, H, D), k, v, m, [0] * (B * m), False, 1.0)
    R.assert_rows(out, ref, slack, "rows that cancel")


@pytest.mark.parametrize("exponent", [8, 15, 24, 31])
@pytest.mark.parametrize("m,H", [(1, 2), (16, 16)])
def test_small_elements_of_a_bf16_query(m, H, exponent):
    """bf16 queries over 8-bit pages: elements 2^-31 times the largest one still count with all of their bits. The largest
    element meets keys of zero in the two rows that take the weight, and their scores, around 1, come from the smallest
    element alone, under a scale that lifts it. Products and scores are exact; a weight is off by 2^-11 and the base-2 exponential."""
    B, D, n = 4, 64, 32
    gen = torch.Generator().manual_seed(m + exponent)
    small = (1 + torch.randint(0, 128, (B * m, H), generator=gen) / 128) * 2.0 ** -exponent
    q = torch.zeros(B * m, H, D)
    q[..., 0], q[..., 9] = 1.0, small
    k, v = torch.zeros(B, n, 2, D), values((B, n, 2, D), "bf16", True, gen)
    k[..., 0] = -1.0
    k[:, :2, :, 0] = 0.0
    k[:, 0, :, 9], k[:, 1, :, 9] = 0.5, -0.75
    out = attend(q.to(torch.bfloat16), k, v, m, [0] * (B * m), True, 2.0 ** exponent)
    score = small.double() * 2.0 ** exponent
    x = torch.stack([0.5 * score, -0.75 * score], dim=-1)  # [B m, H, 2]
    p = torch.softmax(x, -1)
    vv = v[:, :2].double().permute(0, 2, 1, 3).repeat_interleave(m, 0).repeat_interleave(H // 2, 1)  # [B m, H, 2, D]
    ref = torch.einsum("thr,thrd->thd", p, vv)
    mass = torch.einsum("thr,thrd->thd", p, vv.abs())
    R.assert_rows(out, ref, (2.0 ** -11 + 2.0 ** -19) * mass, f"2^-{exponent}")


@FORMS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("m,G", [(2, 4), (16, 8), (64, 4)])
def test_scores_that_rise_from_far_below(m, G, D, dtype, eight):
    """The first 256 rows' scores are -2^28 and less, the others' 80 and less: the sum is of the others, whatever the first
    rows' reference was. Their two largest scores are alike and lie 8 above the next ones, all exact before the factor
    log2 e: a weight is off by its rounding, 2^-8 or 2^-11, and by 2^-22 of a score and 2^-20; the first rows' weights
    are zero."""
    B, n = 160, 512  # (more units than CTAs: a CTA goes through whole ones)
    gen = torch.Generator().manual_seed(m)
    k, v = torch.zeros(B, n, 1, D), values((B, n, 1, D), dtype, eight, gen)
    k[:, :256, 0, 0] = -2.0
    step = torch.randint(0, 9, (B, 256), generator=gen)
    step[:, 100], step[:, 200] = 10, 10
    k[:, 256:, 0, 1] = step.float()
    k[:, n - m:, 0, 1] = 0.0  # (drafts, which nobody sees)
    q = torch.zeros(B * m, G, D)
    q[..., 0], q[..., 1] = 1.0, 2.0 ** -24
    out = attend(q.to(TYPES[dtype]), k, v, m, [0] * (B * m), eight, 2.0 ** 27)
    x = 8.0 * k[:, 256:n - m, 0, 1].double()
    p = torch.softmax(x, -1)
    vv = v[:, 256:n - m, 0].double()
    ref = torch.einsum("bn,bnd->bd", p, vv)[:, None, None].expand(B, m, G, D).reshape(B * m, G, D)
    mass = torch.einsum("bn,bnd->bd", p, vv.abs())[:, None, None].expand(B, m, G, D).reshape(B * m, G, D)
    weight = 2.0 ** -8 if dtype == "bf16" and not eight else 2.0 ** -11
    R.assert_rows(out, ref, (weight + 2.1 * (2.0 ** -22 * 80 * 2 + 2.0 ** -20) + 256 * 2.0 ** -23) * mass, "rising scores")


@FORMS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("m,G", [(3, 4), (16, 8), (64, 4)])
def test_the_largest_scores(m, G, D, dtype, eight):
    """Scores up to 2^21.9: the row of the largest one has all of the weight, 1 but for the rounding of a weight (half a
    step) and of its sum. Looked at are tokens' heads whose largest score is ahead of the others by more than what
    the sum of D products and the roundings of the score leave open, and 20."""
    B, n = 2, 640
    gen = torch.Generator().manual_seed(m + D)
    k, v = values((B, n, 1, D), dtype, eight, gen), values((B, n, 1, D), dtype, eight, gen)
    q = R.randn((B * m, G, D), TYPES[dtype], gen)
    qk = torch.einsum("bmgd,bnd->bmgn", q.double().view(B, m, G, D), k[:, :n - m, 0].double())
    size = torch.einsum("bmgd,bnd->bmgn", q.double().abs().view(B, m, G, D), k[:, :n - m, 0].double().abs()).amax(-1)
    scale = 2.0 ** 21.9 / qk.abs().max().item()
    out = attend(q, k, v, m, [0] * (B * m), eight, scale)
    two = (qk * scale).topk(2, dim=-1)
    ahead = two.values[..., 0] - two.values[..., 1]
    sure = ahead > 2 * scale * ((D + 8) * 2.0 ** -23 * size) + 2 * 2.0 ** -22 * 2.0 ** 22 + 20
    assert sure.double().mean() > 0.5
    top = two.indices[..., 0]
    ref = torch.stack([v[b, :, 0].double()[top[b]] for b in range(B)])  # [B, m, G, D]
    weight = 2.0 ** -8 if dtype == "bf16" and not eight else 2.0 ** -11
    got = out.view(B, m, G, D)
    assert torch.isfinite(got).all()
    R.assert_rows(got[sure], ref[sure], (weight + 2.0 ** -20) * ref[sure].abs(), "largest scores")

"""Decode attention over paged caches (16-bit and 8-bit pages) and under a
sliding window with sinks, against the plain 64-bit form: head layouts, page
sizes and lengths where a tile, a page, a window or a split can go wrong;
nothing outside the visible rows is read (it is NaN there, and unmapped table
entries are invalid page ids)."""
import pytest
import torch

import decode_attention_static_gb300 as da
import paged_reference as R

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    da.load_library()


class Case:
    """Inputs on the CPU: a query, a pool (rows that are not visible NaN) and
    what the operator gives for it."""

    def __init__(self, lens, H, Hkv, D, dtype, page, eight=False, window=0, sinks=0, seed=0, scale=None, max_pages=None,
                 spread=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.window, self.sinks, self.eight = lens, window, sinks, eight
        dt = TYPES[dtype]
        self.scale = D ** -0.5 if scale is None else scale
        self.q = R.randn((len(lens), H, D), dt, gen, spread)
        self.table, pool = R.deal_pages(lens, page, gen)
        if max_pages:
            wide = torch.full((len(lens), max_pages), 1 << 30, dtype=torch.int32)
            wide[:, :self.table.shape[1]] = self.table
            self.table = wide
        self.kv_len = torch.tensor(lens, dtype=torch.int32)
        store = R.E4M3 if eight else dt
        self.k = torch.full((pool, Hkv, page, D), R.NAN).to(store)
        self.v = torch.full((pool, Hkv, page, D), R.NAN).to(store)
        self.ks = torch.full((pool, Hkv), R.NAN)
        self.vs = torch.full((pool, Hkv), R.NAN)
        self.ref, self.slack = torch.zeros(len(lens), H, D).double(), torch.zeros(len(lens), H, D).double()
        for b, n in enumerate(lens):
            rows = R.visible_rows(n, window, sinks)
            if len(rows) == 0:
                continue
            pages = self.table[b].long()[rows // page]
            k, v = torch.randn(len(rows), Hkv, D, generator=gen), torch.randn(len(rows), Hkv, D, generator=gen)
            if eight:
                k, v = (k * 60).clamp(-448, 448).to(store), (v * 60).clamp(-448, 448).to(store)
                for s in (self.ks, self.vs):
                    s[pages.unique()] = torch.exp2(torch.randint(-9, -4, (len(pages.unique()), Hkv), generator=gen).float())
            else:
                k, v = k.to(store), v.to(store)
            R.bits(self.k)  # (contiguous storage)
            self.k.view(torch.uint8 if eight else torch.int16)[pages, :, rows % page] = k.view(
                torch.uint8 if eight else torch.int16)
            self.v.view(torch.uint8 if eight else torch.int16)[pages, :, rows % page] = v.view(
                torch.uint8 if eight else torch.int16)
            kd, vd = k.double(), v.double()
            if eight:
                kd, vd = kd * self.ks[pages].double()[..., None], vd * self.vs[pages].double()[..., None]
            self.ref[b], self.slack[b] = R.attend(self.q[b].double(), kd.transpose(0, 1), vd.transpose(0, 1), self.scale)

    def cuda(self):
        for name in ("q", "k", "v", "ks", "vs", "table", "kv_len"):
            setattr(self, name, getattr(self, name).cuda())
        return self

    def call(self, **kw):
        kw.setdefault("scale", self.scale)
        if self.eight:
            return da.decode_attn_paged_q8_fwd(self.q, self.k, self.v, self.ks, self.vs, self.table, self.kv_len,
                                               window=self.window, sinks=self.sinks, **kw)
        return da.decode_attn_paged_fwd(self.q, self.k, self.v, self.table, self.kv_len, window=self.window,
                                        sinks=self.sinks, **kw)


def check(case, what="", **kw):
    case.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = case.call(err_flag=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0, f"{what}: device error flag {int(err.item())}"
    R.assert_rows(out, case.ref, case.slack, what)
    for b, n in enumerate(case.lens):
        if n == 0:
            assert (out[b] == 0).all(), f"{what}: idle slot {b} is not zero"
    return out


def static_caches(case, capacity):
    """The same rows in the static layout [B, Hkv, capacity, D]."""
    B, (_, Hkv, page, D) = len(case.lens), case.k.shape
    caches = []
    for pool in (case.k, case.v):
        flat = torch.full((B, Hkv, capacity, D), R.NAN, dtype=pool.dtype, device=pool.device)
        for b, n in enumerate(case.lens):
            j = torch.arange(n, device=pool.device)
            if n:
                flat[b, :, :n] = pool[case.table[b].long()[j // page], :, j % page].transpose(0, 1)
        caches.append(flat)
    return caches


LENGTHS = [1, 2, 15, 16, 17, 31, 33, 64, 127, 129, 0, 300]


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,D", [(1, 1, 64), (2, 1, 128), (8, 2, 128), (16, 2, 64), (8, 1, 128), (6, 3, 64)])
def test_heads_and_lengths(H, Hkv, D, dtype, eight):
    check(Case(LENGTHS, H, Hkv, D, dtype, 16, eight, seed=H * D), f"{H}/{Hkv} heads, D {D}")


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(page, eight):
    lens = [page - 1, page, page + 1, 1, 3 * page + 5, 0, 1000]
    check(Case(lens, 8, 2, 128, "bf16", page, eight, seed=page, max_pages=90), f"page {page}")


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (16, 4), (17, 16), (64, 17), (100, 40), (128, 0),
                                          (300, 5), (5000, 2), (33, 1000), (250, 51)])
def test_window_and_sinks(window, sinks, eight):
    lens = [1, 5, 16, 17, 40, 64, 100, 129, 0, 300, 301, 999]
    check(Case(lens, 8, 2, 128 if window % 2 else 64, "f16", 16, eight, window, sinks, seed=window),
          f"window {window}, sinks {sinks}")


@pytest.mark.parametrize("dtype,H,Hkv,D", [("f16", 4, 4, 128), ("bf16", 16, 2, 128), ("bf16", 4, 1, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (37, 16), (200, 33), (4000, 4)])
def test_static_window(dtype, H, Hkv, D, window, sinks):
    lens = [1, 3, 16, 50, 129, 0, 300, 733]
    case = Case(lens, H, Hkv, D, dtype, 32, window=window, sinks=sinks, seed=window + H).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for capacity in (733, 1001):
        k, v = static_caches(case, capacity)
        out = da.decode_attn_window_fwd(case.q, k, v, case.kv_len, window, sinks=sinks, err_flag=err)
        R.assert_rows(out, case.ref, case.slack, f"window {window}, sinks {sinks}, capacity {capacity}")
        assert (out[5] == 0).all()
    assert int(err.item()) == 0


def test_a_window_over_everything_is_decode_attn_fwd():
    case = Case([300, 733, 64], 8, 2, 128, "bf16", 32, seed=4).cuda()
    k, v = static_caches(case, 733)
    out = da.decode_attn_window_fwd(case.q, k, v, case.kv_len, 733)
    R.assert_rows(out, case.ref, case.slack)
    R.assert_rows(da.decode_attn_fwd(case.q, k, v, case.kv_len), case.ref, case.slack)


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("lens,H,Hkv,page", [([20011], 8, 1, 64), ([4093], 16, 16, 16), ([9000, 1, 4097, 0, 33], 8, 4, 32),
                                             ([50] * 300, 4, 2, 16), ([1] * 700, 8, 8, 16)])
def test_splits_and_batches(lens, H, Hkv, page, eight):
    check(Case(lens, H, Hkv, 128, "bf16", page, eight, seed=len(lens)), f"{len(lens)} sequences")


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("lens,H,Hkv,D", [([70001], 8, 1, 128), ([40000], 2, 2, 64), ([30000, 5, 45000], 1, 1, 128)])
def test_groups_in_many_parts(lens, H, Hkv, D, eight):
    """Few heads with long prefixes: a group lies in up to every CTA's share and
    is joined in two rounds; twice, so that every counter is back at zero."""
    case = Case(lens, H, Hkv, D, "bf16", 64, eight, seed=len(lens))
    ws = da.alloc_paged_workspace(H, Hkv, D)
    first = check(case, f"{lens}", workspace=ws).clone()
    assert not ws[:4096].any()
    assert torch.equal(R.bits(case.call(workspace=ws)), R.bits(first))


def test_counters_left_over_are_reported():
    """A workspace that was never zero-filled: groups in parts become NaN and
    the call says so; zero-filled it serves again."""
    case = Case([5000, 30], 8, 1, 128, "f16", 16, seed=30).cuda()
    ws = torch.full((da.decode_attn_paged_workspace_size(8, 1, 128),), 1, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = case.call(workspace=ws, err_flag=err)
    assert int(err.item()) == da.DA_DEVERR_WORKSPACE and out[0].isnan().all()
    da.workspace_init(ws)
    check(case, "zero-filled again", workspace=ws)
    with pytest.raises(da.DecodeAttnError):
        case.call(workspace=ws[:-16])


def test_empty_batch():
    q = torch.empty(0, 8, 64, dtype=torch.float16, device="cuda")
    pool = [torch.zeros(2, 2, 16, 64, dtype=torch.float16, device="cuda") for _ in range(2)]
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    table = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    ws = da.alloc_paged_workspace(8, 2, 64)
    assert da.decode_attn_paged_fwd(q, *pool, table, none, workspace=ws).shape == q.shape
    da.kvcache_append_paged(*pool, q[:, :2].contiguous(), q[:, :2].contiguous(), table, none)
    cache = torch.empty(0, 2, 32, 64, dtype=torch.float16, device="cuda")
    assert da.decode_attn_window_fwd(q, cache, cache.clone(), none, 4, workspace=ws).shape == q.shape


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("longest", [15, 255, 256, 257, 511, 513])
def test_many_short_groups(longest, D, eight):
    """More groups than CTAs, around the length up to which one warp takes a
    whole group; with idle slots, a window, and lengths that make all warps but
    a few idle."""
    gen = torch.Generator().manual_seed(longest)
    for B, H, Hkv, window, sinks in ((70, 8, 4, 0, 0), (20, 16, 16, 9, 3), (200, 2, 1, 0, 0), (31, 40, 5, 0, 0)):
        lens = torch.randint(0, longest + 1, (B,), generator=gen).tolist()
        lens[B // 2] = longest
        check(Case(lens, H, Hkv, D, "bf16", 16, eight, window, sinks, seed=longest), f"{B} up to {longest}")


def test_short_groups_of_bad_lengths_and_pages():
    lens = [30, 17, 100, 5] * 50
    case = Case(lens, 8, 2, 64, "f16", 16, seed=31).cuda()
    kv, table = case.kv_len.clone(), case.table.clone()
    kv[7], kv[60], table[90, 1] = -3, 1 << 20, 1 << 25
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = da.decode_attn_paged_fwd(case.q, case.k, case.v, table, kv, err_flag=err)
    assert int(err.item()) == da.DA_DEVERR_KV_LEN | da.DA_DEVERR_PAGE
    bad = torch.tensor([7, 60, 90])
    assert out[bad.cuda()].isnan().all()
    good = torch.tensor([b for b in range(200) if b not in (7, 60, 90)])
    R.assert_rows(out[good.cuda()], case.ref[good], case.slack[good])


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("longest", [300, 385, 400, 401, 416, 417])
def test_many_groups_of_a_few_hundred_rows(longest, eight):
    """The same around the length up to which one CTA takes a whole group, for
    batches that one scan covers and for one that it does not, with lengths and
    pages that are refused."""
    gen = torch.Generator().manual_seed(longest)
    for B, H, Hkv, D, window, sinks in ((45, 8, 4, 128, 0, 0), (12, 16, 16, 64, 350, 3), (500, 4, 1, 64, 0, 0)):
        lens = torch.randint(0, longest + 1, (B,), generator=gen).tolist()
        lens[B // 2] = longest
        check(Case(lens, H, Hkv, D, "f16", 16, eight, window, sinks, seed=longest), f"{B} up to {longest}")
    lens = [longest, 17, longest // 2, 0] * 40
    case = Case(lens, 8, 2, 64, "f16", 16, eight, seed=31).cuda()
    case.kv_len[4], case.kv_len[61] = -3, 1 << 20
    case.table[90, 1], case.table[120, 0] = 1 << 25, -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = case.call(err_flag=err)
    assert int(err.item()) == da.DA_DEVERR_KV_LEN | da.DA_DEVERR_PAGE
    bad = torch.tensor([4, 61, 90, 120], device="cuda")
    assert out[bad].isnan().all()
    good = torch.tensor([b for b in range(160) if b not in (4, 61, 90, 120)])
    R.assert_rows(out[good.cuda()], case.ref[good], case.slack[good])


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
@pytest.mark.parametrize("H,Hkv,D", [(16, 8, 128), (4, 4, 64), (8, 1, 64), (24, 24, 128), (150, 75, 64)])
def test_groups_of_about_one_length(H, Hkv, D, eight):
    """Groups that get the same number of CTAs each: one, several, all; equal
    lengths, nearly equal ones, and one that is far shorter."""
    for lens in ([16], [64], [129], [300, 290], [511, 513, 512], [700], [1025, 1000, 1], [2600, 0, 2590]):
        check(Case(lens, H, Hkv, D, "bf16", 16, eight, seed=len(lens)), f"{lens}")
        check(Case(lens, H, Hkv, D, "f16", 32, eight, window=250, sinks=5, seed=2), f"{lens}, window")


def test_more_sequences_than_one_scan_covers():
    gen = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 40, (1500,), generator=gen).tolist()
    check(Case(lens, 2, 1, 64, "f16", 16, seed=6), "1500 sequences")
    check(Case(lens, 2, 1, 64, "f16", 16, True, window=9, sinks=2, seed=6), "1500 sequences, window")
    lens = [0] * 300 + [700] + [0] * 400 + [3, 0]
    check(Case(lens, 4, 4, 64, "f16", 16, seed=7), "mostly idle slots")
    check(Case(lens, 4, 4, 64, "bf16", 16, True, seed=7), "mostly idle slots")


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
def test_scores_that_grow_and_spread(eight):
    """Wide scores: the running maximum moves many times, and some weights
    vanish; also a negative and a zero scale."""
    for scale in (1.0, -0.5, 0.0):
        check(Case([700, 33], 8, 2, 64, "f16", 16, eight, scale=scale, seed=8, spread=3.0), f"scale {scale}")


def test_scales_of_far_apart_blocks():
    """V scales from 2^-60 to 2^60 and K scales that differ by page: no block is
    lost to another's range."""
    case = Case([200], 4, 1, 128, "bf16", 16, True, seed=9)
    pages = case.table[0, :13].long()
    old_k, old_v = case.ks.clone(), case.vs.clone()
    case.vs[pages] = torch.exp2(torch.arange(13.0) * 5 - 60)[:, None]
    case.ks[pages] = torch.exp2(-7 - torch.arange(13.0) % 3)[:, None]
    assert not torch.equal(old_k, case.ks) and not torch.equal(old_v, case.vs)
    j = torch.arange(200)
    p = case.table[0].long()[j // 16]
    bits = torch.uint8
    k = case.k.view(bits)[p, :, j % 16].view(R.E4M3).double() * case.ks[p].double()[..., None]
    v = case.v.view(bits)[p, :, j % 16].view(R.E4M3).double() * case.vs[p].double()[..., None]
    ref, slack = R.attend(case.q[0].double(), k.transpose(0, 1), v.transpose(0, 1), case.scale)
    case.ref[0], case.slack[0] = ref, slack
    check(case, "far apart scales")


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
def test_wide_and_tiny_queries(eight):
    """bf16 queries far outside what 16-bit floats hold; the scale brings the
    scores back."""
    for size in (2.0 ** 40, 2.0 ** -60):
        case = Case([100, 17], 8, 2, 64, "bf16", 16, eight, seed=10, spread=size, scale=0.125 / size)
        check(case, f"queries of size {size}")


def test_every_head_and_element_is_its_own():
    """One row: the output is that row of V, exactly, for each head."""
    for eight in (False, True):
        case = Case([1, 1], 16, 4, 64, "f16", 16, eight, seed=11)
        out = check(case, "one row")
        assert torch.equal(out.cpu().double(), case.ref.to(torch.float16).double())


def test_bad_lengths_and_pages_are_reported():
    case = Case([40, 50, 60, 0], 8, 2, 128, "bf16", 16, seed=12).cuda()
    rows = case.table.shape[1] * 16
    for bad in (-1, rows + 1, -(1 << 31), (1 << 31) - 1):
        kv = case.kv_len.clone()
        kv[1] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = da.decode_attn_paged_fwd(case.q, case.k, case.v, case.table, kv, err_flag=err)
        assert int(err.item()) == da.DA_DEVERR_KV_LEN
        assert out[1].isnan().all() and not out[[0, 2, 3]].isnan().any()
        R.assert_rows(out[[0, 2]], case.ref[[0, 2]], case.slack[[0, 2]])
        da.decode_attn_paged_fwd(case.q, case.k, case.v, case.table, kv)  # no flag to report in
    for bad in (-1, case.k.shape[0], 1 << 30, -(1 << 31)):
        table = case.table.clone()
        table[2, 3] = bad  # rows 48..59 of sequence 2
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = da.decode_attn_paged_fwd(case.q, case.k, case.v, table, case.kv_len, err_flag=err)
        assert int(err.item()) == da.DA_DEVERR_PAGE
        assert out[2].isnan().all()
        R.assert_rows(out[:2], case.ref[:2], case.slack[:2])
        # under a window that does not reach it the page is not looked at
        case2 = Case([40, 50, 48, 0], 8, 2, 128, "bf16", 16, seed=12).cuda()
        case2.table = torch.cat([case2.table, torch.full_like(case2.table[:, :1], bad)], dim=1).contiguous()
        check(case2, "unmapped page behind the last row")


def test_bad_static_lengths_are_reported():
    case = Case([40, 50], 8, 2, 128, "bf16", 16, seed=13).cuda()
    k, v = static_caches(case, 50)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = torch.tensor([51, 50], dtype=torch.int32, device="cuda")
    out = da.decode_attn_window_fwd(case.q, k, v, kv, 64, err_flag=err)
    assert int(err.item()) == da.DA_DEVERR_KV_LEN and out[0].isnan().all()
    R.assert_rows(out[1:], case.ref[1:], case.slack[1:])


def test_non_finite_rows_reach_only_their_head():
    """A NaN among the visible rows of one KV head spoils that head's queries
    and nothing else; so does an infinite score."""
    for eight in (False, True):
        case = Case([90, 90], 8, 2, 64, "bf16", 16, eight, seed=14).cuda()
        page = int(case.table[0, 2])
        bits = case.k.view(torch.uint8 if eight else torch.int16)
        bits[page, 1, 5, 7] = 0x7F if eight else 0x7FC0
        out = case.call()
        assert out[0, 4:].isnan().all()
        R.assert_rows(out[0, :4], case.ref[0, :4], case.slack[0, :4])
        R.assert_rows(out[1], case.ref[1], case.slack[1])


def test_workspace_serves_every_shape_in_turn():
    ws = da.alloc_paged_workspace(16, 2, 128)
    for seed, (lens, H, Hkv, D, page) in enumerate([([5000], 16, 2, 128, 16), ([3], 8, 1, 128, 64), ([900, 0, 77], 8, 8, 64, 32),
                                                    ([20000, 1], 16, 2, 128, 128)] * 2):
        check(Case(lens, H, Hkv, D, "f16", page, bool(seed % 2), seed=seed), f"call {seed}", workspace=ws)


def test_results_do_not_change_from_call_to_call():
    case = Case([9001, 350, 4000], 8, 2, 128, "bf16", 16, seed=15).cuda()
    ws = da.alloc_paged_workspace(8, 2, 128)
    first = case.call(workspace=ws).clone()
    for _ in range(20):
        assert torch.equal(R.bits(case.call(workspace=ws)), R.bits(first))


def test_graphs_share_a_workspace_and_follow_the_lengths():
    """Two captured graphs over one workspace, replayed in turn with lengths
    that change between replays, on a stream of their own."""
    a = Case([700, 1200, 33], 8, 2, 128, "bf16", 16, seed=16).cuda()
    b = Case([50, 2500], 16, 2, 128, "f16", 32, True, window=600, sinks=5, seed=17).cuda()
    ws = da.alloc_paged_workspace(16, 2, 128)
    stream = torch.cuda.Stream()
    outs, graphs = [torch.empty_like(a.q), torch.empty_like(b.q)], []
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for c, o in zip((a, b), outs):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                c.call(workspace=ws, out=o)
            graphs.append(g)
        full = a.kv_len.clone()
        for lens in ([700, 1200, 33], [0, 1, 16], [700, 1200, 33]):
            a.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
            for g in graphs:
                g.replay()
            stream.synchronize()
            R.assert_rows(outs[1], b.ref, b.slack)
            if lens[0]:
                R.assert_rows(outs[0], a.ref, a.slack)
            else:
                assert (outs[0][0] == 0).all() and not outs[0].isnan().any()
        assert torch.equal(full, a.kv_len)


def test_a_pool_past_four_gigabytes():
    """Pages whose byte offsets pass 2^32 (and element offsets 2^31)."""
    for eight in (False, True):
        D, Hkv, page = 128, 2, 64
        element = 1 if eight else 2
        pages = (9 << 29) // (Hkv * page * D * element) + 40
        case = Case([150, 90], 8, Hkv, D, "bf16", page, eight, seed=18)
        small = case.k.shape[0]
        far = torch.randperm(40, generator=torch.Generator().manual_seed(1))[:small] + pages - 40
        big = [torch.zeros((pages, Hkv, page, D), dtype=case.k.dtype, device="cuda") for _ in range(2)]
        bits = torch.uint8 if eight else torch.int16
        for dst, src in zip(big, (case.k, case.v)):
            dst.view(bits)[far.cuda()] = src.view(bits).cuda()
        scales = [torch.zeros((pages, Hkv), device="cuda") for _ in range(2)]
        for dst, src in zip(scales, (case.ks, case.vs)):
            dst[far.cuda()] = src.cuda()
        table = torch.where(case.table >= 0, far[case.table.long().clamp(min=0)].to(torch.int32), case.table)
        case.k, case.v, case.ks, case.vs, case.table = *big, *scales, table
        check(case, "far pages")
        del big, case
        torch.cuda.empty_cache()


def test_another_stream_sees_its_own_order():
    case = Case([800], 8, 2, 128, "bf16", 16, seed=19).cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        q = torch.zeros_like(case.q)
        torch.cuda._sleep(20_000_000)
        q.copy_(case.q)
        case.q = q
        out = case.call()
    stream.synchronize()
    R.assert_rows(out, case.ref, case.slack)

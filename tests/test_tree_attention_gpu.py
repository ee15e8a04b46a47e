"""Attention of several drafted tokens of each sequence over paged caches (16-bit
and 8-bit), against the plain 64-bit form: head layouts, page sizes, lengths,
numbers of tokens and masks where a tile, a page, a split or a mask word can go
wrong. Rows that nobody may see are NaN, unmapped table entries invalid page ids."""
import pytest
import torch

import decode_attention_static_gb300 as da
import draft_reference as Q
import paged_reference as R

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
BOTH = pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    da.load_library()


def step_of(dtype, eight):
    """Half a step of a weight: 8-bit pages are multiplied in fp16."""
    return 2.0 ** -8 if dtype == "bf16" and not eight else 2.0 ** -11


def tree_masks(m, gen, kind):
    """m masks: a chain, a tree's ancestors, or any bits (none at all among them)."""
    if kind == "chain":
        return None
    masks = []
    for i in range(m):
        if kind == "tree":
            parent = int(torch.randint(max(0, i - 5), i, (1,), generator=gen)) if i else None
            masks.append((masks[parent] if i else 0) | 1 << i)
        else:
            bits = torch.randint(0, 2, (256,), generator=gen).tolist()  # (bits past the m tokens do not matter)
            masks.append(0 if i % 5 == 4 else sum(b << j for j, b in enumerate(bits)))
    return masks


class Case:
    """lens: rows of each sequence, the drafted ones among them; news: drafted
    tokens. kind: chain, tree or any. lead, trail: packed tokens of nobody."""

    def __init__(self, lens, news, H, Hkv, D, dtype, page, eight=False, kind="tree", words=None, lead=0, trail=0, seed=0,
                 spread=1.0, scale=None):
        gen = torch.Generator().manual_seed(seed)
        dt, store = TYPES[dtype], R.E4M3 if eight else TYPES[dtype]
        self.dtype, self.eight, self.scale = dtype, eight, D ** -0.5 if scale is None else scale
        self.lens, self.news, self.lead = lens, news, lead
        T = lead + sum(news) + trail
        self.q = R.randn((T, H, D), dt, gen, spread)
        if lead:
            self.q[:lead] = R.NAN
        if trail:
            self.q[-trail:] = R.NAN
        self.table, pool = R.deal_pages(lens, page, gen)
        wide = torch.full((len(lens), self.table.shape[1] + 3), 1 << 30, dtype=torch.int32)
        wide[:, :self.table.shape[1]] = self.table
        for b, n in enumerate(lens):
            wide[b, -(-n // page):] = 1 << 30
        self.table = wide
        self.kv_len = torch.tensor(lens, dtype=torch.int32)
        self.start = torch.tensor([lead + sum(news[:b]) for b in range(len(news) + 1)], dtype=torch.int32)
        self.masks = [tree_masks(m, gen, kind) for m in news]
        words = words or max(1, -(-max(news + [1]) // 64))
        self.mask = None
        if kind != "chain":
            packed = [0] * lead + sum(self.masks, []) + [-1 & (1 << 64) - 1] * trail
            self.mask = Q.words_of([x & (1 << 64 * words) - 1 for x in packed], words)
        self.k = torch.full((pool, Hkv, page, D), R.NAN).to(store)
        self.v = torch.full((pool, Hkv, page, D), R.NAN).to(store)
        self.ks, self.vs = torch.full((pool, Hkv), R.NAN), torch.full((pool, Hkv), R.NAN)
        self.ref, self.slack = torch.zeros(T, H, D).double(), torch.zeros(T, H, D).double()
        self.owned = torch.zeros(T, dtype=torch.bool)
        bits = torch.uint8 if eight else torch.int16
        self.rows = []  # (K, V) of each sequence in 64 bits, [Hkv, n, D]
        for b, (n, m) in enumerate(zip(lens, news)):
            rows = torch.arange(n)
            pages = self.table[b].long()[rows // page]
            k, v = torch.randn(n, Hkv, D, generator=gen), torch.randn(n, Hkv, D, generator=gen)
            if eight:
                k, v = (k * 60).clamp(-448, 448).to(store), (v * 60).clamp(-448, 448).to(store)
                for s in (self.ks, self.vs):
                    s[pages.unique()] = torch.exp2(torch.randint(-9, -4, (len(pages.unique()), Hkv), generator=gen).float())
            else:
                k, v = k.to(store), v.to(store)
            self.k.view(bits)[pages, :, rows % page] = k.view(bits)
            self.v.view(bits)[pages, :, rows % page] = v.view(bits)
            kd, vd = k.double(), v.double()
            if eight:
                kd, vd = kd * self.ks[pages].double()[..., None], vd * self.vs[pages].double()[..., None]
            self.rows.append((kd.transpose(0, 1), vd.transpose(0, 1)))
            at = int(self.start[b])
            self.owned[at:at + m] = True
            if m and n >= m:
                seen = Q.seen_rows(n, m, self.masks[b])
                self.ref[at:at + m], self.slack[at:at + m] = Q.attend_seen(
                    self.q[at:at + m].double(), *self.rows[-1], seen, self.scale, step_of(dtype, eight))

    def cuda(self):
        for name in ("q", "k", "v", "ks", "vs", "table", "kv_len", "start", "mask"):
            t = getattr(self, name)
            setattr(self, name, None if t is None else t.cuda())
        return self

    def call(self, **kw):
        kw.setdefault("scale", self.scale)
        kw = dict(token_start=self.start, tree_mask=self.mask) | kw
        if self.eight:
            return da.decode_attn_tree_q8_fwd(self.q, self.k, self.v, self.ks, self.vs, self.table, self.kv_len, **kw)
        return da.decode_attn_tree_fwd(self.q, self.k, self.v, self.table, self.kv_len, **kw)

    def check(self, what="", flag=0, workspace=None):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(self.q, 7.0)
        got = self.call(out=out, err_flag=err, workspace=workspace)
        assert got is out and int(err.item()) == flag, f"{what}: error flag {int(err.item())}"
        R.assert_rows(out[self.owned], self.ref[self.owned], self.slack[self.owned], what)
        assert (out[~self.owned] == 7.0).all(), f"{what}: rows of nobody were written"
        return out


HEADS = [(4, 1, 64), (16, 8, 128), (5, 5, 128), (32, 4, 64), (8, 2, 128), (8, 1, 128), (3, 3, 64), (2, 1, 64)]


@BOTH
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,D", HEADS)
def test_heads_and_types(H, Hkv, D, dtype, eight):
    Case([300, 17, 129, 0, 64, 1000], [8, 3, 1, 0, 64, 33], H, Hkv, D, dtype, 16, eight, seed=H + D).cuda().check()


@BOTH
@pytest.mark.parametrize("kind", ["chain", "tree", "any"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages_and_masks(page, kind, eight):
    lens = [1, 2, 15, 16, 17, 31, 127, 128, 129, 255, 257, 500]
    news = [1, 2, 15, 1, 17, 30, 5, 128 if kind == "chain" else 64, 2, 7, 40, 60]
    news = [min(a, b) for a, b in zip(lens, news)]
    Case(lens, news, 8, 4, 128, "bf16", page, eight, kind, words=None if kind == "tree" else 4, seed=page).cuda().check()


@BOTH
@pytest.mark.parametrize("kind", ["chain", "tree", "any"])
@pytest.mark.parametrize("m", [1, 2, 16, 32, 63, 64, 65, 100, 128, 129, 200, 255, 256])
def test_numbers_of_tokens(m, kind, eight):
    for n, H, Hkv in ((m, 4, 1), (m + 1, 2, 2), (m + 130, 8, 1)):
        Case([n, n + 77], [m, max(1, m - 1)], H, Hkv, 64, "f16", 32, eight, kind, seed=m).cuda().check(f"{n} rows")


@BOTH
@pytest.mark.parametrize("B,n,m,H,Hkv", [(1, 9000, 7, 8, 2), (1, 20000, 64, 4, 1), (2, 6000, 20, 16, 4), (40, 700, 4, 4, 4),
                                         (3, 3000, 256, 8, 1), (200, 40, 3, 4, 2)])
def test_splits(B, n, m, H, Hkv, eight):
    """Long sequences over many CTAs, and many short ones."""
    lens = [n - 13 * b % (n - m) for b in range(B)]
    Case(lens, [max(1, m - b % 3) for b in range(B)], H, Hkv, 128, "bf16", 64, eight, seed=B + n).cuda().check()


@BOTH
def test_packed_rows_of_nobody(eight):
    """Tokens before the first sequence and behind the last one are left alone; a
    workspace that the program keeps."""
    ws = da.alloc_tree_workspace(8, 2, 128)
    for seed in range(3):
        Case([40, 0, 200, 33], [5, 0, 9, 33], 8, 2, 128, "f16", 16, eight, lead=3, trail=70, seed=seed).cuda().check(workspace=ws)


@BOTH
def test_one_token_each_without_bounds(eight):
    case = Case([40, 1, 200, 33, 700], [1] * 5, 8, 2, 128, "bf16", 16, eight, kind="chain").cuda()
    a = case.check()
    assert torch.equal(R.bits(case.call(token_start=None)), R.bits(a))


@BOTH
def test_tokens_of_nothing_see_nothing(eight):
    """Zero rows where a mask leaves a token without rows: no prefix, no bit."""
    case = Case([6, 5], [6, 5], 4, 1, 64, "bf16", 16, eight, kind="any", words=1).cuda()
    case.mask.zero_()
    out = case.call()
    assert (out == 0).all()
    case.mask[3] = 1 << 2
    out = case.call()
    assert (out[[0, 1, 2, 4, 5, 6]] == 0).all()
    want = case.rows[0][1][:, 2].repeat_interleave(4, 0)
    assert torch.equal(out[3].cpu(), want.to(out.dtype))


@BOTH
def test_large_scores(eight):
    """Scores of some thousands, and a scale below zero."""
    Case([400, 77], [9, 30], 8, 2, 128, "bf16", 32, eight, spread=100.0).cuda().check("wide")
    Case([400, 77], [9, 30], 8, 2, 128, "bf16", 32, eight, spread=3.0, scale=-0.2).cuda().check("negative scale")
    Case([400, 77], [9, 30], 8, 2, 128, "bf16", 32, eight, scale=0.0).cuda().check("no scale")


@BOTH
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_hidden_rows_do_not_reach_a_token(bad, eight):
    """NaN and infinities in drafted rows: tokens that do not see them give the
    same bits as without them, tokens that do give NaN or infinities as the plain form does."""
    case = Case([150, 40], [30, 40], 8, 2, 64, "f16", 16, eight, kind="tree").cuda()
    clean = case.check()
    hit = 120 + 11  # the 12th draft of the first sequence
    page, row = int(case.table[0, hit // 16]), hit % 16
    for pool in (case.v, case.k):
        keep = pool[page, 1, row].clone()
        pool[page, 1, row, 5] = bad
        out = case.call()
        pool[page, 1, row] = keep
        seen = torch.tensor([m >> 11 & 1 == 1 for m in case.masks[0]])
        assert seen.any() and not seen.all()
        own = out[:30].view(30, 2, 4, 64)
        assert torch.equal(R.bits(own[~seen]), R.bits(clean[:30].view(30, 2, 4, 64)[~seen]))
        assert torch.equal(R.bits(own[:, 0]), R.bits(clean[:30].view(30, 2, 4, 64)[:, 0]))
        assert torch.equal(R.bits(out[30:]), R.bits(clean[30:]))
        if pool is case.v:
            if eight or bad != bad:  # (8 bits have no infinities: they are NaN)
                assert own[seen][:, 1, :, 5].isnan().all()
            else:
                assert (own[seen][:, 1, :, 5] == bad).all()
            others = torch.arange(64) != 5
            assert torch.equal(R.bits(own[seen][:, 1][..., others]), R.bits(clean[:30].view(30, 2, 4, 64)[seen][:, 1][..., others]))
        elif eight or bad != bad:
            assert own[seen][:, 1].isnan().all()


@BOTH
def test_nan_in_the_prefix_reaches_its_sequence(eight):
    case = Case([150, 40], [30, 40], 8, 2, 64, "f16", 16, eight, kind="tree").cuda()
    clean = case.call()
    case.v[int(case.table[0, 2]), 1, 3, 5] = R.NAN
    out = case.call()
    a, b = out[:30].view(30, 2, 4, 64), clean[:30].view(30, 2, 4, 64)
    assert a[:, 1, :, 5].isnan().all() and torch.equal(R.bits(a[:, 0]), R.bits(b[:, 0]))
    assert torch.equal(R.bits(out[30:]), R.bits(clean[30:]))


def test_scales_of_any_kind():
    """Page scales far apart, zero, negative and no powers of two."""
    case = Case([300, 90], [20, 7], 8, 2, 128, "bf16", 16, True, kind="tree", seed=5)
    gen = torch.Generator().manual_seed(9)
    for b, n in enumerate(case.lens):
        rows = torch.arange(n)
        pages = case.table[b].long()[rows // 16]
        case.ks[pages] = (torch.rand(pages.shape[0], 2, generator=gen) * 0.02 - 0.005)
        case.vs[pages] = torch.exp2(torch.randint(-30, 20, (pages.shape[0], 2), generator=gen).float()) * 1.3
        case.vs[pages[20]] = 0.0
        case.vs[pages[40]] = -0.7
        case.ks[pages[60]] = 0.0
        ks, vs = case.ks[pages].double()[..., None], case.vs[pages].double()[..., None]
        k = case.k.view(torch.uint8)[pages, :, rows % 16].view(R.E4M3).double() * ks
        v = case.v.view(torch.uint8)[pages, :, rows % 16].view(R.E4M3).double() * vs
        at, m = int(case.start[b]), case.news[b]
        case.ref[at:at + m], case.slack[at:at + m] = Q.attend_seen(
            case.q[at:at + m].double(), k.transpose(0, 1), v.transpose(0, 1), Q.seen_rows(n, m, case.masks[b]),
            case.scale, 2.0 ** -11)
    case.cuda().check()


@BOTH
def test_refused_sequences(eight):
    """Lengths, token ranges and pages that only the device sees: NaN rows or
    skipped ones for that sequence alone, and the error bit."""
    def fresh():
        return Case([100, 60, 300, 20], [10, 5, 70, 3], 8, 2, 128, "bf16", 16, eight, kind="tree", words=2, seed=3).cuda()

    clean = fresh().check()

    def outcome(change, bit, nan=(), skipped=()):
        case = fresh()
        change(case)
        err, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full_like(case.q, 7.0)
        case.call(out=out, err_flag=err)
        assert int(err.item()) == bit
        bounds = [0, 10, 15, 85, 88]
        for b in range(4):
            rows, want = out[bounds[b]:bounds[b + 1]], clean[bounds[b]:bounds[b + 1]]
            if b in nan:
                assert rows.isnan().all(), b
            elif b in skipped:
                assert (rows == 7.0).all(), b
            else:
                assert torch.equal(R.bits(rows), R.bits(want)), b

    def length(b, n):
        def change(case):
            case.kv_len[b] = n
        return change

    def page(b, j, value):
        def change(case):
            case.table[b, j] = value
        return change

    def narrow(case):
        case.mask = case.mask[:, :1].contiguous()

    def bounds(*values):
        def change(case):
            case.start.copy_(torch.tensor(values, dtype=torch.int32))
        return change

    outcome(length(1, 4), da.DA_DEVERR_KV_LEN, nan=[1])
    outcome(length(2, -3), da.DA_DEVERR_KV_LEN, nan=[2])
    outcome(length(0, 1 << 30), da.DA_DEVERR_KV_LEN, nan=[0])
    outcome(page(2, 0, -1), da.DA_DEVERR_PAGE, nan=[2])
    outcome(page(0, 6, 1 << 30), da.DA_DEVERR_PAGE, nan=[0])
    outcome(page(3, 2, -7), 0)  # (behind the sequence's rows)
    outcome(narrow, da.DA_DEVERR_TOKENS, nan=[2])
    outcome(bounds(0, 10, 15, 85, 1000), da.DA_DEVERR_TOKENS, skipped=[3])
    outcome(bounds(-1, 10, 15, 85, 88), da.DA_DEVERR_TOKENS, skipped=[0])


@BOTH
def test_too_many_tokens(eight):
    case = Case([300, 50], [256, 20], 2, 1, 64, "f16", 16, eight, kind="chain").cuda()
    case.q = torch.cat([case.q, case.q[:1]])
    case.start = torch.tensor([0, 257, 277], dtype=torch.int32, device="cuda")
    case.kv_len[0] = 300
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = case.call(err_flag=err)
    assert int(err.item()) == da.DA_DEVERR_TOKENS and out[:257].isnan().all() and torch.isfinite(out[257:]).all()


@BOTH
def test_equal_calls_give_equal_bits(eight):
    case = Case([5000, 33, 2000], [60, 33, 5], 16, 4, 128, "bf16", 64, eight, seed=1).cuda()
    first = case.check()
    ws = da.alloc_tree_workspace(16, 4, 128)
    for _ in range(5):
        assert torch.equal(R.bits(case.call(workspace=ws)), R.bits(first))


@BOTH
def test_graph_replays_with_new_lengths(eight):
    """One captured call serves other lengths, masks and tables; two graphs on
    one workspace, replayed in turn, beside calls on another stream with their own."""
    a = Case([900, 40], [20, 9], 8, 2, 128, "bf16", 16, eight, seed=2).cuda()
    b = Case([50, 1200], [9, 20], 8, 2, 128, "bf16", 16, eight, seed=3).cuda()
    most = max(a.k.shape[0], b.k.shape[0]), max(a.table.shape[1], b.table.shape[1])
    names = ("q", "k", "v", "ks", "vs", "table", "kv_len", "start", "mask")
    live = Case.__new__(Case)
    live.eight, live.scale = eight, a.scale

    def grown(t, n):
        out = torch.zeros((n, *t.shape[1:]), dtype=t.dtype, device="cuda")
        out.view(torch.uint8)[:t.shape[0]] = t.contiguous().view(torch.uint8)
        return out

    def fill(case):
        for n in names:
            t = getattr(case, n)
            if n in ("k", "v", "ks", "vs"):
                t = grown(t, most[0])
            if n == "table":
                t = torch.nn.functional.pad(t, (0, most[1] - t.shape[1]), value=1 << 30)
            if hasattr(live, n):
                getattr(live, n).view(torch.uint8).copy_(t.contiguous().view(torch.uint8))
            else:
                setattr(live, n, t.clone())
    fill(a)
    ws = da.alloc_tree_workspace(8, 2, 128)
    out, out2 = torch.empty_like(live.q), torch.empty_like(live.q)
    graphs = []
    for o in (out, out2):
        live.call(out=o, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            live.call(out=o, workspace=ws)
        graphs.append(g)
    side, ws2 = torch.cuda.Stream(), da.alloc_tree_workspace(8, 2, 128)
    want = {id(c): c.call() for c in (a, b)}
    for case in (b, a, b):
        fill(case)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            other = a.call(workspace=ws2)
        for g, o in zip(graphs, (out, out2)):
            o.fill_(7.0)
            g.replay()
        torch.cuda.synchronize()
        for o in (out, out2):
            assert torch.equal(R.bits(o), R.bits(want[id(case)]))
        assert torch.equal(R.bits(other), R.bits(want[id(a)]))


@BOTH
@pytest.mark.parametrize("slot", [0, 1, 4])
def test_a_copy_that_never_comes(slot, eight):
    """One copy of one CTA is left out: its bounded waits run out, NaN rows and the error bit, nothing faults, and the
    next call is right."""
    case = Case([2000, 900], [20, 9], 8, 2, 128, "bf16", 64, eight, seed=4).cuda()
    ws = da.alloc_tree_workspace(8, 2, 128)
    clean = case.check(workspace=ws)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(case.q, 7.0)
    da.test_skip_slot(slot)
    try:
        case.call(out=out, err_flag=err, workspace=ws)
        torch.cuda.synchronize()
    finally:
        da.test_skip_slot(-1)
    bad = out.isnan().all(dim=-1)
    assert (R.bits(out) == R.bits(clean)).all(dim=-1)[~bad.cpu()].all()
    if bad.any():  # (a CTA of fewer copies never comes to a later one)
        assert int(err.item()) & da.DA_DEVERR_TIMEOUT and bad[:20, :4].all()
    else:
        assert slot > 1 and int(err.item()) == 0
    ws.zero_()
    assert torch.equal(R.bits(case.check(workspace=ws)), R.bits(clean))


@BOTH
def test_large_pools(eight):
    """Rows and pages whose offsets pass 32 bits: a pool of more than 2^32 elements, its last pages in use."""
    Hkv, D, page, n = 16, 128, 256, 700
    pages = (1 << 32) // (Hkv * D * page) + 5
    if torch.cuda.mem_get_info()[0] < 5 * pages * Hkv * D * page:
        pytest.skip("not enough free memory")
    small = Case([n], [7], 32, Hkv, D, "f16", page, eight, seed=8)
    dt = small.k.dtype
    big = [torch.zeros(pages, Hkv, page, D, dtype=torch.uint8 if eight else torch.int16, device="cuda") for _ in range(2)]
    scale = [torch.ones(pages, Hkv, device="cuda") for _ in range(2)]
    table = torch.arange(pages - 1, pages - 4, -1, dtype=torch.int32)[None]
    for i in range(3):
        src = int(small.table[0, i])
        for x, pool in zip((small.k, small.v), big):
            pool[pages - 1 - i] = x.view(pool.dtype)[src].cuda()
        for x, s in zip((small.ks, small.vs), scale):
            s[pages - 1 - i] = x[src].cuda()
    small.table, small.k, small.v = table, big[0].view(dt), big[1].view(dt)
    small.ks, small.vs = scale
    small.cuda().check()


def test_concurrent_calls_on_two_streams():
    """Calls with workspaces of their own side by side, longer than the time that a CTA waits for a unit's other parts."""
    cases = [Case([9000, 4000], [64, 40], 16, 4, 128, "bf16", 64, False, seed=s).cuda() for s in (1, 2)]
    want = [c.check() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [da.alloc_tree_workspace(16, 4, 128) for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(c.call(workspace=spaces[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert torch.equal(R.bits(g), R.bits(want[i]))

"""Appending to paged caches with the rotary embedding: bit for bit against
the plain form in the number formats the header states (fp32 products and sums
rounded apart, one rounding to the storage type; e4m3 codes and power-of-two
scales), and nothing but the appended rows is written. Then prompts and decode
steps through append and attention together."""
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


def tables(rows, D):
    angle = torch.arange(rows).double()[:, None] * 10000.0 ** (-torch.arange(0, D, 2).double() / D)
    angle = torch.cat([angle, angle], dim=1)
    return angle.cos().float(), angle.sin().float()


class Inputs:
    def __init__(self, counts, positions, H, Hkv, D, dtype, page, eight, rope=True, with_q=True, lead=0, trail=0, seed=0,
                 packed=True):
        gen = torch.Generator().manual_seed(seed)
        dt = TYPES[dtype]
        self.eight, self.page = eight, page
        tokens = lead + sum(counts) + trail
        reach = [p + n for p, n in zip(positions, counts)]
        self.table, pool = R.deal_pages([max(r, 1) for r in reach], page, gen)
        shape = (pool, Hkv, page, D)
        if eight:
            self.k, self.v = ((torch.randn(shape, generator=gen) * 100).clamp(-448, 448).to(R.E4M3) for _ in range(2))
            self.ks, self.vs = (torch.exp2(torch.randint(-9, -4, (pool, Hkv), generator=gen).float()) for _ in range(2))
        else:
            self.k, self.v = (R.randn(shape, dt, gen) for _ in range(2))
            self.ks = self.vs = None
        self.k_new, self.v_new = (R.randn((tokens, Hkv, D), dt, gen) for _ in range(2))
        self.q = R.randn((tokens, H, D), dt, gen) if with_q else None
        self.cos, self.sin = tables(max(reach + [1]), D) if rope else (None, None)
        self.position = torch.tensor(positions, dtype=torch.int32)
        start = [lead]
        for n in counts:
            start.append(start[-1] + n)
        self.start = torch.tensor(start, dtype=torch.int32) if packed else None

    def plain(self, **kw):
        """The plain form on copies: (k, v, k_scale, v_scale, q_out)."""
        c = [None if t is None else t.clone() for t in (self.k, self.v, self.ks, self.vs)]
        q = R.append(c[0], c[1], self.k_new, self.v_new, self.table, self.position, self.start, self.cos, self.sin,
                     self.q, c[2], c[3], **kw)
        return [*c, q]

    def call(self, q_out=None, err=None, dev=None):
        d = dev or self.cuda()
        kw = dict(token_start=d["start"], rope_cos=d["cos"], rope_sin=d["sin"], q=d["q"], q_out=q_out, err_flag=err)
        if self.eight:
            q = da.kvcache_append_paged_q8(d["k"], d["v"], d["ks"], d["vs"], d["k_new"], d["v_new"], d["table"],
                                           d["position"], **kw)
        else:
            q = da.kvcache_append_paged(d["k"], d["v"], d["k_new"], d["v_new"], d["table"], d["position"], **kw)
        return [d["k"], d["v"], d["ks"], d["vs"], q]

    def cuda(self):
        names = ("k", "v", "ks", "vs", "k_new", "v_new", "q", "cos", "sin", "position", "start", "table")
        return {n: None if getattr(self, n) is None else getattr(self, n).cuda() for n in names}


def same(got, want, what=""):
    for name, g, w in zip(("k_pages", "v_pages", "k_scale", "v_scale"), got, want):
        if w is not None:
            # (the sign of a stored NaN does not matter)
            gb, wb = R.bits(g), R.bits(w)
            if w.dtype == R.E4M3:
                gb, wb = (torch.where((x & 0x7F) == 0x7F, torch.full_like(x, 0x7F), x) for x in (gb, wb))
            assert torch.equal(gb, wb), f"{what}: {name} differs in {(gb != wb).sum().item()} places"


def check(inp, what="", flag=0, lead=0, trail=0, **kw):
    want = inp.plain(**kw)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = None if inp.q is None else torch.full_like(inp.q, 7.0, device="cuda")
    got = inp.call(q_out=q_out, err=err)
    assert int(err.item()) == flag, f"{what}: error flag {int(err.item())}"
    same(got, want, what)
    if inp.q is not None:
        assert got[4].data_ptr() == q_out.data_ptr()
        g, w = got[4].cpu(), want[4]
        assert torch.equal(g.isnan(), w.isnan()), what
        assert torch.equal(R.bits(g.nan_to_num()), R.bits(w.nan_to_num())), f"{what}: rotated q differs"
    return got


BOTH = pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])


@BOTH
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,D,page", [(4, 1, 64, 16), (16, 8, 128, 16), (5, 5, 128, 32), (32, 4, 64, 256)])
def test_one_token_each(H, Hkv, D, page, dtype, eight):
    positions = [0, 1, page - 1, page, page + 1, 3 * page, 37, 500]
    for packed in (False, True):
        check(Inputs([1] * 8, positions, H, Hkv, D, dtype, page, eight, seed=D + page, packed=packed), "one token each")


@BOTH
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_prompts(page, eight):
    counts = [1, page, 2 * page + 3, 0, page - 1, 5, 700]
    positions = [5, 0, page - 2, 9, 1, 2 * page - 1, 3]
    check(Inputs(counts, positions, 8, 2, 128, "bf16", page, eight, seed=page), f"page {page}")
    check(Inputs(counts, positions, 8, 2, 64, "f16", page, eight, rope=False, with_q=False, seed=page), "no rotation")
    check(Inputs(counts, positions, 8, 2, 64, "f16", page, eight, with_q=False, seed=page), "no query")


@BOTH
def test_padding_tokens_are_left_alone(eight):
    inp = Inputs([3, 0, 20], [4, 0, 60], 4, 2, 64, "bf16", 16, eight, lead=2, trail=5, seed=1)
    got = check(inp, "padding")  # q_out rows keep the 7.0 they held, in the plain form as well
    assert (got[4][:2] == 7).all() and (got[4][-5:] == 7).all()


@BOTH
def test_many_sequences(eight):
    gen = torch.Generator().manual_seed(3)
    counts = torch.randint(0, 5, (777,), generator=gen).tolist()
    positions = torch.randint(0, 100, (777,), generator=gen).tolist()
    check(Inputs(counts, positions, 2, 1, 64, "f16", 16, eight, seed=2), "777 sequences")


@BOTH
def test_nothing_to_append(eight):
    check(Inputs([0, 0], [4, 9], 4, 2, 64, "f16", 16, eight, lead=3, seed=3), "no rows")
    check(Inputs([0, 0], [4, 9], 4, 2, 64, "f16", 16, eight, seed=3), "no tokens")


@BOTH
def test_query_rotated_in_place(eight):
    inp = Inputs([9, 30], [2, 14], 8, 2, 128, "bf16", 16, eight, seed=4)
    want, d = inp.plain(), inp.cuda()
    got = inp.call(q_out=d["q"], dev=d)
    assert got[4].data_ptr() == d["q"].data_ptr()
    assert torch.equal(R.bits(got[4]), R.bits(want[4]))


@BOTH
def test_appending_again_changes_nothing(eight):
    inp = Inputs([1, 40], [21, 7], 8, 2, 128, "bf16", 32, eight, seed=5)
    d = inp.cuda()
    first = [None if t is None else t.clone() for t in inp.call(dev=d)]
    same(inp.call(dev=d), first[:4])
    same(first, inp.plain())


@BOTH
def test_bad_positions_are_skipped_whole(eight):
    counts, positions = [3, 4, 2, 1, 5], [2, 0, 0, 15, 40]
    for at, bad in ((1, -1), (1, -(1 << 31)), (2, 1 << 30), (2, (1 << 31) - 1), (4, 44)):
        inp = Inputs(counts, positions, 4, 2, 64, "f16", 16, eight, seed=6)
        inp.position[at] = bad  # (44 + 5 rows pass the 48 that the table maps, and the rope tables' 45)
        check(inp, f"position {bad}", flag=da.DA_DEVERR_POSITION, limit=45)


@BOTH
def test_bad_pages_are_skipped(eight):
    for bad in (-1, 1 << 30, -(1 << 31)):
        inp = Inputs([40, 3], [4, 30], 4, 2, 64, "bf16", 16, eight, seed=7)
        inp.table[0, 1] = bad
        check(inp, f"page {bad}", flag=da.DA_DEVERR_PAGE)
        inp.call()  # and without a flag


@BOTH
@pytest.mark.parametrize("page,Hkv,D,count", [(16, 24, 128, 150), (64, 9, 128, 300), (16, 17, 64, 200),
                                              (128, 6, 128, 500)])
def test_more_pages_and_heads_than_the_device_takes_at_once(page, Hkv, D, count, eight):
    """Every part of the device goes through several pages, over the ends of
    sequences, empty and refused ones, and pages outside the pool."""
    gen = torch.Generator().manual_seed(page + Hkv)
    counts = torch.randint(count // 2, count, (41,), generator=gen).tolist()
    positions = torch.randint(0, 3 * page, (41,), generator=gen).tolist()
    for b in (0, 7, 8, 40):
        counts[b] = 0
    inp = Inputs(counts, positions, Hkv, Hkv, D, "bf16", page, eight, with_q=False, seed=Hkv)
    check(inp, "long runs")
    inp.table[3, positions[3] // page] = -1
    inp.table[20, positions[20] // page + 1] = inp.k.shape[0]
    inp.position[11] = -1
    inp.position[39] = 1 << 30
    check(inp, "refused places", flag=da.DA_DEVERR_POSITION | da.DA_DEVERR_PAGE)


@BOTH
def test_rows_of_a_page_past_the_last_sequence(eight):
    """A token range that leaves the packed tokens is refused on the device."""
    inp = Inputs([3, 4], [2, 0], 4, 2, 64, "f16", 16, eight, seed=8)
    want = inp.plain()
    inp.start = torch.tensor([0, 3, 8], dtype=torch.int32)  # there are 7 tokens
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = inp.call(err=err)
    assert int(err.item()) == da.DA_DEVERR_POSITION
    rows = inp.table[0, 0]
    assert torch.equal(R.bits(got[0])[rows], R.bits(want[0])[rows])
    untouched = inp.table[1, 0]
    assert torch.equal(R.bits(got[0])[untouched], R.bits(inp.k)[untouched])


def test_far_positions_rotate_as_near_ones():
    """Angles come from the tables: position 100001 is as exact as position 1."""
    inp = Inputs([5], [100000], 2, 1, 64, "f16", 64, False, seed=9)
    check(inp, "far positions")


def values(name, shape, gen):
    x = torch.randn(shape, generator=gen)
    if name == "zeros":
        return x * 0
    if name == "tiny":  # bf16 values below 2^-120
        return x * 2.0 ** -124
    if name == "huge":
        return x.sign() * 3.0e38
    if name == "edge":  # on and around 448 times a power of two
        return torch.tensor([448.0, 450.0, 446.0, 224.0, 7.0, 0.875])[torch.randint(0, 6, shape, generator=gen)]
    if name == "halves":  # ties between e4m3 values
        return torch.randint(-64, 65, shape, generator=gen) * 0.125 + 0.0625
    x[torch.rand(shape, generator=gen) < 0.1] = float("nan")
    x[torch.rand(shape, generator=gen) < 0.1] = float("inf")
    x[torch.rand(shape, generator=gen) < 0.1] = -float("inf")
    return x if name == "some" else x * float("nan")


@pytest.mark.parametrize("name", ["zeros", "tiny", "huge", "edge", "halves", "some", "all"])
def test_scales_and_codes_of_odd_values(name):
    """Without rotation (its products are tested elsewhere): scales at their
    floor, at the type's end and at powers of two; NaN and infinities become
    NaN and do not count for the scale."""
    gen = torch.Generator().manual_seed(10)
    for counts, positions in (([1, 1, 1], [0, 5, 20]), ([50, 3, 16], [3, 30, 16])):
        inp = Inputs(counts, positions, 2, 2, 64, "bf16", 16, True, rope=False, with_q=False, seed=11)
        inp.k_new = values(name, inp.k_new.shape, gen).to(torch.bfloat16)
        inp.v_new = values(name, inp.v_new.shape, gen).to(torch.bfloat16)
        check(inp, name)


def test_growing_scales_move_the_older_rows():
    """Rows that double from step to step: every step that passes the scale
    rounds the page's older rows to the new one, down to nothing."""
    H, Hkv, D, page = 2, 2, 64, 16
    inp = Inputs([1], [0], H, Hkv, D, "bf16", page, True, rope=False, with_q=False, seed=12)
    d = inp.cuda()
    for step in range(page + 3):
        inp.position = torch.tensor([step % page if step < page else step - page], dtype=torch.int32)
        gen = torch.Generator().manual_seed(step)
        inp.k_new = (torch.randn(1, Hkv, D, generator=gen) * 2.0 ** step).bfloat16()
        inp.v_new = (torch.randn(1, Hkv, D, generator=gen) * 2.0 ** -step).bfloat16()
        want = inp.plain()
        d["position"], d["k_new"], d["v_new"] = (t.cuda() for t in (inp.position, inp.k_new, inp.v_new))
        got = inp.call(dev=d)
        same(got, want, f"step {step}")
        inp.k, inp.v, inp.ks, inp.vs = want[:4]
    # started anew at row 0 with V of size 2^-16: the scale of the earlier rows (2^-7 or more) is gone
    assert inp.vs[inp.table[0, 0]].max() < 2.0 ** -15


def test_a_pool_past_four_gigabytes():
    for eight in (False, True):
        Hkv, page, D = 2, 64, 128
        pages = (9 << 29) // (Hkv * page * D * (1 if eight else 2)) + 8
        inp = Inputs([70, 1], [60, 127], 4, Hkv, D, "bf16", page, eight, seed=13)
        want, small = inp.plain(), inp.k.shape[0]
        d = inp.cuda()
        bits = torch.uint8 if eight else torch.int16
        for n in ("k", "v"):
            big = torch.zeros((pages, Hkv, page, D), dtype=d[n].dtype, device="cuda")
            big.view(bits)[pages - small:] = d[n].view(bits)
            d[n] = big
        if eight:
            for n in ("ks", "vs"):
                d[n] = torch.cat([torch.zeros((pages - small, Hkv), device="cuda"), d[n]])
        d["table"] = torch.where(d["table"] >= 0, d["table"] + (pages - small), d["table"])
        got = inp.call(dev=d)
        same([None if g is None else g[pages - small:] for g in got[:4]], want, "far pages")
        assert not d["k"].view(bits)[:pages - small].any()
        del d, got
        torch.cuda.empty_cache()


def test_captured_append_follows_its_inputs():
    """A captured append and attention (a decode step), replayed with positions
    and values that change between replays."""
    for eight in (False, True):
        inp = Inputs([1, 1], [3, 40], 8, 2, 128, "bf16", 16, eight, seed=14, packed=False)
        inp.table = torch.cat([inp.table, inp.table.flip(0)], dim=1).contiguous()
        inp.table[:, 3:] = -1
        inp.cos, inp.sin = tables(64, 128)
        d = inp.cuda()
        q_out, out = torch.empty_like(d["q"]), torch.empty_like(d["q"])
        kv_len = d["position"] + 1
        ws = da.alloc_paged_workspace(8, 2, 128)
        torch.cuda.synchronize()
        before = [None if d[n] is None else d[n].clone() for n in ("k", "v", "ks", "vs")]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            inp.call(q_out=q_out, dev=d)
        same(before, [inp.k, inp.v, inp.ks, inp.vs])
        for step, positions in enumerate(([3, 40], [4, 41], [15, 2])):
            inp.position = torch.tensor(positions, dtype=torch.int32)
            gen = torch.Generator().manual_seed(step)
            inp.k_new = R.randn(inp.k_new.shape, torch.bfloat16, gen, 2.0 ** step)
            d["position"].copy_(inp.position)
            d["k_new"].copy_(inp.k_new)
            want = inp.plain()
            graph.replay()
            torch.cuda.synchronize()
            same([d["k"], d["v"], d["ks"], d["vs"]], want, f"replay {step}")
            assert torch.equal(R.bits(q_out), R.bits(want[4]))
            inp.k, inp.v, inp.ks, inp.vs = want[:4]
        del out, kv_len, ws


@BOTH
@pytest.mark.parametrize("dtype,H,Hkv,D,page,window,sinks", [("bf16", 8, 2, 128, 16, 0, 0), ("f16", 4, 4, 64, 32, 40, 4),
                                                            ("bf16", 16, 2, 128, 64, 100, 16)])
def test_prompt_then_decode(dtype, H, Hkv, D, page, window, sinks, eight):
    """A serving run: prompts of three requests, then 40 decode steps of append
    and attention. The pages stay what the plain append makes of them, and
    every step's output is the attention over the rows they hold."""
    gen = torch.Generator().manual_seed(20)
    dt, steps, prompts = TYPES[dtype], 40, [70, 1, 133]
    total = [n + steps for n in prompts]
    table, pool = R.deal_pages(total, page, gen)
    cos, sin = tables(max(total), D)
    shape = (pool, Hkv, page, D)
    store = R.E4M3 if eight else dt
    cpu = [torch.zeros(shape).to(store), torch.zeros(shape).to(store)] + [torch.zeros(pool, Hkv) for _ in range(2)]
    gpu = [t.cuda() for t in cpu]
    dev = {n: t.cuda() for n, t in (("table", table), ("cos", cos), ("sin", sin))}
    ws = da.alloc_paged_workspace(H, Hkv, D)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    position, counts = [0, 0, 0], prompts
    for step in range(steps + 1):
        tokens = sum(counts)
        k_new, v_new = (R.randn((tokens, Hkv, D), dt, gen) for _ in range(2))
        q = R.randn((tokens, H, D), dt, gen)
        start = torch.tensor([0, counts[0], counts[0] + counts[1], tokens], dtype=torch.int32)
        pos = torch.tensor(position, dtype=torch.int32)
        want_q = R.append(cpu[0], cpu[1], k_new, v_new, table, pos, start, cos, sin, q, *(cpu[2:] if eight else (None, None)))
        args = dict(token_start=start.cuda() if step == 0 else None, rope_cos=dev["cos"], rope_sin=dev["sin"], q=q.cuda(),
                    err_flag=err)
        if eight:
            q_rot = da.kvcache_append_paged_q8(*gpu, k_new.cuda(), v_new.cuda(), dev["table"], pos.cuda(), **args)
        else:
            q_rot = da.kvcache_append_paged(*gpu[:2], k_new.cuda(), v_new.cuda(), dev["table"], pos.cuda(), **args)
        assert torch.equal(R.bits(q_rot), R.bits(want_q))
        position = [p + n for p, n in zip(position, counts)]
        if step:
            kv_len = torch.tensor(position, dtype=torch.int32, device="cuda")
            kw = dict(window=window, sinks=sinks, workspace=ws, err_flag=err)
            if eight:
                out = da.decode_attn_paged_q8_fwd(q_rot, *gpu, dev["table"], kv_len, **kw)
            else:
                out = da.decode_attn_paged_fwd(q_rot, *gpu[:2], dev["table"], kv_len, **kw)
            for b, n in enumerate(position):
                j = R.visible_rows(n, window, sinks)
                p = table[b].long()[j // page]
                rows = [t.view(torch.uint8 if eight else torch.int16)[p, :, j % page].view(store).double() for t in cpu[:2]]
                if eight:
                    rows = [r * s[p].double()[..., None] for r, s in zip(rows, cpu[2:])]
                ref, slack = R.attend(want_q[b].double(), *(r.transpose(0, 1) for r in rows), D ** -0.5)
                R.assert_rows(out[b], ref, slack, f"step {step}, sequence {b}")
        counts = [1, 1, 1]
    assert int(err.item()) == 0
    same(gpu, cpu if eight else cpu[:2] + [None, None], "the cache after the run")

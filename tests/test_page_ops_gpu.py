"""Taking, sharing, releasing, copying and compacting pages, against the plain
forms of tests/draft_reference.py: every number and bit equal."""
import pytest
import torch

import decode_attention_static_gb300 as da
import draft_reference as Q
import paged_reference as R

pytestmark = pytest.mark.gpu

BITS = {"full": 128, "page": 16, "pool": 256, "kv_len": 1, "sequence": 64, "position": 2, "tokens": 32}


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    da.load_library()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def flag_of(errors):
    return sum(BITS[e] for e in errors)


class Cache:
    """A table and a pool's state, on the device and as plain lists."""

    def __init__(self, B, max_pages, num_pages, size):
        self.size, self.pool = size, Q.Pool(num_pages)
        self.table = [[-1] * max_pages for _ in range(B)]
        self.kv_len = [0] * B
        self.d_pool = da.alloc_page_pool(num_pages)
        self.d_table, self.d_len = i32(self.table), i32(self.kv_len)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def same(self, what=""):
        assert self.d_table.cpu().tolist() == self.table, f"{what}: table"
        free, counts, order = (t.cpu().tolist() for t in da.page_pool_views(self.d_pool))
        assert free == [self.pool.free], f"{what}: {free} free pages, not {self.pool.free}"
        assert counts == self.pool.counts, f"{what}: counts"
        assert order[:free[0]] == self.pool.list[:free[0]], f"{what}: free pages"
        assert self.d_pool[1:4].tolist() == [0, 0, 0]
        assert int(self.err.item()) == flag_of(self.pool.errors), f"{what}: flag {int(self.err.item())} {self.pool.errors}"

    def push(self):
        """The plain state to the device."""
        self.d_pool.copy_(self.pool.tensor())
        self.d_table.copy_(i32(self.table))
        self.d_len.copy_(i32(self.kv_len))

    def resize(self, held, wanted, what=""):
        Q.resize(self.table, held, wanted, self.pool, self.size)
        da.kvcache_resize_paged(self.d_table, i32(held), i32(wanted), self.d_pool, self.size, err_flag=self.err)
        self.same(what)

    def fork(self, parent, child, what=""):
        want = Q.fork(self.table, self.kv_len, parent, child, self.pool, self.size)
        got = da.kvcache_fork_paged(self.d_table, self.d_len, i32(parent), i32(child), self.d_pool, self.size,
                                    err_flag=self.err)
        assert got.cpu().tolist() == want, f"{what}: copies"
        assert self.d_len.cpu().tolist() == self.kv_len, f"{what}: lengths"
        self.same(what)
        return got


@pytest.mark.parametrize("B,max_pages,num_pages,size", [(1, 1, 1, 16), (3, 8, 20, 16), (64, 30, 1500, 32), (7, 900, 5000, 16),
                                                        (700, 9, 5000, 256), (520, 70, 33000, 16), (1500, 40, 70000, 64)])
def test_resize_at_random(B, max_pages, num_pages, size):
    """Sequences grow, shrink, end and begin; the list runs out at times."""
    gen = torch.Generator().manual_seed(B + num_pages)
    c = Cache(B, max_pages, num_pages, size)
    c.same("fresh")
    held = [0] * B
    for step in range(6):
        wanted = torch.randint(0, max_pages * size + 1, (B,), generator=gen).tolist()
        for b in range(B):
            if step % 2 and b % 3 == 0:
                wanted[b] = held[b] + (b % 5)
            if step % 3 == 2 and b % 4 == 0:
                wanted[b] = 0
            wanted[b] = min(wanted[b], max_pages * size)
        c.resize(held, wanted, f"step {step}")
        held = wanted
    c.resize(held, [0] * B, "end")
    assert c.pool.free == num_pages and not any(c.pool.counts)


def test_resize_of_nothing():
    c = Cache(3, 4, 6, 16)
    c.resize([0, 0, 0], [0, 0, 0])
    c.resize([0, 0, 0], [1, 16, 17])
    c.resize([1, 16, 17], [16, 15, 32])
    assert c.pool.free == 2


def test_resize_refusals():
    """Lengths, entries and counts that only the device sees."""
    c = Cache(4, 4, 12, 16)
    c.resize([0] * 4, [40, 64, 10, 5])
    c.resize([40, 64, -1, 5], [10, 64, 0, 65], "lengths")
    assert c.pool.errors == {"kv_len"}
    c.table[1][2] = 77
    c.push()
    c.resize([10, 64, 10, 5], [10, 0, 10, 5], "entry")
    c.table[3][0] = c.table[2][0]  # held twice, counted once
    c.push()
    c.resize([10, 0, 10, 5], [0, 0, 0, 0], "released twice")
    assert c.pool.errors == {"kv_len", "page", "pool"}


def test_resize_survives_a_broken_list():
    c = Cache(2, 4, 8, 16)
    c.d_pool[4 + 8 + 7] = 99
    c.d_pool[4 + 8 + 6] = -5
    da.kvcache_resize_paged(c.d_table, i32([0, 0]), i32([40, 0]), c.d_pool, 16, err_flag=c.err)
    assert c.d_table.tolist() == [[-1, -1, 5, -1], [-1] * 4] and int(c.err.item()) == da.DA_DEVERR_POOL
    c.d_pool[0] = 1 << 30
    da.kvcache_resize_paged(c.d_table, i32([0, 0]), i32([0, 16]), c.d_pool, 16, err_flag=c.err)
    assert c.d_pool[0].item() == 7
    c.d_pool[0] = -4
    da.kvcache_resize_paged(c.d_table, i32([0, 0]), i32([0, 16]), c.d_pool, 16, err_flag=c.err)
    assert c.d_pool[0].item() == 0 and int(c.err.item()) == da.DA_DEVERR_POOL | da.DA_DEVERR_FULL


@pytest.mark.parametrize("B,max_pages,num_pages,size", [(2, 1, 3, 16), (16, 20, 400, 16), (300, 40, 9000, 32), (40, 1000, 40000, 16),
                                                        (1400, 4, 6000, 16)])
def test_fork_at_random(B, max_pages, num_pages, size):
    gen = torch.Generator().manual_seed(B)
    c = Cache(B, max_pages, num_pages, size)
    kept = max(1, B // 3)
    for step in range(4):
        held = list(c.kv_len)
        lens = torch.randint(0, max_pages * size + 1, (kept,), generator=gen).tolist() + [0] * (B - kept)
        lens[0] = max_pages * size if step % 2 else max_pages * size - 1
        c.kv_len = lens
        c.resize(held, lens, f"step {step}")
        c.push()
        n = int(torch.randint(1, B - kept + 1, (1,), generator=gen))
        child = (torch.randperm(B - kept, generator=gen)[:n] + kept).tolist()
        parent = torch.randint(0, kept, (n,), generator=gen).tolist()
        c.fork(parent, child, f"step {step}")
    c.resize(c.kv_len, [0] * B, "end")
    assert c.pool.free == num_pages


def test_fork_refusals():
    def fresh(free=20):
        c = Cache(8, 3, free, 16)
        c.kv_len = [40, 16, 5, 0, 0, 0, 0, 0]
        c.resize([0] * 8, c.kv_len)
        c.push()
        return c

    for parent, child in (([0, 0], [3, 3]), ([0, 3], [3, 4]), ([0], [0]), ([8], [3]), ([0], [8]), ([-1, 1], [3, 4]),
                          ([0, 0, 1, 2], [3, -5, 4, 5]), ([0, 0, 1], [4, 4, 4])):
        c = fresh()
        c.fork(parent, child, f"{parent} {child}")
        assert c.pool.errors == {"sequence"}
    c = fresh()
    c.kv_len[1] = 49
    c.push()
    c.fork([0, 1, 2], [3, 4, 5], "length")
    assert c.pool.errors == {"kv_len"}
    c = fresh(6)
    c.fork([0, 1, 2, 0], [3, 4, 5, 6], "full")  # one page is left: whole pages alone need none
    assert c.pool.errors == {"full"} and c.kv_len[3:7] == [40, 16, 0, 0]
    c = fresh()
    c.table[0][1], c.table[2][0] = -1, 50
    c.push()
    c.fork([0, 2], [3, 4], "entries")
    assert c.pool.errors == {"page"}


def pools(layers, pages, Hkv, size, D, store, gen):
    shape = ([layers] if layers else []) + [pages, Hkv, size, D]
    k, v = (torch.randn(shape, generator=gen) * (60 if store == R.E4M3 else 1) for _ in range(2))
    k, v = k.clamp(-448, 448).to(store), v.clamp(-448, 448).to(store)
    if store != R.E4M3:
        return [k, v]
    # scales alike for the most part
    return [k, v] + [torch.exp2(torch.randint(-6, -4, shape[:-2], generator=gen).float()) for _ in range(2)]


def stacked(ts):
    return [t if t.dim() in (3, 5) else t[None] for t in ts]


def equal(got, want, what=""):
    for i, (g, w) in enumerate(zip(got, want)):
        gb, wb = R.bits(g), R.bits(w).reshape(g.shape)
        if g.dtype == R.E4M3:
            gb, wb = (torch.where((x & 0x7F) == 0x7F, torch.full_like(x, 0x7F), x) for x in (gb, wb))
        assert torch.equal(gb, wb), f"{what}: array {i} differs in {(gb != wb).sum().item()} places"


STORES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": R.E4M3}


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("layers,Hkv,size,D", [(0, 1, 16, 64), (1, 8, 32, 128), (3, 5, 256, 64), (2, 2, 64, 128)])
def test_copy_pages(layers, Hkv, size, D, store):
    gen = torch.Generator().manual_seed(size)
    ts = pools(layers, 12, Hkv, size, D, STORES[store], gen)
    copies = [[3, -1, 5, 5, 0, 2, 9], [4, -1, 6, 7, 1, 2, 8], [size, 0, 1, size - 1, 0, 5, 7]]
    dev = [t.cuda() for t in ts]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    da.kvcache_copy_pages(dev[0], dev[1], i32(copies), *dev[2:], err_flag=err)
    Q.copy_pages([t.view(torch.uint8) if t.dtype == R.E4M3 else t for t in stacked(ts)], copies)
    equal(dev, ts, store)
    assert int(err.item()) == 0
    for bad in ([[3], [12], [1]], [[99], [1], [1]], [[3], [4], [-1]], [[3], [4], [size + 1]]):
        err.zero_()
        da.kvcache_copy_pages(dev[0], dev[1], i32(bad), *dev[2:], err_flag=err)
        assert int(err.item()) == da.DA_DEVERR_PAGE
    equal(dev, ts, "refused")
    da.kvcache_copy_pages(dev[0], dev[1], i32([[3, 1], [-1, -1], [1, 1]]), *dev[2:])
    equal(dev, ts, "skipped")


def compact(ts, table, keep, start, position, size, what="", errors=None):
    dev = [t.cuda() for t in ts]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    table, keep, start, position = (torch.tensor(x, dtype=torch.int32) for x in (table, keep, start, position))
    args = [x.cuda() for x in (table, keep, start, position)]
    (da.kvcache_compact_paged_q8 if len(ts) == 4 else da.kvcache_compact_paged)(*dev, *args, err_flag=err)
    flat = stacked(ts)
    found = Q.compact(flat[:2], table, keep, start, position, size, flat[2:] or (None, None))
    equal(dev, ts, what)
    assert int(err.item()) == flag_of(found), f"{what}: flag {int(err.item())}, {found}"
    if errors is not None:
        assert found == errors


@pytest.mark.parametrize("store", STORES)
@pytest.mark.parametrize("layers,Hkv,size,D", [(0, 1, 16, 64), (1, 8, 16, 128), (3, 5, 32, 64), (2, 2, 256, 128)])
def test_compact_at_random(layers, Hkv, size, D, store):
    gen = torch.Generator().manual_seed(size + D)
    for seed in range(4):
        B, most = 9, 5
        ts = pools(layers, B * most + 2, Hkv, size, D, STORES[store], gen)
        table = (torch.randperm(B * most + 2, generator=gen)[:B * most]).view(B, most).tolist()
        keep, start, position = [], [2], []
        keep = [0, 0]  # rows of nobody
        for b in range(B):
            p0 = int(torch.randint(0, 3 * size, (1,), generator=gen))
            span = most * size - p0
            n = [0, 1, 2, 9, span, span // 2, 17, 3, size][(b + seed) % 9]
            reach = min(span, n + int(torch.randint(0, span - n + 1, (1,), generator=gen)))
            rows = (torch.randperm(reach, generator=gen)[:n].sort().values + p0).tolist()
            keep += rows
            start.append(len(keep))
            position.append(p0)
        keep += [3]
        compact(ts, table, keep, start, position, size, f"seed {seed}", set())


@pytest.mark.parametrize("store", ["f16", "e4m3"])
def test_compact_refusals(store):
    gen = torch.Generator().manual_seed(1)
    table = [[0, 1, 2], [3, 4, 5]]
    for what, keep, start, position, errors in (
            ("falling", [5, 9, 8, 12, 3, 40], [0, 4, 6], [4, 3], {"position"}),
            ("twice", [5, 9, 9, 12, 3, 40], [0, 4, 6], [4, 3], {"position"}),
            ("up", [5, 6, 9, 12, 3, 40], [0, 4, 6], [6, 3], {"position"}),
            ("outside", [5, 9, 48, 50, 3, 40], [0, 4, 6], [4, 3], {"position"}),
            ("below", [-1, 9, 11, 12, 3, 40], [0, 4, 6], [-1, 3], {"position"}),
            ("far", [5, 9, 11, 12, 3, 40], [0, 4, 6], [(1 << 31) - 1, 3], {"position"}),
            ("range", [5, 9, 11, 12, 3, 40], [0, 4, 60], [4, 3], {"tokens"}),
            ("falling range", [5, 9, 11, 12, 3, 40], [5, 4, 6], [4, 3], {"tokens"})):
        compact(pools(2, 6, 2, 16, 64, STORES[store], gen), table, keep, start, position, 16, what, errors)
    for bad in ([[0, 1, 99], [3, 4, 5]], [[-1, 1, 2], [3, 4, 5]], [[0, -3, 2], [3, 4, 5]]):
        compact(pools(2, 6, 2, 16, 64, STORES[store], gen), bad, [5, 20, 21, 40, 3, 40], [0, 4, 6], [4, 3], 16, str(bad),
                {"page"})


def test_compact_scales():
    """8 bits: one page's scale grows under rows of another's, NaN codes stay NaN, and where scales are
    alike the other rows keep their bits."""
    gen = torch.Generator().manual_seed(1)
    ts = pools(0, 3, 2, 16, 64, R.E4M3, gen)
    ts[2][:] = 2.0 ** -5
    ts[3][:] = 0.013
    ts[2][1] = 2.0 ** -3
    ts[3][1] = 0.02
    ts[0].view(torch.uint8)[0, 0, 3, 5] = 0x7F
    ts[1].view(torch.uint8)[1, 0, 4, 7] = 0xFF
    before = [t.clone() for t in ts]
    compact(ts, [[0, 1, 2]], [13, 20, 22], [0, 3], [12], 16, "grown", set())
    assert torch.equal(ts[2][0], ts[2][1]) and ts[1][0, 0, 13, 7].isnan()
    ts = before
    ts[2][:] = ts[3][:] = 0.25
    compact(ts, [[0, 1, 2]], [13, 20, 22], [0, 3], [12], 16, "alike", set())


def test_pages_in_graphs_and_on_streams():
    """A step of the bookkeeping captured and replayed beside another one on its
    own stream: equal states after each."""
    def make():
        c = Cache(32, 20, 500, 16)
        c.kv_len = [100 + 3 * b for b in range(16)] + [0] * 16
        c.resize([0] * 32, c.kv_len)
        c.push()
        return c

    a, b = make(), make()
    held = [i32(x.kv_len) for x in (a, b)]
    up = [h + 30 for h in held]
    for u in up:
        u[16:] = 0
    side = torch.cuda.Stream()
    copies = [torch.empty((3, 16), dtype=torch.int32, device="cuda") for _ in range(2)]
    fam = i32(list(range(16))), i32(list(range(16, 32)))
    zero = [torch.cat([h[:16], torch.zeros(16, dtype=torch.int32, device="cuda")]) for h in held]

    def step(c, i):
        da.kvcache_resize_paged(c.d_table, held[i], up[i], c.d_pool, 16, err_flag=c.err)
        da.kvcache_resize_paged(c.d_table, up[i], held[i], c.d_pool, 16, err_flag=c.err)
        da.kvcache_fork_paged(c.d_table, c.d_len, *fam, c.d_pool, 16, copies=copies[i], err_flag=c.err)
        da.kvcache_resize_paged(c.d_table, c.d_len, zero[i], c.d_pool, 16, err_flag=c.err)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(b, 1)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(b, 1)
    torch.cuda.synchronize()
    step(a, 0)
    for _ in range(3):
        step(a, 0)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.d_table, b.d_table) and torch.equal(a.d_pool, b.d_pool) and torch.equal(copies[0], copies[1])
    assert int(a.err.item()) == int(b.err.item()) == 0

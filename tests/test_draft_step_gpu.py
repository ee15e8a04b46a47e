"""The operators for drafted tokens together, as a serving step runs them: pages
taken, drafts appended with rotary positions by depth, verified in one call, the
accepted rows moved together and the other pages given back. The cache must then
be what appending the accepted tokens alone would have made it, and the
verification's outputs those of decoding them one by one."""
import pytest
import torch

import decode_attention_static_gb300 as da
import paged_reference as R
from test_paged_append_gpu import tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build_library()
    da.load_library()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


H, HKV, D, PAGE, LAYERS, MOST = 8, 2, 64, 16, 2, 12
# a tree of 7 drafts: parents, and the accepted path
PARENT = [-1, 0, 0, 1, 2, 2, 5]
PATH = [0, 2, 5, 6]


def depth_and_masks():
    depth, masks = [], []
    for i, p in enumerate(PARENT):
        depth.append(0 if p < 0 else depth[p] + 1)
        masks.append((0 if p < 0 else masks[p]) | 1 << i)
    return depth, masks


class Cache:
    def __init__(self, B, eight):
        self.eight = eight
        store = R.E4M3 if eight else torch.float16
        n = B * MOST + 4
        self.pools = [torch.zeros(LAYERS, n, HKV, PAGE, D, device="cuda").to(store) for _ in range(2)]
        if eight:
            self.pools += [torch.zeros(LAYERS, n, HKV, device="cuda") for _ in range(2)]
        self.table = torch.full((B, MOST), -1, dtype=torch.int32, device="cuda")
        self.state = da.alloc_page_pool(n)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cos, self.sin = (t.cuda() for t in tables(MOST * PAGE, D))

    def layer(self, i):
        return [t[i] for t in self.pools]

    def resize(self, held, wanted):
        da.kvcache_resize_paged(self.table, held, wanted, self.state, PAGE, err_flag=self.err)

    def append(self, i, k, v, at, start, turns, q):
        fn = da.kvcache_append_paged_q8_axes if self.eight else da.kvcache_append_paged_axes
        return fn(*self.layer(i), k, v, self.table, at, turns, self.cos, self.sin, token_start=start, q=q, err_flag=self.err)

    def tree(self, i, q, kv_len, start, mask):
        fn = da.decode_attn_tree_q8_fwd if self.eight else da.decode_attn_tree_fwd
        return fn(q, *self.layer(i), self.table, kv_len, token_start=start, tree_mask=mask, err_flag=self.err)

    def decode(self, i, q, kv_len):
        fn = da.decode_attn_paged_q8_fwd if self.eight else da.decode_attn_paged_fwd
        return fn(q, *self.layer(i), self.table, kv_len, err_flag=self.err)

    def rows(self, b, n):
        """K and V of a sequence's first n rows as values, [layers, HKV, n, D]."""
        at = torch.arange(n, device="cuda")
        ids = self.table[b].long()[at // PAGE]
        out = []
        for x in range(2):
            bits = self.pools[x].view(torch.uint8 if self.eight else torch.int16)
            r = bits[:, ids, :, at % PAGE].view(self.pools[x].dtype).double()  # [n, layers, HKV, D]
            if self.eight:
                r = r * self.pools[2 + x][:, ids].transpose(0, 1).double()[..., None]
            out.append(r)
        return out


def fill(cache, lens, gen):
    """Prefixes of `lens` rows in every layer."""
    zero = i32([0] * len(lens))
    cache.resize(zero, i32(lens))
    start = i32([sum(lens[:b]) for b in range(len(lens) + 1)])
    turns = torch.cat([torch.arange(n) for n in lens])[None].to(torch.int32).cuda()
    for i in range(LAYERS):
        k, v = (torch.randn(sum(lens), HKV, D, generator=gen).half().cuda() for _ in range(2))
        cache.append(i, k, v, zero, start, turns, None)


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
def test_a_step_with_drafts(eight):
    lens = [37, 16, 100, 1]
    B, m = len(lens), len(PARENT)
    depth, masks = depth_and_masks()
    gen = torch.Generator().manual_seed(0)
    step, plain = Cache(B, eight), Cache(B, eight)
    for cache in (step, plain):
        fill(cache, lens, torch.Generator().manual_seed(1))
    k, v = (torch.randn(LAYERS, B, m, HKV, D, generator=gen).half().cuda() for _ in range(2))
    q = torch.randn(LAYERS, B, m, H, D, generator=gen).half().cuda()
    base = i32(lens)
    start = i32([m * b for b in range(B + 1)])
    turns = i32([[n + d for n in lens for d in depth]])
    mask = torch.tensor([[x] for _ in lens for x in masks], dtype=torch.int64, device="cuda")
    keep = i32([n + j for n in lens for j in PATH])
    keep_start = i32([len(PATH) * b for b in range(B + 1)])
    outs = []

    def run():
        step.resize(base, base + m)
        outs.clear()
        for i in range(LAYERS):
            rot = step.append(i, k[i].flatten(0, 1), v[i].flatten(0, 1), base, start, turns, q[i].flatten(0, 1))
            outs.append(step.tree(i, rot, base + m, start, mask))
        (da.kvcache_compact_paged_q8 if eight else da.kvcache_compact_paged)(
            *step.pools, step.table, keep, keep_start, base, err_flag=step.err)
        step.resize(base + m, base + len(PATH))

    run()
    # the accepted tokens one by one into the other cache
    want = []
    plain.resize(base, base + len(PATH))
    for d, j in enumerate(PATH):
        at = base + d
        for i in range(LAYERS):
            rot = plain.append(i, k[i][:, j].contiguous(), v[i][:, j].contiguous(), at, None, at[None], q[i][:, j].contiguous())
            want.append(plain.decode(i, rot, at + 1))
    assert int(step.err.item()) == 0 and int(plain.err.item()) == 0
    for b, n in enumerate(lens):
        for x, y in zip(step.rows(b, n + len(PATH)), plain.rows(b, n + len(PATH))):
            if eight:  # a rejected row's scale may have rounded its page once more: a step of 2^-3, of what the scale grew
                assert (x - y).abs().max() <= 2.0 ** -3 * y.abs().max()
                assert (x - y).norm() <= 2.0 ** -4 * y.norm()
            else:
                assert torch.equal(x, y)
    for d, j in enumerate(PATH):
        for i in range(LAYERS):
            got = outs[i].view(B, m, H, D)[:, j].double()
            ref = want[d * LAYERS + i].double()
            # fp16 weights and outputs, half a step of each (2^-11), of values up to max|v|; in 8 bits rows rounded apart
            assert (got - ref).norm() <= (2.0 ** -3 if eight else 2.0 ** -9) * ref.norm()
    assert (step.table >= 0).sum().item() == sum(-(-(n + len(PATH)) // PAGE) for n in lens)
    free, counts, _ = da.page_pool_views(step.state)
    assert free.item() == counts.numel() - int((step.table >= 0).sum()) and counts.max().item() == 1


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
def test_a_captured_step(eight):
    """The step in one graph (each kernel starting under the one before it) gives
    the bits of its calls one by one, replay after replay."""
    lens = [37, 16, 90, 1]
    B, m = len(lens), len(PARENT)
    depth, masks = depth_and_masks()
    mask = torch.tensor([[x] for _ in lens for x in masks], dtype=torch.int64, device="cuda")
    start, keep_start = i32([m * b for b in range(B + 1)]), i32([len(PATH) * b for b in range(B + 1)])
    gen = torch.Generator().manual_seed(0)
    k, v = (torch.randn(LAYERS, B * m, HKV, D, generator=gen).half().cuda() for _ in range(2))
    q = torch.randn(LAYERS, B * m, H, D, generator=gen).half().cuda()
    path, depths = i32(PATH), i32(depth)
    results = []
    for captured in (False, True):
        cache = Cache(B, eight)
        fill(cache, lens, torch.Generator().manual_seed(1))
        base, n_all = i32(lens), i32([0] * B)
        keep, turns = i32([0] * (B * len(PATH))), i32([[0] * (B * m)])
        ws = da.alloc_tree_workspace(H, HKV, D)
        outs = [torch.empty(B * m, H, D, dtype=torch.float16, device="cuda") for _ in range(LAYERS)]

        def step():
            torch.add(base, m, out=n_all)
            cache.resize(base, n_all)
            turns.view(B, m).copy_(base[:, None] + depths)
            keep.view(B, -1).copy_(base[:, None] + path)
            for i in range(LAYERS):
                rot = cache.append(i, k[i], v[i], base, start, turns, q[i])
                (da.decode_attn_tree_q8_fwd if eight else da.decode_attn_tree_fwd)(
                    rot, *cache.layer(i), cache.table, n_all, token_start=start, tree_mask=mask, out=outs[i], workspace=ws,
                    err_flag=cache.err)
            (da.kvcache_compact_paged_q8 if eight else da.kvcache_compact_paged)(
                *cache.pools, cache.table, keep, keep_start, base, err_flag=cache.err)
            base.add_(len(PATH))
            cache.resize(n_all, base)

        if captured:
            side = torch.cuda.Stream()
            saved = [t.clone() for t in (*cache.pools, cache.table, cache.state, base)]
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
            for t, s in zip((*cache.pools, cache.table, cache.state, base), saved):
                t.view(torch.uint8).copy_(s.view(torch.uint8))
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            go = g.replay
        else:
            go = step
        got = []
        for _ in range(6):
            go()
            got += [R.bits(o) for o in outs]
        torch.cuda.synchronize()
        assert int(cache.err.item()) == 0
        results.append(got + [R.bits(t) for t in (*cache.pools, cache.table, base)])
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("eight", [False, True], ids=["16bit", "e4m3"])
def test_samples_of_one_prompt(eight):
    """Forks share the prompt's pages and go on apart."""
    n, B = 41, 4
    cache = Cache(B, eight)
    fill(cache, [n, 0, 0, 0], torch.Generator().manual_seed(1))
    lens = i32([n, 0, 0, 0])
    copies = da.kvcache_fork_paged(cache.table, lens, i32([0, 0, 0]), i32([1, 2, 3]), cache.state, PAGE, err_flag=cache.err)
    da.kvcache_copy_pages(cache.pools[0], cache.pools[1], copies, *cache.pools[2:], err_flag=cache.err)
    assert lens.tolist() == [n] * B and int(cache.err.item()) == 0
    want = cache.rows(0, n)
    for b in range(1, B):
        for x, y in zip(cache.rows(b, n), want):
            assert torch.equal(x, y)
    cache.resize(lens, lens + 10)
    gen = torch.Generator().manual_seed(2)
    for d in range(10):
        for i in range(LAYERS):
            k, v = (torch.randn(B, HKV, D, generator=gen).half().cuda() for _ in range(2))
            cache.append(i, k, v, lens + d, None, (lens + d)[None], None)
    for b in range(1, B):
        for x, y in zip(cache.rows(b, n + 10), cache.rows(0, n + 10)):
            assert not torch.equal(x[n:], y[n:])
            if not eight:
                assert torch.equal(x[:n], y[:n])
    cache.resize(lens + 10, lens * 0)
    free, counts, order = da.page_pool_views(cache.state)
    assert free.item() == counts.numel() and int(counts.abs().max()) == 0
    assert sorted(order.tolist()) == list(range(counts.numel())) and int(cache.err.item()) == 0

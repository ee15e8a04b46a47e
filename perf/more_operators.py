"""What the operators of a serving step with drafted tokens cost, and what they compute.

Five operators around a paged decode cache: attention of several drafted tokens of
each sequence, which form a tree, over the cache that holds their rows already; the
append of new rows with rotary positions of several axes (time, height, width, or a
drafted token's depth); forking sequences, with the copies of the pages that they do
not share; moving the rows of accepted tokens together; and taking and releasing
pages as sequences grow and shrink. ``run`` computes them with elementary torch
operations, or, where ``own`` is true, with the framework's entry points.
"""
import math
import random

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_EXPONENT = -100  # smallest scale of an 8-bit block: 2 ** MIN_EXPONENT
HEADER = 4  # words of a page pool's state before its counts and its list of free pages


# ---------------------------------------------------------------------------
# Cases


def listed():
    return [
        # One user, multi-head attention, a short prefix and a handful of drafts: latency.
        dict(name="tree of 8, 1 x 1024, 16/16 heads", op="tree", B=1, H=16, Hkv=16, D=128, type="f16", page=16,
             longest=1024, ragged=False, drafts=8, chain=False, lens=1),
        # A batch that verifies wide trees.
        dict(name="tree of 64, 16 ragged to 8191, 32/8 heads", op="tree", B=16, H=32, Hkv=8, D=128, type="bf16",
             page=64, longest=8191, ragged=True, drafts=64, chain=False, lens=2, idle=1),
        # Long contexts with short chains of drafts: the most bytes.
        dict(name="chain of 5, 32 ragged to 32768, 32/8 heads", op="tree", B=32, H=32, Hkv=8, D=128, type="bf16",
             page=64, longest=32768, ragged=True, drafts=5, chain=True, lens=3),
        # Eight heads on each KV head over the 8-bit cache: the most products.
        dict(name="tree of 32 over 8 bits, 32 ragged to 16384, 64/8 heads", op="tree8", B=32, H=64, Hkv=8, D=128,
             type="bf16", page=32, longest=16384, ragged=True, drafts=32, chain=False, lens=4),
        # The drafts of one step enter the cache, rotated by their depth in the tree. Latency.
        dict(name="append by depth, 16 sequences, 8 drafts", op="axes", B=16, H=32, Hkv=8, D=128, type="bf16", page=16,
             longest=8, ragged=False, reach=8192, axes=1, split="sections", lens=5),
        # Prompts with images, three axes, into the 8-bit cache.
        dict(name="append 8 bits by three axes, prompts of 20k tokens", op="axes8", B=5, H=32, Hkv=8, D=128,
             type="bf16", page=64, longest=8191, ragged=True, reach=8192, axes=3, split="sections", lens=6),
        # Eight samples from one prompt of odd length, one layer's pools.
        dict(name="fork, 8 samples of one prompt", op="fork", B=8, parents=1, Hkv=8, D=128, type="bf16", page=16,
             layers=1, longest=1021, lens=7),
        # A beam step of 96 sequences over the pools of 12 layers, a third of them kept.
        dict(name="fork, 96 beams, 12 layers", op="fork", B=96, parents=32, Hkv=8, D=128, type="bf16", page=64,
             layers=12, longest=2048, lens=8),
        # The accepted drafts of a small batch, one layer's pools. Latency.
        dict(name="compact, 8 sequences, up to 5 of 16 drafts", op="compact", B=8, Hkv=8, D=128, type="f16", page=16,
             layers=1, longest=4096, drafts=16, most=5, lens=9),
        # The accepted drafts of a large batch, 8 bits, the pools of 36 layers.
        dict(name="compact 8 bits, 64 sequences, 36 layers", op="compact8", B=64, Hkv=8, D=128, type="bf16", page=32,
             layers=36, longest=1024, drafts=32, most=9, lens=10),
        # Pages behind the accepted drafts go back, pages for the next ones are taken.
        dict(name="resize, 64 sequences by a step's drafts", op="resize", B=64, page=16, longest=8192, low=32,
             high=64, whole=False, lens=11),
        # A batch ends and another takes its pages.
        dict(name="resize, 256 sequences come and go", op="resize", B=256, page=16, longest=8192, low=0, high=0,
             whole=True, lens=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree8", "tree8", "axes", "axes8", "fork", "compact", "compact8", "resize"])
    heads_kv = rng.choice([1, 2, 4, 5, 8, 16])
    case = dict(op=op, lens=rng.randrange(1 << 20), page=rng.choice([16, 32, 64, 128, 256]))
    if op == "resize":
        B = _log(rng, 1, 512)
        case.update(B=B, longest=_log(rng, 64, 2000000 // B if B > 60 else 32768))
        if rng.random() < 0.5:
            case.update(low=0, high=0, whole=True)
        else:
            low = _log(rng, 1, 256)
            case.update(low=low, high=low + _log(rng, 1, 256), whole=False)
        return case
    D = rng.choice([64, 128, 128])
    case.update(Hkv=heads_kv, D=D, type=rng.choice(["f16", "bf16"]))
    if op in ("tree", "tree8"):
        group = rng.choice([1, 2, 4, 8])
        drafts = rng.choice([1, 3, 5, 8, 16, 26, 32, 60, 64, 100, 256])
        # cached rows of the batch: so many that the plain form's scores and the products stay within the listed ones
        rows = _log(rng, 64, min(500000, 4000000 // heads_kv, 400000000 // (heads_kv * group * drafts)))
        B = _log(rng, 1, max(1, min(64, rows // drafts)))
        case.update(B=B, H=heads_kv * group, longest=max(drafts, min(32768, rows // B)), ragged=rng.random() < 0.7,
                    drafts=drafts, chain=rng.random() < 0.3)
        if B > 2 and rng.random() < 0.3:
            case["idle"] = 1
    elif op in ("axes", "axes8"):
        axes = rng.choice([1, 2, 3, 3, 4])
        tokens, B = _log(rng, 1, 16384), _log(rng, 1, 64)
        case.update(B=B, H=heads_kv * rng.choice([1, 2, 4, 8]), longest=max(1, tokens // B), ragged=rng.random() < 0.7,
                    reach=_log(rng, 64, 16384), axes=axes, split=rng.choice(["sections", "interleaved"]))
    elif op == "fork":
        B = rng.randint(2, 128)
        case.update(B=B, parents=rng.randint(1, max(1, B // 2)), layers=rng.choice([1, 1, 4, 12]),
                    longest=_log(rng, 1, 4096))
        case["layers"] = min(case["layers"], max(1, 24000000 // (case["parents"] * case["longest"] * heads_kv * 4
                                                                + B * case["page"] * heads_kv * 4)))
    else:
        most = _log(rng, 1, 32)
        case.update(B=_log(rng, 1, 96), layers=rng.choice([1, 1, 4, 36]), longest=_log(rng, 64, 1024),
                    drafts=2 * most + rng.randint(0, 64), most=most)
        case["layers"] = min(case["layers"], max(1, 24000000 // (case["B"] * (case["longest"] + 128) * heads_kv)))
    return case


def counts(case):
    """Rows of each sequence before the call's own ones, and the new or drafted ones."""
    r = random.Random(case["lens"])
    B, longest, op = case["B"], case["longest"], case["op"]
    if op in ("tree", "tree8"):
        new = [case["drafts"]] * B
        if case["ragged"]:
            new = [r.randint(max(1, case["drafts"] // 2), case["drafts"]) for _ in range(B)]
            new[r.randrange(B)] = case["drafts"]
            n = [r.randint(max(1, longest // 8), longest) for _ in range(B)]
            n[r.randrange(B)] = longest
        else:
            n = [longest] * B
        old = [max(0, a - m) for a, m in zip(n, new)]
        if case.get("idle"):
            new[0] = old[0] = 0
        return old, new
    if op in ("axes", "axes8"):
        new = [longest] * B
        if case["ragged"]:
            new = [r.randint(max(1, longest // 8), longest) for _ in range(B)]
            new[r.randrange(B)] = longest
        return [r.randint(0, case["reach"] - 1) for _ in range(B)], new
    if op == "fork":  # parents first, then as many sequences that fork one of them
        n = [r.randint(max(1, longest // 2), longest) for _ in range(case["parents"])]
        n[0] = longest
        return n + [0] * (B - len(n)), [r.randrange(case["parents"]) for _ in range(B - len(n))]
    if op in ("compact", "compact8"):
        return [r.randint(longest // 4, longest) for _ in range(B)], [r.randint(1, case["most"]) for _ in range(B)]
    if case["whole"]:
        return [0] * B, [r.randint(max(1, longest // 8), longest) for _ in range(B)]
    base = [r.randint(max(1, longest // 8), longest) for _ in range(B)]
    return [n + r.randint(0, case["low"]) for n in base], [n + case["high"] for n in base]


def trees(case):
    """For every drafted token of every sequence: its ancestors and itself, as a bit mask, and its depth."""
    r = random.Random(case["lens"] + 1)
    masks, depths = [], []
    for m in counts(case)[1]:
        seen, depth = [], []
        for i in range(m):
            parent = None if i == 0 else i - 1 if case.get("chain") else r.randint(max(0, (i - 1) // 4), i - 1)
            seen.append((0 if parent is None else seen[parent]) | 1 << i)
            depth.append(0 if parent is None else depth[parent] + 1)
        masks += seen
        depths += depth
    return masks, depths


def kept(case):
    """Rows that compaction keeps, of each sequence: its first draft, and as many others as were accepted."""
    r = random.Random(case["lens"] + 1)
    rows = []
    for n, m in zip(*counts(case)):
        rows.append([n] + sorted(n + i for i in r.sample(range(m, case["drafts"]), m - 1)))
    return rows


def work(case):
    op, page = case["op"], case["page"]
    old, new = counts(case)
    if op in ("tree", "tree8"):
        H, Hkv, D, T = case["H"], case["Hkv"], case["D"], sum(new)
        rows = sum(a + b for a, b in zip(old, new))
        element = 1 if op == "tree8" else 2
        pairs = sum(a * b for a, b in zip(old, new)) + sum(m.bit_count() for m in trees(case)[0])
        return {"bytes": 2 * rows * Hkv * D * element + 4 * T * H * D, "flops": 4 * pairs * H * D}
    if op in ("axes", "axes8"):
        H, Hkv, D, T = case["H"], case["Hkv"], case["D"], sum(new)
        store = 2 if op == "axes" else 1
        return {"bytes": 2 * T * Hkv * D * (2 + store) + 4 * T * H * D + 4 * case["axes"] * T, "flops": 3 * T * (H + Hkv) * D}
    if op == "fork":
        forks = [old[p] for p in new]
        moved = sum(n % page for n in forks) * case["layers"] * case["Hkv"] * case["D"] * 4
        entries = sum(n // page for n in forks)  # a table entry read and written, a count read and written
        return {"bytes": 2 * moved + 16 * entries, "flops": entries}
    if op in ("compact", "compact8"):
        moved = sum(a != b for n, rows in zip(old, kept(case)) for a, b in zip(rows, range(n, n + len(rows))))
        element = 1 if op == "compact8" else 2
        return {"bytes": 4 * moved * case["layers"] * case["Hkv"] * case["D"] * element, "flops": 0}
    pages = sum(-(-b // page) - -(-a // page) for a, b in zip(old, new))
    return {"bytes": 2 * 16 * pages + 16 * case["B"], "flops": 2 * pages}


# ---------------------------------------------------------------------------
# Inputs


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pool(rows, page, gen, spare):
    """Pages of a pool, dealt to sequences of these rows in a random order: the table (-1 where a sequence has no
    page), the pages in use, and the others in rising order."""
    need = [-(-r // page) for r in rows]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32).cpu()
    table = torch.full((len(rows), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return table, order[:at], order[at:].sort().values


def _state(used, free, pages, table):
    """State of a page pool: a header (how many pages are free), a count for each page, the list of free pages."""
    state = torch.zeros(HEADER + 2 * pages, dtype=torch.int32)
    state[0] = len(free)
    state[HEADER:HEADER + pages] = torch.bincount(table[table >= 0].long(), minlength=pages).to(torch.int32)
    state[HEADER + pages:HEADER + pages + len(free)] = free
    return state.cuda()


def _fill(s, shape, eight, dt, gen):
    """Page pools of K and V: keys with a few wide channels, in 8 bits with scales of their own."""
    if eight:
        for x in ("k", "v"):
            s[x] = (torch.randn(shape, generator=gen, device="cuda") * 100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3)
            s[x + "_scale"] = torch.exp2(torch.randint(-8, -6, shape[:-2], generator=gen, device="cuda").float())
    else:
        spread = torch.ones(shape[-1], device="cuda")
        spread[torch.randint(0, shape[-1], (3,), generator=gen, device="cuda")] = 4.0
        s["k"] = (torch.randn(shape, generator=gen, device="cuda") * spread).to(dt)
        s["v"] = torch.randn(shape, generator=gen, device="cuda").to(dt)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, B, page = case["op"], case["B"], case["page"]
    old, new = counts(case)
    s = dict(case=case)
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(TYPES[case["type"]])  # noqa: E731
    if op == "resize":
        reach = [max(a, b) for a, b in zip(old, new)]
        table, used, free = _pool(reach, page, gen, 37)
        pages = len(used) + len(free)
        s.update(table=table.cuda(), pool=_state(used, free, pages, table), low=_int32(old), high=_int32(new))
        return s
    Hkv, D, dt = case["Hkv"], case["D"], TYPES[case["type"]]
    if op in ("tree", "tree8"):
        table, used, free = _pool([a + b for a, b in zip(old, new)], page, gen, 3)
        _fill(s, (len(used) + 3, Hkv, page, D), op == "tree8", dt, gen)
        T, H = sum(new), case["H"]
        bounds = [0]
        for m in new:
            bounds.append(bounds[-1] + m)
        words = -(-case["drafts"] // 64)
        mask = None
        if not case["chain"]:
            flat = [(m >> 64 * w) & (1 << 64) - 1 for m in trees(case)[0] for w in range(words)]
            mask = torch.tensor([f - (1 << 64) if f >> 63 else f for f in flat], dtype=torch.int64,
                                device="cuda").view(T, words)
        s.update(q=normal(T, H, D), table=table.cuda(), bounds=_int32(bounds), mask=mask,
                 kv_len=_int32([a + b for a, b in zip(old, new)]), scale=D ** -0.5)
        # the scratch that a program keeps for its attention calls
        s["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    elif op in ("axes", "axes8"):
        table, used, free = _pool([a + b for a, b in zip(old, new)], page, gen, 3)
        _fill(s, (len(used) + 3, Hkv, page, D), op == "axes8", dt, gen)
        T, bounds, axes = sum(new), [0], case["axes"]
        for m in new:
            bounds.append(bounds[-1] + m)
        if axes == 1:  # drafts: their depth in the tree behind the sequence's rows
            depth = trees(case)[1]
            places = [[n + depth[bounds[b] + i] for b, n in enumerate(old) for i in range(new[b])]]
        else:  # image patches: a frame and places of a grid, all behind the sequence's rows
            side = 1 + math.isqrt(max(new))
            unit = [side * side, side, 1, 7]
            places = [[n + i // unit[a] % (side + a) for n, m in zip(old, new) for i in range(m)] for a in range(axes)]
        pair = torch.arange(D // 2)
        axis = pair % axes if case["split"] == "interleaved" else (pair * axes) // (D // 2)
        rows = max(max(p) for p in places) + 1
        angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D))
        angle = torch.cat([angle, angle], dim=1)
        s.update(table=table.cuda(), position=_int32(old), bounds=_int32(bounds), places=_int32(places),
                 axis=_int32(axis.tolist()), cos=angle.cos().float(), sin=angle.sin().float(), k_new=normal(T, Hkv, D),
                 v_new=normal(T, Hkv, D), q=normal(T, case["H"], D))
    elif op == "fork":
        parents = case["parents"]
        table, used, free = _pool(old, page, gen, B - parents + 5)
        pages = len(used) + len(free)
        _fill(s, (case["layers"], pages, Hkv, page, D), False, dt, gen)
        s.update(table=table.cuda(), pool=_state(used, free, pages, table), kv_len=_int32(old), parent=_int32(new),
                 child=_int32(list(range(parents, B))))
        # the sequences that are dropped for the forks (at first they hold nothing)
        s["kept_len"] = _int32(old)
    else:
        table, used, free = _pool([n + case["drafts"] for n in old], page, gen, 3)
        _fill(s, (case["layers"], len(used) + 3, Hkv, page, D), op == "compact8", dt, gen)
        rows = kept(case)
        bounds = [0]
        for r in rows:
            bounds.append(bounds[-1] + len(r))
        s.update(table=table.cuda(), position=_int32(old), bounds=_int32(bounds), keep=_int32(sum(rows, [])))
    return s


# ---------------------------------------------------------------------------
# Plain forms


def _sequence(bounds, T):
    """Sequence of each packed entry, and its number within it."""
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(bounds[1:].contiguous(), t, right=True)
    return b, t - bounds.long()[b]


def _gathered(s, x):
    """K or V of every sequence in 32 bits: [B, Hkv, rows, D]."""
    ids = s["table"].long().clamp(min=0)
    if s[x].dtype == E4M3:
        got = s[x].view(torch.uint8)[ids].view(E4M3).float() * s[x + "_scale"][ids][..., None, None]
    else:
        got = s[x][ids].float()
    return got.transpose(1, 2).flatten(2, 3)


def _plain_tree(s):
    case, q, n = s["case"], s["q"], s["kv_len"].long()
    B, Hkv, D, T = case["B"], case["Hkv"], case["D"], q.shape[0]
    k, v = _gathered(s, "k"), _gathered(s, "v")
    L = k.shape[2]
    b, i = _sequence(s["bounds"], T)
    most = case["drafts"]
    dense = torch.zeros((B, most) + q.shape[1:], device="cuda")
    dense[b, i] = q.float()
    dense = dense.view(B, most, Hkv, -1, D).transpose(1, 2)  # [B, Hkv, most, G, D]
    x = torch.matmul(dense.flatten(2, 3), k.transpose(2, 3)) * s["scale"]
    drafted = torch.arange(L, device="cuda")[None] - (n - (s["bounds"][1:] - s["bounds"][:-1]))[:, None]  # [B, L]
    inside = (drafted >= 0) & (torch.arange(L, device="cuda")[None] < n[:, None])
    if s["mask"] is None:
        seen = drafted[:, None] <= torch.arange(most, device="cuda")[None, :, None]
    else:
        bits = torch.zeros((B, most, s["mask"].shape[1]), dtype=torch.int64, device="cuda")
        bits[b, i] = s["mask"]
        at = drafted.clamp(0, 64 * s["mask"].shape[1] - 1)[:, None].expand(B, most, L)
        seen = (bits.gather(2, at // 64) >> at % 64) & 1 == 1
    seen = (drafted < 0)[:, None] | (seen & inside[:, None])  # [B, most, L]
    G = case["H"] // Hkv
    x = x.view(B, Hkv, most, G, L).masked_fill_(~seen[:, None, :, None], float("-inf"))
    top = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(top.isfinite(), top, torch.zeros_like(top)))
    total = p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), v).view(B, Hkv, most, G, D) / torch.where(total > 0, total, torch.ones_like(total))
    return out.transpose(1, 2).flatten(2, 3)[b, i].to(q.dtype)


def _turned(x, cos, sin):
    half = x.shape[-1] // 2
    x = x.float()
    return x * cos + torch.cat([-x[..., half:], x[..., :half]], dim=-1) * sin


def _plain_axes(s):
    case, page, T = s["case"], s["case"]["page"], s["k_new"].shape[0]
    b, i = _sequence(s["bounds"], T)
    at = s["position"].long()[b] + i
    ids, row = s["table"].long()[b, at // page], at % page
    column = torch.arange(case["D"], device="cuda")
    turn = s["places"].long()[s["axis"].long()].t().repeat(1, 2)  # [T, D]: the table row of every element
    cos, sin = s["cos"][turn, column][:, None], s["sin"][turn, column][:, None]
    k, q = _turned(s["k_new"], cos, sin), _turned(s["q"], cos, sin).to(s["q"].dtype)
    if case["op"] == "axes":
        s["k"][ids, :, row] = k.to(s["k"].dtype)
        s["v"][ids, :, row] = s["v_new"]
        return [s["k"], s["v"], q]
    _plain_store8(s, s["k"], s["k_scale"], k, ids, row)
    _plain_store8(s, s["v"], s["v_scale"], s["v_new"].float(), ids, row)
    return [s["k"], s["v"], s["k_scale"], s["v_scale"], q]


def _plain_store8(s, pool, scale, x, ids, row):
    """x [T, Hkv, D] into its pages in 8 bits; a page whose scale grows has its older rows rounded to the new one."""
    size = s["case"]["page"]
    peak = torch.zeros_like(scale).scatter_reduce_(0, ids[:, None].expand(x.shape[:2]), x.abs().amax(dim=-1), "amax")
    mantissa, exponent = torch.frexp(peak)
    exponent = torch.where(mantissa > 0.875, exponent - 8, exponent - 9)
    exponent = torch.where(peak > 0, exponent, torch.full_like(exponent, MIN_EXPONENT)).clamp(min=MIN_EXPONENT)
    fresh = torch.exp2(exponent.float())
    position = s["position"].long()
    first = s["table"].long().gather(1, (position // size)[:, None])[:, 0]
    older = position % size  # rows before the new ones in a sequence's first page
    before = torch.where((older > 0)[:, None], scale[first], torch.zeros_like(scale[first]))
    grown = torch.maximum(fresh[first], before)
    bits = pool.view(torch.uint8)
    block = bits[first].view(E4M3).float()
    moved = block * (scale[first] / grown)[:, :, None, None]
    old = (torch.arange(size, device="cuda")[None] < older[:, None])[:, None, :, None]
    bits[first] = torch.where(old, moved, block).to(E4M3).view(torch.uint8)
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, ids, True)
    scale.copy_(torch.where(touched[:, None], fresh, scale))
    scale[first] = grown
    bits[ids, :, row] = (x / scale[ids][:, :, None]).to(E4M3).view(torch.uint8)


def _views(pool):
    """Free pages, counts and list of a pool's state."""
    pages = (pool.shape[0] - HEADER) // 2
    return pool[:1], pool[HEADER:HEADER + pages], pool[HEADER + pages:]


def _plain_resize(table, pool, before, after, page):
    """Sequences of `before` rows become sequences of `after` rows: pages that nobody holds any more go to the end of
    the list in rising order, then missing ones are taken from its end, in the order of sequences and rows."""
    free, count, order = _views(pool)
    j = torch.arange(table.shape[1], device="cuda")[None]
    held, wanted = (-(-n.long() // page) for n in (before, after))
    drop = (j < held[:, None]) & (j >= wanted[:, None])
    ids = torch.where(drop, table, torch.zeros_like(table)).long()
    fewer = torch.zeros_like(count).scatter_add_(0, ids.flatten(), drop.int().flatten())
    empty = (fewer > 0) & (count == fewer)
    count.sub_(fewer)
    at = torch.cumsum(empty, 0) - 1 + free
    size = order.shape[0]
    keep = torch.cat([order, order[:1]])
    keep[torch.where(empty, at, torch.full_like(at, size))] = torch.arange(size, dtype=torch.int32, device="cuda")
    order.copy_(keep[:size])
    table.masked_fill_(drop, -1)
    top = free + empty.sum()
    take = (j >= held[:, None]) & (j < wanted[:, None])
    rank = (torch.cumsum(take.flatten(), 0) - 1).view(take.shape)
    given = take & (rank < top)
    got = order[(top - 1 - rank).clamp(0, size - 1)]
    table.copy_(torch.where(given, got, torch.where(take, torch.full_like(table, -1), table)))
    count.scatter_add_(0, torch.where(given, got, torch.zeros_like(got)).long().flatten(), given.int().flatten())
    free.copy_(top - given.sum())


def _plain_fork(s):
    page, table, kv_len = s["case"]["page"], s["table"], s["kv_len"]
    _plain_resize(table, s["pool"], kv_len, s["kept_len"], page)
    free, count, order = _views(s["pool"])
    parent, child = s["parent"].long(), s["child"].long()
    n = kv_len.long()[parent]
    full, rest = n // page, n % page
    j = torch.arange(table.shape[1], device="cuda")[None]
    shared = j < full[:, None]
    rows = table[parent]
    count.scatter_add_(0, torch.where(shared, rows, torch.zeros_like(rows)).long().flatten(), shared.int().flatten())
    rank = torch.cumsum(rest > 0, 0) - 1
    fresh = order[(free - 1 - rank).clamp(min=0)]
    last = rows.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    none = torch.full_like(fresh, -1)
    src, dst = torch.where(rest > 0, last, none), torch.where(rest > 0, fresh, none)
    mine = torch.where(shared, rows, table[child])
    table[child] = torch.where((j == full[:, None]) & (rest > 0)[:, None], fresh[:, None], mine)
    count.scatter_add_(0, torch.where(rest > 0, fresh, torch.zeros_like(fresh)).long(), (rest > 0).int())
    free.sub_((rest > 0).sum())
    kv_len[child] = n.int()
    copies = torch.stack([src, dst, rest.int()])
    # whole pages of every layer, the rows behind the sequence's own left as they are
    a, b = src.long().clamp(min=0), torch.where(rest > 0, dst, src).long().clamp(min=0)
    moved = (torch.arange(page, device="cuda")[None] < rest[:, None])[:, None, :, None]
    for x in ("k", "v"):
        s[x][:, b] = torch.where(moved, s[x][:, a], s[x][:, b])
    return [s["k"], s["v"], table, s["pool"], kv_len, copies]


def _plain_compact(s):
    page, keep = s["case"]["page"], s["keep"].long()
    b, i = _sequence(s["bounds"], keep.shape[0])
    to = s["position"].long()[b] + i
    a_page, a_row = s["table"].long()[b, keep // page], keep % page
    b_page, b_row = s["table"].long()[b, to // page], to % page
    if s["case"]["op"] == "compact":
        for x in ("k", "v"):
            s[x][:, b_page, :, b_row] = s[x][:, a_page, :, a_row]
        return [s["k"], s["v"]]
    for x in ("k", "v"):
        bits, scale = s[x].view(torch.uint8), s[x + "_scale"]
        rows = bits[:, a_page, :, a_row].view(E4M3).float() * scale[:, a_page].transpose(0, 1)[..., None]
        grown = scale.scatter_reduce(1, b_page[None, :, None].expand(scale.shape[0], -1, scale.shape[2]),
                                     scale[:, a_page], "amax")
        # pages that take rows, one entry for each: their other rows are rounded to the new scale
        block = bits[:, b_page].view(E4M3).float() * (scale / grown)[:, b_page][..., None, None]
        bits[:, b_page] = block.to(E4M3).view(torch.uint8)
        scale.copy_(grown)
        bits[:, b_page, :, b_row] = (rows / scale[:, b_page].transpose(0, 1)[..., None]).to(E4M3).view(torch.uint8)
    return [s["k"], s["v"], s["k_scale"], s["v_scale"]]


def run(s):
    case = s["case"]
    op, page = case["op"], case["page"]
    if not own:
        if op in ("tree", "tree8"):
            return _plain_tree(s)
        if op in ("axes", "axes8"):
            return _plain_axes(s)
        if op == "fork":
            return _plain_fork(s)
        if op in ("compact", "compact8"):
            return _plain_compact(s)
        _plain_resize(s["table"], s["pool"], s["high"], s["low"], page)
        _plain_resize(s["table"], s["pool"], s["low"], s["high"], page)
        return [s["table"], s["pool"]]
    import decode_attention_static_gb300 as da

    if op == "tree":
        return da.decode_attn_tree_fwd(s["q"], s["k"], s["v"], s["table"], s["kv_len"], token_start=s["bounds"],
                                       tree_mask=s["mask"], workspace=s["workspace"])
    if op == "tree8":
        return da.decode_attn_tree_q8_fwd(s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["kv_len"],
                                          token_start=s["bounds"], tree_mask=s["mask"], workspace=s["workspace"])
    if op == "axes":
        q = da.kvcache_append_paged_axes(s["k"], s["v"], s["k_new"], s["v_new"], s["table"], s["position"], s["places"],
                                         s["cos"], s["sin"], rope_axis=s["axis"], token_start=s["bounds"], q=s["q"])
        return [s["k"], s["v"], q]
    if op == "axes8":
        q = da.kvcache_append_paged_q8_axes(s["k"], s["v"], s["k_scale"], s["v_scale"], s["k_new"], s["v_new"],
                                            s["table"], s["position"], s["places"], s["cos"], s["sin"],
                                            rope_axis=s["axis"], token_start=s["bounds"], q=s["q"])
        return [s["k"], s["v"], s["k_scale"], s["v_scale"], q]
    if op == "fork":
        da.kvcache_resize_paged(s["table"], s["kv_len"], s["kept_len"], s["pool"], page)
        copies = da.kvcache_fork_paged(s["table"], s["kv_len"], s["parent"], s["child"], s["pool"], page)
        da.kvcache_copy_pages(s["k"], s["v"], copies)
        return [s["k"], s["v"], s["table"], s["pool"], s["kv_len"], copies]
    if op == "compact":
        da.kvcache_compact_paged(s["k"], s["v"], s["table"], s["keep"], s["bounds"], s["position"])
        return [s["k"], s["v"]]
    if op == "compact8":
        da.kvcache_compact_paged_q8(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["keep"], s["bounds"],
                                    s["position"])
        return [s["k"], s["v"], s["k_scale"], s["v_scale"]]
    da.kvcache_resize_paged(s["table"], s["high"], s["low"], s["pool"], page)
    da.kvcache_resize_paged(s["table"], s["low"], s["high"], s["pool"], page)
    return [s["table"], s["pool"]]


# ---------------------------------------------------------------------------
# The definitions in 64 bits


def _grid8(x):
    """x (64 bits) on the grid of e4m3: three bits after the leading one, steps of 2**-9 at least, ties to even."""
    exponent = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6)
    step = torch.exp2(exponent - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    op, page = case["op"], case["page"]
    old, new = counts(case)
    table = s["table"].cpu().tolist()

    def tree():
        Hkv, D = case["Hkv"], case["D"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        masks, at = trees(case)[0], 0
        for b, (n, m) in enumerate(zip(old, new)):
            if m == 0:
                continue
            rows = torch.arange(n + m, device="cuda")
            ids, row = s["table"][b].long()[rows // page], rows % page
            bits = torch.uint8 if op == "tree8" else torch.int16
            k, v = (s[x].view(bits)[ids, :, row].view(s[x].dtype).double() for x in ("k", "v"))  # [rows, Hkv, D]
            if op == "tree8":
                k, v = k * s["k_scale"][ids].double()[..., None], v * s["v_scale"][ids].double()[..., None]
            hidden = torch.tensor([[masks[at + i] >> j & 1 == 0 for j in range(m)] for i in range(m)], device="cuda")
            for g in range(Hkv):
                q = s["q"][at:at + m].double().view(m, Hkv, -1, D)[:, g]
                x = torch.einsum("mhd,rd->mhr", q, k[:, g]) * s["scale"]
                x[:, :, n:].masked_fill_(hidden[:, None], float("-inf"))
                G = q.shape[1]
                out[at:at + m, g * G:(g + 1) * G] = torch.einsum("mhr,rd->mhd", torch.softmax(x, dim=-1), v[:, g])
            at += m
        return out

    def axes():
        D, eight = case["D"], op == "axes8"
        k, v = s["k"].double(), s["v"].double()
        scales = [s["k_scale"].double(), s["v_scale"].double()] if eight else None
        q_out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        axis, at = s["axis"].tolist(), 0
        for b, (p0, m) in enumerate(zip(old, new)):
            cos, sin = (torch.stack([s[c][s["places"][a, at:at + m].long(), i].double() for i, a in enumerate(axis)],
                                    dim=1)[:, None] for c in ("cos", "sin"))

            def turned(x):
                x = x.double()
                a, c = x[..., :D // 2], x[..., D // 2:]
                return torch.cat([a * cos - c * sin, c * cos + a * sin], dim=-1)

            q_out[at:at + m] = turned(s["q"][at:at + m])
            rows = [turned(s["k_new"][at:at + m]), s["v_new"][at:at + m].double()]
            for j in range(p0 // page, (p0 + m - 1) // page + 1):
                lo, hi = max(p0, j * page), min(p0 + m, (j + 1) * page)
                where, r0, r1 = table[b][j], lo - j * page, hi - j * page
                for i, pool in enumerate((k, v)):
                    x = rows[i][lo - p0:hi - p0].transpose(0, 1)  # [Hkv, rows, D]
                    if not eight:
                        pool[where, :, r0:r1] = x
                        continue
                    scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(1, 2)) / E4M3_MAX)).clamp(min=MIN_EXPONENT))
                    if r0 > 0:
                        before = scales[i][where].clone()
                        scale = torch.maximum(scale, before)
                        pool[where, :, :r0] = _grid8(pool[where, :, :r0] * (before / scale)[:, None, None])
                    scales[i][where] = scale
                    pool[where, :, r0:r1] = _grid8(x / scale[:, None, None])
            at += m
        return [k, v, *scales, q_out] if eight else [k, v, q_out]

    def fork():
        k, v = s["k"].double(), s["v"].double()
        free = s["pool"][0].item()
        order = s["pool"][-k.shape[1]:].tolist()
        for p in new:
            if old[p] % page:
                free -= 1
                src, dst = table[p][old[p] // page], order[free]
                for pool in (k, v):
                    pool[:, dst, :, :old[p] % page] = pool[:, src, :, :old[p] % page]
        return [k, v, None, None, None, None]

    def compact():
        eight = op == "compact8"
        pools = [s["k"].double(), s["v"].double()]
        scales = [s["k_scale"].double(), s["v_scale"].double()] if eight else [None, None]
        for b, (n, rows) in enumerate(zip(old, kept(case))):
            for pool, scale in zip(pools, scales):
                for j in range(n // page, (n + len(rows) - 1) // page + 1):
                    moves = [(a, n + i) for i, a in enumerate(rows) if (n + i) // page == j]
                    dst = table[b][j]
                    got = torch.stack([pool[:, table[b][a // page], :, a % page] for a, _ in moves])
                    if eight:
                        from_scale = torch.stack([scale[:, table[b][a // page]] for a, _ in moves])
                        top = torch.maximum(scale[:, dst], from_scale.amax(dim=0))
                        pool[:, dst] = _grid8(pool[:, dst] * (scale[:, dst] / top)[..., None, None])
                        got = _grid8(got * (from_scale / top)[..., None])
                        scale[:, dst] = top
                    for (_, to), row in zip(moves, got):
                        pool[:, dst, :, to % page] = row
        return pools + scales if eight else pools

    if op in ("tree", "tree8"):
        return tree()
    if op in ("axes", "axes8"):
        return axes()
    if op == "fork":
        return fork()
    if op in ("compact", "compact8"):
        return compact()
    return None  # whole numbers alone

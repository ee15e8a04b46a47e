"""What the serving-cache operators cost, and what they compute.

Five operators around a decode cache: appending keys and values to a paged cache
with the rotary embedding on the way, the same into an 8-bit cache with one
scale per page and head, decode attention over either kind of page, and decode
attention with a sliding window and sinks over a static cache. ``run`` computes
them with elementary torch operations, or, where ``own`` is true, with the
framework's entry points.
"""
import math
import random

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3_MAX = 448.0
MIN_EXPONENT = -100  # smallest scale of a block: 2 ** MIN_EXPONENT


# ---------------------------------------------------------------------------
# Cases


def listed():
    return [
        # One decode step of a small batch: every sequence appends one rotated row. Latency.
        dict(name="append, 8 sequences, one token", op="append", B=8, H=16, Hkv=8, D=128, type="bf16", page=16,
             longest=1, reach=8192, lens=1),
        # Prompts of three requests, of odd lengths and starting inside a page, entering the cache at once.
        dict(name="append, prompts of 8k tokens", op="append", B=3, H=32, Hkv=8, D=128, type="f16", page=64,
             longest=4095, reach=16384, lens=2),
        # The decode step of a large batch into the 8-bit cache.
        dict(name="append 8 bits, 64 sequences, one token", op="append8", B=64, H=32, Hkv=8, D=128, type="bf16",
             page=16, longest=1, reach=8192, lens=3),
        # Prompts into the 8-bit cache: the largest append.
        dict(name="append 8 bits, prompts of 20k tokens", op="append8", B=5, H=32, Hkv=8, D=128, type="bf16", page=64,
             longest=8191, reach=8192, lens=4),
        # One user, multi-head attention, a short prefix: latency.
        dict(name="paged, 1 x 1024, 16/16 heads", op="paged", B=1, H=16, Hkv=16, D=128, type="f16", page=16,
             longest=1024, ragged=False, window=0, sinks=0, lens=5),
        # A streaming batch of ragged lengths with one idle slot.
        dict(name="paged, 8 ragged to 8191, 16/8 heads", op="paged", B=8, H=16, Hkv=8, D=128, type="bf16", page=16,
             longest=8191, ragged=True, window=0, sinks=0, lens=6, idle=1),
        # A serving batch with long contexts: the most bytes.
        dict(name="paged, 32 ragged to 32768, 32/8 heads", op="paged", B=32, H=32, Hkv=8, D=128, type="bf16", page=64,
             longest=32768, ragged=True, window=0, sinks=0, lens=7),
        # A small head dimension, four heads on one KV head, an odd length over small pages.
        dict(name="paged 8 bits, 1 x 4093, 4/1 heads, D 64", op="paged8", B=1, H=4, Hkv=1, D=64, type="f16", page=16,
             longest=4093, ragged=False, window=0, sinks=0, lens=8),
        # The same serving batch over the 8-bit cache.
        dict(name="paged 8 bits, 32 ragged to 32768, 32/8 heads", op="paged8", B=32, H=32, Hkv=8, D=128, type="bf16",
             page=64, longest=32768, ragged=True, window=0, sinks=0, lens=7),
        # The 8-bit cache under a window with sinks, eight heads on each KV head.
        dict(name="paged 8 bits, 16 ragged, 64/8 heads, window 4096", op="paged8", B=16, H=64, Hkv=8, D=128,
             type="bf16", page=32, longest=32768, ragged=True, window=4096, sinks=4, lens=10),
        # One user with a long context under a window, over the static cache.
        dict(name="window 4096 of 1 x 32768, 32/8 heads", op="window", B=1, H=32, Hkv=8, D=128, type="bf16",
             longest=32768, ragged=False, window=4096, sinks=4, lens=11),
        # A batch under an odd window that starts inside a tile.
        dict(name="window 1021 of 16 ragged to 16384, 16/8 heads", op="window", B=16, H=16, Hkv=8, D=128, type="f16",
             longest=16384, ragged=True, window=1021, sinks=16, lens=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append8", "paged", "paged8", "window"])
    group = rng.choice([1, 2, 4, 8])
    heads_kv = rng.choice([1, 2, 4, 5, 8, 16])
    case = dict(op=op, Hkv=heads_kv, H=heads_kv * group, D=rng.choice([64, 128, 128]), type=rng.choice(["f16", "bf16"]),
                lens=rng.randrange(1 << 20))
    if op in ("append", "append8"):
        case["page"] = rng.choice([16, 32, 64, 128])
        tokens = _log(rng, 1, 16384)
        if rng.random() < 0.4:
            case.update(B=_log(rng, 1, 256), longest=1, reach=_log(rng, 64, 16384))
        else:
            B = rng.randint(1, 8)
            case.update(B=B, longest=max(1, tokens // B), reach=_log(rng, 64, 16384))
        return case
    rows = _log(rng, 64, min(400000, 4000000 // heads_kv))  # cached rows of the batch
    B = _log(rng, 1, 64)
    longest = max(1, min(32768, rows // B))
    case.update(B=B, longest=longest, ragged=rng.random() < 0.7)
    if B > 2 and rng.random() < 0.3:
        case["idle"] = 1
    windowed = op == "window" or rng.random() < 0.4
    case.update(window=_log(rng, 1, max(2, longest)) if windowed else 0,
                sinks=rng.choice([0, 1, 4, 16, 37]) if windowed else 0)
    if op != "window":
        case["page"] = rng.choice([16, 32, 64, 128])
    return case


def lengths(case):
    """Rows of each sequence: new ones for an append, cached ones for the attention."""
    r = random.Random(case["lens"])
    B, longest = case["B"], case["longest"]
    if longest == 1:
        n = [1] * B
    elif case["op"] in ("append", "append8") or case.get("ragged"):
        n = [r.randint(max(1, longest // 8), longest) for _ in range(B)]
        n[r.randrange(B)] = longest
    else:
        n = [longest] * B
    if case.get("idle") and case["op"] not in ("append", "append8"):
        n[0 if n[0] != longest else B - 1] = 0
    return n


def starts(case):
    """First position of each sequence's new rows."""
    r = random.Random(case["lens"] + 1)
    return [r.randint(0, case["reach"] - 1) for _ in range(case["B"])]


def visible(case, n):
    w = case["window"]
    if w <= 0 or n <= w:
        return n
    return w + min(case["sinks"], n - w)


def work(case):
    n, H, Hkv, D = lengths(case), case["H"], case["Hkv"], case["D"]
    if case["op"] in ("append", "append8"):
        T = sum(n)
        at = {p + i for p, m in zip(starts(case), n) for i in range(m)}
        store = 2 if case["op"] == "append" else 1
        moved = 2 * T * Hkv * D * (2 + store) + 2 * T * H * D * 2 + len(at) * 2 * D * 4
        return {"bytes": moved, "flops": 3 * T * (H + Hkv) * D}
    rows = sum(visible(case, m) for m in n)
    element = 1 if case["op"] == "paged8" else 2
    return {"bytes": 2 * rows * Hkv * D * element + 2 * len(n) * H * D * 2, "flops": 4 * rows * H * D}


# ---------------------------------------------------------------------------
# Inputs


def _values(shape, gen, spread):
    """Normal values with a few wide channels, as keys have."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return x * spread


def _codes(shape, gen):
    """8-bit values of a block scaled to the type's range."""
    return (torch.randn(shape, generator=gen, device="cuda") * 100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def prepare(case, seed):
    def deal(rows):
        """Pages of the pool, dealt in a random order; -1 where a sequence has no page."""
        page = case["page"]
        need = [-(-r // page) for r in rows]
        total = sum(need)
        pool = total + 3
        order = torch.randperm(pool, generator=gen, device="cuda")[:total].to(torch.int32).cpu()
        table = torch.full((len(rows), max(1, max(need))), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = order[at:at + m]
            at += m
        return table.cuda(), pool

    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, H, Hkv, D, dt = case["B"], case["H"], case["Hkv"], case["D"], TYPES[case["type"]]
    n = lengths(case)
    spread = torch.ones(D, device="cuda")
    spread[torch.randint(0, D, (3,), generator=gen, device="cuda")] = 6.0
    s = dict(case=case, scale=D ** -0.5)
    int32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] in ("append", "append8"):
        first, T = starts(case), sum(n)
        table, pool = deal([p + m for p, m in zip(first, n)])
        shape = (pool, Hkv, case["page"], D)
        bounds = [0]
        for m in n:
            bounds.append(bounds[-1] + m)
        rows = max(p + m for p, m in zip(first, n))
        angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D))
        angle = torch.cat([angle, angle], dim=1)
        s.update(table=table, position=int32(first), bounds=None if case["longest"] == 1 else int32(bounds),
                 cos=angle.cos().float(), sin=angle.sin().float(),
                 k_new=_values((T, Hkv, D), gen, spread).to(dt), v_new=_values((T, Hkv, D), gen, 1.0).to(dt),
                 q=_values((T, H, D), gen, 1.0).to(dt))
        if case["op"] == "append":
            s.update(k=_values(shape, gen, 1.0).to(dt), v=_values(shape, gen, 1.0).to(dt))
        else:
            exps = lambda: torch.exp2(torch.randint(-9, -4, (pool, Hkv), generator=gen, device="cuda").float())  # noqa: E731
            s.update(k=_codes(shape, gen), v=_codes(shape, gen), k_scale=exps(), v_scale=exps())
        return s
    s["kv_len"] = int32(n)
    s["q"] = _values((B, H, D), gen, 1.0).to(dt)
    if case["op"] == "window":
        shape = (B, Hkv, case["longest"], D)
        s.update(k=_values(shape, gen, 1.0).to(dt), v=_values(shape, gen, 1.0).to(dt))
    else:
        s["table"], pool = deal(n)
        shape = (pool, Hkv, case["page"], D)
        if case["op"] == "paged":
            s.update(k=_values(shape, gen, 1.0).to(dt), v=_values(shape, gen, 1.0).to(dt))
        else:
            exps = lambda: torch.exp2(torch.randint(-8, -6, (pool, Hkv), generator=gen, device="cuda").float())  # noqa: E731
            s.update(k=_codes(shape, gen), v=_codes(shape, gen), k_scale=exps(), v_scale=exps())
    # the scratch that a program keeps for its attention calls
    s["workspace"] = torch.zeros(8 << 20, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# Plain forms


def _rotate(x, cos, sin):
    half = x.shape[-1] // 2
    x = x.float()
    return x * cos + torch.cat([-x[..., half:], x[..., :half]], dim=-1) * sin


def _places(s):
    """Position, page and row in the page of every new token, and its sequence."""
    page, T = s["case"]["page"], s["k_new"].shape[0]
    t = torch.arange(T, device="cuda")
    if s["bounds"] is None:
        b, at = t, s["position"].long()
    else:
        b = torch.searchsorted(s["bounds"][1:].contiguous(), t, right=True)
        at = s["position"].long()[b] + t - s["bounds"].long()[b]
    return at, s["table"].long()[b, at // page], at % page


def _plain_append(s):
    at, page, row = _places(s)
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    dt = s["k_new"].dtype
    k, v = _rotate(s["k_new"], cos, sin), s["v_new"]
    q = _rotate(s["q"], cos, sin).to(dt)
    if s["case"]["op"] == "append":
        s["k"][page, :, row] = k.to(dt)
        s["v"][page, :, row] = v
        return [s["k"], s["v"], q]
    _plain_store8(s, s["k"], s["k_scale"], k, page, row)
    _plain_store8(s, s["v"], s["v_scale"], v.float(), page, row)
    return [s["k"], s["v"], s["k_scale"], s["v_scale"], q]


def _plain_store8(s, pool, scale, x, page, row):
    """x [T, Hkv, D] into its pages in 8 bits; a page whose scale grows has its older rows rounded to the new one."""
    size = s["case"]["page"]
    peak = x.abs().nan_to_num(nan=0.0, posinf=0.0).amax(dim=-1)
    peak = torch.zeros_like(scale).scatter_reduce_(0, page[:, None].expand_as(peak), peak, "amax")
    mantissa, exponent = torch.frexp(peak)
    exponent = torch.where(mantissa > 0.875, exponent - 8, exponent - 9)
    exponent = torch.where(peak > 0, exponent, torch.full_like(exponent, MIN_EXPONENT)).clamp(min=MIN_EXPONENT)
    fresh = torch.exp2(exponent.float())
    # the first page of each sequence may hold older rows: its scale never shrinks
    position = s["position"].long()
    first = s["table"].long().gather(1, (position // size)[:, None])[:, 0]
    kept = position % size
    old = torch.where((kept > 0)[:, None], scale[first], torch.zeros_like(scale[first]))
    grown = torch.maximum(fresh[first], old)
    older = (torch.arange(size, device="cuda")[None] < kept[:, None])[:, None, :, None]
    bits = pool.view(torch.uint8)
    block = bits[first].view(pool.dtype).float()
    moved = block * (scale[first] / grown)[:, :, None, None]
    bits[first] = torch.where(older, moved, block).to(pool.dtype).view(torch.uint8)
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, page, True)
    scale.copy_(torch.where(touched[:, None], fresh, scale))
    scale[first] = grown
    x = x / scale[page][:, :, None]
    x = torch.where(x.isfinite(), x, torch.full_like(x, float("nan")))
    bits[page, :, row] = x.to(pool.dtype).view(torch.uint8)


def _plain_attention(s):
    case = s["case"]
    if case["op"] == "window":
        k, v = s["k"].float(), s["v"].float()
    else:
        ids = s["table"].long().clamp(min=0)
        if case["op"] == "paged8":
            k, v = ((s[x].view(torch.uint8)[ids].view(s[x].dtype).float() * s[x + "_scale"][ids][..., None, None])
                    for x in ("k", "v"))
        else:
            k, v = s["k"][ids].float(), s["v"][ids].float()  # [B, pages, Hkv, page, D]
        k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))
    B, Hkv, L, D = k.shape
    q = s["q"].float().view(B, Hkv, -1, D)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    j, n = torch.arange(L, device="cuda")[None], s["kv_len"].long()[:, None]
    seen = j < n
    if case["window"] > 0:
        seen = seen & ((j >= n - case["window"]) | (j < case["sinks"]))
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    top = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(top.isfinite(), top, torch.zeros_like(top)))
    total = p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return out.reshape(B, -1, D).to(s["q"].dtype)


def run(s):
    case = s["case"]
    if not own:
        return _plain_append(s) if case["op"] in ("append", "append8") else _plain_attention(s)
    import decode_attention_static_gb300 as da

    if case["op"] == "append":
        q = da.kvcache_append_paged(s["k"], s["v"], s["k_new"], s["v_new"], s["table"], s["position"],
                                    token_start=s["bounds"], rope_cos=s["cos"], rope_sin=s["sin"], q=s["q"])
        return [s["k"], s["v"], q]
    if case["op"] == "append8":
        q = da.kvcache_append_paged_q8(s["k"], s["v"], s["k_scale"], s["v_scale"], s["k_new"], s["v_new"], s["table"],
                                       s["position"], token_start=s["bounds"], rope_cos=s["cos"], rope_sin=s["sin"],
                                       q=s["q"])
        return [s["k"], s["v"], s["k_scale"], s["v_scale"], q]
    if case["op"] == "paged":
        return da.decode_attn_paged_fwd(s["q"], s["k"], s["v"], s["table"], s["kv_len"], window=case["window"],
                                        sinks=case["sinks"], workspace=s["workspace"])
    if case["op"] == "paged8":
        return da.decode_attn_paged_q8_fwd(s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["kv_len"],
                                           window=case["window"], sinks=case["sinks"], workspace=s["workspace"])
    return da.decode_attn_window_fwd(s["q"], s["k"], s["v"], s["kv_len"], case["window"], sinks=case["sinks"],
                                     workspace=s["workspace"])


# ---------------------------------------------------------------------------
# The definitions in 64 bits


def _grid8(x):
    """x (64 bits) on the grid of e4m3: three bits after the leading one, steps of 2**-9 at least, ties to even."""
    exponent = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6)
    step = torch.exp2(exponent - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)

    def append():
        size = case["page"]
        n, first = lengths(case), starts(case)
        D = case["D"]
        k, v = s["k"].double(), s["v"].double()
        eight = case["op"] == "append8"
        scales = [s["k_scale"].double(), s["v_scale"].double()] if eight else None
        q_out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        table = s["table"].cpu().tolist()
        at = 0
        for b, (m, p0) in enumerate(zip(n, first)):
            cos, sin = (s[c][p0:p0 + m].double()[:, None] for c in ("cos", "sin"))

            def turned(x):
                x = x.double()
                a, c = x[..., :D // 2], x[..., D // 2:]
                return torch.cat([a * cos[..., :D // 2] - c * sin[..., :D // 2],
                                  c * cos[..., D // 2:] + a * sin[..., D // 2:]], dim=-1)

            q_out[at:at + m] = turned(s["q"][at:at + m])
            new = [turned(s["k_new"][at:at + m]), s["v_new"][at:at + m].double()]
            for j in range(p0 // size, (p0 + m - 1) // size + 1):
                lo, hi = max(p0, j * size), min(p0 + m, (j + 1) * size)
                page, r0, r1 = table[b][j], lo - j * size, hi - j * size
                for i, pool in enumerate((k, v)):
                    rows = new[i][lo - p0:hi - p0].transpose(0, 1)  # [Hkv, rows, D]
                    if not eight:
                        pool[page, :, r0:r1] = rows
                        continue
                    need = torch.ceil(torch.log2(rows.abs().amax(dim=(1, 2)) / E4M3_MAX)).clamp(min=MIN_EXPONENT)
                    scale = torch.exp2(need)
                    if r0 > 0:
                        before = scales[i][page].clone()
                        scale = torch.maximum(scale, before)
                        pool[page, :, :r0] = _grid8(pool[page, :, :r0] * (before / scale)[:, None, None])
                    scales[i][page] = scale
                    pool[page, :, r0:r1] = _grid8(rows / scale[:, None, None])
            at += m
        return [k, v, *scales, q_out] if eight else [k, v, q_out]

    def attention():
        B, H, Hkv, D = case["B"], case["H"], case["Hkv"], case["D"]
        out = torch.zeros(B, H, D, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lengths(case)):
            if n == 0:
                continue
            rows = torch.arange(n, device="cuda")
            if case["window"] > 0:
                rows = rows[(rows >= n - case["window"]) | (rows < case["sinks"])]
            if case["op"] == "window":
                k, v = s["k"][b][:, rows].double(), s["v"][b][:, rows].double()
            else:
                page, row = s["table"][b].long()[rows // case["page"]], rows % case["page"]
                bits = torch.uint8 if case["op"] == "paged8" else torch.int16
                k, v = (s[x].view(bits)[page, :, row].view(s[x].dtype).double() for x in ("k", "v"))  # [rows, Hkv, D]
                if case["op"] == "paged8":
                    k = k * s["k_scale"][page].double()[..., None]
                    v = v * s["v_scale"][page].double()[..., None]
                k, v = k.transpose(0, 1), v.transpose(0, 1)
            q = s["q"][b].double().view(Hkv, H // Hkv, D)
            p = torch.softmax(torch.einsum("hgd,hrd->hgr", q, k) * s["scale"], dim=-1)
            out[b] = torch.einsum("hgr,hrd->hgd", p, v).reshape(H, D)
        return out

    return append() if case["op"] in ("append", "append8") else attention()

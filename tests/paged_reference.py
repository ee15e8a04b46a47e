"""Plain 64-bit forms of the paged-cache and sliding-window operators, the
error that the kernels' number formats allow, and the inputs of their tests.
CPU only; shares nothing with the library."""
from __future__ import annotations

import math

import torch

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
NAN = float("nan")


def visible_rows(n: int, window: int, sinks: int) -> torch.Tensor:
    j = torch.arange(n)
    return j if window <= 0 else j[(j >= n - window) | (j < sinks)]


def attend(q, k, v, scale):
    """softmax(scale q k^T) v in 64 bits, and how far a kernel may be off.

    q [H, D], k and v [Hkv, n, D] (64 bits, the exact values). The allowance,
    before the rounding to the output type, per output element: with x a
    score, weights err by 2 |dx| relative (numerator and sum), where the dot
    product of D exact products summed in 32 bits (rounded or truncated, half a
    step or a whole one of 2^-23 each) errs by (D + 8) 2^-23 sum|q k|, the
    query's own rounding to an 11-bit format relative to its largest element
    by 2^-25 max|q| sum|k|, and the score's two roundings and the base-2
    exponential by 2^-22 |x| + 2^-20. The sum over n rows, 16 to a step and in
    up to 2 x 152 x 8 parts, errs by (n / 16 + 64) 2^-23 of sum p|v| (a partial
    sum never exceeds it), and weights held in two 8-bit pieces by half a step
    of the second, 2^-18, of it."""
    H, D = q.shape
    Hkv, n, _ = k.shape
    qg = q.view(Hkv, H // Hkv, D)
    x = torch.einsum("hgd,hnd->hgn", qg, k) * scale
    p = torch.softmax(x, dim=-1)
    out = torch.einsum("hgn,hnd->hgd", p, v).reshape(H, D)
    mass = torch.einsum("hgn,hnd->hgd", p, v.abs())
    size = torch.einsum("hgd,hnd->hgn", qg.abs(), k.abs()).amax(-1, keepdim=True)
    peak = qg.abs().amax(-1, keepdim=True) * k.abs().sum(-1).amax(-1)[:, None, None]
    dx = abs(scale) * ((D + 8) * 2.0 ** -23 * size + 2.0 ** -25 * peak)
    dx = dx + 2.0 ** -22 * x.abs().amax(-1, keepdim=True) + 2.0 ** -20
    slack = (2.1 * dx + (n / 16 + 64) * 2.0 ** -23 + 2.0 ** -18) * mass
    return out, slack.reshape(H, D)


def assert_rows(got: torch.Tensor, ref: torch.Tensor, slack: torch.Tensor, what: str = "") -> None:
    """got (16-bit) against ref: the slack, then one rounding of half a step
    (in the subnormal range half the smallest one)."""
    info = torch.finfo(got.dtype)
    g = got.double().cpu()
    allowed = slack * (1 + info.eps) + ref.abs() * info.eps / 2 + info.smallest_normal * info.eps / 2
    off = (g - ref).abs()
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    assert (off <= allowed).all(), f"{what}: off by {(off / allowed).max().item():.3f} of what is allowed"


def deal_pages(lens, page, gen, spare=2):
    """Random pages for sequences of `lens` rows: (table int32 [B, max_pages]
    with -1 where nothing is mapped, pool size)."""
    need = [-(-n // page) for n in lens]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=gen)
    table = torch.full((len(lens), max(1, max(need, default=1))), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m].to(torch.int32)
        at += m
    return table, pool


def grid8(x: torch.Tensor) -> torch.Tensor:
    """64-bit values to the nearest e4m3 one, ties to even."""
    exponent = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6)
    step = torch.exp2(exponent - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def rotate32(x, cos, sin):
    """The rotary embedding in 32 bits, products and sum rounded apart."""
    half = x.shape[-1] // 2
    x = x.float()
    return x * cos + torch.cat([-x[..., half:], x[..., :half]], dim=-1) * sin


def block_scale(x: torch.Tensor) -> float:
    """Smallest power of two s, at least 2^-100, with every finite |x| <= 448 s."""
    finite = x.double().abs()
    finite = finite[torch.isfinite(finite)]
    peak = float(finite.max()) if finite.numel() else 0.0
    if peak == 0.0:
        return 2.0 ** -100
    m, e = math.frexp(peak)  # 448 = 0.875 * 2^9
    return 2.0 ** max(-100, e - (8 if m > 0.875 else 9))


def append(k_pages, v_pages, k_new, v_new, table, position, start=None, cos=None, sin=None, q=None, k_scale=None,
           v_scale=None, limit=None):
    """The append on CPU tensors, in place; returns the rotated q. 16-bit
    pages, or e4m3 ones with their scales."""
    size = k_pages.shape[2]
    limit = table.shape[1] * size if limit is None else limit
    q_out = None if q is None else torch.full_like(q, 7.0)
    pages = k_pages.shape[0]
    for b in range(table.shape[0]):
        lo, hi = (b, b + 1) if start is None else (int(start[b]), int(start[b + 1]))
        n, p0 = hi - lo, int(position[b])
        if n == 0:
            continue
        if p0 < 0 or p0 + n > limit:
            if q is not None:
                q_out[lo:hi] = NAN
            continue
        new = [k_new[lo:hi].float(), v_new[lo:hi].float()]
        if cos is not None:
            c, s = cos[p0:p0 + n, None], sin[p0:p0 + n, None]
            new[0] = rotate32(k_new[lo:hi], c, s)
            if q is not None:
                q_out[lo:hi] = rotate32(q[lo:hi], c, s).to(q.dtype)
        for j in range(p0 // size, (p0 + n - 1) // size + 1):
            a, z = max(p0, j * size), min(p0 + n, (j + 1) * size)
            page, r0, r1 = int(table[b, j]), a - j * size, z - j * size
            if page < 0 or page >= pages:
                continue
            for i, (pool, scale) in enumerate(((k_pages, k_scale), (v_pages, v_scale))):
                rows = new[i][a - p0:z - p0].transpose(0, 1)  # [Hkv, rows, D]
                if scale is None:
                    pool[page, :, r0:r1] = rows.to(pool.dtype)
                    continue
                for g in range(pool.shape[1]):
                    s = block_scale(rows[g])
                    if r0 > 0:
                        before = float(scale[page, g])
                        s = max(s, before)
                        if s != before:
                            old = pool[page, g, :r0].double()
                            moved = grid8(old * (before / s))
                            pool[page, g, :r0] = torch.where(old.isnan(), old, moved).float().to(E4M3)
                    scale[page, g] = s
                    x = rows[g].double()
                    pool[page, g, r0:r1] = torch.where(x.isfinite(), grid8(x / s), torch.full_like(x, NAN)).float().to(E4M3)
    return q_out


def bits(t: torch.Tensor) -> torch.Tensor:
    """The storage of a tensor as integers, on the CPU."""
    t = t.detach().cpu().contiguous()
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def randn(shape, dtype, gen, spread=1.0):
    return (torch.randn(*shape, generator=gen) * spread).to(dtype)

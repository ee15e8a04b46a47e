"""Plain forms of the operators for drafted tokens and for pages, with the error
that the kernels' number formats allow. CPU only; shares nothing with the library."""
from __future__ import annotations

import torch

import paged_reference as R

HEADER = 4


# ---------------------------------------------------------------------------
# Tree attention


def seen_rows(n: int, m: int, masks) -> torch.Tensor:
    """[m, n] truth values: which of n rows the m last ones' tokens see. masks:
    one int for each token (bit i: the i-th of them), or None for a chain."""
    base = n - m
    seen = torch.zeros(m, n, dtype=torch.bool)
    seen[:, :base] = True
    for i in range(m):
        for j in range(m):
            seen[i, base + j] = j <= i if masks is None else bool(masks[i] >> j & 1)
    return seen


def words_of(masks, words: int) -> torch.Tensor:
    """Masks as int64 [tokens, words]."""
    flat = [m >> 64 * w & (1 << 64) - 1 for m in masks for w in range(words)]
    return torch.tensor([f - (1 << 64) if f >> 63 else f for f in flat], dtype=torch.int64).view(len(masks), words)


def attend_seen(q, k, v, seen, scale, weight_step):
    """softmax(scale q k^T) v over the rows seen, in 64 bits, and how far a
    kernel may be off.

    q [m, H, D], k and v [Hkv, n, D] (64 bits, the exact values), seen [m, n].
    The allowance before the rounding to the output type is that of
    paged_reference.attend (scores from exact products summed in 32 bits, an
    11-bit query where it is given to one, the base-2 exponential, sums over n
    rows truncated at 2^-23), with these sums in one accumulator of the n / 16
    steps of a tile's rows and rescaled by running maxima (two roundings, of
    which each is 2^-24, for at most n / 128 tiles: within the n / 16 + 64
    steps counted there), and with weights rounded once to the storage type:
    half a step, weight_step = 2^-8 (bf16) or 2^-11 (fp16), of each, so of sum
    p|v| at most. An fp16 weight below its smallest normal number errs by at most
    2^-25; weights are scaled so that a row's largest one is at least 2^7: 2^-32
    max|v| for each row seen."""
    m, H, D = q.shape
    Hkv, n, _ = k.shape
    G = H // Hkv
    out, slack = torch.zeros(m, H, D).double(), torch.zeros(m, H, D).double()
    for i in range(m):
        rows = seen[i].nonzero()[:, 0]
        if len(rows) == 0:
            continue
        out[i], slack[i] = R.attend(q[i], k[:, rows], v[:, rows], scale)
        kk, vv = k[:, rows], v[:, rows]
        p = torch.softmax(torch.einsum("hgd,hnd->hgn", q[i].view(Hkv, G, D), kk) * scale, dim=-1)
        mass = torch.einsum("hgn,hnd->hgd", p, vv.abs()).reshape(H, D)
        slack[i] += weight_step * mass
        if weight_step < 2.0 ** -9:
            slack[i] += len(rows) * 2.0 ** -32 * vv.abs().amax(dim=1)[:, None].expand(Hkv, G, D).reshape(H, D)
    return out, slack


# ---------------------------------------------------------------------------
# Append by axes


def turn_rows(rope_position_ids, rope_axis, D):
    """Table row of every (token, element): [tokens, D]."""
    axis = torch.zeros(D // 2, dtype=torch.long) if rope_axis is None else rope_axis.long()
    return rope_position_ids.long()[axis].t().repeat(1, 2)


def append_axes(k_pages, v_pages, k_new, v_new, table, position, start, cos, sin, rope_position_ids, rope_axis, q=None,
                k_scale=None, v_scale=None):
    """The append on CPU tensors, in place; returns the rotated q. It is the plain
    append of vectors that have been rotated before, token by token (so that it
    rounds them once more only where that is exact: the rotated values go
    through 32 bits)."""
    D, rows = k_new.shape[2], cos.shape[0]
    places = turn_rows(rope_position_ids, rope_axis, D)
    fine = ((rope_position_ids >= 0) & (rope_position_ids < rows)).all(dim=0)
    turn = places.clamp(0, rows - 1)
    column = torch.arange(D)
    c, s = cos[turn, column][:, None], sin[turn, column][:, None]
    turned = R.rotate32(k_new, c, s)
    q_out = None if q is None else torch.full_like(q, 7.0)
    if q is not None:
        q_all = R.rotate32(q, c, s).to(q.dtype)
    for b in range(table.shape[0]):
        lo, hi = (b, b + 1) if start is None else (int(start[b]), int(start[b + 1]))
        p0, n = int(position[b]), hi - lo
        if n == 0:
            continue
        ok = p0 >= 0 and p0 + n <= table.shape[1] * k_pages.shape[2]
        if q is not None:
            q_out[lo:hi] = q_all[lo:hi] if ok else R.NAN
            q_out[lo:hi][~fine[lo:hi]] = R.NAN
        if not ok:
            continue
        _store(k_pages, v_pages, k_scale, v_scale, [turned[lo:hi], v_new[lo:hi].float()], fine[lo:hi], table[b], p0)
    return q_out


def _store(k_pages, v_pages, k_scale, v_scale, new, fine, pages_of, p0):
    size, n = k_pages.shape[2], new[0].shape[0]
    for j in range(p0 // size, (p0 + n - 1) // size + 1):
        a, z = max(p0, j * size), min(p0 + n, (j + 1) * size)
        page = int(pages_of[j])
        if page < 0 or page >= k_pages.shape[0]:
            continue
        rows = [r for r in range(a, z) if fine[r - p0]]
        for i, (pool, scale) in enumerate(((k_pages, k_scale), (v_pages, v_scale))):
            x = new[i][[r - p0 for r in rows]].transpose(0, 1)  # [Hkv, rows, D]
            at = torch.tensor([r - j * size for r in rows], dtype=torch.long)
            if scale is None:
                pool[page][:, at] = x.to(pool.dtype)
                continue
            r0 = a - j * size
            for g in range(pool.shape[1]):
                t = R.block_scale(x[g])
                if r0 > 0:
                    before = float(scale[page, g])
                    t = max(t, before)
                    if t != before:
                        old = pool[page, g, :r0].double()
                        pool[page, g, :r0] = torch.where(old.isnan(), old, R.grid8(old * (before / t))).float().to(R.E4M3)
                scale[page, g] = t
                y = x[g].double()
                bits = torch.where(y.isfinite(), R.grid8(y / t), torch.full_like(y, R.NAN)).float().to(R.E4M3)
                pool.view(torch.uint8)[page, g, at] = bits.view(torch.uint8)


# ---------------------------------------------------------------------------
# Pages


class Pool:
    """A pool's state as the header describes it."""

    def __init__(self, num_pages, free=None, counts=None):
        self.n = num_pages
        self.list = list(range(num_pages)) if free is None else list(free) + [0] * (num_pages - len(free))
        self.free = num_pages if free is None else len(free)
        self.counts = [0] * num_pages if counts is None else list(counts)
        self.errors = set()

    def tensor(self):
        return torch.tensor([self.free, 0, 0, 0] + self.counts + self.list, dtype=torch.int32)

    def take(self):
        if self.free == 0:
            self.errors.add("full")
            return -1
        self.free -= 1
        page = self.list[self.free]
        self.counts[page] += 1
        return page

    def release(self, ids):
        """Lower counts; the pages that become free, in rising order, to the list."""
        freed = set()
        for page in ids:
            if page < 0 or page >= self.n:
                if page != -1:
                    self.errors.add("page")
            elif self.counts[page] < 1:
                self.errors.add("pool")
            else:
                self.counts[page] -= 1
                if self.counts[page] == 0:
                    freed.add(page)
        for page in sorted(freed):
            self.list[self.free] = page
            self.free += 1


def resize(table, held, wanted, pool, size):
    most = len(table[0]) * size
    spans = []
    for h, w in zip(held, wanted):
        if not (0 <= h <= most and 0 <= w <= most):
            pool.errors.add("kv_len")
            h = w = 0
        spans.append((-(-h // size), -(-w // size)))
    dropped = []
    for row, (h, w) in zip(table, spans):
        for j in range(w, h):
            dropped.append(row[j])
            row[j] = -1
    pool.release(dropped)
    for row, (h, w) in zip(table, spans):
        for j in range(h, w):
            row[j] = pool.take()


def fork(table, kv_len, parent, child, pool, size):
    """copies, as three lists."""
    B, most, n = len(table), len(table[0]) * size, len(parent)
    copies = [[-1] * n, [-1] * n, [0] * n]
    good = []
    for i, (p, c) in enumerate(zip(parent, child)):
        ok = 0 <= p < B and 0 <= c < B and child.count(c) == 1 and p not in child
        if not ok:
            pool.errors.add("sequence")
        elif not 0 <= kv_len[p] <= most:
            pool.errors.add("kv_len")
            ok = False
        good.append(ok)
    for i, (p, c) in enumerate(zip(parent, child)):
        if not good[i]:
            continue
        full, rest = divmod(kv_len[p], size)
        new, there = -1, rest > 0 and 0 <= table[p][full] < pool.n
        if there:
            new = pool.take()
            if new < 0:
                continue
        for j in range(full):
            page = table[p][j]
            table[c][j] = page
            if 0 <= page < pool.n:
                pool.counts[page] += 1
            else:
                pool.errors.add("page")
        if rest:
            table[c][full] = new
            if there:
                copies[0][i], copies[1][i], copies[2][i] = table[p][full], new, rest
            else:
                pool.errors.add("page")
        kv_len[c] = kv_len[p]
    return copies


def copy_pages(pools, copies):
    """pools: [layers, pages, ...] tensors (scales have no rows), in place."""
    for src, dst, rows in zip(*copies):
        if src < 0 or dst < 0 or src == dst:
            continue
        for t in pools:
            if t.dim() == 5:
                t[:, dst, :, :rows] = t[:, src, :, :rows]
            else:
                t[:, dst] = t[:, src]


def compact(pools, table, keep, start, position, size, scales=(None, None)):
    """pools: K and V [layers, pages, Hkv, size, D] (as integers of their bits in
    16 bits; e4m3 with scales [layers, pages, Hkv]), in place. Returns errors."""
    errors = set()
    pages, limit = pools[0].shape[1], table.shape[1] * size
    for b in range(table.shape[0]):
        s0, s1, p0 = int(start[b]), int(start[b + 1]), int(position[b])
        if s0 < 0 or s1 < s0 or s1 > len(keep):
            errors.add("tokens")
            continue
        moves, last = [], p0 - 1
        for i, row in enumerate(keep[s0:s1].tolist()):
            if p0 < 0 or row <= last or row < p0 + i or row >= limit:
                errors.add("position")
                break
            last = row
            moves.append((row, p0 + i))
        for pool, scale in zip(pools, scales):
            was, was_scale = pool.clone(), None if scale is None else scale.clone()
            for j in sorted({to // size for _, to in moves}):
                dst = int(table[b, j])
                here = [(a, to) for a, to in moves if to // size == j]
                if not 0 <= dst < pages:
                    if scale is None:
                        errors.update("page" for a, to in here if a != to)
                    else:
                        errors.add("page")
                    continue
                got = []
                for a, to in here:
                    src = int(table[b, a // size])
                    if not 0 <= src < pages:
                        errors.add("page")
                    elif a != to or scale is not None:
                        got.append((src, a % size, to % size))
                if scale is None:
                    for src, x, y in got:
                        pool[:, dst, :, y] = was[:, src, :, x]
                    continue
                own = was_scale[:, dst]
                top = own.clone()
                for src, _, _ in got:
                    top = torch.maximum(top, was_scale[:, src])

                def moved(codes, old):
                    ratio = (old / top)[..., None]
                    x = codes.double() * ratio.double()
                    y = torch.where(x.isnan(), x, R.grid8(x)).float().to(R.E4M3)
                    same = (old == top)[..., None].expand(codes.shape)
                    return torch.where(same, codes.view(torch.uint8), y.view(torch.uint8))

                bits = pool.view(torch.uint8)
                for r in range(size):
                    bits[:, dst, :, r] = moved(was[:, dst, :, r], own)
                for src, x, y in got:
                    bits[:, dst, :, y] = moved(was[:, src, :, x], was_scale[:, src])
                scale[:, dst] = top
    return errors

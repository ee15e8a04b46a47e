"""The rule by which a paged or window attention call is divided (csrc/
cache_attn.cuh), restated, so that tests can tell which way a batch takes."""
from __future__ import annotations

import numpy as np

F = np.float32


def ways(lens, n_kv_head, D, eight, window=0, sinks=0, sms=152):
    """("teams", warps), ("even", CTAs of each group) or ("shares", CTAs), and
    the number of scans over the lengths."""
    rows = 16 if (D if eight else 2 * D) > 128 else 32
    warps = 12 if eight and D == 64 else 8
    join_turns = 1 if eight else 3
    count = []
    for n in lens:
        w0 = n - window if 0 < window < n else 0
        first = w0 // rows
        count.append(min(-(-min(sinks, w0) // rows), first) + -(-n // rows) - first if n else 0)
    tiles, groups, most = sum(count) * n_kv_head, sum(c > 0 for c in count) * n_kv_head, max(count)
    scans = -(-len(lens) // (warps * 32))
    if groups > sms:
        each = F(1) / F(sms * warps)
        least, team = F(tiles) * each + F(groups) * each * F(warps) + F(6), 0
        for t in (1, 2, 4):
            cost = np.ceil((F(groups) - F(0.5)) * each * F(t)) * F((most + t - 1) // t + 1)
            if cost <= least:
                least, team = cost, t
        if team:
            return ("teams", team), scans
    ctas = min(sms, -(-tiles // 8))
    if 0 < groups <= sms:
        fit = sms // groups
        turns = -(-most // (warps * fit))
        each = 1 if most <= warps * (turns + join_turns) else -(-most // (warps * turns))
        part = -(-most // each)
        if part * ctas * 7 <= (tiles + ctas * (48 if each == 1 else 12)) * 8:
            return ("even", each), scans
    return ("shares", ctas), scans

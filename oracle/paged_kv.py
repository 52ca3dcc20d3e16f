"""A serving step over 16-bit and FP8 paged caches: block tables and slot maps, rotary positions, the
cache write and decode attention, in plain Python and float64.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py). Written from the definitions; no counterpart on the
source pages.
"""

import math

import numpy as np

from . import formats


def plan_step(context, query, table, free, cursor, block_size, num_blocks, T, rows=None, batch=None):
    """Request by request. table, batch: int arrays, changed in place. Returns (seq_lens, starts, positions, slots,
    cursor, flags)."""
    B = len(context)
    cap = table.shape[1] * block_size
    rows = list(range(B)) if rows is None else list(rows)
    flags, seq, starts, pos, slots = 0, [], [0], [], []
    for b in range(B):
        c, n = int(context[b]), 1 if query is None else int(query[b])
        if c < 0 or n < 0:
            flags |= 2
        c, n = max(c, 0), max(n, 0)
        if c + n > cap:
            flags |= 2
        L = min(c + n, cap)
        c = min(c, cap)
        row = rows[b]
        seq.append(L)
        starts.append(starts[-1] + n)
        if not 0 <= row < table.shape[0]:
            flags |= 1
            pos += range(c, c + n)
            slots += [-1] * n
            continue
        need = -(-L // block_size)
        if free is not None:
            for j in range(-(-c // block_size), need):
                if cursor >= len(free):
                    flags |= 32
                    table[row, j] = -1
                else:
                    ok = 0 <= free[cursor] < num_blocks
                    table[row, j] = free[cursor] if ok else -1
                    flags |= 0 if ok else 1
                    cursor += 1
        if batch is not None:
            batch[b, :need] = table[row, :need]
        for p in range(c, c + n):
            pos.append(p)
            block = int(table[row, p // block_size]) if p < L else -1
            held = free is None or p // block_size < -(-c // block_size)
            if p < L and held and not 0 <= block < num_blocks and len(slots) < T:
                flags |= 1
            slots.append(block * block_size + p % block_size if 0 <= block < num_blocks else -1)
    if len(pos) > T:
        flags |= 2
    pos, slots = (x[:T] + [-1] * (T - len(x)) for x in (pos, slots))
    return np.array(seq), np.array(starts), np.array(pos), np.array(slots), cursor, flags


def angles(positions, freqs):
    """positions [T] and freqs [R / 2] (phase advance a position in 2^-64 turns) -> radians [T, R / 2] in (-pi, pi]."""
    turns = [[((int(p) * int(f)) % (1 << 64)) / 2.0 ** 64 for f in freqs] for p in positions]
    turns = np.array(turns).reshape(len(positions), len(freqs))
    return 2 * math.pi * (turns - np.round(turns))


def rotate(x, positions, freqs, interleaved, factor):
    """x [T, H, D] float64 -> rotated, and the size |a| + |b| of each element's pair (for error bounds)."""
    R = 2 * len(freqs)
    a = angles(positions, freqs)[:, None]
    y, size = np.array(x, np.float64), np.abs(np.array(x, np.float64))
    first, second = (np.arange(0, R, 2), np.arange(1, R, 2)) if interleaved else (np.arange(R // 2), np.arange(R // 2, R))
    u, v = x[..., first], x[..., second]
    y[..., first] = (u * np.cos(a) - v * np.sin(a)) * factor
    y[..., second] = (v * np.cos(a) + u * np.sin(a)) * factor
    size[..., first] = size[..., second] = (np.abs(u) + np.abs(v)) * abs(factor)
    return y, size


def e4m3(x):
    """The values that float64 x rounds to in E4M3FN (nearest, ties to even, saturating), one rounding."""
    vals = formats.e4m3fn_to_f64(np.arange(0x7F, dtype=np.uint8))
    a = np.abs(x)
    hi = np.clip(np.searchsorted(vals, a), 0, len(vals) - 1)
    lo = np.clip(hi - 1, 0, None)
    near_lo = (a - vals[lo] < vals[hi] - a) | ((a - vals[lo] == vals[hi] - a) & (lo % 2 == 0))
    y = np.where(a >= 448, 448.0, vals[np.where(near_lo, lo, hi)])
    return np.where(np.isnan(x), np.nan, np.copysign(y, x))


def decode(q, k, v, table, lens, scale, window=0, softcap=0.0, sinks=None, slopes=None):
    """q [B, Hq, D], k / v [num_blocks, block_size, Hk, D] float64 values. Returns (out, lse, size): size is
    sum p |v|, what relative errors of the weights act on."""
    B, Hq, D = q.shape
    bs, Hk = k.shape[1], k.shape[2]
    out, size, lse = np.zeros((B, Hq, D)), np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    for b in range(B):
        L = min(int(lens[b]), table.shape[1] * bs)
        n = np.arange(max(0, L - window) if window else 0, L)
        for h in range(Hq):
            sink = -np.inf if sinks is None else float(sinks[h])
            lse[b, h] = sink
            if len(n) == 0:
                continue
            blocks, kh = table[b, n // bs], h // (Hq // Hk)
            s = k[blocks, n % bs, kh] @ q[b, h] * scale
            if softcap:
                s = softcap * np.tanh(s / softcap)
            if slopes is not None:
                s = s + float(slopes[h]) * (n - (L - 1))
            top = max(s.max(), sink)
            p = np.exp(s - top)
            total = p.sum() + (np.exp(sink - top) if sinks is not None else 0.0)
            vals = v[blocks, n % bs, kh]
            out[b, h], size[b, h] = p @ vals / total, p @ np.abs(vals) / total
            lse[b, h] = top + np.log(total)
    return out, lse, size

"""fp64 definitions of the paged cache around the decode: the page plan of a step, the
append of new tokens (bf16, or 8 bits with one scale per block of rows and 128 columns)
and the load of cached rows.  Test infrastructure, like the rest of this package.
"""
from __future__ import annotations

import numpy as np

from .reference import rope_rotate

TOP = {"int8": 127.0, "e4m3": 448.0}


def e4m3_values() -> np.ndarray:
    """The non-negative e4m3 numbers in the order of their codes 0 .. 126: 3 mantissa bits,
    exponents from -6 (below it subnormals of spacing 2^-9), largest 448."""
    code = np.arange(127)
    e, m = code >> 3, code & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def nearest(y, fmt: str) -> np.ndarray:
    """The format's number nearest to y, the even code on a tie, clamped to the largest."""
    y = np.asarray(y, dtype=np.float64)
    if fmt == "int8":
        return np.clip(np.rint(y), -127, 127)
    grid = e4m3_values()
    size = np.minimum(np.abs(y), 448.0)
    high = np.searchsorted(grid, size)
    low = np.maximum(high - 1, 0)
    up, down = grid[high] - size, size - grid[low]
    code = np.where((up < down) | ((up == down) & (high % 2 == 0)), high, low)
    return np.copysign(grid[code], y)


def block_scale(amax, fmt: str) -> np.ndarray:
    """fl32(amax / top): scales are fp32 numbers by the format's definition."""
    return (np.asarray(amax, dtype=np.float64) / TOP[fmt]).astype(np.float32)


def append_block(codes, scale, x, offsets, fmt: str):
    """One block of rows and 128 columns: codes [rows, 128] (fp64 values of the codes), its
    fp32 scale, new rows x [n, 128] at the given offsets.  Returns the block's codes and scale."""
    codes, x = np.array(codes, dtype=np.float64), np.asarray(x, dtype=np.float64)
    first = min(offsets)
    s = block_scale(np.abs(x).max(), fmt)
    if first > 0:
        s = max(s, np.float32(scale))
        if s > scale:
            codes[:first] = nearest(codes[:first] * float(scale) / float(s), fmt)
    codes[list(offsets)] = nearest(x / float(s), fmt) if s > 0 else 0.0
    return codes, np.float32(s)


def append(codes, scale, krope, x, k, slots, positions, block: int, fmt: str, theta: float = 10000.0):
    """New tokens x [n, d_c], k [n, 64] into a cache of codes [rows, d_c] (fp64 values; the
    latents themselves for fmt "bf16"), scale fp32 [ceil(rows / block), d_c / 128] and krope
    [rows, 64], all copied.  Tokens whose slot is no row are skipped."""
    codes, krope = np.array(codes, dtype=np.float64), np.array(krope, dtype=np.float64)
    scale = None if scale is None else np.array(scale, dtype=np.float32)
    rows = codes.shape[0]
    live = [i for i in range(len(slots)) if 0 <= slots[i] < rows]
    for i in live:
        krope[slots[i]] = rope_rotate(np.asarray(k[i], dtype=np.float64), int(positions[i]), theta)
    if fmt == "bf16":
        for i in live:
            codes[slots[i]] = x[i]
        return codes, scale, krope
    by_block = {}
    for i in live:
        by_block.setdefault(int(slots[i]) // block, []).append(i)
    for b, tokens in by_block.items():
        r0 = b * block
        for g in range(codes.shape[1] // 128):
            c = slice(128 * g, 128 * (g + 1))
            new, scale[b, g] = append_block(codes[r0:r0 + block, c], scale[b, g], np.asarray(x, dtype=np.float64)[tokens, c],
                                            [int(slots[i]) - r0 for i in tokens], fmt)
            codes[r0:r0 + block, c] = new
    return codes, scale, krope


def values(codes, scale, block: int) -> np.ndarray:
    """What an 8-bit cache stands for: codes [rows, d_c] times their block's scales."""
    codes = np.asarray(codes, dtype=np.float64)
    per_row = np.repeat(np.asarray(scale, dtype=np.float64), block, axis=0)[:codes.shape[0]]
    return codes * np.repeat(per_row[:, :codes.shape[1] // 128], 128, axis=1)


def cache_rows_of(length: int, s: int, table, page: int, seq_stride: int) -> np.ndarray:
    t = np.arange(length)
    return s * seq_stride + t if table is None else table[s, t // page].astype(np.int64) * page + t % page


def page_plan(lens, new, table, ring, free, page: int, max_tokens: int):
    """One step's plan, sequence by sequence.  Returns a dict of the outputs of hra_page_plan
    (table and ring copied), with "status" (code, sequence, wanted, limit)."""
    lens, new, table, ring = np.array(lens), np.array(new), np.array(table), np.array(ring)
    head, tail = int(free[0]), int(free[1])
    B, wide = table.shape
    n = len(ring)
    out = dict(lens=lens.copy(), table=table, ring=ring, free=[head, tail], start=np.zeros(B + 1, np.int64),
               slots=np.full(max_tokens, -1), positions=np.full(max_tokens, -1), status=[0, 0, 0, 0])

    def pages(tokens):
        return -(-int(tokens) // page)

    for code, wrong in ((1, lambda b: lens[b] < 0 or pages(lens[b]) > wide or lens[b] > wide * page),
                        (2, lambda b: new[b] >= 0 and int(lens[b]) + int(new[b]) > wide * page)):
        for b in range(B):
            if wrong(b):
                out["status"] = [code, b, 0, 0]
                return out
    need = sum(pages(lens[b] + new[b]) - pages(lens[b]) for b in range(B) if new[b] >= 0)
    back = sum(pages(lens[b]) for b in range(B) if new[b] < 0)
    total = sum(int(x) for x in new if x > 0)
    if head < 0 or tail < head or tail - head + back > n:
        out["status"] = [5, 0, 0, 0]
        return out
    if total > max_tokens:
        out["status"] = [3, 0, total, max_tokens]
        return out
    if need > tail - head:
        out["status"] = [4, 0, need, tail - head]
        return out
    for k in range(head, head + need):
        if not 0 <= ring[k % n] < n:
            out["status"] = [6, 0, k % n, int(ring[k % n])]
            return out
    at = 0
    for b in range(B):
        if new[b] >= 0:
            for p in range(pages(lens[b]), pages(lens[b] + new[b])):
                table[b, p] = ring[head % n]
                head += 1
        for j in range(max(int(new[b]), 0)):
            pos = int(lens[b]) + j
            where = int(table[b, pos // page])
            out["slots"][at] = where * page + pos % page if 0 <= where < n else -1
            out["positions"][at] = pos
            at += 1
        out["start"][b + 1] = at
    for b in range(B):
        if new[b] < 0:
            for p in range(pages(lens[b])):
                ring[tail % n] = table[b, p]
                tail += 1
    out["lens"] = np.where(new < 0, 0, lens + new)
    out["free"] = [head, tail]
    return out

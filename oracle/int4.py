"""Oracle of the 4-bit KV cache and of the page bookkeeping (TEST
INFRASTRUCTURE ONLY), independent of the CUDA library.

Quantisation follows the library's definition in numpy fp32 (include/fd.h,
fd_append_int4), attention is the fp64 definition over the values the codes
stand for, and the page bookkeeping is a plain loop over the requests, one
token and one page at a time.  bf16 tensors are numpy.uint16 bit patterns."""
from __future__ import annotations

import numpy as np


def _bf16(x) -> np.ndarray:
    """Nearest bf16 bits, ties to even, of float32 values."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + np.uint64(0x7FFF) + ((u >> np.uint64(16)) & np.uint64(1))) >> np.uint64(16)).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def _f64(bits) -> np.ndarray:
    return (np.asarray(bits).astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)


def quantise(x_bits: np.ndarray):
    """Rows [..., D] of bf16 bits -> (codes [..., D] of 0..15, record [..., 4] of
    bf16 bits: scale and bias of each half row)."""
    D = x_bits.shape[-1]
    codes = np.empty(x_bits.shape, np.uint8)
    record = np.empty(x_bits.shape[:-1] + (4,), np.uint16)
    with np.errstate(all="ignore"):
        for g in range(2):
            x = _f64(x_bits[..., g * D // 2:(g + 1) * D // 2])
            mn, mx = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
            # halves: mx - mn of the largest entries does not fit fp32
            s = _bf16((mx / 2 - mn / 2).astype(np.float32) / np.float32(7.5))
            b = _bf16((mn + 8 * _f64(s)).astype(np.float32))
            sf, bf = _f64(s).astype(np.float32), _f64(b).astype(np.float32)
            y = np.rint((x.astype(np.float32) - bf) / np.where(sf > 0, sf, np.float32(1)))
            c = np.where(sf > 0, np.clip(y, -8, 7), 0) + 8
            bad = ~np.isfinite(x).all(-1, keepdims=True)
            codes[..., g * D // 2:(g + 1) * D // 2] = np.where(bad, 8, c).astype(np.uint8)
            record[..., 2 * g] = np.where(bad, 0x7FC0, s)[..., 0]
            record[..., 2 * g + 1] = np.where(bad, 0x7FC0, b)[..., 0]
    return codes, record


def pack(codes: np.ndarray) -> np.ndarray:
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def values(packed: np.ndarray, record: np.ndarray):
    """(s (c - 8), b) in fp64, [..., D] each, of packed rows [..., D/2] and the
    four record entries [..., 4] of K or of V."""
    D = 2 * packed.shape[-1]
    c = np.empty(packed.shape[:-1] + (D,))
    c[..., 0::2] = packed & 15
    c[..., 1::2] = packed >> 4
    r = _f64(record)
    s = np.repeat(r[..., 0::2], D // 2, axis=-1)
    b = np.repeat(r[..., 1::2], D // 2, axis=-1)
    return s * (c - 8), np.broadcast_to(b, c.shape)


def rounded_values(packed, record) -> np.ndarray:
    """bf16 bits of what the rows stand for, rounded once: to fp32 with the lowest
    bit set where that is not exact, and from there to bf16."""
    x, b = values(packed, record)
    with np.errstate(all="ignore"):
        y = x + b
        f = y.astype(np.float32)
        u = f.view(np.uint32)
        u = u - (np.abs(f.astype(np.float64)) > np.abs(y)) | (f != y)      # towards zero, inexact
        return _bf16(np.where(np.isfinite(f), u.astype(np.uint32).view(np.float32), f))


def attend(q_bits, kc, kr, vc, vr, scale: float):
    """Attention of G queries [G, D] over n rows: packed codes [n, D/2] and
    records [n, 4] of K and V.  Returns (O [G, D], lse [G], tol_O, tol_lse).

    The tolerances bound what the library's arithmetic may be off by:
      scores  sums of D products in fp32, at most 2^-23 of the magnitudes per
              addition (a tensor core may truncate), of the terms q s (c - 8)
              and b sum q; q entries are held to 2^-25 of the row's largest;
      weights f16(p s / s_max): 2^-11 of each, and at least 2^-25 s_max;
      the rest of the fp32 arithmetic 2^-20 (ex2 and the sums);
      the output, bf16: 2^-8."""
    q = _f64(q_bits)
    G, D = q.shape
    n = kc.shape[0]
    if n == 0:
        return np.zeros((G, D)), np.full(G, -np.inf), np.zeros((G, D)), np.zeros(G)
    kx, kb = values(kc, kr)
    vx, vb = values(vc, vr)
    sc = float(np.float32(scale))
    t = sc * (q @ (kx + kb).T)
    m = t.max(1, keepdims=True)
    e = np.exp(t - m)
    l = e.sum(1, keepdims=True)
    p = e / l
    v = vx + vb
    o = p @ v
    lse = m[:, 0] + np.log(l[:, 0])
    size = np.abs(q) @ (np.abs(kx) + np.abs(kb)).T                       # [G, n]
    top = np.abs(q).max(1, keepdims=True) * (np.abs(kx).max(1) + np.abs(kb).max(1))[None]
    score = sc * ((D + 16) * 2.0 ** -23 * size + D * 2.0 ** -25 * top) + 2.0 ** -22 * np.abs(t)
    worst = score.max(1, keepdims=True)
    rel = 2 * worst + 2.0 ** -20
    s_max = np.abs(_f64(vr)[:, 0::2]).max()
    tol = (2.0 ** -8 * np.abs(o) + (2.0 ** -11 + rel) * (p @ (np.abs(vx) + np.abs(vb)))
           + n * 2.0 ** -22 * s_max / l)
    return o, lse, tol, worst[:, 0] + 2.0 ** -20 * (1 + np.abs(lse))


def alloc(seqlens, new_lens, table, free_pages, free_count, block_size: int, max_tokens: int):
    """fd_alloc_pages, one request, token and page at a time."""
    B, blocks = table.shape
    room, table = min(blocks * block_size, 2 ** 31 - 1), table.copy()
    F = min(max(int(free_count), 0), len(free_pages))
    slots = np.full(max_tokens, -1, np.int64)
    positions = np.zeros(max_tokens, np.int32)
    out, cu, used, at = np.zeros(B, np.int32), np.zeros(B + 1, np.int32), 0, 0
    for b in range(B):
        n = min(max(int(seqlens[b]), 0), room)
        held, end, wanted = -(-n // block_size), n, 0
        for i in range(min(max(int(new_lens[b]), 0), max_tokens - at)):
            t = n + i
            j = t // block_size
            if t < room:
                if j >= held + wanted:
                    wanted += 1
                    if used + wanted <= F:
                        table[b, j] = free_pages[F - used - wanted]
                if j < held or used + (j - held) < F:
                    end = t + 1
                    if table[b, j] >= 0:
                        slots[at] = int(table[b, j]) * block_size + t % block_size
            positions[at] = t
            at += 1
        used += wanted
        out[b], cu[b + 1] = end, at
    return slots, positions, cu, out, F - min(F, used), table


def release(seqlens, done, table, free_pages, free_count, block_size: int):
    """fd_release_pages, one page at a time."""
    B, blocks = table.shape
    free = free_pages.copy()
    F = min(max(int(free_count), 0), len(free))
    out = np.zeros(B, np.int32)
    for b in range(B):
        n = min(max(int(seqlens[b]), 0), blocks * block_size)
        if not done[b]:
            out[b] = n
            continue
        for j in range(-(-n // block_size)):
            if F < len(free):
                free[F] = table[b, j]
                F += 1
    return out, F, free

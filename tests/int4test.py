"""Shared helpers of the 4-bit cache tests: seeded caches in every layout and
their oracle results."""
from __future__ import annotations

import numpy as np

from oracle import int4
from split_kv_decode_attn_b200 import workloads as wl

HND, NHD = 0, 1


def torch():
    import torch as _t
    return _t


def up(a):
    """uint16 arrays are bf16 bits; others keep their type."""
    t = torch()
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return t.from_numpy(a.view(np.int16)).cuda().view(t.bfloat16)
    return t.from_numpy(a).cuda()


def bits(x):
    return x.view(torch().int16).cpu().numpy().view(np.uint16)


def rows(seed, shape, spread=0.4, offset=0.25):
    """bf16 rows with channels of unequal size and mean."""
    D = shape[-1]
    ch = np.exp(spread * wl.normal_f64(seed + 1, D))
    x = wl.normal_f64(seed, int(np.prod(shape))).reshape(shape) * ch + offset * ch
    return wl.f64_to_bf16_bits(x)


class Cache:
    """A seeded 4-bit cache.  Places behind a sequence's length, and pages that
    no sequence holds, get random codes and NaN records."""

    def __init__(self, lens, Hq, Hkv, D, max_len, seed, block_size=0, layout=HND, k=None, v=None):
        B = len(lens)
        self.B, self.Hq, self.Hkv, self.D, self.G = B, Hq, Hkv, D, Hq // Hkv
        self.lens, self.block_size, self.layout = list(lens), block_size, layout
        self.max_len = max_len
        self.scale = 1.0 / D ** 0.5
        self.q = wl.f64_to_bf16_bits(wl.normal_f64(seed + 7, B * Hq * D).reshape(B, Hq, D))
        self.k = rows(seed + 20, (B, Hkv, max(max_len, 1), D)) if k is None else k
        self.v = rows(seed + 40, (B, Hkv, max(max_len, 1), D), offset=0.0) if v is None else v
        self.kc, self.kr = int4.quantise(self.k)
        self.vc, self.vr = int4.quantise(self.v)
        self.kc, self.vc = int4.pack(self.kc), int4.pack(self.vc)
        r = np.random.default_rng(seed)
        self.table = None
        rows_ = max_len
        planes = B
        if block_size:
            rows_, blocks = block_size, -(-max_len // block_size)
            held = [-(-n // block_size) for n in lens]
            planes = sum(held) + 3
            perm = r.permutation(planes).astype(np.int32)
            self.table = np.full((B, blocks), 0x7FFFFFF0, np.int32)
            at = 0
            for b, h in enumerate(held):
                self.table[b, :h] = perm[at:at + h]
                at += h
        self.planes, self.rows = planes, rows_
        shape = (planes, Hkv, rows_) if layout == HND else (planes, rows_, Hkv)
        self.k4 = r.integers(0, 256, shape + (D // 2,), dtype=np.uint8)
        self.v4 = r.integers(0, 256, shape + (D // 2,), dtype=np.uint8)
        self.params = np.full(shape + (8,), 0x7FC0, np.uint16)
        for b in range(B):
            t = np.arange(lens[b])
            plane = self.table[b, t // block_size] if block_size else np.full(lens[b], b)
            row = t % block_size if block_size else t
            for h in range(Hkv):
                at = (plane, h, row) if layout == HND else (plane, row, h)
                self.k4[at], self.v4[at] = self.kc[b, h, t], self.vc[b, h, t]
                self.params[at] = np.concatenate([self.kr[b, h, t], self.vr[b, h, t]], -1)

    def on_device(self):
        self.dq, self.dk, self.dv, self.dp = up(self.q), up(self.k4), up(self.v4), up(self.params)
        self.dl = up(np.array(self.lens, np.int32))
        self.dt = up(self.table)
        return self

    def oracle(self):
        o = np.zeros((self.B, self.Hq, self.D))
        lse = np.zeros((self.B, self.Hq))
        tol, ltol = np.zeros_like(o), np.zeros_like(lse)
        for b, n in enumerate(self.lens):
            for h in range(self.Hkv):
                g = slice(h * self.G, (h + 1) * self.G)
                o[b, g], lse[b, g], tol[b, g], ltol[b, g] = int4.attend(
                    self.q[b, g], self.kc[b, h, :n], self.kr[b, h, :n], self.vc[b, h, :n],
                    self.vr[b, h, :n], self.scale)
        return o, lse, tol, ltol


def check(got, got_lse, ref, what=""):
    """got [B, Hq, D] bf16 tensor and lse against Cache.oracle()'s result."""
    o, lse, tol, ltol = ref
    x = wl.bf16_bits_to_f64(bits(got))
    err = np.abs(x - o)
    assert (err <= tol).all(), (f"{what}: {(err > tol).sum()} outputs beyond the bound, worst "
                                f"{np.max(err / np.maximum(tol, 1e-300)):.2f} of it")
    l = got_lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(l), empty), what
    lerr = np.abs(l[~empty] - lse[~empty])
    assert (lerr <= ltol[~empty]).all(), f"{what}: lse off by {lerr.max():.2e}"
    return err.max(), lerr.max() if lerr.size else 0.0

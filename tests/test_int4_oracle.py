"""The 4-bit oracle against closed forms (CPU): the quantiser's grid, error and
special groups; attention against brute force; the page bookkeeping against
what it promises."""
import numpy as np
import pytest

from oracle import int4
from split_kv_decode_attn_b200 import workloads as wl

from int4test import rows


@pytest.mark.parametrize("D", [64, 128])
def test_quantised_rows_are_within_half_a_step(D):
    x = rows(11, (200, D))
    codes, rec = int4.quantise(x)
    assert codes.max() <= 15
    xc, b = int4.values(int4.pack(codes), rec)
    s = np.repeat(wl.bf16_bits_to_f64(rec[:, 0::2]), D // 2, axis=1)
    xf = wl.bf16_bits_to_f64(x)
    # half a step, the clip at an end (s is off by 2^-8, 15 steps of it), and
    # the bias's rounding, 2^-8 of it
    assert (np.abs(xc + b - xf) <= 0.5 * s + 15 * 2.0 ** -8 * s + 2.0 ** -8 * np.abs(b)).all()


def test_values_on_the_grid_come_back_exactly():
    # s = 1/4, b = 1: the values 1 + (c - 8) / 4 for c = 0 .. 15
    grid = 1 + (np.arange(16) - 8) / 4
    x = wl.f64_to_bf16_bits(np.tile(grid, (1, 4)))
    codes, rec = int4.quantise(x)
    assert np.array_equal(codes[0], np.tile(np.arange(16), 4))
    assert np.array_equal(wl.bf16_bits_to_f64(rec[0]), [0.25, 1.0, 0.25, 1.0])
    assert np.array_equal(int4.rounded_values(int4.pack(codes), rec), x)


def test_special_groups():
    x = np.zeros((4, 64), np.uint16)
    x[0, :] = wl.f64_to_bf16_bits(np.full(64, 3.5))          # constant
    x[1, :32] = wl.f64_to_bf16_bits(np.linspace(-1, 1, 32))
    x[1, 5] = 0x7FC0                                          # NaN in the first group
    x[2, 40] = 0x7F80                                         # infinity in the second
    x[3, :] = np.where(np.arange(64) % 2, 0x7F7F, 0xFF7F)     # +- the largest bf16
    codes, rec = int4.quantise(x)
    v = wl.bf16_bits_to_f64(int4.rounded_values(int4.pack(codes), rec))
    assert (v[0] == 3.5).all()
    assert np.isnan(v[1, :32]).all() and (v[1, 32:] == 0).all()
    assert (v[2, :32] == 0).all() and np.isnan(v[2, 32:]).all()
    assert not np.isnan(v[3]).any() and (np.abs(v[3]) > 3.3e38).all()


def test_attention_matches_brute_force():
    D, n = 64, 5
    x = rows(3, (n, D))
    (kc, kr), (vc, vr) = int4.quantise(x), int4.quantise(rows(4, (n, D)))
    q = wl.f64_to_bf16_bits(wl.normal_f64(5, 2 * D).reshape(2, D))
    o, lse, tol, ltol = int4.attend(q, int4.pack(kc), kr, int4.pack(vc), vr, 0.125)
    for g in range(2):
        s, vals = [], []
        for j in range(n):
            dot, row = 0.0, []
            for d in range(D):
                h = d // (D // 2)
                ks, kb, vs, vb = (float(wl.bf16_bits_to_f64(r[j:j + 1, 2 * h + i])[0])
                                  for r in (kr, vr) for i in range(2))
                dot += float(wl.bf16_bits_to_f64(q[g:g + 1, d])[0]) * (ks * (int(kc[j, d]) - 8) + kb)
                row.append(vs * (int(vc[j, d]) - 8) + vb)
            s.append(0.125 * dot)
            vals.append(row)
        w = np.exp(s)
        assert np.allclose(o[g], w @ np.array(vals) / w.sum(), rtol=1e-12)
        assert np.isclose(lse[g], np.log(w.sum()), rtol=1e-12)
    assert (tol > 0).all() and (ltol > 0).all()


def test_pages_are_taken_once_and_come_back():
    r = np.random.default_rng(0)
    B, bs, blocks, pages = 6, 8, 12, 40
    table = np.full((B, blocks), -1, np.int32)
    free = r.permutation(pages).astype(np.int32)
    lens, count = np.zeros(B, np.int32), pages
    for turn in range(30):
        new = r.integers(0, 12, B).astype(np.int32)
        slots, pos, cu, lens2, count, table = int4.alloc(lens, new, table, free, count, bs, 100)
        assert (lens2 <= lens + new).all() and (lens2 <= blocks * bs).all()
        held = [p for b in range(B) for p in table[b, :-(-int(lens2[b]) // bs)]]
        assert len(set(held)) == len(held) and set(held).isdisjoint(free[:count])
        assert len(held) + count == pages
        good = slots[slots >= 0]
        assert len(set(good.tolist())) == len(good) == (lens2 - lens).sum()
        lens = lens2
        done = r.random(B) < 0.2
        lens, count, free = int4.release(lens, done, table, free, count, bs)
        assert (lens[done] == 0).all()

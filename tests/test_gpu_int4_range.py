"""fd_decode_int4 over the whole range of bf16: rows that fd_append_int4 takes and
fd_expand_int4 gives back finite, up to the largest, against the fp64 oracle and
its derived bounds.  (All scalings are by powers of two, so the bounds of the
ordinary sizes hold unchanged.)"""
import numpy as np
import pytest

import split_kv_decode_attn_b200 as fd
from split_kv_decode_attn_b200 import workloads as wl

from int4test import HND, NHD, Cache, check, rows, torch

pytestmark = pytest.mark.gpu

LARGEST = 3e38      # of a V entry: the values of its codes stay below the largest bf16


@pytest.fixture(autouse=True)
def _gpu(cuda_device):
    yield
    assert fd.fd_check_device_error() == fd.FD_OK


def decode(c, S=None):
    out, lse = fd.decode_int4(c.dq, c.dk, c.dv, c.dp, c.dl, c.dt, kv_layout=c.layout,
                              max_len=c.max_len, scale=c.scale, num_splits=S)
    torch().cuda.synchronize()
    return out, lse


def large(seed, shape, size):
    """V rows of one size, cut off at the largest."""
    v = wl.bf16_bits_to_f64(rows(seed, shape)) * size
    return wl.f64_to_bf16_bits(np.clip(v, -LARGEST, LARGEST))


# ------------------------------------------------------------------------ V

@pytest.mark.parametrize("size", [2e31, 1e33, 1e37, LARGEST])
@pytest.mark.parametrize("G,D", [(8, 128), (16, 128), (1, 64)])
def test_large_values(size, G, D):
    """Clusters, one CTA, ranges of CTAs and of warps, one head or eight at a time."""
    for B, n, Hkv in ((1, 200, 2), (3, 1500, 1), (5, 700, 8)):
        lens = ([n, 1, n - 65, 0, 64] * B)[:B]
        c = Cache(lens, G * Hkv, Hkv, D, n, seed=1000 + G + B,
                  v=large(21, (B, Hkv, n, D), size)).on_device()
        ref = c.oracle()
        assert np.isfinite(ref[0]).all() and np.abs(ref[0]).max() < LARGEST * 1.01
        for S in (None, 1, 2, 3, 40, 400):
            check(*decode(c, S), ref, f"size={size} G={G} D={D} B={B} S={S}")


@pytest.mark.parametrize("value", [1e34, LARGEST, -LARGEST])
@pytest.mark.parametrize("n", [3, 6000])
def test_large_constant_values_of_equal_weight(value, n):
    """Constant rows have scale 0 and all of their size in the bias; with q = 0 every
    token has the same weight, and the result is the value itself."""
    t = torch()
    v = wl.f64_to_bf16_bits(np.full((2, 8, n, 64), value))
    c = Cache([n, max(n - 70, 1)], 16, 8, 64, n, seed=1100, v=v)
    c.q[:] = 0
    c.on_device()
    ref = c.oracle()
    for S in (None, 1, 2, 30, 400):
        out, lse = decode(c, S)
        check(out, lse, ref, f"value={value} n={n} S={S}")
        assert t.equal(out, t.full_like(out, value))


@pytest.mark.parametrize("layout,bs", [(HND, 0), (NHD, 16)])
def test_values_of_every_size_along_one_history(layout, bs):
    """Sizes from 1 to the largest in one history, in random order, rising and
    falling: the weights' reference moves by up to 2^120 and the biases with it."""
    n = 20000
    r = np.random.default_rng(7)
    for gain in (r.uniform(0, 120, n), np.linspace(0, 120, n), np.linspace(120, 0, n)):
        v = wl.bf16_bits_to_f64(rows(31, (1, 1, n, 128)))
        v = np.clip(v * 2.0 ** np.round(gain)[:, None], -LARGEST, LARGEST)
        c = Cache([n], 8, 1, 128, n, seed=1200, block_size=bs, layout=layout,
                  v=wl.f64_to_bf16_bits(v)).on_device()
        ref = c.oracle()
        for S in (1, 2, 37, 300):
            check(*decode(c, S), ref, f"S={S}")


@pytest.mark.parametrize("size", [1e-38, 1e-34])
def test_smallest_values(size):
    """Down to bf16's subnormals, whose step (2^-133) replaces the relative bound."""
    v = wl.f64_to_bf16_bits(wl.bf16_bits_to_f64(rows(41, (2, 2, 900, 64))) * size)
    c = Cache([900, 65], 8, 2, 64, 900, seed=1300, v=v).on_device()
    o, lse, tol, ltol = c.oracle()
    for S in (None, 1, 2, 20):
        check(*decode(c, S), (o, lse, tol + 2.0 ** -133, ltol), f"size={size} S={S}")


@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 24, 2.0 ** 26])
def test_equal_scores_of_any_size_are_merged_alike(size):
    """One warp's 64 tokens and another's single one, all with the same score: the mean
    of V.  A reference of 2^24 and more has no room for a change of it by less than 2."""
    for D, G in ((128, 4), (64, 16)):
        for n in (65, 1000, 3000):
            k = np.ones((1, 1, n, D))
            k[..., 1::2] = -1.0
            c = Cache([n], G, 1, D, n, seed=1250, k=wl.f64_to_bf16_bits(k))
            c.q = wl.f64_to_bf16_bits(np.tile(np.where(np.arange(D) % 2, -1.0, 1.0), (1, G, 1)) * size / D / c.scale)
            c.on_device()
            o = c.oracle()[0]
            out, lse = decode(c, 1)
            got = wl.bf16_bits_to_f64(out.view(torch().int16).cpu().numpy().view(np.uint16))
            # 2^-8 of the result, 2^-11 (a weight in f16) of scale * (code - 8), which is at
            # most 8 / 15 (1 + 2^-8) of the range of V, and fp32's sums
            err = np.abs(got - o) - (2.0 ** -8 * np.abs(o) + 2.0 ** -11 * 1.1 * np.abs(wl.bf16_bits_to_f64(c.v)).max())
            assert err.max() <= 0, f"D={D} n={n}"


# ------------------------------------------------------------------- q and scale

@pytest.mark.parametrize("scale", [1e-38, 1e-12, 3e38])
def test_zero_query_of_any_scale_gives_the_mean(scale):
    """Lengths that end inside a unit: a token that does not count has weight 0."""
    lens = [500, 77, 64, 1, 0, 33]
    for G, D in ((4, 128), (16, 64)):
        c = Cache(lens, 2 * G, 2, D, 500, seed=1400)
        c.q[:] = 0
        c.scale = float(np.float32(scale))
        c.on_device()
        ref = c.oracle()
        for S in (None, 1, 3, 40):
            check(*decode(c, S), ref, f"scale={scale} G={G} S={S}")


@pytest.mark.parametrize("qlog,klog,scale", [
    (-120, 0, 1e-8),       # scores of about 0
    (-120, 0, 2.0 ** 118),
    (-124, 0, 3e37),
    (-126, 0, 3e38),       # scale log2(e) is beyond fp32
    (121, -115, None),
    (125, -127, 0.5),
    (121, -115, 1e-3),
    (60, -60, 1e30),
    (60, 60, 1e-36),
    (122, 0, 2.0 ** -122)])
def test_scores_of_ordinary_size_from_any_q_k_and_scale(qlog, klog, scale):
    lens = [301, 64, 5, 900]
    for G, Hkv, D in ((8, 1, 128), (16, 2, 64), (2, 8, 64)):
        c = Cache(lens, G * Hkv, Hkv, D, 900, seed=1500 + G,
                  k=wl.f64_to_bf16_bits(wl.bf16_bits_to_f64(rows(51, (4, Hkv, 900, D))) * 2.0 ** klog))
        c.q = wl.f64_to_bf16_bits(wl.bf16_bits_to_f64(c.q) * 2.0 ** qlog)
        c.scale = c.scale if scale is None else float(np.float32(scale))
        c.on_device()
        ref = c.oracle()
        for S in (None, 1, 2, 30):
            check(*decode(c, S), ref, f"G={G} S={S}")


def test_scores_next_to_the_largest():
    """Scores of up to 2^125: the row with the largest one is the result.  Heads of
    ordinary size, of size 0 and of the smallest size beside it keep theirs."""
    n, G, D = 700, 8, 128
    c = Cache([n, 130], G, 1, D, n, seed=1600)
    q = wl.bf16_bits_to_f64(c.q) * np.array([1, 2.0 ** 121, 0, 2.0 ** -120, 2.0 ** 118, 1, -2.0 ** 121, 2])[:, None]
    c.q = wl.f64_to_bf16_bits(q)
    c.on_device()
    o, lse, tol, ltol = c.oracle()
    far = [1, 4, 6]
    near = [0, 2, 3, 5, 7]
    vmax = np.abs(wl.bf16_bits_to_f64(c.v)).max()
    for S in (None, 1, 2, 30):
        out, l = decode(c, S)
        check(out[:, near], l[:, near], [x[:, near] for x in (o, lse, tol, ltol)], f"S={S}")
        got = wl.bf16_bits_to_f64(out[:, far].view(torch().int16).cpu().numpy().view(np.uint16))
        # one weight of 1 (the next score is 2^100 away): V's row with the result's 2^-8
        # and 2^-11, the weight's f16 rounding, of scale * (code - 8), which is at most
        # 8 / 15 (1 + 2^-8) of the range of V
        want = o[:, far]
        err = np.abs(got - want) - (2.0 ** -8 * np.abs(want) + 2.0 ** -11 * 1.1 * vmax)
        assert err.max() <= 0
        err = np.abs(l[:, far].cpu().numpy() - lse[:, far]) - ltol[:, far]
        assert err.max() <= 0


@pytest.mark.parametrize("size", [2.0 ** 18, 2.0 ** 21, 2.0 ** 24, 2.0 ** 30, 2.0 ** 60])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_scores_that_differ_by_little(size, sign):
    """Scores of one large size whose differences are the steps of fp32 there: equal
    rows of K, one of them half as large again (or as small) in the middle, so that
    a reference that is not the largest score would lose every weight."""
    n, D = 400, 128
    for at in (0, 70, 399):
        k = np.ones((1, 1, n, D))
        k[0, 0, :, 1::2] = -1.0
        k[0, 0, at] *= 1.5
        c = Cache([n], 4, 1, D, n, seed=1700, k=wl.f64_to_bf16_bits(k))
        q = np.tile(np.where(np.arange(D) % 2, -1.0, 1.0), (1, 4, 1)) * np.array([1, 0.5, 1, 2])[:, None]
        c.q = wl.f64_to_bf16_bits(sign * q * size / D / c.scale)
        c.on_device()
        o, lse, tol, ltol = c.oracle()
        vmax = np.abs(wl.bf16_bits_to_f64(c.v)).max()
        for S in (1, 2, 5):
            out, l = decode(c, S)
            check(out, l, (o, lse, tol, ltol), f"at={at} S={S}")
            if S > 1:       # parts meet by their lse, as good as fp32 holds it
                continue
            got = wl.bf16_bits_to_f64(out.view(torch().int16).cpu().numpy().view(np.uint16))
            # The row in the middle alone, or the mean of all others: equal weights, whatever
            # the reference's rounding makes of them.  2^-8 of the result, 2^-11 of V's size.
            err = np.abs(got - o) - (2.0 ** -8 * np.abs(o) + 2.0 ** -11 * 1.1 * vmax)
            assert err.max() <= 0, f"at={at}"


@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 20, 2.0 ** 30, 2.0 ** 60, 2.0 ** 120])
def test_equal_scores_over_many_units_of_a_warp(size):
    """The same score over and over, in units that each take it relative to a reference
    from an earlier one: finite, within V's range, and within the bound of the oracle."""
    n, D = 9000, 128
    k = np.ones((1, 1, n, D))
    k[..., 1::2] = -1.0
    c = Cache([n], 8, 1, D, n, seed=1800, k=wl.f64_to_bf16_bits(k))
    q = np.tile(np.where(np.arange(D) % 2, -1.0, 1.0), (1, 8, 1)) * np.linspace(0.1, 1, 8)[:, None]
    c.q = wl.f64_to_bf16_bits(q * size / D / c.scale)
    c.on_device()
    ref = c.oracle()
    v = wl.bf16_bits_to_f64(c.v)[0, 0]
    for S in (1, 2, 11):
        out, lse = decode(c, S)
        check(out, lse, ref, f"S={S}")
        got = wl.bf16_bits_to_f64(out.view(torch().int16).cpu().numpy().view(np.uint16))
        # the values of the codes pass V by 2^-7 of its size, the result by 2^-8
        room = 2.0 ** -6 * np.abs(v).max()
        assert (got <= v.max(0) + room).all() and (got >= v.min(0) - room).all()

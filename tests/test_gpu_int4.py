"""GPU parity of the 4-bit cache: fd_append_int4 (bit for bit), fd_expand_int4
(bit for bit) and fd_decode_int4 against the fp64 oracle, whose bounds are
derived from the library's roundings (oracle/int4.py, attend)."""
import numpy as np
import pytest

import split_kv_decode_attn_b200 as fd
from oracle import int4
from split_kv_decode_attn_b200 import workloads as wl

from int4test import HND, NHD, Cache, bits, check, rows, torch, up

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_device):
    yield
    assert fd.fd_check_device_error() == fd.FD_OK


def decode(c, S=None, **kw):
    out, lse = fd.decode_int4(c.dq, c.dk, c.dv, c.dp, c.dl, c.dt, kv_layout=c.layout,
                              max_len=c.max_len, scale=c.scale, num_splits=S, **kw)
    torch().cuda.synchronize()
    return out, lse


# ------------------------------------------------------------------- append

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", [HND, NHD])
@pytest.mark.parametrize("T,Hkv,rows_", [(1, 1, 8), (37, 3, 16), (300, 8, 100)])
def test_append_is_the_oracles_codes_and_touches_nothing_else(D, layout, T, Hkv, rows_):
    t = torch()
    planes = -(-T // rows_) + 3
    shape = (planes, Hkv, rows_) if layout == HND else (planes, rows_, Hkv)
    r = np.random.default_rng(T)
    k4 = r.integers(0, 256, shape + (D // 2,), dtype=np.uint8)
    v4 = r.integers(0, 256, shape + (D // 2,), dtype=np.uint8)
    prm = wl.f64_to_bf16_bits(r.standard_normal(shape + (8,)))
    # K and V as slices of one projection's output
    fused = rows(T + D, (T, (2 + 2 * Hkv), D))
    fused[0, 1, :3] = wl.f64_to_bf16_bits(np.array([1e30, -1e30, 1e-30]))
    fused[T // 2, 2] = fused[T // 2, 2, 0]                      # a constant row
    slots = r.permutation(planes * rows_)[:T].astype(np.int64)
    if T > 5:
        slots[3], slots[4], slots[5] = -1, planes * rows_, -(1 << 40)
    dk4, dv4, dprm, df, ds = up(k4), up(v4), up(prm), up(fused), up(slots)
    fd.append_int4(df[:, 1:1 + Hkv], df[:, 1 + Hkv:1 + 2 * Hkv], ds, dk4, dv4, dprm, kv_layout=layout)
    t.cuda.synchronize()
    kc, kr = int4.quantise(fused[:, 1:1 + Hkv])
    vc, vr = int4.quantise(fused[:, 1 + Hkv:1 + 2 * Hkv])
    for i, s in enumerate(slots):
        if 0 <= s < planes * rows_:
            at = (s // rows_, slice(None), s % rows_) if layout == HND else (s // rows_, s % rows_)
            k4[at], v4[at] = int4.pack(kc[i]), int4.pack(vc[i])
            prm[at] = np.concatenate([kr[i], vr[i]], -1)
    assert np.array_equal(dk4.cpu().numpy(), k4) and np.array_equal(dv4.cpu().numpy(), v4)
    assert np.array_equal(bits(dprm), prm)


def test_append_of_special_and_tied_rows():
    """Infinities, NaN, the largest and smallest entries, ties between codes and
    a bias far larger than the range."""
    D = 128
    x = rows(5, (64, 1, D))
    x[0, 0, 5] = 0x7FC0
    x[1, 0, 100] = 0xFF80
    x[2, 0, :] = np.where(np.arange(D) % 2, 0x7F7F, 0xFF7F)
    x[3, 0, :] = np.arange(D)                                   # subnormals
    x[4, 0, :] = wl.f64_to_bf16_bits(100 + (np.arange(D) % 3) * 0.5)
    r = np.random.default_rng(1)
    for i in range(8, 64):     # many exact ties: multiples of half a step
        half = float(r.choice([0.5, 0.375, 0.625, 0.4375, 1.5]))
        x[i, 0, :] = wl.f64_to_bf16_bits(r.integers(-15, 16, D) * half)
    k4 = torch().zeros((1, 1, 64, D // 2), dtype=torch().uint8, device="cuda")
    v4, prm = torch().zeros_like(k4), up(np.zeros((1, 1, 64, 8), np.uint16))
    fd.append_int4(up(x), up(x), up(np.arange(64)), k4, v4, prm)
    c, rec = int4.quantise(x[:, 0])
    assert np.array_equal(k4[0, 0].cpu().numpy(), int4.pack(c))
    assert np.array_equal(v4[0, 0].cpu().numpy(), int4.pack(c))
    got = bits(prm)[0, 0]
    # the sign of a zero bias is free
    zero = (rec & 0x7FFF) == 0
    for half in (got[:, :4], got[:, 4:]):
        assert np.array_equal(np.where(zero, half & 0x7FFF, half), np.where(zero, rec & 0x7FFF, rec))


@pytest.mark.parametrize("D", [64, 128])
def test_append_next_to_ties(D):
    """Entries that lie on, and a bit off, the border between two codes: integer
    groups of range 15 (scale 1) and 30 (scale 2), entries of all sizes down to
    the smallest beside them, biases up to where codes have to be clamped."""
    n = 2048
    r = np.random.default_rng(D)
    x = np.empty((n, D))
    for i in range(n):
        size = 2.0 ** r.integers(-130, 100)
        kind = i % 4
        if kind == 0:      # borders exactly, and tiny entries
            row = r.integers(-15, 16, D) * 0.5
            tiny = r.random(D) < 0.3
            row[tiny] = r.choice([-1, 1], tiny.sum()) * 2.0 ** -r.integers(1, 40, tiny.sum())
            row[::D // 2], row[1::D // 2] = -7.5, 7.5
        elif kind == 1:    # a narrow band around the borders
            row = (r.integers(-15, 16, D) * 0.5) * (1 + r.integers(-2, 3, D) / 128)
        elif kind == 2:    # an offset that bf16 holds coarsely
            row = 2.0 ** r.integers(0, 9) + r.integers(-8, 8, D) * 0.25
        else:
            row = r.standard_normal(D) * 2.0 ** r.integers(-20, 1, D)
        x[i] = row * size
    x = wl.f64_to_bf16_bits(x).reshape(n, 1, D)
    k4 = torch().zeros((1, 1, n, D // 2), dtype=torch().uint8, device="cuda")
    v4, prm = torch().zeros_like(k4), up(np.zeros((1, 1, n, 8), np.uint16))
    fd.append_int4(up(x), up(x[::-1].copy()), up(np.arange(n)), k4, v4, prm)
    c, rec = int4.quantise(x[:, 0])
    assert np.array_equal(k4[0, 0].cpu().numpy(), int4.pack(c))
    assert np.array_equal(v4[0, 0].cpu().numpy(), int4.pack(c[::-1]))
    # the sign of a zero is free
    assert np.array_equal(rec & 0x7FFF, bits(prm)[0, 0, :, :4] & 0x7FFF)
    nonzero = (rec & 0x7FFF) != 0
    assert np.array_equal(rec[nonzero], bits(prm)[0, 0, :, :4][nonzero])


# ------------------------------------------------------------------- expand

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", [HND, NHD])
@pytest.mark.parametrize("bs", [0, 8, 64])
def test_expand_gives_the_values_and_leaves_the_rest(D, layout, bs):
    t = torch()
    lens = [0, 1, 100, 31, 33, 97]
    c = Cache(lens, 4, 2, D, 104, seed=D + bs, block_size=bs, layout=layout).on_device()
    shape = (c.B, c.Hkv, c.max_len, D) if layout == HND else (c.B, c.max_len, c.Hkv, D)
    k, v = (t.full(shape, 7.0, dtype=t.bfloat16, device="cuda") for _ in range(2))
    fd.expand_int4(c.dk, c.dv, c.dp, c.dl, c.dt, max_len=c.max_len, kv_layout=layout, k_out=k, v_out=v)
    t.cuda.synchronize()
    for got, code, rec in ((k, c.kc, c.kr), (v, c.vc, c.vr)):
        ref = int4.rounded_values(code, rec)
        for b, n in enumerate(lens):
            ref[b, :, n:] = wl.f64_to_bf16_bits(np.full(1, 7.0))[0]
        g = got if layout == HND else got.transpose(1, 2)
        assert np.array_equal(bits(g.contiguous()), ref)


def test_expanded_cache_feeds_decode():
    c = Cache([700, 64, 0, 301], 16, 2, 128, 700, seed=77, block_size=0).on_device()
    k, v = fd.expand_int4(c.dk, c.dv, c.dp, c.dl)
    out, lse = fd.decode(c.dq, k, v, c.dl, scale=c.scale, num_splits=3)
    got, gl = decode(c, 3)
    # bf16 rows against the rows the codes stand for: 2^-8 of each entry
    assert (out.float() - got.float()).abs().max() < 3e-2
    assert (lse[:2] - gl[:2]).abs().max() < 2e-2


def test_a_page_outside_the_pool_reads_zeros():
    t = torch()
    c = Cache([64, 64], 4, 2, 64, 64, seed=5, block_size=16).on_device()
    bad = c.dt.clone()
    bad[0, 1], bad[1, 2], bad[1, 3] = -3, c.planes, 2 ** 31 - 1
    k, v = fd.expand_int4(c.dk, c.dv, c.dp, c.dl, bad)
    t.cuda.synchronize()
    assert (k[0, :, 16:32] == 0).all() and (k[1, :, 32:] == 0).all() and (v[1, :, 32:] == 0).all()
    out, lse = fd.decode_int4(c.dq, c.dk, c.dv, c.dp, c.dl, bad, num_splits=1)
    for code in (c.kc, c.vc, c.kr, c.vr):
        code[0, :, 16:32] = 0
        code[1, :, 32:] = 0
    check(out, lse, c.oracle(), "bad pages")


# ------------------------------------------------------------------- decode

LENS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 130, 400, 777]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
def test_group_sizes_and_ragged_lengths(G, D):
    c = Cache(LENS, 2 * G, 2, D, 777, seed=100 + G + D).on_device()
    ref = c.oracle()
    for S in (1, 2, 3, 7, 13, 1024):
        e = check(*decode(c, S), ref, f"G={G} D={D} S={S}")
    print(f"G={G} D={D}: max|dO| {e[0]:.2e}, max|dlse| {e[1]:.2e}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", [HND, NHD])
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128, 256])
def test_layouts_and_pages_agree_bit_for_bit(bs, layout, D):
    lens = [0, 1, 250, 500, 129]
    base = Cache(lens, 8, 2, D, 512, seed=200 + D).on_device()
    c = Cache(lens, 8, 2, D, 512, seed=200 + D, block_size=bs, layout=layout, k=base.k, v=base.v)
    c.on_device()
    ref = base.oracle()
    for S in (1, 3, 8):
        a, b = decode(base, S), decode(c, S)
        check(*b, ref, f"bs={bs} layout={layout} D={D} S={S}")
        assert torch().equal(a[0], b[0]) and torch().equal(a[1], b[1])


@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_contiguous_token_major_and_odd_lengths(Hkv):
    lens = [3001, 1, 2999, 64, 0]
    for layout in (HND, NHD):
        c = Cache(lens, 4 * Hkv, Hkv, 128, 3001, seed=300 + Hkv, layout=layout).on_device()
        ref = c.oracle()
        for S in (None, 1, 5):
            check(*decode(c, S), ref, f"Hkv={Hkv} layout={layout} S={S}")


@pytest.mark.parametrize("layout", [HND, NHD])
@pytest.mark.parametrize("G,D,Hkv,bs", [(1, 64, 8, 0), (4, 128, 8, 16), (8, 128, 16, 32),
                                        (16, 128, 8, 8), (16, 64, 8, 0)])
def test_eight_heads_at_a_time(G, D, Hkv, bs, layout):
    """KV heads in eights: one row of up to 150 parts, several in one range."""
    lens = [0, 1, 5000, 64, 65, 300, 1000, 0]
    c = Cache(lens, G * Hkv, Hkv, D, 5000 if bs == 0 else 5024, seed=900 + G + D, block_size=bs,
              layout=layout).on_device()
    ref = c.oracle()
    for S in (None, 2, 40, 1024):
        check(*decode(c, S), ref, f"G={G} D={D} Hkv={Hkv} bs={bs} layout={layout} S={S}")


@pytest.mark.parametrize("B,most", [(200, 100), (700, 40)])
def test_eight_heads_of_many_sequences(B, most):
    r = np.random.default_rng(B)
    lens = r.integers(0, most + 1, B).tolist()
    c = Cache(lens, 8, 8, 64, most, seed=B).on_device()
    ref = c.oracle()
    for S in (None, 1, 16):
        check(*decode(c, S), ref, f"B={B} S={S}")


@pytest.mark.parametrize("B,most,G,D,bs,layout", [
    (15, 4096, 4, 128, 0, HND),      # 8 CTAs to a row
    (15, 3400, 16, 64, 8, NHD),      # 7
    (22, 4096, 1, 64, 16, HND),      # 6
    (26, 4100, 8, 128, 0, NHD),      # 5
    (33, 1990, 2, 128, 256, HND),    # 4
    (45, 1300, 16, 128, 32, HND),    # 3
    (74, 1000, 8, 64, 64, NHD)])     # 2
def test_rows_that_a_cluster_shares(B, most, G, D, bs, layout):
    """num_splits = 1 and few rows: lengths that leave CTAs and warps of a cluster
    without a token, none, and one; the result does not depend on the other rows."""
    t = torch()
    lens = np.random.default_rng(B).integers(0, most + 1, B).tolist()
    lens[:10] = [most, 0, 1, 63, 64, 65, 512, 513, most - 1, 0]
    most_rows = most if bs == 0 else -(-most // bs) * bs
    c = Cache(lens, G, 1, D, most_rows, seed=950 + B, block_size=bs, layout=layout).on_device()
    out, lse = decode(c, 1)
    check(out, lse, c.oracle(), f"B={B}")
    c.dl = c.dl.clone()
    c.dl[0], c.dl[3:] = 7, 5
    again, _ = decode(c, 1)
    assert t.equal(again[1:3], out[1:3])


def test_seqlens_are_clamped_and_optional():
    c = Cache([90, 90], 8, 1, 64, 90, seed=9).on_device()
    ref = c.oracle()
    c.dl = None
    check(*decode(c, 2), ref, "no lengths")
    c.dl = up(np.array([2 ** 31 - 1, 90], np.int32))
    check(*decode(c, 2), ref, "clamped")
    c.dl = up(np.array([-5, 90], np.int32))
    out, lse = decode(c, 2)
    assert (out[0] == 0).all() and torch().isneginf(lse[0]).all()


def test_long_history():
    c = Cache([40000, 33], 8, 1, 128, 40000, seed=400).on_device()
    ref = c.oracle()
    for S in (None, 1, 37, 200):
        check(*decode(c, S), ref, f"long S={S}")


def test_a_maximum_that_keeps_growing_and_one_that_falls():
    """Logits that rise (or fall) by several hundred over the history: every
    token moves the running maximum, by less and by more than a rescale."""
    n, D = 600, 128
    for step in (0.05, 0.9, 12.0, -0.9):
        c = Cache([n], 8, 1, D, n, seed=500)
        u = np.zeros(D)
        u[3] = 1.0
        q = np.tile(u * 16.0, (1, 8, 1)) + 0.25 * wl.bf16_bits_to_f64(c.q)
        k = 0.3 * wl.bf16_bits_to_f64(c.k)
        k[0, 0, :, 3] += np.arange(n) * step / (16.0 * c.scale)
        c = Cache([n], 8, 1, D, n, seed=500, k=wl.f64_to_bf16_bits(k))
        c.q = wl.f64_to_bf16_bits(q)
        c.on_device()
        ref = c.oracle()
        for S in (1, 3):
            check(*decode(c, S), ref, f"step={step} S={S}")


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e4, 1e30])
def test_value_rows_of_any_size(size):
    """V rows of one size, and of sizes that rise by 2^20 along the history or
    jump up and down: the weights are held relative to the largest scale."""
    n, D = 200, 64
    v = wl.bf16_bits_to_f64(rows(9, (1, 2, n, D)))
    for gain in (np.ones(n), 2.0 ** np.linspace(-20, 0, n), 2.0 ** np.where(np.arange(n) % 7, -12, 0)):
        c = Cache([n], 4, 2, D, n, seed=600, v=wl.f64_to_bf16_bits(v * size * gain[:, None])).on_device()
        ref = c.oracle()
        for S in (1, 2):
            check(*decode(c, S), ref, f"size={size} S={S}")


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -20, 2.0 ** 60])
def test_query_rows_of_any_size(size):
    n, D = 300, 128
    c = Cache([n], 8, 1, D, n, seed=650)
    c.q = wl.f64_to_bf16_bits(wl.bf16_bits_to_f64(c.q) * size)
    c.scale = float(np.float32(0.09 / size))
    c.on_device()
    check(*decode(c, 2), c.oracle(), f"q size={size}")


def test_zero_query_gives_the_mean():
    c = Cache([500], 4, 1, 128, 500, seed=660)
    c.q[:] = 0
    c.on_device()
    out, lse = decode(c, 3)
    check(out, lse, c.oracle(), "q = 0")
    assert abs(float(lse[0, 0]) - np.log(500)) < 1e-5


def test_nan_rows_inside_a_history_stay_with_their_head():
    for where in (0, 40, 99):
        x = rows(20, (2, 2, 100, 128))
        x[0, 1, where, 7] = 0x7FC0
        for kw in (dict(k=x), dict(v=x)):
            c = Cache([100, 100], 8, 2, 128, 100, seed=670, **kw).on_device()
            for S in (1, 2):
                out, lse = decode(c, S)
                bad = torch().isnan(out).reshape(2, 2, 4, 128)
                assert bad[0, 1].any() and not bad[1].any() and not bad[0, 0].any()
                if "k" in kw:
                    assert bad[0, 1].all() and torch().isnan(lse[0, 4:]).all()


def test_a_history_of_nan_rows_alone_is_nan():
    x = np.full((1, 1, 70, 64), 0x7FC0, np.uint16)
    c = Cache([70], 2, 1, 64, 70, seed=680, k=x).on_device()
    for S in (1, 2):
        out, lse = decode(c, S)
        assert torch().isnan(out).all() and torch().isnan(lse).all()


def test_repeated_calls_give_the_same_bits():
    t = torch()
    for S in (1, 2, 4, 37):
        c = Cache([900, 333, 1200, 5, 0, 64], 32, 4, 128, 1200, seed=700).on_device()
        a = decode(c, S)
        for _ in range(3):
            b = decode(c, S)
            assert t.equal(a[0], b[0]) and t.equal(a[1], b[1])


@pytest.mark.parametrize("B", [1, 31, 33, 70, 300])
def test_ragged_batches_and_ranges_that_end_anywhere(B):
    """Ranges of CTAs and of warps that begin and end inside rows, at their
    edges, hold many rows or part of one; empty sequences at the front, at the
    end and in between."""
    r = np.random.default_rng(B)
    lens = r.integers(0, 260, B)
    lens[r.random(B) < 0.3] = 0
    if B > 1:
        lens[0] = lens[-1] = 0
        lens[B // 2] = 1500
    else:
        lens[:] = 1500
    for Hkv, G, D in ((1, 4, 64), (3, 8, 128), (2, 16, 64)):
        c = Cache(list(lens), Hkv * G, Hkv, D, 1500, seed=800 + B).on_device()
        ref = c.oracle()
        for S in (1, 2, 3, 16, 300):
            check(*decode(c, S), ref, f"B={B} Hkv={Hkv} G={G} S={S}")


def test_ranges_that_end_with_rows():
    """Rows of 1, 2, 4 and 8 units: the ranges' ends fall on the rows' ends."""
    for n in (64, 128, 256, 512, 2048):
        c = Cache([n] * 4, 8, 1, 128, n, seed=850 + n).on_device()
        ref = c.oracle()
        for S in (1, 2, 4, 8, 16, 64):
            check(*decode(c, S), ref, f"n={n} S={S}")


def test_two_streams_and_a_stream_that_is_not_current():
    t = torch()
    cs = [Cache([2000, 700], 16, 2, 128, 2000, seed=710 + i).on_device() for i in range(2)]
    refs = [c.oracle() for c in cs]
    streams = [t.cuda.Stream() for _ in cs]
    t.cuda.synchronize()
    got = []
    for _ in range(5):
        got = [fd.decode_int4(c.dq, c.dk, c.dv, c.dp, c.dl, scale=c.scale, num_splits=6, stream=s)
               for c, s in zip(cs, streams)]
    t.cuda.synchronize()
    for g, r in zip(got, refs):
        check(*g, r, "streams")


def test_outputs_and_workspace_have_exact_bounds():
    t = torch()
    c = Cache([200, 1], 8, 2, 64, 200, seed=720).on_device()
    S, guard = 3, 64
    need = fd.fd_workspace_bytes(c.B, c.Hq, c.D, S)
    ws = t.full((need // 4 + 2 * guard,), 123.0, device="cuda")
    out = t.full((c.B * c.Hq * c.D + 2 * guard,), 5.0, dtype=t.bfloat16, device="cuda")
    lse = t.full((c.B * c.Hq + 2 * guard,), 9.0, device="cuda")
    o = out[guard:-guard].view(c.B, c.Hq, c.D)
    l = lse[guard:-guard].view(c.B, c.Hq)
    decode(c, S, out=o, lse=l, workspace=ws[guard:-guard])
    check(o, l, c.oracle(), "bounds")
    for buf, v in ((ws, 123.0), (out, 5.0), (lse, 9.0)):
        assert (buf[:guard] == v).all() and (buf[-guard:] == v).all()


def test_capture_and_replay_with_other_lengths():
    t = torch()
    c = Cache([500, 130], 16, 2, 128, 1000, seed=730, block_size=16).on_device()
    out, lse = t.empty_like(c.dq), t.empty((c.B, c.Hq), device="cuda")
    ws = t.empty(fd.fd_workspace_bytes(c.B, c.Hq, c.D, 5) // 4, device="cuda")
    run = lambda: fd.decode_int4(c.dq, c.dk, c.dv, c.dp, c.dl, c.dt, max_len=c.max_len,  # noqa: E731
                                 scale=c.scale, num_splits=5, out=out, lse=lse, workspace=ws)
    run()
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        run()
    for lens in ([500, 130], [17, 0], [499, 64]):
        c.dl.copy_(t.tensor(lens, dtype=t.int32))
        c.lens = lens
        out.zero_()
        g.replay()
        t.cuda.synchronize()
        check(out, lse, c.oracle(), f"replay {lens}")


def test_clusters_captured_and_on_two_streams():
    """num_splits = 1 with a cluster per row: one graph replayed with other lengths
    (rows that leave CTAs of the cluster idle among them), while a second stream runs
    the same rows; nothing is shared between the two but the inputs."""
    t = torch()
    c = Cache([3000, 3000, 2999, 2049], 8, 2, 128, 3000, seed=735).on_device()
    outs = [t.empty_like(c.dq) for _ in range(2)]
    lses = [t.empty((c.B, c.Hq), device="cuda") for _ in range(2)]
    side = t.cuda.Stream()
    run = lambda i, s=None: fd.decode_int4(c.dq, c.dk, c.dv, c.dp, c.dl, scale=c.scale,  # noqa: E731
                                           num_splits=1, out=outs[i], lse=lses[i], stream=s)
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        run(0)
    for lens in ([3000, 130, 0, 2049], [1, 0, 0, 64], [0, 0, 0, 0], [65, 3000, 2999, 513]):
        c.dl.copy_(t.tensor(lens, dtype=t.int32))
        c.lens = lens
        for x in outs:
            x.fill_(7.0)
        t.cuda.synchronize()
        for _ in range(20):
            g.replay()
            run(1, side)
        t.cuda.synchronize()
        ref = c.oracle()
        for i in range(2):
            check(outs[i], lses[i], ref, f"{lens} {i}")
        assert t.equal(outs[0], outs[1]) and t.equal(lses[0], lses[1])
    assert fd.fd_check_device_error() == fd.FD_OK


def test_slots_past_32_bits_of_bytes():
    """Rows whose byte offset does not fit 32 bits: a contiguous cache of 4.8 GB
    of codes a tensor, of which the last rows are used."""
    t = torch()
    planes, Hkv, L, D = 3, 8, 3_200_000, 128
    shape = (planes, Hkv, L)
    k4 = t.zeros(shape + (D // 2,), dtype=t.uint8, device="cuda")
    v4, prm = t.zeros_like(k4), t.zeros(shape + (8,), dtype=t.bfloat16, device="cuda")
    n = 70
    c = Cache([n], 8, 8, D, n, seed=740).on_device()
    kx, vx = up(c.k[0].transpose(1, 0, 2).copy()), up(c.v[0].transpose(1, 0, 2).copy())
    # the rows as the first of the last plane
    slots = t.arange(n, device="cuda") + (planes - 1) * L
    fd.append_int4(kx, vx, slots, k4, v4, prm)
    q = t.zeros((planes, 8, D), dtype=t.bfloat16, device="cuda")
    q[-1] = c.dq[0]
    lens = t.tensor([0, 0, n], dtype=t.int32, device="cuda")
    out, lse = fd.decode_int4(q, k4, v4, prm, lens, scale=c.scale, num_splits=4)
    t.cuda.synchronize()
    check(out[-1:], lse[-1:], c.oracle(), "far rows")
    assert (out[:-1] == 0).all()

"""fd_alloc_pages and fd_release_pages against the oracle's plain loops, and a
serving loop that uses them with the 4-bit cache."""
import numpy as np
import pytest

import split_kv_decode_attn_b200 as fd
from oracle import int4
from split_kv_decode_attn_b200 import workloads as wl

from int4test import HND, NHD, bits, check, rows, torch, up

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_device):
    yield


def setting(r, B, bs, blocks, spare, full=0.9):
    """Requests that hold tokens, their table rows (-1 elsewhere) and the stack."""
    lens = r.integers(0, int(full * blocks * bs) + 1, B).astype(np.int32)
    held = -(-lens // bs)
    pages = int(held.sum()) + spare
    perm = r.permutation(pages).astype(np.int32)
    table = np.full((B, blocks), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = np.full(pages, -7, np.int32)
    free[:spare] = perm[at:]
    return lens, table, free, spare


def run_alloc(lens, new, table, free, count, bs, T, in_place):
    t = torch()
    dl, dn, dt, df, dc = up(lens), up(new), up(table), up(free), up(np.array([count], np.int32))
    kw = dict(seqlens_out=dl, free_count_out=dc) if in_place else {}
    slots, pos, cu, out, left = fd.alloc_pages(dl, dn, dt, df, dc, block_size=bs, max_tokens=T, **kw)
    t.cuda.synchronize()
    assert np.array_equal(df.cpu().numpy(), free)
    if not in_place:
        assert np.array_equal(dl.cpu().numpy(), lens) and int(dc) == count
    return [x.cpu().numpy() for x in (slots, pos, cu, out, left, dt)]


def check_alloc(lens, new, table, free, count, bs, T, what=""):
    ref = int4.alloc(lens, new, table, free, count, bs, T)
    for in_place in (False, True):
        got = run_alloc(lens, new, table, free, count, bs, T, in_place)
        for g, x, name in zip(got, ref, ("slots", "positions", "cu", "seqlens", "count", "table")):
            assert np.array_equal(g, np.asarray(x).reshape(g.shape)), f"{what} {name} in_place={in_place}"


@pytest.mark.parametrize("B", [1, 2, 31, 33, 257, 1024, 1025, 2500])
@pytest.mark.parametrize("most", [1, 40])
def test_alloc_matches_the_plain_loop(B, most):
    r = np.random.default_rng(B + most)
    for bs in (8, 32, 256):
        lens, table, free, spare = setting(r, B, bs, 9, spare=B * (2 + most // bs))
        new = r.integers(0 if most > 1 else 1, most + 1, B).astype(np.int32)
        check_alloc(lens, new, table, free, spare, bs, int(new.sum()) + 5, f"B={B} bs={bs}")


def test_alloc_when_the_pool_the_table_or_the_list_runs_out():
    r = np.random.default_rng(3)
    for B in (5, 300, 1500):
        lens, table, free, _ = setting(r, B, 16, 6, spare=B)
        new = r.integers(0, 120, B).astype(np.int32)
        total = int(new.sum())
        for count in (0, 1, B // 2, B):                      # the pool
            check_alloc(lens, new, table, free, count, 16, total, f"pool {count}")
        for T in (0, 1, total // 2, total - 1):              # the list
            check_alloc(lens, new, table, free, B, 16, T, f"list {T}")


def test_alloc_of_odd_inputs():
    r = np.random.default_rng(4)
    lens, table, free, spare = setting(r, 40, 8, 5, spare=60)
    new = r.integers(-3, 9, 40).astype(np.int32)
    lens[3], lens[4], new[5], new[6] = -9, 2 ** 31 - 1, -2 ** 31, 0
    check_alloc(lens, new, table, free, spare, 8, 300, "odd")
    check_alloc(lens, new, table, free, len(free) + 100, 8, 300, "count above the pool")
    check_alloc(lens, new, table, free, -5, 8, 300, "count below 0")
    new[7] = 2 ** 31 - 1                                     # more than the list holds
    check_alloc(lens, new, table, free, spare, 8, 300, "huge")


def test_alloc_of_long_prompts_over_many_ctas():
    r = np.random.default_rng(5)
    for B, most in ((3, 200_000), (70, 9000), (1300, 500)):
        lens, table, free, spare = setting(r, B, 64, 4000, spare=B * (most // 64 + 2), full=0.01)
        new = r.integers(0, most, B).astype(np.int32)
        check_alloc(lens, new, table, free, spare, 64, int(new.sum()) + 3000, f"B={B}")


@pytest.mark.parametrize("B", [1, 40, 1024, 1100, 3000])
def test_release_matches_the_plain_loop(B):
    r = np.random.default_rng(B)
    for blocks, spare in ((4, 10), (200, 3)):
        lens, table, free, _ = setting(r, B, 16, blocks, spare)
        for share in (0.0, 0.3, 1.0):
            done = (r.random(B) < share).astype(np.uint8)
            ref = int4.release(lens, done, table, free, spare, 16)
            for in_place in (False, True):
                dl, df, dc = up(lens), up(free), up(np.array([spare], np.int32))
                kw = dict(seqlens_out=dl, free_count_out=dc) if in_place else {}
                out, left = fd.release_pages(dl, up(done), up(table), df, dc, block_size=16, **kw)
                torch().cuda.synchronize()
                assert np.array_equal(out.cpu().numpy(), ref[0])
                assert int(left) == ref[1] and np.array_equal(df.cpu().numpy(), ref[2])


def test_release_drops_what_does_not_fit():
    r = np.random.default_rng(9)
    lens, table, free, spare = setting(r, 20, 8, 10, 5)
    for room in (spare, spare + 7):
        f = free[:room].copy()
        ref = int4.release(lens, np.ones(20, bool), table, f, spare, 8)
        df = up(f)
        out, left = fd.release_pages(up(lens), up(np.ones(20, np.uint8)), up(table), df,
                                     up(np.array([spare], np.int32)), block_size=8)
        torch().cuda.synchronize()
        assert int(left) == ref[1] == room and np.array_equal(df.cpu().numpy(), ref[2])


@pytest.mark.parametrize("layout", [HND, NHD])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(layout, captured):
    """Requests come, grow by a token a step and leave: pages, slots, quantised
    rows and attention in one run, eager and as one captured graph per step.
    The oracle keeps every request's rows itself."""
    t = torch()
    r = np.random.default_rng(11)
    B, Hkv, G, D, bs, blocks, T = 6, 2, 4, 128, 8, 20, 64
    pages = 70
    scale = 1.0 / D ** 0.5
    shape = (pages, Hkv, bs) if layout == HND else (pages, bs, Hkv)
    k4 = t.zeros(shape + (D // 2,), dtype=t.uint8, device="cuda")
    v4, prm = t.zeros_like(k4), t.zeros(shape + (8,), dtype=t.bfloat16, device="cuda")
    table = t.full((B, blocks), -1, dtype=t.int32, device="cuda")
    free = up(r.permutation(pages).astype(np.int32))
    count = up(np.array([pages], np.int32))
    lens, new = up(np.zeros(B, np.int32)), up(np.zeros(B, np.int32))
    done = up(np.zeros(B, np.uint8))
    k_new, v_new = (t.zeros((T, Hkv, D), dtype=t.bfloat16, device="cuda") for _ in range(2))
    q = t.zeros((B, Hkv * G, D), dtype=t.bfloat16, device="cuda")
    buf = dict(cu_new=t.zeros(B + 1, dtype=t.int32, device="cuda"),
               slots=t.zeros(T, dtype=t.int64, device="cuda"),
               positions=t.zeros(T, dtype=t.int32, device="cuda"))
    out, lse = t.empty_like(q), t.empty((B, Hkv * G), device="cuda")
    S = 3
    ws = t.empty(fd.fd_workspace_bytes(B, Hkv * G, D, S) // 4, device="cuda")

    def one_step():
        fd.release_pages(lens, done, table, free, count, block_size=bs, seqlens_out=lens,
                         free_count_out=count)
        fd.alloc_pages(lens, new, table, free, count, block_size=bs, max_tokens=T,
                       seqlens_out=lens, free_count_out=count, **buf)
        fd.append_int4(k_new, v_new, buf["slots"], k4, v4, prm, kv_layout=layout)
        fd.decode_int4(q, k4, v4, prm, lens, table, kv_layout=layout, scale=scale, num_splits=S,
                       out=out, lse=lse, workspace=ws)

    one_step()                     # nothing held yet: an empty step
    t.cuda.synchronize()
    assert (out == 0).all() and t.isneginf(lse).all()
    go = one_step
    if captured:
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            one_step()
        go = g.replay
    held = [None] * B              # per request: K codes, K records, V codes, V records
    for turn in range(14):
        gone = np.array([h is not None and r.random() < 0.15 for h in held])
        grow = np.array([1 if h is not None and not x else (int(r.integers(0, 9)) if r.random() < 0.6
                         else 0) for h, x in zip(held, gone)], np.int32)
        x, y = rows(1000 + turn, (T, Hkv, D)), rows(2000 + turn, (T, Hkv, D))
        qq = wl.f64_to_bf16_bits(r.standard_normal((B, Hkv * G, D)))
        done.copy_(t.from_numpy(gone.astype(np.uint8)))
        new.copy_(t.from_numpy(grow))
        for dst, src in ((k_new, x), (v_new, y), (q, qq)):
            dst.copy_(up(src))
        go()
        t.cuda.synchronize()
        at = 0
        for b in range(B):
            if gone[b]:
                held[b] = None
            n = int(grow[b])
            if n:
                (kc, kr), (vc, vr) = int4.quantise(x[at:at + n]), int4.quantise(y[at:at + n])
                add = [int4.pack(kc), kr, int4.pack(vc), vr]
                held[b] = add if held[b] is None else [np.concatenate(p) for p in zip(held[b], add)]
                at += n
        ref = [[] for _ in range(4)]
        for b in range(B):
            for h in range(Hkv):
                rowsets = [p[:, h] for p in held[b]] if held[b] is not None else \
                    [np.zeros((0, w), d) for w, d in ((D // 2, np.uint8), (4, np.uint16)) * 2]
                res = int4.attend(qq[b, h * G:(h + 1) * G], *rowsets, scale)
                for lst, v in zip(ref, res):
                    lst.append(v)
        o, l, tol, ltol = (np.concatenate(p).reshape((B, Hkv * G) + p[0].shape[1:]) for p in ref)
        check(out, lse, (o, l, tol, ltol), f"turn {turn}")
        n_held = [0 if h is None else len(h[0]) for h in held]
        assert np.array_equal(lens.cpu().numpy(), n_held)
        assert int(count) == pages - sum(-(-n // bs) for n in n_held)
    assert fd.fd_check_device_error() == fd.FD_OK


FIRST_CALLS = """
import torch, split_kv_decode_attn_b200 as fd
B, Hkv, G, D, bs, blocks = 6, 8, 2, 128, 16, 20
i32 = dict(dtype=torch.int32, device="cuda")
k4 = torch.zeros(B * blocks, Hkv, bs, D // 2, dtype=torch.uint8, device="cuda")
v4, prm = torch.zeros_like(k4), torch.zeros(B * blocks, Hkv, bs, 8, dtype=torch.bfloat16, device="cuda")
torch.manual_seed(0)
x = torch.randn(100 * B, Hkv, D, device="cuda").to(torch.bfloat16)
q = torch.randn(B, Hkv * G, D, device="cuda").to(torch.bfloat16)
lens, new, done = torch.zeros(B, **i32), torch.full((B,), 100, **i32), torch.zeros(B, dtype=torch.uint8, device="cuda")
free, count, table = torch.arange(B * blocks, **i32), torch.full((1,), B * blocks, **i32), torch.full((B, blocks), -1, **i32)
slots, cu = torch.zeros(100 * B, dtype=torch.int64, device="cuda"), torch.zeros(B + 1, **i32)
ko = torch.zeros(B, Hkv, blocks * bs, D, dtype=torch.bfloat16, device="cuda")
vo = torch.zeros_like(ko)
outs = {S: torch.empty_like(q) for S in (1, 2, 60)}
lse = torch.empty(B, Hkv * G, device="cuda")
ws = torch.empty(fd.fd_workspace_bytes(B, Hkv * G, D, 60), dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    fd.release_pages(lens, done, table, free, count, block_size=bs, seqlens_out=lens, free_count_out=count)
    fd.alloc_pages(lens, new, table, free, count, block_size=bs, max_tokens=100 * B, seqlens_out=lens,
                   cu_new=cu, slots=slots, free_count_out=count)
    fd.append_int4(x, x, slots, k4, v4, prm)
    for S, out in outs.items():
        fd.decode_int4(q, k4, v4, prm, lens, table, num_splits=S, out=out, lse=lse, workspace=ws)
    fd.expand_int4(k4, v4, prm, lens, table, k_out=ko, v_out=vo)
for turn in range(3):
    g.replay()
    torch.cuda.synchronize()
    n = 100 * (turn + 1)
    assert lens.tolist() == [n] * B and int(count) == B * (blocks - -(-n // bs))
    assert (ko[:, :, :n].float() - x.view(B, 100, Hkv, D).transpose(1, 2).repeat(1, 1, turn + 1, 1).float()).abs().max() < 0.5
    # Two roundings to bf16, 2^-9 each below 1 and 2^-8 from 1 to 2, and the weights' 2^-11 of |v|, mean 0.8, twice
    # (below 1: 2 2^-9 + 2 2^-11 0.8 = 4.7e-3; from 1 to 2: 2 2^-8 + 2 2^-11 0.8 = 8.6e-3).
    top = outs[1].float().abs().max().item()
    assert top < 2
    for out in outs.values():
        assert (out.float() - outs[1].float()).abs().max() < (6e-3 if top < 1 else 9e-3), turn
assert fd.fd_check_device_error() == fd.FD_OK
print("fine")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    import subprocess
    import sys
    got = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "fine" in got.stdout, got.stderr[-2000:]

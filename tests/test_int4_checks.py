"""Refusals of the 4-bit cache and page entry points (CPU: every call below is
stopped by a check on the host), through the C ABI and the torch wrappers."""
import ctypes

import pytest
import torch

import split_kv_decode_attn_b200 as fd

BAD, UNSUP = fd.FD_ERR_INVALID_ARGUMENT, fd.FD_ERR_UNSUPPORTED
Q, K, V, R, O, W, S, T = (0x10000 * i for i in range(1, 9))   # never dereferenced


def P(B=1, Hq=8, Hkv=8, D=128, L=512, bs=0, nb=0, mb=0, layout=0, kv=fd.FD_KV_INT4):
    return fd.make_problem(B, Hq, Hkv, D, L, bs, nb, mb, layout, kv)


def decode(p, q=Q, k=K, v=V, r=R, sl=None, table=None, scale=0.125, S=1, out=O, lse=None, ws=None,
           wsb=0):
    return fd.load_library().fd_decode_int4(ctypes.byref(p) if p else None, q, k, v, r, sl, table,
                                            scale, S, out, lse, ws, wsb, None)


def test_enum_matches_header_and_other_entry_points_refuse_it():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "fd.h")).read()
    assert int(re.search(r"\bFD_KV_INT4\s*=\s*(\d+)", text).group(1)) == fd.FD_KV_INT4
    lib = fd.load_library()
    p = P()
    assert lib.fd_decode(ctypes.byref(p), Q, K, V, None, None, 0.1, 1, O, None, None, 0, None) == BAD
    assert lib.fd_decode_partial(ctypes.byref(p), Q, K, V, None, None, 0.1, 1, O, W, None, 0,
                                 None) == BAD
    assert lib.fd_quantize_keys(ctypes.byref(p), K, None, V, R, None) == UNSUP


def test_what_the_header_says_other_entry_points_return_for_it():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = " ".join(open(os.path.join(root, "include", "fd.h")).read().replace("\n *", " ").split())
    said = re.search(r"For FD_KV_INT4 ([^.]*) return it too, and (\w+) returns (\w+)", text)
    assert said and said.group(2) == "fd_quantize_keys" and said.group(3) == "FD_ERR_UNSUPPORTED"
    lib, p = fd.load_library(), ctypes.byref(P())
    got = {"fd_decode": lib.fd_decode(p, Q, K, V, None, None, 0.1, 1, O, None, None, 0, None),
           "fd_decode_partial": lib.fd_decode_partial(p, Q, K, V, None, None, 0.1, 1, O, W, None, 0,
                                                      None),
           "fd_decode_sparse": lib.fd_decode_sparse(p, Q, K, V, W, S, None, 0.1, 1.0, 1, O, None,
                                                    None, None, 0, None)}
    for name, status in got.items():     # fd_decode_static_workspace asks the device first
        assert name in said.group(1) and status == BAD, name
    assert lib.fd_quantize_keys(p, K, None, V, R, None) == UNSUP


def test_decode_int4_refusals():
    assert decode(None) == BAD
    for name in ("q", "k", "v", "r", "out"):
        assert decode(P(), **{name: None}) == BAD, name
    for name, at in (("q", Q + 8), ("k", K + 8), ("v", V + 4), ("r", R + 8), ("out", O + 2),
                     ("lse", W + 2), ("sl", W + 1)):
        assert decode(P(), **{name: at}) == BAD, name
    for kv in (fd.FD_KV_BF16, fd.FD_KV_FP8_E4M3, 3, -1):
        assert decode(P(kv=kv)) == BAD
    assert decode(P(layout=2)) == BAD
    assert decode(P(Hq=12)) == BAD and decode(P(B=0)) == BAD and decode(P(L=-1)) == BAD
    assert decode(P(D=96)) == UNSUP and decode(P(Hq=256)) == UNSUP
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert decode(P(), scale=scale) == BAD
    assert decode(P(), S=0) == BAD and decode(P(), S=1025) == BAD
    # paging
    assert decode(P(), table=T) == BAD and decode(P(bs=16, nb=64, mb=32)) == BAD
    assert decode(P(bs=16, nb=64, mb=8), table=T) == BAD       # table too short for max_len
    assert decode(P(bs=16, nb=0, mb=32), table=T) == BAD
    assert decode(P(bs=12, nb=64, mb=64), table=T) == UNSUP
    # workspace
    need = fd.fd_workspace_bytes(1, 8, 128, 8)
    assert decode(P(), S=8) == fd.FD_ERR_WORKSPACE
    assert decode(P(), S=8, ws=W, wsb=need - 1) == fd.FD_ERR_WORKSPACE
    assert decode(P(), S=8, ws=W + 8, wsb=need) == BAD


def test_append_int4_refusals():
    lib = fd.load_library()

    def append(p=P(), n=4, k=Q, ks=1024, v=W, vs=1024, slots=S, k4=K, v4=V, r=R):
        return lib.fd_append_int4(ctypes.byref(p) if p else None, n, k, ks, v, vs, slots, k4, v4, r,
                                  None)
    assert append(p=None) == BAD and append(n=-1) == BAD
    for name in ("k", "v", "slots", "k4", "v4", "r"):
        assert append(**{name: None}) == BAD, name
    for name, at in (("k", Q + 8), ("v", W + 2), ("slots", S + 4), ("k4", K + 8), ("v4", V + 1),
                     ("r", R + 2)):
        assert append(**{name: at}) == BAD, name
    for stride in (1020, 1016, 0, -1024):              # not a multiple of 8; tokens overlap
        assert append(ks=stride) == BAD and append(vs=stride) == BAD, stride
    assert append(p=P(kv=fd.FD_KV_BF16)) == BAD and append(p=P(D=96)) == UNSUP
    assert append(n=0) == fd.FD_OK                     # nothing to do, nothing launched
    assert append(p=P(L=0)) == fd.FD_OK


def test_expand_int4_refusals():
    lib = fd.load_library()

    def expand(p=P(), k4=K, v4=V, r=R, sl=None, table=None, k=Q, v=W):
        return lib.fd_expand_int4(ctypes.byref(p) if p else None, k4, v4, r, sl, table, k, v, None)
    assert expand(p=None) == BAD
    for name in ("k4", "v4", "r", "k", "v"):
        assert expand(**{name: None}) == BAD, name
    assert expand(k=Q + 8) == BAD and expand(v=W + 2) == BAD and expand(sl=S + 2) == BAD
    assert expand(table=T) == BAD and expand(p=P(bs=16, nb=64, mb=32)) == BAD
    assert expand(p=P(kv=fd.FD_KV_FP8_E4M3)) == BAD and expand(p=P(D=32)) == UNSUP
    assert expand(p=P(L=0)) == fd.FD_OK


def test_page_refusals():
    lib = fd.load_library()
    names = ("seqlens", "new_lens", "free_pages", "free_count", "block_table", "seqlens_out",
             "cu_new", "slots", "positions", "free_count_out")

    def alloc(B=4, bs=16, mb=8, mt=64, pages=100, **kw):
        at = {n: 0x1000 * (i + 1) for i, n in enumerate(names)}
        at.update(kw)
        return lib.fd_alloc_pages(B, bs, mb, mt, pages, *[at[n] for n in names], None)
    assert alloc(B=0) == BAD and alloc(B=65536) == BAD and alloc(mb=0) == BAD
    assert alloc(mt=-1) == BAD and alloc(pages=0) == BAD and alloc(bs=0) == BAD
    assert alloc(bs=12) == UNSUP and alloc(bs=512) == UNSUP and alloc(bs=4) == UNSUP
    for n in names:
        if n != "positions":
            assert alloc(**{n: None}) == BAD, n
        assert alloc(**{n: 0x9002}) == BAD, n
    assert alloc(slots=0x9004) == BAD

    rel = ("seqlens", "done", "block_table", "free_pages", "free_count", "seqlens_out",
           "free_count_out")

    def release(B=4, bs=16, mb=8, pages=100, **kw):
        at = {n: 0x1000 * (i + 1) for i, n in enumerate(rel)}
        at.update(kw)
        return lib.fd_release_pages(B, bs, mb, pages, *[at[n] for n in rel], None)
    assert release(B=0) == BAD and release(bs=24) == UNSUP and release(pages=0) == BAD
    for n in rel:
        assert release(**{n: None}) == BAD, n
        if n != "done":
            assert release(**{n: 0x9002}) == BAD, n


def test_planner_takes_4_bit_caches():
    """The least count whose workspace serves a CTA on each of the 148 SMs (two
    partial results each; two for each of eight KV heads with Hkv a multiple of 8
    and five such rows); short histories and few rows keep one cluster per row."""
    def plan(B, Hkv, L, lens=None, D=128):
        return fd.fd_plan_problem(148, fd.make_problem(B, 8 * Hkv, Hkv, D, L, kv_dtype=fd.FD_KV_INT4),
                                  lens)
    for B, Hkv, heads in ((1, 1, 1), (1, 8, 1), (4, 8, 1), (3, 5, 1), (9, 12, 1), (5, 8, 8),
                          (2, 16, 1), (3, 16, 8), (32, 8, 8), (64, 8, 8), (4096, 8, 8)):
        S = plan(B, Hkv, 65536)
        assert 2 <= S <= 1024
        assert B * Hkv * S // (2 * heads) >= 148
        assert S == 2 or B * Hkv * (S - 1) // (2 * heads) < 148
    assert plan(1, 8, 0) == plan(1, 8, 1) == plan(1, 8, 512) == plan(18, 8, 512, D=64) == 1
    assert plan(1, 8, 12288) == 1 and plan(1, 8, 12289) > 1 and plan(19, 8, 512) > 1
    assert plan(2, 8, 65536, [6144, 7]) == 1 and plan(2, 8, 65536, [6145, 7]) > 1
    assert plan(18, 8, 4096) == 1 and plan(18, 8, 65536) > 1
    assert plan(18, 8, 4096, [4096] + 17 * [7]) > 1
    assert plan(2, 8, 65536, [-4, 0]) == 1
    assert fd.fd_plan_problem(148, P(D=96)) == UNSUP


# ---- torch wrappers ------------------------------------------------------------

def cache(planes=2, Hkv=2, rows=256, D=128):
    return (torch.zeros(planes, Hkv, rows, D // 2, dtype=torch.uint8),
            torch.zeros(planes, Hkv, rows, D // 2, dtype=torch.uint8),
            torch.zeros(planes, Hkv, rows, 8, dtype=torch.bfloat16))


def raises(match, f, *a, **kw):
    with pytest.raises(ValueError, match=match):
        f(*a, **kw)


def test_decode_int4_wrapper():
    k4, v4, r = cache()
    q = torch.zeros(2, 16, 128, dtype=torch.bfloat16)
    raises("CUDA device", fd.decode_int4, q, k4, v4, r)
    raises("q: expected", fd.decode_int4, q[0], k4, v4, r)
    raises("q: dtype", fd.decode_int4, q.float(), k4, v4, r)
    raises("k4: dtype", fd.decode_int4, q, k4.int(), v4, r)
    raises("k4: expected 4", fd.decode_int4, q, k4[0], v4, r)
    raises("v4: shape", fd.decode_int4, q, k4, v4[:, :1].contiguous(), r)
    raises("params: shape", fd.decode_int4, q, k4, v4, r[..., :4].contiguous())
    raises("params: dtype", fd.decode_int4, q, k4, v4, r.float())
    raises("head dim", fd.decode_int4, q[..., :64].contiguous(), k4, v4, r)
    raises("sequences", fd.decode_int4, q[:1].contiguous(), k4, v4, r)
    raises("max_len", fd.decode_int4, q, k4, v4, r, max_len=100)
    raises("kv_layout", fd.decode_int4, q, k4, v4, r, kv_layout=3)
    raises("contiguous", fd.decode_int4, q, k4.transpose(1, 2), v4.transpose(1, 2), r)
    raises("seqlens: dtype", fd.decode_int4, q, k4, v4, r, torch.zeros(2))
    raises("block_table: expected", fd.decode_int4, q, *cache(9, 2, 16), None,
           torch.zeros(3, 4, dtype=torch.int32))
    raises("lse: dtype", fd.decode_int4, q, k4, v4, r, lse=torch.zeros(2, 16).double())


def test_append_and_expand_wrappers():
    k4, v4, r = cache(9, 2, 16)
    new = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    raises("CUDA device", fd.append_int4, new, new, slots, k4, v4, r)
    fused = torch.zeros(3, 8 * 128, dtype=torch.bfloat16)
    raises("CUDA device", fd.append_int4, fused[:, :256].unflatten(1, (2, 128)),
           fused[:, 256:512].unflatten(1, (2, 128)), slots, k4, v4, r)
    raises("slots: dtype", fd.append_int4, new, new, slots.int(), k4, v4, r)
    raises("slots: shape", fd.append_int4, new, new, slots[:2], k4, v4, r)
    raises("k_new: dtype", fd.append_int4, new.float(), new, slots, k4, v4, r)
    raises("k_new: shape", fd.append_int4, new[:, :1], new, slots, k4, v4, r)
    raises("v_new: 2 tokens", fd.append_int4, new, new[:2], slots, k4, v4, r)
    raises("dense", fd.append_int4, new, torch.zeros(2, 3, 128, dtype=torch.bfloat16).transpose(0, 1),
           slots, k4, v4, r)
    odd = torch.zeros(3, 300, dtype=torch.bfloat16)[:, :256].unflatten(1, (2, 128))
    raises("token stride 300", fd.append_int4, odd, new, slots, k4, v4, r)
    raises("token stride 0", fd.append_int4, new[:1].expand(3, 2, 128), new, slots, k4, v4, r)
    raises("CUDA device", fd.expand_int4, k4, v4, r)
    raises("k_out: shape", fd.expand_int4, k4, v4, r, k_out=torch.zeros(1, dtype=torch.bfloat16))
    raises("seqlens: shape", fd.expand_int4, k4, v4, r, torch.zeros(3, dtype=torch.int32))


def test_page_wrappers():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    kw = dict(block_size=16, max_tokens=8)
    raises("CUDA device", fd.alloc_pages, i(4), i(4), i(4, 5), i(30), i(1), **kw)
    raises("new_lens: shape", fd.alloc_pages, i(4), i(3), i(4, 5), i(30), i(1), **kw)
    raises("block_table: expected", fd.alloc_pages, i(4), i(4), i(3, 5), i(30), i(1), **kw)
    raises("free_count: shape", fd.alloc_pages, i(4), i(4), i(4, 5), i(30), i(2), **kw)
    raises("seqlens: dtype", fd.alloc_pages, i(4).long(), i(4), i(4, 5), i(30), i(1), **kw)
    raises("slots: dtype", fd.alloc_pages, i(4), i(4), i(4, 5), i(30), i(1), slots=i(8), **kw)
    raises("max_tokens", fd.alloc_pages, i(4), i(4), i(4, 5), i(30), i(1), block_size=16,
           max_tokens=-1)
    raises("done: dtype", fd.release_pages, i(4), i(4), i(4, 5), i(30), i(1), block_size=16)
    raises("CUDA device", fd.release_pages, i(4), torch.zeros(4, dtype=torch.bool), i(4, 5), i(30),
           i(1), block_size=16)

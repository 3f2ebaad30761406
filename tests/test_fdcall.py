"""The native calls behind the 4-bit cache and the page bookkeeping: conversions of
their arguments, and the same status as the C entry point for the same arguments
(CPU: every call is refused before it looks at a device)."""
import ctypes

import pytest
import torch

import split_kv_decode_attn_b200 as fd

X = torch.zeros(64, dtype=torch.int64)
A = X.data_ptr()


def problem(**kw):
    p = fd.make_problem(1, 8, 8, 128, 64, kv_dtype=fd.FD_KV_INT4)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def append(p=None, n=1, k=X, ks=1024, v=X, vs=1024, slots=X, k4=X, v4=X, params=X):
    return (p or problem()), n, k, ks, v, vs, slots, k4, v4, params


def expand(p=None, k4=X, v4=X, params=X, seqlens=X, table=None, k=X, v=X):
    return (p or problem()), k4, v4, params, seqlens, table, k, v


def decode(p=None, q=X, k4=X, v4=X, params=X, seqlens=X, table=None, scale=1.0, splits=2, out=X,
           lse=X, work=X, size=1 << 30):
    return (p or problem()), q, k4, v4, params, seqlens, table, scale, splits, out, lse, work, size


def alloc(B=1, block=16, most=4, tokens=4, pages=4, seqlens=X, new=X, free=X, count=X, table=X,
          out=X, cu=X, slots=X, positions=X, count_out=X):
    return (B, block, most, tokens, pages, seqlens, new, free, count, table, out, cu, slots,
            positions, count_out)


def release(B=1, block=16, most=4, pages=4, seqlens=X, done=X, table=X, free=X, count=X, out=X,
            count_out=X):
    return B, block, most, pages, seqlens, done, table, free, count, out, count_out


# Every pointer on its own: NULL where it is needed, then an address that is not
# aligned, so that an argument in another's place would be seen.
REFUSED = (
    [("fd_append_int4", append(**{k: v})) for k, v in
     [("n", -1), ("k", None), ("k", A + 2), ("ks", 1023), ("ks", 8), ("v", None), ("v", A + 2),
      ("vs", 1023), ("vs", 8), ("slots", None), ("slots", A + 4), ("k4", None), ("v4", None),
      ("params", None), ("k4", A + 8), ("v4", A + 8), ("params", A + 8)]]
    + [("fd_expand_int4", expand(**{k: v})) for k, v in
       [("k4", None), ("v4", A + 8), ("params", None), ("seqlens", A + 2), ("table", X), ("k", None),
        ("v", None), ("k", A + 2), ("v", A + 2)]]
    + [("fd_decode_int4", decode(**{k: v})) for k, v in
       [("q", None), ("k4", A + 8), ("v4", None), ("params", A + 8), ("seqlens", A + 2), ("table", X),
        ("scale", 0.0), ("scale", float("nan")), ("splits", 0), ("splits", 1025), ("out", None),
        ("lse", A + 2), ("work", None), ("size", 64)]]
    + [("fd_alloc_pages", alloc(**{k: v})) for k, v in
       [("B", 0), ("block", 12), ("most", 0), ("tokens", -1), ("pages", 0), ("seqlens", None),
        ("new", None), ("free", None), ("count", None), ("table", None), ("out", None), ("cu", None),
        ("slots", None), ("slots", A + 4), ("positions", A + 2), ("count_out", None)]]
    + [("fd_release_pages", release(**{k: v})) for k, v in
       [("B", 0), ("block", 512), ("most", 0), ("pages", 0), ("seqlens", None), ("done", None),
        ("table", None), ("free", None), ("count", None), ("out", None), ("count_out", A + 1)]]
    + [("fd_decode_int4", decode(p=problem(kv_dtype=fd.FD_KV_BF16))),
       ("fd_expand_int4", expand(p=problem(D=96))), ("fd_append_int4", append(p=problem(B=0)))])


@pytest.mark.parametrize("name,args", REFUSED)
def test_refusals_are_those_of_the_c_entry_point(name, args):
    want = getattr(fd.load_library(), name)(
        *(ctypes.byref(x) if isinstance(x, fd.fd_problem) else fd._ptr(x) if torch.is_tensor(x)
          else x for x in args), 1)
    assert want < 0
    assert getattr(fd, name)(*args, stream=1) == want


CALLS = [("fd_append_int4", append()), ("fd_expand_int4", expand()), ("fd_decode_int4", decode()),
         ("fd_alloc_pages", alloc()), ("fd_release_pages", release())]


@pytest.mark.parametrize("name,args", CALLS)
def test_arguments_of_the_wrong_kind_raise(name, args):
    call = getattr(fd, name)
    for i, x in enumerate(args):
        if isinstance(x, fd.fd_problem):
            wrong, error = [b"short", X, None], (TypeError, BufferError)
        elif torch.is_tensor(x) or x is None:
            wrong, error = ["text", 1.5, object()], AttributeError
        elif isinstance(x, float):
            wrong, error = ["text", None], TypeError
        else:
            wrong, error = ["text", None, 1.5, 1 << 70], (TypeError, OverflowError)
        for w in wrong:
            with pytest.raises(error):
                call(*args[:i], w, *args[i + 1:], stream=1)
    native = getattr(fd._load_calls(), name[3:])
    for bad in (args, args + (1, 1)):
        with pytest.raises(TypeError, match="arguments"):
            native(*bad)


def test_numbers_that_do_not_fit_a_c_int():
    for name, args in CALLS[3:]:
        with pytest.raises(OverflowError):
            getattr(fd, name)(1 << 31, *args[1:], stream=1)
    with pytest.raises(OverflowError):
        fd.fd_append_int4(*append(n=1 << 32), stream=1)
    assert fd.fd_decode_int4(*decode(size=-1), stream=1) == fd.FD_ERR_WORKSPACE

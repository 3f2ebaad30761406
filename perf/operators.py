"""Cases of the 4-bit KV cache operators and of the page bookkeeping beside it.

A row of the cache is one token of one KV head: D = 64 or 128 entries in two groups of D / 2, each
entry a 4-bit code c, each group a bf16 scale s and bias b; an entry stands for s (c - 8) + b.
The codes of K and of V are D / 2 bytes per row (entry 2j in the low nibble of byte j); the scales
and biases of both are one record of 8 bf16 per row: ks0 kb0 ks1 kb1 vs0 vb0 vs1 vb1.

Kinds of a case:
  attend  one query token per sequence attends over its 4-bit history
  step    one serving step: pages and slots for one new token per request, its K/V row quantised
          and written, attention over the history with it
  fill    the K/V rows of prompts are quantised and written, and the cache comes back as the bf16
          values it stands for (what the prompt's own attention reads)
  slots   pages, slots and positions for the new tokens of a batch of requests
  turn    finished requests give their pages back, then the batch's new tokens get theirs
"""
import math
import random

import torch

own = False

HND, NHD, KV_INT4 = 0, 1, 2


def attend(name, B, Hq, Hkv, D, longest, ragged, block_size=0, layout=HND):
    return dict(name=name, kind="attend", B=B, Hq=Hq, Hkv=Hkv, D=D, longest=longest,
                ragged=ragged, block_size=block_size, layout=layout, lens=1)


def step(name, B, Hq, Hkv, D, longest, block_size, layout=HND):
    return dict(name=name, kind="step", B=B, Hq=Hq, Hkv=Hkv, D=D, longest=longest, ragged=True,
                block_size=block_size, layout=layout, lens=2)


def fill(name, B, Hq, Hkv, D, longest, block_size, layout=HND):
    return dict(name=name, kind="fill", B=B, Hq=Hq, Hkv=Hkv, D=D, longest=longest, ragged=True,
                block_size=block_size, layout=layout, lens=3)


def slots(name, kind, B, longest, new, block_size):
    return dict(name=name, kind=kind, B=B, longest=longest, new=new, block_size=block_size, lens=4)


def listed():
    return [
        # one user, a short chat: latency is everything
        attend("attend-1x512", 1, 64, 8, 128, 512, False),
        # one user, a long document: one sequence has to fill the device
        attend("attend-1x64K", 1, 64, 8, 128, 65536, False),
        # a batch of unequal chats in a contiguous cache, an empty one among them
        attend("attend-32-ragged", 32, 32, 8, 128, 8192, True),
        # a few long documents, token-major pages of 16
        attend("attend-8-paged", 8, 32, 8, 128, 40000, True, 16, NHD),
        # multi-head attention with small heads and an odd length
        attend("attend-5-mha64", 5, 8, 8, 64, 3001, False),
        # a serving step of few and of many requests
        step("step-4", 4, 32, 8, 128, 1500, 16),
        step("step-64", 64, 64, 8, 128, 4096, 32, NHD),
        # prompts enter the cache: a short one with small heads, and a full batch
        fill("fill-short", 1, 8, 8, 64, 37, 8, NHD),
        fill("fill-prompts", 8, 64, 8, 128, 6000, 16),
        # page bookkeeping: a small decode batch, a large one, and many prompts
        slots("turn-16", "turn", 16, 2000, 1, 16),
        slots("turn-1024", "turn", 1024, 8000, 1, 16),
        slots("slots-prompts", "slots", 200, 4000, 2500, 64),
    ]


def between(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "step", "fill", "slots", "turn"])
    bs = rng.choice([8, 16, 32, 64, 128, 256])
    if kind in ("slots", "turn"):
        B = between(rng, 1, 1500)
        new = 1 if rng.random() < 0.4 else between(rng, 1, max(1, min(4000, 500000 // B)))
        c = slots("", kind, B, between(rng, 1, min(8000, 8000000 // B)), new, bs)
        return dict({k: v for k, v in c.items() if k != "name"}, lens=rng.randrange(1 << 20))
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    Hq, D, layout = Hkv * rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128, 128]), rng.choice([HND, NHD])
    if kind == "attend":
        B = between(rng, 1, 40)
        longest = between(rng, 1, max(1, min(70000, 1200000 // (B * Hkv))))
        c = attend("", B, Hq, Hkv, D, longest, rng.random() < 0.6, rng.choice([0, 0, bs]), layout)
    elif kind == "step":
        B = between(rng, 1, 128)
        c = step("", B, Hq, Hkv, D, between(rng, 1, max(1, 1200000 // (B * Hkv))), bs, layout)
    else:
        B = between(rng, 1, 16)
        c = fill("", B, Hq, Hkv, D, between(rng, 1, max(1, 180000 // (B * Hkv))), bs, layout)
    return dict({k: v for k, v in c.items() if k != "name"}, lens=rng.randrange(1 << 20))


def lengths(case):
    """Cached tokens of each request: sizes of the case, the same whatever the seed."""
    r, B, most = random.Random(case["lens"]), case["B"], case["longest"]
    if not case.get("ragged", True):
        return [most] * B
    lens = [r.randint(1, most) for _ in range(B)]
    lens[r.randrange(B)] = most
    if B > 3:
        lens[r.randrange(B)] = 0
    if B > 5:
        lens[r.randrange(B)] = 1
    return lens


def news(case):
    """New tokens of each request."""
    r, most = random.Random(case["lens"] + 1), case["new"]
    return [1 if most == 1 else r.randint(0, most) for _ in range(case["B"])]


def finished(case):
    r = random.Random(case["lens"] + 2)
    return [case["kind"] == "turn" and r.random() < 0.25 for _ in range(case["B"])]


def pages_of(n, bs):
    return -(-n // bs)


# ------------------------------------------------------------------- inputs

def rows_like(g, shape, channel):
    """K or V rows as a model makes them: channels of unequal size."""
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * channel).to(torch.bfloat16)


def quantise_rows(x):
    """Codes (0..15) and [scale, bias] of bf16 rows [..., D], two groups a row."""
    h = x.unflatten(-1, (2, x.shape[-1] // 2)).float()
    mn, mx = h.amin(-1, keepdim=True), h.amax(-1, keepdim=True)
    s = ((mx * 0.5 - mn * 0.5) / 7.5).to(torch.bfloat16)
    b = (mn.double() + 8 * s.double()).float().to(torch.bfloat16)
    sf, bf = s.float(), b.float()
    c = torch.where(sf > 0, torch.round((h - bf) / sf), torch.zeros_like(h)).clamp(-8, 7) + 8
    return c.flatten(-2).to(torch.uint8), torch.cat([s, b], -1).flatten(-2)


def pack(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def cache_of(g, shape, D):
    """A filled cache: codes of K and V and the records, planes one after another."""
    k4 = torch.empty(shape + (D // 2,), dtype=torch.uint8, device="cuda")
    v4, prm = torch.empty_like(k4), torch.empty(shape + (8,), dtype=torch.bfloat16, device="cuda")
    channel = torch.exp(0.4 * torch.randn(2, D, generator=g, device="cuda"))
    k, v, p = k4.view(-1, D // 2), v4.view(-1, D // 2), prm.view(-1, 8)
    for at in range(0, k.shape[0], 1 << 20):
        some = slice(at, at + (1 << 20))
        n = k[some].shape[0]
        kc, kp = quantise_rows(rows_like(g, (n, D), channel[0]) + 0.25 * channel[0].to(torch.bfloat16))
        vc, vp = quantise_rows(rows_like(g, (n, D), channel[1]))
        k[some], v[some], p[some] = pack(kc), pack(vc), torch.cat([kp, vp], -1)
    return k4, v4, prm


def shape_of(planes, Hkv, rows, layout):
    return (planes, Hkv, rows) if layout == HND else (planes, rows, Hkv)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def pool(g, lens, most, bs, spare):
    """Block table of requests that hold `lens` tokens, and the stack of free pages."""
    held = [pages_of(n, bs) for n in lens]
    pages = sum(held) + spare
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), most), -1, dtype=torch.int32)
    at, host = 0, perm.cpu()
    for b, n in enumerate(held):
        table[b, :n] = host[at:at + n]
        at += n
    free = torch.zeros(pages, dtype=torch.int32, device="cuda")
    free[:spare] = perm[at:]
    return table.cuda(), free, i32([spare]), pages


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind, B, bs, lens = case["kind"], case["B"], case["block_size"], lengths(case)
    s = dict(case, seqlens=i32(lens))
    if kind in ("slots", "turn"):
        new, done = news(case), finished(case)
        ends = [(0 if d else n) + a for n, a, d in zip(lens, new, done)]
        most = max(1, max(pages_of(max(n, e), bs) for n, e in zip(lens, ends)))
        spare = sum(pages_of(a, bs) + 1 for a in new)
        table, free, count, pages = pool(g, lens, most, bs, spare)
        T = sum(new) + 7
        s.update(new_lens=i32(new), done=torch.tensor(done, dtype=torch.uint8, device="cuda"),
                 table=table, free=free, count=count, pages=pages, most=most, T=T)
        s.update(bookkeeping(B, T))
        return s
    Hq, Hkv, D, layout = case["Hq"], case["Hkv"], case["D"], case["layout"]
    if kind == "fill":
        # K and V are slices of a fused projection's output; two padded rows belong to no request
        total = sum(lens)
        T = total + 2
        most = max(1, pages_of(max(lens), bs))
        table, free, count, pages = pool(g, lens, most, bs, 3)
        qkv = rows_like(g, (T, (Hq + 2 * Hkv) * D), torch.exp(0.4 * torch.randn((Hq + 2 * Hkv) * D, generator=g, device="cuda")))
        k, v = qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:]
        t = torch.cat([torch.arange(n) for n in lens]).cuda()
        b = torch.repeat_interleave(torch.arange(B), torch.tensor(lens)).cuda()
        slot = table[b, t // bs].long() * bs + t % bs
        s.update(k=k.unflatten(-1, (Hkv, D)), v=v.unflatten(-1, (Hkv, D)), qkv=qkv, table=table, pages=pages,
                 slots=torch.cat([slot, torch.full((T - total,), -1, device="cuda")]), T=T)
        shape, rows = shape_of(pages, Hkv, bs, layout), most * bs
        s.update(k4=torch.zeros(shape + (D // 2,), dtype=torch.uint8, device="cuda"),
                 v4=torch.zeros(shape + (D // 2,), dtype=torch.uint8, device="cuda"),
                 params=torch.zeros(shape + (8,), dtype=torch.bfloat16, device="cuda"), max_len=rows, most=most)
        s.update(k_out=torch.zeros(shape_of(B, Hkv, rows, layout) + (D,), dtype=torch.bfloat16, device="cuda"))
        s.update(v_out=torch.zeros_like(s["k_out"]))
        return s
    s["q"] = torch.randn((B, Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    s.update(scale=1.0 / math.sqrt(D), table=None, pages=0, most=0)
    s.update(out=torch.empty_like(s["q"]), lse=torch.empty((B, Hq), device="cuda"))
    if kind == "step":
        most = pages_of(max(lens) + 1, bs)
        s["table"], free, count, s["pages"] = pool(g, lens, most, bs, B + 5)
        k_new, v_new = (rows_like(g, (B, Hkv, D), 1.0) for _ in range(2))
        s.update(new_lens=i32([1] * B), free=free, count=count, most=most, T=B, k=k_new, v=v_new)
        s.update(bookkeeping(B, B))
    elif bs:
        s["most"] = pages_of(max(lens), bs)
        s["table"], _, _, s["pages"] = pool(g, lens, s["most"], bs, 3)
    s["max_len"] = s["most"] * bs if bs else max(lens)
    shape = shape_of(s["pages"], Hkv, bs, layout) if bs else shape_of(B, Hkv, s["max_len"], layout)
    s["k4"], s["v4"], s["params"] = cache_of(g, shape, D)
    return s


def bookkeeping(B, T):
    return dict(seqlens_out=i32([0] * B), kept=i32([0] * B), cu_new=i32([0] * (B + 1)), count_out=i32([0]),
                count_kept=i32([0]), slots=torch.zeros(T, dtype=torch.int64, device="cuda"), positions=i32([0] * T))


# --------------------------------------------------------------- plain forms

def plain_codes(x):
    return torch.stack([x & 15, x >> 4], -1).flatten(-2)


def plain_values(x4, params, first):
    """fp32 values of rows: codes [..., D / 2] with their records [..., 8]."""
    c = (plain_codes(x4).float() - 8).unflatten(-1, (2, x4.shape[-1]))
    p = params[..., first:first + 4].float().unflatten(-1, (2, 2))
    return (p[..., 0:1] * c + p[..., 1:2]).flatten(-2)


def by_token(x, s):
    """A cache [planes, ...] as [B, Hkv, max_len, ...]; pages are gathered."""
    if s["layout"] == NHD:
        x = x.transpose(1, 2)
    if s["table"] is None:
        return x
    x = x[s["table"].long().clamp(0, x.shape[0] - 1)]
    return x.transpose(1, 2).flatten(2, 3)


def plain_attend(s, seqlens):
    B, Hkv, D = s["B"], s["Hkv"], s["D"]
    params = by_token(s["params"], s)
    k = plain_values(by_token(s["k4"], s), params, 0)
    v = plain_values(by_token(s["v4"], s), params, 4)
    q = s["q"].float().unflatten(1, (Hkv, s["Hq"] // Hkv))
    x = (q @ k.transpose(-1, -2)) * s["scale"]
    away = torch.arange(x.shape[-1], device="cuda") >= seqlens[:, None, None, None]
    x = x.masked_fill(away, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.clamp(min=-3e38))
    z = p.sum(-1, keepdim=True)
    o = (p @ v.masked_fill(away.transpose(-1, -2), 0)) / z.clamp(min=1e-30)
    lse = m + torch.log(z)
    return o.reshape(B, s["Hq"], D).to(torch.bfloat16), lse.reshape(B, s["Hq"])


def plain_append(s, slots):
    """New rows into the caches, in place; a negative slot writes nothing."""
    use = slots >= 0
    rows = s["block_size"]
    plane, row = slots[use] // rows, slots[use] % rows
    (kc, kp), (vc, vp) = quantise_rows(s["k"][use]), quantise_rows(s["v"][use])
    at = (plane, slice(None), row) if s["layout"] == HND else (plane, row)
    s["k4"][at], s["v4"][at], s["params"][at] = pack(kc), pack(vc), torch.cat([kp, vp], -1)


def plain_alloc(s, seqlens, count):
    bs, most, T = s["block_size"], s["most"], s["T"]
    F = count.long().clamp(0, s["pages"])
    n = seqlens.long().clamp(0, most * bs)
    cu = torch.cat([torch.zeros_like(n[:1]), s["new_lens"].long().clamp(min=0).cumsum(0)]).clamp(max=T)
    e = (n + cu[1:] - cu[:-1]).clamp(max=most * bs)
    p0 = (n + bs - 1) // bs
    need = (e + bs - 1) // bs - p0
    o = need.cumsum(0) - need
    granted = torch.minimum(torch.clamp(F - o, min=0), need)
    end = torch.minimum(e, (p0 + granted) * bs)
    j = torch.arange(most, device="cuda")[None]
    fresh = (j >= p0[:, None]) & (j < (p0 + granted)[:, None])
    page = s["free"][(F - 1 - (o[:, None] + j - p0[:, None])).clamp(0, s["pages"] - 1)]
    s["table"].copy_(torch.where(fresh, page, s["table"]))
    i = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu, i, right=True).clamp(1, s["B"]) - 1
    t = n[b] + i - cu[b]
    inside = i < cu[-1]
    at = s["table"][b, (t // bs).clamp(0, most - 1)].long()
    slot = torch.where(inside & (t < end[b]) & (at >= 0), at * bs + t % bs, -1)
    return {"slots": slot, "positions": torch.where(inside, t, 0).int(), "cu_new": cu.int(), "seqlens": end.int(),
            "free_count": (F - torch.minimum(F, need.sum())).int(), "table": s["table"]}


def plain_release(s):
    bs, most, pages = s["block_size"], s["most"], s["pages"]
    F = s["count"].long().clamp(0, pages)
    n, done = s["seqlens"].long().clamp(0, most * bs), s["done"].bool()
    r = torch.where(done, (n + bs - 1) // bs, 0)
    o = r.cumsum(0) - r
    j = torch.arange(most, device="cuda")[None]
    to = F + o[:, None] + j
    use = (j < r[:, None]) & (to < pages)
    s["free"][to[use]] = s["table"][use]
    return torch.where(done, 0, n).int(), (F + r.sum()).clamp(max=pages).int()


def plain(s):
    kind = s["kind"]
    if kind == "attend":
        return plain_attend(s, s["seqlens"])
    if kind == "step":
        a = plain_alloc(s, s["seqlens"], s["count"])
        plain_append(s, a["slots"])
        return plain_attend(s, a["seqlens"]) + (dict(a, params=s["params"]),)
    if kind == "fill":
        plain_append(s, s["slots"])
        params = by_token(s["params"], s)
        for out, x, first in ((s["k_out"], s["k4"], 0), (s["v_out"], s["v4"], 4)):
            value = plain_values(by_token(x, s), params, first).to(torch.bfloat16)
            out = out if s["layout"] == HND else out.transpose(1, 2)
            there = torch.arange(s["max_len"], device="cuda") < s["seqlens"][:, None, None]
            out.copy_(torch.where(there[..., None], value, out))
        return s["k_out"], s["v_out"]
    if kind == "slots":
        return plain_alloc(s, s["seqlens"], s["count"])
    kept, count = plain_release(s)
    return dict(plain_alloc(s, kept, count), free_pages=s["free"])


# ------------------------------------------------------- the framework's calls

def problem(fd, s):
    if "prob" not in s:
        s["prob"] = fd.make_problem(s["B"], s["Hq"], s["Hkv"], s["D"], s["max_len"], s["block_size"], s["pages"],
                                    s["most"], s["layout"], fd.FD_KV_INT4)
    return s["prob"]


def checked(fd, status):
    if status != fd.FD_OK:
        raise fd.FdError(status)


def own_attend(fd, s, seqlens):
    """The problem, the split count and the workspace are kept, as a decode loop keeps them."""
    p = problem(fd, s)
    if "splits" not in s:
        after = [n + (s["kind"] == "step") for n in lengths(s)]
        s["splits"] = fd.fd_plan_problem(0, p, after)
        s["bytes"] = fd.fd_workspace_bytes(s["B"], s["Hq"], s["D"], s["splits"])
        s["work"] = torch.empty(max(4, s["bytes"]), dtype=torch.uint8, device="cuda")
    checked(fd, fd.fd_decode_int4(p, s["q"], s["k4"], s["v4"], s["params"], seqlens, s["table"], s["scale"],
                                  s["splits"], s["out"], s["lse"], s["work"], s["bytes"]))
    return s["out"], s["lse"]


def own_append(fd, s, slots):
    k, v = s["k"], s["v"]
    checked(fd, fd.fd_append_int4(problem(fd, s), s["T"], k, k.stride(0), v, v.stride(0), slots, s["k4"], s["v4"],
                                  s["params"]))


def own_alloc(fd, s, seqlens, count):
    checked(fd, fd.fd_alloc_pages(s["B"], s["block_size"], s["most"], s["T"], s["pages"], seqlens, s["new_lens"],
                                  s["free"], count, s["table"], s["seqlens_out"], s["cu_new"], s["slots"],
                                  s["positions"], s["count_out"]))
    return {"slots": s["slots"], "positions": s["positions"], "cu_new": s["cu_new"], "seqlens": s["seqlens_out"],
            "free_count": s["count_out"], "table": s["table"]}


def framework(s):
    import split_kv_decode_attn_b200 as fd
    kind = s["kind"]
    if kind == "attend":
        return own_attend(fd, s, s["seqlens"])
    if kind == "step":
        a = own_alloc(fd, s, s["seqlens"], s["count"])
        own_append(fd, s, a["slots"])
        return own_attend(fd, s, a["seqlens"]) + (dict(a, params=s["params"]),)
    if kind == "fill":
        own_append(fd, s, s["slots"])
        checked(fd, fd.fd_expand_int4(problem(fd, s), s["k4"], s["v4"], s["params"], s["seqlens"], s["table"],
                                      s["k_out"], s["v_out"]))
        return s["k_out"], s["v_out"]
    if kind == "slots":
        return own_alloc(fd, s, s["seqlens"], s["count"])
    checked(fd, fd.fd_release_pages(s["B"], s["block_size"], s["most"], s["pages"], s["seqlens"], s["done"],
                                    s["table"], s["free"], s["count"], s["kept"], s["count_kept"]))
    return dict(own_alloc(fd, s, s["kept"], s["count_kept"]), free_pages=s["free"])


def run(state):
    return framework(state) if own else plain(state)


# ------------------------------------------------------------------ the floor

def work(case):
    kind, B, lens, bs = case["kind"], case["B"], lengths(case), case["block_size"]
    if kind in ("slots", "turn"):
        new, done = news(case), finished(case)
        kept = [0 if d else n for n, d in zip(lens, done)]
        taken = sum(pages_of(n + a, bs) - pages_of(n, bs) for n, a in zip(kept, new))
        back = sum(pages_of(n, bs) for n, d in zip(lens, done) if d)
        # lengths, new lengths, flags; slots and positions; a page id read and written each way
        return {"bytes": 4 * B * (5 if kind == "turn" else 4) + 12 * sum(new) + 8 * (taken + back), "flops": 0}
    Hq, Hkv, D, total = case["Hq"], case["Hkv"], case["D"], sum(lens)
    if kind == "fill":
        return {"bytes": total * Hkv * (4 * D + 2 * (D + 16) + 4 * D) + 8 * total, "flops": 0}
    fresh = B if kind == "step" else 0
    read = (total + fresh) * Hkv * (D + 16) + B * Hq * (4 * D + 4) + sum(4 * pages_of(n, bs) for n in lens if bs)
    return {"bytes": read + fresh * Hkv * (4 * D + D + 16), "flops": 4 * Hq * D * (total + fresh)}


# ------------------------------------------- the definition, in 64 bits

def exact_rows(x4, params, first):
    """Rows [n, D / 2] of codes and their records [n, 8] as 64-bit values, entry by entry."""
    n, half = x4.shape[0], x4.shape[1] // 2
    value = torch.empty((n, 2 * x4.shape[1]), dtype=torch.float64, device=x4.device)
    value[:, 0::2] = (x4 % 16).double()
    value[:, 1::2] = torch.div(x4, 16, rounding_mode="floor").double()
    for group in range(2):
        part = value[:, group * 2 * half:(group + 1) * 2 * half]
        part.sub_(8).mul_(params[:, first + 2 * group, None].double()).add_(params[:, first + 2 * group + 1, None].double())
    return value


def exact_quantised(x):
    """The values that rows [n, D] stand for once they are held in 4 bits, from the definition."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    half = x.shape[1] // 2
    for lo in (0, half):
        part = x[:, lo:lo + half].double()
        low, high = part.min(1, keepdim=True).values, part.max(1, keepdim=True).values
        scale = ((high - low) / 15).bfloat16().double()
        bias = (low + 8 * scale).bfloat16().double()
        code = ((part - bias) / torch.where(scale == 0, 1.0, scale)).round().clamp(-8, 7)
        out[:, lo:lo + half] = scale * torch.where(scale == 0, 0.0, code) + bias
    return out


def exact(case, seed):
    kind, bs, lens = case["kind"], case["block_size"], lengths(case)
    if kind in ("slots", "turn"):
        return None
    s = prepare(case, seed)
    Hkv, D, G = case["Hkv"], case["D"], case["Hq"] // case["Hkv"]
    if kind == "fill":
        outs = []
        for x in (s["k"], s["v"]):
            out, at = torch.zeros(shape_of(case["B"], Hkv, s["max_len"], case["layout"]) + (D,), dtype=torch.float64, device="cuda"), 0
            for b, n in enumerate(lens):
                rows = exact_quantised(x[at:at + n].reshape(n * Hkv, D)).view(n, Hkv, D) if n else None
                if n and case["layout"] == HND:
                    out[b, :, :n] = rows.transpose(0, 1)
                elif n:
                    out[b, :n] = rows
                at += n
            outs.append(out)
        return tuple(outs)
    out = torch.zeros((case["B"], case["Hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"], case["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        for h in range(Hkv):
            where = torch.arange(n, device="cuda")
            if bs:
                page = s["table"][b].long()[where // bs]
                at = (page, h, where % bs) if case["layout"] == HND else (page, where % bs, h)
            else:
                at = (b, h, where) if case["layout"] == HND else (b, where, h)
            prm = s["params"][at]
            k, v = exact_rows(s["k4"][at], prm, 0), exact_rows(s["v4"][at], prm, 4)
            if kind == "step":
                k = torch.cat([k, exact_quantised(s["k"][b, h][None])])
                v = torch.cat([v, exact_quantised(s["v"][b, h][None])])
            if k.shape[0] == 0:
                continue
            heads = slice(h * G, (h + 1) * G)
            x = torch.mv(k, s["q"][b, h * G].double())[None] if G == 1 else s["q"][b, heads].double() @ k.T
            x = x * s["scale"]
            lse[b, heads] = torch.logsumexp(x, 1)
            out[b, heads] = torch.softmax(x, 1) @ v
    return (out, lse) if kind == "attend" else (out, lse, None)

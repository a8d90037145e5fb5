"""Measured cases of the paged key/value cache held in 4 bits: writing it, reading it back, attention over it.

* append: new keys and values quantised as they are written into pages, then the values the pages now stand for.
* read:   keys and values of requests (or of a shared prompt) read back to bf16 rows, for the calls that take such rows.
* paged:  attention of new tokens over the 4-bit pages, whose first ``prefix`` tokens every request shares.

The format: 32 neighbouring channels of a token and head share a scale of 8 bits, (1 + f / 8) 2^(e - 15) with f the lowest
three bits and e the upper five (255: the 32 values were not all finite), and each is a code of 4 bits, code + 8 = 1 .. 15.
A page holds for each head blocks of 16 tokens, of K the codes [group][token][16 bytes], of V [channel][8 bytes], and behind
them scales [group][token].  Eight neighbouring codes lie in a 32-bit word: the even ones in its lower half, the odd ones
in its upper.

Heads, head dims and lengths are those of the workloads in ``bsa_inputs/synthetic.py`` (24/8 and 32/8 heads of 128,
24 heads of 128, heads of 64) and generic serving sizes around them.
"""

import math
import random

import torch

own = False

BF, F32, F64, I32, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8
GROUP, BLOCK = 32, 16


def _append(name, B, T, Hkv, d, page, slots, **kw):
    return {"op": "append", "name": name, "B": B, "T": T, "Hkv": Hkv, "d": d, "page": page, "slots": slots, "ragged": False,
            "spread": 1, **kw}


def _read(name, B, low, high, Hkv, d, page, **kw):
    return {"op": "read", "name": name, "B": B, "low": low, "high": high, "Hkv": Hkv, "d": d, "page": page, "behind": 0,
            "spread": 1, **kw}


def _paged(name, B, T, P, low, high, Hq, Hkv, d, page, **kw):
    return {"op": "paged", "name": name, "B": B, "T": T, "P": P, "low": low, "high": high, "Hq": Hq, "Hkv": Hkv, "d": d,
            "page": page, "ragged": False, "causal": True, "spread": 1, **kw}


def listed():
    return [
        # one token each of 64 running requests
        _append("append_step", 64, 1, 8, 128, 64, 2048),
        # prompts of unequal lengths on their way into small pages
        _append("append_prompts", 5, 4099, 8, 128, 16, 8192, ragged=True),
        # a shared prompt, as the selector and the dense pass take it
        _read("read_prompt", 1, 8209, 8209, 8, 128, 64),
        # requests of unequal lengths with heads of 64, without what each has held since before
        _read("read_ragged_d64", 16, 1, 16384, 2, 64, 16, behind=100),
        # one request, one token: latency alone
        _paged("decode_one", 1, 1, 0, 4097, 4097, 32, 8, 128, 64),
        # 64 requests on one long system prompt, each with its own answer so far
        _paged("decode_shared", 64, 1, 8209, 1, 1024, 32, 8, 128, 64),
        # 16 requests with long contexts of their own, nothing shared
        _paged("decode_long", 16, 1, 0, 1024, 65536, 32, 8, 128, 128),
        # as many key heads as query heads: one row for each pass over a head's keys
        _paged("decode_all_heads", 20, 1, 0, 500, 9000, 24, 24, 128, 32),
        # five drafted tokens a request, heads of 64, small pages, prefix that ends inside a page
        _paged("verify_drafts_d64", 24, 5, 1000, 5, 2500, 4, 2, 64, 16),
        # 256 samples of one 32k prompt: the shared keys meet many rows
        _paged("samples_of_one_prompt", 256, 1, 32768, 1, 512, 32, 8, 128, 64),
        # the next 500 tokens of two prompts over a shared prefix and what each already holds
        _paged("chunk_of_prompt", 2, 500, 4096, 500, 4100, 24, 8, 128, 128),
    ]


HEADS = ((32, 8, 128), (24, 8, 128), (24, 24, 128), (4, 2, 64), (3, 1, 64), (16, 2, 128), (8, 8, 64), (20, 4, 128))


def _log(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    while True:
        op = rng.choice(("append", "read", "paged", "paged"))
        Hq, Hkv, d = rng.choice(HEADS)
        page = rng.choice((16, 32, 64, 128, 256))
        if op == "append":
            T = rng.choice((1, 1, _log(rng, 1, 4096)))
            case = _append("", _log(rng, 1, 128), T, Hkv, d, page, T + _log(rng, 1, 4096), ragged=T > 1 and rng.random() < 0.6,
                           spread=rng.randint(1, 999))
        elif op == "read":
            low = _log(rng, 1, 4000)
            case = _read("", _log(rng, 1, 32), low, low + _log(rng, 1, 20000), Hkv, d, page, behind=rng.choice((0, 0, _log(rng, 1, 500))),
                         spread=rng.randint(1, 999))
        else:
            T = rng.choice((1, 1, 1, _log(rng, 1, 16), _log(rng, 1, 500)))
            low = T + _log(rng, 1, 2000) - 1
            case = _paged("", _log(rng, 1, 256), T, rng.choice((0, _log(rng, 1, 33000))), low, low + _log(rng, 1, 30000), Hq, Hkv, d,
                          page, ragged=T > 1 and rng.random() < 0.5, causal=rng.random() < 0.8, spread=rng.randint(1, 999))
        w = work(case)
        values = 2 * case["B"] * case.get("high", case.get("slots", 0)) * Hkv * d
        scores = 4 * case["B"] * Hq * case["T"] * (case["P"] + case["high"]) if op == "paged" else 0
        if w["bytes"] <= (5.8e8 if op == "paged" else 1.6e8) and w["flops"] <= 1.4e11 and values <= 2.4e9 and scores <= 3e9:
            return case


# ---- lengths and pages ----

def _lens(case):
    """(keys of its own, new tokens, keys left out in front) of every request: fixed by the case alone."""
    r = random.Random(case["spread"] * 7919 + case["B"])
    B = case["B"]
    if case["op"] == "append":
        T = case["T"]
        new = [r.randint(0, T) if case["ragged"] else T for _ in range(B)]
        return [n + r.randint(0, case["slots"] - T) for n in new], new, [0] * B
    keys = [r.randint(case["low"], case["high"]) for _ in range(B)]
    if case["op"] == "read":
        return keys, [0] * B, [min(n, r.randint(0, case["behind"])) for n in keys]
    return keys, [r.randint(0, case["T"]) if case["ragged"] else case["T"] for _ in range(B)], [0] * B


def _pages(slots, page, shared, g):
    """Tables of pages in no order: [B, n] of the requests' own (-1 where a table has no page) and [m] of the shared prefix."""
    need = torch.tensor([-(-s // page) for s in slots])
    m = -(-shared // page)
    total = int(need.sum()) + m + 3
    order = torch.randperm(total, generator=g, device="cuda").to(I32)
    column = torch.arange(max(1, int(need.max())))
    number = torch.cumsum(need, 0)[:, None] - need[:, None] + column
    mine = torch.where(column < need[:, None], number, -1).cuda()
    table = torch.where(mine >= 0, order[mine.clamp(min=0) + m], -1).to(I32)
    return total, table, order[:m].clone()


# ---- the format ----

def _codes(x):
    """(code + 8, scale byte) of x [..., d]: [..., d] and [..., d / 32], uint8."""
    x = x.to(F32).unflatten(-1, (-1, GROUP))
    most = x.abs().amax(-1)
    fine = torch.isfinite(most)
    most = most.masked_fill(~fine, 1.0).to(F64)
    m, e = torch.frexp(most / torch.full_like(most, 7.0))             # by a number it would be a product, off at ties
    m = torch.round(m * 16.0)                                         # four bits of the quotient, ties to even
    byte = ((e + 14) * 8 + m.to(I32) - 8).clamp(0, 254).masked_fill(most == 0, 0)
    scale = torch.ldexp(1.0 + (byte % 8) / 8.0, byte // 8 - 15).to(F32)
    n = torch.floor(x.abs() / scale[..., None] + 0.5).clamp(max=7.0).copysign(x).masked_fill(~fine[..., None], 0.0)
    return (n + 8.0).to(U8).flatten(-2), byte.masked_fill(~fine, 255).to(U8)


def _pack(u):
    """[..., n] codes + 8 to [..., n / 2] bytes."""
    u = u.unflatten(-1, (-1, 4, 2)).transpose(-1, -2).flatten(-3)     # of eight the even ones first
    return u[..., 0::2] | u[..., 1::2] << 4


def _unpack(b):
    u = torch.stack([b & 15, b >> 4], -1).flatten(-2).unflatten(-1, (-1, 2, 4))
    return u.transpose(-1, -2).flatten(-3)


def _scales(byte):
    byte = byte.to(I32)
    return torch.ldexp(1.0 + (byte % 8).to(F32) / 8.0, byte // 8 - 15).masked_fill(byte == 255, math.nan)


def _rows(blocks, d, channels_first):
    """Values [..., n * 16, H, d] fp32 that blocks [..., H, n, bytes] stand for."""
    G = d // GROUP
    codes, byte = blocks.split([BLOCK * d // 2, BLOCK * G], -1)
    s = _scales(byte.unflatten(-1, (G, BLOCK))).transpose(-1, -2)                                # [..., token, group]
    if channels_first:
        c = _unpack(codes.unflatten(-1, (d, BLOCK // 2))).transpose(-1, -2).unflatten(-1, (G, GROUP))
    else:
        c = _unpack(codes.unflatten(-1, (G, BLOCK, GROUP // 2))).transpose(-2, -3)
    x = ((c.to(F32) - 8.0) * s[..., None]).flatten(-2)                                           # [..., H, n, 16, d]
    return x.flatten(-3, -2).transpose(-3, -2)


def _filled(total, page, Hkv, d, channels_first, g):
    """A pool of pages with normally distributed values, an eighth of the channels three times as large."""
    out = torch.empty(total, Hkv, page // BLOCK, 17 * d // 2, dtype=U8, device="cuda")
    wide = torch.where(torch.rand(Hkv, 1, 1, d, generator=g, device="cuda") < 0.125, 3.0, 1.0) if not channels_first else 1.0
    step = max(1, (1 << 26) // (page * Hkv * d))
    for at in range(0, total, step):
        n = min(step, total - at)
        u, s = _codes(torch.randn(n, Hkv, page // BLOCK, BLOCK, d, generator=g, device="cuda") * wide)
        u = u.transpose(-1, -2) if channels_first else u.unflatten(-1, (-1, GROUP)).transpose(-2, -3)
        out[at:at + n] = torch.cat([_pack(u).flatten(3), s.transpose(-1, -2).flatten(3)], -1)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 29)
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    lens, new, first = _lens(case)
    st = {"case": case, "kv_lens": torch.tensor(lens, dtype=I32, device="cuda")}
    slots = [case["slots"]] * B if case["op"] == "append" else lens
    total, st["table"], st["prefix_table"] = _pages(slots, page, case.get("P", 0), g)
    st["k_cache"], st["v_cache"] = (_filled(total, page, Hkv, d, x, g) for x in (False, True))
    if case["op"] == "read":
        st["first"] = torch.tensor(first, dtype=I32, device="cuda") if case["behind"] else None
        rows = max(1, max(n - f for n, f in zip(lens, first)))
        st["k"], st["v"] = (torch.zeros(B, rows, Hkv, d, dtype=BF, device="cuda") for _ in range(2))
        return st
    T = case["T"]
    st["new_lens"] = torch.tensor(new, dtype=I32, device="cuda") if case["ragged"] else None
    if case["op"] == "append":
        kv = torch.randn(B, T, 2 * Hkv, d, generator=g, device="cuda").to(BF)                    # of one projection
        st["k"], st["v"] = kv[:, :, :Hkv], kv[:, :, Hkv:]
        st["k"] *= torch.where(torch.rand(Hkv, d, generator=g, device="cuda") < 0.125, 3.0, 1.0).to(BF)
        st["first"] = torch.tensor([n - t for n, t in zip(lens, new)], dtype=I32, device="cuda")
        st["k_out"], st["v_out"] = (torch.zeros(B, T, Hkv, d, dtype=BF, device="cuda") for _ in range(2))
    else:
        st["q"] = torch.randn(B, T, case["Hq"], d, generator=g, device="cuda").to(BF)
    return st


# ---- the plain forms ----

def _place(token):
    """The byte of a token among the eight of a channel, and whether it is the lower half of it."""
    return (token % 8 // 2 + token % 2 * 4) // 2 + token // 8 * 4, token % 8 // 2 % 2 == 0


def _write_k(cache, x, d, at, token):
    u, s = _codes(x)                                                                             # [n, H, d], [n, H, G]
    G, half = d // GROUP, BLOCK * d // 2
    cache[..., half:].unflatten(-1, (G, BLOCK))[at[0], :, at[1], :, token] = s
    cache[..., :half].unflatten(-1, (G, BLOCK, -1))[at[0], :, at[1], :, token] = _pack(u).unflatten(-1, (G, -1))


def _write_v(cache, x, d, at, token):
    u, s = _codes(x)
    G, half = d // GROUP, BLOCK * d // 2
    cache[..., half:].unflatten(-1, (G, BLOCK))[at[0], :, at[1], :, token] = s
    byte, low = _place(token)
    held = cache[..., :half].unflatten(-1, (d, BLOCK // 2))
    a = (at[0][low], slice(None), at[1][low], slice(None), byte[low])
    held[a] = held[a] & 0xF0 | u[low]
    b = (at[0][~low], slice(None), at[1][~low], slice(None), byte[~low])
    held[b] = held[b] & 0x0F | u[~low] << 4


def _held(cache, d, at, token, channels_first):
    """Values [n, H, d] of tokens."""
    G, half = d // GROUP, BLOCK * d // 2
    s = _scales(cache[..., half:].unflatten(-1, (G, BLOCK))[at[0], :, at[1], :, token])          # [n, H, G]
    if channels_first:
        byte, low = _place(token)
        u = cache[..., :half].unflatten(-1, (d, BLOCK // 2))[at[0], :, at[1], :, byte]
        u = torch.where(low[:, None, None], u & 15, u >> 4).unflatten(-1, (G, GROUP))
    else:
        u = _unpack(cache[..., :half].unflatten(-1, (G, BLOCK, -1))[at[0], :, at[1], :, token])
    return ((u.to(F32) - 8.0) * s[..., None]).flatten(-2).to(BF)


def _plain_append(st):
    case = st["case"]
    T, d, page, kv = case["T"], case["d"], case["page"], st["kv_lens"].long()
    new = torch.full_like(kv, T) if st["new_lens"] is None else st["new_lens"].long()
    t = torch.arange(T, device=kv.device)
    real = t < new[:, None]
    key = ((kv - new)[:, None] + t)[real]
    request = torch.arange(case["B"], device=kv.device)[:, None].expand(-1, T)[real]
    at = st["table"].long()[request, key // page], key % page // BLOCK
    _write_k(st["k_cache"], st["k"][real], d, at, key % BLOCK)
    _write_v(st["v_cache"], st["v"][real], d, at, key % BLOCK)


def _plain_read(st, first, k, v):
    """Row t of request b from key first[b] + t on, where there is one."""
    d, page, kv = st["case"]["d"], st["case"]["page"], st["kv_lens"].long()
    key = torch.arange(k.shape[1], device=k.device).expand(k.shape[0], -1)
    if first is not None:
        key = key + first.long()[:, None]
    real = key < kv[:, None]
    request = torch.arange(k.shape[0], device=k.device)[:, None].expand_as(key)[real]
    key = key[real]
    at = st["table"].long()[request, key // page], key % page // BLOCK
    k[real] = _held(st["k_cache"], d, at, key % BLOCK, False)
    v[real] = _held(st["v_cache"], d, at, key % BLOCK, True)


def _plain_paged(st):
    case = st["case"]
    B, T, P, Hq, Hkv, d = (case[n] for n in ("B", "T", "P", "Hq", "Hkv", "d"))
    kv, new = st["kv_lens"].long(), st["new_lens"]
    new = torch.full_like(kv, T) if new is None else new.long()
    q = st["q"].to(F32).view(B, T, Hkv, Hq // Hkv, d) * d ** -0.5

    def dense(table):
        """Rows of K and V [..., keys, Hkv, d] of the pages of a table [..., pages]."""
        return [_rows(c[table].transpose(-3, -4).flatten(-3, -2), d, x) for c, x in ((st["k_cache"], False), (st["v_cache"], True))]

    own_k, own_v = dense(st["table"].long().clamp(min=0))
    n, dev = own_k.shape[1], kv.device
    key, row = torch.arange(n, device=dev), torch.arange(T, device=dev)
    last = kv[:, None] - new[:, None] + row if case["causal"] else (kv[:, None] - 1).expand(B, T)
    real = row < new[:, None]
    seen = (key <= last[:, :, None]) & (key < kv[:, None, None])                       # [B, T, n]
    s = torch.einsum("bthgd,bnhd->bthgn", q, own_k).masked_fill(~seen[:, :, None, None], -math.inf)
    own_v = own_v.masked_fill((key >= kv[:, None])[:, :, None, None], 0.0)
    if P:
        pk, pv = (x[:P] for x in dense(st["prefix_table"].long()))
        s = torch.cat([torch.einsum("bthgd,nhd->bthgn", q, pk), s], -1)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m.masked_fill(m == -math.inf, 0.0))
    total = p.sum(-1)
    out = torch.einsum("bthgn,bnhd->bthgd", p[..., P:], own_v)
    if P:
        out = out + torch.einsum("bthgn,nhd->bthgd", p[..., :P], pv)
    filled = (total > 0) & real[:, :, None, None]
    out = (out / total[..., None]).masked_fill(~filled[..., None], 0.0)
    lse = (m[..., 0] + torch.log(total)).masked_fill(~filled, -math.inf)
    return {"out": out.reshape(B, T, Hq, d).to(BF), "lse": lse.reshape(B, T, Hq).transpose(1, 2).contiguous()}


def run(st):
    case = st["case"]
    if own:
        import block_sparse_attention_bsa_gb300 as bsa
        pages = (st["k_cache"], st["v_cache"], st["table"], st["kv_lens"])
        if case["op"] == "paged":
            out, lse = bsa.bsa_forward_paged_q4(st["q"], *pages, new_lens=st["new_lens"], prefix_table=st["prefix_table"],
                                                prefix_len=case["P"], causal=case["causal"])
            return {"out": out, "lse": lse}
        if case["op"] == "append":
            bsa.bsa_cache_append_q4(st["k"], st["v"], *pages, new_lens=st["new_lens"])
            k, v = bsa.bsa_cache_read_q4(*pages, case["T"], first=st["first"], k_out=st["k_out"], v_out=st["v_out"])
        else:
            k, v = bsa.bsa_cache_read_q4(*pages, st["k"].shape[1], first=st["first"], k_out=st["k"], v_out=st["v"])
        return {"k": k, "v": v}
    if case["op"] == "paged":
        return _plain_paged(st)
    if case["op"] == "append":
        _plain_append(st)
        _plain_read(st, st["first"], st["k_out"], st["v_out"])
        return {"k": st["k_out"], "v": st["v_out"]}
    _plain_read(st, st["first"], st["k"], st["v"])
    return {"k": st["k"], "v": st["v"]}


def work(case):
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    lens, new, first = _lens(case)
    row = 17 * d // 32                                     # bytes of a token and head: codes and scales
    if case["op"] == "append":
        # K and V are read, their codes and scales written and read, their values written; lengths and a table entry a token
        n = sum(new) * Hkv
        return {"bytes": 2 * n * (4 * d + 2 * row) + 4 * sum(new) + 12 * B, "flops": 2 * n * d * 6}
    if case["op"] == "read":
        n = sum(a - f for a, f in zip(lens, first)) * Hkv
        return {"bytes": 2 * n * (2 * d + row) + 4 * (n // Hkv // case["page"]) + 8 * B, "flops": 2 * n * d}
    T, P, Hq = case["T"], case["P"], case["Hq"]
    seen = sum(new) * P                                    # the prefix once for all, each request's own keys once
    for n, t in zip(lens, new):
        # row i of t sees n - t + i + 1 of its own keys
        seen += sum(max(0, n - t + i + 1) for i in range(t)) if case["causal"] else n * t
    kv = P + sum(n for n, t in zip(lens, new) if t)
    return {"bytes": 2 * kv * Hkv * row + 4 * B * T * Hq * d + 4 * B * Hq * T + 4 * (kv // case["page"]),
            "flops": 4 * seen * Hq * d}


# ---- the definitions in 64 bits ----

def _scale_table():
    return torch.tensor([(1 + b % 8 / 8) * 2.0 ** (b // 8 - 15) for b in range(255)] + [math.nan], dtype=F64, device="cuda")


def _held64(x):
    """What the pages hold of x [n, H, d]: the nearest scale to a seventh of the largest of 32 values, the even one of two;
    then the nearest multiple, the larger one of two."""
    x = x.to(F64).reshape(*x.shape[:-1], -1, GROUP)
    table = _scale_table()[:255]
    want = x.abs().max(-1).values
    want = want / torch.full_like(want, 7)
    upper = torch.searchsorted(table, want.contiguous()).clamp(max=254)
    lower = (upper - 1).clamp(min=0)
    above, below = (table[upper] - want).abs(), (want - table[lower]).abs()
    pick = torch.where((above < below) | ((above == below) & (upper % 2 == 0)), upper, lower)
    scale = table[pick][..., None]
    times = torch.trunc(x / scale)
    rest = (x / scale - times).abs()
    times = torch.where(rest >= 0.5, times + torch.sign(x), times)
    return (torch.minimum(torch.maximum(times, torch.tensor(-7.0, device=x.device, dtype=F64)),
                          torch.tensor(7.0, device=x.device, dtype=F64)) * scale).reshape(*x.shape[:-2], -1)


def _read64(blocks, n, d, channels_first):
    """Values of n tokens in 64 bits: blocks [m, H, bytes] of 16 tokens in their order."""
    table, G = _scale_table(), d // GROUP
    token = torch.arange(n, device="cuda")
    at, i = token // BLOCK, token % BLOCK
    out = torch.empty(n, blocks.shape[1], d, dtype=F64, device="cuda")
    for c in range(d):
        s = table[blocks[at, :, BLOCK * d // 2 + c // GROUP * BLOCK + i].long()]
        if channels_first:
            number, base = i, c * (BLOCK // 2)
        else:
            number, base = torch.full_like(i, c % GROUP), (c // GROUP * BLOCK + i) * (GROUP // 2)
        bit = 4 * (number % 8 // 2) + 16 * (number % 2)                        # of its word of 32
        byte = blocks[at, :, base + number // 8 * 4 + bit // 8].long()
        out[:, :, c] = ((byte >> (bit % 8)[:, None] & 15) - 8).to(F64) * s
    return out


def exact(case, seed):
    st = prepare(case, seed)
    lens, new, first = _lens(case)
    d, page = case["d"], case["page"]
    if case["op"] == "append":
        k, v = torch.zeros_like(st["k"], dtype=F64), torch.zeros_like(st["v"], dtype=F64)
        for b, n in enumerate(new):
            k[b, :n], v[b, :n] = _held64(st["k"][b, :n]), _held64(st["v"][b, :n])
        return {"k": k, "v": v}

    def dense(cache, table, n, channels_first):
        pages = cache[table[:-(-n // page)].long()]                            # [pages, H, blocks, bytes]
        return _read64(pages.transpose(1, 2).flatten(0, 1), n, d, channels_first)

    if case["op"] == "read":
        k, v = torch.zeros_like(st["k"], dtype=F64), torch.zeros_like(st["v"], dtype=F64)
        for b, (n, f) in enumerate(zip(lens, first)):
            k[b, :n - f] = dense(st["k_cache"], st["table"][b], n, False)[f:]
            v[b, :n - f] = dense(st["v_cache"], st["table"][b], n, True)[f:]
        return {"k": k, "v": v}
    B, T, P, Hq, Hkv = (case[n] for n in ("B", "T", "P", "Hq", "Hkv"))
    G = Hq // Hkv
    if work(case)["flops"] > 2e12:
        return None
    out = torch.zeros(B, T, Hq, d, dtype=F64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=F64, device="cuda")
    pk, pv = (dense(st[c], st["prefix_table"], P, x) for c, x in (("k_cache", False), ("v_cache", True)))
    for b in range(B):
        n, t = lens[b], new[b]
        if t == 0:
            continue
        k = torch.cat([pk, dense(st["k_cache"], st["table"][b], n, False)])
        v = torch.cat([pv, dense(st["v_cache"], st["table"][b], n, True)])
        hidden = None
        if case["causal"]:
            hidden = torch.arange(P + n, device="cuda")[None] > P + n - t + torch.arange(t, device="cuda")[:, None]
        for h in range(Hq):
            z = st["q"][b, :t, h].to(F64) @ k[:, h // G].T / math.sqrt(d)
            if hidden is not None:
                z[hidden] = -math.inf
            lse[b, h, :t] = torch.logsumexp(z, -1)
            keyed = torch.isfinite(lse[b, h, :t])
            out[b, :t, h][keyed] = torch.softmax(z[keyed], -1) @ v[:, h // G]
    return {"out": out, "lse": lse}

"""Measured cases of the operators that serve and train the positions and the key/value cache of the attention calls.

* rope:   rotary positions with several axes (time, height, width) on Q and K, forward and backward.
* append: new keys and values written into a paged cache, K rotated on the way, Q rotated beside it.
* paged:  attention of new tokens over a paged cache whose first ``prefix`` tokens every request shares.

Heads, head dims and lengths are those of the workloads in ``bsa_inputs/synthetic.py`` (24/8 and 32/8 heads of 128,
heads of 64, the 480p and 720p latents behind a text prefix) and generic serving sizes around them.
"""

import math
import random

import torch

own = False

BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
AXES = 3


def _rope(name, B, S, P, Hq, Hkv, d, grid, **kw):
    return {"op": "rope", "name": name, "B": B, "S": S, "P": P, "Hq": Hq, "Hkv": Hkv, "d": d, "pairs": d // 2, "fy": grid[0],
            "fx": grid[1], "far": 0, "interleaved": False, "fused": False, "backward": False, **kw}


def _append(name, B, T, Hq, Hkv, d, page, slots, **kw):
    return {"op": "append", "name": name, "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "slots": slots,
            "ragged": False, "interleaved": False, "spread": 1, **kw}


def _paged(name, B, T, P, low, high, Hq, Hkv, d, page, **kw):
    return {"op": "paged", "name": name, "B": B, "T": T, "P": P, "low": low, "high": high, "Hq": Hq, "Hkv": Hkv, "d": d,
            "page": page, "ragged": False, "causal": True, "spread": 1, **kw}


def listed():
    return [
        # one more text token of 16 requests, far along a stream: the smallest rotation, where the launch counts
        _rope("rope_step", 16, 1, 0, 32, 8, 128, (1, 1), far=100000, fused=True),
        # two pictures with their captions from one fused projection: heads of 64, 48 of the channels rotated, neighbours paired
        _rope("rope_image_d64", 2, 1337, 0, 4, 2, 64, (30, 52), pairs=24, interleaved=True, fused=True),
        # the 480p latent behind its text prefix, as the selector and the attention read it
        _rope("rope_480p", 1, 48360, 512, 24, 8, 128, (30, 52)),
        # the same rotation's backward pass in a training step on the 720p latent
        _rope("rope_720p_backward", 1, 172800, 1024, 32, 8, 128, (45, 80), backward=True),
        # one token each of 64 running requests
        _append("append_step", 64, 1, 32, 8, 128, 64, 2048),
        # prompts of unequal lengths on their way into small pages
        _append("append_prompts", 5, 4099, 24, 8, 128, 16, 8192, ragged=True),
        # one request, one token: latency alone
        _paged("decode_one", 1, 1, 0, 4097, 4097, 32, 8, 128, 64),
        # 64 requests on one long system prompt, each with its own answer so far
        _paged("decode_shared", 64, 1, 8209, 1, 1024, 32, 8, 128, 64),
        # 16 requests with long contexts of their own, nothing shared
        _paged("decode_long", 16, 1, 0, 1024, 65536, 32, 8, 128, 128),
        # five drafted tokens a request, heads of 64, small pages, prefix that ends inside a page
        _paged("verify_drafts_d64", 24, 5, 1000, 5, 2500, 4, 2, 64, 16),
        # 256 samples of one 32k prompt: the shared keys meet more query rows than memory bounds
        _paged("samples_of_one_prompt", 256, 1, 32768, 1, 512, 32, 8, 128, 64),
        # the next 500 tokens of two prompts over a shared prefix and what each already holds
        _paged("chunk_of_prompt", 2, 500, 4096, 500, 4100, 24, 8, 128, 128),
    ]


HEADS = ((32, 8, 128), (24, 8, 128), (24, 24, 128), (4, 2, 64), (3, 1, 64), (16, 2, 128), (8, 8, 64))


def _log(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    most = {"rope": 3.6e9, "append": 3.0e8, "paged": 2.0e9}
    while True:
        op = rng.choice(("rope", "append", "paged", "paged"))
        Hq, Hkv, d = rng.choice(HEADS)
        if op == "rope":
            P = rng.choice((0, 0, _log(rng, 1, 2000)))
            case = _rope("", rng.choice((1, 1, 2, 3, 16)), _log(rng, 1, 170000), P, Hq, Hkv, d, (rng.randint(1, 60), rng.randint(1, 90)),
                         pairs=rng.choice((d // 2, d // 2, 3 * d // 8, d // 4)), far=rng.choice((0, 0, rng.randint(1, 1000000))),
                         interleaved=rng.random() < 0.4, fused=P == 0 and rng.random() < 0.5, backward=rng.random() < 0.4)
        elif op == "append":
            T = rng.choice((1, 1, _log(rng, 1, 4096)))
            case = _append("", _log(rng, 1, 128), T, Hq, Hkv, d, rng.choice((16, 32, 64, 128)), T + _log(rng, 1, 4096),
                           ragged=T > 1 and rng.random() < 0.6, interleaved=rng.random() < 0.4, spread=rng.randint(1, 999))
        else:
            T = rng.choice((1, 1, 1, _log(rng, 1, 16), _log(rng, 1, 500)))
            low = T + _log(rng, 1, 2000) - 1
            case = _paged("", _log(rng, 1, 256), T, rng.choice((0, _log(rng, 1, 33000))), low, low + _log(rng, 1, 30000), Hq, Hkv, d,
                          rng.choice((16, 32, 64, 128)), ragged=T > 1 and rng.random() < 0.5, causal=rng.random() < 0.8,
                          spread=rng.randint(1, 999))
        w = work(case)
        pool = 2 * case["B"] * case["high"] * Hkv * d * 2 if op == "paged" else 2 * case["B"] * case["slots"] * Hkv * d * 2 if op == "append" else 0
        scores = 4 * case["B"] * Hq * case["T"] * (case["P"] + case["high"]) if op == "paged" else 0
        if w["bytes"] <= most[op] and w["flops"] <= 1.4e11 and pool <= 5e9 and scores <= 3e9:
            return case


# ---- what the cases share: lengths, positions, frequencies ----

def _lens(case):
    """(keys of its own, new tokens) of every request: fixed by the case alone."""
    r = random.Random(case["spread"] * 7919 + case["B"])
    T = case["T"]
    if case["op"] == "append":
        new = [r.randint(0, T) if case["ragged"] else T for _ in range(case["B"])]
        return [n + r.randint(0, case["slots"] - T) for n in new], new
    own_keys = [r.randint(case["low"], case["high"]) for _ in range(case["B"])]
    new = [r.randint(0, T) if case["ragged"] else T for _ in range(case["B"])]
    return own_keys, new


def _frequencies(pairs, dev):
    """One spectrum over all pairs, cut into a time, a height and a width section."""
    inv = 10000.0 ** (-torch.arange(pairs, dtype=F64, device=dev) / pairs)
    i = torch.arange(pairs, device=dev)
    axes = (i >= pairs // 4).to(I32) + (i >= pairs // 4 + (pairs - pairs // 4) // 2).to(I32)
    return inv, axes


def _grid_positions(n, text, fy, fx, far, dev):
    """Positions (t, h, w) of `text` tokens in a row and of n latent tokens behind them."""
    i = torch.arange(n, device=dev)
    t = torch.arange(text, device=dev)
    latent = torch.stack([i // (fy * fx), i // fx % fy, i % fx], 1) + text
    return (torch.cat([t[:, None].expand(text, AXES), latent]) + far).to(I32)


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=F32).to(BF) if math.prod(shape) < 1 << 28 else \
        torch.randn(shape, generator=g, device="cuda", dtype=BF)


def _pages(B, slots, page, shared, g):
    """Tables of pages in no order: [B, n] of the requests' own (-1 where a table has no page) and [m] of the shared prefix."""
    need = torch.tensor([-(-s // page) for s in slots])
    m = -(-shared // page)
    width = max(1, int(need.max()))
    total = int(need.sum()) + m + 3
    order = torch.randperm(total, generator=g, device="cuda").to(I32)
    column = torch.arange(width)
    number = torch.cumsum(need, 0)[:, None] - need[:, None] + column
    mine = torch.where(column < need[:, None], number, -1).cuda()
    table = torch.where(mine >= 0, order[mine.clamp(min=0) + m], -1).to(I32)
    return total, table, order[:m].clone()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    st = {"case": case}
    if case["op"] == "rope":
        S, P = case["S"], case["P"]
        if case["fused"]:
            qkv = _randn((B, S, Hq + 2 * Hkv, d), g)
            st["q"], st["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
        else:
            st["q"], st["k"] = _randn((B, S, Hq, d), g), _randn((B, P + S, Hkv, d), g)
        start = torch.randint(0, 50, (B,), generator=g, device="cuda", dtype=I32)     # each request stands elsewhere
        st["pos_k"] = _grid_positions(S, P, case["fy"], case["fx"], case["far"], "cuda")[None] + start[:, None, None]
        st["pos_q"] = st["pos_k"][:, P:]
        st["inv_freq"], st["axes"] = _frequencies(case["pairs"], "cuda")
        return st
    lens, new = _lens(case)
    T, page = case["T"], case["page"]
    st["kv_lens"] = torch.tensor(lens, dtype=I32, device="cuda")
    st["new_lens"] = torch.tensor(new, dtype=I32, device="cuda") if case["ragged"] else None
    if case["op"] == "append":
        total, st["table"], _ = _pages(B, [case["slots"]] * B, page, 0, g)
        qkv = _randn((B, T, Hq + 2 * Hkv, d), g)
        st["q"], st["k"], st["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        first = st["kv_lens"] - torch.tensor(new, dtype=I32, device="cuda")
        steps = torch.arange(T, dtype=I32, device="cuda")
        away = torch.randint(0, 90, (B, T, AXES), generator=g, device="cuda", dtype=I32)
        st["pos"] = (first[:, None] + steps)[:, :, None] + away
        st["inv_freq"], st["axes"] = _frequencies(d // 2, "cuda")
    else:
        total, st["table"], st["prefix_table"] = _pages(B, lens, page, case["P"], g)
        st["q"] = _randn((B, T, Hq, d), g)
    st["k_cache"], st["v_cache"] = _randn((total, page, Hkv, d), g), _randn((total, page, Hkv, d), g)
    return st


# ---- the plain forms ----

def _rotate(x, pos, inv_freq, axes, interleaved, back):
    angle = pos[:, :, axes.long()].to(F64) * inv_freq                 # far positions: the angle needs 64 bits
    c, s = torch.cos(angle).to(F32)[:, :, None], torch.sin(angle).to(F32)[:, :, None]
    s = -s if back else s
    n, half = axes.numel(), x.shape[3] // 2
    y = x.to(F32, copy=True)
    if interleaved:
        a, b = y[..., 0:2 * n:2], y[..., 1:2 * n:2]
    else:
        a, b = y[..., :n], y[..., n:2 * n]
    a0 = a.clone()
    a.copy_(a0 * c - b * s)
    b.copy_(b * c + a0 * s)
    return y.to(BF)


def _plain_append(st):
    T = st["case"]["T"]
    kv, new, page = st["kv_lens"].long(), st["new_lens"], st["case"]["page"]
    new = torch.full_like(kv, T) if new is None else new.long()
    k = _rotate(st["k"], st["pos"], st["inv_freq"], st["axes"], st["case"]["interleaved"], False)
    q = _rotate(st["q"], st["pos"], st["inv_freq"], st["axes"], st["case"]["interleaved"], False)
    t = torch.arange(T, device=kv.device)
    slot = (kv - new)[:, None] + t
    real = t < new[:, None]
    where = torch.gather(st["table"].long(), 1, (slot // page).clamp(0, st["table"].shape[1] - 1))
    st["k_cache"][where[real], slot[real] % page] = k[real]
    st["v_cache"][where[real], slot[real] % page] = st["v"][real]
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"], "q": q}


def _plain_paged(st):
    case = st["case"]
    B, T, P, Hq, Hkv, d = (case[n] for n in ("B", "T", "P", "Hq", "Hkv", "d"))
    kv, new = st["kv_lens"].long(), st["new_lens"]
    new = torch.full_like(kv, T) if new is None else new.long()
    q = st["q"].to(F32).view(B, T, Hkv, Hq // Hkv, d) * d ** -0.5
    table = st["table"].long().clamp(min=0)
    own_k, own_v = st["k_cache"][table].to(F32).flatten(1, 2), st["v_cache"][table].to(F32).flatten(1, 2)
    n, dev = own_k.shape[1], kv.device
    key, row = torch.arange(n, device=dev), torch.arange(T, device=dev)
    last = kv[:, None] - new[:, None] + row if case["causal"] else (kv[:, None] - 1).expand(B, T)
    real = row < new[:, None]
    seen = (key <= last[:, :, None]) & (key < kv[:, None, None])                       # [B, T, n]
    s = torch.einsum("bthgd,bnhd->bthgn", q, own_k).masked_fill(~seen[:, :, None, None], -math.inf)
    own_v = own_v.masked_fill((key >= kv[:, None])[:, :, None, None], 0.0)
    if P:
        pk = st["k_cache"][st["prefix_table"].long()].to(F32).flatten(0, 1)[:P]
        pv = st["v_cache"][st["prefix_table"].long()].to(F32).flatten(0, 1)[:P]
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
        if case["op"] == "rope":
            call = bsa.bsa_rope_axes_backward if case["backward"] else bsa.bsa_rope_axes
            q, k = call(st["q"], st["k"], st["pos_q"], st["pos_k"], st["inv_freq"], st["axes"], interleaved=case["interleaved"])
            return {"q": q, "k": k}
        if case["op"] == "append":
            q = bsa.bsa_cache_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["kv_lens"],
                                     new_lens=st["new_lens"], q=st["q"], positions=st["pos"], inv_freq=st["inv_freq"],
                                     axes=st["axes"], interleaved=case["interleaved"])
            return {"k_cache": st["k_cache"], "v_cache": st["v_cache"], "q": q}
        out, lse = bsa.bsa_forward_paged(st["q"], st["k_cache"], st["v_cache"], st["table"], st["kv_lens"],
                                         new_lens=st["new_lens"], prefix_table=st["prefix_table"], prefix_len=case["P"],
                                         causal=case["causal"])
        return {"out": out, "lse": lse}
    if case["op"] == "rope":
        back = case["backward"]
        return {"q": _rotate(st["q"], st["pos_q"], st["inv_freq"], st["axes"], case["interleaved"], back),
                "k": _rotate(st["k"], st["pos_k"], st["inv_freq"], st["axes"], case["interleaved"], back)}
    return _plain_append(st) if case["op"] == "append" else _plain_paged(st)


def work(case):
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "rope":
        S, P = case["S"], case["P"]
        values = B * d * (S * Hq + (P + S) * Hkv)
        turned = values // d * 2 * case["pairs"]
        return {"bytes": 4 * values + 4 * AXES * B * (P + S) + 12 * case["pairs"], "flops": 3 * turned}
    lens, new = _lens(case)
    T = case["T"]
    if case["op"] == "append":
        # q is rotated whole, k and v are read and written where a token is real; positions and one table entry a token
        values = sum(new) * 2 * Hkv * d + B * T * Hq * d
        return {"bytes": 4 * values + 4 * (AXES + 1) * B * T + 8 * B, "flops": 3 * (sum(new) * Hkv * d + B * T * Hq * d)}
    P = case["P"]
    # the prefix once for all, each request's own keys once
    seen = sum(new) * P
    for n, t in zip(lens, new):
        # row i of t sees n - t + i + 1 of its own keys
        seen += sum(max(0, n - t + i + 1) for i in range(t)) if case["causal"] else n * t
    kv = P + sum(n for n, t in zip(lens, new) if t)
    return {"bytes": 4 * kv * Hkv * d + 4 * B * T * Hq * d + 4 * B * Hq * T + 4 * (kv // case["page"]), "flops": 4 * seen * Hq * d}


# ---- the definitions in 64 bits ----

def _turn64(x, pos, inv_freq, axes, interleaved, back):
    """Each pair is a complex number; its rotation is a product with exp(i angle)."""
    n = axes.numel()
    out = x.to(F64)
    place = torch.arange(n, device=x.device)
    lo, hi = (2 * place, 2 * place + 1) if interleaved else (place, place + n)
    angle = torch.stack([pos[:, :, a].to(F64) for a in axes.tolist()], -1) * inv_freq
    turn = torch.polar(torch.ones_like(angle), -angle if back else angle)
    for h in range(x.shape[2]):
        z = torch.complex(out[:, :, h][..., lo], out[:, :, h][..., hi]) * turn
        out[:, :, h, lo], out[:, :, h, hi] = z.real, z.imag
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        args = (st["inv_freq"], st["axes"], case["interleaved"], case["backward"])
        return {"q": _turn64(st["q"], st["pos_q"], *args), "k": _turn64(st["k"], st["pos_k"], *args)}
    lens, new = _lens(case)
    page = case["page"]
    if case["op"] == "append":
        args = (st["inv_freq"], st["axes"], case["interleaved"], False)
        k, q = _turn64(st["k"], st["pos"], *args), _turn64(st["q"], st["pos"], *args)
        kc, vc = st["k_cache"].to(F64), st["v_cache"].to(F64)
        for b in range(case["B"]):
            slot = torch.arange(lens[b] - new[b], lens[b], device="cuda")
            at = st["table"][b, slot // page].long()
            kc[at, slot % page] = k[b, :new[b]]
            vc[at, slot % page] = st["v"][b, :new[b]].to(F64)
        return {"k_cache": kc, "v_cache": vc, "q": q}
    B, T, P, Hq, Hkv, d = (case[n] for n in ("B", "T", "P", "Hq", "Hkv", "d"))
    G = Hq // Hkv
    if work(case)["flops"] > 2e12:
        return None
    out = torch.zeros(B, T, Hq, d, dtype=F64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=F64, device="cuda")

    def dense(cache, table, n):
        return cache[table[:-(-n // page)].long()].reshape(-1, Hkv, d)[:n].to(F64)

    pk, pv = dense(st["k_cache"], st["prefix_table"], P), dense(st["v_cache"], st["prefix_table"], P)
    for b in range(B):
        n, t = lens[b], new[b]
        if t == 0:
            continue
        k, v = torch.cat([pk, dense(st["k_cache"], st["table"][b], n)]), torch.cat([pv, dense(st["v_cache"], st["table"][b], n)])
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

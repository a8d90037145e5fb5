"""Multi-axis rotation, paged append and paged attention on the GPU against
plain 64-bit forms (bounds: paged_utils)."""

import math
from decimal import Decimal, getcontext

import pytest
import torch

import block_sparse_attention_bsa_gb300 as bsa
from paged_utils import BF, Pool, attend64, check_attention, rotate64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    bsa.build()


def randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF)


# ------------------------------------------------------------ rotation ---

ROPE_CASES = [
    # B, S, Hq, Hkv, d, sections, interleaved
    (1, 1, 1, 1, 64, (8, 0, 0), False),
    (3, 1, 32, 8, 128, (16, 24, 24), False),
    (2, 37, 4, 2, 64, (8, 12, 12), True),
    (2, 129, 3, 1, 64, (4, 2, 2), False),         # 16 of 64 channels
    (1, 1000, 5, 5, 128, (40,), True),            # 80 of 128 channels, one axis
    (1, 515, 24, 8, 128, (8, 16, 16, 8), False),  # four axes, 96 of 128 channels
    (1, 20011, 2, 1, 128, (16, 24, 24), False),
]


@pytest.mark.parametrize("B,S,Hq,Hkv,d,sections,inter", ROPE_CASES)
@pytest.mark.parametrize("back", [False, True])
def test_rotation_matches_64_bits(B, S, Hq, Hkv, d, sections, inter, back):
    q, k = randn((B, S, Hq, d), 1), randn((B, S + 3, Hkv, d), 2)
    A = len(sections)
    g = torch.Generator().manual_seed(3)
    pq = torch.randint(-2000, 2000000, (B, S, A), generator=g, dtype=torch.int32)
    pk = torch.randint(0, 50, (B, S + 3, A), generator=g, dtype=torch.int32)
    inv, axes = bsa.bsa_axis_frequencies(sections, 10000.0, "cycled", DEV)
    call = bsa.bsa_rope_axes_backward if back else bsa.bsa_rope_axes
    gq, gk = call(q.to(DEV), k.to(DEV), pq.to(DEV), pk.to(DEV), inv, axes, interleaved=inter)
    for got, x, pos in ((gq, q, pq), (gk, k, pk)):
        assert got.is_contiguous() and got.dtype == BF
        y, bound = rotate64(x, pos, inv.cpu(), axes.cpu(), inter, back)
        err = (got.double().cpu() - y).abs()
        assert (err <= bound).all(), float((err - bound).max())


def test_rotation_is_exact_at_far_positions():
    """Positions up to 2^31 - 1 and frequencies above one turn, against turns
    reduced in 60 decimal digits."""
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    freqs = [1.0, 0.1, 1e-4, 3.7e-7, 7.25, 900.5, -0.3, 2.0 ** -60]
    pos = [0, 1, -1, 12345, 1 << 20, (1 << 31) - 1, -(1 << 31), 999999937]
    x = randn((1, len(pos), 1, 64), 4)
    inv = torch.tensor(freqs, dtype=torch.float64, device=DEV)
    axes = torch.zeros(8, dtype=torch.int32, device=DEV)
    p = torch.tensor(pos, dtype=torch.int32, device=DEV)[:, None]
    got, _ = bsa.bsa_rope_axes(x.to(DEV), None, p, None, inv, axes)
    got = got.double().cpu()
    for s, w in enumerate(pos):
        for i, f in enumerate(freqs):
            angle = float((Decimal(w) * Decimal(f)) % two_pi)
            a, b = float(x[0, s, 0, i]), float(x[0, s, 0, i + 8])
            for ch, y in ((i, a * math.cos(angle) - b * math.sin(angle)), (i + 8, b * math.cos(angle) + a * math.sin(angle))):
                assert abs(float(got[0, s, 0, ch]) - y) <= 2.0 ** -8 * abs(y) + (abs(a) + abs(b)) * 2.0 ** -20, (w, f)
    assert torch.equal(got[..., 16:], x[..., 16:].double())


def test_rotation_reads_strided_broadcast_and_permuted_inputs():
    B, S, Hq, Hkv, d = 2, 33, 6, 2, 64
    inv, axes = bsa.bsa_axis_frequencies((8, 12, 12), device=DEV)
    pos = torch.randint(0, 999, (3, B, S), dtype=torch.int32, generator=torch.Generator().manual_seed(5)).to(DEV)
    qkv = randn((B, S, Hq + 2 * Hkv, d), 6).to(DEV)
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
    p = pos.permute(1, 2, 0)                                    # positions kept as [axes, B, S]
    a = bsa.bsa_rope_axes(q, k, p, p, inv, axes)
    b = bsa.bsa_rope_axes(q.contiguous(), k.contiguous(), p.contiguous(), p.contiguous(), inv, axes)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    one = randn((1, 1, 1, d), 7).to(DEV)                        # a broadcast gradient, positions shared by the batch
    got, none = bsa.bsa_rope_axes_backward(one.expand(B, S, Hq, d), None, p[0], None, inv, axes)
    want, _ = bsa.bsa_rope_axes_backward(one.expand(B, S, Hq, d).contiguous(), None, p[:1].expand(B, S, 3).contiguous(),
                                         None, inv, axes)
    assert none is None and torch.equal(got, want)


def test_rotation_in_place_equals_out_of_place_and_refuses_other_overlap():
    q = randn((2, 50, 9, 128), 8).to(DEV)
    inv, axes = bsa.bsa_axis_frequencies((16, 24, 24), device=DEV)
    pos = torch.arange(150, dtype=torch.int32, device=DEV).view(50, 3)
    want, _ = bsa.bsa_rope_axes(q, None, pos, None, inv, axes)
    mine = q.clone()
    got, _ = bsa.bsa_rope_axes(mine, None, pos, None, inv, axes, q_out=mine)
    assert got is mine and torch.equal(mine, want)
    flat = torch.zeros(q.numel() + 64, dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="overlaps"):
        bsa.bsa_rope_axes(flat[64:].view(q.shape), None, pos, None, inv, axes, q_out=flat[:-64].view(q.shape))
    with pytest.raises(ValueError, match="overlaps"):
        bsa.bsa_rope_axes(q, q, pos, pos, inv, axes, q_out=want, k_out=want)


def test_rotation_gradient_against_differences():
    """The backward pass is the transpose: <R x, g> = <x, R^T g>, and it agrees
    with differences of the forward pass (linear in x, so a difference of any
    length is exact up to the outputs' roundings)."""
    B, S, H, d = 1, 7, 2, 64
    inv, axes = bsa.bsa_axis_frequencies((8, 8, 8), 100.0, "per_axis", DEV)
    pos = torch.randint(0, 4000, (B, S, 3), dtype=torch.int32, generator=torch.Generator().manual_seed(9)).to(DEV)
    x, g = randn((B, S, H, d), 10).to(DEV), randn((B, S, H, d), 11).to(DEV)
    dx, _ = bsa.bsa_rope_axes_backward(g, None, pos, None, inv, axes)
    base, _ = bsa.bsa_rope_axes(x, None, pos, None, inv, axes)
    f0 = (base.double() * g.double()).sum((1, 2, 3))
    for ch in (0, 5, 23, 24, 40, 47, 48, 63):
        step = torch.zeros_like(x)
        step[0, 3, 1, ch] = 4.0                                  # x + step is rounded: take the step that was made
        moved = x + step
        made = float(moved[0, 3, 1, ch] - x[0, 3, 1, ch])
        y, _ = bsa.bsa_rope_axes(moved, None, pos, None, inv, axes)
        diff = float(((y.double() - base.double()) * g.double()).sum()) / made
        # at most two outputs change, by at most `made`; each of the two calls rounds them by 2^-8
        touched = (y != base).nonzero()
        assert len(touched) <= 2
        slack = sum(2.0 ** -8 * (abs(float(y[tuple(t)])) + abs(float(base[tuple(t)]))) * abs(float(g[tuple(t)]))
                    for t in touched) / abs(made)
        assert abs(diff - float(dx[0, 3, 1, ch])) <= slack + 2.0 ** -8 * abs(float(dx[0, 3, 1, ch])) + 1e-5, ch
    assert torch.isfinite(f0).all()


# ------------------------------------------------------------- append ---

APPEND_CASES = [
    # T, new_lens, kv_lens (with the new ones), Hkv, d, page, layout
    (1, None, [1, 16, 17, 300], 8, 128, 16, "slots"),
    (1, [1, 0, 1, 1], [64, 0, 65, 200], 2, 64, 64, "heads"),
    (70, [70, 0, 33, 1], [70, 5, 128, 129], 3, 64, 32, "pairs"),
    (300, None, [300, 557], 1, 128, 256, "slots"),
    (129, [129, 64], [129, 500], 2, 128, 128, "heads"),
]


@pytest.mark.parametrize("T,new,kv,Hkv,d,page,layout", APPEND_CASES)
@pytest.mark.parametrize("turned", ["no", "half", "neighbours"])
def test_append_writes_the_new_tokens_and_nothing_else(T, new, kv, Hkv, d, page, layout, turned):
    B, Hq = len(kv), 2 * Hkv
    pool = Pool(kv, 0, Hkv, d, page, DEV, 20, layout=layout, fill=-7.0)
    qkv = randn((B, T, Hq + 2 * Hkv, d), 21)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    before_k, before_v = pool.gk.clone(), pool.gv.clone()
    gq, gk, gv = qkv.to(DEV)[:, :, :Hq], qkv.to(DEV)[:, :, Hq:Hq + Hkv], qkv.to(DEV)[:, :, Hq + Hkv:]
    pos = torch.randint(0, 3000, (B, T, 3), dtype=torch.int32, generator=torch.Generator().manual_seed(22))
    inv, axes = bsa.bsa_axis_frequencies((8, 8, 8), device=DEV)
    kw = {} if turned == "no" else dict(q=gq, positions=pos.to(DEV), inv_freq=inv, axes=axes,
                                        interleaved=turned == "neighbours")
    new_t = None if new is None else torch.tensor(new, dtype=torch.int32, device=DEV)
    got = bsa.bsa_cache_append(gk, gv, pool.gk, pool.gv, pool.gtable, pool.kv_lens, new_lens=new_t, **kw)
    bsa.bsa_device_status()
    if turned == "no":
        assert got is None
        ky, kb = k.double(), torch.zeros(k.shape, dtype=torch.float64)
    else:
        ky, kb = rotate64(k, pos, inv.cpu(), axes.cpu(), turned == "neighbours")
        qy, qb = rotate64(q, pos, inv.cpu(), axes.cpu(), turned == "neighbours")
        assert ((got.double().cpu() - qy).abs() <= qb).all()
    ck, cv = pool.gk.cpu(), pool.gv.cpu()
    touched = torch.zeros(pool.total, page, dtype=torch.bool)
    for b in range(B):
        n = T if new is None else new[b]
        for t in range(n):
            j = kv[b] - n + t
            at, slot = int(pool.table[b, j // page]), j % page
            touched[at, slot] = True
            assert ((ck[at, slot].double() - ky[b, t]).abs() <= kb[b, t]).all(), (b, t)
            assert torch.equal(cv[at, slot], v[b, t])
    assert torch.equal(ck[~touched], before_k.cpu()[~touched])
    assert torch.equal(cv[~touched], before_v.cpu()[~touched])


def test_append_drops_and_reports_tokens_without_a_page():
    pool = Pool([40, 40, 40], 0, 2, 64, 16, DEV, 23, fill=1.0)
    k = randn((3, 8, 2, 64), 24).to(DEV)
    table = pool.gtable.clone()
    table[1, 2] = pool.total                                     # names no page: tokens at 32..39 of request 1
    table[2, 2] = -1
    lens = torch.tensor([52, 40, 40], dtype=torch.int32, device=DEV)   # request 0: tokens at 44..51, 48.. behind the table
    before = pool.gk.clone()
    bsa.bsa_cache_append(k, k, pool.gk, pool.gv, table, lens)
    with pytest.raises(bsa.BsaError, match="BSA_ERR_INVALID_INDICES.*bsap_cache_append"):
        bsa.bsa_device_status()
    bsa.bsa_device_status()                                       # reported once
    want = before.clone()
    want[int(table[0, 2]), 12:16] = k[0, :4]
    assert torch.equal(pool.gk, want)
    lens[:] = torch.tensor([3, 8, 8])                             # request 0: 8 new tokens, positions -5 .. 2
    bsa.bsa_cache_append(k, k, pool.gk, pool.gv, table, lens)
    with pytest.raises(bsa.BsaError, match="BSA_ERR_INVALID_INDICES"):
        bsa.bsa_device_status()
    want[int(table[0, 0]), :3] = k[0, 5:]
    want[int(table[1, 0]), :8], want[int(table[2, 0]), :8] = k[1], k[2]
    assert torch.equal(pool.gk, want)


# ---------------------------------------------------------- attention ---

ATTEND_CASES = [
    # lens (own keys), T, new_lens, prefix, Hq, Hkv, d, page, causal, layout
    ([1], 1, None, 0, 1, 1, 64, 16, True, "slots"),
    ([128], 1, None, 0, 4, 1, 128, 64, True, "slots"),
    ([129, 0, 1, 127], 1, [1, 1, 1, 0], 0, 8, 2, 128, 32, True, "heads"),
    ([5, 0, 300], 1, None, 1, 8, 2, 64, 16, True, "pairs"),
    ([7, 260, 64], 1, None, 300, 6, 2, 128, 128, True, "slots"),
    ([40, 9, 513], 5, [5, 0, 3], 77, 4, 2, 64, 16, True, "slots"),
    ([40, 2, 140], 5, None, 0, 3, 3, 128, 16, True, "heads"),      # 2 keys for 5 tokens: rows before them are empty
    ([40, 2, 140], 5, None, 129, 8, 1, 128, 256, False, "slots"),
    ([300, 130], 130, [130, 60], 200, 4, 2, 64, 64, True, "slots"),  # several row tiles a request
    ([257], 257, None, 0, 6, 2, 128, 128, True, "pairs"),
    ([257, 600], 200, [0, 200], 128, 2, 2, 128, 32, False, "slots"),
    ([3000], 1, None, 0, 16, 1, 128, 64, True, "slots"),
    ([0, 0], 3, None, 500, 5, 1, 64, 256, True, "slots"),
    ([0, 0], 2, None, 0, 5, 1, 128, 16, True, "slots"),              # no key at all
    ([20] * 70, 1, None, 130, 4, 1, 64, 16, True, "slots"),          # more than one block of requests, 3 row tiles
    ([1, 2, 3, 128, 129, 255, 256, 257], 2, None, 127, 64, 1, 64, 16, True, "slots"),
    ([50, 300], 1, None, 40, 256, 1, 64, 16, True, "heads"),          # one token fills two jobs' rows
    ([200, 70, 66], 65, [65, 30, 64], 0, 2, 1, 128, 32, True, "slots"),   # rows of one request in two jobs, of another in one
    ([33], 1, None, 5, 256, 256, 64, 16, True, "slots"),
    ([300], 1, None, 1000, 4, 2, 64, 64, True, "slots"),              # one request: prefix and own keys in one segment
    ([0], 3, None, 129, 4, 2, 128, 16, True, "heads"),
    ([2], 9, None, 128, 4, 2, 64, 16, True, "pairs"),
]


@pytest.mark.parametrize("lens,T,new,prefix,Hq,Hkv,d,page,causal,layout", ATTEND_CASES)
def test_attention_matches_64_bits(lens, T, new, prefix, Hq, Hkv, d, page, causal, layout):
    pool = Pool(lens, prefix, Hkv, d, page, DEV, 30, layout=layout)
    q = randn((len(lens), T, Hq, d), 31)
    if T > 1:                                     # padded rows of q hold anything
        for b, n in enumerate(new or []):
            q[b, n:] = float("nan")
    new_t = None if new is None else torch.tensor(new, dtype=torch.int32, device=DEV)
    out, lse = bsa.bsa_forward_paged(q.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens, new_lens=new_t,
                                     prefix_table=pool.gprefix, prefix_len=prefix, causal=causal)
    bsa.bsa_device_status()
    check_attention(out, lse, attend64(q, pool, new, causal))
    again, lse2 = bsa.bsa_forward_paged(q.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens, new_lens=new_t,
                                        prefix_table=pool.gprefix, prefix_len=prefix, causal=causal)
    assert torch.equal(out, again) and torch.equal(lse, lse2)      # nothing depends on scheduling


def test_attention_of_large_logits_and_given_scale():
    """Logits of hundreds, keys in rising order (the running maximum grows at
    every tile), a scale of its own, strided q, no lse."""
    pool = Pool([700], 400, 2, 128, 64, DEV, 32)
    q = randn((1, 1, 4, 128), 33)
    for rows in (pool.pre_k, pool.own_k[0]):
        for h in range(2):
            order = torch.argsort((rows[:, h].float() @ q[0, 0, 2 * h].float()))
            rows[:, h] = rows[order, h]
    for j in range(400):
        pool.gk[int(pool.prefix_table[j // 64]), j % 64] = pool.pre_k[j].to(DEV)
    for j in range(700):
        pool.gk[int(pool.table[0, j // 64]), j % 64] = pool.own_k[0][j].to(DEV)
    wide = torch.empty(1, 1, 9, 128, dtype=BF, device=DEV)
    wide[:, :, 3:7] = q.to(DEV)
    for scale in (3.0, 0.01):
        out, lse = bsa.bsa_forward_paged(wide[:, :, 3:7], pool.gk, pool.gv, pool.gtable, pool.kv_lens,
                                         prefix_table=pool.gprefix, prefix_len=400, softmax_scale=scale)
        check_attention(out, lse, attend64(q, pool, scale=scale))
        only, none = bsa.bsa_forward_paged(wide[:, :, 3:7], pool.gk, pool.gv, pool.gtable, pool.kv_lens,
                                           prefix_table=pool.gprefix, prefix_len=400, softmax_scale=scale,
                                           return_lse=False)
        assert none is None and torch.equal(only, out)


def test_attention_reports_tables_that_name_no_page():
    pool = Pool([100, 30], 50, 1, 64, 16, DEV, 34, fill=0.0)
    q = randn((2, 1, 2, 64), 35).to(DEV)
    good, _ = bsa.bsa_forward_paged(q, pool.gk, pool.gv, pool.gtable, pool.kv_lens, prefix_table=pool.gprefix,
                                    prefix_len=50)
    bsa.bsa_device_status()
    for what in ("own", "prefix", "length"):
        table, shared, lens = pool.gtable.clone(), pool.gprefix.clone(), pool.kv_lens.clone()
        if what == "own":
            table[0, 3] = pool.total
        elif what == "prefix":
            shared[1] = -5
        else:
            lens[0] = table.shape[1] * 16 + 1
        out, _ = bsa.bsa_forward_paged(q, pool.gk, pool.gv, table, lens, prefix_table=shared, prefix_len=50)
        with pytest.raises(bsa.BsaError, match="BSA_ERR_INVALID_INDICES.*bsap_forward"):
            bsa.bsa_device_status()
        if what != "prefix":
            assert torch.equal(out[1], good[1])                   # the other request is as it was


def attend64_one(q, k, v, lens, prefix_k, prefix_v):
    """One token per request, all requests at once on the GPU in 64 bits:
    k, v [B, n, Hkv, d] (rows behind lens hold zeros).  (out, lse, bounds)"""
    B, _, Hq, d = q.shape
    Hkv, n = k.shape[2], k.shape[1]
    qq = q.double().view(B, Hkv, Hq // Hkv, d)
    z = torch.einsum("bhgd,bnhd->bhgn", qq, k.double()) * d ** -0.5
    za = torch.einsum("bhgd,bnhd->bhgn", qq.abs(), k.double().abs()) * d ** -0.5
    hidden = (torch.arange(n, device=q.device) >= lens[:, None])[:, None, None]
    z, za = z.masked_fill(hidden, -math.inf), za.masked_fill(hidden, 0.0)
    zp = torch.einsum("bhgd,nhd->bhgn", qq, prefix_k.double()) * d ** -0.5
    zpa = torch.einsum("bhgd,nhd->bhgn", qq.abs(), prefix_k.double().abs()) * d ** -0.5
    z, dz = torch.cat([zp, z], -1), 2.0 ** -15 * torch.cat([zpa, za], -1).amax(-1)
    w = torch.softmax(z, -1)
    P = prefix_k.shape[0]

    def mix(f):
        return torch.einsum("bhgn,bnhd->bhgd", w[..., P:], f(v.double())) + \
            torch.einsum("bhgn,nhd->bhgd", w[..., :P], f(prefix_v.double()))

    out, reach, lse = mix(lambda x: x), mix(torch.abs), torch.logsumexp(z, -1)
    ob = 2.0 ** -8 * out.abs() + (2 * dz[..., None] + 2.0 ** -8 + 2.0 ** -12) * reach
    lb = dz + 2.0 ** -19 * (lse.abs() + 1)
    return tuple(x.cpu() for x in (out.reshape(B, 1, Hq, d), lse.reshape(B, Hq, 1), ob.reshape(B, 1, Hq, d), lb.reshape(B, Hq, 1)))


@pytest.mark.parametrize("B,prefix,low,high,Hq,Hkv,d,page", [
    (300, 0, 1, 300, 8, 4, 128, 64),          # many short segments in every CTA, none of them cut or joined but few
    (300, 257, 0, 140, 8, 4, 64, 16),         # one or two tiles each, beside a prefix with ten row tiles
    (700, 129, 100, 128, 4, 4, 128, 128),     # single tiles only
    (6, 20000, 1000, 9000, 32, 2, 128, 128),  # long runs of tiles, cut many times
    (64, 0, 4096, 4096, 16, 8, 128, 128),
    (4096, 100, 0, 40, 2, 1, 64, 16),         # the largest batch
    (97, 0, 30, 31, 8, 8, 64, 32),            # fewer tiles than a CTA has warps, many requests without a cut
])
def test_attention_over_many_segments_matches_64_bits(B, prefix, low, high, Hq, Hkv, d, page):
    g = torch.Generator(device=DEV).manual_seed(B + high)
    lens = torch.randint(low, high + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    width, shared = -(-high // page), -(-prefix // page)
    total = B * width + shared + 1
    kc, vc = (torch.randn(total, page, Hkv, d, generator=g, device=DEV).to(BF) for _ in range(2))
    order = torch.randperm(total, generator=g, device=DEV).int()
    table, pt = order[:B * width].view(B, width), order[B * width:B * width + shared]
    q = torch.randn(B, 1, Hq, d, generator=g, device=DEV).to(BF)
    k, v = (c[table.long()].flatten(1, 2) for c in (kc, vc))
    pk, pv = (c[pt.long()].flatten(0, 1)[:prefix] for c in (kc, vc))
    ref = attend64_one(q, k, v, lens, pk, pv)
    out, lse = bsa.bsa_forward_paged(q, kc, vc, table, lens, prefix_table=pt, prefix_len=prefix)
    bsa.bsa_device_status()
    check_attention(out, lse, ref)
    for _ in range(3):
        again, lse2 = bsa.bsa_forward_paged(q, kc, vc, table, lens, prefix_table=pt, prefix_len=prefix)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    bsa.bsa_device_status()


@pytest.mark.parametrize("T,new,kv,prefix,Hq,Hkv,d,page,causal", [
    (1500, [1500, 700], [1500, 2100], 300, 4, 1, 128, 64, True),      # 24 row tiles a request, a prefix beside them
    (1100, [1100, 0, 257], [1300, 40, 257], 0, 6, 2, 64, 16, True),   # no prefix: whole segments are written at once
    (600, [600, 431], [900, 431], 129, 3, 3, 128, 256, False),
    (8200, [8200], [8200], 0, 1, 1, 64, 128, True),                   # 33 row tiles
    (700, [700, 700, 333], [700, 1000, 333], 128, 2, 1, 64, 32, True),    # a prefix of one whole tile at the head of each
    (512, [512, 0, 100, 512], [512, 7, 100, 600], 1000, 8, 2, 128, 16, True),
])
def test_attention_of_long_chunks_matches_64_bits(T, new, kv, prefix, Hq, Hkv, d, page, causal):
    g = torch.Generator(device=DEV).manual_seed(T)
    B, G = len(kv), Hq // Hkv
    width, shared = -(-max(kv) // page), -(-prefix // page)
    total = B * width + shared + 1
    kc, vc = (torch.randn(total, page, Hkv, d, generator=g, device=DEV).to(BF) for _ in range(2))
    order = torch.randperm(total, generator=g, device=DEV).int()
    table, pt = order[:B * width].view(B, width), order[B * width:B * width + shared]
    q = torch.randn(B, T, Hq, d, generator=g, device=DEV).to(BF)
    lens, new_t = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (kv, new))
    out, lse = bsa.bsa_forward_paged(q, kc, vc, table, lens, new_lens=new_t, prefix_table=pt, prefix_len=prefix,
                                     causal=causal)
    bsa.bsa_device_status()
    for b in range(B):
        n = new[b]
        assert (out[b, n:] == 0).all() and torch.isneginf(lse[b, :, n:]).all()
        if n == 0:
            continue
        k, v = (torch.cat([c[pt.long()].flatten(0, 1)[:prefix], c[table[b].long()].flatten(0, 1)[:kv[b]]]).double()
                for c in (kc, vc))
        hidden = None
        if causal:
            hidden = torch.arange(prefix + kv[b], device=DEV) > prefix + kv[b] - n + torch.arange(n, device=DEV)[:, None]
        for h in range(Hq):
            qq, kk, vv = q[b, :n, h].double(), k[:, h // G], v[:, h // G]
            z = qq @ kk.T * d ** -0.5
            za = qq.abs() @ kk.abs().T * d ** -0.5
            if hidden is not None:
                z, za = z.masked_fill(hidden, -math.inf), za.masked_fill(hidden, 0.0)
            dz = 2.0 ** -15 * za.amax(-1)
            w, ref_lse = torch.softmax(z, -1), torch.logsumexp(z, -1)
            ref = w @ vv
            bound = 2.0 ** -8 * ref.abs() + (2 * dz[:, None] + 2.0 ** -8 + 2.0 ** -12) * (w @ vv.abs())
            assert ((out[b, :n, h].double() - ref).abs() <= bound).all(), (b, h)
            assert ((lse[b, h, :n].double() - ref_lse).abs() <= dz + 2.0 ** -19 * (ref_lse.abs() + 1)).all(), (b, h)


def test_attention_over_the_prefix_alone():
    """A table without pages: no own keys at all."""
    pool = Pool([0, 0, 0], 333, 2, 64, 32, DEV, 40)
    q = randn((3, 2, 6, 64), 41)
    none = torch.empty((3, 0), dtype=torch.int32, device=DEV)
    out, lse = bsa.bsa_forward_paged(q.to(DEV), pool.gk, pool.gv, none, pool.kv_lens, prefix_table=pool.gprefix,
                                     prefix_len=333)
    bsa.bsa_device_status()
    check_attention(out, lse, attend64(q, pool))


def test_append_rotates_queries_in_place():
    pool = Pool([9, 30], 0, 2, 128, 16, DEV, 42, fill=0.0)
    q, k = randn((2, 5, 4, 128), 43).to(DEV), randn((2, 5, 2, 128), 44).to(DEV)
    pos = torch.randint(0, 99, (2, 5, 2), dtype=torch.int32, generator=torch.Generator().manual_seed(45)).to(DEV)
    inv, axes = bsa.bsa_axis_frequencies((20, 12), layout="per_axis", device=DEV)
    want, _ = bsa.bsa_rope_axes(q, None, pos, None, inv, axes)
    mine = q.clone()
    got = bsa.bsa_cache_append(k, k, pool.gk, pool.gv, pool.gtable, pool.kv_lens, q=mine, q_out=mine, positions=pos,
                               inv_freq=inv, axes=axes)
    assert got is mine and torch.equal(mine, want)
    bsa.bsa_device_status()


@pytest.mark.parametrize("prefix,Hq,Hkv,d,page", [(0, 8, 2, 128, 64), (0, 4, 4, 64, 16), (300, 8, 2, 128, 32)])
def test_attention_of_single_tokens_beside_chunks(prefix, Hq, Hkv, d, page):
    """Single tokens and chunks of up to 80 in turn: blocks go from segments of a
    few rows to segments of several row tiles and back, with ends inside tiles."""
    g = torch.Generator().manual_seed(prefix + page)
    new = [(1, 80, 2, 33, 1, 1, 64, 17, 0, 40)[b % 10] for b in range(100)]
    lens = [max(n, int(torch.randint(0, 400, (1,), generator=g))) for n in new]
    pool = Pool(lens, prefix, Hkv, d, page, DEV, 40)
    q = randn((100, 80, Hq, d), 41)
    for b, n in enumerate(new):
        q[b, n:] = float("nan")
    new_t = torch.tensor(new, dtype=torch.int32, device=DEV)
    out, lse = bsa.bsa_forward_paged(q.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens, new_lens=new_t,
                                     prefix_table=pool.gprefix, prefix_len=prefix)
    bsa.bsa_device_status()
    check_attention(out, lse, attend64(q, pool, new, True))
    for _ in range(20):
        again, lse2 = bsa.bsa_forward_paged(q.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens, new_lens=new_t,
                                            prefix_table=pool.gprefix, prefix_len=prefix)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    bsa.bsa_device_status()

"""The 4-bit cache's calls against the format and the formulas in 64 bits: what
is written (bytes), what is read (values), attention over it."""

import math

import pytest
import torch

import block_sparse_attention_bsa_gb300 as bsa
from paged_utils import BF, attend64, check_attention
from quant_utils import QPool, U8, held, quantise64, values64, write

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    bsa.build()


def randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF)


def ints(x):
    return None if x is None else torch.tensor(x, dtype=I32, device=DEV)


# ---- append ----

# T, new, kv (the new ones included), Hkv, d, page, layout
APPEND_CASES = [
    (1, None, [1], 1, 128, 16, "pages"),
    (1, None, [16, 17, 700, 33], 8, 128, 64, "pages"),
    (1, [1, 0, 1], [5, 9, 64], 3, 64, 16, "heads"),
    (2, None, [16, 17], 2, 128, 16, "beside"),
    (15, None, [15, 16, 31], 2, 64, 32, "pages"),
    (16, None, [16, 40], 5, 128, 128, "pages"),
    (37, [37, 0, 20, 36, -3, 99], [50, 10, 20, 90, 4, 40], 2, 128, 32, "heads"),
    (100, None, [300, 100], 1, 64, 256, "beside"),
    (130, [1, 129], [1, 257], 3, 64, 64, "pages"),
]


@pytest.mark.parametrize("T,new,kv,Hkv,d,page,layout", APPEND_CASES)
def test_append_writes_the_new_tokens_and_nothing_else(T, new, kv, Hkv, d, page, layout):
    """Every byte of both caches, those of slots that are not written included."""
    B = len(kv)
    n = [T if new is None else min(max(new[b], 0), T) for b in range(B)]
    pool = QPool([max(x, 1) for x in kv], 0, Hkv, d, page, DEV, 200, layout=layout)
    before = [pool.gk.cpu().clone(), pool.gv.cpu().clone()]
    qkv = randn((B, T, 3 * Hkv + 1, d), 201) * 3.0
    k, v = qkv[:, :, 1:1 + Hkv], qkv[:, :, 2 * Hkv:3 * Hkv]                    # views of a wider tensor
    x = qkv.to(DEV)
    assert bsa.bsa_cache_append_q4(x[:, :, 1:1 + Hkv], x[:, :, 2 * Hkv:3 * Hkv], pool.gk, pool.gv, pool.gtable, ints(kv),
                                   new_lens=ints(new)) is None
    bsa.bsa_device_status()
    for cache, rows, got, channels_first in ((before[0], k, pool.gk, False), (before[1], v, pool.gv, True)):
        for b in range(B):
            write(cache, pool.table[b], kv[b] - n[b], rows[b, :n[b]], channels_first)
        assert torch.equal(got.cpu(), cache)


@pytest.mark.parametrize("d", [64, 128])
def test_append_of_odd_numbers(d):
    """Zeros of both signs, subnormal, tiny, huge and largest numbers, exact ties of
    scales and of codes, infinities and NaN: the bytes of the format."""
    T, H = 61, 2
    x = randn((1, T, H, d), 202)
    x[0, 0] = 0.0
    x[0, 1] = -0.0
    x[0, 2] = 1e-39
    x[0, 3, :, ::3] = 2.0 ** -18
    x[0, 4] = 3.3e38
    x[0, 5] = -3.3e38
    x[0, 6, :, 5] = 7 * 114688.0
    x[0, 7, :, 9] = 8e5
    for i in range(16):                               # scales of 1 + i / 16: every other one is a tie
        x[0, 8 + i] = x[0, 8 + i].clamp(-7, 7)
        x[0, 8 + i, :, 0::32] = 7 * (1 + i / 16)
        x[0, 24 + i] = torch.arange(d).remainder(32) * 0.25 * (1 + (i // 2) / 8) * (-1) ** i      # codes of n / 4
        x[0, 24 + i, :, 0::32] = 7 * (1 + (i // 2) / 8)
    x[0, 40, 0, 3] = float("nan")
    x[0, 41, 1, 40] = float("inf")
    x[0, 42] = -float("inf")
    for i in range(43, T):
        x[0, i] *= 10.0 ** (i - 52)
    cache = [torch.zeros(4, H, 1, 17 * d // 2, dtype=U8) for _ in range(2)]
    gpu = [c.to(DEV) for c in cache]
    table = torch.tensor([[2, 0, 3, 1]], dtype=I32)
    bsa.bsa_cache_append_q4(x.to(DEV), x.flip(2).to(DEV), *gpu, table.to(DEV), ints([T]))
    bsa.bsa_device_status()
    for c, rows, got, channels_first in ((cache[0], x[0], gpu[0], False), (cache[1], x[0].flip(1), gpu[1], True)):
        codes, byte = quantise64(rows)
        write(c, table[0], 0, rows, channels_first)
        # the codes of a group that is not finite are not defined: its values are
        k, v = bsa.bsa_cache_read_q4(*gpu, table.to(DEV), ints([T]), T)
        y = (v if channels_first else k)[0].double().cpu()
        want = values64(codes, byte)
        bad = (y != want) & ~(torch.isnan(y) & torch.isnan(want))
        assert not bad.any(), (bad.nonzero()[:4].tolist(), y[bad][:4].tolist(), want[bad][:4].tolist())
        half = 16 * d // 2
        assert bool((got.cpu()[..., half:] == c[..., half:]).all())
        assert torch.isnan(want).any()
    bsa.bsa_device_status()


def test_append_in_pieces_equals_append_at_once():
    """A prompt in one call, and token by token and in uneven chunks: the same bytes."""
    H, d, page, n = 2, 128, 32, 150
    k, v = randn((1, n, H, d), 203).to(DEV), randn((1, n, H, d), 204).to(DEV)
    table = ints([[4, 1, 0, 3, 2]])
    caches = []
    for cuts in ((0, n), (0, 1, 2, 3, 20, 21, 64, 65, 100, 117, n)):
        kc, vc = (torch.full(bsa.bsa_cache_q4_shape(5, page, H, d), 77, dtype=U8, device=DEV) for _ in range(2))
        for a, z in zip(cuts, cuts[1:]):
            bsa.bsa_cache_append_q4(k[:, a:z], v[:, a:z], kc, vc, table, ints([z]))
        caches.append((kc, vc))
    bsa.bsa_device_status()
    assert all(torch.equal(x, y) for x, y in zip(*caches))


def test_append_and_read_report_tokens_without_a_page():
    H, d, page = 2, 64, 16
    kc, vc = (torch.zeros(bsa.bsa_cache_q4_shape(3, page, H, d), dtype=U8, device=DEV) for _ in range(2))
    x = randn((1, 20, H, d), 205).to(DEV)
    for table, kv in (([[0, 3]], [20]), ([[0, -1]], [20]), ([[0, 1]], [40]), ([[0, 1]], [7]), ([[1 << 30, 1]], [20])):
        bsa.bsa_device_status()
        bsa.bsa_cache_append_q4(x, x, kc, vc, ints(table), ints(kv))
        with pytest.raises(bsa.BsaError, match="BSA_ERR_INVALID_INDICES.*bsaq_cache_append"):
            bsa.bsa_device_status()
    bsa.bsa_device_status()
    assert int(kc[2].count_nonzero()) == 0
    bsa.bsa_cache_read_q4(kc, vc, ints([[0, 3]]), ints([20]), 20)
    with pytest.raises(bsa.BsaError, match="BSA_ERR_INVALID_INDICES.*bsaq_cache_read"):
        bsa.bsa_device_status()
    bsa.bsa_cache_read_q4(kc, vc, ints([[0, 3]]), ints([16]), 20)              # the entry behind is not looked at
    bsa.bsa_device_status()


# ---- read ----

# lens, first, length, Hkv, d, page, layout
READ_CASES = [
    ([1], None, 1, 1, 128, 16, "pages"),
    ([300], None, 300, 8, 128, 64, "pages"),
    ([5, 0, 77, 130], [0, 0, 30, 129], 140, 2, 64, 16, "heads"),
    ([129, 257], [17, 300], 200, 3, 128, 128, "beside"),
    ([400, 20], [-5, 19], 50, 3, 64, 256, "pages"),
    ([33, 47], [15, 16], 20, 1, 64, 32, "pages"),
]


@pytest.mark.parametrize("lens,first,length,Hkv,d,page,layout", READ_CASES)
def test_read_gives_the_held_values_and_leaves_other_rows(lens, first, length, Hkv, d, page, layout):
    B = len(lens)
    pool = QPool(lens, 0, Hkv, d, page, DEV, 210, layout=layout)
    args = (pool.gk, pool.gv, pool.gtable, pool.kv_lens, length)
    k, v = bsa.bsa_cache_read_q4(*args, first=ints(first))
    room = torch.full((B, length + 3, 2 * Hkv + 1, d), 7.0, dtype=BF, device=DEV)       # outputs inside a wider tensor
    ko, vo = room[:, 1:length + 1, :Hkv], torch.full((B, length, Hkv, d), 7.0, dtype=BF, device=DEV)
    got = bsa.bsa_cache_read_q4(*args, first=ints(first), k_out=ko, v_out=vo)
    bsa.bsa_device_status()
    assert got[0] is ko and got[1] is vo
    want_room = torch.full_like(room, 7.0).cpu()
    for b in range(B):
        f = 0 if first is None else max(first[b], 0)
        n = max(0, min(length, lens[b] - f))
        for got, other, rows in ((k, ko, pool.own_k[b]), (v, vo, pool.own_v[b])):
            assert torch.equal(got[b, :n].cpu(), rows[f:f + n]) and torch.equal(other[b, :n].cpu(), rows[f:f + n])
            assert (got[b, n:] == 0).all() and (other[b, n:] == 7).all()
        want_room[b, 1:1 + n, :Hkv] = pool.own_k[b][f:f + n]
    assert torch.equal(room.cpu(), want_room)


# ---- attention ----

# lens, T, new, prefix, Hq, Hkv, d, page, causal, layout
ATTEND_CASES = [
    ([1], 1, None, 0, 1, 1, 64, 16, True, "pages"),
    ([700], 1, None, 0, 8, 2, 128, 64, True, "pages"),
    ([5, 0, 333], 1, None, 0, 4, 4, 64, 16, True, "heads"),
    ([0, 0], 1, None, 0, 8, 2, 128, 64, True, "pages"),
    ([130, 1, 128, 129], 1, None, 200, 8, 2, 128, 32, True, "beside"),
    ([300, 40], 5, None, 131, 6, 2, 64, 16, True, "pages"),
    ([300, 40, 3], 5, [5, 0, 2], 0, 24, 8, 128, 128, True, "pages"),
    ([40, 2], 7, [3, 7], 0, 3, 1, 64, 32, True, "heads"),
    ([140, 40], 5, None, 129, 8, 1, 128, 256, False, "pages"),
    ([260, 100], 90, [90, 33], 64, 8, 2, 64, 64, True, "pages"),
    ([200], 40, None, 1000, 16, 2, 128, 16, True, "pages"),
    ([90, 30], 70, None, 0, 3, 3, 128, 16, False, "beside"),
    ([1000, 3, 500, 90, 17] * 8, 1, None, 300, 32, 8, 128, 64, True, "pages"),
    ([20, 90] * 40, 1, None, 40, 16, 2, 64, 16, True, "pages"),
    ([70], 1, None, 0, 40, 1, 128, 64, True, "pages"),
    ([256, 384], 3, None, 256, 20, 1, 128, 128, True, "pages"),
]


def run_case(lens, T, new, prefix, Hq, Hkv, d, page, causal, layout, seed=220, **kw):
    pool = QPool(lens, prefix, Hkv, d, page, DEV, seed, layout=layout)
    q = randn((len(lens), T, Hq, d), seed + 1)
    out, lse = bsa.bsa_forward_paged_q4(q.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens, new_lens=ints(new),
                                        prefix_table=pool.gprefix, prefix_len=prefix, causal=causal, **kw)
    bsa.bsa_device_status()
    return pool, q, out, lse


@pytest.mark.parametrize("lens,T,new,prefix,Hq,Hkv,d,page,causal,layout", ATTEND_CASES)
def test_attention_matches_64_bits(lens, T, new, prefix, Hq, Hkv, d, page, causal, layout):
    pool, q, out, lse = run_case(lens, T, new, prefix, Hq, Hkv, d, page, causal, layout)
    check_attention(out, lse, attend64(q, pool, new, causal))


@pytest.mark.parametrize("scale", [0.5, 4.0, 1e-4])
def test_attention_of_a_given_scale(scale):
    pool, q, out, lse = run_case([300, 77], 2, None, 140, 8, 2, 64, 32, True, "pages", softmax_scale=scale)
    check_attention(out, lse, attend64(q, pool, scale=scale))


def test_attention_strided_queries_and_no_lse():
    pool = QPool([90, 200], 0, 2, 128, 32, DEV, 230)
    wide = randn((2, 3, 13, 128), 231)
    q = wide[:, 1:3, 2:10]
    out, lse = bsa.bsa_forward_paged_q4(wide.to(DEV)[:, 1:3, 2:10], pool.gk, pool.gv, pool.gtable, pool.kv_lens)
    bare, none = bsa.bsa_forward_paged_q4(q.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens, return_lse=False)
    assert none is None and torch.equal(out, bare)
    check_attention(out, lse, attend64(q, pool))


def test_attention_over_the_prefix_alone():
    pool = QPool([1, 1, 1], 333, 2, 64, 64, DEV, 232)
    q = randn((3, 2, 8, 64), 233)
    empty = torch.empty(3, 0, dtype=I32, device=DEV)
    out, lse = bsa.bsa_forward_paged_q4(q.to(DEV), pool.gk, pool.gv, empty, pool.kv_lens, prefix_table=pool.gprefix,
                                        prefix_len=333)
    bsa.bsa_device_status()
    pool.lens, pool.own_k, pool.own_v = [0] * 3, [pool.own_k[0][:0]] * 3, [pool.own_v[0][:0]] * 3
    check_attention(out, lse, attend64(q, pool))


def test_attention_reports_tables_that_name_no_page():
    pool = QPool([40], 20, 2, 64, 16, DEV, 234)
    x = randn((1, 1, 4, 64), 235).to(DEV)
    for at, page in ((1, -1), (0, pool.total), (2, 1 << 30)):
        table = pool.gtable.clone()
        table[0, at] = page
        bsa.bsa_device_status()
        bsa.bsa_forward_paged_q4(x, pool.gk, pool.gv, table, pool.kv_lens)
        with pytest.raises(bsa.BsaError, match="BSA_ERR_INVALID_INDICES.*bsaq_forward"):
            bsa.bsa_device_status()
    shared = pool.gprefix.clone()
    shared[1] = -7
    bsa.bsa_forward_paged_q4(x, pool.gk, pool.gv, pool.gtable, pool.kv_lens, prefix_table=shared, prefix_len=20)
    with pytest.raises(bsa.BsaError, match="BSA_ERR_INVALID_INDICES.*bsaq_forward"):
        bsa.bsa_device_status()
    for kv in (-1, 49):
        bsa.bsa_forward_paged_q4(x, pool.gk, pool.gv, pool.gtable, ints([kv]))
        with pytest.raises(bsa.BsaError, match="BSA_ERR_INVALID_INDICES.*bsaq_forward"):
            bsa.bsa_device_status()
    bsa.bsa_device_status()


# lens, T, new, prefix, Hq, Hkv, d, page, causal
WAYS = {
    "few rows": ([100, 77], 1, None, 0, 8, 2, 128, 64, True),
    "one row": ([300], 1, None, 0, 3, 3, 64, 32, True),
    "many tiles": ([3000], 1, None, 0, 16, 1, 128, 64, True),
    "prefix": ([5, 300] * 30, 1, None, 300, 16, 2, 64, 16, True),
    "chunks": ([40, 130] * 20, 40, [40, 3] * 20, 200, 8, 2, 128, 32, True),
    "not causal": ([140, 40], 5, None, 129, 8, 1, 128, 256, False),
}


@pytest.mark.parametrize("kind", ["nan", "inf", "3e38"])
@pytest.mark.parametrize("way", WAYS)
def test_rows_of_numbers_that_are_not_finite_come_out_as_nan(way, kind):
    """As in the attention over bf16 pages: a row whose scores hold a NaN or a +inf,
    or are all -inf, is NaN, and no other row feels it.  A channel of 3e38 makes
    those products infinite that pass fp32's largest number."""
    lens, T, new, prefix, Hq, Hkv, d, page, causal = WAYS[way]
    B = len(lens)
    pool = QPool(lens, prefix, Hkv, d, page, DEV, 240)
    q = randn((B, T, Hq, d), 241)

    def attend(x):
        out, lse = bsa.bsa_forward_paged_q4(x.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens, new_lens=ints(new),
                                            prefix_table=pool.gprefix, prefix_len=prefix, causal=causal)
        bsa.bsa_device_status()
        return out.cpu(), lse.cpu()

    want, want_lse = attend(q)
    g = torch.Generator().manual_seed(242)
    hit = torch.zeros(B, T, Hq, dtype=torch.bool)
    bad = q.clone()
    for b in range(0, B, 1 if B < 5 else 7):
        n = T if new is None else new[b]
        i, h = int(torch.randint(0, n, (1,), generator=g)), int(torch.randint(0, Hq, (1,), generator=g))
        c = int(torch.randint(0, d, (1,), generator=g))
        bad[b, i, h] = 0
        bad[b, i, h, c] = float(kind)
        keys = torch.cat([pool.pre_k, pool.own_k[b]])[:, h // (Hq // Hkv), c].float()
        if causal:
            keys = keys[:prefix + lens[b] - n + i + 1]
        z = keys * float(torch.tensor(float(kind)).to(BF))     # one product: the others are with 0
        if torch.isnan(torch.softmax(z.float(), 0)).any():
            hit[b, i, h] = True
        else:
            bad[b, i, h] = q[b, i, h]                    # no product of this row passes fp32's range
    assert hit.any()
    out, lse = attend(bad)
    assert torch.isnan(out[hit]).all()
    assert not torch.isfinite(lse.transpose(1, 2)[hit]).any()
    if kind == "nan":
        assert torch.isnan(lse.transpose(1, 2)[hit]).all()
    assert torch.equal(out[~hit], want[~hit])
    assert torch.equal(lse.transpose(1, 2)[~hit], want_lse.transpose(1, 2)[~hit])
    assert torch.isfinite(want).all()


def test_rows_without_a_key_stay_empty_whatever_their_q_holds():
    for lens in ([2, 40], [2]):
        pool = QPool(lens, 0, 2, 64, 16, DEV, 243)
        q = randn((len(lens), 5, 4, 64), 244)
        args = (pool.gk, pool.gv, pool.gtable, pool.kv_lens)
        want, want_lse = (x.cpu() for x in bsa.bsa_forward_paged_q4(q.to(DEV), *args))
        q[0, 0], q[0, 1], q[0, 2] = float("nan"), float("inf"), 3e38
        out, lse = (x.cpu() for x in bsa.bsa_forward_paged_q4(q.to(DEV), *args))
        bsa.bsa_device_status()
        assert (out[0, :3] == 0).all() and torch.isneginf(lse[0, :, :3]).all()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_scores_far_apart_and_growing_along_the_keys():
    """Scores that rise by hundreds from tile to tile, and fall: the running maximum
    moves in every tile, or lies in the first one."""
    n, d = 900, 64
    for sign in (1.0, -1.0):
        k = torch.zeros(n, 1, d)
        k[:, 0, 0] = sign * torch.arange(n) * 0.5
        k[:, 0, 32] = torch.randn(n, generator=torch.Generator().manual_seed(246))
        k = held(k.to(BF))
        v = held(randn((n, 1, d), 247))
        pool = QPool([n], 0, 1, d, 64, DEV, 245)
        write(pool.k, pool.table[0], 0, k, False)        # what is held is held again as it is
        write(pool.v, pool.table[0], 0, v, True)
        pool.own_k, pool.own_v = [held(k)], [held(v)]
        q = torch.zeros(1, 1, 4, d, dtype=BF)
        q[..., 0] = torch.tensor([8.0, 16.0, 30.0, 0.0])
        q[..., 32] = 1.0
        out, lse = bsa.bsa_forward_paged_q4(q.to(DEV), pool.k.to(DEV), pool.v.to(DEV), pool.gtable, pool.kv_lens)
        bsa.bsa_device_status()
        check_attention(out, lse, attend64(q, pool))
        assert math.isfinite(float(lse.sum()))

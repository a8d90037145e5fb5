"""The 4-bit cache's calls as they are used together: a prompt, a chunk and single
tokens over one cache with rotated keys, read back for the calls that take rows,
captured steps, streams, batches that split over several kernels, caches past 32
bits."""

import math

import pytest
import torch

import block_sparse_attention_bsa_gb300 as bsa
from paged_utils import BF, attend64, check_attention
from quant_utils import QPool, U8, held, write

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    bsa.build()


def randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF)


def ints(x):
    return torch.tensor(x, dtype=I32, device=DEV)


class Serving:
    """Three requests behind one prompt of 150 tokens: the rotated tokens of each (Q,
    K, V), and a 4-bit cache with pages for all of them, every byte poisoned."""

    B, P, Hq, Hkv, d, page = 3, 150, 8, 2, 64, 32
    total = 90                                   # own tokens of each request in the end

    def __init__(self):
        n = self.P + self.B * self.total
        qkv = randn((n, self.Hq + 2 * self.Hkv, self.d), 300).to(DEV)
        pos = torch.randint(0, 700, (n, 3), generator=torch.Generator().manual_seed(301), dtype=I32).to(DEV)
        inv, axes = bsa.bsa_axis_frequencies((8, 12, 12), device=DEV)
        q, k = bsa.bsa_rope_axes(qkv[None, :, :self.Hq], qkv[None, :, self.Hq:self.Hq + self.Hkv], pos, pos, inv, axes)
        self.q, self.k, self.v = q[0], k[0], qkv[:, self.Hq + self.Hkv:]
        per, shared = -(-self.total // self.page), -(-self.P // self.page)
        pages = self.B * per + shared + 1
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(302)).int().to(DEV)
        self.kc, self.vc = (torch.full(bsa.bsa_cache_q4_shape(pages, self.page, self.Hkv, self.d), 255, dtype=U8, device=DEV)
                            for _ in range(2))
        self.prefix_table = order[:shared]
        wide = torch.full((self.B, per + 5), 1 << 30, dtype=I32, device=DEV)
        wide[:, :per] = order[shared:shared + self.B * per].view(self.B, per)
        self.table = wide[:, :per]               # rows of a wider table

    def rows(self, first, T):
        """q, k, v [B, T, H, d] of own tokens first .. first + T of every request."""
        at = self.P + torch.arange(self.B, device=DEV)[:, None] * self.total + first + torch.arange(T, device=DEV)
        return self.q[at], self.k[at], self.v[at]

    def store_prompt(self):
        bsa.bsa_cache_append_q4(self.k[None, :self.P], self.v[None, :self.P], self.kc, self.vc, self.prefix_table[None],
                                ints([self.P]))

    def reference(self):
        pool = QPool.__new__(QPool)
        k, v = held(self.k.cpu()), held(self.v.cpu())
        pool.prefix_len, pool.pre_k, pool.pre_v = self.P, k[:self.P], v[:self.P]
        own = [slice(self.P + b * self.total, self.P + (b + 1) * self.total) for b in range(self.B)]
        return pool, [k[o] for o in own], [v[o] for o in own]


def test_prompt_chunk_and_single_tokens_over_one_cache():
    s = Serving()
    s.store_prompt()
    pool, k_all, v_all = s.reference()
    at = 0
    for T in (33, 1, 1, 5, 1):
        q, k, v = s.rows(at, T)
        at += T
        lens = ints([at] * s.B)
        bsa.bsa_cache_append_q4(k, v, s.kc, s.vc, s.table, lens)
        out, lse = bsa.bsa_forward_paged_q4(q, s.kc, s.vc, s.table, lens, prefix_table=s.prefix_table, prefix_len=s.P)
        pool.lens = [at] * s.B
        pool.own_k, pool.own_v = [x[:at] for x in k_all], [x[:at] for x in v_all]
        check_attention(out, lse, attend64(q.cpu(), pool))
    kr, vr = bsa.bsa_cache_read_q4(s.kc, s.vc, s.table, lens, at)
    assert all(torch.equal(kr[b].cpu(), k_all[b][:at]) and torch.equal(vr[b].cpu(), v_all[b][:at]) for b in range(s.B))
    bsa.bsa_device_status()


def test_rows_read_back_go_through_the_other_calls():
    """A prompt in pages, read back to rows: the causal pass over them agrees with the
    attention over the pages, and the selector and the forward take them as the
    protected prefix of a generation stream."""
    s = Serving()
    s.store_prompt()
    k, v = bsa.bsa_cache_read_q4(s.kc, s.vc, s.prefix_table[None], ints([s.P]), s.P)
    pool, _, _ = s.reference()
    assert torch.equal(k[0].cpu(), pool.pre_k) and torch.equal(v[0].cpu(), pool.pre_v)
    q = s.q[None, :s.P]
    dense, dense_lse = bsa.bsa_forward_causal(q.contiguous(), k, v, 128, 128)
    out, lse = bsa.bsa_forward_paged_q4(q, s.kc, s.vc, s.prefix_table[None], ints([s.P]))
    pool.prefix_len, pool.lens, pool.own_k, pool.own_v = 0, [s.P], [pool.pre_k], [pool.pre_v]
    pool.pre_k, pool.pre_v = pool.pre_k[:0], pool.pre_v[:0]
    ref = attend64(q.cpu(), pool)
    check_attention(out, lse, ref)
    check_attention(dense, dense_lse, ref)
    # generation tokens behind the prefix that was read into the front of their K and V
    n = 200
    gen_q, gen = randn((1, n, s.Hq, s.d), 310).to(DEV), randn((1, n, 2 * s.Hkv, s.d), 311).to(DEV)
    room = torch.empty(2, 1, s.P + n, s.Hkv, s.d, dtype=BF, device=DEV)
    room[0, :, s.P:], room[1, :, s.P:] = gen[:, :, :s.Hkv], gen[:, :, s.Hkv:]
    bsa.bsa_cache_read_q4(s.kc, s.vc, s.prefix_table[None], ints([s.P]), s.P, k_out=room[0, :, :s.P], v_out=room[1, :, :s.P])
    idx, cnt = bsa.bsa_select(gen_q, room[0], s.P, [n], 128, 128, 1.0)
    o1, l1 = bsa.bsa_forward(gen_q, room[0], room[1], idx, cnt, s.P, [n], 128, 128)
    whole = torch.cat([k, gen[:, :, :s.Hkv]], 1), torch.cat([v, gen[:, :, s.Hkv:]], 1)
    o2, l2 = bsa.bsa_forward(gen_q, *whole, None, None, s.P, [n], 128, 128)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    bsa.bsa_device_status()


def test_captured_steps_follow_lengths_and_tables():
    """One captured step (lengths + 1, append, attention) replayed for many tokens gives
    the bits of the eager calls; its workspace is shared with a second captured step."""
    s, eager = Serving(), Serving()
    s.store_prompt()
    eager.store_prompt()
    stream = torch.cuda.Stream()
    B = s.B
    lens = torch.zeros(B, dtype=I32, device=DEV)
    q, k, v = (torch.empty_like(x) for x in eager.rows(0, 1))
    outs = [torch.empty(B, 1, s.Hq, s.d, dtype=BF, device=DEV) for _ in range(2)]
    lses = [torch.empty(B, s.Hq, 1, device=DEV) for _ in range(2)]
    need = bsa.bsa_forward_paged_q4_workspace_size(B, 1, s.Hq, s.Hkv, s.d, True)
    ws = torch.empty(need, dtype=U8, device=DEV)

    def step():
        lens.add_(1)
        bsa.bsa_cache_append_q4(k, v, s.kc, s.vc, s.table, lens)
        bsa.bsa_forward_paged_q4(q, s.kc, s.vc, s.table, lens, prefix_table=s.prefix_table, prefix_len=s.P, out=outs[0],
                                 lse=lses[0], workspace=ws)

    def again():
        bsa.bsa_forward_paged_q4(q, s.kc, s.vc, s.table, lens, prefix_table=s.prefix_table, prefix_len=s.P - 7, out=outs[1],
                                 lse=lses[1], workspace=ws)

    for a, b in zip((q, k, v), eager.rows(0, 1)):
        a.copy_(b)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step()                                    # sets the kernels' attributes once
        again()
        stream.synchronize()
        lens.zero_()
        graphs = []
        for f in (step, again):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                f()
            graphs.append(g)
        for i in range(70):
            x = eager.rows(i, 1)
            for a, b in zip((q, k, v), x):
                a.copy_(b)
            graphs[0].replay()
            graphs[1].replay()
            n = torch.full((B,), i + 1, dtype=I32, device=DEV)
            bsa.bsa_cache_append_q4(x[1], x[2], eager.kc, eager.vc, eager.table, n)
            for j, P in enumerate((s.P, s.P - 7)):
                out, lse = bsa.bsa_forward_paged_q4(x[0], eager.kc, eager.vc, eager.table, n, prefix_table=eager.prefix_table,
                                                    prefix_len=P)
                assert torch.equal(out, outs[j]) and torch.equal(lse, lses[j]), (i, j)
    stream.synchronize()
    assert torch.equal(s.kc, eager.kc) and torch.equal(s.vc, eager.vc)
    bsa.bsa_device_status()


# B, T, prefix, low, high, Hq, Hkv, d, page: one kernel, the other, and both of them
SPLITS = [
    (5, 1, 0, 1, 900, 8, 2, 128, 64),
    (3, 2, 40, 3, 500, 8, 2, 128, 16),
    (2, 3, 130, 3, 300, 10, 2, 64, 32),
    (2, 4, 0, 300, 400, 16, 4, 128, 32),
    (3, 6, 0, 7, 300, 16, 4, 64, 64),
    (9, 1, 700, 1, 300, 32, 8, 128, 64),
    (40, 1, 1500, 0, 100, 32, 4, 64, 128),
    (20, 2, 257, 0, 40, 16, 2, 128, 16),
    (2, 150, 300, 150, 400, 6, 2, 128, 64),
    (70, 1, 64, 1, 2, 3, 3, 64, 16),
]


@pytest.mark.parametrize("B,T,prefix,low,high,Hq,Hkv,d,page", SPLITS)
def test_every_way_of_splitting_a_batch(B, T, prefix, low, high, Hq, Hkv, d, page):
    g = torch.Generator().manual_seed(320)
    lens = torch.randint(low, high + 1, (B,), generator=g).tolist()
    pool = QPool(lens, prefix, Hkv, d, page, DEV, 321)
    q = randn((B, T, Hq, d), 322)
    new = torch.randint(0, T + 1, (B,), generator=g).tolist()
    for n, causal in ((None, True), (new, True), (new, False)):
        out, lse = bsa.bsa_forward_paged_q4(q.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens,
                                            new_lens=None if n is None else ints(n), prefix_table=pool.gprefix,
                                            prefix_len=prefix, causal=causal)
        bsa.bsa_device_status()
        check_attention(out, lse, attend64(q, pool, n, causal))
        more, more_lse = bsa.bsa_forward_paged_q4(q.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens,
                                                  new_lens=None if n is None else ints(n), prefix_table=pool.gprefix,
                                                  prefix_len=prefix, causal=causal)
        assert torch.equal(out, more) and torch.equal(lse, more_lse)


def test_calls_on_two_streams_at_once():
    """Calls that overlap, each with its own workspace and outputs, give the bits of
    calls that do not: narrow, wide and both beside one another."""
    pool = QPool([900, 33, 2000], 700, 2, 128, 64, DEV, 330)
    args = (pool.gk, pool.gv, pool.gtable, pool.kv_lens)
    calls = [(randn((3, T, 8, 128), 331 + T).to(DEV), P) for T, P in ((1, 0), (4, 700), (40, 700), (2, 700))]

    def run(q, P, **kw):
        return bsa.bsa_forward_paged_q4(q, *args, prefix_table=pool.gprefix, prefix_len=P, **kw)

    want = [run(*c) for c in calls]
    rows = bsa.bsa_cache_read_q4(*args, 2000)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got, reads = [], []
    for i in range(12):
        for j, st in enumerate(streams):
            c = (i + j) % len(calls)
            got.append((c, run(*calls[c], stream=st)))
            reads.append(bsa.bsa_cache_read_q4(*args, 2000, stream=st.cuda_stream))
    torch.cuda.synchronize()
    for c, (out, lse) in got:
        assert torch.equal(out, want[c][0]) and torch.equal(lse, want[c][1]), c
    for k, v in reads:
        assert torch.equal(k, rows[0]) and torch.equal(v, rows[1])
    bsa.bsa_device_status()


def test_a_workspace_of_any_content_and_calls_behind_one_another():
    """Every byte that counts is written by the call: NaN in the workspace, and calls of
    other shapes on it, change nothing."""
    pool = QPool([300, 40, 0, 129], 260, 2, 64, 32, DEV, 340)
    args = (pool.gk, pool.gv, pool.gtable, pool.kv_lens)
    shapes = [(1, 0), (1, 260), (3, 260), (20, 260), (5, 0), (30, 0)]
    ws = torch.full((64 << 20,), 255, dtype=U8, device=DEV)
    for T, P in shapes * 2:
        q = randn((4, T, 8, 64), 341 + T)
        out, lse = bsa.bsa_forward_paged_q4(q.to(DEV), *args, prefix_table=pool.gprefix, prefix_len=P, workspace=ws)
        bsa.bsa_device_status()
        mine = QPool.__new__(QPool)
        mine.__dict__.update(pool.__dict__)
        mine.prefix_len, mine.pre_k, mine.pre_v = P, pool.pre_k[:P], pool.pre_v[:P]
        check_attention(out, lse, attend64(q, mine))


def test_cache_past_32_bits():
    """A cache of more than 2^32 bytes with a request in its last pages, checked at its ends."""
    page, Hkv, d = 128, 8, 128
    unit = page // 16 * Hkv * 17 * d // 2
    total = (1 << 32) // unit + 40
    kc = torch.zeros(bsa.bsa_cache_q4_shape(total, page, Hkv, d), dtype=U8, device=DEV)
    vc = torch.zeros_like(kc)
    n = 700
    k, v = randn((1, n, Hkv, d), 350), randn((1, n, Hkv, d), 351)
    table = torch.arange(total - 6, total, dtype=I32, device=DEV).flip(0)[None]
    lens = ints([n])
    bsa.bsa_cache_append_q4(k.to(DEV), v.to(DEV), kc, vc, table, lens)
    assert not bool(kc[:total - 6].any()) and not bool(vc[:total - 6].any())
    kr, vr = bsa.bsa_cache_read_q4(kc, vc, table, lens, n)
    hk, hv = held(k[0]), held(v[0])
    assert torch.equal(kr[0].cpu(), hk) and torch.equal(vr[0].cpu(), hv)
    pool = QPool.__new__(QPool)
    pool.prefix_len, pool.pre_k, pool.pre_v = 0, hk[:0], hv[:0]
    pool.lens, pool.own_k, pool.own_v = [n], [hk], [hv]
    for T in (1, 30):
        q = randn((1, T, 16, d), 352 + T)
        out, lse = bsa.bsa_forward_paged_q4(q.to(DEV), kc, vc, table, lens)
        check_attention(out, lse, attend64(q, pool))
    bsa.bsa_device_status()


def test_calls_right_behind_what_writes_their_inputs():
    """Lengths, tables and rows written by the kernel just before a call, eager and
    captured, give the bits of calls with a synchronisation after every operation."""
    B, Hq, Hkv, d, page, steps, P = 12, 8, 2, 128, 64, 30, 300
    g = torch.Generator(device=DEV).manual_seed(360)
    shape = bsa.bsa_cache_q4_shape(150, page, Hkv, d)
    start_k, start_v = (torch.randint(0, 120, shape, generator=g, device=DEV, dtype=I32).to(U8) for _ in range(2))
    tables = [torch.randperm(144, generator=g, device=DEV)[:96].int().view(B, 8) for _ in range(3)]
    prefix = torch.arange(144, 149, device=DEV, dtype=I32)
    rows = torch.randn(B, 1, Hq + 2 * Hkv, d, generator=g, device=DEV).to(BF)
    table, lens = tables[0].clone(), torch.zeros(B, dtype=I32, device=DEV)
    x, kc, vc = rows.clone(), start_k.clone(), start_v.clone()

    def start():
        lens.fill_(100), x.copy_(rows), kc.copy_(start_k), vc.copy_(start_v)

    def step(i, between=lambda: None):
        x.mul_(1.0625 if i % 2 else 0.9375)
        between()
        table.copy_(tables[i % 3])
        lens.add_(1)
        between()
        bsa.bsa_cache_append_q4(x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], kc, vc, table, lens)
        between()
        out, lse = bsa.bsa_forward_paged_q4(x[:, :, :Hq], kc, vc, table, lens, prefix_table=prefix, prefix_len=P)
        between()
        x[:, :, :Hq].add_(out.clamp(-1, 1))
        k, v = bsa.bsa_cache_read_q4(kc, vc, table, lens, 8, first=lens - 4)
        between()
        return out, lse, k, v

    def same(a, b):
        return all(torch.equal(s, t) for p, q in zip(a, b) for s, t in zip(p, q))

    start()
    want = [step(i, torch.cuda.synchronize) for i in range(steps)]
    assert all(bool(torch.isfinite(w[0]).all()) for w in want)
    run = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(run):
        for _ in range(4):
            start()
            got = [step(i) for i in range(steps)]
            run.synchronize()
            assert same(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=run):
            start()
            got = [step(i) for i in range(steps)]
        for _ in range(4):
            graph.replay()
            run.synchronize()
            assert same(got, want)
    bsa.bsa_device_status()


def test_results_do_not_depend_on_memory_order_or_padding():
    """The same keys in pages of another size and order, in tables of another width,
    with K and V of a page beside each other: the values of the formula; and rows from
    new_lens on leave no trace."""
    lens, T, Hq, Hkv, d = [200, 77], 3, 8, 2, 128
    q = randn((2, T, Hq, d), 370)
    ref = None
    for page, layout, width in ((16, "pages", None), (64, "heads", 9), (256, "beside", 3)):
        pool = QPool(lens, 0, Hkv, d, page, DEV, 371, max_pages=width, layout=layout)
        if ref is None:
            k, v, ref = pool.own_k, pool.own_v, attend64(q, pool, [3, 1])
        for b in range(2):
            write(pool.k, pool.table[b], 0, k[b], False)
            write(pool.v, pool.table[b], 0, v[b], True)
        if layout == "beside":
            both = torch.stack([pool.k, pool.v], 1).to(DEV)
            gk, gv = both[:, 0], both[:, 1]
        else:
            gk, gv = pool.k.to(DEV), pool.v.to(DEV)
        x = q.clone()
        x[1, 1:] = float("nan")                        # padding
        out, lse = bsa.bsa_forward_paged_q4(x.to(DEV), gk, gv, pool.gtable, pool.kv_lens, new_lens=ints([3, 1]))
        bsa.bsa_device_status()
        check_attention(out, lse, ref)
    assert math.isfinite(float(out.float().sum()))


def test_binding_refusals_on_the_gpu():
    pool = QPool([40, 20], 30, 2, 64, 16, DEV, 380)
    q, k = randn((2, 1, 4, 64), 381).to(DEV), randn((2, 1, 2, 64), 382).to(DEV)
    args = (pool.gk, pool.gv, pool.gtable, pool.kv_lens)
    bad = [
        (lambda: bsa.bsa_forward_paged_q4(q.float(), *args), "q must be torch.bfloat16"),
        (lambda: bsa.bsa_forward_paged_q4(q, pool.gk.cpu(), *args[1:]), "k_cache is on cpu"),
        (lambda: bsa.bsa_forward_paged_q4(q, pool.gk.view(torch.int8), *args[1:]), "k_cache must be torch.uint8"),
        (lambda: bsa.bsa_forward_paged_q4(q, pool.gk[..., :540], *args[1:]), "17 d / 2"),
        (lambda: bsa.bsa_forward_paged_q4(q, pool.gk, pool.gv[:, :1], *args[2:]), "v_cache shape"),
        (lambda: bsa.bsa_forward_paged_q4(q, *args[:3], pool.kv_lens.long()), "kv_lens must be torch.int32"),
        (lambda: bsa.bsa_forward_paged_q4(q, *args[:2], pool.gtable[:1], pool.kv_lens), "page_table must be"),
        (lambda: bsa.bsa_forward_paged_q4(q, *args, prefix_len=30), "prefix_table is None"),
        (lambda: bsa.bsa_forward_paged_q4(q, *args, prefix_len=49, prefix_table=pool.gprefix[:3]), "prefix_len is 49"),
        (lambda: bsa.bsa_forward_paged_q4(q, *args, out=q), "overlaps"),
        (lambda: bsa.bsa_forward_paged_q4(q, *args, workspace=torch.empty(64, device=DEV)), "workspace"),
        (lambda: bsa.bsa_cache_append_q4(k, k[:, :, :1], *args), "v shape differs"),
        (lambda: bsa.bsa_cache_append_q4(k, k, pool.gk, pool.gk, *args[2:]), "shares memory"),
        (lambda: bsa.bsa_cache_append_q4(k, k, *args[:3], pool.kv_lens[:1]), "kv_lens must be contiguous"),
        (lambda: bsa.bsa_cache_read_q4(*args, 0), "length 0"),
        (lambda: bsa.bsa_cache_read_q4(*args, 5, k_out=k), "k_out must have shape"),
        (lambda: bsa.bsa_cache_read_q4(*args, 1, k_out=k, v_out=k), "shares memory"),
        (lambda: bsa.bsa_cache_read_q4(*args, 1, first=pool.kv_lens[:1]), "first must be contiguous"),
    ]
    for call, needle in bad:
        with pytest.raises((ValueError, bsa.BsaError), match=needle):
            call()
    with pytest.raises(bsa.BsaError, match="BSA_ERR_WORKSPACE"):
        bsa.bsa_forward_paged_q4(q, *args, workspace=torch.empty(256, dtype=U8, device=DEV))
    with pytest.raises(bsa.BsaError, match="not a multiple of Hkv"):
        bsa.bsa_forward_paged_q4(q[:, :, :3], *args)
    bsa.bsa_device_status()
    assert math.isfinite(float(bsa.bsa_forward_paged_q4(q, *args)[0].float().sum()))


@pytest.mark.parametrize("B,T,prefix,Hq,Hkv,d", [(200, 2, 0, 4, 2, 64), (1100, 1, 0, 4, 1, 128), (1100, 1, 300, 4, 1, 64),
                                                 (170, 3, 150, 8, 2, 128)])
def test_more_requests_than_one_pass_over_the_lengths_takes(B, T, prefix, Hq, Hkv, d):
    """Batches whose lengths five warps, or one warp's 32 sums of 32, do not take at
    once: runs of requests without a key, and the last one with the most."""
    g = torch.Generator().manual_seed(330)
    lens = torch.randint(0, 40, (B,), generator=g)
    lens[40:110] = 0
    lens[-1] = 500
    pool = QPool(lens.tolist(), prefix, Hkv, d, 16, DEV, 331)
    q = randn((B, T, Hq, d), 332)
    out, lse = bsa.bsa_forward_paged_q4(q.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens, prefix_table=pool.gprefix,
                                        prefix_len=prefix)
    bsa.bsa_device_status()
    check_attention(out, lse, attend64(q, pool))


def test_a_prefix_alone_needs_no_table_and_no_lengths():
    """max_pages 0 with null pointers for the table and the lengths: few rows, many rows
    in either kernel or beside one another, and chunks."""
    from block_sparse_attention_bsa_gb300._lib import load
    from block_sparse_attention_bsa_gb300.paged import _tensor
    from block_sparse_attention_bsa_gb300.quant import _caches
    lib = load()
    pool = QPool([1, 1], 333, 2, 64, 64, DEV, 340)
    for B, T in ((1, 1), (70, 1), (200, 1), (2, 40)):
        x = randn((B, T, 8, 64), 341)
        q = x.to(DEV)
        out, lse = torch.empty_like(q), torch.empty(B, 8, T, device=DEV)
        n = bsa.bsa_forward_paged_q4_workspace_size(B, T, 8, 2, 64, True)
        ws = torch.empty(n, dtype=U8, device=DEV)
        kc, vc, _ = _caches(pool.gk, pool.gv, 0)
        assert lib.bsaq_forward(_tensor(q, "q", 0), kc, vc, None, 0, 0, None, None, pool.gprefix.data_ptr(), 333, 1, 0.0,
                                out.data_ptr(), lse.data_ptr(), ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == 0
        bsa.bsa_device_status()
        ref = QPool.__new__(QPool)
        ref.prefix_len, ref.pre_k, ref.pre_v, ref.lens = 333, pool.pre_k, pool.pre_v, [0] * B
        ref.own_k, ref.own_v = [pool.pre_k[:0]] * B, [pool.pre_v[:0]] * B
        check_attention(out, lse, attend64(x, ref))


# B, T, new, prefix, Hq, Hkv, d, page, causal: prefixes whose tiles, of segments of few
# rows, are more than the GPU's 608 blocks, beside own keys of few rows
BESIDE = {
    "4 rows": (160, 1, False, 700, 8, 2, 128, 64, True),
    "4 rows, 120 in all": (30, 1, False, 2000, 8, 2, 128, 16, True),
    "8 rows": (64, 2, True, 613, 8, 2, 64, 32, True),
    "12 rows": (80, 3, True, 700, 8, 2, 128, 128, False),
    "10 rows of 64": (70, 5, True, 1300, 4, 2, 64, 16, True),
}


def beside(name, seed):
    B, T, ragged, prefix, Hq, Hkv, d, page, causal = BESIDE[name]
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, 300, (B,), generator=g)
    lens[3:7] = 0
    new = torch.minimum(torch.randint(0, T + 1, (B,), generator=g), lens).tolist() if ragged else None
    pool = QPool(lens.tolist(), prefix, Hkv, d, page, DEV, seed + 1)
    q, counts = randn((B, T, Hq, d), seed + 2), ints(new) if ragged else None

    def attend(x, **kw):
        return bsa.bsa_forward_paged_q4(x, pool.gk, pool.gv, pool.gtable, pool.kv_lens, new_lens=counts,
                                        prefix_table=pool.gprefix, prefix_len=prefix, causal=causal, **kw)

    return pool, q, new, causal, attend


@pytest.mark.parametrize("name", BESIDE)
def test_a_long_prefix_beside_own_keys_of_few_rows(name):
    pool, q, new, causal, attend = beside(name, 350)
    out, lse = attend(q.to(DEV))
    bsa.bsa_device_status()
    check_attention(out, lse, attend64(q, pool, new, causal))
    # a row that is not finite is felt by no other
    i = next(b for b in range(len(pool.lens) - 1, 0, -1) if pool.lens[b] > 0 and (new is None or new[b] > 0))
    bad = q.clone()
    bad[i, 0, 1, 5] = float("nan")
    out2, lse2 = attend(bad.to(DEV))
    bsa.bsa_device_status()
    assert torch.isnan(out2[i, 0, 1]).all() and torch.isnan(lse2[i, 1, 0])
    out2[i, 0, 1], lse2[i, 1, 0] = out[i, 0, 1], lse[i, 1, 0]
    assert torch.equal(out2, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("name", ["4 rows", "8 rows"])
def test_long_prefixes_captured_on_two_streams_and_behind_one_another(name):
    """Kernels that start before the ones in front of them have left: twenty calls in a
    row with one workspace, in two graphs on two streams at once, and eager ones beside
    them, each with inputs that are written right before; the same bits every time."""
    pool, q, _, _, attend = beside(name, 360)
    xs = [q.to(DEV), q.flip(0).contiguous().to(DEV)]
    want = [attend(x) for x in xs]
    B, T, Hq, d = q.shape
    n = bsa.bsa_forward_paged_q4_workspace_size(B, T, Hq, pool.gk.shape[1], d, True)
    streams, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [], []
    for s, x in zip(streams, xs):
        room, ws = torch.empty_like(x), torch.empty(n, dtype=U8, device=DEV)
        out = [torch.empty_like(x) for _ in range(20)]
        lse = [torch.empty(B, Hq, T, device=DEV) for _ in range(20)]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for i in range(20):
                room.fill_(float("nan"))
                room.copy_(x)
                attend(room, out=out[i], lse=lse[i], workspace=ws)
        graphs.append(g)
        outs.append((out, lse, room, ws))
    torch.cuda.synchronize()
    for _ in range(3):
        for o, l, *_ in outs:
            for t in (*o, *l):
                t.fill_(7.0)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = [attend(x) for x in xs]
        torch.cuda.synchronize()
        for (o, l, *_), (wo, wl), (eo, el) in zip(outs, want, eager):
            assert torch.equal(eo, wo) and torch.equal(el, wl)
            assert all(torch.equal(t, wo) for t in o) and all(torch.equal(t, wl) for t in l)
    bsa.bsa_device_status()

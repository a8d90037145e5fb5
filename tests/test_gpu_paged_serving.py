"""The position, cache and paged-attention calls as they are used together: a
prompt, a chunk and single tokens over one cache, captured steps, streams, a
training step through the selector and the attention, tensors past 32 bits."""

import math

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


class Serving:
    """Three requests behind one prompt of 150 tokens: the tokens of each (Q, K,
    V, positions), a cache with pages for all of them, and frequencies."""

    B, P, Hq, Hkv, d, page = 3, 150, 8, 2, 64, 32
    total = 90                                   # own tokens of each request in the end

    def __init__(self):
        n = self.P + self.B * self.total
        self.qkv = randn((n, self.Hq + 2 * self.Hkv, self.d), 50).to(DEV)
        self.pos = torch.randint(0, 700, (n, 3), generator=torch.Generator().manual_seed(51), dtype=torch.int32).to(DEV)
        self.inv, self.axes = bsa.bsa_axis_frequencies((8, 12, 12), device=DEV)
        per, shared = -(-self.total // self.page), -(-self.P // self.page)
        pages = self.B * per + shared + 1
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(52)).int().to(DEV)
        self.kc = torch.full((pages, self.page, self.Hkv, self.d), float("nan"), dtype=BF, device=DEV)
        self.vc = self.kc.clone()
        self.prefix_table = order[:shared]
        wide = torch.full((self.B, per + 5), 1 << 30, dtype=torch.int32, device=DEV)
        wide[:, :per] = order[shared:shared + self.B * per].view(self.B, per)
        self.table = wide[:, :per]               # rows of a wider table

    def rows(self, first, T):
        """q, k, v [B, T, H, d] and positions of own tokens first .. first + T of every request."""
        at = self.P + torch.arange(self.B, device=DEV)[:, None] * self.total + first + torch.arange(T, device=DEV)
        x = self.qkv[at]
        return (x[:, :, :self.Hq], x[:, :, self.Hq:self.Hq + self.Hkv], x[:, :, self.Hq + self.Hkv:], self.pos[at])

    def rope(self):
        return dict(inv_freq=self.inv, axes=self.axes)

    def store_prompt(self):
        x = self.qkv[None, :self.P]
        q = bsa.bsa_cache_append(x[:, :, self.Hq:self.Hq + self.Hkv], x[:, :, self.Hq + self.Hkv:], self.kc, self.vc,
                                 self.prefix_table[None], torch.tensor([self.P], dtype=torch.int32, device=DEV),
                                 q=x[:, :, :self.Hq], positions=self.pos[None, :self.P], **self.rope())
        return q

    def reference(self):
        """A Pool whose keys are those the cache should hold (turned by the same
        kernel, whose values test_gpu_paged pins), and the turned queries."""
        pool = Pool.__new__(Pool)
        k, q = self.qkv[None, :, self.Hq:self.Hq + self.Hkv], self.qkv[None, :, :self.Hq]
        q, k = bsa.bsa_rope_axes(q, k, self.pos, self.pos, self.inv, self.axes)
        v = self.qkv[:, self.Hq + self.Hkv:]
        q, k, v = q[0].cpu(), k[0].cpu(), v.cpu()
        pool.prefix_len, pool.pre_k, pool.pre_v = self.P, k[:self.P], v[:self.P]
        own = [slice(self.P + b * self.total, self.P + (b + 1) * self.total) for b in range(self.B)]
        return pool, q, k, v, own


def test_prompt_chunk_and_single_tokens_over_one_cache():
    s = Serving()
    s.store_prompt()
    pool, q_all, k_all, v_all, own = s.reference()
    at = 0
    for T in (33, 1, 1, 5, 1):
        q, k, v, pos = s.rows(at, T)
        at += T
        lens = torch.full((s.B,), at, dtype=torch.int32, device=DEV)
        q = bsa.bsa_cache_append(k, v, s.kc, s.vc, s.table, lens, q=q, positions=pos, **s.rope())
        out, lse = bsa.bsa_forward_paged(q, s.kc, s.vc, s.table, lens, prefix_table=s.prefix_table, prefix_len=s.P)
        pool.lens = [at] * s.B
        pool.own_k = [k_all[o][:at] for o in own]
        pool.own_v = [v_all[o][:at] for o in own]
        qr = torch.stack([q_all[o][at - T:at] for o in own])
        assert torch.equal(q.cpu(), qr)
        check_attention(out, lse, attend64(qr, pool))
    bsa.bsa_device_status()


def test_prompt_rows_agree_with_the_causal_forward():
    """The prompt attended through its pages (a request with no prefix) and by
    bsa_forward_causal: two kernels, one definition."""
    s = Serving()
    q = s.store_prompt()
    k, v = (c[s.prefix_table.long()].flatten(0, 1)[None, :s.P].contiguous() for c in (s.kc, s.vc))
    dense, dense_lse = bsa.bsa_forward_causal(q, k, v, 128, 128)
    out, lse = bsa.bsa_forward_paged(q, s.kc, s.vc, s.prefix_table[None],
                                     torch.tensor([s.P], dtype=torch.int32, device=DEV))
    pool, q_all, k_all, v_all, _ = s.reference()
    pool.prefix_len, pool.pre_k, pool.pre_v = 0, k_all[:0], v_all[:0]
    pool.lens, pool.own_k, pool.own_v = [s.P], [k_all[:s.P]], [v_all[:s.P]]
    ref = attend64(q.cpu(), pool)
    check_attention(out, lse, ref)
    check_attention(dense, dense_lse, ref)


def test_captured_steps_follow_lengths_tables_and_positions():
    """One captured step (lengths + 1, append, attention) replayed for many
    tokens gives the bits of the eager calls; its buffers are its own, its
    workspace is shared with a second captured step."""
    s = Serving()
    s.store_prompt()
    eager = Serving()
    eager.store_prompt()
    stream = torch.cuda.Stream()
    B, dev = s.B, DEV
    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    step_qkv = torch.empty(B, 1, s.Hq + 2 * s.Hkv, s.d, dtype=BF, device=dev)
    step_pos = torch.empty(B, 1, 3, dtype=torch.int32, device=dev)
    q_out = torch.empty(B, 1, s.Hq, s.d, dtype=BF, device=dev)
    outs = [torch.empty(B, 1, s.Hq, s.d, dtype=BF, device=dev) for _ in range(2)]
    lses = [torch.empty(B, s.Hq, 1, device=dev) for _ in range(2)]
    ws = torch.empty(bsa.bsa_forward_paged_workspace_size(B, 1, s.Hq, s.Hkv, s.d, True), dtype=torch.uint8, device=dev)
    q, k, v = step_qkv[:, :, :s.Hq], step_qkv[:, :, s.Hq:s.Hq + s.Hkv], step_qkv[:, :, s.Hq + s.Hkv:]

    def step():
        lens.add_(1)
        bsa.bsa_cache_append(k, v, s.kc, s.vc, s.table, lens, q=q, positions=step_pos, q_out=q_out, **s.rope())
        bsa.bsa_forward_paged(q_out, s.kc, s.vc, s.table, lens, prefix_table=s.prefix_table, prefix_len=s.P, out=outs[0],
                              lse=lses[0], workspace=ws)

    def again():                                  # the same rows without their own keys' last one, after the step
        bsa.bsa_forward_paged(q_out, s.kc, s.vc, s.table, lens, prefix_table=s.prefix_table, prefix_len=s.P - 7,
                              out=outs[1], lse=lses[1], workspace=ws)

    x = torch.cat([t for t in eager.rows(0, 1)[:3]], 2)
    step_qkv.copy_(x)
    step_pos.copy_(eager.rows(0, 1)[3])
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
            qi, ki, vi, pi = eager.rows(i, 1)
            step_qkv.copy_(torch.cat([qi, ki, vi], 2))
            step_pos.copy_(pi)
            graphs[0].replay()
            graphs[1].replay()
            n = torch.full((B,), i + 1, dtype=torch.int32, device=dev)
            qe = bsa.bsa_cache_append(ki, vi, eager.kc, eager.vc, eager.table, n, q=qi, positions=pi, **s.rope())
            for j, P in enumerate((s.P, s.P - 7)):
                out, lse = bsa.bsa_forward_paged(qe, eager.kc, eager.vc, eager.table, n, prefix_table=eager.prefix_table,
                                                 prefix_len=P)
                assert torch.equal(out, outs[j]) and torch.equal(lse, lses[j]), (i, j)
    stream.synchronize()
    assert torch.equal(s.kc.nan_to_num(), eager.kc.nan_to_num())
    bsa.bsa_device_status()


def test_calls_on_two_streams_at_once():
    """Calls that overlap, each with its own workspace and outputs, give the bits
    of calls that do not."""
    pool = Pool([900, 33, 2000], 700, 2, 128, 64, DEV, 60)
    q = randn((3, 4, 8, 128), 61).to(DEV)
    pos = torch.arange(12, dtype=torch.int32, device=DEV).view(3, 4, 1)
    inv, axes = bsa.bsa_axis_frequencies((64,), device=DEV)
    args = (pool.gk, pool.gv, pool.gtable, pool.kv_lens)
    kw = dict(prefix_table=pool.gprefix, prefix_len=700)
    want = bsa.bsa_forward_paged(q, *args, **kw)
    turned, _ = bsa.bsa_rope_axes(q, None, pos, None, inv, axes)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for st in streams:
            got.append((bsa.bsa_forward_paged(q, *args, stream=st, **kw),
                        bsa.bsa_rope_axes(q, None, pos, None, inv, axes, stream=st.cuda_stream)[0]))
    torch.cuda.synchronize()
    for (out, lse), t in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(t, turned)
    bsa.bsa_device_status()


def test_training_step_through_rotation_selection_and_attention():
    """dL/dq and dL/dk through rotation, selection (everything kept), attention
    and their backward passes, against autograd of the dense formula in 64
    bits.  Tolerance, relative in the 2-norm: 1e-2, the bound that smoke() holds
    the attention's gradients to, and three more bf16 roundings (rotated inputs,
    attention gradients, turned gradients): 1e-2 + 3 * 2^-8."""
    B, S, P, Hq, Hkv, d = 1, 300, 90, 4, 2, 64
    q, k, v = randn((B, S, Hq, d), 70), randn((B, P + S, Hkv, d), 71), randn((B, P + S, Hkv, d), 72)
    g = randn((B, S, Hq, d), 73)
    pos_k = torch.randint(0, 300, (B, P + S, 3), generator=torch.Generator().manual_seed(74), dtype=torch.int32)
    inv, axes = bsa.bsa_axis_frequencies((8, 12, 12), device=DEV)
    gq, gk, gv, gg, gp = (t.to(DEV) for t in (q, k, v, g, pos_k))
    rq, rk = bsa.bsa_rope_axes(gq, gk, gp[:, P:], gp, inv, axes)
    idx, cnt = bsa.bsa_select(rq, rk, P, None, 128, 128, 1.0)
    out, lse = bsa.bsa_forward(rq, rk, gv, idx, cnt, P, None, 128, 128)
    dq, dk, dv = bsa.bsa_backward(rq, rk, gv, out, gg, lse, idx, cnt, P, None, 128, 128)
    dq, dk = bsa.bsa_rope_axes_backward(dq, dk, gp[:, P:], gp, inv, axes, dq_out=dq, dk_out=dk)
    bsa.bsa_device_status()

    leaves = [t.double().requires_grad_() for t in (q, k, v)]

    def turn(x, pos):
        n = axes.numel()
        angle = pos[..., axes.cpu().long()].double() * inv.cpu()
        c, s = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]
        a, b = x[..., :n], x[..., n:2 * n]
        return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * n:]], -1)

    tq, tk = turn(leaves[0], pos_k[:, P:]), turn(leaves[1], pos_k)
    tk, tv = (t.repeat_interleave(Hq // Hkv, 2) for t in (tk, leaves[2]))
    w = torch.softmax(torch.einsum("bihd,bjhd->bhij", tq, tk) * d ** -0.5, -1)
    (torch.einsum("bhij,bjhd->bihd", w, tv) * g.double()).sum().backward()
    for got, leaf in zip((dq, dk, dv), leaves):
        rel = float((got.double().cpu() - leaf.grad).norm() / leaf.grad.norm())
        assert rel <= 1e-2 + 3 * 2.0 ** -8, rel


def test_cache_and_rows_past_32_bits():
    """A cache of more than 2^31 values with a request in its last pages, and a
    rotation of more than 2^31 values, checked at their ends."""
    page, Hkv, d = 128, 8, 128
    total = (1 << 31) // (page * Hkv * d) + 40
    kc = torch.zeros(total, page, Hkv, d, dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)
    n = 700
    k, v = randn((1, n, Hkv, d), 80), randn((1, n, Hkv, d), 81)
    table = torch.arange(total - 6, total, dtype=torch.int32, device=DEV).flip(0)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    bsa.bsa_cache_append(k.to(DEV), v.to(DEV), kc, vc, table, lens)
    assert torch.equal(kc[table[0].long()].flatten(0, 1)[:n].cpu(), k[0])
    assert int(kc[:total - 6].count_nonzero()) == 0
    q = randn((1, 1, 16, d), 82)
    out, lse = bsa.bsa_forward_paged(q.to(DEV), kc, vc, table, lens)
    pool = Pool.__new__(Pool)
    pool.prefix_len, pool.pre_k, pool.pre_v = 0, k[0, :0], v[0, :0]
    pool.lens, pool.own_k, pool.own_v = [n], [k[0]], [v[0]]
    check_attention(out, lse, attend64(q, pool))
    bsa.bsa_device_status()
    del kc, vc

    S, H = (1 << 31) // (32 * 128) + 100, 32
    x = torch.zeros(1, S, H, d, dtype=BF, device=DEV)
    tail = randn((1, 200, H, d), 83)
    x[:, -200:] = tail.to(DEV)
    pos = torch.arange(S, dtype=torch.int32, device=DEV)[:, None]
    inv, axes = bsa.bsa_axis_frequencies((64,), device=DEV)
    y, _ = bsa.bsa_rope_axes(x, None, pos, None, inv, axes, q_out=x)
    ref, bound = rotate64(tail, pos[None, -200:].cpu(), inv.cpu(), axes.cpu())
    assert ((y[:, -200:].double().cpu() - ref).abs() <= bound).all()
    assert int(y[:, :-200].count_nonzero()) == 0


def test_binding_refusals_on_the_gpu():
    pool = Pool([40, 20], 30, 2, 64, 16, DEV, 90)
    q, k = randn((2, 1, 4, 64), 91).to(DEV), randn((2, 1, 2, 64), 92).to(DEV)
    args = (pool.gk, pool.gv, pool.gtable, pool.kv_lens)
    bad = [
        (lambda: bsa.bsa_forward_paged(q.float(), *args), "q must be torch.bfloat16"),
        (lambda: bsa.bsa_forward_paged(q, pool.gk.cpu(), *args[1:]), "k_cache is on cpu"),
        (lambda: bsa.bsa_forward_paged(q, *args[:3], pool.kv_lens.long()), "kv_lens must be torch.int32"),
        (lambda: bsa.bsa_forward_paged(q, *args[:3], pool.kv_lens[:1]), "kv_lens must be contiguous"),
        (lambda: bsa.bsa_forward_paged(q, *args[:2], pool.gtable[:1], pool.kv_lens), "page_table must be"),
        (lambda: bsa.bsa_forward_paged(q, *args, prefix_len=30), "prefix_table is None"),
        (lambda: bsa.bsa_forward_paged(q, *args, prefix_len=49, prefix_table=pool.gprefix[:3]), "prefix_len is 49"),
        (lambda: bsa.bsa_forward_paged(q, *args, out=q), "overlaps"),
        (lambda: bsa.bsa_forward_paged(q, *args, workspace=torch.empty(64, device=DEV)), "workspace"),
        (lambda: bsa.bsa_forward_paged(q.transpose(2, 3), *args), "contiguous last dim"),
        (lambda: bsa.bsa_cache_append(k, k, *args, q=q), "without positions"),
        (lambda: bsa.bsa_cache_append(k, k, *args, q_out=q), "without q"),
        (lambda: bsa.bsa_cache_append(k, k[:, :, :1], *args), "v shape differs"),
    ]
    for call, needle in bad:
        with pytest.raises((ValueError, bsa.BsaError), match=needle):
            call()
    with pytest.raises(bsa.BsaError, match="BSA_ERR_WORKSPACE"):
        bsa.bsa_forward_paged(q, *args, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(bsa.BsaError, match="not a multiple of Hkv"):
        bsa.bsa_forward_paged(q[:, :, :3], *args)
    bsa.bsa_device_status()
    assert math.isfinite(float(bsa.bsa_forward_paged(q, *args)[0].float().sum()))


def test_calls_right_behind_what_writes_their_inputs():
    """Lengths, tables, positions and rows written by the kernel just before a
    call, eager, captured, and behind a join of two streams: the bits of calls
    with a synchronisation after every operation."""
    B, Hq, Hkv, d, page, steps = 8, 8, 2, 128, 64, 40
    g = torch.Generator(device=DEV).manual_seed(70)
    kc0, vc0 = (torch.randn(100, page, Hkv, d, generator=g, device=DEV).to(BF) for _ in range(2))
    tables = [torch.randperm(100, generator=g, device=DEV)[:64].int().view(8, 8) for _ in range(3)]
    rows = torch.randn(B, 1, Hq + 2 * Hkv, d, generator=g, device=DEV).to(BF)
    inv, axes = bsa.bsa_axis_frequencies((16, 24, 24), device=DEV)
    table, lens, pos = tables[0].clone(), torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(
        B, 1, 3, dtype=torch.int32, device=DEV)
    x, kc, vc = rows.clone(), kc0.clone(), vc0.clone()
    side = torch.cuda.Stream()

    def start():
        lens.fill_(100), pos.zero_(), x.copy_(rows), kc.copy_(kc0), vc.copy_(vc0)

    def step(i, between=lambda: None):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):                 # the rows come from another stream
            x.mul_(1.0625 if i % 2 else 0.9375)
        between()
        table.copy_(tables[i % 3])
        between()
        pos.add_(3)
        main.wait_stream(side)
        lens.add_(1)
        between()
        q = bsa.bsa_cache_append(x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], kc, vc, table, lens, q=x[:, :, :Hq],
                                 positions=pos, inv_freq=inv, axes=axes)
        between()
        out, lse = bsa.bsa_forward_paged(q, kc, vc, table, lens)
        between()
        x[:, :, :Hq].add_(out)
        between()
        return out, lse

    def same(a, b):
        return all(torch.equal(s, t) for x, y in zip(a, b) for s, t in zip(x, y))

    start()
    want = [step(i, torch.cuda.synchronize) for i in range(steps)]
    run = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(run):
        for _ in range(5):
            start()
            got = [step(i) for i in range(steps)]
            run.synchronize()
            assert same(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=run):
            start()
            got = [step(i) for i in range(steps)]
        for _ in range(5):
            graph.replay()
            run.synchronize()
            assert same(got, want)
    bsa.bsa_device_status()

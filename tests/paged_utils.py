"""Plain 64-bit forms of the multi-axis rotation, the paged append and the
paged attention, and the bounds their kernels are held to.

Bounds, from the arithmetic of the kernels (bf16 rounding: at most 2^-8 of the
value; fp32: 2^-24):

* rotation y = a cos - b sin: sine and cosine are off by at most pi 2^-24 (the
  half-turn count is rounded to fp32) + 2^-22 (sincospif) < 2^-21; the two
  products and their sum round three times in fp32; the result once to bf16:
      |err| <= 2^-8 |y| + (|a| + |b|) 2^-20.
* logits z_j = scale sum_e q_e k_je: at most d <= 128 fp32 additions, each off
  by 2^-23 of the running magnitude (accumulators may truncate), and one
  product with scale log2 e:
      dz <= 2^-15 max_j scale sum_e |q_e k_je|.
* weights: relative 2 dz (own logit and maximum) + 2^-8 (bf16 weights against
  fp32 sums) + 2^-12 (2^x to 2 units in the last place, fp32 sums and joins of
  up to 2^10 partial results); the output once to bf16:
      |err| <= 2^-8 |o| + (2 dz + 2^-8 + 2^-12) sum_j w_j |v_j|.
* lse: |err| <= dz + 2^-19 (|lse| + 1)  (fp32 log, sums and joins).
"""

from __future__ import annotations

import math

import torch

BF = torch.bfloat16


def rotate64(x, pos, inv_freq, axes, interleaved=False, back=False):
    """(y, bound) of the rotation of x [B, S, H, d] at pos [B, S, A], 64 bits."""
    y = x.double().clone()
    bound = torch.zeros_like(y)
    for p in range(axes.numel()):
        a = int(axes[p])
        if not 0 <= a < pos.shape[-1]:
            continue
        lo, hi = (2 * p, 2 * p + 1) if interleaved else (p, p + axes.numel())
        angle = (pos[..., a].double() * inv_freq[p].double())[:, :, None]
        c, s = torch.cos(angle), torch.sin(angle) * (-1 if back else 1)
        u, w = x[..., lo].double(), x[..., hi].double()
        y[..., lo], y[..., hi] = u * c - w * s, w * c + u * s
        for ch in (lo, hi):
            bound[..., ch] = 2.0 ** -8 * y[..., ch].abs() + (u.abs() + w.abs()) * 2.0 ** -20
    return y, bound


class Pool:
    """A paged cache with every slot poisoned, tables in no order, and lists of
    the keys that stand in it."""

    def __init__(self, lens, prefix, Hkv, d, page, device, seed, max_pages=None, layout="slots", fill=float("nan")):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        shared = -(-prefix // page)
        total = sum(need) + shared + 2
        self.page, self.total = page, total
        shape = (total, page, Hkv, d)
        if layout == "slots":            # [pages, page, H, d]
            self.k, self.v = (torch.full(shape, fill, dtype=BF) for _ in range(2))
        elif layout == "heads":          # [pages, H, page, d]
            self.k, self.v = (torch.full((total, Hkv, page, d), fill, dtype=BF).transpose(1, 2) for _ in range(2))
        else:                            # K and V of a page beside each other
            both = torch.full((total, 2, page, Hkv, d), fill, dtype=BF)
            self.k, self.v = both[:, 0], both[:, 1]
        order = torch.randperm(total, generator=g).tolist()
        width = max(1, max(need)) if max_pages is None else max_pages
        # entries behind a request's length are never read: 2^30 would be far outside
        self.table = torch.full((len(lens), width), 1 << 30, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.prefix_table = torch.tensor(order[at:at + shared] + [1 << 30], dtype=torch.int32)
        self.prefix_len, self.lens = prefix, list(lens)

        def put(cache, table, rows):
            for j in range(rows.shape[0]):
                cache[int(table[j // page]), j % page] = rows[j]

        self.own_k = [torch.randn(n, Hkv, d, generator=g).to(BF) for n in lens]
        self.own_v = [torch.randn(n, Hkv, d, generator=g).to(BF) for n in lens]
        self.pre_k, self.pre_v = (torch.randn(prefix, Hkv, d, generator=g).to(BF) for _ in range(2))
        for b in range(len(lens)):
            put(self.k, self.table[b], self.own_k[b])
            put(self.v, self.table[b], self.own_v[b])
        put(self.k, self.prefix_table, self.pre_k)
        put(self.v, self.prefix_table, self.pre_v)
        self.gk, self.gv = self.k.to(device), self.v.to(device)
        assert self.gk.stride() == self.k.stride() or layout == "pairs"
        if layout == "pairs":
            both = both.to(device)
            self.gk, self.gv = both[:, 0], both[:, 1]
        self.gtable, self.gprefix = self.table.to(device), self.prefix_table.to(device)
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32, device=device)


def attend64(q, pool: Pool, new_lens=None, causal=True, scale=None):
    """(out, lse, out bound, lse bound) in 64 bits; q [B, T, Hq, d] on the CPU."""
    B, T, Hq, d = q.shape
    Hkv = pool.pre_k.shape[1] if pool.prefix_len else pool.own_k[0].shape[1]
    G = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros(B, T, Hq, d, dtype=torch.float64)
    bound = torch.zeros_like(out)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64)
    lbound = torch.zeros_like(lse)
    for b in range(B):
        n = T if new_lens is None else min(max(new_lens[b], 0), T)
        k = torch.cat([pool.pre_k, pool.own_k[b]]).double()
        v = torch.cat([pool.pre_v, pool.own_v[b]]).double()
        kv = pool.lens[b]
        for i in range(n):
            own = max(0, min(kv, kv - n + i + 1)) if causal else kv
            m = pool.prefix_len + own
            if m == 0:
                continue
            for h in range(Hq):
                qq, kk, vv = q[b, i, h].double(), k[:m, h // G], v[:m, h // G]
                z = kk @ qq * scale
                dz = 2.0 ** -15 * float((kk.abs() @ qq.abs()).max()) * scale
                w = torch.softmax(z, 0)
                out[b, i, h] = w @ vv
                lse[b, h, i] = torch.logsumexp(z, 0)
                bound[b, i, h] = 2.0 ** -8 * out[b, i, h].abs() + (2 * dz + 2.0 ** -8 + 2.0 ** -12) * (w @ vv.abs())
                lbound[b, h, i] = dz + 2.0 ** -19 * (abs(float(lse[b, h, i])) + 1)
    return out, lse, bound, lbound


def check_attention(out, lse, ref):
    o, l, ob, lb = ref
    out, lse = out.double().cpu(), lse.double().cpu()
    empty = torch.isneginf(l)
    assert torch.isfinite(out).all()
    assert (torch.isneginf(lse) == empty).all()
    assert (out.transpose(1, 2)[empty] == 0).all()
    bad = (out - o).abs() > ob
    assert not bad.any(), (bad.nonzero()[:4].tolist(), float((out - o).abs()[bad].max()), int(bad.sum()))
    off = (lse - l).abs()[~empty]
    assert (off <= lb[~empty]).all(), float(off.max())

"""The 4-bit format in plain 64-bit arithmetic, packed and unpacked byte by byte
from its description, and a cache of it with lists of what stands in it.

Values that pages hold are exact in bf16, so that what is written and read back
is compared for equality; attention over them has the bounds of ``paged_utils``
(the kernels' products are of the same bf16 numbers).
"""

from __future__ import annotations

import torch

from paged_utils import BF, Pool

U8 = torch.uint8
# the values of the 255 scale bytes
SCALES = torch.tensor([(1 + b % 8 / 8) * 2.0 ** (b // 8 - 15) for b in range(255)], dtype=torch.float64)


def quantise64(x):
    """(codes -7 .. 7, scale bytes) of x [..., d]; bytes [..., d / 32]."""
    x = x.double().unflatten(-1, (-1, 32))
    fine = torch.isfinite(x).all(-1)
    x = x.masked_fill(~fine[..., None], 0.0)
    want = torch.clamp(x.abs().amax(-1) / 7, max=float(SCALES[-1]))
    # the nearest scale, of two as near the one with an even byte
    off = (want[..., None] - SCALES).abs()
    near = off == off.amin(-1, keepdim=True)
    byte = torch.where(near, torch.arange(255), 255).amin(-1)
    last = torch.where(near, torch.arange(255), -1).amax(-1)
    byte = torch.where(byte % 2 == 0, byte, last)
    byte = torch.where(want == 0, 0, byte)
    codes = torch.sign(x) * torch.clamp(torch.floor(x.abs() / SCALES[byte][..., None] + 0.5), max=7)
    return codes.to(torch.int64).flatten(-2), torch.where(fine, byte, 255)


def values64(codes, byte):
    s = torch.cat([SCALES, torch.tensor([float("nan")], dtype=torch.float64)])[byte]
    return (codes.double().unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def held(x):
    """What a cache holds of x, as bf16."""
    y = values64(*quantise64(x))
    assert ((y.to(BF).double() == y) | torch.isnan(y)).all()
    return y.to(BF)


def _nibbles(u):
    """[..., 8 m] codes + 8 to [..., 4 m] bytes: number e of eight in bits 4 (e / 2 + 4 (e mod 2))."""
    out = torch.zeros(*u.shape[:-1], u.shape[-1] // 2, dtype=torch.int64)
    for e in range(u.shape[-1]):
        n = e % 8 // 2 + 4 * (e % 2)
        out[..., e // 8 * 4 + n // 2] |= u[..., e] << (4 * (n % 2))
    return out


def _block(codes, byte, channels_first):
    """Bytes [H, 17 d / 2] of a block from codes [16, H, d] and scale bytes [16, H, d / 32]."""
    d = codes.shape[-1]
    u = codes + 8
    if channels_first:
        c = _nibbles(u.permute(1, 2, 0))                                       # [H, d, 8]
    else:
        c = _nibbles(u.unflatten(-1, (d // 32, 32)).permute(1, 2, 0, 3))       # [H, G, 16, 16]
    return torch.cat([c.flatten(1), byte.permute(1, 2, 0).flatten(1)], 1).to(U8)


def _mask(slots, H, d, channels_first):
    """Bits of a block that belong to the given slots."""
    codes = torch.full((16, H, d), -8, dtype=torch.int64)
    codes[slots] = 7
    byte = torch.zeros(16, H, d // 32, dtype=torch.int64)
    byte[slots] = 255
    return _block(codes, byte, channels_first)


def write(cache, table, first, x, channels_first):
    """Rows x [n, H, d] into keys first .. first + n of a request's pages, the rest of the cache kept."""
    n, H, d = x.shape
    if n == 0:
        return
    codes, byte = quantise64(x)
    blocks = cache.shape[2]
    for blk in range(first // 16, (first + n - 1) // 16 + 1):
        slots = [i for i in range(16) if first <= blk * 16 + i < first + n]
        rows = [blk * 16 + i - first for i in slots]
        c, s = torch.zeros(16, H, d, dtype=torch.int64), torch.zeros(16, H, d // 32, dtype=torch.int64)
        c[slots], s[slots] = codes[rows], byte[rows]
        m = _mask(slots, H, d, channels_first)
        at = cache[int(table[blk // blocks]), :, blk % blocks]
        at.copy_((at & ~m) | (_block(c, s, channels_first) & m))


class QPool(Pool):
    """A 4-bit cache with every byte poisoned (0xFF: scales that read as NaN),
    tables in no order, and lists of the values that stand in it."""

    def __init__(self, lens, prefix, Hkv, d, page, device, seed, max_pages=None, layout="pages", wide=1.0):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        shared = -(-prefix // page)
        total = sum(need) + shared + 2
        self.page, self.total = page, total
        shape = (total, Hkv, page // 16, 17 * d // 2)
        if layout == "pages":
            self.k, self.v = (torch.full(shape, 255, dtype=U8) for _ in range(2))
        elif layout == "heads":          # [H, pages, ..]
            self.k, self.v = (torch.full((shape[1], shape[0], *shape[2:]), 255, dtype=U8).transpose(0, 1) for _ in range(2))
        else:                            # K and V of a page beside each other
            both = torch.full((total, 2, *shape[1:]), 255, dtype=U8)
            self.k, self.v = both[:, 0], both[:, 1]
        order = torch.randperm(total, generator=g).tolist()
        width = max(1, max(need)) if max_pages is None else max_pages
        self.table = torch.full((len(lens), width), 1 << 30, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.prefix_table = torch.tensor(order[at:at + shared] + [1 << 30], dtype=torch.int32)
        self.prefix_len, self.lens = prefix, list(lens)

        def fill(table, n, cache, channels_first):
            x = torch.randn(n, Hkv, d, generator=g).to(BF) * (1.0 if channels_first else wide)
            write(cache, table, 0, x, channels_first)
            return held(x) if n else x

        self.own_k = [fill(self.table[b], n, self.k, False) for b, n in enumerate(lens)]
        self.own_v = [fill(self.table[b], n, self.v, True) for b, n in enumerate(lens)]
        self.pre_k, self.pre_v = fill(self.prefix_table, prefix, self.k, False), fill(self.prefix_table, prefix, self.v, True)
        if layout == "beside":
            both = both.to(device)
            self.gk, self.gv = both[:, 0], both[:, 1]
        else:
            self.gk, self.gv = self.k.to(device), self.v.to(device)
            assert self.gk.stride() == self.k.stride()
        self.gtable, self.gprefix = self.table.to(device), self.prefix_table.to(device)
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32, device=device)

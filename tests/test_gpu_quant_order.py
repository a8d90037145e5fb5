"""Attention over 4-bit pages whose prefix and own keys run in two kernels side by side:
what the calls in front have written is read, whichever of the kernels reads it."""

import pytest
import torch

import block_sparse_attention_bsa_gb300 as bsa
from paged_utils import BF
from quant_utils import U8

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    bsa.build()


# B, T, prefix, Hq, Hkv, d, page: prefixes of more tiles than one kernel takes for both
@pytest.mark.parametrize("B,T,prefix,Hq,Hkv,d,page", [(160, 1, 700, 8, 2, 128, 64), (64, 2, 613, 8, 2, 64, 32)])
def test_all_inputs_of_a_long_prefix_beside_own_keys_written_right_before(B, T, prefix, Hq, Hkv, d, page):
    """Rows, tables, lengths, numbers of new tokens and both parts of the cache change in
    every step, by the kernels just before the attention; eager and captured steps give
    the bits of steps with a synchronisation after every operation."""
    steps, own = 20, -(-200 // page)
    shared = -(-prefix // page)
    g = torch.Generator(device=DEV).manual_seed(500)
    shape = bsa.bsa_cache_q4_shape(B * own + 2 * shared, page, Hkv, d)
    start_k, start_v = (torch.randint(0, 120, shape, generator=g, device=DEV, dtype=I32).to(U8) for _ in range(2))
    order = torch.arange(B * own + 2 * shared, device=DEV, dtype=I32)
    tables = [torch.randperm(B * own, generator=g, device=DEV).int().view(B, own) for _ in range(3)]
    prefixes = [order[B * own:B * own + shared], order[B * own + shared:].flip(0)]
    counts = [torch.randint(0, T + 1, (B,), generator=g, device=DEV).int() for _ in range(3)]
    wide = torch.randn(B, T, Hq + 2 * Hkv, d, generator=g, device=DEV).to(BF)
    prompt = torch.randn(1, prefix, 2 * Hkv, d, generator=g, device=DEV).to(BF)
    x, kc, vc, rows = wide.clone(), start_k.clone(), start_v.clone(), prompt.clone()
    table, lens, new, pre = tables[0].clone(), torch.zeros(B, dtype=I32, device=DEV), counts[0].clone(), prefixes[0].clone()
    whole = torch.tensor([prefix], dtype=I32, device=DEV)

    def start():
        lens.fill_(90), x.copy_(wide), rows.copy_(prompt), kc.copy_(start_k), vc.copy_(start_v)

    def step(i, between=lambda: None):
        x.mul_(1.0625 if i % 2 else 0.9375)
        rows.mul_(0.9375 if i % 2 else 1.0625)
        between()
        bsa.bsa_cache_append_q4(rows[:, :, :Hkv], rows[:, :, Hkv:], kc, vc, prefixes[i % 2][None], whole)
        between()
        table.copy_(tables[i % 3]), pre.copy_(prefixes[i % 2]), new.copy_(counts[i % 3])
        lens.add_(new)
        between()
        bsa.bsa_cache_append_q4(x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], kc, vc, table, lens, new_lens=new)
        between()
        out, lse = bsa.bsa_forward_paged_q4(x[:, :, :Hq], kc, vc, table, lens, new_lens=new, prefix_table=pre,
                                            prefix_len=prefix)
        between()
        lens.add_(1)                                  # written right behind, too
        x[:, :, :Hq].add_(out.clamp(-1, 1))
        between()
        again = bsa.bsa_forward_paged_q4(x[:, :, :Hq], kc, vc, table, lens, prefix_table=pre, prefix_len=prefix)
        between()
        return (out, lse, *again)

    def same(a, b):
        return all(torch.equal(s, t) for p, q in zip(a, b) for s, t in zip(p, q))

    start()
    want = [step(i, torch.cuda.synchronize) for i in range(steps)]
    assert all(bool(torch.isfinite(w[2]).all()) for w in want)
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

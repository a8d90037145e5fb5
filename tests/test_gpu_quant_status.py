"""What bsa_device_status reports of the 4-bit cache's calls."""

import pytest
import torch

import block_sparse_attention_bsa_gb300 as bsa
from paged_utils import BF, Pool, attend64, check_attention
from quant_utils import QPool, U8

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
I32 = torch.int32
FAR = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def built():
    bsa.build()


def randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF)


def ints(x):
    return torch.tensor(x, dtype=I32, device=DEV)


@pytest.mark.parametrize("lens,first,length", [
    ([5, 300, 0], [FAR, FAR, FAR], 1),
    ([5, 300, 0], [FAR, FAR - 300, FAR], 400),
    ([5, 300, 33], [FAR, 290, FAR], 3000),
])
def test_read_from_far_behind_the_last_key_reads_nothing(lens, first, length):
    """No key lies below the length there, whatever the number of rows: none is written
    and none missing."""
    pool = QPool(lens, 0, 2, 64, 16, DEV, 405)
    out = [torch.full((3, length, 2, 64), 7.0, dtype=BF, device=DEV) for _ in range(2)]
    bsa.bsa_device_status()
    bsa.bsa_cache_read_q4(pool.gk, pool.gv, pool.gtable, pool.kv_lens, length, first=ints(first), k_out=out[0], v_out=out[1])
    bsa.bsa_device_status()
    for got, rows in zip(out, (pool.own_k, pool.own_v)):
        for b in range(3):
            n = max(0, min(lens[b] - first[b], length))
            assert torch.equal(got[b, :n].cpu(), rows[b][first[b]:first[b] + n])
            assert (got[b, n:] == 7).all()


def test_read_reports_a_negative_length():
    """As the append and the attention do; other requests are read."""
    pool = QPool([40, 20], 0, 2, 64, 16, DEV, 406)
    for first in (None, ints([0, 3])):
        bsa.bsa_device_status()
        k, v = bsa.bsa_cache_read_q4(pool.gk, pool.gv, pool.gtable, ints([-1, 20]), 30, first=first)
        with pytest.raises(bsa.BsaError, match="BSA_ERR_INVALID_INDICES.*bsaq_cache_read"):
            bsa.bsa_device_status()
        f = 0 if first is None else 3
        assert torch.equal(k[1, :20 - f].cpu(), pool.own_k[1][f:]) and torch.equal(v[1, :20 - f].cpu(), pool.own_v[1][f:])
        assert (k[0] == 0).all()
    bsa.bsa_device_status()


# lens, T, prefix, Hq, Hkv, d, page: a kernel of few rows, the one of many rows, both beside one another
WAYS = {
    "few rows": ([70, 40], 1, 40, 8, 2, 128, 32),
    "a chunk": ([70, 40], 17, 40, 8, 2, 64, 32),
    "a chunk and its prefix": ([200] * 3, 100, 300, 16, 2, 128, 64),
    "a long prefix beside own keys": ([70, 3] * 80, 1, 700, 8, 2, 128, 64),
}


@pytest.mark.parametrize("bad", ["table", "prefix", "length"])
@pytest.mark.parametrize("way", WAYS)
def test_bad_pages_are_reported_under_the_call_that_met_them(way, bad):
    lens, T, prefix, Hq, Hkv, d, page = WAYS[way]
    pool = QPool(lens, prefix, Hkv, d, page, DEV, 400)
    q = randn((len(lens), T, Hq, d), 401).to(DEV)
    table, shared, kv = pool.gtable.clone(), pool.gprefix.clone(), pool.kv_lens.clone()
    if bad == "table":
        table[0, 0] = pool.total
    elif bad == "prefix":
        shared[-(-prefix // page) - 1] = -1
    else:
        kv[0] = table.shape[1] * page + 1
    bsa.bsa_device_status()
    bsa.bsa_forward_paged_q4(q, pool.gk, pool.gv, table, kv, prefix_table=shared, prefix_len=prefix)
    with pytest.raises(bsa.BsaError, match="BSA_ERR_INVALID_INDICES.*reached bsaq_forward") as e:
        bsa.bsa_device_status()
    assert "bsap_forward" not in str(e.value)
    bsa.bsa_device_status()


def test_bad_pages_of_both_caches_attentions_are_told_apart():
    x = randn((1, 40, 4, 64), 402).to(DEV)
    plain, packed = Pool([60], 0, 2, 64, 16, DEV, 403, fill=1.0), QPool([60], 0, 2, 64, 16, DEV, 404)
    plain.gtable[0, 1] = packed.gtable[0, 1] = -1
    bsa.bsa_device_status()
    bsa.bsa_forward_paged(x, plain.gk, plain.gv, plain.gtable, plain.kv_lens)
    with pytest.raises(bsa.BsaError, match="reached bsap_forward") as e:
        bsa.bsa_device_status()
    assert "bsaq" not in str(e.value)
    bsa.bsa_forward_paged(x, plain.gk, plain.gv, plain.gtable, plain.kv_lens)
    bsa.bsa_forward_paged_q4(x, packed.gk, packed.gv, packed.gtable, packed.kv_lens)
    with pytest.raises(bsa.BsaError, match="reached bsap_forward and bsaq_forward"):
        bsa.bsa_device_status()
    bsa.bsa_device_status()


def test_tables_and_lengths_right_beside_what_is_written():
    """In one allocation with the outputs of a read, and with the caches of an append,
    one element before the first byte and one behind the last."""
    pool = QPool([40, 20], 0, 2, 64, 16, DEV, 407)
    want = bsa.bsa_cache_read_q4(pool.gk, pool.gv, pool.gtable, pool.kv_lens, 40)
    n = want[0].numel() * 2
    for at in (16, 16 + n):
        room = torch.zeros(n + 64, dtype=U8, device=DEV)
        out = room[16:16 + n].view(BF).view(want[0].shape)
        lens = room[at - 8 if at == 16 else at:][:8].view(I32)
        lens.copy_(pool.kv_lens)
        k, v = bsa.bsa_cache_read_q4(pool.gk, pool.gv, pool.gtable, lens, 40, k_out=out)
        assert k is out and torch.equal(k, want[0]) and torch.equal(v, want[1])
        with pytest.raises(bsa.BsaError, match="k_out shares memory with kv_lens"):
            bsa.bsa_cache_read_q4(pool.gk, pool.gv, pool.gtable, room[12:20].view(I32), 40, k_out=out)
    m = pool.gk.numel()
    room = torch.zeros(m + 64, dtype=U8, device=DEV)
    kc, vc = room[16:16 + m].view(pool.gk.shape), torch.zeros_like(pool.gv)
    lens = room[16 + m:16 + m + 8].view(I32)
    lens.copy_(pool.kv_lens)
    bsa.bsa_cache_append_q4(*want, kc, vc, pool.gtable, lens, new_lens=pool.kv_lens)
    k, v = bsa.bsa_cache_read_q4(kc, vc, pool.gtable, lens, 40)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    with pytest.raises(bsa.BsaError, match="k_cache shares memory with kv_lens"):
        bsa.bsa_cache_append_q4(*want, kc, vc, pool.gtable, room[16:24].view(I32))
    bsa.bsa_device_status()


def test_a_wait_that_gave_up_is_reported_once_and_the_next_call_is_right():
    """One thread waits, with the kernels' bounded wait and a limit of 20 ms, for a phase
    that nothing completes, and leaves: the word of the kernel of few rows."""
    pool = QPool([300, 5], 130, 2, 64, 16, DEV, 408)
    q = randn((2, 1, 4, 64), 409)
    args = (q.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens)
    bsa.bsa_device_status()
    bsa.bsa_debug_paged_q4_wait_probe(20_000_000)
    with pytest.raises(bsa.BsaError, match="BSA_ERR_TIMEOUT.*in the paged attention kernels"):
        bsa.bsa_device_status()
    bsa.bsa_device_status()
    bsa.bsa_debug_paged_q4_wait_probe(20_000_000)
    bsa.bsa_debug_wait_probe(1, 20_000_000)
    with pytest.raises(bsa.BsaError, match="BSA_ERR_TIMEOUT.*in the paged attention and other kernels"):
        bsa.bsa_device_status()
    table = pool.gtable.clone()
    table[0, 1] = -1
    bsa.bsa_forward_paged_q4(*args[:3], table, pool.kv_lens)
    bsa.bsa_debug_paged_q4_wait_probe(20_000_000)
    with pytest.raises(bsa.BsaError, match="BSA_ERR_INVALID_INDICES.*bsaq_forward; a bounded device wait also gave up"):
        bsa.bsa_device_status()
    bsa.bsa_device_status()
    out, lse = bsa.bsa_forward_paged_q4(*args, prefix_table=pool.gprefix, prefix_len=130)
    bsa.bsa_device_status()
    check_attention(out, lse, attend64(q, pool))

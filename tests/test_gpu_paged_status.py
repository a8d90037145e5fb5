"""What bsa_device_status reports of the cache append and the paged attention."""

import pytest
import torch

import block_sparse_attention_bsa_gb300 as bsa
from bsa_inputs import CONFIGS, make_inputs
from paged_utils import Pool, attend64, check_attention

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    bsa.build()


def test_a_wait_that_gave_up_is_reported_once_and_the_next_call_is_right():
    """One thread waits, with the kernels' bounded wait and a limit of 20 ms, for
    a phase that nothing completes, and leaves."""
    bsa.bsa_device_status()
    bsa.bsa_debug_paged_wait_probe(20_000_000)
    with pytest.raises(bsa.BsaError, match="BSA_ERR_TIMEOUT.*in the paged attention kernels"):
        bsa.bsa_device_status()
    bsa.bsa_device_status()
    bsa.bsa_debug_paged_wait_probe(20_000_000)
    bsa.bsa_debug_wait_probe(0, 20_000_000)
    with pytest.raises(bsa.BsaError, match="BSA_ERR_TIMEOUT.*in the paged attention and other kernels"):
        bsa.bsa_device_status()
    bsa.bsa_device_status()
    pool = Pool([300, 5], 130, 2, 64, 16, DEV, 111)
    q = torch.randn(2, 1, 4, 64, generator=torch.Generator().manual_seed(112)).to(torch.bfloat16)
    out, lse = bsa.bsa_forward_paged(q.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens, prefix_table=pool.gprefix,
                                     prefix_len=130)
    bsa.bsa_device_status()
    check_attention(out, lse, attend64(q, pool))


def test_a_wait_that_gave_up_is_told_of_beside_a_bad_page():
    bsa.bsa_device_status()
    pool = Pool([40], 0, 2, 64, 16, DEV, 113, fill=1.0)
    table = pool.gtable.clone()
    table[0, 1] = -1
    x = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device=DEV)
    bsa.bsa_forward_paged(x, pool.gk, pool.gv, table, pool.kv_lens)
    bsa.bsa_debug_paged_wait_probe(20_000_000)
    with pytest.raises(bsa.BsaError, match="BSA_ERR_INVALID_INDICES.*bsap_forward; a bounded device wait also gave up"):
        bsa.bsa_device_status()
    bsa.bsa_device_status()


def test_bad_pages_are_reported_beside_malformed_lists(monkeypatch):
    """With BSA_DEBUG, an index list out of order and a page table entry that
    names no page between two status calls: both are told of, once."""
    monkeypatch.setenv("BSA_DEBUG", "1")
    bsa.bsa_device_status()
    cfg = CONFIGS["small_gqa"]
    inp = make_inputs(cfg, "cuda", pad_fill=0.0)
    q, k, v, lens = inp["q"], inp["k"], inp["v"], inp["seq_lens"]
    idx, cnt = bsa.bsa_select(q, k, cfg.prefix, lens, cfg.block_q, cfg.block_k, inp["keep_ratio"])
    bad = idx.clone()
    assert int(cnt[0, 0, 0]) >= 2
    bad[0, 0, 0, 0], bad[0, 0, 0, 1] = idx[0, 0, 0, 1], idx[0, 0, 0, 0]
    pool = Pool([40, 20], 0, 2, 64, 16, DEV, 110, fill=1.0)
    table = pool.gtable.clone()
    table[0, 1] = pool.total
    x = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16, device=DEV)
    new = torch.zeros(2, 20, 2, 64, dtype=torch.bfloat16, device=DEV)
    bsa.bsa_forward(q, k, v, bad, cnt, cfg.prefix, lens, cfg.block_q, cfg.block_k)
    bsa.bsa_forward_paged(x, pool.gk, pool.gv, table, pool.kv_lens)
    with pytest.raises(bsa.BsaError, match="BSA_ERR_INVALID_INDICES: 1 malformed.*bsap_forward"):
        bsa.bsa_device_status()
    bsa.bsa_device_status()
    bsa.bsa_forward(q, k, v, bad, cnt, cfg.prefix, lens, cfg.block_q, cfg.block_k)
    bsa.bsa_cache_append(new, new, pool.gk, pool.gv, table, pool.kv_lens)
    with pytest.raises(bsa.BsaError, match="BSA_ERR_INVALID_INDICES: 1 malformed.*bsap_cache_append"):
        bsa.bsa_device_status()
    bsa.bsa_device_status()

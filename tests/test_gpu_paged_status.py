"""What bsa_device_status reports of the cache append and the paged attention."""

import pytest
import torch

import block_sparse_attention_bsa_gb300 as bsa
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

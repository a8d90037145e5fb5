"""What bsa_device_status reports of the 4-bit cache's calls."""

import pytest
import torch

import block_sparse_attention_bsa_gb300 as bsa
from paged_utils import BF
from quant_utils import QPool

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
I32 = torch.int32
FAR = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def built():
    bsa.build()


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

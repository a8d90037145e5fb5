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

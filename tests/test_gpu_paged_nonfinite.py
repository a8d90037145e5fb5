"""Numbers that are not finite in the paged attention and the rotation: a row of
Q that holds them comes out of the attention as NaN (0 and -inf mean "no key" and
nothing else), and no other row feels it; a pair without an axis keeps them.

The rows' scores, from the formula alone: a NaN in q makes every score NaN; an
infinity in one channel makes them infinite with the signs of that channel of K;
3e38 (finite in bf16) in one channel makes those infinite whose K channel is
above 1.14 in size, since the product is past fp32's 3.4e38.  softmax of scores
with a NaN or a +inf among them, or all -inf, is NaN.
"""

import pytest
import torch

import block_sparse_attention_bsa_gb300 as bsa
from paged_utils import BF, Pool, rotate64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    bsa.build()


def randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF)


# lens, T, new, prefix, Hq, Hkv, d, page, causal
WAYS = {
    "direct, few rows": ([100, 77], 1, None, 0, 8, 2, 128, 64, True),
    "direct, two tiles": ([256] * 40, 3, None, 0, 8, 8, 64, 32, True),
    "direct and cut, wide": ([300] * 60, 90, None, 0, 8, 4, 64, 64, True),
    "join by eight warps": ([3000], 1, None, 0, 16, 1, 128, 64, True),
    "join by a warp": ([5, 300] * 30, 1, None, 300, 16, 2, 64, 16, True),
    "join by eight lanes": ([40, 130] * 20, 40, [40, 3] * 20, 200, 8, 2, 128, 32, True),
    "prefix folded": ([300], 1, None, 1000, 4, 2, 64, 64, True),
    "not causal": ([140, 40], 5, None, 129, 8, 1, 128, 256, False),
}


@pytest.mark.parametrize("kind", ["nan", "inf", "3e38"])
@pytest.mark.parametrize("way", WAYS)
def test_rows_of_numbers_that_are_not_finite_come_out_as_nan(way, kind):
    lens, T, new, prefix, Hq, Hkv, d, page, causal = WAYS[way]
    B = len(lens)
    pool = Pool(lens, prefix, Hkv, d, page, DEV, 100)
    q = randn((B, T, Hq, d), 101)
    new_t = None if new is None else torch.tensor(new, dtype=torch.int32, device=DEV)

    def attend(x):
        out, lse = bsa.bsa_forward_paged(x.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens, new_lens=new_t,
                                         prefix_table=pool.gprefix, prefix_len=prefix, causal=causal)
        bsa.bsa_device_status()
        return out.cpu(), lse.cpu()

    want, want_lse = attend(q)
    g = torch.Generator().manual_seed(102)
    hit = torch.zeros(B, T, Hq, dtype=torch.bool)
    bad = q.clone()
    for b in range(0, B, 1 if B < 5 else 7):
        n = T if new is None else new[b]
        i, h = int(torch.randint(0, n, (1,), generator=g)), int(torch.randint(0, Hq, (1,), generator=g))
        c = int(torch.randint(0, d, (1,), generator=g))
        bad[b, i, h] = 0
        bad[b, i, h, c] = float(kind)
        keys = torch.cat([pool.pre_k, pool.own_k[b]])[:, h // (Hq // Hkv), c].float()
        if causal:
            keys = keys[:prefix + lens[b] - n + i + 1]
        z = keys * float(torch.tensor(float(kind)).to(BF))     # one product: the others are with 0
        if torch.isnan(torch.softmax(z.float(), 0)).any():
            hit[b, i, h] = True
        else:
            bad[b, i, h] = q[b, i, h]                    # no product of this row passes fp32's range
    assert hit.any()
    out, lse = attend(bad)
    assert torch.isnan(out[hit]).all()
    assert not torch.isfinite(lse.transpose(1, 2)[hit]).any()
    if kind == "nan":
        assert torch.isnan(lse.transpose(1, 2)[hit]).all()
    assert torch.equal(out[~hit], want[~hit])
    assert torch.equal(lse.transpose(1, 2)[~hit], want_lse.transpose(1, 2)[~hit])
    assert torch.isfinite(want).all()


@pytest.mark.parametrize("prefix,lens", [(0, [2, 40]), (0, [2])])
def test_rows_without_a_key_stay_empty_whatever_their_q_holds(prefix, lens):
    """Five tokens of which the first three stand before the first key."""
    B, T = len(lens), 5
    pool = Pool(lens, prefix, 2, 64, 16, DEV, 103)
    q = randn((B, T, 4, 64), 104)
    want, want_lse = (x.cpu() for x in bsa.bsa_forward_paged(q.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens))
    q[0, 0], q[0, 1], q[0, 2] = float("nan"), float("inf"), 3e38
    out, lse = (x.cpu() for x in bsa.bsa_forward_paged(q.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens))
    bsa.bsa_device_status()
    assert (out[0, :3] == 0).all() and torch.isneginf(lse[0, :, :3]).all()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_scores_of_minus_infinity_alone_are_no_empty_row():
    """3e38 times keys of -2: every score is -inf, softmax of which is NaN; its
    log-sum-exp is -inf by the formula."""
    pool = Pool([20], 0, 1, 64, 16, DEV, 105)
    pool.gk[..., 5] = -2.0
    q = torch.zeros(1, 1, 2, 64, dtype=BF)
    q[0, 0, 0, 5], q[0, 0, 1, 5] = 3e38, 0.5
    out, lse = bsa.bsa_forward_paged(q.to(DEV), pool.gk, pool.gv, pool.gtable, pool.kv_lens)
    bsa.bsa_device_status()
    assert torch.isnan(out[0, 0, 0]).all() and torch.isneginf(lse[0, 0, 0])
    assert torch.isfinite(out[0, 0, 1]).all() and torch.isfinite(lse[0, 1, 0])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("back", [False, True])
def test_pairs_without_an_axis_pass_through_bit_for_bit(inter, back):
    """Axes -1 and 3 of three: infinities, NaN and zeros of either sign go through
    as they are, as in the channels behind the pairs; in place, too."""
    B, S, H, d, pairs = 2, 5, 7, 64, 16
    x = randn((B, S, H, d), 106)
    odd = torch.tensor([float("inf"), float("nan"), -0.0, 0.0, -float("inf"), -1.5], dtype=BF)
    lo = [2 * p for p in range(pairs)] if inter else list(range(pairs))
    hi = [2 * p + 1 for p in range(pairs)] if inter else list(range(pairs, 2 * pairs))
    axes = torch.tensor([0, -1, 2, 3, 1, 5, -7, 1 << 30] * 2, dtype=torch.int32)
    free = [p for p in range(pairs) if not 0 <= int(axes[p]) < 3]
    for n, p in enumerate(free):
        x[..., lo[p]], x[..., hi[p]] = odd[n % 6], odd[(n // 6 + n + 1) % 6]
    x[0, 0, :, 2 * pairs:] = odd[1]
    pos = torch.randint(-50, 50, (B, S, 3), generator=torch.Generator().manual_seed(107), dtype=torch.int32)
    inv, _ = bsa.bsa_axis_frequencies((pairs,), device=DEV)
    call = bsa.bsa_rope_axes_backward if back else bsa.bsa_rope_axes
    y, _ = call(x.to(DEV), None, pos.to(DEV), None, inv, axes.to(DEV), interleaved=inter)
    through = [ch for p in free for ch in (lo[p], hi[p])] + list(range(2 * pairs, d))
    bits = torch.int16
    assert torch.equal(y.cpu()[..., through].view(bits), x[..., through].view(bits))
    turned = [ch for p in range(pairs) if p not in free for ch in (lo[p], hi[p])]
    ref, bound = rotate64(x, pos, inv.cpu(), axes, inter, back)
    assert ((y.double().cpu() - ref).abs() <= bound)[..., turned].all()
    mine = x.to(DEV)
    out = dict(dq_out=mine) if back else dict(q_out=mine)
    call(mine, None, pos.to(DEV), None, inv, axes.to(DEV), interleaved=inter, **out)
    assert torch.equal(mine.view(bits), y.view(bits))

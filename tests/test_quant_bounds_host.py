"""How far what the 4-bit format holds may be from what it was given, at the ends of its
range (CPU, 64-bit form; the kernels' bytes are compared with that form's elsewhere)."""

import torch

from quant_utils import SCALES, held, quantise64, values64

BF = torch.bfloat16


def group(most, n=32):
    x = torch.linspace(-1, 1, n) * most
    x[0] = most
    return x.to(BF)[None]


def test_small_groups_are_off_by_half_the_smallest_scale_and_read_as_0_below_it():
    for e in range(-40, -11):
        for f in (1.0, 1.5, 1.9921875):
            x = group(f * 2.0 ** e)
            off = (held(x).double() - x.double()).abs().max()
            assert off <= max(float(x.double().abs().max()) / 13, 2.0 ** -16)
            assert bool((held(x) == 0).all()) == (f * 2.0 ** e < 2.0 ** -16)


def test_large_groups_saturate_at_7_times_the_largest_scale():
    end = 7 * float(SCALES[-1])
    assert end == 802816.0
    for most in (7e5, 802816.0, 811008.0, 1e6, 1e20, 3e38):
        x = group(most)
        codes, byte = quantise64(x)
        y = values64(codes, byte)
        want = x.double().clamp(-end, end)
        assert (y - want).abs().max() <= SCALES[byte].max() / 2
        assert float(y.abs().max()) <= end

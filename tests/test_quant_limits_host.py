"""Limits of the attention over 4-bit pages, those of the one over bf16 pages (CPU only:
every call below fails host-side validation, so fake device pointers are never
dereferenced)."""

import ctypes

import pytest

from block_sparse_attention_bsa_gb300 import _lib, build

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


# B, T, Hq, Hkv, pages of 128 slots of a request, prefix, refused: 2^28 tiles and just below,
# with own keys, a prefix read with them and one of its own
SIZES = [
    (64, 32768, 32, 8, 1024, 0, True),
    (64, 32768, 32, 8, 1016, 0, False),
    (42, 32768, 32, 8, 512, 512 * 128, False),        # 42 x 8 x 512 x (512 + 512) + 8 x 21,504 x 512 = 264,241,152
    (43, 32768, 32, 8, 512, 512 * 128, True),
    (63, 32768, 32, 8, 512, 512 * 128, True),
    (4096, 1, 32, 8, 8191, 0, False),
    (4096, 1, 32, 8, 8192, 0, True),
    (4096, 1, 32, 8, 4095, 4000 * 128, False),
    (16, 1, 1, 1, 8000, 8000 * 128, False),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,pages,prefix,refused", SIZES)
def test_both_attentions_over_pages_take_the_same_sizes(lib, B, T, Hq, Hkv, pages, prefix, refused):
    """A workspace of 16 bytes: sizes that are taken are refused for that (3)."""
    q = _lib.BsaTensor(1 << 40, B, T, Hq, 128, T * Hq * 128, Hq * 128, 128)
    unit = 128 * Hkv * 128
    plain = [_lib.BsaTensor(p, 8192, 128, Hkv, 128, unit, Hkv * 128, 128) for p in (1 << 30, 1 << 36)]
    packed = [_lib.BsaqCache(p, 8192, Hkv, 8, 128, Hkv * 8 * 1088, 8 * 1088) for p in (1 << 30, 1 << 36)]
    for fn, caches in ((lib.bsap_forward, plain), (lib.bsaq_forward, packed)):
        st = fn(ctypes.byref(q), *map(ctypes.byref, caches), FAKE, pages, pages, FAKE, None, FAKE if prefix else None, prefix, 1,
                0.0, 1 << 45, None, 1 << 47, 16, None)
        assert st == (2 if refused else 3), lib.bsa_get_last_error().decode()


@pytest.mark.parametrize("limit", [0, 999_999, 10_000_000_001])
def test_wait_probe_refuses_limits_out_of_range(lib, limit):
    assert lib.bsaq_debug_wait_probe(limit, None) == 1
    assert lib.bsa_get_last_error().decode().startswith("bsaq_debug_wait_probe: limit_ns")

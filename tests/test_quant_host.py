"""The 4-bit format's own properties, and refusals and host logic of the 4-bit
cache's calls (CPU only: every call below fails host-side validation, so fake
device pointers are never dereferenced)."""

import ctypes
import os
import re

import pytest
import torch

import block_sparse_attention_bsa_gb300 as bsa
from block_sparse_attention_bsa_gb300 import _lib, build, quant
from quant_utils import SCALES, held, quantise64, values64, write

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000
BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def err(lib):
    return lib.bsa_get_last_error().decode()


def T(B=2, S=4, H=4, D=128, sb=None, ss=None, sh=None, ptr=FAKE):
    sh = D if sh is None else sh
    ss = H * D if ss is None else ss
    sb = S * H * D if sb is None else sb
    return _lib.BsaTensor(ptr, B, S, H, D, sb, ss, sh)


def C(pages=8, heads=2, blocks=1, D=128, sp=None, sh=None, ptr=FAKE):
    unit = blocks * 17 * D // 2
    sh = unit if sh is None else sh
    sp = heads * unit if sp is None else sp
    return _lib.BsaqCache(ptr, pages, heads, blocks, D, sp, sh)


def ref(x):
    return None if x is None else ctypes.byref(x)


# ---- the format ----

def test_scales_fill_four_bits_of_every_octave():
    assert float(SCALES[0]) == 2.0 ** -15 and float(SCALES[254]) == 1.75 * 2 ** 16
    assert (SCALES[1:] > SCALES[:-1]).all()
    assert all(float(SCALES[b]) == float(torch.tensor(float(SCALES[b])).to(BF)) for b in range(255))


def test_every_code_times_every_scale_is_exact_in_bf16():
    c = torch.arange(-7, 8).double()[:, None] * SCALES
    assert (c.to(BF).double() == c).all()


@pytest.mark.parametrize("scale", [1e-6, 1e-3, 1.0, 300.0, 1e5])
def test_what_is_held_is_within_half_a_scale(scale):
    x = (torch.randn(64, 3, 128, generator=torch.Generator().manual_seed(1)) * scale).to(BF)
    codes, byte = quantise64(x)
    y = values64(codes, byte)
    a = x.double().unflatten(-1, (-1, 32)).abs().amax(-1)
    off = (y - x.double()).unflatten(-1, (-1, 32)).abs().amax(-1)
    assert (off <= SCALES[byte] / 2).all()
    assert (off <= torch.clamp(a / 13, min=2.0 ** -16)).all()
    assert codes.abs().max() <= 7


def test_ties_go_to_the_even_scale_and_to_the_larger_code():
    x = torch.zeros(1, 32, dtype=BF)
    x[0, 0] = 7 * 1.0625                                  # half way between scales of 1 (byte 120) and 1.125 (121)
    assert int(quantise64(x)[1]) == 120
    x[0, 0] = 7 * 1.1875                                  # 1.125 and 1.25
    assert int(quantise64(x)[1]) == 122
    x[0, 0] = 7.0
    x[0, 1:5] = torch.tensor([0.5, -0.5, 2.5, 0.498046875])
    assert quantise64(x)[0][0, :5].tolist() == [7, 1, -1, 3, 0]


def test_a_group_that_is_not_finite_reads_as_nan_and_its_neighbours_do_not():
    x = torch.ones(1, 64, dtype=BF)
    x[0, 3] = float("inf")
    y = held(x)
    # 1/7 lies between the scales 9/64 and 10/64, nearer the first; 7 * 9/64 = 63/64
    assert torch.isnan(y[0, :32]).all() and (y[0, 32:] == 63 / 64).all()


def test_writing_keeps_what_other_slots_hold():
    g = torch.Generator().manual_seed(2)
    for channels_first in (False, True):
        whole = torch.zeros(4, 2, 2, 17 * 64 // 2, dtype=torch.uint8)
        parts = whole.clone()
        table = torch.tensor([2, 0, 3])
        x = torch.randn(90, 2, 64, generator=g).to(BF)
        write(whole, table, 0, x, channels_first)
        for a, z in ((0, 5), (5, 37), (37, 38), (38, 90)):
            write(parts, table, a, x[a:z], channels_first)
        assert torch.equal(whole, parts)


# ---- host checks ----

def test_header_signatures_and_exports_agree(lib):
    import subprocess
    txt = open(os.path.join(ROOT, "include", "bsa_quant.h")).read()
    declared = sorted(set(re.findall(r"BSA_API\s+[\w\s\*]+?\b(bsaq_\w+)\s*\(", txt)))
    assert declared == sorted(_lib.QUANT_SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.lib_path()], capture_output=True, text=True).stdout
    assert declared == sorted({x.split()[-1] for x in out.splitlines() if x.split() and x.split()[-1].startswith("bsaq_")})


def test_shape_of_a_cache():
    assert bsa.bsa_cache_q4_shape(10, 64, 8, 128) == (10, 8, 4, 1088)
    assert bsa.bsa_cache_q4_shape(1, 16, 3, 64) == (1, 3, 1, 544)
    for bad in ((1, 24, 8, 128), (1, 512, 8, 128), (1, 64, 8, 96)):
        with pytest.raises(ValueError):
            bsa.bsa_cache_q4_shape(*bad)


CACHE_REFUSALS = [
    (dict(kc=None), 1, "k_cache descriptor is NULL"),
    (dict(vc=None), 1, "v_cache descriptor is NULL"),
    (dict(kc=C(ptr=None)), 1, "k_cache->ptr is NULL"),
    (dict(kc=C(pages=0)), 1, "non-positive size"),
    (dict(vc=C(blocks=-1)), 1, "non-positive size"),
    (dict(kc=C(D=96)), 2, "head dim 96"),
    (dict(kc=C(heads=257)), 2, "257 heads"),
    (dict(kc=C(blocks=3)), 2, "page size 48"),
    (dict(kc=C(blocks=32)), 2, "page size 512"),
    (dict(kc=C(pages=1 << 27)), 2, "2^30 slots"),
    (dict(kc=C(ptr=FAKE + 8)), 1, "16-byte aligned"),
    (dict(kc=C(sh=1096)), 1, "multiples of 16"),
    (dict(kc=C(sp=-2176)), 1, "positive multiples"),
    (dict(kc=C(sp=1088)), 1, "blocks overlap"),
    (dict(kc=C(sh=1072)), 1, "blocks overlap"),
    (dict(kc=C(sp=1088, sh=7 * 1088)), 1, "blocks overlap"),
    (dict(kc=C(sp=0)), 1, "blocks overlap"),
    (dict(vc=C(pages=9, ptr=1 << 24)), 1, "v_cache shape"),
    (dict(vc=C(D=64, ptr=1 << 24)), 1, "v_cache shape"),
    (dict(table=None), 1, "page_table and kv_lens"),
    (dict(lens=None), 1, "page_table and kv_lens"),
    (dict(stride=3), 1, "table_stride 3"),
    (dict(pages=-1), 1, "max_pages -1"),
    (dict(pages=1 << 27), 1, "max_pages"),
    (dict(table=FAKE + 2), 1, "page_table is not 4-byte aligned"),
    (dict(lens=FAKE + 1), 1, "kv_lens is not 4-byte aligned"),
]
ROWS_REFUSALS = [
    (dict(k=None), 1, "descriptor is NULL"),
    (dict(k=T(H=2, D=96)), 2, "head dim 96"),
    (dict(v=T(H=2, S=5, ptr=1 << 28)), 1, "shape differs"),
    (dict(k=T(H=2, ptr=FAKE + 8)), 1, "16-byte aligned"),
    (dict(k=T(H=2, ss=260)), 1, "multiples of 8"),
    (dict(k=T(H=3, ptr=1 << 27), v=T(H=3, ptr=1 << 28)), 1, "the cache has 2 heads"),
    (dict(k=T(B=4097, S=1, H=2, ptr=1 << 27), v=T(B=4097, S=1, H=2, ptr=1 << 28)), 2, "batch 4097"),
    (dict(pages=0), 1, "max_pages is 0"),
    (dict(k=T(H=2, ptr=1 << 24)), 1, "k_cache shares memory"),
    (dict(v=T(H=2, ptr=(1 << 25) + 16)), 1, "v_cache shares memory"),
]


def rows_args(change, written):
    a = dict(k=T(H=2, ptr=1 << 27), v=T(H=2, ptr=1 << 28), kc=C(ptr=1 << 24), vc=C(ptr=1 << 25), table=FAKE, stride=8, pages=8,
             lens=FAKE, other=None)
    a.update(change)
    pages = (ref(a["kc"]), ref(a["vc"]), a["table"], a["stride"], a["pages"], a["lens"], a["other"])
    rows = (ref(a["k"]), ref(a["v"]))
    return (*pages, *rows, None) if written else (*rows, *pages, None)


@pytest.mark.parametrize("change,status,needle", CACHE_REFUSALS + ROWS_REFUSALS)
@pytest.mark.parametrize("name", ["bsaq_cache_append", "bsaq_cache_read"])
def test_append_and_read_refuse(lib, name, change, status, needle):
    st = getattr(lib, name)(*rows_args(change, name == "bsaq_cache_read"))
    assert st == status and needle in err(lib) and err(lib).startswith(name + ": "), err(lib)


def test_refusals_of_one_call_only(lib):
    assert lib.bsaq_cache_append(*rows_args(dict(vc=C(ptr=1 << 24)), False)) == 1 and "v_cache shares memory" in err(lib)
    assert lib.bsaq_cache_append(*rows_args(dict(other=FAKE + 2), False)) == 1 and "new_lens is not 4-byte" in err(lib)
    assert lib.bsaq_cache_read(*rows_args(dict(other=FAKE + 2), True)) == 1 and "first is not 4-byte" in err(lib)
    assert lib.bsaq_cache_read(*rows_args(dict(v=T(H=2, ptr=(1 << 27) + 512)), True)) == 1
    assert "v_out shares memory with k_out" in err(lib)
    assert lib.bsaq_cache_read(*rows_args(dict(k=T(H=2, sb=0, ptr=1 << 27)), True)) == 1 and "strides" in err(lib)


FORWARD_REFUSALS = [
    (dict(q=None), 1, "q descriptor is NULL"),
    (dict(q=T(D=64)), 1, "head dim of q (64)"),
    (dict(q=T(H=3)), 1, "not a multiple of Hkv"),
    (dict(q=T(B=1 << 20, S=1)), 2, "batch 1048576"),
    (dict(q=T(B=4096, S=1 << 16)), 2, "too many for one call"),
    (dict(new=FAKE + 2), 1, "new_lens is not 4-byte aligned"),
    (dict(plen=-1), 1, "prefix_len -1"),
    (dict(plen=1 << 30), 1, "out of range"),
    (dict(plen=5), 1, "prefix_table is NULL"),
    (dict(plen=5, shared=FAKE + 2), 1, "prefix_table is not 4-byte aligned"),
    (dict(out=None), 1, "out is NULL"),
    (dict(out=FAKE + 8), 1, "out is not 16-byte aligned"),
    (dict(lse=FAKE + 2), 1, "lse is not 4-byte aligned"),
    (dict(scale=float("nan")), 1, "softmax_scale is not finite"),
    (dict(scale=float("inf")), 1, "softmax_scale is not finite"),
    (dict(scale=1e-40), 1, "subnormal"),
    (dict(scale=3e38), 1, "half the largest"),
    (dict(ws=None), 3, "workspace is NULL"),
    (dict(ws_bytes=16), 3, "smaller than"),
    (dict(ws=FAKE + 128), 3, "256-byte aligned"),
]


def call_forward(lib, change):
    a = dict(q=T(ptr=1 << 26), kc=C(ptr=1 << 24), vc=C(ptr=1 << 25), table=FAKE, stride=8, pages=8, lens=FAKE, new=None,
             shared=None, plen=0, causal=1, scale=0.0, out=1 << 27, lse=None, ws=1 << 28, ws_bytes=1 << 40)
    a.update(change)
    return lib.bsaq_forward(ref(a["q"]), ref(a["kc"]), ref(a["vc"]), a["table"], a["stride"], a["pages"], a["lens"], a["new"],
                            a["shared"], a["plen"], a["causal"], a["scale"], a["out"], a["lse"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("change,status,needle", CACHE_REFUSALS + FORWARD_REFUSALS)
def test_forward_refuses(lib, change, status, needle):
    st = call_forward(lib, change)
    assert st == status and needle in err(lib) and err(lib).startswith("bsaq_forward: "), err(lib)


@pytest.mark.parametrize("change,needle", [
    (dict(out=(1 << 26) + 4096), "out shares memory with q"),
    (dict(out=(1 << 24) + 16), "out shares memory with k_cache"),
    (dict(out=(1 << 25) - 16), "out shares memory with v_cache"),
    (dict(lse=(1 << 27) + 64), "lse shares memory with out"),
    (dict(lse=FAKE + 4), "lse shares memory with page_table"),
    (dict(out=FAKE - 4096, lens=1 << 20), "out shares memory with page_table"),
    (dict(ws=1 << 26), "workspace shares memory with q"),
    (dict(ws=1 << 27), "workspace shares memory with out"),
    (dict(new=1 << 28), "workspace shares memory with new_lens"),
    (dict(plen=20, shared=1 << 28), "workspace shares memory with prefix_table"),
])
def test_forward_refuses_results_in_what_it_reads_or_in_one_another(lib, change, needle):
    assert call_forward(lib, change) == 1 and needle in err(lib), err(lib)


def test_forward_workspace_size(lib):
    size = bsa.bsa_forward_paged_q4_workspace_size
    assert size(2, 1, 8, 2, 128, False, 152) > 0
    for bad in ((0, 1, 8, 2, 128), (2, 0, 8, 2, 128), (2, 1, 7, 2, 128), (2, 1, 8, 2, 96), (4097, 1, 8, 2, 128),
                (2, 1, 512, 2, 128), (4096, 1 << 18, 32, 1, 128)):
        assert size(*bad, False, 152) == 0


def test_binding_refusals():
    x, c = torch.zeros(1, 1, 4, 64, dtype=BF), torch.zeros(2, 2, 1, 544, dtype=torch.uint8)
    ints = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        bsa.bsa_forward_paged_q4(x, c, c, ints[None], ints)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        bsa.bsa_cache_append_q4(x, x, c, c, ints[None], ints)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        bsa.bsa_cache_read_q4(c, c, ints[None], ints, 5)
    for scale in (5e-324, 1e-40):
        with pytest.raises(ValueError, match="softmax_scale"):
            bsa.bsa_forward_paged_q4(x, c, c, ints[None], ints, softmax_scale=scale)
    with pytest.raises(ValueError, match="prefix_len"):
        bsa.bsa_forward_paged_q4(x, c, c, ints[None], ints, prefix_len=1 << 32)
    with pytest.raises(TypeError, match="workspace must be a torch.Tensor"):
        quant._forward_launch(x, c, c, (), torch.zeros_like(x), None, False, bytearray(256), 0)

"""Refusals and host logic of the position, cache and paged-attention calls
(CPU only: every call below fails host-side validation, so fake device
pointers are never dereferenced)."""

import ctypes
import os
import re

import pytest
import torch

import block_sparse_attention_bsa_gb300 as bsa
from block_sparse_attention_bsa_gb300 import _lib, build, paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000


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


def R(pairs=64, n_axes=3, inv=FAKE, axes=FAKE):
    return _lib.BsapRope(inv, axes, pairs, n_axes, 0)


def P(ptr=FAKE, sb=12, ss=3, sa=1):
    return _lib.BsapPositions(ptr, sb, ss, sa)


def ref(x):
    return None if x is None else ctypes.byref(x)


def test_header_signatures_and_exports_agree(lib):
    import subprocess
    txt = open(os.path.join(ROOT, "include", "bsa_paged.h")).read()
    declared = sorted(set(re.findall(r"BSA_API\s+[\w\s\*]+?\b(bsap_\w+)\s*\(", txt)))
    assert declared == sorted(_lib.PAGED_SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.lib_path()], capture_output=True, text=True).stdout
    assert declared == sorted({x.split()[-1] for x in out.splitlines() if x.split() and x.split()[-1].startswith("bsap_")})


ROPE_REFUSALS = [
    (dict(q=None), 1, "q descriptor is NULL"),
    (dict(q=T(D=96)), 2, "head dim 96"),
    (dict(q=T(ptr=FAKE + 2)), 1, "16-byte aligned"),
    (dict(q=T(ss=516)), 1, "multiples of 8"),
    (dict(q=T(sb=-8)), 1, "not be negative"),
    (dict(q=T(H=257)), 2, "257 heads"),
    (dict(q=T(S=0)), 1, "non-positive dim"),
    (dict(q=T(B=1 << 20, S=1 << 11)), 2, "2^30 rows"),
    (dict(k=T(D=64)), 1, "head dim of q"),
    (dict(pos_q=None), 1, "pos_q is NULL"),
    (dict(pos_q=P(ptr=None)), 1, "pos_q is NULL"),
    (dict(pos_k=None), 1, "pos_k is NULL"),
    (dict(pos_k=P(ss=-1)), 1, "pos_k strides"),
    (dict(rope=None), 1, "rope is NULL"),
    (dict(rope=R(inv=None)), 1, "inv_freq and axes"),
    (dict(rope=R(inv=FAKE + 4)), 1, "8-byte aligned"),
    (dict(rope=R(pairs=72)), 1, "72 pairs"),
    (dict(rope=R(pairs=0)), 1, "0 pairs"),
    (dict(rope=R(pairs=20)), 2, "not a multiple of 8"),
    (dict(rope=R(n_axes=5)), 2, "n_axes 5"),
    (dict(rope=R(n_axes=0)), 2, "n_axes 0"),
    (dict(q_out=None), 1, "q_out is NULL"),
    (dict(k_out=FAKE + 8), 1, "k_out is not 16-byte aligned"),
]


@pytest.mark.parametrize("change,status,needle", ROPE_REFUSALS)
def test_rope_refusals(lib, change, status, needle):
    a = dict(q=T(), k=T(H=2), pos_q=P(), pos_k=P(), rope=R(), q_out=FAKE, k_out=FAKE)
    a.update(change)
    st = lib.bsap_rope_axes(ref(a["q"]), ref(a["k"]), ref(a["pos_q"]), ref(a["pos_k"]), ref(a["rope"]), 0, a["q_out"],
                            a["k_out"], None)
    assert st == status and needle in err(lib) and err(lib).startswith("bsap_rope_axes: "), err(lib)


CACHE = T(B=10, S=64, H=2, D=128)
APPEND_REFUSALS = [
    (dict(k=None), 1, "k descriptor is NULL"),
    (dict(v=T(H=4)), 1, "v shape differs"),
    (dict(kc=T(B=10, S=48, H=2), vc=T(B=10, S=48, H=2)), 2, "page size 48"),
    (dict(vc=T(B=9, S=64, H=2)), 1, "v_cache shape differs"),
    (dict(kc=T(B=10, S=64, H=3), vc=T(B=10, S=64, H=3)), 1, "the cache has 3 heads"),
    (dict(kc=T(B=10, S=64, H=2, sb=0)), 1, "strides must be positive"),
    (dict(kc=T(B=10, S=64, H=2, sb=64)), 1, "slots overlap"),
    (dict(table=None), 1, "page_table and kv_lens"),
    (dict(lens=None), 1, "page_table and kv_lens"),
    (dict(stride=4), 1, "table_stride 4"),
    (dict(pages=-1), 1, "max_pages -1"),
    (dict(pages=0), 1, "max_pages is 0"),
    (dict(pages=1 << 28, stride=1 << 28), 1, "out of range"),
    (dict(k=T(B=4097, H=2), v=T(B=4097, H=2)), 2, "batch 4097"),
    (dict(rope=None, pos=None), 1, "q is given without rope"),
    (dict(pos=None), 1, "pos is NULL"),
    (dict(rope=R(pairs=65)), 1, "65 pairs"),
    (dict(q=T(S=5, H=4)), 1, "q's batch, length or head dim"),
    (dict(q_out=None), 1, "q_out is NULL"),
]


@pytest.mark.parametrize("change,status,needle", APPEND_REFUSALS)
def test_append_refusals(lib, change, status, needle):
    a = dict(k=T(H=2), v=T(H=2), kc=CACHE, vc=CACHE, table=FAKE, stride=8, pages=8, lens=FAKE, new=None, rope=R(), pos=P(),
             q=T(H=4), q_out=FAKE)
    a.update(change)
    st = lib.bsap_cache_append(ref(a["k"]), ref(a["v"]), ref(a["kc"]), ref(a["vc"]), a["table"], a["stride"], a["pages"],
                               a["lens"], a["new"], ref(a["rope"]), ref(a["pos"]), ref(a["q"]), a["q_out"], None)
    assert st == status and needle in err(lib) and err(lib).startswith("bsap_cache_append: "), err(lib)


FORWARD_REFUSALS = [
    (dict(q=None), 1, "q descriptor is NULL"),
    (dict(q=T(D=64)), 1, "head dim of q (64)"),
    (dict(q=T(H=3)), 1, "not a multiple of Hkv"),
    (dict(kc=T(B=10, S=512, H=2), vc=T(B=10, S=512, H=2)), 2, "page size 512"),
    (dict(prefix=-1), 1, "prefix_len -1"),
    (dict(prefix=5, shared=None), 1, "prefix_table is NULL"),
    (dict(out=None), 1, "out is NULL"),
    (dict(out=FAKE + 8), 1, "out is not 16-byte aligned"),
    (dict(scale=float("inf")), 1, "softmax_scale"),
    (dict(lens=None), 1, "page_table and kv_lens"),
    (dict(ws=None), 3, "workspace is NULL"),
    (dict(ws_bytes=8), 3, "smaller than"),
    (dict(ws=FAKE + 128), 3, "256-byte aligned"),
]


@pytest.mark.parametrize("change,status,needle", FORWARD_REFUSALS)
def test_forward_refusals(lib, change, status, needle):
    a = dict(q=T(), kc=CACHE, vc=CACHE, table=FAKE, stride=8, pages=8, lens=FAKE, new=None, shared=FAKE, prefix=100, scale=0.0,
             out=FAKE, ws=FAKE, ws_bytes=1 << 40)
    a.update(change)
    st = lib.bsap_forward(ref(a["q"]), ref(a["kc"]), ref(a["vc"]), a["table"], a["stride"], a["pages"], a["lens"], a["new"],
                          a["shared"], a["prefix"], 1, a["scale"], a["out"], None, a["ws"], a["ws_bytes"], None)
    assert st == status and needle in err(lib) and err(lib).startswith("bsap_forward: "), err(lib)


def test_binding_refuses_cpu_tensors_and_wrong_types():
    q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    pos = torch.zeros(1, 3, dtype=torch.int32)
    inv, axes = bsa.bsa_axis_frequencies((8, 8, 8), device="cpu")
    cpu = q.get_device()                      # -1: the checks below are the ones that follow the first tensor's
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        bsa.bsa_rope_axes(q, None, pos, None, inv, axes)
    with pytest.raises(ValueError, match="k must be a CUDA tensor"):
        bsa.bsa_cache_append(q, q, q, q, pos, pos)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        bsa.bsa_forward_paged(q, q, q, pos, pos)
    with pytest.raises(TypeError, match="q must be a torch.Tensor"):
        bsa.bsa_forward_paged(None, q, q, pos, pos)
    with pytest.raises(ValueError, match="CUDA tensor"):
        paged._tensor(q, "q", cpu)
    with pytest.raises(ValueError, match="the call's first tensor on device 0"):
        paged._tensor(q, "v", 0)
    with pytest.raises(TypeError, match="inv_freq"):
        paged._rope(None, axes, 3, False, cpu)
    with pytest.raises(ValueError, match="float64"):
        paged._rope(inv.float(), axes, 3, False, cpu)
    with pytest.raises(ValueError, match="24 pairs, axes 23"):
        paged._rope(inv, axes[:23], 3, False, cpu)
    with pytest.raises(ValueError, match="int32"):
        paged._positions(pos.long(), "pos_q", cpu, 1, 1)
    with pytest.raises(ValueError, match="B = 1, S = 2"):
        paged._positions(pos, "pos_q", cpu, 1, 2)
    with pytest.raises(ValueError, match="kv_lens"):
        paged._ints(pos, "kv_lens", cpu, 1)
    with pytest.raises(ValueError, match="kv_lens"):
        paged._ints(torch.zeros(8, dtype=torch.int32)[::2], "kv_lens", cpu, 4)
    with pytest.raises(ValueError, match="contiguous last dim"):
        paged._table(torch.zeros(4, 3, dtype=torch.int32).t(), 3, cpu)
    with pytest.raises(ValueError, match="page_table must be"):
        paged._table(torch.zeros(4, 3, dtype=torch.int32), 3, cpu)


def test_overlap_check():
    flat = torch.zeros(1000, dtype=torch.bfloat16)
    a, b = flat[:512].view(1, 2, 4, 64), flat[488:].view(1, 2, 4, 64)
    with pytest.raises(ValueError, match="overlaps"):
        paged._check_overlap("out", a, (b,), b)
    paged._check_overlap("out", a, (a,), a)
    with pytest.raises(ValueError, match="overlaps"):
        paged._check_overlap("out", a, (a,), None)
    wide = flat[:512].view(1, 1, 8, 64)
    with pytest.raises(ValueError, match="overlaps"):
        paged._check_overlap("out", flat[:256].view(1, 1, 4, 64), (wide[:, :, ::2],), wide)


def test_overlap_check_of_one_tensor_as_two_inputs():
    x, y = (torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16) for _ in range(2))
    with pytest.raises(ValueError, match="overlaps"):
        paged._check_overlap("q_out", x, (x, x), x)
    with pytest.raises(ValueError, match="overlaps"):
        paged._check_overlap("k_out", x, (x, x, y), x)
    paged._check_overlap("k_out", y, (x, x), x)


@pytest.mark.parametrize("scale", [1e-40, 3e38, float("nan")])
def test_attention_refuses_scales_out_of_range(lib, scale):
    st = lib.bsap_forward(ref(T()), ref(CACHE), ref(CACHE), FAKE, 8, 8, FAKE, None, None, 0, 1, scale, FAKE, None, FAKE,
                          1 << 40, None)
    assert st == 1 and "softmax_scale" in err(lib)


# q 2 x 4 x 4 heads of 128 (8,192 bytes), k half of it; where the outputs lie
@pytest.mark.parametrize("q,k,qo,ko,needle", [
    (0, 1 << 16, 256, 1 << 17, "q_out shares memory with q"),
    (0, 1 << 16, 8192 - 16, 1 << 17, "q_out shares memory with q"),
    (0, 0, 0, 1 << 17, "q_out shares memory with k"),
    (0, 0, 1 << 17, 0, "k_out shares memory with q"),
    (0, 8192, 1 << 16, 8192 + 16, "k_out shares memory with k"),
    (0, 1 << 16, 1 << 17, (1 << 17) + 8192 - 16, "k_out shares memory with q_out"),
])
def test_rotation_refuses_shared_memory(lib, q, k, qo, ko, needle):
    st = lib.bsap_rope_axes(ref(T(ptr=FAKE + q)), ref(T(H=2, ptr=FAKE + k)), ref(P()), ref(P()), ref(R()), 0,
                            FAKE + qo, FAKE + ko, None)
    assert st == 1 and needle in err(lib)


def test_rotation_in_place_takes_contiguous_inputs_only(lib):
    st = lib.bsap_rope_axes(ref(T(ss=1024, sb=4096)), None, ref(P()), None, ref(R()), 0, FAKE, None, None)
    assert st == 1 and "q_out shares memory with q" in err(lib)


# caches of 8 pages of 16 slots, 2 heads of 128: 65,536 bytes
@pytest.mark.parametrize("change,needle", [
    (dict(vc=0), "v_cache shares memory with k_cache"),
    (dict(k=256), "k_cache shares memory with k"),
    (dict(v=(1 << 20) + 65536 - 16), "v_cache shares memory with v"),
    (dict(q=65536 - 16), "k_cache shares memory with q"),
    (dict(qo=1 << 20), "v_cache shares memory with q_out"),
    (dict(qo=(2 << 20) + 16), "q_out shares memory with k"),
    (dict(qo=3 << 20), "q_out shares memory with v"),
    (dict(qo=(4 << 20) + 16), "q_out shares memory with q"),
])
def test_append_refuses_shared_memory(lib, change, needle):
    at = dict(kc=0, vc=1 << 20, k=2 << 20, v=3 << 20, q=4 << 20, qo=5 << 20)
    at.update(change)
    at = {name: FAKE + x for name, x in at.items()}
    st = lib.bsap_cache_append(ref(T(H=2, ptr=at["k"])), ref(T(H=2, ptr=at["v"])),
                               ref(T(B=8, S=16, H=2, ptr=at["kc"])), ref(T(B=8, S=16, H=2, ptr=at["vc"])), FAKE, 4, 4,
                               FAKE, None, ref(R()), ref(P()), ref(T(ptr=at["q"])), at["qo"], None)
    assert st == 1 and needle in err(lib)


@pytest.mark.parametrize("out,needle", [(4 << 20, "out shares memory with q"), (65536 - 16, "out shares memory with k_cache"),
                                        ((1 << 20) + 256, "out shares memory with v_cache")])
def test_attention_refuses_an_output_in_its_inputs(lib, out, needle):
    st = lib.bsap_forward(ref(T(ptr=FAKE + (4 << 20))), ref(T(B=8, S=16, H=2)), ref(T(B=8, S=16, H=2, ptr=FAKE + (1 << 20))),
                          FAKE, 4, 4, FAKE, None, None, 0, 1, 0.0, FAKE + out, None, FAKE, 1 << 40, None)
    assert st == 1 and needle in err(lib)


@pytest.mark.parametrize("prefix_len", [-1, 1 << 31, (1 << 32) + 5])
def test_binding_refuses_prefix_lengths_that_do_not_fit(prefix_len):
    x = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="prefix_len"):
        bsa.bsa_forward_paged(x, x, x, x, x, prefix_len=prefix_len)


def test_axis_frequencies():
    inv, axes = bsa.bsa_axis_frequencies((2, 3, 3), 100.0, device="cpu")
    assert axes.tolist() == [0, 0, 1, 1, 1, 2, 2, 2]
    assert inv.dtype == torch.float64 and torch.allclose(inv, 100.0 ** (-torch.arange(8, dtype=torch.float64) / 8))
    inv, axes = bsa.bsa_axis_frequencies((2, 3, 3), 100.0, "cycled", "cpu")
    assert axes.tolist() == [0, 1, 2, 0, 1, 2, 1, 2]
    inv, axes = bsa.bsa_axis_frequencies((1, 3), 100.0, "per_axis", "cpu")
    assert axes.tolist() == [0, 1, 1, 1]
    assert inv.tolist() == [1.0, 1.0, 100.0 ** (-1 / 3), 100.0 ** (-2 / 3)]
    for bad in ((), (1, 2, 3, 4, 5), (-1, 4), (0, 0)):
        with pytest.raises(ValueError, match="sections"):
            bsa.bsa_axis_frequencies(bad, device="cpu")
    with pytest.raises(ValueError, match="layout"):
        bsa.bsa_axis_frequencies((8,), layout="rows", device="cpu")


def test_workspace_size_refuses_what_the_call_refuses(lib):
    f = bsa.bsa_forward_paged_workspace_size
    assert f(1, 1, 32, 8, 128, True, 152) > 0
    for bad in ((0, 1, 32, 8, 128), (1, 0, 32, 8, 128), (1, 1, 30, 8, 128), (1, 1, 32, 8, 96), (4097, 1, 32, 8, 128)):
        assert f(*bad, True, 152) == 0


@pytest.mark.parametrize("limit", [999_999, 10 ** 10 + 1])
def test_wait_probe_refuses_limits_out_of_range(lib, limit):
    assert lib.bsap_debug_wait_probe(limit, None) == 1
    assert err(lib).startswith("bsap_debug_wait_probe: limit_ns")


# q, out 4,096 values each; caches of 8 pages of 16 slots, 2 heads of 128; lse 2 x 4 x 4 floats; tables of 2 x 4 pages;
# a workspace of megabytes, by the number of SMs (one is assumed where there is no GPU): 16 MB for each
@pytest.mark.parametrize("change,needle", [
    (dict(lse=(4 << 24) + 8192 - 4), "lse shares memory with q"),
    (dict(lse=65536 - 64), "lse shares memory with k_cache"),
    (dict(lse=1 << 24), "lse shares memory with v_cache"),
    (dict(lse=(5 << 24) + 128), "lse shares memory with out"),
    (dict(lse=(8 << 24) + 4), "lse shares memory with kv_lens"),
    (dict(lse=(9 << 24) + 28), "lse shares memory with page_table"),
    (dict(ws=4 << 24), "workspace shares memory with q"),
    (dict(ws=65536 - 256), "workspace shares memory with k_cache"),
    (dict(ws=(1 << 24) + 256), "workspace shares memory with v_cache"),
    (dict(ws=5 << 24), "workspace shares memory with out"),
    (dict(ws=(6 << 24) - 256), "workspace shares memory with lse"),
    (dict(new=(7 << 24) + 4), "workspace shares memory with new_lens"),
    (dict(shared=(7 << 24) + 64), "workspace shares memory with prefix_table"),
    (dict(out=9 << 24), "out shares memory with page_table"),
])
def test_attention_refuses_results_and_workspaces_in_what_it_reads_or_in_one_another(lib, change, needle):
    at = dict(kc=0, vc=1, q=4, out=5, lse=6, ws=7, lens=8, table=9, new=10, shared=11)
    at = {name: x << 24 for name, x in at.items()}
    at.update(change)
    at = {name: FAKE + x for name, x in at.items()}
    need = lib.bsap_forward_workspace_size(2, 4, 4, 2, 128, 1, 0)
    assert 512 < need < 1 << 24
    st = lib.bsap_forward(ref(T(ptr=at["q"])), ref(T(B=8, S=16, H=2, ptr=at["kc"])), ref(T(B=8, S=16, H=2, ptr=at["vc"])),
                          at["table"], 4, 4, at["lens"], at["new"], at["shared"], 33, 1, 0.0, at["out"], at["lse"], at["ws"],
                          need, None)
    assert st == 1 and needle in err(lib), err(lib)


@pytest.mark.parametrize("name", ["page_table", "kv_lens", "new_lens", "prefix_table", "lse"])
def test_attention_refuses_misaligned_arrays(lib, name):
    at = {n: FAKE * (i + 2) + (2 if n == name else 0)
          for i, n in enumerate(("page_table", "kv_lens", "new_lens", "prefix_table", "lse"))}
    st = lib.bsap_forward(ref(T(ptr=1 << 30)), ref(T(B=8, S=16, H=2, ptr=1 << 31)), ref(T(B=8, S=16, H=2, ptr=1 << 32)),
                          at["page_table"], 4, 4, at["kv_lens"], at["new_lens"], at["prefix_table"], 33, 1, 0.0, 1 << 33,
                          at["lse"], 1 << 34, 1 << 30, None)
    assert st == 1 and f"{name} is not 4-byte aligned" in err(lib)


@pytest.mark.parametrize("name", ["page_table", "kv_lens", "new_lens", "axes", "pos"])
def test_append_refuses_misaligned_arrays(lib, name):
    at = {n: FAKE * (i + 2) + (1 if n == name else 0)
          for i, n in enumerate(("page_table", "kv_lens", "new_lens", "axes", "pos"))}
    st = lib.bsap_cache_append(ref(T(H=2, ptr=1 << 30)), ref(T(H=2, ptr=1 << 31)), ref(T(B=8, S=16, H=2, ptr=1 << 32)),
                               ref(T(B=8, S=16, H=2, ptr=1 << 33)), at["page_table"], 4, 4, at["kv_lens"], at["new_lens"],
                               ref(R(axes=at["axes"])), ref(P(ptr=at["pos"])), None, None, None)
    assert st == 1 and f"{name} is not 4-byte aligned" in err(lib)


@pytest.mark.parametrize("change,needle", [(dict(pos_q=P(ptr=FAKE + 2)), "pos_q"), (dict(pos_k=P(ptr=FAKE + 3)), "pos_k"),
                                           (dict(rope=R(axes=FAKE + 2)), "axes")])
def test_rotation_refuses_misaligned_arrays(lib, change, needle):
    a = dict(pos_q=P(), pos_k=P(), rope=R())
    a.update(change)
    st = lib.bsap_rope_axes(ref(T()), ref(T(H=2, ptr=1 << 20)), ref(a["pos_q"]), ref(a["pos_k"]), ref(a["rope"]), 0, 1 << 21,
                            1 << 22, None)
    assert st == 1 and f"{needle} is not 4-byte aligned" in err(lib)


@pytest.mark.parametrize("scale", [5e-324, 1e-300, 1e-46, 1e-40])
def test_binding_refuses_scales_that_round_to_zero(scale):
    """0 selects d^-1/2; a scale that a float cannot hold must not."""
    x = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="softmax_scale"):
        bsa.bsa_forward_paged(x, x, x, x, x, softmax_scale=scale)


def test_binding_refuses_a_workspace_that_is_no_tensor(lib):
    q, out = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="workspace must be a torch.Tensor"):
        paged._forward_launch(q, q, q, (), out, None, False, bytearray(256), 0)

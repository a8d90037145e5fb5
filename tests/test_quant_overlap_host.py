"""Append and read of the 4-bit cache refuse tables and lengths that lie in what they
write (CPU only: every call fails host-side validation, so fake device pointers are never
dereferenced)."""

import ctypes

import pytest

from block_sparse_attention_bsa_gb300 import _lib, build

ROWS, CACHES = (1 << 27, 1 << 28), (1 << 24, 1 << 25)


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def call(lib, written, table, lens, other):
    """An append or a read (``written``) of 2 requests of 4 rows, 2 heads of 128, tables of 8 pages."""
    rows = [ctypes.byref(_lib.BsaTensor(p, 2, 4, 2, 128, 1024, 256, 128)) for p in ROWS]
    caches = [ctypes.byref(_lib.BsaqCache(p, 8, 2, 1, 128, 2176, 1088)) for p in CACHES]
    pages = (*caches, table, 8, 8, lens, other)
    fn = lib.bsaq_cache_read if written else lib.bsaq_cache_append
    st = fn(*pages, *rows, None) if written else fn(*rows, *pages, None)
    return st, lib.bsa_get_last_error().decode()


@pytest.mark.parametrize("written", [False, True])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("name", ["table", "lens", "other"])
def test_tables_and_lengths_inside_what_is_written_are_refused(lib, written, which, name):
    at = (ROWS if written else CACHES)[which]
    size = 2 * 4 * 2 * 256 if written else 8 * 2 * 1088
    label = {"table": "page_table", "lens": "kv_lens", "other": "first" if written else "new_lens"}[name]
    out = (("k_out", "v_out") if written else ("k_cache", "v_cache"))[which]
    own = 64 if name == "table" else 8
    for p in (at, at + size - 4, at - own + 4):
        args = dict(table=1 << 16, lens=1 << 17, other=1 << 18)
        args[name] = p
        st, msg = call(lib, written, **args)
        assert st == 1 and out in msg and label in msg and "shares memory" in msg, msg

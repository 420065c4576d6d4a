"""Argument checks of the paged-store calls (no GPU needed: every call here
fails validation before anything would be launched, or has nothing to do)."""

import ctypes

import pytest

import sparse_dictionary_coded_b200 as sdk


def _at(k):
    """Distinct, well-aligned addresses that are never dereferenced."""
    return ctypes.c_void_p((1 << 32) * (k + 1))


OFF = ctypes.c_void_p((1 << 40) + 2)


@pytest.fixture(scope="module")
def lib():
    return sdk.load()


def _call(fn, base, kw):
    a = dict(base)
    assert set(kw) <= set(a)
    a.update(kw)
    return fn(*a.values(), None)


TABLES = dict(lens=_at(0), n_new=_at(1), B=4, free=_at(2), n_stack=100, n_free=_at(3), n_pages=100,
              page_size=16, table=_at(4), max_pages=10, max_new=64, slots=_at(5), cu=_at(6),
              new_lens=_at(7), n_free_out=_at(8), ws=_at(9), ws_bytes=0)


@pytest.mark.parametrize("kw,status", [
    ({}, 3),                                   # every check passes but the workspace's size
    (dict(B=0), 1), (dict(B=4097), 1), (dict(B=-1), 1), (dict(max_pages=0), 1),
    (dict(max_new=0), 1), (dict(max_new=1 << 31), 1), (dict(page_size=0), 1),
    (dict(page_size=65537), 1), (dict(n_pages=0), 1), (dict(n_stack=0), 1),
    (dict(n_pages=1 << 20, page_size=4096), 1),
    (dict(lens=None), 1), (dict(n_new=None), 1), (dict(free=None), 1), (dict(n_free=None), 1),
    (dict(table=None), 1), (dict(slots=None), 1), (dict(cu=None), 1), (dict(new_lens=None), 1),
    (dict(n_free_out=None), 1), (dict(ws=None), 1), (dict(ws=OFF), 1), (dict(lens=OFF), 1),
    (dict(slots=ctypes.c_void_p((1 << 40) + 4)), 1),
    (dict(new_lens=_at(0)), 1),                # outputs may not lie on inputs
    (dict(n_free_out=_at(3)), 1), (dict(cu=_at(1)), 1), (dict(table=_at(2)), 1),
    (dict(cu=_at(7)), 1),                      # nor on one another
    (dict(new_lens=ctypes.c_void_p((1 << 32) + 12)), 1),
])
def test_block_tables_arguments(lib, kw, status):
    assert _call(lib.sdk_block_tables, TABLES, kw) == status


STORE = dict(ck=_at(0), cv=_at(1), n_tok=5, Hkv=8, slots=_at(2), pages=_at(3), n_pages=10,
             page_size=64, ws=_at(4), ws_bytes=0)


@pytest.mark.parametrize("kw,status", [
    ({}, 3), (dict(n_tok=-1), 1), (dict(Hkv=0), 1), (dict(pages=None), 1), (dict(pages=OFF), 1),
    (dict(n_pages=0), 1), (dict(page_size=0), 1), (dict(ws=None), 1),
    (dict(ck=None, ws_bytes=256), 1), (dict(cv=OFF, ws_bytes=256), 1),
    (dict(slots=None, ws_bytes=256), 1), (dict(slots=ctypes.c_void_p(12), ws_bytes=256), 1),
    (dict(n_tok=0, ck=None, cv=None, slots=None, ws_bytes=256), 0),
])
def test_paged_store_arguments(lib, kw, status):
    assert _call(lib.sdk_paged_store, STORE, kw) == status


APPEND = dict(xk=_at(0), xv=_at(1), dt=1, n_tok=5, Hkv=8, d=128, dk=_at(2), dv=_at(3), n=32768,
              slots=_at(4), pages=_at(5), n_pages=10, page_size=64, ws=_at(6), ws_bytes=0)


@pytest.mark.parametrize("kw,status", [
    ({}, 3), (dict(d=96), 2), (dict(dt=5), 1), (dict(n=0), 1), (dict(n=32769), 1),
    (dict(xk=None), 1), (dict(xv=ctypes.c_void_p(1)), 1), (dict(dk=OFF), 1), (dict(slots=None), 1),
    (dict(pages=None), 1), (dict(n_tok=-1), 1), (dict(ws_bytes=4096), 3),
    (dict(n_tok=0, xk=None, xv=None, ws_bytes=256), 0),
])
def test_paged_append_arguments(lib, kw, status):
    assert _call(lib.sdk_paged_append, APPEND, kw) == status


CHUNK = dict(q=_at(0), n_tok=7, B=3, Hq=32, Hkv=8, d=128, dk=_at(1), dv=_at(2), n=32768,
             pages=_at(3), n_pages=100, page_size=64, table=_at(4), max_pages=20, lens=_at(5),
             cu=_at(6), max_q=5, max_len=1200, total=0, window=0, flags=1, scale=0.1, out=_at(7),
             lse=None, ws=_at(8), ws_bytes=0)


@pytest.mark.parametrize("kw,status", [
    ({}, 3), (dict(B=0), 1), (dict(B=4097), 1), (dict(Hq=30), 1), (dict(Hkv=0), 1),
    (dict(d=96), 2), (dict(n=0), 1), (dict(n=40000), 1), (dict(max_q=0), 1), (dict(max_len=0), 1),
    (dict(max_len=1281), 1),                   # 20 pages of 64 hold 1280 tokens
    (dict(max_pages=0), 1), (dict(total=-1), 1), (dict(window=-1), 1),
    (dict(window=5, flags=0), 1),              # a window needs the causal order
    (dict(n_pages=1 << 25, page_size=32, Hkv=8), 1),   # 2^33 records
    (dict(flags=2), 1), (dict(flags=0), 3), (dict(scale=0.0), 1), (dict(scale=float("inf")), 1),
    (dict(scale=float("nan")), 1), (dict(q=None), 1), (dict(q=OFF), 1), (dict(out=None), 1),
    (dict(out=OFF), 1), (dict(lse=OFF, ws_bytes=0), 1), (dict(dk=None), 1), (dict(dv=OFF), 1),
    (dict(pages=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(cu=None), 1),
    (dict(ws=None), 1), (dict(ws=OFF), 1), (dict(n_tok=-1), 1), (dict(n_tok=1 << 27), 1),
    (dict(n_tok=0, q=None, out=None, ws_bytes=1 << 40), 0),
])
def test_chunk_attn_arguments(lib, kw, status):
    a = dict(CHUNK)
    a.update(kw)
    # lse alignment is 4 bytes: OFF is 2 past a multiple of 4
    assert lib.sdk_chunk_attn(*a.values(), None) == status


def test_chunk_attn_overlapping_outputs(lib):
    """out may be q, and pass on to the next check; not lie across it."""
    at = lambda x: ctypes.c_void_p(x)
    base, size = 1 << 32, 7 * 32 * 128 * 2
    call = lambda **kw: lib.sdk_chunk_attn(*dict(CHUNK, **kw).values(), None)
    assert call(out=at(base)) == 3
    assert call(out=at(base + size)) == 3 and call(out=at(base - size)) == 3
    assert call(out=at(base + size - 16)) == 1 and call(out=at(base - 16)) == 1
    assert call(lse=at(base + size)) == 3 and call(lse=at(base + size - 4)) == 1
    assert call(out=at(base), lse=at(base)) == 1


def test_workspace_sizes(lib):
    assert lib.sdk_block_tables_workspace_bytes(0) == 0
    assert lib.sdk_block_tables_workspace_bytes(64) >= 256
    assert lib.sdk_paged_store_workspace_bytes() >= 256
    assert lib.sdk_paged_append_workspace_bytes(-1, 8, 128, 32768) == 0
    f = sdk.sdk_chunk_attn_workspace_bytes
    assert f(0, 1, 32, 8, 128, 32768, 1, 100) == 0
    assert f(1, 1, 30, 8, 128, 32768, 1, 100) == 0
    assert f(1, 1, 32, 8, 80, 32768, 1, 100) == 0
    assert f(4096, 1, 32, 8, 128, 32768, 1, 1 << 30) == 0      # over the call's limit
    few = f(64, 64, 32, 8, 128, 32768, 1, 32768, 100000)
    assert 0 < few < f(64, 64, 32, 8, 128, 32768, 1, 32768)    # a bound on all contexts saves memory


def test_python_argument_checks():
    import torch
    with pytest.raises(ValueError, match="CUDA tensor"):
        sdk.sdk_paged_store(torch.zeros(1, 1, 4, 2, 16, dtype=torch.int32), None, None, None)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sdk.sdk_block_tables(torch.zeros(2, dtype=torch.int32), None, None, None, None, 16, 1)

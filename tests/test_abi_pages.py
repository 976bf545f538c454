"""Host-only checks of the page entry points (kv8_copy_pages, kv8_free,
kv8_reserve, kv8_fork, kv8_compact): what they refuse before touching the GPU,
and pins of their oracle."""

import ctypes
import os

import pytest

from bit_weight_only_gemm_amd import _lib
from oracle import kv8_pages as oracle

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libw4a16.so not built", allow_module_level=True)

L = _lib.load()
NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(0x10000)        # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x10008)         # misaligned
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 5


def arrays(count=2, at=0x10000, odd=None, null=None):
    a = [at + 0x1000 * i for i in range(4 * count)]
    if odd is not None:
        a[odd] += 8
    if null is not None:
        a[null] = None
    return (ctypes.c_void_p * len(a))(*a)


def copy(caches=None, count=2, pages=8, T=16, Hkv=2, D=64, src=FAKE, dst=FAKE, n=3):
    return L.kv8_copy_pages(arrays() if caches is None else caches, count, pages, T, Hkv, D, src, dst, n, NULL)


def free(refs=FAKE, pages=8, T=16, table=FAKE, width=4, lens=FAKE, B=3, rows=FAKE, n=2):
    return L.kv8_free(refs, pages, T, table, width, lens, B, rows, n, NULL)


def reserve(refs=FAKE, pages=8, T=16, table=FAKE, width=4, lens=FAKE, B=3, added=FAKE, status=FAKE,
            space=FAKE, nbytes=1 << 20):
    return L.kv8_reserve(refs, pages, T, table, width, lens, B, added, status, space, nbytes, NULL)


def fork(caches=None, count=2, pages=8, T=16, Hkv=2, D=64, refs=FAKE, table=FAKE, width=4, lens=FAKE, B=3,
         src=FAKE, dst=FAKE, n=2, status=FAKE, space=FAKE, nbytes=1 << 20):
    return L.kv8_fork(arrays() if caches is None else caches, count, pages, T, Hkv, D, refs, table, width, lens,
                      B, src, dst, n, status, space, nbytes, NULL)


def compact(caches=None, count=2, pages=8, T=16, Hkv=2, D=64, refs=FAKE, refs_out=FAKE, table=FAKE,
            table_out=FAKE, width=4, lens=FAKE, B=3, used=FAKE, space=FAKE, nbytes=1 << 20):
    return L.kv8_compact(arrays() if caches is None else caches, count, pages, T, Hkv, D, refs, refs_out, table,
                         table_out, width, lens, B, used, space, nbytes, NULL)


@pytest.mark.parametrize("call", [copy, fork, compact])
def test_caches_are_checked(call):
    for bad in (dict(count=0), dict(count=-1), dict(pages=0), dict(Hkv=0), dict(caches=arrays(null=6)),
                dict(caches=ctypes.cast(None, ctypes.POINTER(ctypes.c_void_p)))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(T=24), dict(D=96), dict(pages=(1 << 30) + 1), dict(Hkv=1025), dict(count=65537)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(caches=arrays(odd=7)) == MISALIGNED


@pytest.mark.parametrize("call", [free, reserve, fork, compact])
def test_pools_are_checked(call):
    for bad in (dict(width=0), dict(B=-1), dict(refs=NULL), dict(table=NULL), dict(lens=NULL)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(B=(1 << 20) + 1), dict(width=1 << 27), dict(T=8)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(refs=ODD) == MISALIGNED and call(table=ODD) == MISALIGNED and call(lens=ODD) == MISALIGNED


def test_what_only_one_call_takes():
    for call, names in ((copy, ("src", "dst")), (free, ("rows",)), (reserve, ("added", "status")),
                        (fork, ("src", "dst", "status")), (compact, ("refs_out", "table_out", "used"))):
        for name in names:
            assert call(**{name: NULL}) == INVALID and call(**{name: ODD}) == MISALIGNED, (call, name)
    for call in (copy, free, fork):
        assert call(n=-1) == INVALID
        assert call(n=(1 << 20) + 1) == UNSUPPORTED
    assert copy(n=0) == OK and free(n=0) == OK and free(B=0) == OK


@pytest.mark.parametrize("call,n", [(reserve, 0), (fork, 2), (compact, 0)])
def test_workspace(call, n):
    need = L.kv8_pages_workspace_bytes(8, 3, n)
    assert need >= 4 * max(3 + 8, 7 + 4 * n)
    assert call(nbytes=need - 1) == WORKSPACE and call(space=NULL, nbytes=0) == WORKSPACE
    assert call(space=ODD) == MISALIGNED


def test_workspace_bytes():
    assert L.kv8_pages_workspace_bytes(0, 3, 0) == -1 and L.kv8_pages_workspace_bytes(8, -1, 0) == -1
    assert L.kv8_pages_workspace_bytes(8, 3, -1) == -1
    assert L.kv8_pages_workspace_bytes(1 << 30, 1 << 20, 1 << 20) >= 4 * (4 + 3 * (1 << 30))


# ------------------------------------------------------------------ oracle ---
def pool(refs, table, lens, T=16):
    return {"refs": refs, "table": table, "lens": lens, "T": T}


def test_oracle_fork_shares_whole_pages_and_copies_the_last():
    p = pool([1, 0, 0, 1, 0, 0], [[3, 0, -1], [-1] * 3, [-1] * 3], [20, 0, 0])
    assert oracle.fork(p, [0, 0], [2, 1]) == (0, [(0, 1), (0, 2)])
    assert p["refs"] == [1, 1, 1, 3, 0, 0] and p["lens"] == [20, 20, 20]
    assert p["table"] == [[3, 0, -1], [3, 2, -1], [3, 1, -1]]
    assert oracle.fork(p, [0], [1]) == (-1, []) and oracle.fork(p, [0], [0]) == (-1, [])
    oracle.free(p, [1, 1, 7])
    assert p["refs"] == [1, 1, 0, 2, 0, 0] and p["table"][1] == [-1] * 3
    p["refs"] = [1] * 6
    assert oracle.fork(p, [0], [1]) == (1, []) and p["lens"][1] == 0


def test_oracle_reserve_takes_the_lowest_in_order_of_the_rows():
    p = pool([0, 1, 0, 0, 0], [[1, -1], [-1, -1], [-1, -1]], [16, 0, 0])
    assert oracle.reserve(p, [0, 17, 1]) == (0, [])
    assert p["table"] == [[1, -1], [0, 2], [3, -1]] and p["refs"] == [1, 1, 1, 1, 0] and p["lens"] == [16, 17, 1]
    assert oracle.reserve({**p, "refs": [*p["refs"]], "lens": [*p["lens"]], "table": [[*t] for t in p["table"]]},
                          [-1, 0, 0])[0] == 0
    assert oracle.reserve(p, [1, 0, 16]) == (1, []) and oracle.reserve(p, [17, 0, 0]) == (-1, [])
    assert p["lens"] == [16, 17, 1]


def test_oracle_compact_moves_the_high_pages_down_in_order():
    p = pool([0, 1, 0, 2, 0, 1], [[3, 5, 9], [3, 1, 5]], [17, 32])
    assert oracle.compact(p) == (3, [(3, 0), (5, 2)])
    assert p["refs"] == [2, 1, 1, 0, 0, 0] and p["table"] == [[0, 2, 9], [0, 1, 5]]

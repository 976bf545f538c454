"""Rows whose lengths are below 0 hold nothing, for every page operator (on the GPU
against lists)."""

import pytest
import torch

import bit_weight_only_gemm_amd as w4
from gpu_util import DEV
from oracle import kv8_pages as oracle

pytestmark = pytest.mark.gpu
LENS = [20, -3, 0, -(2 ** 31), 16, -1]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def make():
    pool = {"refs": [1, 0, 1, 1, 0, 0, 0, 0], "table": [[3, 0, -1], [-1] * 3, [-1] * 3, [5, 5, 5], [2, -1, -1], [7, 7, 7]],
            "lens": list(LENS), "T": 16}
    return pool, {n: ints(pool[n]) for n in ("refs", "table", "lens")}, w4.kv8_cache(8, 16, 1, 64, DEV)


def check(pool, d):
    for n in ("refs", "table", "lens"):
        assert d[n].tolist() == pool[n], n


def test_fork_into_rows_below_0():
    pool, d, cache = make()
    cache["k"][0] = 9
    status, moves = oracle.fork(pool, [0, 4, 0], [3, 5, 1])
    got = w4.kv8_fork(cache, d["refs"], d["table"], d["lens"], ints([0, 4, 0]), ints([3, 5, 1]))
    assert got.tolist() == [status] == [0]
    check(pool, d)
    assert len(moves) == 2 and all((cache["k"][b] == 9).all() for _, b in moves)


def test_fork_from_rows_below_0():
    pool, d, cache = make()
    status, moves = oracle.fork(pool, [1, 3], [2, 5])
    got = w4.kv8_fork(cache, d["refs"], d["table"], d["lens"], ints([1, 3]), ints([2, 5]))
    assert got.tolist() == [status] == [0] and not moves
    check(pool, d)


def test_reserve_free_and_compact():
    pool, d, cache = make()
    added = [0, 17, -5, 1, 0, 0]
    assert oracle.reserve(pool, added)[0] == 0
    assert w4.kv8_reserve(d["refs"], d["table"], d["lens"], ints(added), 16).tolist() == [0]
    check(pool, d)
    pool["lens"][1] = -7
    d["lens"][1] = -7
    oracle.free(pool, [1, 3])
    w4.kv8_free(d["refs"], d["table"], d["lens"], ints([1, 3]), 16)
    check(pool, d)
    used, _ = oracle.compact(pool)
    table, refs, got = w4.kv8_compact(cache, d["refs"], d["table"], d["lens"])
    assert got.tolist() == [used]
    check(pool, {"table": table, "refs": refs, "lens": d["lens"]})


def test_a_row_that_holds_tokens_is_still_refused():
    pool, d, cache = make()
    assert oracle.fork(pool, [0], [4]) == (-1, [])
    assert w4.kv8_fork(cache, d["refs"], d["table"], d["lens"], ints([0]), ints([4])).tolist() == [-1]
    check(pool, d)

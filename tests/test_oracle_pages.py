"""Pins of the pages' oracle that its other tests leave open."""

from oracle import kv8_pages as oracle


def pool(refs, table, lens, T=16):
    return {"refs": refs, "table": table, "lens": lens, "T": T}


def test_a_length_below_0_is_a_row_that_holds_nothing():
    p = pool([1, 0, 0], [[0, -1], [-1, -1], [-1, -1]], [16, -4, 0])
    assert oracle.fork(p, [0], [1]) == (0, []) and p["lens"] == [16, 16, 0] and p["refs"] == [2, 0, 0]
    p = pool([1, 0, 0], [[0, -1], [-1, -1], [-1, -1]], [16, -4, 0])
    assert oracle.fork(p, [1], [2]) == (0, []) and p["lens"] == [16, -4, 0]
    assert oracle.reserve(p, [0, 3, 0]) == (0, []) and p["lens"] == [16, 3, 0] and p["table"][1] == [1, -1]

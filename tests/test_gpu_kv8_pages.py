"""The page operators on the GPU against lists: every counter, table entry,
length and byte of the caches after each call."""

import numpy as np
import pytest
import torch

import bit_weight_only_gemm_amd as w4
from gpu_util import DEV, say
from oracle import kv8_pages as oracle

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(np.asarray(v, np.int64).astype(np.int32), device=DEV)


def make(seed, lens, width, pages, T, Hkv=2, D=64, layers=1, stray=()):
    """A pool whose rows hold random pages, and the same on the device."""
    r = np.random.RandomState(seed)
    order, at = r.permutation(pages), 0
    p = {"refs": [0] * pages, "table": [[-1] * width for _ in lens], "lens": list(lens), "T": T}
    for b in range(len(lens)):
        for i in range(-(-lens[b] // T)):
            p["table"][b][i] = int(order[at])
            p["refs"][order[at]] += 1
            at += 1
    for b, i, page in stray:
        p["table"][b][i] = page
    caches = []
    for _ in range(layers):
        c = w4.kv8_cache(pages, T, Hkv, D, DEV)
        for n in ("k", "v"):
            c[n].copy_(torch.from_numpy(r.randint(0, 256, c[n].shape).astype(np.uint8)))
        for n in ("k_scale", "v_scale"):
            c[n].copy_(torch.from_numpy(r.rand(*c[n].shape).astype(np.float32)))
        caches.append(c)
    d = {"refs": ints(p["refs"]), "table": ints(p["table"]), "lens": ints(p["lens"])}
    return p, d, caches, [{n: c[n].clone() for n in ("k", "v", "k_scale", "v_scale")} for c in caches]


def check(p, d, caches, want, moves=()):
    for c, w in zip(caches, want):
        for n, t in w.items():
            for a, b in moves:
                t[b] = t[a]
            assert torch.equal(c[n], t), n
    assert d["refs"].tolist() == p["refs"]
    assert d["table"].tolist() == p["table"]
    assert d["lens"].tolist() == p["lens"]


SHAPES = [  # lens, width, pages, T, Hkv, D, layers
    ([1], 1, 2, 16, 1, 64, 1),
    ([16, 0, 0], 1, 4, 16, 1, 64, 1),
    ([33, 64, 5, 0, 0, 0, 0], 5, 24, 32, 3, 128, 2),
    ([700, 1, 128, 1000, 0, 0, 0, 0, 0], 8, 64, 128, 2, 64, 3),
    ([2000, 900, 0, 0, 0], 130, 5003, 16, 1, 64, 1),        # the pool takes several turns of the plan
]


@pytest.mark.parametrize("shape", SHAPES)
def test_fork_reserve_free(shape):
    lens, width, pages, T, Hkv, D, layers = shape
    say("fork", shape)
    p, d, caches, want = make(1, lens, width, pages, T, Hkv, D, layers)
    full = [b for b, n in enumerate(lens) if n]
    empty = [b for b, n in enumerate(lens) if not n]
    src, dst = [full[i % len(full)] for i in range(len(empty))], empty[::-1]
    if dst:
        status, moves = oracle.fork(p, src, dst)
        got = w4.kv8_fork(caches, d["refs"], d["table"], d["lens"], ints(src), ints(dst))
        assert got.tolist() == [status]
        check(p, d, caches, want, moves)
    added = [min(b % 3 * T // 2 + b % 2, width * T - n) for b, n in enumerate(p["lens"])]
    status, _ = oracle.reserve(p, added)
    assert w4.kv8_reserve(d["refs"], d["table"], d["lens"], ints(added), T).tolist() == [status]
    check(p, d, caches, want)
    rows = [full[0], len(lens), -1, full[0], *dst[:2]]
    oracle.free(p, rows)
    w4.kv8_free(d["refs"], d["table"], d["lens"], ints(rows), T)
    check(p, d, caches, want)


def test_many_rows_and_many_caches():
    lens = [(37 * b) % 90 for b in range(1500)] + [0] * 1500     # rows past one turn of the plan
    p, d, caches, want = make(2, lens, 8, 12000, 16, 1, 64, 35)  # caches past one launch
    src = [b for b in range(1500)]
    dst = [1500 + (7 * b) % 1500 for b in range(1500)]
    dst = [x for i, x in enumerate(dst)]
    assert len(set(dst)) == 1500
    live = [(s, t) for s, t in zip(src, dst)]
    status, moves = oracle.fork(p, *map(list, zip(*live)))
    got = w4.kv8_fork(caches, d["refs"], d["table"], d["lens"], *(ints(x) for x in zip(*live)))
    assert got.tolist() == [status] == [0]
    a, b = (torch.tensor(x, device=DEV) for x in zip(*moves))
    for w in want:
        for t in w.values():
            t[b] = t[a]
    check(p, d, caches, want)
    added = [b % 5 * 7 for b in range(3000)]
    status, _ = oracle.reserve(p, added)
    assert w4.kv8_reserve(d["refs"], d["table"], d["lens"], ints(added), 16).tolist() == [status]
    check(p, d, caches, want)
    rows = list(range(0, 3000, 2))
    oracle.free(p, rows)
    w4.kv8_free(d["refs"], d["table"], d["lens"], ints(rows), 16)
    check(p, d, caches, want)


@pytest.mark.parametrize("case", ["missing", "twice", "source", "held", "range", "range_src"])
def test_fork_refused_on_the_device(case):
    p, d, caches, want = make(3, [17, 20, 0, 0], 3, 6, 16)
    src, dst = [0, 1], [2, 3]
    if case == "missing":
        p["refs"] = [max(n, 1) for n in p["refs"]][:5] + [0]
        d["refs"] = ints(p["refs"])
    elif case == "twice":
        dst = [2, 2]
    elif case == "source":
        src, dst = [0, 3], [3, 2]
    elif case == "held":
        dst = [2, 1]
    elif case == "range":
        dst = [2, 4]
    else:
        src = [0, -1]
    status, moves = oracle.fork(p, src, dst)
    assert status != 0 and not moves
    got = w4.kv8_fork(caches, d["refs"], d["table"], d["lens"], ints(src), ints(dst))
    assert got.tolist() == [status]
    check(p, d, caches, want)


@pytest.mark.parametrize("added,status", [([0, 0, 0], 0), ([-5, 0, 1], 0), ([0, 0, 49], -1), ([33, 0, 0], -1),
                                          ([0, 33, 33], 2), ([2 ** 31 - 1, 0, 0], -1)])
def test_reserve_refused_on_the_device(added, status):
    p, d, caches, want = make(4, [16, 1, 0], 3, 5, 16)
    assert oracle.reserve(p, added)[0] == status
    got = torch.full((1,), 77, dtype=torch.int32, device=DEV)
    assert w4.kv8_reserve(d["refs"], d["table"], d["lens"], ints(added), 16, status=got) is got
    assert got.tolist() == [status]
    check(p, d, caches, want)


DROPS = [([-1, -1, -1, 20, -1], 0), ([-40, -16, -7, 0, 0], 0), ([-2 ** 31, -1000, 5, -1, -2 ** 31], 0),
         ([-33, 0, -8, 70, 1], 0),    # to the end of a page; all tokens; takes beside it
         ([0, -3, 0, 200, 0], 1)]     # 13 pages, 12 free: nothing is dropped either


@pytest.mark.parametrize("added,status", DROPS)
def test_reserve_drops_tokens(added, status):
    p, d, caches, want = make(14, [49, 16, 8, 0, 90], 16, 24, 16, stray=[(4, 5, -9)])
    assert oracle.reserve(p, added)[0] == status
    assert w4.kv8_reserve(d["refs"], d["table"], d["lens"], ints(added), 16).tolist() == [status]
    check(p, d, caches, want)
    more = [3, 30, 0, 1, 17]          # what was given back can be taken again
    if status == 0:
        assert oracle.reserve(p, more)[0] == 0
        assert w4.kv8_reserve(d["refs"], d["table"], d["lens"], ints(more), 16).tolist() == [0]
        check(p, d, caches, want)


def test_reserve_does_not_end_rows_in_shared_pages():
    for added, status in (([-1, 0, 0], 0), ([-10, 0, 0], -1), ([0, 0, -17], -1), ([-9, 0, -25], 0), ([-41, 0, 0], 0),
                          ([1, 1, -9], 0)):
        p, d, caches, want = make(15, [41, 7, 0], 4, 9, 16)
        status_f, moves = oracle.fork(p, [0], [2])
        assert w4.kv8_fork(caches, d["refs"], d["table"], d["lens"], ints([0]), ints([2])).tolist() == [status_f] == [0]
        assert oracle.reserve(p, added)[0] == status
        assert w4.kv8_reserve(d["refs"], d["table"], d["lens"], ints(added), 16).tolist() == [status]
        check(p, d, caches, want, moves)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_compact(shape, in_place):
    lens, width, pages, T, Hkv, D, layers = shape
    say("compact", shape)
    p, d, caches, want = make(5, lens, width, pages, T, Hkv, D, layers)
    empty = [b for b, n in enumerate(lens) if not n]
    if empty:      # shared pages
        oracle.fork(p, [0], [empty[0]])
        w4.kv8_fork(caches, d["refs"], d["table"], d["lens"], ints([0]), ints([empty[0]]))
        want = [{n: c[n].clone() for n in w} for c, w in zip(caches, want)]
    before = {n: t.clone() for n, t in d.items()}
    used, moves = oracle.compact(p)
    out = dict(page_table_out=d["table"], refs_out=d["refs"]) if in_place else {}
    table, refs, got = w4.kv8_compact(caches, d["refs"], d["table"], d["lens"], **out)
    assert got.tolist() == [used]
    if in_place:
        assert table is d["table"] and refs is d["refs"]
    else:
        assert all(torch.equal(d[n], before[n]) for n in d)
    check(p, {"table": table, "refs": refs, "lens": d["lens"]}, caches, want, moves)
    # nothing left to move
    again, refs2, got = w4.kv8_compact(caches, refs, table, d["lens"])
    assert got.tolist() == [used] and torch.equal(again, table) and torch.equal(refs, refs2)
    check(p, {"table": again, "refs": refs2, "lens": d["lens"]}, caches, want)


def test_compact_of_empty_and_full_pools():
    for lens, pages in (([0, 0], 7), ([112, 0], 7)):
        p, d, caches, want = make(6, lens, 7, pages, 16)
        used, moves = oracle.compact(p)
        table, refs, got = w4.kv8_compact(caches, d["refs"], d["table"], d["lens"])
        assert got.tolist() == [used] == [sum(lens) // 16] and not moves
        check(p, {"table": table, "refs": refs, "lens": d["lens"]}, caches, want)


def test_entries_and_lengths_out_of_range():
    """Strays in the table and lengths past its rows change nothing else."""
    stray = [(0, 1, -7), (1, 0, 1 << 29), (2, 2, 99)]
    p, d, caches, want = make(7, [40, 16, 3, 0, 0], 3, 16, 16, stray=stray)
    p["lens"][2] = 10000
    d["lens"] = ints(p["lens"])
    status, moves = oracle.fork(p, [0, 1], [3, 4])
    assert w4.kv8_fork(caches, d["refs"], d["table"], d["lens"], ints([0, 1]), ints([3, 4])).tolist() == [status]
    check(p, d, caches, want, moves)
    table, refs, used = w4.kv8_compact(caches, d["refs"], d["table"], d["lens"])
    n, moves = oracle.compact(p)
    assert used.tolist() == [n]
    d = {"table": table, "refs": refs, "lens": d["lens"]}
    check(p, d, caches, want, moves)
    oracle.free(p, [2, 1, 0])
    w4.kv8_free(d["refs"], d["table"], d["lens"], ints([2, 1, 0]), 16)
    check(p, d, caches, want)


@pytest.mark.parametrize("T,Hkv,D", [(16, 1, 64), (32, 5, 128), (128, 8, 128)])
def test_copy_pages(T, Hkv, D):
    p, d, caches, want = make(8, [1], 1, 9, T, Hkv, D, 2)
    pairs = [(0, 3), (8, 1), (0, 7), (-1, 2), (4, 9), (5, 5), (1 << 30, 6)]
    w4.kv8_copy_pages(caches, *(ints(x) for x in zip(*pairs)))
    check(p, d, caches, want, [(0, 3), (8, 1), (0, 7)])
    w4.kv8_copy_pages(caches[0], ints([4]), ints([0]))
    check(p, d, caches[:1], want[:1], [(4, 0)])
    w4.kv8_copy_pages(caches, ints([]), ints([]))
    check(p, d, caches, want)


def test_calls_without_rows():
    p, d, caches, want = make(9, [5], 1, 3, 16)
    none = ints([])
    assert w4.kv8_fork(caches, d["refs"], d["table"], d["lens"], none, none).tolist() == [0]
    w4.kv8_free(d["refs"], d["table"], d["lens"], none, 16)
    check(p, d, caches, want)
    empty = torch.zeros(0, 4, dtype=torch.int32, device=DEV)
    assert w4.kv8_reserve(d["refs"], empty, none, none, 16).tolist() == [0]
    table, refs, used = w4.kv8_compact(caches, d["refs"], empty, none)
    assert table.shape == (0, 4) and used.tolist() == [1]


def test_captured_in_a_graph():
    """A beam's step, replayed: free, fork, reserve, with lengths that change in between."""
    T, width = 16, 6
    p, d, caches, want = make(10, [20, 47, 0, 0, 0, 0], width, 40, T, layers=2)
    src, dst, added = [0, 0, 1, 1], [2, 3, 4, 5], [0, 0, 1, 17, 1, 0]
    gs, gd, ga = ints(src), ints(dst), ints(added)
    s1, s2 = (torch.empty(1, dtype=torch.int32, device=DEV) for _ in range(2))
    space = w4.workspace(w4.kv8_pages_workspace_bytes(40, 6, 4), DEV)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        w4.kv8_free(d["refs"], d["table"], d["lens"], gd, T)
        w4.kv8_fork(caches, d["refs"], d["table"], d["lens"], gs, gd, status=s1, workspace=space)
        w4.kv8_reserve(d["refs"], d["table"], d["lens"], ga, T, status=s2, workspace=space)
    for i in range(4):
        g.replay()
        torch.cuda.synchronize()
        oracle.free(p, dst)
        status, moves = oracle.fork(p, src, dst)
        assert (status, oracle.reserve(p, added)[0]) == (0, 0)
        assert s1.tolist() == s2.tolist() == [0]
        check(p, d, caches, want, moves)
        assert torch.zeros(8, device=DEV).sum().item() == 0      # other work in between
        more = [3, 1, 0, 0, 0, 0]
        oracle.reserve(p, more)
        assert w4.kv8_reserve(d["refs"], d["table"], d["lens"], ints(more), T).tolist() == [0]


def test_on_another_stream():
    p, d, caches, want = make(11, [20, 0], 2, 6, 16)
    st = torch.cuda.Stream()
    src, dst, added = ints([0]), ints([1]), ints([1, 13])
    torch.cuda.synchronize()
    oracle_status, moves = oracle.fork(p, [0], [1])
    a = w4.kv8_fork(caches, d["refs"], d["table"], d["lens"], src, dst, stream=st)
    b = w4.kv8_reserve(d["refs"], d["table"], d["lens"], added, 16, stream=st)
    st.synchronize()
    # 20 + 13 tokens pass the 2 x 16 of a row
    assert oracle.reserve(p, [1, 13])[0] == -1 and oracle_status == 0
    assert a.tolist() == [0] and b.tolist() == [-1]
    check(p, d, caches, want, moves)


def test_refusals():
    p, d, caches, _ = make(12, [20, 0], 2, 6, 16)
    refs, table, lens = d["refs"], d["table"], d["lens"]
    one = ints([0])
    with pytest.raises(ValueError, match="no cache"):
        w4.kv8_copy_pages([], one, one)
    with pytest.raises(ValueError, match="differ"):
        w4.kv8_copy_pages([caches[0], w4.kv8_cache(7, 16, 2, 64, DEV)], one, one)
    with pytest.raises(ValueError):
        w4.kv8_copy_pages(caches, one, ints([0, 1]))
    with pytest.raises(TypeError):
        w4.kv8_copy_pages(caches, one, one.long())
    with pytest.raises(ValueError):
        w4.kv8_fork(caches, refs[:-1], table, lens, one, one)
    with pytest.raises(ValueError):
        w4.kv8_fork(caches, refs, table, lens[:1], one, one)
    with pytest.raises(ValueError):
        w4.kv8_free(refs, table.t(), lens, one, 16)
    with pytest.raises(w4.W4A16Error, match="status 2"):
        w4.kv8_free(refs, table, lens, one, 24)
    with pytest.raises(TypeError):
        w4.kv8_reserve(refs, table, lens, ints([0, 0]).cpu(), 16)
    with pytest.raises(w4.W4A16Error, match="status 5"):
        w4.kv8_reserve(refs, table, lens, ints([0, 0]), 16, workspace=torch.empty(4, device=DEV))
    with pytest.raises(ValueError):
        w4.kv8_compact(caches, refs, table, lens, refs_out=torch.empty(5, dtype=torch.int32, device=DEV))
    with pytest.raises(w4.W4A16Error):
        w4.kv8_pages_workspace_bytes(0, 1)


def test_offsets_beyond_32_bits():
    """Pages past 4 GB of keys are shared, copied and moved."""
    T, Hkv, D, pages = 128, 32, 128, 9000
    cache = w4.kv8_cache(pages, T, Hkv, D, DEV)
    assert cache["k"].numel() > 1 << 32
    refs, table, lens = ints([0] * pages), ints([[8990, 8995], [-1, -1], [-1, -1]]), ints([200, 0, 0])
    refs[8990] = refs[8995] = 1
    refs[2:8980] = 1                                # held by rows of another table
    g = torch.Generator(device=DEV).manual_seed(1)
    page = {}
    for p in (8990, 8995):
        for n in ("k", "v"):
            cache[n][p] = torch.randint(0, 256, cache[n][p].shape, generator=g, device=DEV, dtype=torch.uint8)
        for n in ("k_scale", "v_scale"):
            cache[n][p] = torch.rand(Hkv, generator=g, device=DEV)
        page[p] = {n: cache[n][p].clone() for n in ("k", "v", "k_scale", "v_scale")}

    def holds(at, of):
        return all(torch.equal(cache[n][at], page[of][n]) for n in page[of])

    assert w4.kv8_fork(cache, refs, table, lens, ints([0, 0]), ints([1, 2])).tolist() == [0]
    assert table.tolist() == [[8990, 8995], [8990, 0], [8990, 1]] and holds(0, 8995) and holds(1, 8995)
    w4.kv8_free(refs, table, lens, ints([1]), T)
    table, refs, used = w4.kv8_compact(cache, refs, table, lens)
    assert used.tolist() == [8981] and table.tolist() == [[0, 8980], [-1, -1], [0, 1]]
    assert holds(0, 8990) and holds(8980, 8995) and holds(1, 8995)
    w4.kv8_copy_pages(cache, ints([8980]), ints([8999]))
    assert holds(8999, 8995)

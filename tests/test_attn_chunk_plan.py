"""The plan of attention of new tokens: the library's own code run on the CPU (chunk_plan_host.cpp), wave by wave.  Every key tile that a
row tile sees is walked once, parts are where the join reads them, and row numbers that do not ascend stay within memory."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FIELDS = ("joined", "run", "b", "head", "tile", "q0", "row0", "row1", "off", "lk", "n", "sinks", "lo", "u0", "u1", "whole", "part", "parts")
ARGS = ("tile_rows", "tokens", "tile_heads", "head_tiles", "heads", "runs", "single", "parts")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so, csrc = str(tmp_path_factory.mktemp("plan") / "plan.so"), os.path.join(ROOT, "flatquant_transform_quant_amd", "csrc")
    subprocess.run(["g++", "-O1", "-fwrapv", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
                    "-I" + csrc, os.path.join(ROOT, "tests", "chunk_plan_host.cpp"), os.path.join(csrc, "attn", "fq_attn_chunk_host.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.plan_of.restype = ctypes.c_int64
    return lib


def plan(lib, cu, lengths, Tq, Hq, H, D=64, P=16, width=64, window=0, sinks=0, most=400000):
    """({argument: value}, records as a structured array)"""
    i32 = lambda v: np.ascontiguousarray(v, np.int32)  # noqa: E731
    sizes, cu, lengths, args, out = i32([Tq, len(lengths), Hq, H, D, P, width, window, sinks]), i32(cu), i32(lengths), i32([0] * 8), np.empty((most, len(FIELDS)), np.int32)
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    n = lib.plan_of(p(sizes), p(cu), p(lengths), p(args), p(out), ctypes.c_int64(most))
    assert n >= 0, n
    return dict(zip(ARGS, args.tolist())), np.rec.fromarrays(out[:n].T.copy(), names=FIELDS)


def in_memory(a, r, Tq, reach):
    """What the kernels index with: rows of q and out, keys of the table, parts of the workspace."""
    assert (r.q0 >= 0).all() and (r.row0 >= 0).all() and (r.row1 >= r.row0).all() and (r.q0 + r.row1 < Tq).all()
    assert (r.row1 - r.row0 < a["tokens"]).all() and (r.head >= 0).all() and (r.head < a["heads"]).all()
    assert (r.lk >= 0).all() and (r.lk <= reach).all() and (r.u0 >= 0).all() and (r.u1 <= r.n).all()
    last = np.where(r.u1 - 1 < r.sinks, r.u1 - 1, r.lo + r.u1 - 1 - r.sinks)  # the last tile of a share begins at a key of the sequence
    assert (64 * last < np.maximum(r.lk, 1))[r.u1 > r.u0].all() and (r.sinks >= 0).all() and (r.lo >= 0).all()
    parts = r[(r.joined == 0) & (r.whole == 0)]
    assert (parts.part >= 0).all() and (parts.part < a["parts"]).all()
    joins = r[r.joined == 1]
    assert (joins.parts >= 1).all() and (joins.run + joins.parts < a["runs"]).all() and 2 * (joins.run + joins.parts).max(initial=0) + 1 < max(a["parts"], 2)


def check(lib, sizes, Hq, H, **kw):
    cu = np.concatenate([[0], np.cumsum([r for r, _ in sizes])])
    Tq, lens = int(cu[-1]) + 3, [n for _, n in sizes]
    a, r = plan(lib, cu, lens, Tq, Hq, H, **kw)
    reach = kw.get("width", 64) * kw.get("P", 16)
    in_memory(a, r, Tq, reach)
    walks, joins = r[r.joined == 0], r[r.joined == 1]
    window, sinks = kw.get("window", 0), kw.get("sinks", 0)
    want = {(b, h, t) for b, (rows, _) in enumerate(sizes) for h in range(a["heads"]) for t in range(-(-rows // a["tokens"]))}
    by = {}
    for x in walks:
        by.setdefault((int(x.b), int(x.head), int(x.tile)), []).append(x)
    assert set(by) == want
    joined = {(int(x.b), int(x.head), int(x.tile)): x for x in joins}
    assert len(joined) == len(joins)
    for key, xs in by.items():
        rows, n = sizes[key[0]]
        x = xs[0]
        first, end = key[2] * a["tokens"], min((key[2] + 1) * a["tokens"], rows)
        assert (x.q0, x.row0, x.row1) == (cu[key[0]], first, end - 1) and x.lk == min(n, reach) and x.off == x.lk - rows
        # every key that a row of the tile sees is in a tile of the walk, which has each tile once
        tiles = [u if u < x.sinks else x.lo + u - x.sinks for u in range(x.n)]
        assert len(set(tiles)) == len(tiles)
        seen = set()
        for i in range(first, end):
            p = x.off + i
            w = window if 0 < window < reach else 0
            seen |= set(range((max(0, p - w + 1) if w else 0) // 64, p // 64 + 1)) if p >= 0 else set()
            seen |= set(range(0, -(-min(sinks, p + 1) // 64))) if w and p >= 0 else set()
        assert seen <= set(tiles)
        # the shares: one whole walk, or parts one behind the other in the order of the runs, which the join finds
        if len(xs) == 1 and xs[0].whole:
            assert key not in joined and (x.u0, x.u1) == (0, x.n)
            continue
        xs.sort(key=lambda y: y.u0)
        assert [y.u0 for y in xs] == [0] + [y.u1 for y in xs[:-1]] and xs[-1].u1 == x.n and not any(y.whole for y in xs)
        j = joined.pop(key)
        assert [y.run for y in xs] == list(range(j.run, j.run + j.parts + 1)) and [y.part for y in xs] == [2 * j.run + 1] + [2 * (j.run + i) for i in range(1, j.parts + 1)]
    assert not joined
    used = walks.part[walks.whole == 0]
    assert len(set(used.tolist())) == len(used)
    return a


MIXED = [(1, 1), (3, 0), (0, 40), (1, 17), (5, 64), (2, 65), (4, 3), (33, 130), (64, 64), (20, 300)]


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (37, 4), (64, 64), (129, 200), (100000, 7)])
def test_a_workgroup_a_walk(lib, window, sinks):
    for Hq, H in ((4, 4), (14, 2), (130, 1)):
        assert check(lib, MIXED, Hq, H, window=window, sinks=sinks)["single"] == 1


@pytest.mark.parametrize("window,sinks", [(0, 0), (1700, 5), (1700, 300)])
@pytest.mark.parametrize("Hq,H,D", [(8, 1, 128), (6, 2, 64), (4, 1, 256), (300, 1, 64)])
def test_walks_in_parts(lib, window, sinks, Hq, H, D):
    a = check(lib, [(2, 5000), (1, 1), (0, 0), (40, 2500), (3, 777), (300, 4000)], Hq, H, D=D, width=400, window=window, sinks=sinks)
    assert a["single"] == 0 and a["runs"] > 8


def test_long_walks_of_single_rows(lib):
    """Runs that lie within one segment."""
    check(lib, [(1, 60000)], 1, 1, width=4096)
    check(lib, [(1, 60000), (0, 5), (1, 100)], 8, 2, width=4096, window=40000, sinks=70)


def test_more_sequences_than_lanes(lib):
    """Several rounds of 64 sequences in each plan, idle places among them, alone and beside long ones."""
    many = [((i * i) % 4, (37 * i) % 400) for i in range(150)]
    check(lib, many, 4, 2, width=26)
    check(lib, many, 4, 2, width=26, window=50, sinks=5)
    check(lib, many[:70] + [(2, 3000)] + many[:70] + [(30, 1800)], 4, 2, width=200)
    check(lib, [(0, 9)] * 64 + [(1, 3000)] + [(0, 0)] * 130 + [(7, 2000)], 2, 1, width=200)


def test_nothing_but_idle_places(lib):
    a, r = plan(lib, [0] * 71, [5] * 70, 9, 4, 2)
    assert len(r) == 0 and a["single"] == 1


def test_drawn(lib):
    g = random.Random(7)
    for _ in range(12):
        H = g.choice([1, 2, 3])
        Hq = H * g.choice([1, 2, 5, 8, 33])
        width = g.choice([4, 60, 300])
        sizes = [(g.choice([0, 1, 1, 2, 5, 40, 200]), g.randint(0, width * 16 + 20)) for _ in range(g.choice([1, 5, 70]))]
        if sum(r for r, _ in sizes):
            check(lib, sizes, Hq, H, D=g.choice([64, 256]), width=width, window=g.choice([0, 0, 1, 100, 2000]), sinks=g.choice([0, 4, 90]))


@pytest.mark.parametrize("width,window", [(30, 0), (30, 9), (400, 0), (400, 1800), (4096, 0)])
def test_row_numbers_that_do_not_ascend(lib, width, window):
    """Whatever cu_q and lengths hold, the kernels index no row, key or part that is not there, and every walk ends."""
    g = random.Random(8)
    for i in range(8):
        B, Tq = g.choice([1, 3, 70, 130]), g.choice([1, 40, 700])
        wild = lambda most: g.choice([-2 ** 31, -1, 0, 1, most // 2, most, most + 1, 2 ** 31 - 1, g.randint(0, most)])  # noqa: E731
        cu, lengths = [wild(Tq) for _ in range(B + 1)], [wild(16 * width) for _ in range(B)]
        a, r = plan(lib, cu, lengths, Tq, 8, 2, width=width, window=window, sinks=g.choice([0, 5]), most=4000000)
        in_memory(a, r, Tq, 16 * width)


def test_sequences_that_all_have_every_row(lib):
    """Far more places than the sizes allow for: from row 0 to the last and back, 130 times."""
    for width, Tq in ((4096, 700), (30, 700)):
        cu = [0, Tq] * 65 + [0]
        a, r = plan(lib, cu, [16 * width] * 130, Tq, 8, 2, width=width, most=4000000)
        in_memory(a, r, Tq, 16 * width)

"""Where each XCD's range of weight-gradient tiles begins (csrc/tile_ranges.h),
compiled for the host: whatever offsets a caller gives, the eight ranges cover
every tile once, from 0 to the tile count.  And the slots through which a
workgroup's waves learn their next tile."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_feed_amd", "csrc")

SOURCE = """
#include "tile_ranges.h"
extern "C" {
void starts(int based, const int32_t* poff, int E, int S, int per_p, int K_s, int* out) {
    const int tiles = (E + S) * per_p;
    for (int x = 0; x <= 8; ++x)
        out[x] = based ? inkling::wgrad_range_start<true>(x, poff, E, S, per_p, K_s, tiles)
                       : inkling::wgrad_range_start<false>(x, poff, E, S, per_p, K_s, tiles);
}
int tile_cost() { return inkling::kWgradEpi; }
int next_slot(int turn) { return inkling::next_slot(turn); }
int next_slots() { return inkling::kNextSlots; }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("c++") or shutil.which("g++") or "/opt/rocm/llvm/bin/clang++"
    d = tmp_path_factory.mktemp("ranges")
    src, so = d / "ranges.cpp", d / "ranges.so"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{CSRC}", str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


def _safe(offsets, rows):
    """The plan's offsets: clamped to the rows, non-decreasing."""
    return np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, rows)).astype(np.int32)


def _starts(lib, poff, per_p, S=0, K_s=0, based=True):
    poff = np.ascontiguousarray(poff, np.int32)
    out = np.zeros(9, np.int32)
    lib.starts(int(based), poff.ctypes.data_as(ctypes.c_void_p), len(poff) - 1, S, per_p, K_s,
               out.ctypes.data_as(ctypes.c_void_p))
    return out


def _check(lib, poff, per_p):
    """Monotone from 0 to the tile count, and an eighth of the cost each but for one tile at either end."""
    E = len(poff) - 1
    s = _starts(lib, poff, per_p)
    assert s[0] == 0 and s[8] == E * per_p and (np.diff(s) >= 0).all(), (poff.tolist(), per_p, s.tolist())
    tile = np.repeat(np.diff(poff.astype(np.int64)) + lib.tile_cost(), per_p)
    cost = np.concatenate([[0], np.cumsum(tile)])
    share = cost[-1] / 8
    for x in range(8):
        assert abs(cost[s[x]] - x * share) <= tile.max() + 1, (poff.tolist(), per_p, s.tolist())


def _uniform(E, rows_each):
    return np.arange(E + 1, dtype=np.int64) * rows_each


def test_slices_of_the_offsets(lib):
    """A rank's own experts: the offsets of the later ones begin far from 0."""
    full = _uniform(16, 512)
    per_p = (6144 // 256) * (2048 // 128)
    whole = _starts(lib, full, per_p)
    for first in range(16):
        part = full[first:]
        _check(lib, part.astype(np.int32), per_p)
        # where the rows begin makes no difference
        assert np.array_equal(_starts(lib, part, per_p), _starts(lib, part - part[0], per_p))
    assert np.array_equal(whole, _starts(lib, full, per_p, based=False))


@pytest.mark.parametrize("rows", [0, 1, 2000, 24576, (1 << 31) - 257])
def test_offsets_of_any_kind(lib, rows):
    g = np.random.default_rng(rows & 0xFFFF)
    sets = [[rows] * 9, [0] * 9, [0] * 8 + [rows], [rows // 2] * 4 + [rows] * 5, [-5, 30, 12, 1 << 30, -(1 << 30)],
            [(1 << 31) - 1] * 5, [-(1 << 31)] * 5, [rows, 0, rows, 0], [rows, rows], [0, rows]]
    for E in (1, 2, 7, 64, 512):
        sets.append(np.sort(g.integers(0, rows + 1, E + 1)).tolist())
        sets.append(g.integers(-rows - 1, 2 * rows + 2, E + 1).clip(-(1 << 31), (1 << 31) - 1).tolist())
        late = np.full(E + 1, rows)
        late[:1] = rows - rows // 8
        sets.append(late.tolist())
    for offsets in sets:
        for per_p in (1, 2, 3, 64, 384):
            _check(lib, _safe(offsets, rows), per_p)


def test_largest_tile_counts(lib):
    """One expert of 2^20 x 2^20 weights, 2^31 - 257 rows; 512 experts just below the tile limit."""
    top = (1 << 31) - 257
    for poff in ([0, top], [top, top], [top - 1, top], [top // 2, top]):
        s = _starts(lib, _safe(poff, top), 4096 * 8192)
        assert s[0] == 0 and s[8] == 4096 * 8192 and (np.diff(s) >= 0).all()
    per_p = ((1 << 31) - 4097) // 512
    for first in (0, top // 2, top):
        s = _starts(lib, np.linspace(first, top, 513).astype(np.int64), per_p)
        assert s[0] == 0 and s[8] == 512 * per_p and (np.diff(s.astype(np.int64)) >= 0).all()


def test_the_layers_padded_counts(lib):
    """Without a base: padded counts from 0, shared problems behind them."""
    g = np.random.default_rng(2)
    for E, S, K_s in ((1, 0, 0), (8, 2, 512), (64, 1, 4096), (128, 2, 64)):
        poff = np.concatenate([[0], np.cumsum(g.integers(0, 9, E) * 64)])
        for per_p in (1, 6, 384):
            s = _starts(lib, poff, per_p, S, K_s, based=False)
            assert s[0] == 0 and s[8] == (E + S) * per_p and (np.diff(s) >= 0).all()
            tile = np.concatenate([np.repeat(np.diff(poff), per_p), np.full(S * per_p, K_s)]) + lib.tile_cost()
            cost = np.concatenate([[0], np.cumsum(tile)])
            assert all(abs(cost[s[x]] - x * cost[-1] / 8) <= tile.max() + 1 for x in range(8))


def test_row_offsets_need_the_base(lib):
    """What the base is for: taken as costs from 0, the offsets of 8 later experts give ranges before the first tile."""
    late = _uniform(16, 512)[8:]
    assert _starts(lib, late, 384, based=False).min() < 0
    assert _starts(lib, late, 384).min() == 0


def _wrong_reads(slot_of, slots, turns=4):
    """Every order in which thread 0's wave (write, barrier, read) and another (barrier, read) can take their
    steps over `turns` tiles without a K loop: the turns at which a wave can read another turn's tile."""
    programs = [[step for t in range(turns) for step in (("write", t), ("wait", t), ("read", t))],
                [step for t in range(turns) for step in (("wait", t), ("read", t))]]
    wrong, seen = set(), set()
    todo = [((0, 0), (None,) * slots)]
    while todo:
        at, held = state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        steps = [p[i] if i < len(p) else None for p, i in zip(programs, at)]
        if all(s is not None and s[0] == "wait" for s in steps):
            todo.append(((at[0] + 1, at[1] + 1), held))   # the barrier lets both go
            continue
        for w, s in enumerate(steps):
            if s is None or s[0] == "wait":
                continue
            now = list(held)
            if s[0] == "write":
                now[slot_of(s[1])] = s[1]
            elif held[slot_of(s[1])] != s[1]:
                wrong.add(s[1])
            todo.append(((at[0] + (w == 0), at[1] + (w == 1)), tuple(now)))
    return wrong


def test_every_wave_reads_its_turns_tile(lib):
    assert lib.next_slots() == 2 and {lib.next_slot(t) for t in range(9)} == {0, 1}
    assert _wrong_reads(lib.next_slot, lib.next_slots()) == set()
    assert _wrong_reads(lambda t: 0, 1)      # one slot: a slow wave can read the next turn's tile

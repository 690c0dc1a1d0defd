// Where each XCD's range of weight-gradient tiles begins, and where a workgroup
// finds its next tile.  Plain constexpr arithmetic, so that a host program can
// run it over offsets of any kind.
#pragma once

#include <algorithm>
#include <cstdint>

namespace inkling {

constexpr int kWgradEpi = 128;    // K-equivalent cost of a weight-gradient tile's fp32 epilogue

// First tile of XCD x of 8 (x = 8: the end), with an eighth of the tiles' cost
// in every range.  Tiles are those of `E` problems, per_p each, then those of
// `S` shared problems of K_s rows.  A tile of problem p costs its K plus
// kWgradEpi; the K of problem p is poff[p + 1] - poff[p].
// BASED: poff holds row offsets, whose first may be any row: costs count from
// poff[0].  Otherwise poff[0] is 0.
// poff must not decrease.  The starts do not decrease with x either, from 0 to
// tiles = (E + S) * per_p.
template <bool BASED>
constexpr int wgrad_range_start(int x, const int32_t* poff, int E, int S, int per_p, int K_s, int tiles) {
    if (x >= 8) return tiles;
    const long long base = BASED ? poff[0] : 0;
    const long long routed = (long long)per_p * (poff[E] - base + (long long)E * kWgradEpi);
    const long long total = routed + (long long)per_p * S * (K_s + kWgradEpi);
    const long long c = total * x / 8;
    if (c <= 0) return 0;
    if (c >= routed) {
        const long long per_tile = K_s + kWgradEpi;
        const int at = E * per_p + (int)((c - routed + per_tile - 1) / per_tile);
        return tiles < at ? tiles : at;
    }
    int lo = 0, hi = E - 1;   // last problem p with cost(problems < p) <= c
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((long long)per_p * (poff[mid] - base + (long long)mid * kWgradEpi) <= c) lo = mid;
        else hi = mid - 1;
    }
    const long long before = (long long)per_p * (poff[lo] - base + (long long)lo * kWgradEpi);
    const long long per_tile = (long long)(poff[lo + 1] - poff[lo]) + kWgradEpi;
    const long long all = per_p, in = (c - before + per_tile - 1) / per_tile;   // tiles of problem lo
    const int at = lo * per_p + (int)(in < all ? in : all);
    // (BASED: whatever the offsets hold, no range starts before the first tile)
    return BASED ? std::clamp(at, 0, tiles) : tiles < at ? tiles : at;
}

// The LDS slot that hands the workgroup's tile of this turn from thread 0 to the
// other waves: write, barrier, read.  A weight-gradient tile of an expert without
// rows has no K loop, so no other barrier: in one slot, thread 0 could write the
// next turn's tile before a slower wave has read this one's.  With two in turn,
// it writes a slot again only after the barrier of the turn between, which every
// wave reaches after its read.
constexpr int kNextSlots = 2;
constexpr int next_slot(int turn) { return turn % kNextSlots; }

}  // namespace inkling

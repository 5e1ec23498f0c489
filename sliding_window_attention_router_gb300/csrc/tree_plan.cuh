// What the kernels of the tree attention share: the plan that the first of them
// leaves in the workspace, and the walk over the work it lays down.
//
// A sequence's n drafted tokens times the G query heads of a key head are rows,
// the routed tokens' first; rows are cut into tiles of R, keys into tiles of K from
// the cache's start.  A row tile of routed tokens walks all key tiles, one of others
// those of the anchors and of the window; where all rows fit one tile, that walks all
// key tiles if any token is routed.  A unit is the walk of one
// row tile of one key head of one sequence; the units' key tiles, laid end to end (with
// what a unit costs beside), are dealt out to the CTAs in equal shares, whatever units
// they belong to.  So a unit is a run of consecutive CTAs' parts, one of each; the join adds them up.
// All of a head's units come before the next head's: CTAs a head's number of shares
// apart then read the same tokens at the same time, whose heads lie side by side in
// memory (16 sequences of 32K with 16 key heads: 622 us; a sequence's heads one
// after another, 676).
#pragma once

#include "swiattn_internal.h"

namespace swi {

struct TreeSeq {
    int first, n, base;           // packed tokens [first, first + n), cached ones before them
    int far_rows;                 // rows of the tiles that walk all key tiles
    int lo, na;                   // a window token reads none of [na, lo)
    int far_tiles, near_tiles;    // key tiles of a row tile with routed tokens, and of one without
};
static_assert(sizeof(TreeSeq) == 32, "TreeSeq is read as two int4");

// Row tiles of one key head: the far ones, then the others.
template <int R>
__device__ __forceinline__ int far_tiles(const TreeSeq& s) { return (s.far_rows + R - 1) / R; }
template <int R>
__device__ __forceinline__ int row_tiles(const TreeSeq& s, int G) { return far_tiles<R>(s) + (s.n * G - s.far_rows + R - 1) / R; }
// Key tiles of all its units of one head.
template <int R>
__device__ __forceinline__ int64_t seq_tiles(const TreeSeq& s, int G) {
    const int far = far_tiles<R>(s), all = row_tiles<R>(s, G);
    return static_cast<int64_t>(far) * s.far_tiles + static_cast<int64_t>(all - far) * s.near_tiles;
}

// Rows that the parts of a tile are laid out for: on the tensor cores two halves of
// the keys have one each.
template <int R>
constexpr int kPartRows = R == kTreeTcRows ? 2 * R : R;

// What a unit costs a CTA beside its key tiles (its rows, its first scores, its part
// written out), in key tiles: it counts in the shares as so many before its first,
// unless there are CTAs enough for a tile each.  On the tensor cores two (33 ragged
// trees: 90 us, without 97, with three 92; 7 x 8K, 255 drafts, 16/2 heads: 103, 119, 103;
// 59 ragged sequences, 3 drafts, 16/16 heads: 87, 90, 89).
template <int R>
__device__ __forceinline__ int unit_cost(int64_t tiles, int ctas) { return R == kTreeTcRows && tiles > ctas ? 2 : 0; }

// The CTAs that the work is dealt out to: as many as there are, and no share empty.
// CTA c takes [total c / n, total (c + 1) / n).
__device__ __forceinline__ int64_t share_count(int64_t total, int ctas) { return min(total, static_cast<int64_t>(ctas)); }

// First key of key tile kt of a walk.
template <int K>
__device__ __forceinline__ int tile_key(const TreeSeq& s, bool far, int kt) {
    if (far) return kt * K;
    const int anchors = min((s.na + K - 1) / K, s.lo / K);   // tiles before the window's first
    return (kt < anchors ? kt : s.lo / K + kt - anchors) * K;
}

// One unit's share of a CTA: key tiles [kt0, kt1) of the walk.
struct TreeWork {
    TreeSeq s;
    int b, h, slot;
    int row0, rows;   // rows [row0, row0 + rows) of the head's, row i being token order[i / G], head i % G
    int kt0, kt1;
    bool far;
};

// Where a CTA's share of the work begins, and what it needs to walk it.
struct TreeStart {
    int64_t at, end;      // [at, end) of all the work, key tiles and units' costs
    int64_t head_work;    // of one head
    int64_t before;       // of the head, before sequence b
    int h, b, cost;       // a unit's
    int head_units, units;   // units of one head, and of the head before sequence b
};

// A CTA's share of the work, unit by unit.
template <int R>
struct TreeWalk {
    const TreeDecodeArgs& a;
    TreeStart s;
    __device__ __forceinline__ bool next(TreeWork& w) {
        if (s.at >= s.end) return false;
        const int G = a.Hq / a.Hkv;
        int64_t in = s.at - s.h * s.head_work;
        if (in >= s.head_work) {   // the next head
            ++s.h;
            s.b = s.units = 0;
            s.before = 0;
            in -= s.head_work;
        }
        for (;;) {   // ends: the head has more than `in`
            const int4* p = reinterpret_cast<const int4*>(a.plan.seqs + s.b);
            const int4 x = p[0], y = p[1];
            w.s = TreeSeq{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            const int units = row_tiles<R>(w.s, G);
            const int64_t work = seq_tiles<R>(w.s, G) + static_cast<int64_t>(units) * s.cost;
            if (in < s.before + work || s.b + 1 >= a.B) break;
            s.before += work;
            s.units += units;
            ++s.b;
        }
        const int far = far_tiles<R>(w.s);
        int64_t rest = in - s.before;
        const int64_t far_all = static_cast<int64_t>(far) * (w.s.far_tiles + s.cost);
        w.far = rest < far_all;
        const int len = (w.far ? w.s.far_tiles : w.s.near_tiles) + s.cost;
        if (!w.far) rest -= far_all;
        const int tile = static_cast<int>(rest / len);   // of its kind
        w.row0 = tile * R + (w.far ? 0 : w.s.far_rows);
        w.rows = min(R, (w.far ? w.s.far_rows : w.s.n * G) - w.row0);
        const int from = static_cast<int>(rest - static_cast<int64_t>(tile) * len);
        const int to = static_cast<int>(min(static_cast<int64_t>(len), from + s.end - s.at));
        w.kt0 = max(from - s.cost, 0);
        w.kt1 = to - s.cost;
        w.b = s.b;
        w.h = s.h;
        w.slot = blockIdx.x + s.h * s.head_units + s.units + tile + (w.far ? 0 : far);
        s.at += to - from;
        return w.kt1 > w.kt0;   // none: the share ends before the unit's first tile
    }
};

// The walk of this CTA, by one warp over all sequences; CTA 0 leaves their
// running sums for the join.
template <int R>
__device__ __forceinline__ TreeStart start_walk(const TreeDecodeArgs& a) {
    const int lane = threadIdx.x & 31, G = a.Hq / a.Hkv;
    // Key tiles and units of up to 32 sequences, and of those before each.
    struct Sums {
        int64_t tiles, sum;
        int units, usum;
    };
    auto sums_of = [&](int from) {
        Sums x = {0, 0, 0, 0};
        if (from + lane < a.B) {
            const int4* p = reinterpret_cast<const int4*>(a.plan.seqs + from + lane);
            const int4 lo = p[0], hi = p[1];
            const TreeSeq s{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            x.tiles = x.sum = seq_tiles<R>(s, G);
            x.units = x.usum = row_tiles<R>(s, G);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x.sum, o);
            const int z = __shfl_up_sync(0xffffffffu, x.usum, o);
            if (lane >= o) {
                x.sum += y;
                x.usum += z;
            }
        }
        return x;
    };
    const Sums first = sums_of(0);
    int64_t tiles = 0;
    int units = 0;
    for (int from = 0; from < a.B; from += 32) {
        const Sums x = from == 0 ? first : sums_of(from);
        tiles += __shfl_sync(0xffffffffu, x.sum, 31);
        units += __shfl_sync(0xffffffffu, x.usum, 31);
    }
    TreeStart w;
    w.cost = unit_cost<R>(tiles * a.Hkv, gridDim.x);
    w.head_units = units;
    const int64_t total = w.head_work = tiles + static_cast<int64_t>(units) * w.cost;
    const int64_t all = total * a.Hkv, ctas = share_count(all, gridDim.x), c = blockIdx.x;
    w.at = c < ctas ? all * c / ctas : 0;
    w.end = c < ctas ? all * (c + 1) / ctas : 0;
    w.h = total > 0 ? static_cast<int>(w.at / total) : 0;
    w.before = 0;
    w.b = w.units = 0;
    const int64_t in = w.at - w.h * total;
    int64_t before = 0;
    int units_before = 0;
    bool found = false;
    for (int from = 0; from < a.B && !(found && blockIdx.x > 0); from += 32) {
        const Sums x = from == 0 ? first : sums_of(from);
        const int64_t sum = x.sum + static_cast<int64_t>(x.usum) * w.cost, start = sum - x.tiles - static_cast<int64_t>(x.units) * w.cost;
        if (blockIdx.x == 0 && from + lane < a.B) {
            a.plan.start[from + lane] = before + start;
            a.plan.unit[from + lane] = units_before + x.usum - x.units;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + sum > in);
        if (hit && !found) {
            const int who = __ffs(hit) - 1;
            w.b = from + who;
            w.before = before + __shfl_sync(0xffffffffu, start, who);
            w.units = units_before + __shfl_sync(0xffffffffu, x.usum - x.units, who);
            found = true;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
        units_before += __shfl_sync(0xffffffffu, x.usum, 31);
    }
    if (blockIdx.x == 0 && lane == 0) {
        a.plan.start[a.B] = total;
        a.plan.unit[a.B] = units;
        a.plan.cost[0] = w.cost;
    }
    return w;
}

}  // namespace swi

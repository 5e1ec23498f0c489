// What the kernels of the tree attention share: the plan that the first of them
// leaves in the workspace, and the walk over the work it lays down.
//
// A sequence's n drafted tokens times the G query heads of a key head are rows,
// the routed tokens' first; rows are cut into tiles of R, keys into tiles of K from
// the cache's start.  A row tile that holds a routed token walks all key tiles, one
// without walks those of the anchors and of the window.  A unit is the walk of one
// row tile of one key head of one sequence; the units' key tiles, laid end to end,
// are dealt out to the CTAs in equal shares, whatever units they belong to.  So a
// unit is a run of consecutive CTAs' parts, one of each; the join adds them up.
#pragma once

#include "swiattn_internal.h"

namespace swi {

struct TreeSeq {
    int first, n, base, routed;   // packed tokens [first, first + n), cached ones before them, routed among the n
    int lo, na;                   // a window token reads none of [na, lo)
    int far_tiles, near_tiles;    // key tiles of a row tile with routed tokens, and of one without
};
static_assert(sizeof(TreeSeq) == 32, "TreeSeq is read as two int4");

template <int R>
__device__ __forceinline__ int row_tiles(int tokens, int G) { return (tokens * G + R - 1) / R; }
template <int R>
__device__ __forceinline__ int64_t seq_tiles(const TreeSeq& s, int G, int Hkv) {
    const int far = row_tiles<R>(s.routed, G), all = row_tiles<R>(s.n, G);
    return (static_cast<int64_t>(far) * s.far_tiles + static_cast<int64_t>(all - far) * s.near_tiles) * Hkv;
}

// Rows of each of the copies in which a tile on the tensor cores holds its rows: 32,
// 64 or, once, all.
__device__ __forceinline__ int tree_copy_rows(int rows) { return rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

// The CTAs that the key tiles are dealt out to: as many as there are, and no share
// empty.  CTA c takes [total c / n, total (c + 1) / n).
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
    int b, h, rt, slot;
    int kt0, kt1;
    bool far;
};

// A CTA's share of the work, unit by unit.
template <int R>
struct TreeWalk {
    const TreeDecodeArgs& a;
    int64_t at, end;      // key tiles [at, end) of all
    int64_t before;       // those of the sequences before b
    int b, units;         // units before sequence b's
    int G;
    // `first`: the sequence that the share begins in, and what lies before it.
    __device__ __forceinline__ bool next(TreeWork& w) {
        if (at >= end) return false;
        int64_t tiles;
        for (;;) {   // ends: `end` is no further than all sequences' tiles
            const int4* p = reinterpret_cast<const int4*>(a.plan.seqs + b);
            const int4 x = p[0], y = p[1];
            w.s = TreeSeq{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            tiles = seq_tiles<R>(w.s, G, a.Hkv);
            if (at < before + tiles || b + 1 >= a.B) break;
            before += tiles;
            units += row_tiles<R>(w.s.n, G) * a.Hkv;
            ++b;
        }
        const int far = row_tiles<R>(w.s.routed, G), all = row_tiles<R>(w.s.n, G);
        const int64_t head = tiles / a.Hkv, in = at - before;   // of one head
        w.h = static_cast<int>(in / head);
        int64_t rest = in - w.h * head;
        const int64_t far_all = static_cast<int64_t>(far) * w.s.far_tiles;
        w.far = rest < far_all;
        const int len = w.far ? w.s.far_tiles : w.s.near_tiles;
        if (!w.far) rest -= far_all;
        w.rt = static_cast<int>(rest / len) + (w.far ? 0 : far);
        w.kt0 = static_cast<int>(rest % len);
        w.kt1 = static_cast<int>(min(static_cast<int64_t>(len), w.kt0 + end - at));
        w.b = b;
        w.slot = blockIdx.x + units + w.h * all + w.rt;
        at += w.kt1 - w.kt0;
        return true;
    }
};

// The walk of this CTA, by one warp over all sequences; CTA 0 leaves their
// running sums for the join.
template <int R>
__device__ __forceinline__ void start_walk(const TreeDecodeArgs& a, TreeWalk<R>& w) {
    const int lane = threadIdx.x & 31, G = a.Hq / a.Hkv;
    int64_t total = 0;
    for (int i = lane; i < a.B; i += 32) total += seq_tiles<R>(a.plan.seqs[i], G, a.Hkv);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    w.G = G;
    const int64_t ctas = share_count(total, gridDim.x), c = blockIdx.x;
    w.at = c < ctas ? total * c / ctas : 0;
    w.end = c < ctas ? total * (c + 1) / ctas : 0;
    w.before = 0;
    w.b = w.units = 0;
    int64_t before = 0;
    int units = 0;
    bool found = false;
    for (int from = 0; from < a.B && (blockIdx.x == 0 || !found); from += 32) {
        const int i = from + lane;
        int64_t mine = 0;
        int u = 0;
        if (i < a.B) {
            const TreeSeq s = a.plan.seqs[i];
            mine = seq_tiles<R>(s, G, a.Hkv);
            u = row_tiles<R>(s.n, G) * a.Hkv;
        }
        int64_t sum = mine;
        int usum = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
            const int z = __shfl_up_sync(0xffffffffu, usum, o);
            if (lane >= o) {
                sum += y;
                usum += z;
            }
        }
        if (blockIdx.x == 0 && i < a.B) {
            a.plan.start[i] = before + sum - mine;
            a.plan.unit[i] = units + usum - u;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + sum > w.at);
        if (hit && !found) {
            const int who = __ffs(hit) - 1;
            w.b = from + who;
            w.before = before + __shfl_sync(0xffffffffu, sum - mine, who);
            w.units = units + __shfl_sync(0xffffffffu, usum - u, who);
            found = true;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
        units += __shfl_sync(0xffffffffu, usum, 31);
    }
    if (blockIdx.x == 0 && lane == 0) {
        a.plan.start[a.B] = total;
        a.plan.unit[a.B] = units;
    }
}

}  // namespace swi

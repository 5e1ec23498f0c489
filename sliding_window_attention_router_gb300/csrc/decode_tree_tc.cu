// The products of the tree attention on the 5th-generation tensor cores: 128 rows
// (drafted tokens times the query heads of a key head) by 128 keys at a time.
//
// Per key tile: S = Q K^T into TMEM, softmax weights P written back over S as two
// bf16 each, O += P V with P from TMEM.  What bounds it is the cache's bytes: a tile
// of 128 keys is 64 KiB (bf16, d = 128), 1466 ns of an SM's share of the copy
// bandwidth, against 1536 tensor cycles (0.8 us) and about as many of the softmax,
// overlapped: S of the next tile is computed while the weights of this one are.
//
// The weights go in as two bf16, the nearest and what it leaves, right to 2^-17 of
// each: the products of fp32 weights to less than the result's own rounding.  With
// the first alone, 2^-9 of each, errors would be of the size of that rounding.  The
// tensor cores have the time.
//
// Where a unit has 64 rows or fewer, Q holds them two or four times, and each copy
// takes the weights of its own half or quarter of every tile's keys, the others
// being zero to it: all four softmax warps work, each on fewer keys, and the join
// adds up the copies as it does parts.
//
//   warps 0-3   softmax: thread r owns row r, TMEM lane r
//   warp 4      TMEM and MMA issue (converged, elected issue)
//   warp 5      Q: gathers a unit's rows
//   warps 8-11  K and V: a ring of tiles in the order in which they are used (K0,
//               K1, V0, K2, V1, ...), 32 rows of each tile a warp
//   (warps 6, 7 fill up a warpgroup, the unit that registers are moved by)
// TMEM: S at [0, 128) and [128, 256), O at [256, 256 + d).

#include "swiattn.h"
#include "ptx.cuh"
#include "tree_plan.cuh"

#include <cuda_bf16.h>
#include <math.h>
#include <atomic>

namespace swi {
namespace {

constexpr int R = kTreeTcRows, K = kTreeTcKeys;
constexpr int kWords = kMaxTree / 32;
constexpr int kLoaders = 4;
constexpr int kThreads = 384;   // 3 warpgroups, launched at 168 registers a thread,
constexpr uint32_t kRegsSoftmax = 232, kRegsOther = 136;   // of 3 * 168
constexpr int kHalf = R * 128;   // 128 rows of 64 bf16 columns, 128-byte swizzled
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;

template <int D>
struct Sizes {
    static constexpr int kTile = R * D * 2;            // Q, and a slot of the ring
    static constexpr int kSlots = 6 * 128 / D;
    static constexpr int kLag = 4 * 128 / D;           // slots between a copy's start and the look whether it has come
    static constexpr int kBars = 2 * kSlots + 2 + 2 + 2 + 3 + 1;
    static constexpr int kOffBar = (1 + kSlots) * kTile;
    static constexpr int kOffMisc = kOffBar + kBars * 8;
    static constexpr int kBytes = kOffMisc + 64 + 1024;   // and room to align
};
static_assert(Sizes<128>::kBytes <= 232448 && Sizes<64>::kBytes <= 232448, "shared memory budget");

struct Start {   // where the CTA's share of the work begins
    int64_t at, end, before;
    int b, units;
};

template <int D>
struct Ctx {
    uint8_t* smem;
    uint64_t* bar;
    volatile int* abort_flag;
    const Start* start;
    static constexpr int kFull = 0, kEmpty = Sizes<D>::kSlots, kQFull = 2 * Sizes<D>::kSlots, kQEmpty = kQFull + 1,
                         kSFull = kQEmpty + 1, kPFull = kSFull + 2, kODone = kPFull + 2, kOFull = kODone + 1,
                         kOFree = kOFull + 1, kDrain = kOFree + 1;
};

__device__ __forceinline__ TreeWalk<R> walk_of(const TreeDecodeArgs& a, const Start& s) {
    TreeWalk<R> w{a};
    w.at = s.at;
    w.end = s.end;
    w.before = s.before;
    w.b = s.b;
    w.units = s.units;
    w.G = a.Hq / a.Hkv;
    return w;
}

// As mbar_wait_w, with a first try that does not suspend, so that a lowered limit
// reaches waits that would end within it.
__device__ __forceinline__ bool wait_w(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    const bool ok = mbar_wait_on(bar, parity, abort_flag, err);
    return __all_sync(0xffffffffu, ok);
}

// ---- K and V -----------------------------------------------------------------------
// A warp's 32 rows of a tile: lane l finds the place of row 32 w + l (a page's row of
// this head, as a row of the pool) and whether any token of the walk reads it; what
// none reads comes as zeros, whatever is there.
struct Rows {
    uint32_t row;     // lane's
    uint32_t read;    // the warp's, a bit a row
};
__device__ __forceinline__ Rows rows_of(const TreeDecodeArgs& a, const TreeWork& w, int kt, int row32) {
    const int tok = tile_key<K>(w.s, w.far, kt) + row32 + (threadIdx.x & 31);
    const bool on = tok < w.s.base + w.s.n && (w.far || tok >= w.s.lo || tok < w.s.na);
    Rows r;
    r.row = 0;
    if (on) {
        const int p = a.block_table[static_cast<int64_t>(w.b) * a.max_pages + (tok >> a.page_lg)];
        const bool in = p >= 0 && p < a.num_pages;
        if (!in) atomicOr(a.err, kDevErrInput);
        r.row = (static_cast<uint32_t>(in ? p : 0) << a.page_lg) + (tok & ((1 << a.page_lg) - 1));
    }
    r.read = __ballot_sync(0xffffffffu, on);
    return r;
}

template <int D>
__device__ __forceinline__ void copy_rows(const TreeDecodeArgs& a, const void* pages, const Rows& rows, int h, uint32_t dst) {
    constexpr int P = D / 8, kPer = 32 / P;   // 16-byte pieces of a row; rows at a time
    const int lane = threadIdx.x & 31, piece = lane % P;
    const char* src = static_cast<const char*>(pages) + static_cast<size_t>(h) * (D * 2) + piece * 16;
    const size_t step = static_cast<size_t>(a.Hkv) * (D * 2);
    const uint32_t col = dst + (piece >> 3) * kHalf;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int r = i * kPer + lane / P;
        const uint32_t row = __shfl_sync(0xffffffffu, rows.row, r);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(col + r * 128 + (((piece & 7) ^ (r & 7)) << 4)),
                     "l"(src + row * step), "r"(rows.read >> r & 1 ? 16u : 0u)
                     : "memory");
    }
}

template <int D>
__device__ bool loader(const TreeDecodeArgs& a, const Ctx<D>& c, int w32) {
    constexpr int S = Sizes<D>::kSlots, kLag = Sizes<D>::kLag;
    const int lane = threadIdx.x & 31;
    const uint32_t ring = smem_u32(c.smem) + Sizes<D>::kTile + w32 * 32 * 128;
    uint32_t g = 0;   // slots filled (or, at the end, passed)
    // Starts slot g's copies; then slot g - kLag's have come, and are announced.
    auto fill = [&](const void* pages, const Rows* rows, int h) -> bool {
        if (rows) {
            const uint32_t slot = g % S;
            if (!wait_w(&c.bar[c.kEmpty + slot], (g / S & 1) ^ 1, c.abort_flag, a.err)) return false;
            copy_rows<D>(a, pages, *rows, h, ring + slot * Sizes<D>::kTile);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
        if (g >= kLag) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.bar[c.kFull + (g - kLag) % S]);
        }
        ++g;
        return true;
    };
    TreeWalk<R> walk = walk_of(a, *c.start);
    TreeWork w;
    while (walk.next(w)) {
        Rows next = rows_of(a, w, w.kt0, w32 * 32), now = next;
        for (int kt = w.kt0; kt <= w.kt1; ++kt) {
            const Rows last = now;
            now = next;
            if (kt + 1 < w.kt1) next = rows_of(a, w, kt + 1, w32 * 32);   // the page numbers are on their way during the copies
            if (kt < w.kt1 && !fill(a.k_pages, &now, w.h)) return false;
            if (kt > w.kt0 && !fill(a.v_pages, &last, w.h)) return false;
        }
    }
#pragma unroll 1
    for (int i = 0; i < kLag; ++i) fill(nullptr, nullptr, 0);
    return true;
}

// ---- Q ---------------------------------------------------------------------------------
template <int D>
__device__ bool q_loader(const TreeDecodeArgs& a, const Ctx<D>& c) {
    constexpr int P = D / 8, kPer = 32 / P;
    const int lane = threadIdx.x & 31, piece = lane % P;
    const uint32_t col = smem_u32(c.smem) + (piece >> 3) * kHalf;
    TreeWalk<R> walk = walk_of(a, *c.start);
    TreeWork w;
    for (uint32_t u = 0; walk.next(w); ++u) {
        if (!wait_w(&c.bar[c.kQEmpty], (u & 1) ^ 1, c.abort_flag, a.err)) return false;
        const int rows = min(R, w.s.n * walk.G - w.rt * R), each = tree_copy_rows(rows);
        for (int r0 = 0; r0 < R; r0 += 32) {
            const int in = (r0 & (each - 1)) + lane, mine = w.rt * R + in;
            int64_t at = -1;   // the lane's row of q
            if (in < rows)
                at = static_cast<int64_t>(w.s.first + a.plan.order[w.s.first + mine / walk.G]) * a.Hq + w.h * walk.G + mine % walk.G;
#pragma unroll 4
            for (int i = 0; i < P; ++i) {
                const int r = i * kPer + lane / P;
                const int64_t from = __shfl_sync(0xffffffffu, at, r);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(col + (r0 + r) * 128 + (((piece & 7) ^ (r & 7)) << 4)),
                             "l"(static_cast<const __nv_bfloat16*>(a.q) + max(from, static_cast<int64_t>(0)) * D + piece * 8), "r"(from >= 0 ? 16u : 0u)
                             : "memory");
            }
        }
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.bar[c.kQFull]);
    }
    return true;
}

// ---- MMA -----------------------------------------------------------------------------------
// Step j of a unit: S of tile j, then, its weights being there, O += P V of tile j - 1.
// A tile's S buffer is written again two tiles on, by this thread after the PV that
// read it.
template <int D>
__device__ bool mma_issuer(const TreeDecodeArgs& a, const Ctx<D>& c, uint32_t tmem) {
    constexpr int S = Sizes<D>::kSlots;
    constexpr uint32_t kIdescS = idesc_bf16_f32(R, K, false, false), kIdescO = idesc_bf16_f32(R, D, false, true);
    const uint64_t q = sdesc_sw128(smem_u32(c.smem), 16, 1024);
    const uint64_t k0 = sdesc_sw128(smem_u32(c.smem) + Sizes<D>::kTile, 16, 1024);
    const uint64_t v0 = sdesc_sw128(smem_u32(c.smem) + Sizes<D>::kTile, kHalf, 1024);
    uint32_t g = 0, tiles = 0, u = 0;
    auto full = [&]() { return wait_w(&c.bar[c.kFull + g % S], g / S & 1, c.abort_flag, a.err); };
    TreeWalk<R> walk = walk_of(a, *c.start);
    TreeWork w;
    for (; walk.next(w); ++u) {
        const int n = w.kt1 - w.kt0;
        if (!wait_w(&c.bar[c.kQFull], u & 1, c.abort_flag, a.err)) return false;
        for (int j = 0; j <= n; ++j) {
            if (j < n) {
                if (!full()) return false;
                tc_fence_after();
                const uint64_t k = k0 + (g % S) * (Sizes<D>::kTile >> 4);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint64_t off = ((i >> 2) * kHalf + (i & 3) * 32) >> 4;
                    umma_bf16_w(tmem + (tiles & 1) * K, q + off, k + off, kIdescS, i > 0 ? 1u : 0u);
                }
                umma_commit_w(&c.bar[c.kSFull + (tiles & 1)]);
                umma_commit_w(&c.bar[c.kEmpty + g % S]);
                if (j == n - 1) umma_commit_w(&c.bar[c.kQEmpty]);
                ++g;
                ++tiles;
            }
            if (j > 0) {
                const uint32_t t = tiles - (j < n ? 2 : 1);   // tile j - 1
                if (!wait_w(&c.bar[c.kPFull + (t & 1)], t >> 1 & 1, c.abort_flag, a.err)) return false;
                if (j == 1 && !wait_w(&c.bar[c.kOFree], (u & 1) ^ 1, c.abort_flag, a.err)) return false;
                if (!full()) return false;
                tc_fence_after();
                const uint64_t v = v0 + (g % S) * (Sizes<D>::kTile >> 4);
#pragma unroll
                for (int i = 0; i < 2 * K / 16; ++i)   // the nearest bf16, then what they leave
                    umma_bf16_ts_w(tmem + kColO, tmem + (t & 1) * K + i * 8, v + ((i % (K / 16)) * 16 * 128 >> 4), kIdescO,
                                   j == 1 && i == 0 ? 0u : 1u);
                umma_commit_w(&c.bar[c.kEmpty + g % S]);
                umma_commit_w(&c.bar[j == n ? c.kOFull : c.kODone]);
                ++g;
            }
        }
    }
    return true;
}

// ---- softmax ---------------------------------------------------------------------------------
// Bits of word [k0, k0 + 32) at keys [from, to).
__device__ __forceinline__ uint32_t below(int x) { return x <= 0 ? 0u : x >= 32 ? ~0u : (1u << x) - 1; }
__device__ __forceinline__ uint32_t bits_of(int k0, int from, int to) { return below(to - k0) & ~below(from - k0); }

// What a softmax thread knows of its row.
struct RowOf {
    const uint32_t* mask;
    int lo, base, anchors, n;
    bool on;
    float m, l;
};

// Weights of columns [C0, C0 + N) of the tile at key0, whose scores are in TMEM at
// ts, written over them with zeros for the other columns.  Returns the factor that
// the sums so far have to be scaled by.
template <int N>
__device__ __forceinline__ float weigh(RowOf& row, uint32_t ts, int c0, int key0, float sl) {
    uint32_t sr[N];
#pragma unroll
    for (int i = 0; i < N; i += 32) tmem_ld32(ts + c0 + i, sr + i);
    tmem_ld_wait();
    float* s = reinterpret_cast<float*>(sr);
    key0 += c0;
    const bool full = !row.on || (key0 + N <= row.base && (key0 >= row.lo || key0 + N <= row.anchors));
    if (!__all_sync(0xffffffffu, full)) {
#pragma unroll
        for (int i = 0; i < N / 32; ++i) {
            const int k0 = key0 + 32 * i, at = k0 - row.base;
            uint32_t bits = bits_of(k0, row.lo, row.base) | bits_of(k0, 0, row.anchors);
            if (row.on && at > -32 && at < row.n) {   // the tree's tokens at .. at + 31
                const int word = at >> 5;
                const uint32_t x = word >= 0 ? row.mask[word] : 0u, y = word + 1 < kWords ? row.mask[word + 1] : 0u;
                bits |= __funnelshift_r(x, y, at & 31);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) s[32 * i + e] = bits >> e & 1 ? s[32 * i + e] : -INFINITY;
        }
    }
    float m8[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) m8[t] = s[t];
#pragma unroll
    for (int i = 8; i < N; i += 16)
#pragma unroll
        for (int t = 0; t < 8; ++t) m8[t] = i + 8 + t < N ? fmax3(m8[t], s[i + t], s[i + 8 + t]) : fmaxf(m8[t], s[i + t]);
    const float mx = fmaxf(fmax3(m8[0], m8[1], m8[2]), fmax3(fmax3(m8[3], m8[4], m8[5]), m8[6], m8[7]));
    // The reference of the weights follows the maximum where that is over it by more
    // than 2^8: weights stay under 2^8, O is rescaled seldom.
    const float mn = fmaxf(row.m, mx * sl);
    float f = 1.f;
    if (mn > row.m + 8.f) {
        f = ex2_approx(row.m - mn);
        row.m = mn;
    }
    const float ref = row.m == -INFINITY ? 0.f : row.m;
    const float2 sl2 = make_float2(sl, sl), off = make_float2(-ref, -ref);
    float2 sum[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) sum[t] = make_float2(0.f, 0.f);
    constexpr int kAt = N == 128 ? 64 : N, kWide = kAt / 2;   // columns at a time, and those of TMEM they become
#pragma unroll
    for (int part = 0; part < N / kAt; ++part) {
        uint32_t hi[kWide], rest[kWide];
#pragma unroll
        for (int i = 0; i < kWide; ++i) {
            const int at = part * kAt + 2 * i;
            const float2 x = ffma2(make_float2(s[at], s[at + 1]), sl2, off);
            const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            sum[i & 3] = fadd2(sum[i & 3], p);
            hi[i] = pack_bf16x2(p.x, p.y);
            rest[i] = pack_bf16x2(p.x - __uint_as_float(hi[i] << 16), p.y - __uint_as_float(hi[i] & 0xffff0000u));
        }
        const uint32_t to = ts + c0 / 2 + part * kWide;
        if constexpr (kWide == 32) {
            tmem_st32(to, hi);
            tmem_st32(to + K / 2, rest);
        } else {
            tmem_st16(to, hi);
            tmem_st16(to + K / 2, rest);
        }
    }
    if constexpr (N < K) {
        uint32_t zero[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) zero[i] = 0;
#pragma unroll
        for (int i = 0; i < K / N; ++i) {
            if (i * N == c0) continue;
            if constexpr (N == 64) {
                tmem_st32(ts + i * 32, zero);
                tmem_st32(ts + K / 2 + i * 32, zero);
            } else {
                tmem_st16(ts + i * 16, zero);
                tmem_st16(ts + K / 2 + i * 16, zero);
            }
        }
    }
    const float2 s2 = fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3]));
    const bool had = row.l > 0.f;
    row.l = row.l * f + (s2.x + s2.y);
    return had ? f : 1.f;
}

template <int D>
__device__ bool softmax(const TreeDecodeArgs& a, const Ctx<D>& c, uint32_t tmem, int warp) {
    const int lane = threadIdx.x & 31, r = warp * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const uint32_t to = lanes + kColO;
    uint32_t tiles = 0, done = 0;
    TreeWalk<R> walk = walk_of(a, *c.start);
    TreeWork w;
    for (uint32_t u = 0; walk.next(w); ++u) {
        const int rows = min(R, w.s.n * walk.G - w.rt * R), each = tree_copy_rows(rows);
        const int in = r & (each - 1), first = (warp * 32) & (each - 1);
        const bool any = first < rows;   // the warp has rows
        const int c0 = warp * 32 / each * each;   // its copy's columns, as many as the copy has rows
        RowOf row{nullptr, 0, w.s.base, min(a.n_anchor, w.s.base), w.s.n, in < rows, -INFINITY, 0.f};
        if (row.on) {
            const int tok = w.s.first + a.plan.order[w.s.first + (w.rt * R + in) / walk.G];
            row.lo = a.plan.lo[tok];
            row.mask = a.plan.mask + static_cast<size_t>(tok) * kWords;
        }
        for (int kt = w.kt0; kt < w.kt1; ++kt, ++tiles) {
            const int key0 = tile_key<K>(w.s, w.far, kt);
            if (!wait_w(&c.bar[c.kSFull + (tiles & 1)], tiles >> 1 & 1, c.abort_flag, a.err)) return false;
            tc_fence_after();
            if (any) {
                const uint32_t ts = lanes + (tiles & 1) * K;
                const float f = each == 32   ? weigh<32>(row, ts, c0, key0, a.scale_log2)
                                : each == 64 ? weigh<64>(row, ts, c0, key0, a.scale_log2)
                                             : weigh<128>(row, ts, 0, key0, a.scale_log2);
                // O may be rescaled once the last tile's PV has landed; every PV but a
                // unit's last one arrives at kODone.
                if (__any_sync(0xffffffffu, row.on && f != 1.f)) {
                    if (!wait_w(&c.bar[c.kODone], done & 1, c.abort_flag, a.err)) return false;
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < D; i += 32) {
                        uint32_t o[32];
                        tmem_ld32(to + i, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int t = 0; t < 32; ++t) o[t] = __float_as_uint(__uint_as_float(o[t]) * f);
                        tmem_st32(to + i, o);
                    }
                }
                tmem_st_wait();
            }
            if (kt > w.kt0) ++done;
            tc_fence_before();
            mbar_arrive(&c.bar[c.kPFull + (tiles & 1)]);
        }
        if (!wait_w(&c.bar[c.kOFull], u & 1, c.abort_flag, a.err)) return false;
        tc_fence_after();
        if (any) {
            float* part = a.plan.part + static_cast<size_t>(w.slot) * R * (D + 2);
#pragma unroll
            for (int i = 0; i < D; i += 32) {
                uint32_t o[32];
                tmem_ld32(to + i, o);
                tmem_ld_wait();
                if (row.on)
#pragma unroll
                    for (int t = 0; t < 32; t += 4)
                        *reinterpret_cast<uint4*>(part + r * D + i + t) = make_uint4(o[t], o[t + 1], o[t + 2], o[t + 3]);
            }
            if (row.on) reinterpret_cast<float2*>(part + R * D)[r] = make_float2(row.m, row.l);
        }
        tc_fence_before();
        mbar_arrive(&c.bar[c.kOFree]);
    }
    return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) tree_tc_kernel(const __grid_constant__ TreeDecodeArgs a) {
    extern __shared__ uint8_t raw[];
    using Z = Sizes<D>;
    Ctx<D> c;
    c.smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
    c.bar = reinterpret_cast<uint64_t*>(c.smem + Z::kOffBar);
    Start* start = reinterpret_cast<Start*>(c.smem + Z::kOffMisc);
    c.start = start;
    c.abort_flag = reinterpret_cast<volatile int*>(c.smem + Z::kOffMisc + 40);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(c.smem + Z::kOffMisc + 44);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < Z::kSlots; ++i) {
            mbar_init(&c.bar[c.kFull + i], kLoaders);
            mbar_init(&c.bar[c.kEmpty + i], 1);
        }
        mbar_init(&c.bar[c.kQFull], 1);
        mbar_init(&c.bar[c.kQEmpty], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c.bar[c.kSFull + i], 1);
            mbar_init(&c.bar[c.kPFull + i], R);
        }
        mbar_init(&c.bar[c.kODone], 1);
        mbar_init(&c.bar[c.kOFull], 1);
        mbar_init(&c.bar[c.kOFree], R);
        mbar_init(&c.bar[c.kDrain], 1);
        *c.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 4) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");   // for the plan
    if (warp == 0) {
        TreeWalk<R> walk{a};
        start_walk<R>(a, walk);
        if (lane == 0) *start = Start{walk.at, walk.end, walk.before, walk.b, walk.units};
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (warp < 4) {
        warpgroup_reg_inc<kRegsSoftmax>();
        softmax<D>(a, c, tmem, warp);
    } else {
        warpgroup_reg_dec<kRegsOther>();
        if (warp == 4) {
            mma_issuer<D>(a, c, tmem);
            umma_commit_w(&c.bar[c.kDrain]);   // all that was issued
            mbar_drain(&c.bar[c.kDrain], 0);
        } else if (warp == 5) {
            q_loader<D>(a, c);
        } else if (warp >= 8) {
            loader<D>(a, c, warp - 8);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D>
cudaError_t launch(const TreeDecodeArgs& a, int ctas, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_dynamic_smem(tree_tc_kernel<D>, Sizes<D>::kBytes, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = dependent_launch(ctas, kThreads, s, attr);
    cfg.dynamicSmemBytes = Sizes<D>::kBytes;
    return cudaLaunchKernelEx(&cfg, tree_tc_kernel<D>, a);
}

}  // namespace

cudaError_t launch_tree_tc(const TreeDecodeArgs& a, int d, int ctas, cudaStream_t s) {
    return d == 128 ? launch<128>(a, ctas, s) : launch<64>(a, ctas, s);
}

cudaError_t tree_set_wait_limit(uint64_t ns) { return set_wait_limit_of_unit(ns); }

}  // namespace swi

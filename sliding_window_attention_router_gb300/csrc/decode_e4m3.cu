// Decode over a paged cache of 8-bit keys and values: one query a sequence
// against the window, the anchors and the window, or the whole history, of
// e4m3 rows that each carry a power of two.
//
// The mathematics, for one query head and the visited keys j, in base 2:
//   s_j = scale log2(e) 2^(ku_j - 127) <q, k8_j>,   t_j = s_j + vu_j - 127,
//   l = sum_j 2^(s_j - m),      a = sum_j 2^(t_j - n) v8_j,
//   o = 2^(n - m) a / l,        lse = ln 2 (m + log2 l),
// with m and n the largest s_j and t_j.  Folding a value row's power of two
// into its weight leaves the e4m3 bytes as they are; the weights then have a
// maximum of their own, n, so that what is rounded to 16 bits is always of
// order 1 at the largest contribution, whatever the rows' sizes.  Parts (m,
// n, l, a) of the key set join by their maxima.
//
// The products run on mma.sync m16n8k16 (fp16 in, fp32 accumulate).  An e4m3
// value is exact in fp16, and q is made so by a power of two per head (exact
// for every element within 2^31 of the head's largest).  The weights are
// rounded to fp16, 2^-11 of each, under the bf16 result's own 2^-8.  The
// bound is the cache's bytes, not the products: 16 keys of one head (4 KiB at
// d = 128) take 16 products for up to 8 query heads, a small part of the
// tensor rate, so the register path (no shared-memory staging, no TMEM) is
// the short one:
//   S^T [16 keys x 8 heads] = K Q^T: a thread's 16-byte pieces of two key rows
//   are its A fragments after conversion, the order of d being free as long
//   as q's fragments follow it;
//   O^T [d x 8 heads] += V^T W^T: a thread's 16-byte pieces of four value rows
//   are its A fragments after pairing bytes of neighbouring rows (one byte
//   permute for two registers), and W^T comes from S^T by two 8 x 8
//   transposes inside the warp.

#include "swiattn.h"
#include "swiattn_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>
#include <atomic>

namespace swi {
namespace {

constexpr int kTile = 16;        // keys of one product tile
constexpr int kWarps = 4;        // warps of a block; they take a chunk's tiles in turn
constexpr int kStages = 3;       // tiles a warp holds: one at work, two on their way
constexpr int kBlocksPerSm = 4;
constexpr int kMinChunk = 64;    // keys of a chunk (one block's work at a time)
constexpr int kMaxChunk = 512;
constexpr int kChunksWanted = 8; // of a visit shorter than kChunksWanted * kMaxChunk
constexpr float kSlack = 8.f;    // base-2 units a score may pass its reference (weights up to 256)

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What to subtract from scores whose maximum is x: a maximum of -inf (no key
// yet, or scores that are all -inf or NaN) must not make -inf - -inf.
__device__ __forceinline__ float finite_or_0(float x) { return x == -INFINITY ? 0.f : x; }

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes the 8 x 8 matrix of 16-bit elements that the warp's registers hold.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Two e4m3 bytes (the low or high half of w) as a pair of fp16.
__device__ __forceinline__ uint32_t half2_of(uint32_t w, int high) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(high ? w >> 16 : w & 0xffffu),
                                                     __NV_E4M3);
    return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {   // zeros where not on
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global.L2::128B [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(on ? 8 : 0)
                 : "memory");
}

// Keys sequence b visits: anchors [0, na) and [lo, len).  Chunks are runs of
// `tiles` 16-key tiles at multiples of 16 from the cache's start, so that a
// tile never straddles a page of 16 or more; the first nca chunks are
// anchors'.  The chunk length depends on the visit alone, so a sequence's
// result does not depend on the rest of the batch.
struct Visit {
    int len, lo, na;
    int tiles;      // tiles of a chunk
    int nca, nc;    // chunks: anchors', all
};
__device__ __forceinline__ Visit visit_of(const DecodeE4m3Args& a, int raw_len, int gate) {
    Visit v;
    v.len = min(max(raw_len, 0), a.max_pages << a.page_lg);
    v.lo = gate ? 0 : max(0, v.len - a.W);
    v.na = min(a.n_anchor, v.lo);
    const int m = v.na + v.len - v.lo;
    int chunk = kMinChunk;
    while (chunk < kMaxChunk && chunk * kChunksWanted < m) chunk <<= 1;
    v.tiles = chunk / kTile;
    const int ta = (v.na + kTile - 1) / kTile;
    const int tw = v.len > 0 ? (v.len + kTile - 1) / kTile - v.lo / kTile : 0;
    v.nca = (ta + v.tiles - 1) / v.tiles;
    v.nc = v.nca + (tw + v.tiles - 1) / v.tiles;
    return v;
}

// Shared memory of a block: each thread's own queue of the 16-byte pieces it
// loads (piece p of stage s of a warp: 32 lanes side by side), so nothing is
// exchanged through it and no bank is met twice; after the last tile the same
// bytes hold the warps' sums.
template <int D>
constexpr int kStageBytes = kTile * 2 * D;   // of one warp
template <int D>
constexpr int kSharedBytes = kWarps * kStages * kStageBytes<D>;

// A unit of work: chunk c of KV head h of sequence b.  Blocks are persistent
// and take units blockIdx.x, blockIdx.x + gridDim.x, ... of the batch's (a
// unit's heads side by side, so that neighbouring blocks read neighbouring
// bytes of the same tokens).  Each warp finds its block's units by itself: it
// holds the visits of 32 sequences, one a lane, and moves on to the next 32
// when the unit lies behind them.
struct Units {
    Visit mine;        // of sequence first + lane
    int first;         // first sequence held
    int before, total; // chunks of the held sequences: before this lane's, of all
    unsigned c;        // the unit: chunk index from the first held sequence's first
    int h;

    __device__ void hold(const DecodeE4m3Args& a, int from) {
        const int lane = threadIdx.x & 31, b = from + lane;
        first = from;
        mine = visit_of(a, b < a.B ? a.seq_lens[b] : 0, b < a.B ? a.gate[b] : 0);
        int sum = mine.nc;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        before = sum - mine.nc;
        total = __shfl_sync(0xffffffffu, sum, 31);
    }
    // Finds the unit's sequence; false: there are no more.
    __device__ bool find(const DecodeE4m3Args& a, int& b, int& chunk, Visit& v) {
        while (c >= static_cast<unsigned>(total)) {
            c -= total;
            if (first + 32 >= a.B) return false;
            hold(a, first + 32);
        }
        const int ci = static_cast<int>(c);
        const int at = __ffs(__ballot_sync(0xffffffffu, ci >= before && ci < before + mine.nc)) - 1;
        b = first + at;
        chunk = ci - __shfl_sync(0xffffffffu, before, at);
        v.len = __shfl_sync(0xffffffffu, mine.len, at);
        v.lo = __shfl_sync(0xffffffffu, mine.lo, at);
        v.na = __shfl_sync(0xffffffffu, mine.na, at);
        v.tiles = __shfl_sync(0xffffffffu, mine.tiles, at);
        v.nca = __shfl_sync(0xffffffffu, mine.nca, at);
        return true;
    }
};

// NH: groups of eight query heads (1: Hq/Hkv <= 8, 2: <= 16).
template <int D, int NH>
__global__ void __launch_bounds__(kWarps * 32, NH == 1 ? kBlocksPerSm : 2) decode_e4m3_split_kernel(DecodeE4m3Args a) {
    constexpr int KS = D / 16;    // 16-deep steps of the score product, and 16-row tiles of O^T
    constexpr int KW = D / 64;    // 16-byte pieces of a key row a thread holds
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint8_t s_exp[kWarps][kStages][32];
    __shared__ float s_m[kWarps][NH * 8], s_n[kWarps][NH * 8], s_l[kWarps][NH * 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int G = a.Hq / a.Hkv;
    uint8_t* const queue = smem + warp * kStages * kStageBytes<D>;
    const uint32_t queue_s = static_cast<uint32_t>(__cvta_generic_to_shared(queue));

    if (blockIdx.x == 0)   // lengths that are clamped
        for (int i = threadIdx.x; i < a.B; i += kWarps * 32) {
            const int raw = a.seq_lens[i];
            if (raw < 0 || raw > (a.max_pages << a.page_lg)) atomicOr(a.err, kDevErrInput);
        }

    Units unit;
    unit.hold(a, 0);
    unit.c = blockIdx.x / a.Hkv;
    unit.h = blockIdx.x % a.Hkv;
    const unsigned step_c = gridDim.x / a.Hkv;
    const int step_h = gridDim.x % a.Hkv;
    int b, c;
    Visit vis;
    for (; unit.find(a, b, c, vis);) {
    const int h = unit.h;
    unit.c += step_c;
    unit.h += step_h;
    if (unit.h >= a.Hkv) {
        unit.h -= a.Hkv;
        ++unit.c;
    }

    // This chunk's tiles and the keys of them that are visited, [from, to);
    // this warp's are tile0, tile0 + kWarps, ..., `count` of them.
    int tile0, from, to;
    if (c < vis.nca) {
        from = 0;
        to = vis.na;
        tile0 = c * vis.tiles;
    } else {
        from = vis.lo;
        to = vis.len;
        tile0 = vis.lo / kTile + (c - vis.nca) * vis.tiles;
    }
    const int tile1 = min(tile0 + vis.tiles, (to + kTile - 1) / kTile);
    tile0 += warp;
    const int count = max(0, (tile1 - tile0 + kWarps - 1) / kWarps);

    // Pool row of key (lane & 15) of this warp's i-th tile (a key that is not
    // visited: of one that is, and its bytes are not copied).
    const int32_t* table = a.block_table + static_cast<size_t>(b) * a.max_pages;
    auto row_of = [&](int i) -> uint32_t {
        const int tok = min(max((tile0 + i * kWarps) * kTile + (lane & 15), from), to - 1);
        int p = table[tok >> a.page_lg];
        if (p < 0 || p >= a.num_pages) {
            atomicOr(a.err, kDevErrInput);
            p = 0;
        }
        return (static_cast<uint32_t>(p) << a.page_lg) + (tok & ((1 << a.page_lg) - 1));
    };
    // Starts the copies of tile i, whose rows are `row` (lane by lane).
    auto issue = [&](int i, uint32_t row) {
        const int base = (tile0 + i * kWarps) * kTile;
        const uint32_t dst = queue_s + (i % kStages) * kStageBytes<D>;
#pragma unroll
        for (int r = 0; r < 2; ++r) {   // keys g and 8 + g
            const int j = g + 8 * r;
            const size_t at = static_cast<size_t>(__shfl_sync(0xffffffffu, row, j)) * a.Hkv + h;
            const bool on = base + j >= from && base + j < to;
#pragma unroll
            for (int w = 0; w < KW; ++w)
                copy16(dst + ((r * KW + w) * 32 + lane) * 16, a.k_pages + at * D + w * 64 + t * 16, on);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {   // values of keys 2t, 2t + 1, 2t + 8, 2t + 9
            const int j = 2 * t + (r & 1) + 8 * (r >> 1);
            const size_t at = static_cast<size_t>(__shfl_sync(0xffffffffu, row, j)) * a.Hkv + h;
            const bool on = base + j >= from && base + j < to;
            const uint8_t* src = a.v_pages + at * D + g * (D / 8);
            const uint32_t to_s = dst + 2 * KW * 512 + (r * 32 + lane) * (D / 8);
            if constexpr (D == 128) copy16(to_s, src, on);
            else copy8(to_s, src, on);
        }
    };
    // Exponent byte of key (lane & 15): of its K row in lanes 0-15, its V row in 16-31.
    auto exponent_of = [&](uint32_t row) -> uint32_t {
        const size_t at = ((static_cast<size_t>(row >> a.page_lg) * a.Hkv + h) << a.page_lg) +
                          (row & ((1u << a.page_lg) - 1));
        return (lane < 16 ? a.k_exp : a.v_exp)[at];
    };

    uint32_t first_row[kStages - 1], next_row = 0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) first_row[i] = i < count ? row_of(i) : 0;
    if (kStages - 1 < count) next_row = row_of(kStages - 1);

    // Query fragments: head g (and 8 + g), dims 16 t .. 16 t + 15 of each 64.
    uint32_t qf[NH][KS][2];
    float fs[NH][2];   // scale log2(e) 2^-qe of the thread's columns, heads 2t and 2t + 1
#pragma unroll
    for (int n = 0; n < NH; ++n) {
        const int head = n * 8 + g;
        float x[KW * 16];
        float amax = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            uint4 u[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            if (head < G) {
                const uint4* src = reinterpret_cast<const uint4*>(
                    static_cast<const __nv_bfloat16*>(a.q) + (static_cast<size_t>(b) * a.Hq + h * G + head) * D + w * 64 + t * 16);
                u[0] = src[0];
                u[1] = src[1];
            }
            const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(u);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 f = __bfloat1622float2(p[e]);
                x[w * 16 + 2 * e] = f.x;
                x[w * 16 + 2 * e + 1] = f.y;
                amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^qe takes the head's largest element to [2^14, 2^15).
        const int qe = min(126, 14 + 127 - static_cast<int>(__float_as_uint(amax) >> 23));
        const float up = __uint_as_float(static_cast<uint32_t>(qe + 127) << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int r = 0; r < 2; ++r) qf[n][s][r] = pack_half2(x[4 * s + 2 * r] * up, x[4 * s + 2 * r + 1] * up);
        const float down = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - qe) << 23);
        fs[n][0] = __shfl_sync(0xffffffffu, down, (2 * t) * 4);
        fs[n][1] = __shfl_sync(0xffffffffu, down, (2 * t + 1) * 4);
    }

    float acc[NH][KS][4];
    float m[NH][2], nmax[NH][2], l[NH][2];
#pragma unroll
    for (int n = 0; n < NH; ++n) {
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][j][e] = 0.f;
        m[n][0] = m[n][1] = nmax[n][0] = nmax[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
    }

    uint32_t last_exp = 0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        if (i < count) issue(i, first_row[i]);
        if (i > 0 && i - 1 < count) s_exp[warp][i - 1][lane] = static_cast<uint8_t>(last_exp);
        if (i < count) last_exp = exponent_of(first_row[i]);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    for (int i = 0; i < count; ++i) {
        // The exponents of the tile issued last have arrived by now; then the
        // next tile's copies start, in the stage that the last one left.
        const int ahead = i + kStages - 1;
        if (ahead - 1 < count) s_exp[warp][(ahead - 1) % kStages][lane] = static_cast<uint8_t>(last_exp);
        if (ahead < count) {
            issue(ahead, next_row);
            last_exp = exponent_of(next_row);
            if (ahead + 1 < count) next_row = row_of(ahead + 1);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();
        const int base = (tile0 + i * kWarps) * kTile;
        const uint8_t* stage = queue + (i % kStages) * kStageBytes<D>;
        uint4 kw[2][KW];
        uint32_t vw[4][D / 32];
        int ku[2], vu[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int w = 0; w < KW; ++w)
                kw[r][w] = *reinterpret_cast<const uint4*>(stage + ((r * KW + w) * 32 + lane) * 16);
            ku[r] = s_exp[warp][i % kStages][g + 8 * r];
            vu[r] = s_exp[warp][i % kStages][16 + g + 8 * r];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint8_t* src = stage + 2 * KW * 512 + (r * 32 + lane) * (D / 8);
            if constexpr (D == 128) {
                const uint4 u = *reinterpret_cast<const uint4*>(src);
                vw[r][0] = u.x, vw[r][1] = u.y, vw[r][2] = u.z, vw[r][3] = u.w;
            } else {
                const uint2 u = *reinterpret_cast<const uint2*>(src);
                vw[r][0] = u.x, vw[r][1] = u.y;
            }
        }
        __syncwarp();   // every lane has read the stage's exponents

        // Scores: rows key g and 8 + g, columns heads 2t and 2t + 1.
        float s[NH][4];
#pragma unroll
        for (int n = 0; n < NH; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        const uint32_t* k0 = reinterpret_cast<const uint32_t*>(kw[0]);
        const uint32_t* k1 = reinterpret_cast<const uint32_t*>(kw[1]);
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const uint32_t a0 = half2_of(k0[i], 0), a1 = half2_of(k1[i], 0);
            const uint32_t a2 = half2_of(k0[i], 1), a3 = half2_of(k1[i], 1);
#pragma unroll
            for (int n = 0; n < NH; ++n) mma_f16(s[n], a0, a1, a2, a3, qf[n][i][0], qf[n][i][1]);
        }
        // s_j and t_j, and whether one is over kSlack above the reference it
        // would be subtracted from.
        float x[NH][4], y[NH][4];
        bool over = false;
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = e >> 1, tok = base + g + 8 * r;
                const bool on = tok >= from && tok < to;
                x[n][e] = on ? s[n][e] * fs[n][e & 1] * __uint_as_float(static_cast<uint32_t>(ku[r]) << 23) : -INFINITY;
                y[n][e] = x[n][e] + static_cast<float>(vu[r] - 127);
                over |= x[n][e] > m[n][e & 1] + kSlack || y[n][e] > nmax[n][e & 1] + kSlack;
            }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int col = 0; col < 2; ++col) {
                    float xm = fmaxf(x[n][col], x[n][col + 2]), ym = fmaxf(y[n][col], y[n][col + 2]);
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        xm = fmaxf(xm, __shfl_xor_sync(0xffffffffu, xm, o));
                        ym = fmaxf(ym, __shfl_xor_sync(0xffffffffu, ym, o));
                    }
                    const float mn = fmaxf(m[n][col], xm), nn = fmaxf(nmax[n][col], ym);
                    l[n][col] *= ex2f(m[n][col] - finite_or_0(mn));
                    const float ca = ex2f(nmax[n][col] - finite_or_0(nn));
#pragma unroll
                    for (int j = 0; j < KS; ++j) {
                        acc[n][j][col] *= ca;
                        acc[n][j][col + 2] *= ca;
                    }
                    m[n][col] = mn;
                    nmax[n][col] = nn;
                }
        }
        uint32_t wt[NH][2];
#pragma unroll
        for (int n = 0; n < NH; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = e & 1;
                l[n][col] += ex2f(x[n][e] - finite_or_0(m[n][col]));
                y[n][e] = ex2f(y[n][e] - finite_or_0(nmax[n][col]));
            }
            wt[n][0] = transpose8x8(pack_half2(y[n][0], y[n][1]));
            wt[n][1] = transpose8x8(pack_half2(y[n][2], y[n][3]));
        }
        // O^T: tile i holds dims D/8 g + 2 i (rows g) and + 1 (rows 8 + g).
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const uint32_t sel = (i & 1) ? 0x7362 : 0x5140;
            const uint32_t lo = __byte_perm(vw[0][i / 2], vw[1][i / 2], sel);
            const uint32_t hi = __byte_perm(vw[2][i / 2], vw[3][i / 2], sel);
            const uint32_t a0 = half2_of(lo, 0), a1 = half2_of(lo, 1), a2 = half2_of(hi, 0), a3 = half2_of(hi, 1);
#pragma unroll
            for (int n = 0; n < NH; ++n) mma_f16(acc[n][i], a0, a1, a2, a3, wt[n][0], wt[n][1]);
        }
    }

    // Join the warps: their references, then their sums relative to the
    // block's, through the queue's bytes.
    float* part = a.part + ((static_cast<size_t>(b) * a.Hq + h * G) * a.max_chunks + c) * (D + 4);
    const size_t head_step = static_cast<size_t>(a.max_chunks) * (D + 4);
    float* const s_acc = reinterpret_cast<float*>(smem);
    static_assert(kSharedBytes<D> >= kWarps * 8 * D * 4, "the sums of eight heads fit the queue");
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int col = 0; col < 2; ++col) {
            float ls = l[n][col];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
            if (g == 0) {
                s_m[warp][n * 8 + 2 * t + col] = m[n][col];
                s_n[warp][n * 8 + 2 * t + col] = nmax[n][col];
                s_l[warp][n * 8 + 2 * t + col] = ls;
            }
        }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NH; ++n) {
#pragma unroll
        for (int col = 0; col < 2; ++col) {
            const int head = 2 * t + col;
            float top = s_n[0][n * 8 + head];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_n[w][n * 8 + head]);
            const float f = ex2f(nmax[n][col] - finite_or_0(top));   // 0 for a warp without a tile
            if (n * 8 + head < G) {
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    s_acc[(warp * 8 + head) * D + g * (D / 8) + 2 * j] = acc[n][j][col] * f;
                    s_acc[(warp * 8 + head) * D + g * (D / 8) + 2 * j + 1] = acc[n][j][col + 2] * f;
                }
            }
        }
        __syncthreads();
        const int heads = min(8, G - n * 8);
        for (int i = threadIdx.x; i < heads * D; i += kWarps * 32) {
            const int head = i / D, col = i % D;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += s_acc[(w * 8 + head) * D + col];
            part[(n * 8 + head) * head_step + col] = sum;
        }
        __syncthreads();
    }
    if (threadIdx.x < G) {
        const int head = threadIdx.x;
        float top = s_m[0][head], topn = s_n[0][head];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            top = fmaxf(top, s_m[w][head]);
            topn = fmaxf(topn, s_n[w][head]);
        }
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += s_l[w][head] * ex2f(s_m[w][head] - finite_or_0(top));
        float* dst = part + head * head_step + D;
        dst[0] = top;
        dst[1] = topn;
        dst[2] = sum;
    }
    __syncthreads();   // s_m, s_n, s_l and the queue are free again
    }   // next unit
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Joins the chunks of one (query head, sequence): block (hq, b), kJoin groups
// of D threads; group i sums chunks i, i + kJoin, ..., and the groups' sums are
// added in order.  Launched as a programmatic dependent of the split kernel:
// it reads the visit, an input, and then waits for that grid's memory.
constexpr int kJoin = 4;
template <int D>
__global__ void __launch_bounds__(kJoin * D) decode_e4m3_join_kernel(DecodeE4m3Args a) {
    __shared__ float s_top[2][kJoin * D / 32];
    __shared__ float s_sum[kJoin][D], s_l[kJoin];
    const int hq = blockIdx.x, b = blockIdx.y, col = threadIdx.x % D, grp = threadIdx.x / D;
    const Visit vis = visit_of(a, a.seq_lens[b], a.gate[b]);
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + (static_cast<size_t>(b) * a.Hq + hq) * D;
    const float* part = a.part + (static_cast<size_t>(b) * a.Hq + hq) * a.max_chunks * (D + 4);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (vis.nc == 0) {   // an empty slot
        if (grp == 0) o[col] = __float2bfloat16_rn(0.f);
        if (a.lse && threadIdx.x == 0) a.lse[static_cast<size_t>(b) * a.Hq + hq] = -INFINITY;
        return;
    }
    float m = -INFINITY, n = -INFINITY;
    for (int c = threadIdx.x; c < vis.nc; c += kJoin * D) {
        const float2 p = *reinterpret_cast<const float2*>(part + static_cast<size_t>(c) * (D + 4) + D);
        m = fmaxf(m, p.x);
        n = fmaxf(n, p.y);
    }
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
        n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, i));
    }
    if ((threadIdx.x & 31) == 0) {
        s_top[0][threadIdx.x / 32] = m;
        s_top[1][threadIdx.x / 32] = n;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoin * D / 32; ++i) {
        m = fmaxf(m, s_top[0][i]);
        n = fmaxf(n, s_top[1][i]);
    }
    const float mr = finite_or_0(m), nr = finite_or_0(n);
    float l = 0.f, sum = 0.f;
#pragma unroll 4
    for (int c = grp; c < vis.nc; c += kJoin) {
        const float* p = part + static_cast<size_t>(c) * (D + 4);
        const float4 st = *reinterpret_cast<const float4*>(p + D);
        l += st.z * ex2f(st.x - mr);
        sum += p[col] * ex2f(st.y - nr);
    }
    s_sum[grp][col] = sum;
    if (col == 0) s_l[grp] = l;
    __syncthreads();
    if (grp != 0) return;
#pragma unroll
    for (int i = 1; i < kJoin; ++i) {
        sum += s_sum[i][col];
        l += s_l[i];
    }
    o[col] = __float2bfloat16_rn(sum / l * ex2f(n - m));
    if (a.lse && col == 0) a.lse[static_cast<size_t>(b) * a.Hq + hq] = (m + __log2f(l)) * 0.69314718055994531f;
}

template <int D, int NH>
cudaError_t launch_split(const DecodeE4m3Args& a, int sms, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_dynamic_smem(decode_e4m3_split_kernel<D, NH>, kSharedBytes<D>, done);
    if (e != cudaSuccess) return e;
    const int64_t units = static_cast<int64_t>(a.B) * a.Hkv * a.max_chunks;
    const int64_t most = static_cast<int64_t>(sms) * kBlocksPerSm;
    decode_e4m3_split_kernel<D, NH><<<static_cast<unsigned>(units < most ? units : most), kWarps * 32, kSharedBytes<D>, s>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const DecodeE4m3Args& a, int sms, cudaStream_t s) {
    prof_start(s);
    cudaError_t e = a.Hq / a.Hkv <= 8 ? launch_split<D, 1>(a, sms, s) : launch_split<D, 2>(a, sms, s);
    prof_stop(s);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.Hq, a.B);
    cfg.blockDim = dim3(kJoin * D);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, decode_e4m3_join_kernel<D>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// A visit of v keys (v <= max_len + min(n_anchor, max_len)) has at most
// v / chunk + 2.75 chunks (two segments, each cut at multiples of 16 keys, of
// at least four tiles a chunk): kChunksWanted + 2 where the chunk is below
// kMaxChunk (then kChunksWanted chunks hold v), else ceil(v / kMaxChunk) + 2.
int decode_e4m3_max_chunks(int64_t max_len, int n_anchor) {
    const int64_t v = max_len + (n_anchor < max_len ? n_anchor : max_len);
    const int64_t longest = (v + kMaxChunk - 1) / kMaxChunk;
    return static_cast<int>((longest > kChunksWanted ? longest : kChunksWanted) + 3);
}

size_t decode_e4m3_workspace_bytes(int B, int Hq, int d, int max_chunks) {
    const size_t n = sizeof(float) * static_cast<size_t>(B) * Hq * max_chunks * (d + 4);
    return (n + 255) & ~static_cast<size_t>(255);
}

cudaError_t launch_decode_e4m3(const DecodeE4m3Args& a, int d, int sms, cudaStream_t s) {
    return d == 128 ? launch_d<128>(a, sms, s) : launch_d<64>(a, sms, s);
}

}  // namespace swi

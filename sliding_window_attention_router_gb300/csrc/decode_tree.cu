// Attention of drafted tokens that form a tree, over a paged cache: the plan, the
// products on CUDA cores, the join, and the choice between these products and the
// tensor cores' (decode_tree_tc.cu).
//
// The mathematics, for a row (token t, query head) and the entries j it reads, in
// base 2:  s_j = scale log2(e) <q, k_j>,  m = max s_j,  l = sum 2^(s_j - m),
//   o = sum 2^(s_j - m) v_j / l,   lse = ln 2 (m + log2 l).
// Parts (m, l, o l) over disjoint sets of entries join by their maxima.
// Token t at depth x of the tree after `base` cached tokens stands at position
// base + x.  It reads the cached entries j < base and those of the tokens on its
// path, itself among them, that a decode step at its position would: with its gate
// set all of them, else those whose positions are above base + x - W or below the
// number of anchors.

#include "swiattn.h"
#include "ptx.cuh"
#include "tree_plan.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>
#include <algorithm>
#include <atomic>

namespace swi {
namespace {

constexpr int kWords = kMaxTree / 32;

// ---- the plan ----------------------------------------------------------------
// The r > 0 lowest set bits of x (a call: 16 copies in line made the plan of trees that do not
// need it 1 us slower).
__device__ __noinline__ uint32_t lowest(uint32_t x, int r) {
    if (r >= __popc(x)) return x;
    int p = 0;   // the most bits of which no more than r are set
#pragma unroll
    for (int step = 16; step > 0; step >>= 1)
        if (__popc(x & ((1u << (p + step)) - 1)) <= r) p += step;
    return x & ((1u << p) - 1);
}

// Block b: sequence b's tokens, one a thread.  The paths come by doubling: after r
// rounds mask[t] holds the 2^r last tokens of t's path, and up[t] the one before
// them.
__global__ void __launch_bounds__(kMaxTree) tree_plan_kernel(const __grid_constant__ TreeDecodeArgs a, int rows, int keys) {
    __shared__ uint32_t s_mask[2][kWords][kMaxTree];
    __shared__ short s_up[2][kMaxTree];
    __shared__ int s_count[kMaxTree / 32], s_bad;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    if (t == 0) s_bad = 0;
    const int first = a.starts[b], after = a.starts[b + 1], len = a.seq_lens[b];   // on their way while the others are looked at
    __syncthreads();
    // Sequences must not overlap: the workspace has room for each token once.
    bool bad = t == 0 && (a.starts[0] < 0 || a.starts[a.B] > a.T);
    for (int i = t; i < a.B; i += kMaxTree) bad |= a.starts[i + 1] < a.starts[i];
    if (bad) s_bad = 1;
    __syncthreads();
    bad = s_bad != 0;
    int n = bad ? 0 : after - first;
    if (!bad && len != 0 && (n > kMaxTree || len < n || len > (a.max_pages << a.page_lg))) bad = true;   // with or without drafts
    if (bad || len == 0) n = 0;   // an empty slot has no tokens to look at
    const int base = len - n;

    const bool on = t < n;
    const bool gate = on && a.gate[first + t] != 0;
    int up = -1;
    if (on) {
        up = a.parents ? a.parents[first + t] : t - 1;
        if (up >= t) bad = true;
        if (up >= t || up < 0) up = -1;
    }
    if (bad) atomicOr(a.err, kDevErrInput);
#pragma unroll
    for (int w = 0; w < kWords; ++w) s_mask[0][w][t] = on && w == warp ? 1u << lane : 0u;
    s_up[0][t] = static_cast<short>(up);
    __syncthreads();
    int cur = 0;
    for (int reach = 1; reach < n; reach *= 2, cur ^= 1) {
        const int p = s_up[cur][t];
#pragma unroll
        for (int w = 0; w < kWords; ++w) s_mask[cur ^ 1][w][t] = s_mask[cur][w][t] | (p >= 0 ? s_mask[cur][w][p] : 0u);
        s_up[cur ^ 1][t] = p >= 0 ? s_up[cur][p] : static_cast<short>(-1);
        __syncthreads();
    }
    uint32_t mask[kWords];
    int depth = -1;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        mask[w] = s_mask[cur][w][t];
        depth += __popc(mask[w]);
    }
    // Routed tokens first, each kind in its order.
    const unsigned routed = __ballot_sync(0xffffffffu, gate);
    if (lane == 0) s_count[warp] = __popc(routed);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kMaxTree / 32; ++w) {
        before += w < warp ? s_count[w] : 0;
        all += s_count[w];
    }
    before += __popc(routed & ((1u << lane) - 1));   // routed tokens before this one
    if (on) {
        if (!gate && depth >= a.W) {   // the top of the path has left the window
            // A path's tokens come in the order of their depths: of them the anchors stay,
            // and those from depth - W + 1 on.
            int stay = min(max(a.n_anchor - base, 0), kMaxTree), gone = depth - a.W + 1;
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                if (w * 32 >= n) break;
                const uint32_t x = mask[w];
                mask[w] = x & ((stay > 0 ? lowest(x, stay) : 0u) | ~(gone > 0 ? lowest(x, gone) : 0u));
                stay -= __popc(x);
                gone -= __popc(x);
            }
        }
        a.plan.order[first + (gate ? before : all + t - before)] = t;
        a.plan.lo[first + t] = gate ? 0 : min(max(0, base + depth - a.W + 1), base);
        uint4* to = reinterpret_cast<uint4*>(a.plan.mask + static_cast<size_t>(first + t) * kWords);
        to[0] = make_uint4(mask[0], mask[1], mask[2], mask[3]);
        to[1] = make_uint4(mask[4], mask[5], mask[6], mask[7]);
    }
    if (t == 0) {
        TreeSeq s = {};
        if (n > 0) {
            s.first = first;
            s.n = n;
            s.base = base;
            const int G = a.Hq / a.Hkv;
            s.far_rows = (n * G > rows || all == 0 ? all : n) * G;
            s.lo = max(0, base - a.W + 1);
            s.na = min(a.n_anchor, s.lo);
            s.far_tiles = (len + keys - 1) / keys;
            s.near_tiles = min((s.na + keys - 1) / keys, s.lo / keys) + s.far_tiles - s.lo / keys;
        }
        a.plan.seqs[b] = s;
    }
}

// ---- elements of a page row ---------------------------------------------------
// Four elements of a row as floats; `up` is an e4m3 row's power of two, 2^(byte - 127) for every
// exponent byte as the tensor cores' tiles have it, in two factors as one would not reach its ends.
template <int KIND>
__device__ __forceinline__ float4 four_of(const void* row, int at, float2 up) {
    if constexpr (KIND == SWIATTN_F32) {
        return reinterpret_cast<const float4*>(row)[at];
    } else if constexpr (KIND == SWIATTN_BF16) {
        const uint2 u = reinterpret_cast<const uint2*>(row)[at];
        const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
        const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
        return make_float4(x.x, x.y, y.x, y.y);
    } else {
        const uint32_t u = reinterpret_cast<const uint32_t*>(row)[at];
        const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u & 0xffff), __NV_E4M3);
        const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u >> 16), __NV_E4M3);
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        return make_float4(x.x * up.x * up.y, x.y * up.x * up.y, y.x * up.x * up.y, y.y * up.x * up.y);
    }
}
template <int KIND>
__host__ __device__ constexpr int bytes_of() { return KIND == SWIATTN_F32 ? 4 : KIND == SWIATTN_BF16 ? 2 : 1; }

// Page of a token (a bad table entry: page 0, reported).
__device__ __forceinline__ int page_of(const TreeDecodeArgs& a, int b, int tok) {
    const int p = a.block_table[static_cast<int64_t>(b) * a.max_pages + (tok >> a.page_lg)];
    if (p >= 0 && p < a.num_pages) return p;
    atomicOr(a.err, kDevErrInput);
    return 0;
}

// Key (0) or value (1) row of token tok for key head h, and its power of two.
template <int KIND, int D>
struct Row {
    const void* at;
    float2 up;
};
template <int KIND, int D>
__device__ __forceinline__ Row<KIND, D> row_of(const TreeDecodeArgs& a, int which, int page, int tok, int h) {
    const int slot = tok & ((1 << a.page_lg) - 1);
    const int64_t row = ((static_cast<int64_t>(page) << a.page_lg) + slot) * a.Hkv + h;
    Row<KIND, D> r;
    r.at = static_cast<const char*>(which ? a.v_pages : a.k_pages) + row * (D * bytes_of<KIND>());
    r.up = make_float2(1.f, 1.f);
    if (KIND == SWIATTN_E4M3) {
        const uint32_t e = (which ? a.v_exp : a.k_exp)[((static_cast<int64_t>(page) * a.Hkv + h) << a.page_lg) + slot];
        r.up = make_float2(__uint_as_float((e / 2 + 64) << 23), __uint_as_float((e - e / 2 + 63) << 23));
    }
    return r;
}

// ---- products on CUDA cores ------------------------------------------------------
// For fp32, exact where the tensor cores are not: 32 rows by 64 keys, a thread 4 x 4
// scores, then 4 rows by D/16 dimensions.  A tile's K is copied while the last one's
// values are added, its V while its scores are formed, one buffer each; four CTAs an SM
// where they fit, d = 64 (32 ragged sequences of up to 83 drafts, 64/4 heads, d = 64: 141
// us, by two CTAs that copied first 248).  A lane looks one row up, not each piece of it,
// and takes four keys' weights at once (45 sequences of 196 drafts, 8/1 heads, d = 128: 353
// us, without 440): eight warps an SM, which is what d = 128 leaves room for, are bound by
// the instructions beside the products.
constexpr int kR = kTreeRows, kK = kTreeKeys, kSimtThreads = 128;
template <int D>
struct SimtShared {
    float q[kR][D], k[kK][D + 4], v[kK][D], p[kR][kK + 4];   // rows of 16-byte multiples
    uint32_t mask[kR][kWords];
    int lo[kR];
    TreeStart start;
};

template <int D>
__global__ void __launch_bounds__(kSimtThreads, kTreeCtas<D> / 152) tree_simt_kernel(const __grid_constant__ TreeDecodeArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    SimtShared<D>& s = *reinterpret_cast<SimtShared<D>*>(raw);
    constexpr int F = D / 4;      // float4 of a row
    constexpr int C = D / 64;     // float4 of a thread's output row
    constexpr int KIND = SWIATTN_F32;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, G = a.Hq / a.Hkv;
    if (tid < 32) {
        const TreeStart start = start_walk<kR>(a);
        if (tid == 0) s.start = start;
    }
    __syncthreads();
    TreeWalk<kR> walk{a, s.start};
    const float sl = a.scale_log2;

    TreeWork w;
    while (walk.next(w)) {
        const int rows = w.rows;
        const int anchors = min(a.n_anchor, w.s.base), len = w.s.base + w.s.n;
        __syncthreads();   // the last unit's tiles have been read
        for (int i = tid; i < kR * F; i += kSimtThreads) {
            const int r = i / F, c = i % F, R = w.row0 + r;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const int tok = w.s.first + a.plan.order[w.s.first + R / G];
                x = four_of<KIND>(static_cast<const float*>(a.q) + (static_cast<int64_t>(tok) * a.Hq + w.h * G + R % G) * D, c, make_float2(1.f, 1.f));
            }
            reinterpret_cast<float4*>(s.q[r])[c] = x;
        }
        for (int i = tid; i < kR * kWords; i += kSimtThreads) {
            const int r = i / kWords, R = w.row0 + r;
            uint32_t m = 0;
            if (r < rows) {
                const int tok = w.s.first + a.plan.order[w.s.first + R / G];
                m = a.plan.mask[static_cast<size_t>(tok) * kWords + i % kWords];
                if (i % kWords == 0) s.lo[r] = a.plan.lo[tok];
            }
            s.mask[r][i % kWords] = m;
        }
        float m[4], l[4], acc[4][4 * C];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < 4 * C; ++c) acc[i][c] = 0.f;
        }
        // K (0) or V (1) of key tile kt, a warp a row at a time or two: 16 rows in all, one
        // looked up by each lane.  What no row of the walk reads comes as zeros.
        auto copy = [&](int which, int kt) {
            constexpr int H = 32 / F;
            const int key0 = tile_key<kK>(w.s, w.far, kt), lane = tid & 31, l = lane & 15, first = tid / 32 * H;
            const int tok = key0 + first + l % H + l / H * (kSimtThreads / 32 * H);
            unsigned long long row = 0;
            if (tok < len && (w.far || tok >= w.s.lo || tok < w.s.na))
                row = reinterpret_cast<unsigned long long>(row_of<KIND, D>(a, which, page_of(a, w.b, tok), tok, w.h).at);
            const int stride = which ? sizeof(s.v[0]) : sizeof(s.k[0]);
            uint32_t to = smem_u32(which ? s.v[0] : s.k[0]) + (first + lane / F) * stride + lane % F * 16;
#pragma unroll 4
            for (int n = 0; n < 16 / H; ++n, to += kSimtThreads / 32 * H * stride) {
                const unsigned long long from = __shfl_sync(0xffffffffu, row, n * H + lane / F);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                             "l"(from ? from + lane % F * 16 : reinterpret_cast<unsigned long long>(a.q)), "r"(from ? 16u : 0u)
                             : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        static_assert(kK == 16 * (kSimtThreads / 32), "16 rows a warp");
        copy(0, w.kt0);
        copy(1, w.kt0);
        for (int kt = w.kt0; kt < w.kt1; ++kt) {
            const int key0 = tile_key<kK>(w.s, w.far, kt);
            asm volatile("cp.async.wait_group 1;" ::: "memory");   // K
            __syncthreads();
            float x[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
#pragma unroll 4
            for (int c = 0; c < F; ++c) {
                float4 q[4], k[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = reinterpret_cast<const float4*>(s.q[ty * 4 + i])[c];
#pragma unroll
                for (int j = 0; j < 4; ++j) k[j] = reinterpret_cast<const float4*>(s.k[tx + 16 * j])[c];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[i][j] = fmaf(q[i].x, k[j].x, x[i][j]);
                        x[i][j] = fmaf(q[i].y, k[j].y, x[i][j]);
                        x[i][j] = fmaf(q[i].z, k[j].z, x[i][j]);
                        x[i][j] = fmaf(q[i].w, k[j].w, x[i][j]);
                    }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = ty * 4 + i;
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int tok = key0 + tx + 16 * j, u = tok - w.s.base;
                    const bool seen = r < rows && (u < 0 ? tok >= s.lo[r] || tok < anchors
                                                         : u < w.s.n && (s.mask[r][u >> 5] >> (u & 31) & 1));
                    x[i][j] = seen ? x[i][j] * sl : -INFINITY;
                    top = fmaxf(top, x[i][j]);
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float mn = fmaxf(m[i], top), ref = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(m[i] - ref);
                m[i] = mn;
                l[i] *= f;
#pragma unroll
                for (int c = 0; c < 4 * C; ++c) acc[i][c] *= f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = exp2f(x[i][j] - ref);
                    l[i] += p;
                    s.p[r][tx + 16 * j] = p;
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");   // V
            __syncthreads();   // and K has been read
            if (kt + 1 < w.kt1) copy(0, kt + 1);
#pragma unroll 1
            for (int k0 = 0; k0 < kK; k0 += 4) {
                float4 p[4];   // four keys' weights of a row at once
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(&s.p[ty * 4 + i][k0]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float4 v[C];
#pragma unroll
                    for (int c = 0; c < C; ++c) v[c] = reinterpret_cast<const float4*>(s.v[k0 + k])[tx + 16 * c];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float w = k == 0 ? p[i].x : k == 1 ? p[i].y : k == 2 ? p[i].z : p[i].w;
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            acc[i][4 * c] = fmaf(w, v[c].x, acc[i][4 * c]);
                            acc[i][4 * c + 1] = fmaf(w, v[c].y, acc[i][4 * c + 1]);
                            acc[i][4 * c + 2] = fmaf(w, v[c].z, acc[i][4 * c + 2]);
                            acc[i][4 * c + 3] = fmaf(w, v[c].w, acc[i][4 * c + 3]);
                        }
                    }
                }
            }
            if (kt + 1 < w.kt1) {
                __syncthreads();   // V has been read
                copy(1, kt + 1);
            }
        }
        static_assert(kPartRows<kR> == kR, "a part has the tile's rows");
        float* part = a.plan.part + static_cast<size_t>(w.slot) * kR * (D + 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
            if (r < rows) {
#pragma unroll
                for (int c = 0; c < C; ++c)
                    reinterpret_cast<float4*>(part)[(tx + 16 * c) * kR + r] =
                        make_float4(acc[i][4 * c], acc[i][4 * c + 1], acc[i][4 * c + 2], acc[i][4 * c + 3]);
                if (tx == 0) reinterpret_cast<float2*>(part + kR * D)[r] = make_float2(m[i], l[i]);
            }
        }
    }
}

// ---- the join ---------------------------------------------------------------------
// A block 32 rows of a row tile at a time, lane r row r, warp w the (w % 8)-th eighth of
// the dimensions and, of 16 warps, every other part of the rows' unit; where there are
// 16 rows or 8, two or four lanes share a row's parts.  Parts join by their maxima,
// in an order that the numbers of rows and parts decide.  They lie four dimensions of
// all rows together, then the next four, so that lanes read (and the threads that own
// a row write) neighbouring 16 bytes.
//
// Every row of a tile multiplies every value row that the tile's walk reads, with
// weight 0 where the row itself does not read it; where that value is not finite, 0
// times it is a NaN that is none of the row's.  So a row that comes out not finite is
// computed again, key by key over what it does read (slow, and right whatever the
// reason).
constexpr int kJoinThreads = 512;   // at most, or half of them

template <int N>
struct Dims {
    float x[N];
};

template <int KIND, int D>
__device__ __noinline__ void row_again(const TreeDecodeArgs& a, int b, int h, int tok, const TreeSeq& s, const float* q, Dims<D / 32>& o, float& m, float& l) {
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) o.x[i] = 0.f;
    const int lo = a.plan.lo[tok], anchors = min(a.n_anchor, lo);
    const uint32_t* mask = a.plan.mask + static_cast<size_t>(tok) * kWords;
    for (int j = anchors > 0 ? 0 : lo; j < s.base + s.n; ++j) {
        if (j == anchors && j < lo) {
            j = lo - 1;
            continue;
        }
        const int u = j - s.base;
        if (u >= 0 && !(mask[u >> 5] >> (u & 31) & 1)) continue;
        const int page = page_of(a, b, j);
        const Row<KIND, D> k = row_of<KIND, D>(a, 0, page, j, h), v = row_of<KIND, D>(a, 1, page, j, h);
        // lane's dimensions: N side by side
        float x = 0.f, vv[N];
        const float4 kx = four_of<KIND>(k.at, lane * N / 4, k.up), vx = four_of<KIND>(v.at, lane * N / 4, v.up);
        if (N == 4) {
            x = q[0] * kx.x + q[1] * kx.y + q[2] * kx.z + q[3] * kx.w;
            vv[0] = vx.x, vv[1] = vx.y, vv[N - 2] = vx.z, vv[N - 1] = vx.w;
        } else {
            x = lane & 1 ? q[0] * kx.z + q[1] * kx.w : q[0] * kx.x + q[1] * kx.y;
            vv[0] = lane & 1 ? vx.z : vx.x;
            vv[1] = lane & 1 ? vx.w : vx.y;
        }
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
        x *= a.scale_log2;
        // The maximum passes over a NaN, whose weight is one; nothing is forgotten, whatever the
        // maximum was, so that it stays.  Scores of -infinity weigh 0 before a finite one, too.
        const float mn = fmaxf(m, x), ref = mn == -INFINITY ? 0.f : mn, f = exp2f(m - ref), p = exp2f(x - ref);
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < N; ++i) o.x[i] = o.x[i] * f + p * vv[i];
        m = mn;
    }
}

__device__ __forceinline__ void add(float4& o, const float4& x, float w) {
    o = make_float4(fmaf(x.x, w, o.x), fmaf(x.y, w, o.y), fmaf(x.z, w, o.z), fmaf(x.w, w, o.w));
}

template <int KIND, int D, int R>
__global__ void __launch_bounds__(kJoinThreads, 2) tree_join_kernel(const __grid_constant__ TreeDecodeArgs a, int ctas) {
    constexpr int N = D / 32, kAcross = 8, kGroups = D / 4 / kAcross;   // warps across the dimensions; fours of a warp
    const int warps = blockDim.x / 32, downs = warps / kAcross;   // 8 or 16; 1 or 2
    constexpr int kAtOnce = 8 / kGroups;   // parts on their way: 32 registers
    constexpr int kPart = kPartRows<R>;
    using T = typename std::conditional<KIND == SWIATTN_F32, float, __nv_bfloat16>::type;
    __shared__ float s_o[32][D + 4];
    __shared__ float2 s_stats[32];   // of the second warps
    __shared__ float s_lse[32];
    __shared__ unsigned s_bad[2];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x / 32, G = a.Hq / a.Hkv;
    const int across = warp % kAcross, down = warp / kAcross;
    const TreeSeq s = a.plan.seqs[b];
    if (s.n == 0) return;
    const int far = far_tiles<R>(s), near_rows = s.n * G - s.far_rows;
    const int64_t head = a.plan.start[a.B], total = head * a.Hkv, start = a.plan.start[b];   // work of a head, of all
    const int unit = a.plan.unit[b], head_units = a.plan.unit[a.B], cost = a.plan.cost[0];
    const int64_t shares = share_count(total, ctas);
    auto cta_of = [&](int64_t at) {   // a division of 64 bits takes several times one of 32, and few calls need it
        const int64_t x = (at + 1) * shares - 1;
        return static_cast<int>((x | total) >> 32 ? x / total : static_cast<uint32_t>(x) / static_cast<uint32_t>(total));
    };
    const int far_chunks = (s.far_rows + 31) / 32, chunks = far_chunks + (near_rows + 31) / 32;
    if (threadIdx.x < 2) s_bad[threadIdx.x] = 0;
    __syncthreads();
    int turn = 0;
    for (int i = blockIdx.y; i < chunks * a.Hkv; i += gridDim.y, turn ^= 1) {
        const int h = i / chunks, chunk = i - h * chunks;
        const bool is_far = chunk < far_chunks;
        const int in = (is_far ? chunk : chunk - far_chunks) * 32, rows = is_far ? s.far_rows : near_rows;   // of its kind
        const int here = min(32, rows - in), lanes = here <= 8 ? 8 : here <= 16 ? 16 : 32, at_row = lane & (lanes - 1);
        const int rt = in / R, r = in % R + at_row;
        const bool on = at_row < here;
        const int row = on ? in + at_row + (is_far ? 0 : s.far_rows) : 0;
        const int tok = s.first + a.plan.order[s.first + row / G];
        const int64_t out = static_cast<int64_t>(tok) * a.Hq + h * G + row % G;
        const int len = is_far ? s.far_tiles : s.near_tiles;
        const int64_t from = h * head + start + cost + static_cast<int64_t>(rt) * (len + cost) + (is_far ? 0 : static_cast<int64_t>(far) * (s.far_tiles + cost));   // its first key tile
        const int c0 = cta_of(from);
        constexpr int kOf = kPart / R;   // parts of a CTA
        const int n = (cta_of(from + len - 1) - c0 + 1) * kOf;
        const float* part = a.plan.part + static_cast<size_t>(c0 + h * head_units + unit + rt + (is_far ? 0 : far)) * kPart * (D + 2);
        float m = -INFINITY, l = 0.f;
        float4 o[kGroups];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) o[g] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int step = downs * (32 / lanes);   // this lane's parts: the first, and how far apart
        for (int p0 = down * (32 / lanes) + lane / lanes; p0 < n; p0 += kAtOnce * step) {
            float2 st[kAtOnce];
            float4 x[kAtOnce][kGroups];
#pragma unroll
            for (int p = 0; p < kAtOnce; ++p) {
                st[p] = make_float2(-INFINITY, 0.f);
                const int q = p0 + p * step;
                if (on && q < n) {
                    const float* at = part + static_cast<size_t>(q / kOf) * kPart * (D + 2);
                    const int in_part = r + q % kOf * R;
                    st[p] = __ldcg(reinterpret_cast<const float2*>(at + kPart * D) + in_part);
#pragma unroll
                    for (int g = 0; g < kGroups; ++g)
                        x[p][g] = __ldcg(reinterpret_cast<const float4*>(at) + (across * kGroups + g) * kPart + in_part);
                }
            }
            float mn = m;
#pragma unroll
            for (int p = 0; p < kAtOnce; ++p) mn = fmaxf(mn, st[p].x);
            const float ref = mn == -INFINITY ? 0.f : mn, f = exp2f(m - ref);
            l *= f;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) o[g] = make_float4(o[g].x * f, o[g].y * f, o[g].z * f, o[g].w * f);
#pragma unroll
            for (int p = 0; p < kAtOnce; ++p)
                if (on && p0 + p * step < n) {
                    const float w = exp2f(st[p].x - ref);
                    l = fmaf(st[p].y, w, l);
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) add(o[g], x[p][g], w);
                }
            m = mn;
        }
        // The row's other lanes, then its other warps.
        auto join = [&](float m2, float l2, auto other) {
            const float mn = fmaxf(m, m2), ref = mn == -INFINITY ? 0.f : mn, f = exp2f(m - ref), w = exp2f(m2 - ref);
            l = l * f + l2 * w;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const float4 x = other(g);
                o[g] = make_float4(o[g].x * f, o[g].y * f, o[g].z * f, o[g].w * f);
                add(o[g], x, w);
            }
            m = mn;
        };
        for (int w = lanes; w < 32; w *= 2)
            join(__shfl_xor_sync(0xffffffffu, m, w), __shfl_xor_sync(0xffffffffu, l, w), [&](int g) {
                return make_float4(__shfl_xor_sync(0xffffffffu, o[g].x, w), __shfl_xor_sync(0xffffffffu, o[g].y, w),
                                   __shfl_xor_sync(0xffffffffu, o[g].z, w), __shfl_xor_sync(0xffffffffu, o[g].w, w));
            });
        if (downs == 2) {
            if (down == 1) {
#pragma unroll
                for (int g = 0; g < kGroups; ++g) *reinterpret_cast<float4*>(&s_o[lane][(across * kGroups + g) * 4]) = o[g];
                if (across == 0) s_stats[lane] = make_float2(m, l);
            }
            __syncthreads();
            if (down == 0) {
                const float2 st = s_stats[lane];
                join(st.x, st.y, [&](int g) { return *reinterpret_cast<const float4*>(&s_o[lane][(across * kGroups + g) * 4]); });
            }
        }
        bool fine = true;
        if (down == 0) {
            const float inv = 1.f / l;
            fine = l - l == 0.f && l > 0.f;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                o[g] = make_float4(o[g].x * inv, o[g].y * inv, o[g].z * inv, o[g].w * inv);
                fine &= (o[g].x - o[g].x == 0.f) & (o[g].y - o[g].y == 0.f) & (o[g].z - o[g].z == 0.f) & (o[g].w - o[g].w == 0.f);
                *reinterpret_cast<float4*>(&s_o[lane][(across * kGroups + g) * 4]) = o[g];
            }
            if (across == 0) s_lse[lane] = (m + log2f(l)) * 0.69314718055994531f;
        }
        const unsigned odd = __ballot_sync(0xffffffffu, lane < here && !fine);
        if (odd && lane == 0) atomicOr(&s_bad[turn], odd);
        if (threadIdx.x == 0) s_bad[turn ^ 1] = 0;
        __syncthreads();
        const unsigned bad = s_bad[turn];
        // A warp's rows, lanes side by side along the dimensions.
        for (int at = warp; at < here; at += warps) {
            const int64_t to = __shfl_sync(0xffffffffu, out, at & (lanes - 1));
            float y[N];
#pragma unroll
            for (int e = 0; e < N; ++e) y[e] = s_o[at][lane * N + e];
            float lse = s_lse[at];
            if (bad >> at & 1) {
                Dims<N> again;
                float q[N], am, al;
                const T* src = static_cast<const T*>(a.q) + to * D + lane * N;
#pragma unroll
                for (int e = 0; e < N; ++e) q[e] = static_cast<float>(src[e]);
                row_again<KIND, D>(a, b, h, static_cast<int>(to / a.Hq), s, q, again, am, al);
                lse = (am + log2f(al)) * 0.69314718055994531f;
#pragma unroll
                for (int e = 0; e < N; ++e) y[e] = again.x[e] / al;
            }
            T* dst = static_cast<T*>(a.o) + to * D + lane * N;
            if constexpr (KIND == SWIATTN_F32) {
                if constexpr (N == 4) *reinterpret_cast<float4*>(dst) = make_float4(y[0], y[1], y[2], y[3]);
                else *reinterpret_cast<float2*>(dst) = make_float2(y[0], y[1]);
            } else {
                if constexpr (N == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
                else *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(y[0], y[1]);
            }
            if (a.lse && lane == 0) a.lse[to] = lse;
        }
        __syncthreads();   // s_o is written again
    }
}

template <int D>
cudaError_t launch_simt(const TreeDecodeArgs& a, int ctas, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_dynamic_smem(tree_simt_kernel<D>, sizeof(SimtShared<D>), done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = dependent_launch(ctas, kSimtThreads, s, attr);
    cfg.dynamicSmemBytes = sizeof(SimtShared<D>);
    return cudaLaunchKernelEx(&cfg, tree_simt_kernel<D>, a);
}

template <int KIND, int D>
cudaError_t launch_all(const TreeDecodeArgs& a, int sms, cudaStream_t s) {
    constexpr bool kTc = KIND != SWIATTN_F32;
    constexpr int kRows = kTc ? kTreeTcRows : kTreeRows;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = dependent_launch(a.B, kMaxTree, s, attr);
    cudaError_t e = cudaLaunchKernelEx(&cfg, tree_plan_kernel, a, kRows, kTc ? kTreeTcKeys : kTreeKeys);
    if (e != cudaSuccess) return e;
    const int ctas = kTc ? std::min(sms, kTreeTcCtas) : std::min(kTreeCtas<D> / 152 * sms, kTreeCtas<D>);
    prof_start(s);
    if constexpr (kTc) e = launch_tree_tc(a, D, KIND == SWIATTN_E4M3, ctas, s);
    else e = launch_simt<D>(a, ctas, s);
    prof_stop(s);
    if (e != cudaSuccess) return e;
    // About the chunks of a sequence of mean size (blocks without one cost time too), or, as
    // one may be larger, what runs at once (2 ragged sequences of 16K: 31 us, without 44).
    const int64_t G = a.Hq / a.Hkv, mean = (static_cast<int64_t>(a.T) * G / a.B / 32 + 1) * a.Hkv;
    const int64_t most = ((std::min(a.T, kMaxTree) * G + 31) / 32 + 1) * a.Hkv;
    const int64_t y = std::max(mean, std::min<int64_t>(most, 2 * sms / a.B));
    // Many chunks want many blocks at once, few their parts read by more warps (33
    // ragged trees, 1400 chunks: 100 us, by 512 threads each 114; 8 x 32K with 64 rows,
    // 64 chunks: 110 us by 256 threads, 103 by 512).
    const bool many = mean * a.B > 4 * sms;
    cfg = dependent_launch(dim3(a.B, static_cast<unsigned>(std::min<int64_t>(y, std::max(1, 8192 / a.B)))), many ? kJoinThreads / 2 : kJoinThreads, s, attr);
    e = cudaLaunchKernelEx(&cfg, tree_join_kernel<KIND, D, kRows>, a, ctas);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int KIND>
cudaError_t launch_kind(const TreeDecodeArgs& a, int d, int sms, cudaStream_t s) {
    return d == 128 ? launch_all<KIND, 128>(a, sms, s) : launch_all<KIND, 64>(a, sms, s);
}

}  // namespace

TreeWs tree_ws_layout(int T, int B, int Hq, int Hkv, int d, int dtype) {
    auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    const size_t t = T, b = B, G = Hq / Hkv;
    TreeWs L;
    L.seqs = 0;
    L.start = up(sizeof(int) * 8 * b);
    L.unit = up(L.start + sizeof(int64_t) * (b + 1));
    L.cost = L.unit + sizeof(int) * (b + 1);
    L.order = up(L.cost + sizeof(int));
    L.lo = up(L.order + sizeof(int) * t);
    L.mask = up(L.lo + sizeof(int) * t);
    L.part = up(L.mask + sizeof(uint32_t) * kWords * t);
    // Units: a key head's row tiles, of which each sequence with tokens has at most
    // two that are not full.
    const size_t rows = dtype == SWIATTN_BF16 ? kTreeTcRows : kTreeRows, ctas = dtype == SWIATTN_BF16 ? kTreeTcCtas : d == 64 ? kTreeCtas<64> : kTreeCtas<128>;
    const size_t units = Hkv * (t * G / rows + 2 * std::min(b, t));
    const size_t part_rows = dtype == SWIATTN_BF16 ? kPartRows<kTreeTcRows> : kPartRows<kTreeRows>;
    L.total = up(L.part + (ctas + units) * part_rows * (d + 2) * sizeof(float));
    return L;
}

cudaError_t launch_decode_tree(const TreeDecodeArgs& a, int d, int page_dtype, int sms, cudaStream_t s) {
    if (page_dtype == SWIATTN_F32) return launch_kind<SWIATTN_F32>(a, d, sms, s);
    if (page_dtype == SWIATTN_BF16) return launch_kind<SWIATTN_BF16>(a, d, sms, s);
    return launch_kind<SWIATTN_E4M3>(a, d, sms, s);
}

}  // namespace swi

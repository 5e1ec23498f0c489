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

namespace swi {
namespace {

constexpr int kTile = 16;        // keys of one product tile
constexpr int kWarps = 4;        // warps of a block; they take a chunk's tiles in turn
constexpr int kMinChunk = 64;    // keys of a chunk (one block's work)
constexpr int kMaxChunk = 512;
constexpr int kBlocksWanted = 304;   // chunks x KV heads that fill the GPU (two blocks an SM)

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

// Keys sequence b visits: anchors [0, na) and [lo, len).  Chunks are runs of
// `tiles` 16-key tiles at multiples of 16 from the cache's start, so that a
// tile never straddles a page of 16 or more; the first nca chunks are
// anchors'.  The chunk length depends on the sequence and the shapes alone,
// so a sequence's result does not depend on the rest of the batch.
struct Visit {
    int len, lo, na;
    int tiles;      // tiles of a chunk
    int nca, nc;    // chunks: anchors', all
};
__host__ __device__ inline int chunks_wanted(int Hkv) { return (kBlocksWanted + Hkv - 1) / Hkv; }
__device__ __forceinline__ Visit visit_of(const DecodeE4m3Args& a, int b) {
    Visit v;
    const int max_len = a.max_pages << a.page_lg;
    v.len = min(max(a.seq_lens[b], 0), max_len);
    v.lo = a.gate[b] ? 0 : max(0, v.len - a.W);
    v.na = min(a.n_anchor, v.lo);
    const int m = v.na + v.len - v.lo;
    int chunk = kMinChunk;
    while (chunk < kMaxChunk && static_cast<int64_t>(chunk) * chunks_wanted(a.Hkv) < m) chunk <<= 1;
    v.tiles = chunk / kTile;
    const int ta = (v.na + kTile - 1) / kTile;
    const int tw = v.len > 0 ? (v.len + kTile - 1) / kTile - v.lo / kTile : 0;
    v.nca = (ta + v.tiles - 1) / v.tiles;
    v.nc = v.nca + (tw + v.tiles - 1) / v.tiles;
    return v;
}

// One block: chunk blockIdx.x of KV head blockIdx.y of sequence blockIdx.z.
// NH: groups of eight query heads (1: Hq/Hkv <= 8, 2: <= 16).
template <int D, int NH>
__global__ void __launch_bounds__(kWarps * 32) decode_e4m3_split_kernel(DecodeE4m3Args a) {
    constexpr int KS = D / 16;    // 16-deep steps of the score product, and 16-row tiles of O^T
    constexpr int KW = D / 64;    // 16-byte pieces of a key row a thread holds
    const int b = blockIdx.z, h = blockIdx.y, c = blockIdx.x;
    const Visit vis = visit_of(a, b);
    if (c == 0 && h == 0 && threadIdx.x == 0) {
        const int raw = a.seq_lens[b];
        if (raw < 0 || raw > (a.max_pages << a.page_lg)) atomicOr(a.err, kDevErrInput);
    }
    if (c >= vis.nc) return;
    const int G = a.Hq / a.Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;

    // This chunk's tiles and the keys of them that are visited, [from, to).
    int tile0, tile1, from, to;
    if (c < vis.nca) {
        from = 0;
        to = vis.na;
        tile0 = c * vis.tiles;
    } else {
        from = vis.lo;
        to = vis.len;
        tile0 = vis.lo / kTile + (c - vis.nca) * vis.tiles;
    }
    tile1 = min(tile0 + vis.tiles, (to + kTile - 1) / kTile);

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

    const int32_t* table = a.block_table + static_cast<size_t>(b) * a.max_pages;
    const int mask = (1 << a.page_lg) - 1;
    auto page_of = [&](int tok) {
        int p = table[tok >> a.page_lg];
        if (p < 0 || p >= a.num_pages) {
            atomicOr(a.err, kDevErrInput);
            p = 0;
        }
        return p;
    };

    for (int tile = tile0 + warp; tile < tile1; tile += kWarps) {
        const int base = tile * kTile;
        // Keys base + g and base + 8 + g: rows and exponents.
        uint4 kw[2][KW];
        int ku[2], vu[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int tok = base + g + 8 * r;
            const bool on = tok >= from && tok < to;
            ku[r] = vu[r] = 127;
#pragma unroll
            for (int w = 0; w < KW; ++w) kw[r][w] = make_uint4(0, 0, 0, 0);
            if (on) {
                const size_t page = page_of(tok);
                const size_t row = ((page << a.page_lg) + (tok & mask)) * a.Hkv + h;
                const uint4* src = reinterpret_cast<const uint4*>(a.k_pages + row * D) + t;
#pragma unroll
                for (int w = 0; w < KW; ++w) kw[r][w] = src[4 * w];
                const size_t ex = ((page * a.Hkv + h) << a.page_lg) + (tok & mask);
                ku[r] = a.k_exp[ex];
                vu[r] = a.v_exp[ex];
            }
        }
        // Values of keys 2t, 2t + 1, 2t + 8, 2t + 9, dims D/8 g on.  Keys that are
        // not visited hold zeros (a weight of zero would not cancel a NaN).
        uint32_t vw[4][D / 32];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int tok = base + 2 * t + (r & 1) + 8 * (r >> 1);
#pragma unroll
            for (int w = 0; w < D / 32; ++w) vw[r][w] = 0;
            if (tok >= from && tok < to) {
                const size_t row = ((static_cast<size_t>(page_of(tok)) << a.page_lg) + (tok & mask)) * a.Hkv + h;
                const uint8_t* src = a.v_pages + row * D + g * (D / 8);
                if constexpr (D == 128) {
                    const uint4 u = *reinterpret_cast<const uint4*>(src);
                    vw[r][0] = u.x, vw[r][1] = u.y, vw[r][2] = u.z, vw[r][3] = u.w;
                } else {
                    const uint2 u = *reinterpret_cast<const uint2*>(src);
                    vw[r][0] = u.x, vw[r][1] = u.y;
                }
            }
        }

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
        uint32_t wt[NH][2];
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            float x[4], y[4];   // s_j and t_j
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = e >> 1;
                const int tok = base + g + 8 * r;
                const bool on = tok >= from && tok < to;
                x[e] = on ? s[n][e] * fs[n][e & 1] * __uint_as_float(static_cast<uint32_t>(ku[r]) << 23) : -INFINITY;
                y[e] = x[e] + static_cast<float>(vu[r] - 127);
            }
#pragma unroll
            for (int col = 0; col < 2; ++col) {
                float xm = fmaxf(x[col], x[col + 2]), ym = fmaxf(y[col], y[col + 2]);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    xm = fmaxf(xm, __shfl_xor_sync(0xffffffffu, xm, o));
                    ym = fmaxf(ym, __shfl_xor_sync(0xffffffffu, ym, o));
                }
                const float mn = fmaxf(m[n][col], xm), nn = fmaxf(nmax[n][col], ym);
                const float mr = finite_or_0(mn), nr = finite_or_0(nn);
                const float cl = ex2f(m[n][col] - mr), ca = ex2f(nmax[n][col] - nr);
                m[n][col] = mn;
                nmax[n][col] = nn;
                l[n][col] = l[n][col] * cl + ex2f(x[col] - mr) + ex2f(x[col + 2] - mr);
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    acc[n][j][col] *= ca;
                    acc[n][j][col + 2] *= ca;
                }
                y[col] = ex2f(y[col] - nr);
                y[col + 2] = ex2f(y[col + 2] - nr);
            }
            wt[n][0] = transpose8x8(pack_half2(y[0], y[1]));
            wt[n][1] = transpose8x8(pack_half2(y[2], y[3]));
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

    // Join the warps: their maxima, then their sums relative to the block's.
    __shared__ float s_m[kWarps][NH * 8], s_n[kWarps][NH * 8], s_l[kWarps][NH * 8];
    __shared__ float s_acc[kWarps][8][D];
    float* part = a.part + ((static_cast<size_t>(b) * a.Hq + h * G) * a.max_chunks + c) * (D + 4);
    const size_t head_step = static_cast<size_t>(a.max_chunks) * (D + 4);
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
                    s_acc[warp][head][g * (D / 8) + 2 * j] = acc[n][j][col] * f;
                    s_acc[warp][head][g * (D / 8) + 2 * j + 1] = acc[n][j][col + 2] * f;
                }
            }
        }
        __syncthreads();
        const int heads = min(8, G - n * 8);
        for (int i = threadIdx.x; i < heads * D; i += kWarps * 32) {
            const int head = i / D, col = i % D;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += s_acc[w][head][col];
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
}

// Joins the chunks of one (query head, sequence): block (hq, b), thread = dim.
template <int D>
__global__ void __launch_bounds__(D) decode_e4m3_join_kernel(DecodeE4m3Args a) {
    const int hq = blockIdx.x, b = blockIdx.y, col = threadIdx.x;
    const Visit vis = visit_of(a, b);
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + (static_cast<size_t>(b) * a.Hq + hq) * D;
    const float* part = a.part + (static_cast<size_t>(b) * a.Hq + hq) * a.max_chunks * (D + 4);
    float m = -INFINITY, n = -INFINITY;
    for (int c = 0; c < vis.nc; ++c) {
        m = fmaxf(m, part[c * (D + 4) + D]);
        n = fmaxf(n, part[c * (D + 4) + D + 1]);
    }
    const float mr = finite_or_0(m), nr = finite_or_0(n);
    float l = 0.f, sum = 0.f;
    for (int c = 0; c < vis.nc; ++c) {
        const float* p = part + c * (D + 4);
        l += p[D + 2] * ex2f(p[D] - mr);
        sum += p[col] * ex2f(p[D + 1] - nr);
    }
    if (vis.nc == 0) {   // an empty slot
        o[col] = __float2bfloat16_rn(0.f);
        if (a.lse && col == 0) a.lse[static_cast<size_t>(b) * a.Hq + hq] = -INFINITY;
        return;
    }
    o[col] = __float2bfloat16_rn(sum / l * ex2f(n - m));
    if (a.lse && col == 0) a.lse[static_cast<size_t>(b) * a.Hq + hq] = (m + __log2f(l)) * 0.69314718055994531f;
}

template <int D>
cudaError_t launch_d(const DecodeE4m3Args& a, cudaStream_t s) {
    const dim3 grid(a.max_chunks, a.Hkv, a.B);
    prof_start(s);
    if (a.Hq / a.Hkv <= 8) decode_e4m3_split_kernel<D, 1><<<grid, kWarps * 32, 0, s>>>(a);
    else decode_e4m3_split_kernel<D, 2><<<grid, kWarps * 32, 0, s>>>(a);
    prof_stop(s);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    decode_e4m3_join_kernel<D><<<dim3(a.Hq, a.B), D, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

// A visit of v keys (v <= max_len + min(n_anchor, max_len)) has at most
// ceil(v / chunk) + 2 chunks (16-key alignment and the two segments), and the
// chunk is kMaxChunk or at least v / chunks_wanted.
int decode_e4m3_max_chunks(int64_t max_len, int n_anchor, int Hkv) {
    const int64_t v = max_len + (n_anchor < max_len ? n_anchor : max_len);
    const int64_t longest = (v + kMaxChunk - 1) / kMaxChunk;
    const int64_t wanted = chunks_wanted(Hkv);
    return static_cast<int>((longest > wanted ? longest : wanted) + 3);
}

size_t decode_e4m3_workspace_bytes(int B, int Hq, int d, int max_chunks) {
    const size_t n = sizeof(float) * static_cast<size_t>(B) * Hq * max_chunks * (d + 4);
    return (n + 255) & ~static_cast<size_t>(255);
}

cudaError_t launch_decode_e4m3(const DecodeE4m3Args& a, int d, cudaStream_t s) {
    return d == 128 ? launch_d<128>(a, s) : launch_d<64>(a, s);
}

}  // namespace swi

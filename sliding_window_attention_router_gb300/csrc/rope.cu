// Position rotation of queries and keys, its gradient, and the append of new
// tokens' keys and values to a paged cache with the rotation on the way.
//
// The mathematics: frequency f < r/2 turns the pair (a, b) of a head's
// dimensions at position p by the angle p w_f,
//   a' = m (a cos - b sin),   b' = m (b cos + a sin),
// with (a, b) = (x[f], x[f + r/2]) or, interleaved, (x[2f], x[2f+1]); the
// dimensions from r on pass through.  The gradient is the transposed map: the
// same with the sine negated.
//
// The angle: w_f / 2pi is held as a 64-bit binary fraction of a turn F, so
// p F mod 2^64 is the angle modulo a whole turn without any rounding (a float
// product would be off by p w_f 2^-24: 0.06 rad at position 10^6).  The nearest
// quarter turn comes off its top 32 bits as a whole number; what is left is
// within an eighth of a turn, where rounding it to a float costs at most 2^-28
// of a turn, and goes to the Taylor polynomials of sine and cosine.

#include "swiattn.h"
#include "swiattn_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <algorithm>

namespace swi {
namespace {

constexpr int kMaxThreads = 256;  // of a block
constexpr int kMaxHalf = 64;      // rotated pairs of a head: d <= 128
constexpr int kMaxTokens = 8;     // of a block

// ---- eight elements of T: as loaded, as floats ------------------------------
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float* x) const {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __bfloat1622float2(h[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p + 4));
    }
    __device__ __forceinline__ void get(float* x) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
    uint4 u;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
// Round to nearest even, the largest finite value beyond it, NaN kept.
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float* x) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// ---- angles ----------------------------------------------------------------
// Frequency w (radians a position) as a 64-bit fraction of a turn, modulo a
// whole turn (positions are whole numbers, so whole turns do not matter).  With
// w = M 2^E, M of 53 bits, it is M * (2^66 / 2pi) * 2^(E - 2), a 128-bit whole
// number shifted, right to 2^-63 of the turns it stands for and, up to a radian a
// position, to the last bit but one.  Whole-number arithmetic, as the
// double-precision pipe is a sixty-fourth as wide.  `factor`, of the cosine and
// sine, becomes a NaN where w is not finite.
__device__ __forceinline__ uint64_t turn_fraction(double w, float& factor) {
    const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(w));
    const int e = static_cast<int>(bits >> 52 & 2047);
    const uint64_t m = (bits & 0xfffffffffffffull) | (e ? 1ull << 52 : 0ull);
    constexpr uint64_t kInv = 0xa2f9836e4e44152aull;   // 2^66 / 2pi
    const uint64_t hi = __umul64hi(m, kInv), lo = m * kInv;
    if (e == 2047) factor = __int_as_float(0x7fffffff);
    const int shift = 1077 - (e ? e : 1);   // right, 2 - E
    uint64_t f;
    if (shift >= 128) f = 0;
    else if (shift >= 64) f = hi >> (shift - 64);
    else if (shift > 0) f = (hi << (64 - shift)) | (lo >> shift);
    else f = shift > -64 ? lo << -shift : 0;
    return bits >> 63 ? 0 - f : f;
}
// m cos and m sin of position p times frequency F.  With |z| <= pi/4 the first
// terms left out are z^11/11! < 2^-29 of the sine and z^12/12! < 2^-32.  (With
// sincospif in their place the tables were a sixth of the append's instructions.)
__device__ __forceinline__ float2 cos_sin(uint64_t F, int p, float m) {
    const uint64_t turn = F * static_cast<uint64_t>(static_cast<int64_t>(p));
    const uint32_t top = static_cast<uint32_t>(turn >> 32);
    const uint32_t quarter = (top + 0x20000000u) >> 30;
    const float z = static_cast<float>(static_cast<int32_t>(top - (quarter << 30))) * 1.46291807927e-9f;   // 2 pi 2^-32
    const float q = z * z;
    const float sp = fmaf(q, fmaf(q, fmaf(q, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6);
    const float cp = fmaf(q, fmaf(q, fmaf(q, fmaf(q, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f);
    float s = fmaf(z * q, sp, z), c = fmaf(q, cp, 1.f);
    if (quarter & 1) {   // a quarter turn on: (c, s) -> (-s, c)
        const float o = c;
        c = -s;
        s = o;
    }
    if (quarter & 2) m = -m;
    return make_float2(m * c, m * s);
}

// ---- where a new token goes --------------------------------------------------
// Largest b in [0, B) with starts[b] <= t, by one warp (32 probes a step), or
// -1.  Every probe is inside [0, B) whatever the array holds.
__device__ __forceinline__ int find_sequence(const int32_t* starts, int B, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B;
    for (;;) {
        const int step = (n + 31) / 32;
        const int at = lane * step;
        const unsigned hit = __ballot_sync(0xffffffffu, at < n && starts[lo + at] <= t);
        if (hit == 0) return -1;
        const int j = 31 - __clz(hit);
        lo += j * step;
        n = min(step, n - j * step);
        if (step == 1) return lo;
    }
}

// New token t: its sequence b and position; b < 0 where it is not stored (a
// padding row, an empty slot, or a position off the table, which is reported).
// Called by a whole warp.  Up to 32 sequences take one round trip to memory.
struct Place {
    int b, pos;
};
__device__ __forceinline__ Place place_of(const RotateArgs& a, int t) {
    int b = t, after = 1, len;   // tokens of the sequence from t on, its length
    if (!a.starts) {
        len = a.seq_lens[t];
    } else if (a.B <= 32) {
        const int lane = threadIdx.x & 31, i = min(lane, a.B - 1);
        const int from = a.starts[i], to = a.starts[i + 1], mine = a.seq_lens[i];
        const unsigned hit = __ballot_sync(0xffffffffu, lane < a.B && from <= t && t < to);
        if (hit == 0) return {-1, 0};
        b = 31 - __clz(hit);
        after = __shfl_sync(0xffffffffu, to, b) - t;
        len = __shfl_sync(0xffffffffu, mine, b);
    } else {
        b = find_sequence(a.starts, a.B, t);
        if (b < 0) return {-1, 0};
        after = a.starts[b + 1] - t;
        len = a.seq_lens[b];
        if (after <= 0) return {-1, 0};
    }
    if (len == 0) return {-1, 0};
    const int64_t pos = static_cast<int64_t>(len) - after;
    if (pos >= 0 && (pos >> a.page_lg) < a.max_pages) return {b, static_cast<int>(pos)};
    if ((threadIdx.x & 31) == 0) atomicOr(a.err, kDevErrInput);
    return {-1, 0};
}

// Exponent e of the smallest power of two with amax <= 448 * 2^e, within
// [-126, 127]: amax = m 2^x with m in [1, 2) and 448 = 1.75 * 2^8.
__device__ __forceinline__ int row_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(-126, min(127, e));
}

// ---- the kernel ------------------------------------------------------------
// A token's heads (q's, k's, v's) are cut into slots of 16 elements, d/16 to a
// head: a rotated slot holds eight whole pairs, as two groups of eight
// elements (rot/2 apart, or side by side when interleaved), the others two
// groups that pass through.
//
// HBM-bound: 6 operations on 4 bytes (bf16).  A block takes U tokens a thread of
// one slot, `span` tokens side by side, and
//   1. starts all its loads, which need no position,
//   2. finds the tokens' places and their cosines and sines, once for all
//      heads, in shared memory (a warp a token and 32 frequencies),
//   3. after one barrier rotates, converts and stores.
// Blocks are small and many: while some wait in 2, others load and store.
// Persistent blocks that prefetch, tiles of more tokens and warps on their own
// all came out slower (84 to 115 us for the first figure below).
//
// Measured (one GB300, copy rate 6787 GB/s): rotation of 32K tokens of 16 + 16
// heads, 537 MB, 79 us, the copy rate; gradient of 2 x 8K tokens of 16 + 4 heads,
// 168 MB, 27 us (92 % of it); append of five prompts, 4.7K tokens of 16 + 4 + 4
// heads, 57 MB, 10 us; append of 32K tokens of 16 + 16 + 16 heads to e4m3 pages, 672 MB,
// 118 us (84 %; it issues in 71 % of the cycles: maxima, scaling and conversion
// on top of the rotation); to bf16 pages, 805 MB, 125 us (95 %);
// fp32, one token a thread, to fp32 pages, 1611 MB, 264 us (90 %).  One token: 2.5 us.
enum Mode { kRope, kRopeBackward, kAppend, kAppendE4m3 };

// U.  The e4m3 append, bound by instructions, shares its addressing among four
// tokens (118 us, with two 129); the others want the registers for more blocks.
template <typename T, int MODE>
constexpr int kAtOnce = sizeof(T) == 4 ? 1 : MODE == kAppendE4m3 ? 4 : 2;

// cos and sin of frequency f: two frequencies (c, c, s, s) to 16 bytes, laid out
// so that the lanes of a head read neighbouring 16 bytes.
__device__ __forceinline__ int table_at(int f) { return ((f & 7) >> 1) * 32 + (f >> 3) * 4 + (f & 1); }

template <bool BACKWARD>
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    if (BACKWARD) s = -s;
    const float y = a * c - b * s;
    b = b * c + a * s;
    a = y;
}

template <typename T, int MODE, int D>
__global__ void __launch_bounds__(kMaxThreads) rotate_kernel(const __grid_constant__ RotateArgs a) {
    constexpr bool kStored = MODE >= kAppend;   // k and v go to pages
    constexpr bool kBackward = MODE == kRopeBackward;
    constexpr int U = kAtOnce<T, MODE>, lph = D / 16;
    __shared__ __align__(16) float s_table[kMaxTokens][2 * kMaxHalf];
    __shared__ int64_t s_row[kMaxTokens];
    // What waits for this grid may be set up now; this grid waits for the one
    // before it.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int half = a.rot / 2;
    const int t0 = blockIdx.x * (U * a.span), part = blockIdx.y;
    const int tokens = min(a.tokens - t0, U * a.span);

    // This thread's slot: of the part's slots, side by side with other tokens'.
    const int beside = a.span == 1 ? threadIdx.x >= a.part_slots : threadIdx.x / a.part_slots;   // token of the span
    const int i = part * a.part_slots + threadIdx.x - beside * a.part_slots;
    int head = i / lph;   // q's, then k's, then v's
    const int sub = i % lph;
    const bool on = beside < a.span && head < a.Hq + (kStored ? 2 : 1) * a.Hkv;
    const int which = head < a.Hq ? 0 : head < a.Hq + a.Hkv ? 1 : 2;
    head -= which == 0 ? 0 : which == 1 ? a.Hq : a.Hq + a.Hkv;
    const bool turned = which < 2 && sub * 16 < a.rot;
    const bool apart = turned && !a.interleaved;
    const int lo = head * D + (apart ? sub * 8 : sub * 16), apart_by = apart ? half : 8;

    Eight<T> raw[U][2];
    {
        const int64_t stride = which == 0 ? a.q_stride : which == 1 ? a.k_stride : a.v_stride;
        const T* src = static_cast<const T*>(which == 0 ? a.q : which == 1 ? a.k : a.v) + (t0 + beside) * stride + lo;
#pragma unroll
        for (int u = 0; u < U; ++u, src += a.span * stride)
            if (on && u * a.span + beside < tokens) {
                raw[u][0].load(src);
                raw[u][1].load(src + apart_by);
            }
    }

    // Places and tables: task x is token x / pieces, frequencies 32 (x % pieces) on.
    const bool table_used = part * (a.part_slots / lph) < a.Hq + a.Hkv;   // a part may hold values alone
    const int pieces = table_used ? max((half + 31) / 32, 1) : 1;
    for (int x = threadIdx.x / 32; x < tokens * pieces; x += blockDim.x / 32) {
        const int j = pieces == 2 ? x >> 1 : x, f = (pieces == 2 ? (x & 1) * 32 : 0) + (threadIdx.x & 31);
        const int t = t0 + j;
        Place place = {0, 0};
        int page = 0;
        if (kStored) {
            place = place_of(a, t);
            page = place.b < 0 ? -1 : a.block_table[static_cast<int64_t>(place.b) * a.max_pages + (place.pos >> a.page_lg)];
        } else {
            place.pos = a.positions ? a.positions[t] : t % a.N;
        }
        if (table_used && f < half) {   // while the page number is on its way
            float factor = a.factor;
            const uint64_t fraction = turn_fraction(a.inv_freq[f], factor);
            const float2 cs = cos_sin(fraction, place.pos, factor);
            s_table[j][table_at(f)] = cs.x;
            s_table[j][table_at(f) + 2] = cs.y;
        }
        if ((threadIdx.x & 31) == 0) {   // the pieces of a token agree
            int64_t row = 0;
            if (kStored) {
                row = page < 0 || page >= a.num_pages ? -1 : (static_cast<int64_t>(page) << a.page_lg) + (place.pos & ((1 << a.page_lg) - 1));
                if (row < 0 && place.b >= 0) atomicOr(a.err, kDevErrInput);
            }
            s_row[j] = row;
        }
    }
    __syncthreads();

    const bool paged = kStored && which > 0;
    const int size = MODE == kAppendE4m3 && paged ? 1 : static_cast<int>(sizeof(T));
    char* const dst = static_cast<char*>(which == 0 ? a.q_out : which == 1 ? a.k_out : a.v_out) + lo * size;
    const int64_t out_stride = (paged ? a.Hkv * D : which == 0 ? a.q_out_stride : a.k_out_stride) * size;
    const unsigned paged_lanes = MODE == kAppendE4m3 ? __ballot_sync(0xffffffffu, paged) : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int token = u * a.span + beside;
        const bool mine = on && token < tokens;
        float x[16];
        int64_t row = -1;
        if (mine) {
            row = s_row[token];
            raw[u][0].get(x);
            raw[u][1].get(x + 8);
            if (turned) {
                const float4* table = reinterpret_cast<const float4*>(s_table[token]) + sub;
                if (a.interleaved) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float4 cs = table[e / 2 * 8];
                        turn<kBackward>(x[2 * e], x[2 * e + 1], cs.x, cs.z);
                        turn<kBackward>(x[2 * e + 2], x[2 * e + 3], cs.y, cs.w);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float4 cs = table[e / 2 * 8];
                        turn<kBackward>(x[e], x[8 + e], cs.x, cs.z);
                        turn<kBackward>(x[e + 1], x[9 + e], cs.y, cs.w);
                    }
                }
            }
        }
        if (MODE == kAppendE4m3 && paged) {
            float amax = 0.f;   // a NaN does not enter it
            if (mine) {
#pragma unroll
                for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
            }
#pragma unroll
            for (int o = lph / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(paged_lanes, amax, o));
            if (row >= 0) {
                const int e = row_exponent(amax);
                const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                for (int c = 0; c < 16; ++c) x[c] *= inv;
                uint8_t* to = reinterpret_cast<uint8_t*>(dst + row * out_stride);
                store8_e4m3(to, x);
                store8_e4m3(to + apart_by, x + 8);
                if (sub == 0) {
                    const int64_t page = row >> a.page_lg, at = row & ((1 << a.page_lg) - 1);
                    (which == 1 ? a.k_exp : a.v_exp)[((page * a.Hkv + head) << a.page_lg) + at] = static_cast<uint8_t>(e + 127);
                }
            }
        } else if (row >= 0) {
            T* to = reinterpret_cast<T*>(dst + (paged ? row : t0 + token) * out_stride);
            store8(to, x);
            store8(to + apart_by, x + 8);
        }
    }
}

// A block covers all slots of a token, as many tokens side by side as 128
// threads hold; more than kMaxThreads slots are cut into parts of whole heads
// and at most 128 slots (16 + 16 + 16 heads: bf16 append 126 us, in two parts 130,
// whole 161, as then only two blocks fit an SM; 16 + 4 heads: whole 27 us, in two
// parts 29).
template <typename T, int MODE, int D>
cudaError_t launch(RotateArgs a, cudaStream_t s) {
    constexpr int U = kAtOnce<T, MODE>, lph = D / 16;
    const int heads = a.Hq + (MODE >= kAppend ? 2 : 1) * a.Hkv;
    const int parts = heads * lph <= kMaxThreads ? 1 : (heads * lph + 127) / 128;
    a.part_slots = (heads + parts - 1) / parts * lph;
    a.span = std::max(1, std::min({128 / a.part_slots, kMaxTokens / U, (a.tokens + U - 1) / U}));
    const int threads = (a.part_slots * a.span + 31) / 32 * 32;
    const dim3 grid((a.tokens - 1) / (U * a.span) + 1, parts);
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = dependent_launch(grid, threads, s, attr);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, rotate_kernel<T, MODE, D>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int MODE>
cudaError_t launch(const RotateArgs& a, cudaStream_t s) {
    return a.d == 128 ? launch<T, MODE, 128>(a, s) : launch<T, MODE, 64>(a, s);
}

}  // namespace

cudaError_t launch_rope(const RotateArgs& a, int dtype, bool backward, cudaStream_t s) {
    if (dtype == SWIATTN_BF16)
        return backward ? launch<__nv_bfloat16, kRopeBackward>(a, s) : launch<__nv_bfloat16, kRope>(a, s);
    return backward ? launch<float, kRopeBackward>(a, s) : launch<float, kRope>(a, s);
}

cudaError_t launch_append(const RotateArgs& a, int dtype, int page_dtype, cudaStream_t s) {
    if (page_dtype == SWIATTN_E4M3) return launch<__nv_bfloat16, kAppendE4m3>(a, s);
    return dtype == SWIATTN_BF16 ? launch<__nv_bfloat16, kAppend>(a, s) : launch<float, kAppend>(a, s);
}

}  // namespace swi

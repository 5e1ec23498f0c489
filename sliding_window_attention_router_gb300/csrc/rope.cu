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
// quarter turn comes off its top 32 bits as a whole number, so what goes to
// sincospif is within an eighth of a turn and its rounding to a float costs
// at most 2^-28 of a turn.

#include "swiattn.h"
#include "swiattn_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp8.h>

namespace swi {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = 64;   // rotated pairs of a head: d <= 128

// ---- eight elements of T as floats -----------------------------------------
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(h[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void load8(const float* p, float* x) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
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
// whole turn (positions are whole numbers, so whole turns do not matter).
// 1/2pi is held in two doubles, so the fraction is right to 2^-63 for |w| <= 1.
__device__ __forceinline__ uint64_t turn_fraction(double w) {
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;   // 1/2pi = kHi + kLo
    const double p = w * kHi;
    const double e = fma(w, kHi, -p) + w * kLo;
    const double f = p - floor(p);                     // exact, in [0, 1)
    const double hi = floor(f * 4294967296.0);         // first 32 bits
    const double lo = (f * 4294967296.0 - hi) * 4294967296.0 + e * 18446744073709551616.0;
    return (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(static_cast<int64_t>(rint(lo)));
}
// m cos and m sin of position p times frequency F.
__device__ __forceinline__ float2 cos_sin(uint64_t F, int p, float m) {
    const uint64_t turn = F * static_cast<uint64_t>(static_cast<int64_t>(p));
    const uint32_t top = static_cast<uint32_t>(turn >> 32);
    const uint32_t quarter = (top + 0x20000000u) >> 30;
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(top - (quarter << 30))) * 0x1p-31f, &s, &c);
    if (quarter & 1) {   // a quarter turn on: (c, s) -> (-s, c)
        const float o = c;
        c = -s;
        s = o;
    }
    if (quarter & 2) m = -m;
    return make_float2(m * c, m * s);
}

// A slot is 16 elements of one head: lane `sub` of the head's d/16 lanes.
// Rotated slots (sub < rot/16) hold eight pairs, the others pass through.
struct Slot {
    int lo, hi;   // element offsets of its two groups of eight
};
__device__ __forceinline__ Slot slot_of(int sub, int rot, bool interleaved) {
    if (!interleaved && sub * 16 < rot) return {sub * 8, rot / 2 + sub * 8};
    return {sub * 16, sub * 16 + 8};
}

// Rotates the 16 elements of a slot; cs holds (m cos, m sin) of its eight pairs.
template <bool BACKWARD>
__device__ __forceinline__ void rotate(float* x, const float2* cs, bool interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float c = cs[e].x, s = BACKWARD ? -cs[e].y : cs[e].y;
        if (interleaved) {
            const float a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = a * c - b * s;
            x[2 * e + 1] = b * c + a * s;
        } else {
            const float a = x[e], b = x[8 + e];
            x[e] = a * c - b * s;
            x[8 + e] = b * c + a * s;
        }
    }
}

// ---- rotation of q and k ---------------------------------------------------
// One token a block: the block's first threads take the token's cosines and
// sines, then each thread rotates slot after slot of its heads.
template <typename T, bool BACKWARD>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a) {
    __shared__ float2 cs[kMaxHalf];
    const int64_t t = blockIdx.x;
    const int pos = a.positions ? a.positions[t] : static_cast<int>(t % a.N);
    if (threadIdx.x < a.rot / 2) cs[threadIdx.x] = cos_sin(turn_fraction(a.inv_freq[threadIdx.x]), pos, a.factor);
    __syncthreads();
    const int lph = a.d / 16;
    const int slots = (a.Hq + a.Hkv) * lph;
    for (int i = threadIdx.x; i < slots; i += kThreads) {
        const int head = i / lph, sub = i % lph;
        const Slot sl = slot_of(sub, a.rot, a.interleaved);
        const bool isq = head < a.Hq;
        const T* src = isq ? static_cast<const T*>(a.q) + t * a.q_stride + head * a.d
                           : static_cast<const T*>(a.k) + t * a.k_stride + (head - a.Hq) * a.d;
        T* dst = isq ? static_cast<T*>(a.q_out) + t * a.q_out_stride + head * a.d
                     : static_cast<T*>(a.k_out) + t * a.k_out_stride + (head - a.Hq) * a.d;
        float x[16];
        load8(src + sl.lo, x);
        load8(src + sl.hi, x + 8);
        if (sub * 16 < a.rot) rotate<BACKWARD>(x, cs + sub * 8, a.interleaved);
        store8(dst + sl.lo, x);
        store8(dst + sl.hi, x + 8);
    }
}

// ---- append ----------------------------------------------------------------
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

// Position and pool row (page * page_size + slot) of new token t; row < 0: the
// token is not stored (a padding row, an empty slot, or bad input, which is
// reported).  Called by a whole warp.
struct Place {
    int pos;
    int64_t row;
};
__device__ __forceinline__ Place place_of(const AppendArgs& a, int t, unsigned int* err) {
    int b = t, after = 1;   // tokens of the sequence from t on
    if (a.starts) {
        b = find_sequence(a.starts, a.B, t);
        if (b < 0) return {0, -1};
        after = a.starts[b + 1] - t;
        if (after <= 0) return {0, -1};
    }
    const int len = a.seq_lens[b];
    if (len == 0) return {0, -1};
    const int64_t pos = static_cast<int64_t>(len) - after;
    if (pos >= 0 && (pos >> a.page_lg) < a.max_pages) {
        const int32_t page = a.block_table[static_cast<int64_t>(b) * a.max_pages + (pos >> a.page_lg)];
        if (page >= 0 && page < a.num_pages)
            return {static_cast<int>(pos),
                    (static_cast<int64_t>(page) << a.page_lg) + (pos & ((1 << a.page_lg) - 1))};
    }
    if ((threadIdx.x & 31) == 0) atomicOr(err, kDevErrInput);
    return {0, -1};
}

// Exponent e of the smallest power of two with amax <= 448 * 2^e, within
// [-126, 127]: amax = m 2^x with m in [1, 2) and 448 = 1.75 * 2^8.
__device__ __forceinline__ int row_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(-126, min(127, e));
}

// One token a block.
template <typename T, bool E4M3>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a, unsigned int* err) {
    __shared__ float2 cs[kMaxHalf];
    __shared__ Place where;
    const int t = blockIdx.x;
    if (threadIdx.x < 32) {
        const Place p = place_of(a, t, err);
        if (threadIdx.x == 0) where = p;
    }
    __syncthreads();
    const int pos = where.pos;
    const int64_t row = where.row;
    if (row < 0) return;
    if (threadIdx.x < a.rot / 2) cs[threadIdx.x] = cos_sin(turn_fraction(a.inv_freq[threadIdx.x]), pos, a.factor);
    __syncthreads();
    const int lph = a.d / 16;
    const int nq = a.Hq * lph, nk = a.Hkv * lph;
    const int slots = nq + 2 * nk;
    // Whole warps go round together, for the shuffles of the row maximum.
    for (int i0 = threadIdx.x & ~31; i0 < slots; i0 += kThreads) {
        const int i = i0 + (threadIdx.x & 31);
        const bool active = i < slots;
        const int which = i < nq ? 0 : i < nq + nk ? 1 : 2;
        const int j = which == 0 ? i : which == 1 ? i - nq : i - nq - nk;
        const int head = j / lph, sub = j % lph;
        const Slot sl = slot_of(sub, which == 2 ? 0 : a.rot, a.interleaved);
        float x[16];
        if (active) {
            const T* src = which == 0   ? static_cast<const T*>(a.q) + t * a.q_stride
                           : which == 1 ? static_cast<const T*>(a.k) + t * a.k_stride
                                        : static_cast<const T*>(a.v) + t * a.v_stride;
            src += head * a.d;
            load8(src + sl.lo, x);
            load8(src + sl.hi, x + 8);
            if (which < 2 && sub * 16 < a.rot) rotate<false>(x, cs + sub * 8, a.interleaved);
        }
        if (which == 0) {
            if (active) {
                T* dst = static_cast<T*>(a.q_out) + (static_cast<int64_t>(t) * a.Hq + head) * a.d;
                store8(dst + sl.lo, x);
                store8(dst + sl.hi, x + 8);
            }
        }
        if constexpr (E4M3) {
            float amax = 0.f;   // a NaN does not enter it
            if (active) {
#pragma unroll
                for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
            }
            for (int o = lph / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            if (active && which > 0) {
                const int e = row_exponent(amax);
                const float inv = __uint_as_float(static_cast<uint32_t>(127 - max(e, -126)) << 23);
                uint8_t* dst = static_cast<uint8_t*>(which == 1 ? a.k_pages : a.v_pages) + (row * a.Hkv + head) * a.d;
#pragma unroll
                for (int c = 0; c < 16; ++c) x[c] *= inv;
                store8_e4m3(dst + sl.lo, x);
                store8_e4m3(dst + sl.hi, x + 8);
                if (sub == 0) {
                    uint8_t* ex = which == 1 ? a.k_exp : a.v_exp;
                    const int64_t page = row >> a.page_lg, slot = row & ((1 << a.page_lg) - 1);
                    ex[((page * a.Hkv + head) << a.page_lg) + slot] = static_cast<uint8_t>(e + 127);
                }
            }
        } else {
            if (active && which > 0) {
                T* dst = static_cast<T*>(which == 1 ? a.k_pages : a.v_pages) + (row * a.Hkv + head) * a.d;
                store8(dst + sl.lo, x);
                store8(dst + sl.hi, x + 8);
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int dtype, bool backward, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(a.tokens);
    if (dtype == SWIATTN_BF16) {
        if (backward) rope_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, s>>>(a);
        else rope_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (backward) rope_kernel<float, true><<<grid, kThreads, 0, s>>>(a);
        else rope_kernel<float, false><<<grid, kThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_append(const AppendArgs& a, int dtype, int page_dtype, unsigned int* err,
                          cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(a.tokens);
    if (page_dtype == SWIATTN_E4M3) append_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, s>>>(a, err);
    else if (dtype == SWIATTN_BF16) append_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, s>>>(a, err);
    else append_kernel<float, false><<<grid, kThreads, 0, s>>>(a, err);
    return cudaGetLastError();
}

}  // namespace swi

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
#include <algorithm>
#include <atomic>

namespace swi {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = 64;     // rotated pairs of a head: d <= 128
constexpr int kMaxTile = 16;     // tokens of a tile
template <typename T>
constexpr int kAtOnce = sizeof(T) == 2 ? 4 : 2;   // slots a thread loads before it rotates one (64 bytes each in fp32)

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

// Position and pool row (page * page_size + slot) of new token t; row < 0: the
// token is not stored (a padding row, an empty slot, or bad input, which is
// reported).  Called by a whole warp.
struct Place {
    int pos;
    int64_t row;
};
__device__ __forceinline__ Place place_of(const RotateArgs& a, int t) {
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
    if ((threadIdx.x & 31) == 0) atomicOr(a.err, kDevErrInput);
    return {0, -1};
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
// groups that pass through.  One thread loads a slot with two 16-byte loads (bf16).
//
// HBM-bound: 6 operations on 4 bytes.  A block takes tiles of `tile` tokens,
// one after another (so the frequencies' 64-bit fractions are taken once a
// block), and per tile
//   1. starts the loads of kAtOnce slots a thread, which need no position,
//   2. works out the tile's cosines and sines in shared memory, one for all
//      heads, and the places of the next tile's tokens,
//   3. after one barrier rotates, converts and stores.
// One barrier a tile is enough: a warp that is ahead writes the table of a tile
// on (two tables) and the places of two tiles on (three) while others still read.
enum Mode { kRope, kRopeBackward, kAppend, kAppendE4m3 };

// Where a thread's slot is within a tile; the same for every tile.
struct Slot {
    int token;    // in the tile; -1: none
    int which;    // 0 q, 1 k, 2 v
    int head, sub;
    int lo, hi;   // element offsets of its two groups within the head
    bool turned;
};
__device__ __forceinline__ Slot slot_of(int i, int slots, const RotateArgs& a) {
    const int lph = a.d / 16, nq = a.Hq * lph, nk = a.Hkv * lph;
    Slot s;
    s.token = i / slots;
    const int j = i - s.token * slots;
    s.which = j < nq ? 0 : j < nq + nk ? 1 : 2;
    const int k = s.which == 0 ? j : s.which == 1 ? j - nq : j - nq - nk;
    s.head = k / lph;
    s.sub = k - s.head * lph;
    s.turned = s.which < 2 && s.sub * 16 < a.rot;
    const bool apart = s.turned && !a.interleaved;
    s.lo = apart ? s.sub * 8 : s.sub * 16;
    s.hi = apart ? a.rot / 2 + s.sub * 8 : s.sub * 16 + 8;
    if (s.token >= a.tile) s.token = -1;
    return s;
}

// (m cos, m sin) of frequency f of a token, two frequencies to 16 bytes, laid
// out so that the lanes of a head read neighbouring 16 bytes.
__device__ __forceinline__ int table_at(int f) { return ((f & 7) >> 1) * 16 + (f >> 3) * 2 + (f & 1); }

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const __grid_constant__ RotateArgs a) {
    constexpr bool kStored = MODE == kAppend || MODE == kAppendE4m3;   // k and v go to pages
    constexpr int U = kAtOnce<T>;
    __shared__ __align__(16) float2 s_table[2][kMaxTile][kMaxHalf];
    __shared__ Place s_place[3][kMaxTile];
    __shared__ uint64_t s_freq[kMaxHalf];
    const int lph = a.d / 16;
    const int slots = (a.Hq + (kStored ? 2 : 1) * a.Hkv) * lph;
    const int tiles = (a.tokens - 1) / a.tile + 1;
    const int warp = threadIdx.x / 32;

    auto places = [&](int tile, int at) {   // of a tile's tokens, a warp a token
        for (int j = warp; j < a.tile; j += kThreads / 32) {
            const int t = tile * a.tile + j;
            Place p = {0, -1};
            if (t < a.tokens) {
                if (kStored) p = place_of(a, t);
                else p = {a.positions ? a.positions[t] : t % a.N, 0};
            }
            if (threadIdx.x % 32 == 0) s_place[at][j] = p;
        }
    };
    if (static_cast<int>(threadIdx.x) < a.rot / 2) s_freq[threadIdx.x] = turn_fraction(a.inv_freq[threadIdx.x]);
    places(blockIdx.x, 0);
    __syncthreads();

    int buf = 0, now = 0;   // this tile's table and places
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1, now = now == 2 ? 0 : now + 1) {
        const int64_t t0 = static_cast<int64_t>(tile) * a.tile;
        const int left = a.tokens - tile * a.tile;   // tokens from t0 on
        for (int i0 = 0; i0 < a.tile * slots; i0 += U * kThreads) {
            Slot slot[U];
            Eight<T> raw[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                slot[u] = slot_of(i0 + u * kThreads + threadIdx.x, slots, a);
                if (slot[u].token >= left) slot[u].token = -1;
                if (slot[u].token >= 0) {
                    const int64_t t = t0 + slot[u].token;
                    const T* src = slot[u].which == 0   ? static_cast<const T*>(a.q) + t * a.q_stride
                                   : slot[u].which == 1 ? static_cast<const T*>(a.k) + t * a.k_stride
                                                        : static_cast<const T*>(a.v) + t * a.v_stride;
                    src += slot[u].head * a.d;
                    raw[u][0].load(src + slot[u].lo);
                    raw[u][1].load(src + slot[u].hi);
                }
            }
            if (i0 == 0) {
                const int half = a.rot / 2, n = min(left, a.tile) * half;
                for (int i = threadIdx.x; i < n; i += kThreads) {
                    const int j = i / half, f = i - j * half;
                    s_table[buf][j][table_at(f)] = cos_sin(s_freq[f], s_place[now][j].pos, a.factor);
                }
                if (tile + gridDim.x < tiles) places(tile + gridDim.x, now == 2 ? 0 : now + 1);
                __syncthreads();
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Slot& s = slot[u];
                float x[16];
                const int64_t row = s.token >= 0 ? s_place[now][s.token].row : -1;
                if (s.token >= 0) {
                    raw[u][0].get(x);
                    raw[u][1].get(x + 8);
                }
                if (s.token >= 0 && s.turned) {
                    const float4* table = reinterpret_cast<const float4*>(s_table[buf][s.token]) + s.sub;
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float4 cs = table[e / 2 * 8];
                        const float c[2] = {cs.x, cs.z};
                        const float sn[2] = {MODE == kRopeBackward ? -cs.y : cs.y, MODE == kRopeBackward ? -cs.w : cs.w};
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            if (a.interleaved) {
                                float &p = x[2 * (e + r)], &q = x[2 * (e + r) + 1];
                                const float y = p * c[r] - q * sn[r];
                                q = q * c[r] + p * sn[r];
                                p = y;
                            } else {
                                float &p = x[e + r], &q = x[8 + e + r];
                                const float y = p * c[r] - q * sn[r];
                                q = q * c[r] + p * sn[r];
                                p = y;
                            }
                        }
                    }
                }
                const int64_t t = t0 + s.token;
                if (s.which == 0 || !kStored) {
                    if (row >= 0) {
                        T* dst = s.which == 0 ? static_cast<T*>(a.q_out) + t * a.q_out_stride
                                              : static_cast<T*>(a.k_out) + t * a.k_out_stride;
                        dst += s.head * a.d;
                        store8(dst + s.lo, x);
                        store8(dst + s.hi, x + 8);
                    }
                }
                if constexpr (MODE == kAppend) {
                    if (s.which > 0 && row >= 0) {
                        T* dst = static_cast<T*>(s.which == 1 ? a.k_out : a.v_out) + (row * a.Hkv + s.head) * a.d;
                        store8(dst + s.lo, x);
                        store8(dst + s.hi, x + 8);
                    }
                }
                if constexpr (MODE == kAppendE4m3) {
                    float amax = 0.f;   // a NaN does not enter it
                    if (s.token >= 0) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
                    }
                    for (int o = lph / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    if (s.which > 0 && row >= 0) {
                        const int e = row_exponent(amax);
                        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                        uint8_t* dst = static_cast<uint8_t*>(s.which == 1 ? a.k_out : a.v_out) + (row * a.Hkv + s.head) * a.d;
#pragma unroll
                        for (int c = 0; c < 16; ++c) x[c] *= inv;
                        store8_e4m3(dst + s.lo, x);
                        store8_e4m3(dst + s.hi, x + 8);
                        if (s.sub == 0) {
                            const int64_t page = row >> a.page_lg, at = row & ((1 << a.page_lg) - 1);
                            (s.which == 1 ? a.k_exp : a.v_exp)[((page * a.Hkv + s.head) << a.page_lg) + at] =
                                static_cast<uint8_t>(e + 127);
                        }
                    }
                }
            }
        }
        if (tile + gridDim.x >= tiles) break;
    }
}

// Tokens of a tile: what kAtOnce slots a thread cover, less where that would
// leave SMs without a tile.  Blocks: what is resident at once.
template <typename T, int MODE>
cudaError_t launch(RotateArgs a, int sms, cudaStream_t s) {
    const int slots = (a.Hq + (MODE >= kAppend ? 2 : 1) * a.Hkv) * (a.d / 16);
    int tile = std::max(1, std::min(kMaxTile, kAtOnce<T> * kThreads / slots));
    a.tile = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(tile, a.tokens / (2 * sms))));
    static std::atomic<int> resident[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int per_sm = dev < 64 ? resident[dev].load(std::memory_order_relaxed) : 0;
    if (per_sm == 0) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, rotate_kernel<T, MODE>, kThreads, 0);
        if (e != cudaSuccess) return e;
        per_sm = std::max(per_sm, 1);
        if (dev < 64) resident[dev].store(per_sm, std::memory_order_relaxed);
    }
    const int64_t tiles = (a.tokens - 1) / a.tile + 1;
    rotate_kernel<T, MODE><<<static_cast<unsigned>(std::min<int64_t>(tiles, static_cast<int64_t>(sms) * per_sm)), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RotateArgs& a, int dtype, bool backward, int sms, cudaStream_t s) {
    if (dtype == SWIATTN_BF16)
        return backward ? launch<__nv_bfloat16, kRopeBackward>(a, sms, s) : launch<__nv_bfloat16, kRope>(a, sms, s);
    return backward ? launch<float, kRopeBackward>(a, sms, s) : launch<float, kRope>(a, sms, s);
}

cudaError_t launch_append(const RotateArgs& a, int dtype, int page_dtype, int sms, cudaStream_t s) {
    if (page_dtype == SWIATTN_E4M3) return launch<__nv_bfloat16, kAppendE4m3>(a, sms, s);
    return dtype == SWIATTN_BF16 ? launch<__nv_bfloat16, kAppend>(a, sms, s) : launch<float, kAppend>(a, sms, s);
}

}  // namespace swi

// Decode over a paged cache of 8-bit keys and values: one query a sequence
// against the window, the anchors and the window, or the whole history, of
// e4m3 rows that each carry a power of two.
//
// The mathematics, for one query head and the visited keys j, in base 2:
//   s_j = scale log2(e) 2^(ku_j - 127) <q, k8_j>,   x_j = s_j - m,
//   l = sum_j 2^x_j,            a = sum_j 2^(x_j + vu_j - 127 - n) v8_j,
//   o = 2^n a / l,              lse = ln 2 (m + log2 l),
// with m the largest s_j and n the largest x_j + vu_j - 127.  Folding a value
// row's power of two into its weight leaves the e4m3 bytes as they are; the
// weights then have a maximum of their own, n, so that what is rounded to 16
// bits is always of order 1 at the largest contribution, whatever the rows'
// sizes.  n is relative to m: beside a score of 2^24 and more a row's power of
// two would be rounded away.  Parts (m, n, l, a) of the key set join by their
// maxima; where m rises, n falls by as much.
//
// The bound is the cache's bytes: 16 keys of one head are 4 KiB (d = 128), and
// with up to 8 query heads to a key head 16 tensor-core products.  So the work
// is to keep bytes on their way, and the instructions per byte few:
//  - a warp streams tiles of 16 keys of one head, key and value rows and their
//    exponents by asynchronous copies (TMA where pages hold a whole tile) into a
//    ring of its own; it waits for no other warp.  Copies by the threads
//    themselves (16 bytes each) took 145 requests to the L2 a tile and 68 us
//    where these took 58 (8 sequences of 32K, 4 key heads, all visited; 50 us
//    with what came after).
//  - the products are mma.sync m16n8k16, fp16 with fp32 accumulation, and not
//    tcgen05: an e4m3 value is exact in fp16, a tcgen05 product of e4m3 would want
//    q and the weights in e4m3 too, and the tensor pipe is busy 25 % of the time.
//    q is made exact by a power of two per head (every element within 2^31 of
//    the head's largest); the weights go in as two fp16, the nearest value and
//    what it leaves, right to 2^-22 of each or 2^-32 of the largest (kRoom).  With
//    the first alone, 2^-11 of each, one bf16 result in twenty was the neighbour
//    of the one that fp32 weights give, for 16 x 32K in 58.1 us in place of 59.4.
//      S^T [16 keys x 8 heads] = K Q^T: a thread's 16-byte pieces of two key rows
//      are its A fragments after conversion, the order of d being free as long
//      as q's fragments follow it;
//      O^T [d x 8 heads] += V^T W^T: a thread's 16-byte pieces of four value
//      rows are its A fragments after pairing bytes of neighbouring rows (one
//      byte permute for two registers), and W^T comes from S^T by 8 x 8
//      transposes inside the warp.
//
// Measured (one GB300, copy rate 6787 GB/s): 16 sequences of 32K, 16 heads, two
// of them whole and fourteen in windows of 1024, 330 MB: 59.5 us, of which this
// kernel 54 (first data after 3 us, warps ending within 3 us of one another) and
// the join the rest; 8 whole sequences of 32K with 16 query and 4 key heads, 271
// MB: 50.5 us.  One sequence of 777 tokens: 8.0 us, a chain of dependent reads
// (lengths, page numbers, rows) and two launches.  A captured graph of ten calls;
// 33 million warp instructions for the first (issue 54 %).  Further from their
// bytes: two groups of heads (the second case with 48 query heads: 64 us; half
// the warps, each with a ring of the same depth), pages under a tile (with pages
// of 8, 4 and 1 tokens: 60, 61 and 66 us; page number and exponents waited for in
// each tile), and batches whose (sequence, key head)s come near the number of
// warps (64, 96 and 160 windows of 1024, 16 heads: 71, 94 and 147 us for 40, 60
// and 100 us of bytes; blocks of unequal length, a last round of few).
// Comparisons beside the constants below are of the time when they were chosen,
// on the first case unless they say otherwise.

#include "swiattn.h"
#include "ptx.cuh"
#include "swiattn_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>
#include <algorithm>
#include <atomic>
#include <cstring>

namespace swi {
namespace {

constexpr int kTile = 16;        // keys of one product tile
constexpr int kWarps = 4;        // warps of a block (they share nothing)
constexpr int kStages = 2;       // tiles a warp holds: one at work, one on its way (3: 59.1 us become 61.0)
template <int NH>
constexpr int kBlocksPerSm = NH == 1 ? 4 : 2;   // by registers, 128 or 255 a thread (5 at 96, spilling: 58 us become 78)
constexpr int kMaxWarps = 152 * 4 * kWarps;     // workers of one call: what fills a GB300
constexpr int kMinRun = 2;       // tiles a warp takes at least (one sequence of 777 tokens: 8.2 us, at 4 10.3, at 8 12.3)
// The values' weights go to fp16: their reference lies kRoom below the largest
// (base 2), and they pass it by up to kSlack before it is raised, so that they
// end at 2^15 and reach down to 2^-31 of the largest (smaller ones are lost to
// the result, not to its sum of weights: under a bf16 half step of it unless
// 2^23 such keys meet in one warp's part).
constexpr float kRoom = 7.f;
constexpr float kSlack = 15.f;

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Where references and maxima start: the lowest finite value, below no score
// but -inf (scores that are all -inf leave it), and finite, so that no
// difference of it and a score or a maximum is a NaN.
constexpr float kLow = -FLT_MAX;

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same onto zeros.
__device__ __forceinline__ void mma_f16_first(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Transposes the 8 x 8 matrix of 16-bit elements that the warp's registers hold.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Four e4m3 bytes as two pairs of fp16 (exact).
__device__ __forceinline__ void halves_of(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {   // zeros where not on
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

// What sequence b's query visits: anchors [0, na) and [lo, len), as 16-key
// tiles at multiples of 16 from the cache's start (so a tile never straddles a
// page of 16 or more): `ta` anchor tiles, then the others, `tiles` in all.
struct Visit {
    int len, lo, na;
    int ta, tiles;
};
__device__ __forceinline__ Visit visit_of(const DecodeE4m3Args& a, int b) {
    Visit v;
    v.len = min(max(a.seq_lens[b], 0), a.max_pages << a.page_lg);
    v.lo = a.gate[b] ? 0 : max(0, v.len - a.W);
    v.na = min(a.n_anchor, v.lo);
    v.ta = (v.na + kTile - 1) / kTile;
    v.tiles = v.ta + (v.len > 0 ? (v.len + kTile - 1) / kTile - v.lo / kTile : 0);
    return v;
}

// The work: every sequence's tiles are cut into blocks of `run` tiles, and a
// warp takes one block of one KV head at a time: item (blocks before it) * Hkv +
// head.  So neighbouring warps read neighbouring heads of the same tokens,
// which lie side by side in memory (16 heads: 66 us, against 74 with equal runs
// cut without regard to the heads).  `run` is the least that gives each warp at
// most one item, where the batch has fewer (sequence, head)s than half the
// warps; else items come round by round.  Items' sums are joined in the order
// of the blocks.
//
// The plan that the split kernel leaves for the join: plan[b] blocks of the
// sequences before b, plan[B] tiles of a block.
__device__ __forceinline__ int inclusive_sum(int x) {   // over the warp's lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if ((threadIdx.x & 31) >= o) x += y;
    }
    return x;
}

// Shared memory of a warp: a ring of tiles, each 16 key rows, then 16 value
// rows, of D bytes.  A row's 16-byte pieces lie swizzled, as a tile copy of
// that width leaves them (128-byte rows: piece ^ (row & 7); 64-byte rows: piece ^
// (row / 2 & 3)), so that the eight rows a quarter of a warp reads at once
// spread over the banks.
template <int D>
constexpr int kStageBytes = kTile * 2 * D;
template <int D>
constexpr int kSharedBytes = kWarps * kStages * kStageBytes<D> + 1024;   // and room to align
template <int D>
__device__ __forceinline__ int piece_at(int row, int piece) {
    return row * D + ((D == 128 ? piece ^ (row & 7) : piece ^ ((row >> 1) & 3)) << 4);
}

// NH: groups of eight query heads (1: Hq/Hkv <= 8, 2: <= 16).  WIDE: pages of
// 16 tokens or more, where a tile's rows follow one another.
template <int D, int NH, bool WIDE>
__global__ void __launch_bounds__(kWarps * 32, kBlocksPerSm<NH>)
decode_e4m3_split_kernel(const __grid_constant__ DecodeE4m3Args a, const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map) {
    constexpr int KS = D / 16;    // 16-deep steps of the score product, and 16-row tiles of O^T
    constexpr int KW = D / 64;    // 16-byte pieces of a key row a thread holds
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(16) uint8_t s_exp[kWarps][kStages][32];   // of a tile's 16 K rows, then V rows
    __shared__ uint64_t s_full[kWarps][kStages];
    __shared__ int s_abort[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int G = a.Hq / a.Hkv;
    uint8_t* const queue = smem + ((1024 - (smem_u32(smem) & 1023)) & 1023) + warp * kStages * kStageBytes<D>;
    const uint32_t queue_s = smem_u32(queue);
    const uint32_t mask = (1u << a.page_lg) - 1;
    const size_t token_bytes = static_cast<size_t>(a.Hkv) * D;
    if (WIDE && lane == 0) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) mbar_init(&s_full[warp][i], 1);
        s_abort[warp] = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    __syncwarp();

    asm volatile("griddepcontrol.wait;" ::: "memory");   // for the kernel before this one

    // The length of a block, from all sequences' tiles.
    int64_t total = 0;
    for (int i = lane; i < a.B; i += 32) total += visit_of(a, i).tiles;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const int worker = blockIdx.x * kWarps + warp, workers = gridDim.x * kWarps;
    const int64_t share = max(workers - static_cast<int64_t>(a.B) * a.Hkv, static_cast<int64_t>(workers) / 2);
    const int run = static_cast<int>(
        min(max((total * a.Hkv + share - 1) / share, static_cast<int64_t>(kMinRun)), static_cast<int64_t>(1) << 27));

    // Blocks of sequence from + lane, and of all up to it.
    auto blocks_of = [&](int from, int& sum) {
        const int i = from + lane, n = i < a.B ? (visit_of(a, i).tiles + run - 1) / run : 0;
        sum = inclusive_sum(n);
        return n;
    };
    if (worker == 0) {   // leaves the plan and reports lengths that are clamped
        int before = 0;
        for (int from = 0; from < a.B; from += 32) {
            const int i = from + lane;
            int sum;
            const int n = blocks_of(from, sum);
            if (i < a.B) {
                a.plan[i] = before + sum - n;
                if (a.seq_lens[i] < 0 || a.seq_lens[i] > (a.max_pages << a.page_lg)) atomicOr(a.err, kDevErrInput);
            }
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (lane == 0) a.plan[a.B] = run;
    }

    int slot = 0;             // stage of the next tile to work on,
    uint32_t phase = 0;       // and the parity its barrier completes with
    int from = 0, before = 0; // the 32 sequences last looked at, and the blocks before them
    for (int item = worker;; item += workers) {
        // The item's head, sequence and block.
        const int h = item % a.Hkv;
        int b = -1, block = 0;
        for (; from < a.B; from += 32) {
            int sum;
            const int n = blocks_of(from, sum), left = item / a.Hkv - before;
            const unsigned hit = __ballot_sync(0xffffffffu, left < sum);
            if (hit) {
                const int who = __ffs(hit) - 1;
                block = left - __shfl_sync(0xffffffffu, sum - n, who);
                b = from + who;
                break;
            }
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (b < 0) break;
        const Visit vis = visit_of(a, b);
        const int at = block * run;   // first tile of the block
        const int count = min(run, vis.tiles - at);
        // The query's head g (and 8 + g), dims 16 t .. 16 t + 15 of each 64.
        uint4 q_raw[NH][2 * KW];
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int p = 0; p < 2 * KW; ++p) {
                q_raw[n][p] = make_uint4(0, 0, 0, 0);
                if (n * 8 + g < G)
                    q_raw[n][p] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                        (static_cast<size_t>(b) * a.Hq + h * G + n * 8 + g) * D + (p / 2) * 64 + t * 16)[p % 2];
            }
        struct Keys {
            int base, from, to;   // first key of the tile; visited: [from, to)
        };
        auto keys_of = [&](int i) -> Keys {
            const int j = at + i;
            if (j < vis.ta) return {j * kTile, 0, vis.na};
            return {(vis.lo / kTile + j - vis.ta) * kTile, vis.lo, vis.len};
        };
        // Page of a token (a bad table entry: page 0).
        auto page_of = [&](int tok) -> int {
            const int p = a.block_table[static_cast<size_t>(b) * a.max_pages + (tok >> a.page_lg)];
            if (p >= 0 && p < a.num_pages) return p;
            atomicOr(a.err, kDevErrInput);
            return 0;
        };
        // WIDE: lane i holds the page of tile i (from the last multiple of 32 on),
        // looked up 32 tiles at once.  Otherwise: of key (lane & 15) of one tile, a
        // key not visited standing for one that is (its bytes are not copied).
        int pages = 0;
        // Starts the copies of tile i into stage `slot`.
        auto issue = [&](int i, int slot) {
            const Keys k = keys_of(i);
            const uint32_t dst = queue_s + slot * kStageBytes<D>;
            if constexpr (WIDE) {
                if (i % 32 == 0) pages = i + lane < count ? page_of(keys_of(i + lane).base) : 0;
                const int page = __shfl_sync(0xffffffffu, pages, i % 32);
                if (lane == 0) {
                    const int at_page = k.base & mask;
                    const size_t ex = ((static_cast<size_t>(page) * a.Hkv + h) << a.page_lg) + at_page;
                    uint64_t* bar = &s_full[warp][slot];
                    mbar_arrive_expect_tx(bar, kStageBytes<D> + 32);
                    tma_load_3d(dst, &k_map, bar, h * D, at_page, page);
                    tma_load_3d(dst + kTile * D, &v_map, bar, h * D, at_page, page);
                    bulk_load(smem_u32(s_exp[warp][slot]), a.k_exp + ex, 16, bar);
                    bulk_load(smem_u32(s_exp[warp][slot]) + 16, a.v_exp + ex, 16, bar);
                }
            } else {
                const int tok = min(max(k.base + (lane & 15), k.from), k.to - 1);
                pages = page_of(tok);
                const size_t row = (static_cast<size_t>(pages) << a.page_lg) + (tok & mask);
                constexpr int P = D / 16;   // pieces of a row
#pragma unroll
                for (int x = 0; x < P / 2; ++x) {
                    const int j = x * (32 / P) + lane / P, piece = lane % P;
                    const bool on = k.base + j >= k.from && k.base + j < k.to;
                    const size_t src = __shfl_sync(0xffffffffu, row, j) * token_bytes + h * D + piece * 16;
                    copy16(dst + piece_at<D>(j, piece), a.k_pages + src, on);
                    copy16(dst + kTile * D + piece_at<D>(j, piece), a.v_pages + src, on);
                }
                const size_t ex = ((static_cast<size_t>(pages) * a.Hkv + h) << a.page_lg) + (tok & mask);
                s_exp[warp][slot][lane] = (lane < 16 ? a.k_exp : a.v_exp)[ex];
            }
        };

        // The first tiles, from stage `slot` on.
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            if (i < count) issue(i, slot + i < kStages ? slot + i : slot + i - kStages);
            if (!WIDE) asm volatile("cp.async.commit_group;" ::: "memory");
        }

        // Query fragments and the factors of their scores, scale log2(e) 2^-qe
        // of the thread's columns, heads 2t and 2t + 1, as fa fb: a sum of
        // products (2^-33 to 2^31) times fa, then times the key row's power of
        // two, then times fb stays inside fp32 where the score is, and is off
        // by no more than 2^-23 where one of the three is subnormal.
        uint32_t qf[NH][KS][2];
        float fa[NH][2], fb[NH][2];
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            float x[KW * 16];
            float amax = 0.f;
            const __nv_bfloat162* pairs = reinterpret_cast<const __nv_bfloat162*>(q_raw[n]);
#pragma unroll
            for (int e = 0; e < KW * 8; ++e) {
                const float2 f = __bfloat1622float2(pairs[e]);
                x[2 * e] = f.x;
                x[2 * e + 1] = f.y;
                amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
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
            const int down = a.scale_e - qe;   // large: after the key's power; small: some of it, as much as scores leave room
            const int late = down < -90 ? -60 : min(max(down - 60, 0), 127);
            const float f0 = a.scale_m * __uint_as_float(static_cast<uint32_t>(max(down - late, -126) + 127) << 23);
            const float f1 = __uint_as_float(static_cast<uint32_t>(late + 127) << 23);
#pragma unroll
            for (int col = 0; col < 2; ++col) {
                fa[n][col] = __shfl_sync(0xffffffffu, f0, (2 * t + col) * 4);
                fb[n][col] = __shfl_sync(0xffffffffu, f1, (2 * t + col) * 4);
            }
        }

        float acc[NH][KS][4];
        float m[NH][2], nr[NH][2], l[NH][2];   // reference of s, that of the values' weights beyond it, and the sum
#pragma unroll
        for (int n = 0; n < NH; ++n) {
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[n][j][e] = 0.f;
            m[n][0] = m[n][1] = nr[n][0] = nr[n][1] = kLow;
            l[n][0] = l[n][1] = 0.f;
        }

        for (int i = 0; i < count; ++i) {
            // The next tile's copies start, in the stage that the last one left.
            const int ahead = i + kStages - 1;
            if (ahead < count) issue(ahead, slot == 0 ? kStages - 1 : slot - 1);
            if constexpr (WIDE) {
                // One lane's time-out is every lane's: the warp leaves together.  (With
                // a first try that may suspend 16 x 32K takes 57.8 us in place of 58.1,
                // but a lowered limit does not reach these waits.)
                if (!__all_sync(0xffffffffu, mbar_wait_short(&s_full[warp][slot], phase, &s_abort[warp], a.err))) {
                    for (int j = i; j < min(ahead + 1, count); ++j) {   // the copies in flight
                        mbar_drain(&s_full[warp][slot], phase);
                        if (++slot == kStages) slot = 0, phase ^= 1;
                    }
                    return;
                }
            } else {
                asm volatile("cp.async.commit_group;" ::: "memory");
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
                __syncwarp();
            }
            const uint8_t* stage = queue + slot * kStageBytes<D>;
            const Keys keys = keys_of(i);
            uint4 kw[2][KW];
            uint32_t vw[4][D / 32];
            int ku[2], vu[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = g + 8 * r;
#pragma unroll
                for (int p = 0; p < KW; ++p)
                    kw[r][p] = *reinterpret_cast<const uint4*>(stage + piece_at<D>(row, 4 * p + t));
                ku[r] = s_exp[warp][slot][row];
                vu[r] = s_exp[warp][slot][16 + row];
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {   // value rows 2t, 2t + 1, 2t + 8, 2t + 9
                const int row = 2 * t + (r & 1) + 8 * (r >> 1);
                if constexpr (D == 128) {
                    const uint4 u = *reinterpret_cast<const uint4*>(stage + kTile * D + piece_at<D>(row, g));
                    vw[r][0] = u.x, vw[r][1] = u.y, vw[r][2] = u.z, vw[r][3] = u.w;
                } else {
                    const uint2 u = *reinterpret_cast<const uint2*>(stage + kTile * D + piece_at<D>(row, g / 2) + (g & 1) * 8);
                    vw[r][0] = u.x, vw[r][1] = u.y;
                }
            }
            __syncwarp();   // every lane has read the stage
            if (++slot == kStages) slot = 0, phase ^= 1;
            if (keys.base < keys.from || keys.base + kTile > keys.to) {
                // Rows that are not visited: a weight of zero would not cancel a NaN.
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int tok = keys.base + 2 * t + (r & 1) + 8 * (r >> 1);
                    if (tok < keys.from || tok >= keys.to) {
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) vw[r][w] = 0;
                    }
                }
            }

            // Scores: rows key g and 8 + g, columns heads 2t and 2t + 1.
            // Two chains of products, to wait less on either.
            float s[NH][4], s2[NH][4];
            const uint32_t* k0 = reinterpret_cast<const uint32_t*>(kw[0]);
            const uint32_t* k1 = reinterpret_cast<const uint32_t*>(kw[1]);
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                uint32_t a0, a1, a2, a3;
                halves_of(k0[j], a0, a2);
                halves_of(k1[j], a1, a3);
#pragma unroll
                for (int n = 0; n < NH; ++n) {
                    float* chain = j & 1 ? s2[n] : s[n];
                    if (j < 2) mma_f16_first(chain, a0, a1, a2, a3, qf[n][j][0], qf[n][j][1]);
                    else mma_f16(chain, a0, a1, a2, a3, qf[n][j][0], qf[n][j][1]);
                }
            }
            // Both exponents less their references, which are raised first where one
            // is over them by more than kSlack (a NaN is not).
            float x[NH][4], y[NH][4], ve[2];
            float over = -INFINITY;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int tok = keys.base + g + 8 * r;
                const bool on = static_cast<unsigned>(tok - keys.from) < static_cast<unsigned>(keys.to - keys.from);
                const float kf = __uint_as_float(static_cast<uint32_t>(ku[r]) << 23);
                ve[r] = static_cast<float>(vu[r] - 127);
#pragma unroll
                for (int n = 0; n < NH; ++n)
#pragma unroll
                    for (int col = 0; col < 2; ++col) {
                        const int e = 2 * r + col;
                        s[n][e] = on ? (s[n][e] + s2[n][e]) * fa[n][col] * kf : -INFINITY;   // but for fb
                        x[n][e] = fmaf(s[n][e], fb[n][col], -m[n][col]);
                        y[n][e] = x[n][e] + (ve[r] - nr[n][col]);
                        over = fmaxf(over, fmaxf(x[n][e], y[n][e]));
                    }
            }
            if (__any_sync(0xffffffffu, over > kSlack)) {
#pragma unroll
                for (int n = 0; n < NH; ++n)
#pragma unroll
                    for (int col = 0; col < 2; ++col) {
                        float top = fmaxf(s[n][col], s[n][col + 2]) * fb[n][col];
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const float mn = fmaxf(m[n][col], top), fall = m[n][col] - mn;
                        x[n][col] = fmaf(s[n][col], fb[n][col], -mn);
                        x[n][col + 2] = fmaf(s[n][col + 2], fb[n][col], -mn);
                        top = fmaxf(x[n][col] + ve[0], x[n][col + 2] + ve[1]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const float nn = fmaxf(nr[n][col] + fall, top - kRoom);
                        l[n][col] *= ex2f(fall);
                        const float ca = ex2f(nr[n][col] + fall - nn);
#pragma unroll
                        for (int j = 0; j < KS; ++j) {
                            acc[n][j][col] *= ca;
                            acc[n][j][col + 2] *= ca;
                        }
                        m[n][col] = mn;
                        nr[n][col] = nn;
                        y[n][col] = x[n][col] + (ve[0] - nn);
                        y[n][col + 2] = x[n][col + 2] + (ve[1] - nn);
                    }
            }
            uint32_t wt[NH][2], wl[NH][2];   // and what rounding left
#pragma unroll
            for (int n = 0; n < NH; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    l[n][e & 1] += ex2f(x[n][e]);
                    y[n][e] = ex2f(y[n][e]);
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t hi = pack_half2(y[n][2 * r], y[n][2 * r + 1]);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                    wt[n][r] = transpose8x8(hi);
                    wl[n][r] = transpose8x8(pack_half2(y[n][2 * r] - f.x, y[n][2 * r + 1] - f.y));
                }
            }
            // O^T: tile j holds dims D/8 g + 2 j (rows g) and + 1 (rows 8 + g).
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                const uint32_t sel = (j & 1) ? 0x7362 : 0x5140;
                uint32_t a0, a1, a2, a3;
                halves_of(__byte_perm(vw[0][j / 2], vw[1][j / 2], sel), a0, a1);
                halves_of(__byte_perm(vw[2][j / 2], vw[3][j / 2], sel), a2, a3);
#pragma unroll
                for (int n = 0; n < NH; ++n) {
                    mma_f16(acc[n][j], a0, a1, a2, a3, wt[n][0], wt[n][1]);
                    mma_f16(acc[n][j], a0, a1, a2, a3, wl[n][0], wl[n][1]);
                }
            }
        }

        // The item's part.
        float* part = a.part + static_cast<size_t>(item) * G * (D + 4);
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int col = 0; col < 2; ++col) {
                float ls = l[n][col];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
                const int head = n * 8 + 2 * t + col;
                if (head < G) {
                    float* dst = part + head * (D + 4);
#pragma unroll
                    for (int j = 0; j < KS; j += 2)
                        *reinterpret_cast<float4*>(dst + g * (D / 8) + 2 * j) =
                            make_float4(acc[n][j][col], acc[n][j][col + 2], acc[n][j + 1][col], acc[n][j + 1][col + 2]);
                    if (g == 0) *reinterpret_cast<float4*>(dst + D) = make_float4(m[n][col], nr[n][col], ls, 0.f);
                }
            }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Joins the parts of one (query head, sequence), block (hq, b): groups of D/4
// threads, four dimensions a thread.  A group takes every kJoinThreads/(D/4)-th
// part, kAtOnce of them loaded together, with running maxima; the groups join
// in order.  Launched as a programmatic dependent of the split kernel: it reads
// the visit, an input, and then waits for that grid's memory.  Bound by latency,
// so small enough that 1024 blocks (64 sequences of 16 heads) run at once: 16.9
// us for that batch, 19.7 with 4 parts at once, 17.4 with 128 threads, 23.5 with
// 512; 8 sequences of 32K: 49.4, 51.3, 51.2, 49.1.
constexpr int kJoinThreads = 256;
constexpr int kAtOnce = 2;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) decode_e4m3_join_kernel(const __grid_constant__ DecodeE4m3Args a) {
    constexpr int kLanes = D / 4, kGroups = kJoinThreads / kLanes;
    __shared__ float4 s_sum[kGroups][kLanes];
    __shared__ float3 s_top[kGroups];
    const int hq = blockIdx.x, b = blockIdx.y, col = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
    const int G = a.Hq / a.Hkv, h = hq / G;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tiles = visit_of(a, b).tiles;
    uint2* o = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + (static_cast<size_t>(b) * a.Hq + hq) * D) + col;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tiles == 0) {   // an empty slot
        if (grp == 0) *o = make_uint2(0, 0);
        if (a.lse && threadIdx.x == 0) a.lse[static_cast<size_t>(b) * a.Hq + hq] = -INFINITY;
        return;
    }
    const int run = a.plan[a.B], parts = (tiles + run - 1) / run;
    const size_t step = static_cast<size_t>(a.Hkv) * G * (D + 4);   // from block to block
    const float* part = a.part + (static_cast<size_t>(a.plan[b]) * a.Hkv + h) * G * (D + 4) + (hq % G) * (D + 4);
    float m = kLow, n = kLow, l = 0.f;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c0 = grp; c0 < parts; c0 += kGroups * kAtOnce) {
        float4 st[kAtOnce], v[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int c = c0 + i * kGroups;
            st[i] = make_float4(kLow, kLow, 0.f, 0.f);
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < parts) {
                const float4* p = reinterpret_cast<const float4*>(part + c * step);
                st[i] = __ldcg(p + kLanes);
                v[i] = __ldcg(p + col);
            }
        }
        float mn = m;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) mn = fmaxf(mn, st[i].x);
        n += m - mn;   // from here on beyond the new maximum
        float nn = n;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) nn = fmaxf(nn, st[i].y + (st[i].x - mn));
        l *= ex2f(m - mn);
        const float f = ex2f(n - nn);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] *= f;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            l += st[i].z * ex2f(st[i].x - mn);
            const float w = ex2f(st[i].y + (st[i].x - mn) - nn);
            sum[0] += v[i].x * w;
            sum[1] += v[i].y * w;
            sum[2] += v[i].z * w;
            sum[3] += v[i].w * w;
        }
        m = mn;
        n = nn;
    }
    if (parts > 1) {   // else group 0 has it all
        s_sum[grp][col] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        if (col == 0) s_top[grp] = make_float3(m, n, l);
        __syncthreads();
        if (grp != 0) return;
        float mn = m;
#pragma unroll
        for (int i = 1; i < kGroups; ++i) mn = fmaxf(mn, s_top[i].x);
        n += m - mn;
        float nn = n;
#pragma unroll
        for (int i = 1; i < kGroups; ++i) nn = fmaxf(nn, s_top[i].y + (s_top[i].x - mn));
        l *= ex2f(m - mn);
        const float f = ex2f(n - nn);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] *= f;
#pragma unroll
        for (int i = 1; i < kGroups; ++i) {
            l += s_top[i].z * ex2f(s_top[i].x - mn);
            const float w = ex2f(s_top[i].y + (s_top[i].x - mn) - nn);
            const float4 v = s_sum[i][col];
            sum[0] += v.x * w;
            sum[1] += v.y * w;
            sum[2] += v.z * w;
            sum[3] += v.w * w;
        }
        m = mn;
        n = nn;
    }
    if (grp != 0) return;
    const float f = ex2f(n + kRoom);   // in [2^-126, 2^127], which 2^n is not
    const float lr = l * (1 << static_cast<int>(kRoom));
    const __nv_bfloat162 lo = __floats2bfloat162_rn(sum[0] / lr * f, sum[1] / lr * f);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(sum[2] / lr * f, sum[3] / lr * f);
    *o = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    if (a.lse && col == 0) a.lse[static_cast<size_t>(b) * a.Hq + hq] = (m + __log2f(l)) * 0.69314718055994531f;
}

template <int D, int NH, bool WIDE>
cudaError_t launch_split(const DecodeE4m3Args& a, int sms, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_dynamic_smem(decode_e4m3_split_kernel<D, NH, WIDE>, kSharedBytes<D>, done);
    if (e != cudaSuccess) return e;
    // At most what is resident at once, and what the longest visits can use.
    const int64_t visit = (static_cast<int64_t>(a.max_pages) << a.page_lg) / kTile + 1;
    const int64_t units = (visit * a.B * a.Hkv + kMinRun * kWarps - 1) / (kMinRun * kWarps);
    const int64_t most = std::min<int64_t>(static_cast<int64_t>(sms) * kBlocksPerSm<NH>, kMaxWarps / kWarps);
    CUtensorMap k_map, v_map;
    std::memset(&k_map, 0, sizeof(k_map));
    std::memset(&v_map, 0, sizeof(v_map));
    if (WIDE && (!make_tmap_pages_u8(&k_map, a.k_pages, static_cast<uint64_t>(a.Hkv) * D, 1ull << a.page_lg, a.num_pages, D, kTile) ||
                 !make_tmap_pages_u8(&v_map, a.v_pages, static_cast<uint64_t>(a.Hkv) * D, 1ull << a.page_lg, a.num_pages, D, kTile)))
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = dependent_launch(static_cast<unsigned>(units < most ? units : most), kWarps * 32, s, attr);
    cfg.dynamicSmemBytes = kSharedBytes<D>;
    e = cudaLaunchKernelEx(&cfg, decode_e4m3_split_kernel<D, NH, WIDE>, a, k_map, v_map);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <int D, int NH>
cudaError_t launch_split(const DecodeE4m3Args& a, int sms, cudaStream_t s) {
    return (1 << a.page_lg) >= kTile ? launch_split<D, NH, true>(a, sms, s) : launch_split<D, NH, false>(a, sms, s);
}

template <int D>
cudaError_t launch_d(const DecodeE4m3Args& a, int sms, cudaStream_t s) {
    prof_start(s);
    cudaError_t e = a.Hq / a.Hkv <= 8 ? launch_split<D, 1>(a, sms, s) : launch_split<D, 2>(a, sms, s);
    prof_stop(s);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = dependent_launch(dim3(a.Hq, a.B), kJoinThreads, s, attr);
    e = cudaLaunchKernelEx(&cfg, decode_e4m3_join_kernel<D>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// The parts of all items, then the plan.
DecodeE4m3Ws decode_e4m3_ws_layout(int B, int Hq, int Hkv, int d) {
    DecodeE4m3Ws L;
    const size_t parts = static_cast<size_t>(kMaxWarps) + static_cast<size_t>(B) * Hkv;
    L.plan = sizeof(float) * parts * (Hq / Hkv) * (d + 4);
    L.plan = (L.plan + 255) & ~static_cast<size_t>(255);
    L.total = (L.plan + sizeof(int) * (static_cast<size_t>(B) + 1) + 255) & ~static_cast<size_t>(255);
    return L;
}

cudaError_t decode_e4m3_set_wait_limit(uint64_t ns) { return set_wait_limit_of_unit(ns); }

cudaError_t launch_decode_e4m3(const DecodeE4m3Args& a, int d, int sms, cudaStream_t s) {
    return d == 128 ? launch_d<128>(a, sms, s) : launch_d<64>(a, sms, s);
}

}  // namespace swi

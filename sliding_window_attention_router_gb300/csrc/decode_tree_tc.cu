// The products of the tree attention on the 5th-generation tensor cores: 128 rows
// (drafted tokens times the query heads of a key head) by 128 keys at a time.
//
// Per key tile: S = Q K^T into TMEM, softmax weights P written back over S as two
// bf16 each, O += P V with P from TMEM.  What bounds it over bf16 pages is the cache's
// bytes: a tile of 128 keys is 64 KiB (d = 128), 1466 ns of an SM's share of the copy
// bandwidth, against 1536 tensor cycles (0.8 us) and about as many of the softmax,
// overlapped: S of the next tile is computed while the weights of this one are.  16
// sequences of 32K, 16 key heads of one row tile, 4.03 GB: 605 to 618 us by the box, 96
// to 98 % of the copy rate (without a pause, under the power cap, 644 to 671).  33
// ragged trees (d = 64, 408 units, 36 key tiles a CTA): 88 us, 20 %, 1.7 us a tile of
// 128 rows, which is the chain of its softmax, and not its bytes (0.7 us).
// Over e4m3 pages it is bound by instructions: 8 sequences of 32K with 4 key heads of
// 128 rows, 273 MB: 138 us (29 %); a tile's bytes would take 733 ns, its conversion and
// its softmax, on the same four schedulers, are about 2600 cycles each.
//
// The weights go in as two bf16, the nearest and what it leaves, right to 2^-17 of
// each: the products of fp32 weights to less than the result's own rounding.  With
// the first alone, 2^-9 of each, errors would be of the size of that rounding.  The
// tensor cores have the time.
//
// A tile's keys are two halves of 64, each with softmax warps, weights and an O of
// its own: neither waits for the other, and the join adds the two up as it does
// parts.  (Q with few rows held two or four times, each copy with a part of the keys,
// so that all softmax warps work on fewer: 8 x 32K, 32 rows, 137 us, without 110; the
// join of the copies and the longer code cost more than they saved.)
//
//   warps 0-7   softmax: four warps a half; thread r of them owns row r, TMEM lane r
//   warp 8      TMEM and MMA issue (converged, elected issue)
//   warp 9      Q: gathers a unit's rows
//   warps 12-15 K and V: a ring of tiles in the order in which they are used (K0,
//               K1, V0, K2, V1, ...), 32 rows of each tile a warp
//   (warps 10, 11 fill up a warpgroup, the unit that registers are moved by)
// e4m3 pages come through a ring of their own: warps 10 and 11 have K and V copied,
// warps 12-19 write them as bf16 to the ring that the products read.
// TMEM: S at [0, 128) and [128, 256), the halves' O at [256, 256 + d) and from 256 + d.

#include "swiattn.h"
#include "ptx.cuh"
#include "tree_plan.cuh"

#include <cuda_bf16.h>
#include <math.h>
#include <algorithm>
#include <atomic>
#include <cstring>

namespace swi {
namespace {

constexpr int R = kTreeTcRows, K = kTreeTcKeys;
constexpr int kWords = kMaxTree / 32;
constexpr int kLoaders = 4;   // warps that fill a slot
// 4 warpgroups, launched at 128 registers a thread, or 5 at 96: of these the two that
// do the softmax take their share, 2 * 168 + 2 * 88 = 4 * 128, 2 * 144 + 3 * 64 = 5 * 96.
template <bool E4M3>
constexpr int kThreads = E4M3 ? 640 : 512;
template <bool E4M3>
constexpr uint32_t kRegsSoftmax = E4M3 ? 144 : 168;
template <bool E4M3>
constexpr uint32_t kRegsOther = E4M3 ? 64 : 88;
constexpr int kHalf = R * 128;   // 128 rows of 64 bf16 columns, 128-byte swizzled
constexpr uint32_t kTmemCols = 512;
constexpr int kHalfKeys = K / 2;
constexpr uint32_t kColO = 256;

template <int D, bool E4M3>
struct Sizes {
    static constexpr int kTile = R * D * 2;                    // Q, and a slot of the ring
    // Q's tiles: two, so that a unit's comes while the one before is worked on, where
    // there is room (33 ragged trees, D 64: 120 us with one, 118 with two).
    static constexpr int kQ = E4M3 && D == 128 ? 1 : 2;
    static constexpr int kSlots = E4M3 ? 4 * 128 / D : 6 * 128 / D - (kQ - 1);
    static constexpr int kRaw = E4M3 ? 4 * 128 / D : 0;        // tiles as they are in the pages
    // e4m3: the first half of either ring for K, the second for V.  They are filled by
    // different warps, and a wait by parity is sound only for one that waited for every
    // use of the slot before.
    static constexpr int kOwn = kSlots / 2;
    [[maybe_unused]] static constexpr int kOwnRaw = kRaw / 2;
    static constexpr int kBars = 2 * kSlots + 2 * kQ + 2 + 4 + 3 + 1 + 2 * kRaw;
    static constexpr int kOffRing = kQ * kTile;
    static constexpr int kOffRaw = kOffRing + kSlots * kTile;
    static constexpr int kOffExp = kOffRaw + kRaw * (R * D);   // their rows' exponent bytes,
    static constexpr int kOffRead = kOffExp + kRaw * R;        // and, a bit a row, which are read
    static constexpr int kOffBar = kOffRead + kRaw * (R / 8);
    static constexpr int kOffMisc = kOffBar + kBars * 8;
    static constexpr int kBytes = kOffMisc + 80 + 1024;        // and room to align
};
static_assert(sizeof(TreeStart) + 8 <= 80, "what follows the barriers");
template <int D, bool E4M3>
constexpr bool kFits = Sizes<D, E4M3>::kBytes <= 232448;
static_assert(kFits<128, false> && kFits<64, false> && kFits<128, true> && kFits<64, true>, "shared memory budget");

template <int D, bool E4M3>
struct Ctx {
    using Z = Sizes<D, E4M3>;
    uint8_t* smem;
    uint64_t* bar;
    volatile int* abort_flag;
    const TreeStart* start;
    static constexpr int kFull = 0, kEmpty = Z::kSlots, kQFull = 2 * Z::kSlots, kQEmpty = kQFull + Z::kQ,
                         kSFull = kQEmpty + Z::kQ, kPFull = kSFull + 2, kODone = kPFull + 4, kOFull = kODone + 1,
                         kOFree = kOFull + 1, kDrain = kOFree + 1,
                         kRawFull = kDrain + 1, kRawEmpty = kRawFull + Z::kRaw;
};

// As mbar_wait_w, but that a lowered limit, which polls, reaches waits that would end
// within it: the try that suspends the warp comes only under limits that do not.
__device__ __forceinline__ bool wait_w(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
    const bool there = mbar_test_wait(bar, parity) || (g_wait_limit_ns >= kPollBelowNs && mbar_try_wait(bar, parity));
    if (__all_sync(0xffffffffu, there)) return true;
    const bool ok = mbar_wait_on(bar, parity, abort_flag, err);
    return __all_sync(0xffffffffu, ok);
}

// As tma_load_4d, by shared-memory address.
__device__ __forceinline__ void tma_load_4d_at(uint32_t smem_dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                               int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

// Four steps of 16 along K by one election: D (+)= A B with A and B in shared memory,
// `step` (a descriptor's units, bytes / 16) apart.  `accumulate` is the first step's.
__device__ __forceinline__ void umma_bf16_x4_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t step,
                                               uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 a1, a2, a3, b1, b2, b3, s;\n\t"
        "cvt.u64.u32 s, %5;\n\tadd.s64 a1, %1, s;\n\tadd.s64 b1, %2, s;\n\tadd.s64 a2, a1, s;\n\tadd.s64 b2, b1, s;\n\t"
        "add.s64 a3, a2, s;\n\tadd.s64 b3, b2, s;\n\t"
        "setp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(step)
        : "memory");
}

// The same with A in TMEM, 8 columns a step.
__device__ __forceinline__ void umma_bf16_ts_x4_w(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t step,
                                                  uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 b1, b2, b3, s;\n\t.reg .b32 a1, a2, a3;\n\t"
        "cvt.u64.u32 s, %5;\n\tadd.s64 b1, %2, s;\n\tadd.s64 b2, b1, s;\n\tadd.s64 b3, b2, s;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
        "setp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, 1;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(step)
        : "memory");
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

// The tiles of the ring in their order, one by one; the next key tile's page numbers
// are looked up while the last one's rows are copied.
struct SlotWalk {
    const TreeDecodeArgs& a;
    TreeWalk<R> walk;
    int row32;
    TreeWork w;
    int kt = 0, which = 2;   // K (0) of key tile kt or V (1) of the one before it comes next, or (2) a new unit
    Rows before, now, ahead;
    // Whether there is a next one: K (0) or V (1), its rows and their head in w.h.
    __device__ __forceinline__ bool next(int& kind, Rows& rows) {
        for (;;) {
            if (which == 2) {
                if (!walk.next(w)) return false;
                kt = w.kt0;
                which = 0;
                now = ahead = rows_of(a, w, kt, row32);
                if (kt + 1 < w.kt1) ahead = rows_of(a, w, kt + 1, row32);
            }
            if (which == 0) {
                which = 1;
                if (kt < w.kt1) {
                    kind = 0;
                    rows = now;
                    return true;
                }
            }
            const bool v = kt > w.kt0;
            kind = 1;
            rows = before;
            before = now;
            now = ahead;
            ++kt;
            which = kt > w.kt1 ? 2 : 0;
            if (kt + 1 < w.kt1) ahead = rows_of(a, w, kt + 1, row32);
            if (v) return true;
        }
    }
};

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

// All but the last `left` groups of copies have come.
__device__ __forceinline__ void copies_but(int left) {
    switch (left) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;   // fewer left than asked for
    }
}

// A warp fills its 32 rows of every slot: by TMA, which announces itself, where a
// page holds `box` of them (16 or 32) and all are read; else by copies of its own
// threads, which it announces, in their order, three slots later or when it has no
// slot to fill.
template <int D>
__device__ bool loader(const TreeDecodeArgs& a, const Ctx<D, false>& c, const CUtensorMap* maps, int box, int w32, uint32_t& g) {
    using Z = Sizes<D, false>;
    constexpr int S = Z::kSlots;
    const int lane = threadIdx.x & 31;
    const uint32_t ring = smem_u32(c.smem) + Z::kOffRing + w32 * 32 * 128;
    uint32_t first = 0;              // of the slots with copies not announced, which follow one another
    uint32_t own = 0;                // bit i: slot first + i is one of them
    auto announce = [&]() {          // slot `first`
        copies_but(__popc(own) - 1);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.bar[c.kFull + first % S]);
        own >>= 1;
        ++first;
        if (own) {
            const int skip = __ffs(own) - 1;
            own >>= skip;
            first += skip;
        }
    };
    SlotWalk slots{a, TreeWalk<R>{a, *c.start}, w32 * 32};
    Rows rows;
    for (int which; slots.next(which, rows); ++g) {
        const uint32_t slot = g % S, dst = ring + slot * Z::kTile, parity = (g / S & 1) ^ 1;
        uint64_t* empty = &c.bar[c.kEmpty + slot];
        while (own && (g - first >= 3 || !__all_sync(0xffffffffu, mbar_test_wait(empty, parity)))) announce();
        if (!wait_w(empty, parity, c.abort_flag, a.err)) return false;
        if (box && rows.read == 0xffffffffu) {
            uint64_t* full = &c.bar[c.kFull + slot];
            if (lane == 0) mbar_arrive_expect_tx(full, 32 * D * 2);
            __syncwarp();
            for (int r = 0; r < 32; r += box) {
                const int row = __shfl_sync(0xffffffffu, rows.row, r);
                if (lane == 0)
#pragma unroll
                    for (int half = 0; half < D / 64; ++half)
                        tma_load_4d_at(dst + half * kHalf + r * 128, maps + which, full, half * 64, slots.w.h, row, 0);
            }
        } else {
            copy_rows<D>(a, which ? a.v_pages : a.k_pages, rows, slots.w.h, dst);
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (!own) first = g;
            own |= 1u << (g - first);
        }
    }
    while (own) announce();
    return true;
}

// e4m3 to bf16, exact where a bf16 reaches: powers of two from 2^-133 to below 2^128.
__device__ __forceinline__ uint32_t times(uint32_t x, uint32_t y) {   // two bf16
    uint32_t z;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
    return z;
}

// 16 e4m3 bytes of a row, times `scale` (two bf16), as 16 bf16 whose every four are in
// the order 0 2 1 3 (Q's elements are laid out alike, and so come O's).  A byte's sign
// goes to a bf16's, its exponent and mantissa to the lowest bits of theirs: that is the
// value over 2^120.  Bit 11 of a half of `nan` is set where one of them is a NaN, which
// comes out as 480.
__device__ __forceinline__ void row_piece(const uint4& raw, uint32_t scale, uint32_t* x, uint32_t& nan) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = (w[i] << 8 & 0x80008000u) | (w[i] << 4 & 0x07f007f0u);
        const uint32_t hi = (w[i] & 0x80008000u) | (w[i] >> 4 & 0x07f007f0u);
        nan |= (lo + 0x00100010u) | (hi + 0x00100010u);
        x[2 * i] = times(lo, scale);
        x[2 * i + 1] = times(hi, scale);
    }
}

// For any exponent byte: over 134 its power of two takes a second factor; and NaN.
__device__ __forceinline__ void row_piece_rest(const uint4& raw, uint32_t e, uint32_t* x) {
    const uint32_t more = e > 134 ? e - 134 + 127 : 127;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 one = make_uint4(i == 0 ? raw.x : i == 1 ? raw.y : i == 2 ? raw.z : raw.w, 0, 0, 0);
        uint32_t y[8], nan = 0;
        row_piece(one, min(e + 120, 254u) * 0x00800080u, y, nan);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t both = k ? one.x >> 8 : one.x;   // bytes 0 and 2, or 1 and 3
            x[2 * i + k] = times(y[k], more * 0x00800080u) | ((both & 0x7fu) == 0x7fu ? 0x7fffu : 0u) |
                           ((both & 0x7f0000u) == 0x7f0000u ? 0x7fff0000u : 0u);
        }
    }
}

// The ring of tiles as they are in e4m3 pages: rows of D bytes, their 16-byte pieces
// swizzled as a tile copy of that width leaves them.
template <int D>
__device__ __forceinline__ int raw_piece(int row, int piece) {
    return row * D + ((D == 128 ? piece ^ (row & 7) : piece ^ ((row >> 1) & 3)) << 4);
}

// Fills it, one warp K's tiles and one V's: by TMA and bulk copies `box` rows at a time
// where a page holds 16 rows or more, else row by row.  Boxes of which no row is read
// are left as they were.
template <int D>
__device__ bool raw_loader(const TreeDecodeArgs& a, const Ctx<D, true>& c, const CUtensorMap* map, int box, int which,
                           uint32_t& filled) {
    using Z = Sizes<D, true>;
    const int lane = threadIdx.x & 31;
    const uint32_t ring = smem_u32(c.smem) + Z::kOffRaw;
    uint8_t* exps = c.smem + Z::kOffExp;
    uint32_t* read = reinterpret_cast<uint32_t*>(c.smem + Z::kOffRead);
    const uint8_t* from = which ? a.v_exp : a.k_exp;
    const int mask = (1 << a.page_lg) - 1;
    uint32_t t = 0;   // tiles filled
    TreeWalk<R> walk{a, *c.start};
    TreeWork w;
    while (walk.next(w)) {
        const int len = w.s.base + w.s.n, n = w.kt1 - w.kt0;
        // Page of a token of the tile, or -1 where it is not read.
        auto page_of = [&](int tok, bool on) {
            int p = -1;
            if (on) {
                p = a.block_table[static_cast<int64_t>(w.b) * a.max_pages + (tok >> a.page_lg)];
                if (p < 0 || p >= a.num_pages) {
                    p = 0;
                    atomicOr(a.err, kDevErrInput);
                }
            }
            return p;
        };
        auto is_read = [&](int tok) { return tok < len && (w.far || tok >= w.s.lo || tok < w.s.na); };
        // Lane i looks up the page of box i of key tile kt.
        auto box_page = [&](int kt) {
            const int tok = tile_key<K>(w.s, w.far, kt) + lane * box;
            bool on = false;   // any of its rows
            if (kt < w.kt1 && lane * box < K) on = tok < len && (w.far || tok + box > w.s.lo || tok < w.s.na);
            return page_of(min(tok, len - 1), on);
        };
        int page = box ? box_page(w.kt0) : 0;
        for (int j = 0; j < n; ++j) {
            const int ahead = box ? box_page(w.kt0 + j + 1) : 0;
            const uint32_t slot = which * Z::kOwnRaw + t % Z::kOwnRaw, dst = ring + slot * (R * D);
            const int key0 = tile_key<K>(w.s, w.far, w.kt0 + j);
            uint64_t* full = &c.bar[c.kRawFull + slot];
            if (!wait_w(&c.bar[c.kRawEmpty + slot], (t / Z::kOwnRaw & 1) ^ 1, c.abort_flag, a.err)) return false;
            uint32_t bits = 0xffffffffu;   // lane i: of rows 32 i .. 32 i + 31
            if (!(key0 + K <= len && (w.far || key0 >= w.s.lo || key0 + K <= w.s.na))) {
                for (int i = 0; i < R / 32; ++i) {
                    const uint32_t x = __ballot_sync(0xffffffffu, is_read(key0 + i * 32 + lane));
                    if (lane == i) bits = x;
                }
            }
            if (lane < R / 32) read[slot * (R / 32) + lane] = bits;
            __syncwarp();
            if (box) {
                const unsigned boxes = __ballot_sync(0xffffffffu, page >= 0);
                if (lane == 0) mbar_arrive_expect_tx(full, __popc(boxes) * box * (D + 1));
                __syncwarp();
                if (page >= 0) {
                    const int at = (key0 + lane * box) & mask;
                    tma_load_3d(dst + lane * box * D, map, full, w.h * D, at, page);
                    bulk_load(smem_u32(exps + slot * R) + lane * box, from + (((static_cast<int64_t>(page) * a.Hkv + w.h) << a.page_lg) + at), box, full);
                }
            } else {
                const uint8_t* pages = static_cast<const uint8_t*>(which ? a.v_pages : a.k_pages);
#pragma unroll 1
                for (int r = lane; r < R; r += 32) {
                    const int tok = key0 + r;
                    const int p = page_of(tok, is_read(tok));
                    if (p < 0) continue;
                    const int64_t row = ((static_cast<int64_t>(p) << a.page_lg) + (tok & mask)) * a.Hkv + w.h;
                    exps[slot * R + r] = from[((static_cast<int64_t>(p) * a.Hkv + w.h) << a.page_lg) + (tok & mask)];
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + raw_piece<D>(r, i)), "l"(pages + row * D + i * 16) : "memory");
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(full)) : "memory");
                mbar_arrive(full);
            }
            page = ahead;
            filled = ++t;
        }
    }
    return true;
}

// From that ring to the products': four warps K's tiles, four V's, 32 rows a warp.  The
// conversion is bound by the instructions that it issues (the SM's own rate, shared with
// the softmax: shifts written as products, which another pipe runs, changed nothing), so
// its addresses are constants: a lane has one row a of every eight and one of four
// pieces of half a row.  Eight lanes hold rows a and a ^ 5, whose pieces differ in
// their banks both in the pages' layout and, two for one, in the products'.
template <int D>
__device__ bool converter(const TreeDecodeArgs& a, const Ctx<D, true>& c, int which, int w32) {
    using Z = Sizes<D, true>;
    constexpr int kHalves = D / 64;
    const int lane = threadIdx.x & 31, quarter = lane & 3, row = (lane >> 3) ^ (lane & 4 ? 5 : 0);
    const uint32_t raw0 = smem_u32(c.smem) + Z::kOffRaw + raw_piece<D>(w32 * 32 + row, quarter);
    const uint32_t raw1 = smem_u32(c.smem) + Z::kOffRaw + raw_piece<D>(w32 * 32 + row, quarter + (D == 128 ? 4 : 0));
    const uint32_t to = smem_u32(c.smem) + Z::kOffRing + (w32 * 32 + row) * 128;
    const uint32_t to0 = to + ((2 * quarter ^ row) << 4), to1 = to + (((2 * quarter + 1) ^ row) << 4);
    const uint8_t* exps = c.smem + Z::kOffExp + w32 * 32 + row;
    const uint32_t* read = reinterpret_cast<const uint32_t*>(c.smem + Z::kOffRead) + w32;
    TreeWalk<R> walk{a, *c.start};
    uint32_t left = 0;   // of the unit's tiles
    for (uint32_t t = 0;; ++t, --left) {
        if (left == 0) {
            TreeWork w;
            if (!walk.next(w)) return true;
            left = w.kt1 - w.kt0;
        }
        const uint32_t slot = which * Z::kOwn + t % Z::kOwn, from = which * Z::kOwnRaw + t % Z::kOwnRaw;
        if (!wait_w(&c.bar[c.kRawFull + from], t / Z::kOwnRaw & 1, c.abort_flag, a.err)) return false;
        if (!wait_w(&c.bar[c.kEmpty + slot], (t / Z::kOwn & 1) ^ 1, c.abort_flag, a.err)) return false;
        const uint32_t bits = read[from * (R / 32)], in = from * (R * D), out = slot * Z::kTile;
        uint32_t nan = 0, large = 0;
#pragma unroll 1
        for (int i = 0; i < 2 * kHalves; ++i) {   // two rows, eight apart: loads first
            const uint32_t from_row = in + (i & 1) * (16 * D), to_row = out + (i >> 1) * kHalf + (i & 1) * 2048;
            uint4 x4[2];
            uint32_t e[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                x4[k] = ld_shared_v4((i >> 1 ? raw1 : raw0) + from_row + k * (8 * D));
                e[k] = exps[from * R + (i & 1) * 16 + k * 8];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                large = max(large, e[k]);
                uint32_t x[8];
                row_piece(x4[k], (e[k] + 120) * 0x00800080u, x, nan);   // 2^(e - 127 + 120)
                st_shared_v4(to0 + to_row + k * 1024, x[0], x[1], x[2], x[3]);
                st_shared_v4(to1 + to_row + k * 1024, x[4], x[5], x[6], x[7]);
            }
        }
        if (bits != 0xffffffffu || large > 134 || (nan & 0x08000800u)) {
            // Once more, with what that leaves out.
#pragma unroll 1
            for (int i = 0; i < 4 * kHalves; ++i) {
                const int half = i >> 2, at = i & 3;
                const bool on = bits >> (row + at * 8) & 1;
                uint4 bytes = ld_shared_v4((half ? raw1 : raw0) + in + at * (8 * D));
                if (!on) bytes = make_uint4(0, 0, 0, 0);
                uint32_t x[8];
                row_piece_rest(bytes, on ? exps[from * R + at * 8] : 127u, x);
                st_shared_v4(to0 + out + half * kHalf + at * 1024, x[0], x[1], x[2], x[3]);
                st_shared_v4(to1 + out + half * kHalf + at * 1024, x[4], x[5], x[6], x[7]);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&c.bar[c.kFull + slot]);
            mbar_arrive(&c.bar[c.kRawEmpty + from]);
        }
    }
}

// Waits for a loader's last copies where any warp gave up: those whose tiles none waits for
// any more would else write to memory that is the next CTA's by then.
template <int S>
__device__ void drain(uint64_t* full, uint32_t filled) {
    for (uint32_t back = 1; back <= S && back <= filled; ++back) {
        const uint32_t g = filled - back;
        mbar_drain(&full[g % S], g / S & 1);
    }
}

// ---- Q ---------------------------------------------------------------------------------
// One warp gathers a unit's rows, kPer of them an instruction; what lies in the tile's
// others reaches no row but themselves.
template <int D, bool E4M3>
__device__ bool q_loader(const TreeDecodeArgs& a, const Ctx<D, E4M3>& c) {
    using Z = Sizes<D, E4M3>;
    constexpr int P = D / 8, kPer = 32 / P;
    const int lane = threadIdx.x & 31, piece = lane % P, G = a.Hq / a.Hkv;
    // Row i kPer + lane / P of 32: its piece's place but for what i adds and flips.
    const uint32_t col0 = smem_u32(c.smem) + (piece >> 3) * kHalf + lane / P * 128, swizzle = ((piece & 7) ^ (lane / P)) << 4;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + piece * 8;
    TreeWalk<R> walk{a, *c.start};
    TreeWork w;
    for (uint32_t u = 0; walk.next(w); ++u) {
        const uint32_t buf = u % Z::kQ, col = col0 + buf * Z::kTile;
        int at[R / 32];   // the lane's rows of q
#pragma unroll
        for (int k = 0; k < R / 32; ++k) {
            const int in = k * 32 + lane, mine = w.row0 + in;
            at[k] = in < w.rows ? (w.s.first + a.plan.order[w.s.first + mine / G]) * a.Hq + w.h * G + mine % G : 0;
        }
        if (!wait_w(&c.bar[c.kQEmpty + buf], (u / Z::kQ & 1) ^ 1, c.abort_flag, a.err)) return false;
#pragma unroll
        for (int k = 0; k < R / 32; ++k) {
            if (k * 32 >= w.rows) break;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int row = __shfl_sync(0xffffffffu, at[k], i * kPer + lane / P);
                const uint32_t to = col + (k * 32 + i * kPer) * 128 + (swizzle ^ ((i * kPer & 7) << 4));
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(q + static_cast<int64_t>(row) * D) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        if (E4M3) {   // every four elements in the order that the pages' come in; each lane its own copies
#pragma unroll 4
            for (int i = 0; i < R / kPer; ++i) {
                if (i * kPer >= w.rows) break;
                const uint32_t at = col + i * kPer * 128 + (swizzle ^ ((i * kPer & 7) << 4));
                const uint4 x = ld_shared_v4(at);
                st_shared_v4(at, __byte_perm(x.x, x.y, 0x5410), __byte_perm(x.x, x.y, 0x7632), __byte_perm(x.z, x.w, 0x5410),
                             __byte_perm(x.z, x.w, 0x7632));
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.bar[c.kQFull + buf]);
    }
    return true;
}

// ---- MMA -----------------------------------------------------------------------------------
// Step j of a unit: S of tile j, then, its weights being there, O += P V of tile j - 1.
// A tile's S buffer is written again two tiles on, by this thread after the PV that
// read it.
template <int D, bool E4M3>
__device__ bool mma_issuer(const TreeDecodeArgs& a, const Ctx<D, E4M3>& c, uint32_t tmem) {
    using Z = Sizes<D, E4M3>;
    constexpr int S = Z::kSlots;
    constexpr uint32_t kIdescS = idesc_bf16_f32(R, K, false, false), kIdescO = idesc_bf16_f32(R, D, false, true);
    const uint64_t q0 = sdesc_sw128(smem_u32(c.smem), 16, 1024);
    const uint64_t k0 = sdesc_sw128(smem_u32(c.smem) + Z::kOffRing, 16, 1024);
    const uint64_t v0 = sdesc_sw128(smem_u32(c.smem) + Z::kOffRing, kHalf, 1024);
    uint32_t g = 0, tiles = 0, u = 0;
    // K (0) or V (1) of the CTA's t-th key tile: its slot, once it is full.
    uint32_t slot;
    auto full = [&](int which, uint32_t t) {
        slot = E4M3 ? which * Z::kOwn + t % Z::kOwn : g % S;
        return wait_w(&c.bar[c.kFull + slot], (E4M3 ? t / Z::kOwn : g / S) & 1, c.abort_flag, a.err);
    };
    TreeWalk<R> walk{a, *c.start};
    TreeWork w;
    for (; walk.next(w); ++u) {
        const int n = w.kt1 - w.kt0;
        const uint32_t buf = u % Z::kQ;
        const uint64_t q = q0 + buf * (Z::kTile >> 4);
        if (!wait_w(&c.bar[c.kQFull + buf], u / Z::kQ & 1, c.abort_flag, a.err)) return false;
        for (int j = 0; j <= n; ++j) {
            if (j < n) {
                if (!full(0, tiles)) return false;
                tc_fence_after();
                const uint64_t k = k0 + slot * (Z::kTile >> 4);
#pragma unroll
                for (int i = 0; i < D / 64; ++i)
                    umma_bf16_x4_w(tmem + (tiles & 1) * K, q + i * (kHalf >> 4), k + i * (kHalf >> 4), 2, kIdescS, i > 0 ? 1u : 0u);
                umma_commit_w(&c.bar[c.kSFull + (tiles & 1)]);
                umma_commit_w(&c.bar[c.kEmpty + slot]);
                if (j == n - 1) umma_commit_w(&c.bar[c.kQEmpty + buf]);
                ++g;
                ++tiles;
            }
            if (j > 0) {
                const uint32_t t = tiles - (j < n ? 2 : 1);   // tile j - 1
                if (j == 1 && !wait_w(&c.bar[c.kOFree], (u & 1) ^ 1, c.abort_flag, a.err)) return false;
                if (!full(1, t)) return false;
                const uint64_t v = v0 + slot * (Z::kTile >> 4);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!wait_w(&c.bar[c.kPFull + (t & 1) * 2 + half], t >> 1 & 1, c.abort_flag, a.err)) return false;
                    tc_fence_after();
                    static_assert(kHalfKeys == 64, "four steps");
#pragma unroll
                    for (int i = 0; i < 2; ++i)   // the nearest bf16, then what they leave
                        umma_bf16_ts_x4_w(tmem + kColO + half * D, tmem + (t & 1) * K + half * kHalfKeys + i * 32,
                                          v + (half * kHalfKeys * 128 >> 4), 16 * 128 >> 4, kIdescO, j == 1 && i == 0 ? 0u : 1u);
                }
                umma_commit_w(&c.bar[c.kEmpty + slot]);
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

// Which of a half tile's keys, from key0 on, the row reads, a bit a key; whether any
// row of the warp leaves one out.
struct Reads {
    uint32_t bits[kHalfKeys / 32];
    bool some;
};
__device__ __forceinline__ Reads reads_of(const RowOf& row, int key0) {
    Reads x;
    x.bits[0] = x.bits[1] = 0xffffffffu;
    const bool full = !row.on || (key0 + kHalfKeys <= row.base && (key0 >= row.lo || key0 + kHalfKeys <= row.anchors));
    x.some = !__all_sync(0xffffffffu, full);
    if (x.some) {
        const int at = key0 - row.base, word = at >> 5;   // the tree's tokens at ...
        uint32_t w[3] = {0, 0, 0};
        if (row.on && at > -kHalfKeys && at < row.n) {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (word + i >= 0 && word + i < kWords) w[i] = row.mask[word + i];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k0 = key0 + 32 * i;
            x.bits[i] = bits_of(k0, row.lo, row.base) | bits_of(k0, 0, row.anchors) | __funnelshift_r(w[i], w[i + 1], at & 31);
        }
    }
    return x;
}

// Weights of a half tile whose scores are in TMEM at ts, written over them: the nearest
// bf16 of every two keys to a column, then what they leave.  Returns the factor that
// the sums so far have to be scaled by.
__device__ __forceinline__ float weigh(RowOf& row, const Reads& reads, uint32_t ts, float sl) {
    constexpr int N = kHalfKeys;
    uint32_t sr[N];
    tmem_ld32(ts, sr);
    tmem_ld32(ts + 32, sr + 32);
    tmem_ld_wait();
    float* s = reinterpret_cast<float*>(sr);
    if (reads.some) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = reads.bits[i / 32] >> (i % 32) & 1 ? s[i] : -INFINITY;
    }
    float m4[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) m4[t] = fmaxf(s[t], s[4 + t]);
#pragma unroll
    for (int i = 8; i < N; i += 8)
#pragma unroll
        for (int t = 0; t < 4; ++t) m4[t] = fmax3(m4[t], s[i + t], s[i + 4 + t]);
    const float mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
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
#pragma unroll
    for (int at = 0; at < N; at += 32) {
        uint32_t hi[16], rest[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 x = ffma2(make_float2(s[at + 2 * i], s[at + 2 * i + 1]), sl2, off);
            const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            sum[i & 3] = fadd2(sum[i & 3], p);
            hi[i] = pack_bf16x2(p.x, p.y);
            rest[i] = pack_bf16x2(p.x - __uint_as_float(hi[i] << 16), p.y - __uint_as_float(hi[i] & 0xffff0000u));
        }
        tmem_st16(ts + at / 2, hi);
        tmem_st16(ts + N / 2 + at / 2, rest);
    }
    const float2 s2 = fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3]));
    const bool had = row.l > 0.f;
    row.l = row.l * f + (s2.x + s2.y);
    return had ? f : 1.f;
}

template <int D, bool E4M3>
__device__ bool softmax(const TreeDecodeArgs& a, const Ctx<D, E4M3>& c, uint32_t tmem, int half, int warp) {
    const int lane = threadIdx.x & 31, r = warp * 32 + lane, G = a.Hq / a.Hkv;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const uint32_t to = lanes + kColO + half * D;
    uint32_t tiles = 0, done = 0;
    TreeWalk<R> walk{a, *c.start};
    TreeWork w, next;
    // The place of this thread's row of a unit among the packed tokens, -1: none.
    auto token_of = [&](const TreeWork& w) { return r < w.rows ? w.s.first + a.plan.order[w.s.first + (w.row0 + r) / G] : -1; };
    bool more = walk.next(next);
    int next_tok = more ? token_of(next) : -1;
    for (uint32_t u = 0; more; ++u) {
        w = next;
        const int tok = next_tok;
        const bool any = warp * 32 < w.rows;   // the warp has rows
        RowOf row{nullptr, 0, w.s.base, min(a.n_anchor, w.s.base), w.s.n, tok >= 0, -INFINITY, 0.f};
        if (row.on) {
            row.lo = a.plan.lo[tok];
            row.mask = a.plan.mask + static_cast<size_t>(tok) * kWords;
        }
        for (int kt = w.kt0; kt < w.kt1; ++kt, ++tiles) {
            const int key0 = tile_key<K>(w.s, w.far, kt) + half * kHalfKeys;
            const Reads reads = reads_of(row, key0);   // while the scores are on their way
            if (!wait_w(&c.bar[c.kSFull + (tiles & 1)], tiles >> 1 & 1, c.abort_flag, a.err)) return false;
            tc_fence_after();
            if (any) {
                const uint32_t ts = lanes + (tiles & 1) * K + half * kHalfKeys;
                const float f = weigh(row, reads, ts, a.scale_log2);
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
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.bar[c.kPFull + (tiles & 1) * 2 + half]);
        }
        // The next unit, looked up while the last product runs.
        more = walk.next(next);
        next_tok = more ? token_of(next) : -1;
        if (!wait_w(&c.bar[c.kOFull], u & 1, c.abort_flag, a.err)) return false;
        tc_fence_after();
        if (any) {
            // Parts lie four dimensions of all rows together: lanes write side by side
            // (row by row, 128 rows took 8 to 10 thousand cycles).
            float* part = a.plan.part + static_cast<size_t>(w.slot) * kPartRows<R> * (D + 2);
            const int at = half * R + r;
#pragma unroll
            for (int i = 0; i < D; i += 32) {
                uint32_t o[32];
                tmem_ld32(to + i, o);
                tmem_ld_wait();
                if (row.on)
#pragma unroll
                    for (int t = 0; t < 32; t += 4)
                        reinterpret_cast<uint4*>(part)[(i + t) / 4 * kPartRows<R> + at] =
                            E4M3 ? make_uint4(o[t], o[t + 2], o[t + 1], o[t + 3]) : make_uint4(o[t], o[t + 1], o[t + 2], o[t + 3]);
            }
            if (row.on) reinterpret_cast<float2*>(part + kPartRows<R> * D)[at] = make_float2(row.m, row.l);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.bar[c.kOFree]);
    }
    return true;
}

struct TreeMaps {
    CUtensorMap of[2];   // K's pages, V's
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads<E4M3>, 1) tree_tc_kernel(const __grid_constant__ TreeDecodeArgs a, const __grid_constant__ TreeMaps maps, int box) {
    extern __shared__ uint8_t raw[];
    using Z = Sizes<D, E4M3>;
    Ctx<D, E4M3> c;
    c.smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
    c.bar = reinterpret_cast<uint64_t*>(c.smem + Z::kOffBar);
    TreeStart* start = reinterpret_cast<TreeStart*>(c.smem + Z::kOffMisc);
    c.start = start;
    c.abort_flag = reinterpret_cast<volatile int*>(c.smem + Z::kOffMisc + sizeof(TreeStart));
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(c.smem + Z::kOffMisc + sizeof(TreeStart) + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < Z::kSlots; ++i) {
            mbar_init(&c.bar[c.kFull + i], kLoaders);
            mbar_init(&c.bar[c.kEmpty + i], 1);
        }
        for (int i = 0; i < 2 * Z::kQ; ++i) mbar_init(&c.bar[c.kQFull + i], 1);   // and kQEmpty
        for (int i = 0; i < 2; ++i) mbar_init(&c.bar[c.kSFull + i], 1);
        for (int i = 0; i < 4; ++i) mbar_init(&c.bar[c.kPFull + i], 4);   // warps
        mbar_init(&c.bar[c.kODone], 1);
        mbar_init(&c.bar[c.kOFull], 1);
        mbar_init(&c.bar[c.kOFree], 8);
        mbar_init(&c.bar[c.kDrain], 1);
        for (int i = 0; i < Z::kRaw; ++i) {
            mbar_init(&c.bar[c.kRawFull + i], box ? 1 : 64);
            mbar_init(&c.bar[c.kRawEmpty + i], kLoaders);
        }
        *c.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 8) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");   // for the plan
    if (warp == 0) {
        const TreeStart begin = start_walk<R>(a);
        if (lane == 0) *start = begin;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    uint32_t filled = 0;   // by a loader
    if (warp < 8) {
        warpgroup_reg_inc<kRegsSoftmax<E4M3>>();
        softmax<D, E4M3>(a, c, tmem, warp >> 2, warp & 3);
    } else {
        warpgroup_reg_dec<kRegsOther<E4M3>>();
        if (warp == 8) {
            mma_issuer<D, E4M3>(a, c, tmem);
            umma_commit_w(&c.bar[c.kDrain]);   // all that was issued
            mbar_drain(&c.bar[c.kDrain], 0);
        } else if (warp == 9) {
            q_loader<D, E4M3>(a, c);
        } else if (warp >= 12) {
            if constexpr (E4M3) {
                converter<D>(a, c, (warp - 12) / kLoaders, (warp - 12) % kLoaders);
            } else {
                loader<D>(a, c, maps.of, box, warp - 12, filled);
            }
        } else if constexpr (E4M3) {
            raw_loader<D>(a, c, &maps.of[warp - 10], box, warp - 10, filled);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    } else if (*c.abort_flag && filled) {   // all have left their roles: it does not change any more
        // (Behind each loader, aborted or not, e4m3 8 x 32K took 139.7 us, here 137.9.)
        if constexpr (E4M3) drain<Z::kOwnRaw>(&c.bar[c.kRawFull + (warp - 10) * Z::kOwnRaw], filled);
        else drain<Z::kSlots>(&c.bar[c.kFull], filled);
    }
}

template <int D, bool E4M3>
cudaError_t launch(const TreeDecodeArgs& a, int ctas, cudaStream_t s) {
    using Z = Sizes<D, E4M3>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_dynamic_smem(tree_tc_kernel<D, E4M3>, Z::kBytes, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = dependent_launch(ctas, kThreads<E4M3>, s, attr);
    cfg.dynamicSmemBytes = Z::kBytes;
    // Rows that a copy takes, by what pages hold; none in pages of fewer than 16, or
    // (bf16) where a row's number in the pool does not fit a coordinate.
    const int64_t rows = static_cast<int64_t>(a.num_pages) << a.page_lg;
    int box = a.page_lg < 4 || (!E4M3 && rows >= (int64_t(1) << 31)) ? 0 : std::min(1 << a.page_lg, E4M3 ? K : 32);
    TreeMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    if (box) {
        const void* pages[2] = {a.k_pages, a.v_pages};
        for (int i = 0; i < 2; ++i)
            if (!(E4M3 ? make_tmap_pages_u8(&maps.of[i], pages[i], static_cast<uint64_t>(a.Hkv) * D, 1ull << a.page_lg, a.num_pages, D, box)
                       : make_tmap_4d_bf16(&maps.of[i], pages[i], D, a.Hkv, rows, 1, 64, box)))
                return cudaErrorInvalidValue;
    }
    return cudaLaunchKernelEx(&cfg, tree_tc_kernel<D, E4M3>, a, maps, box);
}

}  // namespace

cudaError_t launch_tree_tc(const TreeDecodeArgs& a, int d, bool e4m3, int ctas, cudaStream_t s) {
    if (e4m3) return d == 128 ? launch<128, true>(a, ctas, s) : launch<64, true>(a, ctas, s);
    return d == 128 ? launch<128, false>(a, ctas, s) : launch<64, false>(a, ctas, s);
}

cudaError_t tree_set_wait_limit(uint64_t ns) { return set_wait_limit_of_unit(ns); }

}  // namespace swi

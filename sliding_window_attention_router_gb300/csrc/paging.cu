// Keeping the accepted path of a drafted tree, and forking sequences, in a paged
// cache: rows of keys and values (with their exponent bytes) moved inside the
// pools of all layers, lengths and block tables brought along.  Nothing is
// computed; the bound is the bytes moved, and for the few rows of an ordinary step
// the chain of dependent reads before them (starts and length, parents, table,
// rows), about 0.6 us each.

#include "swiattn.h"
#include "swiattn_internal.h"

#include <algorithm>

namespace swi {
namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 8;   // 16-byte loads a thread starts before it stores

// Sequence b of a call on drafted trees: its first token among the packed ones,
// its tokens n and its cached tokens before them.
struct Tree {
    int first, n, base;
    bool ok;   // and nothing to report
};
__device__ __forceinline__ Tree tree_of(const int32_t* starts, const int32_t* seq_lens, int b, int T, int capacity) {
    Tree t;
    t.first = starts[b];
    const int after = starts[b + 1], len = seq_lens[b];
    t.n = len == 0 ? 0 : after - t.first;   // an empty slot has no tokens to look at
    t.base = len - t.n;
    t.ok = len >= 0 && len <= capacity && t.first >= 0 && after >= t.first && after <= T && t.n <= kMaxTree && t.base >= 0;
    return t;
}

// ---- the accepted path ------------------------------------------------------
// The path's token i goes to slot i of the tree's, its own slot being no earlier;
// its token j > i comes from a later slot still.  So a thread that moves one
// 16-byte column of all rows in order, each batch loaded before it is stored,
// reads every row before it is overwritten, and threads share nothing.  (16 trees of
// 22 layers, 6 MB: 4.8 us, of which an empty kernel is 2.3; one tree of 8 layers 2.9.)
__global__ void __launch_bounds__(kThreads) accept_kernel(const __grid_constant__ PagingArgs a, int parts) {
    __shared__ int s_parent[kMaxTree];
    __shared__ int s_path[kMaxTree];   // from its end: the leaf in the last place
    __shared__ int64_t s_from[kMaxTree], s_to[kMaxTree];   // rows of a layer's pool, -1: not moved
    __shared__ int s_first, s_bad;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.x / parts, part = blockIdx.x % parts;
    const Tree t = tree_of(a.starts, a.seq_lens, b, a.T, a.max_pages << a.page_lg);
    int leaf = t.n == 0 ? -1 : a.leaf[b];
    const bool reports = part == 0 && threadIdx.x == 0;
    if (!t.ok || (leaf >= t.n && t.n > 0)) {   // left as it is, and reported
        if (reports) {
            a.lens_out[b] = a.seq_lens[b];
            atomicOr(a.err, kDevErrInput);
        }
        return;
    }
    if (!a.parents || leaf < 0) {   // a chain's tokens are where they belong
        if (reports) a.lens_out[b] = t.base + max(leaf, -1) + 1;
        return;
    }
    if (threadIdx.x == 0) s_bad = 0;
    for (int i = threadIdx.x; i < t.n; i += kThreads) s_parent[i] = a.parents[t.first + i];
    __syncthreads();
    if (threadIdx.x == 0) {
        int at = kMaxTree;
        while (leaf >= 0) {   // ends: a parent comes before its token
            s_path[--at] = leaf;
            int next = s_parent[leaf];
            if (next >= leaf) {
                next = -1;
                s_bad = 1;
            }
            leaf = next;
        }
        s_first = at;
    }
    __syncthreads();
    const int at = s_first, count = kMaxTree - at;
    bool bad = s_bad != 0;
    const int mask = (1 << a.page_lg) - 1;
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const int from = t.base + s_path[at + i], to = t.base + i;
        const int32_t* table = a.block_table + static_cast<int64_t>(b) * a.max_pages;
        const int p = from == to ? 0 : table[from >> a.page_lg], q = from == to ? 0 : table[to >> a.page_lg];
        const bool in = p >= 0 && p < a.num_pages && q >= 0 && q < a.num_pages;
        bad |= !in;
        s_from[i] = in && from != to ? (static_cast<int64_t>(p) << a.page_lg) + (from & mask) : -1;
        s_to[i] = (static_cast<int64_t>(q) << a.page_lg) + (to & mask);
    }
    if (part == 0 && bad) atomicOr(a.err, kDevErrInput);
    if (reports) a.lens_out[b] = t.base + count;
    // The first tokens of the path that stay where they are.
    int stay = count;
    for (int i0 = 0; i0 < count && stay == count; i0 += 32) {
        const int i = i0 + (threadIdx.x & 31);
        const unsigned off = __ballot_sync(0xffffffffu, i < count && s_path[at + i] != i);
        if (off) stay = i0 + __ffs(off) - 1;
    }
    __syncthreads();
    if (stay == count) return;

    // Columns: of 16 bytes, layer by layer, keys then values; then single
    // exponent bytes, a head each.
    const int64_t wide = static_cast<int64_t>(a.row_bytes / 16), pool = static_cast<int64_t>(a.num_pages) << a.page_lg;
    const int64_t columns = 2 * a.layers * wide, all = columns + (a.k_exp ? 2 * a.layers * a.Hkv : 0);
    for (int64_t c = static_cast<int64_t>(part) * kThreads + threadIdx.x; c < all; c += static_cast<int64_t>(parts) * kThreads) {
        if (c < columns) {
            const int64_t unit = c / wide;   // 2 layer + (0 keys, 1 values)
            char* at_row = static_cast<char*>(unit & 1 ? a.v_pages : a.k_pages) + (unit >> 1) * pool * a.row_bytes + (c - unit * wide) * 16;
            for (int i0 = stay; i0 < count; i0 += kAtOnce) {
                uint4 x[kAtOnce];
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
                    if (i0 + i < count && s_from[i0 + i] >= 0) x[i] = *reinterpret_cast<const uint4*>(at_row + s_from[i0 + i] * a.row_bytes);
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
                    if (i0 + i < count && s_from[i0 + i] >= 0) *reinterpret_cast<uint4*>(at_row + s_to[i0 + i] * a.row_bytes) = x[i];
            }
        } else {
            const int64_t e = c - columns, unit = e / a.Hkv, h = e - unit * a.Hkv;
            uint8_t* exps = (unit & 1 ? a.v_exp : a.k_exp) + (unit >> 1) * pool * a.Hkv;
            auto byte_of = [&](int64_t row) { return exps + ((((row >> a.page_lg) * a.Hkv + h) << a.page_lg) + (row & mask)); };
            for (int i = stay; i < count; ++i)
                if (s_from[i] >= 0) *byte_of(s_to[i]) = *byte_of(s_from[i]);
        }
    }
}

// ---- forks -------------------------------------------------------------------
// Blocks (c, y): child c, and of the pieces of its copies (of all layers' keys and
// values) every gridDim.y-th from y on.  Children come first in the grid, so that those
// of one source read its page while the L2 holds it; a block takes many pieces, as
// each begins with three reads that wait for one another, but not so many that a child
// with little to copy leaves the others waiting (64 children of four prompts, 22 layers,
// 317 MB: 52 us, 6.1 TB/s; a piece a block 67, blocks for 8 a SM 65, for 16, 32 and 128 57,
// 53 and 59).
__global__ void __launch_bounds__(kThreads) fork_kernel(const __grid_constant__ PagingArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x;
    const int b = a.source[c];
    int32_t* table_out = a.table_out + static_cast<int64_t>(c) * a.max_pages;
    int len = 0, to = -1;
    bool bad = false;
    if (b >= 0) {
        bad = b >= a.B;
        if (!bad) {
            len = a.seq_lens[b];
            to = a.new_page[c];
            bad = len < 0 || len > (a.max_pages << a.page_lg) || to >= a.num_pages;
        }
    }
    const int at = len >> a.page_lg, rest = len & ((1 << a.page_lg) - 1);
    int from = 0;
    if (b >= 0 && !bad && rest > 0 && to >= 0) {
        from = a.block_table[static_cast<int64_t>(b) * a.max_pages + at];
        bad = from < 0 || from >= a.num_pages;
    }
    const bool empty = b < 0 || bad;   // an empty slot, or a child that is made one and reported
    if (blockIdx.y == 0 && threadIdx.x == 0) {
        a.lens_out[c] = empty ? 0 : len;
        if (bad) atomicOr(a.err, kDevErrInput);
    }
    const int32_t* table = a.block_table + static_cast<int64_t>(empty ? 0 : b) * a.max_pages;
    for (int64_t i = static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x; i < a.max_pages; i += static_cast<int64_t>(gridDim.y) * kThreads)
        table_out[i] = empty ? 0 : i == at && to >= 0 ? to : table[i];
    if (empty || rest == 0 || to < 0) return;

    const int64_t pool = static_cast<int64_t>(a.num_pages) << a.page_lg;   // rows of a layer
    const int64_t n = static_cast<int64_t>(rest) * (a.row_bytes / 16);     // 16-byte columns of a copy
    const int64_t pieces = (n + kThreads * kAtOnce - 1) / (kThreads * kAtOnce), units = 2 * a.layers;
    const int64_t src_at = (static_cast<int64_t>(from) << a.page_lg) * a.row_bytes, dst_at = (static_cast<int64_t>(to) << a.page_lg) * a.row_bytes;
    for (int64_t p = blockIdx.y; p < units * pieces; p += gridDim.y) {
        const int64_t unit = p / pieces, i0 = (p - unit * pieces) * (kThreads * kAtOnce) + threadIdx.x;
        char* rows = static_cast<char*>(unit & 1 ? a.v_pages : a.k_pages) + (unit >> 1) * pool * a.row_bytes;
        const uint4* src = reinterpret_cast<const uint4*>(rows + src_at);
        uint4* dst = reinterpret_cast<uint4*>(rows + dst_at);
        uint4 x[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (i0 + i * kThreads < n) x[i] = src[i0 + i * kThreads];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (i0 + i * kThreads < n) __stcs(dst + i0 + i * kThreads, x[i]);
    }
    if (a.k_exp) {
        const int64_t s = (static_cast<int64_t>(from) * a.Hkv) << a.page_lg, d = (static_cast<int64_t>(to) * a.Hkv) << a.page_lg;
        const int bytes = a.Hkv << a.page_lg;
        for (int64_t unit = blockIdx.y; unit < units; unit += gridDim.y) {
            uint8_t* exps = (unit & 1 ? a.v_exp : a.k_exp) + (unit >> 1) * pool * a.Hkv;
            for (int i = threadIdx.x; i < bytes; i += kThreads)
                if ((i & ((1 << a.page_lg) - 1)) < rest) exps[d + i] = exps[s + i];
        }
    }
}

}  // namespace

cudaError_t launch_accept(const PagingArgs& a, cudaStream_t s) {
    const int64_t columns = 2ll * a.layers * (a.row_bytes / 16 + (a.k_exp ? a.Hkv : 0));
    const int64_t most = std::max<int64_t>(1, (1 << 30) / a.B);   // blocks of the grid
    const int parts = static_cast<int>(std::min<int64_t>({(columns + kThreads - 1) / kThreads, most, 4096}));
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = dependent_launch(dim3(a.B * parts), kThreads, s, attr);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, accept_kernel, a, parts);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_fork(const PagingArgs& a, int sms, cudaStream_t s) {
    // Eight times as many blocks as run at once, and no more than there can be pieces.
    const int64_t pieces = (static_cast<int64_t>(a.row_bytes / 16) << a.page_lg) / (kThreads * kAtOnce) + 1;
    const int64_t most = std::min<int64_t>(2 * a.layers * pieces, 65535);
    const int64_t y = std::max<int64_t>(1, std::min<int64_t>(most, (64 * sms + a.C - 1) / a.C));
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = dependent_launch(dim3(a.C, static_cast<unsigned>(y)), kThreads, s, attr);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fork_kernel, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace swi

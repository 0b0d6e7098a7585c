// Shared by the kernels of the paged cache: finding a row's sequence, the division of
// attention's work over the blocks of a persistent grid, and the joining of
// what several of them computed of one item.
//
// Work. A tile is up to TQ = R / G new tokens of a sequence with the G query heads
// that share a key head: R or fewer rows (token, head) of one product with the key head's keys.
// An item is a tile of one key head, a unit is KB keys of an item. The units of
// the call, sequence by sequence, tile by tile, head by head, key block by key block, form
// one line, and each block of the grid takes an equal stretch of it. What an item costs beside its
// units (its queries, its output) stands on the line as `lead` units before the first, in which nothing happens. Lengths lie
// on the device, so every block adds up the sequences' units itself. An item that a
// stretch's end cuts is computed in parts: each block leaves its rows' sums (not
// divided), maxima and totals in the workspace, and a second kernel joins them in the order of
// the blocks. Which block has which units depends on the lengths and the grid alone, so
// results repeat bit for bit, and no block waits for another.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "device_common.cuh"
#include "internal.h"
#include "tc_common.cuh"

namespace lin {

// The sequence that row n belongs to: the last b with q_start[b] <= n, or -1, with
// end = q_start[b + 1] and kv = kv_len[b]. By one warp, 32 entries a step. Nothing but the entries is
// read, whatever they hold.
__device__ __forceinline__ int find_sequence(const int* q_start, const int* kv_len, int B, int n, int& end, int& kv) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = B;
    while (hi - lo > 32) {
        const int step = (hi - lo + 31) / 32, i = lo + lane * step;
        const int c = __popc(__ballot_sync(0xffffffffu, i < hi && q_start[i] <= n));
        if (c == 0) return -1;
        lo += (c - 1) * step;
        hi = hi < lo + step ? hi : lo + step;
    }
    const bool in = lo + lane < hi;
    const int from = in ? q_start[lo + lane] : 0, to = in ? q_start[lo + lane + 1] : 0, held = in ? kv_len[lo + lane] : 0;
    const int c = __popc(__ballot_sync(0xffffffffu, in && from <= n));
    end = __shfl_sync(0xffffffffu, to, c > 0 ? c - 1 : 0);
    kv = __shfl_sync(0xffffffffu, held, c > 0 ? c - 1 : 0);
    return c == 0 ? -1 : lo + c - 1;
}

// What a block leaves of an item that starts in its stretch and ends in a later
// block's: the combining kernel's work list.
struct PagedCut {
    int row0, tokens;  // the tile's rows of q
    int h;             // key head
    int last;          // the block that ends it; 0 when the block cuts no item
};

struct PagedArgs {
    lin_kv_batch batch;
    int pages, page_size, page_shift;  // page_size = 1 << page_shift
    int Hkv, G, TQ;            // key heads, query heads of each, tokens of a tile
    int causal;
    int lead;                  // units that an item's start and end cost
    float scale_log2;          // softmax scale times log2(e)
    uint16_t* out;             // row n, head h at n * ldo + h * D
    long long ldo;
    float* lse;                // N x H, or null
    PagedCut* cuts;            // one a block
    float2* stats;             // slots x R: maximum (of the scores in base-2 units) and total
    float* sums;               // slots x R x D; block c has slot 2c for an item that it continues, 2c + 1 for one that it starts
    int* status;
};

// A sequence's new rows and what they see.
struct PagedSeq {
    int row0, n;   // rows of q
    int held;      // keys that can be read
    int pos0;      // position of the first new token
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs& a, int b) {
    const int s = a.batch.q_start[b], e = a.batch.q_start[b + 1], kv = a.batch.kv_len[b];
    PagedSeq q;
    q.row0 = min(max(s, 0), a.batch.tokens);
    q.n = max(min(e, a.batch.tokens) - q.row0, 0);
    const int room = a.batch.table_pages * a.page_size;  // at most 2^30
    q.held = min(max(kv, 0), room);
    const long long pos = (long long)kv - e + q.row0;
    q.pos0 = (int)max(min(pos, (1ll << 30) + (1ll << 29)), -(1ll << 30));
    return q;
}
// Keys that some row of tile t sees, and its units (at least one: rows that see
// nothing are written too).
__device__ __forceinline__ int tile_seen(const PagedArgs& a, const PagedSeq& q, int t) {
    const int end = min((t + 1) * a.TQ, q.n);
    return a.causal ? max(min(q.held, q.pos0 + end), 0) : q.held;
}
template <int KB>
__device__ __forceinline__ int tile_units(const PagedArgs& a, const PagedSeq& q, int t) {
    return max((tile_seen(a, q, t) + KB - 1) / KB, 1);
}

// This block's stretch [lo, hi) of the line, and where it starts: unit `off` of
// sequence b. By all THREADS threads of the block.
struct PagedStretch {
    long long lo, hi, per;
    int b;
    long long off;
};
template <int KB, int THREADS>
__device__ __forceinline__ PagedStretch paged_stretch(const PagedArgs& a) {
    static_assert(THREADS % 32 == 0, "whole warps");
    constexpr int W = THREADS / 32;
    __shared__ long long s_sum[W];
    __shared__ long long s_off;
    __shared__ int s_b;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int B = a.batch.sequences, each = (B + THREADS - 1) / THREADS;
    const int b0 = min((int)threadIdx.x * each, B), b1 = min(b0 + each, B);
    auto tiles = [&](const PagedSeq& q) { return (q.n + a.TQ - 1) / a.TQ; };
    auto some = [&](const PagedSeq& q, int t, int n, int step) {
        long long u = 0;
        for (; t < n; t += step) u += tile_units<KB>(a, q, t) + a.lead;
        return u;
    };
    long long mine = 0;
    for (int i = 0; i < each; ++i) {
        PagedSeq q = {0, 0, 0, 0};
        if (b0 + i < b1) q = paged_seq(a, b0 + i);
        const int n = tiles(q);
        if (n <= 4) mine += some(q, 0, n, 1);
        // a long prompt's tiles by the whole warp
        for (unsigned many = __ballot_sync(0xffffffffu, n > 4); many; many &= many - 1) {
            const int from = __ffs(many) - 1;
            PagedSeq o;
            o.row0 = 0;
            o.n = __shfl_sync(0xffffffffu, q.n, from);
            o.held = __shfl_sync(0xffffffffu, q.held, from);
            o.pos0 = __shfl_sync(0xffffffffu, q.pos0, from);
            long long u = some(o, lane, __shfl_sync(0xffffffffu, n, from), 32);
#pragma unroll
            for (int d = 16; d > 0; d /= 2) u += __shfl_xor_sync(0xffffffffu, u, d);
            if (lane == from) mine += u;
        }
    }
    mine *= a.Hkv;
    long long upto = mine;  // inclusive over the threads
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < W; ++w) {
        if (w < warp) upto += s_sum[w];
        total += s_sum[w];
    }
    PagedStretch r;
    r.per = (total + gridDim.x - 1) / gridDim.x;
    r.lo = min((long long)blockIdx.x * r.per, total);
    r.hi = min(r.lo + r.per, total);
    long long at = upto - mine;
    if (r.lo < r.hi && at <= r.lo && r.lo < upto) {
        int b = b0;
        for (; b + 1 < b1; ++b) {
            const PagedSeq q = paged_seq(a, b);
            const long long u = some(q, 0, tiles(q), 1) * a.Hkv;
            if (at + u > r.lo) break;
            at += u;
        }
        s_b = b;
        s_off = r.lo - at;
    }
    __syncthreads();
    r.b = s_b;
    r.off = s_off;
    return r;
}

// Walks a stretch item by item; by a whole warp. After start(), and after next(), part()
// says whether there is another part of an item in the stretch, and which.
template <int KB>
struct PagedWalk {
    PagedSeq q;
    int b, t, h, n;   // sequence, tile, key head, units of the item
    long long u, hi;  // place on the line, end of the stretch
    int j;            // place in the item: `lead` units, then n
    int lead;
    __device__ __forceinline__ void start(const PagedArgs& a, const PagedStretch& r) {
        const int lane = threadIdx.x & 31;
        u = r.lo;
        hi = r.hi;
        lead = a.lead;
        b = r.b;
        t = h = j = n = 0;
        if (u >= hi) return;
        q = paged_seq(a, b);
        long long off = r.off;
        for (int t0 = 0; t0 * a.TQ < q.n; t0 += 32) {
            const bool some = (t0 + lane) * a.TQ < q.n;
            const long long mine = some ? (long long)(tile_units<KB>(a, q, t0 + lane) + lead) * a.Hkv : 0;
            long long upto = mine;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const long long v = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += v;
            }
            const unsigned in = __ballot_sync(0xffffffffu, off < upto);
            if (in) {
                const int at = __ffs(in) - 1;
                t = t0 + at;
                off -= __shfl_sync(0xffffffffu, upto - mine, at);
                break;
            }
            off -= __shfl_sync(0xffffffffu, upto, 31);
        }
        n = tile_units<KB>(a, q, t);
        h = (int)(off / (n + lead));
        j = (int)(off - (long long)h * (n + lead));
    }
    // The next part: units j0 .. j0 + k - 1 of the item.
    __device__ __forceinline__ bool part(const PagedArgs& a, int& j0, int& k) {
        while (u < hi) {
            if (j < lead) {
                const int skip = (int)min((long long)(lead - j), hi - u);
                u += skip;
                j += skip;
                continue;
            }
            j0 = j - lead;
            k = (int)min((long long)(n - j0), hi - u);
            return true;
        }
        return false;
    }
    // Past the part.
    __device__ __forceinline__ void next(const PagedArgs& a, int k) {
        u += k;
        j = 0;
        if (u >= hi || ++h < a.Hkv) return;
        h = 0;
        if ((++t) * a.TQ >= q.n) {
            t = 0;
            do {
                q = paged_seq(a, ++b);
            } while (q.n == 0 && b + 1 < a.batch.sequences);
        }
        n = tile_units<KB>(a, q, t);
    }
    // What the block that starts the item and does not end it notes of it.
    __device__ __forceinline__ int last_block(long long per) const { return (int)((u + n - 1) / per); }
};

// A row's result: sums over its maximum's scale divided by the total; a row that saw
// no key (total 0) is zero, with lse -inf.
__device__ __forceinline__ float row_lse(float m, float l) {
    return l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
}

// The workspace of a grid of C blocks whose tiles have R rows.
inline size_t paged_workspace(int C, int R, int D) {
    return align_up(sizeof(PagedCut) * (size_t)C, 256) + (size_t)C * 2 * R * (sizeof(float2) + (size_t)D * sizeof(float));
}

// A box of the key block at key0: KEYS keys in boxes of a page each (or all of them, when a page
// holds more). Lane `at` of the first KEYS >> shift lanes, and those as far apart again, has box `at`.
template <int KEYS>
struct PagedBox {
    int shift;       // keys of a box: 1 << shift
    int at, group;   // this lane's box, and its group of lanes
    __device__ __forceinline__ explicit PagedBox(const PagedArgs& a) {
        constexpr int top = KEYS == 128 ? 7 : 6;
        const int lane = threadIdx.x & 31;
        shift = min(a.page_shift, top);
        at = lane & ((KEYS >> shift) - 1);
        group = lane >> (top - shift);
    }
    // The table's entry for this lane's box, 0 when no key of the box is seen. Not looked at here: it
    // is asked for a block ahead, and the first use of a load waits for it.
    __device__ __forceinline__ int entry(const PagedArgs& a, const int* table, int key0, int seen) const {
        const int key = key0 + (at << shift);
        return key < seen ? table[key >> a.page_shift] : 0;
    }
    // Its page: `pages` (outside the map: zeros) where the table names none.
    __device__ __forceinline__ static int page(const PagedArgs& a, int entry) {
        return entry < 0 || entry > a.pages ? a.pages : entry;
    }
    __device__ __forceinline__ bool holds(int key0, int seen) const { return key0 + (at << shift) < seen; }
    __device__ __forceinline__ int slot(const PagedArgs& a, int key0) const {
        return (key0 + (at << shift)) & (a.page_size - 1);
    }
    __device__ __forceinline__ int count(int key0, int seen) const {
        return (min(max(seen - key0, 0), KEYS) + (1 << shift) - 1) >> shift;
    }
};

// Host side (paged_rows.cu). Maps of the pages of `base` (box: 64 elements x a page's tokens,
// at most `keys`) and of q (box: 64 elements x the heads of a key head x `tokens`), 128-byte
// swizzle, what lies outside reads as zeros; and the kernels' arguments for a grid whose tiles have
// R rows (false: the workspace is too small).
bool paged_kv_map(CUtensorMap* map, const PagedProblem& p, const void* base, int keys);
bool paged_q_map(CUtensorMap* map, const PagedProblem& p, int tokens);
bool paged_args(const PagedProblem& p, int grid, int R, PagedArgs* a);
// The joining kernel, behind an attention kernel of `grid` blocks (paged_join.cu).
int launch_paged_join(const PagedProblem& p, const PagedArgs& a, int grid, int R);

// 4-D TMA load of a box at (element, slot, head, page), 3-D at (element, head, row).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

}  // namespace lin

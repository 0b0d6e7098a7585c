// Joins the parts of the items that the ends of the blocks' stretches cut (paged.cuh):
//   m = max_i m_i,  w_i = 2^(m_i - m),  out = sum_i w_i O_i / sum_i w_i l_i
// for each row, in an order that the parts' number fixes. Blocks (c, y) take the item that block c of the
// attention kernel started and did not end, if there is one. A thread has four columns of a row; with
// few parts (nearly always two) the block's threads have different rows, with many (a long context
// on few heads is cut into as many parts as there are blocks) they share a row's parts.
// Bound by latency: the parts lie in the L2, and everything that a thread reads is asked
// for at once, past the L1 (not by loads of constant data: this kernel may have started before the
// attention kernel wrote the parts). (A warp per row with a loop over the parts took 19 us behind the 69 of
// 4 x 512 tokens over 8704 keys, 12 heads of 64.)
#include <math.h>

#include "paged.cuh"

namespace lin {
namespace {

constexpr int kPjThreads = 256;
constexpr int kPjFew = 4, kPjMany = 6;  // parts that a thread asks for at once

template <int D>
__global__ void __launch_bounds__(kPjThreads, 4) paged_join_kernel(const PagedArgs a, int R) {
    constexpr int LANES = D / 4, SLOTS = kPjThreads / LANES;
    __shared__ float4 s_acc[SLOTS][LANES];
    __shared__ float2 s_stat[SLOTS];
    pdl_wait();
    pdl_launch_dependents();
    const int c = blockIdx.x;
    const PagedCut cut = a.cuts[c];
    if (cut.last <= c) return;
    const int col = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    const int parts = cut.last - c + 1, rows = cut.tokens * a.G;
    // part i of the item: block c started it, the others continue it
    auto at = [&](int i) { return (size_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * R; };
    auto store = [&](int row, float m, float total, float4 v) {
        const int tok = row / a.G, head = cut.h * a.G + row - tok * a.G;
        const float inv = 1.f / total;
        const bool none = total == 0.f;  // a row without keys is 0
        *reinterpret_cast<uint2*>(a.out + (size_t)(cut.row0 + tok) * a.ldo + (size_t)head * D + 4 * col) =
            make_uint2(none ? 0u : pack_bf16x2(v.x * inv, v.y * inv), none ? 0u : pack_bf16x2(v.z * inv, v.w * inv));
        if (a.lse && col == 0) a.lse[(size_t)(cut.row0 + tok) * (a.Hkv * a.G) + head] = row_lse(m, total);
    };
    auto add = [](float4& v, const float4& x, float w) {
        v.x = fmaf(x.x, w, v.x);
        v.y = fmaf(x.y, w, v.y);
        v.z = fmaf(x.z, w, v.z);
        v.w = fmaf(x.w, w, v.w);
    };
    const float4* sums = reinterpret_cast<const float4*>(a.sums) + col;
    if (parts <= kPjFew) {
        for (int row = blockIdx.y * SLOTS + slot; row < rows; row += gridDim.y * SLOTS) {
            float2 st[kPjFew];
            float4 x[kPjFew];
#pragma unroll
            for (int i = 0; i < kPjFew; ++i) {
                st[i] = i < parts ? __ldcg(a.stats + at(i) + row) : make_float2(-INFINITY, 0.f);
                x[i] = i < parts ? __ldcg(sums + (at(i) + row) * LANES) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float m = st[0].x, total = 0.f;
#pragma unroll
            for (int i = 1; i < kPjFew; ++i) m = fmaxf(m, st[i].x);
            const float base = m == -INFINITY ? 0.f : m;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kPjFew; ++i) {
                const float w = exp2f(st[i].x - base);
                total = fmaf(st[i].y, w, total);
                add(v, x[i], w);
            }
            store(row, m, total, v);
        }
        return;
    }
    for (int row = blockIdx.y; row < rows; row += gridDim.y) {
        float m = -INFINITY, total = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = slot; i0 < parts; i0 += SLOTS * kPjMany) {
            float2 st[kPjMany];
            float4 x[kPjMany];
            float top = m;
#pragma unroll
            for (int k = 0; k < kPjMany; ++k) {
                const int i = i0 + k * SLOTS;
                st[k] = i < parts ? __ldcg(a.stats + at(i) + row) : make_float2(-INFINITY, 0.f);
                x[k] = i < parts ? __ldcg(sums + (at(i) + row) * LANES) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int k = 0; k < kPjMany; ++k) top = fmaxf(top, st[k].x);
            const float base = top == -INFINITY ? 0.f : top, old = exp2f(m - base);
            total *= old;
            v = make_float4(v.x * old, v.y * old, v.z * old, v.w * old);
            m = top;
#pragma unroll
            for (int k = 0; k < kPjMany; ++k) {
                const float w = exp2f(st[k].x - base);
                total = fmaf(st[k].y, w, total);
                add(v, x[k], w);
            }
        }
        s_acc[slot][col] = v;
        if (col == 0) s_stat[slot] = make_float2(m, total);
        __syncthreads();
        if (slot == 0) {
            m = -INFINITY;
            total = 0.f;
            v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) m = fmaxf(m, s_stat[i].x);
            const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                const float w = exp2f(s_stat[i].x - base);
                total = fmaf(s_stat[i].y, w, total);
                add(v, s_acc[i][col], w);
            }
            store(row, m, total, v);
        }
        __syncthreads();
    }
}

}  // namespace

int launch_paged_join(const PagedProblem& p, const PagedArgs& a, int grid, int R) {
    if (grid < 2) return LIN_OK;  // one block cuts nothing
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid - 1, R > kPagedRowsMax ? 16 : 8);
    cfg.blockDim = dim3(kPjThreads);
    cfg.stream = p.stream;
    cfg.attrs = &attr;
    cfg.numAttrs = p.early_start ? 1 : 0;
    const cudaError_t e = p.cache.head_dim == 64 ? cudaLaunchKernelEx(&cfg, paged_join_kernel<64>, a, R)
                                                 : cudaLaunchKernelEx(&cfg, paged_join_kernel<128>, a, R);
    if (e != cudaSuccess) return LIN_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? LIN_OK : LIN_ERR_CUDA;
}

}  // namespace lin

// Joins the parts of the items that the ends of the blocks' stretches cut (paged.cuh):
//   m = max_i m_i,  w_i = 2^(m_i - m),  out = sum_i w_i O_i / sum_i w_i l_i
// for each row, parts in the order of the blocks. Blocks (c, y) take the item that block c of
// the attention kernel started and did not end, if there is one. With few parts a warp takes a
// row; with many (a long context on few heads is cut into as many parts as there are blocks) the
// block's eight warps share a row's parts, whose loads would otherwise stand one behind the other.
// Bound by latency: the parts lie in the L2.
#include <math.h>

#include "paged.cuh"

namespace lin {
namespace {

constexpr int kPjWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kPjWarps) paged_join_kernel(const PagedArgs a, int R) {
    constexpr int V = D / 32;  // columns of a lane
    __shared__ float s_acc[kPjWarps][D];
    __shared__ float s_total[kPjWarps];
    pdl_wait();
    pdl_launch_dependents();
    const int c = blockIdx.x;
    const PagedCut cut = a.cuts[c];
    if (cut.last <= c) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = cut.last - c + 1, rows = cut.tokens * a.G;
    const bool share = parts > kPjWarps;
    const int first = share ? warp : 0, step = share ? kPjWarps : 1;      // this warp's parts
    auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * R; };
    const int r0 = share ? blockIdx.y : blockIdx.y * kPjWarps + warp, rstep = gridDim.y * (share ? 1 : kPjWarps);
    for (int row = r0; row < rows; row += rstep) {
        float m = -INFINITY;
        for (int i = lane; i < parts; i += 32) m = fmaxf(m, a.stats[slot(i) + row].x);
#pragma unroll
        for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float base = m == -INFINITY ? 0.f : m;
        float acc[V] = {}, total = 0.f;
#pragma unroll 8
        for (int i = first; i < parts; i += step) {
            const float2 s = a.stats[slot(i) + row];
            const float w = exp2f(s.x - base);
            const float* src = a.sums + (slot(i) + row) * D + lane * V;
            float x[V];
            if constexpr (V == 2) {
                *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(src);
            } else {
                *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(src);
            }
            total = fmaf(s.y, w, total);
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = fmaf(x[e], w, acc[e]);
        }
        if (share) {
            __syncthreads();  // the row before has been read
#pragma unroll
            for (int e = 0; e < V; ++e) s_acc[warp][lane * V + e] = acc[e];
            if (lane == 0) s_total[warp] = total;
            __syncthreads();
            if (warp > 0) continue;
            total = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll
            for (int w = 0; w < kPjWarps; ++w) {
                total += s_total[w];
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] += s_acc[w][lane * V + e];
            }
        }
        const int tok = row / a.G, head = cut.h * a.G + row % a.G;
        const float inv = 1.f / total;
        uint32_t y[V / 2];
#pragma unroll
        for (int e = 0; e < V; e += 2)  // a row without keys is 0
            y[e / 2] = total == 0.f ? 0u : pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
        uint16_t* dst = a.out + (size_t)(cut.row0 + tok) * a.ldo + (size_t)head * D + lane * V;
        if constexpr (V == 2)
            *reinterpret_cast<uint32_t*>(dst) = y[0];
        else
            *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
        if (a.lse && lane == 0) a.lse[(size_t)(cut.row0 + tok) * (a.Hkv * a.G) + head] = row_lse(m, total);
    }
}

}  // namespace

int launch_paged_join(const PagedProblem& p, const PagedArgs& a, int grid, int R) {
    if (grid < 2) return LIN_OK;  // one block cuts nothing
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid - 1, R > 32 ? R / 8 : 4);
    cfg.blockDim = dim3(32 * kPjWarps);
    cfg.stream = p.stream;
    cfg.attrs = &attr;
    cfg.numAttrs = p.early_start ? 1 : 0;
    const cudaError_t e = p.cache.head_dim == 64 ? cudaLaunchKernelEx(&cfg, paged_join_kernel<64>, a, R)
                                                 : cudaLaunchKernelEx(&cfg, paged_join_kernel<128>, a, R);
    if (e != cudaSuccess) return LIN_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? LIN_OK : LIN_ERR_CUDA;
}

}  // namespace lin

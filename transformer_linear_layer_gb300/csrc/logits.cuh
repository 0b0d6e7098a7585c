// Shared pieces of the operators on the LM head's logits (R rows of V values,
// rows ld apart): token log probabilities and distillation.
//
// Their floor is memory's: a row is read once (and its gradient written once),
// and what is kept of it is a running maximum m and the sum
// s = sum exp((z - m) / tau) of a softmax. The differences z - m are formed
// before they are scaled, so that neither an offset common to a row nor a mask of
// the type's lowest value costs accuracy (a gradient from a given lse keeps to that
// by computing the two again where lse is too large to stand for them); maximum, sums
// and statistics are fp32.
//
// A row is cut into 16-byte units on the address grid, since rows of an odd
// vocabulary start anywhere: whole units move as one 16-byte access, the (at
// most two) units that stick out of the row element by element. A cluster of CL
// blocks takes a row: one block when there are rows enough to fill the SMs, more
// when there are few, with the partial statistics exchanged through distributed
// shared memory and joined in rank order (identical inputs give identical bits).
#pragma once

#include <limits.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "device_common.cuh"
#include "internal.h"
#include "tc_common.cuh"

namespace lin {
namespace {

constexpr int kLgMaxCluster = 8;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFarBelow = -200.f;  // 2^-200 is zero in fp32: stands in for -inf where 0 * -inf would be NaN

__device__ __forceinline__ float lg_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t lg_pack(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void lg_unpack(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t lg_add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t lg_mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t lg_fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// 16 bytes of memory (not kept in L1) or of shared memory where `read`; else r is left as it is.
__device__ __forceinline__ void lg_ldg16_if(uint4& r, bool read, const void* p) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w)
        : "l"(p), "r"((uint32_t)read)
        : "memory");
}
__device__ __forceinline__ void lg_lds16_if(uint4& r, bool read, uint32_t addr) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "@p ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w)
        : "r"(addr), "r"((uint32_t)read)
        : "memory");
}

// One row on the 16-byte address grid.
template <bool BF16>
struct Row {
    static constexpr int E = BF16 ? 8 : 4;  // elements of a unit
    static constexpr int SZ = BF16 ? 2 : 4;
    const char* a0;  // address of unit 0, at or below the row's first element
    int off;         // elements of unit 0 before the row
    int V;
    int units;
    __device__ __forceinline__ Row(const void* base, long long row, long long ld, int v) : V(v) {
        const char* p = static_cast<const char*>(base) + row * ld * SZ;
        off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) / SZ;
        a0 = p - off * SZ;
        units = (V + off + E - 1) / E;
    }
    __device__ __forceinline__ int first(int u) const { return u * E - off; }  // index of the unit's first element
    __device__ __forceinline__ bool whole(int u) const { return first(u) >= 0 && first(u) + E <= V; }
    __device__ __forceinline__ float at(int i) const {
        const char* p = a0 + (long long)(i + off) * SZ;
        if constexpr (BF16) return bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(p));
        else return *reinterpret_cast<const float*>(p);
    }
    // What stands for an element that is not there.
    static __device__ __forceinline__ uint4 nothing() {
        constexpr uint32_t x = BF16 ? 0xFF80FF80u : 0xFF800000u;  // -inf
        return make_uint4(x, x, x, x);
    }
    // Raw bits of a unit that sticks out of the row, -inf outside it.
    __device__ __noinline__ uint4 load_edge(int u) const {
        constexpr uint32_t fill = BF16 ? 0xFF80FF80u : 0xFF800000u;
        uint32_t w[4] = {fill, fill, fill, fill};
        const int i0 = first(u);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int i = i0 + j;
            if (i < 0 || i >= V) continue;
            const char* p = a0 + ((long long)u * E + j) * SZ;
            if constexpr (BF16) {
                const uint32_t h = *reinterpret_cast<const uint16_t*>(p);
                w[j >> 1] = (j & 1) ? (w[j >> 1] & 0xFFFFu) | (h << 16) : (w[j >> 1] & 0xFFFF0000u) | h;
            } else {
                w[j] = *reinterpret_cast<const uint32_t*>(p);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // The elements of a unit that lie in a row, stored one by one.
    __device__ __noinline__ void store_edge(char* p, int u, uint4 o) const {
        const uint32_t w[4] = {o.x, o.y, o.z, o.w};
        const int i0 = first(u);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            if (i0 + j < 0 || i0 + j >= V) continue;
            if constexpr (BF16)
                reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)((j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu);
            else
                reinterpret_cast<uint32_t*>(p)[j] = w[j];
        }
    }
    // Raw bits of the units u, u + stride, ... from memory; -inf past the row.
    template <int N>
    __device__ __forceinline__ void load(uint4 (&r)[N], int u, int stride) const {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            r[k] = nothing();
            lg_ldg16_if(r[k], u + k * stride < units && whole(u + k * stride), a0 + (long long)(u + k * stride) * 16);
        }
        if (u >= stride && u + N * stride <= units) return;  // no unit at the row's ends among them
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (u + k * stride < units && !whole(u + k * stride)) r[k] = load_edge(u + k * stride);
    }
};

// The fp32 values of a unit, as pairs.
template <bool BF16>
__device__ __forceinline__ void lg_values(const uint4& r, uint64_t (&v)[Row<BF16>::E / 2]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if constexpr (BF16) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = lg_pack(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
    } else {
        v[0] = lg_pack(__uint_as_float(w[0]), __uint_as_float(w[1]));
        v[1] = lg_pack(__uint_as_float(w[2]), __uint_as_float(w[3]));
    }
}

// Largest value of a unit (NaN ignored).
template <bool BF16>
__device__ __forceinline__ float lg_unit_max(const uint4& r) {
    if constexpr (BF16) {
        auto mx = [](uint32_t a, uint32_t b) {
            uint32_t d;
            asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
            return d;
        };
        const uint32_t h = mx(mx(r.x, r.y), mx(r.z, r.w));
        return fmaxf(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u));
    } else {
        return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)),
                     fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
    }
}

// Statistics of a set of logits: their maximum m, s = sum 2^((z - m) c) and, for
// the entropy, t = sum 2^((z - m) c) (z - m) c, with c = log2(e) / tau.
struct Stats {
    float m, s, t;
    uint32_t bound;  // key of the top selection's bound (token log probabilities only)
};
// A maximum of -inf (nothing visible) is replaced by 0 before it is subtracted.
__device__ __forceinline__ float lg_base(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ Stats lg_rebase(const Stats& a, float m, float c) {
    const float d = (a.m - lg_base(m)) * c;  // <= 0; -inf for an empty set
    const float f = lg_ex2(d);
    return {m, a.s * f, (a.t + a.s * fmaxf(d, kFarBelow)) * f, a.bound};
}
__device__ __forceinline__ Stats lg_join(const Stats& a, const Stats& b, float c) {
    const float m = fmaxf(a.m, b.m);
    const Stats x = lg_rebase(a, m, c), y = lg_rebase(b, m, c);
    return {m, x.s + y.s, x.t + y.t, max(x.bound, y.bound)};
}

// The sums over the first n units against one maximum. CLAMP: (z - m) c may be -inf.
template <bool BF16, bool ENTROPY, bool CLAMP, int N>
__device__ __forceinline__ void lg_sums(Stats& st, const uint4 (&r)[N], int n, float c) {
    const float nb = -lg_base(st.m);
    const uint64_t nb2 = lg_pack(nb, nb), c2 = lg_pack(c, c);
    uint64_t s2 = 0ull, t2 = 0ull;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (k >= n) break;
        uint64_t v[Row<BF16>::E / 2];
        lg_values<BF16>(r[k], v);
#pragma unroll
        for (int j = 0; j < Row<BF16>::E / 2; ++j) {
            uint64_t d = lg_mul2(lg_add2(v[j], nb2), c2);
            float d0, d1;
            lg_unpack(d, d0, d1);
            const uint64_t e = lg_pack(lg_ex2(d0), lg_ex2(d1));
            s2 = lg_add2(s2, e);
            if constexpr (ENTROPY) {
                if constexpr (CLAMP) d = lg_pack(fmaxf(d0, kFarBelow), fmaxf(d1, kFarBelow));
                t2 = lg_fma2(e, d, t2);
            }
        }
    }
    float a, b;
    lg_unpack(s2, a, b);
    st.s += a + b;
    if constexpr (ENTROPY) {
        lg_unpack(t2, a, b);
        st.t += a + b;
    }
}

// Add the first n units to the running statistics (n is the same for a warp).
// Returns their largest value.
template <bool BF16, bool ENTROPY, int N>
__device__ __forceinline__ float lg_accumulate(Stats& st, const uint4 (&r)[N], int n, float c) {
    float m = lg_unit_max<BF16>(r[0]);
#pragma unroll
    for (int k = 1; k < N; ++k) {
        if (k >= n) break;
        m = fmaxf(m, lg_unit_max<BF16>(r[k]));
    }
    if (m > st.m) st = lg_rebase(st, m, c);
    if constexpr (ENTROPY && BF16) {
        // the smallest value in pairs costs less than a clamp of every term
        uint32_t low = r[0].x;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (k >= n) break;
            const uint32_t w[4] = {r[k].x, r[k].y, r[k].z, r[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) asm("min.bf16x2 %0, %0, %1;" : "+r"(low) : "r"(w[j]));
        }
        const float least = fminf(__uint_as_float(low << 16), __uint_as_float(low & 0xFFFF0000u));
        if (__all_sync(0xffffffffu, (least - lg_base(st.m)) * c > kFarBelow)) {
            lg_sums<BF16, true, false>(st, r, n, c);
            return m;
        }
    }
    lg_sums<BF16, ENTROPY, true>(st, r, n, c);
    return m;
}

__device__ __forceinline__ Stats lg_warp_join(Stats st, float c) {
    float m = st.m;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    st = lg_rebase(st, m, c);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        st.s += __shfl_xor_sync(0xffffffffu, st.s, o);
        st.t += __shfl_xor_sync(0xffffffffu, st.t, o);
    }
    return st;
}

// A thread's share of a row's statistics, read straight from memory: the units u0,
// u0 + stride, ... in batches of N. seen(largest value) is called after every batch.
template <bool BF16, bool ENTROPY, int N, class Seen>
__device__ __forceinline__ Stats lg_stream(const Row<BF16>& row, int u0, int stride, float c, Seen seen) {
    Stats st{-INFINITY, 0.f, 0.f, 0u};
    for (int u = u0; u - (int)(threadIdx.x & 31) < row.units; u += stride * N) {
        uint4 raw[N];
        row.load(raw, u, stride);
        seen(lg_accumulate<BF16, ENTROPY>(st, raw, (row.units - (u - (int)(threadIdx.x & 31)) + stride - 1) / stride, c));
    }
    return st;
}

template <int NT>
struct LgExchange {
    Stats warp[NT / 32];
    Stats rank[kLgMaxCluster];
};

// The block's, then the cluster's statistics, in every thread. The bound is the
// least of a block's warps', and the largest of the blocks'. The cluster's
// blocks have arrived (relaxed) at its barrier once, when they started.
template <int NT, int CL>
__device__ __forceinline__ Stats lg_join_blocks(Stats st, float c, LgExchange<NT>& x, uint32_t rank) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    st = lg_warp_join(st, c);
    if (lane == 0) x.warp[warp] = st;
    __syncthreads();
    st = lg_warp_join(lane < NT / 32 ? x.warp[lane] : Stats{-INFINITY, 0.f, 0.f, 0xFFFFFFFFu}, c);
    st.bound = __reduce_min_sync(0xffffffffu, st.bound);
    if constexpr (CL > 1) {
        cluster_wait();  // the peers are running
        if (warp == 0) {
            if (lane < CL) {
                const uint32_t dst = dsmem_map(smem_u32(&x.rank[rank]), lane);
                dsmem_st_f32(dst, st.m);
                dsmem_st_f32(dst + 4, st.s);
                dsmem_st_f32(dst + 8, st.t);
                dsmem_st_f32(dst + 12, __uint_as_float(st.bound));
            }
            __syncwarp();
        }
        cluster_sync_all();
        st = x.rank[0];
#pragma unroll
        for (int k = 1; k < CL; ++k) st = lg_join(st, x.rank[k], c);
    }
    return st;
}

__device__ __forceinline__ int lg_load_id(const void* ids, bool wide, long long i) {
    if (!wide) return static_cast<const int*>(ids)[i];
    const long long v = static_cast<const long long*>(ids)[i];
    return v < 0 ? -1 : v > INT_MAX ? INT_MAX : static_cast<int>(v);
}

// Blocks per row for kernels of NT threads a block: enough to give every SM
// `per_sm` blocks when there are few rows, as long as every thread keeps a unit.
inline int lg_cluster(const LogitsProblem& p, int nt, int per_sm) {
    const long long units = ((long long)p.V * (p.bf16 ? 2 : 4) + 15) / 16;
    int cl = 1;
    while (cl < kLgMaxCluster && p.R * cl * 2 <= (long long)per_sm * p.sm_count && units >= 2ll * cl * nt) cl *= 2;
    return cl;
}

template <class... Params, class... Args>
int lg_launch(void (*kern)(Params...), long long blocks, int threads, size_t smem, int cl, const LogitsProblem& p,
              const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = p.stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cl > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cl;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (p.early_start) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) return LIN_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? LIN_OK : LIN_ERR_CUDA;
}

template <class F>
int lg_by_cluster(int cl, F f) {
    switch (cl) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 4: return f(std::integral_constant<int, 4>{});
        default: return f(std::integral_constant<int, 8>{});
    }
}

}  // namespace
}  // namespace lin

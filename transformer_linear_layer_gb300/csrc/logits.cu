// Operators on the LM head's logits (R rows of V values, rows ld apart):
//
//   token log probabilities   lse_r = log sum_j exp(z_rj / tau),
//       logprob_r = z_r,token / tau - lse_r,  H_r = - sum_j p_rj log p_rj,
//       and the `top` largest logits of a row with their log probabilities,
//       ordered by value, equal values by the lowest index;
//   distillation towards a teacher's top logits: with q = softmax(t / tau) over
//       a row's valid teacher entries and p = softmax(z / tau) over the row,
//       loss_r = tau^2 sum_i q_i (log q_i - log p_id(i)),
//       dz_rj  = g_r tau (p_rj - sum of q_i with id(i) = j).
//
// All of them are bound by memory: a row is read once (and its gradient
// written once), and what is kept of it is a running maximum m and the sum
// s = sum exp((z - m) / tau) of a softmax. The differences z - m are formed
// before they are scaled, so that an offset common to a row costs no accuracy;
// maximum, sums and statistics are fp32.
//
// Layout. A row is cut into 16-byte units on the address grid, since rows of an
// odd vocabulary start anywhere: interior units move as one 16-byte access, the
// (at most two) units that stick out of the row element by element. The units
// are dealt in turn to the threads of a cluster of CL blocks: CL = 1 when there
// are rows enough to fill the SMs, more when there are few, with the partial
// statistics exchanged through distributed shared memory in rank order
// (identical inputs give identical bits).
#include <limits.h>
#include <math.h>

#include <type_traits>

#include "device_common.cuh"
#include "internal.h"
#include "tc_common.cuh"

namespace lin {
namespace {

constexpr int kLgThreads = 256;
constexpr int kLgWarps = kLgThreads / 32;
constexpr int kLgMaxCluster = 8;
constexpr int kLgBatch = 4;       // units a thread loads before it uses the first
constexpr int kLgList = 1024;     // candidates of the top selection held in shared memory
constexpr float kLog2e = 1.4426950408889634f;
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
__device__ __forceinline__ uint4 lg_ld16(const char* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ void dsmem_st_u64(uint32_t addr, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
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
    // Raw bits of N units `stride` apart; elements outside the row (and units
    // past its end) read as -inf. The whole units' loads are issued first.
    template <int N>
    __device__ __forceinline__ void load(uint4 (&r)[N], int u, int stride) const {
        constexpr uint32_t fill = BF16 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            r[k] = make_uint4(fill, fill, fill, fill);
            const int w = u + k * stride;
            if (w < units && whole(w)) r[k] = lg_ld16(a0 + (long long)w * 16);
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int w = u + k * stride;
            if (w < units && !whole(w)) r[k] = load_edge(w);
        }
    }
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

// Statistics of a set of logits: their maximum m, s = sum 2^((z - m) c) and,
// for the entropy, t = sum 2^((z - m) c) (z - m) c, with c = log2(e) / tau.
struct Stats {
    float m, s, t;
};
// A maximum of -inf (nothing visible) is replaced by 0 before it is subtracted.
__device__ __forceinline__ float lg_base(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ Stats lg_rebase(const Stats& a, float m, float c) {
    const float d = (a.m - lg_base(m)) * c;  // <= 0; -inf for an empty set
    const float f = lg_ex2(d);
    return {m, a.s * f, (a.t + a.s * fmaxf(d, kFarBelow)) * f};
}
__device__ __forceinline__ Stats lg_join(const Stats& a, const Stats& b, float c) {
    const float m = fmaxf(a.m, b.m);
    const Stats x = lg_rebase(a, m, c), y = lg_rebase(b, m, c);
    return {m, x.s + y.s, x.t + y.t};
}

// Add N units to the running statistics: their maximum first, then the sums
// against it.
template <bool BF16, bool ENTROPY, int N>
__device__ __forceinline__ void lg_accumulate(Stats& st, const uint4 (&r)[N], float c) {
    float m = st.m;
#pragma unroll
    for (int k = 0; k < N; ++k) m = fmaxf(m, lg_unit_max<BF16>(r[k]));
    if (m > st.m) st = lg_rebase(st, m, c);
    const float nb = -lg_base(m);
    const uint64_t nb2 = lg_pack(nb, nb), c2 = lg_pack(c, c);
    uint64_t s2 = 0ull, t2 = 0ull;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        uint64_t v[Row<BF16>::E / 2];
        lg_values<BF16>(r[k], v);
#pragma unroll
        for (int j = 0; j < Row<BF16>::E / 2; ++j) {
            float d0, d1;
            lg_unpack(lg_mul2(lg_add2(v[j], nb2), c2), d0, d1);
            const uint64_t e = lg_pack(lg_ex2(d0), lg_ex2(d1));
            s2 = lg_add2(s2, e);
            if constexpr (ENTROPY) t2 = lg_fma2(e, lg_pack(fmaxf(d0, kFarBelow), fmaxf(d1, kFarBelow)), t2);
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

struct LgShared {
    Stats warp[kLgWarps];
    Stats rank[kLgMaxCluster];
};

// Statistics of the whole row in every thread of the cluster. `started` says
// that the cluster's blocks have all arrived at its start-up barrier.
template <int CL>
__device__ __forceinline__ Stats lg_row_stats(Stats st, float c, LgShared& sh, uint32_t rank) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    st = lg_warp_join(st, c);
    if (lane == 0) sh.warp[warp] = st;
    __syncthreads();
    st = lg_warp_join(lane < kLgWarps ? sh.warp[lane] : Stats{-INFINITY, 0.f, 0.f}, c);
    if constexpr (CL > 1) {
        cluster_wait();  // the peers are running
        if (warp == 0 && lane < CL) {
            const uint32_t dst = dsmem_map(smem_u32(&sh.rank[rank]), lane);
            dsmem_st_f32(dst, st.m);
            dsmem_st_f32(dst + 4, st.s);
            dsmem_st_f32(dst + 8, st.t);
        }
        __syncwarp();
        cluster_sync_all();
        st = sh.rank[0];
#pragma unroll
        for (int k = 1; k < CL; ++k) st = lg_join(st, sh.rank[k], c);
    }
    return st;
}

__device__ __forceinline__ int lg_load_id(const void* ids, bool wide, long long i) {
    if (!wide) return static_cast<const int*>(ids)[i];
    const long long v = static_cast<const long long*>(ids)[i];
    return v < 0 ? -1 : v > INT_MAX ? INT_MAX : static_cast<int>(v);
}

// ------------------------------------------------------- token log probabilities

// Whole-number order of the values: a larger value has a larger key, zeros of
// either sign are equal, NaN ranks with -inf, and 0 is below every value.
__device__ __forceinline__ uint32_t lg_key(float x) {
    if (x != x) x = -INFINITY;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float lg_key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

struct LogprobArgs {
    const void* z;
    long long ld;
    int V, top;
    const void* tokens;  // null: no tokens
    bool wide;           // 64-bit tokens
    float inv_tau;
    float* logprob;
    float* entropy;      // or null
    float* lse;          // or null
    float* top_logprob;
    int* top_ids;
};

struct TopShared {
    uint64_t list[kLgList];
    uint64_t best[kLgMaxCluster * kLogprobMaxTop];
    uint64_t warp[kLgWarps];
    int count;
};

// The `top` largest of the n unique keys in `list`, in order, to out[0..top);
// places that the keys do not fill are 0. The keys are ranked by counting.
__device__ __forceinline__ void lg_rank(const uint64_t* list, int n, int top, uint64_t* out) {
    for (int i = threadIdx.x; i < top; i += kLgThreads)
        if (i >= n) out[i] = 0;
    for (int i = threadIdx.x; i < n; i += kLgThreads) {
        const uint64_t mine = list[i];
        int above = 0;
        for (int j = 0; j < n; ++j) above += list[j] > mine;
        if (above < top && mine != 0) out[above] = mine;
    }
}

template <bool BF16, int CL>
__global__ void __launch_bounds__(kLgThreads) logprob_kernel(const LogprobArgs a) {
    __shared__ LgShared sh;
    __shared__ TopShared tp;
    if constexpr (CL > 1) cluster_arrive_relaxed();
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t rank = CL > 1 ? cluster_ctarank() : 0;
    const long long r = blockIdx.x / CL;
    const Row<BF16> row(a.z, r, a.ld, a.V);
    const float c = a.inv_tau * kLog2e;
    constexpr int stride = kLgThreads * CL;
    const int u0 = rank * kLgThreads + threadIdx.x;

    Stats st{-INFINITY, 0.f, 0.f};
    for (int u = u0; u < row.units; u += stride * kLgBatch) {
        uint4 raw[kLgBatch];
        row.load(raw, u, stride);
        lg_accumulate<BF16, true>(st, raw, c);
    }
    const float mine = st.m;
    st = lg_row_stats<CL>(st, c, sh, rank);
    const float base = lg_base(st.m), logs = logf(st.s);
    auto logprob = [&](float z) { return st.s == 0.f ? -INFINITY : (z - base) * a.inv_tau - logs; };
    if (rank == 0 && threadIdx.x == 0) {
        if (a.logprob) {
            const int tok = lg_load_id(a.tokens, a.wide, r);
            a.logprob[r] = tok < 0 ? 0.f : tok >= a.V ? NAN : logprob(row.at(tok));
        }
        if (a.entropy) a.entropy[r] = st.s == 0.f ? 0.f : logs - st.t / st.s * 0.6931471805599453f;
        if (a.lse) a.lse[r] = st.s == 0.f ? -INFINITY : base * a.inv_tau + logs;
    }
    if (a.top == 0) return;

    // A lower bound of the block's top-th largest value: the largest key (its
    // upper 16 bits, all that bf16 has) that `top` of the threads' own maxima
    // reach. Only threads whose maximum reaches it look at their units again.
    const uint32_t have = u0 < row.units ? lg_key(mine) : 0u;
    if (threadIdx.x == 0) tp.count = 0;
    uint32_t bound = 0;
#pragma unroll 1
    for (int b = 31; b >= 16; --b) {
        const uint32_t cand = bound | (1u << b);
        if (__syncthreads_count(have >= cand) >= a.top) bound = cand;
    }
    if (have != 0 && have >= bound) {
        for (int u = u0; u < row.units; u += stride) {
            uint4 raw[1];
            row.load(raw, u, stride);
            if (lg_key(lg_unit_max<BF16>(raw[0])) < bound) continue;
            uint64_t v[Row<BF16>::E / 2];
            lg_values<BF16>(raw[0], v);
#pragma unroll
            for (int j = 0; j < Row<BF16>::E; ++j) {
                float lo, hi;
                lg_unpack(v[j >> 1], lo, hi);
                const int i = row.first(u) + j;
                const uint32_t key = lg_key((j & 1) ? hi : lo);
                if (i < 0 || i >= a.V || key < bound) continue;
                const int n = atomicAdd(&tp.count, 1);
                if (n < kLgList) tp.list[n] = (uint64_t)key << 32 | (0xFFFFFFFFu - (uint32_t)i);
            }
        }
    }
    __syncthreads();
    const int n = tp.count;
    uint64_t* own = tp.best + rank * a.top;
    if (n <= kLgList) {
        lg_rank(tp.list, n, a.top, own);
    } else {
        // More equal values than the list holds (a row that is mostly one
        // value): the largest key below the one before it, `top` times.
        uint64_t last = ~0ull;
#pragma unroll 1
        for (int j = 0; j < a.top; ++j) {
            uint64_t best = 0;
            for (int u = u0; u < row.units; u += stride) {
                uint4 raw[1];
                row.load(raw, u, stride);
                uint64_t v[Row<BF16>::E / 2];
                lg_values<BF16>(raw[0], v);
#pragma unroll
                for (int e = 0; e < Row<BF16>::E; ++e) {
                    float lo, hi;
                    lg_unpack(v[e >> 1], lo, hi);
                    const int i = row.first(u) + e;
                    if (i < 0 || i >= a.V) continue;
                    const uint64_t key = (uint64_t)lg_key((e & 1) ? hi : lo) << 32 | (0xFFFFFFFFu - (uint32_t)i);
                    if (key < last && key > best) best = key;
                }
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const uint64_t x = __shfl_xor_sync(0xffffffffu, best, o);
                if (x > best) best = x;
            }
            if ((threadIdx.x & 31) == 0) tp.warp[threadIdx.x >> 5] = best;
            __syncthreads();
            best = 0;
#pragma unroll
            for (int w = 0; w < kLgWarps; ++w)
                if (tp.warp[w] > best) best = tp.warp[w];
            if (threadIdx.x == 0) own[j] = best;
            last = best;
            __syncthreads();
        }
    }
    __syncthreads();
    const uint64_t* best = own;
    if constexpr (CL > 1) {
        // the ranks' lists to rank 0, which ranks them together
        if (rank != 0)
            for (int i = threadIdx.x; i < a.top; i += kLgThreads)
                dsmem_st_u64(dsmem_map(smem_u32(own + i), 0), own[i]);
        __syncwarp();
        cluster_sync_all();
        if (rank != 0) return;
        lg_rank(tp.best, CL * a.top, a.top, tp.list);
        __syncthreads();
        best = tp.list;
    }
    for (int i = threadIdx.x; i < a.top; i += kLgThreads) {
        const uint64_t k = best[i];
        const float z = lg_key_value((uint32_t)(k >> 32));
        a.top_logprob[r * a.top + i] = logprob(z);
        a.top_ids[r * a.top + i] = (int)(0xFFFFFFFFu - (uint32_t)k);
    }
}

// ------------------------------------------------------------------ distillation

struct DistillArgs {
    const void* z;
    long long ld;
    int V, K;
    const void* ids;
    bool wide;           // 64-bit ids
    const void* teacher;
    bool teacher_bf16;
    float tau, inv_tau;
    const float* weight; // upstream gradient of a row's loss, or null (1)
    const float* lse_in; // backward alone
    float* loss;         // or null (backward alone)
    float* lse;          // or null
    void* dz;            // or null (forward alone)
    long long ldd;
};

struct TeacherShared {
    int id[kDistillMaxEntries];       // -1: no entry
    float q[kDistillMaxEntries];      // probability
    float z[kDistillMaxEntries];      // the student's logit there
    float red[kLgWarps];
    int flag[kLgWarps];
};

template <class Op>
__device__ __forceinline__ float lg_block_reduce(float v, float* red, Op op) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();  // `red` is free again
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < kLgWarps; ++w) v = op(v, red[w]);
    return v;
}

// The row's teacher entries in shared memory. Returns the sum of their
// exponentials against the largest valid logit (0: no entry carries weight)
// and, in *top, that logit. *bad: an id lies past the vocabulary.
template <bool BF16>
__device__ __forceinline__ float lg_teacher(const DistillArgs& a, long long r, const Row<BF16>& row,
                                            TeacherShared& te, float* top, bool* bad) {
    float m = -INFINITY;
    int over = 0;
    for (int i = threadIdx.x; i < a.K; i += kLgThreads) {
        const int id = lg_load_id(a.ids, a.wide, r * a.K + i);
        float t = -INFINITY, z = 0.f;
        if (id >= a.V) over = 1;
        const bool held = id >= 0 && id < a.V;
        if (held) {
            t = a.teacher_bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(a.teacher)[r * a.K + i])
                               : static_cast<const float*>(a.teacher)[r * a.K + i];
            z = row.at(id);
        }
        te.id[i] = held ? id : -1;
        te.q[i] = t;
        te.z[i] = z;
        m = fmaxf(m, t);
    }
    m = lg_block_reduce(m, te.red, [](float x, float y) { return fmaxf(x, y); });
    *bad = __syncthreads_or(over) != 0;
    *top = m;
    float sum = 0.f;
    for (int i = threadIdx.x; i < a.K; i += kLgThreads)
        if (te.id[i] >= 0)
            sum += m != -INFINITY || te.q[i] != te.q[i] ? exp2f((te.q[i] - m) * (a.inv_tau * kLog2e)) : 0.f;
    return lg_block_reduce(sum, te.red, [](float x, float y) { return x + y; });
}

// dz = coef 2^((z - base) c) for a unit's values (0 where coef is 0, whatever
// the logits are), stored; elements outside the row are left alone.
template <bool BF16>
__device__ __forceinline__ void lg_store_grad(const Row<BF16>& row, char* d0, bool vec, int u, const uint4& raw,
                                              float base, float c, float coef) {
    if (u >= row.units) return;
    uint64_t v[Row<BF16>::E / 2];
    lg_values<BF16>(raw, v);
    const uint64_t nb2 = lg_pack(-base, -base), c2 = lg_pack(c, c), k2 = lg_pack(coef, coef);
    float x[Row<BF16>::E];
#pragma unroll
    for (int j = 0; j < Row<BF16>::E / 2; ++j) {
        float d0_, d1_;
        lg_unpack(lg_mul2(lg_add2(v[j], nb2), c2), d0_, d1_);
        lg_unpack(lg_mul2(lg_pack(lg_ex2(d0_), lg_ex2(d1_)), k2), x[2 * j], x[2 * j + 1]);
    }
    if (coef == 0.f) {
#pragma unroll
        for (int j = 0; j < Row<BF16>::E; ++j) x[j] = 0.f;
    }
    uint4 o;
    if constexpr (BF16)
        o = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                       pack_bf16x2(x[6], x[7]));
    else
        o = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    char* p = d0 + (long long)u * 16;
    if (vec && row.whole(u)) {
        *reinterpret_cast<uint4*>(p) = o;
        return;
    }
    const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int j = 0; j < Row<BF16>::E; ++j) {
        const int i = row.first(u) + j;
        if (i < 0 || i >= row.V) continue;
        if constexpr (BF16)
            reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)((j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu);
        else
            reinterpret_cast<uint32_t*>(p)[j] = w[j];
    }
}

// FORWARD: loss and lse. GRAD: dz. With both, a row is read once: a thread
// keeps its first `HELD` units in registers between the statistics and the
// gradient and reads the rest again (they are in the L2 by then). GRAD alone
// takes the lse it is given.
template <bool BF16, bool FORWARD, bool GRAD, int HELD, int CL>
__global__ void __launch_bounds__(kLgThreads) distill_kernel(const DistillArgs a) {
    __shared__ LgShared sh;
    __shared__ TeacherShared te;
    if constexpr (CL > 1 && FORWARD) cluster_arrive_relaxed();
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t rank = CL > 1 ? cluster_ctarank() : 0;
    const long long r = blockIdx.x / CL;
    const Row<BF16> row(a.z, r, a.ld, a.V);
    const float c = a.inv_tau * kLog2e;
    constexpr int stride = kLgThreads * CL;
    const int u0 = rank * kLgThreads + threadIdx.x;

    // the first units are on their way while the teacher's entries are read
    uint4 held[HELD];
    row.load(held, u0, stride);
    float t_max;
    bool bad;
    const float t_sum = lg_teacher<BF16>(a, r, row, te, &t_max, &bad);

    float base, inv_s = 1.f;  // p = 2^((z - base) c) inv_s
    if constexpr (FORWARD) {
        Stats st{-INFINITY, 0.f, 0.f};
        lg_accumulate<BF16, false>(st, held, c);
        for (int u = u0 + HELD * stride; u < row.units; u += stride * kLgBatch) {
            uint4 raw[kLgBatch];
            row.load(raw, u, stride);
            lg_accumulate<BF16, false>(st, raw, c);
        }
        st = lg_row_stats<CL>(st, c, sh, rank);
        base = lg_base(st.m);
        inv_s = 1.0f / st.s;
        const float logs = logf(st.s);
        if (rank == 0) {
            float part = 0.f;
            const float logt = logf(t_sum);
            for (int i = threadIdx.x; i < a.K; i += kLgThreads) {
                if (te.id[i] < 0 || t_sum == 0.f) continue;
                const float lq = (te.q[i] - t_max) * a.inv_tau;
                const float q = exp2f(lq * kLog2e) / t_sum;
                if (q != 0.f) part += q * ((lq - logt) - ((te.z[i] - base) * a.inv_tau - logs));
            }
            part = lg_block_reduce(part, te.red, [](float x, float y) { return x + y; });
            if (threadIdx.x == 0) {
                if (a.loss) a.loss[r] = bad ? NAN : a.tau * a.tau * part;
                if (a.lse) a.lse[r] = st.s == 0.f ? -INFINITY : base * a.inv_tau + logs;
            }
        }
    } else {
        base = a.lse_in[r] * a.tau;  // p = exp((z - lse tau) / tau)
    }
    if constexpr (GRAD) {
        const float g = bad ? NAN : t_sum == 0.f ? 0.f : (a.weight ? a.weight[r] : 1.f) * a.tau;
        const float coef = g == 0.f ? 0.f : g * inv_s;
        char* d0 = static_cast<char*>(a.dz) + r * a.ldd * Row<BF16>::SZ - row.off * Row<BF16>::SZ;
        const bool vec = (reinterpret_cast<uintptr_t>(d0) & 15) == 0;
#pragma unroll
        for (int k = 0; k < HELD; ++k) lg_store_grad<BF16>(row, d0, vec, u0 + k * stride, held[k], base, c, coef);
        for (int u = u0 + HELD * stride; u < row.units; u += stride * kLgBatch) {
            uint4 raw[kLgBatch];
            row.load(raw, u, stride);
#pragma unroll
            for (int k = 0; k < kLgBatch; ++k) lg_store_grad<BF16>(row, d0, vec, u + k * stride, raw[k], base, c, coef);
        }
        __syncthreads();
        // the teacher's tokens again, from unrounded values, by the block that
        // owns their unit; an id that appears twice is written once, with both weights
        for (int i = threadIdx.x; i < a.K; i += kLgThreads) {
            const int id = te.id[i];
            if (id < 0 || t_sum == 0.f || ((id + row.off) / Row<BF16>::E / kLgThreads) % CL != (int)rank) continue;
            float w = 0.f;
            bool first = true;
            for (int j = 0; j < a.K; ++j) {
                if (te.id[j] != id) continue;
                if (j < i) first = false;
                w += exp2f((te.q[j] - t_max) * c);
            }
            if (!first) continue;
            const float x = g == 0.f ? 0.f : g * (lg_ex2((te.z[i] - base) * c) * inv_s - w / t_sum);
            if constexpr (BF16) reinterpret_cast<uint16_t*>(d0)[id + row.off] = f32_to_bf16_bits(x);
            else reinterpret_cast<float*>(d0)[id + row.off] = x;
        }
    }
}

// ------------------------------------------------------------------ launches

template <class Args>
int lg_launch(void (*kern)(const Args), const Args& a, long long blocks, int cl, cudaStream_t st, bool early) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kLgThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cl > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cl;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (early) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return LIN_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? LIN_OK : LIN_ERR_CUDA;
}

// Blocks per row: enough to give every SM four blocks when there are few rows,
// as long as every thread keeps a unit.
int lg_cluster(long long rows, int V, int esz, int sm_count) {
    const long long units = ((long long)V * esz + 15) / 16;
    int cl = 1;
    while (cl < kLgMaxCluster && rows * cl * 2 <= 4ll * sm_count && units >= 2ll * cl * kLgThreads) cl *= 2;
    return cl;
}

template <bool BF16>
int launch_logprobs_t(const LogprobArgs& a, long long rows, int cl, cudaStream_t st, bool early) {
    switch (cl) {
        case 1: return lg_launch(logprob_kernel<BF16, 1>, a, rows, 1, st, early);
        case 2: return lg_launch(logprob_kernel<BF16, 2>, a, rows * 2, 2, st, early);
        case 4: return lg_launch(logprob_kernel<BF16, 4>, a, rows * 4, 4, st, early);
        default: return lg_launch(logprob_kernel<BF16, 8>, a, rows * 8, 8, st, early);
    }
}

template <bool BF16, bool FORWARD, bool GRAD, int HELD>
int launch_distill_t(const DistillArgs& a, long long rows, int cl, cudaStream_t st, bool early) {
    switch (cl) {
        case 1: return lg_launch(distill_kernel<BF16, FORWARD, GRAD, HELD, 1>, a, rows, 1, st, early);
        case 2: return lg_launch(distill_kernel<BF16, FORWARD, GRAD, HELD, 2>, a, rows * 2, 2, st, early);
        case 4: return lg_launch(distill_kernel<BF16, FORWARD, GRAD, HELD, 4>, a, rows * 4, 4, st, early);
        default: return lg_launch(distill_kernel<BF16, FORWARD, GRAD, HELD, 8>, a, rows * 8, 8, st, early);
    }
}

}  // namespace

int launch_logprobs(const LogitsProblem& p) {
    LogprobArgs a;
    a.z = p.z;
    a.ld = p.ld;
    a.V = p.V;
    a.top = p.top;
    a.tokens = p.ids;
    a.wide = p.wide_ids;
    a.inv_tau = 1.0f / p.tau;
    a.logprob = p.logprob;
    a.entropy = p.entropy;
    a.lse = p.lse;
    a.top_logprob = p.top_logprob;
    a.top_ids = p.top_ids;
    const int cl = lg_cluster(p.R, p.V, p.bf16 ? 2 : 4, p.sm_count);
    return p.bf16 ? launch_logprobs_t<true>(a, p.R, cl, p.stream, p.early_start)
                  : launch_logprobs_t<false>(a, p.R, cl, p.stream, p.early_start);
}

int launch_distill(const LogitsProblem& p) {
    DistillArgs a;
    a.z = p.z;
    a.ld = p.ld;
    a.V = p.V;
    a.K = p.K;
    a.ids = p.ids;
    a.wide = p.wide_ids;
    a.teacher = p.teacher;
    a.teacher_bf16 = p.teacher_bf16;
    a.tau = p.tau;
    a.inv_tau = 1.0f / p.tau;
    a.weight = p.weight;
    a.lse_in = p.lse_in;
    a.loss = p.loss;
    a.lse = p.lse;
    a.dz = p.dz;
    a.ldd = p.ldd;
    const bool forward = p.lse_in == nullptr, grad = p.dz != nullptr;
    int cl = lg_cluster(p.R, p.V, p.bf16 ? 2 : 4, p.sm_count);
    auto go = [&](auto bf16) {
        constexpr bool B = decltype(bf16)::value;
        if (!grad) return launch_distill_t<B, true, false, kLgBatch>(a, p.R, cl, p.stream, p.early_start);
        // a row's units in the cluster's registers, as far as they go
        const long long units = ((long long)p.V * (B ? 2 : 4) + 31) / 16;
        while (cl < kLgMaxCluster && units > (long long)cl * kLgThreads * 8) cl *= 2;
        if (!forward) return launch_distill_t<B, false, true, 8>(a, p.R, cl, p.stream, p.early_start);
        return launch_distill_t<B, true, true, 8>(a, p.R, cl, p.stream, p.early_start);
    };
    return p.bf16 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace lin

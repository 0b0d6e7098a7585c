// Log probabilities of given tokens, with the entropy of their distribution and
// its top alternatives:
//   lse_r = log sum_j exp(z_rj / tau),  logprob_r = z_r,token / tau - lse_r,
//   H_r = - sum_j p_rj log p_rj,  and the `top` largest logits of a row with
//   their log probabilities, ordered by value, equal values by the lowest index.
// A row is read once, straight into registers; many small blocks an SM keep
// enough loads in flight (see logits.cuh). The top selection looks again only at
// the few threads that can hold one of the top values.
//
// Measured (GB300): 8192 x 50257 bf16 without a top 150 us (5.5 TB/s), top 8 180 us;
// 301 x 128001 fp32, top 32, 53 us; one row of 50257, top 20, 11 us. 2048 rows
// of the first issue in 64 % of the cycles with DRAM at 52 % (45 % with the top) of
// its nominal rate: neither is full, the warps wait for memory and for the
// instruction before. The small cases are bound by latency.
#include "logits.cuh"

namespace lin {
namespace {

constexpr int kLpThreads = 128;
constexpr int kLpWarps = kLpThreads / 32;
// Units a thread loads before it uses the first, and blocks an SM. fp32 units hold
// half the elements, so more of them have to be on their way for the same time
// (2048 x 50257 fp32, top 8: 82 us, with 4 and 10 96 us); bf16 has more to compute
// and gains from more warps (8192 x 50257 bf16, top 8: 178 us, with 8 and 8 196 us;
// without a top 156 and 150 in that run).
constexpr int lp_batch(bool bf16) { return bf16 ? 4 : 8; }
constexpr int lp_blocks(bool bf16) { return bf16 ? 10 : 8; }
constexpr int kLpFolds = 16;   // maxima kept of a thread's batches (batch n in place n % 16)
constexpr int kLpList = 512;   // candidates of the top selection held in shared memory

// Whole-number order of the values: a larger value has a larger key, zeros of
// either sign are equal, NaN ranks with -inf, and 0 is below every value.
__device__ __forceinline__ uint32_t lg_key(float x) {
    if (x != x) x = -INFINITY;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float lg_key_value(uint32_t k) {  // (NaN for 0)
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

struct LogprobArgs {
    const void* z;
    long long ld;
    int V, top;
    const void* tokens;  // null: no tokens
    bool wide;           // 64-bit tokens
    float c, inv_tau;    // log2(e) / tau, 1 / tau
    float* logprob;
    float* entropy;      // or null
    float* lse;          // or null
    float* top_logprob;
    int* top_ids;
};

struct TopShared {
    uint64_t list[kLpList];
    uint64_t best[kLgMaxCluster * kLogprobMaxTop];  // a list of `top` from each block
    float seen[kLpFolds][kLpThreads];               // largest value of a thread's batches
    int count;
};

__device__ __forceinline__ void dsmem_st_u64(uint32_t addr, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// The `top` largest of the n unique keys in `list`, in order, to out[0..top);
// places that the keys do not fill are 0. The keys are ranked by counting.
__device__ __forceinline__ void lp_rank(const uint64_t* list, int n, int top, uint64_t* out) {
    for (int i = threadIdx.x; i < top; i += kLpThreads)
        if (i >= n) out[i] = 0;
    for (int i = threadIdx.x; i < n; i += kLpThreads) {
        const uint64_t mine = list[i];
        int above = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) above += list[j] > mine;
        if (above < top && mine != 0) out[above] = mine;
    }
}

__device__ __forceinline__ uint64_t lp_full_key(float x, int i) {
    return (uint64_t)lg_key(x) << 32 | (0xFFFFFFFFu - (uint32_t)i);
}

// Element j of a unit.
template <bool BF16>
__device__ __forceinline__ float lp_element(const uint4& r, int j) {
    const int k = BF16 ? j >> 1 : j;
    const uint32_t w = k == 0 ? r.x : k == 1 ? r.y : k == 2 ? r.z : r.w;
    if constexpr (BF16) return __uint_as_float((j & 1) ? w & 0xFFFF0000u : w << 16);
    else return __uint_as_float(w);
}

template <bool BF16, int CL>
__global__ void __launch_bounds__(kLpThreads, lp_blocks(BF16)) logprob_kernel(const LogprobArgs a) {
    __shared__ LgExchange<kLpThreads> sh;
    __shared__ TopShared tp;
    if constexpr (CL > 1) cluster_arrive_relaxed();
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t rank = CL > 1 ? cluster_ctarank() : 0;
    const long long r = blockIdx.x / CL;
    const Row<BF16> row(a.z, r, a.ld, a.V);
    constexpr int stride = kLpThreads * CL, kLpBatch = lp_batch(BF16);
    const int u0 = rank * kLpThreads + threadIdx.x, warp = threadIdx.x >> 5;

    const bool asked = rank == 0 && threadIdx.x == 0;
    int tok = -1;
    float z_tok = 0.f;
    if (asked && a.logprob) {  // on its way while the row is read
        tok = lg_load_id(a.tokens, a.wide, r);
        if (tok >= 0 && tok < a.V) z_tok = row.at(tok);
    }
    int batches = 0;
    Stats st = lg_stream<BF16, true, kLpBatch>(row, u0, stride, a.c, [&](float m) {
        if (a.top > 0) {
            float& kept = tp.seen[batches % kLpFolds][threadIdx.x];
            kept = batches < kLpFolds ? m : fmaxf(kept, m);
            ++batches;
        }
    });

    // A lower bound of the row's top-th largest value: of the W warps whose threads
    // all have units, each finds the largest key (its upper 16 bits, all that bf16
    // has) that ceil(top / W) of its threads' own maxima reach; `top` values of the
    // block reach the least of them, and the row's bound is the best of its
    // blocks'. Only threads whose maximum reaches it look at their units again.
    const uint32_t have = u0 < row.units ? lg_key(st.m) : 0u;
    if (a.top > 0) {
        const int mine = row.units - (int)rank * kLpThreads;  // units in the block's first turn, if less than its threads
        const int W = mine <= 0 ? 0 : min(kLpWarps, mine / 32);
        const int q = W > 0 ? (a.top + W - 1) / W : 33;
        st.bound = warp < W ? 0u : W > 0 ? 0xFFFFFFFFu : 0u;
        if (warp < W) {
#pragma unroll
            for (int b = 31; b >= 16; --b) {
                const uint32_t cand = st.bound | (1u << b);
                if (__popc(__ballot_sync(0xffffffffu, have >= cand)) >= q) st.bound = cand;
            }
        }
        if (threadIdx.x == 0) tp.count = 0;
    }
    st = lg_join_blocks<kLpThreads, CL>(st, a.c, sh, rank);
    const float base = lg_base(st.m), logs = log2f(st.s);
    auto logprob = [&](float z) { return st.s == 0.f ? -INFINITY : fmaf(-logs, kLn2, (z - base) * a.inv_tau); };
    if (asked) {
        if (a.logprob) a.logprob[r] = tok < 0 ? 0.f : tok >= a.V ? NAN : logprob(z_tok);
        if (a.entropy) a.entropy[r] = st.s == 0.f ? 0.f : (logs - st.t / st.s) * kLn2;
        if (a.lse) a.lse[r] = st.s == 0.f ? -INFINITY : fmaf(logs, kLn2, base * a.inv_tau);
    }
    if (a.top == 0) return;

    const uint32_t bound = st.bound;
    const float least_value = lg_key_value(bound);
    uint32_t folds = 0;  // batches of this thread that reach the bound
    if (have != 0)
        for (int f = 0; f < min(batches, kLpFolds); ++f)
            if (!(tp.seen[f][threadIdx.x] < least_value)) folds |= 1u << f;
    for (; folds; folds &= folds - 1) {
        for (int f = __ffs(folds) - 1; f < batches; f += kLpFolds) {
            const int u = u0 + f * stride * kLpBatch;
            uint4 raw[kLpBatch];
            row.load(raw, u, stride);
            uint32_t in = 0;
#pragma unroll
            for (int k = 0; k < kLpBatch; ++k)
                if (!(lg_unit_max<BF16>(raw[k]) < least_value)) in |= 1u << k;
            for (; in; in &= in - 1) {  // few: their code stands here once
                const int v = u + (__ffs(in) - 1) * stride;
                if (v >= row.units) break;
                uint4 one = Row<BF16>::nothing();
                if (!row.whole(v)) one = row.load_edge(v);
                else lg_ldg16_if(one, true, row.a0 + (long long)v * 16);
#pragma unroll
                for (int j = 0; j < Row<BF16>::E; ++j) {
                    const float x = lp_element<BF16>(one, j);
                    const int i = row.first(v) + j;
                    if (i < 0 || i >= a.V || lg_key(x) < bound) continue;
                    const int n = atomicAdd(&tp.count, 1);
                    if (n < kLpList) tp.list[n] = lp_full_key(x, i);
                }
            }
        }
    }
    __syncthreads();
    const int n = tp.count;
    uint64_t* own = tp.best + rank * a.top;
    if (n <= kLpList) {
        lp_rank(tp.list, n, a.top, own);
    } else {
        // More candidates than the list holds (a row that is mostly one value). In
        // the order of the units, one element of each thread at a time: what beats
        // the top-th best so far joins the list, which is then cut to `top`.
        __syncthreads();  // tp.count has been read
        if (threadIdx.x == 0) tp.count = 0;
        uint64_t least = (uint64_t)bound << 32;
        for (int ub = rank * kLpThreads; ub < row.units; ub += stride * kLpBatch) {
            uint4 raw[kLpBatch];
            row.load(raw, ub + (int)threadIdx.x, stride);
#pragma unroll
            for (int k = 0; k < kLpBatch; ++k) {
                const int v = ub + k * stride + (int)threadIdx.x;
                if (__syncthreads_or(v < row.units && lg_key(lg_unit_max<BF16>(raw[k])) >= (uint32_t)(least >> 32)) == 0)
                    continue;
#pragma unroll 1
                for (int j = 0; j < Row<BF16>::E; ++j) {
                    const int i = v < row.units ? row.first(v) + j : -1;
                    const uint64_t key = lp_full_key(lp_element<BF16>(raw[k], j), i);
                    const bool in = i >= 0 && i < a.V && key > least;
                    if (__syncthreads_or(in) == 0) continue;
                    if (in) tp.list[atomicAdd(&tp.count, 1)] = key;  // at most top + 128
                    __syncthreads();
                    const int now = tp.count;
                    if (now < a.top) continue;
                    lp_rank(tp.list, now, a.top, own);
                    __syncthreads();
                    for (int q = threadIdx.x; q < a.top; q += kLpThreads) tp.list[q] = own[q];
                    if (threadIdx.x == 0) tp.count = a.top;
                    least = own[a.top - 1];
                    __syncthreads();
                }
            }
        }
        __syncthreads();
        lp_rank(tp.list, tp.count, a.top, own);
    }
    __syncthreads();
    const uint64_t* best = own;
    if constexpr (CL > 1) {
        // the ranks' lists to rank 0, which ranks them together
        if (rank != 0)
            for (int i = threadIdx.x; i < a.top; i += kLpThreads)
                dsmem_st_u64(dsmem_map(smem_u32(own + i), 0), own[i]);
        __syncwarp();
        cluster_sync_all();
        if (rank != 0) return;
        lp_rank(tp.best, CL * a.top, a.top, tp.list);
        __syncthreads();
        best = tp.list;
    }
    for (int i = threadIdx.x; i < a.top; i += kLpThreads) {
        const uint64_t k = best[i];
        a.top_logprob[r * a.top + i] = logprob(lg_key_value((uint32_t)(k >> 32)));
        a.top_ids[r * a.top + i] = (int)(0xFFFFFFFFu - (uint32_t)k);
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
    a.c = (float)(1.4426950408889634 / p.tau);
    a.inv_tau = 1.0f / p.tau;
    a.logprob = p.logprob;
    a.entropy = p.entropy;
    a.lse = p.lse;
    a.top_logprob = p.top_logprob;
    a.top_ids = p.top_ids;
    const int cl = lg_cluster(p, kLpThreads, lp_blocks(p.bf16));
    return lg_by_cluster(cl, [&](auto c) {
        constexpr int CL = decltype(c)::value;
        return p.bf16 ? lg_launch(logprob_kernel<true, CL>, p.R * CL, kLpThreads, 0, CL, p, a)
                      : lg_launch(logprob_kernel<false, CL>, p.R * CL, kLpThreads, 0, CL, p, a);
    });
}

}  // namespace lin

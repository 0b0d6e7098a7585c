// Distillation towards a teacher's top logits: with q = softmax(t / tau) over a
// row's valid teacher entries and p = softmax(z / tau) over the row,
//   loss_r = tau^2 sum_i q_i (log q_i - log p_id(i)),
//   dz_rj  = g_r tau (p_rj - sum of q_i with id(i) = j).
// The loss alone streams a row through registers (many small blocks an SM). The
// gradient, with or without the loss, runs persistent blocks:
//   warps 0-7   the row's statistics, then its gradient;
//   warp 8      bulk copies into a ring of chunks in shared memory, ahead of the
//               rows; a row stays in the ring from its statistics to its
//               gradient, so that it is read from memory once;
//   warps 9-12  the teacher's entries of the rows to come (two dependent reads of
//               memory that nothing else waits for), and, when a row's gradient is
//               stored, its loss and its teacher's tokens again.
// The row's way through warps 0-7 then has one barrier. Every wait is bounded
// (about 1 s); a block that gives up sets the device status word.
//
// Measured (GB300, 8192 x 50257 bf16, 32 entries): loss 138 us (6.0 TB/s), loss and
// gradient 345 us (4.8 TB/s), gradient 292 us (5.6 TB/s); 2048 x 50257 fp32, 64
// entries: gradient 161 us, loss and gradient 176 us (5.1 and 4.7 TB/s). Of 2048 bf16
// rows the gradient kernel issues in 46 % of the cycles (58 % with the loss) with DRAM
// at 61 % (48 %) of its nominal rate: neither is full. Its warps wait, for memory and
// for the instruction before, and the ring in shared memory leaves room for 26 of them
// an SM. That ring is what the loss and gradient together need; the gradient from a
// given lse shares the kernel, and has not been built as a stream through registers.
#include "logits.cuh"

namespace lin {
namespace {

constexpr int kDfThreads = 128;   // loss alone
constexpr int kDfBatch = 8;
constexpr int kDgThreads = 256;   // gradient: the threads that compute
constexpr int kDgWarps = kDgThreads / 32;
constexpr int kDgHelpers = 4;     // (32768 x 8000 bf16, gradient: 283 us with 2, 200 with 4; loss and gradient of
                                  // 8192 x 50257 348 and 354)
constexpr int kDgAll = kDgThreads + 32 + 32 * kDgHelpers;
// Units of a thread in a chunk, at most. A slice goes in as few chunks as that allows,
// all of about one size, which often is less than the limit: the kernel is there for
// chunks of up to four units, whose code is shorter, and for five. Loss and gradient, in
// us, with a limit of 4 and of 5: where five means fewer chunks, 7959 x 50257 bf16 388
// and 347, 3999 x 100003 bf16 427 and 377, 32768 x 5003 fp32 509 and 407, 19989 x 20011
// bf16 522 and 540; where it does not, code for 4 and for 5, 32768 x 8000 bf16 313 and
// 329, 12498 x 32003 bf16 409 and 427, 3124 x 128001 bf16 451 and 478. (Eight, at 8192 x
// 50257: 393 against 354.)
constexpr int kDgBatch = 5, kDgSmallBatch = 4;
constexpr int kDgRing = 32;       // chunks of the ring, at most
constexpr int kDgRows = 2 * kDgHelpers;  // rows between their teacher's entries and their loss
// Shared memory of a block when two share an SM (228 KB, 1 KB of it reserved for each block).
constexpr size_t kDgSmem = 113 * 1024;

struct DistillArgs {
    const void* z;
    long long ld;
    int V, K;
    const void* ids;
    bool wide;              // 64-bit ids
    const void* teacher;
    bool teacher_bf16;
    float tau, c, inv_tau;  // temperature, log2(e) / tau, 1 / tau
    const float* weight;    // upstream gradient of a row's loss, or null (1)
    const float* lse_in;    // backward alone
    float* loss;            // or null
    float* lse;             // or null
    void* dz;
    long long ldd;
};

// A row's teacher entries in shared memory, padded to a multiple of four.
struct Teacher {
    int* id;      // -1: no entry
    float* t;     // the teacher's logit
    float* z;     // the student's logit there
};
__host__ __device__ __forceinline__ int lg_padded(int K) { return (K + 3) & ~3; }
__device__ __forceinline__ Teacher lg_teacher_at(void* mem, int K, int n) {
    int* p = static_cast<int*>(mem) + (size_t)n * 3 * lg_padded(K);
    return {p, reinterpret_cast<float*>(p + lg_padded(K)), reinterpret_cast<float*>(p + 2 * lg_padded(K))};
}
struct TeacherSums {
    float top, sum;  // largest valid logit; sum of exponentials against it (0: no entry carries weight)
    bool bad;        // an id lies past the vocabulary
};

// One warp reads a row's entries.
template <bool BF16>
__device__ __forceinline__ TeacherSums lg_teacher(const DistillArgs& a, long long r, Teacher te) {
    const Row<BF16> row(a.z, r, a.ld, a.V);
    const int lane = threadIdx.x & 31;
    float m = -INFINITY;
    bool over = false;
#pragma unroll 2
    for (int i = lane; i < lg_padded(a.K); i += 32) {
        const int id = i < a.K ? lg_load_id(a.ids, a.wide, r * a.K + i) : -1;
        float t = -INFINITY, z = 0.f;
        if (id >= a.V) over = true;
        const bool held = id >= 0 && id < a.V;
        if (held) {
            t = a.teacher_bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(a.teacher)[r * a.K + i])
                               : static_cast<const float*>(a.teacher)[r * a.K + i];
            z = row.at(id);
        }
        te.id[i] = held ? id : -1;
        te.t[i] = t;
        te.z[i] = z;
        m = fmaxf(m, t);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float sum = 0.f;
    for (int i = lane; i < a.K; i += 32)
        if (te.id[i] >= 0) sum += m != -INFINITY || te.t[i] != te.t[i] ? exp2f((te.t[i] - m) * a.c) : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return {m, sum, __any_sync(0xffffffffu, over) != 0};
}

// One warp: the loss from the row's statistics (p = 2^((z - base) c - logs)). With the
// temperature drawn out of the logarithms, tau^2 (log q - log p) is tau times
// (t - top) - (z - base) + tau ln 2 (logs - logt), where t and z are in their own units:
// a teacher's token that the student masks with the type's lowest value then costs what
// it costs, and does not overflow on the way.
__device__ __forceinline__ float lg_loss(const DistillArgs& a, Teacher te, const TeacherSums& s, float base,
                                         float logs) {
    float part = 0.f;
    const float rest = a.tau * kLn2 * (logs - log2f(s.sum));
    for (int i = threadIdx.x & 31; i < a.K; i += 32) {
        if (te.id[i] < 0 || s.sum == 0.f) continue;
        const float t = te.t[i] - s.top;
        const float q = exp2f(t * a.c) / s.sum;
        if (q != 0.f) part += q * (t - (te.z[i] - base) + rest);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    return s.bad ? NAN : a.tau * part;
}

// ------------------------------------------------------------------ loss alone

template <bool BF16, int CL>
__global__ void __launch_bounds__(kDfThreads, 8) distill_loss_kernel(const DistillArgs a) {
    extern __shared__ __align__(16) uint8_t entries[];
    __shared__ LgExchange<kDfThreads> sh;
    if constexpr (CL > 1) cluster_arrive_relaxed();
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t rank = CL > 1 ? cluster_ctarank() : 0;
    const long long r = blockIdx.x / CL;
    const Row<BF16> row(a.z, r, a.ld, a.V);
    const Teacher te = lg_teacher_at(entries, a.K, 0);
    TeacherSums s{0.f, 0.f, false};
    if (rank == 0 && threadIdx.x < 32) s = lg_teacher<BF16>(a, r, te);
    Stats st = lg_stream<BF16, false, kDfBatch>(row, rank * kDfThreads + threadIdx.x, kDfThreads * CL, a.c, [](float) {});
    st = lg_join_blocks<kDfThreads, CL>(st, a.c, sh, rank);
    if (rank != 0 || threadIdx.x >= 32) return;
    const float base = lg_base(st.m), logs = log2f(st.s);
    const float loss = lg_loss(a, te, s, base, logs);
    if (threadIdx.x == 0) {
        a.loss[r] = loss;
        if (a.lse) a.lse[r] = st.s == 0.f ? -INFINITY : fmaf(logs, kLn2, base * a.inv_tau);
    }
}

// ------------------------------------------------------------------ gradient

__device__ __forceinline__ void dg_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kDgThreads) : "memory"); }
// Untiled copy; addresses and size are multiples of 16 bytes.
__device__ __forceinline__ void lg_bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

struct DgShared {
    uint64_t full[kDgRing], empty[kDgRing];  // chunks of the ring
    uint64_t stats_in;                       // statistics of the cluster's blocks
    uint64_t teacher[kDgRows];               // a row's teacher entries are there
    uint64_t stored[kDgRows];                // its gradient is stored
    Stats warp[2][kDgWarps];                 // of this row and the one before
    Stats rank[2][kLgMaxCluster];
    float weight[kDgRows];                   // g tau; 0 without entries, NaN for an id past the vocabulary
    float base[kDgRows], logs[kDgRows];
    int abort;
};

// How a launch cuts its rows.
struct DgRing {
    int chunk;   // units of a chunk
    int slots;   // chunks of the ring
    int whole;   // a slice fits the ring and stays there until its gradient is stored
    long long rows;
    int* status;
};

// A block's slice of its cluster's rows. Chunks are numbered in the order in
// which they pass through the ring; `slot` and `phase` follow that order.
template <bool BF16, int CL, int BATCH>
struct Slice {
    DgShared& sh;
    const DgRing& g;
    uint4* ring;
    uint32_t rank;
    int slot, phase;

    __device__ __forceinline__ Slice(DgShared& s, const DgRing& r, void* mem, uint32_t k)
        : sh(s), g(r), ring(static_cast<uint4*>(mem)), rank(k), slot(0), phase(0) {}
    __device__ __forceinline__ int begin(const Row<BF16>& row) const {
        return CL == 1 ? 0 : min(row.units, (int)rank * ((row.units + CL - 1) / CL));
    }
    __device__ __forceinline__ int end(const Row<BF16>& row) const {
        return CL == 1 ? row.units : min(row.units, (int)(rank + 1) * ((row.units + CL - 1) / CL));
    }
    __device__ __forceinline__ void step() {
        if (++slot == g.slots) {
            slot = 0;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ void give_up() const {
        atomicExch(&sh.abort, 1);
        atomicExch(g.status, (int)LIN_ERR_DEVICE_TIMEOUT);
    }
    __device__ __forceinline__ bool aborted() const { return *(volatile int*)&sh.abort != 0; }
    // Bounded wait; once one has run out nothing is waited for any more.
    __device__ __forceinline__ void wait(uint64_t& bar, int parity) const {
        if (!mbar_try_wait(smem_u32(&bar), parity) && !aborted() && !mbar_wait(smem_u32(&bar), parity)) give_up();
    }
    __device__ __forceinline__ void arrive(uint64_t& bar) const {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bar));
    }
    // The units that this thread's warp has in a chunk [c0, c1) (a thread takes every 256th).
    __device__ __forceinline__ static int count(int c0, int c1) {
        return (c1 - c0 - (int)(threadIdx.x & ~31u) + kDgThreads - 1) / kDgThreads;
    }
    // This thread's units of a chunk; units past its end read as -inf. `again`: from memory.
    __device__ __forceinline__ void units(const Row<BF16>& row, int which, int c0, int c1, uint4 (&r)[BATCH],
                                          bool again = false) const {
        const int n = c1 - c0 - (int)threadIdx.x;
        if (!again) {
            const uint32_t at = smem_u32(ring) + ((uint32_t)which * g.chunk + threadIdx.x) * 16u;
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                r[k] = Row<BF16>::nothing();
                lg_lds16_if(r[k], n > k * kDgThreads, at + k * (kDgThreads * 16u));
            }
        } else {
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int u = c0 + threadIdx.x + k * kDgThreads;
                r[k] = Row<BF16>::nothing();
                lg_ldg16_if(r[k], n > k * kDgThreads && row.whole(u), row.a0 + (long long)u * 16);
            }
        }
        if (c0 > 0 && c1 < row.units) return;  // (as most chunks) no unit sticks out
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int u = c0 + threadIdx.x + k * kDgThreads;
            if (u < c1 && !row.whole(u)) r[k] = row.load_edge(u);
        }
    }
    // The copying thread: the whole units of every chunk of every row.
    __device__ void copy(const void* z, long long ld, int V) {
        bool ok = true;
        uint32_t issued = 0;
        for (long long r = blockIdx.x / CL; ok && r < g.rows; r += gridDim.x / CL) {
            const Row<BF16> row(z, r, ld, V);
            const int e = end(row);
            for (int c0 = begin(row); c0 < e; c0 += g.chunk) {
                if (aborted() || !mbar_wait(smem_u32(&sh.empty[slot]), phase ^ 1)) {
                    ok = false;
                    break;
                }
                int a = c0, b = min(c0 + g.chunk, e);
                uint4* dst = ring + (size_t)slot * g.chunk;
                if (a == 0 && !row.whole(0)) {
                    ++a;
                    ++dst;
                }
                if (b == row.units && b > a && !row.whole(b - 1)) --b;
                const uint32_t bytes = b > a ? (uint32_t)(b - a) * 16u : 0u;
                mbar_expect_tx(smem_u32(&sh.full[slot]), bytes);
                if (bytes) lg_bulk_load(smem_u32(dst), row.a0 + (long long)a * 16, bytes, smem_u32(&sh.full[slot]));
                ++issued;
                step();
            }
        }
        if (!ok) {
            give_up();
            // let the copies still in flight land
            for (int k = 0; k < g.slots && k < (int)issued; ++k) {
                if (--slot < 0) {
                    slot = g.slots - 1;
                    phase ^= 1;
                }
                mbar_wait(smem_u32(&sh.full[slot]), phase);
            }
        }
    }
};

// Statistics of the whole row in every computing thread of the cluster; `seq` counts the calls.
template <bool BF16, int CL, int BATCH>
__device__ __forceinline__ Stats dg_row_stats(const Slice<BF16, CL, BATCH>& sl, Stats st, float c, uint32_t seq) {
    DgShared& sh = sl.sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Stats* parts = sh.warp[seq & 1];
    st = lg_warp_join(st, c);
    if (lane == 0) parts[warp] = st;
    dg_sync();
    st = lg_warp_join(lane < kDgWarps ? parts[lane] : Stats{-INFINITY, 0.f, 0.f, 0u}, c);
    if constexpr (CL > 1) {
        Stats* slots = sh.rank[seq & 1];
        if (warp == 0) {
            if (lane < CL) {
                const uint32_t dst = dsmem_map(smem_u32(&slots[sl.rank]), lane);
                dsmem_st_f32(dst, st.m);
                dsmem_st_f32(dst + 4, st.s);
                mbar_arrive_remote(dsmem_map(smem_u32(&sh.stats_in), lane));
            }
            __syncwarp();
        }
        if (!sl.aborted() && !mbar_wait_cluster(smem_u32(&sh.stats_in), seq & 1)) sl.give_up();
        st = Stats{slots[0].m, slots[0].s, 0.f, 0u};
#pragma unroll
        for (int k = 1; k < CL; ++k) st = lg_join(st, Stats{slots[k].m, slots[k].s, 0.f, 0u}, c);
    }
    return st;
}

// coef 2^((z - base) c) for a unit's values, in the logits' type; 0 where `keep` is 0.
template <bool BF16>
__device__ __forceinline__ uint4 dg_unit(const uint4& raw, float base, float c, float coef, uint32_t keep) {
    uint64_t v[Row<BF16>::E / 2];
    lg_values<BF16>(raw, v);
    const uint64_t nb2 = lg_pack(-base, -base), c2 = lg_pack(c, c), k2 = lg_pack(coef, coef);
    float x[Row<BF16>::E];
#pragma unroll
    for (int j = 0; j < Row<BF16>::E / 2; ++j) {
        float e0, e1;
        lg_unpack(lg_mul2(lg_add2(v[j], nb2), c2), e0, e1);
        lg_unpack(lg_mul2(lg_pack(lg_ex2(e0), lg_ex2(e1)), k2), x[2 * j], x[2 * j + 1]);
    }
    if constexpr (BF16)
        return make_uint4(pack_bf16x2(x[0], x[1]) & keep, pack_bf16x2(x[2], x[3]) & keep, pack_bf16x2(x[4], x[5]) & keep,
                          pack_bf16x2(x[6], x[7]) & keep);
    else
        return make_uint4(__float_as_uint(x[0]) & keep, __float_as_uint(x[1]) & keep, __float_as_uint(x[2]) & keep,
                          __float_as_uint(x[3]) & keep);
}

// Element 0 of the gradient's row, less the units' offset: unit u lies at + 16 u.
template <bool BF16>
__device__ __forceinline__ char* dg_row(const DistillArgs& a, long long r, const Row<BF16>& row) {
    return static_cast<char*>(a.dz) + (r * a.ldd - row.off) * Row<BF16>::SZ;
}

// The largest |lse| from which the gradient alone takes p = exp(z / tau - lse). A given
// lse is right to half a step of fp32, and its product with tau to another: 2^-23 |lse|
// relative on every p of the row, which is 1/64 of a bf16 half step (2^-8) at 512 and
// 128 roundings of fp32 at 64. Past it (logits that lie far from zero, a mask of the
// type's lowest value on all of them) lse has lost the digits that p needs, and the
// row's maximum and sum are computed again (7959 rows of 50257 bf16, all of them past
// it: 440 us against 288).
template <bool BF16>
constexpr float dg_lse_limit() { return BF16 ? 512.f : 64.f; }

// FORWARD: the statistics (and the loss) are computed; else lse is given.
template <bool BF16, bool FORWARD, int CL, int BATCH>
__global__ void __launch_bounds__(kDgAll, 2) distill_grad_kernel(const DistillArgs a, const DgRing g) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ DgShared sh;
    const uint32_t rank = CL > 1 ? cluster_ctarank() : 0;
    if (threadIdx.x == 0) {
        for (int k = 0; k < g.slots; ++k) {
            mbar_init(smem_u32(&sh.full[k]), 1);
            mbar_init(smem_u32(&sh.empty[k]), kDgWarps);
        }
        mbar_init(smem_u32(&sh.stats_in), CL);
        for (int k = 0; k < kDgRows; ++k) {
            mbar_init(smem_u32(&sh.teacher[k]), 1);
            mbar_init(smem_u32(&sh.stored[k]), kDgWarps);
        }
        sh.abort = 0;
        mbar_fence_init();
    }
    if constexpr (CL > 1) cluster_sync_all();  // the peers' barriers are ready
    else __syncthreads();
    pdl_wait();  // first, so that a call after this one never runs beside one before it
    pdl_launch_dependents();
    Slice<BF16, CL, BATCH> sl(sh, g, smem, rank);
    void* entries = smem + (size_t)g.slots * g.chunk * 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long r0 = blockIdx.x / CL, step = gridDim.x / CL;

    if (warp == kDgWarps) {
        if (lane == 0) sl.copy(a.z, a.ld, a.V);
    } else if (warp > kDgWarps) {
        // ---- the teacher's entries ahead of a row, its loss and tokens after it ----
        const int h = warp - kDgWarps - 1;
        auto ahead = [&](uint32_t seq) {
            const long long r = r0 + seq * step;
            if (r >= g.rows) return TeacherSums{0.f, 0.f, false};
            const int b = seq % kDgRows;
            const TeacherSums s = lg_teacher<BF16>(a, r, lg_teacher_at(entries, a.K, b));
            if (lane == 0) sh.weight[b] = s.bad ? NAN : s.sum == 0.f ? 0.f : (a.weight ? a.weight[r] : 1.f) * a.tau;
            sl.arrive(sh.teacher[b]);
            return s;
        };
        TeacherSums now = ahead(h);
        for (uint32_t seq = h; r0 + seq * step < g.rows; seq += kDgHelpers) {
            const long long r = r0 + seq * step;
            const TeacherSums next = ahead(seq + kDgHelpers);
            const int b = seq % kDgRows;
            const Row<BF16> row(a.z, r, a.ld, a.V);
            const Teacher te = lg_teacher_at(entries, a.K, b);
            sl.wait(sh.stored[b], (seq / kDgRows) & 1);
            const float base = sh.base[b], logs = sh.logs[b], w = sh.weight[b];
            if (FORWARD && rank == 0 && a.loss) {
                const float loss = lg_loss(a, te, now, base, logs);
                if (lane == 0) a.loss[r] = loss;
            }
            // The teacher's tokens, from unrounded values, by the block that has their
            // unit; a token that appears twice is written once, with both weights.
            const int u0 = sl.begin(row), u1 = sl.end(row);
            char* d0 = dg_row(a, r, row);
            for (int i = lane; i < a.K; i += 32) {
                const int id = te.id[i], u = (id + row.off) / Row<BF16>::E;
                if (id < 0 || now.sum == 0.f || u < u0 || u >= u1) continue;
                float q = 0.f;
                bool first = true;
                for (int j = 0; j < a.K; j += 4) {
                    const int4 x = *reinterpret_cast<const int4*>(te.id + j);
                    const int e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (e[k] == id) {
                            if (j + k < i) first = false;
                            q += exp2f((te.t[j + k] - now.top) * a.c);
                        }
                }
                if (!first) continue;
                const float x = w == 0.f ? 0.f : w * (exp2f((te.z[i] - base) * a.c - logs) - q / now.sum);
                if constexpr (BF16) reinterpret_cast<uint16_t*>(d0)[id + row.off] = f32_to_bf16_bits(x);
                else reinterpret_cast<float*>(d0)[id + row.off] = x;
            }
            __syncwarp();
            now = next;
        }
    } else {
        uint32_t seq = 0, renewed = 0;  // rows; those whose statistics are computed although lse is given
        for (long long r = r0; r < g.rows; r += step, ++seq) {
            const Row<BF16> row(a.z, r, a.ld, a.V);
            const int u0 = sl.begin(row), u1 = sl.end(row), b = seq % kDgRows;
            float base, logs = 0.f, inv_s = 1.f;  // p = 2^((z - base) c) inv_s
            int slot = sl.slot;
            if constexpr (FORWARD) {
                Stats st{-INFINITY, 0.f, 0.f, 0u};
                for (int c0 = u0; c0 < u1; c0 += g.chunk) {
                    const int c1 = min(c0 + g.chunk, u1);
                    sl.wait(sh.full[sl.slot], sl.phase);
                    uint4 raw[BATCH];
                    sl.units(row, sl.slot, c0, c1, raw);
                    if (!g.whole) sl.arrive(sh.empty[sl.slot]);
                    lg_accumulate<BF16, false>(st, raw, sl.count(c0, c1), a.c);
                    sl.step();
                }
                // The teacher's warp has read the row's logits in this block, so that
                // the statistics tell the peers that they may write to it.
                sl.wait(sh.teacher[b], (seq / kDgRows) & 1);
                st = dg_row_stats(sl, st, a.c, seq);
                base = lg_base(st.m);
                logs = log2f(st.s);
                inv_s = 1.0f / st.s;
            } else {
                const float lse = a.lse_in[r];
                base = lse * a.tau;
                sl.wait(sh.teacher[b], (seq / kDgRows) & 1);
                if (!(fabsf(lse) <= dg_lse_limit<BF16>())) {
                    Stats st{-INFINITY, 0.f, 0.f, 0u};
                    for (int c0 = u0; c0 < u1; c0 += g.chunk) {
                        const int c1 = min(c0 + g.chunk, u1);
                        uint4 raw[BATCH];
                        sl.units(row, 0, c0, c1, raw, true);
                        lg_accumulate<BF16, false>(st, raw, sl.count(c0, c1), a.c);
                    }
                    st = dg_row_stats(sl, st, a.c, renewed++);
                    base = lg_base(st.m);
                    logs = log2f(st.s);
                    inv_s = 1.0f / st.s;
                }
            }
            const float w = sh.weight[b], coef = w * inv_s;
            const uint32_t keep = w == 0.f ? 0u : ~0u;
            if (threadIdx.x == 0) {
                sh.base[b] = base;
                sh.logs[b] = logs;
            }
            char* d0 = dg_row(a, r, row);
            const bool vec = (reinterpret_cast<uintptr_t>(d0) & 15) == 0;
            for (int c0 = u0; c0 < u1; c0 += g.chunk) {
                const int c1 = min(c0 + g.chunk, u1);
                if constexpr (!FORWARD) sl.wait(sh.full[sl.slot], sl.phase);
                uint4 raw[BATCH];
                sl.units(row, slot, c0, c1, raw, FORWARD && !g.whole);
                if (!FORWARD || g.whole) sl.arrive(sh.empty[slot]);
                const bool plain = vec && c0 > 0 && c1 < row.units;
                const int n = sl.count(c0, c1);
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    if (k >= n) break;
                    const int u = c0 + threadIdx.x + k * kDgThreads;
                    const uint4 o = dg_unit<BF16>(raw[k], base, a.c, coef, keep);
                    char* p = d0 + (long long)u * 16;
                    if (u < c1) {
                        if (plain || (vec && row.whole(u))) *reinterpret_cast<uint4*>(p) = o;
                        else row.store_edge(p, u, o);
                    }
                }
                if constexpr (!FORWARD) sl.step();
                if (++slot == g.slots) slot = 0;
            }
            sl.arrive(sh.stored[b]);
        }
    }
    if constexpr (CL > 1) {
        __syncwarp();
        cluster_sync_all();  // no peer writes to this block any more
    }
}

struct DgPlan {
    DgRing ring;
    int cl;
    size_t smem;  // dynamic
};

DgPlan dg_plan(const LogitsProblem& p, bool whole, size_t extra) {
    const long long most = ((long long)p.V * (p.bf16 ? 2 : 4) + 15) / 16 + 1;  // units of a row
    const long long budget = ((long long)kDgSmem - (long long)sizeof(DgShared) - (long long)extra) / 16;
    DgPlan q;
    q.cl = lg_cluster(p, kDgThreads, 1);
    auto slice = [&]() { return (most + q.cl - 1) / q.cl; };
    // Chunks of whole unit rows (a unit of every thread), as large as a batch, or
    // smaller where that lets a slice fit; more blocks a row where nothing else does.
    long long size = 1;
    auto chunk = [&]() { return size * kDgThreads; };
    auto need = [&]() { return (slice() + chunk() - 1) / chunk(); };
    auto fit = [&]() {
        const long long rows = (slice() + kDgThreads - 1) / kDgThreads;
        for (long long n = (rows + kDgBatch - 1) / kDgBatch; n <= kDgRing; ++n) {
            size = (rows + n - 1) / n;
            if (!whole || need() * chunk() <= budget) return true;
        }
        size = kDgBatch / 2;
        return false;
    };
    while (!fit() && q.cl < kLgMaxCluster) q.cl *= 2;
    q.ring.chunk = (int)chunk();
    q.ring.slots = (int)std::min({budget / chunk(), 4 * need(), (long long)kDgRing});
    q.ring.whole = need() <= q.ring.slots;
    q.ring.rows = p.R;
    q.ring.status = p.dev_status;
    q.smem = (size_t)q.ring.slots * chunk() * 16 + extra;
    return q;
}

// What a kernel has been told about the devices: its shared-memory limit, and
// how many clusters of a configuration fit at once (the last one asked for, on a
// device).
struct DgKernelState {
    std::atomic<unsigned long long> attr_set{0};
    std::atomic<unsigned long long> fits{0};  // dynamic shared memory << 32 | device << 16 | clusters
};

template <bool BF16, bool FORWARD, int CL, int BATCH>
int launch_grad(const LogitsProblem& p, const DistillArgs& a, const DgPlan& q) {
    static DgKernelState state;
    const auto kern = distill_grad_kernel<BF16, FORWARD, CL, BATCH>;
    if (ensure_smem_attr(state.attr_set, kern, kDgSmem) != LIN_OK) return LIN_ERR_CUDA;
    long long clusters = std::max(1, 2 * p.sm_count / CL);
    if (CL > 1 && p.R > 1) {
        // Clusters stay within a part of the SMs, so fewer may fit: a block of a
        // second wave would take its share of the rows after all others are done.
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return LIN_ERR_CUDA;
        const unsigned long long asked = ((unsigned long long)q.smem << 16 | (unsigned)(dev & 0xFFFF)) << 16;
        const unsigned long long known = state.fits.load(std::memory_order_relaxed);
        int fit = (int)(known & 0xFFFFu);
        if ((known ^ asked) >> 16 != 0) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)(clusters * CL));
            cfg.blockDim = dim3(kDgAll);
            cfg.dynamicSmemBytes = q.smem;
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = CL;
            attr.val.clusterDim.y = 1;
            attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&fit, kern, &cfg) != cudaSuccess) return LIN_ERR_CUDA;
            fit = std::min(fit, 0xFFFF);
            state.fits.store(asked | (unsigned)fit, std::memory_order_relaxed);
        }
        clusters = std::min(clusters, (long long)std::max(1, fit));
    }
    return lg_launch(kern, std::min(clusters, p.R) * CL, kDgAll, q.smem, CL, p, a, q.ring);
}

template <int CL, int BATCH>
int launch_grad_of(const LogitsProblem& p, const DistillArgs& a, const DgPlan& q) {
    const bool forward = p.lse_in == nullptr;
    if (p.bf16)
        return forward ? launch_grad<true, true, CL, BATCH>(p, a, q) : launch_grad<true, false, CL, BATCH>(p, a, q);
    return forward ? launch_grad<false, true, CL, BATCH>(p, a, q) : launch_grad<false, false, CL, BATCH>(p, a, q);
}

}  // namespace

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
    a.c = (float)(1.4426950408889634 / p.tau);
    a.inv_tau = 1.0f / p.tau;
    a.weight = p.weight;
    a.lse_in = p.lse_in;
    a.loss = p.loss;
    a.lse = p.lse;
    a.dz = p.dz;
    a.ldd = p.ldd;
    const size_t entries = (size_t)lg_padded(p.K) * 12;
    if (p.dz == nullptr)
        return lg_by_cluster(lg_cluster(p, kDfThreads, 8), [&](auto cl) {
            constexpr int CL = decltype(cl)::value;
            return p.bf16 ? lg_launch(distill_loss_kernel<true, CL>, p.R * CL, kDfThreads, entries, CL, p, a)
                          : lg_launch(distill_loss_kernel<false, CL>, p.R * CL, kDfThreads, entries, CL, p, a);
        });
    const DgPlan q = dg_plan(p, p.lse_in == nullptr, kDgRows * entries);
    return lg_by_cluster(q.cl, [&](auto cl) {
        constexpr int CL = decltype(cl)::value;
        return q.ring.chunk <= kDgSmallBatch * kDgThreads ? launch_grad_of<CL, kDgSmallBatch>(p, a, q)
                                                          : launch_grad_of<CL, kDgBatch>(p, a, q);
    });
}

}  // namespace lin

// Attention of few new tokens (single ones, short drafts) over a paged cache: tiles of
// up to 16 rows (token, query head of one key head).
//
//   s_rj = (q_r . k_j) scale,  out_r = sum_j exp(s_rj - m) v_j / sum_j exp(s_rj - m)
//
// over the keys j that row r sees, with the running maximum and sum of a softmax.
// Memory bounds it: a key and its value are 4 D bytes and are used for 4 D G flops a
// token, so that K and V should stream once, whatever the products run on. A
// block holds a ring of units of 64 keys, filled by TMA through a 4-D map of the pages
// (element, slot, head, page), one box per page (each of the producer warp's lanes
// looks up and issues its own), 64 columns wide with the 128-byte swizzle. Two
// blocks an SM keep about 190 KB of copies in flight.
//
// Few rows: the products are mma.sync with the rows as M = 16 (tcgen05's least M, 64, and
// its trip through TMEM would cost a chain of waits for every unit and save nothing
// where memory is the bound). Each of the four warps takes 16 of the unit's 64 keys and
// keeps its own maxima, totals and sums O (rows x D) in registers, so that no warp waits
// for another until the item ends; P stays in registers, the accumulators of S being
// the A operand of P V, rounded to bf16 (the error against 64 bits is 0.0018 of the norm, 0.0017 of it the output's
// rounding). At the item's end the four sums are joined in the unit's shared memory.
//
// Measured (GB300, with the joining kernel): 64 sequences of 100 to 8000 keys, 32 heads of 128 on 8,
// pages of 16: 159 us, 6.6 TB/s (up to 164 on another board; DRAM reads what is needed, issue slots 28 %); 2 of 131072 keys, 16
// heads of 128 on 2: 49 us, 5.4 TB/s, of which this kernel 45; one of 1000 keys, 12 heads of 64: 7.9 us.
#include <math.h>

#include "paged.cuh"

namespace lin {
namespace {

constexpr int kPrWarps = 4;                        // consumer warps
constexpr int kPrThreads = 32 * (kPrWarps + 1);    // and the producer
constexpr int kPrKeys = 16 * kPrWarps;             // keys of a unit

constexpr int kPrRows = kPagedRowsMax;             // rows of a tile
static_assert(kPrRows == 16, "the products' M");

template <int D>
struct PrShape {
    static constexpr uint32_t kK = kPrKeys * D * 2, kQ = kPrRows * D * 2, kStage = 2 * kK + kQ;
    static constexpr int kRoom = 111 * 1024 / (int)kStage, S = kRoom < 6 ? kRoom : 6;  // two blocks an SM
    static constexpr size_t kSmem = 1024 + S * kStage;
};

struct PrUnit {       // what the consumers have to know of a unit
    int key0;         // first key
    int seen;         // keys that some row of the tile sees
    int first, last;  // of this block's part of the item
    int row0, tokens; // the tile's rows of q
    int h;
    int pos0;         // position of its first token
    int slot;         // the workspace's slot, or -1: the item is whole
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// D (16 x 8 fp32) += A (16 x 16) B (16 x 8), bf16.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float pr_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int D>
__global__ void __launch_bounds__(kPrThreads, 2)
paged_rows_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const PagedArgs a) {
    using P = PrShape<D>;
    constexpr int R = kPrRows, S = P::S, HALVES = D / 64;
    extern __shared__ uint8_t raw[];
    __shared__ alignas(8) uint64_t bars[2 * S + 1];
    __shared__ PrUnit units[S];
    __shared__ float2 s_stat[2][kPrWarps][R];
    __shared__ int s_abort;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * S, join = empty0 + 8 * S;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, kPrWarps);
        }
        mbar_init(join, kPrWarps);
        s_abort = 0;
        mbar_fence_init();
        tma_prefetch_map(&tmQ);
        tma_prefetch_map(&tmK);
        tma_prefetch_map(&tmV);
    }
    pdl_wait();
    pdl_launch_dependents();
    const PagedStretch r = paged_stretch<kPrKeys, kPrThreads>(a);  // syncs the block

    auto give_up = [&]() {
        atomicExch(&s_abort, 1);
        atomicExch(a.status, (int)LIN_ERR_DEVICE_TIMEOUT);
    };
    auto aborted = [&]() { return *(volatile int*)&s_abort != 0; };

    if (warp == kPrWarps) {
        // ---- producer: the whole warp walks the stretch ----
        PagedCut cut = {0, 0, 0, 0};
        uint32_t g = 0;
        bool ok = true;
        {
            const PagedBox<kPrKeys> box(a);
            const int half = box.group % HALVES, isv = box.group / HALVES;
            const uint32_t q_bytes = (uint32_t)(a.TQ * a.G) * D * 2;
            uint32_t s = 0, ph = 1;
            PagedWalk<kPrKeys> w;
            w.start(a, r);
            for (int j0, k; ok && w.part(a, j0, k); w.next(a, k)) {
                const int seen = tile_seen(a, w.q, w.t);
                const int row0 = w.q.row0 + w.t * a.TQ, tokens = min(a.TQ, w.q.n - w.t * a.TQ);
                const int slot = k == w.n ? -1 : 2 * (int)blockIdx.x + (j0 == 0 ? 1 : 0);
                if (j0 == 0 && k < w.n) cut = {row0, tokens, w.h, w.last_block(r.per)};
                const int* table = a.batch.block_table + w.b * a.batch.table_stride;
                int key0 = j0 * kPrKeys, next = box.entry(a, table, key0, seen);
                for (int i = 0; i < k; ++i, key0 += kPrKeys) {
                    const int entry = next;
                    if (i + 1 < k) next = box.entry(a, table, key0 + kPrKeys, seen);
                    if (!__all_sync(0xffffffffu, !aborted() && mbar_wait(empty0 + 8 * s, ph))) {
                        ok = false;
                        break;
                    }
                    uint8_t* stage = smem + s * P::kStage;
                    if (lane == 0) {
                        units[s] = PrUnit{key0, seen, i == 0, i == k - 1, row0, tokens, w.h, w.q.pos0 + w.t * a.TQ, slot};
                        mbar_expect_tx(full0 + 8 * s,
                                       (uint32_t)(box.count(key0, seen) * HALVES * 2) * (128u << box.shift) + (i == 0 ? q_bytes : 0));
                    }
                    __syncwarp();
                    if (isv < 2 && box.holds(key0, seen))
                        tma_load_4d(smem_u32(stage + isv * P::kK + half * (kPrKeys * 128) + ((box.at << box.shift) * 128)),
                                    isv ? &tmV : &tmK, full0 + 8 * s, 64 * half, box.slot(a, key0), w.h, box.page(a, entry));
                    if (i == 0 && lane < HALVES)
                        tma_load_3d(smem_u32(stage + 2 * P::kK + lane * (R * 128)), &tmQ, full0 + 8 * s, 64 * lane,
                                    w.h * a.G, row0);
                    ++g;
                    if (++s == S) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
        }
        if (lane == 0) a.cuts[blockIdx.x] = cut;
        if (!ok) {
            if (lane == 0) give_up();
            // the copies in flight land before the block ends
            for (uint32_t n = g > (uint32_t)S ? g - S : 0; n < g; ++n) mbar_wait(full0 + 8 * (n % S), (n / S) & 1);
        }
        return;
    }

    // ---- consumers: warp w has keys 16 w .. 16 w + 15 of each unit ----
    float m[2], l[2], o[D / 8][4];
    uint32_t qf[D / 16][4];
    int lim[2];            // keys that this lane's rows see
    uint32_t joins = 0, items = 0;
    bool ok = true;
    const int r8 = lane & 7;
    // Wait for all consumer warps (bounded, unlike a block barrier).
    auto all_warps = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(join);
        return __all_sync(0xffffffffu, !aborted() && mbar_wait(join, joins++ & 1));
    };
    const int stretch = (int)(r.hi - r.lo);
    uint32_t s = 0, ph = 0;
    for (int g = 0; g < stretch; ++g) {
        if (!__all_sync(0xffffffffu, !aborted() && mbar_wait(full0 + 8 * s, ph))) {
            ok = false;
            break;
        }
        const PrUnit u = units[s];
        uint8_t* stage = smem + s * P::kStage;
        const uint32_t sk = smem_u32(stage), sv = sk + P::kK, sq = sk + 2 * P::kK;
        if (u.first) {
            const int row = ((lane >> 3) & 1) * 8 + r8;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const int chunk = (2 * kk + (lane >> 4)) & 7;
                ldsm4(sq + (kk >> 2) * (R * 128) + row * 128 + ((chunk ^ (row & 7)) << 4), qf[kk]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[e] = -INFINITY;
                l[e] = 0.f;
                const int tok = ((lane >> 2) + 8 * e) / a.G;
                lim[e] = a.causal ? min(u.pos0 + tok + 1, u.seen) : u.seen;
            }
#pragma unroll
            for (int d = 0; d < D / 8; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
        }
        const int k0 = u.key0 + 16 * warp;
        bool zeroed = false;
        if (k0 < u.seen) {
            if (k0 + 16 > u.seen) {
                // keys that nobody sees: their values (a page's slots that were never
                // written) must not meet a probability of 0 as NaN
                const int bad = k0 + 16 - u.seen;
                for (int i = lane; i < bad * (D / 8); i += 32) {
                    const int row = 16 * warp + 16 - bad + i / (D / 8), c = i % (D / 8);
                    *reinterpret_cast<uint4*>(stage + P::kK + (c >> 3) * (kPrKeys * 128) + row * 128 + ((c & 7) << 4)) =
                        make_uint4(0, 0, 0, 0);
                }
                zeroed = true;
                __syncwarp();
            }
            float sc[2][4] = {};
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t kf[4];
                const int key = 16 * warp + (lane >> 4) * 8 + r8, chunk = (2 * kk + ((lane >> 3) & 1)) & 7;
                ldsm4(sk + (kk >> 2) * (kPrKeys * 128) + key * 128 + ((chunk ^ r8) << 4), kf);
                mma16816(sc[0], qf[kk], kf[0], kf[1]);
                mma16816(sc[1], qf[kk], kf[2], kf[3]);
            }
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = k0 + nt * 8 + 2 * (lane & 3) + (e & 1);
                    float& x = sc[nt][e];
                    x = key < lim[e >> 1] ? x * a.scale_log2 : -INFINITY;
                    mx[e >> 1] = fmaxf(mx[e >> 1], x);
                }
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
                const float now = fmaxf(m[e], mx[e]);
                const float base = now == -INFINITY ? 0.f : now;
                alpha[e] = pr_ex2(m[e] - base);
                m[e] = now;
                float sum = 0.f;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        float& x = sc[nt][2 * e + f];
                        x = pr_ex2(x - base);
                        sum += x;
                    }
                l[e] = fmaf(l[e], alpha[e], sum);
            }
            const uint32_t pf[4] = {pack_bf16x2(sc[0][0], sc[0][1]), pack_bf16x2(sc[0][2], sc[0][3]),
                                    pack_bf16x2(sc[1][0], sc[1][1]), pack_bf16x2(sc[1][2], sc[1][3])};
            if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
                for (int d = 0; d < D / 8; ++d)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[d][e] *= alpha[e >> 1];
            }
#pragma unroll
            for (int dd = 0; dd < D / 16; ++dd) {
                uint32_t vf[4];
                const int key = 16 * warp + ((lane >> 3) & 1) * 8 + r8, chunk = (2 * dd + (lane >> 4)) & 7;
                ldsm4_t(sv + (dd >> 2) * (kPrKeys * 128) + key * 128 + ((chunk ^ r8) << 4), vf);
                mma16816(o[2 * dd], pf, vf[0], vf[1]);
                mma16816(o[2 * dd + 1], pf, vf[2], vf[3]);
            }
        }
        if (u.last) {
            // ---- the item's end here: the warps' sums at one maximum, joined in the stage ----
            float2(&stat)[kPrWarps][R] = s_stat[items & 1];
            ++items;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if ((lane & 3) == 0) stat[warp][(lane >> 2) + 8 * e] = make_float2(m[e], sum);
            }
            if (!all_warps()) {  // the stage's keys and values have been read, too
                ok = false;
                break;
            }
            float* part = reinterpret_cast<float*>(stage);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = (lane >> 2) + 8 * e;
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kPrWarps; ++w) top = fmaxf(top, stat[w][row].x);
                const float f = pr_ex2(m[e] - (top == -INFINITY ? 0.f : top));
#pragma unroll
                for (int d = 0; d < D / 8; ++d)  // groups of 8 columns swizzled by the row: no two lanes on a bank
                    *reinterpret_cast<float2*>(part + (warp * 16 + row) * D + ((d ^ (row & 7)) << 3) + 2 * (lane & 3)) =
                        make_float2(o[d][2 * e] * f, o[d][2 * e + 1] * f);
            }
            if (!all_warps()) {
                ok = false;
                break;
            }
            for (int i = threadIdx.x; i < 16 * D / 4; i += 32 * kPrWarps) {
                const int row = i / (D / 4), col = 4 * (i % (D / 4));
                if (row >= u.tokens * a.G) break;
                float top = -INFINITY, total = 0.f;
#pragma unroll
                for (int w = 0; w < kPrWarps; ++w) top = fmaxf(top, stat[w][row].x);
                const float base = top == -INFINITY ? 0.f : top;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kPrWarps; ++w) {
                    const float2 st = stat[w][row];
                    total = fmaf(st.y, pr_ex2(st.x - base), total);
                    const float4 x = *reinterpret_cast<const float4*>(
                        part + (w * 16 + row) * D + (((col >> 3) ^ (row & 7)) << 3) + (col & 7));
                    v.x += x.x;
                    v.y += x.y;
                    v.z += x.z;
                    v.w += x.w;
                }
                if (u.slot < 0) {
                    const bool none = total == 0.f;  // a row without keys is 0
                    const float inv = 1.f / total;
                    const int tok = row / a.G, head = u.h * a.G + row - tok * a.G;
                    *reinterpret_cast<uint2*>(a.out + (size_t)(u.row0 + tok) * a.ldo + (size_t)head * D + col) =
                        make_uint2(none ? 0u : pack_bf16x2(v.x * inv, v.y * inv), none ? 0u : pack_bf16x2(v.z * inv, v.w * inv));
                    if (a.lse && col == 0) a.lse[(size_t)(u.row0 + tok) * (a.Hkv * a.G) + head] = row_lse(top, total);
                } else {
                    *reinterpret_cast<float4*>(a.sums + ((size_t)u.slot * R + row) * D + col) = v;
                    if (col == 0) a.stats[(size_t)u.slot * R + row] = make_float2(top, total);
                }
            }
            zeroed = true;
        }
        if (zeroed) fence_proxy_async_smem();  // written here, then by the next copy
        __syncwarp();
        if (lane == 0) mbar_arrive(empty0 + 8 * s);
        if (++s == S) {
            s = 0;
            ph ^= 1;
        }
    }
    if (!ok && lane == 0) give_up();
}

template <int D>
int start(const PagedProblem& p) {
    using P = PrShape<D>;
    constexpr int R = kPrRows;
    const int grid = 2 * p.sm_count;
    PagedArgs a;
    if (!paged_args(p, grid, R, &a)) return LIN_ERR_WORKSPACE;
    CUtensorMap tq, tk, tv;
    if (!paged_q_map(&tq, p, a.TQ) || !paged_kv_map(&tk, p, p.cache.k, kPrKeys) || !paged_kv_map(&tv, p, p.cache.v, kPrKeys))
        return LIN_ERR_CUDA;
    static std::atomic<unsigned long long> attr_set{0};
    if (ensure_smem_attr(attr_set, paged_rows_kernel<D>, P::kSmem) != LIN_OK) return LIN_ERR_CUDA;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kPrThreads);
    cfg.dynamicSmemBytes = P::kSmem;
    cfg.stream = p.stream;
    cfg.attrs = &attr;
    cfg.numAttrs = p.early_start ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, paged_rows_kernel<D>, tq, tk, tv, a) != cudaSuccess) return LIN_ERR_CUDA;
    if (cudaGetLastError() != cudaSuccess) return LIN_ERR_CUDA;
    return launch_paged_join(p, a, grid, R);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

}  // namespace

bool paged_kv_map(CUtensorMap* map, const PagedProblem& p, const void* base, int keys) {
    auto fn = encode_fn();
    if (!fn) return false;
    const lin_kv_cache& c = p.cache;
    const cuuint64_t D = c.head_dim;
    cuuint64_t dims[4] = {D, (cuuint64_t)c.page_size, (cuuint64_t)c.heads, (cuuint64_t)c.pages};
    // the strides of a single head or page do not matter; they have to be valid
    const cuuint64_t token = (cuuint64_t)c.token_stride * 2;
    cuuint64_t strides[3] = {token, c.heads > 1 ? (cuuint64_t)c.head_stride * 2 : token,
                             c.pages > 1 ? (cuuint64_t)c.page_stride * 2 : token};
    cuuint32_t box[4] = {64, (cuuint32_t)(c.page_size < keys ? c.page_size : keys), 1, 1};
    cuuint32_t one[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool paged_q_map(CUtensorMap* map, const PagedProblem& p, int tokens) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t D = p.cache.head_dim;
    cuuint64_t dims[3] = {D, (cuuint64_t)p.H, (cuuint64_t)p.batch.tokens};
    cuuint64_t strides[2] = {D * 2, (cuuint64_t)p.ldq * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)(p.H / p.cache.heads), (cuuint32_t)tokens};
    cuuint32_t one[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.q), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool paged_args(const PagedProblem& p, int grid, int R, PagedArgs* a) {
    const int D = p.cache.head_dim;
    if (paged_workspace(grid, R, D) > p.workspace_bytes) return false;
    a->batch = p.batch;
    a->pages = p.cache.pages;
    a->page_size = p.cache.page_size;
    a->page_shift = 0;
    while ((1 << a->page_shift) < p.cache.page_size) ++a->page_shift;
    a->Hkv = p.cache.heads;
    a->G = p.H / p.cache.heads;
    a->TQ = R / a->G;
    a->causal = p.causal ? 1 : 0;
    a->lead = 0;
    a->scale_log2 = p.scale * 1.4426950408889634f;
    a->out = static_cast<uint16_t*>(p.out);
    a->ldo = p.ldo;
    a->lse = p.lse;
    uint8_t* ws = static_cast<uint8_t*>(p.workspace);
    a->cuts = reinterpret_cast<PagedCut*>(ws);
    ws += align_up(sizeof(PagedCut) * (size_t)grid, 256);
    a->sums = reinterpret_cast<float*>(ws);
    a->stats = reinterpret_cast<float2*>(ws + (size_t)grid * 2 * R * D * sizeof(float));
    a->status = p.dev_status;
    return true;
}

size_t paged_rows_workspace(int sm_count, int D) { return paged_workspace(2 * sm_count, kPrRows, D); }

int launch_paged_rows(const PagedProblem& p) { return p.cache.head_dim == 64 ? start<64>(p) : start<128>(p); }

}  // namespace lin

// Backward pass of the fused self-attention, in the forward's layouts: from
// qkv ((B*T) x 3C), the forward's out and dout ((B*T) x C) and lse (B x H x T)
// it writes dqkv ((B*T) x 3C). The probabilities are rebuilt from lse, so the
// score matrix reaches memory in neither direction ("Writing a CUDA matmul that
// catches cuBLAS", section "Fusing attention: the score matrix never exists"):
//
//   s_ij  = (q_i . k_j) scale,   p_ij = exp(s_ij - lse_i)   (0 where masked)
//   delta_i = dout_i . out_i     (= sum_j p_ij dp_ij)
//   dv_j  = sum_i p_ij dout_i,   dp_ij = dout_i . v_j
//   ds_ij = p_ij (dp_ij - delta_i)
//   dq_i  = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i
//
// For one block of 128 keys and one of 128 queries these are five products of
// 128 x 128 x 64 on the tensor cores, scores transposed (keys on the TMEM lanes):
//   S'  = K Q',  dP' = V dO'      operands in shared memory as they were loaded
//   dV += P' dO                   P' (bf16) from TMEM, dO read MN-major
//   dK += dS' Q                   dS' (bf16) in shared memory, read K-major,
//   dQ  = dS K                    and the same tile read MN-major as dS
// With the keys on the lanes P' needs no trip through shared memory, whose
// bandwidth the five products' operands otherwise exceed. For the same reason lse
// and delta are not read by the threads (one value for all lanes costs shared
// memory as much as 32): S' and dP' have one more step of 16, in which a row of
// ones meets -lse / scale and -delta of the queries, each split into three bf16
// parts that carry 24 bits. What the threads read from TMEM is then
//   (s_ij - lse_i) / scale   and   dp_ij - delta_i.
//
// Sequences of one block (T <= 128): attn_bwd_short_kernel, a block per
// (sequence, head), two blocks an SM so that one's loads and stores run under the
// other's products and exponentials.
//
// Longer ones: three kernels:
//   attn_bwd_prep    delta and lse, a row of eight bf16 a query, padded to whole
//                    blocks of 128 queries.
//   attn_bwd_kernel  a persistent block per SM draws work items (sequence, head,
//                    block of 128 keys) by a ticket; an item walks the query blocks
//                    that see its keys, with dk and dv accumulating in TMEM. dq is
//                    summed over the key blocks in fp32 in the workspace.
//   attn_bwd_dq      the fp32 sums to bf16.
//
// attn_bwd_kernel's warps: 0 TMA; 1 tcgen05.mma issuer; 2 and 3 send what is staged
// for memory; 4-19 four groups that turn S' and dP' into P' and dS' (a thread has one
// key and 32 of the block's queries); 20-23 dQ out of TMEM, and dK and dV at an
// item's end. When P'(n) is written, S'(n+1), dV and dP'(n+1) are issued and run while
// dS'(n) is formed; dK and dQ of step n run under the exponentials of step n+1. A step
// has three commits (S', dV with the next dP', dK with dQ); what else waits for products
// is told by the warps that saw them.
//
// Order of the dq sums: the key blocks of a head form `chains` chains (block j in
// chain j % chains), each with its own fp32 copy of dq; within a chain block j
// adds to a tile after block j - chains has (a counter per tile, waited for). The
// sums' order is thus fixed, results are repeatable bit for bit whichever block has an
// item, and a wait is only ever for an item that was drawn earlier, by a block that
// runs. A tile is added by one bulk reduction from shared memory, whose completion is
// looked for a step later. Every wait is bounded (about 1 s); a block that gives up sets
// the device status word.
//
// Measured (GB300): 64 sequences of 128, 12 heads, causal 29 us (3.5 TB/s of
// operands); 2 of 4096 202 us (640 TF/s of the visible pairs' products), of which
// attn_bwd_kernel about 170 (profiled alone); a step takes 2700 cycles when nothing
// waits, 1660 of them products. Tensor pipe 37 % active, DRAM 6 %: bound by the
// steps' chain of products, exponentials and additions. T <= 128: DRAM 28 %, tensor
// pipe 15 %: bound by the latency of a block's own chain, two blocks an SM.
#include <math.h>

#include <algorithm>

#include "device_common.cuh"
#include "internal.h"
#include "tc_common.cuh"

namespace lin {
namespace {

constexpr int kAbB = 128;                          // keys, and queries, of a block
constexpr int kAbD = 64;                           // head width
constexpr int kAbGroups = 4;                       // groups of four warps that make P' and dS', 32 queries each
constexpr int kAbThreads = 128 * (kAbGroups + 2);
constexpr uint32_t kAbTile = kAbB * kAbD * 2;      // 16 KiB: 128 rows of 128 bytes, 128-byte swizzle
constexpr uint32_t kAbStat = kAbB * 16;            // eight bf16 of 128 queries: -lse / scale and -delta, in three parts each
constexpr uint32_t kAbOnes = 512;                  // the rows that meet them
constexpr int kAbKStages = 2, kAbQStages = 3;      // (V has one)
constexpr uint32_t kAbQStage = 2 * kAbTile + kAbStat;
constexpr int kAbItems = 4;                        // work items between the ticket and the last role that takes them
constexpr uint32_t kAbDs = kAbB * kAbB * 2;        // dS': two 64-query K-major blocks of 16 KiB
constexpr uint32_t kAbDqTile = kAbB * kAbD * 4;    // fp32 dq of a query block: [column / 4][row][4]
constexpr int kAbBars = 2 * kAbKStages + 2 + 2 * kAbQStages + 10 + 2 * kAbItems;
constexpr size_t kAbSmem = 1024 + (kAbKStages + 1) * kAbTile + kAbQStages * kAbQStage + kAbDs + kAbDqTile + kAbOnes +
                           kAbBars * 8 + kAbItems * 8 + 16;
static_assert(kAbSmem <= 227 * 1024, "shared memory");
// TMEM columns
constexpr uint32_t kAbS = 0, kAbDp = 128, kAbDv = 256, kAbDk = 320, kAbDq = 384, kAbP = 448, kAbTmem = 512;
// and of the short kernel, where dV and dK take dP's place and dQ half of S's
constexpr int kAsThreads = 256;
constexpr uint32_t kAsP = 0, kAsDq = 64, kAsDp = 128, kAsDv = 128, kAsDk = 192, kAsTmem = 256;
constexpr size_t kAsSmem = 1024 + 4 * kAbTile + kAbDs + kAbStat + kAbOnes + 6 * 8 + 16;
static_assert(2 * (kAsSmem + 1024) <= 228 * 1024, "two blocks an SM");
// Register split (setmaxnreg, per warpgroup): launched at 80 a thread; the groups that
// hold 32 probabilities and 32 dp a thread take what the others give back.
constexpr int kAbLaunchRegs = 80, kAbRegsIssue = 64, kAbRegsSoftmax = 88, kAbRegsOut = 64;
static_assert(kAbRegsIssue + kAbGroups * kAbRegsSoftmax + kAbRegsOut <= (kAbGroups + 2) * kAbLaunchRegs, "register split");
constexpr float kAbLog2e = 1.4426950408889634f;

struct AbArgs {
    int T, H, C;
    int nb;              // blocks of 128 in a sequence
    int bh0, heads;      // the launch's (sequence, head) pairs: bh0 .. bh0 + heads - 1
    int items;           // heads * nb
    int chains;
    int ahead;           // blocks that run at once (short kernel)
    int causal;
    float scale, scale_log2, inv_scale;
    unsigned* ticket;    // the next item, counted by the blocks that run
    const uint4* stats;  // heads x nb x 128
    unsigned* flags;     // heads x chains x nb
    float* dq;           // heads x chains x nb tiles
    int* status;
};

__device__ __forceinline__ float ab_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t ab_pack(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void ab_unpack(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t ab_mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// 128 tokens x 64 columns of a (B, T, columns) tensor; tokens past T read as zero.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void ab_prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void ab_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
// Untiled copy; addresses and size are multiples of 16 bytes.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// True in one lane. The issuing warp runs its loop whole and issues inside such a
// branch, which the compiler knows to be one thread's: descriptors stay in uniform
// registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e != 0;
}
// D (+)= A B with A (bf16, two to a 32-bit column) in TMEM.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
constexpr uint32_t kIdescS = make_idesc(1u, kAbB, kAbB);                  // both K-major
constexpr uint32_t kIdescDkv = make_idesc(1u, kAbB, kAbD, false, true);   // A K-major (or TMEM), B MN-major
constexpr uint32_t kIdescDq = make_idesc(1u, kAbB, kAbD, true, true);     // both MN-major
// 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void ab_tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The dS' tile read MN-major (rows are keys = K, 64-query chunks 16 KiB apart).
__device__ __forceinline__ uint64_t ab_ds_mn_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((kAbDs / 2) >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}
// A tile of the workspace from shared memory: stored, or added to what is there.
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_add_f32(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.reduce.async.bulk.global.shared::cta.bulk_group.add.f32 [%0], [%1], %2;" ::"l"(dst), "r"(src),
                 "r"(bytes)
                 : "memory");
}
// Wait until this thread's bulk operations have completed, not only read their source.
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- one thread's key and 32 of the block's queries ----

// p = 2^(s scale log2(e)), s less lse / scale already.
__device__ __forceinline__ void ab_probs(const uint32_t (&s)[32], uint64_t sl2, uint64_t (&p)[16]) {
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        float x0, x1;
        ab_unpack(ab_mul2(ab_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sl2), x0, x1);
        p[c] = ab_pack(ab_ex2(x0), ab_ex2(x1));
    }
}
// Only queries from `from` on see the key.
__device__ __forceinline__ void ab_hide(uint64_t (&p)[16], int from) {
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        float x0, x1;
        ab_unpack(p[c], x0, x1);
        p[c] = ab_pack(2 * c >= from ? x0 : 0.f, 2 * c + 1 >= from ? x1 : 0.f);
    }
}
// P' in bf16 to 16 columns of TMEM.
__device__ __forceinline__ void ab_put_p(uint32_t taddr, const uint64_t (&p)[16]) {
    uint32_t pk[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        float x0, x1;
        ab_unpack(p[c], x0, x1);
        pk[c] = pack_bf16x2(x0, x1);
    }
    tmem_st16(taddr, pk);
}
// ds = p dp (dp less delta already) in bf16 to pieces `first`.. of the thread's row
// of dS'. MASKED: a hidden pair takes nothing from dp, whatever it is.
template <bool MASKED>
__device__ __forceinline__ void ab_put_ds(const uint32_t (&dp)[32], const uint64_t (&p)[16], uint8_t* ds_row, int r,
                                          int first, int from) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        uint32_t pk[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = 8 * v + 2 * k;
            float x0, x1;
            ab_unpack(ab_mul2(p[c / 2], ab_pack(__uint_as_float(dp[c]), __uint_as_float(dp[c + 1]))), x0, x1);
            if constexpr (MASKED) {
                x0 = c >= from ? x0 : 0.f;
                x1 = c + 1 >= from ? x1 : 0.f;
            }
            pk[k] = pack_bf16x2(x0, x1);
        }
        *reinterpret_cast<uint4*>(ds_row + (((first + v) ^ (r & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    }
}
// 8 * N fp32 values, scaled, in bf16 to pieces `first`.. of row r of a 128-byte-swizzled tile.
template <int N>
__device__ __forceinline__ void ab_stage(uint8_t* tile, int r, int first, const uint32_t* v, float f) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const uint32_t* x = v + 8 * k;
        *reinterpret_cast<uint4*>(tile + r * 128 + (((first + k) ^ (r & 7)) << 4)) =
            make_uint4(pack_bf16x2(__uint_as_float(x[0]) * f, __uint_as_float(x[1]) * f),
                       pack_bf16x2(__uint_as_float(x[2]) * f, __uint_as_float(x[3]) * f),
                       pack_bf16x2(__uint_as_float(x[4]) * f, __uint_as_float(x[5]) * f),
                       pack_bf16x2(__uint_as_float(x[6]) * f, __uint_as_float(x[7]) * f));
    }
}

// Statistics of 128 queries of one head by 256 threads (two a query), a row of
// eight bf16 each: -lse / scale (far below everything past the sequence's end and
// for a query that sees no key: probability 0) and -delta, in three parts.
__device__ __forceinline__ void ab_stats(const uint16_t* out, const uint16_t* dout, const float* lse, int T, int H,
                                         int b, int h, int i, float inv_scale, uint4* st) {
    const int row = threadIdx.x >> 1, half = threadIdx.x & 1;
    const int t = i * kAbB + row;
    float sum = 0.f;
    if (t < T) {
        const size_t off = ((size_t)b * T + t) * ((size_t)H * kAbD) + h * kAbD + 32 * half;
        uint4 o[4], g[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            o[k] = *reinterpret_cast<const uint4*>(out + off + 8 * k);
            g[k] = *reinterpret_cast<const uint4*>(dout + off + 8 * k);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t x[4] = {o[k].x, o[k].y, o[k].z, o[k].w}, y[4] = {g[k].x, g[k].y, g[k].z, g[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sum = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(y[e] << 16), sum);
                sum = fmaf(__uint_as_float(x[e] & 0xFFFF0000u), __uint_as_float(y[e] & 0xFFFF0000u), sum);
            }
        }
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    if (half == 0) {
        // finite, so that it is 0 where it meets a 0, and 0 as a probability: e scale <= -256
        const float far = -fmaxf(1e30f, 256.f * inv_scale);
        const float l = t < T ? lse[((size_t)b * H + h) * T + t] : -INFINITY;
        const float e = l == -INFINITY || l == INFINITY ? far : -l * inv_scale;
        const float e0 = bf16_bits_to_f32(f32_to_bf16_bits(e)), e1 = bf16_bits_to_f32(f32_to_bf16_bits(e - e0));
        const bool cut = e == far;
        if (cut) sum = 0.f;  // its out may be anything, a 0 / 0 as well
        const float d0 = bf16_bits_to_f32(f32_to_bf16_bits(-sum)), d1 = bf16_bits_to_f32(f32_to_bf16_bits(-sum - d0));
        st[row] = make_uint4(pack_bf16x2(e0, cut ? 0.f : e1), pack_bf16x2(cut ? 0.f : (e - e0) - e1, d0),
                             pack_bf16x2(d1, (-sum - d0) - d1), 0u);
    }
}
// The rows that meet them: ones in places 0-2 (lse) and 3-5 (delta). Eight equal
// rows and eight of zeros stand for all 128 (the descriptor's strides are 0).
__device__ __forceinline__ void ab_ones(uint4* ones) {
    const int i = threadIdx.x;
    if (i < 32) {
        const bool rows = (i & 8) == 0;
        ones[i] = !rows    ? make_uint4(0u, 0u, 0u, 0u)
                  : i < 16 ? make_uint4(0x3F803F80u, 0x00003F80u, 0u, 0u)
                           : make_uint4(0u, 0x3F800000u, 0x3F803F80u, 0u);
    }
}
// Descriptors without swizzle: 8 x 16-byte cores, `k` bytes apart along K, `mn` along the rows.
__device__ __forceinline__ uint64_t ab_flat_desc(uint32_t saddr, uint32_t k, uint32_t mn) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(k >> 4) << 16;
    d |= static_cast<uint64_t>(mn >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    return d;
}
// S' and dP' with their extra step. The second half of its K is zero on the ones'
// side, so the statistics' side may repeat its first half there.
__device__ __forceinline__ void ab_mma_scores(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t ones, uint32_t stat) {
    const uint64_t ad = sw128_kmajor_desc(a), bd = sw128_kmajor_desc(b);
#pragma unroll
    for (int kk = 0; kk < kAbD / 16; ++kk) tc_mma<true>(d_tmem, ad + 2u * kk, bd + 2u * kk, kIdescS, kk != 0 ? 1u : 0u);
    tc_mma<true>(d_tmem, ab_flat_desc(ones, 128, 0), ab_flat_desc(stat, 0, 128), kIdescS, 1u);
}

__device__ __forceinline__ int2 ab_lds_item(uint32_t addr) {
    int2 x;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ void ab_sts_item(uint32_t addr, int j, int bh) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(j), "r"(bh) : "memory");
}

// A role's place in the block's items. The TMA warp draws them by a ticket and passes
// them on through a ring in shared memory. Items are ordered by key block, then by head
// (their lengths fall along the order when causal), and only a block that runs draws
// one. So an item whose sums another one waits for has started and goes on, whichever
// blocks are resident: with the items dealt out by block index, a block that another
// stream's kernel keeps off its SM held up all the others. Against dealing them out,
// every second round in reverse where chains were many (calls in a CUDA graph): 2 x 4096
// x 12 heads causal 211 -> 200 us, 16 x 4096 x 12 1562 -> 1494, 40 x 256 x 12 61.0 -> 59.4,
// 3 x 777 x 5 full 25.3 both, and 8 x 200 x 12, 192 items of one or two steps whose
// reversed round was even, 17.4 -> 19.8.
struct AbWalker {
    unsigned m = ~0u;  // number of the item within the block
    int j = -1, bh;    // key block (-1 past the last item), launch-local (sequence, head)
    int i;             // query block
    __device__ __forceinline__ void set(const AbArgs& a, int2 x) {
        j = x.x;
        bh = x.y;
        i = first(a);
    }
    __device__ __forceinline__ bool valid() const { return j >= 0; }
    __device__ __forceinline__ int first(const AbArgs& a) const { return a.causal ? j : 0; }
    __device__ __forceinline__ bool last(const AbArgs& a) const { return i == a.nb - 1; }
};

__global__ void __launch_bounds__(kAbThreads, 1)
attn_bwd_kernel(const __grid_constant__ CUtensorMap tmQkv, const __grid_constant__ CUtensorMap tmDo,
                const __grid_constant__ CUtensorMap tmDqkv, const AbArgs a) {
    constexpr int KS = kAbKStages, QS = kAbQStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sK = smem;
    uint8_t* sV = sK + KS * kAbTile;
    uint8_t* sQ = sV + kAbTile;                // stage: Q, dO, statistics
    uint8_t* sDS = sQ + QS * kAbQStage;
    uint8_t* sOut = sDS + kAbDs;               // dq on its way out; dk and dv at an item's end
    uint8_t* sOnes = sOut + kAbDqTile;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sOnes + kAbOnes);
    // (the items' ring lies behind the barriers: key block, -1 for no more, and head)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kAbBars + kAbItems);
    int* s_abort = reinterpret_cast<int*>(tmem_slot + 1);

    // Full / empty of the stages; then, once a step: sfull, dpfull, done (the
    // products of S', of dV and dP', of dK and dQ), pready, dsready (the groups'
    // warps), dqfree, accfree (the four); outfull (the four; of even and of odd
    // messages), outfree (a sender) once a message; full / empty of the items' ring.
    const uint32_t kfull = smem_u32(bars), kempty = kfull + 8 * KS, vfull = kempty + 8 * KS, vempty = vfull + 8,
                   qfull = vempty + 8, qempty = qfull + 8 * QS, one_a_step = qempty + 8 * QS;
    const uint32_t sfull = one_a_step, dpfull = one_a_step + 8, done = one_a_step + 16, pready = one_a_step + 24,
                   dsready = one_a_step + 32, dqfree = one_a_step + 40, accfree = one_a_step + 48,
                   outfull = one_a_step + 56, outfree = one_a_step + 72, ifull = outfree + 8,
                   iempty = ifull + 8 * kAbItems, items = iempty + 8 * kAbItems;

    // (the same in every lane, and known to be: roles branch without divergence)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < KS; ++s) {
            mbar_init(kfull + 8 * s, 1);
            mbar_init(kempty + 8 * s, 4);
        }
        mbar_init(vfull, 1);
        mbar_init(vempty, 4 * kAbGroups);
        for (int s = 0; s < QS; ++s) {
            mbar_init(qfull + 8 * s, 1);
            mbar_init(qempty + 8 * s, 4);
        }
        mbar_init(sfull, 1);
        mbar_init(dpfull, 1);
        mbar_init(done, 1);
        mbar_init(pready, 4 * kAbGroups);
        mbar_init(dsready, 4 * kAbGroups);
        mbar_init(dqfree, 4);
        mbar_init(accfree, 4);
        mbar_init(outfull, 4);
        mbar_init(outfull + 8, 4);
        mbar_init(outfree, 1);
        for (int k = 0; k < kAbItems; ++k) {
            mbar_init(ifull + 8 * k, 1);
            mbar_init(iempty + 8 * k, 1 + 2 + 4 * kAbGroups + 4);  // issuer, senders, the groups' and the last warps
        }
        *s_abort = 0;
        mbar_fence_init();
        tma_prefetch_map(&tmQkv);
        tma_prefetch_map(&tmDo);
        tma_prefetch_map(&tmDqkv);
    }
    ab_ones(reinterpret_cast<uint4*>(sOnes));
    fence_proxy_async_smem();
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), kAbTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    if (threadIdx.x == 0) pdl_launch_dependents();

    auto give_up = [&]() {
        atomicExch(s_abort, 1);
        atomicExch(a.status, (int)LIN_ERR_DEVICE_TIMEOUT);
    };
    // A warp's wait: false when it has run out.
    auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0; };
    auto aborted = [&]() { return __any_sync(0xffffffffu, *(volatile int*)s_abort != 0) != 0; };
    auto arrive = [&](uint32_t bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    // The next item, by a whole warp and by one thread; false when the wait has run out.
    auto take = [&](AbWalker& w) {
        const uint32_t k = ++w.m % kAbItems;
        if (!wait(ifull + 8 * k, (w.m / kAbItems) & 1)) return false;
        w.set(a, ab_lds_item(items + 8 * k));
        arrive(iempty + 8 * k);
        return true;
    };
    auto take_alone = [&](AbWalker& w) {
        const uint32_t k = ++w.m % kAbItems;
        if (!mbar_wait(ifull + 8 * k, (w.m / kAbItems) & 1)) return false;
        w.set(a, ab_lds_item(items + 8 * k));
        mbar_arrive(iempty + 8 * k);
        return true;
    };

    if (warp < 4) regs_dec<kAbRegsIssue>();
    if (warp == 0) {
        // ---- TMA ----
        pdl_wait();  // the statistics and the ticket are the previous kernel's output
        uint32_t m = 0, n = 0;
        bool ok = true;
        for (;; ++m) {
            unsigned drawn = 0;
            if (lane == 0) drawn = atomicAdd(a.ticket, 1u);
            const unsigned idx = __shfl_sync(0xffffffffu, drawn, 0);
            AbWalker w;
            const bool more = idx < (unsigned)a.items;
            w.set(a, more ? make_int2((int)(idx / a.heads), (int)(idx % a.heads)) : make_int2(-1, 0));
            const uint32_t is = m % kAbItems;
            if (aborted() || !wait(iempty + 8 * is, ((m / kAbItems) & 1) ^ 1)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                ab_sts_item(items + 8 * is, w.j, w.bh);
                mbar_arrive(ifull + 8 * is);
            }
            if (!more) break;
            const int bh = a.bh0 + w.bh, b = bh / a.H, h = bh % a.H;
            const uint32_t ks = m % KS;
            if (aborted() || !wait(kempty + 8 * ks, ((m / KS) & 1) ^ 1)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                mbar_expect_tx(kfull + 8 * ks, kAbTile);
                tma_load_3d(smem_u32(sK + ks * kAbTile), &tmQkv, kfull + 8 * ks, a.C + h * kAbD, w.j * kAbB, b);
            }
            for (int i = w.first(a); i < a.nb; ++i, ++n) {
                const uint32_t qs = n % QS;
                if (aborted() || !wait(qempty + 8 * qs, ((n / QS) & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                uint8_t* q = sQ + qs * kAbQStage;
                if (lane == 0) {
                    mbar_expect_tx(qfull + 8 * qs, kAbQStage);
                    tma_load_3d(smem_u32(q), &tmQkv, qfull + 8 * qs, h * kAbD, i * kAbB, b);
                    tma_load_3d(smem_u32(q + kAbTile), &tmDo, qfull + 8 * qs, h * kAbD, i * kAbB, b);
                    bulk_load(smem_u32(q + 2 * kAbTile), a.stats + ((size_t)w.bh * a.nb + i) * kAbB, kAbStat,
                              qfull + 8 * qs);
                }
                if (i == w.first(a)) {  // V's one stage frees when the item before has its last dP'
                    if (!wait(vempty, (m & 1) ^ 1)) {
                        ++n;
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        mbar_expect_tx(vfull, kAbTile);
                        tma_load_3d(smem_u32(sV), &tmQkv, vfull, 2 * a.C + h * kAbD, w.j * kAbB, b);
                    }
                }
            }
            if (!ok) {
                ++m;  // its K is in flight, and V if it came that far
                break;
            }
        }
        if (!ok) {
            if (lane == 0) {
                give_up();
                // let the copies still in flight land before the block exits
                for (uint32_t k = m > (uint32_t)KS ? m - KS : 0; k < m; ++k) mbar_wait(kfull + 8 * (k % KS), (k / KS) & 1);
                for (uint32_t k = n > (uint32_t)QS ? n - QS : 0; k < n; ++k) mbar_wait(qfull + 8 * (k % QS), (k / QS) & 1);
                if (m > 0) mbar_wait(vfull, (m - 1) & 1);
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        // ---- tcgen05.mma ----
        // (This thread's own instructions count: its loop is about as long as the
        // groups'. Stages, phases and the steps left are kept, not computed.)
        if (elect_one()) {
            AbWalker lead;  // the item of the step whose scores are issued next
            bool ok = take_alone(lead);
            const uint64_t k_desc = sw128_kmajor_desc(smem_u32(sK)), km_desc = sw128_mnmajor_desc(smem_u32(sK));
            const uint64_t v_desc = sw128_kmajor_desc(smem_u32(sV));
            const uint64_t q_desc = sw128_kmajor_desc(smem_u32(sQ)), qm_desc = sw128_mnmajor_desc(smem_u32(sQ));
            const uint64_t dsk = sw128_kmajor_desc(smem_u32(sDS)), dsm = ab_ds_mn_desc(smem_u32(sDS));
            const uint64_t ones = ab_flat_desc(smem_u32(sOnes), 128, 0);
            const uint64_t stat = ab_flat_desc(smem_u32(sQ) + 2 * kAbTile, 0, 128);
            constexpr uint32_t kTile16 = kAbTile >> 4, kStage16 = kAbQStage >> 4;
            uint32_t n = 0;                        // step whose gradients are issued
            uint32_t s_stage = 0, s_phase = 0;     // Q stage of the next scores
            uint32_t g_stage = 0;                  // and of the gradients
            uint32_t lead_k = 0, lead_kphase = 0, lead_vphase = 0, cur_k = 0, acc_phase = 1;
            int lead_left = lead.valid() ? a.nb - lead.first(a) : 0, cur_left = lead_left, lead_len = lead_left;
            bool lead_first = true, first = true, any = lead_left > 0;
            auto scores = [&](uint32_t d_tmem, uint64_t ad, uint64_t bd, uint64_t one_rows) {
#pragma unroll
                for (int kk = 0; kk < kAbD / 16; ++kk)
                    tc_mma<true>(d_tmem, ad + 2u * kk, bd + 2u * kk, kIdescS, kk != 0 ? 1u : 0u);
                tc_mma<true>(d_tmem, one_rows, stat + s_stage * kStage16, kIdescS, 1u);
            };
            // the operands of the next scores have landed
            auto loaded = [&]() {
                return mbar_wait(qfull + 8 * s_stage, s_phase) && (!lead_first || mbar_wait(kfull + 8 * lead_k, lead_kphase));
            };
            auto issue_s = [&]() {
                scores(tmem + kAbS, k_desc + lead_k * kTile16, q_desc + s_stage * kStage16, ones);
                tc_commit(sfull);
            };
            auto issue_dp = [&]() {  // and on to the next step's scores
                scores(tmem + kAbDp, v_desc, q_desc + (s_stage * kStage16 + kTile16), ones + 16u);
                tc_commit(dpfull);
                lead_first = false;
                if (++s_stage == QS) {
                    s_stage = 0;
                    s_phase ^= 1;
                }
                if (--lead_left == 0) {
                    ok = take_alone(lead);
                    lead_len = lead_left = ok && lead.valid() ? a.nb - lead.first(a) : 0;
                    lead_first = true;
                    lead_vphase ^= 1;
                    if (++lead_k == KS) {
                        lead_k = 0;
                        lead_kphase ^= 1;
                    }
                }
            };
            if (any) {
                ok = loaded() && mbar_wait(vfull, 0);
                if (ok) {
                    issue_s();
                    issue_dp();
                }
            }
            while (ok && any) {
                const uint32_t parity = n & 1;
                // P' of step n is written, S' and dP' are read: S' of the next step,
                // dV += P' dO, dP' of the next step (whose commit covers dV too)
                if (!mbar_wait(pready, parity) || (lead_left > 0 && !loaded()) ||
                    (first && n > 0 && (*(volatile int*)s_abort != 0 || !mbar_wait(accfree, acc_phase)))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (lead_left > 0) issue_s();
                const uint64_t qm = qm_desc + g_stage * kStage16;
#pragma unroll
                for (int kk = 0; kk < kAbB / 16; ++kk)
                    tc_mma_ts(tmem + kAbDv, tmem + kAbP + 8u * kk, qm + kTile16 + 128u * kk, kIdescDkv,
                              (kk != 0 || !first) ? 1u : 0u);
                // (a new item's V is still on its way here: its dP' comes after dK and dQ)
                const bool turn = lead_first && lead_left > 0;
                if (lead_left > 0 && !turn) issue_dp();
                // dS' of step n is written: dK += dS' Q, dQ = dS K
                if (!ok || !mbar_wait(dsready, parity) || (n > 0 && !mbar_wait(dqfree, parity ^ 1))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t km = km_desc + cur_k * kTile16;
#pragma unroll
                for (int kk = 0; kk < kAbB / 16; ++kk)
                    tc_mma<true>(tmem + kAbDk, dsk + 1024u * (kk >> 2) + 2u * (kk & 3), qm + 128u * kk, kIdescDkv,
                                 (kk != 0 || !first) ? 1u : 0u);
#pragma unroll
                for (int kk = 0; kk < kAbB / 16; ++kk)
                    tc_mma<true>(tmem + kAbDq, dsm + 128u * kk, km + 128u * kk, kIdescDq, kk != 0 ? 1u : 0u);
                tc_commit(done);
                ++n;
                if (turn) {
                    if (!mbar_wait(vfull, lead_vphase)) {
                        ok = false;
                        break;
                    }
                    cur_left = lead_len + 1;  // (the item that follows)
                    issue_dp();
                    if (!ok) break;
                }
                if (++g_stage == QS) g_stage = 0;
                first = false;
                if (--cur_left == 0) break;
                if (turn) {
                    first = true;
                    acc_phase ^= 1;
                    if (++cur_k == KS) cur_k = 0;
                }
            }
            if (!ok) {
                give_up();
                // the products issued so far end before the block does
                tc_commit(done);
                mbar_wait(done, n & 1);
            }
        }
        __syncwarp();
    } else if (warp == 2 || warp == 3) {
        // ---- two senders, in turn: what the last group has staged in sOut. One waits
        // for its tile's addition to complete, and tells the chain, while the other
        // sends the next. ----
        pdl_wait();
        if (elect_one()) {
            uint32_t msg = 0;
            AbWalker w;
            bool ok = take_alone(w);
            for (; ok && w.valid(); ok = ++w.i < a.nb || take_alone(w)) {
                const int bh = a.bh0 + w.bh, b = bh / a.H, h = bh % a.H;
                if (w.last(a) && (msg++ & 1) == (uint32_t)(warp & 1)) {
                    // dk and dv; tokens past T lie outside the map and are not written
                    ok = mbar_wait(outfull + 8 * ((msg - 1) & 1), ((msg - 1) >> 1) & 1);
                    if (!ok) break;
                    for (int y = 0; y < kAbB; y += 32) {
                        ab_store_3d(&tmDqkv, smem_u32(sOut + y * 128), a.C + h * kAbD, w.j * kAbB + y, b);
                        ab_store_3d(&tmDqkv, smem_u32(sOut + kAbTile + y * 128), 2 * a.C + h * kAbD, w.j * kAbB + y, b);
                    }
                    bulk_commit();
                    bulk_wait_read_all();
                    mbar_arrive(outfree);
                }
                if ((msg++ & 1) == (uint32_t)(warp & 1)) {
                    if (*(volatile int*)s_abort != 0 || !mbar_wait(outfull + 8 * ((msg - 1) & 1), ((msg - 1) >> 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const int chain = w.j % a.chains, pos = w.j / a.chains;
                    const size_t slot = ((size_t)w.bh * a.chains + chain) * a.nb + w.i;
                    float* tile = a.dq + slot * (kAbDqTile / 4);
                    if (pos == 0) {
                        bulk_store(tile, smem_u32(sOut), kAbDqTile);
                    } else {
                        // until the chain's earlier block has added to this tile
                        bool there = ld_acquire_gpu(a.flags + slot) == (unsigned)pos;
                        const unsigned long long t0 = global_ns();
                        for (uint32_t k = 1; !there && k < kWaitIters; ++k) {
                            there = ld_acquire_gpu(a.flags + slot) == (unsigned)pos;
                            if ((k & 63u) == 63u && (*(volatile int*)s_abort != 0 || global_ns() - t0 > kWaitNs)) break;
                        }
                        if (!there) {
                            ok = false;
                            break;
                        }
                        fence_proxy_async_global();
                        bulk_add_f32(tile, smem_u32(sOut), kAbDqTile);
                    }
                    bulk_commit();
                    bulk_wait_read_all();
                    mbar_arrive(outfree);
                    if (w.j + a.chains <= (a.causal ? w.i : a.nb - 1)) {
                        bulk_wait_all();
                        fence_proxy_async_global();
                        st_release_gpu(a.flags + slot, (unsigned)pos + 1u);
                    }
                }
            }
            if (!ok) give_up();
            bulk_wait_all();
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 4 + 4 * kAbGroups) {
        // ---- P' and dS' ----
        regs_inc<kAbRegsSoftmax>();
        const int grp = (warp - 4) >> 2, quad = warp & 3;
        const int r = 32 * quad + lane;  // key within the block, TMEM lane
        const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
        const uint32_t tS = tmem + lanes + kAbS + 32u * grp, tDp = tmem + lanes + kAbDp + 32u * grp,
                       tP = tmem + lanes + kAbP + 16u * grp;
        uint8_t* ds_row = sDS + (grp >> 1) * (kAbDs / 2) + r * 128;
        const uint64_t sl2 = ab_pack(a.scale_log2, a.scale_log2);
        uint32_t n = 0;
        AbWalker w;
        bool ok = take(w);
        for (; ok && w.valid(); ok = ++w.i < a.nb || take(w), ++n) {
            const bool diag = a.causal && w.i == w.j;
            const bool masked = diag || (w.j + 1) * kAbB > a.T;
            // query c of this group is visible to the thread's key from `from` on
            const int from = w.j * kAbB + r >= a.T ? 32 : diag ? r - 32 * grp : 0;
            ok = wait(sfull, n & 1);
            if (!ok) break;
            tc_fence_after();
            uint32_t s[32];
            tmem_ld32_async(tS, s);
            tmem_wait_ld(s);
            uint64_t p[16];
            ab_probs(s, sl2, p);
            if (masked) ab_hide(p, from);
            // dP' of this step, and so dV of the step before: P' may be rewritten
            ok = wait(dpfull, n & 1);
            if (!ok) break;
            tc_fence_after();
            tmem_ld32_async(tDp, s);
            ab_put_p(tP, p);
            ab_tmem_wait_st();
            tmem_wait_ld(s);
            tc_fence_before();
            arrive(pready);
            if (w.last(a)) arrive(vempty);
            // dK and dQ of the step before: dS' may be rewritten
            ok = n == 0 || wait(done, (n - 1) & 1);
            if (!ok) break;
            if (masked) ab_put_ds<true>(s, p, ds_row, r, 4 * (grp & 1), from);
            else ab_put_ds<false>(s, p, ds_row, r, 4 * (grp & 1), from);
            fence_proxy_async_smem();
            tc_fence_before();
            arrive(dsready);
        }
        if (!ok && lane == 0) give_up();
    } else if (warp >= 4 + 4 * kAbGroups) {
        // ---- dq, dk and dv out of TMEM ----
        regs_dec<kAbRegsOut>();
        const int quad = warp & 3;
        const int r = 32 * quad + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
        uint32_t n = 0, msg = 0;
        AbWalker w;
        bool ok = take(w);
        for (; ok && w.valid(); ok = ++w.i < a.nb || take(w), ++n) {
            const bool last = w.last(a);
            ok = wait(done, n & 1) && (msg == 0 || wait(outfree, (msg - 1) & 1));
            if (!ok) break;
            tc_fence_after();
            arrive(qempty + 8 * (n % QS));
            if (last) arrive(kempty + 8 * (w.m % KS));
            uint32_t v[32];
            if (last) {  // first, since the next item's dV waits for it
#pragma unroll
                for (int part = 0; part < 4; ++part) {  // dk, then dv
                    tmem_ld32_async(tmem + lanes + (part < 2 ? kAbDk : kAbDv) + 32u * (part & 1), v);
                    tmem_wait_ld(v);
                    ab_stage<4>(sOut + (part >> 1) * kAbTile, r, 4 * (part & 1), v, part < 2 ? a.scale : 1.0f);
                }
                tc_fence_before();
                arrive(accfree);
                fence_proxy_async_smem();
                arrive(outfull + 8 * (msg & 1));
                ++msg;
                ok = wait(outfree, (msg - 1) & 1);
                if (!ok) break;
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                tmem_ld32_async(tmem + lanes + kAbDq + 32u * half, v);
                tmem_wait_ld(v);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    *reinterpret_cast<uint4*>(sOut + (8 * half + c) * (kAbB * 16) + r * 16) =
                        make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
            }
            tc_fence_before();
            arrive(dqfree);
            fence_proxy_async_smem();
            arrive(outfull + 8 * (msg & 1));
            ++msg;
        }
        if (!ok && lane == 0) give_up();
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kAbTmem);
    }
}

// T <= 128: a block per (sequence, head). Thread: a key (TMEM lane) and 64 queries.
__global__ void __launch_bounds__(kAsThreads, 2)
attn_bwd_short_kernel(const __grid_constant__ CUtensorMap tmQkv, const __grid_constant__ CUtensorMap tmDo,
                      const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmDqkv,
                      const uint16_t* out, const uint16_t* dout, const float* lse, const AbArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sK = smem, *sQ = sK + kAbTile, *sV = sQ + kAbTile, *sDO = sV + kAbTile, *sDS = sDO + kAbTile;
    uint8_t *sStat = sDS + kAbDs, *sOnes = sStat + kAbStat;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sOnes + kAbOnes);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 6);
    const uint32_t kq = smem_u32(bars), vdo = kq + 8, sfull = kq + 16, dpfull = kq + 24, done = kq + 32;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H;
    if (threadIdx.x == 0) {
        for (int k = 0; k < 5; ++k) mbar_init(kq + 8 * k, 1);
        mbar_fence_init();
        tma_prefetch_map(&tmQkv);
        tma_prefetch_map(&tmDo);
        tma_prefetch_map(&tmDqkv);
    }
    if (warp == 0) tmem_alloc(smem_u32(tmem_slot), kAsTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    pdl_wait();
    if (threadIdx.x == 0) {
        pdl_launch_dependents();
        mbar_expect_tx(kq, 2 * kAbTile);
        tma_load_3d(smem_u32(sK), &tmQkv, kq, a.C + h * kAbD, 0, b);
        tma_load_3d(smem_u32(sQ), &tmQkv, kq, h * kAbD, 0, b);
        mbar_expect_tx(vdo, 2 * kAbTile);
        tma_load_3d(smem_u32(sV), &tmQkv, vdo, 2 * a.C + h * kAbD, 0, b);
        tma_load_3d(smem_u32(sDO), &tmDo, vdo, h * kAbD, 0, b);
    }
    __syncwarp();
    ab_ones(reinterpret_cast<uint4*>(sOnes));
    ab_stats(out, dout, lse, a.T, a.H, b, h, 0, a.inv_scale, reinterpret_cast<uint4*>(sStat));
    fence_proxy_async_smem();
    __syncthreads();
    // A wait that runs out sets the status word; the block then goes on with what
    // it has, and its outputs are not to be used.
    auto wait = [&](uint32_t bar) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar, 0))) {
            if (lane == 0) atomicExch(a.status, (int)LIN_ERR_DEVICE_TIMEOUT);
            mbar_wait(bar, 0);  // what is in flight once more before the block goes on
            __syncwarp();
        }
    };
    wait(kq);
    if (warp == 0) {
        if (elect_one()) {
            ab_mma_scores(tmem + kAbS, smem_u32(sK), smem_u32(sQ), smem_u32(sOnes), smem_u32(sStat));
            tc_commit(sfull);
        }
        __syncwarp();
    }
    wait(vdo);
    if (warp == 0) {
        if (elect_one()) {
            ab_mma_scores(tmem + kAsDp, smem_u32(sV), smem_u32(sDO), smem_u32(sOnes) + 256, smem_u32(sStat));
            tc_commit(dpfull);
        }
        __syncwarp();
    }
    if (threadIdx.x == 32 && bh + a.ahead < (int)gridDim.x) {
        // The inputs of the block that comes after this one on its place are asked for
        // while this one computes: its loads then find them in the L2. Without it all
        // blocks load and compute at the same time (64 x 128 x 12 heads: 33 us).
        const int next = bh + a.ahead, nb_ = next / a.H, x = (next % a.H) * kAbD;
        ab_prefetch_3d(&tmQkv, x, 0, nb_);
        ab_prefetch_3d(&tmQkv, a.C + x, 0, nb_);
        ab_prefetch_3d(&tmQkv, 2 * a.C + x, 0, nb_);
        ab_prefetch_3d(&tmDo, x, 0, nb_);
        ab_prefetch_3d(&tmOut, x, 0, nb_);
    }
    __syncwarp();
    const int grp = warp >> 2, quad = warp & 3;
    const int r = 32 * quad + lane;  // key, TMEM lane
    const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
    const bool masked = a.causal || a.T < kAbB;
    wait(sfull);
    tc_fence_after();
    uint32_t s[2][32];
    tmem_ld32_async(tmem + lanes + kAbS + 64u * grp, s[0]);
    tmem_ld32_async(tmem + lanes + kAbS + 64u * grp + 32u, s[1]);
    tmem_wait_ld(s[0]);
    tmem_wait_ld(s[1]);
    tc_fence_before();
    __syncthreads();  // S' has been read (P' and dQ take its place)
    tc_fence_after();
    uint64_t p[2][16];
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
        const int q0 = 64 * grp + 32 * ch;  // the chunk's first query; visible from `from` on
        const int from = r >= a.T ? 32 : a.causal ? r - q0 : 0;
        ab_probs(s[ch], ab_pack(a.scale_log2, a.scale_log2), p[ch]);
        if (masked) ab_hide(p[ch], from);
        ab_put_p(tmem + lanes + kAsP + 32u * grp + 16u * ch, p[ch]);
    }
    ab_tmem_wait_st();
    wait(dpfull);
    tc_fence_after();
    uint8_t* ds_row = sDS + grp * (kAbDs / 2) + r * 128;
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
        const int q0 = 64 * grp + 32 * ch;
        const int from = r >= a.T ? 32 : a.causal ? r - q0 : 0;
        tmem_ld32_async(tmem + lanes + kAsDp + q0, s[0]);
        tmem_wait_ld(s[0]);
        if (masked) ab_put_ds<true>(s[0], p[ch], ds_row, r, 4 * ch, from);
        else ab_put_ds<false>(s[0], p[ch], ds_row, r, 4 * ch, from);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) {
        const uint64_t od = sw128_mnmajor_desc(smem_u32(sDO)), qd = sw128_mnmajor_desc(smem_u32(sQ)),
                       kd = sw128_mnmajor_desc(smem_u32(sK));
        const uint64_t dsk = sw128_kmajor_desc(smem_u32(sDS)), dsm = ab_ds_mn_desc(smem_u32(sDS));
        if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kAbB / 16; ++kk) {
                const uint32_t add = kk != 0 ? 1u : 0u;
                tc_mma_ts(tmem + kAsDv, tmem + kAsP + 8u * kk, od + 128u * kk, kIdescDkv, add);
                tc_mma<true>(tmem + kAsDk, dsk + 1024u * (kk >> 2) + 2u * (kk & 3), qd + 128u * kk, kIdescDkv, add);
                tc_mma<true>(tmem + kAsDq, dsm + 128u * kk, kd + 128u * kk, kIdescDq, add);
            }
            tc_commit(done);
        }
        __syncwarp();
    }
    wait(done);
    tc_fence_after();
    // Group 0 takes dk and half of dq, group 1 dv and the rest, through the tiles
    // of K, V and Q.
    uint32_t* v = &s[0][0];
    tmem_ld32_async(tmem + lanes + (grp ? kAsDv : kAsDk), s[0]);
    tmem_ld32_async(tmem + lanes + (grp ? kAsDv : kAsDk) + 32u, s[1]);
    uint32_t q[32];
    tmem_ld32_async(tmem + lanes + kAsDq + 32u * grp, q);
    tmem_wait_ld(s[0]);
    tmem_wait_ld(s[1]);
    tmem_wait_ld(q);
    ab_stage<8>(grp ? sV : sK, r, 0, v, grp ? 1.0f : a.scale);
    ab_stage<4>(sQ, r, 4 * grp, q, a.scale);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kAsTmem);
    }
    // tokens past T lie outside the map and are not written
    if (lane == 0 && 32 * quad < a.T) {
        if (grp == 0) {
            ab_store_3d(&tmDqkv, smem_u32(sK + quad * 4096), a.C + h * kAbD, 32 * quad, b);
            ab_store_3d(&tmDqkv, smem_u32(sQ + quad * 4096), h * kAbD, 32 * quad, b);
        } else {
            ab_store_3d(&tmDqkv, smem_u32(sV + quad * 4096), 2 * a.C + h * kAbD, 32 * quad, b);
        }
        bulk_commit();
        bulk_wait_read_all();
    }
}

// The statistics of every query block; its dq counters and the ticket zeroed.
__global__ void __launch_bounds__(256) attn_bwd_prep(const uint16_t* out, const uint16_t* dout, const float* lse, int T,
                                                     int H, int nb, int bh0, int chains, float inv_scale,
                                                     uint4* stats, unsigned* flags, unsigned* ticket) {
    pdl_wait();
    pdl_launch_dependents();
    const int local = blockIdx.x / nb, i = blockIdx.x % nb;
    const int bh = bh0 + local;
    ab_stats(out, dout, lse, T, H, bh / H, bh % H, i, inv_scale, stats + (size_t)blockIdx.x * kAbB);
    for (int g = threadIdx.x; g < chains; g += 256) flags[((size_t)local * chains + g) * nb + i] = 0u;
    if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0u;
}

// dq of 128 queries of one head: the chains' fp32 sums added in order, scaled,
// rounded once. A thread has 16 columns of a row.
__global__ void __launch_bounds__(kAbB) attn_bwd_dq(const float* dq, uint16_t* dqkv, int T, int H, int nb, int bh0,
                                                   int chains, int causal, float scale) {
    pdl_wait();
    pdl_launch_dependents();
    const int part = blockIdx.x & 3, tile = blockIdx.x >> 2, local = tile / nb, i = tile % nb;
    const int bh = bh0 + local, b = bh / H, h = bh % H;
    const int row = threadIdx.x;
    const int t = i * kAbB + row;
    if (t >= T) return;
    const int used = min(chains, causal ? i + 1 : nb);
    float4 s[4];
    for (int g = 0; g < used; ++g) {
        const float4* p = reinterpret_cast<const float4*>(dq + (((size_t)local * chains + g) * nb + i) * (kAbDqTile / 4)) +
                          4 * part * kAbB + row;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 x = p[k * kAbB];
            if (g == 0) {
                s[k] = x;
            } else {
                s[k].x += x.x;
                s[k].y += x.y;
                s[k].z += x.z;
                s[k].w += x.w;
            }
        }
    }
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        o[2 * k] = pack_bf16x2(s[k].x * scale, s[k].y * scale);
        o[2 * k + 1] = pack_bf16x2(s[k].z * scale, s[k].w * scale);
    }
    uint4* dst = reinterpret_cast<uint4*>(dqkv + ((size_t)b * T + t) * ((size_t)3 * H * kAbD) + h * kAbD + 16 * part);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

PFN_cuTensorMapEncodeTiled_v12000 ab_encode_fn() {
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

// (B, T, cols) bf16, box = 64 columns x `rows` tokens of one sequence, 128-byte swizzle.
bool ab_map(CUtensorMap* map, const void* base, int B, int T, int cols, int rows) {
    auto fn = ab_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(T), static_cast<cuuint64_t>(B)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, static_cast<cuuint64_t>(T) * cols * 2};
    cuuint32_t box[3] = {kAbD, static_cast<cuuint32_t>(rows), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int launch_attention_backward(const AttnBwdProblem& p) {
    const int C = p.H * kAbD;
    const int nb = (p.T + kAbB - 1) / kAbB;
    const long long bh_all = (long long)p.B * p.H;

    CUtensorMap tq, tdo, tdq;
    if (!ab_map(&tq, p.qkv, p.B, p.T, 3 * C, kAbB) || !ab_map(&tdo, p.dout, p.B, p.T, C, kAbB) ||
        !ab_map(&tdq, p.dqkv, p.B, p.T, 3 * C, 32))
        return LIN_ERR_CUDA;
    const uint16_t* out = static_cast<const uint16_t*>(p.out);
    const uint16_t* dout = static_cast<const uint16_t*>(p.dout);
    AbArgs a = {};
    a.T = p.T;
    a.H = p.H;
    a.C = C;
    a.nb = nb;
    a.causal = p.causal ? 1 : 0;
    a.scale = p.scale;
    a.scale_log2 = p.scale * kAbLog2e;
    a.inv_scale = 1.0f / p.scale;
    a.status = p.dev_status;

    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = p.stream;
    cfg.attrs = &attr;
    cfg.numAttrs = p.early_start ? 1 : 0;

    if (nb == 1) {
        static std::atomic<unsigned long long> attr_set{0};
        if (ensure_smem_attr(attr_set, attn_bwd_short_kernel, kAsSmem) != LIN_OK) return LIN_ERR_CUDA;
        cfg.gridDim = dim3((unsigned)bh_all);
        cfg.blockDim = dim3(kAsThreads);
        cfg.dynamicSmemBytes = kAsSmem;
        CUtensorMap to;
        if (!ab_map(&to, p.out, p.B, p.T, C, kAbB)) return LIN_ERR_CUDA;
        a.ahead = 2 * p.sm_count;
        if (cudaLaunchKernelEx(&cfg, attn_bwd_short_kernel, tq, tdo, to, tdq, out, dout, p.lse, a) != cudaSuccess)
            return LIN_ERR_CUDA;
        return cudaGetLastError() == cudaSuccess ? LIN_OK : LIN_ERR_CUDA;
    }

    // Workspace after the counter block: ticket, statistics, counters, dq sums (a
    // kilobyte stands for the first and for alignment). Heads go in as many launches
    // as it takes.
    const size_t avail = p.workspace_bytes > kCounterBytes + 1024 ? p.workspace_bytes - kCounterBytes - 1024 : 0;
    const size_t stat = (size_t)nb * kAbStat;
    const size_t chain = (size_t)nb * (kAbDqTile + sizeof(unsigned));
    if (stat + chain > avail) return LIN_ERR_WORKSPACE;
    const long long heads = std::min(bh_all, (long long)(avail / (stat + chain)));
    // Chains: as many of a head's key blocks as run at the same time, so that
    // none waits, where the workspace has room for their sums.
    const long long together = (p.sm_count + heads - 1) / heads;
    const long long room = (long long)((avail / heads - stat) / chain);
    a.chains = (int)std::max(1ll, std::min({together, room, (long long)nb}));

    static std::atomic<unsigned long long> attr_set{0};
    if (ensure_smem_attr(attr_set, attn_bwd_kernel, kAbSmem) != LIN_OK) return LIN_ERR_CUDA;
    // The register split needs the kernel launched at kAbLaunchRegs a thread (else the
    // increase would wait forever): refuse otherwise.
    static const int regs = []() {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, attn_bwd_kernel) == cudaSuccess ? fa.numRegs : 0;
    }();
    if (regs < kAbLaunchRegs) return LIN_ERR_UNSUPPORTED;
    a.ticket = reinterpret_cast<unsigned*>(static_cast<char*>(p.workspace) + kCounterBytes);
    char* ws = static_cast<char*>(p.workspace) + kCounterBytes + 256;
    for (long long bh0 = 0; bh0 < bh_all; bh0 += heads) {
        const int count = (int)std::min(heads, bh_all - bh0);
        a.bh0 = (int)bh0;
        a.heads = count;
        a.items = count * nb;
        uint4* stats = reinterpret_cast<uint4*>(ws);
        char* rest = ws + align_up((size_t)count * stat, 256);
        a.stats = stats;
        a.flags = reinterpret_cast<unsigned*>(rest);
        a.dq = reinterpret_cast<float*>(rest + align_up((size_t)count * a.chains * nb * sizeof(unsigned), 256));
        cfg.gridDim = dim3((unsigned)a.items);
        cfg.blockDim = dim3(256);
        cfg.dynamicSmemBytes = 0;
        if (cudaLaunchKernelEx(&cfg, attn_bwd_prep, out, dout, p.lse, p.T, p.H, nb, a.bh0, a.chains,
                               a.inv_scale, stats, a.flags, a.ticket) !=
            cudaSuccess)
            return LIN_ERR_CUDA;
        cfg.gridDim = dim3((unsigned)std::min(a.items, p.sm_count));
        cfg.blockDim = dim3(kAbThreads);
        cfg.dynamicSmemBytes = kAbSmem;
        if (cudaLaunchKernelEx(&cfg, attn_bwd_kernel, tq, tdo, tdq, a) != cudaSuccess) return LIN_ERR_CUDA;
        cfg.gridDim = dim3((unsigned)a.items * 4u);
        cfg.blockDim = dim3(kAbB);
        cfg.dynamicSmemBytes = 0;
        if (cudaLaunchKernelEx(&cfg, attn_bwd_dq, static_cast<const float*>(a.dq), static_cast<uint16_t*>(p.dqkv), p.T,
                               p.H, nb, a.bh0, a.chains, a.causal, a.scale) != cudaSuccess)
            return LIN_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? LIN_OK : LIN_ERR_CUDA;
}

}  // namespace lin

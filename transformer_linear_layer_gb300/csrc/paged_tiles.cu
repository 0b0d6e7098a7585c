// Attention of many new tokens (chunks of prompts, whole prompts, the queries of a
// cross attention) over a paged cache, on the tensor cores: tiles of two groups of up
// to 128 rows (token, query head of one key head).
//
//   s_rj = (q_r . k_j) scale,  out_r = sum_j exp(s_rj - m) v_j / sum_j exp(s_rj - m)
//
// 4 D flops a row and key against 4 D bytes a key: with 256 rows a tile the products and the
// exponentials bound it, not memory. Both groups work on the same keys, so that
// a block of 128 keys, brought in once, serves 256 rows (two tiles apart would ask the
// L2 for 60 bytes a cycle and SM); and one group's softmax runs under the other's products.
//   warps 0, 3  TMA. K and V of 128 keys are tiles of a ring each,
//               a box per page and 64 columns, each lane its own (pages of 8 tokens take 32
//               boxes a tile, so that K and V have a warp each); Q per group.
//   warps 1, 2  tcgen05.mma, an elected thread per group: S = Q K^T (128 x 128) into the
//               group's 128 TMEM columns, then O += P V with P (bf16) as the TMEM operand, beside S
//               (heads of 64) or in its columns: nothing of the scores passes through shared memory.
//   warps 4-7,  softmax of group 0 and 1, a thread per row: scores out of TMEM, scaled to
//   warps 8-11  base-2 units by a packed FMA, exponentiated, rounded to bf16, back into TMEM.
//               The reference for the exponents need not be the maximum: it is that of an
//               item's first 64 keys (when they all score -inf, of the first that do not), and stays
//               while 64 probabilities of a row add up to at most 2^16
//               (bf16 keeps its relative precision; the argument of an exponential stays below 16, and its
//               rounding below 2^-20). So nothing waits for a maximum and none is taken; in the
//               rare case that the scores have risen, O is scaled and the 64 keys are exponentiated again.
//               The price: the probability of a row's top key is rounded like the others and not 1 (error against
//               64 bits 0.0023 of the norm where a maximum gives 0.0018; the output's rounding alone is 0.0017).
// Keys past the last one that a row of the tile sees are not loaded where they fill a box, and their
// values are set to zero in shared memory where they do not: a probability of 0 must not meet a
// NaN in slots that were never written.
// Every wait is bounded (about 1 s); a block that gives up sets the status word.
//
// Measured (GB300, with the joining kernel): 2 prompts of 4096 tokens, 16 heads of 128 on 2: 138 us, 992
// TF/s of the visible pairs' products; 4 chunks of 512 over 8704 keys, 16 heads of 128 on 2: 114 us, 1240 TF/s
// (3300 cycles a block of 256 x 128 in a long item, with stamps, 2070 of them products when
// nothing else is done); the same chunks, 12 heads of 64: 68 us, 780 TF/s (2500 cycles a
// block, 2700 with stamps, 1160 of products and 1250 of exponentials with two warps a scheduler). Tensor pipe 51 %
// (prompts) and 35 % (heads of 64), DRAM 4 and 23 %: bound by a group's chain of scores, exponentials and products, and by the waits
// between them, which queue behind the exponentials.
#include <math.h>

#include <type_traits>

#include "paged.cuh"

namespace lin {
namespace {

constexpr int kPtThreads = 384;
constexpr int kPtKeys = 128;            // keys of a block, and rows of a group
// Registers: launched at kPtLaunch a thread; warps 0-3 go down to kPtLow and the softmax
// warps up to kPtHigh (128 * 72 + 256 * 216 = 384 * 168). The host refuses a kernel
// compiled to fewer than kPtLaunch: the increase could not be granted.
constexpr int kPtLaunch = 168, kPtLow = 72, kPtHigh = 216;
static_assert(128 * kPtLow + 256 * kPtHigh <= kPtThreads * kPtLaunch, "register split");
constexpr uint32_t kPtTmem = 512;
constexpr int kPtParts = 4;             // parts of items that are described at a time
// Blocks that an item's start and end cost. Measured (us) with              0    1    2    3    4    6
//     2 prompts of 4096, 16 heads of 128 on 2                             209  164  136  131  132  133
//     4 prompts of 2048, 12 heads of 64                                    74   63   59   59   58   58
//     4 chunks of 512 over 8704, 12 heads of 64                            68   67   67   68   68   70
//     the same, 16 heads of 128 on 2                                      114  115  114  114  114  116
//     8 x 77 to 101 queries over 1500, 12 heads of 64, full              21.6 22.2 21.3 22.8 22.3 23.4
//     the same, 16 heads of 128 on 4                                     26.9 31.2 29.6 29.3 28.6 29.8
//     33 sequences, a quarter with 200 to 301 tokens, 20 heads of 64 on 4   59   55   53   53   53   55
//     the same, 32 heads of 128 on 8                                      123  114  110  104  104  106
constexpr int kPtLead = 2;
constexpr float kPtRise = 65536.f;      // what 64 probabilities may add up to before their reference moves

template <int D>
struct PtShape {
    static constexpr uint32_t kTile = kPtKeys * D * 2;      // K, V or Q: halves of 64 columns, 16 KiB each
    // Tiles of K's ring and of V's. A barrier's wait tells odd phases from even ones only, so whoever waits for a slot
    // may be at most one phase ahead of it: each ring has one producer, which fills every phase of its
    // slots itself, and each group releases every tile of both. (Were a slot to alternate between the two producers, one of them
    // would wait for it two phases after its last fill, and take the release before that for the one it waits for.)
    // Heads of 128 with 2 slots for K and 3 for V: the same times (2 x 4096 tokens 135.8 us and 136.4).
    static constexpr int KS = D == 64 ? 5 : 3, VS = D == 64 ? 5 : 2, S = KS + VS;
    static constexpr size_t kSmem = 1024 + (2 + S) * (size_t)kTile;
    // TMEM columns of a group: S (128), O (D) and P (64). Heads of 64 leave room for P beside
    // S, so that the next block's S is computed while this one's exponentials are; with
    // 128 columns of O a group P takes the place of the S that it came from.
    static constexpr bool kApart = D == 64;
    // The groups take turns with a block's exponentials, warp by warp of a scheduler, where P lies in S's
    // place: that keeps one group's products under the other's softmax (2 x 4096 tokens, 16 heads of 128 on
    // 2: 146 -> 137 us). With the next scores ready early it only adds waits (4 x 512 over 8704, 12 heads of
    // 64: 67 us without, 91 with a turn a block, 82 with one per 64 keys).
    static constexpr bool kTurns = !kApart;
    static constexpr uint32_t kS = 0, kP = kApart ? 256 : 0, kO = kApart ? 384 : 256, kPStep = kApart ? 64 : 128;
};

struct PtPart {       // a block's part of an item
    int h, row0;      // key head, first row of q
    int tokens;
    int pos0;         // position of the first token
    int seen;         // keys that some row sees
    int j0, n;        // first key block, blocks
    int slot;         // the workspace's slot, or -1: the item is whole
};

__device__ __forceinline__ float pt_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t pt_pack(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void pt_unpack(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t pt_fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t pt_add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float pt_max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ void pt_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void pt_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D (+)= A B with A (bf16, two to a 32-bit column) in TMEM.
__device__ __forceinline__ void pt_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// True in one lane of the warp.
__device__ __forceinline__ bool pt_elect() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e != 0;
}
// A V tile read MN-major: 64-column halves 16 KiB apart, groups of 8 keys 1 KiB.
__device__ __forceinline__ uint64_t pt_v_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(16384u >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// What group grp does of a part: tokens of its own, keys that they see, key blocks.
struct PtShare {
    int tokens, seen, n;
};
__device__ __forceinline__ PtShare pt_share(const PagedArgs& a, const PtPart& p, int grp) {
    const int each = a.TQ / 2;
    PtShare s;
    s.tokens = min(max(p.tokens - grp * each, 0), each);
    s.seen = a.causal ? max(min(p.seen, p.pos0 + grp * each + s.tokens), 0) : p.seen;
    s.n = s.tokens == 0 ? 0 : min(max((s.seen + kPtKeys - 1) / kPtKeys - p.j0, 0), p.n);
    return s;
}

template <int D>
__global__ void __launch_bounds__(kPtThreads, 1)
paged_tiles_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const PagedArgs a) {
    using P = PtShape<D>;
    constexpr int KS = P::KS, VS = P::VS, S = P::S, HALVES = D / 64;  // slots: K's, then V's
    constexpr uint32_t kHalf = kPtKeys * 128;
    constexpr uint32_t IDESC_S = make_idesc(1u, 128, kPtKeys);
    constexpr uint32_t IDESC_O = make_idesc(1u, 128, D, false, true);

    extern __shared__ uint8_t raw[];
    __shared__ alignas(8) uint64_t bars[2 * S + 2 * kPtParts + 28];
    __shared__ PtPart parts[kPtParts];
    __shared__ uint32_t s_tmem;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;
    uint8_t* ring = smem + 2 * P::kTile;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * S, pfull0 = empty0 + 8 * S,
                   pempty0 = pfull0 + 8 * kPtParts, qfull0 = pempty0 + 8 * kPtParts, qempty0 = qfull0 + 16,
                   sfull0 = qempty0 + 16, sread0 = sfull0 + 16, probs0 = sread0 + 16, pv0 = probs0 + 32, pvhalf0 = pv0 + 16,
                   ofull0 = pvhalf0 + 16,
                   done0 = ofull0 + 16, turn0 = done0 + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 2);          // both groups
        }
        for (int s = 0; s < kPtParts; ++s) {
            mbar_init(pfull0 + 8 * s, 1);
            mbar_init(pempty0 + 8 * s, 2 + 8);     // both MMA threads, the softmax warps
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(qfull0 + 8 * g, 1);
            mbar_init(qempty0 + 8 * g, 1);
            mbar_init(sfull0 + 8 * g, 1);
            mbar_init(sread0 + 8 * g, 4);
            mbar_init(probs0 + 16 * g, 4);         // keys 0-63 and 64-127 of the block
            mbar_init(probs0 + 16 * g + 8, 4);
            mbar_init(pv0 + 8 * g, 1);
            mbar_init(pvhalf0 + 8 * g, 1);
            mbar_init(ofull0 + 8 * g, 1);
            mbar_init(done0 + 8 * g, 1);
            for (int w = 0; w < 4; ++w) mbar_init(turn0 + 32 * g + 8 * w, 1);
        }
        mbar_fence_init();
        tma_prefetch_map(&tmQ);
        tma_prefetch_map(&tmK);
        tma_prefetch_map(&tmV);
    }
    if (warp == 1) tmem_alloc(smem_u32(&s_tmem), kPtTmem);
    tc_fence_before();
    pdl_wait();
    pdl_launch_dependents();
    const PagedStretch r = paged_stretch<kPtKeys, kPtThreads>(a);  // syncs the block
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    auto give_up = [&]() { atomicExch(a.status, (int)LIN_ERR_DEVICE_TIMEOUT); };
    // A warp's wait: all lanes agree on whether it ended.
    auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
    };

    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPtLow));
    if (warp == 0 || warp == 3) {
        // ---- TMA: warp 0 the parts, Q and K, warp 3 V; whole warps walk the stretch ----
        const bool keys = warp == 0;
        PagedCut cut = {0, 0, 0, 0};
        const uint32_t first = keys ? 0 : KS, slots = keys ? KS : VS;             // this warp's ring
        uint32_t st = first, ph = 1, issued = 0, np = 0, nq[2] = {0, 0};          // the next tile; what has been issued
        bool ok = true;
        const int each = a.TQ / 2;
        const PagedBox<kPtKeys> box(a);
        const bool mine = box.group < HALVES;
        const uint32_t to = smem_u32(ring) + box.group * kHalf + ((box.at << box.shift) * 128);
        PagedWalk<kPtKeys> w;
        w.start(a, r);
        for (int j0, k; ok && w.part(a, j0, k); w.next(a, k)) {
            PtPart p;
            p.h = w.h;
            p.row0 = w.q.row0 + w.t * a.TQ;
            p.tokens = min(a.TQ, w.q.n - w.t * a.TQ);
            p.pos0 = w.q.pos0 + w.t * a.TQ;
            p.seen = tile_seen(a, w.q, w.t);
            p.j0 = j0;
            p.n = k;
            p.slot = k == w.n ? -1 : 2 * (int)blockIdx.x + (j0 == 0 ? 1 : 0);
            const int* table = a.batch.block_table + w.b * a.batch.table_stride;
            int key0 = j0 * kPtKeys, next = box.entry(a, table, key0, p.seen);
            if (keys) {
                if (j0 == 0 && k < w.n) cut = {p.row0, p.tokens, p.h, w.last_block(r.per)};
                const uint32_t ps = np % kPtParts;
                if (!wait(pempty0 + 8 * ps, ((np / kPtParts) & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    parts[ps] = p;
                    mbar_arrive(pfull0 + 8 * ps);
                }
                ++np;
            }
            for (int i = 0; i < k; ++i, key0 += kPtKeys) {
                const int entry = next;
                if (i + 1 < k) next = box.entry(a, table, key0 + kPtKeys, p.seen);
                if (!wait(empty0 + 8 * st, ph)) {
                    ok = false;
                    break;
                }
                if (lane == 0)
                    mbar_expect_tx(full0 + 8 * st, (uint32_t)(box.count(key0, p.seen) * HALVES) * (128u << box.shift));
                __syncwarp();
                if (mine && box.holds(key0, p.seen))
                    tma_load_4d(to + st * P::kTile, keys ? &tmK : &tmV, full0 + 8 * st, 64 * box.group, box.slot(a, key0),
                                p.h, box.page(a, entry));
                ++issued;
                if (++st == first + slots) {
                    st = first;
                    ph ^= 1;
                }
                if (i > 0 || !keys) continue;
                // the part's Q, once its predecessor's last S is done
                for (int grp = 0; ok && grp < 2; ++grp) {
                    if (pt_share(a, p, grp).n == 0) continue;
                    if (!wait(qempty0 + 8 * grp, (nq[grp] & 1) ^ 1)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_expect_tx(qfull0 + 8 * grp, (uint32_t)(each * a.G) * D * 2);
                    __syncwarp();
                    if (lane < HALVES)
                        tma_load_3d(smem_u32(sQ + grp * P::kTile + lane * kHalf), &tmQ, qfull0 + 8 * grp, 64 * lane,
                                    p.h * a.G, p.row0 + grp * each);
                    ++nq[grp];
                }
                if (!ok) break;
            }
        }
        if (keys && ok) {  // the end
            const uint32_t ps = np % kPtParts;
            ok = wait(pempty0 + 8 * ps, ((np / kPtParts) & 1) ^ 1);
            if (ok && lane == 0) {
                parts[ps].n = 0;
                mbar_arrive(pfull0 + 8 * ps);
            }
        }
        if (keys && lane == 0) a.cuts[blockIdx.x] = cut;
        if (!ok) {
            if (lane == 0) give_up();
            // the copies in flight land before the block ends
            for (int grp = 0; grp < 2; ++grp)
                if (nq[grp] > 0) mbar_wait(qfull0 + 8 * grp, (nq[grp] - 1) & 1);
            for (uint32_t back = 1; back <= issued && back <= slots; ++back) {
                const uint32_t g = issued - back;
                mbar_wait(full0 + 8 * (first + g % slots), (g / slots) & 1);
            }
        }
    } else if (warp < 3) {
        // ---- the products of group warp - 1: the whole warp waits, one thread, which the
        // compiler knows to be one, issues (descriptors stay in uniform registers) ----
        const int grp = warp - 1;
        const uint32_t tS = tmem + P::kS + 128u * grp, tP = tmem + P::kP + P::kPStep * grp, tO = tmem + P::kO + P::kPStep * grp;
        const uint64_t qd = sw128_kmajor_desc(smem_u32(sQ + grp * P::kTile));
        const uint64_t kd0 = sw128_kmajor_desc(smem_u32(ring)), vd0 = pt_v_desc(smem_u32(ring));
        uint32_t ks = 0, kph = 0, vs = KS, vph = 0;  // the next K and V tile
        uint32_t nq = 0, cs = 0, c = 0;              // Q tiles, blocks whose S is issued, blocks
        bool ok = true;
        auto step_k = [&]() {
            if (++ks == KS) {
                ks = 0;
                kph ^= 1;
            }
        };
        auto step_v = [&]() {
            if (++vs == S) {
                vs = KS;
                vph ^= 1;
            }
        };
        // S of the group's next block, issued by one thread once its keys are there and, with
        // P beside it, its columns have been read
        auto ready = [&]() {
            return wait(full0 + 8 * ks, kph) && (!P::kApart || cs == 0 || wait(sread0 + 8 * grp, (cs - 1) & 1));
        };
        auto issue = [&](bool last) {
            const uint64_t kd = kd0 + ks * (P::kTile >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                tc_mma<true>(tS, qd + 1024u * (kk >> 2) + 2u * (kk & 3), kd + 1024u * (kk >> 2) + 2u * (kk & 3), IDESC_S,
                             kk != 0 ? 1u : 0u);
            tc_commit(sfull0 + 8 * grp);  // S, and every product before it
            tc_commit(empty0 + 8 * ks);
            if (last) tc_commit(qempty0 + 8 * grp);
        };
        auto issued = [&]() {
            __syncwarp();
            step_k();
            ++cs;
        };
        for (uint32_t np = 0; ok; ++np) {
            const uint32_t ps = np % kPtParts;
            if (!wait(pfull0 + 8 * ps, (np / kPtParts) & 1)) {
                ok = false;
                break;
            }
            const PtPart p = parts[ps];
            if (p.n == 0) break;
            const int n = pt_share(a, p, grp).n;
            if (n > 0) {
                ok = wait(qfull0 + 8 * grp, nq++ & 1) && ready();
                if (!ok) break;
                tc_fence_after();
                if (pt_elect()) issue(n == 1);
                issued();
            }
            for (int i = 0; ok && i < n; ++i) {
                const bool more = i + 1 < n;
                if (P::kApart && more) {
                    if (!(ok = ready())) break;
                    tc_fence_after();
                    if (pt_elect()) issue(i + 2 == n);
                    issued();
                }
                // the first 64 keys while the others are exponentiated
                if (!(ok = wait(full0 + 8 * vs, vph) && wait(probs0 + 16 * grp, c & 1))) break;
                tc_fence_after();
                const uint64_t vd = vd0 + vs * (P::kTile >> 4);
                if (pt_elect()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        pt_mma_ts(tO, tP + 8u * kk, vd + 128u * kk, IDESC_O, (kk != 0 || i != 0) ? 1u : 0u);
                    tc_commit(pvhalf0 + 8 * grp);
                }
                __syncwarp();
                if (!P::kApart && more && !(ok = ready())) break;
                if (!(ok = wait(probs0 + 16 * grp + 8, c & 1))) break;
                tc_fence_after();
                if (pt_elect()) {
#pragma unroll
                    for (int kk = 4; kk < 8; ++kk) pt_mma_ts(tO, tP + 8u * kk, vd + 128u * kk, IDESC_O, 1u);
                    if (P::kApart) tc_commit(pv0 + 8 * grp);
                    if (!more) tc_commit(ofull0 + 8 * grp);
                    if (!P::kApart && more) issue(i + 2 == n);
                    tc_commit(empty0 + 8 * vs);
                }
                if (!P::kApart && more)
                    issued();
                else
                    __syncwarp();
                ++c;
                step_v();
            }
            for (int i = n; ok && i < p.n; ++i) {  // the other group's blocks only
                if (!wait(full0 + 8 * ks, kph) || !wait(full0 + 8 * vs, vph)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive(empty0 + 8 * ks);
                    mbar_arrive(empty0 + 8 * vs);
                }
                step_k();
                step_v();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(pempty0 + 8 * ps);
        }
        if (!ok && lane == 0) give_up();
        // all products are done before the block ends
        if (pt_elect()) tc_commit(done0 + 8 * grp);
        __syncwarp();
        mbar_wait(done0 + 8 * grp, 0);
    } else if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPtHigh));
        // ---- softmax and output of a group: thread = row ----
        const int grp = (warp - 4) >> 2, q = warp & 3, row = 32 * q + lane;
        const int each = a.TQ / 2, tok = row / a.G, sub = row - tok * a.G;
        const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
        const uint32_t tS = tmem + lanes + P::kS + 128u * grp, tP = tmem + lanes + P::kP + P::kPStep * grp,
                       tO = tmem + lanes + P::kO + P::kPStep * grp;
        const float NEG = -INFINITY, sl2 = a.scale_log2;
        const uint64_t sl2x2 = pt_pack(sl2, sl2);
        uint32_t g = 0, np = 0, c = 0, no = 0;  // blocks of the parts so far, parts, blocks and outputs of the group
        uint32_t turns = 0;                     // blocks that both groups have taken turns with
        bool ok = true;
        for (; ok; ++np) {
            const uint32_t ps = np % kPtParts;
            if (!wait(pfull0 + 8 * ps, (np / kPtParts) & 1)) {
                ok = false;
                break;
            }
            const PtPart p = parts[ps];
            if (p.n == 0) break;
            const PtShare sh = pt_share(a, p, grp);
            // rows that are none see what the last one does (their results go nowhere)
            const bool live = tok < sh.tokens;
            const int lim = a.causal && live ? min(p.pos0 + grp * each + tok + 1, sh.seen) : sh.seen;
            const int wmin = __reduce_min_sync(0xffffffffu, lim);
            const int shared = P::kTurns ? min(sh.n, pt_share(a, p, grp ^ 1).n) : 0;  // blocks of both groups
            float m = NEG, l = 0.f;  // the reference of the exponents (raw score), the total
            // One block; MASKED: some of the warp's rows do not see all of its keys. Two copies of the
            // code, so that the one that nearly always runs is short and straight.
            auto block = [&](int i, auto masked) {
                const int k0 = (p.j0 + i) * kPtKeys;
                if (!wait(sfull0 + 8 * grp, c & 1)) return false;
                tc_fence_after();
                uint32_t sv[2][2][32];
                tmem_ld32_async(tS, sv[0][0]);
                tmem_ld32_async(tS + 32u, sv[0][1]);
                tmem_wait_ld(sv[0][0]);
                tmem_wait_ld(sv[0][1]);
                tmem_ld32_async(tS + 64u, sv[1][0]);
                tmem_ld32_async(tS + 96u, sv[1][1]);
                if (decltype(masked)::value && k0 + kPtKeys > p.seen) {
                    // values of keys that nobody sees
                    const uint32_t v = g + (uint32_t)i, vs = KS + v % VS;
                    if (!wait(full0 + 8 * vs, (v / VS) & 1)) return false;
                    if (k0 + row >= p.seen) {
                        uint8_t* dst = ring + vs * P::kTile + row * 128;
#pragma unroll
                        for (int x = 0; x < D / 8; ++x)
                            *reinterpret_cast<uint4*>(dst + (x >> 3) * kHalf + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                // group 0's turn comes first, for this block as for all before it
                if (P::kTurns && i < shared &&
                    (grp == 0 ? turns > 0 && !wait(turn0 + 32 + 8 * q, (turns - 1) & 1) : !wait(turn0 + 8 * q, turns & 1)))
                    return false;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t(&x)[2][32] = sv[half];
                    if (half == 1) {
                        tmem_wait_ld(x[0]);
                        tmem_wait_ld(x[1]);
                        if (P::kApart) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(sread0 + 8 * grp);
                        }
                    }
                    const int c0 = k0 + 64 * half;
                    if constexpr (decltype(masked)::value) {
#pragma unroll
                        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (c0 + 32 * ch + e >= lim) x[ch][e] = __float_as_uint(NEG);
                    }
                    auto top = [&]() {
                        float mx[4] = {NEG, NEG, NEG, NEG};
#pragma unroll
                        for (int e = 0; e < 16; e += 2)
#pragma unroll
                            for (int ch = 0; ch < 4; ++ch)
                                mx[ch] = pt_max3(mx[ch], __uint_as_float(x[ch >> 1][16 * (ch & 1) + e]),
                                                 __uint_as_float(x[ch >> 1][16 * (ch & 1) + e + 1]));
                        return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    };
                    uint32_t pk[2][16];
                    float sum;
                    auto exponentials = [&](float ref) {
                        const uint64_t nref = pt_pack(-ref * sl2, -ref * sl2);
                        uint64_t s2[2] = {0ull, 0ull};
#pragma unroll
                        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                float x0, x1;
                                pt_unpack(pt_fma2(pt_pack(__uint_as_float(x[ch][e]), __uint_as_float(x[ch][e + 1])), sl2x2,
                                                  nref),
                                          x0, x1);
                                const float p0 = pt_ex2(x0), p1 = pt_ex2(x1);
                                s2[(e >> 1) & 1] = pt_add2(s2[(e >> 1) & 1], pt_pack(p0, p1));
                                pk[ch][e >> 1] = pack_bf16x2(p0, p1);
                            }
                        float la, lb;
                        pt_unpack(pt_add2(s2[0], s2[1]), la, lb);
                        sum = la + lb;
                    };
                    // A row that has no reference yet (its scores so far were all -inf) sums up inf or NaN and so
                    // looks for one, except among keys that it does not see.
                    const bool first = half == 0 && i == 0, sees = !decltype(masked)::value || c0 < lim;
                    if (first) m = top();
                    exponentials((first || !sees) && m == NEG ? 0.f : m);
                    if (__builtin_expect(!first && __any_sync(0xffffffffu, live && !(sum <= kPtRise)), 0)) {
                        // The reference moves: the products so far are done, what they summed is scaled, and
                        // these keys are exponentiated again. (Rows that are none have no say: their q
                        // is whatever the shared memory held, and results would not repeat.)
                        if (half == 1 ? !wait(pvhalf0 + 8 * grp, c & 1)
                                      : P::kApart && !wait(pv0 + 8 * grp, (c - 1) & 1)) return false;
                        tc_fence_after();
                        const float now = fmaxf(m, top());
                        const float alpha = pt_ex2((m - (now == NEG ? 0.f : now)) * sl2);
                        m = now;
                        l *= alpha;
#pragma unroll 1
                        for (int h = 0; h < D; h += 16) {
                            uint32_t ov[16];
                            tmem_ld16(tO + h, ov);
#pragma unroll
                            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                            pt_st16(tO + h, ov);
                        }
                        exponentials(m == NEG ? 0.f : m);
                    }
                    l += sum;
                    if (P::kTurns && half == 1 && i < shared) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(turn0 + 32 * grp + 8 * q);
                        ++turns;
                    }
                    // with P beside S, the product that read the last block's probabilities is done
                    if (P::kApart && half == 0 && c > 0) {
                        if (!wait(pv0 + 8 * grp, (c - 1) & 1)) return false;
                        tc_fence_after();
                    }
                    pt_st16(tP + 32u * half, pk[0]);
                    pt_st16(tP + 32u * half + 16u, pk[1]);
                    pt_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(probs0 + 16 * grp + 8 * half);
                }
                return true;
            };
            for (int i = 0; ok && i < sh.n; ++i, ++c)
                ok = (p.j0 + i + 1) * kPtKeys > wmin ? block(i, std::true_type()) : block(i, std::false_type());
            if (!ok) break;
            if (sh.tokens > 0) {
                if (sh.n > 0) {
                    if (!wait(ofull0 + 8 * grp, no++ & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                }
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const int head = p.h * a.G + sub, at = grp * each * a.G + row;  // row of the tile
                const size_t n = (size_t)p.row0 + grp * each + tok;
#pragma unroll
                for (int h = 0; h < D / 32; ++h) {
                    uint32_t ov[32];
                    if (sh.n > 0) {
                        tmem_ld32_async(tO + 32u * h, ov);
                        tmem_wait_ld(ov);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] = 0u;
                    }
                    if (!live) continue;
                    if (p.slot < 0) {
                        uint4* dst = reinterpret_cast<uint4*>(a.out + n * a.ldo + (size_t)head * D + 32 * h);
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            uint32_t x[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)  // a row without keys is 0 whatever O holds
                                x[e] = l == 0.f ? 0u : pack_bf16x2(__uint_as_float(ov[8 * v + 2 * e]) * inv,
                                                                   __uint_as_float(ov[8 * v + 2 * e + 1]) * inv);
                            dst[v] = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(a.sums + ((size_t)p.slot * 256 + at) * D + 32 * h);
#pragma unroll
                        for (int v = 0; v < 8; ++v) dst[v] = make_uint4(ov[4 * v], ov[4 * v + 1], ov[4 * v + 2], ov[4 * v + 3]);
                    }
                }
                if (live) {
                    const float base2 = m == NEG ? NEG : m * sl2;
                    if (p.slot >= 0)
                        a.stats[(size_t)p.slot * 256 + at] = make_float2(base2, l);
                    else if (a.lse)
                        a.lse[n * (a.Hkv * a.G) + head] = row_lse(base2, l);
                }
                tc_fence_before();
            }
            g += (uint32_t)p.n;
            __syncwarp();
            if (lane == 0) mbar_arrive(pempty0 + 8 * ps);
        }
        if (!ok && lane == 0) give_up();
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kPtTmem);
    }
}

template <int D>
int start(const PagedProblem& p) {
    using P = PtShape<D>;
    const int grid = p.sm_count;
    PagedArgs a;
    if (!paged_args(p, grid, 256, &a)) return LIN_ERR_WORKSPACE;
    const int each = 128 / a.G;  // tokens of a group
    a.TQ = 2 * each;
    a.lead = kPtLead;
    CUtensorMap tq, tk, tv;
    if (!paged_q_map(&tq, p, each) || !paged_kv_map(&tk, p, p.cache.k, kPtKeys) || !paged_kv_map(&tv, p, p.cache.v, kPtKeys))
        return LIN_ERR_CUDA;
    static std::atomic<unsigned long long> attr_set{0};
    if (ensure_smem_attr(attr_set, paged_tiles_kernel<D>, P::kSmem) != LIN_OK) return LIN_ERR_CUDA;
    static const int regs = []() {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, paged_tiles_kernel<D>) == cudaSuccess ? fa.numRegs : 0;
    }();
    if (regs < kPtLaunch) return LIN_ERR_UNSUPPORTED;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kPtThreads);
    cfg.dynamicSmemBytes = P::kSmem;
    cfg.stream = p.stream;
    cfg.attrs = &attr;
    cfg.numAttrs = p.early_start ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, paged_tiles_kernel<D>, tq, tk, tv, a) != cudaSuccess) return LIN_ERR_CUDA;
    if (cudaGetLastError() != cudaSuccess) return LIN_ERR_CUDA;
    return launch_paged_join(p, a, grid, 256);
}

}  // namespace

size_t paged_tiles_workspace(int sm_count, int D) { return paged_workspace(sm_count, 256, D); }

int launch_paged_tiles(const PagedProblem& p) {
    return p.cache.head_dim == 64 ? start<64>(p) : start<128>(p);
}

}  // namespace lin

// C ABI of the linear-layer library: context, argument validation, the
// per-shape dispatch table and the launches. No host fallback exists: when a
// kernel cannot run, the call returns an error.
//
// Dispatch ("Optimizing a GPT-2-class transformer on a GPU", Act II: route each
// shape to its measured winner; "Writing a CUDA matmul that catches cuBLAS",
// "One kernel was never going to be enough": tile and split chosen per shape):
//   BF16, M <= 16        -> skinny W stream (HBM-bound), split-K inside a
//                           thread-block cluster, reduced through DSMEM
//   BF16, M > 16 ; TF32  -> tcgen05 kernel, N tile chosen for wave efficiency
//   FP32                 -> FFMA kernel; 64x64 tiles + split-K when 128x128
//                           tiles cannot fill the SMs
//   K == 0               -> fill Y = act(bias)
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <vector>
#include <new>
#include <utility>

#include "internal.h"
#include "device_common.cuh"

// A measured winner installed for one exact call signature.
struct lin_override {
    int M, N, K, precision, epilogue;
    lin_plan plan;
};

struct lin_ctx {
    int device;
    int sm_count;
    void* workspace;
    size_t workspace_bytes;
    int* dev_status;
    int early_level;   // LIN_OPT_EARLY_START: 0 none, 1 W and bias, 2 also X
    bool programmatic; // LIN_OPT_PROGRAMMATIC_LAUNCH
    bool adaptive;     // LIN_OPT_ADAPTIVE_PLANS
    lin_plan last_plan;
    std::mutex override_mu;
    std::vector<lin_override> overrides;  // consulted by lin_forward before the table
};

namespace lin {
namespace {

template <bool BF16, bool GELU>
__global__ void fill_kernel(int M, int N, const float* bias, const void* R, void* Y) {
    const size_t total = (size_t)M * N;
    for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < total; i += (size_t)gridDim.x * blockDim.x) {
        const int n = (int)(i % N);
        const float v = epilogue<GELU>(0.f, bias ? bias[n] : 0.f);
        if constexpr (BF16)
            static_cast<uint16_t*>(Y)[i] =
                f32_to_bf16_bits(v + (R ? bf16_bits_to_f32(static_cast<const uint16_t*>(R)[i]) : 0.f));
        else
            static_cast<float*>(Y)[i] = v + (R ? static_cast<const float*>(R)[i] : 0.f);
    }
}

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

void plan_common(lin_plan* p, int kernel, int variant) {
    std::memset(p, 0, sizeof(*p));
    p->kernel = kernel;
    p->variant = variant;
    p->splits = 1;
}

int make_skinny(int sm, int variant, int splits, int M, int N, int K, size_t /*ws*/, lin_plan* p) {
    if (variant < 0 || variant >= kSkinnyVariants || M > 16 || M < 1 || N < 1 || K < 1) return LIN_ERR_UNSUPPORTED;
    const SkinnyCfg c = kSkinnyCfg[variant];
    const int tiles = ceil_div(N, 128);
    const int kblocks = ceil_div(K, 64 * c.kbox);
    int S = splits;
    if (S <= 0) {
        // Cluster split-K: the largest power of two (<= 8, the portable cluster
        // size) keeping the grid within the CTAs the SMs hold at once (one per SM,
        // two for the small ring), with >= 2 K stages per CTA.
        const long long slots = variant == kSkinnyTwoPerSm ? 2LL * sm : (long long)sm;
        S = 1;
        while (S < 8 && (long long)tiles * S * 2 <= slots && 2 * S <= kblocks) S *= 2;
    }
    if (S != 1 && S != 2 && S != 4 && S != 8) return LIN_ERR_UNSUPPORTED;
    plan_common(p, LIN_KERNEL_SKINNY, variant);
    p->bm = 16;
    p->bn = 128;
    p->bk = 64 * c.kbox;
    p->splits = S;
    p->stages = c.stages;
    p->grid_x = tiles;
    p->grid_y = S;
    p->grid_z = 1;
    p->threads = kSkinnyThreads;
    p->workspace_bytes = 0;
    return LIN_OK;
}

// `min_steps`: the fewest K steps of 32 a split keeps (4 for a call that runs
// alone; a call that overlaps an independent predecessor passes more, see run()).
int make_ffma(int sm, int variant, int splits, int M, int N, int K, size_t ws, lin_plan* p, int min_steps = 4) {
    if (M < 1 || N < 1 || K < 1) return LIN_ERR_UNSUPPORTED;
    if (variant < 0) {
        // 128x128 tiles when they give at least one full wave, else 64x64 + split-K.
        // The 128x128 tiles take K in steps of 64 over 3 stages (variant 2):
        // half the barriers of steps of 32 (4096^3: 50.2 -> 53.2 TF/s).
        const long long big = (long long)ceil_div(M, kFfmaCfg[0].bm) * ceil_div(N, kFfmaCfg[0].bn);
        variant = big >= sm ? 2 : 1;
    }
    if (variant >= kFfmaVariants) return LIN_ERR_UNSUPPORTED;
    const FfmaCfg c = kFfmaCfg[variant];
    const int gx = ceil_div(N, c.bn), gy = ceil_div(M, c.bm);
    const int tiles = gx * gy;
    const int nkb = ceil_div(K, c.bk);
    int S = splits;
    if (S <= 0) {
        // Fill the resident slots (one 128x128 CTA per SM, two 64x64 CTAs per
        // SM) without starting a second wave, keeping >= 4 K steps per split
        // (measured on the GPT-2 M = 128 shapes: qkv 22 -> 17 us, fc1 29 -> 23 us
        // against rounding the split up to one CTA per SM).
        const int slots = (variant == 1 || variant == 3) ? 2 * sm : sm;  // resident CTAs
        S = tiles >= slots ? 1 : slots / tiles;
        // A short reduction is not split (256^3, 8 steps: 9.8 us whole against
        // 12.1 us in two halves, measured as isolated calls).
        const int max_s = nkb >= 16 && nkb / min_steps > 1 ? nkb / min_steps : 1;
        if (S > max_s) S = max_s;
        if (S < 1) S = 1;
        while (S > 1 && splitk_workspace_bytes(S, M, N) > ws) --S;
    }
    if (S > nkb) S = nkb;
    if (tiles > kMaxSplitTiles) S = 1;
    plan_common(p, LIN_KERNEL_FFMA, variant);
    p->bm = c.bm;
    p->bn = c.bn;
    p->bk = c.bk;
    p->splits = S;
    p->grid_x = gx;
    p->grid_y = gy;
    p->grid_z = S;
    p->threads = 256;
    p->workspace_bytes = (long long)splitk_workspace_bytes(S, M, N);
    return LIN_OK;
}

// GEMV (FP32 / TF32 M <= 8, BF16 M <= 4): X padded to 1, 2, 4 or 8 rows in shared memory;
// `width` CTAs of 8 warps (0 = as many as fit on the SMs at once, by shared
// memory and by threads) take the rows of W in turn.
int gemv_rows(int M) { return M <= 1 ? 1 : M <= 2 ? 2 : M <= 4 ? 4 : 8; }
bool gemv_fits(int M, int K, bool bf16) {
    return M >= 1 && M <= (bf16 ? kGemvMaxRowsBf16 : kGemvMaxRows) && K % (bf16 ? 8 : 4) == 0 &&
           (size_t)gemv_rows(M) * K * sizeof(float) <= (size_t)kGemvMaxSmem;
}
int make_gemv(int sm, int width, int M, int N, int K, bool bf16, lin_plan* p) {
    if (N < 1 || K < 1 || !gemv_fits(M, K, bf16)) return LIN_ERR_UNSUPPORTED;
    const int rows = gemv_rows(M);
    const long long smem = (long long)rows * K * 4 + 1024;
    long long per_sm = (228 * 1024) / smem;
    if (per_sm > 8) per_sm = 8;  // 2048 threads per SM
    if (per_sm < 1) per_sm = 1;
    long long grid = width > 0 ? width : (long long)sm * per_sm;
    const long long need = ((long long)N + 7) / 8;  // one row per warp and pass
    if (grid > need) grid = need;
    plan_common(p, LIN_KERNEL_GEMV, 0);
    p->bm = rows;
    p->bn = 8;
    p->bk = 0;
    p->splits = 1;
    p->stages = 0;
    p->grid_x = (int)grid;
    p->grid_y = 1;
    p->grid_z = 1;
    p->threads = 256;
    p->workspace_bytes = 0;
    return LIN_OK;
}

// Persistent tcgen05 kernel: `width` CTAs walk the 128 x BN output tiles
// (0 = one CTA per SM) in static round robin; pair variants walk 256 x BN
// tiles with one 2-CTA cluster (an SM pair) per tile (grid rounded down to
// even). `stream_k` (single-CTA variants, at least one tile per CTA): every CTA
// takes an equal share of the (tile, K stage) sequence instead (splits = 2).
// Default, from the measured M = 8192 GPT-2 shapes, the LM head and
// 4096^3 / 8192^3:
// * SM pair when each tile runs at least 64 K stages (K >= 4096 bf16 or 2048
//   tf32): there the pair's lighter shared-memory traffic wins (8192^3 bf16
//   1.91 vs 1.62 PF/s); with shorter K its per-tile synchronisation costs
//   more than it saves.
// * Otherwise whole single-CTA tiles, the N tile minimising rounds_eff(BN) x
//   r(BN), where rounds_eff is the mean of the average and the maximum tiles
//   per CTA (a back-to-back caller overlaps part of a ragged last round with
//   its next call) and r = 1, 0.9, 0.75 for BN = 256, 192, 128 is the measured
//   time of one round relative to BN = 256 (A is reloaded for every N tile, so
//   narrow tiles are slower per column).
// * Never stream-K by default: on the M = 8192 GPT-2 shapes it measured slower
//   than whole tiles both back to back (where the SMs that a ragged last round
//   frees start the next call early) and with the early start off (the cut
//   tiles' hand-over sits on the critical path). Explicit plans reach it.
int make_tc(int sm, int variant, int width, bool stream_k, int M, int N, int K, int esz, lin_plan* p,
            size_t ksplit_ws = 0) {
    if (M < 1 || N < 1 || K < 1 || width < 0) return LIN_ERR_UNSUPPORTED;
    const long long w0 = width > 0 ? width : sm;
    if (variant < 0) {
        // SM pairs for long K, unless the single-CTA tiles are so few that a K
        // split (below) is what fills the SMs.
        const long long tiles256 = (long long)ceil_div(M, 128) * ceil_div(N, 256);
        const bool want_pair = ceil_div(K, 128 / esz) >= 64 && !(ksplit_ws > 0 && tiles256 * 2 <= sm);
        double best = 0.0;
        for (int v = 0; v < kTcVariants; ++v) {
            if (kTcCfg[v].pair != want_pair) continue;
            const int bn = kTcCfg[v].bn;
            const long long items =
                (long long)(want_pair ? ceil_div(ceil_div(M, 128), 2) : ceil_div(M, 128)) * ceil_div(N, bn);
            long long slots = w0;
            if (want_pair) slots = slots / 2 > 0 ? slots / 2 : 1;
            const double avg = (double)items / (double)slots;
            const double mx = (double)((items + slots - 1) / slots);
            const double rel = bn == 256 ? 1.0 : bn == 192 ? 0.9 : 0.75;
            const double cost = 0.5 * (avg + mx) * rel;
            if (variant < 0 || cost < best) {
                best = cost;
                variant = v;
            }
        }
    }
    if (variant >= kTcVariants) return LIN_ERR_UNSUPPORTED;
    const bool pair = kTcCfg[variant].pair;
    const long long items = (long long)(pair ? ceil_div(ceil_div(M, 128), 2) : ceil_div(M, 128)) *
                            ceil_div(N, kTcCfg[variant].bn);
    long long w = w0;
    if (pair) {
        if (stream_k) return LIN_ERR_UNSUPPORTED;
        w = (w / 2 < items ? w / 2 : items) * 2;
        if (w < 2) w = 2;
    } else if (w > items) {
        w = items;
    }
    if (stream_k && (items < w || w > kTcMaxStreamKCtas)) return LIN_ERR_UNSUPPORTED;
    plan_common(p, LIN_KERNEL_TC, variant);
    p->bm = 128;
    p->bn = kTcCfg[variant].bn;
    p->bk = 0;  // 128 bytes of K: 64 bf16 or 32 fp32
    p->splits = stream_k ? 2 : 1;
    p->stages = 0;  // derived in the kernel from the shared-memory budget
    p->grid_x = (int)w;
    p->grid_y = 1;
    p->grid_z = 1;
    p->threads = kTcThreads;
    p->workspace_bytes = stream_k ? (long long)tc_streamk_workspace_bytes((int)w, p->bn) : 0;
    // Few tiles with a long K (and room in the workspace): split K so that
    // the (tile, split) items fill the SMs; grid_z = splits.
    if (!pair && !stream_k && ksplit_ws > 0) {
        const int S = tc_ksplits(items, ceil_div(K, 128 / esz), sm, ksplit_ws, p->bn);
        if (S > 1) {
            const long long w2 = width > 0 ? width : sm;
            p->grid_z = S;
            p->grid_x = (int)(items * S < w2 ? items * S : w2);
            p->workspace_bytes = (long long)tc_ksplit_workspace_bytes(items, S, p->bn);
        }
        // A ragged last round (more tiles than CTAs) is not split by default:
        // measured on GB300 as isolated calls, splitting the last round's tiles
        // in K was slower than running them whole (8192 x 768 x 768: 20.7 against
        // 13.8 us; 8192 x 3072 x 768 with GELU: 43.0 against 36.3 us; 8192 x 768 x
        // 3072: 37.6 against 36.5 us): the split pieces' partial sums pass through
        // the L2 and the last piece's reduction sits on the critical path.
        // Explicit plans (grid_z > 1 with more tiles than CTAs) still run it.
    }
    return LIN_OK;
}

bool valid_enums(int epilogue, int precision) {
    return (epilogue == LIN_EPI_NONE || epilogue == LIN_EPI_GELU_TANH) &&
           (precision == LIN_PREC_FP32 || precision == LIN_PREC_TF32 || precision == LIN_PREC_BF16);
}

int plan_default(int sm, int M, int N, int K, int precision, size_t ws, lin_plan* p) {
    if (M == 0 || N == 0) {
        plan_common(p, LIN_KERNEL_NONE, 0);
        return LIN_OK;
    }
    if (K == 0) {
        plan_common(p, LIN_KERNEL_FILL, 0);
        p->grid_x = ceil_div((long long)M * N, 256) < 4 * sm ? ceil_div((long long)M * N, 256) : 4 * sm;
        p->grid_y = p->grid_z = 1;
        p->threads = 256;
        return LIN_OK;
    }
    switch (precision) {
        case LIN_PREC_BF16:
            // The GEMV only for one row and at most one 128-row tile of W per
            // SM; measured back to back, the skinny tensor-core kernel wins
            // everywhere else (4 x 50257 x 768: 12.1 against 41.5 us; one row
            // of 50257: 11.9 against 14.3 us; one row of 2304: 1.9 against 1.3 us).
            if (M == 1 && ceil_div(N, 128) <= sm && gemv_fits(M, K, true)) return make_gemv(sm, 0, M, N, K, true, p);
            // More row tiles than SMs: the 6 x 1 ring (two CTAs per SM) without a
            // split, so the tiles run in fewer waves (measured on the last
            // token's logits, 50257 rows: 15.7 -> 12.1 us). Otherwise the 5 x 1
            // ring split over a cluster (two CTAs per SM): the next call's CTAs
            // start beside this call's and stream their W into L2 meanwhile.
            if (M <= 16) return make_skinny(sm, ceil_div(N, 128) > sm ? 1 : kSkinnyTwoPerSm, 0, M, N, K, ws, p);
            return make_tc(sm, -1, 0, false, M, N, K, 2, p, ws);
        case LIN_PREC_TF32:
            // A few rows are a weight stream: the exact-fp32 GEMV is as fast as
            // any tensor-core tile there, and more accurate than TF32.
            if (gemv_fits(M, K, false)) return make_gemv(sm, 0, M, N, K, false, p);
            return make_tc(sm, -1, 0, false, M, N, K, 4, p, ws);
        default:
            if (gemv_fits(M, K, false)) return make_gemv(sm, 0, M, N, K, false, p);
            return make_ffma(sm, -1, 0, M, N, K, ws, p);
    }
}

bool overlaps(const void* a, size_t an, const void* b, size_t bn) {
    if (!a || !b || an == 0 || bn == 0) return false;
    const char* pa = static_cast<const char*>(a);
    const char* pb = static_cast<const char*>(b);
    return pa < pb + bn && pb < pa + an;
}

// Makes `dev` the thread's current device, and its context the current one.
struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) != cudaSuccess) { ok = false; return; }
        if ((prev != dev || !thread_has_context()) && cudaSetDevice(dev) != cudaSuccess) ok = false;
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

struct Range {
    const void* p;
    size_t bytes;
};

// What the calls on each stream (process-wide) may still be writing. A kernel that
// lets its successor start before its own dependency wait is behind it while the call
// before both still runs, so a call's inputs are compared with the outputs of all calls
// since the last one that is known to start, or to let others start, only when
// everything before it has finished. Such a call begins the list anew.
constexpr int kOutputs = 64;
struct StreamOutputs {
    cudaStream_t stream;
    int n;
    bool more;  // there are outputs that the list has no place for
    uintptr_t lo[kOutputs], hi[kOutputs];
};
std::mutex g_outputs_mu;
StreamOutputs g_outputs[64];
int g_streams = 0;

// The stream's list, under the mutex. A new one is empty; once the table has been full,
// it may be one that had to make room for another.
StreamOutputs& outputs_of(cudaStream_t st, bool* known) {
    for (int i = 0; i < std::min(g_streams, 64); ++i)
        if (g_outputs[i].stream == st) {
            *known = true;
            return g_outputs[i];
        }
    *known = false;
    StreamOutputs& o = g_outputs[g_streams % 64];
    o.stream = st;
    o.n = 0;
    o.more = g_streams >= 64;
    if (++g_streams == 128) g_streams = 64;
    return o;
}

void add_output(StreamOutputs& o, Range y) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(y.p), hi = lo + y.bytes;
    for (int i = 0; i < o.n; ++i)
        if (o.lo[i] <= lo && hi <= o.hi[i]) {  // there already: now the newest
            std::swap(o.lo[i], o.lo[o.n - 1]);
            std::swap(o.hi[i], o.hi[o.n - 1]);
            return;
        }
    if (o.n == kOutputs) {
        o.more = true;
        return;
    }
    o.lo[o.n] = lo;
    o.hi[o.n++] = hi;
}

struct EarlyReads {
    bool w = false;        // W and bias may be read before the dependency wait
    bool x = false;        // and X
    bool known = false;    // the stream has had a call
    bool ordered = false;  // the call has to be launched in plain stream order
};

// Which inputs a call may read early, at the context's level; records Y. An input that
// the newest call writes is read after the wait, which is for that call. One that
// an older call writes, or that cannot be told from one, makes the call an ordered one.
EarlyReads early_reads(cudaStream_t st, int level, Range w, Range bias, Range x, Range y) {
    std::lock_guard<std::mutex> lk(g_outputs_mu);
    EarlyReads r;
    StreamOutputs& o = outputs_of(st, &r.known);
    if (level >= 1) {
        bool older = o.more || o.n == kOutputs;
        auto hits = [&](Range in) {
            const uintptr_t lo = reinterpret_cast<uintptr_t>(in.p), hi = lo + in.bytes;
            bool hit = false;
            for (int i = 0; in.p && in.bytes && i < o.n; ++i)
                if (lo < o.hi[i] && o.lo[i] < hi) {
                    hit = true;
                    older = older || i != o.n - 1;
                }
            return hit;
        };
        const bool bias_hit = hits(bias);
        r.w = !hits(w) && !bias_hit;
        r.x = level >= 2 && r.w && !hits(x);
        if (older) {
            r.w = r.x = false;
            r.ordered = true;
            o.n = 0;
            o.more = false;
        }
    }
    add_output(o, y);
    return r;
}

// Record another output of a call on `st`.
void note_output(cudaStream_t st, Range y) {
    std::lock_guard<std::mutex> lk(g_outputs_mu);
    bool known;
    add_output(outputs_of(st, &known), y);
}

}  // namespace

void note_ordered_output(cudaStream_t st, const void* p, size_t bytes) {
    std::lock_guard<std::mutex> lk(g_outputs_mu);
    bool known;
    StreamOutputs& o = outputs_of(st, &known);
    o.n = 0;
    o.more = false;
    add_output(o, Range{p, bytes});
}

namespace {

int check_plan_fits(const lin_plan& p, int M, int N, int K, int precision) {
    switch (p.kernel) {
        case LIN_KERNEL_NONE: return (M == 0 || N == 0) ? LIN_OK : LIN_ERR_UNSUPPORTED;
        case LIN_KERNEL_FILL: return (K == 0 && p.grid_x > 0) ? LIN_OK : LIN_ERR_UNSUPPORTED;
        case LIN_KERNEL_SKINNY: {
            if (precision != LIN_PREC_BF16 || M > 16 || K == 0) return LIN_ERR_UNSUPPORTED;
            if (p.variant < 0 || p.variant >= kSkinnyVariants) return LIN_ERR_UNSUPPORTED;
            if (p.splits != 1 && p.splits != 2 && p.splits != 4 && p.splits != 8) return LIN_ERR_UNSUPPORTED;
            if (p.grid_x != ceil_div(N, 128) || p.grid_y != p.splits) return LIN_ERR_UNSUPPORTED;
            return LIN_OK;
        }
        case LIN_KERNEL_FFMA: {
            if (precision != LIN_PREC_FP32 || K == 0) return LIN_ERR_UNSUPPORTED;
            if (p.variant < 0 || p.variant >= kFfmaVariants || p.splits < 1) return LIN_ERR_UNSUPPORTED;
            const FfmaCfg c = kFfmaCfg[p.variant];
            if (p.bk != c.bk || p.grid_x != ceil_div(N, c.bn) || p.grid_y != ceil_div(M, c.bm) ||
                p.grid_z != p.splits || p.splits > ceil_div(K, c.bk) ||
                (p.splits > 1 && (long long)p.grid_x * p.grid_y > kMaxSplitTiles))
                return LIN_ERR_UNSUPPORTED;
            return LIN_OK;
        }
        case LIN_KERNEL_TC: {
            if (precision == LIN_PREC_FP32 || K == 0) return LIN_ERR_UNSUPPORTED;
            if (p.variant < 0 || p.variant >= kTcVariants || (p.splits != 1 && p.splits != 2))
                return LIN_ERR_UNSUPPORTED;
            const bool pair = kTcCfg[p.variant].pair;
            const long long items = (long long)(pair ? ceil_div(ceil_div(M, 128), 2) : ceil_div(M, 128)) *
                                    ceil_div(N, kTcCfg[p.variant].bn);
            const long long ctas = pair ? 2 * items : items * (p.grid_z > 1 ? p.grid_z : 1);
            if (p.bn != kTcCfg[p.variant].bn || p.grid_x < 1 || p.grid_x > ctas || p.grid_y != 1 ||
                (pair && p.grid_x % 2 != 0))
                return LIN_ERR_UNSUPPORTED;
            if (p.splits == 2 &&
                (pair || p.grid_x > kTcMaxStreamKCtas ||
                 p.workspace_bytes < (long long)tc_streamk_workspace_bytes(p.grid_x, p.bn)))
                return LIN_ERR_UNSUPPORTED;
            if (p.grid_z > 1) {  // K split (of every tile, or of the tiles past the whole rounds)
                const long long tiles = (long long)ceil_div(M, 128) * ceil_div(N, p.bn);
                const long long split_tiles = tiles - tc_tail_whole(tiles, p.grid_x);
                if (pair || p.splits != 1 || p.grid_z > 16 || split_tiles < 1 || split_tiles > kTcMaxKSplitTiles ||
                    ceil_div(K, precision == LIN_PREC_BF16 ? 64 : 32) < p.grid_z ||
                    p.workspace_bytes < (long long)tc_ksplit_workspace_bytes(split_tiles, p.grid_z, p.bn))
                    return LIN_ERR_UNSUPPORTED;
            } else if (p.grid_z != 1) {
                return LIN_ERR_UNSUPPORTED;
            }
            return LIN_OK;
        }
        case LIN_KERNEL_GEMV: {
            if (K == 0 || !gemv_fits(M, K, precision == LIN_PREC_BF16)) return LIN_ERR_UNSUPPORTED;
            if (p.bm != gemv_rows(M) || p.grid_x < 1 || p.grid_y != 1 || p.grid_z != 1) return LIN_ERR_UNSUPPORTED;
            return LIN_OK;
        }
        default: return LIN_ERR_UNSUPPORTED;
    }
}

int run(lin_ctx* ctx, const lin_plan& plan_in, int M, int N, int K, const void* X, const void* W, const float* bias,
        void* Y, int epilogue, int precision, void* stream, bool adaptive, const void* R = nullptr) {
    lin_plan plan = plan_in;
    if (!ctx || M < 0 || N < 0 || K < 0 || !valid_enums(epilogue, precision)) return LIN_ERR_ARG;
    if (M == 0 || N == 0) return plan.kernel == LIN_KERNEL_NONE ? LIN_OK : LIN_ERR_UNSUPPORTED;
    if (!Y || (K > 0 && (!X || !W))) return LIN_ERR_ARG;
    const size_t ein = precision == LIN_PREC_BF16 ? 2 : 4;
    const size_t eout = ein;
    const size_t ybytes = (size_t)M * N * eout;
    if (overlaps(Y, ybytes, X, (size_t)M * K * ein) || overlaps(Y, ybytes, W, (size_t)N * K * ein) ||
        overlaps(Y, ybytes, bias, bias ? (size_t)N * 4 : 0))
        return LIN_ERR_ARG;
    if (R && R != Y && overlaps(Y, ybytes, R, ybytes)) return LIN_ERR_ARG;  // in place, or apart
    if (K > 0 && (((uintptr_t)X | (uintptr_t)W) % 16 != 0 || ((size_t)K * ein) % 16 != 0)) return LIN_ERR_ALIGN;
    if ((((uintptr_t)Y | (uintptr_t)R) % eout) != 0 || ((uintptr_t)bias % 4) != 0) return LIN_ERR_ALIGN;
    const int fit = check_plan_fits(plan, M, N, K, precision);
    if (fit != LIN_OK) return fit;
    if ((size_t)plan.workspace_bytes > ctx->workspace_bytes) return LIN_ERR_WORKSPACE;

    DeviceGuard guard(ctx->device);
    if (!guard.ok) return LIN_ERR_CUDA;
    Problem p;
    p.M = M;
    p.N = N;
    p.K = K;
    p.X = X;
    p.W = W;
    p.bias = bias;
    p.Y = Y;
    p.residual = R;
    p.epilogue = epilogue;
    p.precision = precision;
    p.stream = static_cast<cudaStream_t>(stream);
    p.workspace = ctx->workspace;
    p.workspace_bytes = ctx->workspace_bytes;
    p.dev_status = ctx->dev_status;
    p.sm_count = ctx->sm_count;
    const EarlyReads early = early_reads(p.stream, ctx->early_level, Range{W, (size_t)N * K * ein},
                                         Range{bias, bias ? (size_t)N * 4 : 0}, Range{X, (size_t)M * K * ein},
                                         Range{Y, ybytes});
    const bool known = early.known;
    p.early_start = ctx->programmatic && !early.ordered;
    p.early_w = p.early_start && early.w;
    p.early_x = p.early_w && early.x;
    // An independent call right after another call on this stream overlaps it:
    // the skinny stream then needs no K split to fill the SMs (the concurrent
    // calls do), and skipping the split saves its reduction.
    // The two-per-SM ring keeps its variant (the same summation order, so the
    // same bits) and takes the split that leaves one CTA slot per SM to the
    // neighbouring call (measured on 16 x 4096 x 4096: cluster 4 5.4 us per
    // call back to back against 7.2 us for cluster 8); the deep rings drop the
    // split altogether.
    if (adaptive && ctx->adaptive && known && p.early_x && plan.kernel == LIN_KERNEL_SKINNY && plan.splits > 1) {
        lin_plan narrow;
        int S = 1;
        if (plan.variant == kSkinnyTwoPerSm) {
            const long long tiles = ceil_div(N, 128), kblocks = ceil_div(K, 64);
            while (S < 8 && tiles * S * 2 <= ctx->sm_count && 2 * S <= kblocks) S *= 2;
        }
        if (S < plan.splits && make_skinny(ctx->sm_count, plan.variant, S, M, N, K, ctx->workspace_bytes, &narrow) == LIN_OK)
            plan = narrow;
    }
    // Likewise a tensor-core K split (measured: it helps an isolated call and
    // costs a back-to-back one).
    if (adaptive && ctx->adaptive && known && p.early_x && plan.kernel == LIN_KERNEL_TC && plan.grid_z > 1) {
        lin_plan whole;
        if (make_tc(ctx->sm_count, -1, 0, false, M, N, K, precision == LIN_PREC_BF16 ? 2 : 4, &whole) == LIN_OK)
            plan = whole;
    }
    // And the FFMA split: back to back, the next call's CTAs fill the SMs that
    // a split would, so a split must now pay for its reduction with a long K
    // (>= 24 steps of 32 each; measured on the GPT-2 M = 128 layers: proj
    // 8.6 -> 4.1 us, qkv 14.7 -> 11.9 us, fc2 keeps a split of 4).
    // Without a split, wide outputs of a few rows take 128 x 64 tiles (two CTAs
    // per SM; measured back to back at M = 128, K = 768: N = 2304 10.5 -> 9.4 us,
    // N = 3072 14.3 -> 13.4 us; N = 768 unchanged).
    if (adaptive && ctx->adaptive && known && p.early_x && plan.kernel == LIN_KERNEL_FFMA && plan.splits > 1) {
        lin_plan fewer;
        if (make_ffma(ctx->sm_count, -1, 0, M, N, K, ctx->workspace_bytes, &fewer, 24) == LIN_OK) {
            plan = fewer;
            lin_plan wide;
            if (plan.splits == 1 && plan.variant == 1 && M <= 128 && N >= 2048 &&
                make_ffma(ctx->sm_count, 3, 1, M, N, K, ctx->workspace_bytes, &wide) == LIN_OK)
                plan = wide;
        }
    }
    ctx->last_plan = plan;
    switch (plan.kernel) {
        case LIN_KERNEL_FILL: return launch_fill(p);
        case LIN_KERNEL_SKINNY: return launch_skinny(p, plan);
        case LIN_KERNEL_FFMA: return launch_ffma(p, plan);
        case LIN_KERNEL_TC: return launch_tc(p, plan);
        case LIN_KERNEL_GEMV: return launch_gemv(p, plan);
        default: return LIN_ERR_UNSUPPORTED;
    }
}

}  // namespace

int launch_fill(const Problem& p) {
    const long long total = (long long)p.M * p.N;
    int grid = (int)((total + 255) / 256);
    if (grid > 4 * p.sm_count) grid = 4 * p.sm_count;
    if (grid < 1) grid = 1;
    const bool bf16 = p.precision == LIN_PREC_BF16, gelu = p.epilogue == LIN_EPI_GELU_TANH;
    const void* R = p.residual;
    if (bf16 && gelu) fill_kernel<true, true><<<grid, 256, 0, p.stream>>>(p.M, p.N, p.bias, R, p.Y);
    else if (bf16) fill_kernel<true, false><<<grid, 256, 0, p.stream>>>(p.M, p.N, p.bias, R, p.Y);
    else if (gelu) fill_kernel<false, true><<<grid, 256, 0, p.stream>>>(p.M, p.N, p.bias, R, p.Y);
    else fill_kernel<false, false><<<grid, 256, 0, p.stream>>>(p.M, p.N, p.bias, R, p.Y);
    return cudaGetLastError() == cudaSuccess ? LIN_OK : LIN_ERR_CUDA;
}

}  // namespace lin

extern "C" {

int lin_abi_version(void) { return LIN_ABI_VERSION; }

int lin_timeline(int kernel, void* host_dst, size_t bytes, int clear) {
    if ((host_dst == nullptr) != (bytes == 0)) return LIN_ERR_ARG;
    switch (kernel) {
        case LIN_KERNEL_TC: return lin::timeline_copy_tc(host_dst, bytes, clear != 0);
        case LIN_KERNEL_SKINNY: return lin::timeline_copy_skinny(host_dst, bytes, clear != 0);
        case LIN_TIMELINE_ATTENTION: return lin::timeline_copy_attn(host_dst, bytes, clear != 0);
        default: return LIN_ERR_ARG;
    }
}

const char* lin_strerror(int status) {
    switch (status) {
        case LIN_OK: return "success";
        case LIN_ERR_ARG: return "invalid argument (NULL pointer, negative size, unknown enum, or Y overlapping an input)";
        case LIN_ERR_ALIGN: return "misaligned operand (X and W need 16-byte alignment and K*element size a multiple of 16)";
        case LIN_ERR_WORKSPACE: return "plan needs more workspace than the context holds";
        case LIN_ERR_CUDA: return "CUDA runtime error or kernel launch failure";
        case LIN_ERR_DEVICE_TIMEOUT: return "a kernel gave up a bounded wait; its output is incomplete";
        case LIN_ERR_UNSUPPORTED: return "the plan's kernel cannot run this shape or precision";
        default: return "unknown status";
    }
}

int lin_create(lin_ctx** out, int device, size_t max_workspace_bytes) {
    if (!out) return LIN_ERR_ARG;
    *out = nullptr;
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || device < 0 || device >= ndev) {
        cudaGetLastError();
        return LIN_ERR_CUDA;
    }
    lin::DeviceGuard guard(device);
    if (!guard.ok) return LIN_ERR_CUDA;
    lin_ctx* c = new (std::nothrow) lin_ctx();
    if (!c) return LIN_ERR_CUDA;
    c->device = device;
    c->early_level = 0;
    c->programmatic = true;
    c->adaptive = true;
    std::memset(&c->last_plan, 0, sizeof(c->last_plan));
    c->workspace_bytes = max_workspace_bytes ? max_workspace_bytes : ((size_t)64 << 20);
    if (cudaDeviceGetAttribute(&c->sm_count, cudaDevAttrMultiProcessorCount, device) != cudaSuccess ||
        cudaMalloc(&c->workspace, c->workspace_bytes) != cudaSuccess ||
        cudaMemset(c->workspace, 0, c->workspace_bytes) != cudaSuccess ||
        cudaMalloc(reinterpret_cast<void**>(&c->dev_status), sizeof(int)) != cudaSuccess ||
        cudaMemset(c->dev_status, 0, sizeof(int)) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
        if (c->workspace) cudaFree(c->workspace);
        if (c->dev_status) cudaFree(c->dev_status);
        delete c;
        cudaGetLastError();
        return LIN_ERR_CUDA;
    }
    *out = c;
    return LIN_OK;
}

int lin_destroy(lin_ctx* ctx) {
    if (!ctx) return LIN_OK;
    int rc = LIN_OK;
    {
        lin::DeviceGuard guard(ctx->device);
        if (cudaDeviceSynchronize() != cudaSuccess) rc = LIN_ERR_CUDA;
        cudaFree(ctx->workspace);
        cudaFree(ctx->dev_status);
    }
    delete ctx;
    return rc;
}

int lin_ctx_last_plan(const lin_ctx* ctx, lin_plan* out) {
    if (!ctx || !out) return LIN_ERR_ARG;
    *out = ctx->last_plan;
    return LIN_OK;
}

int lin_set_option(lin_ctx* ctx, int option, long long value) {
    if (!ctx) return LIN_ERR_ARG;
    switch (option) {
        case LIN_OPT_EARLY_START:
            if (value < 0 || value > 2) return LIN_ERR_ARG;
            ctx->early_level = (int)value;
            return LIN_OK;
        case LIN_OPT_ADAPTIVE_PLANS:
            if (value != 0 && value != 1) return LIN_ERR_ARG;
            ctx->adaptive = value != 0;
            return LIN_OK;
        case LIN_OPT_PROGRAMMATIC_LAUNCH:
            if (value != 0 && value != 1) return LIN_ERR_ARG;
            ctx->programmatic = value != 0;
            return LIN_OK;
        default: return LIN_ERR_ARG;
    }
}

int lin_ctx_info(const lin_ctx* ctx, int* device, int* sm_count, size_t* workspace_bytes) {
    if (!ctx) return LIN_ERR_ARG;
    if (device) *device = ctx->device;
    if (sm_count) *sm_count = ctx->sm_count;
    if (workspace_bytes) *workspace_bytes = ctx->workspace_bytes;
    return LIN_OK;
}

int lin_plan_query(int sm_count, int M, int N, int K, int precision, int epilogue, size_t workspace_bytes,
                   lin_plan* out) {
    if (!out || sm_count < 1 || M < 0 || N < 0 || K < 0 || !lin::valid_enums(epilogue, precision)) return LIN_ERR_ARG;
    return lin::plan_default(sm_count, M, N, K, precision, workspace_bytes, out);
}

int lin_plan_check(const lin_plan* plan, int M, int N, int K, int precision, size_t workspace_bytes) {
    if (!plan || M < 0 || N < 0 || K < 0 || !lin::valid_enums(0, precision)) return LIN_ERR_ARG;
    if (M == 0 || N == 0) return plan->kernel == LIN_KERNEL_NONE ? LIN_OK : LIN_ERR_UNSUPPORTED;
    const int fit = lin::check_plan_fits(*plan, M, N, K, precision);
    if (fit != LIN_OK) return fit;
    return (size_t)plan->workspace_bytes > workspace_bytes ? LIN_ERR_WORKSPACE : LIN_OK;
}

int lin_plan_make(int sm_count, int kernel, int variant, int splits, int M, int N, int K, int precision,
                  lin_plan* out) {
    if (!out || sm_count < 1 || M < 0 || N < 0 || K < 0 || !lin::valid_enums(0, precision)) return LIN_ERR_ARG;
    const size_t unlimited = (size_t)1 << 62;
    switch (kernel) {
        case LIN_KERNEL_SKINNY:
            if (precision != LIN_PREC_BF16) return LIN_ERR_UNSUPPORTED;
            return lin::make_skinny(sm_count, variant, splits, M, N, K, unlimited, out);
        case LIN_KERNEL_FFMA:
            if (precision != LIN_PREC_FP32) return LIN_ERR_UNSUPPORTED;
            return lin::make_ffma(sm_count, variant, splits, M, N, K, unlimited, out);
        case LIN_KERNEL_TC:
            if (precision == LIN_PREC_FP32) return LIN_ERR_UNSUPPORTED;
            // splits >= 0: CTAs walking whole tiles (0 = one per SM); -1: stream-K with
            // one CTA per SM; -c (c >= 2): stream-K with c CTAs.
            return lin::make_tc(sm_count, variant, splits >= 0 ? splits : (splits == -1 ? 0 : -splits), splits < 0,
                                M, N, K, precision == LIN_PREC_BF16 ? 2 : 4, out);
        case LIN_KERNEL_GEMV:  // splits = CTAs (0 = as many as fit)
            return lin::make_gemv(sm_count, splits > 0 ? splits : 0, M, N, K, precision == LIN_PREC_BF16, out);
        case LIN_KERNEL_NONE:
        case LIN_KERNEL_FILL:
            return lin::plan_default(sm_count, M, N, K, precision, unlimited, out);
        default: return LIN_ERR_ARG;
    }
}

namespace {

// lin_forward and lin_forward_residual: an installed plan for the call
// signature, else the built-in table (adapted to the call's neighbour).
int forward_dispatch(lin_ctx* ctx, int M, int N, int K, const void* X, const void* W, const float* bias,
                     const void* R, void* Y, int epilogue, int precision, void* stream) {
    if (!ctx || M < 0 || N < 0 || K < 0 || !lin::valid_enums(epilogue, precision)) return LIN_ERR_ARG;
    lin_plan plan;
    bool installed = false;
    {
        std::lock_guard<std::mutex> lk(ctx->override_mu);  // copy the entry; launch outside the lock
        for (const lin_override& o : ctx->overrides)
            if (o.M == M && o.N == N && o.K == K && o.precision == precision && o.epilogue == epilogue) {
                plan = o.plan;
                installed = true;
                break;
            }
    }
    if (installed) return lin::run(ctx, plan, M, N, K, X, W, bias, Y, epilogue, precision, stream, false, R);
    const int rc = lin::plan_default(ctx->sm_count, M, N, K, precision, ctx->workspace_bytes, &plan);
    if (rc != LIN_OK) return rc;
    return lin::run(ctx, plan, M, N, K, X, W, bias, Y, epilogue, precision, stream, true, R);
}

}  // namespace

int lin_forward(lin_ctx* ctx, int M, int N, int K, const void* X, const void* W, const float* bias, void* Y,
                int epilogue, int precision, void* stream) {
    return forward_dispatch(ctx, M, N, K, X, W, bias, nullptr, Y, epilogue, precision, stream);
}

int lin_forward_residual(lin_ctx* ctx, int M, int N, int K, const void* X, const void* W, const float* bias,
                         const void* R, void* Y, int epilogue, int precision, void* stream) {
    if (!R && M > 0 && N > 0) return LIN_ERR_ARG;
    return forward_dispatch(ctx, M, N, K, X, W, bias, R, Y, epilogue, precision, stream);
}

int lin_set_plan_override(lin_ctx* ctx, int M, int N, int K, int precision, int epilogue, const lin_plan* plan) {
    if (!ctx || M < 0 || N < 0 || K < 0 || !lin::valid_enums(epilogue, precision)) return LIN_ERR_ARG;
    if (plan) {  // a refused plan leaves the table as it was
        const int fit = lin::check_plan_fits(*plan, M, N, K, precision);
        if (fit != LIN_OK) return fit;
        if ((size_t)plan->workspace_bytes > ctx->workspace_bytes) return LIN_ERR_WORKSPACE;
    }
    std::lock_guard<std::mutex> lk(ctx->override_mu);
    auto& v = ctx->overrides;
    for (size_t i = 0; i < v.size(); ++i)
        if (v[i].M == M && v[i].N == N && v[i].K == K && v[i].precision == precision && v[i].epilogue == epilogue) {
            v.erase(v.begin() + (long)i);
            break;
        }
    if (plan) v.push_back(lin_override{M, N, K, precision, epilogue, *plan});
    return LIN_OK;
}

int lin_clear_plan_overrides(lin_ctx* ctx) {
    if (!ctx) return LIN_ERR_ARG;
    std::lock_guard<std::mutex> lk(ctx->override_mu);
    ctx->overrides.clear();
    return LIN_OK;
}

namespace {

// Shared checks of the two backward GEMMs: returns LIN_OK and fills q, or an error.
int backward_setup(lin_ctx* ctx, int which, int M, int N, int K, const void* dZ, const void* B, void* out,
                   int precision, void* stream, lin::BwdProblem* q) {
    using namespace lin;
    if (!ctx || M < 0 || N < 0 || K < 0 || !valid_enums(0, precision)) return LIN_ERR_ARG;
    const size_t esz = precision == LIN_PREC_BF16 ? 2 : 4;
    const int Mo = which == 1 ? M : N;
    const size_t out_bytes = (size_t)Mo * K * esz;
    if (Mo == 0 || K == 0) return LIN_OK;
    if (!out || (M > 0 && N > 0 && (!dZ || !B))) return LIN_ERR_ARG;
    const size_t dz_bytes = (size_t)M * N * esz;
    const size_t b_bytes = (size_t)(which == 1 ? N : M) * K * esz;
    if (overlaps(out, out_bytes, dZ, dz_bytes) || overlaps(out, out_bytes, B, b_bytes)) return LIN_ERR_ARG;
    if ((((uintptr_t)dZ | (uintptr_t)B | (uintptr_t)out) % 16) != 0 || ((size_t)K * esz) % 16 != 0) return LIN_ERR_ALIGN;
    if (precision == LIN_PREC_BF16 && ((size_t)N * esz) % 16 != 0) return LIN_ERR_ALIGN;  // dZ rows by TMA
    q->which = which;
    q->M = M;
    q->N = N;
    q->K = K;
    q->dZ = dZ;
    q->B = B;
    q->out = out;
    q->stream = static_cast<cudaStream_t>(stream);
    q->dev_status = ctx->dev_status;
    q->sm_count = ctx->sm_count;
    const EarlyReads early = early_reads(q->stream, ctx->early_level, Range{B, b_bytes}, Range{nullptr, 0},
                                         Range{dZ, dz_bytes}, Range{out, out_bytes});
    q->early_start = ctx->programmatic && !early.ordered;
    q->early_x = q->early_start && early.x;
    q->workspace = ctx->workspace;
    q->workspace_bytes = ctx->workspace_bytes;
    // Right after an independent call the two overlap (early start) and fill
    // the SMs together: a K split would only add its round trip.
    q->ksplit_ok = !(ctx->adaptive && early.known && q->early_x);
    q->aux = nullptr;
    return LIN_OK;
}

int backward_run(const lin::BwdProblem& q, int precision, lin_ctx* ctx) {
    using namespace lin;
    const int R = q.which == 1 ? q.N : q.M;
    const int Mo = q.which == 1 ? q.M : q.N;
    if (R == 0)
        return cudaMemsetAsync(q.out, 0, (size_t)Mo * q.K * (precision == LIN_PREC_BF16 ? 2 : 4), q.stream) == cudaSuccess
                   ? LIN_OK
                   : LIN_ERR_CUDA;
    if (precision == LIN_PREC_BF16) return launch_tc_backward(q);
    const int S = bwd_ffma_splits(q.which, q.M, q.N, q.K, ctx->sm_count, ctx->workspace_bytes);
    return launch_bwd_ffma(q.which, q.M, q.N, q.K, static_cast<const float*>(q.dZ), static_cast<const float*>(q.B),
                           static_cast<float*>(q.out), S, ctx->workspace, q.stream, q.early_start,
                           static_cast<const float*>(q.aux));
}

}  // namespace

int lin_backward_data(lin_ctx* ctx, int M, int N, int K, const void* dZ, const void* W, void* dX, int precision,
                      void* stream) {
    lin::BwdProblem q;
    q.which = 0;
    const int rc = backward_setup(ctx, 1, M, N, K, dZ, W, dX, precision, stream, &q);
    if (rc != LIN_OK || q.which == 0) return rc;
    lin::DeviceGuard guard(ctx->device);
    if (!guard.ok) return LIN_ERR_CUDA;
    return backward_run(q, precision, ctx);
}

int lin_backward_data_gelu(lin_ctx* ctx, int M, int N, int K, const void* dZ, const void* W, const void* Zp,
                           void* dX, int precision, void* stream) {
    lin::BwdProblem q;
    q.which = 0;
    if (!ctx || !lin::valid_enums(0, precision)) return LIN_ERR_ARG;
    const size_t esz = precision == LIN_PREC_BF16 ? 2 : 4;
    const size_t bytes = (size_t)(M > 0 ? M : 0) * (K > 0 ? K : 0) * esz;
    if (bytes > 0 && !Zp) return LIN_ERR_ARG;
    if (Zp != dX && lin::overlaps(Zp, bytes, dX, bytes)) return LIN_ERR_ARG;  // in place, or apart
    if ((uintptr_t)Zp % esz != 0) return LIN_ERR_ALIGN;
    const int rc = backward_setup(ctx, 1, M, N, K, dZ, W, dX, precision, stream, &q);
    if (rc != LIN_OK || q.which == 0) return rc;
    q.aux = Zp;
    lin::DeviceGuard guard(ctx->device);
    if (!guard.ok) return LIN_ERR_CUDA;
    return backward_run(q, precision, ctx);
}

int lin_backward_weight(lin_ctx* ctx, int M, int N, int K, const void* dZ, const void* X, void* dW, float* db,
                        int precision, void* stream) {
    using namespace lin;
    lin::BwdProblem q;
    q.which = 0;
    int rc = backward_setup(ctx, 2, M, N, K, dZ, X, dW, precision, stream, &q);
    if (rc != LIN_OK) return rc;
    if (db) {
        if ((uintptr_t)db % 4 != 0) return LIN_ERR_ALIGN;
        const size_t esz = precision == LIN_PREC_BF16 ? 2 : 4;
        if (overlaps(db, (size_t)N * 4, dZ, (size_t)M * N * esz) || overlaps(db, (size_t)N * 4, X, (size_t)M * K * esz) ||
            overlaps(db, (size_t)N * 4, dW, (size_t)N * K * esz))
            return LIN_ERR_ARG;
        if (M > 0 && N > 0 && colsum_workspace_bytes(M, N) > ctx->workspace_bytes) return LIN_ERR_WORKSPACE;
    }
    lin::DeviceGuard guard(ctx->device);
    if (!guard.ok) return LIN_ERR_CUDA;
    if (q.which != 0) {
        rc = backward_run(q, precision, ctx);
        if (rc != LIN_OK) return rc;
    }
    if (db && N > 0) {
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        rc = launch_colsum(M, N, dZ, db, precision == LIN_PREC_BF16, ctx->workspace, st);
        if (rc != LIN_OK) return rc;
        note_output(st, Range{db, (size_t)N * 4});
    }
    return LIN_OK;
}

int lin_gelu_backward(lin_ctx* ctx, long long count, const void* dY, const void* Z, void* dZ, int precision,
                      void* stream) {
    using namespace lin;
    if (!ctx || count < 0 || !valid_enums(0, precision)) return LIN_ERR_ARG;
    if (count == 0) return LIN_OK;
    if (!dY || !Z || !dZ) return LIN_ERR_ARG;
    const size_t esz = precision == LIN_PREC_BF16 ? 2 : 4;
    const size_t bytes = (size_t)count * esz;
    if (overlaps(dZ, bytes, Z, bytes)) return LIN_ERR_ARG;  // dZ may overwrite dY in place
    if ((((uintptr_t)dY | (uintptr_t)Z | (uintptr_t)dZ) % esz) != 0) return LIN_ERR_ALIGN;
    DeviceGuard guard(ctx->device);
    if (!guard.ok) return LIN_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    note_output(st, Range{dZ, bytes});
    return launch_gelu_backward(count, dY, Z, dZ, precision == LIN_PREC_BF16, ctx->sm_count, st,
                                ctx->programmatic);
}

int lin_fold_layernorm(lin_ctx* ctx, int N, int K, const float* W, const float* bias, const float* gamma,
                       const float* beta, void* W_out, float* bias_out, int precision, void* stream) {
    using namespace lin;
    if (!ctx || N < 0 || K < 0 || !valid_enums(0, precision)) return LIN_ERR_ARG;
    if (N == 0) return LIN_OK;
    if (!W_out || !bias_out || (K > 0 && (!W || !gamma))) return LIN_ERR_ARG;
    const size_t eout = precision == LIN_PREC_BF16 ? 2 : 4;
    const size_t wbytes = (size_t)N * K * 4, wobytes = (size_t)N * K * eout;
    // In place: W_out = W (fp32 storage) and bias_out = bias are allowed; no other overlap.
    if (!(W_out == W && eout == 4) && overlaps(W_out, wobytes, W, wbytes)) return LIN_ERR_ARG;
    if (overlaps(W_out, wobytes, gamma, (size_t)K * 4) || overlaps(W_out, wobytes, beta, beta ? (size_t)K * 4 : 0) ||
        overlaps(W_out, wobytes, bias, bias ? (size_t)N * 4 : 0) || overlaps(W_out, wobytes, bias_out, (size_t)N * 4))
        return LIN_ERR_ARG;
    if (bias_out != bias && overlaps(bias_out, (size_t)N * 4, bias, bias ? (size_t)N * 4 : 0)) return LIN_ERR_ARG;
    if (overlaps(bias_out, (size_t)N * 4, W, wbytes) || overlaps(bias_out, (size_t)N * 4, gamma, (size_t)K * 4) ||
        overlaps(bias_out, (size_t)N * 4, beta, beta ? (size_t)K * 4 : 0))
        return LIN_ERR_ARG;
    if ((((uintptr_t)W | (uintptr_t)bias | (uintptr_t)gamma | (uintptr_t)beta | (uintptr_t)bias_out) % 4) != 0 ||
        ((uintptr_t)W_out % eout) != 0)
        return LIN_ERR_ALIGN;
    DeviceGuard guard(ctx->device);
    if (!guard.ok) return LIN_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int rc = launch_fold_layernorm(N, K, W, bias, gamma, beta, W_out, bias_out, precision == LIN_PREC_BF16,
                                         ctx->sm_count, st);
    if (rc == LIN_OK) {
        note_output(st, Range{W_out, wobytes});
    }
    return rc;
}

int lin_forward_plan(lin_ctx* ctx, const lin_plan* plan, int M, int N, int K, const void* X, const void* W,
                     const float* bias, void* Y, int epilogue, int precision, void* stream) {
    if (!plan) return LIN_ERR_ARG;
    return lin::run(ctx, *plan, M, N, K, X, W, bias, Y, epilogue, precision, stream, false);
}

int lin_probe_ffma(lin_ctx* ctx, int iters, float* out, double* flops, void* stream) {
    if (!ctx || iters < 1 || !out) return LIN_ERR_ARG;
    if ((uintptr_t)out % 4 != 0) return LIN_ERR_ALIGN;
    lin::DeviceGuard guard(ctx->device);
    if (!guard.ok) return LIN_ERR_CUDA;
    return lin::launch_ffma_probe(ctx->sm_count, iters, out, static_cast<cudaStream_t>(stream), flops);
}

int lin_attention_forward(lin_ctx* ctx, int B, int T, int H, int D, const void* qkv, void* out, float* lse,
                          int causal, float scale, void* stream) {
    using namespace lin;
    if (!ctx || B < 0 || T < 0 || H < 0 || D < 0 || (causal != 0 && causal != 1)) return LIN_ERR_ARG;
    if (!(scale >= 0.f) || isinf(scale)) return LIN_ERR_ARG;  // NaN, negative or infinite
    if (B == 0 || T == 0 || H == 0) return LIN_OK;
    if (D != 64) return LIN_ERR_UNSUPPORTED;
    const long long rows = (long long)B * T;
    const long long nqb = (T + 127) / 128;
    if (rows > INT_MAX || (long long)H * D * 3 > INT_MAX || (long long)B * H * nqb > INT_MAX) return LIN_ERR_UNSUPPORTED;
    if (!qkv || !out) return LIN_ERR_ARG;
    const size_t C = (size_t)H * D;
    const size_t in_bytes = (size_t)rows * 3 * C * 2, out_bytes = (size_t)rows * C * 2;
    const size_t lse_bytes = lse ? (size_t)B * H * T * 4 : 0;
    if (overlaps(out, out_bytes, qkv, in_bytes) || overlaps(lse, lse_bytes, qkv, in_bytes) ||
        overlaps(lse, lse_bytes, out, out_bytes))
        return LIN_ERR_ARG;
    if ((((uintptr_t)qkv | (uintptr_t)out) % 16) != 0 || ((uintptr_t)lse % 4) != 0) return LIN_ERR_ALIGN;
    DeviceGuard guard(ctx->device);
    if (!guard.ok) return LIN_ERR_CUDA;
    AttnProblem p;
    p.B = B;
    p.T = T;
    p.H = H;
    p.qkv = qkv;
    p.out = out;
    p.lse = lse;
    p.causal = causal != 0;
    p.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)D);
    p.stream = static_cast<cudaStream_t>(stream);
    p.dev_status = ctx->dev_status;
    p.sm_count = ctx->sm_count;
    p.early_start = ctx->programmatic;
    // Its output is a later call's input: note it for the early-read checks.
    note_output(p.stream, Range{out, out_bytes});
    if (lse) note_output(p.stream, Range{lse, lse_bytes});
    return launch_attention(p);
}

namespace {

bool float_type(int t) { return t == LIN_TYPE_FP32 || t == LIN_TYPE_BF16; }
bool index_type(int t) { return t == LIN_TYPE_INT32 || t == LIN_TYPE_INT64; }
size_t type_bytes(int t) { return t == LIN_TYPE_BF16 ? 2 : t == LIN_TYPE_INT64 ? 8 : 4; }
size_t row_bytes(int R, int V, long long ld, size_t esz) { return ((size_t)(R - 1) * (size_t)ld + (size_t)V) * esz; }

// A range, its element size and whether the call writes it.
struct Operand {
    const void* p;
    size_t bytes, esz;
    bool written;
};

// Alignment, and no output over another operand. Records the outputs of the call on the
// stream; *hull is where they all lie.
int check_operands(const Operand* o, int N, cudaStream_t st, lin::Range* hull) {
    using namespace lin;
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < N; ++j)
            if (i != j && o[i].written && overlaps(o[i].p, o[i].p ? o[i].bytes : 0, o[j].p, o[j].p ? o[j].bytes : 0))
                return LIN_ERR_ARG;
    uintptr_t lo = UINTPTR_MAX, hi = 0;
    for (int i = 0; i < N; ++i) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(o[i].p);
        if (!a) continue;
        if (a % o[i].esz != 0) return LIN_ERR_ALIGN;
        if (!o[i].written) continue;
        if (a < lo) lo = a;
        if (a + o[i].bytes > hi) hi = a + o[i].bytes;
    }
    *hull = Range{reinterpret_cast<const void*>(lo), hi - lo};
    note_output(st, *hull);
    return LIN_OK;
}

// These calls' kernels wait for what is before them before they let others start.
int launched(int rc, cudaStream_t st, const lin::Range& hull) {
    if (rc == LIN_OK) lin::note_ordered_output(st, hull.p, hull.bytes);
    return rc;
}

int logits_setup(lin_ctx* ctx, int R, int V, const void* logits, long long ld, int type, float tau, void* stream,
                 lin::LogitsProblem* p) {
    // log2(e) / tau has to be finite in fp32 too
    if (!ctx || R < 0 || V < 0 || !float_type(type) || !(tau > 0.f) || isinf(tau) ||
        isinf((float)(1.4426950408889634 / tau)))
        return LIN_ERR_ARG;
    if (R == 0) return LIN_OK;
    if (V == 0 || ld < V || !logits) return LIN_ERR_ARG;
    if (V > (1 << 30) || R > (1 << 27) || ld > (1ll << 40)) return LIN_ERR_UNSUPPORTED;
    p->R = R;
    p->V = V;
    p->ld = ld;
    p->z = logits;
    p->bf16 = type == LIN_TYPE_BF16;
    p->tau = tau;
    p->stream = static_cast<cudaStream_t>(stream);
    p->dev_status = ctx->dev_status;
    p->sm_count = ctx->sm_count;
    p->early_start = ctx->programmatic;
    return LIN_OK;
}

int distill_run(lin_ctx* ctx, int R, int V, int K, const void* logits, long long ld, int logits_type, const void* ids,
                int ids_type, const void* teacher, int teacher_type, float tau, const float* weight,
                const float* lse_in, float* loss, float* lse, void* dz, long long ldd, bool grad, void* stream) {
    lin::LogitsProblem p;
    const int rc = logits_setup(ctx, R, V, logits, ld, logits_type, tau, stream, &p);
    if (rc != LIN_OK) return rc;
    if (K < 0 || !index_type(ids_type) || !float_type(teacher_type)) return LIN_ERR_ARG;
    if (R == 0) return LIN_OK;
    if (K > lin::kDistillMaxEntries) return LIN_ERR_UNSUPPORTED;
    if ((K > 0 && (!ids || !teacher)) || (grad && (!dz || ldd < V))) return LIN_ERR_ARG;
    if (ldd > (1ll << 40)) return LIN_ERR_UNSUPPORTED;
    const size_t esz = type_bytes(logits_type), rk = (size_t)R * K, r4 = (size_t)R * 4;
    const bool in_place = grad && dz == logits && ldd == ld;
    const Operand ops[] = {
        {in_place ? nullptr : logits, row_bytes(R, V, ld, esz), esz, false},
        {ids, rk * type_bytes(ids_type), type_bytes(ids_type), false},
        {teacher, rk * type_bytes(teacher_type), type_bytes(teacher_type), false},
        {weight, r4, 4, false},
        {lse_in, r4, 4, false},
        {loss, r4, 4, true},
        {lse, r4, 4, true},
        {grad ? dz : nullptr, grad ? row_bytes(R, V, ldd, esz) : 0, esz, true},
    };
    lin::Range hull;
    const int ok = check_operands(ops, (int)(sizeof(ops) / sizeof(ops[0])), p.stream, &hull);
    if (ok != LIN_OK) return ok;
    lin::DeviceGuard guard(ctx->device);
    if (!guard.ok) return LIN_ERR_CUDA;
    p.K = K;
    p.ids = ids;
    p.wide_ids = ids_type == LIN_TYPE_INT64;
    p.teacher = teacher;
    p.teacher_bf16 = teacher_type == LIN_TYPE_BF16;
    p.weight = weight;
    p.lse_in = lse_in;
    p.loss = loss;
    p.lse = lse;
    p.dz = grad ? dz : nullptr;
    p.ldd = ldd;
    return launched(lin::launch_distill(p), p.stream, hull);
}

}  // namespace

int lin_attention_backward(lin_ctx* ctx, int B, int T, int H, int D, const void* qkv, const void* out,
                           const float* lse, const void* dout, void* dqkv, int causal, float scale, void* stream) {
    using namespace lin;
    if (!ctx || B < 0 || T < 0 || H < 0 || D < 0 || (causal != 0 && causal != 1)) return LIN_ERR_ARG;
    if (!(scale >= 0.f) || isinf(scale)) return LIN_ERR_ARG;  // NaN, negative or infinite
    if (B == 0 || T == 0 || H == 0) return LIN_OK;
    if (D != 64) return LIN_ERR_UNSUPPORTED;
    const long long rows = (long long)B * T, nb = (T + 127ll) / 128;
    if (rows > INT_MAX || (long long)H * D * 3 > INT_MAX || (long long)B * H > INT_MAX ||
        (long long)B * H * nb > INT_MAX)
        return LIN_ERR_UNSUPPORTED;
    if (!qkv || !out || !lse || !dout || !dqkv) return LIN_ERR_ARG;
    // lse / scale, and what stands for no key, are fp32
    if (scale > 0.f && !(scale >= 0x1p-100f && scale <= 0x1p100f)) return LIN_ERR_ARG;
    const size_t bytes = (size_t)rows * H * D * 2;
    const Operand ops[] = {
        {qkv, 3 * bytes, 16, false}, {out, bytes, 16, false},      {lse, (size_t)B * H * T * 4, 4, false},
        {dout, bytes, 16, false},    {dqkv, 3 * bytes, 16, true},
    };
    Range hull;
    const int ok = check_operands(ops, (int)(sizeof(ops) / sizeof(ops[0])), static_cast<cudaStream_t>(stream), &hull);
    if (ok != LIN_OK) return ok;
    DeviceGuard guard(ctx->device);
    if (!guard.ok) return LIN_ERR_CUDA;
    AttnBwdProblem p;
    p.B = B;
    p.T = T;
    p.H = H;
    p.qkv = qkv;
    p.out = out;
    p.lse = lse;
    p.dout = dout;
    p.dqkv = dqkv;
    p.causal = causal != 0;
    p.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)D);
    p.stream = static_cast<cudaStream_t>(stream);
    p.workspace = ctx->workspace;
    p.workspace_bytes = ctx->workspace_bytes;
    p.dev_status = ctx->dev_status;
    p.sm_count = ctx->sm_count;
    p.early_start = ctx->programmatic;
    return launched(launch_attention_backward(p), p.stream, hull);
}

int lin_token_logprobs(lin_ctx* ctx, int R, int V, const void* logits, long long ld, int logits_type,
                       const void* tokens, int tokens_type, float tau, int top, float* logprob, float* entropy,
                       float* lse, float* top_logprob, int* top_ids, void* stream) {
    lin::LogitsProblem p;
    const int rc = logits_setup(ctx, R, V, logits, ld, logits_type, tau, stream, &p);
    if (rc != LIN_OK) return rc;
    if (top < 0 || (tokens && !index_type(tokens_type)) || (R > 0 && (tokens == nullptr) != (logprob == nullptr)))
        return LIN_ERR_ARG;
    if (R == 0) return LIN_OK;
    if (top > lin::kLogprobMaxTop) return LIN_ERR_UNSUPPORTED;
    if (top > V || (top > 0 && (!top_logprob || !top_ids))) return LIN_ERR_ARG;
    if (!logprob && !entropy && !lse && top == 0) return LIN_OK;
    if (top == 0) {
        top_logprob = nullptr;
        top_ids = nullptr;
    }
    const size_t esz = type_bytes(logits_type), r4 = (size_t)R * 4;
    const Operand ops[] = {
        {logits, row_bytes(R, V, ld, esz), esz, false},
        {tokens, (size_t)R * type_bytes(tokens_type), type_bytes(tokens_type), false},
        {logprob, r4, 4, true},
        {entropy, r4, 4, true},
        {lse, r4, 4, true},
        {top_logprob, r4 * top, 4, true},
        {top_ids, r4 * top, 4, true},
    };
    lin::Range hull;
    const int ok = check_operands(ops, (int)(sizeof(ops) / sizeof(ops[0])), p.stream, &hull);
    if (ok != LIN_OK) return ok;
    lin::DeviceGuard guard(ctx->device);
    if (!guard.ok) return LIN_ERR_CUDA;
    p.ids = tokens;
    p.wide_ids = tokens_type == LIN_TYPE_INT64;
    p.top = top;
    p.logprob = logprob;
    p.entropy = entropy;
    p.lse = lse;
    p.top_logprob = top_logprob;
    p.top_ids = top_ids;
    return launched(lin::launch_logprobs(p), p.stream, hull);
}

int lin_distill_forward(lin_ctx* ctx, int R, int V, int K, const void* logits, long long ld, int logits_type,
                        const void* ids, int ids_type, const void* teacher, int teacher_type, float tau, float* loss,
                        float* lse, void* stream) {
    if (R > 0 && !loss) return LIN_ERR_ARG;
    return distill_run(ctx, R, V, K, logits, ld, logits_type, ids, ids_type, teacher, teacher_type, tau, nullptr,
                       nullptr, loss, lse, nullptr, 0, false, stream);
}

int lin_distill_backward(lin_ctx* ctx, int R, int V, int K, const void* logits, long long ld, int logits_type,
                         const void* ids, int ids_type, const void* teacher, int teacher_type, float tau,
                         const float* lse, const float* grad_loss, void* dlogits, long long ldd, void* stream) {
    if (R > 0 && (!lse || !grad_loss)) return LIN_ERR_ARG;
    return distill_run(ctx, R, V, K, logits, ld, logits_type, ids, ids_type, teacher, teacher_type, tau, grad_loss,
                       lse, nullptr, nullptr, dlogits, ldd, true, stream);
}

int lin_distill_forward_backward(lin_ctx* ctx, int R, int V, int K, const void* logits, long long ld, int logits_type,
                                 const void* ids, int ids_type, const void* teacher, int teacher_type, float tau,
                                 const float* weight, float* loss, void* dlogits, long long ldd, void* stream) {
    return distill_run(ctx, R, V, K, logits, ld, logits_type, ids, ids_type, teacher, teacher_type, tau, weight,
                       nullptr, loss, nullptr, dlogits, ldd, true, stream);
}

// ---- rotary positions and the paged cache ----

int lin_rotary_turns(const double* frequencies, int n, unsigned long long* turns) {
    if (n < 0 || (n > 0 && (!frequencies || !turns))) return LIN_ERR_ARG;
    for (int i = 0; i < n; ++i)
        if (!std::isfinite(frequencies[i])) return LIN_ERR_ARG;
    for (int i = 0; i < n; ++i) {
        // f / 2 pi as the sum of a double and what it lacks, 1 / 2 pi being the sum of two: 106 bits, so that the
        // 64 of the fraction are right (to 0.6 of the last, with its rounding) up to f = 2^40.
        constexpr double kInv = 0x1.45f306dc9c883p-3, kInvRest = -0x1.6b01ec5417056p-57;
        const double f = std::fabs(frequencies[i]);
        const double t = f * kInv, rest = std::fmod(std::fma(f, kInv, -t) + f * kInvRest, 1.0);
        const double part = std::ldexp(std::fmod(t, 1.0), 64), whole = std::floor(part);
        const double low = (part - whole) + std::ldexp(rest, 64);  // below 2^64 in size
        const unsigned long long add = static_cast<unsigned long long>(std::floor(std::fabs(low) + 0.5));
        const unsigned long long turn = static_cast<unsigned long long>(whole) + (low < 0.0 ? 0ull - add : add);
        turns[i] = std::signbit(frequencies[i]) ? 0ull - turn : turn;
    }
    return LIN_OK;
}

namespace {

constexpr int kMaxHeadDim = 1024;

// N rows of `width` elements of `esz` bytes, `ld` elements apart.
struct Rows {
    const void* p;
    long long N, width, ld;
    size_t esz;
};

size_t rows_extent(const Rows& r) { return r.p && r.N > 0 && r.width > 0 ? ((size_t)(r.N - 1) * r.ld + r.width) * r.esz : 0; }

// Whether two sets of rows share an element. Rows of the same stride may interleave
// (columns of one matrix); others overlap when their extents do.
bool rows_overlap(const Rows& a, const Rows& b) {
    if (!lin::overlaps(a.p, rows_extent(a), b.p, rows_extent(b))) return false;
    const long long la = a.ld * (long long)a.esz, lb = b.ld * (long long)b.esz;
    const bool same = la == lb || a.N == 1 || b.N == 1;
    if (!same) return true;
    const long long ld = a.N == 1 ? lb : la;
    if (a.N == 1 && b.N == 1) return true;
    const long long wa = a.width * (long long)a.esz, wb = b.width * (long long)b.esz;
    long long d = (long long)(reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p)) % ld;
    if (d < 0) d += ld;
    return !(d >= wa && ld - d >= wb);
}

int rotary_ok(const lin_rotary* r, int D) {
    if (!r || r->dim < 0 || r->dim > D || r->dim % 2 != 0 || (r->dim > 0 && !r->turns) || !std::isfinite(r->scale) ||
        (r->layout != LIN_ROTARY_HALF && r->layout != LIN_ROTARY_INTERLEAVED))
        return LIN_ERR_ARG;
    return (uintptr_t)r->turns % 8 != 0 ? LIN_ERR_ALIGN : LIN_OK;
}

// Largest row stride that is taken, extent of a cache (elements).
constexpr long long kMaxStride = 1ll << 30, kMaxCache = 1ll << 46;
// A tensor map's strides are below 2^40 bytes.
constexpr long long kMaxCacheStride = 1ll << 38;

int rotary_run(lin_ctx* ctx, int N, int H, int D, const void* x, long long ldx, void* y, long long ldy, int type,
               const void* positions, int positions_type, const lin_rotary* rotary, bool inverse, void* stream) {
    using namespace lin;
    if (!ctx || N < 0 || H < 0 || D < 0 || !float_type(type) || !index_type(positions_type)) return LIN_ERR_ARG;
    if (D > kMaxHeadDim) return LIN_ERR_UNSUPPORTED;
    const int ok = rotary_ok(rotary, D);
    if (ok != LIN_OK) return ok;
    if (N == 0 || H == 0 || D == 0) return LIN_OK;
    const long long width = (long long)H * D;
    if (!x || !y || !positions || ldx < width || ldy < width) return LIN_ERR_ARG;
    if (width > (1 << 27) || ldx > kMaxStride || ldy > kMaxStride) return LIN_ERR_UNSUPPORTED;
    const size_t esz = type_bytes(type), psz = type_bytes(positions_type);
    const Rows in{x, N, width, ldx, esz}, out{y, N, width, ldy, esz};
    const bool in_place = x == y && (ldx == ldy || N == 1);
    if (!in_place && rows_overlap(out, in)) return LIN_ERR_ARG;
    const size_t turn_bytes = (size_t)rotary->dim / 2 * 8;
    if (rows_overlap(out, Rows{positions, 1, N, N, psz}) ||
        rows_overlap(out, Rows{rotary->turns, 1, (long long)turn_bytes, (long long)turn_bytes, 1}))
        return LIN_ERR_ARG;
    if (((uintptr_t)x | (uintptr_t)y) % esz != 0 || (uintptr_t)positions % psz != 0) return LIN_ERR_ALIGN;
    // Nothing turns and everything is in its place. No kernel runs, so what the stream's earlier calls may still
    // be writing stays on its list.
    if (in_place && rotary->dim == 0) return LIN_OK;
    DeviceGuard guard(ctx->device);
    if (!guard.ok) return LIN_ERR_CUDA;
    RotaryProblem p;
    p.N = N;
    p.D = D;
    p.rot = rotary->dim;
    p.interleaved = rotary->layout == LIN_ROTARY_INTERLEAVED;
    p.inverse = inverse;
    p.bf16 = type == LIN_TYPE_BF16;
    p.part[0] = RotaryPart{x, y, ldx, ldy, H};
    p.positions = positions;
    p.wide = positions_type == LIN_TYPE_INT64;
    p.turns = rotary->turns;
    p.scale = rotary->scale;
    p.stream = static_cast<cudaStream_t>(stream);
    p.sm_count = ctx->sm_count;
    p.early_start = ctx->programmatic;
    const Range hull{y, rows_extent(out)};
    note_output(p.stream, hull);
    return launched(launch_rotary(p), p.stream, hull);
}

// Elements from a cache's first to its last.
size_t cache_extent(const lin_kv_cache& c) {
    return ((size_t)(c.pages - 1) * c.page_stride + (size_t)(c.heads - 1) * c.head_stride +
            (size_t)(c.page_size - 1) * c.token_stride + c.head_dim) * 2;
}

// Whether the cache's rows of head_dim elements, k's and v's, lie apart: strides taken
// from the smallest, each at least the extent of those below it. Strides of a
// single page, head or slot do not count; v is a second copy at its distance from k.
bool cache_rows_apart(const lin_kv_cache& c) {
    const uintptr_t k = reinterpret_cast<uintptr_t>(c.k), v = reinterpret_cast<uintptr_t>(c.v);
    const uintptr_t apart = (k < v ? v - k : k - v) / 2;
    long long n[4] = {c.pages, c.heads, c.page_size, 2};
    long long s[4] = {c.page_stride, c.head_stride, c.token_stride, (long long)(apart > (uintptr_t)kMaxCache * 4 ? kMaxCache * 4 : apart)};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (s[j] < s[i]) {
                std::swap(s[i], s[j]);
                std::swap(n[i], n[j]);
            }
    long long extent = c.head_dim;
    for (int i = 0; i < 4; ++i) {
        if (n[i] == 1) continue;
        if (s[i] < extent) return false;
        extent = (n[i] - 1) * s[i] + extent;
    }
    return true;
}

int cache_ok(const lin_kv_cache* c, const lin_kv_batch* b) {
    if (!c || !b || c->pages < 1 || c->heads < 1 || c->page_size < 1 || c->head_dim < 1 || b->sequences < 0 ||
        b->tokens < 0 || b->table_pages < 0 || b->table_stride < b->table_pages)
        return LIN_ERR_ARG;
    if ((c->page_size & (c->page_size - 1)) != 0 || c->page_size < 8 || c->page_size > 4096 ||
        (c->head_dim != 64 && c->head_dim != 128) || c->heads > 65535 || b->table_stride > kMaxStride ||
        (long long)b->table_pages * c->page_size > (1 << 30) || b->sequences > (1 << 30))
        return LIN_ERR_UNSUPPORTED;
    if (b->tokens > 0 && b->sequences > 0 && (!b->q_start || !b->kv_len || (b->table_pages > 0 && !b->block_table)))
        return LIN_ERR_ARG;
    if (((uintptr_t)b->q_start | (uintptr_t)b->kv_len | (uintptr_t)b->block_table) % 4 != 0) return LIN_ERR_ALIGN;
    if (!c->k || !c->v) return LIN_ERR_ARG;
    const long long strides[] = {c->page_stride, c->head_stride, c->token_stride};
    const int counts[] = {c->pages, c->heads, c->page_size};
    for (int i = 0; i < 3; ++i) {
        if (strides[i] < 0) return LIN_ERR_ARG;
        if (strides[i] > kMaxCacheStride || strides[i] > kMaxCache / counts[i]) return LIN_ERR_UNSUPPORTED;
    }
    if (!cache_rows_apart(*c)) return LIN_ERR_ARG;
    if (((uintptr_t)c->k | (uintptr_t)c->v) % 16 != 0 || c->token_stride % 8 != 0 ||
        (c->heads > 1 && c->head_stride % 8 != 0) || (c->pages > 1 && c->page_stride % 8 != 0))
        return LIN_ERR_ALIGN;
    return LIN_OK;
}

// Rows of table entries as an operand of the overlap checks.
Rows table_rows(const lin_kv_batch& b) {
    return Rows{b.block_table, b.sequences, b.table_pages, b.table_stride, 4};
}

}  // namespace

int lin_rotary_forward(lin_ctx* ctx, int N, int H, int D, const void* x, long long ldx, void* y, long long ldy,
                       int type, const void* positions, int positions_type, const lin_rotary* rotary, void* stream) {
    return rotary_run(ctx, N, H, D, x, ldx, y, ldy, type, positions, positions_type, rotary, false, stream);
}

int lin_rotary_backward(lin_ctx* ctx, int N, int H, int D, const void* dy, long long lddy, void* dx, long long lddx,
                        int type, const void* positions, int positions_type, const lin_rotary* rotary, void* stream) {
    return rotary_run(ctx, N, H, D, dy, lddy, dx, lddx, type, positions, positions_type, rotary, true, stream);
}

int lin_cache_append(lin_ctx* ctx, const lin_kv_cache* cache, const lin_kv_batch* batch, int H, const void* q,
                     long long ldq, void* q_out, long long ldqo, const void* k, long long ldk, const void* v,
                     long long ldv, const void* positions, int positions_type, const lin_rotary* rotary,
                     void* stream) {
    using namespace lin;
    if (!ctx || H < 0 || (positions && !index_type(positions_type))) return LIN_ERR_ARG;
    int ok = cache_ok(cache, batch);
    if (ok != LIN_OK) return ok;
    const int D = cache->head_dim;
    if (rotary && (ok = rotary_ok(rotary, D)) != LIN_OK) return ok;
    if (H > 0 ? !rotary : (q || q_out)) return LIN_ERR_ARG;
    if (batch->tokens == 0 || batch->sequences == 0) return LIN_OK;
    const long long N = batch->tokens, wq = (long long)H * D, wk = (long long)cache->heads * D;
    if (!k || !v || ldk < wk || ldv < wk || (H > 0 && (!q || !q_out || ldq < wq || ldqo < wq))) return LIN_ERR_ARG;
    if (wq > (1 << 27) || ldk > kMaxStride || ldv > kMaxStride || (H > 0 && (ldq > kMaxStride || ldqo > kMaxStride)))
        return LIN_ERR_UNSUPPORTED;
    const size_t psz = positions ? type_bytes(positions_type) : 4;
    const size_t held = cache_extent(*cache);
    auto flat = [](const void* p, size_t bytes) { return Rows{p, 1, (long long)bytes, (long long)bytes, 1}; };
    const Rows rq{H > 0 ? q : nullptr, N, wq, ldq, 2}, rqo{H > 0 ? q_out : nullptr, N, wq, ldqo, 2};
    const Rows rk{k, N, wk, ldk, 2}, rv{v, N, wk, ldv, 2};
    const Rows kc = flat(cache->k, held), vc = flat(cache->v, held);
    const Rows inputs[] = {rk, rv, table_rows(*batch), flat(batch->q_start, 4 * ((size_t)batch->sequences + 1)),
                           flat(batch->kv_len, 4 * (size_t)batch->sequences), flat(positions, positions ? N * psz : 0),
                           flat(rotary ? rotary->turns : nullptr, rotary ? (size_t)rotary->dim / 2 * 8 : 0)};
    for (const Rows& r : inputs)
        if (rows_overlap(rqo, r) || rows_overlap(kc, r) || rows_overlap(vc, r)) return LIN_ERR_ARG;
    if (!(q == q_out && (ldq == ldqo || N == 1)) && rows_overlap(rqo, rq)) return LIN_ERR_ARG;
    if (rows_overlap(kc, rq) || rows_overlap(vc, rq) || rows_overlap(kc, rqo) || rows_overlap(vc, rqo)) return LIN_ERR_ARG;
    if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)q | (uintptr_t)q_out) % 2 != 0 || (uintptr_t)positions % psz != 0)
        return LIN_ERR_ALIGN;
    DeviceGuard guard(ctx->device);
    if (!guard.ok) return LIN_ERR_CUDA;
    RotaryProblem p;
    p.N = N;
    p.D = D;
    p.rot = rotary ? rotary->dim : 0;
    p.interleaved = rotary && rotary->layout == LIN_ROTARY_INTERLEAVED;
    p.append = true;
    p.part[0] = RotaryPart{q, q_out, ldq, ldqo, H};
    p.part[1] = RotaryPart{k, cache->k, ldk, cache->token_stride, cache->heads};
    p.part[2] = RotaryPart{v, cache->v, ldv, cache->token_stride, cache->heads};
    p.positions = positions;
    p.wide = positions_type == LIN_TYPE_INT64;
    p.turns = rotary ? rotary->turns : nullptr;
    p.scale = rotary ? rotary->scale : 1.f;
    p.cache = *cache;
    p.batch = *batch;
    p.stream = static_cast<cudaStream_t>(stream);
    p.sm_count = ctx->sm_count;
    p.early_start = ctx->programmatic;
    uintptr_t lo = UINTPTR_MAX, hi = 0;
    for (const Rows& r : {rqo, kc, vc}) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(r.p);
        const size_t n = rows_extent(r);
        if (n == 0) continue;
        lo = a < lo ? a : lo;
        hi = a + n > hi ? a + n : hi;
    }
    const Range hull{hi ? reinterpret_cast<const void*>(lo) : nullptr, hi ? hi - lo : 0};
    note_output(p.stream, hull);
    return launched(launch_rotary(p), p.stream, hull);
}

namespace {

// Rows of a tile that the call is made for: the new tokens of a sequence with
// the query heads of a key head.
int paged_rows(const lin_kv_cache& cache, const lin_kv_batch* batch, int H, int max_new) {
    long long n = max_new;
    if (n == 0 && batch && batch->sequences > 0)
        n = ((long long)batch->tokens + batch->sequences - 1) / batch->sequences;
    const long long rows = (n < 1 ? 1 : n) * (H / cache.heads);
    return rows > INT_MAX ? INT_MAX : (int)rows;
}

size_t paged_bytes(const lin_ctx& ctx, const lin_kv_cache& cache, int rows) {
    return rows <= lin::kPagedRowsMax ? lin::paged_rows_workspace(ctx.sm_count, cache.head_dim)
                                      : lin::paged_tiles_workspace(ctx.sm_count, cache.head_dim);
}

int paged_heads_ok(const lin_kv_cache* c, int H, int max_new) {
    if (!c || H < 1 || c->heads < 1 || max_new < 0 || H % c->heads != 0) return LIN_ERR_ARG;
    if ((c->head_dim != 64 && c->head_dim != 128) || H / c->heads > lin::kPagedGroupMax || H > 65535)
        return LIN_ERR_UNSUPPORTED;
    return LIN_OK;
}

}  // namespace

int lin_paged_attention_workspace(const lin_ctx* ctx, const lin_kv_cache* cache, const lin_kv_batch* batch, int H,
                                  int max_new, size_t* bytes) {
    if (!ctx || !bytes || (max_new == 0 && !batch)) return LIN_ERR_ARG;
    const int ok = paged_heads_ok(cache, H, max_new);
    if (ok != LIN_OK) return ok;
    *bytes = paged_bytes(*ctx, *cache, paged_rows(*cache, batch, H, max_new));
    return LIN_OK;
}

int lin_paged_attention(lin_ctx* ctx, const lin_kv_cache* cache, const lin_kv_batch* batch, int H, const void* q,
                        long long ldq, void* out, long long ldo, float* lse, int causal, float scale, int max_new,
                        void* workspace, size_t workspace_bytes, void* stream) {
    using namespace lin;
    if (!ctx || (causal != 0 && causal != 1) || !(scale >= 0.f) || std::isinf(scale) || H < 0) return LIN_ERR_ARG;
    int ok = cache_ok(cache, batch);
    if (ok != LIN_OK) return ok;
    if (H == 0 || batch->tokens == 0 || batch->sequences == 0) return LIN_OK;
    if ((ok = paged_heads_ok(cache, H, max_new)) != LIN_OK) return ok;
    const long long N = batch->tokens, width = (long long)H * cache->head_dim;
    if (!q || !out || ldq < width || ldo < width) return LIN_ERR_ARG;
    // scaled scores and their differences are fp32
    if (scale > 0.f && !(scale >= 0x1p-100f && scale <= 0x1p100f)) return LIN_ERR_ARG;
    // positions, clipped to +-1.5 * 2^30, plus a row's number are 32 bits in the kernels
    if (ldq > kMaxStride || ldo > kMaxStride || batch->sequences > (1 << 24) || N > (1 << 28)) return LIN_ERR_UNSUPPORTED;
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) % 16 != 0 || ldq % 8 != 0 || ldo % 8 != 0 ||
        (uintptr_t)lse % 4 != 0)
        return LIN_ERR_ALIGN;
    if (!workspace) {
        workspace_bytes = ctx->workspace_bytes > kCounterBytes ? ctx->workspace_bytes - kCounterBytes : 0;
        workspace = static_cast<char*>(ctx->workspace) + kCounterBytes;
    }
    const int rows = paged_rows(*cache, batch, H, max_new);
    if (workspace_bytes < paged_bytes(*ctx, *cache, rows)) return LIN_ERR_WORKSPACE;
    auto flat = [](const void* p, size_t bytes) { return Rows{p, 1, (long long)bytes, (long long)bytes, 1}; };
    const size_t held = cache_extent(*cache), lse_bytes = lse ? (size_t)N * H * 4 : 0;
    const Rows ro{out, N, width, ldo, 2}, rl = flat(lse, lse_bytes), rw = flat(workspace, workspace_bytes);
    const Rows inputs[] = {Rows{q, N, width, ldq, 2}, flat(cache->k, held), flat(cache->v, held), table_rows(*batch),
                           flat(batch->q_start, 4 * ((size_t)batch->sequences + 1)),
                           flat(batch->kv_len, 4 * (size_t)batch->sequences)};
    for (const Rows& r : inputs)
        if (rows_overlap(ro, r) || rows_overlap(rl, r) || rows_overlap(rw, r)) return LIN_ERR_ARG;
    if (rows_overlap(ro, rl) || rows_overlap(ro, rw) || rows_overlap(rl, rw)) return LIN_ERR_ARG;
    DeviceGuard guard(ctx->device);
    if (!guard.ok) return LIN_ERR_CUDA;
    PagedProblem p;
    p.cache = *cache;
    p.batch = *batch;
    p.H = H;
    p.q = q;
    p.ldq = ldq;
    p.out = out;
    p.ldo = ldo;
    p.lse = lse;
    p.causal = causal != 0;
    p.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)cache->head_dim);
    p.stream = static_cast<cudaStream_t>(stream);
    p.workspace = workspace;
    p.workspace_bytes = workspace_bytes;
    p.dev_status = ctx->dev_status;
    p.sm_count = ctx->sm_count;
    p.early_start = ctx->programmatic;
    Range hull{out, rows_extent(ro)};
    if (lse) {
        const char* lo = std::min(static_cast<const char*>(out), reinterpret_cast<const char*>(lse));
        const char* hi = std::max(static_cast<const char*>(out) + hull.bytes, reinterpret_cast<const char*>(lse) + lse_bytes);
        hull = Range{lo, (size_t)(hi - lo)};
    }
    note_output(p.stream, hull);
    return launched(rows <= kPagedRowsMax ? launch_paged_rows(p) : launch_paged_tiles(p), p.stream, hull);
}

int lin_check_device(lin_ctx* ctx, void* stream) {
    if (!ctx) return LIN_ERR_ARG;
    lin::DeviceGuard guard(ctx->device);
    if (!guard.ok) return LIN_ERR_CUDA;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return LIN_ERR_CUDA;
    int status = 0;
    if (cudaMemcpy(&status, ctx->dev_status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return LIN_ERR_CUDA;
    if (status != 0) {
        if (cudaMemset(ctx->dev_status, 0, sizeof(int)) != cudaSuccess) return LIN_ERR_CUDA;
        return status;
    }
    return LIN_OK;
}

}  // extern "C"

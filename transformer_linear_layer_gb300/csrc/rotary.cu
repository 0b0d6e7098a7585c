// Rotary positions, and the append of new keys and values to a paged cache with
// the rotation applied on the way.
//
//   pair i of a head's first `rot` elements (a, b = elements 2i and 2i + 1, or i
//   and i + rot/2) at position p:  theta = p f_i,
//     y_a = s (x_a cos theta - x_b sin theta),  y_b = s (x_a sin theta + x_b cos theta)
//   (the gradient: theta negated). The head's other elements are copied.
//
// Angles: f_i comes as turns per position in units of 2^-64 (f_i / 2 pi mod 1), so
// that the low 64 bits of p times it are p times the table's entry mod one turn, exactly, however
// far the position. The entry is off by 0.6 of a unit at most, so the angle is by p 2^-62
// radians: 3 10^-13 at position 10^6, 3 10^-4 at 2^50 (an fp32 product p f_i is off by 2^-24 p f_i
// radians: 0.06 at position 10^6). The nearest quarter turn is taken off in integers and
// sincospif sees at most an eighth of a turn.
//
// Memory bounds both: each element is read and written once. A thread has one place in a head (16
// bytes of pairs; with halves paired two times 16, rot/2 apart) and up to K heads of a row, which
// it asks for at once before the angles are computed; the cosines and sines of a block's rows are computed once,
// into shared memory, and read once a thread. v's heads are places of the same kind that do not turn.
// Element by element where sizes, strides or addresses do not allow 16 bytes. bf16 moves two to a word
// (with single elements converted and stored the kernel was bound by its instructions, 13 us for the
// first of the sizes below).
// Measured (GB300): 8192 x 24 heads of 64, bf16, halves 7.9 us (6.4 TB/s); 2331 x 10 heads of 128, fp32,
// half of each head, neighbours 3.9 us (6.2 TB/s); one row 1.4 us; append of 5757 rows of 32 + 16
// heads of 128 26.0 us (5.4 TB/s), of 64 rows of 12 + 24 heads of 64 2.7 us.
#include <limits.h>
#include <math.h>

#include "device_common.cuh"
#include "internal.h"
#include "paged.cuh"
#include "tc_common.cuh"

namespace lin {
namespace {

constexpr int kRtThreads = 256;
constexpr int kRtHeads = 4;         // heads a thread asks for at once
constexpr int kRtMaxRows = 8;       // rows a block takes, a warp each for where they go

struct RotaryArgs {
    RotaryProblem p;
    int heads;                      // of a row: q, k and v
    int turning;                    // q and k: those that turn
    int rot_units, units;           // places of a head that rotate, all
    int span;                       // places that a block takes (gridDim.z spans)
    int each;                       // head groups of a row: a thread has heads g, g + each, ...
    int chunk;                      // head groups that a block takes (gridDim.y chunks)
    int rows;                       // rows a block takes
};

// cos and sin at position p, modulo 2^64 (turns in units of 2^-64 of a turn per position).
__device__ __forceinline__ void turn(unsigned long long p, unsigned long long turns, float& c, float& s) {
    const unsigned long long t = p * turns;
    const unsigned q = static_cast<unsigned>((t + (1ull << 61)) >> 62);                  // nearest quarter
    const long long rest = static_cast<long long>(t - (static_cast<unsigned long long>(q) << 62));  // +- 2^61
    float c0, s0;
    sincospif(__ll2float_rn(rest) * 0x1p-63f, &s0, &c0);
    const float ca = (q & 1) ? s0 : c0, sa = (q & 1) ? c0 : s0;
    c = (q == 1 || q == 2) ? -ca : ca;
    s = q >= 2 ? -sa : sa;
}

// The pairs of a place turned, 16 bytes of each of x0 and x1 (halves paired) or of x0 alone: bf16
// two to a word, unpacked by shifts and rounded two at a time.
template <class T, bool INTER>
__device__ __forceinline__ void turn_words(uint32_t (&x0)[4], uint32_t (&x1)[4], const float* c, const float* s) {
    auto pair = [&](float& a, float& b, int e) {
        const float xa = a, xb = b;
        a = fmaf(xa, c[e], -(xb * s[e]));
        b = fmaf(xa, s[e], xb * c[e]);
    };
    if constexpr (sizeof(T) == 4 && !INTER) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float a = __uint_as_float(x0[w]), b = __uint_as_float(x1[w]);
            pair(a, b, w);
            x0[w] = __float_as_uint(a);
            x1[w] = __float_as_uint(b);
        }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int w = 0; w < 4; w += 2) {
            float a = __uint_as_float(x0[w]), b = __uint_as_float(x0[w + 1]);
            pair(a, b, w / 2);
            x0[w] = __float_as_uint(a);
            x0[w + 1] = __float_as_uint(b);
        }
    } else if constexpr (!INTER) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float a0 = __uint_as_float(x0[w] << 16), a1 = __uint_as_float(x0[w] & 0xffff0000u);
            float b0 = __uint_as_float(x1[w] << 16), b1 = __uint_as_float(x1[w] & 0xffff0000u);
            pair(a0, b0, 2 * w);
            pair(a1, b1, 2 * w + 1);
            x0[w] = pack_bf16x2(a0, a1);
            x1[w] = pack_bf16x2(b0, b1);
        }
    } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float a = __uint_as_float(x0[w] << 16), b = __uint_as_float(x0[w] & 0xffff0000u);
            pair(a, b, w);
            x0[w] = pack_bf16x2(a, b);
        }
    }
}

// V elements a thread's access holds; INTER: neighbours are paired; K heads a thread.
template <class T, int V, bool INTER, int K, bool APPEND>
__global__ void __launch_bounds__(kRtThreads) rotary_kernel(const RotaryArgs a) {
    extern __shared__ __align__(16) float s_turn[];  // cos then sin: rows x rot/2 each
    __shared__ long long s_dst[kRtMaxRows];   // append: the row's place in its page, < 0 for none
    __shared__ long long s_pos[kRtMaxRows];
    __shared__ int s_live[kRtMaxRows];
    const RotaryProblem& p = a.p;
    const int half = p.rot >> 1;
    const long long row0 = (long long)blockIdx.x * a.rows;
    const int rows = (int)(p.N - row0 < a.rows ? p.N - row0 : a.rows);
    const int g0 = blockIdx.y * a.chunk, chunk = min(a.chunk, a.each - g0);

    // This thread's row, head group and place.
    const int per_row = chunk * a.span;
    const int row = (unsigned)threadIdx.x / (unsigned)per_row, rest = threadIdx.x - row * per_row;
    const int in_row = (unsigned)rest / (unsigned)a.span;
    const int group = g0 + in_row, place = blockIdx.z * a.span + rest - in_row * a.span;
    const bool mine = row < rows && place < a.units, rot = place < a.rot_units;
    // its first element: past the rotated ones for the rest of the head; a scalar pair of neighbours starts at 2 place
    const int first = (V == 1 && INTER && rot) ? 2 * place : (rot ? place : place + p.rot / V - a.rot_units) * V;
    // The second access of a rotating place: rot/2 further, or the neighbour.
    constexpr bool TWO = !INTER || V == 1;
    const int apart = INTER ? 1 : half;

    pdl_wait();
    pdl_launch_dependents();

    uint32_t x0[K][4], x1[K][4];  // V == 1: the element's bits in the first
    auto load = [&](const T* src, uint32_t (&x)[4]) {
        if constexpr (V == 1) {
            if constexpr (sizeof(T) == 2)
                x[0] = (uint32_t)*reinterpret_cast<const uint16_t*>(src) << 16;
            else
                x[0] = *reinterpret_cast<const uint32_t*>(src);
        } else {
            const uint4 v = *reinterpret_cast<const uint4*>(src);
            x[0] = v.x;
            x[1] = v.y;
            x[2] = v.z;
            x[3] = v.w;
        }
    };
    // (a scalar that is only copied keeps its bits: a bf16 is its fp32's upper half)
    auto store = [&](T* dst, const uint32_t (&x)[4], bool turned) {
        if constexpr (V == 1) {
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<uint16_t*>(dst) =
                    turned ? f32_to_bf16_bits(__uint_as_float(x[0])) : (uint16_t)(x[0] >> 16);
            else
                *reinterpret_cast<uint32_t*>(dst) = x[0];
        } else {
            *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
        }
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int h = group + k * a.each;
        if (mine && h < a.heads) {
            const int part = !APPEND || h < p.part[0].heads ? 0 : h < a.turning ? 1 : 2;
            const int in = h - (part == 0 ? 0 : part == 1 ? p.part[0].heads : a.turning);
            const T* src = static_cast<const T*>(p.part[part].src) + (row0 + row) * p.part[part].ld_src + (in * p.D + first);
            load(src, x0[k]);
            if (TWO && rot) load(src + apart, x1[k]);
        }
    }

    // Positions, and the places in the cache.
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if constexpr (APPEND) {
        for (int r = warp; r < rows; r += blockDim.x >> 5) {
            const int n = (int)(row0 + r);
            int end, kv;
            const int b = find_sequence(p.batch.q_start, p.batch.kv_len, p.batch.sequences, n, end, kv);
            if (lane == 0) {
                long long pos = -1, dst = -1;
                const bool live = b >= 0 && n < end;
                if (live) {
                    pos = (long long)kv - end + n;
                    const int shift = 31 - __clz(p.cache.page_size);  // a power of two
                    if (pos >= 0 && pos < (long long)p.batch.table_pages << shift) {
                        const int page = p.batch.block_table[b * p.batch.table_stride + (pos >> shift)];
                        if (page >= 0 && page < p.cache.pages)
                            dst = page * p.cache.page_stride + (pos & (p.cache.page_size - 1)) * p.cache.token_stride;
                    }
                }
                s_live[r] = live;
                s_dst[r] = dst;
                s_pos[r] = pos;
            }
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < rows * half; i += blockDim.x) {
        const int r = (unsigned)i / (unsigned)half, f = i - r * half;
        long long pos;
        if (!APPEND || p.positions)
            pos = p.wide ? static_cast<const long long*>(p.positions)[row0 + r]
                         : (long long)static_cast<const int*>(p.positions)[row0 + r];
        else
            pos = s_pos[r];
        float c, s;
        turn(p.inverse ? 0ull - (unsigned long long)pos : (unsigned long long)pos, p.turns[f], c, s);
        s_turn[i] = c * p.scale;
        s_turn[rows * half + i] = s * p.scale;
    }
    __syncthreads();
    if (!mine) return;

    constexpr int P = TWO ? V : V / 2;  // pairs of a place
    alignas(16) float c[P], s[P];
    if (rot) {
        const float* cs = s_turn + row * half + place * P;
        const float* sn = cs + rows * half;
        if constexpr (P % 4 == 0) {
#pragma unroll
            for (int e = 0; e < P; e += 4) {
                *reinterpret_cast<float4*>(c + e) = *reinterpret_cast<const float4*>(cs + e);
                *reinterpret_cast<float4*>(s + e) = *reinterpret_cast<const float4*>(sn + e);
            }
        } else {
#pragma unroll
            for (int e = 0; e < P; ++e) {
                c[e] = cs[e];
                s[e] = sn[e];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int h = group + k * a.each;
        if (h >= a.heads) break;
        T* dst;
        if (!APPEND || h < p.part[0].heads) {
            if (APPEND && !s_live[row]) continue;
            dst = static_cast<T*>(p.part[0].dst) + (row0 + row) * p.part[0].ld_dst + h * p.D;
        } else {
            if (s_dst[row] < 0) continue;
            dst = h < a.turning ? static_cast<T*>(p.cache.k) + (h - p.part[0].heads) * p.cache.head_stride
                                : static_cast<T*>(p.cache.v) + (h - a.turning) * p.cache.head_stride;
            dst += s_dst[row];
        }
        dst += first;
        const bool turned = rot && (!APPEND || h < a.turning);
        if (turned) {
            if constexpr (V == 1) {
                const float xa = __uint_as_float(x0[k][0]), xb = __uint_as_float(x1[k][0]);
                x0[k][0] = __float_as_uint(fmaf(xa, c[0], -(xb * s[0])));
                x1[k][0] = __float_as_uint(fmaf(xa, s[0], xb * c[0]));
            } else {
                turn_words<T, INTER>(x0[k], x1[k], c, s);
            }
        }
        store(dst, x0[k], turned);
        if (TWO && rot) store(dst + apart, x1[k], turned);
    }
}

template <class T, int V, bool INTER, int K>
int start(const RotaryProblem& p) {
    RotaryArgs a;
    a.p = p;
    const int pair = p.rot / 2;
    a.turning = p.part[0].heads + p.part[1].heads;
    a.heads = a.turning + p.part[2].heads;
    a.rot_units = INTER ? (V == 1 ? pair : p.rot / V) : pair / V;
    // in place the rest of the head stays where it is
    const bool rest = p.append || p.part[0].src != p.part[0].dst;
    a.units = a.rot_units + (rest ? (p.D - p.rot) / V : 0);
    if (a.heads == 0 || a.units == 0) return LIN_OK;
    a.each = (a.heads + K - 1) / K;
    a.span = a.units < kRtThreads ? a.units : kRtThreads;
    a.chunk = a.each < kRtThreads / a.span ? a.each : kRtThreads / a.span;
    const int per_row = a.chunk * a.span;
    long long rows = kRtThreads / per_row;
    if (rows > kRtMaxRows) rows = kRtMaxRows;
    if (rows > p.N) rows = p.N;
    a.rows = (int)rows;
    const int chunks = (a.each + a.chunk - 1) / a.chunk;
    if (chunks > 65535) return LIN_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.N + rows - 1) / rows), (unsigned)chunks, (unsigned)((a.units + a.span - 1) / a.span));
    cfg.blockDim = dim3((unsigned)((rows * per_row + 31) / 32 * 32));
    cfg.dynamicSmemBytes = (size_t)rows * pair * 2 * sizeof(float);
    cfg.stream = p.stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = p.early_start ? 1 : 0;
    cudaError_t e;
    if constexpr (sizeof(T) == 2)
        e = p.append ? cudaLaunchKernelEx(&cfg, rotary_kernel<T, V, INTER, K, true>, a)
                     : cudaLaunchKernelEx(&cfg, rotary_kernel<T, V, INTER, K, false>, a);
    else
        e = cudaLaunchKernelEx(&cfg, rotary_kernel<T, V, INTER, K, false>, a);
    if (e != cudaSuccess) return LIN_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? LIN_OK : LIN_ERR_CUDA;
}

template <class T, bool INTER>
int start_width(const RotaryProblem& p) {
    constexpr int V = 16 / sizeof(T);
    bool wide = p.D % V == 0 && (INTER ? p.rot : p.rot / 2) % V == 0;
    auto fits = [&](const void* q, long long ld) { return (uintptr_t)q % 16 == 0 && ld % V == 0; };
    for (const RotaryPart& part : p.part)
        if (part.heads > 0) wide = wide && fits(part.src, part.ld_src) && fits(part.dst, part.ld_dst);
    // the cache's own addresses and strides are multiples of 16 bytes
    if (!wide) return start<T, 1, INTER, 1>(p);
    // Few rows: one head a thread, so that the row is done by as many threads as it has. Many: accesses in
    // flight count. Measured (us, with one head a thread and with four; device time):
    //     rows                          64         400         608        1024        2048        5760
    //     append, 12 + 24 heads of 64   2.6 3.8    2.9 3.9     3.1 4.0    3.8 4.0     5.7 4.6    12.0  9.5
    //     append, 32 + 16 heads of 128  2.7 3.4    3.8 3.8     5.7 4.1    8.2 5.6    14.0 8.9    38.1 26.9
    //     rotary, 24 heads of 64        1.7 2.2    1.8 2.3     2.1 2.4    2.5 2.4     3.0 3.1     5.6  4.8
    //     rotary, 10 of 128 in fp32     1.9 2.3    2.0 2.3     2.2 2.4    2.9 3.0     3.7 4.0     7.3  6.9
    // so that the border, 608 rows here, is late for wide rows and early for narrow ones, by 1.6 us at most.
    return p.N < 4 * p.sm_count ? start<T, V, INTER, 1>(p) : start<T, V, INTER, kRtHeads>(p);
}

}  // namespace

int launch_rotary(const RotaryProblem& p) {
    if (p.bf16) return p.interleaved ? start_width<uint16_t, true>(p) : start_width<uint16_t, false>(p);
    return p.interleaved ? start_width<float, true>(p) : start_width<float, false>(p);
}

}  // namespace lin

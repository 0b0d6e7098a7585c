// Rotary positions, and the append of new keys and values to a paged cache with
// the rotation applied on the way.
//
//   pair i of a head's first `rot` elements (a, b = elements 2i and 2i + 1, or i
//   and i + rot/2) at position p:  theta = p f_i,
//     y_a = s (x_a cos theta - x_b sin theta),  y_b = s (x_a sin theta + x_b cos theta)
//   (the gradient: theta negated). The head's other elements are copied.
//
// Angles: f_i comes as turns per position in units of 2^-64 (f_i / 2 pi mod 1), so
// that the low 64 bits of p times it are the angle mod one turn, exactly, however
// far the position (an fp32 product p f_i is off by 2^-24 p f_i radians: 0.06 at
// position 10^6). The nearest quarter turn is taken off in integers and
// sincospif sees at most an eighth of a turn.
//
// Memory bounds both: each element is read and written once. A block of 256
// threads takes a few rows (their cosines and sines are computed once for all
// heads, into shared memory) and moves 16-byte units: with neighbours paired a unit
// holds its pairs, with halves paired a thread moves two units, rot/2 apart. The
// first units are asked for before the angles are computed. Element by element where
// sizes, strides or addresses do not allow 16 bytes.
#include <limits.h>
#include <math.h>

#include "device_common.cuh"
#include "internal.h"
#include "paged.cuh"
#include "tc_common.cuh"

namespace lin {
namespace {

constexpr int kRtThreads = 256;
constexpr int kRtMaxRows = 8;       // rows a block takes

struct RotaryArgs {
    RotaryProblem p;
    int rows;                       // rows a block takes
    int rot_units, units;           // of a rotated head: units that rotate, all
    int copy_units;                 // of a head that is only copied (v)
    int row_units;                  // of a row
    int chunk;                      // units of a row that a block takes (gridDim.y chunks)
};

// cos and sin of p turns (turns in units of 2^-64 of a turn per position).
__device__ __forceinline__ void turn(long long p, unsigned long long turns, float& c, float& s) {
    const unsigned long long t = static_cast<unsigned long long>(p) * turns;
    const unsigned q = static_cast<unsigned>((t + (1ull << 61)) >> 62);                  // nearest quarter
    const long long rest = static_cast<long long>(t - (static_cast<unsigned long long>(q) << 62));  // +- 2^61
    float c0, s0;
    sincospif(__ll2float_rn(rest) * 0x1p-63f, &s0, &c0);
    const float ca = (q & 1) ? s0 : c0, sa = (q & 1) ? c0 : s0;
    c = (q == 1 || q == 2) ? -ca : ca;
    s = q >= 2 ? -sa : sa;
}

template <class T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(uint16_t v) { return bf16_bits_to_f32(v); }
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f(float v) { return f32_to_bf16_bits(v); }

// A unit: V elements that move as one access.
template <class T, int V>
struct alignas(V * sizeof(T)) Unit {
    T e[V];
};

// V elements a thread's access holds; INTER: neighbours are paired.
template <class T, int V, bool INTER>
__global__ void __launch_bounds__(kRtThreads) rotary_kernel(const RotaryArgs a) {
    using U = Unit<T, V>;
    extern __shared__ float s_turn[];  // cos then sin: rows x rot/2 each
    __shared__ long long s_dst[kRtMaxRows];   // append: the row's place in its page, < 0 for none
    __shared__ long long s_pos[kRtMaxRows];
    __shared__ int s_live[kRtMaxRows];
    const RotaryProblem& p = a.p;
    const int half = p.rot >> 1;
    const long long row0 = (long long)blockIdx.x * a.rows;
    const int rows = (int)(p.N - row0 < a.rows ? p.N - row0 : a.rows);
    const int u0 = blockIdx.y * a.chunk;
    const int chunk = a.row_units - u0 < a.chunk ? a.row_units - u0 : a.chunk;
    const int total = rows * chunk;
    const int q_units = p.part[0].heads * a.units, k_units = p.part[1].heads * a.units;

    pdl_wait();
    pdl_launch_dependents();

    // Where unit i of the block's lies: part, head, element, and whether it rotates.
    struct Place {
        const T* src;
        int part, head, u, row;
        bool rot;
    };
    auto place = [&](int i) {
        Place w;
        w.row = (unsigned)i / (unsigned)chunk;
        int r = u0 + (i - w.row * chunk);
        w.part = r < q_units ? 0 : r < q_units + k_units ? 1 : 2;
        if (w.part > 0) r -= q_units;
        if (w.part > 1) r -= k_units;
        const int per = w.part == 2 ? a.copy_units : a.units;
        w.head = (unsigned)r / (unsigned)per;
        w.u = r - w.head * per;
        w.rot = w.part != 2 && w.u < a.rot_units;
        if (w.part != 2 && !w.rot) w.u += p.rot / V - a.rot_units;  // past the rotated elements
        // unit u starts at element u V, but a scalar pair of neighbours at 2u
        const int e = (V == 1 && INTER && w.rot) ? 2 * w.u : w.u * V;
        w.src = static_cast<const T*>(p.part[w.part].src) + (row0 + w.row) * p.part[w.part].ld_src +
                (long long)w.head * p.D + e;
        return w;
    };
    // The second access of a rotating unit: rot/2 further, or the neighbour.
    constexpr bool TWO = !INTER || V == 1;
    const int apart = INTER ? 1 : half;

    U x0, x1;
    Place w;
    if (threadIdx.x < total) {
        w = place(threadIdx.x);
        x0 = *reinterpret_cast<const U*>(w.src);
        if (TWO && w.rot) x1 = *reinterpret_cast<const U*>(w.src + apart);
    }

    // Positions, and the places in the cache.
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (p.append) {
        if (warp < rows) {
            const int n = (int)(row0 + warp);
            const int b = find_sequence(p.batch.q_start, p.batch.sequences, n);
            if (lane == 0) {
                long long pos = -1, dst = -1;
                int live = 0;
                if (b >= 0) {
                    const int end = p.batch.q_start[b + 1];
                    if (n < end) {
                        live = 1;
                        pos = (long long)p.batch.kv_len[b] - end + n;
                        const long long slots = (long long)p.batch.table_pages * p.cache.page_size;
                        if (pos >= 0 && pos < slots) {
                            const int page = p.batch.block_table[b * p.batch.table_stride + pos / p.cache.page_size];
                            if (page >= 0 && page < p.cache.pages)
                                dst = page * p.cache.page_stride + pos % p.cache.page_size * p.cache.token_stride;
                        }
                    }
                }
                s_live[warp] = live;
                s_dst[warp] = dst;
                s_pos[warp] = pos;
            }
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < rows * half; i += kRtThreads) {
        const int r = (unsigned)i / (unsigned)half, f = i - r * half;
        long long pos;
        if (p.positions)
            pos = p.wide ? static_cast<const long long*>(p.positions)[row0 + r]
                         : (long long)static_cast<const int*>(p.positions)[row0 + r];
        else
            pos = s_pos[r];
        float c, s;
        turn(p.inverse ? -pos : pos, p.turns[f], c, s);
        s_turn[i] = c * p.scale;
        s_turn[rows * half + i] = s * p.scale;
    }
    __syncthreads();

    for (int i = threadIdx.x; i < total;) {
        T* dst = nullptr;
        if (!p.append) {
            dst = static_cast<T*>(p.part[0].dst) + (row0 + w.row) * p.part[0].ld_dst;
        } else if (w.part == 0) {
            if (s_live[w.row]) dst = static_cast<T*>(p.part[0].dst) + (row0 + w.row) * p.part[0].ld_dst;
        } else if (s_dst[w.row] >= 0) {
            dst = static_cast<T*>(w.part == 1 ? p.cache.k : p.cache.v) + s_dst[w.row];
        }
        if (dst) {
            dst += w.part == 0 ? (long long)w.head * p.D : w.head * p.cache.head_stride;
            dst += (V == 1 && INTER && w.rot) ? 2 * w.u : w.u * V;
            if (w.rot) {
                const float* cs = s_turn + w.row * half;
                const float* sn = cs + rows * half;
                if constexpr (TWO) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float c = cs[w.u * V + e], s = sn[w.u * V + e];
                        const float xa = to_f(x0.e[e]), xb = to_f(x1.e[e]);
                        x0.e[e] = from_f<T>(fmaf(xa, c, -(xb * s)));
                        x1.e[e] = from_f<T>(fmaf(xa, s, xb * c));
                    }
                    *reinterpret_cast<U*>(dst + apart) = x1;
                } else {
#pragma unroll
                    for (int e = 0; e < V; e += 2) {
                        const float c = cs[(w.u * V + e) >> 1], s = sn[(w.u * V + e) >> 1];
                        const float xa = to_f(x0.e[e]), xb = to_f(x0.e[e + 1]);
                        x0.e[e] = from_f<T>(fmaf(xa, c, -(xb * s)));
                        x0.e[e + 1] = from_f<T>(fmaf(xa, s, xb * c));
                    }
                }
            }
            *reinterpret_cast<U*>(dst) = x0;
        }
        i += kRtThreads;
        if (i < total) {
            w = place(i);
            x0 = *reinterpret_cast<const U*>(w.src);
            if (TWO && w.rot) x1 = *reinterpret_cast<const U*>(w.src + apart);
        }
    }
}

template <class T, int V, bool INTER>
int start(const RotaryProblem& p) {
    RotaryArgs a;
    a.p = p;
    const int pair = p.rot / 2;
    a.rot_units = INTER ? (V == 1 ? pair : p.rot / V) : pair / V;
    // in place the rest of the head stays where it is
    const bool rest = p.append || p.part[0].src != p.part[0].dst;
    a.units = a.rot_units + (rest ? (p.D - p.rot) / V : 0);
    a.copy_units = p.D / V;
    const long long row_units =
        (long long)(p.part[0].heads + p.part[1].heads) * a.units + (long long)p.part[2].heads * a.copy_units;
    if (row_units == 0) return LIN_OK;
    if (row_units > INT_MAX / kRtMaxRows) return LIN_ERR_UNSUPPORTED;
    a.row_units = (int)row_units;
    // Rows enough for three accesses a thread, but blocks enough for two an SM;
    // few rows: their units are spread over blocks of one access a thread.
    long long rows = 3 * kRtThreads / row_units;
    if (rows > p.N / (2 * p.sm_count)) rows = p.N / (2 * p.sm_count);
    if (rows > kRtMaxRows) rows = kRtMaxRows;
    if (rows < 1) rows = 1;
    a.rows = (int)rows;
    long long chunks = 1;
    if (p.N < 2 * p.sm_count) {
        chunks = (row_units + kRtThreads - 1) / kRtThreads;
        if (chunks > 64) chunks = 64;
    }
    a.chunk = (int)((row_units + chunks - 1) / chunks);
    chunks = (row_units + a.chunk - 1) / a.chunk;
    const long long grid = (p.N + rows - 1) / rows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, (unsigned)chunks);
    cfg.blockDim = dim3(kRtThreads);
    cfg.dynamicSmemBytes = (size_t)rows * pair * 2 * sizeof(float);
    cfg.stream = p.stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = p.early_start ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, rotary_kernel<T, V, INTER>, a) != cudaSuccess) return LIN_ERR_CUDA;
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
    return wide ? start<T, V, INTER>(p) : start<T, 1, INTER>(p);
}

}  // namespace

int launch_rotary(const RotaryProblem& p) {
    if (p.bf16) return p.interleaved ? start_width<uint16_t, true>(p) : start_width<uint16_t, false>(p);
    return p.interleaved ? start_width<float, true>(p) : start_width<float, false>(p);
}

}  // namespace lin

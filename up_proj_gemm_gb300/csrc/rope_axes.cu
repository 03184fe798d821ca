// Rotary positions with several axes (time, height, width, ...): every
// rotation pair i of a head follows one axis a(i), and token t turns it by
// the table row of its position on that axis, p_i = pos[a(i)][t]. With
// h = Dr/2 and column j of the cos/sin tables for rope channel j,
//   apply    out_i = x_i cos[p_i][i] - x_{i+h} sin[p_i][i]
//            out_{i+h} = x_{i+h} cos[p_i][i+h] + x_i sin[p_i][i+h]
//   inverse  out_i = g_i cos[p_i][i] + g_{i+h} sin[p_i][i+h]
//            out_{i+h} = g_{i+h} cos[p_i][i+h] - g_i sin[p_i][i]
// (the Jacobian transpose of apply: its gradient). The sum mode turns the
// sum of all heads' gradients, the gradient of a key part that the heads
// share. Products and sums are float32, one rounding at the store.
//
// All of it is bound by HBM: each element is read and written once, by
// 16-byte accesses where pointers and strides allow.
#include <cuda_runtime.h>

#include <cstdint>

#include "checks.h"
#include "internal.h"
#include "launch.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace mlaq {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;        // rows in flight per thread (two vectors each)
constexpr int kRowBlocks = 4;     // resident blocks per SM: with kUnroll, 64 KB of loads in flight
constexpr int kRunRows = 8;       // rows per thread at most
constexpr int kFill = 4;          // table entries in flight per thread
constexpr int kTableBytes = 16384;  // the gathered entries of a block's tokens at most
constexpr int kMaxPairs = 128;    // Dr <= 256
constexpr int64_t kMaxD = 8192;

struct RopeParams {
    const void* in;
    void* out;
    int64_t T, rows;              // rows = T * H
    int64_t in_t, in_h, out_t, out_h;
    int H, Dn, Dr;
    int inverse;
    const float* cos_tab;
    const float* sin_tab;
    int64_t cs_rows, cs_width;
    const int32_t* pos;           // [axes][T]
    int* status;
    int rows_per_block;
    uint8_t axis[kMaxPairs];
};

// VE elements in 32-bit registers as they lie in memory (16 bytes when VE > 1).
template <typename E, int VE>
struct Raw {
    uint32_t u[VE == 1 ? 1 : 4];

    __device__ __forceinline__ void load(const E* p) {
        if constexpr (VE == 1) {
            if constexpr (sizeof(E) == 2) u[0] = *p;
            else u[0] = __float_as_uint(*p);
        } else {
            const uint4 w = *reinterpret_cast<const uint4*>(p);
            u[0] = w.x;
            u[1] = w.y;
            u[2] = w.z;
            u[3] = w.w;
        }
    }
    __device__ __forceinline__ void store(E* p) const {
        if constexpr (VE == 1) {
            if constexpr (sizeof(E) == 2) *p = (uint16_t)u[0];
            else *p = __uint_as_float(u[0]);
        } else {
            st_global_v4(p, u[0], u[1], u[2], u[3]);
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(E) == 4) return __uint_as_float(u[i]);
        else return i & 1 ? bf16hi_to_f32(u[i / 2]) : bf16lo_to_f32(u[i / 2]);
    }
    __device__ __forceinline__ void set(const float (&v)[VE]) {
        if constexpr (sizeof(E) == 4) {
#pragma unroll
            for (int i = 0; i < VE; ++i) u[i] = __float_as_uint(v[i]);
        } else if constexpr (VE == 1) {
            u[0] = pack_bf16x2(v[0], 0.f);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        }
    }
};

// The position of token t on the axis of rope channel j (j < Dr).
__device__ __forceinline__ int64_t position(const RopeParams& p, int j, int64_t t) {
    const int half = p.Dr / 2;
    return p.pos[p.axis[j < half ? j : j - half] * p.T + t];
}
__device__ __forceinline__ bool in_table(const RopeParams& p, int64_t row) { return row >= 0 && row < p.cs_rows; }

// VE floats of shared memory (by 16 bytes when VE > 1).
template <int VE>
__device__ __forceinline__ void from_table(const float* q, float (&v)[VE]) {
    if constexpr (VE == 1) {
        v[0] = *q;
    } else {
#pragma unroll
        for (int k = 0; k < VE; k += 4) {
            const float4 f = *reinterpret_cast<const float4*>(q + k);
            v[k] = f.x;
            v[k + 1] = f.y;
            v[k + 2] = f.z;
            v[k + 3] = f.w;
        }
    }
}

// apply and inverse. A block takes a run of (token, head) rows. It gathers
// the cos/sin entries of the run's tokens into shared memory once (a thread
// that kept its own in registers had room for too few loads in flight: 1.7
// against 5.x TB/s); a thread then owns one slot of a row, two vectors of VE
// elements: a pair vector (channels i.. and i+h..), or two vectors of the
// pass-through channels, and walks the rows, kUnroll in flight. The first
// rows are on their way while the table is gathered.
template <typename E, int VE>
__global__ void __launch_bounds__(kThreads, kRowBlocks) rope_axes_kernel(const __grid_constant__ RopeParams p) {
    extern __shared__ float4 table4[];  // [token of the run][cos Dr | sin Dr]
    grid_launch_next();
    grid_wait_previous();
    float* table = reinterpret_cast<float*>(table4);
    const int half = p.Dr / 2;
    const int n_pair = half / VE, n_copy = p.Dn / VE;
    const int n_copy2 = (n_copy + 1) / 2;
    const int slots = n_copy2 + n_pair;
    const bool narrow = slots <= kThreads;
    const int lanes = narrow ? kThreads / slots : 1;  // rows walked side by side
    const int lane = narrow ? (int)threadIdx.x / slots : 0;
    const int64_t r_begin = (int64_t)blockIdx.x * p.rows_per_block;
    const int64_t r_end = r_begin + p.rows_per_block < p.rows ? r_begin + p.rows_per_block : p.rows;
    const int t_first = (int)((uint32_t)r_begin / (uint32_t)p.H);
    const int toks = (int)((uint32_t)(r_end - 1) / (uint32_t)p.H) - t_first + 1;
    const int h_first = (int)((uint32_t)r_begin - (uint32_t)t_first * (uint32_t)p.H);
    const int step_t = lanes / p.H, step_h = lanes - step_t * p.H;
    const E* in = static_cast<const E*>(p.in) + t_first * p.in_t;
    E* out = static_cast<E*>(p.out) + t_first * p.out_t;
    bool filled = false;
    const int rounds = narrow ? 1 : (slots + kThreads - 1) / kThreads;
    for (int k0 = 0; k0 < rounds; ++k0) {
        // threads without a slot only help to fill the table
        const int s = (int)threadIdx.x - lane * slots + k0 * kThreads;
        const bool works = s < slots && lane < lanes;
        const bool pair = s >= n_copy2;
        const int i0 = pair ? (s - n_copy2) * VE : 0;
        const int ca = pair ? p.Dn + i0 : s * VE;
        const int cb = pair ? ca + half : (s + n_copy2) * VE;
        const bool two = works && (pair || s + n_copy2 < n_copy);
        // the lane's next row, in tokens of the run and heads, and how far it moves
        int left = works ? ((int)(r_end - r_begin) - lane + lanes - 1) / lanes : 0;  // rows of this lane
        int tn = (h_first + lane) / p.H, hn = h_first + lane - tn * p.H;
        do {
            Raw<E, VE> a[kUnroll], b[kUnroll];
            int t[kUnroll], h[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                t[u] = tn;
                h[u] = hn;
                tn += step_t;
                hn += step_h;
                if (hn >= p.H) {
                    hn -= p.H;
                    ++tn;
                }
                if (u >= left) continue;
                const E* x = in + t[u] * p.in_t + h[u] * p.in_h;
                a[u].load(x + ca);
                if (two) b[u].load(x + cb);
            }
            if (!filled) {
                const int n = toks * p.Dr;
                for (int i0f = threadIdx.x; i0f < n; i0f += kFill * kThreads) {
                    int64_t row[kFill];
                    float cv[kFill], sv[kFill];
#pragma unroll
                    for (int q = 0; q < kFill; ++q) {
                        const int i = i0f + q * kThreads, tt = i / p.Dr;
                        row[q] = i < n ? position(p, i - tt * p.Dr, t_first + tt) : 0;
                    }
#pragma unroll
                    for (int q = 0; q < kFill; ++q) {
                        const int i = i0f + q * kThreads, j = i % p.Dr;
                        const bool ok = i < n && in_table(p, row[q]);
                        cv[q] = ok ? p.cos_tab[row[q] * p.cs_width + j] : 0.f;
                        sv[q] = ok ? p.sin_tab[row[q] * p.cs_width + j] : 0.f;
                    }
#pragma unroll
                    for (int q = 0; q < kFill; ++q) {
                        const int i = i0f + q * kThreads, tt = i / p.Dr, j = i - tt * p.Dr;
                        if (i >= n) break;
                        if (!in_table(p, row[q])) record_status(p.status, MLA_ERR_POS_RANGE);
                        table[tt * 2 * p.Dr + j] = cv[q];
                        table[tt * 2 * p.Dr + p.Dr + j] = sv[q];
                    }
                }
                __syncthreads();
                filled = true;
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (u >= left) continue;
                if (pair) {
                    const float* c = table + t[u] * 2 * p.Dr + i0;
                    float c0[VE], s0[VE], c1[VE], s1[VE], x[VE], y[VE];
                    from_table<VE>(c, c0);
                    from_table<VE>(c + half, c1);
                    from_table<VE>(c + p.Dr, s0);
                    from_table<VE>(c + p.Dr + half, s1);
#pragma unroll
                    for (int k = 0; k < VE; ++k) {
                        const float v = a[u].get(k), w = b[u].get(k);
                        x[k] = p.inverse ? v * c0[k] + w * s1[k] : v * c0[k] - w * s0[k];
                        y[k] = p.inverse ? w * c1[k] - v * s0[k] : w * c1[k] + v * s1[k];
                    }
                    a[u].set(x);
                    b[u].set(y);
                }
                E* o = out + t[u] * p.out_t + h[u] * p.out_h;
                a[u].store(o + ca);
                if (two) b[u].store(o + cb);
            }
            left -= kUnroll;
        } while (left > 0);
    }
}

// The same without a block's table, one slot of one row per thread: for
// tensors of few heads, whose tokens' entries serve too few rows to be gathered
// first ([8190, 1, 64] bf16 3.4 against 8.1 us, [8190, 16, 64] 11.0 against 12.3,
// but [8190, 32, 64] 20.0 against 17.6), and for whatever is resident at once
// ([30, 100, 32 + 96] 2.7 against 3.3).
constexpr int kFewHeads = 16;

template <typename E, int VE>
__global__ void __launch_bounds__(kThreads) rope_few_kernel(const __grid_constant__ RopeParams p) {
    grid_launch_next();
    grid_wait_previous();
    const int half = p.Dr / 2;
    const int n_copy = p.Dn / VE, n_copy2 = (n_copy + 1) / 2;
    const uint32_t slots = n_copy2 + half / VE;
    const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t r = item / slots;
    if (r >= p.rows) return;
    const int s = (int)(item - r * slots);
    const int t = (int)((uint32_t)r / (uint32_t)p.H), h = (int)((uint32_t)r - (uint32_t)t * (uint32_t)p.H);
    const bool pair = s >= n_copy2;
    const int i0 = pair ? (s - n_copy2) * VE : 0;
    const int ca = pair ? p.Dn + i0 : s * VE;
    const int cb = pair ? ca + half : (s + n_copy2) * VE;
    const bool two = pair || s + n_copy2 < n_copy;
    const E* x = static_cast<const E*>(p.in) + t * p.in_t + h * p.in_h;
    E* o = static_cast<E*>(p.out) + t * p.out_t + h * p.out_h;
    Raw<E, VE> a, b;
    a.load(x + ca);
    if (two) b.load(x + cb);
    if (pair) {
        int64_t row[VE];
#pragma unroll
        for (int k = 0; k < VE; ++k) row[k] = position(p, i0 + k, t);
        float v[VE], w[VE];
        bool ok = true;  // reported behind the loads: none of them may pass the report
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            const bool in = in_table(p, row[k]);
            ok &= in;
            const int64_t at = (in ? row[k] : 0) * p.cs_width + i0 + k;
            const float c0 = p.cos_tab[at], c1 = p.cos_tab[at + half];
            const float s0 = p.sin_tab[at], s1 = p.sin_tab[at + half];
            const float u = a.get(k), y = b.get(k);
            v[k] = p.inverse ? u * c0 + y * s1 : u * c0 - y * s0;
            w[k] = p.inverse ? y * c1 - u * s0 : y * c1 + u * s1;
        }
        if (!ok) record_status(p.status, MLA_ERR_POS_RANGE);
        a.set(v);
        b.set(w);
    }
    a.store(o + ca);
    if (two) b.store(o + cb);
}

// The sum over heads, turned. Warps work alone: a lane owns one slot of a
// token's row (two vectors of VE channels, as in rope_axes_kernel) and every
// hl-th head, adds them in float32 in its registers, and the hl lanes of a slot
// meet by shuffles, in an order that does not depend on scheduling. hl is the
// largest power of two that fits the warp beside the slots; the rest of the
// warp takes other tokens. (A block per token with sums in shared memory waited
// for itself: [8190, 8, 128] bf16 18.1 us.)
// [4096, 128, 64] of 192 channels' rows, bf16: 15.8 us, 4.4 TB/s (blocks of 128
// 15.9; positions read pair by pair 16.9; [300, 100, 64] 3.7, 3.9, 4.5).
constexpr int kSumThreads = 64;
constexpr int kSumHeads = 4;  // heads in flight per lane (20 warps per SM; 32 with 2 heads lost a third at D = 192)

template <typename E, int VE>
__global__ void __launch_bounds__(kSumThreads, 10) rope_sum_kernel(const __grid_constant__ RopeParams p, int hl, int per_warp) {
    grid_launch_next();
    grid_wait_previous();
    const int half = p.Dr / 2;
    const int n_copy = p.Dn / VE, n_copy2 = (n_copy + 1) / 2;
    const int slots = n_copy2 + half / VE;
    const int lane = threadIdx.x & 31;
    const int64_t warp = ((int64_t)blockIdx.x * kSumThreads + threadIdx.x) >> 5;
    const int width = slots < 32 ? slots : 32;            // lanes side by side over the slots
    const int tw = lane / (width * hl);                   // token of the warp
    const int h0 = (lane - tw * width * hl) / width;      // first head of the lane
    const int64_t t = warp * per_warp + tw;
    const bool works = tw < per_warp && t < p.T;
    const E* x = static_cast<const E*>(p.in) + t * p.in_t;
    E* out = static_cast<E*>(p.out) + t * p.out_t;
    for (int s0 = 0; s0 < slots; s0 += width) {
        const int s = s0 + lane - (tw * hl + h0) * width;
        const bool mine = works && s < slots;
        const bool pair = s >= n_copy2;
        const int i0 = pair ? (s - n_copy2) * VE : 0;
        const int ca = pair ? p.Dn + i0 : s * VE;
        const int cb = pair ? ca + half : (s + n_copy2) * VE;
        const bool two = mine && (pair || s + n_copy2 < n_copy);
        float a[VE], b[VE];
#pragma unroll
        for (int k = 0; k < VE; ++k) a[k] = b[k] = 0.f;
        for (int h = h0; h < (mine ? p.H : 0); h += hl * kSumHeads) {
            Raw<E, VE> va[kSumHeads], vb[kSumHeads];
#pragma unroll
            for (int u = 0; u < kSumHeads; ++u) {
                if (h + u * hl >= p.H) continue;
                const E* q = x + (int64_t)(h + u * hl) * p.in_h;
                va[u].load(q + ca);
                if (two) vb[u].load(q + cb);
            }
#pragma unroll
            for (int u = 0; u < kSumHeads; ++u) {
                if (h + u * hl >= p.H) continue;
#pragma unroll
                for (int k = 0; k < VE; ++k) {
                    a[k] += va[u].get(k);
                    if (two) b[k] += vb[u].get(k);
                }
            }
        }
        // the positions all at once, and under the shuffles; then all the table's entries
        const bool turns = mine && pair && h0 == 0;
        int row[VE];
#pragma unroll
        for (int k = 0; k < VE; ++k) row[k] = turns ? (int)position(p, i0 + k, t) : 0;
        __syncwarp();
        for (int d = hl / 2; d >= 1; d /= 2)
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                a[k] += __shfl_down_sync(0xffffffffu, a[k], d * width);
                b[k] += __shfl_down_sync(0xffffffffu, b[k], d * width);
            }
        if (!mine || h0 != 0) continue;
        if (pair) {
            float c0[VE], c1[VE], n0[VE], n1[VE];
            bool ok = true;
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                const bool in = in_table(p, row[k]);
                ok &= in;
                const int64_t at = (in ? row[k] : 0) * p.cs_width + i0 + k;
                c0[k] = p.cos_tab[at];
                c1[k] = p.cos_tab[at + half];
                n0[k] = p.sin_tab[at];
                n1[k] = p.sin_tab[at + half];
            }
            if (!ok) record_status(p.status, MLA_ERR_POS_RANGE);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                const float u = a[k], w = b[k];
                a[k] = u * c0[k] + w * n1[k];
                b[k] = w * c1[k] - u * n0[k];
            }
        }
        Raw<E, VE> ra, rb;
        ra.set(a);
        ra.store(out + ca);
        if (two) {
            rb.set(b);
            rb.store(out + cb);
        }
    }
}

// The cos/sin rows of every token, gathered per pair: a table for the fused
// projection, whose positions are then the token numbers. A thread owns N
// columns (4 when the tables allow 16-byte accesses) of U tokens: their positions
// are all asked for first, then their table entries, since the time is these two
// latencies. (A loop over single elements: T = 16384, Dr = 64 7.5 us; U = 1, 2, 4:
// 6.0, 5.3, 6.6. T = 100: 2.9; 2.1, 2.7, 3.6. T = 131072, Dr = 128: 99; 109, 64, 51.)
template <int N, int U>
__global__ void __launch_bounds__(kThreads) rope_table_kernel(const __grid_constant__ RopeParams p,
                                                              float* cos_out, float* sin_out) {
    grid_launch_next();
    grid_wait_previous();
    const int half = p.Dr / 2;
    const int cols = p.Dr / N, tokens = kThreads / cols;  // of a block at a time
    const int mine = threadIdx.x / cols, c = (threadIdx.x - mine * cols) * N;
    const int64_t t0 = (int64_t)blockIdx.x * tokens * U + mine;
    if (mine >= tokens) return;
    const int i = c < half ? c : c - half;
    bool same = true;
#pragma unroll
    for (int k = 1; k < N; ++k) same &= c < half == c + k < half && p.axis[i + k] == p.axis[i];
    int64_t at[U][N];
    bool ok[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t t = t0 + u * tokens;
        if (t >= p.T) break;
#pragma unroll
        for (int k = 0; k < N; ++k) at[u][k] = k > 0 && same ? at[u][0] : position(p, c + k, t);
    }
    float cv[U][N], sv[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (t0 + u * tokens >= p.T) break;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            ok[u][k] = in_table(p, at[u][k]);
            at[u][k] = (ok[u][k] ? at[u][k] : 0) * p.cs_width + c;
        }
        if (N == 4 && same) {
            const float4 a = *reinterpret_cast<const float4*>(p.cos_tab + at[u][0]);
            const float4 b = *reinterpret_cast<const float4*>(p.sin_tab + at[u][0]);
            cv[u][0] = a.x, cv[u][1 % N] = a.y, cv[u][2 % N] = a.z, cv[u][3 % N] = a.w;
            sv[u][0] = b.x, sv[u][1 % N] = b.y, sv[u][2 % N] = b.z, sv[u][3 % N] = b.w;
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                cv[u][k] = p.cos_tab[at[u][k] + k];
                sv[u][k] = p.sin_tab[at[u][k] + k];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t t = t0 + u * tokens;
        if (t >= p.T) break;
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (!ok[u][k]) {  // reported behind the loads: none of them may pass the report
                record_status(p.status, MLA_ERR_POS_RANGE);
                cv[u][k] = sv[u][k] = 0.f;
            }
        float* co = cos_out + t * p.Dr + c;
        float* so = sin_out + t * p.Dr + c;
        if constexpr (N == 4) {
            *reinterpret_cast<float4*>(co) = make_float4(cv[u][0], cv[u][1], cv[u][2], cv[u][3]);
            *reinterpret_cast<float4*>(so) = make_float4(sv[u][0], sv[u][1], sv[u][2], sv[u][3]);
        } else {
            *co = cv[u][0];
            *so = sv[u][0];
        }
    }
}

template <typename E, int VE>
int launch_rows(RopeParams p, bool sum, int num_sms, cudaStream_t stream) {
    if (sum) {
        const int slots = (p.Dn / VE + 1) / 2 + p.Dr / 2 / VE;
        const int width = slots < 32 ? slots : 32;
        int hl = 1;
        while (2 * hl * width <= 32 && hl < p.H) hl *= 2;
        const int per_warp = 32 / (width * hl);
        const int64_t warps = (p.T + per_warp - 1) / per_warp;
        const int64_t grid = (warps * 32 + kSumThreads - 1) / kSumThreads;
        return launch_overlapped(rope_sum_kernel<E, VE>, (unsigned)grid, kSumThreads, 0, 0, stream, p, hl, per_warp);
    } else if (p.H <= kFewHeads || p.rows * ((p.Dn / VE + 1) / 2 + p.Dr / 2 / VE) <= (int64_t)num_sms * 2048) {
        const int slots = (p.Dn / VE + 1) / 2 + p.Dr / 2 / VE;
        const int64_t grid = (p.rows * slots + kThreads - 1) / kThreads;
        if (grid > kI32Max) return MLA_ERR_UNSUPPORTED;
        return launch_overlapped(rope_few_kernel<E, VE>, (unsigned)grid, kThreads, 0, 0, stream, p);
    } else {
        const int slots = (p.Dn / VE + 1) / 2 + p.Dr / 2 / VE;
        const int lanes = kThreads / slots > 0 ? kThreads / slots : 1;
        // up to kRunRows rows per thread, fewer when the grid would not fill the SMs or the table its room
        const int64_t tok_rows = kTableBytes / (8 * p.Dr);  // tokens whose entries fit
        int64_t per = (p.rows + (int64_t)lanes * num_sms * kRowBlocks - 1) / ((int64_t)lanes * num_sms * kRowBlocks);
        per = per < 1 ? 1 : (per > kRunRows ? kRunRows : per);
        int64_t run = per * lanes;
        if ((run + p.H - 2) / p.H + 1 > tok_rows) run = (tok_rows - 1) * p.H;
        p.rows_per_block = (int)run;
        const int64_t grid = (p.rows + run - 1) / run;
        const int64_t most = (run + p.H - 2) / p.H + 1;  // tokens that a run may touch
        return launch_overlapped(rope_axes_kernel<E, VE>, (unsigned)grid, kThreads, (size_t)(most * 8 * p.Dr), 0, stream, p);
    }
}

// The checks that the entry points share; fills the parameters.
int check_axes(const mla_rope_axes_shape* s, const float* cos_tab, const float* sin_tab, const int32_t* pos,
               const uint8_t* pair_axis, const int* dev_status, RopeParams* p) {
    if (!s) return MLA_ERR_INVALID_ARG;
    if (s->T < 0 || s->H <= 0 || s->Dn < 0 || s->Dr <= 0 || (s->Dr & 1) || s->axes <= 0 || s->cs_rows < 0 ||
        s->cs_width < 0 || s->reserved != 0)
        return MLA_ERR_INVALID_ARG;
    if (s->T > kI32Max || s->T * s->H > kI32Max || s->cs_rows > kI32Max || s->cs_width > kI32Max || !pair_axis)
        return MLA_ERR_INVALID_ARG;
    if (s->cs_width < s->Dr) return MLA_ERR_ROPE_WIDTH;
    if (s->T > 0 && (!cos_tab || !sin_tab || !pos)) return MLA_ERR_INVALID_ARG;
    if (s->cs_rows == 0 && s->T > 0) return MLA_ERR_POS_RANGE;
    if (s->Dr > 2 * kMaxPairs || (int64_t)s->Dn + s->Dr > kMaxD || s->axes > 16) return MLA_ERR_UNSUPPORTED;
    for (int i = 0; i < s->Dr / 2; ++i)
        if (pair_axis[i] >= s->axes) return MLA_ERR_INVALID_ARG;
    if (!aligned(cos_tab, 4) || !aligned(sin_tab, 4) || !aligned(pos, 4) || !aligned(dev_status, 4))
        return MLA_ERR_ALIGNMENT;
    p->T = s->T;
    p->H = s->H;
    p->rows = s->T * s->H;
    p->Dn = s->Dn;
    p->Dr = s->Dr;
    p->cos_tab = cos_tab;
    p->sin_tab = sin_tab;
    p->cs_rows = s->cs_rows;
    p->cs_width = s->cs_width;
    p->pos = pos;
    p->status = const_cast<int*>(dev_status);
    for (int i = 0; i < s->Dr / 2; ++i) p->axis[i] = pair_axis[i];
    return MLA_OK;
}

// Bytes that rows of D elements at these strides span.
int64_t extent(int64_t T, int64_t st, int64_t H, int64_t sh, int64_t D, int64_t size) {
    return T == 0 ? 0 : ((T - 1) * st + (H - 1) * sh + D) * size;
}

}  // namespace
}  // namespace mlaq

using namespace mlaq;

extern "C" {

MLAQ_API int mla_rope_axes(const mla_rope_axes_shape* shape, int dtype, int mode, const void* in,
                           const float* cos_tab, const float* sin_tab, const int32_t* pos,
                           const uint8_t* pair_axis, void* out, int* dev_status, void* stream) {
    RopeParams p{};
    const int st = check_axes(shape, cos_tab, sin_tab, pos, pair_axis, dev_status, &p);
    if (st != MLA_OK) return st;
    const mla_rope_axes_shape& s = *shape;
    const bool sum = mode == MLA_ROPE_INVERSE_SUM;
    if ((dtype != MLA_IN_F32 && dtype != MLA_IN_BF16) || mode < MLA_ROPE_APPLY || mode > MLA_ROPE_INVERSE_SUM)
        return MLA_ERR_INVALID_ARG;
    if (s.T > 0 && (!in || !out)) return MLA_ERR_INVALID_ARG;
    const int64_t D = (int64_t)s.Dn + s.Dr;
    const int64_t Ho = sum ? 1 : s.H;
    if (!inside(s.T, s.in_t) || !inside(s.H, s.in_h) || !inside(s.T, s.out_t) || !inside(Ho, s.out_h))
        return MLA_ERR_INVALID_ARG;
    // no two output rows share an element: heads inside a token, or tokens inside a head
    const bool heads_in = (Ho == 1 || s.out_h >= D) && (s.T <= 1 || s.out_t >= (Ho - 1) * s.out_h + D);
    const bool tokens_in = (s.T <= 1 || s.out_t >= D) && (Ho == 1 || s.out_h >= (s.T - 1) * s.out_t + D);
    if (!heads_in && !tokens_in) return MLA_ERR_INVALID_ARG;
    const int64_t size = dtype == MLA_IN_F32 ? 4 : 2;
    if (!aligned(in, size) || !aligned(out, size)) return MLA_ERR_ALIGNMENT;
    const int64_t table = s.cs_rows * s.cs_width * 4;
    const Range outs[] = {rng(out, extent(s.T, s.out_t, Ho, s.out_h, D, size)), rng(dev_status, 4)};
    const Range ins[] = {rng(in, extent(s.T, s.in_t, s.H, s.in_h, D, size)), rng(cos_tab, table),
                         rng(sin_tab, table), rng(pos, (int64_t)s.axes * s.T * 4)};
    if (any_alias(outs, ins)) return MLA_ERR_ALIAS;
    if (s.T == 0) return MLA_OK;
    DeviceInfo di;
    const int ds = current_device_info(&di);
    if (ds != MLA_OK) return ds;
    p.in = in;
    p.out = out;
    p.in_t = s.in_t;
    p.in_h = s.in_h;
    p.out_t = s.out_t;
    p.out_h = s.out_h;
    p.inverse = mode != MLA_ROPE_APPLY;
    const int ve = (int)(16 / size);
    // 16-byte accesses: every row and both halves of every pair start on 16 bytes
    const bool vec = aligned(in, 16) && aligned(out, 16) && s.in_t % ve == 0 && s.in_h % ve == 0 &&
                     s.out_t % ve == 0 && s.out_h % ve == 0 && s.Dn % ve == 0 && s.Dr / 2 % ve == 0;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (dtype == MLA_IN_F32)
        return vec ? launch_rows<float, 4>(p, sum, di.num_sms, cs) : launch_rows<float, 1>(p, sum, di.num_sms, cs);
    return vec ? launch_rows<uint16_t, 8>(p, sum, di.num_sms, cs) : launch_rows<uint16_t, 1>(p, sum, di.num_sms, cs);
}

MLAQ_API int mla_rope_axes_table(const mla_rope_axes_shape* shape, const float* cos_tab, const float* sin_tab,
                                 const int32_t* pos, const uint8_t* pair_axis, float* cos_out, float* sin_out,
                                 int* dev_status, void* stream) {
    RopeParams p{};
    const int st = check_axes(shape, cos_tab, sin_tab, pos, pair_axis, dev_status, &p);
    if (st != MLA_OK) return st;
    const mla_rope_axes_shape& s = *shape;
    if (s.T > 0 && (!cos_out || !sin_out)) return MLA_ERR_INVALID_ARG;
    if (!aligned(cos_out, 16) || !aligned(sin_out, 16)) return MLA_ERR_ALIGNMENT;
    const int64_t table = s.cs_rows * s.cs_width * 4, bytes = s.T * s.Dr * 4;
    const Range outs[] = {rng(cos_out, bytes), rng(sin_out, bytes), rng(dev_status, 4)};
    const Range ins[] = {rng(cos_tab, table), rng(sin_tab, table), rng(pos, (int64_t)s.axes * s.T * 4)};
    if (any_alias(outs, ins)) return MLA_ERR_ALIAS;
    if (s.T == 0) return MLA_OK;
    DeviceInfo di;
    const int ds = current_device_info(&di);
    if (ds != MLA_OK) return ds;
    // tables read and written by float4
    const bool cs_vec = aligned(cos_tab, 16) && aligned(sin_tab, 16) && s.cs_width % 4 == 0 && s.Dr / 2 % 4 == 0;
    const int cols = cs_vec ? s.Dr / 4 : s.Dr;
    // tokens of a thread: one while that leaves SMs room, four once they come in several waves (see the kernel)
    const int64_t threads = s.T * cols;
    const int u = threads <= (int64_t)di.num_sms * 512 ? 1 : threads <= (int64_t)di.num_sms * 8192 ? 2 : 4;
    const int64_t run = (int64_t)(kThreads / cols) * u;
    const auto kernel = cs_vec ? (u == 1   ? rope_table_kernel<4, 1>
                                  : u == 2 ? rope_table_kernel<4, 2>
                                           : rope_table_kernel<4, 4>)
                               : (u == 1   ? rope_table_kernel<1, 1>
                                  : u == 2 ? rope_table_kernel<1, 2>
                                           : rope_table_kernel<1, 4>);
    return launch_overlapped(kernel, (unsigned)((s.T + run - 1) / run), kThreads, 0, 0, static_cast<cudaStream_t>(stream),
                             p, cos_out, sin_out);
}

}  // extern "C"

// RMS norm of token rows, with the residual's addition in front of it and an
// MXFP8 result for the block-scaled projections behind it:
//   h = x + r,  rstd = (mean_k h_k^2 + eps)^(-1/2),  y_k = h_k rstd w_k
// and its gradient, with g = dy w and the normed row n = h rstd,
//   dx = rstd (g - n mean_k(g_k n_k)) + dh,   dw = sum_t dy n.
// Sums are float32; y is made of the unrounded sum x + r, and each result is
// rounded once, at its store.
//
// All of it is bound by HBM once there is enough of it: a row is read once and
// stays in registers, eight channels to a granule (see Layout). A row belongs to a
// warp (no barrier; several rows in flight per block) or to a block; a thread's
// weights stay in its registers for all of its rows. In a graph, bf16 with the
// residual: 8192 x 7168 75.6 us (6.2 TB/s, 93% of a copy's rate), its gradient with
// dh 83 to 86 (by box; 5.6 TB/s); short calls are a launch and one row's chain of
// load, sum and store: 1 x 1536 as MXFP8 2.1 us, 4099 x 1536 8.3. A
// large MXFP8 call is bound by the rows that an SM's registers hold: 8192 x 7168 66
// us, of 26 for its bytes, with one block of 448 threads and 88 registers an SM (64
// registers and two blocks 65, packed products and these 64).
#include <cuda_runtime.h>

#include <cstdint>

#include "checks.h"
#include "internal.h"
#include "launch.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace mlaq {
namespace {

constexpr int kG = 8;                // channels of a granule
constexpr int64_t kMaxK = 32768;     // 512 threads of eight granules
constexpr int kWarpRows = 8;         // rows (warps) of a block that gives each row a warp

struct NormParams {
    const void *x, *res, *w;         // backward: h, dh, weight
    const void* dy;
    void *h, *y;                     // backward: y is dx
    uint8_t* scales;
    float* rstd;
    float* partials;                 // backward: [blocks][K]
    int64_t T, ld_x, ld_res, ld_dy;
    int K;
    int x_bf16, w_bf16, tiled;
    float eps, inv_k;
};

// Which channels are granule j of lane i. kWhole: the eight from (j * lanes + i) * 8,
// by 16-byte accesses, where rows start on 16 bytes. kSingle: the same, one by one
// (an MXFP8 block is four lanes' granules). kStrided: j * 8 * lanes + i and every
// lanes-th behind it, so that single accesses of a warp lie side by side (777 x 1001
// float32 gradient: 14.0 us with kSingle, so 10.6).
enum Layout { kWhole, kSingle, kStrided };

struct Lanes {
    int lane, lanes, K;
    template <Layout L>
    __device__ __forceinline__ int channel(int j, int i) const {
        return L == kStrided ? (j * kG + i) * lanes + lane : (j * lanes + lane) * kG + i;
    }
};

// Eight channels in registers, as they lie in memory; zeros behind the row's end.
template <typename E, Layout L>
struct Granule {
    uint32_t u[sizeof(E) == 2 ? 4 : 8];

    __device__ __forceinline__ void load(const E* row, const Lanes& l, int j) {
        if constexpr (L == kWhole) {
            zero();
            const int c = l.channel<L>(j, 0);
            if (c >= l.K) return;
            const uint4 a = *reinterpret_cast<const uint4*>(row + c);
            u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w;
            if constexpr (sizeof(E) == 4) {
                const uint4 b = *reinterpret_cast<const uint4*>(row + c + 4);
                u[4] = b.x, u[5] = b.y, u[6] = b.z, u[7] = b.w;
            }
        } else if constexpr (sizeof(E) == 2) {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = l.channel<L>(j, i);
                v[i] = c < l.K ? (uint32_t)row[c] : 0u;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = v[2 * i] | (v[2 * i + 1] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = l.channel<L>(j, i);
                u[i] = c < l.K ? __float_as_uint(row[c]) : 0u;
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (sizeof(E) == 2 ? 4 : 8); ++i) u[i] = 0u;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(E) == 4) return __uint_as_float(u[i]);
        else return i & 1 ? bf16hi_to_f32(u[i / 2]) : bf16lo_to_f32(u[i / 2]);
    }
    __device__ __forceinline__ void set(const float (&v)[kG]) {
#pragma unroll
        for (int i = 0; i < (sizeof(E) == 2 ? 4 : 8); ++i)
            u[i] = sizeof(E) == 2 ? pack_bf16x2(v[2 * i % kG], v[(2 * i + 1) % kG]) : __float_as_uint(v[i % kG]);
    }
    __device__ __forceinline__ void store(E* row, const Lanes& l, int j) const {
        if constexpr (L == kWhole) {
            const int c = l.channel<L>(j, 0);
            if (c >= l.K) return;
            st_global_v4(row + c, u[0], u[1], u[2], u[3]);
            if constexpr (sizeof(E) == 4) st_global_v4(row + c + 4, u[4], u[5], u[6], u[7]);
        } else {
#pragma unroll
            for (int i = 0; i < kG; ++i) {
                const int c = l.channel<L>(j, i);
                if (c < l.K) {
                    if constexpr (sizeof(E) == 2) row[c] = (uint16_t)(i & 1 ? u[i / 2] >> 16 : u[i / 2] & 0xFFFFu);
                    else row[c] = __uint_as_float(u[i]);
                }
            }
        }
    }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The sum over the threads of a row: a warp's, or (WARP false) the block's,
// through a buffer that alternates with the row so that one barrier is enough.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* buf, int turn) {
    v = warp_sum(v);
    if constexpr (WARP) return v;
    float* b = buf + (turn & 1) * 32;
    const int warps = blockDim.x / 32;
    if (threadIdx.x % 32 == 0) b[threadIdx.x / 32] = v;
    __syncthreads();
    const int lane = threadIdx.x % 32;
    return warp_sum(lane < warps ? b[lane] : 0.f);  // every warp the same sum, in the same order
}

// The weights of a granule, as 32-bit values.
template <Layout L>
__device__ __forceinline__ void load_weights(const NormParams& p, const Lanes& l, int j, float (&w)[kG]) {
    if (p.w_bf16) {
        Granule<uint16_t, L> g;
        g.load(static_cast<const uint16_t*>(p.w), l, j);
#pragma unroll
        for (int i = 0; i < kG; ++i) w[i] = g.get(i);
    } else {
        Granule<float, L> g;
        g.load(static_cast<const float*>(p.w), l, j);
#pragma unroll
        for (int i = 0; i < kG; ++i) w[i] = g.get(i);
    }
}

// Threads of a block at most: with more than one granule each, half as many and twice the registers.
template <bool WARP, int GPT>
constexpr int kMaxThreads = WARP ? 32 * kWarpRows : GPT == 1 ? 1024 : 512;

// E: x, r, h and y (bf16 as uint16_t, or float). GPT granules per thread. MX:
// y as E4M3 codes with a scale for each 32 channels, four granules that lie
// side by side in four lanes.
template <typename E, int GPT, bool MX, Layout L, bool WARP>
__global__ void __launch_bounds__(kMaxThreads<WARP, GPT>) rms_norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ float buf[64];
    grid_launch_next();
    grid_wait_previous();
    const Lanes l{WARP ? (int)threadIdx.x % 32 : (int)threadIdx.x, WARP ? 32 : (int)blockDim.x, p.K};
    const int rows = WARP ? kWarpRows : 1;
    const int64_t step = (int64_t)gridDim.x * rows;
    const E* x = static_cast<const E*>(p.x);
    const E* res = static_cast<const E*>(p.res);
    constexpr bool kHold = GPT <= 4;   // weights stay in registers; else each row reads them again
    constexpr bool kAhead = GPT <= 2;  // the next row is on its way while this one is worked on
    float w[kHold ? GPT : 1][kG];
    if constexpr (kHold) {
#pragma unroll
        for (int j = 0; j < GPT; ++j) load_weights<L>(p, l, j, w[j]);
    }
    // tiled scales: the last 128-row tile's missing rows get scale bytes of zero
    const int64_t end = MX && p.tiled ? (p.T + 127) / 128 * 128 : p.T;
    const int64_t nkt = (p.K / 32 + 3) / 4;
    Granule<E, L> raw[GPT], add[GPT], raw2[kAhead ? GPT : 1], add2[kAhead ? GPT : 1];
    int64_t t = (int64_t)blockIdx.x * rows + (WARP ? threadIdx.x / 32 : 0);
    auto fetch = [&](int64_t t, auto& a, auto& b) {
#pragma unroll
        for (int j = 0; j < GPT; ++j) {
            a[j].zero();
            b[j].zero();
            if (t < p.T) {
                a[j].load(x + t * p.ld_x, l, j);
                if (res) b[j].load(res + t * p.ld_res, l, j);
            }
        }
    };
    if constexpr (kAhead) fetch(t, raw2, add2);
    int turn = 0;
    for (; t < end; t += step, ++turn) {
        if (MX && t >= p.T) {  // uniform over the row's threads
            for (int c = l.lane; c < nkt * 4; c += l.lanes) p.scales[sf_tiled_offset(t, c, 128, nkt)] = 0;
            continue;
        }
        if constexpr (kAhead) {
#pragma unroll
            for (int j = 0; j < GPT; ++j) raw[j] = raw2[j], add[j] = add2[j];
            fetch(t + step, raw2, add2);
        } else {
            fetch(t, raw, add);
        }
        float v[GPT][kG], sum = 0.f;
#pragma unroll
        for (int j = 0; j < GPT; ++j) {
#pragma unroll
            for (int i = 0; i < kG; ++i) v[j][i] = raw[j].get(i);
            if (res) {
#pragma unroll
                for (int i = 0; i < kG; ++i) v[j][i] += add[j].get(i);
            }
#pragma unroll
            for (int i = 0; i < kG; ++i) sum = fmaf(v[j][i], v[j][i], sum);
            if (res) {
                raw[j].set(v[j]);
                raw[j].store(static_cast<E*>(p.h) + t * p.K, l, j);
            }
        }
        const float rstd = __frsqrt_rn(fmaf(row_sum<WARP>(sum, buf, turn), p.inv_k, p.eps));
        if (p.rstd && l.lane == 0) p.rstd[t] = rstd;
        uint8_t* row_scales = MX && p.tiled ? p.scales + sf_tiled_offset(t, 0, 128, nkt) : nullptr;
#pragma unroll
        for (int j = 0; j < GPT; ++j) {
            if constexpr (!kHold) load_weights<L>(p, l, j, w[0]);
#pragma unroll
            for (int i = 0; i < kG; ++i) v[j][i] = v[j][i] * rstd * w[kHold ? j : 0][i];
            if constexpr (MX) {
                const int c = l.channel<L>(j, 0);
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < kG; ++i) {
                    m = max(m, __float_as_uint(v[j][i]) & 0x7FFFFFFFu);  // a block's four lanes are inside K or behind it
                }
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
                uint32_t codes[2];
                const uint32_t s = quantize8_block_scale(v[j], m, codes);
                if (c < p.K) {
                    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + t * p.K + c) = make_uint2(codes[0], codes[1]);
                    if (l.lane % 4 == 0) {
                        if (p.tiled) row_scales[(c >> 7) * 512 + ((c >> 5) & 3)] = (uint8_t)s;  // as sf_tiled_offset
                        else p.scales[t * (p.K / 32) + c / 32] = (uint8_t)s;
                    }
                }
            } else {
                Granule<E, L> o;
                o.set(v[j]);
                o.store(static_cast<E*>(p.y) + t * p.K, l, j);
            }
        }
        if (MX && p.tiled)  // and so the last tile's missing columns
            for (int c = p.K / 32 + l.lane; c < nkt * 4; c += l.lanes) p.scales[sf_tiled_offset(t, c, 128, nkt)] = 0;
    }
}

// The gradient. dw's sum over the rows stays in the threads' registers; each
// block adds its rows' in a fixed order and leaves one partial row.
template <typename E, int GPT, Layout L, bool WARP>
__global__ void __launch_bounds__(kMaxThreads<WARP, GPT>) rms_norm_bwd_kernel(const __grid_constant__ NormParams p) {
    extern __shared__ float4 dyn[];
    __shared__ float buf[64];
    grid_launch_next();
    grid_wait_previous();
    const Lanes l{WARP ? (int)threadIdx.x % 32 : (int)threadIdx.x, WARP ? 32 : (int)blockDim.x, p.K};
    const int rows = WARP ? kWarpRows : 1;
    const int64_t step = (int64_t)gridDim.x * rows;
    const E* h = static_cast<const E*>(p.x);
    const E* dh = static_cast<const E*>(p.res);
    const E* dy = static_cast<const E*>(p.dy);
    constexpr bool kHold = GPT <= 4;
    float w[kHold ? GPT : 1][kG], dw[GPT][kG];
#pragma unroll
    for (int j = 0; j < GPT; ++j) {
#pragma unroll
        for (int i = 0; i < kG; ++i) dw[j][i] = 0.f;
        if constexpr (kHold) load_weights<L>(p, l, j, w[j]);
    }
    int turn = 0;
    for (int64_t t = (int64_t)blockIdx.x * rows + (WARP ? threadIdx.x / 32 : 0); t < p.T; t += step, ++turn) {
        Granule<E, L> a[GPT], b[GPT], d[GPT];
#pragma unroll
        for (int j = 0; j < GPT; ++j) {
            a[j].load(dy + t * p.ld_dy, l, j);
            b[j].load(h + t * p.ld_x, l, j);
        }
        if (dh) {
#pragma unroll
            for (int j = 0; j < GPT; ++j) d[j].load(dh + t * p.ld_res, l, j);
        }
        const float rstd = p.rstd[t];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < GPT; ++j) {
            if constexpr (!kHold) load_weights<L>(p, l, j, w[0]);
#pragma unroll
            for (int i = 0; i < kG; ++i) {
                const float n = b[j].get(i) * rstd, e = a[j].get(i);
                sum = fmaf(e * w[kHold ? j : 0][i], n, sum);
                dw[j][i] = fmaf(e, n, dw[j][i]);
            }
        }
        if (!p.y) continue;
        const float mean = row_sum<WARP>(sum, buf, turn) * p.inv_k;
#pragma unroll
        for (int j = 0; j < GPT; ++j) {
            if constexpr (!kHold) load_weights<L>(p, l, j, w[0]);
            float o[kG];
#pragma unroll
            for (int i = 0; i < kG; ++i) {
                const float n = b[j].get(i) * rstd;
                o[i] = rstd * fmaf(-n, mean, a[j].get(i) * w[kHold ? j : 0][i]) + (dh ? d[j].get(i) : 0.f);
            }
            a[j].set(o);
            a[j].store(static_cast<E*>(p.y) + t * p.K, l, j);
        }
    }
    if (!p.partials) return;
    float* out = p.partials + (int64_t)blockIdx.x * p.K;
    float* part = WARP ? reinterpret_cast<float*>(dyn) + (threadIdx.x / 32) * p.K : out;
#pragma unroll
    for (int j = 0; j < GPT; ++j)
#pragma unroll
        for (int i = 0; i < kG; ++i) {
            const int c = l.channel<L>(j, i);
            if (c < p.K) part[c] = dw[j][i];
        }
    if constexpr (WARP) {  // the warps' sums through shared memory, [warp][K]
        __syncthreads();
        part = reinterpret_cast<float*>(dyn);
        for (int c = threadIdx.x; c < p.K; c += blockDim.x) {
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < kWarpRows; ++r) s += part[r * p.K + c];
            out[c] = s;
        }
    }
}

// The gradient of wide rows that start on 16 bytes. Rows come by asynchronous
// copies into a ring of shared memory, several ahead of the one that is worked on:
// with the loads in registers a block had one row in flight and waited for it (8192
// x 7168 with dh: 138 us, so 85 us). A thread copies the granules that it reads
// itself, so it waits for its own copies and for no barrier. (By bulk copies and
// barriers: 85 us as well, without dh 80 for 75, in float32 5% less.)
constexpr int kMaxStages = 8, kRingGranules = 2;  // granules of a thread: norm_grid's for a block to a row of more rows than SMs
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// Until all groups of copies but the youngest n are there.
__device__ __forceinline__ void copies_wait(int n) {
    static_assert(kMaxStages == 8, "a case for each number of stages");
    switch (n) {
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
        case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
        case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
        case 7: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
}
template <typename E>
__global__ void __launch_bounds__(512) rms_norm_bwd_ring_kernel(const __grid_constant__ NormParams p, int stages, int pitch) {
    constexpr int GPT = kRingGranules;
    extern __shared__ __align__(128) uint8_t ring[];  // [stage][dy | h | dh], rows of `pitch` bytes
    __shared__ float buf[64];
    const int tid = threadIdx.x, parts = p.res ? 3 : 2;
    const uint32_t ring0 = smem_u32(ring);
    grid_launch_next();
    grid_wait_previous();
    const int64_t step = gridDim.x;
    const Lanes l{tid, (int)blockDim.x, p.K};
    // this thread's granules of row t into stage s: a group of copies, empty behind the last row
    auto load = [&](int64_t t, int s) {
        if (t < p.T) {
            const E* rows[3] = {static_cast<const E*>(p.dy) + t * p.ld_dy, static_cast<const E*>(p.x) + t * p.ld_x,
                                static_cast<const E*>(p.res) + t * p.ld_res};
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                if (k == 2 && !p.res) break;
                const uint32_t to = ring0 + (s * parts + k) * pitch;
#pragma unroll
                for (int j = 0; j < GPT; ++j) {
                    const int c = l.channel<kWhole>(j, 0);
                    if (c >= p.K) continue;
#pragma unroll
                    for (int i = 0; i < kG; i += 16 / (int)sizeof(E)) copy16(to + (c + i) * (int)sizeof(E), rows[k] + c + i);
                }
            }
        }
        cp_async_commit();
    };
    for (int s = 0; s < stages; ++s) load(blockIdx.x + s * step, s);
    float w[GPT][kG], dw[GPT][kG];
#pragma unroll
    for (int j = 0; j < GPT; ++j) {
#pragma unroll
        for (int i = 0; i < kG; ++i) dw[j][i] = 0.f;
        load_weights<kWhole>(p, l, j, w[j]);
    }
    int turn = 0, s = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += step, ++turn) {
        copies_wait(stages - 1);
        const float rstd = p.rstd[t];
        const uint8_t* row = ring + s * parts * pitch;
        Granule<E, kWhole> a[GPT], b[GPT], d[GPT];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < GPT; ++j) {
            a[j].load(reinterpret_cast<const E*>(row), l, j);
            b[j].load(reinterpret_cast<const E*>(row + pitch), l, j);
            if (p.res) d[j].load(reinterpret_cast<const E*>(row + 2 * pitch), l, j);
#pragma unroll
            for (int i = 0; i < kG; ++i) {
                const float n = b[j].get(i) * rstd, e = a[j].get(i);
                sum = fmaf(e * w[j][i], n, sum);
                dw[j][i] = fmaf(e, n, dw[j][i]);
            }
        }
        load(t + stages * step, s);  // what lay there is in this thread's registers, and no other thread's
        if (++s == stages) s = 0;
        const float mean = row_sum<false>(sum, buf, turn) * p.inv_k;
        if (!p.y) continue;
#pragma unroll
        for (int j = 0; j < GPT; ++j) {
            float o[kG];
#pragma unroll
            for (int i = 0; i < kG; ++i) {
                const float n = b[j].get(i) * rstd;
                o[i] = rstd * fmaf(-n, mean, a[j].get(i) * w[j][i]) + (p.res ? d[j].get(i) : 0.f);
            }
            a[j].set(o);
            a[j].store(static_cast<E*>(p.y) + t * p.K, l, j);
        }
    }
    if (!p.partials) return;
    float* out = p.partials + (int64_t)blockIdx.x * p.K;
#pragma unroll
    for (int j = 0; j < GPT; ++j) {
        const int c = l.channel<kWhole>(j, 0);
        if (c >= p.K) continue;
#pragma unroll
        for (int i = 0; i < kG; i += 4) *reinterpret_cast<float4*>(out + c + i) = make_float4(dw[j][i], dw[j][i + 1], dw[j][i + 2], dw[j][i + 3]);
    }
}

// dw from the blocks' partial rows: 32 columns to a block, 32 threads to a
// column, each a fixed share of the rows.
constexpr int kDwShares = 32;
__global__ void __launch_bounds__(32 * kDwShares) rms_norm_dw_kernel(const float* partials, int parts, int K, int w_bf16, void* dw) {
    __shared__ float sums[kDwShares][33];
    grid_launch_next();
    grid_wait_previous();
    const int c = blockIdx.x * 32 + threadIdx.x % 32, r = threadIdx.x / 32;
    float s = 0.f;
    if (c < K) {
#pragma unroll 8
        for (int i = r; i < parts; i += kDwShares) s += partials[(int64_t)i * K + c];
    }
    sums[r][threadIdx.x % 32] = s;
    __syncthreads();
    s = warp_sum(sums[threadIdx.x % 32][r]);  // column r of the block's, in a fixed order
    const int k = blockIdx.x * 32 + r;
    if (threadIdx.x % 32 == 0 && k < K) {
        if (w_bf16) static_cast<uint16_t*>(dw)[k] = (uint16_t)pack_bf16x2(s, 0.f);
        else static_cast<float*>(dw)[k] = s;
    }
}

struct NormGrid {
    bool warp;      // a warp to a row
    int gpt;        // granules per thread
    unsigned threads, blocks;
};

// How rows are shared out. Up to 32 granules a warp to a row; up to 128 also, of
// as many granules per lane as it takes, in the gradient, whose sum would be a
// barrier for each row (300 x 1024: 5.0 us, by blocks 6.1; 8192 x 512: 8.9, by
// blocks 17.0), and forward where the rows fill the SMs (8192 x 1024: 10.4 us, by
// blocks 11.0; but 300 x 1024: 2.5, by blocks 1.9). Else a block to a row: one
// granule per thread for up to 128, or while there are fewer rows than SMs (128 x
// 7168: 2.6 us, with two 3.1), then two (8192 x 7168: 75.6 us, with one 102.6; 8192
// x 2048: 20.9, with one 24.7; its gradient 27.2, with one 32.0), and four or eight
// where the block would pass 512 threads.
NormGrid norm_grid(int64_t T, int64_t K, int num_sms, bool bwd, bool mx = false) {
    const int64_t granules = (K + kG - 1) / kG;
    NormGrid g{};
    if (granules <= 32 || (granules <= 128 && (bwd || T >= (int64_t)num_sms * kWarpRows))) {
        g.warp = true;
        g.gpt = granules <= 32 ? 1 : granules <= 64 ? 2 : 4;
        g.threads = 32 * kWarpRows;
        const int64_t need = (T + kWarpRows - 1) / kWarpRows, room = (int64_t)num_sms * (bwd ? 2 : 4);
        g.blocks = (unsigned)(need < room ? need : room);
        return g;
    }
    g.gpt = granules <= 1024 && (T < num_sms || granules <= 128) ? 1 : granules <= 1024 ? 2 : granules <= 2048 ? 4 : 8;
    g.threads = (unsigned)((granules + 32 * g.gpt - 1) / (32 * g.gpt) * 32);
    // Blocks to an SM: as its threads allow; MXFP8 with more than one granule as its registers do (88 a thread), so that a
    // block goes on to its next row, already on its way, instead of others' first ones (8192 x 1536: 14.1 us, else 15.7;
    // 8192 x 7168: 66.4, else 69.5). Results in x's type want the threads (8192 x 1536: 15.2, with fewer 20.0).
    const int fill = mx && g.gpt > 1 ? 640 : 2048, per = fill / (int)g.threads < 1 ? 1 : fill / (int)g.threads;
    const int64_t room = (int64_t)num_sms * (bwd ? (per > 4 ? 4 : per) : per);
    g.blocks = (unsigned)(T < room ? T : room);
    return g;
}

template <typename E, bool MX, Layout L>
int launch_fwd_rows(const NormParams& p, const NormGrid& g, cudaStream_t s) {
    const auto kernel = g.warp ? (g.gpt == 1   ? rms_norm_kernel<E, 1, MX, L, true>
                                  : g.gpt == 2 ? rms_norm_kernel<E, 2, MX, L, true>
                                               : rms_norm_kernel<E, 4, MX, L, true>)
                               : (g.gpt == 1   ? rms_norm_kernel<E, 1, MX, L, false>
                                  : g.gpt == 2 ? rms_norm_kernel<E, 2, MX, L, false>
                                  : g.gpt == 4 ? rms_norm_kernel<E, 4, MX, L, false>
                                               : rms_norm_kernel<E, 8, MX, L, false>);
    return launch_overlapped(kernel, g.blocks, g.threads, 0, 0, s, p);
}

// The ring of rows for a block-to-a-row backward of more rows than SMs: as many
// blocks to an SM as keep it busy (a row of 48 KB, read and written, takes longer
// to come than to work on; a shorter one wants others beside it), the rest of
// shared memory for rows ahead.
struct NormRing {
    int stages, pitch;  // stages 0: not this way
    unsigned blocks;
    size_t smem;
};
NormRing norm_ring(const NormParams& p, const NormGrid& g, int64_t size, const DeviceInfo& di) {
    NormRing r{};
    const int64_t row = p.K * size, parts = p.res ? 3 : 2;
    if (g.warp || g.gpt != kRingGranules || g.threads > 512 || p.T < 4 * (int64_t)di.num_sms) return r;
    const int per = 4 * row >= 48 * 1024 ? 1 : 4 * row >= 24 * 1024 ? 2 : 4;  // with dh or without: dw's sum is the same
    r.pitch = (int)((row + 127) / 128 * 128);
    const int64_t room = ((int64_t)di.max_smem_optin / per - 2048) / (parts * r.pitch);
    if (room < 2) return r;
    r.stages = (int)(room > kMaxStages ? kMaxStages : room);
    r.smem = (size_t)r.stages * parts * r.pitch;
    const int64_t blocks = (int64_t)di.num_sms * per;
    r.blocks = (unsigned)(blocks < g.blocks ? blocks : g.blocks);  // no more than the workspace is for
    return r;
}

template <typename E>
int launch_bwd_ring(const NormParams& p, const NormGrid& g, const NormRing& r, cudaStream_t s) {
    const auto kernel = rms_norm_bwd_ring_kernel<E>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)r.smem) != cudaSuccess) return MLA_ERR_CUDA;
    return launch_overlapped(kernel, r.blocks, g.threads, r.smem, 0, s, p, r.stages, r.pitch);
}

template <typename E, Layout L>
int launch_bwd_rows(const NormParams& p, const NormGrid& g, cudaStream_t s) {
    const auto kernel = g.warp ? (g.gpt == 1   ? rms_norm_bwd_kernel<E, 1, L, true>
                                  : g.gpt == 2 ? rms_norm_bwd_kernel<E, 2, L, true>
                                               : rms_norm_bwd_kernel<E, 4, L, true>)
                               : (g.gpt == 1   ? rms_norm_bwd_kernel<E, 1, L, false>
                                  : g.gpt == 2 ? rms_norm_bwd_kernel<E, 2, L, false>
                                  : g.gpt == 4 ? rms_norm_bwd_kernel<E, 4, L, false>
                                               : rms_norm_bwd_kernel<E, 8, L, false>);
    const size_t smem = g.warp && p.partials ? (size_t)kWarpRows * p.K * sizeof(float) : 0;
    return launch_overlapped(kernel, g.blocks, g.threads, smem, 0, s, p);
}

// What forward and backward check alike; *p gets the sizes.
int check_norm(const mla_norm_shape* s, NormParams* p) {
    if (!s) return MLA_ERR_INVALID_ARG;
    if (s->T < 0 || s->K <= 0 || s->T > kI32Max || s->K > kI32Max || s->reserved != 0) return MLA_ERR_INVALID_ARG;
    if ((s->dtype != MLA_IN_F32 && s->dtype != MLA_IN_BF16) || (s->w_dtype != MLA_IN_F32 && s->w_dtype != MLA_IN_BF16))
        return MLA_ERR_INVALID_ARG;
    if (!(s->eps >= 0.f) || s->eps > 3.402823466e38f) return MLA_ERR_INVALID_ARG;
    for (const int64_t ld : {s->ld_x, s->ld_res, s->ld_dy})
        if (ld != 0 && (ld < s->K || !inside(s->T, ld))) return MLA_ERR_INVALID_ARG;
    p->T = s->T;
    p->K = (int)s->K;
    p->ld_x = s->ld_x ? s->ld_x : s->K;
    p->ld_res = s->ld_res ? s->ld_res : s->K;
    p->ld_dy = s->ld_dy ? s->ld_dy : s->K;
    p->x_bf16 = s->dtype == MLA_IN_BF16;
    p->w_bf16 = s->w_dtype == MLA_IN_BF16;
    p->eps = s->eps;
    p->inv_k = 1.f / (float)s->K;
    if (s->K > kMaxK) return MLA_ERR_UNSUPPORTED;
    return MLA_OK;
}

int64_t span(int64_t T, int64_t ld, int64_t K, int64_t size) { return T > 0 ? ((T - 1) * ld + K) * size : 0; }

}  // namespace
}  // namespace mlaq

using namespace mlaq;

extern "C" {

MLAQ_API int mla_rms_norm_fwd(const mla_norm_shape* shape, const void* x, const void* residual, const void* weight,
                              void* h, void* y, uint8_t* y_scales, float* rstd, void* stream) {
    NormParams p{};
    const int st = check_norm(shape, &p);
    if (st != MLA_OK && st != MLA_ERR_UNSUPPORTED) return st;
    const mla_norm_shape& s = *shape;
    if (s.out_mode < MLA_NORM_OUT_SAME || s.out_mode > MLA_NORM_OUT_MXFP8_TILED) return MLA_ERR_INVALID_ARG;
    const bool mx = s.out_mode != MLA_NORM_OUT_SAME;
    if ((residual != nullptr) != (h != nullptr) || mx != (y_scales != nullptr) || !weight) {
        if (s.T > 0 || !weight) return MLA_ERR_INVALID_ARG;
    }
    if (s.T > 0 && (!x || !y)) return MLA_ERR_INVALID_ARG;
    if (mx && s.K % 32 != 0) return MLA_ERR_UNSUPPORTED;
    if (st != MLA_OK) return st;
    const int64_t size = p.x_bf16 ? 2 : 4, wsize = p.w_bf16 ? 2 : 4, n = s.T * s.K;
    if (!aligned(x, size) || !aligned(residual, size) || !aligned(h, size) || !aligned(weight, wsize) ||
        !aligned(rstd, 4) || !aligned(y, mx ? 8 : size))
        return MLA_ERR_ALIGNMENT;
    const bool tiled = s.out_mode == MLA_NORM_OUT_MXFP8_TILED;
    const int64_t marks = tiled ? sf_tiled_bytes(s.T, s.K / 32, 128) : n / 32;
    const Range outs[] = {rng(h, n * size), rng(y, mx ? n : n * size), rng(y_scales, marks), rng(rstd, s.T * 4)};
    const Range ins[] = {rng(x, span(s.T, p.ld_x, s.K, size)), rng(residual, span(s.T, p.ld_res, s.K, size)),
                         rng(weight, s.K * wsize)};
    if (any_alias(outs, ins)) return MLA_ERR_ALIAS;
    if (s.T == 0) return MLA_OK;
    DeviceInfo di;
    const int ds = current_device_info(&di);
    if (ds != MLA_OK) return ds;
    p.x = x, p.res = residual, p.w = weight, p.h = h, p.y = y, p.scales = y_scales, p.rstd = rstd, p.tiled = tiled;
    const int64_t ve = 16 / size;
    const bool vec = s.K % kG == 0 && aligned(x, 16) && aligned(residual, 16) && aligned(weight, 16) &&
                     aligned(h, 16) && (mx || aligned(y, 16)) && p.ld_x % ve == 0 && p.ld_res % ve == 0;
    const NormGrid g = norm_grid(s.T, s.K, di.num_sms, false, mx);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (p.x_bf16)
        return mx ? (vec ? launch_fwd_rows<uint16_t, true, kWhole>(p, g, cs) : launch_fwd_rows<uint16_t, true, kSingle>(p, g, cs))
                  : (vec ? launch_fwd_rows<uint16_t, false, kWhole>(p, g, cs) : launch_fwd_rows<uint16_t, false, kStrided>(p, g, cs));
    return mx ? (vec ? launch_fwd_rows<float, true, kWhole>(p, g, cs) : launch_fwd_rows<float, true, kSingle>(p, g, cs))
              : (vec ? launch_fwd_rows<float, false, kWhole>(p, g, cs) : launch_fwd_rows<float, false, kStrided>(p, g, cs));
}

MLAQ_API size_t mla_rms_norm_bwd_workspace_size(const mla_norm_shape* shape) {
    NormParams p{};
    DeviceInfo di;
    if (check_norm(shape, &p) != MLA_OK || current_device_info(&di) != MLA_OK) return 0;
    return (size_t)norm_grid(p.T, p.K, di.num_sms, true).blocks * p.K * sizeof(float);
}

MLAQ_API int mla_rms_norm_bwd(const mla_norm_shape* shape, const void* dy, const void* h, const void* weight,
                              const float* rstd, const void* dh, void* dx, void* dw, void* workspace, size_t ws_bytes,
                              void* stream) {
    NormParams p{};
    const int st = check_norm(shape, &p);
    if (st != MLA_OK && st != MLA_ERR_UNSUPPORTED) return st;
    const mla_norm_shape& s = *shape;
    if (s.out_mode != MLA_NORM_OUT_SAME || (!dx && !dw) || !weight || (dh && !dx)) return MLA_ERR_INVALID_ARG;
    if (s.T > 0 && (!dy || !h || !rstd)) return MLA_ERR_INVALID_ARG;
    if (st != MLA_OK) return st;
    const int64_t size = p.x_bf16 ? 2 : 4, wsize = p.w_bf16 ? 2 : 4, n = s.T * s.K;
    if (!aligned(dy, size) || !aligned(h, size) || !aligned(dh, size) || !aligned(dx, size) || !aligned(weight, wsize) ||
        !aligned(dw, wsize) || !aligned(rstd, 4) || !aligned(workspace, 16))
        return MLA_ERR_ALIGNMENT;
    const Range outs[] = {rng(dx, n * size), rng(dw, s.K * wsize), rng(workspace, (int64_t)ws_bytes)};
    const Range ins[] = {rng(dy, span(s.T, p.ld_dy, s.K, size)), rng(h, span(s.T, p.ld_x, s.K, size)),
                         rng(dh, span(s.T, p.ld_res, s.K, size)), rng(weight, s.K * wsize), rng(rstd, s.T * 4)};
    if (any_alias(outs, ins)) return MLA_ERR_ALIAS;
    if (s.T == 0 && !dw) return MLA_OK;
    DeviceInfo di;
    const int ds = current_device_info(&di);
    if (ds != MLA_OK) return ds;
    const NormGrid g = norm_grid(s.T, s.K, di.num_sms, true);
    if (dw && (ws_bytes < (size_t)g.blocks * s.K * sizeof(float) || (g.blocks > 0 && !workspace))) return MLA_ERR_WORKSPACE;
    p.x = h, p.res = dh, p.w = weight, p.dy = dy, p.y = dx, p.rstd = const_cast<float*>(rstd);
    p.partials = dw ? static_cast<float*>(workspace) : nullptr;
    const int64_t ve = 16 / size;
    const bool vec = s.K % kG == 0 && aligned(dy, 16) && aligned(h, 16) && aligned(dh, 16) && aligned(weight, 16) &&
                     aligned(dx, 16) && p.ld_x % ve == 0 && p.ld_res % ve == 0 && p.ld_dy % ve == 0;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const NormRing ring = vec ? norm_ring(p, g, size, di) : NormRing{};
    int parts = (int)g.blocks;
    if (s.T > 0 && ring.stages > 0) {
        const int r = p.x_bf16 ? launch_bwd_ring<uint16_t>(p, g, ring, cs) : launch_bwd_ring<float>(p, g, ring, cs);
        if (r != MLA_OK) return r;
        parts = (int)ring.blocks;
    } else if (s.T > 0) {
        const int r = p.x_bf16 ? (vec ? launch_bwd_rows<uint16_t, kWhole>(p, g, cs) : launch_bwd_rows<uint16_t, kStrided>(p, g, cs))
                               : (vec ? launch_bwd_rows<float, kWhole>(p, g, cs) : launch_bwd_rows<float, kStrided>(p, g, cs));
        if (r != MLA_OK) return r;
    }
    if (!dw) return MLA_OK;
    return launch_overlapped(rms_norm_dw_kernel, (unsigned)((s.K + 31) / 32), 32 * kDwShares, 0, 0, cs, p.partials, parts,
                             p.K, p.w_bf16, dw);
}

}  // extern "C"

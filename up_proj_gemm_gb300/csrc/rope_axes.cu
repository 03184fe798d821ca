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
#include "mx.cuh"
#include "ptx.cuh"

namespace mlaq {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;        // rows in flight per thread
constexpr int kMaxPairs = 128;    // Dr <= 256
constexpr int64_t kMaxD = 8192;   // the sum kernel's shared sums: at most 32 KB

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
    int cs_vec;                   // tables read by float4
    const int32_t* pos;           // [axes][T]
    int* status;
    int rows_per_block;
    uint8_t axis[kMaxPairs];
};

template <typename E>
struct Elem;
template <>
struct Elem<float> {
    static __device__ float up(float v) { return v; }
    static __device__ float down(float v) { return v; }
};
template <>
struct Elem<uint16_t> {
    static __device__ float up(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ uint16_t down(float v) { return (uint16_t)pack_bf16x2(v, 0.f); }
};

// VE elements at p (16 bytes together when VE > 1) as float32.
template <typename E, int VE>
__device__ __forceinline__ void load_vec(const E* p, float (&v)[VE]) {
    if constexpr (VE == 1) {
        v[0] = Elem<E>::up(*p);
    } else {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (VE == 4) {
                v[i] = __uint_as_float(u[i]);
            } else {
                v[2 * i] = bf16lo_to_f32(u[i]);
                v[2 * i + 1] = bf16hi_to_f32(u[i]);
            }
        }
    }
}

template <typename E, int VE>
__device__ __forceinline__ void store_vec(E* p, const float (&v)[VE]) {
    if constexpr (VE == 1) {
        *p = Elem<E>::down(v[0]);
    } else if constexpr (VE == 4) {
        st_global_v4(p, __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    } else {
        st_global_v4(p, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                     pack_bf16x2(v[6], v[7]));
    }
}

// The table entries of the VE pairs from i0 on, for token t: c0/s0 of the
// low channels, c1/s1 of the high ones. A position outside the table is
// reported and its entries are 0.
template <int VE>
struct Turn {
    float c0[VE], s0[VE], c1[VE], s1[VE];

    __device__ __forceinline__ void load(const RopeParams& p, int i0, bool one_axis, int64_t t) {
        const int h = p.Dr / 2;
        if (VE > 1 && one_axis && p.cs_vec) {  // the pairs share an axis, so a row: read it by float4
            const int64_t row = __ldg(p.pos + p.axis[i0] * p.T + t);
            const bool ok = row >= 0 && row < p.cs_rows;
            if (!ok) record_status(p.status, MLA_ERR_POS_RANGE);
            const int64_t at = (ok ? row : 0) * p.cs_width + i0;
#pragma unroll
            for (int k = 0; k + 4 <= VE; k += 4) {
                four(p.cos_tab + at + k, ok, c0 + k);
                four(p.sin_tab + at + k, ok, s0 + k);
                four(p.cos_tab + at + h + k, ok, c1 + k);
                four(p.sin_tab + at + h + k, ok, s1 + k);
            }
            return;
        }
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            const int64_t row = __ldg(p.pos + p.axis[i0 + k] * p.T + t);
            const bool ok = row >= 0 && row < p.cs_rows;
            if (!ok) record_status(p.status, MLA_ERR_POS_RANGE);
            const int64_t at = (ok ? row : 0) * p.cs_width + i0 + k;
            c0[k] = ok ? __ldg(p.cos_tab + at) : 0.f;
            s0[k] = ok ? __ldg(p.sin_tab + at) : 0.f;
            c1[k] = ok ? __ldg(p.cos_tab + at + h) : 0.f;
            s1[k] = ok ? __ldg(p.sin_tab + at + h) : 0.f;
        }
    }

    __device__ __forceinline__ void turn(bool inverse, float (&a)[VE], float (&b)[VE]) const {
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            const float x = a[k], y = b[k];
            a[k] = inverse ? x * c0[k] + y * s1[k] : x * c0[k] - y * s0[k];
            b[k] = inverse ? y * c1[k] - x * s0[k] : y * c1[k] + x * s1[k];
        }
    }

private:
    static __device__ __forceinline__ void four(const float* q, bool ok, float* d) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(q));
        d[0] = ok ? f.x : 0.f;
        d[1] = ok ? f.y : 0.f;
        d[2] = ok ? f.z : 0.f;
        d[3] = ok ? f.w : 0.f;
    }
};

template <int VE>
__device__ __forceinline__ bool same_axis(const RopeParams& p, int i0) {
    bool same = true;
#pragma unroll
    for (int k = 1; k < VE; ++k) same &= p.axis[i0 + k] == p.axis[i0];
    return same;
}

// apply and inverse. A thread owns one slot of a (token, head) row, two
// vectors of VE elements: a pair vector (channels i.. and i+h..), or two
// vectors of the pass-through channels. It walks the rows of its block, four
// in flight, and reloads the table entries only when the token changes.
template <typename E, int VE>
__global__ void __launch_bounds__(kThreads) rope_axes_kernel(const __grid_constant__ RopeParams p) {
    const int half = p.Dr / 2;
    const int n_pair = half / VE, n_copy = p.Dn / VE;
    const int n_copy2 = (n_copy + 1) / 2;
    const int slots = n_copy2 + n_pair;
    const int lanes = kThreads / slots > 0 ? kThreads / slots : 1;  // rows walked side by side
    const int lane = threadIdx.x / slots;
    if (lane >= lanes && slots <= kThreads) return;
    const int64_t r_begin = (int64_t)blockIdx.x * p.rows_per_block;
    const int64_t r_end = r_begin + p.rows_per_block < p.rows ? r_begin + p.rows_per_block : p.rows;
    const E* in = static_cast<const E*>(p.in);
    E* out = static_cast<E*>(p.out);
    for (int s = slots <= kThreads ? (int)threadIdx.x - lane * slots : (int)threadIdx.x; s < slots; s += kThreads) {
        const bool pair = s >= n_copy2;
        const int i0 = pair ? (s - n_copy2) * VE : 0;
        const int ca = pair ? p.Dn + i0 : s * VE;
        const int cb = pair ? ca + half : (s + n_copy2) * VE;
        const bool two = pair || s + n_copy2 < n_copy;
        const bool one_axis = pair && same_axis<VE>(p, i0);
        int64_t cur = -1;
        Turn<VE> tab;
        const int64_t first = r_begin + (slots <= kThreads ? lane : 0);
        for (int64_t r = first; r < r_end; r += (int64_t)lanes * kUnroll) {
            float a[kUnroll][VE], b[kUnroll][VE];
            int64_t t[kUnroll], h[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t ru = r + (int64_t)u * lanes;
                if (ru >= r_end) continue;
                t[u] = (uint32_t)ru / (uint32_t)p.H;
                h[u] = (uint32_t)ru - (uint32_t)t[u] * (uint32_t)p.H;
                const E* x = in + t[u] * p.in_t + h[u] * p.in_h;
                load_vec<E, VE>(x + ca, a[u]);
                if (two) load_vec<E, VE>(x + cb, b[u]);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (r + (int64_t)u * lanes >= r_end) continue;
                if (pair) {
                    if (t[u] != cur) {
                        cur = t[u];
                        tab.load(p, i0, one_axis, cur);
                    }
                    tab.turn(p.inverse != 0, a[u], b[u]);
                }
                E* o = out + t[u] * p.out_t + h[u] * p.out_h;
                store_vec<E, VE>(o + ca, a[u]);
                if (two) store_vec<E, VE>(o + cb, b[u]);
            }
        }
    }
}

// The sum over heads, turned. A block takes `toks` tokens at a time; a
// thread adds one vector of VE channels over every hl-th head in float32,
// the partial sums meet in shared memory and are added in lane order, so the
// result does not depend on scheduling.
template <typename E, int VE>
__global__ void __launch_bounds__(kThreads) rope_sum_kernel(const __grid_constant__ RopeParams p) {
    extern __shared__ float part[];  // [lanes][D]
    const int D = p.Dn + p.Dr, half = p.Dr / 2;
    const int slots = D / VE;
    const int lanes = kThreads / slots > 0 ? kThreads / slots : 1;
    const int hl = p.H < lanes ? p.H : lanes;  // threads over the heads of one token
    const int toks = lanes / hl;               // tokens side by side
    const int lane = slots <= kThreads ? (int)threadIdx.x / slots : 0;
    const E* in = static_cast<const E*>(p.in);
    E* out = static_cast<E*>(p.out);
    for (int64_t t0 = (int64_t)blockIdx.x * toks; t0 < p.T; t0 += (int64_t)gridDim.x * toks) {
        const int tl = lane / hl, h0 = lane - tl * hl;
        if (tl < toks && t0 + tl < p.T) {
            const E* x = in + (t0 + tl) * p.in_t;
            for (int s = slots <= kThreads ? (int)threadIdx.x - lane * slots : (int)threadIdx.x; s < slots;
                 s += kThreads) {
                float acc[VE];
#pragma unroll
                for (int k = 0; k < VE; ++k) acc[k] = 0.f;
                for (int h = h0; h < p.H; h += hl * kUnroll) {
                    float v[kUnroll][VE];
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u)
                        if (h + u * hl < p.H) load_vec<E, VE>(x + (int64_t)(h + u * hl) * p.in_h + s * VE, v[u]);
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u)
                        if (h + u * hl < p.H)
#pragma unroll
                            for (int k = 0; k < VE; ++k) acc[k] += v[u][k];
                }
#pragma unroll
                for (int k = 0; k < VE; ++k) part[(int64_t)lane * D + s * VE + k] = acc[k];
            }
        }
        __syncthreads();
        const int per = p.Dn + half;  // outputs of a token: pass-through channels, then pairs
        for (int i = threadIdx.x; i < toks * per; i += kThreads) {
            const int tt = i / per, c = i - tt * per;
            const int64_t t = t0 + tt;
            if (t >= p.T) continue;
            const float* q = part + (int64_t)tt * hl * D + c;
            float a = 0.f, b = 0.f;
            for (int l = 0; l < hl; ++l) {
                a += q[l * D];
                if (c >= p.Dn) b += q[l * D + half];
            }
            E* o = out + t * p.out_t + c;
            if (c >= p.Dn) {
                Turn<1> tab;
                tab.load(p, c - p.Dn, false, t);
                float av[1] = {a}, bv[1] = {b};
                tab.turn(true, av, bv);
                store_vec<E, 1>(o, av);
                store_vec<E, 1>(o + half, bv);
            } else {
                const float av[1] = {a};
                store_vec<E, 1>(o, av);
            }
        }
        __syncthreads();
    }
}

// The cos/sin rows of every token, gathered per pair: a table for the fused
// projection, whose positions are then the token numbers.
__global__ void __launch_bounds__(kThreads) rope_table_kernel(const __grid_constant__ RopeParams p,
                                                              float* __restrict__ cos_out,
                                                              float* __restrict__ sin_out) {
    const int half = p.Dr / 2;
    const int quads = p.cs_vec ? p.Dr / 4 : p.Dr;
    const int64_t items = p.T * quads;
    for (int64_t it = (int64_t)blockIdx.x * kThreads + threadIdx.x; it < items; it += (int64_t)gridDim.x * kThreads) {
        const int64_t t = it / quads;
        const int c = (int)(it - t * quads) * (p.cs_vec ? 4 : 1);
        const int i = c < half ? c : c - half;
        const int n = p.cs_vec ? 4 : 1;
        bool same = true;
        for (int k = 1; k < n; ++k) same &= p.axis[i + k] == p.axis[i];
        if (n == 4 && same) {
            const int64_t row = __ldg(p.pos + p.axis[i] * p.T + t);
            const bool ok = row >= 0 && row < p.cs_rows;
            if (!ok) record_status(p.status, MLA_ERR_POS_RANGE);
            const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
            const int64_t at = (ok ? row : 0) * p.cs_width + c;
            const float4 cv = __ldg(reinterpret_cast<const float4*>(p.cos_tab + at));
            const float4 sv = __ldg(reinterpret_cast<const float4*>(p.sin_tab + at));
            *reinterpret_cast<float4*>(cos_out + t * p.Dr + c) = ok ? cv : z;
            *reinterpret_cast<float4*>(sin_out + t * p.Dr + c) = ok ? sv : z;
        } else {
            for (int k = 0; k < n; ++k) {
                const int64_t row = __ldg(p.pos + p.axis[i + k] * p.T + t);
                const bool ok = row >= 0 && row < p.cs_rows;
                if (!ok) record_status(p.status, MLA_ERR_POS_RANGE);
                const int64_t at = (ok ? row : 0) * p.cs_width + c + k;
                cos_out[t * p.Dr + c + k] = ok ? __ldg(p.cos_tab + at) : 0.f;
                sin_out[t * p.Dr + c + k] = ok ? __ldg(p.sin_tab + at) : 0.f;
            }
        }
    }
}

template <typename E, int VE>
int launch_rows(RopeParams p, bool sum, int num_sms, cudaStream_t stream) {
    if (sum) {
        const int D = p.Dn + p.Dr, slots = D / VE;
        const int lanes = kThreads / slots > 0 ? kThreads / slots : 1;
        const int toks = lanes / (p.H < lanes ? p.H : lanes);
        int64_t grid = (p.T + toks - 1) / toks;
        if (grid > (int64_t)num_sms * 8) grid = (int64_t)num_sms * 8;
        rope_sum_kernel<E, VE><<<(unsigned)grid, kThreads, (size_t)lanes * D * sizeof(float), stream>>>(p);
    } else {
        const int slots = (p.Dn / VE + 1) / 2 + p.Dr / 2 / VE;
        const int lanes = kThreads / slots > 0 ? kThreads / slots : 1;
        // enough rows per block to reuse table entries, fewer when the grid would not fill the SMs
        int64_t per = p.rows / ((int64_t)lanes * num_sms * 8);
        per = per < 1 ? 1 : (per > 2 * kUnroll ? 2 * kUnroll : per);
        p.rows_per_block = (int)(per * lanes);
        const int64_t grid = (p.rows + p.rows_per_block - 1) / p.rows_per_block;
        rope_axes_kernel<E, VE><<<(unsigned)grid, kThreads, 0, stream>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
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
    const int64_t lim = (int64_t)1 << 40;  // keeps every extent inside int64
    for (int64_t v : {s.in_t, s.in_h, s.out_t, s.out_h})
        if (v < 0 || v > lim) return MLA_ERR_INVALID_ARG;
    const int64_t Ho = sum ? 1 : s.H;
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
    p.cs_vec = aligned(cos_tab, 16) && aligned(sin_tab, 16) && s.cs_width % 4 == 0 && s.Dr / 2 % 4 == 0;
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
    p.cs_vec = aligned(cos_tab, 16) && aligned(sin_tab, 16) && s.cs_width % 4 == 0 && s.Dr / 2 % 4 == 0;
    const int64_t items = s.T * (p.cs_vec ? s.Dr / 4 : s.Dr);
    int64_t grid = (items + kThreads - 1) / kThreads;
    if (grid > (int64_t)di.num_sms * 8) grid = (int64_t)di.num_sms * 8;
    rope_table_kernel<<<(unsigned)grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p, cos_out, sin_out);
    return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"

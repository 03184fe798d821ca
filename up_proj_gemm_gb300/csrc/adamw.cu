// One AdamW step over many tensors in one launch, moments in float32 or in
// MXFP8. For every element, in float32, each operation rounded once and in
// this order (so a moment's bits do not depend on the compiler):
//   g  = grad * grad_scale
//   p  = p * (1 - lr wd)
//   m' = m b1 + g (1 - b1)
//   v' = v b2 + (g (1 - b2)) g
//   p' = p - (m' / (sqrt(v') c + eps)) s,   s = lr / (1 - b1^t), c = (1 - b2^t)^-1/2
// (the last line's quotient to 2 ulp). In MXFP8 the moments are m and the
// ROOT of v, each as E4M3 codes and one E8M0 scale per 32 elements (the
// quantizer's rule): the root halves the exponent range that v needs, and a
// root above zero never gets code 0, since a vanished denominator would blow
// up the step. The update uses the moments before they are rounded.
//
// With a seed, codes (and bf16 parameters without a float32 master) are
// rounded up with the probability of their fraction: at b2 = 0.999 a step
// moves v by a thousandth, far below half an E4M3 step, and rounding to
// nearest would hold it still for ever. The random bits are a
// multiplicative mix of the seed and the element's place, so a step is
// reproducible; 16 bits each for m, v and p.
//
// Bound by HBM: one pass, every operand read and written once.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <vector>

#include "checks.h"
#include "internal.h"
#include "mx.cuh"
#include "ptx.cuh"

namespace mlaq {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;  // elements per block: 4 rounds of 8 per thread

struct PlanTensor {
    mla_adamw_tensor t;
    int64_t place;  // first random place: a multiple of 64
};

// The plan: a header, the tensors, then for each chunk its tensor and the
// chunk's number inside it.
struct PlanHeader {
    uint64_t magic;
    int64_t count, chunks, bytes;
    int32_t param_dtype, grad_dtype, bits, reserved;
};
constexpr uint64_t kMagic = 0x3177616461716c6dull;
struct PlanChunk {
    int32_t tensor, number;
};

int64_t plan_bytes(int64_t count, int64_t chunks) {
    return (int64_t)sizeof(PlanHeader) + count * (int64_t)sizeof(PlanTensor) + chunks * (int64_t)sizeof(PlanChunk);
}

struct StepParams {
    const PlanTensor* tensors;
    const PlanChunk* chunks;
    const float* grad_scale;
    float decay, b1, ob1, b2, ob2, root, eps, size;
    uint32_t seed;
    int stochastic;
};

// 32 mixed bits of a place: the upper and lower halves serve m and v.
__device__ __forceinline__ uint32_t mix32(uint32_t place, uint32_t seed) {
    uint32_t x = place * 0x9E3779B1u + seed;
    x = (x ^ (x >> 15)) * 0x6A09E667u;
    x = (x ^ (x >> 13)) * 0xBB67AE85u;
    return x ^ (x >> 16);
}

template <typename E>
__device__ __forceinline__ float get(const E* p) {
    if constexpr (sizeof(E) == 2) return __uint_as_float((uint32_t)*p << 16);
    else return *p;
}
template <typename E>
__device__ __forceinline__ void put(E* p, float v) {
    if constexpr (sizeof(E) == 2) *p = (uint16_t)pack_bf16x2(v, 0.f);
    else *p = v;
}

// N elements at p (16-byte aligned runs when VEC), of which n exist.
template <int N, bool VEC, typename E>
__device__ __forceinline__ void load_n(const E* p, int n, float (&v)[N]) {
    if constexpr (VEC) {
        if constexpr (sizeof(E) == 4) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 f = *reinterpret_cast<const float4*>(p + i);
                v[i] = f.x;
                v[i + 1] = f.y;
                v[i + 2] = f.z;
                v[i + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const uint2 w = *reinterpret_cast<const uint2*>(p + i);
                v[i] = bf16lo_to_f32(w.x);
                v[i + 1] = bf16hi_to_f32(w.x);
                v[i + 2] = bf16lo_to_f32(w.y);
                v[i + 3] = bf16hi_to_f32(w.y);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < n ? get(p + i) : 0.f;
    }
}

template <int N, bool VEC, typename E>
__device__ __forceinline__ void store_n(E* p, int n, const float (&v)[N]) {
    if constexpr (VEC) {
        if constexpr (sizeof(E) == 4) {
#pragma unroll
            for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 4)
                *reinterpret_cast<uint2*>(p + i) = make_uint2(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) put(p + i, v[i]);
    }
}

// The moments and the parameter of one element; r: the root of v'.
template <bool EXACT_ROOT>
__device__ __forceinline__ void update(const StepParams& q, float g, float& p, float& m, float& v, float& r) {
    p = __fmul_rn(p, q.decay);
    m = __fadd_rn(__fmul_rn(m, q.b1), __fmul_rn(g, q.ob1));
    v = __fadd_rn(__fmul_rn(v, q.b2), __fmul_rn(__fmul_rn(g, q.ob2), g));
    // the stored root is rounded once; one that only feeds the step may be off by an ulp
    if constexpr (EXACT_ROOT) r = __fsqrt_rn(v);
    else asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    p = __fsub_rn(p, __fmul_rn(__fdividef(m, __fadd_rn(__fmul_rn(r, q.root), q.eps)), q.size));
}

// bf16 parameters rounded up or down at random, by the low 16 bits.
__device__ __forceinline__ float bf16_random(float p, uint32_t mixed) {
    const uint32_t bits = __float_as_uint(p);
    if ((bits & 0x7F800000u) == 0x7F800000u) return p;
    return __uint_as_float((bits + ((mixed * 0x3C6EF373u) >> 16)) & 0xFFFF0000u);
}

// N elements of a tensor from idx on, moments in float32.
template <int N, bool VEC, typename P, typename G>
__device__ __forceinline__ void step_f32(const StepParams& q, const PlanTensor& T, float gs, int64_t idx, int n) {
    P* param = static_cast<P*>(T.t.param) + idx;
    float* em = static_cast<float*>(T.t.exp_avg) + idx;
    float* ev = static_cast<float*>(T.t.exp_avg_sq) + idx;
    float* ma = T.t.master ? T.t.master + idx : nullptr;
    float g[N], p[N], m[N], v[N];
    load_n<N, VEC>(static_cast<const G*>(T.t.grad) + idx, n, g);
    load_n<N, VEC>(em, n, m);
    load_n<N, VEC>(ev, n, v);
    if (ma) load_n<N, VEC>(ma, n, p);
    else load_n<N, VEC>(param, n, p);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float r;
        update<false>(q, __fmul_rn(g[i], gs), p[i], m[i], v[i], r);
    }
    store_n<N, VEC>(em, n, m);
    store_n<N, VEC>(ev, n, v);
    if (ma) store_n<N, VEC>(ma, n, p);
    else if (sizeof(P) == 2 && q.stochastic) {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = bf16_random(p[i], mix32((uint32_t)(T.place + idx + i), q.seed));
    }
    store_n<N, VEC>(param, n, p);
}

template <typename P, typename G>
__global__ void __launch_bounds__(kThreads) adamw_f32_kernel(const StepParams q) {
    const PlanChunk c = q.chunks[blockIdx.x];
    const PlanTensor& T = q.tensors[c.tensor];
    const float gs = q.grad_scale ? __ldg(q.grad_scale) : 1.f;
    const int64_t base = (int64_t)c.number * kChunk;
    const int64_t left = T.t.n - base;
    const int n = left < kChunk ? (int)left : kChunk;
    // groups of 4: 16-byte accesses of the float32 operands, 8-byte ones of bf16
    const uintptr_t at = reinterpret_cast<uintptr_t>(T.t.exp_avg) | reinterpret_cast<uintptr_t>(T.t.exp_avg_sq) |
                         reinterpret_cast<uintptr_t>(T.t.master) |
                         (reinterpret_cast<uintptr_t>(T.t.param) * (4 / sizeof(P))) |
                         (reinterpret_cast<uintptr_t>(T.t.grad) * (4 / sizeof(G)));
    const bool vec = (at & 15) == 0;
    const int whole = vec ? n & ~3 : 0;
    for (int i = threadIdx.x * 4; i < whole; i += kThreads * 4) step_f32<4, true, P, G>(q, T, gs, base + i, 4);
    for (int i = whole + threadIdx.x; i < n; i += kThreads) step_f32<1, false, P, G>(q, T, gs, base + i, 1);
}

// 8 code bytes at 16 random bits each: E4M3 of v * 2^-e, rounded up where
// the 20-bit fraction below its 3 mantissa bits is above rnd * 2^-16. Values
// below the smallest normal, 2^-6, are moved into its octave, where the
// step is the same; adding upwards keeps "fraction above rnd" exact.
__device__ __forceinline__ uint32_t e4m3_random(float v, float scale, uint32_t rnd) {
    const float s = fabsf(v) * scale;
    const bool sub = s < 0.015625f;
    const float t = sub ? __fadd_ru(s, 0.015625f) : s;
    const uint32_t code = ((__float_as_uint(t) + 0xFFFFFu - (rnd << 4)) >> 20) - (sub ? 968u : 960u);
    return code | ((__float_as_uint(v) >> 24) & 0x80u);
}

// 8 of a block's 32 values (the other 24 in three neighbouring lanes).
template <bool ROOT>
__device__ __forceinline__ uint32_t encode8(const StepParams& q, const float (&v)[8], const uint32_t (&mixed)[8],
                                            uint32_t (&codes)[2]) {
    float am = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) am = amax_nan(am, v[i]);
    am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, 2));
    const uint32_t bits = __float_as_uint(am);
    uint32_t sf;
    if (!q.stochastic || bits >= 0x7F800000u) {
        sf = quantize8_block_scale(v, bits, codes);
    } else {
        const int e = e8m0_exponent_f32(am);
        const float scale = exp2_neg(e);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint32_t c = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x = mixed[4 * w + j];
                c |= e4m3_random(v[4 * w + j], scale, ROOT ? x & 0xFFFFu : x >> 16) << (8 * j);
            }
            codes[w] = c;
        }
        sf = (uint32_t)(e + 127);
    }
    if constexpr (ROOT) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (v[i] > 0.f && ((codes[i / 4] >> (8 * (i % 4))) & 0xFFu) == 0) codes[i / 4] |= 1u << (8 * (i % 4));
    }
    return sf;
}

// 2^(byte - 127); byte 255 marks a block that held a NaN or an infinity.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

// Two E4M3 codes as float32 (exact).
__device__ __forceinline__ void e4m3x2_to_f32(uint32_t two, float& a, float& b) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
        : "=f"(a), "=f"(b)
        : "r"(h));
}

template <bool VEC>
__device__ __forceinline__ void load_codes(const uint8_t* p, int n, uint32_t (&c)[2]) {
    if constexpr (VEC) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        c[0] = w.x;
        c[1] = w.y;
    } else {
        c[0] = c[1] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) c[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
    }
}

template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* p, int n, const uint32_t (&c)[2]) {
    if constexpr (VEC) {
        *reinterpret_cast<uint2*>(p) = make_uint2(c[0], c[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint8_t)(c[i / 4] >> (8 * (i % 4)));
    }
}

__device__ __forceinline__ void decode8(const uint32_t (&c)[2], float scale, float (&v)[8]) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        e4m3x2_to_f32((c[w / 2] >> (16 * (w % 2))) & 0xFFFFu, v[2 * w], v[2 * w + 1]);
        v[2 * w] *= scale;
        v[2 * w + 1] *= scale;
    }
}

// 8 elements of a tensor from idx on (n of them exist), moments in MXFP8.
// All lanes of a warp take part (the block scales are shared by shuffles).
template <bool VEC, typename P, typename G>
__device__ __forceinline__ void step_mx(const StepParams& q, const PlanTensor& T, float gs, int64_t idx, int n) {
    P* param = static_cast<P*>(T.t.param) + idx;
    uint8_t* em = static_cast<uint8_t*>(T.t.exp_avg) + idx;
    uint8_t* ev = static_cast<uint8_t*>(T.t.exp_avg_sq) + idx;
    float* ma = T.t.master ? T.t.master + idx : nullptr;
    float g[8], p[8], m[8], r[8];
    uint32_t cm[2], cv[2], mixed[8];
    uint32_t sm = 0, sv = 0;
    if (VEC || n > 0) {
        sm = T.t.exp_avg_scales[idx >> 5];
        sv = T.t.exp_avg_sq_scales[idx >> 5];
    }
    load_n<8, VEC>(static_cast<const G*>(T.t.grad) + idx, n, g);
    load_codes<VEC>(em, n, cm);
    load_codes<VEC>(ev, n, cv);
    if (ma) load_n<8, VEC>(ma, n, p);
    else load_n<8, VEC>(param, n, p);
    decode8(cm, e8m0_value(sm), m);
    decode8(cv, e8m0_value(sv), r);
    const uint32_t place = (uint32_t)(T.place + idx);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v = __fmul_rn(r[i], r[i]);
        update<true>(q, __fmul_rn(g[i], gs), p[i], m[i], v, r[i]);
        mixed[i] = q.stochastic ? mix32(place + i, q.seed) : 0;
    }
    // the partial group of a tensor's end: elements past it count for nothing in the block's scale
    if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i >= n) m[i] = r[i] = 0.f;
    }
    sm = encode8<false>(q, m, mixed, cm);
    sv = encode8<true>(q, r, mixed, cv);
    if (!VEC && n <= 0) return;
    store_codes<VEC>(em, n, cm);
    store_codes<VEC>(ev, n, cv);
    if ((idx & 31) == 0) {
        T.t.exp_avg_scales[idx >> 5] = (uint8_t)sm;
        T.t.exp_avg_sq_scales[idx >> 5] = (uint8_t)sv;
    }
    if (ma) store_n<8, VEC>(ma, n, p);
    else if (sizeof(P) == 2 && q.stochastic) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = bf16_random(p[i], mixed[i]);
    }
    store_n<8, VEC>(param, n, p);
}

template <typename P, typename G>
__global__ void __launch_bounds__(kThreads) adamw_mx_kernel(const StepParams q) {
    const PlanChunk c = q.chunks[blockIdx.x];
    const PlanTensor& T = q.tensors[c.tensor];
    const float gs = q.grad_scale ? __ldg(q.grad_scale) : 1.f;
    const int64_t base = (int64_t)c.number * kChunk;
    const int64_t left = T.t.n - base;
    const int n = left < kChunk ? (int)left : kChunk;
    const uintptr_t at = reinterpret_cast<uintptr_t>(T.t.master) | reinterpret_cast<uintptr_t>(T.t.param) |
                         reinterpret_cast<uintptr_t>(T.t.grad) | (reinterpret_cast<uintptr_t>(T.t.exp_avg) * 2) |
                         (reinterpret_cast<uintptr_t>(T.t.exp_avg_sq) * 2);
    const bool vec = (at & 15) == 0;
    // whole warps walk the chunk 256 elements at a time; a warp whose 256
    // elements all exist takes the wide path
    for (int i = threadIdx.x * 8; i - (int)(threadIdx.x & 31) * 8 < n; i += kThreads * 8) {
        const int w0 = i - (int)(threadIdx.x & 31) * 8;
        if (vec && w0 + 256 <= n) step_mx<true, P, G>(q, T, gs, base + i, 8);
        else step_mx<false, P, G>(q, T, gs, base + i, n - i < 0 ? 0 : (n - i > 8 ? 8 : n - i));
    }
}

template <typename P, typename G>
int launch(const PlanHeader& h, const StepParams& q, cudaStream_t stream) {
    if (h.bits == 32) adamw_f32_kernel<P, G><<<(unsigned)h.chunks, kThreads, 0, stream>>>(q);
    else adamw_mx_kernel<P, G><<<(unsigned)h.chunks, kThreads, 0, stream>>>(q);
    return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int64_t count_chunks(const mla_adamw_tensor* t, int64_t count) {
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (t[i].n < 0 || t[i].n > ((int64_t)1 << 40)) return -1;
        chunks += (t[i].n + kChunk - 1) / kChunk;
    }
    return count <= kI32Max && chunks <= kI32Max ? chunks : -1;
}

struct Span {
    uintptr_t lo, hi;
    bool out;
};

// Whether a written range meets any other range (gradients may share memory).
bool spans_alias(std::vector<Span>& spans) {
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
    uintptr_t any_hi = 0, out_hi = 0;
    for (const Span& s : spans) {
        if (s.lo < out_hi || (s.out && s.lo < any_hi)) return true;
        any_hi = std::max(any_hi, s.hi);
        if (s.out) out_hi = std::max(out_hi, s.hi);
    }
    return false;
}

}  // namespace
}  // namespace mlaq

using namespace mlaq;

extern "C" {

MLAQ_API size_t mla_adamw_plan_bytes(const mla_adamw_tensor* tensors, int64_t count) {
    if (!tensors || count <= 0 || count > kI32Max) return 0;
    const int64_t chunks = count_chunks(tensors, count);
    return chunks < 0 ? 0 : (size_t)plan_bytes(count, chunks);
}

MLAQ_API int mla_adamw_plan_build(const mla_adamw_tensor* tensors, int64_t count, int param_dtype, int grad_dtype,
                                  int state_bits, void* plan, size_t plan_size) {
    if (!tensors || count <= 0 || count > kI32Max || !plan) return MLA_ERR_INVALID_ARG;
    if ((param_dtype != MLA_IN_F32 && param_dtype != MLA_IN_BF16) ||
        (grad_dtype != MLA_IN_F32 && grad_dtype != MLA_IN_BF16) || (state_bits != 32 && state_bits != 8))
        return MLA_ERR_INVALID_ARG;
    const int64_t chunks = count_chunks(tensors, count);
    if (chunks < 0) return MLA_ERR_INVALID_ARG;
    if (plan_size < (size_t)plan_bytes(count, chunks)) return MLA_ERR_WORKSPACE;
    const int64_t ps = param_dtype == MLA_IN_F32 ? 4 : 2, gs = grad_dtype == MLA_IN_F32 ? 4 : 2;
    const int64_t ss = state_bits / 8;
    for (int64_t i = 0; i < count; ++i) {
        const mla_adamw_tensor& t = tensors[i];
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return MLA_ERR_INVALID_ARG;
        if (state_bits == 8 && (!t.exp_avg_scales || !t.exp_avg_sq_scales)) return MLA_ERR_INVALID_ARG;
        if (state_bits == 32 && (t.exp_avg_scales || t.exp_avg_sq_scales)) return MLA_ERR_INVALID_ARG;
    }
    for (int64_t i = 0; i < count; ++i) {
        const mla_adamw_tensor& t = tensors[i];
        if (!aligned(t.param, ps) || !aligned(t.grad, gs) || !aligned(t.exp_avg, ss) || !aligned(t.exp_avg_sq, ss) ||
            !aligned(t.master, 4))
            return MLA_ERR_ALIGNMENT;
    }
    std::vector<Span> spans;
    auto add = [&spans](const void* p, int64_t bytes, bool out) {
        const Range r = rng(p, bytes);
        if (r.lo != r.hi) spans.push_back({r.lo, r.hi, out});
    };
    for (int64_t i = 0; i < count; ++i) {
        const mla_adamw_tensor& t = tensors[i];
        add(t.grad, t.n * gs, false);
        add(t.param, t.n * ps, true);
        add(t.exp_avg, t.n * ss, true);
        add(t.exp_avg_sq, t.n * ss, true);
        add(t.exp_avg_scales, (t.n + 31) / 32, true);
        add(t.exp_avg_sq_scales, (t.n + 31) / 32, true);
        add(t.master, t.n * 4, true);
    }
    if (spans_alias(spans)) return MLA_ERR_ALIAS;

    PlanHeader h{};
    h.magic = kMagic;
    h.count = count;
    h.chunks = chunks;
    h.bytes = plan_bytes(count, chunks);
    h.param_dtype = param_dtype;
    h.grad_dtype = grad_dtype;
    h.bits = state_bits;
    char* at = static_cast<char*>(plan);
    std::memcpy(at, &h, sizeof(h));
    at += sizeof(h);
    int64_t place = 0;
    for (int64_t i = 0; i < count; ++i) {
        const PlanTensor pt{tensors[i], place};
        std::memcpy(at, &pt, sizeof(pt));
        at += sizeof(pt);
        place += (tensors[i].n + 63) / 64 * 64;
    }
    for (int64_t i = 0; i < count; ++i)
        for (int64_t k = 0; k * kChunk < tensors[i].n; ++k) {
            const PlanChunk c{(int32_t)i, (int32_t)k};
            std::memcpy(at, &c, sizeof(c));
            at += sizeof(c);
        }
    return MLA_OK;
}

MLAQ_API int mla_adamw_step(const void* plan_host, const void* plan_device, const mla_adamw_args* args,
                            const float* grad_scale, void* stream) {
    if (!plan_host || !plan_device || !args) return MLA_ERR_INVALID_ARG;
    PlanHeader h;
    std::memcpy(&h, plan_host, sizeof(h));
    if (h.magic != kMagic) return MLA_ERR_INVALID_ARG;
    const mla_adamw_args& a = *args;
    if (!(a.beta1 >= 0.0 && a.beta1 < 1.0) || !(a.beta2 >= 0.0 && a.beta2 < 1.0) || !(a.eps >= 0.0) ||
        !std::isfinite(a.lr) || !std::isfinite(a.weight_decay) || !std::isfinite(a.eps) || a.step < 1 ||
        (a.stochastic != 0 && a.stochastic != 1))
        return MLA_ERR_INVALID_ARG;
    if (!aligned(plan_device, 16) || !aligned(grad_scale, 4)) return MLA_ERR_ALIGNMENT;
    if (h.chunks == 0) return MLA_OK;
    DeviceInfo di;
    const int ds = current_device_info(&di);
    if (ds != MLA_OK) return ds;
    StepParams q{};
    const char* base = static_cast<const char*>(plan_device) + sizeof(PlanHeader);
    q.tensors = reinterpret_cast<const PlanTensor*>(base);
    q.chunks = reinterpret_cast<const PlanChunk*>(base + h.count * (int64_t)sizeof(PlanTensor));
    q.grad_scale = grad_scale;
    q.decay = (float)(1.0 - a.lr * a.weight_decay);
    q.b1 = (float)a.beta1;
    q.ob1 = (float)(1.0 - a.beta1);
    q.b2 = (float)a.beta2;
    q.ob2 = (float)(1.0 - a.beta2);
    q.size = (float)(a.lr / (1.0 - std::pow(a.beta1, (double)a.step)));
    q.root = (float)std::pow(1.0 - std::pow(a.beta2, (double)a.step), -0.5);
    q.eps = (float)a.eps;
    q.seed = a.seed;
    q.stochastic = a.stochastic;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (h.param_dtype == MLA_IN_F32)
        return h.grad_dtype == MLA_IN_F32 ? launch<float, float>(h, q, cs) : launch<float, uint16_t>(h, q, cs);
    return h.grad_dtype == MLA_IN_F32 ? launch<uint16_t, float>(h, q, cs) : launch<uint16_t, uint16_t>(h, q, cs);
}

}  // extern "C"

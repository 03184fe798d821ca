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
// One pass, every operand read and written once. With float32 moments HBM is
// the bound: 100 M elements at 6.86 TB/s, a plain copy's rate. With MXFP8 moments
// an element is 10 bytes and 67 instructions: 5.13 TB/s (300 M elements in
// 592 us), issue slots 75% taken.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "checks.h"
#include "internal.h"
#include "launch.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace mlaq {
namespace {

constexpr int kThreads = 256;
// Elements per block: with MXFP8 moments 8 rounds of 8 per thread where that
// leaves at least 8 blocks for each that is resident at once (5 on each of 152
// SMs; 300 M elements: 654 -> 634 us against 4 rounds; 20 M elements, 1.6 blocks
// for each: 50 -> 53; float32 moments of 100 M: 408 -> 414). Else 4, halved until there are as many blocks as are resident:
// 100,000 elements in 10 tensors 6.5 -> 3.1 us with MXFP8 moments, 4.6 -> 2.5
// with float32 ones; twice as many blocks lost again (3 M elements in 40 tensors:
// 15.3 against 17.2).
constexpr int kChunkMost = 16384, kChunkLeast = 1024;
constexpr int64_t kChunkBlocks = 760;

struct PlanTensor {
    mla_adamw_tensor t;
    int64_t place;  // first random place: a multiple of 64
};

// The plan: a header, the tensors, then for each chunk its tensor and the
// chunk's number inside it.
struct PlanHeader {
    uint64_t magic;
    int64_t count, chunks, bytes;
    int32_t param_dtype, grad_dtype, bits, chunk;
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
    int chunk;  // elements per block
};

// The complement of 32 mixed bits of a place: its upper and lower halves serve
// m and v. (What is added to a magnitude is the complement of a random number.)
__device__ __forceinline__ uint32_t mix_not(uint32_t place, uint32_t seed) {
    uint32_t x = place * 0x9E3779B1u + seed;
    x = (x ^ (x >> 15)) * 0x6A09E667u;
    x = (x ^ (x >> 13)) * 0xBB67AE85u;
    return ~(x ^ (x >> 16));
}
// The upper halves of another mix of two of them (their complements times a
// constant): the parameters' bits.
__device__ __forceinline__ uint32_t mix_param(uint32_t lo, uint32_t hi) {
    return __byte_perm(~lo * 0x3C6EF373u, ~hi * 0x3C6EF373u, 0x7632);
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

// Two float32 values in one register pair: the packed instructions round
// each half as the scalar ones do, at half the issue slots.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// A product that stays rounded where it feeds an addition: the compiler
// contracts the packed forms into one rounding.
__device__ __forceinline__ f32x2 mul2_rounded(f32x2 a, f32x2 b) {
    float a0, a1, b0, b1;
    unpack2(a, a0, a1);
    unpack2(b, b0, b1);
    return pack2(__fmul_rn(a0, b0), __fmul_rn(a1, b1));
}
__device__ __forceinline__ f32x2 both(float v) { return pack2(v, v); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Roots of two values >= 0 (or NaN), within an ulp: a reciprocal root y of 2
// ulp, r = v y, and one Heron correction r + (v - r^2) y / 2, whose residual
// is exact by fused arithmetic. Values below 2^-126 count as 2^-126 for y
// (their root then comes out at most as large as it is, and a zero's is 0); an
// infinite one, of gradients above 10^19, counts as the largest float32 up to
// the residual, which then makes the root infinite (and the quotient 0).
__device__ __forceinline__ f32x2 root2(f32x2 v) {
    float v0, v1, y0, y1;
    unpack2(v, v0, v1);
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(v0) : "f"(3.402823466e38f));
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(v1) : "f"(3.402823466e38f));
    y0 = max_nan(v0, 1.17549435e-38f);
    y1 = max_nan(v1, 1.17549435e-38f);
    asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(y0));
    asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(y1));
    const f32x2 y = pack2(y0, y1), r = mul2(pack2(v0, v1), y);
    const f32x2 left = fma2(mul2(r, both(-1.f)), r, v);
    return fma2(left, mul2(y, both(0.5f)), r);
}
// The moments and the parameters of two elements; v is v' on return, r its
// root.
__device__ __forceinline__ void update2(const StepParams& q, f32x2 g, f32x2& p, f32x2& m, f32x2& v, f32x2& r) {
    p = mul2(p, both(q.decay));
    m = add2(mul2_rounded(m, both(q.b1)), mul2_rounded(g, both(q.ob1)));
    v = add2(mul2_rounded(v, both(q.b2)), mul2_rounded(mul2(g, both(q.ob2)), g));
    r = root2(v);
    float d0, d1;
    unpack2(fma2(r, both(q.root), both(q.eps)), d0, d1);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(d0));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(d1));
    p = fma2(mul2(m, pack2(d0, d1)), both(-q.size), p);
}

// N elements at once (an odd one is paired with itself).
template <int N>
__device__ __forceinline__ void update(const StepParams& q, float gs, const float (&g)[N], float (&p)[N], float (&m)[N],
                                       float (&v)[N], float (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const int j = i + 1 < N ? i + 1 : i;
        f32x2 pp = pack2(p[i], p[j]), mm = pack2(m[i], m[j]), vv = pack2(v[i], v[j]), rr;
        update2(q, mul2(pack2(g[i], g[j]), both(gs)), pp, mm, vv, rr);
        unpack2(pp, p[i], p[j]);
        unpack2(mm, m[i], m[j]);
        unpack2(vv, v[i], v[j]);
        unpack2(rr, r[i], r[j]);
    }
}

// Two values rounded to bf16, up or down at random by 16 bits each (lo: the
// lower halves of the result and of the bits); NaNs and infinities stay.
__device__ __forceinline__ uint32_t bf16x2_random(float lo, float hi, uint32_t mixed) {
    uint32_t r;
    asm("cvt.rs.bf16x2.f32 %0, %1, %2, %3;" : "=r"(r) : "f"(hi), "f"(lo), "r"(mixed));
    return r;
}

// The largest of three magnitudes, NaN when one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// N parameters of a bf16 tensor rounded at random and stored.
template <int N, bool VEC>
__device__ __forceinline__ void store_random(uint16_t* p, int n, const float (&v)[N], const uint32_t (&mixed)[N]) {
    if constexpr (N == 1) {
        if (n) p[0] = (uint16_t)bf16x2_random(v[0], v[0], mix_param(mixed[0], mixed[0]));
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint32_t a = bf16x2_random(v[i], v[i + 1], mix_param(mixed[i], mixed[i + 1]));
            const uint32_t b = bf16x2_random(v[i + 2], v[i + 3], mix_param(mixed[i + 2], mixed[i + 3]));
            if constexpr (VEC) {
                *reinterpret_cast<uint2*>(p + i) = make_uint2(a, b);
            } else {
                if (i < n) p[i] = (uint16_t)a;
                if (i + 1 < n) p[i + 1] = (uint16_t)(a >> 16);
                if (i + 2 < n) p[i + 2] = (uint16_t)b;
                if (i + 3 < n) p[i + 3] = (uint16_t)(b >> 16);
            }
        }
    }
}

// N elements of a tensor from idx on (n of them exist), moments in float32.
template <int N, bool VEC, typename P, typename G>
struct GroupF32 {
    float g[N], p[N], m[N], v[N];

    __device__ __forceinline__ void load(const PlanTensor& T, int64_t idx, int n) {
        load_n<N, VEC>(static_cast<const G*>(T.t.grad) + idx, n, g);
        load_n<N, VEC>(static_cast<const float*>(T.t.exp_avg) + idx, n, m);
        load_n<N, VEC>(static_cast<const float*>(T.t.exp_avg_sq) + idx, n, v);
        if (T.t.master) load_n<N, VEC>(T.t.master + idx, n, p);
        else load_n<N, VEC>(static_cast<const P*>(T.t.param) + idx, n, p);
    }
    __device__ __forceinline__ void step(const StepParams& q, const PlanTensor& T, float gs, int64_t idx, int n) {
        float r[N];
        update<N>(q, gs, g, p, m, v, r);
        store_n<N, VEC>(static_cast<float*>(T.t.exp_avg) + idx, n, m);
        store_n<N, VEC>(static_cast<float*>(T.t.exp_avg_sq) + idx, n, v);
        P* param = static_cast<P*>(T.t.param) + idx;
        if (T.t.master) store_n<N, VEC>(T.t.master + idx, n, p);
        if constexpr (sizeof(P) == 2) {
            if (!T.t.master && q.stochastic) {
                const uint32_t place = (uint32_t)(T.place + idx);
                uint32_t mixed[N];
#pragma unroll
                for (int i = 0; i < N; ++i) mixed[i] = mix_not(place + i, q.seed);
                store_random<N, VEC>(param, n, p, mixed);
                return;
            }
        }
        store_n<N, VEC>(param, n, p);
    }
};

template <typename P, typename G>
__global__ void __launch_bounds__(kThreads) adamw_f32_kernel(const StepParams q) {
    grid_launch_next();
    grid_wait_previous();
    const PlanChunk c = q.chunks[blockIdx.x];
    const PlanTensor T = q.tensors[c.tensor];
    const float gs = q.grad_scale ? *q.grad_scale : 1.f;
    const int64_t base = (int64_t)c.number * q.chunk;
    const int64_t left = T.t.n - base;
    const int n = left < q.chunk ? (int)left : q.chunk;
    // groups of 4: 16-byte accesses of the float32 operands, 8-byte ones of bf16
    const uintptr_t at = reinterpret_cast<uintptr_t>(T.t.exp_avg) | reinterpret_cast<uintptr_t>(T.t.exp_avg_sq) |
                         reinterpret_cast<uintptr_t>(T.t.master) |
                         (reinterpret_cast<uintptr_t>(T.t.param) * (4 / sizeof(P))) |
                         (reinterpret_cast<uintptr_t>(T.t.grad) * (4 / sizeof(G)));
    const bool vec = (at & 15) == 0;
    const int whole = vec ? n & ~3 : 0;
    for (int i = threadIdx.x * 4; i < whole; i += kThreads * 8) {  // two groups in flight
        const int j = i + kThreads * 4;
        GroupF32<4, true, P, G> a, b;
        a.load(T, base + i, 4);
        if (j < whole) b.load(T, base + j, 4);
        a.step(q, T, gs, base + i, 4);
        if (j < whole) b.step(q, T, gs, base + j, 4);
    }
    for (int i = whole + threadIdx.x; i < n; i += 4 * kThreads) {  // the rest one by one, four in flight
        GroupF32<1, false, P, G> a[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i + u * kThreads < n) a[u].load(T, base + i + u * kThreads, 1);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i + u * kThreads < n) a[u].step(q, T, gs, base + i + u * kThreads, 1);
    }
}

constexpr int kLeastExponent = -120;  // 2^(e-6) is a normal float32 from here on

// E4M3 codes of 8 values * 2^-e, each rounded up where the 20-bit fraction
// below its 3 mantissa bits carries when a random 16-bit number * 16 + 15 is
// added: with the probability of the fraction, to 2^-16, and never for a
// fraction of zero. Bits 20.. of the float32 less (e + 120) * 8 are then the
// code. All of it is one multiply-add: 16 * bits (the sign falls out at the
// top) + the word of the random number, 15 * 16 below it and the exponent's
// difference in its top byte, where the code then stands.
//
// Values below the smallest normal, 2^(e-6), are moved into its octave, where
// the step is the same, and 8 codes back; adding upwards keeps the fraction
// exact. That form is the larger one below 2^(e-6) and the smaller one above
// it, so the maximum of both picks the right one. LOW: there may be such
// values; a root above zero then keeps a code above zero.
template <bool ROOT, bool LOW>
__device__ __forceinline__ void codes_random(const float (&v)[8], int e, const uint32_t (&mixed)[8],
                                             uint32_t (&codes)[2]) {
    const float least = __uint_as_float((uint32_t)(e + 121) << 23);  // 2^(e-6), e >= kLeastExponent
    const uint32_t ends = ((uint32_t)(-(e + 120) * 8) << 24) | 0xF0u;
    uint32_t top[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t bits = __float_as_uint(v[i]);
        if constexpr (LOW) {
            const float a = fabsf(v[i]);
            bits = (uint32_t)__viaddmax_s32(__float_as_int(__fadd_ru(a, least)), -(8 << 20), __float_as_int(a));
        }
        top[i] = bits * 16u + __byte_perm(ends, mixed[i], ROOT ? 0x3540 : 0x3760);
        if constexpr (!ROOT) top[i] |= __float_as_uint(v[i]) & 0x80000000u;
        else if (LOW && v[i] > 0.f) top[i] = max(top[i], 1u << 24);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w)  // the top bytes of four words
        codes[w] = __byte_perm(__byte_perm(top[4 * w], top[4 * w + 1], 0x0073),
                               __byte_perm(top[4 * w + 2], top[4 * w + 3], 0x0073), 0x5410);
}

// The smallest of three magnitudes.
__device__ __forceinline__ float min3_abs(float a, float b, float c) {
    float r;
    asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

constexpr float kLargestRoot = 1.8446743e19f;  // of the largest float32

// 8 of a block's 32 values (the other 24 in three neighbouring lanes); v may
// be scaled on return.
template <bool ROOT>
__device__ __forceinline__ uint32_t encode8(const StepParams& q, float (&v)[8], const uint32_t (&mixed)[8],
                                            uint32_t (&codes)[2]) {
    float am = max3_nan(max3_nan(v[0], v[1], v[2]), max3_nan(v[3], v[4], v[5]), amax_nan(fabsf(v[6]), v[7]));
    am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, 2));
    uint32_t bits = __float_as_uint(am);
    if (q.stochastic && bits < 0x7F800000u) {
        const int e = e8m0_exponent_f32(am);
        int left = e;  // what the codes still have to be scaled by
        if (e < kLeastExponent) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= exp2_neg(e);
            left = 0;
        }
        const float lo = min3_abs(min3_abs(v[0], v[1], v[2]), min3_abs(v[3], v[4], v[5]), fminf(fabsf(v[6]), fabsf(v[7])));
        if (lo < __uint_as_float((uint32_t)(left + 121) << 23)) codes_random<ROOT, true>(v, left, mixed, codes);
        else codes_random<ROOT, false>(v, left, mixed, codes);
        return (uint32_t)(e + 127);
    }
    if (ROOT && bits == 0x7F800000u) {  // an infinite root is kept as that of the largest float32
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fminf(v[i], kLargestRoot);
        bits = __float_as_uint(kLargestRoot);
    }
    const uint32_t sf = quantize8_block_scale(v, bits, codes);
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

// Words of memory at p: NW of them, or the n bytes that exist.
template <int NW, bool VEC>
__device__ __forceinline__ void load_words(const void* p, int n, uint32_t (&w)[NW]) {
    if constexpr (VEC) {
        if constexpr (NW == 2) {
            const uint2 v = *static_cast<const uint2*>(p);
            w[0] = v.x;
            w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < NW; i += 4) {
                const uint4 v = static_cast<const uint4*>(p)[i / 4];
                w[i] = v.x;
                w[i + 1] = v.y;
                w[i + 2] = v.z;
                w[i + 3] = v.w;
            }
        }
    } else if constexpr (NW == 8) {  // float32
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = i < n ? static_cast<const uint32_t*>(p)[i] : 0u;
    } else if constexpr (NW == 4) {  // bf16
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = 2 * i < n ? static_cast<const uint16_t*>(p)[2 * i] : 0u;
            if (2 * i + 1 < n) w[i] |= (uint32_t)static_cast<const uint16_t*>(p)[2 * i + 1] << 16;
        }
    } else {  // codes
        w[0] = w[1] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i / 4] |= (uint32_t)static_cast<const uint8_t*>(p)[i] << (8 * (i % 4));
    }
}

template <int NW>
__device__ __forceinline__ void to_float(const uint32_t (&w)[NW], float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (NW == 8) v[i] = __uint_as_float(w[i]);
        else v[i] = i & 1 ? bf16hi_to_f32(w[i / 2]) : bf16lo_to_f32(w[i / 2]);
    }
}

// 8 elements of a tensor from idx on (n of them exist), moments in MXFP8, as
// they lie in memory. All lanes of a warp step together (the block scales
// are shared by shuffles). MASTER: the parameter is read from its master.
template <bool MASTER, typename P, typename G>
struct GroupMx {
    uint32_t g[2 * sizeof(G)], p[MASTER ? 8 : 2 * sizeof(P)], cm[2], cv[2], sm, sv;

    template <bool VEC>
    __device__ __forceinline__ void load(const PlanTensor& T, int64_t idx, int n) {
        sm = sv = 0;
        if (VEC || n > 0) {
            sm = T.t.exp_avg_scales[idx >> 5];
            sv = T.t.exp_avg_sq_scales[idx >> 5];
        }
        load_words<2 * sizeof(G), VEC>(static_cast<const G*>(T.t.grad) + idx, n, g);
        load_words<2, VEC>(static_cast<const uint8_t*>(T.t.exp_avg) + idx, n, cm);
        load_words<2, VEC>(static_cast<const uint8_t*>(T.t.exp_avg_sq) + idx, n, cv);
        if constexpr (MASTER) load_words<8, VEC>(T.t.master + idx, n, p);
        else load_words<2 * sizeof(P), VEC>(static_cast<const P*>(T.t.param) + idx, n, p);
    }

    template <bool VEC>
    __device__ __forceinline__ void step(const StepParams& q, const PlanTensor& T, float gs, int64_t idx, int n) {
        float gf[8], pf[8], m[8], v[8], r[8];
        uint32_t mixed[8];
        to_float(g, gf);
        to_float(p, pf);
        decode8(cm, e8m0_value(sm), m);
        decode8(cv, e8m0_value(sv), r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(r[i], r[i]);
        update<8>(q, gs, gf, pf, m, v, r);
        const uint32_t place = (uint32_t)(T.place + idx);
#pragma unroll
        for (int i = 0; i < 8; ++i) mixed[i] = q.stochastic ? mix_not(place + i, q.seed) : 0;
        // the partial group of a tensor's end: elements past it count for nothing in the block's scale
        if constexpr (!VEC) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i >= n) m[i] = r[i] = 0.f;
        }
        const uint32_t em = encode8<false>(q, m, mixed, cm);
        const uint32_t ev = encode8<true>(q, r, mixed, cv);
        if (!VEC && n <= 0) return;
        store_codes<VEC>(static_cast<uint8_t*>(T.t.exp_avg) + idx, n, cm);
        store_codes<VEC>(static_cast<uint8_t*>(T.t.exp_avg_sq) + idx, n, cv);
        if ((idx & 31) == 0) {
            T.t.exp_avg_scales[idx >> 5] = (uint8_t)em;
            T.t.exp_avg_sq_scales[idx >> 5] = (uint8_t)ev;
        }
        P* param = static_cast<P*>(T.t.param) + idx;
        if constexpr (MASTER) store_n<8, VEC>(T.t.master + idx, n, pf);
        if constexpr (sizeof(P) == 2 && !MASTER) {
            if (q.stochastic) {
                store_random<8, VEC>(param, n, pf, mixed);
                return;
            }
        }
        store_n<8, VEC>(param, n, pf);
    }
};

// Whole warps walk the chunk 256 elements at a time; a warp whose 256 elements
// all exist takes the wide path, where the next group's loads are in flight
// while this one is computed. (Fetching the group after it into L2 as well cost
// more issue slots than it saved waiting: 300 M elements 586 -> 633 us.)
template <bool MASTER, typename P, typename G>
__device__ __forceinline__ void walk_mx(const StepParams& q, const PlanTensor& T, float gs, int64_t base, int n, bool vec) {
    const int lane8 = (int)(threadIdx.x & 31) * 8;
    int i = threadIdx.x * 8;
    GroupMx<MASTER, P, G> cur, next;
    if (vec && i - lane8 + 256 <= n) {
        const int step = kThreads * 8;
        cur.template load<true>(T, base + i, 8);
        for (;;) {
            const int j = i + step;
            const bool more = j - lane8 + 256 <= n;
            if (more) next.template load<true>(T, base + j, 8);
            cur.template step<true>(q, T, gs, base + i, 8);
            i = j;
            if (!more) break;
            cur = next;
        }
    }
    for (; i - lane8 < n; i += kThreads * 8) {
        const int k = n - i < 0 ? 0 : (n - i > 8 ? 8 : n - i);
        cur.template load<false>(T, base + i, k);
        cur.template step<false>(q, T, gs, base + i, k);
    }
}

template <typename P, typename G>
__global__ void __launch_bounds__(kThreads, 4) adamw_mx_kernel(const StepParams q) {
    grid_launch_next();
    grid_wait_previous();
    const PlanChunk c = q.chunks[blockIdx.x];
    const PlanTensor& T = q.tensors[c.tensor];
    const float gs = q.grad_scale ? *q.grad_scale : 1.f;
    const int64_t base = (int64_t)c.number * q.chunk;
    const int64_t left = T.t.n - base;
    const int n = left < q.chunk ? (int)left : q.chunk;
    const uintptr_t at = reinterpret_cast<uintptr_t>(T.t.master) | reinterpret_cast<uintptr_t>(T.t.param) |
                         reinterpret_cast<uintptr_t>(T.t.grad) | (reinterpret_cast<uintptr_t>(T.t.exp_avg) * 2) |
                         (reinterpret_cast<uintptr_t>(T.t.exp_avg_sq) * 2);
    const bool vec = (at & 15) == 0;
    if (T.t.master) walk_mx<true, P, G>(q, T, gs, base, n, vec);
    else walk_mx<false, P, G>(q, T, gs, base, n, vec);
}

template <typename P, typename G>
int launch(const PlanHeader& h, const StepParams& q, cudaStream_t stream) {
    return launch_overlapped(h.bits == 32 ? adamw_f32_kernel<P, G> : adamw_mx_kernel<P, G>, (unsigned)h.chunks, kThreads, 0,
                             0, stream, q);
}

// The number of chunks and (out) their size; -1: invalid sizes. Never more of
// them with 8 bits than with 32.
int64_t count_chunks(const mla_adamw_tensor* t, int64_t count, int bits, int* size) {
    int64_t chunks = 0, total = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (t[i].n < 0 || t[i].n > ((int64_t)1 << 40)) return -1;
        total = std::min(total + t[i].n, (int64_t)1 << 60);
    }
    for (*size = bits == 8 && total / kChunkMost >= 8 * kChunkBlocks ? kChunkMost : kChunkMost / 2;; *size /= 2) {
        chunks = 0;
        for (int64_t i = 0; i < count; ++i) chunks += (t[i].n + *size - 1) / *size;
        if (chunks >= kChunkBlocks || *size <= kChunkLeast) break;
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

// The same for a plan's tensors, ps, gs and ss bytes for each element of a
// parameter, a gradient and a moment. No exception leaves it.
int written_overlap(const mla_adamw_tensor* tensors, int64_t count, int64_t ps, int64_t gs, int64_t ss) {
    try {
        std::vector<Span> spans;
        spans.reserve((size_t)count * 7);
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
        return spans_alias(spans) ? MLA_ERR_ALIAS : MLA_OK;
    } catch (const std::bad_alloc&) {
        return MLA_ERR_MEMORY;
    }
}

}  // namespace
}  // namespace mlaq

using namespace mlaq;

extern "C" {

MLAQ_API size_t mla_adamw_plan_bytes(const mla_adamw_tensor* tensors, int64_t count) {
    if (!tensors || count <= 0 || count > kI32Max) return 0;
    int chunk;
    const int64_t chunks = count_chunks(tensors, count, 32, &chunk);
    return chunks < 0 ? 0 : (size_t)plan_bytes(count, chunks);
}

MLAQ_API int mla_adamw_plan_build(const mla_adamw_tensor* tensors, int64_t count, int param_dtype, int grad_dtype,
                                  int state_bits, void* plan, size_t plan_size) {
    if (!tensors || count <= 0 || count > kI32Max || !plan) return MLA_ERR_INVALID_ARG;
    if ((param_dtype != MLA_IN_F32 && param_dtype != MLA_IN_BF16) ||
        (grad_dtype != MLA_IN_F32 && grad_dtype != MLA_IN_BF16) || (state_bits != 32 && state_bits != 8))
        return MLA_ERR_INVALID_ARG;
    int chunk;
    const int64_t chunks = count_chunks(tensors, count, state_bits, &chunk);
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
    const int alias = written_overlap(tensors, count, ps, gs, ss);
    if (alias != MLA_OK) return alias;

    PlanHeader h{};
    h.magic = kMagic;
    h.count = count;
    h.chunks = chunks;
    h.bytes = plan_bytes(count, chunks);
    h.param_dtype = param_dtype;
    h.grad_dtype = grad_dtype;
    h.bits = state_bits;
    h.chunk = chunk;
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
        for (int64_t k = 0; k * chunk < tensors[i].n; ++k) {
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
    q.chunk = h.chunk;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (h.param_dtype == MLA_IN_F32)
        return h.grad_dtype == MLA_IN_F32 ? launch<float, float>(h, q, cs) : launch<float, uint16_t>(h, q, cs);
    return h.grad_dtype == MLA_IN_F32 ? launch<uint16_t, float>(h, q, cs) : launch<uint16_t, uint16_t>(h, q, cs);
}

}  // extern "C"

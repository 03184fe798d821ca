// The cache of keys and values in 8 bits, as its kernels see it: pages of
// E4M3 codes [pages, H, page, D] with one E8M0 scale for each block of tokens
// and head [pages, H, page / block]; sequence b's position t lies in page
// table[b][t / page].
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "checks.h"
#include "mlaq.h"
#include "mx.cuh"
#include "ptx.cuh"

namespace mlaq {

// 2^(byte - 127); 255 is NaN.
__device__ __forceinline__ float e8m0_to_f32(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

// Two E4M3 codes (lo in bits 0..7) as f32.
__device__ __forceinline__ void e4m3x2_to_f32(uint32_t codes, float& lo, float& hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
}

// The largest b < B with first(b) <= at, for a first() that never falls: 32 candidates a round, the same answer in
// every lane. (One that does fall gives some b < B.)
template <typename First>
__device__ __forceinline__ int find_sequence(int B, int64_t at, const First& first) {
    const int lane = threadIdx.x % 32;
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int stride = (hi - lo + 31) / 32, i = lo + lane * stride;
        const uint32_t below = __ballot_sync(0xFFFFFFFFu, i < hi && first(i < hi ? i : lo) <= at);
        const int n = below ? 31 - __clz(below) : 0;
        lo += n * stride;
        hi = lo + stride < hi ? lo + stride : hi;
    }
    return lo;
}

// The checks of a cache and of the table of B sequences. *codes_k, *marks_k, ... get their bytes.
struct CacheBytes {
    int64_t k = 0, k_scales = 0, v = 0, v_scales = 0;
};
inline int check_cache(const mla_kv_cache* c, int64_t B, const int32_t* table, int64_t table_width, CacheBytes* n) {
    if (!c || c->pages < 0 || c->page < 16 || c->page > 1024 || (c->page & (c->page - 1)) || c->block < 1 ||
        c->block > c->page || (c->block & (c->block - 1)) || c->H <= 0 || c->Dk <= 0 || c->Dv <= 0 || c->reserved != 0)
        return MLA_ERR_INVALID_ARG;
    if (c->pages > kI32Max || c->H > 65535 || c->Dk > 4096 || c->Dv > 4096) return MLA_ERR_INVALID_ARG;
    if (B < 0 || B > kI32Max || table_width < 0 || table_width > kI32Max || (B > 0 && table_width > 0 && !table))
        return MLA_ERR_INVALID_ARG;
    const bool shared = !c->v;
    if (shared != !c->v_scales || (c->pages > 0 && (!c->k || !c->k_scales))) return MLA_ERR_INVALID_ARG;
    if (shared && c->Dv > c->Dk) return MLA_ERR_INVALID_ARG;
    const int64_t rows = c->pages * c->H * c->page, marks = rows / c->block;
    if (c->pages > 0 && rows > ((int64_t)1 << 50)) return MLA_ERR_INVALID_ARG;
    n->k = rows * c->Dk, n->k_scales = marks;
    n->v = shared ? 0 : rows * c->Dv, n->v_scales = shared ? 0 : marks;
    if (c->Dk % 16 != 0 || c->Dv % 16 != 0) return MLA_ERR_UNSUPPORTED;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(table, 4)) return MLA_ERR_ALIGNMENT;
    return MLA_OK;
}

}  // namespace mlaq

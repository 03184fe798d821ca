// Keys and values into a paged 8-bit cache, and back. Each block of `block`
// tokens of a head has one power-of-two scale 2^e, the smallest with
// amax <= 448 * 2^e over what the block holds, and E4M3 codes v * 2^-e to
// nearest even. A write that continues a block keeps its exponent or raises
// it: e' = max(e, e(new)); codes that were there then become
// rne(code * 2^(e - e')), which touches no other token's block. NaN and Inf get
// NaN codes (with their sign) and leave the scale to the others: one bad
// token does not take its block with it.
//
// Both directions are bound by HBM: two bytes read and one written per
// element, or the reverse (ragged prompts of 128 heads of 192 + 128, 278 MB: 54 us,
// 5.1 TB/s, 77% of a copy's rate; what is left is the wait from a unit's place to its
// rows and from their largest to their codes). Short calls are latency: one token
// of 64 sequences 4.5 us, 9 MB of latents read back 9.7. Work is dealt out by (run of tokens, head, keys or
// values); a run lies in one page, so its codes are contiguous. Run i of
// sequence b is slot first(b) + i with first(b) = cu[b] / run + 2 b: n tokens
// touch at most n / run + 2 runs, so the host knows a bound on the slots
// without knowing the lengths; a slot past its sequence's runs does nothing.
#include "cache.cuh"
#include "internal.h"
#include "launch.cuh"

namespace mlaq {
namespace {

constexpr int kHeld = 12;    // granules of eight values that a thread keeps between the two passes
constexpr int kUnits = 8;    // units (warps) of a block where a warp has a unit

struct CacheParams {
    uint8_t *k, *k_scales, *v, *v_scales;
    const int32_t *table, *start, *cu;
    void *ek, *ev;               // the dense side
    int64_t k_t, k_h, v_t, v_h;  // its strides in elements
    int64_t pages, T, slots, units;
    int B, width, page, block, block_shift, run, H, Dk, Dv, both, heads;  // heads: of one unit
    int out_bf16;
    int* status;
};

// A unit of work: rows [first, first + n) of the dense side are positions
// [at, at + n) of sequence b, all in one run.
struct Unit {
    int64_t row, cell;  // dense row; code row in the cache (of this head)
    int n, place;       // rows; place of the first in its page
    int64_t marks;      // first scale of this page and head
    int head;           // the first of the unit's
    bool values;
};

__device__ __forceinline__ bool find_unit(const CacheParams& p, int64_t unit, Unit& u) {
    const int groups = (p.H + p.heads - 1) / p.heads, per = groups * p.both;
    const int slot = (int)unit / per, r = (int)unit - slot * per;
    u.values = r >= groups;
    u.head = (u.values ? r - groups : r) * p.heads;
    int64_t b = slot, lo = slot, n = 1, i = 0;
    if (p.cu) b = find_sequence(p.B, slot, [&](int s) { return (int64_t)(p.cu[s] / p.run) + 2 * (int64_t)s; });
    const int64_t start = p.start[b];  // beside cu's entries: one wait for memory
    if (p.cu) {
        lo = p.cu[b];
        n = (int64_t)p.cu[b + 1] - lo;
        i = slot - (lo / p.run + 2 * b);
        if (lo < 0 || n < 0 || lo + n > p.T || i < 0) {
            record_status(p.status, MLA_ERR_INVALID_ARG);
            return false;
        }
    }
    if (n == 0) return false;
    const int64_t first = start / p.run + i;  // the run's number in its sequence
    int64_t a = first * p.run, e = a + p.run;
    a = a < start ? start : a;
    e = e > start + n ? start + n : e;
    if (start >= 0 && e <= a) return false;
    const int64_t at = a / p.page;
    const int64_t page = start >= 0 && at < p.width ? p.table[b * p.width + at] : -1;
    if (page < 0 || page >= p.pages) {
        record_status(p.status, MLA_ERR_POS_RANGE);
        return false;
    }
    u.row = lo + (a - start);
    u.n = (int)(e - a);
    u.place = (int)(a - at * p.page);
    u.cell = (page * p.H + u.head) * p.page + u.place;
    u.marks = (page * p.H + u.head) * (p.page / p.block);
    return true;
}

// Eight bf16 of the dense side.
template <bool VEC>
__device__ __forceinline__ uint4 load_granule(const uint16_t* q) {
    if constexpr (VEC) {
        return *reinterpret_cast<const uint4*>(q);
    } else {
        uint4 r;
        r.x = q[0] | ((uint32_t)q[1] << 16);
        r.y = q[2] | ((uint32_t)q[3] << 16);
        r.z = q[4] | ((uint32_t)q[5] << 16);
        r.w = q[6] | ((uint32_t)q[7] << 16);
        return r;
    }
}

// The largest magnitudes, bit for bit, of the even and the odd elements among eight bf16 and m; NaN or Inf where one is.
__device__ __forceinline__ uint32_t amax2(const uint4& g, uint32_t m) {
    const uint32_t w[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7FFF7FFFu));
    return m;
}
// The magnitude bits (of f32) of the largest finite element among eight bf16 and m.
__device__ __forceinline__ uint32_t finite_amax(const uint4& g, uint32_t m) {
    const uint32_t w[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = (w[i] << 16) & 0x7FFFFFFFu, hi = w[i] & 0x7FFF0000u;
        m = max(m, lo < 0x7F800000u ? lo : 0u);
        m = max(m, hi < 0x7F800000u ? hi : 0u);
    }
    return m;
}

// Eight values times s as codes; bad: there are NaN or Inf among the unit's.
__device__ __forceinline__ uint2 encode_granule(const uint4& g, float s, bool bad) {
    const uint32_t w[4] = {g.x, g.y, g.z, g.w};
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float v[4] = {bf16lo_to_f32(w[2 * i]), bf16hi_to_f32(w[2 * i]), bf16lo_to_f32(w[2 * i + 1]),
                            bf16hi_to_f32(w[2 * i + 1])};
        c[i] = pack_e4m3x4(v[0] * s, v[1] * s, v[2] * s, v[3] * s);
        if (bad) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if ((__float_as_uint(v[j]) & 0x7FFFFFFFu) >= 0x7F800000u)
                    c[i] = (c[i] & ~(0xFFu << (8 * j))) | (nan_code(v[j]) << (8 * j));
        }
    }
    return make_uint2(c[0], c[1]);
}

// Granules lane, lane + lanes, ... of rows of `per`, without a division for each.
struct Steps {
    int row, col, rows, cols, per;
    __device__ __forceinline__ Steps(int lane, int lanes, int per)
        : row(lane / per), col(lane % per), rows(lanes / per), cols(lanes % per), per(per) {}
    __device__ __forceinline__ void next() {
        row += rows;
        col += cols;
        if (col >= per) {
            col -= per;
            ++row;
        }
    }
};

// A warp (WARP) or a block per unit. First pass: the new rows' amax, the first
// kHeld granules of each thread staying in registers; second pass: codes.
template <bool WARP, bool VEC>
__global__ void __launch_bounds__(256) kv_cache_write_kernel(const __grid_constant__ CacheParams p) {
    __shared__ uint32_t top[8];
    grid_launch_next();
    grid_wait_previous();
    const int lanes = WARP ? 32 : (int)blockDim.x;
    const int lane = WARP ? (int)threadIdx.x % 32 : (int)threadIdx.x;
    const int64_t unit = WARP ? (int64_t)blockIdx.x * kUnits + threadIdx.x / 32 : (int64_t)blockIdx.x;
    if (unit >= p.units) return;
    Unit u;
    if (!find_unit(p, unit, u)) return;  // the same in every thread of the unit
    const int D = u.values ? p.Dv : p.Dk, per = D / 8, total = u.n * per;
    const int64_t st = u.values ? p.v_t : p.k_t;
    const int64_t sh = u.values ? p.v_h : p.k_h;
    const uint16_t* src = static_cast<const uint16_t*>(u.values ? p.ev : p.ek) + u.row * st + (int64_t)u.head * sh;
    uint8_t* codes = (u.values ? p.v : p.k) + u.cell * D;
    uint8_t* mark = (u.values ? p.v_scales : p.k_scales) + u.marks + u.place / p.block;
    const int heads = p.H - u.head < p.heads ? p.H - u.head : p.heads;
    for (int head = 0; head < heads; ++head, src += sh, codes += (int64_t)p.page * D, mark += p.page / p.block) {
    uint4 held[kHeld];
    uint32_t m2 = 0;
    Steps at(lane, lanes, per);
#pragma unroll
    for (int j = 0; j < kHeld; ++j, at.next()) {
        held[j] = make_uint4(0, 0, 0, 0);
        if (j * lanes + lane < total) held[j] = load_granule<VEC>(src + at.row * st + at.col * 8);
    }
#pragma unroll
    for (int j = 0; j < kHeld; ++j) m2 = amax2(held[j], m2);
    const Steps rest = at;
    for (int g = kHeld * lanes + lane; g < total; g += lanes, at.next()) m2 = amax2(load_granule<VEC>(src + at.row * st + at.col * 8), m2);
    uint32_t m = max((m2 << 16) & 0x7FFFFFFFu, m2 & 0x7FFF0000u);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if constexpr (!WARP) {
        if (threadIdx.x % 32 == 0) top[threadIdx.x / 32] = m;
        __syncthreads();
        for (int i = 0; i < (int)blockDim.x / 32; ++i) m = max(m, top[i]);
    }
    const bool bad = m >= 0x7F800000u;  // the same in every thread of the unit
    if (bad) {  // the others' largest
        m = 0;
#pragma unroll
        for (int j = 0; j < kHeld; ++j) m = finite_amax(held[j], m);
        at = rest;
        for (int g = kHeld * lanes + lane; g < total; g += lanes, at.next())
            m = finite_amax(load_granule<VEC>(src + at.row * st + at.col * 8), m);
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if constexpr (!WARP) {
            __syncthreads();
            if (threadIdx.x % 32 == 0) top[threadIdx.x / 32] = m;
            __syncthreads();
            for (int i = 0; i < (int)blockDim.x / 32; ++i) m = max(m, top[i]);
        }
    }
    int e = e8m0_exponent_f32(__uint_as_float(m)) + 127;
    const int old_rows = u.place % p.block;
    if (old_rows > 0) {
        const int old = *mark;
        if constexpr (WARP) __syncwarp();
        else __syncthreads();  // read by all before it is written
        if (e > old && old != 255) {  // the older codes follow the exponent
            uint8_t* before = codes - (int64_t)old_rows * D;
            const float f = e - old > 126 ? 0.f : __uint_as_float((uint32_t)(127 - (e - old)) << 23);
            for (int g = lane; g < old_rows * per; g += lanes) {
                uint2 c = *reinterpret_cast<const uint2*>(before + g * 8);
                uint32_t w[2] = {c.x, c.y};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float v[4];
                    e4m3x2_to_f32(w[i] & 0xFFFFu, v[0], v[1]);
                    e4m3x2_to_f32(w[i] >> 16, v[2], v[3]);
                    uint32_t r = pack_e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
#pragma unroll
                    for (int j = 0; j < 4; ++j)  // NaN codes stay as they are
                        if (((w[i] >> (8 * j)) & 0x7Fu) == 0x7Fu) r = (r & ~(0xFFu << (8 * j))) | (w[i] & (0xFFu << (8 * j)));
                    w[i] = r;
                }
                *reinterpret_cast<uint2*>(before + g * 8) = make_uint2(w[0], w[1]);
            }
        } else {
            e = old;
        }
    }
    // 2^-(e - 127): e <= 127 + 120 for finite bf16, and a kept exponent may be any
    const float s = e == 255 ? 0.f : e == 254 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int g = j * lanes + lane;
        if (g < total) *reinterpret_cast<uint2*>(codes + g * 8) = encode_granule(held[j], s, bad);
    }
    at = rest;
    for (int g = kHeld * lanes + lane; g < total; g += lanes, at.next())
        *reinterpret_cast<uint2*>(codes + g * 8) = encode_granule(load_granule<VEC>(src + at.row * st + at.col * 8), s, bad);
    if (lane == 0) *mark = (uint8_t)e;
    if constexpr (!WARP) __syncthreads();  // top, for the next head
    }
}

// A warp per unit: 16 codes to a step, four steps in flight.
template <typename E>
__global__ void __launch_bounds__(256) kv_cache_read_kernel(const __grid_constant__ CacheParams p) {
    grid_launch_next();
    grid_wait_previous();
    const int lane = threadIdx.x % 32;
    const int64_t unit = (int64_t)blockIdx.x * kUnits + threadIdx.x / 32;
    if (unit >= p.units) return;
    Unit u;
    if (!find_unit(p, unit, u)) return;
    const int D = u.values ? p.Dv : p.Dk, per = D / 16, total = u.n * per;
    const int64_t st = u.values ? p.v_t : p.k_t;
    E* dst = static_cast<E*>(u.values ? p.ev : p.ek) + u.row * st + (int64_t)u.head * D;
    const uint8_t* codes = (u.values ? p.v : p.k) + u.cell * D;
    const uint8_t* marks = (u.values ? p.v_scales : p.k_scales) + u.marks;
    constexpr int kFlight = 4;
    Steps at(lane, 32, per);
    for (int base = lane; base < total; base += 32 * kFlight) {
        int row[kFlight], col[kFlight];
        uint4 c[kFlight];
        uint32_t e[kFlight];
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
            const int g = base + 32 * j;
            row[j] = at.row, col[j] = at.col;
            at.next();
            if (g < total) {
                c[j] = *reinterpret_cast<const uint4*>(codes + (int64_t)g * 16);
                e[j] = marks[(u.place + row[j]) >> p.block_shift];
            }
        }
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
            const int g = base + 32 * j;
            if (g >= total) break;
            const float s = e8m0_to_f32(e[j]);
            E* q = dst + row[j] * st + col[j] * 16;
            const uint32_t w[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
            if constexpr (sizeof(E) == 2) {
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float lo, hi;
                    e4m3x2_to_f32(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu, lo, hi);
                    o[i] = pack_bf16x2(lo * s, hi * s);
                }
                st_global_v4(q, o[0], o[1], o[2], o[3]);
                st_global_v4(q + 8, o[4], o[5], o[6], o[7]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v[4];
                    e4m3x2_to_f32(w[i] & 0xFFFFu, v[0], v[1]);
                    e4m3x2_to_f32(w[i] >> 16, v[2], v[3]);
                    st_global_v4(q + 4 * i, __float_as_uint(v[0] * s), __float_as_uint(v[1] * s),
                                 __float_as_uint(v[2] * s), __float_as_uint(v[3] * s));
                }
            }
        }
    }
}

// What both directions check alike; *p gets everything but the dense side's strides. run: tokens of a unit.
int check_call(const mla_kv_cache* c, int64_t B, const int32_t* table, int64_t width, const int32_t* start,
               const int32_t* cu, int64_t T, const int* status, int64_t run, CacheBytes* n, CacheParams* p) {
    const int st = check_cache(c, B, table, width, n);
    if (st != MLA_OK && st != MLA_ERR_UNSUPPORTED && st != MLA_ERR_ALIGNMENT) return st;
    if (T < 0 || T > kI32Max || (!cu && T != B) || (T > 0 && (B == 0 || !start))) return MLA_ERR_INVALID_ARG;
    if (st != MLA_OK) return st;
    if (!aligned(start, 4) || !aligned(cu, 4) || !aligned(status, 4)) return MLA_ERR_ALIGNMENT;
    p->k = c->k, p->k_scales = c->k_scales, p->v = c->v, p->v_scales = c->v_scales;
    p->table = table, p->start = start, p->cu = cu, p->status = const_cast<int*>(status);
    p->pages = c->pages, p->T = T;
    p->B = (int)B, p->width = (int)width, p->page = c->page, p->block = c->block, p->block_shift = __builtin_ctz(c->block), p->run = (int)run;
    p->H = c->H, p->Dk = c->Dk, p->Dv = c->Dv, p->both = c->v ? 2 : 1;
    p->slots = cu ? T / run + 2 * B : B;
    p->heads = 1;
    p->units = p->slots * p->H * p->both;
    return p->units > kI32Max ? MLA_ERR_UNSUPPORTED : MLA_OK;
}

int64_t extent2(int64_t T, int64_t st, int64_t H, int64_t sh, int64_t D, int64_t size) {
    return T > 0 ? ((T - 1) * st + (H - 1) * sh + D) * size : 0;
}

}  // namespace
}  // namespace mlaq

using namespace mlaq;

extern "C" {

MLAQ_API int mla_kv_cache_write(const mla_kv_cache* cache, const void* k, int64_t k_t, int64_t k_h, const void* v,
                                int64_t v_t, int64_t v_h, int64_t T, int64_t B, const int32_t* table,
                                int64_t table_width, const int32_t* start, const int32_t* cu, int* dev_status,
                                void* stream) {
    CacheParams p{};
    CacheBytes n;
    const int st = check_call(cache, B, table, table_width, start, cu, T, dev_status, cache ? cache->block : 1, &n, &p);
    if (st != MLA_OK && st != MLA_ERR_UNSUPPORTED && st != MLA_ERR_ALIGNMENT) return st;
    const mla_kv_cache& c = *cache;
    const bool shared = !c.v;
    if (T > 0 && (!k || shared == (v != nullptr))) return MLA_ERR_INVALID_ARG;
    for (const int64_t q : {k_t, k_h, v_t, v_h})
        if (!inside(T > c.H ? T : c.H, q)) return MLA_ERR_INVALID_ARG;
    if (st != MLA_OK) return st;
    if (!aligned(k, 2) || !aligned(v, 2)) return MLA_ERR_ALIGNMENT;
    const Range outs[] = {rng(c.k, n.k), rng(c.k_scales, n.k_scales), rng(c.v, n.v), rng(c.v_scales, n.v_scales),
                          rng(dev_status, 4)};
    const Range ins[] = {rng(k, extent2(T, k_t, c.H, k_h, c.Dk, 2)), rng(v, extent2(T, v_t, c.H, v_h, c.Dv, 2)),
                         rng(table, B * table_width * 4), rng(start, B * 4), rng(cu, (B + 1) * 4)};
    if (any_alias(outs, ins)) return MLA_ERR_ALIAS;
    if (T == 0) return MLA_OK;
    DeviceInfo di;
    const int ds = current_device_info(&di);
    if (ds != MLA_OK) return ds;
    p.ek = const_cast<void*>(k), p.ev = const_cast<void*>(v);
    p.k_t = k_t, p.k_h = k_h, p.v_t = v_t, p.v_h = v_h;
    const bool vec = aligned(k, 16) && aligned(v, 16) && k_t % 8 == 0 && k_h % 8 == 0 && v_t % 8 == 0 && v_h % 8 == 0;
    // a warp per unit while its granules fit into a warp's registers, else as many warps as that takes, eight at most (28672
    // tokens of latents in blocks of 64: 12 us, by warps 42; 4096 tokens of 8 heads in blocks of 256: 8.1, by warps 40);
    // a call of single tokens has units of one row
    const int D = p.Dk > p.Dv || shared ? p.Dk : p.Dv;
    const int granules = (cu ? p.block : 1) * (D / 8), warps = (granules + 32 * kHeld - 1) / (32 * kHeld);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    // finding a unit's place takes as long as its memory: several heads to a unit once that leaves enough of them (5000
    // tokens of 128 heads: 110 us, with one head 152; single tokens of 512 sequences: 82, with one 174)
    const int64_t enough = (int64_t)di.num_sms * (warps == 1 ? 32 : 8);
    while (p.heads < 8 && p.heads < p.H && p.units / (2 * p.heads) >= enough) p.heads *= 2;
    p.units = p.slots * ((p.H + p.heads - 1) / p.heads) * p.both;
    if (warps == 1) {
        const unsigned grid = (unsigned)((p.units + kUnits - 1) / kUnits);
        return vec ? launch_overlapped(kv_cache_write_kernel<true, true>, grid, 32 * kUnits, 0, 0, cs, p)
                   : launch_overlapped(kv_cache_write_kernel<true, false>, grid, 32 * kUnits, 0, 0, cs, p);
    }
    const unsigned threads = 32 * (warps > 8 ? 8 : warps);
    return vec ? launch_overlapped(kv_cache_write_kernel<false, true>, (unsigned)p.units, threads, 0, 0, cs, p)
               : launch_overlapped(kv_cache_write_kernel<false, false>, (unsigned)p.units, threads, 0, 0, cs, p);
}

MLAQ_API int mla_kv_cache_read(const mla_kv_cache* cache, void* k, void* v, int dtype, int64_t T, int64_t B,
                               const int32_t* table, int64_t table_width, const int32_t* start, const int32_t* cu,
                               int* dev_status, void* stream) {
    CacheParams p{};
    CacheBytes n;
    // tokens of a unit: 16 (2 to 9 KB of codes; two would take 405 us where 5000 tokens of 128 heads take 111), fewer while
    // that leaves SMs without work (512 tokens of latents: 3.6 us, with 16 8.2)
    int64_t run = 16;
    DeviceInfo sms;
    if (cache && current_device_info(&sms) == MLA_OK)
        while (run > 2 && T / run * cache->H * (cache->v ? 2 : 1) < (int64_t)sms.num_sms * 32) run /= 2;
    const int st = check_call(cache, B, table, table_width, start, cu, T, dev_status, run, &n, &p);
    if (st != MLA_OK && st != MLA_ERR_UNSUPPORTED && st != MLA_ERR_ALIGNMENT) return st;
    const mla_kv_cache& c = *cache;
    const bool shared = !c.v;
    if (dtype != MLA_IN_F32 && dtype != MLA_IN_BF16) return MLA_ERR_INVALID_ARG;
    if (T > 0 && (!k || shared == (v != nullptr))) return MLA_ERR_INVALID_ARG;
    if (st != MLA_OK) return st;
    if (!aligned(k, 16) || !aligned(v, 16)) return MLA_ERR_ALIGNMENT;
    const int64_t size = dtype == MLA_IN_F32 ? 4 : 2;
    const Range outs[] = {rng(k, T * c.H * c.Dk * size), rng(v, T * c.H * c.Dv * size), rng(dev_status, 4)};
    const Range ins[] = {rng(c.k, n.k), rng(c.k_scales, n.k_scales), rng(c.v, n.v), rng(c.v_scales, n.v_scales),
                         rng(table, B * table_width * 4), rng(start, B * 4), rng(cu, (B + 1) * 4)};
    if (any_alias(outs, ins)) return MLA_ERR_ALIAS;
    if (T == 0) return MLA_OK;
    DeviceInfo di;
    const int ds = current_device_info(&di);
    if (ds != MLA_OK) return ds;
    p.ek = k, p.ev = v;
    p.k_t = (int64_t)c.H * c.Dk, p.v_t = (int64_t)c.H * c.Dv;
    const unsigned grid = (unsigned)((p.units + kUnits - 1) / kUnits);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return dtype == MLA_IN_F32 ? launch_overlapped(kv_cache_read_kernel<float>, grid, 32 * kUnits, 0, 0, cs, p)
                               : launch_overlapped(kv_cache_read_kernel<uint16_t>, grid, 32 * kUnits, 0, 0, cs, p);
}

}  // extern "C"

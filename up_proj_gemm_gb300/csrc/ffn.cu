// Gated feed-forward block, forward and backward (T tokens, K channels, F
// hidden channels, all bf16 with float32 accumulation):
//   forward   [g | u] = x Wgu^T   (Wgu [2F, K]: F gate rows, then F up rows)
//             h = act(g) u,  y = h Wd^T                       (Wd [K, F])
//   backward  dh = dy Wd,  dg = dh u act'(g),  du = dh act(g)
//             dx = [dg | du] Wgu,  dWgu = [dg | du]^T x,  dWd = dy^T h
// Six products on one GEMM kernel: both projections, the activation and the
// product are one launch (a tile holds the same 128 hidden channels of gate
// and up), and so are dh and the activation's gradient.
//
// The GEMM: a cluster of two CTAs computes a 256 x 256 tile with
// tcgen05.mma.cta_group::2 (M = 256: each CTA accumulates its 128 rows over
// all 256 columns in its own TMEM; each stages its 128 rows of A and its half
// of B, so an operand byte is fetched once per pair). 64-element K steps,
// operands by TMA into a ring of 32 KB stages per CTA, two accumulators of
// 256 TMEM columns, so a tile's epilogue runs under the next one's products.
// Operands come K-major (rows contiguous along the reduction) or MN-major
// (the reduction runs over rows): no transposed copy is made.
// Warps: 0 producer, 1 MMA issuer (of the pair's even CTA), 2-9 epilogue.
// Bound by the tensor cores when T is in the thousands.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "checks.h"
#include "internal.h"
#include "launch.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace mlaq {
namespace {

constexpr int kThreads = 320;
constexpr int kBK = 64;
constexpr uint32_t kHalfBytes = 128u * 128u;       // 128 rows (or columns) of one K step, one operand
constexpr uint32_t kStageBytes = 2u * kHalfBytes;  // A and B of one CTA
constexpr uint32_t kChunkBytes = 64u * 128u;       // MN-major: 64 columns of 64 K rows
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSlotBytes = 32u * 64u;         // 32 rows x 32 columns of a result, 64-byte swizzle (kStore: two, as one)
constexpr int kEpiWarps = 8;
constexpr int kSplitSteps = 12;                     // K steps that adding up a split reduction costs
constexpr int kTailSteps = 16;                     // K steps that a grid for the last tiles costs
constexpr int kTileSteps = 4;                      // K steps that a tile costs beside its own
constexpr int kMaxSplits = 4;                      // clusters of 8 CTAs

enum Epilogue { kStore = 0, kGate = 1, kGateGrad = 2 };

// Ring stages and each epilogue warp's slots: results leave by TMA from a slot
// (a lane writing its own row of the result instead took 32 cache lines per
// instruction: 25 against 9 us for one tile of kGateGrad), and kGateGrad's gate
// and up products arrive in three pairs of slots, two pairs ahead.
template <int EPI>
struct Smem {
    static constexpr int kStages = EPI == kGateGrad ? 4 : 5;
    static constexpr int kSlots = EPI == kGateGrad ? 6 : 4;
    static constexpr uint32_t kRing = kStages * kStageBytes;
    static constexpr size_t kBytes = 1024 + kRing + (size_t)kEpiWarps * kSlots * kSlotBytes + 512;
};

// How a product stands to the grid before it on the stream: the first of a call
// waits for it; one with an operand from it waits before its loads; and one that
// needs nothing of it, but of the grid before that (the weight gradients after
// dx), runs in the SMs it leaves idle and waits at its own end, so that whoever
// waits for this grid has waited for both.
enum After { kFirst = 0, kAfter = 1, kBeside = 2 };

// A result and its tiles; kGate: N = F (a tile holds 128 of them).
struct Result {
    int M, N, m_tiles, n_tiles;
};

struct GemmParams {
    // Both weight gradients are one launch: their tiles (over the same T) fill
    // the last wave together. One result otherwise, and no tiles in the second.
    Result r[2];
    int tiles0, tiles;        // of the first result, of both
    int k_tiles;
    int splits;               // parts of the reduction, each a pair of the cluster
    int after;                // kFirst, kAfter or kBeside
    int late;                 // the next grid runs beside this one: it starts after this one's wait
    int early, head;          // the first `early` clusters share `head` tiles before all share the rest (0: not in this grid)
    int F, act;
    uint16_t* gate_up_out;    // kGate: [M, 2F] or null
    const uint16_t* gate_up;  // kGateGrad: [M, 2F]
    int* status;
};

// A shared-memory matrix descriptor moved by a number of bytes. Its address
// field is address / 16 in 14 bits and shared addresses stay below 2^18, so
// the addition never carries out of it. The issuing thread of the products
// adds to descriptors built once: built anew, four MMAs took it 280 cycles of
// a K step's 512.
__device__ __forceinline__ uint64_t desc_at(uint64_t desc, uint32_t bytes) {
    return (desc & 0xFFFFFFFF00000000ull) | (uint32_t)((uint32_t)desc + (bytes >> 4));
}
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return MN ? desc_mnmajor_sw128(addr, kChunkBytes) : desc_kmajor_sw128(addr);
}
// Bytes from one 16-element K slice of a stage's operand to the next.
template <bool MN>
constexpr uint32_t kSlice = MN ? 2048u : 32u;

// ------------------------------------------------------- two-CTA primitives
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ int cluster_id() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
    return (int)r;
}
__device__ __forceinline__ int cluster_count() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%nclusterid.x;" : "=r"(r));
    return (int)r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
// without a release (360 cycles): for warps that wrote nothing another CTA reads
__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
// The address of another CTA's copy of a shared-memory location.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void tma_store_3d(const void* tmap, int32_t c0, int32_t c1, int32_t c2, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(tmap),
                 "r"(c0), "r"(c1), "r"(c2), "r"(src)
                 : "memory");
}
// Relaxed: the arrival says that TMEM was read (ordered by the tcgen05 fence);
// a release would wait for the warp's stores to shared memory.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* tmap, int32_t c0, int32_t c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on the same barrier of both CTAs (mask: their cluster ranks) once the MMAs issued so far are done.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar, uint32_t mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)mask)
        : "memory");
}

// ------------------------------------------------------------- activations
// act(g) and its derivative. The sigmoid is 1 / (1 + 2^(-z log2 e)) by the
// hardware's exponential and reciprocal (a few ulp of float32, far below the
// bf16 results; 2^x overflows to infinity, whose reciprocal is 0). The
// activation is a template argument: an epilogue is bound by its instructions.
__device__ __forceinline__ float sigmoid(float z) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

// The normal distribution (1 + erf(g / sqrt 2)) / 2 and e = exp(-g^2 / 2). With
// x = |g| / sqrt 2, erfc(x) = t P(t) exp(-x^2), t = 1 / (1 + 0.3 x): P is a
// polynomial of degree 8 fitted to exp(x^2) erfc(x) / t over 0 <= x <= 14 for
// the least relative error (4e-8; in float32 1e-6 for |g| < 5). erfcf takes
// three times the instructions, and the gradient shares e.
__device__ __forceinline__ float normal_cdf(float g, float& e) {
    const float x = fabsf(g);
    float t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(x, 0.21213203f, 1.f)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * g * -0.72134752f));
    float p = -0.126616612f;
    p = fmaf(p, t, 0.471826404f);
    p = fmaf(p, t, -0.484692097f);
    p = fmaf(p, t, 0.517049134f);
    p = fmaf(p, t, -0.0740492865f);
    p = fmaf(p, t, 0.20638521f);
    p = fmaf(p, t, 0.150468856f);
    p = fmaf(p, t, 0.170423716f);
    p = fmaf(p, t, 0.169204757f);
    const float tail = 0.5f * t * p * e;
    return g < 0.f ? tail : 1.f - tail;
}

template <int ACT>
__device__ __forceinline__ float activate(float g) {
    float e;
    if constexpr (ACT == MLA_ACT_SILU) return g * sigmoid(g);
    else if constexpr (ACT == MLA_ACT_GELU) return g * normal_cdf(g, e);
    // 0.5 g (1 + tanh(z)) = g sigmoid(2 z), z = sqrt(2/pi) (g + 0.044715 g^3)
    else return g * sigmoid(g * fmaf(0.0713548162f, g * g, 1.59576912f));
}

template <int ACT>
__device__ __forceinline__ void activate_grad(float g, float& a, float& da) {
    if constexpr (ACT == MLA_ACT_SILU) {
        const float s = sigmoid(g);
        a = g * s;
        da = fmaf(a, 1.f - s, s);
    } else if constexpr (ACT == MLA_ACT_GELU) {
        float e;
        const float c = normal_cdf(g, e);
        a = g * c;
        da = fmaf(g * 0.39894228f, e, c);
    } else {
        const float g2 = g * g, s = sigmoid(g * fmaf(0.0713548162f, g2, 1.59576912f));
        a = g * s;
        da = fmaf(a * (1.f - s), fmaf(0.214064449f, g2, 1.59576912f), s);
    }
}

// f with the activation as a compile-time constant.
template <int ACT>
struct ActTag {
    static constexpr int value = ACT;
};
template <typename Fn>
__device__ __forceinline__ void with_act(int act, Fn&& f) {
    if (act == MLA_ACT_SILU) f(ActTag<MLA_ACT_SILU>{});
    else if (act == MLA_ACT_GELU) f(ActTag<MLA_ACT_GELU>{});
    else f(ActTag<MLA_ACT_GELU_TANH>{});
}

__device__ __forceinline__ void unpack8(uint4 w, float (&v)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16lo_to_f32(u[i]);
        v[2 * i + 1] = bf16hi_to_f32(u[i]);
    }
}

// Which result a tile is of, and where. Tiles in groups of 8 row tiles, columns inside a group: the tiles that run
// at the same time span about as many rows of A as of B, which L2 holds.
constexpr int kGroupM = 8;
__device__ __forceinline__ int tile_at(const GemmParams& p, int tile, int& mt, int& nt) {
    const int job = tile >= p.tiles0;
    tile -= job ? p.tiles0 : 0;
    const int m_tiles = job ? p.r[1].m_tiles : p.r[0].m_tiles;
    const int per = kGroupM * (job ? p.r[1].n_tiles : p.r[0].n_tiles);
    const int g = tile / per, r = tile - g * per;
    const int rows = m_tiles - g * kGroupM < kGroupM ? m_tiles - g * kGroupM : kGroupM;
    nt = r / rows;
    mt = g * kGroupM + (r - nt * rows);
    return job;
}

// One epilogue warp: rows row0 .. row0 + 31 of the tile, lane = row. Its chunks
// of 32 columns come from TMEM, or (splits > 1) as the sum of the pairs' partial
// sums in distributed shared memory.
template <int EPI>
struct Epi {
    const GemmParams& p;
    const CUtensorMap* tmO;   // kStore [M, N], kGate h [M, F]; kGateGrad: {F, 2, T} view of [dg | du]
    const CUtensorMap* tmG;   // kGate, kGateGrad: {F, 2, T} view of the gate and up products
    uint32_t slots, bars;     // this warp's slots; kGateGrad: a barrier per pair of them
    uint32_t sums;            // splits > 1: this CTA's partial sums, float4 [column / 4][128 rows]
    int lane, quad, half, prank, srank;
    int used = 0;             // pairs of slots this warp has used so far
    int asked = 0;            // kGateGrad: chunks whose loads are under way
    volatile int* abort_flag;
    int M = 0, N = 0;         // of the tile's result

    // chunks of this warp: of the tile's 8 (kGate: 4 of gates with their 4 of up products; kStore: 4 of 64 columns)
    static constexpr int kChunks = EPI == kGateGrad ? 8 : 4;
    static constexpr int kWidth = EPI == kStore ? 64 : 32;
    __device__ __forceinline__ int chunk(int i) const { return srank + p.splits * (half + 2 * i); }

    template <int S>
    __device__ __forceinline__ void add_up(uint32_t at, uint32_t (&v)[32]) const {
        uint32_t from[S];
#pragma unroll
        for (int s = 0; s < S; ++s) from[s] = map_to_rank(at, 2 * s + prank);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {  // 2 S loads in flight
            float4 f[S][2];
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int k = 0; k < 2; ++k) f[s][k] = ld_cluster_v4(from[s] + 2048u * (i + k));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float4 a = f[0][k];
#pragma unroll
                for (int s = 1; s < S; ++s) {
                    a.x += f[s][k].x;
                    a.y += f[s][k].y;
                    a.z += f[s][k].z;
                    a.w += f[s][k].w;
                }
                v[4 * (i + k)] = __float_as_uint(a.x);
                v[4 * (i + k) + 1] = __float_as_uint(a.y);
                v[4 * (i + k) + 2] = __float_as_uint(a.z);
                v[4 * (i + k) + 3] = __float_as_uint(a.w);
            }
        }
    }

    // The 32 columns from col on of this lane's row (TMEM: complete after tmem_ld_wait).
    __device__ __forceinline__ void values(uint32_t tacc, int col, uint32_t (&v)[32]) const {
        const uint32_t at = sums + 16u * ((col / 4) * 128 + quad * 32 + lane);
        switch (p.splits) {
            case 1: tmem_ld32(tacc + col, v); break;
            case 2: add_up<2>(at, v); break;
            case 3: add_up<3>(at, v); break;
            default: add_up<kMaxSplits>(at, v); break;
        }
    }

    // Splits > 1: this warp's part of the accumulator, for the other CTAs to add.
    __device__ __forceinline__ void share(uint32_t tacc) const {
        for (int c = 0; c < 128; c += 32) {
            uint32_t v[32];
            __syncwarp();
            tmem_ld32(tacc + half * 128 + c, v);
            tmem_ld_wait();
            const uint32_t at = sums + 16u * ((half * 32 + c / 4) * 128 + quad * 32 + lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) sts_v4(at + 2048u * i, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
    }

    // 16 bytes (8 columns) of this lane's row inside a slot
    __device__ __forceinline__ uint32_t piece(uint32_t slot, int k) const {
        return slot + 64u * lane + 16u * (k ^ ((lane >> 1) & 3));
    }
    __device__ __forceinline__ void write(uint32_t slot, const float (&v)[32]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            sts_v4(piece(slot, k), pack_bf16x2(v[8 * k], v[8 * k + 1]), pack_bf16x2(v[8 * k + 2], v[8 * k + 3]),
                   pack_bf16x2(v[8 * k + 4], v[8 * k + 5]), pack_bf16x2(v[8 * k + 6], v[8 * k + 7]));
    }
    // The slots written by the warp are ready for a TMA store by lane 0.
    __device__ __forceinline__ void written() const {
        fence_proxy_async_smem();
        __syncwarp();
    }
    // All but the newest N groups of stores have been read.
    template <int N>
    __device__ __forceinline__ void stores_read() const {
        if (lane == 0) bulk_wait_group_read<N>();
        __syncwarp();
    }

    // kGateGrad: fetch chunk i's gate and up products into the pair of slots of
    // the chunk three before it, whose stores must have been read: all but the
    // newest one's, since no more than two chunks are asked for ahead.
    __device__ __forceinline__ void ask(int n0, int64_t row0, int i) {
        const int f = n0 + 32 * chunk(i), pair = asked % 3;
        if (lane == 0) {
            bulk_wait_group_read<1>();  // one group per chunk
            const uint32_t slot = slots + kSlotBytes * (2 * pair), bar = bars + 8u * pair;
            mbar_arrive_expect_tx(bar, 2 * kSlotBytes);
            tma_load_3d(slot, tmG, f, 0, (int32_t)row0, bar);
            tma_load_3d(slot + kSlotBytes, tmG, f, 1, (int32_t)row0, bar);
        }
        ++asked;
    }
    __device__ __forceinline__ bool has(int n0, int64_t row0, int i) const {
        return chunk(i) < kChunks && n0 + kWidth * chunk(i) < N && row0 < M;
    }

    // Before the tile's accumulator is ready.
    __device__ __forceinline__ void ahead(int n0, int64_t row0) {
        if constexpr (EPI == kGateGrad)
            for (int i = 0; i < 2; ++i)
                if (has(n0, row0, i)) ask(n0, row0, i);
    }

    // The tile's chunks; `release` is called once its last TMEM read is done.
    template <typename Release>
    __device__ __forceinline__ bool tile(uint32_t tacc, int n0, int64_t row0, Release&& release) {
        if (!has(n0, row0, 0)) release();
        for (int i = 0; chunk(i) < kChunks; ++i) {
            const int c = chunk(i), n = n0 + kWidth * c;
            if (!has(n0, row0, i)) break;  // this and the later chunks lie outside the result
            uint32_t r[32];
            float v[32];
            if constexpr (EPI == kGate) {
                uint32_t ru[32];
                float u[32];
                __syncwarp();
                values(tacc, 32 * c, r);
                values(tacc, 128 + 32 * c, ru);
                tmem_ld_wait();
                if (!has(n0, row0, i + 1)) release();
                stores_read<0>();  // one group per chunk, in the same three slots
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    v[j] = __uint_as_float(r[j]);
                    u[j] = __uint_as_float(ru[j]);
                }
                if (p.gate_up_out) {
                    write(slots, v);
                    write(slots + kSlotBytes, u);
                }
                with_act(p.act, [&](auto act) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = activate<decltype(act)::value>(v[j]) * u[j];
                });
                write(slots + 2 * kSlotBytes, v);
                written();
                if (lane == 0) {
                    if (p.gate_up_out) {
                        tma_store_3d(tmG, n, 0, (int32_t)row0, slots);
                        tma_store_3d(tmG, n, 1, (int32_t)row0, slots + kSlotBytes);
                    }
                    tma_store_2d(tmO, n, (int32_t)row0, slots + 2 * kSlotBytes);
                    bulk_commit_group();
                }
            } else if constexpr (EPI == kStore) {
                // rows of 128 bytes (128-byte swizzle) in the two pairs of slots in turn: one store per 64 columns
                uint32_t r2[32];
                __syncwarp();
                values(tacc, 64 * c, r);
                values(tacc, 64 * c + 32, r2);
                tmem_ld_wait();
                if (!has(n0, row0, i + 1)) release();
                const uint32_t slot = slots + 2 * kSlotBytes * (used++ & 1);
                stores_read<1>();
                const uint32_t row = slot + 128u * lane;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t* q = k < 4 ? r + 8 * k : r2 + 8 * (k - 4);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(q[j]);
                    sts_v4(row + 16u * (k ^ (lane & 7)), pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                           pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
                }
                written();
                if (lane == 0) {
                    tma_store_2d(tmO, n, (int32_t)row0, slot);
                    bulk_commit_group();
                }
            } else {
                __syncwarp();
                values(tacc, 32 * c, r);
                tmem_ld_wait();
                if (!has(n0, row0, i + 1)) release();
                const int pair = used % 3;
                const bool ok = mbar_wait(bars + 8u * pair, (uint32_t)(used / 3) & 1u, abort_flag);
                if (__any_sync(0xffffffffu, !ok)) return false;
                ++used;
                const uint32_t slot = slots + kSlotBytes * (2 * pair);
                with_act(p.act, [&](auto act) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float g[8], u[8];
                        unpack8(lds_v4(piece(slot, k)), g);
                        unpack8(lds_v4(piece(slot + kSlotBytes, k)), u);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float d = __uint_as_float(r[8 * k + j]);
                            float a, da;
                            activate_grad<decltype(act)::value>(g[j], a, da);
                            g[j] = d * u[j] * da;
                            u[j] = d * a;
                        }
                        sts_v4(piece(slot, k), pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]),
                               pack_bf16x2(g[4], g[5]), pack_bf16x2(g[6], g[7]));
                        sts_v4(piece(slot + kSlotBytes, k), pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]),
                               pack_bf16x2(u[4], u[5]), pack_bf16x2(u[6], u[7]));
                    }
                });
                written();
                if (lane == 0) {
                    tma_store_3d(tmO, n, 0, (int32_t)row0, slot);
                    tma_store_3d(tmO, n, 1, (int32_t)row0, slot + kSlotBytes);
                    bulk_commit_group();
                }
                if (has(n0, row0, i + 2)) ask(n0, row0, i + 2);
            }
        }
        return true;
    }

    // Every load has landed and every store has been read when the warp leaves.
    __device__ __forceinline__ void finish() {
        if constexpr (EPI == kGateGrad)
            for (; used < asked; ++used) mbar_wait(bars + 8u * (used % 3), (uint32_t)(used / 3) & 1u, nullptr, 200000000ull);
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
    }
};

// AMN / BMN: the operand is MN-major (its reduction runs over rows). A cluster
// holds `splits` pairs; with one, pairs walk the tiles, with more, a cluster
// has one tile and each pair a part of its reduction.
template <bool AMN, bool BMN, int EPI>
__global__ void __launch_bounds__(kThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmG,
                    const __grid_constant__ CUtensorMap tmA1, const __grid_constant__ CUtensorMap tmB1,
                    const __grid_constant__ CUtensorMap tmO1, const GemmParams p) {
    constexpr int kStages = Smem<EPI>::kStages, kSlots = Smem<EPI>::kSlots;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t staging = base + Smem<EPI>::kRing;
    const uint32_t bars = staging + kEpiWarps * kSlots * kSlotBytes;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (kStages + s); };
    auto tfull = [&](int b) { return bars + 8u * (2 * kStages + b); };
    auto tempty = [&](int b) { return bars + 8u * (2 * kStages + 2 + b); };
    const uint32_t drain = bars + 8u * (2 * kStages + 4);
    const uint32_t loads = drain + 8u;  // kGateGrad: 3 per epilogue warp
    uint8_t* tail = smem_raw + (loads - raw) + 8u * 3 * kEpiWarps;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(tail);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = (int)cluster_rank();
    const int prank = crank & 1, leader = crank & ~1, srank = crank >> 1;
    const int cluster = cluster_id(), clusters = cluster_count();
    const int tiles = p.tiles, first = cluster < p.early ? cluster : p.head + cluster;

    // The setup runs once per tile when there are few: the lanes of a warp
    // write the barriers together, nothing is divided, nothing released that
    // nobody reads (2,000 cycles before the first load became 500).
    if (warp == 0) {
        for (int i = lane; i < 2 * kStages + 5 + 3 * kEpiWarps; i += 32) {
            const bool te = i == 2 * kStages + 2 || i == 2 * kStages + 3;  // tempty: the epilogue warps of both CTAs
            mbar_init(bars + 8u * i, te ? 2 * kEpiWarps : 1);
        }
        if (lane == 0) *abort_flag = 0;
        fence_mbarrier_init();
    } else if (warp == 2 && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmO);
    }
    // First cluster barrier: the barriers exist (all that the producers need).
    // Second: the TMEM of both CTAs does; it is allocated while the first loads
    // are on their way.
    __syncwarp();
    cluster_arrive_relaxed();
    if (warp == 1) {
        tmem_alloc_pair(smem_u32((const void*)tmem_slot), kTmemCols);
        tc_fence_before();
        cluster_wait();
        cluster_arrive();
    } else {
        cluster_wait();
        cluster_arrive_relaxed();
    }
    // The first product of a call waits here, and lets the next one start only
    // then: that one may read its weights before it waits itself. (In the others
    // the producer waits; nothing else reads what the grid before writes. With a
    // grid to come that does not wait for this one, it lets that one start, too.)
    if (p.after == kFirst) grid_wait_previous();
    if (!p.late) grid_launch_next();
    int kb = 0, ke = p.k_tiles;
    if (p.splits > 1) {
        kb = p.k_tiles * srank / p.splits;
        ke = p.k_tiles * (srank + 1) / p.splits;
    }

    const int quad = warp & 3, half = (warp - 2) >> 2;
    Epi<EPI> epi{p,
                 &tmO,
                 &tmG,
                 staging + (uint32_t)(warp - 2) * kSlots * kSlotBytes,
                 loads + 24u * (warp - 2),
                 base,
                 lane,
                 quad,
                 half,
                 prank,
                 srank,
                 0,
                 0,
                 abort_flag};

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0, issued = 0, par = 0;
            bool ok = true;
            if (p.after == kAfter) grid_wait_previous();
            if (p.late) grid_launch_next();
            for (int tile = first; ok && tile < tiles; tile += tile < p.head ? p.early : clusters) {
                int mt, nt;
                const int job = tile_at(p, tile, mt, nt);
                const CUtensorMap *mapA = AMN && job ? &tmA1 : &tmA, *mapB = AMN && job ? &tmB1 : &tmB;
                const int a0 = mt * 256 + prank * 128;
                // kGate: the even CTA brings the tile's 128 gate rows, the odd one its up rows
                const int b0 = EPI == kGate ? prank * p.F + nt * 128 : nt * 256 + prank * 128;
                for (int kt = kb; kt < ke; ++kt) {
                    if (!mbar_wait(empty(s), ph ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = base + s * kStageBytes, sb = sa + kHalfBytes;
                    const uint32_t bar = map_to_rank(full(s), leader);
                    if (prank == 0) mbar_arrive_expect_tx(full(s), 2 * kStageBytes);
                    if constexpr (AMN) {
                        tma_load_2d_pair(sa, mapA, a0, kt * kBK, bar);
                        tma_load_2d_pair(sa + kChunkBytes, mapA, a0 + 64, kt * kBK, bar);
                    } else {
                        tma_load_2d_pair(sa, mapA, kt * kBK, a0, bar);
                    }
                    if constexpr (BMN) {
                        tma_load_2d_pair(sb, mapB, b0, kt * kBK, bar);
                        tma_load_2d_pair(sb + kChunkBytes, mapB, b0 + 64, kt * kBK, bar);
                    } else {
                        tma_load_2d_pair(sb, mapB, kt * kBK, b0, bar);
                    }
                    issued |= 1u << s;
                    par = (par & ~(1u << s)) | (ph << s);
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok && prank == 0)  // copies in flight (both CTAs') land before the pair leaves
                for (int q = 0; q < kStages; ++q)
                    if (issued & (1u << q)) mbar_wait(full(q), (par >> q) & 1u, nullptr, 200000000ull);
        }
        __syncwarp();
        cluster_wait();
    } else if (warp == 1) {
        cluster_wait();
        tc_fence_after();
        const uint32_t tmem = *tmem_slot;
        // ---------------------------------------------------------- MMA issuer
        if (lane == 0 && prank == 0) {
            const uint32_t idesc = idesc_bf16(256, 256, AMN, BMN);
            const uint64_t ad = operand_desc<AMN>(base), bd = operand_desc<BMN>(base + kHalfBytes);
            const uint32_t both = 3u << leader;
            int s = 0, local = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int tile = first; ok && tile < tiles; tile += tile < p.head ? p.early : clusters, ++local) {
                const int b = local & 1;
                if (!mbar_wait(tempty(b), (((uint32_t)local >> 1) & 1u) ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                for (int kt = kb; kt < ke; ++kt) {
                    if (!mbar_wait(full(s), ph, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = s * kStageBytes;
#pragma unroll
                    for (int j = 0; j < kBK / 16; ++j)
                        mma_bf16_pair(tmem + 256u * b, desc_at(ad, at + kSlice<AMN> * j), desc_at(bd, at + kSlice<BMN> * j),
                                      idesc, kt != kb || j != 0);
                    mma_commit_pair(empty(s), both);
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (ok) mma_commit_pair(tfull(b), both);
            }
            if (!ok) {
                mma_commit_pair(drain, both);
                mbar_wait(drain, 0, nullptr, 200000000ull);
            }
        }
        __syncwarp();
    } else {
        cluster_wait();
        tc_fence_after();
        const uint32_t tmem = *tmem_slot;
        // ------------------------------------------------------------ epilogue
        int local = 0;
        for (int tile = first; tile < tiles; tile += tile < p.head ? p.early : clusters, ++local) {
            const int b = local & 1;
            int mt, nt;
            const int job = tile_at(p, tile, mt, nt);
            epi.M = job ? p.r[1].M : p.r[0].M;
            epi.N = job ? p.r[1].N : p.r[0].N;
            if (AMN) epi.tmO = job ? &tmO1 : &tmO;
            const int n0 = nt * (EPI == kGate ? 128 : 256);
            const int64_t row0 = (int64_t)mt * 256 + prank * 128 + quad * 32;
            epi.ahead(n0, row0);
            const bool ok = mbar_wait(tfull(b), ((uint32_t)local >> 1) & 1u, abort_flag);
            if (__any_sync(0xffffffffu, !ok)) break;
            tc_fence_after();
            const uint32_t tacc = tmem + ((uint32_t)(quad * 32) << 16) + 256u * b;
            if (p.splits > 1) {
                epi.share(tacc);  // the ring is free: this was the cluster's only tile
                tc_fence_before();
                continue;
            }
            const bool done = epi.tile(tacc, n0, row0, [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(map_to_rank(tempty(b), leader));
            });
            if (!done) break;
        }
    }

    if (p.splits > 1) {
        __syncthreads();
        cluster_sync();  // every pair's partial sums are in place
        if (warp >= 2 && *abort_flag == 0) {
            int mt, nt;
            tile_at(p, first, mt, nt);
            epi.tile(0, nt * (EPI == kGate ? 128 : 256), (int64_t)mt * 256 + prank * 128 + quad * 32, [] {});
        }
    }
    if (warp >= 2) epi.finish();

    // --------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) record_status(p.status, MLA_ERR_TIMEOUT);
    cluster_sync();  // no CTA leaves while another may still signal it or read its sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(*tmem_slot, kTmemCols);
    }
    if (p.after == kBeside) grid_wait_previous();
}

// Clusters of `splits` pairs that can be resident at once (a GPC may hold a
// number of SMs that clusters do not divide).
template <bool AMN, bool BMN, int EPI>
int resident_clusters(const DeviceInfo& di, int splits, int* out) {
    static std::mutex mu;
    static int cache[64][kMaxSplits + 1];
    std::lock_guard<std::mutex> lock(mu);
    int& n = cache[di.device][splits];
    if (n == 0) {
        const auto k = (const void*)ffn_gemm_kernel<AMN, BMN, EPI>;
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Smem<EPI>::kBytes) != cudaSuccess)
            return MLA_ERR_CUDA;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)(di.num_sms / (2 * splits) * 2 * splits));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Smem<EPI>::kBytes;
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = 2u * splits;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        int got = 0;
        if (cudaOccupancyMaxActiveClusters(&got, k, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            got = 0;
        }
        n = got > 0 ? got : -1;
    }
    *out = n;
    return n > 0 || splits > 1 ? MLA_OK : MLA_ERR_CUDA;
}

// ------------------------------------------------------------ few tokens
// With few tokens a product reads its weights once and does little else: the
// bound is HBM. The operands change places, 128 weight rows are the M of a
// tcgen05.mma and all T tokens (padded to N, a multiple of 16) its N, so the
// weights stream through every SM's ring of TMA stages and are padded by
// nothing. The reduction is split over a cluster of S CTAs (S so that all SMs
// stream); their float32 sums meet in distributed shared memory and are added
// in rank order, so results do not depend on scheduling. A product that follows
// another (y after h) starts under it: it fills its ring with weights first and
// waits for the other grid only before it reads the tokens.
// kGate: 64 gate rows and the same channels' 64 up rows make the 128.
// Warps: 0 producer, 1 MMA issuer, 2-5 read TMEM; all six add and store.
constexpr int kNarrowThreads = 192;
constexpr int kNarrowMax = 128;                       // tokens
constexpr uint32_t kNarrowABytes = 128u * 128u;       // 128 weight rows of one K step
constexpr size_t kNarrowRing = 108 * 1024;            // two CTAs fit an SM

struct NarrowParams {
    int T, N, R;              // tokens, tokens of a tile (a multiple of 16), weight rows (kGate: channels)
    int token_tiles;
    int k_tiles, stages, splits;
    uint32_t stage_bytes, tmem_cols;
    int after;                // kFirst or kAfter: the tokens come from the grid before this one
    int late;                 // as in GemmParams
    int F, act;
    uint16_t* out;
    uint16_t* gate_up_out;
    const uint16_t* gate_up;
    int* status;
};

__device__ __forceinline__ void store4(uint16_t* p, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void load4(const uint16_t* p, float (&v)[4]) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    v[0] = bf16lo_to_f32(w.x);
    v[1] = bf16hi_to_f32(w.x);
    v[2] = bf16lo_to_f32(w.y);
    v[3] = bf16hi_to_f32(w.y);
}

template <bool AMN, int EPI>
__global__ void __launch_bounds__(kNarrowThreads)
    ffn_narrow_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const NarrowParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t bars = base + p.stages * p.stage_bytes;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (p.stages + s); };
    const uint32_t done = bars + 16u * p.stages, drain = done + 8u;
    uint8_t* tail = smem_raw + (done - raw) + 16u;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(tail);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.splits > 1 ? (int)cluster_rank() : 0;
    const int tile = cluster_id() / p.token_tiles, t0 = (cluster_id() - tile * p.token_tiles) * p.N;
    const int kb = p.splits > 1 ? p.k_tiles * rank / p.splits : 0;
    const int steps = (p.splits > 1 ? p.k_tiles * (rank + 1) / p.splits : p.k_tiles) - kb;
    const int r0 = tile * (EPI == kGate ? 64 : 128);

    // weights that one token tile reads are gone after it
    const uint64_t weights_once = p.token_tiles == 1 ? l2_evict_first_policy() : l2_evict_last_policy();
    auto load_a = [&](int i, int s) {
        const uint32_t sa = base + s * p.stage_bytes;
        const int k = (kb + i) * kBK;
        mbar_arrive_expect_tx(full(s), p.stage_bytes);
        if constexpr (EPI == kGate) {
            tma_load_2d_hint(sa, &tmA, k, r0, full(s), weights_once);
            tma_load_2d_hint(sa + kNarrowABytes / 2, &tmA, k, p.F + r0, full(s), weights_once);
        } else if constexpr (AMN) {
            tma_load_2d_hint(sa, &tmA, r0, k, full(s), weights_once);
            tma_load_2d_hint(sa + kChunkBytes, &tmA, r0 + 64, k, full(s), weights_once);
        } else {
            tma_load_2d_hint(sa, &tmA, k, r0, full(s), weights_once);
        }
    };
    auto load_b = [&](int i, int s) {
        tma_load_2d(base + s * p.stage_bytes + kNarrowABytes, &tmB, (kb + i) * kBK, t0, full(s));
    };
    const int ahead = steps < p.stages ? steps : p.stages;

    if (p.after == kFirst) grid_wait_previous();  // before grid_launch_next(): see ffn_gemm_kernel
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(done, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
        for (int i = 0; i < ahead; ++i) load_a(i, i);  // under the rest of the setup
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc(smem_u32((const void*)tmem_slot), p.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (!p.late) grid_launch_next();

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            if (p.after == kAfter) grid_wait_previous();
            if (p.late) grid_launch_next();
            for (int i = 0; i < ahead; ++i) load_b(i, i);
            bool ok = true;
            int s = 0;
            uint32_t ph = 0;  // of the stage's first refill
            int i = ahead;
            for (; i < steps; ++i) {
                if (!mbar_wait(empty(s), ph, abort_flag)) {
                    ok = false;
                    break;
                }
                load_a(i, s);
                load_b(i, s);
                if (++s == p.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (!ok)  // copies in flight land before the CTA leaves: the last fill of each stage is one of
                for (int j = i > p.stages ? i - p.stages : 0; j < i; ++j)
                    mbar_wait(full(j % p.stages), (uint32_t)(j / p.stages) & 1u, nullptr, 200000000ull);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issuer
        if (lane == 0) {
            const uint32_t idesc = idesc_bf16(128, (uint32_t)p.N, AMN, 0), stage_bytes = p.stage_bytes;
            const uint64_t ad = operand_desc<AMN>(base), bd = operand_desc<false>(base + kNarrowABytes);
            const int stages = p.stages;
            uint32_t at = 0;
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int i = 0; i < steps; ++i) {
                if (!mbar_wait(full(s), ph, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < kBK / 16; ++j)
                    mma_bf16(tmem, desc_at(ad, at + kSlice<AMN> * j), desc_at(bd, at + kSlice<false> * j), idesc,
                             (i | j) != 0);
                mma_commit(empty(s));
                at += stage_bytes;
                if (++s == stages) {
                    s = 0;
                    at = 0;
                    ph ^= 1u;
                }
            }
            mma_commit(ok ? done : drain);
            if (!ok) mbar_wait(drain, 0, nullptr, 200000000ull);
        }
        __syncwarp();
    } else {
        // partial sums to shared memory (the ring is free once every MMA is done): [token][128 rows]
        const bool ok = mbar_wait(done, 0, abort_flag);
        if (!__any_sync(0xffffffffu, !ok)) {
            tc_fence_after();
            const int quad = warp & 3;
            const uint32_t dst = base + 4u * (quad * 32 + lane);
            for (int c = 0; c < p.N; c += 16) {
                uint32_t v[16];
                __syncwarp();
                tmem_ld16(tmem + ((uint32_t)(quad * 32) << 16) + c, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + 512u * (c + i)), "r"(v[i]) : "memory");
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, p.tmem_cols);
    }
    if (p.splits > 1) cluster_sync();

    // this CTA adds and finishes its share of the tokens
    const int n_tok = p.T - t0 < p.N ? p.T - t0 : p.N;
    const int t_begin = n_tok * rank / p.splits, t_end = n_tok * (rank + 1) / p.splits;
    constexpr int kQuads = EPI == kGate ? 16 : 32;
    const bool failed = *abort_flag != 0;
    for (int i = threadIdx.x; i < (t_end - t_begin) * kQuads && !failed; i += kNarrowThreads) {
        const int tl = t_begin + i / kQuads, t = t0 + tl, q = i % kQuads, r = r0 + 4 * q;
        if (r >= p.R) continue;
        const uint32_t at = base + 512u * tl + 16u * q;
        float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < p.splits; ++s) {
            const uint32_t from = p.splits > 1 ? map_to_rank(at, s) : at;
            const float4 v = ld_cluster_v4(from);
            a[0] += v.x;
            a[1] += v.y;
            a[2] += v.z;
            a[3] += v.w;
            if constexpr (EPI == kGate) {
                const float4 w = ld_cluster_v4(from + 256u);
                b[0] += w.x;
                b[1] += w.y;
                b[2] += w.z;
                b[3] += w.w;
            }
        }
        if constexpr (EPI == kGate) {
            float h[4];
            with_act(p.act, [&](auto act) {
#pragma unroll
                for (int j = 0; j < 4; ++j) h[j] = activate<decltype(act)::value>(a[j]) * b[j];
            });
            store4(p.out + (int64_t)t * p.F + r, h);
            if (p.gate_up_out) {
                store4(p.gate_up_out + (int64_t)t * 2 * p.F + r, a);
                store4(p.gate_up_out + (int64_t)t * 2 * p.F + p.F + r, b);
            }
        } else if constexpr (EPI == kGateGrad) {
            float g[4], u[4], dg[4], du[4];
            load4(p.gate_up + (int64_t)t * 2 * p.F + r, g);
            load4(p.gate_up + (int64_t)t * 2 * p.F + p.F + r, u);
            with_act(p.act, [&](auto act) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float v, dv;
                    activate_grad<decltype(act)::value>(g[j], v, dv);
                    dg[j] = a[j] * u[j] * dv;
                    du[j] = a[j] * v;
                }
            });
            store4(p.out + (int64_t)t * 2 * p.F + r, dg);
            store4(p.out + (int64_t)t * 2 * p.F + p.F + r, du);
        } else {
            store4(p.out + (int64_t)t * p.R + r, a);
        }
    }

    // --------------------------------------------------------------- teardown
    if (threadIdx.x == 0 && failed) record_status(p.status, MLA_ERR_TIMEOUT);
    if (p.splits > 1) {  // the others have read this CTA's sums
        cluster_arrive_relaxed();
        cluster_wait();
    }
}

struct Operand {
    const void* p;
    int64_t rows, cols, ld;  // as stored, ld in elements
};

// C = A B^T over `red` elements. A is [M, red] (or [red, M] when AMN), B is
// [N, red] (or [red, N]); kGate's B holds the gate rows, then the up rows.
struct Product {
    Operand a, b;
    int64_t M, N;
    void* out;
};

int64_t pair_tiles(int64_t M, int64_t N) { return ((M + 255) / 256) * ((N + 255) / 256); }

// The pairs that a grid leaves idle in its last wave, and for how many K steps.
struct Idle {
    int64_t pairs = 0, steps = 0;
};

// How many tiles each of the idle pairs takes before the others come, so that
// all end soonest. cost: K steps of a tile.
int64_t tiles_ahead(int64_t tiles, int64_t clusters, const Idle& idle, int64_t cost) {
    int64_t best = 0, best_end = INT64_MAX;
    for (int64_t n = 0; n * idle.pairs <= tiles && n * cost <= idle.steps + 2 * cost; ++n) {
        const int64_t shared = tiles - n * idle.pairs, each = shared / clusters, more = shared % clusters;
        const int64_t first = (n + each + (more > 0)) * cost - idle.steps;
        const int64_t others = (each + (more > idle.pairs)) * cost;
        const int64_t end = first > others ? first : others;
        if (end < best_end) {
            best_end = end;
            best = n;
        }
        if (idle.pairs == 0) break;
    }
    return best;
}

// One product, or (AMN) two over the same reduction. `beside`: tiles of a
// product that could have been in the launch and is not; it counts where the
// split is chosen, so a gradient's bits do not depend on which others are asked
// for. leaves (out): the next grid runs beside this one; idle: what the grid
// before left (kBeside). Blocks start in their order, so the first ones get the
// idle pairs and take tiles before the others come (both gradients' calls against
// equal shares after dx: T = 777, K = 1536, F = 4096, 28 pairs idle for 76 steps,
// 67.1 -> 59.0 us; T = 3000, K = 2048, F = 8192 402 -> 360; T = 4096, K = 4096,
// F = 14336 1593 -> 1522; T = 8192, K = 1024, F = 2816, no time for one, 184-191
// either way).
template <bool AMN, bool BMN, int EPI>
int gemm(const Product* jobs, int count, GemmParams p, int64_t red, After after, const DeviceInfo& di,
         cudaStream_t stream, int64_t beside = 0, Idle* leaves = nullptr, const Idle* idle = nullptr, bool tail = false) {
    int64_t tiles = 0;
    for (int j = 0; j < count; ++j) {
        Result& r = p.r[j];
        r.M = (int)jobs[j].M;
        r.N = (int)jobs[j].N;
        r.m_tiles = (r.M + 255) / 256;
        r.n_tiles = EPI == kGate ? (r.N + 127) / 128 : (r.N + 255) / 256;
        tiles += (int64_t)r.m_tiles * r.n_tiles;
        if (j == 0) p.tiles0 = (int)tiles;
    }
    if (tiles > kI32Max / 8) return MLA_ERR_UNSUPPORTED;
    p.tiles = (int)tiles;
    p.k_tiles = (int)((red + kBK - 1) / kBK);
    p.after = after;
    // Split the reduction when the tiles leave pairs idle: in K steps, a pair's
    // time is its share of them plus what the exchange of the sums costs. With
    // `tail`, the tiles of a last wave that is nearly empty are split too, in a
    // grid of their own beside the others (forward, T = 1100, K = F = 4096 103 ->
    // 93 us; T = 256, K = 4096, F = 11008 75.8 -> 72.5; T = 512, K = 2048, F =
    // 10240, whose 32 steps are too few for it, 63 -> 65). Not for dx: there the
    // weights' gradients fill the idle pairs.
    int clusters = 0, tail_splits = 0;
    int64_t best = 0, pairs = 0, last = 0;
    for (int s = 1; s <= kMaxSplits; ++s) {
        int n = 0;
        const int st = resident_clusters<AMN, BMN, EPI>(di, s, &n);
        if (st != MLA_OK) return st;
        const int64_t all = tiles + beside;
        if (s == 1) {
            pairs = n;
            last = all % n;
        } else if (tail && all > pairs && last && last <= n && p.k_tiles >= 4 * s) {
            const int64_t cost = (p.k_tiles + s - 1) / s + kSplitSteps + kTailSteps;
            if (cost < (tail_splits ? best : (int64_t)p.k_tiles)) {
                best = cost;
                tail_splits = s;
            }
        }
        if (s > 1 && (all > n || p.k_tiles < 4 * s)) continue;
        const int64_t cost = s == 1 ? (all + n - 1) / n * p.k_tiles : (p.k_tiles + s - 1) / s + kSplitSteps;
        if (s == 1 || cost < best) {
            best = cost;
            p.splits = s;
            clusters = tiles < n ? (int)tiles : n;
        }
    }
    if (leaves) {
        p.late = 1;
        last = tiles * p.splits % pairs;
        leaves->pairs = last ? pairs - last : 0;
        leaves->steps = p.splits > 1 ? p.k_tiles / p.splits + kSplitSteps : p.k_tiles;
    }
    if (idle && p.splits == 1 && idle->pairs < clusters) {
        const int64_t ahead = tiles_ahead(tiles, clusters, *idle, p.k_tiles + kTileSteps);
        p.early = ahead ? (int)idle->pairs : 0;
        p.head = (int)(ahead * idle->pairs);
    }
    alignas(64) CUtensorMap ta[2]{}, tb[2]{}, to[2]{}, tg{};
    const uint64_t F = (uint64_t)p.F, T = (uint64_t)jobs[0].M;
    for (int j = 0; j < count; ++j) {
        const Operand &a = jobs[j].a, &b = jobs[j].b;
        const uint64_t M = (uint64_t)jobs[j].M, N = (uint64_t)jobs[j].N;
        int st = make_tmap_2d(&ta[j], a.p, 1, (uint64_t)a.cols, (uint64_t)a.rows, (uint64_t)a.ld * 2, 64,
                              AMN ? kBK : 128, true);
        if (st == MLA_OK)
            st = make_tmap_2d(&tb[j], b.p, 1, (uint64_t)b.cols, (uint64_t)b.rows, (uint64_t)b.ld * 2, 64,
                              BMN ? kBK : 128, true);
        if (st == MLA_OK)
            st = EPI == kGateGrad ? make_tmap_3d(&to[j], jobs[j].out, F, 2, T, 2 * F, 4 * F, 32, 1, 32, true)
                                  : make_tmap_2d(&to[j], jobs[j].out, 1, N, M, N * 2, EPI == kStore ? 64 : 32, 32,
                                                 EPI == kStore, true);
        if (st != MLA_OK) return st;
    }
    const void* gu = EPI == kGateGrad ? p.gate_up : p.gate_up_out;
    if (EPI != kStore && gu) {
        const int st = make_tmap_3d(&tg, gu, F, 2, T, 2 * F, 4 * F, 32, 1, 32, true);
        if (st != MLA_OK) return st;
    }
    auto launch = [&](const GemmParams& q, int64_t n) {
        return launch_overlapped(ffn_gemm_kernel<AMN, BMN, EPI>, (unsigned)(2 * q.splits * n), kThreads,
                                 Smem<EPI>::kBytes, 2u * q.splits, stream, ta[0], tb[0], to[0], tg, ta[1], tb[1], to[1],
                                 q);
    };
    if (!tail_splits) return launch(p, clusters);
    GemmParams whole = p, rest = p;
    whole.tiles = rest.head = (int)(tiles - last);
    whole.late = 1;
    rest.splits = tail_splits;
    rest.after = kBeside;
    const int st = launch(whole, clusters);
    return st == MLA_OK ? launch(rest, last) : st;
}

// Whether a product of T tokens and `rows` weight rows (kGate: channels) takes
// the few-token kernel. Up to 128 tokens the bound is reading the weights; up
// to three of its token tiles it serves as a kernel of smaller tiles while they
// fill half the SMs at most (T = 260, K = 1024, F = 2048: forward 16.8 against
// 18.7 us, backward 24.9 against 28.0; T = 384, K = 2048, F = 800: 17.6 and 18.3,
// 25.5 and 30.4; with all SMs full T = 200, K = 2048, F = 5632 backward 61.1
// against 58.4). Beyond, the pairs' larger tiles win even where they are few (T =
// 512, K = 2048, F = 512: 16.9 against 20.1, 22.1 against 24.2).
template <int EPI>
bool few_tokens(int64_t T, int64_t rows, const DeviceInfo& di) {
    if (T <= kNarrowMax) return true;
    const int64_t tiles = EPI == kGate ? (rows + 63) / 64 : (rows + 127) / 128;
    return T <= 3 * kNarrowMax && 2 * tiles * ((T + kNarrowMax - 1) / kNarrowMax) <= di.num_sms;
}

// The same product for few tokens (see ffn_narrow_kernel): w is [R, red] (or
// [red, R] when AMN), tokens [T, red]. after: the tokens are the output of the
// launch before this one.
template <bool AMN, int EPI>
int narrow(const Product& job, const GemmParams& g, int64_t red, After after, const DeviceInfo& di, cudaStream_t stream,
           bool late = false) {
    const Operand &w = job.b, &tokens = job.a;
    NarrowParams p{};
    p.T = (int)job.M;
    p.token_tiles = (p.T + kNarrowMax - 1) / kNarrowMax;
    p.N = ((p.T + p.token_tiles - 1) / p.token_tiles + 15) / 16 * 16;
    p.R = (int)job.N;
    p.F = g.F;
    p.act = g.act;
    p.out = static_cast<uint16_t*>(job.out);
    p.gate_up_out = g.gate_up_out;
    p.gate_up = g.gate_up;
    p.status = g.status;
    p.after = after;
    p.late = late;
    p.k_tiles = (int)((red + kBK - 1) / kBK);
    p.stage_bytes = kNarrowABytes + 128u * p.N;
    p.stages = (int)(kNarrowRing / p.stage_bytes);
    p.tmem_cols = 32;
    while ((int)p.tmem_cols < p.N) p.tmem_cols *= 2;
    const int tiles = EPI == kGate ? (p.R + 63) / 64 : (p.R + 127) / 128;
    p.splits = 1;
    const int64_t ctas = (int64_t)tiles * p.token_tiles;
    if (ctas > kI32Max / 8) return MLA_ERR_UNSUPPORTED;
    while (p.splits < 8 && ctas * p.splits < di.num_sms && p.k_tiles >= 4 * p.splits) p.splits *= 2;
    alignas(64) CUtensorMap ta, tb;
    const uint32_t box_rows = AMN ? kBK : (EPI == kGate ? 64 : 128);
    int st = make_tmap_2d(&ta, w.p, 1, (uint64_t)w.cols, (uint64_t)w.rows, (uint64_t)w.ld * 2, 64, box_rows, true);
    if (st == MLA_OK)
        st = make_tmap_2d(&tb, tokens.p, 1, (uint64_t)tokens.cols, (uint64_t)tokens.rows, (uint64_t)tokens.ld * 2, 64,
                          (uint32_t)p.N, true);
    if (st != MLA_OK) return st;
    const auto kernel = ffn_narrow_kernel<AMN, EPI>;
    const size_t smem = 1024 + kNarrowRing + 512;
    static std::atomic<uint64_t> allowed{0};  // devices whose kernel has its shared-memory limit set
    const uint64_t bit = 1ull << di.device;
    if (!(allowed.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
            return MLA_ERR_CUDA;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_overlapped(kernel, (unsigned)(ctas * p.splits), kNarrowThreads, smem, (unsigned)p.splits, stream, ta, tb,
                             p);
}

int check_ffn(const mla_ffn_shape* s) {
    if (!s) return MLA_ERR_INVALID_ARG;
    if (s->T < 0 || s->K <= 0 || s->F <= 0 || s->ld_x < 0 || s->reserved != 0) return MLA_ERR_INVALID_ARG;
    if (s->act < MLA_ACT_SILU || s->act > MLA_ACT_GELU_TANH) return MLA_ERR_INVALID_ARG;
    if (s->T > kI32Max - 512 || s->K > kI32Max / 2 - 512 || s->F > kI32Max / 2 - 512) return MLA_ERR_INVALID_ARG;
    if (s->ld_x != 0 && (s->ld_x < s->K || s->ld_x > ((int64_t)1 << 36) || !inside(s->T, s->ld_x)))
        return MLA_ERR_INVALID_ARG;
    if (s->K % 8 || s->F % 8 || s->ld_x % 8) return MLA_ERR_ALIGNMENT;
    return MLA_OK;
}

}  // namespace
}  // namespace mlaq

using namespace mlaq;

extern "C" {

MLAQ_API int mla_gated_ffn_fwd(const mla_ffn_shape* shape, const void* x, const void* w_gate_up, const void* w_down,
                               void* gate_up, void* h, void* y, int* dev_status, void* stream) {
    int st = check_ffn(shape);
    if (st != MLA_OK) return st;
    const mla_ffn_shape& s = *shape;
    if (s.T > 0 && (!x || !w_gate_up || !w_down || !h || !y)) return MLA_ERR_INVALID_ARG;
    for (const void* q : {x, w_gate_up, w_down, (const void*)gate_up, (const void*)h, (const void*)y})
        if (!aligned(q, 16)) return MLA_ERR_ALIGNMENT;
    if (!aligned(dev_status, 4)) return MLA_ERR_ALIGNMENT;
    const int64_t ld = s.ld_x ? s.ld_x : s.K;
    const Range outs[] = {rng(gate_up, s.T * s.F * 4), rng(h, s.T * s.F * 2), rng(y, s.T * s.K * 2), rng(dev_status, 4)};
    const Range ins[] = {rng(x, s.T ? ((s.T - 1) * ld + s.K) * 2 : 0), rng(w_gate_up, s.F * s.K * 4),
                         rng(w_down, s.F * s.K * 2)};
    if (any_alias(outs, ins)) return MLA_ERR_ALIAS;
    if (s.T == 0) return MLA_OK;
    DeviceInfo di;
    st = current_device_info(&di);
    if (st != MLA_OK) return st;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    GemmParams p{};
    p.F = (int)s.F;
    p.act = s.act;
    p.status = dev_status;
    p.gate_up_out = static_cast<uint16_t*>(gate_up);
    const Product up{{x, s.T, s.K, ld}, {w_gate_up, 2 * s.F, s.K, s.K}, s.T, s.F, h};
    const Product down{{h, s.T, s.F, s.F}, {w_down, s.K, s.F, s.F}, s.T, s.K, y};
    st = few_tokens<kGate>(s.T, s.F, di) ? narrow<false, kGate>(up, p, s.K, kFirst, di, cs)
                       : gemm<false, false, kGate>(&up, 1, p, s.K, kFirst, di, cs, 0, nullptr, nullptr, true);
    if (st != MLA_OK) return st;
    return few_tokens<kStore>(s.T, s.K, di) ? narrow<false, kStore>(down, p, s.F, kAfter, di, cs)
                         : gemm<false, false, kStore>(&down, 1, p, s.F, kAfter, di, cs, 0, nullptr, nullptr, true);
}

MLAQ_API int mla_gated_ffn_bwd(const mla_ffn_shape* shape, const void* dy, const void* x, const void* w_gate_up,
                               const void* w_down, const void* gate_up, const void* h, void* dgate_up, void* dx,
                               void* dw_gate_up, void* dw_down, int* dev_status, void* stream) {
    int st = check_ffn(shape);
    if (st != MLA_OK) return st;
    const mla_ffn_shape& s = *shape;
    const bool hidden = dx || dw_gate_up;  // the gradients that go through the activation
    if (!dx && !dw_gate_up && !dw_down) return MLA_ERR_INVALID_ARG;
    if (s.T > 0) {
        if (!dy || (hidden && (!w_down || !gate_up || !dgate_up)) || (dx && !w_gate_up) || (dw_gate_up && !x) ||
            (dw_down && !h))
            return MLA_ERR_INVALID_ARG;
    }
    for (const void* q : {dy, x, w_gate_up, w_down, gate_up, h, (const void*)dgate_up, (const void*)dx,
                          (const void*)dw_gate_up, (const void*)dw_down})
        if (!aligned(q, 16)) return MLA_ERR_ALIGNMENT;
    if (!aligned(dev_status, 4)) return MLA_ERR_ALIGNMENT;
    const int64_t ld = s.ld_x ? s.ld_x : s.K;
    const Range outs[] = {rng(dgate_up, s.T * s.F * 4), rng(dx, s.T * s.K * 2), rng(dw_gate_up, s.F * s.K * 4),
                          rng(dw_down, s.F * s.K * 2), rng(dev_status, 4)};
    const Range ins[] = {rng(dy, s.T * s.K * 2), rng(x, s.T ? ((s.T - 1) * ld + s.K) * 2 : 0),
                         rng(w_gate_up, s.F * s.K * 4), rng(w_down, s.F * s.K * 2), rng(gate_up, s.T * s.F * 4),
                         rng(h, s.T * s.F * 2)};
    if (any_alias(outs, ins)) return MLA_ERR_ALIAS;
    DeviceInfo di;
    st = current_device_info(&di);
    if (st != MLA_OK) return st;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (s.T == 0) {  // empty sums: the weights' gradients are zero
        if (dw_gate_up && cudaMemsetAsync(dw_gate_up, 0, (size_t)(s.F * s.K * 4), cs) != cudaSuccess) return MLA_ERR_CUDA;
        if (dw_down && cudaMemsetAsync(dw_down, 0, (size_t)(s.F * s.K * 2), cs) != cudaSuccess) return MLA_ERR_CUDA;
        return MLA_OK;
    }
    GemmParams p{};
    p.F = (int)s.F;
    p.act = s.act;
    p.status = dev_status;
    p.gate_up = static_cast<const uint16_t*>(gate_up);
    const Operand oy{dy, s.T, s.K, s.K}, og{dgate_up, s.T, 2 * s.F, 2 * s.F};
    if (hidden) {
        const Product q{oy, {w_down, s.K, s.F, s.F}, s.T, s.F, dgate_up};
        st = few_tokens<kGateGrad>(s.T, s.F, di) ? narrow<true, kGateGrad>(q, p, s.K, kFirst, di, cs)
                           : gemm<false, true, kGateGrad>(&q, 1, p, s.K, kFirst, di, cs, 0, nullptr, nullptr, true);
        if (st != MLA_OK) return st;
    }
    Idle idle;
    const bool dw_beside = dx && (dw_gate_up || dw_down);
    if (dx) {
        const Product q{og, {w_gate_up, 2 * s.F, s.K, s.K}, s.T, s.K, dx};
        st = few_tokens<kStore>(s.T, s.K, di)
                 ? narrow<true, kStore>(q, p, 2 * s.F, kAfter, di, cs, dw_beside)
                 : gemm<false, true, kStore>(&q, 1, p, 2 * s.F, kAfter, di, cs, 0, dw_beside ? &idle : nullptr);
        if (st != MLA_OK) return st;
    }
    Product dw[2];
    int count = 0;
    if (dw_gate_up) dw[count++] = {og, {x, s.T, s.K, ld}, 2 * s.F, s.K, dw_gate_up};
    if (dw_down) dw[count++] = {oy, {h, s.T, s.F, s.F}, s.K, s.F, dw_down};
    const int64_t beside = (dw_gate_up ? 0 : pair_tiles(2 * s.F, s.K)) + (dw_down ? 0 : pair_tiles(s.K, s.F));
    if (count)
        return gemm<true, true, kStore>(dw, count, p, s.T, dw_beside ? kBeside : hidden ? kAfter : kFirst, di, cs, beside,
                                        nullptr, dw_beside ? &idle : nullptr);
    return MLA_OK;
}

}  // extern "C"

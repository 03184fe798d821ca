// Attention over the 8-bit cache: out = softmax(scale q k^T) v with keys and
// values as E4M3 codes and one power-of-two scale per block of tokens.
//
// The codes go to the tensor cores as they are. The query is split into two
// E4M3 numbers instead: with a row scaled to amax in [128, 256), hi = e4m3(q)
// leaves a residual of at most four bits of a bf16 q, so lo = e4m3(32 (q - hi))
// holds the rest and q = hi + lo / 32 exactly (down to 2^-14 of the row's
// largest; below that to 2^-22 of it). Both go by way of f16, whose eleven bits
// are more than the two keep. Probabilities, as f32, are split the same way and
// enter the second product with eight bits, the precision of bf16: the rounding
// of a result to bf16 is as large. So no cached byte is ever converted, and both
// products run at the 8-bit rate.
//
// Both products have the cached tokens as their 128 rows:
//   S^T [128 tokens, 2R] = K [128, Dk] x [q_hi | q_lo]^T   (R query rows)
//   O^T [128 channels, 2R] += V^T [128, 128 tokens] x [p_hi | p_lo]^T
// A query tile is R = 8 to 64 rows, the heads of a group times the new tokens, so
// one token of a few heads costs an N of 16, not an M of 128; a thread owns a
// token: its scales are two registers. V^T is read from the same [token][channel]
// tiles as an MN-major operand; with values in the keys (latents) the keys' tile
// serves both. The scale of K multiplies the score in the thread that owns the
// token, that of V the probability: a weight is p 2^(e - E), E an exponent of the
// warps that share the token's rows.
//
// The reference of a row is its largest s + max(e - E, -90), s the score in powers
// of two: the largest weight, not the largest probability, since weights are what
// the two E4M3 numbers hold. (With the largest s, and E the largest e, a row whose
// probability lies on small values lost them: a block 2^20 larger that it gives no
// weight, or does not even see, took all of its result.) The floor of -90 keeps the
// sum of the probabilities, at most 2^94 each, within float32. Weights may pass the
// reference by 2^4: one vote per tile, and only a tile that passes it pays for
// reductions and for rescaling O in tensor memory; E then becomes the largest e of
// the tokens that passed, and references fall by as much. The factor 2^4 and E4M3's
// range leave the weights ten binades of eight bits below the reference; further
// down they are held in steps of 2^-18 of it. A row keeps its eight bits while a
// block to which another row of its tile gives weight is up to 2^90 larger.
//
// Work is tiles of 128 tokens of all (head, query tile) pairs in one line, cut into
// equal shares, one per SM: lengths live on the device, and a ragged batch or one
// long sequence fills every SM alike. A share's first and last pair may be
// parts; their O (divided by the sum), reference and sum go to the workspace and a
// second kernel adds the parts in the order of the shares.
//
// What bounds it, by calls in a graph:
// - Tokens over keys and values of their own: HBM. 64 sequences of up to 8192
//   tokens, 8 heads of 128 + 128 (608 MB): 104.5 us, 5.8 TB/s, 87% of a copy's rate;
//   in pages of 128 and more 100 us. Pages of 32 and 16 take 114 and 136: a copy's
//   fixed 50 ns. 512 sequences of 1024: 178 us; a piece of eight tiles is too short
//   to hide bringing its queries in and its result out.
// - Latents (576 channels, 512 of them values, 128 query heads): the chain copy (2600
//   clocks) -> first product (1100) -> softmax (1100) -> second product (1300, and
//   600 until it starts), with room for two tiles of 80 KB. 48 sequences of up to 4096:
//   105 us, of which a third is the first queries, the results of parts and
//   their addition; 256 sequences: 366 us, 0.45 PFLOP/s, four blocks reading the
//   same tiles from L2 for 32 rows each.
// - A chunk of 2048 tokens, 128 heads of 192 + 128, over 4096 positions: 1465 us, 587
//   TFLOP/s. The softmax: 128 x 64 scores are 32 a thread, with four conversions for
//   each two of them (the 8-bit pairs), at a quarter of the rate of an addition.
#include <cuda.h>

#include <type_traits>

#include "cache.cuh"
#include "internal.h"
#include "launch.cuh"

namespace mlaq {
namespace {

constexpr int kTokens = 128;           // tokens of a tile
constexpr uint32_t kChunk = 16384;     // 128 tokens x 128 channels
// Sixteen warps: eight for the softmax, two that load codes, one that issues the
// products, one that loads scales and deals out the pieces of work, and four that
// bring a piece's queries in and its result out, beside the tiles of the pieces after
// and before. (A copy holds up the warp that issues it, 50 ns and 2.8 ns per 128-byte
// row: two warps take turns. One alone reads 5.2 TB/s in boxes of 64 rows on all SMs,
// from L2 or not, two 10 from L2.)
constexpr int kSoftWarps = 8, kLoader = 8, kIssuer = 9, kMarker = 10, kLoader2 = 11, kHelper = 12;
constexpr int kThreads = 512, kHelpers = 128;
constexpr int64_t kMaxLength = 0x7FFFFF80;  // whole tiles within an int
constexpr int kMarkTiles = 16;         // tiles whose scales are in shared memory
constexpr int kPieces = 4;             // pieces that are dealt out ahead
constexpr int kPieceReaders = kSoftWarps + 3 + 4;  // warps
// Four softmax warps hold a tile's tokens, a token to a thread. With few query rows
// a tile is a chain of waits, and the two fours take turns (two streams, each with
// its own references, sums and O, joined in the end); with many it is arithmetic,
// and they halve the rows, each with its references and at its own pace. (Two streams
// need O twice, which tensor memory has up to R = 16 for every size. In the version that
// brought them a decode batch went from 205 to 183 us and a chunk, whose fours halve the
// rows, from 7.7 to 2.9 ms, with the weights stored whole per token as the rest of it.)
template <int R>
constexpr int kStreams = R <= 16 ? 2 : 1;
constexpr float kPass = 4.f;           // log2 of how far weights may pass the reference
constexpr float kNothing = -3.0e38f;   // the reference of a row that has seen nothing
constexpr int kNoScale = -1000;
constexpr int kFar = -90;              // what a scale counts for that is further below the largest
constexpr float kMostSum = 100.f;      // log2 of what a thread's sums may become where references fall
constexpr int kFailed = 1 << 20;       // among the votes: a wait that gave up
constexpr int kMaxQueryChunks = 5;
constexpr int kCombineThreads = 512, kMaxShares = 256;

// The parts of a share: place 0 of the workspace has the one that begins inside
// its pair of slot and head (it may go on into the next share), place 1 the one
// that begins with its pair and does not end it.
enum { kNoPart = 0, kOpens = 1, kGoesOn = 2, kEnds = 3 };

struct AttnParams {
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    const int32_t *table, *length, *cu;
    const uint8_t *k_scales, *v_scales;
    float* part_o;    // [2 * shares][R][Dv], on 16 bytes
    float2* part_ml;  // [2 * shares][R]
    int4* meta;       // [shares][2]
    int64_t q_t, q_h, T, pages;
    int slots;
    int B, width, page_shift, page, block_shift, marks, H, Hq, group, per_seq, Dk, Dv, nk, nv;
    int k_stages, v_stages, q_bufs, o_bufs, tmem_cols;  // buffers of the keys' tiles, the values', of queries, of O
    uint32_t group_mul, group_shift;      // n / group = n * group_mul >> group_shift for n < 2^31
    int q_vec;
    float scale_log2;
    int* status;
};

// ------------------------------------------------------------- pieces of PTX
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// kind::f8f6f4, E4M3 x E4M3, f32 sums (the fields of idesc_bf16, formats 0)
__host__ __device__ constexpr uint32_t idesc_f8(uint32_t M, uint32_t N, uint32_t mn_major) {
    return (1u << 4) | (mn_major << 15) | (mn_major << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// The probabilities: MN-major without swizzle, [16 query rows of one block][token] of 16 bytes: 8 tokens are a core
// matrix of 128 bytes, the next 8 the next; blocks are 128 tokens apart. A thread stores its token's bytes whole.
__device__ __forceinline__ uint64_t desc_weights(uint32_t saddr) { return smem_desc(saddr, 128, 2048, kLayoutNone); }
// A descriptor `bytes` further on. They are built once and added to: an MMA whose descriptors were built in front of it
// took the issuing thread 170 clocks, so 48 (N <= 64) to 68 (N = 128).
__device__ __forceinline__ uint64_t desc_at(uint64_t desc, uint32_t bytes) {
    return (desc & 0xFFFFFFFF00000000ull) | (uint32_t)((uint32_t)desc + (bytes >> 4));
}
// One lane of a converged warp, the same each time. Code that it alone runs keeps its operands in uniform registers, as
// the MMA and TMA instructions want them; behind lane == 0 they were moved there one by one, 100 clocks of an MMA.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// mbar_wait in few instructions: some thirty waits share the instruction cache with the loop over the tiles (a call in
// place of the loop would put the values that live across it on the stack).
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 15) == 0 && (*abort || globaltimer_ns() - t0 > MLAQ_WAIT_NS)) break;
    }
    *abort = 1;
    return false;
}
// The same with the waiting itself out of line (FAR), for warps that hold few values across it. Which warps' waits are
// out of line was measured for each R, the softmax's and the loaders' never: the issuer's up to R = 16 (64 sequences of 8192
// tokens 104.7 -> 103.4 us; at R = 64 slower, 1497 -> 1509), the helpers' at R = 64 (a chunk of 128 heads 1497 -> 1457;
// at R = 32 nothing).
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort) { return wait(bar, parity, abort); }
template <bool FAR>
__device__ __forceinline__ bool wait_by(uint32_t bar, uint32_t parity, volatile int* abort) {
    if constexpr (FAR) return mbar_try_wait(bar, parity) || wait_on(bar, parity, abort);
    else return wait(bar, parity, abort);
}
__device__ __forceinline__ void tma_load_page(uint32_t dst, const void* map, int c, int place, int h, int page,
                                              uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(c), "r"(place), "r"(h), "r"(page), "r"(bar)
        : "memory");
}
// Columns of a lane, W at a time.
template <int W>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[W]) {
    if constexpr (W == 16) {
        tmem_ld16(taddr, r);
    } else {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
    }
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// ln(2^m sum). A sum may be 2^94 with a reference as far below: its exponent goes to m first. (Out of line, for the loop's
// instructions to stay in their cache: a chunk 1498 us with this and the division below inline, so 1467.)
__device__ __noinline__ float log_sum(float m, float sum) {
    const uint32_t u = __float_as_uint(sum);
    const bool normal = u >= 0x00800000u && u < 0x7F800000u;
    if (normal) m += (float)((int)(u >> 23) - 127);
    return (m + log2f(normal ? __uint_as_float((u & 0x7FFFFFu) | 0x3F800000u) : sum)) * 0.693147180559945309f;
}
// The largest of the warp's values (NaN counts for nothing).
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Which of two phases completes first (the first where both have): 0 or 1, or -1 when neither does in time.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ int wait_either(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1, volatile int* abort) {
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    for (uint32_t it = 1;; ++it) {
        if (mbar_test(bar0, parity0)) return 0;
        if (mbar_test(bar1, parity1)) return 1;
        if ((it & 63) == 0 && (*abort || globaltimer_ns() - t0 > MLAQ_WAIT_NS)) break;
    }
    *abort = 1;
    return -1;
}
// Two f32 operations in one instruction.
__device__ __forceinline__ void fma2(float& r0, float& r1, float a0, float a1, float b0, float b1, float c0, float c1) {
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r0), "=f"(r1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mul2(float& r0, float& r1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r0), "=f"(r1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void add2(float& r0, float& r1, float a0, float a1) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(r0), "+f"(r1)
        : "f"(a0), "f"(a1));
}
// Sums of 2N values a lane over the warp: at each step a lane hands half of its values to its partner and keeps the sums
// of the others. l[0] becomes the sum of the values whose number is returned.
template <int N, int O, int M>
__device__ __forceinline__ int fold_rows(float (&l)[M], int lane) {
    const bool upper = (lane & O) != 0;
    if constexpr (N > 0) {
#pragma unroll
        for (int r = 0; r < N; ++r)
            l[r] = (upper ? l[r + N] : l[r]) + __shfl_xor_sync(0xFFFFFFFFu, upper ? l[r] : l[r + N], O);
    } else {
        l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], O);
    }
    int row = upper ? N : 0;
    if constexpr (O > 1) row += fold_rows<N / 2, O / 2>(l, lane);
    return row;
}
// Two numbers (up to 256) as two E4M3 numbers each: hi, and 32 times what it leaves, by way of f16 (eleven bits, of
// which the two keep eight; of a bf16 number from 2^-14 up, all). The first in bits 0-7.
__device__ __forceinline__ void split8(float x, float y, uint32_t& hi, uint32_t& lo) {
    uint16_t a, b;
    asm("{\n\t.reg .b32 w, h, d, k;\n\t"
        "cvt.rn.f16x2.f32 w, %3, %2;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 %0, w;\n\t"
        "cvt.rn.f16x2.e4m3x2 h, %0;\n\t"
        "sub.rn.f16x2 d, w, h;\n\t"
        "mov.b32 k, 0x50005000;\n\t"  // 32, 32
        "mul.rn.f16x2 d, d, k;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 %1, d;\n\t}"
        : "=&h"(a), "=h"(b)
        : "f"(x), "f"(y));
    hi = a;
    lo = b;
}
__device__ __forceinline__ void sts_v2(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// A query row's token.
__device__ __forceinline__ int token_of(const AttnParams& p, int rho) {
    return (int)((uint64_t)(uint32_t)rho * p.group_mul >> p.group_shift);
}

// ------------------------------------------------------------ work in a line
// A slot is a tile of R query rows of one sequence (row = token * group + head in
// the group); slots of sequence b start at first(b) = cu[b] * group / R + b.
struct Slot {
    int lo;  // the sequence's first row of q
    int b, n, len, rho0, rows, tiles;
};

template <int R>
__device__ __forceinline__ int first_slot(const AttnParams& p, int b) {
    return (int)((int64_t)p.cu[b] * p.group / R) + b;
}

// What slot holds; b: a sequence at or before the slot's. (Out of line, as all that is not done at every tile is kept
// small: what sixteen warps do in one tile's time has to fit into the 32 KB of an SM's instruction cache. When it did
// not, half of all cycles went into fetching instructions.)
template <int R>
__device__ __noinline__ Slot read_slot(const AttnParams& p, int slot, int b) {
    Slot x;
    int j;
    if (p.cu) {
        while (b + 1 < p.B && first_slot<R>(p, b + 1) <= slot) ++b;
        x.lo = p.cu[b];
        const int64_t n = (int64_t)p.cu[b + 1] - x.lo;
        const bool fine = x.lo >= 0 && n >= 0 && x.lo + n <= p.T;
        if (!fine) record_status(p.status, MLA_ERR_INVALID_ARG);
        x.n = fine ? (int)n : 0;
        j = fine ? slot - first_slot<R>(p, b) : 0;
    } else {
        b = slot / p.per_seq;
        j = slot - b * p.per_seq;
        x.lo = b;
        x.n = 1;
    }
    x.b = b;
    const int64_t left = (int64_t)x.n * p.group - (int64_t)j * R;
    x.rho0 = j * R;
    x.rows = j < 0 || left <= 0 ? 0 : left < R ? (int)left : R;
    const int64_t table = (int64_t)p.width << p.page_shift, room = table < kMaxLength ? table : kMaxLength;
    const int len = p.length[b];
    x.len = len < 0 ? 0 : len > room ? (int)room : len;
    if (x.rows > 0 && x.len != len) record_status(p.status, MLA_ERR_POS_RANGE);
    int limit = x.len - x.n + token_of(p, x.rho0 + x.rows - 1) + 1;
    limit = limit < 0 ? 0 : limit > x.len ? x.len : limit;
    x.tiles = x.rows == 0 ? 0 : limit == 0 ? 1 : (limit + kTokens - 1) / kTokens;
    return x;
}

__device__ __noinline__ int64_t divide(int64_t a, int64_t b) { return a / b; }

// A piece of a share: tiles [t0, t1) of a slot and head. t1 == 0: no more.
struct Piece {
    Slot x;
    int h, t0, t1;
};

// A buffer of a ring and its phase.
struct Ring {
    int i = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step(int n) {
        if (++i == n) {
            i = 0;
            phase ^= 1u;
        }
    }
};
constexpr int kMaxStages = 8;

template <int R, bool SHARED>
struct Shared {  // behind the ring, the queries and the probabilities
    uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
    uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2], m_full[kMarkTiles], m_empty[kMarkTiles];
    // by piece: dealt out; its queries; the rows' numbers below; its sums; its O
    uint64_t piece_full[kPieces], piece_empty[kPieces], q_full[2], q_empty[2], rows_full[2], sums_full[2], sums_empty[2];
    uint64_t o_full[2], o_empty[2], drain;
    Piece piece[kPieces];
    uint8_t marks[kMarkTiles][SHARED ? 1 : 2][kTokens];  // a tile's scale bytes, one for each block: keys', values'
    // query rows, by the piece's parity
    alignas(16) int row_at[2][R];                // row of out
    alignas(16) float unit[2][R];                // 2^-exponent of the row
    int limit[2][R];                             // the last position that it sees
    alignas(16) float ref[2][kStreams<R>][R];    // minus the reference of the row's scores
    float sums[2][kStreams<R>][4][R];            // of probabilities, by the four warps
    int top_e[2][2];                             // the exponent E, by the four warps
    int nan_at[2][512];                          // by channel: the first position with a NaN that not every row sees
    int nan_seen[2];
    alignas(16) float out_factor[kStreams<R>][R];
    float factor[kStreams<R>][R];
    float warp_row[kStreams<R>][4][R];
    float warp_l[2][4];
    int vote[2][3];
    uint32_t tmem;
    volatile int abort;
    int64_t scan[kThreads / 32];
    int start_slot;
};
static_assert(sizeof(Shared<32, true>) <= 10240, "latents of five chunks: two tiles, the queries and the rest fill shared memory");

template <int R, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                      const __grid_constant__ AttnParams p) {
    constexpr int N2 = 2 * R, kStreams = mlaq::kStreams<R>, kFour = kSoftWarps / kStreams;  // kFour: warps of a stream
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t v_base = base + p.k_stages * p.nk * kChunk;  // the keys' tiles, then the values'
    const uint32_t q_base = v_base + (SHARED ? 0 : p.v_stages * p.nv * kChunk), q_bytes = p.nk * (N2 * 128);
    const uint32_t p_base = q_base + p.q_bufs * q_bytes;
    Shared<R, SHARED>& sh = *reinterpret_cast<Shared<R, SHARED>*>(smem_raw + (p_base - raw) + 2 * N2 * 128);
    const uint32_t k_full = smem_u32(&sh.k_full[0]), k_empty = smem_u32(&sh.k_empty[0]);
    const uint32_t v_full = smem_u32(&sh.v_full[0]), v_empty = smem_u32(&sh.v_empty[0]);
    const uint32_t s_full = smem_u32(&sh.s_full[0]), s_empty = smem_u32(&sh.s_empty[0]);
    const uint32_t p_full = smem_u32(&sh.p_full[0]), p_empty = smem_u32(&sh.p_empty[0]);
    const uint32_t m_full = smem_u32(&sh.m_full[0]), m_empty = smem_u32(&sh.m_empty[0]);
    const uint32_t piece_full = smem_u32(&sh.piece_full[0]), piece_empty = smem_u32(&sh.piece_empty[0]);
    const uint32_t q_full = smem_u32(&sh.q_full[0]), q_empty = smem_u32(&sh.q_empty[0]);
    const uint32_t rows_full = smem_u32(&sh.rows_full[0]);
    const uint32_t sums_full = smem_u32(&sh.sums_full[0]), sums_empty = smem_u32(&sh.sums_empty[0]);
    const uint32_t o_full = smem_u32(&sh.o_full[0]), o_empty = smem_u32(&sh.o_empty[0]);
    const uint32_t drain = smem_u32(&sh.drain);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // known to be the same in the whole warp
    volatile int* abort_flag = &sh.abort;

    if (tid < kMaxStages) {
        mbar_init(k_full + 8 * tid, 2);
        mbar_init(k_empty + 8 * tid, 1);
        mbar_init(v_full + 8 * tid, 2);
        mbar_init(v_empty + 8 * tid, 1);
    } else if (tid < kMaxStages + kMarkTiles) {
        mbar_init(m_full + 8 * (tid - kMaxStages), 1);
        mbar_init(m_empty + 8 * (tid - kMaxStages), kFour);
    } else if (tid < kMaxStages + kMarkTiles + kPieces) {
        mbar_init(piece_full + 8 * (tid - kMaxStages - kMarkTiles), 1);
        mbar_init(piece_empty + 8 * (tid - kMaxStages - kMarkTiles), kPieceReaders);
    } else if (tid >= 64 && tid < 66) {
        const int i = tid - 64;
        mbar_init(s_full + 8 * i, 1);
        mbar_init(s_empty + 8 * i, kFour);
        mbar_init(p_full + 8 * i, kFour);
        mbar_init(p_empty + 8 * i, 1);
        mbar_init(q_full + 8 * i, 4);
        mbar_init(q_empty + 8 * i, 1);
        mbar_init(rows_full + 8 * i, 4);
        mbar_init(sums_full + 8 * i, kSoftWarps);
        mbar_init(sums_empty + 8 * i, 4);
        mbar_init(o_full + 8 * i, 1);
        mbar_init(o_empty + 8 * i, 4);
        sh.nan_seen[i] = 0;
        sh.vote[i][0] = sh.vote[i][1] = sh.vote[i][2] = 0;
    } else if (tid == 96) {
        mbar_init(drain, 1);
        sh.abort = 0;
        tma_prefetch_desc(&k_map);
        if (!SHARED) tma_prefetch_desc(&v_map);
    }
    fence_mbarrier_init();
    if (warp == kIssuer) {
        tmem_alloc(smem_u32(&sh.tmem), p.tmem_cols);
        tmem_relinquish();
    }
    // columns of the queries past Dk meet zeros of the cache: they have to be numbers
#pragma unroll 1
    for (uint32_t i = tid * 16; i < p.q_bufs * q_bytes; i += kThreads * 16) sts_v4(q_base + i, 0, 0, 0, 0);
    sh.nan_at[0][tid] = sh.nan_at[1][tid] = 0x7FFFFFFF;
    grid_launch_next();
    grid_wait_previous();

    // ------------------------------------------------------------ the share
    const int per_thread = (p.slots + kThreads - 1) / kThreads, my_slot = per_thread * tid;
    int64_t mine = 0;
    int my_b = 0;
    if (my_slot < p.slots) {
        if (p.cu) {  // the last b with first(b) <= my_slot
            int hi = p.B;
            while (hi - my_b > 1) {
                const int mid = (my_b + hi) / 2;
                if (first_slot<R>(p, mid) <= my_slot) my_b = mid;
                else hi = mid;
            }
        }
        int b = my_b;
#pragma unroll 1
        for (int i = my_slot; i < my_slot + per_thread && i < p.slots; ++i) {
            const Slot x = read_slot<R>(p, i, b);
            b = x.b;
            mine += x.tiles;
        }
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) sh.scan[warp] = upto;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int64_t line = lane < kThreads / 32 ? sh.scan[lane] : 0;  // tiles of one head
#pragma unroll
    for (int o = 1; o < kThreads / 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, line, o);
        if (lane >= o) line += v;
    }
    if (warp > 0) upto += __shfl_sync(0xFFFFFFFFu, line, warp - 1);
    line = __shfl_sync(0xFFFFFFFFu, line, kThreads / 32 - 1);
    // equal shares, the first `all % shares` one tile longer
    const int64_t all = line * p.H;
    const int64_t most_shares = gridDim.x, shares = all < most_shares ? all : most_shares;
    const int c = blockIdx.x;
    int tiles = 0, h0 = 0;
    if (c < shares) {
        int64_t each, w0;
        if (all < kI32Max) {
            each = (uint32_t)all / (uint32_t)shares;
            const int more = (int)(all - each * shares);
            w0 = c * each + (c < more ? c : more);
            tiles = (int)each + (c < more);
            h0 = (int)((uint32_t)w0 / (uint32_t)line);
        } else {
            each = divide(all, shares);
            const int64_t more = all - each * shares;
            w0 = c * each + (c < more ? c : more);
            tiles = (int)(each + (c < more));
            h0 = (int)divide(w0, line);
        }
        const int64_t at = w0 - h0 * line;
        if (at >= upto - mine && at < upto) {  // one thread's
            int64_t before = upto - mine;
            int b = my_b;
            for (int i = my_slot;; ++i) {
                const Slot x = read_slot<R>(p, i, b);
                b = x.b;
                if (at < before + x.tiles) {
                    const int t0 = (int)(at - before), n = x.tiles - t0;
                    sh.start_slot = i;
                    sh.piece[0] = Piece{x, h0, t0, t0 + (n < tiles ? n : tiles)};
                    mbar_arrive(piece_full);
                    break;
                }
                before += x.tiles;
            }
        }
    }
    __syncthreads();
    const uint32_t tmem = sh.tmem;
    const uint32_t s_tmem = tmem, o_tmem = tmem + 2 * N2, o_cols = kStreams * p.nv * N2;  // o_cols: of one O buffer
    // Piece i as its readers get it; each warp says that it has read it.
    auto get_piece = [&](int i, Piece& x) {
        const bool ok = wait(piece_full + 8 * (i % kPieces), (uint32_t)(i / kPieces) & 1u, abort_flag);
        x = sh.piece[i % kPieces];
        if (!ok) x.t0 = x.t1 = 0;
        return ok;
    };

    if (warp == kLoader || warp == kLoader2) {
        // --------------------------------------------------------- producers
        // tile t's keys, then tile t - 1's values: the order in which they are used. Each of the two brings every second
        // chunk of 128 channels and arrives at the tile's barrier with its bytes.
        const int odd = warp == kLoader2;
        Ring k_ring, v_ring;
        bool ok = true;
        const int box = p.page < kTokens ? p.page : kTokens, boxes = kTokens / box;
        struct Tile {  // this lane's box of a tile: its page's entry of the table; the tile's first place in its page
            int entry, place, h;
            bool have;
        };
        Piece x;
        int i = 0;
        Tile now{}, before{}, next{};
        int k_filled = 0, v_filled = 0;
        x.t1 = 0;
        int tile = -1;
#pragma unroll 1
        for (int t = -1; t <= tiles && ok && tiles > 0; ++t) {
            if (t + 1 < tiles) {  // the next tile's entry is on its way while this one waits for room
                if (++tile == x.t1) {
                    ok = __all_sync(0xFFFFFFFFu, get_piece(i, x));
                    __syncwarp();  // all have read it: a vote orders no memory
                    if (lane == 0) mbar_arrive(piece_empty + 8 * (i % kPieces));
                    ++i;
                    tile = x.t0;
                }
                const int at = tile * kTokens + lane * box;
                next.have = ok && lane < boxes && at < x.x.len;
                next.entry = next.have ? p.table[(int64_t)x.x.b * p.width + (at >> p.page_shift)] : 0;
                next.place = (tile * kTokens) & (p.page - 1);
                next.h = x.h;
            }
#pragma unroll 1
            for (int values = 0; values < (SHARED ? 1 : 2); ++values) {
                if (values ? t < 1 : t < 0 || t == tiles) continue;
                const CUtensorMap* map = values ? &v_map : &k_map;
                const Tile& k = values ? before : now;
                Ring& ring = values ? v_ring : k_ring;
                const int stages = values ? p.v_stages : p.k_stages, chunks = values ? p.nv : p.nk, tile_no = values ? t - 1 : t;
                const uint32_t full = (values ? v_full : k_full) + 8 * ring.i, empty = (values ? v_empty : k_empty) + 8 * ring.i;
                const int count = __popc(__ballot_sync(0xFFFFFFFFu, k.have));
                const int first = (values ? p.nk + odd : odd) & 1;  // chunks first, first + 2, ...
                int page = k.entry;
                if (page < 0 || page >= p.pages) {
                    record_status(p.status, MLA_ERR_POS_RANGE);
                    page = (int)p.pages;  // reads as zeros
                }
                ok = __all_sync(0xFFFFFFFFu, tile_no < stages || wait(empty, ring.phase ^ 1u, abort_flag));
                if (!ok) break;
                if (elect_one()) mbar_arrive_expect_tx(full, (chunks - first + 1) / 2 * count * box * 128);
                __syncwarp();
                const uint32_t to = (values ? v_base : base) + ring.i * chunks * kChunk;
#pragma unroll 1
                for (int j = first; j < chunks; j += 2)
#pragma unroll 1
                    for (int e = 0; e < count; ++e) {
                        const int from = __shfl_sync(0xFFFFFFFFu, page, e);
                        if (elect_one()) tma_load_page(to + j * kChunk + e * box * 128, map, j * 128, k.place, k.h, from, full);
                    }
                if (values) ++v_filled;
                else ++k_filled;
                ring.step(stages);
            }
            before = now;
            now = next;
        }
        if (!ok && lane == 0) {  // copies in flight land before the block leaves
            for (int j = k_filled > p.k_stages ? k_filled - p.k_stages : 0; j < k_filled; ++j)
                mbar_wait(k_full + 8 * (j % p.k_stages), (uint32_t)(j / p.k_stages) & 1u, nullptr, 200000000ull);
            for (int j = v_filled > p.v_stages ? v_filled - p.v_stages : 0; j < v_filled; ++j)
                mbar_wait(v_full + 8 * (j % p.v_stages), (uint32_t)(j / p.v_stages) & 1u, nullptr, 200000000ull);
        }
        __syncwarp();
    } else if (warp == kIssuer) {
        // -------------------------------------------------------- MMA issuer
        if (tiles > 0 && elect_one()) {
            const uint32_t i_s = idesc_f8(128, N2, 0), i_o = idesc_f8(128, N2, 1);
            const uint64_t dk = desc_kmajor_sw128(base), dv = desc_mnmajor_sw128(SHARED ? base : v_base, kChunk);
            const uint64_t dq = desc_kmajor_sw128(q_base), dw = desc_weights(p_base);
            const int whole = p.Dk / 128, rest = (p.Dk % 128 + 31) / 32;  // chunks of 128 channels, steps of 32 behind them
            Ring k_ring, v_ring;       // the next tiles' buffers
            int tq = 0, tp = 0;        // tiles whose first product, and whose second, was issued
            int i = -1, left = 0, len = 0, len_before = 0;  // the first's piece, its tiles that are left; the piece's length
            int vi = 0, v_at = 0, v_len = 0;                // the second's piece, its tiles so far
            bool ok = true;
            // The first product is up to two tiles ahead. Latents hold both tiles until the second product, so theirs
            // goes first when its weights are there before the next keys are.
            while (tp < tiles && ok) {
                bool scores = tq < tiles && tq - tp < 2;
                if (SHARED && scores && tq > tp) {
                    if (left == 0) {
                        scores = false;  // the next piece's queries may be long in coming
                    } else {
                        const int w = wait_either(k_full + 8 * k_ring.i, k_ring.phase, p_full + 8 * (tp & 1), (uint32_t)(tp >> 1) & 1u, abort_flag);
                        ok = w >= 0;
                        scores = w == 0;
                    }
                    if (!ok) break;
                }
                if (scores) {
                    const uint32_t buf = tq & 1;
                    if (left == 0) {
                        Piece x;
                        ++i;
                        ok = get_piece(i, x);
                        mbar_arrive(piece_empty + 8 * (i % kPieces));
                        len_before = len;
                        len = left = x.t1 - x.t0;
                        const int use = p.q_bufs == 2 ? i >> 1 : i;
                        ok = ok && wait_by<(R <= 16)>(q_full + 8 * (p.q_bufs == 2 ? i & 1 : 0), (uint32_t)use & 1u, abort_flag);
                    }
                    ok = ok && (tq < 2 || wait_by<(R <= 16)>(s_empty + 8 * buf, (uint32_t)((tq >> 1) - 1) & 1u, abort_flag));
                    const uint32_t d = s_tmem + buf * N2, qb = p.q_bufs == 2 ? (i & 1) : 0;
                    ok = ok && wait_by<(R <= 16)>(k_full + 8 * k_ring.i, k_ring.phase, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t qt = qb * q_bytes, at = k_ring.i * p.nk * kChunk;
                    uint32_t add = 0;
#pragma unroll 1
                    for (int j = 0; j < whole; ++j) {
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            mma_f8(d, desc_at(dk, at + 32 * s), desc_at(dq, qt + 32 * s), i_s, s == 0 ? add : 1u);
                        add = 1;
                        qt += N2 * 128;
                        at += kChunk;
                    }
#pragma unroll 1
                    for (int s = 0; s < rest; ++s) {
                        mma_f8(d, desc_at(dk, at), desc_at(dq, qt), i_s, add);
                        add = 1;
                        qt += 32;
                        at += 32;
                    }
                    if (!SHARED) mma_commit(k_empty + 8 * k_ring.i);
                    k_ring.step(p.k_stages);
                    mma_commit(s_full + 8 * buf);
                    if (--left == 0) mma_commit(q_empty + 8 * qb);
                    ++tq;
                } else {
                    const uint32_t ub = tp & 1, ob = p.o_bufs == 2 ? (vi & 1) : 0;
                    const int use = p.o_bufs == 2 ? vi >> 1 : vi;
                    if (v_at == 0) {
                        v_len = i == vi ? len : len_before;
                        ok = use == 0 || wait_by<(R <= 16)>(o_empty + 8 * ob, (uint32_t)(use - 1) & 1u, abort_flag);
                    }
                    ok = ok && wait_by<(R <= 16)>(p_full + 8 * ub, (uint32_t)(tp >> 1) & 1u, abort_flag);
                    if (!SHARED) ok = ok && wait_by<(R <= 16)>(v_full + 8 * v_ring.i, v_ring.phase, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t pt = ub * (N2 * 128), slot = SHARED ? tp % p.k_stages : v_ring.i;
                    uint32_t d = o_tmem + ob * o_cols + (kStreams == 2 ? ub * p.nv * N2 : 0);
                    uint32_t at = slot * (SHARED ? p.nk : p.nv) * kChunk;
                    const uint32_t old = v_at < kStreams ? 0u : 1u;  // not the stream's first tile of the piece
#pragma unroll 1
                    for (int j = 0; j < p.nv; ++j) {
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            mma_f8(d, desc_at(dv, at + 4096 * s), desc_at(dw, pt + 512 * s), i_o, s == 0 ? old : 1u);
                        d += N2;
                        at += kChunk;
                    }
                    mma_commit((SHARED ? k_empty : v_empty) + 8 * slot);
                    if (!SHARED) v_ring.step(p.v_stages);
                    mma_commit(p_empty + 8 * ub);
                    if (++v_at == v_len) {
                        mma_commit(o_full + 8 * ob);
                        v_at = 0;
                        ++vi;
                    }
                    ++tp;
                }
            }
            if (!ok) {
                mma_commit(drain);
                mbar_wait(drain, 0, nullptr, 200000000ull);
            }
        }
        __syncwarp();
    } else if (warp == kMarker) {
        // ------------------------------------------------------------- scales
        // By plain loads, one byte to a lane, of up to eight tiles at a time, so that memory is waited for once. (A softmax
        // thread that fetched its own token's waited at every tile.)
        const int shift = p.block_shift < 7 ? p.block_shift : 7;  // log2 of the tokens of a byte
        const int m_shift = 7 - shift, rounds = m_shift > 5 ? 1 << (m_shift - 5) : 1;
        const int most = m_shift >= 5 ? 1 : m_shift < 2 ? 8 : 32 >> m_shift;
        Piece x;
        x.t1 = 0;
        int i = 0, tile = 0, slot = 0;
        bool ok = true;
        auto deal = [&]() {  // piece i, to all that read it; the first lies there
            if (i >= kPieces) ok = wait(piece_empty + 8 * (i % kPieces), (uint32_t)(i / kPieces - 1) & 1u, abort_flag);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (ok && lane == 0) {
                sh.piece[i % kPieces] = x;
                mbar_arrive(piece_full + 8 * (i % kPieces));
            }
            ++i;
        };
#pragma unroll 1
        for (int t = 0;;) {
            if (tile == x.t1) {
                if (t == tiles || !ok) break;
                if (t == 0) {
                    slot = sh.start_slot;
                    x = sh.piece[0];
                    tile = x.t0;
                    ++i;
                    continue;  // to its scales
                } else {
                    x.t0 = 0;
                    do {
                        if (++slot == p.slots) {
                            slot = 0;
                            x.x.b = 0;
                            if (++x.h == p.H) {  // a cu that falls: the slots' tiles are not those that the share was made from
                                record_status(p.status, MLA_ERR_INVALID_ARG);
                                *abort_flag = 1;
                                ok = false;
                                break;
                            }
                        }
                        x.x = read_slot<R>(p, slot, x.x.b);
                    } while (x.x.tiles == 0);
                    if (!ok) break;
                }
                const int left = tiles - t, n = x.x.tiles - x.t0;
                x.t1 = x.t0 + (n < left ? n : left);
                tile = x.t0;
                deal();
                if (!ok) break;
            }
            const int n = x.t1 - tile < most ? x.t1 - tile : most;
#pragma unroll 1
            for (int r = 0; r < rounds; ++r) {
                const int e = lane + 32 * r, of = e >> m_shift, m = e & ((1 << m_shift) - 1), to = (t + of) % kMarkTiles;
                const int pos = (tile + of) * kTokens + (m << shift);
                uint32_t k = 0, v = 0;
                if (of < n && pos < x.x.len) {
                    const int page = p.table[(int64_t)x.x.b * p.width + (pos >> p.page_shift)];
                    if (page >= 0 && page < p.pages) {  // a bad one is recorded by the producer and reads as zeros
                        const int64_t at = ((int64_t)page * p.H + x.h) * p.marks + ((pos & (p.page - 1)) >> p.block_shift);
                        k = p.k_scales[at];
                        if (!SHARED) v = p.v_scales[at];
                    }
                }
                if (of < n) {
                    if (t + of >= kMarkTiles)
                        ok = wait(m_empty + 8 * to, (uint32_t)((t + of) / kMarkTiles - 1) & 1u, abort_flag);
                    sh.marks[to][0][m] = (uint8_t)k;
                    if (!SHARED) sh.marks[to][SHARED ? 0 : 1][m] = (uint8_t)v;
                }
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
            __syncwarp();  // the lanes' bytes lie there: a vote orders no memory
            if (lane < n) mbar_arrive(m_full + 8 * ((t + lane) % kMarkTiles));
            t += n;
            tile += n;
            if (!ok) break;
        }
        x.t0 = x.t1 = 0;
        if (ok) deal();  // no more
        __syncwarp();
    } else if (warp >= kHelper) {
        // ------------------------------------------- queries in, results out
        const int quad = warp & 3, htid = tid - 32 * kHelper;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        bool failed = false;
        int parts = 0;  // which of the share's two places in the workspace it has filled
        constexpr int kG = SHARED ? (kMaxQueryChunks * 128 / 8 + 31) / 32 : 1;
        const int gran = p.Dk / 8;
        // eight bf16 at a time of a piece's query row r, as many as a lane has
        auto fetch = [&](const Piece& x, int r, uint4 (&g)[kG]) {
            const int rho = x.x.rho0 + r, tok = token_of(p, rho);
            const uint16_t* src = p.q + (int64_t)(x.x.lo + tok) * p.q_t + (int64_t)(x.h * p.group + rho - tok * p.group) * p.q_h;
#pragma unroll
            for (int k = 0; k < kG; ++k) {
                const int at = k * 32 + lane;
                g[k] = make_uint4(0, 0, 0, 0);
                if (r < x.x.rows && at < gran) {
                    const uint16_t* q = src + at * 8;
                    if (p.q_vec) {
                        g[k] = *reinterpret_cast<const uint4*>(q);
                    } else {
                        g[k].x = q[0] | ((uint32_t)q[1] << 16);
                        g[k].y = q[2] | ((uint32_t)q[3] << 16);
                        g[k].z = q[4] | ((uint32_t)q[5] << 16);
                        g[k].w = q[6] | ((uint32_t)q[7] << 16);
                    }
                }
            }
        };
        // Piece i's query rows as two E4M3 numbers each, row r at r and R + r; a warp takes every fourth, the next one's
        // memory on its way.
        auto load_q = [&](const Piece& x, int i) {
            const int par = i & 1;
            const uint32_t qb = p.q_bufs == 2 ? par : 0;
            const int use = p.q_bufs == 2 ? i >> 1 : i;
            if constexpr (SHARED) {
                // all of the rows' lines at once: one by one they queue behind the first tiles of all SMs
#pragma unroll 1
                for (int r = quad; r < x.x.rows; r += 4) {
                    const int rho = x.x.rho0 + r, tok = token_of(p, rho);
                    const uint16_t* src = p.q + (int64_t)(x.x.lo + tok) * p.q_t + (int64_t)(x.h * p.group + rho - tok * p.group) * p.q_h;
                    if (lane * 64 < p.Dk) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + lane * 64));
                }
            }
            uint4 g[kG], g2[kG];
#pragma unroll 1
            for (int r = quad - 4; r < R; r += 4) {
                fetch(x, r + 4, g2);
                if (r < 0) {
                    if (use > 0) failed |= !wait_by<(R == 64)>(q_empty + 8 * qb, (uint32_t)(use - 1) & 1u, abort_flag);
#pragma unroll
                    for (int k = 0; k < kG; ++k) g[k] = g2[k];
                    continue;
                }
                uint32_t m = 0;
#pragma unroll
                for (int k = 0; k < kG; ++k) {
                    const uint32_t u[4] = {g[k].x, g[k].y, g[k].z, g[k].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) m = max(m, max((u[e] << 16) & 0x7FFFFFFFu, u[e] & 0x7FFF0000u));
                }
                m = __reduce_max_sync(0xFFFFFFFFu, m);
                // a factor 2^f that brings the row's largest into [128, 256); NaN and Inf make the row's scale NaN
                int f = 134 - (int)(m >> 23);
                f = m == 0 ? 0 : f > 120 ? 120 : f;
                const bool bad = m >= 0x7F800000u;
                const float up = bad ? 0.f : __uint_as_float((uint32_t)(127 + f) << 23);
#pragma unroll
                for (int k = 0; k < kG; ++k) {
                    const int at = k * 32 + lane;
                    if (at < gran) {
                        const uint32_t u[4] = {g[k].x, g[k].y, g[k].z, g[k].w};
                        uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t h2, l2;
                            split8(bad ? 0.f : bf16lo_to_f32(u[e]) * up, bad ? 0.f : bf16hi_to_f32(u[e]) * up, h2, l2);
                            hi[e / 2] |= h2 << (16 * (e & 1));
                            lo[e / 2] |= l2 << (16 * (e & 1));
                        }
                        const uint32_t to = q_base + qb * q_bytes + (at >> 4) * (N2 * 128) + (((at & 15) >> 1 ^ (r & 7)) << 4) + (at & 1) * 8;
                        sts_v2(to + r * 128, hi[0], hi[1]);
                        sts_v2(to + (R + r) * 128, lo[0], lo[1]);
                    }
                    g[k] = g2[k];
                }
                if (lane == 0) {
                    const int rr = r < x.x.rows ? r : x.x.rows - 1, rho = x.x.rho0 + rr, tok = token_of(p, rho);
                    sh.unit[par][r] = bad ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(127 - f) << 23);
                    for (int k = 0; k < kStreams; ++k) sh.ref[par][k][r] = -kNothing;
                    sh.limit[par][r] = x.x.len - x.x.n + tok;
                    sh.row_at[par][r] = (x.x.lo + tok) * p.Hq + x.h * p.group + rho - tok * p.group;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(q_full + 8 * qb);
                mbar_arrive(rows_full + 8 * par);
            }
        };
        Piece now, next;
        next.t1 = 1;
        // at turn i the queries of piece i, then the result of piece i - 1; every warp leaves with the others
#pragma unroll 1
        for (int i = -1; next.t1 > 0; ++i) {
            now = next;
            failed |= !get_piece(i + 1, next);
            if (!named_bar_and(3, kHelpers, !failed)) break;
            if (lane == 0) mbar_arrive(piece_empty + 8 * ((i + 1) % kPieces));
            if (next.t1 > 0) load_q(next, i + 1);
            if (i < 0) continue;
            const int par = i & 1;
            const uint32_t ob = p.o_bufs == 2 ? par : 0;
            const int use = p.o_bufs == 2 ? i >> 1 : i;
            failed |= !wait_by<(R == 64)>(sums_full + 8 * par, (uint32_t)(i >> 1) & 1u, abort_flag);
            const bool whole = now.t0 == 0 && now.t1 == now.x.tiles;
            const int part = 2 * (int)blockIdx.x + (now.t0 == 0 ? 1 : 0);
            if (htid < R) {
                float m = kNothing, sum = 0.f, f[kStreams];
                for (int k = 0; k < kStreams; ++k) m = fmaxf(m, -sh.ref[par][k][htid]);
#pragma unroll
                for (int k = 0; k < kStreams; ++k) {
                    const float(&row)[4][R] = sh.sums[par][k];
                    const float up = exp2_fast(-sh.ref[par][k][htid] - m);
                    sum = fmaf(up, (row[0][htid] + row[1][htid]) + (row[2][htid] + row[3][htid]), sum);
                    const int e = sh.top_e[par][kStreams == 2 ? k : htid / (R / 2)];
                    f[k] = ldexpf(up, e < 0 ? -131 : e - 131);
                }
                const float over = sum == 0.f ? 0.f : __fdividef(1.f, sum);  // of a part too: sums of large values may overflow; 2 ulp
#pragma unroll
                for (int k = 0; k < kStreams; ++k) sh.out_factor[k][htid] = f[k] * over;
                if (!whole) p.part_ml[(int64_t)part * R + htid] = make_float2(m, sum);
                else if (p.lse && htid < now.x.rows)
                    p.lse[sh.row_at[par][htid]] = sum == 0.f ? -INFINITY : log_sum(m, sum);
            }
            failed |= !wait_by<(R == 64)>(o_full + 8 * ob, (uint32_t)use & 1u, abort_flag);
            if (!named_bar_and(3, kHelpers, !failed)) break;
            tc_fence_after();
            const bool nans = *(volatile int*)&sh.nan_seen[par] != 0;
            constexpr int kStep = R < 16 ? R : 16;
            const uint32_t from0 = o_tmem + ob * o_cols + lanes;
#pragma unroll 1
            for (int j = 0; j < p.nv; ++j) {
                const int ch = j * 128 + quad * 32 + lane;
#pragma unroll 1
                for (int r0 = 0; r0 < now.x.rows; r0 += kStep) {
                    float o[kStep];
                    int at[kStep];
#pragma unroll
                    for (int e = 0; e < kStep; e += 4) {
                        const int4 v = *reinterpret_cast<const int4*>(&sh.row_at[par][r0 + e]);
                        at[e] = v.x, at[e + 1] = v.y, at[e + 2] = v.z, at[e + 3] = v.w;
                        o[e] = o[e + 1] = o[e + 2] = o[e + 3] = 0.f;
                    }
#pragma unroll
                    for (int k = 0; k < kStreams; ++k) {
                        if (sh.top_e[par][k] == 2 * kNoScale) continue;  // the same in every thread: a stream without a tile
                        uint32_t v[16], u[16];
                        const uint32_t from = from0 + (k * p.nv + j) * N2 + r0;
                        __syncwarp();
                        tmem_ld16(from, v);
                        if constexpr (R > 8) tmem_ld16(from + R, u);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < kStep; e += 4) {
                            const float4 f4 = *reinterpret_cast<const float4*>(&sh.out_factor[k][r0 + e]);
                            const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
                            for (int i2 = 0; i2 < 4; ++i2)
                                o[e + i2] = fmaf(fmaf(__uint_as_float(R > 8 ? u[e + i2] : v[(8 + e + i2) & 15]), 0.03125f,
                                                      __uint_as_float(v[e + i2])),
                                                 f[i2], o[e + i2]);
                        }
                    }
                    if (nans) {
                        const int nan_at = sh.nan_at[par][ch & 511];
#pragma unroll
                        for (int e = 0; e < kStep; ++e)
                            if (nan_at <= sh.limit[par][r0 + e]) o[e] = __uint_as_float(0x7FC00000u);
                    }
                    if (ch < p.Dv) {
                        const int n = now.x.rows - r0;
                        if (whole) {
                            uint16_t* out = p.out + ch;
#pragma unroll
                            for (int e = 0; e < kStep; ++e)
                                if (e < n) out[(int64_t)at[e] * p.Dv] = (uint16_t)pack_bf16x2(o[e], 0.f);
                        } else {
                            float* out = p.part_o + ((int64_t)part * R + r0) * p.Dv + ch;
#pragma unroll
                            for (int e = 0; e < kStep; ++e)
                                if (e < n) out[e * p.Dv] = o[e];
                        }
                    }
                }
            }
            __syncwarp();
            tc_fence_before();
            if (nans) {  // the same in every thread: set before its sums were
                named_bar_sync(3, kHelpers);
                for (int k = htid; k < 512; k += kHelpers) sh.nan_at[par][k] = 0x7FFFFFFF;
                if (htid == 0) sh.nan_seen[par] = 0;
            }
            named_bar_sync(3, kHelpers);  // out_factor and the rows are read
            if (lane == 0) {
                mbar_arrive(o_empty + 8 * ob);
                mbar_arrive(sums_empty + 8 * par);
            }
            if (htid == 0 && !whole) {
                p.meta[part] = make_int4(now.t0 == 0 ? kOpens : now.t1 == now.x.tiles ? kEnds : kGoesOn, now.x.rho0,
                                         now.x.rows, now.x.lo * p.H + now.h);
                parts |= 1 << (part & 1);
            }
        }
        if (htid == 0)
            for (int k = 0; k < 2; ++k)
                if (!(parts >> k & 1)) p.meta[2 * blockIdx.x + k] = make_int4(kNoPart, 0, 0, 0);
    } else {
        // ------------------------------------------------------------ softmax
        constexpr int kFours = kFour / 4, RT = R / kFours;  // rows of a thread
        constexpr int kWide = RT > 16 ? 8 : 16;             // scores read at a time (with sixteen of 32, registers ran out)
        const int tok = tid & 127, quad = warp & 3, four = warp >> 2, stream = kStreams == 2 ? four : 0;
        const int r_lo = kStreams == 2 ? 0 : four * RT;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;  // this warp's lanes of tensor memory
        const uint32_t my_bar = 1 + four;
        const int mark = tok >> (p.block_shift < 7 ? p.block_shift : 7);  // of the token's byte among its tile's
        int t = 0, turn = 0;  // t: tiles of the share so far; turn: of the four warps' votes
        // A wait that gave up is reported with the next vote, so that the four warps leave together: until then a
        // thread that saw it goes on, through every barrier.
        bool failed = false, leave = false;
#pragma unroll 1
        for (int i = 0; !leave; ++i) {
            Piece w;
            if (!named_bar_and(my_bar, 128, get_piece(i, w))) break;
            if (lane == 0) mbar_arrive(piece_empty + 8 * (i % kPieces));
            if (w.t1 == 0) break;
            const int par = i & 1;
            failed |= !wait(rows_full + 8 * par, (uint32_t)(i >> 1) & 1u, abort_flag);
            const float *unit = &sh.unit[par][r_lo], *ref = &sh.ref[par][stream][r_lo];
            const int* limit = &sh.limit[par][r_lo];
            const uint32_t o_mine = o_tmem + lanes + (p.o_bufs == 2 ? par : 0) * o_cols + stream * p.nv * N2;
            float l[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) l[r] = 0.f;
            int top_e = kNoScale;
            bool any = false;  // the stream has had a tile of the piece
            const int least = w.x.len - w.x.n + token_of(p, w.x.rho0);  // the last position that every row sees
            const int t_end = t + w.t1 - w.t0, to_tile = w.t0 - t;
#pragma unroll 1
            for (; t < t_end; ++t) {
                if (kStreams == 2 && (t & 1) != stream) continue;
                const int tile = to_tile + t, buf = t & 1, pos = tile * kTokens + tok, slot = t % kMarkTiles;
                const bool masked = (tile + 1) * kTokens - 1 > least;
                const bool valid = pos < w.x.len;
                failed |= !wait(m_full + 8 * slot, (uint32_t)(t / kMarkTiles) & 1u, abort_flag);
                const uint32_t ke = sh.marks[slot][0][mark];
                const int ve = SHARED ? (int)ke : sh.marks[slot][SHARED ? 0 : 1][mark];
                // a value's scale of NaN makes the scores NaN of those who see it
                const float ks = e8m0_to_f32(ve == 255 ? 255u : ke) * p.scale_log2;
                const int e = valid && ve != 255 ? ve : 0;
                // what the token's scores may be, less their references, before a vote: kPass less the difference of the
                // exponents (1.5 2^23 + 4 in the last bits of a float)
                const float most = valid ? __int_as_float(0x4B400000 + (int)kPass - max(e - top_e, kFar)) - 12582912.f : INFINITY;
                __syncwarp();
                if (lane == 0) mbar_arrive(m_empty + 8 * slot);
                failed |= !wait(s_full + 8 * buf, (uint32_t)(t >> 1) & 1u, abort_flag);
                __syncwarp();
                tc_fence_after();
                // x = the rows' scores, less their references; -inf where a row does not see the token
                float x[RT];
                auto scores = [&](auto less) {
                    const uint32_t from = s_tmem + lanes + buf * N2 + r_lo;
#pragma unroll
                    for (int r0 = 0; r0 < RT; r0 += kWide) {
                        uint32_t v[kWide], u[kWide];
                        tmem_ld<kWide>(from + r0, v);
                        if constexpr (R > 8) tmem_ld<kWide>(from + R + r0, u);
                        tmem_ld_wait();
#pragma unroll
                        for (int r = 0; r < (RT < kWide ? RT : kWide); r += 4) {
                            const float4 q = *reinterpret_cast<const float4*>(unit + r0 + r);
                            const float4 m = *reinterpret_cast<const float4*>(ref + r0 + r);
                            const float qs[4] = {q.x, q.y, q.z, q.w}, ms[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
                            for (int e = 0; e < 4; e += 2) {
                                const uint32_t *h = &v[r + e], *o = R > 8 ? &u[r + e] : &v[(8 + r + e) % kWide];
                                float &x0 = x[r0 + r + e], &x1 = x[r0 + r + e + 1];
                                float k0, k1;
                                mul2(k0, k1, qs[e], qs[e + 1], ks, ks);
                                fma2(x0, x1, __uint_as_float(o[0]), __uint_as_float(o[1]), 0.03125f, 0.03125f,
                                     __uint_as_float(h[0]), __uint_as_float(h[1]));
                                if constexpr (decltype(less)::value) fma2(x0, x1, x0, x1, k0, k1, ms[e], ms[e + 1]);
                                else mul2(x0, x1, x0, x1, k0, k1);
                            }
                        }
                    }
                    if (masked && w.x.n > 1) {
#pragma unroll
                        for (int r = 0; r < RT; ++r) x[r] = pos <= limit[r] ? x[r] : -INFINITY;
                    }
                };
                scores(std::true_type{});
                float over = max3(x[0], x[1], x[2]), over2 = max3(x[3], x[4], x[5]);
#pragma unroll
                for (int r = 6; r + 3 < RT; r += 4) {
                    over = max3(over, x[r], x[r + 1]);
                    over2 = max3(over2, x[r + 2], x[r + 3]);
                }
                over = max3(max3(over, over2, kNothing), x[RT - 2], x[RT - 1]);
                if (__any_sync(0xFFFFFFFFu, over > most || failed)) {  // a vote: one more than the largest scale among those who pass
                    const int word = 1 + __reduce_max_sync(0xFFFFFFFFu, failed ? kFailed : over > most ? e : 0);
                    if (lane == 0) atomicMax(&sh.vote[four][turn], word);
                }
                named_bar_sync(my_bar, 128);
                const int vote = *(volatile int*)&sh.vote[four][turn];
                turn = turn == 2 ? 0 : turn + 1;
                // the place two turns on was read by all before this barrier and is written by none before the next
                if (tok == 0) sh.vote[four][turn == 2 ? 0 : turn + 1] = 0;
                if (vote > kFailed) {
                    leave = true;
                    break;
                }
                if (vote) {
                    // a larger exponent for all, and a new reference for every row: its largest weight so far
                    const int old_e = top_e;
                    top_e = max(top_e, vote - 1);
                    const float low = valid ? (float)max(e - top_e, kFar) : -INFINITY;
                    const bool raised = any && top_e > old_e;
                    if (raised) {  // how far the references may fall with the larger scale: the sums so far grow as much
                        float sum = l[0];
#pragma unroll
                        for (int r = 1; r < RT; ++r) sum = fmaxf(sum, l[r]);
                        sum = warp_max(sum);
                        if (lane == 0) sh.warp_l[four][quad] = __log2f(sum);
                    }
                    scores(std::false_type{});
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const float m = warp_max(x[r] + low);
                        if (lane == (r & 31)) sh.warp_row[stream][quad][r_lo + r] = m;
                    }
                    named_bar_sync(my_bar, 128);
                    const int r = r_lo + tok;
                    if (tok < RT) {
                        const float old = -sh.ref[par][stream][r];
                        float m = old;
                        if (raised) {
                            const float *w = sh.warp_l[four], sum = fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3]));
                            m -= fmaxf(fminf((float)(top_e - old_e), kMostSum - sum), 0.f);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) m = fmaxf(m, sh.warp_row[stream][k][r]);
                        sh.ref[par][stream][r] = -m;
                        sh.factor[stream][r] = exp2_fast(old - m);  // above 1, by 2^90 at most, where a larger scale lowers the reference
                    }
                    named_bar_sync(my_bar, 128);
#pragma unroll
                    for (int k = 0; k < RT; ++k) {
                        l[k] *= sh.factor[stream][r_lo + k];
                        x[k] += ref[k];
                    }
                    if (any) {
                        const float down = old_e == top_e ? 1.f : old_e < top_e - 126 ? 0.f : __uint_as_float((uint32_t)(127 + old_e - top_e) << 23);
                        const int u = t - kStreams;  // the stream's tile before
                        failed |= !wait(p_empty + 8 * (u & 1), (uint32_t)(u >> 1) & 1u, abort_flag);
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int j = 0; j < p.nv; ++j)
#pragma unroll 1
                            for (int r0 = 0; r0 < 2 * RT; r0 += 16) {
                                uint32_t v[16];
                                const int col = R == 8 ? 0 : r_lo + (r0 < RT ? r0 : R + r0 - RT), row = col < R ? col : col - R;
                                const uint32_t at = o_mine + j * N2 + col;
                                tmem_ld16(at, v);
                                tmem_ld_wait();
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    v[k] = __float_as_uint(__uint_as_float(v[k]) * (sh.factor[stream][R == 8 ? k % 8 : row + k] * down));
                                tmem_st16(at, v);
                            }
                        tmem_st_wait();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_empty + 8 * buf);
                any = true;
                // The probabilities, times the value's scale, as two E4M3 numbers; nothing behind the last position. (Their
                // buffer is free: the scores came behind the product that read it, tile t - 2's.)
                const uint32_t to = p_base + buf * (N2 * 128) + tok * 16;
                const float f = __int_as_float(min(max(e - top_e + 4 + 127, 0), 254) << 23);
#pragma unroll
                for (int r0 = 0; r0 < RT; r0 += 16) {
                    constexpr int kRows = RT < 16 ? RT : 16;
                    uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
                    if (valid) {
#pragma unroll
                        for (int r = 0; r < kRows; r += 4) {
                            uint32_t h[2], o[2];
#pragma unroll
                            for (int k = 0; k < 4; k += 2) {
                                const float a = exp2_fast(x[r0 + r + k]), b = exp2_fast(x[r0 + r + k + 1]);
                                add2(l[r0 + r + k], l[r0 + r + k + 1], a, b);
                                float y, z;
                                mul2(y, z, a, b, f, f);
                                split8(y, z, h[k / 2], o[k / 2]);
                            }
                            hi[r / 4] = __byte_perm(h[0], h[1], 0x5410);
                            lo[r / 4] = __byte_perm(o[0], o[1], 0x5410);
                        }
                    }
                    if constexpr (R == 8) {
                        sts_v4(to, hi[0], hi[1], lo[0], lo[1]);
                    } else {
                        sts_v4(to + (r_lo + r0) / 16 * 2048, hi[0], hi[1], hi[2], hi[3]);
                        sts_v4(to + (R + r_lo + r0) / 16 * 2048, lo[0], lo[1], lo[2], lo[3]);
                    }
                }
                if (r_lo == 0 && ((tile + 1) * kTokens > w.x.len || (masked && w.x.n > 1))) {
                    // What lies behind the last position may be anything, also NaN: zeros. And a NaN that some rows see
                    // and others do not must not meet their zero probability: it is noted and put into the result.
                    const int stages = SHARED ? p.k_stages : p.v_stages, at = t % stages;
                    failed |= !wait((SHARED ? k_full : v_full) + 8 * at, (uint32_t)(t / stages) & 1u, abort_flag);
                    uint32_t mem = (SHARED ? base : v_base) + at * (SHARED ? p.nk : p.nv) * kChunk + tok * 128;
#pragma unroll 1
                    for (int j = 0; j < p.nv; ++j, mem += kChunk) {
                        if (!valid) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) sts_v4(mem + k * 16, 0, 0, 0, 0);
                        } else if (pos > least) {
#pragma unroll 1
                            for (int k = 0; k < 8; ++k) {
                                const uint32_t place = mem + ((k ^ (tok & 7)) << 4);
                                const uint4 v = lds_v4(place);
                                uint32_t u[4] = {v.x, v.y, v.z, v.w};
                                bool found = false;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    uint32_t nan = __vcmpeq4(u[e] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                                    u[e] &= ~nan;
                                    found |= nan != 0;
#pragma unroll 1
                                    for (int f = 0; nan != 0; ++f, nan >>= 8)
                                        if (nan & 1u) atomicMin(&sh.nan_at[par][(j * 128 + k * 16 + e * 4 + f) & 511], pos);
                                }
                                if (!found) continue;
                                sts_v4(place, u[0], u[1], u[2], u[3]);
                                sh.nan_seen[par] = 1;
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * buf);
            }
            if (leave) break;
            // the piece's sums
            if (i >= 2) failed |= !wait(sums_empty + 8 * par, (uint32_t)((i >> 1) - 1) & 1u, abort_flag);
            const int row = fold_rows<RT / 2, 16>(l, lane);
            sh.sums[par][stream][quad][r_lo + row] = l[0];  // a row's lanes the same
            if (tok == 0) sh.top_e[par][four] = any ? top_e : 2 * kNoScale;
            __syncwarp();
            if (lane == 0) mbar_arrive(sums_full + 8 * par);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) record_status(p.status, MLA_ERR_TIMEOUT);
    if (warp == kIssuer) {
        tc_fence_after();
        tmem_dealloc(tmem, p.tmem_cols);
    }
}

// Adds the parts of the pair that share blockIdx.x / (R / 8) opens, eight query
// rows to a block. (One row to a block were 4864 blocks of latents, 33 us; these
// are 608, 6 us.)
constexpr int kCombineRows = 8;
template <int R>
__global__ void __launch_bounds__(kCombineThreads) cache_attn_combine_kernel(const __grid_constant__ AttnParams p, int shares) {
    __shared__ float weight[kMaxShares][kCombineRows], sums[kMaxShares][kCombineRows];
    __shared__ float4 halves[kCombineThreads];
    __shared__ int64_t row_at[kCombineRows];
    __shared__ int ends;
    grid_launch_next();
    grid_wait_previous();
    const int c = blockIdx.x / (R / kCombineRows), r0 = blockIdx.x % (R / kCombineRows) * kCombineRows, tid = threadIdx.x;
    const int4 m = p.meta[2 * c + 1];
    const int rows = m.z - r0 < kCombineRows ? m.z - r0 : kCombineRows;
    if (m.x != kOpens || rows <= 0) return;
    // the shares behind go on with the pair until one ends it
    const int behind = shares - 1 - c;
    if (tid == 0) ends = behind;
    __syncthreads();
    for (int i = 1 + tid; i <= behind; i += kCombineThreads)
        if (p.meta[2 * (c + i)].x == kEnds) atomicMin(&ends, i);
    __syncthreads();
    const int n = ends + 1;  // parts
    auto place = [&](int i) { return (int64_t)(2 * (c + i) + (i == 0)) * R + r0; };
    for (int e = tid; e < n * kCombineRows; e += kCombineThreads) {
        const int i = e / kCombineRows, r = e % kCombineRows;
        const float2 ml = r < rows ? p.part_ml[place(i) + r] : make_float2(kNothing, 0.f);
        weight[i][r] = ml.x;
        sums[i][r] = ml.y;
    }
    __syncthreads();
    const int r = tid / 32, lane = tid % 32;
    if (r < kCombineRows) {  // a warp to a row
        float top = kNothing, l = 0.f;
        for (int i = lane; i < n; i += 32) top = fmaxf(top, weight[i][r]);
        top = warp_max(top);
        for (int i = lane; i < n; i += 32) {
            const float w = exp2_fast(weight[i][r] - top) * sums[i][r];
            weight[i][r] = w;
            l += w;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        for (int i = lane; i < n; i += 32) weight[i][r] *= inv;
        if (lane == 0) {
            const int rho = m.y + r0 + r, tok = token_of(p, rho);
            const int64_t row = (int64_t)(m.w / p.H + tok) * p.Hq + (int64_t)(m.w % p.H) * p.group + rho - tok * p.group;
            row_at[r] = row;
            if (p.lse && r < rows) p.lse[row] = l == 0.f ? -INFINITY : log_sum(top, l);
        }
    }
    __syncthreads();
    // four channels to a thread; where that leaves threads, they share the parts
    const int per = p.Dv / 4, all = rows * per;
    int groups = 1;
    while (groups < 8 && 2 * groups * all <= kCombineThreads) groups *= 2;
    const int lanes = kCombineThreads / groups, group = tid / lanes;
    for (int e0 = 0; e0 < all; e0 += lanes) {
        const int e = e0 + tid % lanes, row = e / per, ch = (e - row * per) * 4;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e < all) {
#pragma unroll 8
            for (int i = group; i < n; i += groups) {
                const float4 v = *reinterpret_cast<const float4*>(p.part_o + (place(i) + row) * p.Dv + ch);
                const float w = weight[i][row];
                o.x = fmaf(w, v.x, o.x);
                o.y = fmaf(w, v.y, o.y);
                o.z = fmaf(w, v.z, o.z);
                o.w = fmaf(w, v.w, o.w);
            }
        }
        if (groups > 1) {
            halves[tid] = o;
            __syncthreads();
            for (int g = 1; g < groups && group == 0; ++g) {
                const float4 v = halves[tid + g * lanes];
                o.x += v.x;
                o.y += v.y;
                o.z += v.z;
                o.w += v.w;
            }
        }
        if (group == 0 && e < all) {
            uint16_t* out = p.out + row_at[row] * p.Dv + ch;
            const uint32_t a = pack_bf16x2(o.x, o.y), b = pack_bf16x2(o.z, o.w);
            out[0] = (uint16_t)a;
            out[1] = (uint16_t)(a >> 16);
            out[2] = (uint16_t)b;
            out[3] = (uint16_t)(b >> 16);
        }
    }
}

// -------------------------------------------------------------------- host
struct AttnPlan {
    int R, nk, nv, k_stages, v_stages, q_bufs, o_bufs, tmem_cols;
    size_t smem;
};

// Query rows of a tile: as many as a head of the cache has for a sequence (the
// group times the new tokens, on average), up to 64; with more than two value
// tiles up to 32, for tensor memory's sake: 2 score buffers and nv sums of 2R
// columns each, 512 in all. (More rows than there are would only add to both
// products and the softmax: eight rows over latents take 29 us with R = 8, and 32
// take 42 with R = 32. Fewer would read the cache again for the others.)
template <int R>
size_t shared_bytes(bool shared) { return shared ? sizeof(Shared<R, true>) : sizeof(Shared<R, false>); }

bool attn_plan(const mla_attn_shape& s, const mla_kv_cache& c, int max_smem, AttnPlan* out) {
    const bool shared = !c.v;
    if (shared ? (c.Dk > 128 * kMaxQueryChunks || c.Dv > 512) : (c.Dk > 256 || c.Dv > 256)) return false;
    AttnPlan a{};
    a.nk = (c.Dk + 127) / 128;
    a.nv = (c.Dv + 127) / 128;
    const int64_t group = s.Hq / c.H, rows = group * (s.B > 0 ? (s.T + s.B - 1) / s.B : 1);
    // half as many rows where two tiles find no room beside them (latents of more than 384 channels, up to 256 of them values)
    for (a.R = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 || a.nv > 2 ? 32 : 64; a.R >= 8; a.R /= 2) {
        const size_t tail = a.R == 8    ? shared_bytes<8>(shared)
                            : a.R == 16 ? shared_bytes<16>(shared)
                            : a.R == 32 ? shared_bytes<32>(shared)
                                        : shared_bytes<64>(shared);
        const size_t q = (size_t)a.nk * 2 * a.R * 128, fixed = 1024 + 2 * 2 * a.R * 128 + tail;
        const int tile = shared ? a.nk : a.nk + a.nv;
        // two buffers of queries where two tiles are left, else one beside a tile (latents: two)
        for (a.q_bufs = 2; a.q_bufs > 0; --a.q_bufs) {
            const int64_t left = (int64_t)max_smem - (int64_t)(fixed + a.q_bufs * q);
            const int room = (int)(left / kChunk), stages = room / tile;
            if (stages < (shared || a.q_bufs == 2 ? 2 : 1)) continue;
            a.v_stages = shared ? 0 : stages > kMaxStages ? kMaxStages : stages;
            a.k_stages = (room - a.v_stages * a.nv) / a.nk;
            if (a.k_stages > kMaxStages) a.k_stages = kMaxStages;
            break;
        }
        if (a.q_bufs == 0) continue;
        a.smem = fixed + a.q_bufs * q + ((size_t)a.k_stages * a.nk + (size_t)a.v_stages * a.nv) * kChunk;
        break;
    }
    if (a.R < 8) return false;
    const int s_cols = 2 * 2 * a.R, o_cols = a.nv * (a.R <= 16 ? 2 : 1) * 2 * a.R;
    a.o_bufs = s_cols + 2 * o_cols <= 512 ? 2 : 1;
    const int cols = s_cols + a.o_bufs * o_cols;
    a.tmem_cols = 32;
    while (a.tmem_cols < cols) a.tmem_cols *= 2;
    if (a.tmem_cols > 512) return false;
    *out = a;
    return true;
}

int check_attn(const mla_attn_shape* s, const mla_kv_cache* c, const int32_t* table, CacheBytes* n) {
    if (!s) return MLA_ERR_INVALID_ARG;
    const int st = check_cache(c, s->B, table, s->table_width, n);
    if (st != MLA_OK && st != MLA_ERR_UNSUPPORTED && st != MLA_ERR_ALIGNMENT) return st;
    if (s->T < 0 || s->T > kI32Max || s->Hq <= 0 || s->Hq % c->H != 0 || s->reserved != 0 || (s->T > 0 && s->B == 0))
        return MLA_ERR_INVALID_ARG;
    if (!(s->scale >= -3.402823466e38f && s->scale <= 3.402823466e38f)) return MLA_ERR_INVALID_ARG;
    const int64_t most = s->T > s->Hq ? s->T : s->Hq;
    if (!inside(most, s->q_t) || !inside(most, s->q_h)) return MLA_ERR_INVALID_ARG;
    if (st != MLA_OK) return st;
    if (s->T * s->Hq > kI32Max) return MLA_ERR_UNSUPPORTED;
    return MLA_OK;
}

size_t workspace_bytes(int R, int Dv, int shares) {
    return (size_t)shares * 2 * (R * ((size_t)Dv * 4 + 8) + 16);
}

template <int R, bool SHARED>
int launch_attn(const AttnParams& p, const AttnPlan& a, const CUtensorMap& k, const CUtensorMap& v, int shares,
                cudaStream_t s) {
    if (cudaFuncSetAttribute(cache_attn_kernel<R, SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)a.smem) != cudaSuccess)
        return MLA_ERR_CUDA;
    const int st = launch_overlapped(cache_attn_kernel<R, SHARED>, (unsigned)shares, kThreads, a.smem, 0, s, k, v, p);
    if (st != MLA_OK) return st;
    return launch_overlapped(cache_attn_combine_kernel<R>, (unsigned)(shares * (R / kCombineRows)), kCombineThreads, 0, 0, s, p, shares);
}

}  // namespace
}  // namespace mlaq

using namespace mlaq;

extern "C" {

MLAQ_API size_t mla_cache_attn_workspace_size(const mla_attn_shape* shape, const mla_kv_cache* cache) {
    CacheBytes n;
    DeviceInfo di;
    AttnPlan a;
    static const int32_t some = 0;  // the table is not looked at
    if (check_attn(shape, cache, &some, &n) != MLA_OK || current_device_info(&di) != MLA_OK ||
        !attn_plan(*shape, *cache, di.max_smem_optin, &a))
        return 0;
    return workspace_bytes(a.R, cache->Dv, di.num_sms);
}

MLAQ_API int mla_cache_attn(const mla_attn_shape* shape, const mla_kv_cache* cache, const void* q,
                            const int32_t* table, const int32_t* length, const int32_t* cu, void* out, float* lse,
                            void* workspace, size_t ws_bytes, int* dev_status, void* stream) {
    CacheBytes n;
    const int st = check_attn(shape, cache, table, &n);
    if (st != MLA_OK && st != MLA_ERR_UNSUPPORTED && st != MLA_ERR_ALIGNMENT) return st;
    const mla_attn_shape& s = *shape;
    const mla_kv_cache& c = *cache;
    if ((!cu && s.T != s.B) || (s.T > 0 && (!q || !out || !length || c.pages == 0 || s.table_width == 0)))
        return MLA_ERR_INVALID_ARG;
    if (st != MLA_OK) return st;
    const bool shared = !c.v;
    if (shared ? (c.Dk > 128 * kMaxQueryChunks || c.Dv > 512) : (c.Dk > 256 || c.Dv > 256)) return MLA_ERR_UNSUPPORTED;
    if (!aligned(q, 2) || !aligned(out, 2) || !aligned(lse, 4) || !aligned(length, 4) || !aligned(cu, 4) ||
        !aligned(dev_status, 4) || !aligned(workspace, 16))
        return MLA_ERR_ALIGNMENT;
    const int64_t q_bytes = s.T > 0 ? ((s.T - 1) * s.q_t + (s.Hq - 1) * s.q_h + c.Dk) * 2 : 0;
    const Range outs[] = {rng(out, s.T * s.Hq * c.Dv * 2), rng(lse, s.T * s.Hq * 4), rng(workspace, (int64_t)ws_bytes),
                          rng(dev_status, 4)};
    const Range ins[] = {rng(q, q_bytes), rng(c.k, n.k), rng(c.k_scales, n.k_scales), rng(c.v, n.v),
                         rng(c.v_scales, n.v_scales), rng(table, s.B * s.table_width * 4), rng(length, s.B * 4),
                         rng(cu, (s.B + 1) * 4)};
    if (any_alias(outs, ins)) return MLA_ERR_ALIAS;
    if (s.T == 0) return MLA_OK;
    DeviceInfo di;
    const int ds = current_device_info(&di);
    if (ds != MLA_OK) return ds;
    AttnPlan a;
    if (!attn_plan(s, c, di.max_smem_optin, &a)) return MLA_ERR_UNSUPPORTED;
    const int shares = di.num_sms < kMaxShares ? di.num_sms : kMaxShares;
    if (!workspace || ws_bytes < workspace_bytes(a.R, c.Dv, di.num_sms)) return MLA_ERR_WORKSPACE;

    AttnParams p{};
    p.q = static_cast<const uint16_t*>(q), p.out = static_cast<uint16_t*>(out), p.lse = lse;
    p.table = table, p.length = length, p.cu = cu, p.k_scales = c.k_scales, p.v_scales = c.v_scales;
    p.meta = static_cast<int4*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(p.meta + 2 * shares);
    p.part_o = reinterpret_cast<float*>(p.part_ml + 2 * (size_t)shares * a.R);
    p.q_t = s.q_t, p.q_h = s.q_h, p.T = s.T, p.pages = c.pages;
    p.B = (int)s.B, p.width = (int)s.table_width, p.page = c.page, p.page_shift = __builtin_ctz(c.page);
    p.block_shift = __builtin_ctz(c.block), p.marks = c.page / c.block, p.H = c.H, p.Hq = s.Hq, p.group = s.Hq / c.H;
    p.per_seq = (p.group + a.R - 1) / a.R;
    const int64_t slots = cu ? s.T * p.group / a.R + s.B : s.B * p.per_seq;
    if (slots > kI32Max) return MLA_ERR_UNSUPPORTED;
    p.slots = (int)slots;
    p.Dk = c.Dk, p.Dv = c.Dv, p.nk = a.nk, p.nv = a.nv, p.k_stages = a.k_stages, p.v_stages = a.v_stages, p.tmem_cols = a.tmem_cols;
    p.q_bufs = a.q_bufs, p.o_bufs = a.o_bufs;
    const Divisor by = divisor(p.group);
    p.group_mul = by.mul, p.group_shift = by.shift;
    p.q_vec = aligned(q, 16) && s.q_t % 8 == 0 && s.q_h % 8 == 0;
    p.scale_log2 = s.scale * 1.44269504088896341f;
    p.status = dev_status;
    const uint32_t box = c.page < kTokens ? c.page : kTokens;
    CUtensorMap km, vm;
    int ms = make_tmap_pages(&km, c.k, c.Dk, c.page, c.H, c.pages, box);
    if (ms != MLA_OK) return ms;
    vm = km;
    if (!shared) ms = make_tmap_pages(&vm, c.v, c.Dv, c.page, c.H, c.pages, box);
    if (ms != MLA_OK) return ms;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (shared)
        return a.R == 8    ? launch_attn<8, true>(p, a, km, vm, shares, cs)
               : a.R == 16 ? launch_attn<16, true>(p, a, km, vm, shares, cs)
               : a.R == 32 ? launch_attn<32, true>(p, a, km, vm, shares, cs)
                           : launch_attn<64, true>(p, a, km, vm, shares, cs);
    return a.R == 8    ? launch_attn<8, false>(p, a, km, vm, shares, cs)
           : a.R == 16 ? launch_attn<16, false>(p, a, km, vm, shares, cs)
           : a.R == 32 ? launch_attn<32, false>(p, a, km, vm, shares, cs)
                       : launch_attn<64, false>(p, a, km, vm, shares, cs);
}

}  // extern "C"

// Attention of a chunk of new tokens over the 8-bit paged cache, on the
// fifth-generation tensor cores (tcgen05, TMEM accumulators).
//
// What it computes: query i of sequence b sits at position L_b - n_b + i and
// attends causally to positions [0, p] of the sequence's 8-bit cache
// (int8_cache.cuh), query head h reading KV head h / G. A key enters the
// products as its codes less 128, exact in f16, and its scale as a factor of
// the logit in fp32. A cached value is (code - 128) * scale. It is staged for
// the tensor cores as (code - 128) * scale * 2^-e, rounded to f16 (half a step,
// 2^-11), with e of its half of the KV tile chosen by the half's largest scale
// (value_exponent): whatever the scales, no value leaves the f16 range, and
// one is below its normal part only where it is 2^-21 of the half's largest scale.
// The weights make up for it: 2^(x + e - m) for a token of logit x, m being the
// row's running maximum of x + e, and the row's sum takes them times 2^-e. (With
// the keys rounded to f16 as well the output's error was 0.00032 of its norm,
// where f16 outputs alone are off by 0.00019; it is 0.00025 so, at nearly the
// same speed. With the values as exact codes too, their scales multiplied into the
// weights, it was 0.00021, but 210 and 68 us instead of 170 and 59 for the two cases
// below, timed as calls in a row: the second factor per token doubles the reads
// of factors by every softmax thread.)
//
// Structure (one CTA per SM, persistent):
//  * A query tile is T = floor(128 / G) query tokens x the G heads of one KV
//    head, row r = (token r / G, head r % G). A KV tile is 128 tokens. S = Q K^T
//    and O += P V are M = N = K = 128 products, P over S in TMEM; two softmax
//    streams (S, O and four warps each) keep the tensor cores on one stream's
//    products while the other's softmax runs.
//  * Wide (chunks longer than T): the streams are two query tiles that share
//    every KV tile. Narrow (chunks that fit one query tile, such as drafted
//    tokens): the streams are the even and the odd KV tiles of one query tile,
//    so that the cache is read at twice the rate of one stream's chain of
//    products and softmax; the two partial results of a row meet in TMEM (softmax
//    warps w and w + 4 share its lanes).
//  * Load balance: the items (query group, KV head, sequence) form a row of
//    KV tiles, every CTA takes an equal run of it, an item cut between CTAs is
//    computed in pieces that store (max, sum, O) per row, and whoever takes the
//    last ticket merges them in their order: wide warp by warp behind the next
//    item's products, narrow all warps of the CTA at its end. Nobody waits on
//    another CTA.
//  * Staging: one TMA warp brings the codes of K (128-byte swizzle), the scales
//    and Q, one the codes of V; four warps convert them, one token (row) per
//    thread: a code becomes an exact f16 integer (a byte permute and a
//    subtraction), and for V, whose scale (times 2^-e) is thus a register, code * scale
//    is formed in f16x2 as code * hi + (code * lo) with scale = hi + lo split into
//    two f16, so that the scale's own rounding does not add to the value's
//    (RowScale). The f16 tiles are written in the 128-byte swizzled layout the
//    tensor cores read: K and V are double-buffered. Codes are finite and rows
//    past the context get scale 0, so no row needs clearing.
//  * Softmax: a row per thread, half a KV tile at a time, on logits read from
//    TMEM once. The running maximum (exp2 domain) is raised only by more than
//    8 (15 in a tile's second half), so most tiles rescale nothing; the row sum
//    adds the fp32 probabilities before they are rounded to f16 for P V. Warps
//    with no live row do no work.
// Every wait is bounded; one that runs out flags PKV_DEVERR_WAIT_TIMEOUT and
// every role stops, drains what it has in flight and leaves; TMEM is freed.
//
// Measured at 28 / 4 heads, in a graph: 512 new tokens of 8 sequences on 2048-token
// contexts 165 us, 0.38 of the measured dense rate; 5 new tokens of 64 sequences on
// contexts of 32 to 2048 tokens 57.7 us. Bound: neither memory nor the tensor cores.
// A CTA takes about 5900 cycles per KV tile (wide: 280 thousand for 47.6 tiles, with
// the launch, the scan and the merges), of which its tensor pipe is busy for 2050, as
// long as the products take, and the threads' loads and stores keep shared memory busy
// for 1690 beside the operands' 1536; narrow about 5800 and 1010. The rest is the
// streams' chains S -> softmax -> P V, whose warps wait for tensor memory and for one
// another more than for anything else, and the instruction cache, which the roles
// compete for; how it divides among these has not been measured. Tried and not kept, us for the two, against 160 / 54 of
// the form they started from (keys rounded to f16): logits in halves of 64 tokens,
// double-buffered, one issuing warp 212 / 58 (products of N = 64 read Q twice); the
// same with an issuing warp per stream 154 / 59; logits taken out of TMEM at once
// and P in its own columns 164 / 62; an issuing warp per stream with N = 128
// 172 / 54 (the streams run in step and wait for the same units); 16 TMEM columns
// per load instead of 64, 182 (against 167 then); eight converter warps 167 / 61.
// Against 164 / 56 of the present form: the waits' slow path inlined 176 / 65;
// registers moved to the softmax (setmaxnreg, inlined waits) 170 / 63; the scales
// brought in by a warp of their own 195 / 71; four warps each for K and V 183 / 67;
// the conversion rolled up to 16 channels 174 / 63; double-buffered halves with an
// issuing warp per stream 162 / 57 (timed in turn: no difference).
#pragma once

#include "int8_cache.cuh"
#include "prefill_tc.cuh"
#include "stream_int8.cuh"

namespace pkv {

struct ChunkInt8Params {
    __half* out;                  // [total, Hq, 128]
    const int32_t* block_tables;  // [B, max_blocks_per_seq]
    const int32_t* context_lens;  // [B]
    const int32_t* query_start;   // [B + 1]
    uint8_t* parts;               // [2 * CTAs][2 streams][kPartBytes]
    unsigned int* tickets;        // [CTAs] (narrow) or [CTAs][2 streams][4 warps], zero between calls
    int32_t batch, total, max_query_len;
    int32_t Hq, Hkv, G;
    int32_t max_blocks_per_seq, num_blocks, max_context_len;
    int32_t tokens;               // T: query tokens of a tile
    float logit_scale_log2;       // softmax_scale * log2(e)
};

struct ChunkInt8Shape {
    static constexpr int kKvTok = 128;
    static constexpr int kChunk = 128 * 128;            // 64 channels of 128 rows, f16: 16 KiB
    static constexpr int kTile = 2 * kChunk;            // a 128 x 128 f16 tile
    static constexpr int kRaw = 128 * 128;              // codes of K or V of a KV tile
    static constexpr int kScales = 8 * 128;             // scales of a KV tile: 8 pages x (16 K, 16 V)
    static constexpr int kBarBytes = 320;
    static constexpr int kFactors = 128 * 4 + 2 * 8;    // logit factors of a KV tile's tokens; e, 2^-e of its halves
    static constexpr int kFactorSlots = 3;
    // Q A | Q B or a second raw stage | K x 2 | V x 2 | raw K, V | scales | factors x 3 | barriers and words.
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = 2 * kTile;
    static constexpr int kOffV = kOffK + 2 * kTile;
    static constexpr int kOffRaw = kOffV + 2 * kTile;
    static constexpr int kOffScales = kOffRaw + 2 * kRaw;
    static constexpr int kOffFactors = kOffScales + kScales;
    static constexpr int kOffBars = kOffFactors + kFactorSlots * kFactors;
    static constexpr int kOffWords = kOffBars + kBarBytes;   // first sequence [2], abort flag, cut items
    static constexpr int kSmemBytes = kOffWords + 96;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory of one SM");
    static constexpr int kSoftmaxWarps = 8;
    static constexpr int kConvertWarp = 8;              // 8..11
    static constexpr int kTmaKWarp = 12, kTmaVWarp = 13, kMmaWarp = 14;
    static constexpr int kThreads = 32 * 15;
    static constexpr uint32_t kTmemCols = 512;
    // log2 of the largest probability of a KV tile's first half (64 tokens), and of its second half: f16 holds it
    static constexpr float kRescaleThreshold = 8.f, kSecondThreshold = 15.f;
    static constexpr int kPartBytes = 128 * 128 * 4 + 128 * 8;
};

// The power of two that the V scales of half a KV tile (64 tokens; `most` the largest) are brought to f16 by:
// scale * 2^-e is below 2^8, so that no code takes it past the f16 range, and the largest at least 2^7 unless e is
// at its least. (Rows of scales below 2^-33 are zeros in any f16 output.)
__device__ __forceinline__ int value_exponent(float most) {
    return max((int)((__float_as_uint(most) >> 23) & 0xff) - 127 - 7, -40);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// A token's scale for the conversion: scale = (hi + lo) * post, hi and lo f16. post is 1 unless the
// scale is small (below 2^-10, where lo would lose bits to the subnormal range): then hi + lo is the
// scale brought into [2^-7, 2^-6) and post the power of two that takes it back. A value so formed is
// off by at most 1.04 half steps of f16 (1 but for what lo loses), and by half a subnormal step more
// where a small row's value is subnormal (a second rounding, by post).
struct RowScale {
    __half2 hi, lo, post;
    bool small;
};
__device__ __forceinline__ RowScale split_scale(float s) {
    RowScale r;
    r.small = fabsf(s) < 9.765625e-4f && s != 0.f;
    float post = 1.f;
    if (r.small) {
        const int e = max((int)((__float_as_uint(s) >> 23) & 0xff) - 127 + 7, -24);   // post = 2^e >= 2^-24
        post = __uint_as_float((uint32_t)(e + 127) << 23);
        s *= __uint_as_float((uint32_t)(127 - e) << 23);
    }
    const __half hi = __float2half_rn(s);
    r.hi = __half2half2(hi);
    r.lo = __half2half2(__float2half_rn(s - __half2float(hi)));
    r.post = __half2half2(__float2half_rn(post));
    return r;
}
// Two integers times (hi + lo), rounded to f16.
__device__ __forceinline__ uint32_t scaled(uint32_t a, const RowScale& s) {
    const __half2 x = *reinterpret_cast<const __half2*>(&a), u = __hfma2(x, s.hi, __hmul2(x, s.lo));
    return *reinterpret_cast<const uint32_t*>(&u);
}
__device__ __forceinline__ uint32_t times(uint32_t a, __half2 f) {
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&a), f);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Untiled bulk copy global -> shared of a multiple of 16 bytes, completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// Packed fp32 pairs: one instruction for two lanes of arithmetic.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// 32 factors (pairs) at shared address `f`.
__device__ __forceinline__ void load_factors(uint32_t f, uint64_t (&v)[16]) {
#pragma unroll
    for (int e = 0; e < 16; e += 2)
        asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[e]), "=l"(v[e + 1]) : "r"(f + 8 * e) : "memory");
}
// x[e] = x[e] * factor[e] + m over 32 tokens from q on.
template <int kCols>
__device__ __forceinline__ void relative_logits(float (&x)[kCols], int q, const uint64_t (&v)[16], uint64_t m) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
        unpack_f32x2(fma_f32x2(pack_f32x2(x[q + 2 * e], x[q + 2 * e + 1]), v[e], m), x[q + 2 * e], x[q + 2 * e + 1]);
}
// Logits of consecutive tokens, those past number `left` hidden.
template <int kCols>
__device__ __forceinline__ void mask_past(float (&x)[kCols], int left) {
#pragma unroll
    for (int e = 0; e < kCols; ++e) x[e] = e <= left ? x[e] : -INFINITY;
}

// The products of a KV tile, executed by the whole warp: one elected lane issues each. (Issued from a branch of
// one lane, every operand is moved to the uniform registers one product at a time, through a queue that the
// softmax keeps full: 100 to 250 cycles a product, where the product itself takes 72.)
// D = A B^T over 128 channels: A and B K-major 128-byte-swizzled tiles of two 64-channel halves.
__device__ __forceinline__ void umma_tile_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred e, z, o;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 z, 0, 0;\n\tsetp.eq.u32 o, 0, 0;\n\t"
        "add.s64 a, %1, 0;\n\tadd.s64 b, %2, 0;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, z;\n\t"
        "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, o;\n\t"
        "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, o;\n\t"
        "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, o;\n\t"
        "add.s64 a, %1, 1024;\n\tadd.s64 b, %2, 1024;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, o;\n\t"
        "add.s64 a, %1, 1026;\n\tadd.s64 b, %2, 1026;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, o;\n\t"
        "add.s64 a, %1, 1028;\n\tadd.s64 b, %2, 1028;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, o;\n\t"
        "add.s64 a, %1, 1030;\n\tadd.s64 b, %2, 1030;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, o;\n\t"
        "}"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc) : "memory");
}
// D (+)= P V over 64 tokens: P in TMEM (two per column), V MN-major; `accumulate` 0 overwrites D.
__device__ __forceinline__ void umma_half_ts(uint32_t d, uint32_t p, uint64_t v, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, f, o;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 f, %4, 0;\n\tsetp.eq.u32 o, 0, 0;\n\t"
        "add.s32 a, %1, 0;\n\tadd.s64 b, %2, 0;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, f;\n\t"
        "add.s32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, o;\n\t"
        "add.s32 a, %1, 16;\n\tadd.s64 b, %2, 256;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, o;\n\t"
        "add.s32 a, %1, 24;\n\tadd.s64 b, %2, 384;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, o;\n\t"
        "}"
        :: "r"(d), "r"(p), "l"(v), "r"(idesc), "r"(accumulate) : "memory");
}
// Arrives on `bar` when all products issued before (by the same elected lane) have completed.
__device__ __forceinline__ void umma_commit_elected(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        :: "r"(bar) : "memory");
}

// 16 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        :: "r"(taddr), "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
           "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
           "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
           "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
           "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
           "r"(__float_as_uint(v[15]))
        : "memory");
}

// 32 or 64 TMEM columns of this thread's lane, in one round trip.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&v)[32]) { tmem_ld32(taddr, v); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&v)[64]) {
    tmem_ld32x2(taddr, *reinterpret_cast<float (*)[32]>(&v[0]), taddr + 32, *reinterpret_cast<float (*)[32]>(&v[32]));
}

// The rest of a bounded wait, out of line (the many places that wait would fill the instruction cache with it):
// false, and the abort flag at shared address `abort` set, when the limit has run out, or another role's has.
__device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, uint32_t abort) {
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 0;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 63u) {
            uint32_t given_up;
            asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(given_up) : "r"(abort) : "memory");
            if (given_up) return false;
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                flag_error(PKV_DEVERR_WAIT_TIMEOUT);
                asm volatile("st.volatile.shared.u32 [%0], %1;" :: "r"(abort), "r"(1u) : "memory");
                return false;
            }
        }
    }
}

template <bool kNarrow>
__global__ void __launch_bounds__(ChunkInt8Shape::kThreads, 1)
chunk_int8_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_s,
                  const ChunkInt8Params p) {
    using S = ChunkInt8Shape;
    constexpr int kCols = 64;                            // logits a softmax thread holds
    constexpr int kRawStages = kNarrow ? 2 : 1;
    constexpr int kQTiles = kNarrow ? 1 : 2;             // query tiles of an item
    constexpr int kMinTiles = kNarrow ? 2 : 4;           // fewest KV tiles a CTA is given
    extern __shared__ uint8_t smem_raw[];
    // Without a static part the dynamic shared memory starts at a multiple of 1024 bytes, and its 226.5 KiB
    // leave no room to align it here. (An alignment on the declaration would pad every kernel of the library.)
    const uint32_t base = smem_u32(smem_raw);
    if (base & 1023u) {
        flag_error(PKV_DEVERR_WAIT_TIMEOUT);             // never seen: no operand tile could be addressed
        return;
    }
    long long* s_red = reinterpret_cast<long long*>(smem_raw + S::kOffFactors);   // [15], before the first factors
    long long* s_first = reinterpret_cast<long long*>(smem_raw + S::kOffWords);   // [2]
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_first + 2);
    // the items this CTA holds a piece of, as the softmax meets them
    struct CutItem { long long u; int row0, nq, g, ntiles; };
    CutItem* s_cut = reinterpret_cast<CutItem*>(smem_raw + S::kOffWords + 32);    // [2]
    int* s_cuts = reinterpret_cast<int*>(smem_raw + S::kOffWords + 20);           // how many
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.G, T = p.tokens;
    const int per_item = kQTiles * T;                    // query tokens of an item

    grid_dependency_wait();
    grid_dependents_launch();
    const int cap = min(p.max_context_len, p.max_blocks_per_seq * kPageRows);
    // lengths of sequence b; false (no queries) when they are inconsistent
    auto lengths = [&](int b, int& qs0, int& n, int& L) -> bool {
        qs0 = __ldg(p.query_start + b);
        const int qs1 = __ldg(p.query_start + b + 1);
        L = __ldg(p.context_lens + b);
        n = qs1 - qs0;
        return !(qs0 < 0 || qs1 < qs0 || qs1 > p.total || n > p.max_query_len || L < n || L > cap);
    };
    // KV tiles of all items of sequence b under one KV head
    auto seq_tiles = [&](int b) -> int64_t {
        int qs0, n, L;
        if (!lengths(b, qs0, n, L)) return 0;
        int64_t s = 0;
        for (int i0 = 0; i0 < n; i0 += per_item) s += (L - n + min(i0 + per_item, n) - 1) / S::kKvTok + 1;
        return s;
    };
    // inclusive scan of x over the block; total: the block's sum (ends synchronised)
    auto block_scan = [&](int64_t x, int64_t& total) -> int64_t {
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        if (lane == 31) s_red[warp] = x;
        __syncthreads();
        int64_t before = 0;
        total = 0;
        for (int i = 0; i < S::kThreads / 32; ++i) {
            before += i < warp ? s_red[i] : 0;
            total += s_red[i];
        }
        __syncthreads();
        return before + x;
    };
    // ---- the batch's KV tiles ("units") and this CTA's run of them ----
    int64_t U = 0, u_lo, u_hi;
    int ctas;
    {
        int64_t my_w = 0, my_incl = 0, first_total = 0;
        for (int b0 = 0; b0 < p.batch; b0 += S::kThreads) {
            const int b = b0 + (int)threadIdx.x;
            int64_t w = 0;
            if (b < p.batch) {
                w = seq_tiles(b) * p.Hkv;
                int qs0, n, L;
                if (blockIdx.x == 0 && !lengths(b, qs0, n, L)) flag_error(PKV_DEVERR_CONTEXT_LEN);
            }
            int64_t total;
            const int64_t incl = U + block_scan(w, total);
            if (b0 == 0) {
                my_w = w;
                my_incl = incl;
                first_total = total;
            }
            U += total;
        }
        ctas = (int)max((int64_t)1, min((int64_t)gridDim.x, U / kMinTiles));
        u_lo = blockIdx.x < ctas ? (int64_t)blockIdx.x * U / ctas : U;
        u_hi = blockIdx.x < ctas ? ((int64_t)blockIdx.x + 1) * U / ctas : U;
        if (u_lo < u_hi) {
            if (my_w > 0 && my_incl - my_w <= u_lo && u_lo < my_incl) {
                s_first[0] = threadIdx.x;
                s_first[1] = my_incl - my_w;
            }
            int64_t base = first_total;                  // more sequences than threads: scan again
            for (int b0 = S::kThreads; b0 < p.batch && base <= u_lo; b0 += S::kThreads) {
                const int b = b0 + (int)threadIdx.x;
                const int64_t w = b < p.batch ? seq_tiles(b) * p.Hkv : 0;
                int64_t total;
                const int64_t incl = base + block_scan(w, total);
                if (w > 0 && incl - w <= u_lo && u_lo < incl) {
                    s_first[0] = b;
                    s_first[1] = incl - w;
                }
                base += total;
            }
        }
        __syncthreads();
    }
    if (u_lo >= u_hi) return;                            // no work for this CTA (uniform)
    auto range_lo = [&](int c) -> int64_t { return (int64_t)c * U / ctas; };
    auto cta_of = [&](int64_t u) -> int {
        int c = (int)min((int64_t)ctas - 1, u * ctas / U);
        while (c > 0 && range_lo(c) > u) --c;
        while (c + 1 < ctas && range_lo(c + 1) <= u) ++c;
        return c;
    };
    // The CTA's pieces, in order: KV tiles [j0, j1) of an item.
    struct Cursor { int b, g, q; int64_t u; };
    struct Piece { int b, g, row0, nq, pos0, ntiles, npages, L, j0, j1; int64_t u; };
    Cursor start;
    {
        start.b = (int)s_first[0];
        const int64_t per_g = seq_tiles(start.b);
        start.g = (int)((u_lo - s_first[1]) / per_g);
        start.u = s_first[1] + start.g * per_g;
        start.q = 0;
        int qs0, n, L;
        lengths(start.b, qs0, n, L);
        for (int i0 = 0; i0 < n; i0 += per_item) {
            const int ntiles = (L - n + min(i0 + per_item, n) - 1) / S::kKvTok + 1;
            if (start.u + ntiles > u_lo) break;
            start.u += ntiles;
            ++start.q;
        }
    }
    // where CTA c keeps its piece of an item (stream t): slot 0 if the piece starts the CTA's run, as it does in every
    // CTA behind the item's first one, else slot 1 (the CTA's last piece)
    auto part_of = [&](int c, int slot, int t) -> uint8_t* {
        return p.parts + ((int64_t)(2 * c + slot) * 2 + t) * S::kPartBytes;
    };
    auto next_piece = [&](Cursor& cu, Piece& pc) -> bool {
        while (cu.u < u_hi && cu.b < p.batch) {
            int qs0, n, L;
            const bool ok = lengths(cu.b, qs0, n, L);
            const int i0 = cu.q * per_item;
            if (!ok || i0 >= n) {                        // next KV head, or next sequence
                cu.q = 0;
                if (!ok || n == 0 || ++cu.g == p.Hkv) {
                    cu.g = 0;
                    ++cu.b;
                }
                continue;
            }
            pc.b = cu.b;
            pc.g = cu.g;
            pc.row0 = qs0 + i0;
            pc.nq = min(per_item, n - i0);
            pc.pos0 = L - n + i0;
            const int p_max = pc.pos0 + pc.nq - 1;
            pc.ntiles = p_max / S::kKvTok + 1;
            pc.npages = p_max / kPageRows + 1;
            pc.L = L;
            pc.u = cu.u;
            pc.j0 = (int)(max(cu.u, u_lo) - cu.u);
            pc.j1 = (int)(min(cu.u + pc.ntiles, u_hi) - cu.u);
            cu.u += pc.ntiles;
            ++cu.q;
            return true;
        }
        return false;
    };

    // ---- shared memory, barriers, TMEM ----
    auto q_s = [&](int t) { return base + S::kOffQ + t * S::kTile; };
    auto k_s = [&](int s) { return base + S::kOffK + s * S::kTile; };
    auto v_s = [&](int s) { return base + S::kOffV + s * S::kTile; };
    // raw stage 0 has its own place, stage 1 (narrow) that of the second query tile
    auto raw_k = [&](int s) { return base + (s ? S::kOffQ + S::kTile : S::kOffRaw); };
    auto raw_v = [&](int s) { return raw_k(s) + S::kRaw; };
    const uint32_t raw_sc = base + S::kOffScales;
    auto factors = [&](int s) { return base + S::kOffFactors + s * S::kFactors; };
    const uint32_t bars = base + S::kOffBars;
    const uint32_t q_full = bars, q_empty = bars + 8, drain = bars + 16;
    auto s_full = [&](int t) { return bars + 24 + 8u * t; };
    auto p_full = [&](int t, int h) { return bars + 40 + 8u * t + (h ? 192u : 0u); };   // halves of 64 tokens
    auto o_done = [&](int t) { return bars + 56 + 8u * t; };
    auto o_free = [&](int t) { return bars + 72 + 8u * t; };
    auto k_full = [&](int s) { return bars + 88 + 8u * s; };
    auto k_empty = [&](int s) { return bars + 104 + 8u * s; };
    auto v_full = [&](int s) { return bars + 120 + 8u * s; };
    auto v_empty = [&](int s) { return bars + 136 + 8u * s; };
    auto rk_full = [&](int s) { return bars + 152 + 8u * s; };
    auto rk_empty = [&](int s) { return bars + 168 + 8u * s; };
    auto rv_full = [&](int s) { return bars + 184 + 8u * s; };
    auto rv_empty = [&](int s) { return bars + 200 + 8u * s; };
    // narrow: the odd stream's (m, l) of a piece are in TMEM; the even stream has read them
    const uint32_t x_full = bars + 216, x_read = bars + 224;
    const uint32_t tmem_slot = bars + 248;
    // scales of a KV tile: raw, and as the logit factors of its tokens; O_t has the first half of P V
    const uint32_t rs_full = bars + 256, rs_empty = bars + 264;
    auto f_full = [&](int s) { return bars + 272 + 8u * s; };
    auto o_half = [&](int t) { return bars + 296 + 8u * t; };
    const uint32_t merge_bar = bars + 312;
    const int rows = G * T;                              // rows of Q the TMA fills; the rest stay zero
    if (threadIdx.x == 0) {
        *s_abort = 0;
        *s_cuts = 0;
        mbar_init(x_full, 128);
        mbar_init(x_read, 128);
        mbar_init(merge_bar, 1);
        mbar_init(rs_full, 1);
        mbar_init(rs_empty, 4);
        for (int s = 0; s < S::kFactorSlots; ++s) mbar_init(f_full(s), 4);
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(drain, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(p_full(t, 0), 128);
            mbar_init(p_full(t, 1), 128);
            mbar_init(o_done(t), 1);
            mbar_init(o_half(t), 1);
            mbar_init(o_free(t), 128);
            mbar_init(k_full(t), 4);
            mbar_init(k_empty(t), 1);
            mbar_init(v_full(t), 4);
            mbar_init(v_empty(t), 1);
            mbar_init(rk_full(t), 1);
            mbar_init(rk_empty(t), 4);
            mbar_init(rv_full(t), 1);
            mbar_init(rv_empty(t), 4);
        }
        mbar_init_fence();
    }
    for (int i = threadIdx.x; i < kQTiles * (128 - rows) * 16; i += S::kThreads) {
        const int t = i / ((128 - rows) * 16), k = i % ((128 - rows) * 16);
        const int r = rows + k / 16, part = k % 16;
        const uint32_t a = q_s(t) + (part >> 3) * S::kChunk + r * 128 + (part & 7) * 16;
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" :: "r"(a), "r"(0u) : "memory");
    }
    fence_proxy_async_shared();
    if (warp == S::kMmaWarp) {
        tmem_alloc(tmem_slot, S::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot) : "memory");
    auto tmem_s = [&](int t) { return tmem + 128u * t; };
    auto tmem_o = [&](int t) { return tmem + 256u + 128u * t; };

    // Bounded wait that also gives up once another role has given up.
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        return mbar_try_wait(bar, parity) || wait_longer(bar, parity, smem_u32(const_cast<int*>(s_abort)));
    };
    auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(bar, parity)); };

    if (warp == S::kTmaKWarp || warp == S::kTmaVWarp) {
        // ================= TMA: codes of K (with Q and the scales), or of V =================
        const bool is_k = warp == S::kTmaKWarp;
        const CUtensorMap* map = is_k ? &tm_k : &tm_v;
        if (lane == 0) {
            prefetch_tensormap(map);
            if (is_k) {
                prefetch_tensormap(&tm_q);
                prefetch_tensormap(&tm_s);
            }
        }
        auto full = [&](int s) { return is_k ? rk_full(s) : rv_full(s); };
        auto empty = [&](int s) { return is_k ? rk_empty(s) : rv_empty(s); };
        int gj = 0, k = 0, scales_short = 0;             // KV tiles, pieces; a tile whose scales were not asked for
        bool ok = true;
        Cursor cu = start;
        Piece pc;
        while (ok && next_piece(cu, pc)) {
            const int32_t* bt = p.block_tables + (int64_t)pc.b * p.max_blocks_per_seq;
            for (int j = pc.j0; j < pc.j1; ++j, ++gj) {
                const int s = gj % kRawStages;
                // a page per lane; pages past the item's last position are not loaded (their scales are
                // taken as 0 by position)
                const int pages = min(8, pc.npages - 8 * j);
                int pb = -1;
                if (lane < pages) {
                    pb = __ldg(bt + 8 * j + lane);
                    if (pb < 0 || pb >= p.num_blocks) {  // outside the pool: codes and scales read as zeros
                        if (is_k) flag_error(PKV_DEVERR_BLOCK_ID);
                        pb = -1;
                    }
                }
                if (gj >= kRawStages && !(ok = wait_all(empty(s), ((gj / kRawStages) - 1) & 1))) break;
                if (lane == 0) mbar_arrive_expect_tx(full(s), pages * 2048);
                __syncwarp();
                if (lane < pages) {
                    fence_proxy_async_shared();          // the converters' reads of the stage come first
                    const uint32_t dst = (is_k ? raw_k(s) : raw_v(s)) + lane * 2048;
                    tma_load_3d_reused(dst, map, full(s), 0, pc.g, pb * kPageRows);
                }
                __syncwarp();
                if (is_k) {                              // the scales' one stage, behind the codes
                    if (gj >= 1 && !(ok = wait_all(rs_empty, (gj - 1) & 1))) {
                        ++gj;
                        ++scales_short;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(rs_full, pages * 128);
                    __syncwarp();
                    if (lane < pages) {
                        fence_proxy_async_shared();
                        tma_load_3d_reused(raw_sc + lane * 128, &tm_s, rs_full, 0, pc.g, pb);
                    }
                    __syncwarp();
                }
                if (is_k && j == pc.j0) {                // the piece's Q, behind its first K
                    if (k >= 1 && !(ok = wait_all(q_empty, (k - 1) & 1))) {
                        ++gj;
                        break;
                    }
                    if (lane == 0) {
                        mbar_arrive_expect_tx(q_full, kQTiles * 2 * 128 * rows);
                        for (int t = 0; t < kQTiles; ++t) {
                            tma_load_3d_reused(q_s(t), &tm_q, q_full, 0, pc.g * G, pc.row0 + t * T);
                            tma_load_3d_reused(q_s(t) + S::kChunk, &tm_q, q_full, 64, pc.g * G, pc.row0 + t * T);
                        }
                    }
                    __syncwarp();
                    ++k;
                }
            }
        }
        // nothing of ours may be in flight when the CTA leaves
        for (int j = max(0, gj - kRawStages); j < gj; ++j) mbar_wait(full(j % kRawStages), (j / kRawStages) & 1);
        if (is_k && gj > scales_short) mbar_wait(rs_full, (gj - scales_short - 1) & 1);
        if (is_k && k >= 1) mbar_wait(q_full, (k - 1) & 1);
    } else if (warp >= S::kConvertWarp && warp < S::kConvertWarp + 4) {
        // ========================= codes to f16 tiles: a token per thread =========================
        const int row = 32 * (warp & 3) + lane;                    // token of the KV tile
        const uint32_t sw = (uint32_t)(row & 7);
        // the raw tile at `src` into the f16 tile at `dst`, 64 channels at a time (kept as a loop: the roles' code
        // competes for the instruction cache): K as the codes' integers, V times this row's scale
        auto convert = [&](bool is_k, uint32_t src, uint32_t dst, float scale) {
            const RowScale s = split_scale(scale);
            const bool any_small = __any_sync(0xffffffffu, s.small);
            const uint32_t in = src + row * 128, out = dst + row * 128;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                uint4 w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) w[c] = lds128(in + (((4 * h + c) ^ sw) << 4));
#pragma unroll
                for (int c = 0; c < 4; ++c) {                      // 16 channels
                    uint32_t d[8];
                    codes_to_half2x2(w[c].x, d[0], d[1]);
                    codes_to_half2x2(w[c].y, d[2], d[3]);
                    codes_to_half2x2(w[c].z, d[4], d[5]);
                    codes_to_half2x2(w[c].w, d[6], d[7]);
                    if (!is_k) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) d[e] = scaled(d[e], s);
                        if (any_small) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) d[e] = times(d[e], s.post);
                        }
                    }
                    const uint32_t o = out + h * S::kChunk;
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                                 :: "r"(o + (((2 * c) ^ sw) << 4)), "r"(d[0]), "r"(d[1]), "r"(d[2]), "r"(d[3]) : "memory");
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                                 :: "r"(o + (((2 * c + 1) ^ sw) << 4)), "r"(d[4]), "r"(d[5]), "r"(d[6]), "r"(d[7]) : "memory");
                }
            }
        };
        // the scale of KV tile j's row r (`which` 0: K, 64: V): 0 past the context; outside [0, 2^60] flagged and 0
        auto row_scale = [&](const Piece& pc, int j, int r, uint32_t which) -> float {
            const float s = lds32(raw_sc + (uint32_t)((r >> 4) * 128 + (r & 15) * 4) + which);
            const bool live = j * S::kKvTok + r < min(pc.L, pc.npages * kPageRows);
            const bool fine = s >= 0.f && s <= kScaleMax;
            if (live && !fine) flag_error(PKV_DEVERR_SCALE);
            return live && fine ? s : 0.f;
        };
        // stages the K (with its tokens' logit factors) or V of KV tile g, the piece's `first` or not; false when a
        // wait ran out
        auto stage_tile = [&](bool is_k, int g, bool first, float scale, int exponent) -> bool {
            const int s = g % kRawStages, d = g & 1;
            if (!wait_all(is_k ? rk_full(s) : rv_full(s), (g / kRawStages) & 1)) return false;
            if (g >= 2 && !wait_all(is_k ? k_empty(d) : v_empty(d), ((g >> 1) - 1) & 1)) return false;
            if (is_k) {
                // Tile g - 3, whose slot this is, has left the softmax: wide, as both streams' S of tile g - 2 is
                // there; narrow, when its P V is done. (A piece's first K comes behind V of tile g - 1, which waited
                // for just that, and whose own P V may have taken the barrier a phase further by now.)
                if (kNarrow && !first && g >= 3 && !wait_all(v_empty(d ^ 1), ((g - 3) >> 1) & 1)) return false;
                const int slot = g % S::kFactorSlots;
                asm volatile("st.shared.f32 [%0], %1;" :: "r"(factors(slot) + 4 * row), "f"(scale) : "memory");
                if ((row & 63) == 0)
                    asm volatile("st.shared.v2.f32 [%0], {%1, %2};"
                                 :: "r"(factors(slot) + 512 + (row >> 3)), "f"((float)exponent), "f"(power_of_two(-exponent))
                                 : "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(f_full(slot));
            }
            convert(is_k, is_k ? raw_k(s) : raw_v(s), is_k ? k_s(d) : v_s(d), scale);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(is_k ? rk_empty(s) : rv_empty(s));
                mbar_arrive(is_k ? k_full(d) : v_full(d));
            }
            return true;
        };
        Cursor cu = start;
        Piece pc;
        int gj = 0;                                                // KV tiles of earlier pieces
        bool ok = true;
        while (ok && next_piece(cu, pc)) {
            const int n = pc.j1 - pc.j0;
            // K(0), K(1), V(0), K(2), V(1), ..., K(n - 1), V(n - 2), V(n - 1)
            float v_scale = 0.f, v_next = 0.f;                     // in units of their half's 2^e
            for (int step = 0; step < 2 * n; ++step) {
                const bool is_k = step < 2 * n - 1 && (step == 0 || (step & 1));
                const int i = is_k ? (step + 1) >> 1 : step == 2 * n - 1 ? n - 1 : (step >> 1) - 1;
                float scale = v_scale;
                int exponent = 0;
                if (is_k) {
                    if (!(ok = wait_all(rs_full, (gj + i) & 1))) break;
                    scale = row_scale(pc, pc.j0 + i, row, 0) * p.logit_scale_log2;
                    v_next = row_scale(pc, pc.j0 + i, row, 64);
                    // (the half's other 32 tokens are another warp's: both come to the same exponent)
                    exponent = value_exponent(warp_max(fmaxf(v_next, row_scale(pc, pc.j0 + i, row ^ 32, 64))));
                    v_next *= power_of_two(-exponent);
                    if (i == 0) v_scale = v_next;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(rs_empty);
                }
                if (!(ok = stage_tile(is_k, gj + i, i == 0, scale, exponent))) break;
                if (!is_k) v_scale = v_next;
            }
            gj += n;
        }
    } else if (warp == S::kMmaWarp) {
        // ===================================== MMA =====================================
        constexpr uint32_t kIdescS = umma_idesc_f16(128, 128, 0);    // Q K^T: both K-major
        constexpr uint32_t kIdescPV = umma_idesc_f16(128, 128, 1);   // P V: V is MN-major
        // S_t = Q K(gg)^T, once stream t's previous O_t += P_t V (its cnt-th) has read P_t out of S_t
        auto issue_s = [&](int t, int gg, int cnt, bool free_k, bool last) -> bool {
            if (cnt >= 1 && !wait_all(o_done(t), (cnt - 1) & 1)) return false;
            tc_fence_after();
            const int s = gg & 1;
            umma_tile_ss(tmem_s(t), umma_desc_sw128(q_s(kNarrow ? 0 : t), 16, 1024), umma_desc_sw128(k_s(s), 16, 1024),
                         kIdescS);
            umma_commit_elected(s_full(t));
            if (free_k) umma_commit_elected(k_empty(s));
            if (last) umma_commit_elected(q_empty);
            return true;
        };
        // O_t += P_t V(gg); `first`: the piece's first product on the stream overwrites O_t
        auto issue_pv = [&](int t, int gg, int cnt, bool free_v, bool first) -> bool {
            const int s = gg & 1;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {                // as each half of P (64 tokens) comes in
                if (!wait_all(p_full(t, h), cnt & 1)) return false;
                tc_fence_after();
                umma_half_ts(tmem_o(t), tmem_s(t) + 32 * h, umma_desc_sw128(v_s(s) + 8192 * h, S::kChunk, 1024), kIdescPV,
                             first && h == 0 ? 0u : 1u);
                umma_commit_elected(h ? o_done(t) : o_half(t));
            }
            if (free_v) umma_commit_elected(v_empty(s));
            return true;
        };
        int gj = 0, k = 0;
        int cnt[2] = {0, 0}, used[2] = {0, 0};           // products and pieces of each stream so far
        bool ok = true;
        Cursor cu = start;
        Piece pc;
        while (ok && next_piece(cu, pc)) {
            int n = pc.j1 - pc.j0;
            asm volatile("" : "+r"(n));                  // kept in a register for the issue loop
            if (!(ok = wait_all(q_full, k & 1))) break;
            if constexpr (kNarrow) {
                // KV tile i on stream i & 1: S(0), S(1), then P V(i), S(i + 2)
                auto s_of = [&](int i) -> bool {
                    return wait_all(k_full((gj + i) & 1), ((gj + i) >> 1) & 1) &&
                           issue_s(i & 1, gj + i, (i & 1 ? cnt[1] : cnt[0]) + (i >> 1), true, i == n - 1);
                };
                ok = s_of(0);
                // the first S on the odd stream overwrites the (m, l) of its previous piece
                if (ok && n > 1 && used[1] >= 1) ok = wait_all(x_read, (used[1] - 1) & 1);
                if (ok && n > 1) ok = s_of(1);
                for (int i = 0; ok && i < n; ++i) {
                    const int t = i & 1;
                    if (!(ok = wait_all(v_full((gj + i) & 1), ((gj + i) >> 1) & 1))) break;
                    const int u = t ? used[1] : used[0];
                    if (i < 2 && u >= 1 && !(ok = wait_all(o_free(t), (u - 1) & 1))) break;
                    ok = issue_pv(t, gj + i, (t ? cnt[1] : cnt[0]) + (i >> 1), true, i < 2);
                    if (ok && i + 2 < n) ok = s_of(i + 2);
                }
                cnt[0] += (n + 1) >> 1;
                cnt[1] += n >> 1;
                ++used[0];
                used[1] += n > 1 ? 1 : 0;
            } else {
                if (!(ok = wait_all(k_full(gj & 1), (gj >> 1) & 1))) break;
                for (int t = 0; ok && t < 2; ++t) ok = issue_s(t, gj, gj, t == 1, t == 1 && n == 1);
                // per KV tile: O_A += P_A V, S_A of the next, O_B += P_B V, S_B of the next
                for (int i = 0; ok && i < n; ++i) {
                    const int gg = gj + i;
                    if (!(ok = wait_all(v_full(gg & 1), (gg >> 1) & 1))) break;
                    const bool more = i + 1 < n;
                    for (int t = 0; ok && t < 2; ++t) {
                        if (i == 0 && k >= 1 && !(ok = wait_all(o_free(t), (k - 1) & 1))) break;
                        ok = issue_pv(t, gg, gg, t == 1, i == 0);
                        if (ok && more && t == 0) ok = wait_all(k_full((gg + 1) & 1), ((gg + 1) >> 1) & 1);
                        if (ok && more) ok = issue_s(t, gg + 1, gg + 1, t == 1, t == 1 && i + 2 == n);
                    }
                }
            }
            gj += n;
            ++k;
        }
        umma_commit_elected(drain);                      // every product has completed before TMEM is freed
        __syncwarp();
        mbar_wait(drain, 0);
    } else {
        // =================================== softmax ===================================
        const int quarter = warp & 3, t = warp >> 2;             // rows, and the stream served
        const int r = 32 * quarter + lane;                       // row = TMEM lane
        const int ti = r / G, hh = r - ti * G;
        const int qi = (kNarrow ? 0 : t * T) + ti;               // query within the item
        const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
        const uint32_t s_row = tmem_s(t) + lane_base, o_row = tmem_o(t) + lane_base;
        int gj = 0, cnt = 0, exchanges = 0;                              // the stream's KV tiles; rows handed over
        bool ok = true;
        Cursor cu = start;
        Piece pc;
        while (ok && next_piece(cu, pc)) {
            const int n = pc.j1 - pc.j0;
            const int mine = kNarrow ? (n + 1 - t) >> 1 : n;     // KV tiles of this stream
            const int g0 = gj + (kNarrow ? t : 0);               // the CTA's number of the stream's first tile
            gj += n;
            if (mine == 0) continue;                             // a one-tile piece has no odd stream
            const bool valid = r < rows && qi < pc.nq;
            const bool idle = !__any_sync(0xffffffffu, valid);
            const int prow = pc.pos0 + min(qi, pc.nq - 1);       // causal limit of the row
            const int first_pos = pc.pos0 + (kNarrow ? 0 : t * T);
            float m_run = -INFINITY, l_run = 0.f;
            for (int i = 0; i < mine; ++i, ++cnt) {
                if (!(ok = wait_all(s_full(t), cnt & 1))) break;
                if (idle) {                                      // no live row in this warp: P is not used
                    mbar_arrive(p_full(t, 0));
                    mbar_arrive(p_full(t, 1));
                    continue;
                }
                tc_fence_after();
                const int t0 = (pc.j0 + (kNarrow ? 2 * i + t : i)) * S::kKvTok;
                const bool edge = t0 + S::kKvTok - 1 > first_pos;
                const int g = g0 + (kNarrow ? 2 * i : i);
                if (!(ok = wait_all(f_full(g % S::kFactorSlots), (g / S::kFactorSlots) & 1))) break;
                // The tile's halves of 64 tokens, each a step of the online softmax on logits read once (a loop, not
                // unrolled code: see the conversion), so that P V starts on the first while the second is worked
                // on. The logits, the sums over the codes times the tokens' factors, plus the half's e, are taken
                // relative to the running maximum at once; where one lies above it by more than 8 (in the second half
                // 15) the maximum is raised, and O and the sum are scaled, unless they are 0: in the second half the
                // P V of the first has to be in O by then.
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const uint32_t f = factors(g % S::kFactorSlots) + 4 * kCols * h;
                    // e and 2^-e of the half's V scales (before the logits: read behind them, e costs 100 bytes of spills)
                    const uint32_t ex = factors(g % S::kFactorSlots) + 512 + 8 * h;
                    const float e_half = lds32(ex);
                    uint64_t v[16];
                    load_factors(f, v);                          // (behind the logits' round trip)
                    float x[kCols];
                    tmem_ld_cols(s_row + kCols * h, x);
                    const bool fresh = m_run == -INFINITY;       // the row has seen no position
                    const float m_use = fresh ? 0.f : m_run;
                    const float e_less_m = e_half - m_use;
                    const uint64_t m2 = pack_f32x2(e_less_m, e_less_m);
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    relative_logits(x, 0, v, m2);
                    load_factors(f + 128, v);
                    relative_logits(x, 32, v, m2);
                    if (edge) mask_past(x, prow - t0 - kCols * h);   // (after the product: a factor may be 0)
#pragma unroll
                    for (int e = 0; e < kCols / 2; ++e) mx[e & 3] = max3(mx[e & 3], x[2 * e], x[2 * e + 1]);
                    const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const bool raise = mt > (fresh ? -INFINITY : h ? S::kSecondThreshold : S::kRescaleThreshold);
                    if (__any_sync(0xffffffffu, raise)) {
                        const float up = raise ? mt : 0.f;
                        const float alpha = raise ? fresh ? 0.f : fast_exp2(-mt) : 1.f;
                        if (i + h > 0) {
                            if (h && !(ok = wait_all(o_half(t), cnt & 1))) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < 4; ++c) {
                                float o[32];
                                tmem_ld32(o_row + 32 * c, o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] *= alpha;
                                tmem_st32(o_row + 32 * c, o);
                            }
                        }
                        l_run *= alpha;
                        if (raise) m_run = m_use + mt;
                        const uint64_t up2 = pack_f32x2(-up, -up);
#pragma unroll
                        for (int e = 0; e < kCols; e += 2)
                            unpack_f32x2(add_f32x2(pack_f32x2(x[e], x[e + 1]), up2), x[e], x[e + 1]);
                    }
                    // probabilities exp2 of that to f16 for the products, and to the row sum before that rounding
                    // (its errors, half a step each, average out over the row), two at a time
                    uint64_t sum0 = 0, sum1 = 0;                 // two packed partial sums each
#pragma unroll
                    for (int q = 0; q < kCols; q += 32) {
                        float w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float y0 = fast_exp2(x[q + 2 * e]), y1 = fast_exp2(x[q + 2 * e + 1]);
                            if (e & 1) sum1 = add_f32x2(sum1, pack_f32x2(y0, y1));
                            else sum0 = add_f32x2(sum0, pack_f32x2(y0, y1));
                            w[e] = __uint_as_float(pack_half2(y0, y1));
                        }
                        tmem_st16(s_row + (kCols * h + q) / 2, w);   // P over logits already read
                    }
                    float u0, u1;
                    unpack_f32x2(add_f32x2(sum0, sum1), u0, u1);
                    l_run = fmaf(u0 + u1, lds32(ex + 4), l_run);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(p_full(t, h));
                }
                if (!ok) break;
            }
            if (!ok) break;
            if (!(ok = wait_all(o_done(t), (cnt - 1) & 1))) break;
            tc_fence_after();
            // narrow: the odd stream hands its rows to the even one, whose warp reads both from TMEM
            const bool both = kNarrow && n > 1;
            float wa = 1.f, wb = 0.f;
            if constexpr (kNarrow) {
                const uint32_t ml_col = tmem_s(1) + lane_base + 126;   // past P in the odd stream's S
                if (t == 1) {
                    tmem_st1(ml_col, m_run);
                    tmem_st1(ml_col + 1, l_run);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(x_full);
                    continue;
                }
                if (both) {
                    if (!(ok = wait_all(x_full, exchanges & 1))) break;
                    ++exchanges;
                    tc_fence_after();
                    const float2 ml = make_float2(tmem_ld1(ml_col), tmem_ld1(ml_col + 1));
                    tc_fence_before();
                    mbar_arrive(x_read);
                    const float M = fmaxf(fmaxf(m_run, ml.x), kLogitFloor);
                    wa = fast_exp2(m_run - M);
                    wb = fast_exp2(ml.x - M);
                    l_run = l_run * wa + ml.y * wb;
                    m_run = fmaxf(m_run, ml.x);
                }
            }
            const uint32_t ob_row = tmem_o(1) + lane_base;
            // columns 32 c .. 32 c + 31 of the row's unnormalised output
            auto load_o = [&](int c, float (&o)[32]) {
                if (both) {
                    float ob[32];
                    tmem_ld32x2(o_row + 32 * c, o, ob_row + 32 * c, ob);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = o[e] * wa + ob[e] * wb;
                } else {
                    tmem_ld32(o_row + 32 * c, o);
                }
            };
            auto release_o = [&]() {                             // O may be overwritten
                tc_fence_before();
                mbar_arrive(o_free(t));
                if (both) mbar_arrive(o_free(1));
            };
            if (idle) {
                release_o();
                continue;
            }
            __half* dst = p.out + ((int64_t)(pc.row0 + qi) * p.Hq + (int64_t)pc.g * G + hh) * kHeadDim;
            auto store_out = [&](int c, const float (&o)[32], float inv) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint4 u;
                    u.x = pack_half2(o[8 * q + 0] * inv, o[8 * q + 1] * inv);
                    u.y = pack_half2(o[8 * q + 2] * inv, o[8 * q + 3] * inv);
                    u.z = pack_half2(o[8 * q + 4] * inv, o[8 * q + 5] * inv);
                    u.w = pack_half2(o[8 * q + 6] * inv, o[8 * q + 7] * inv);
                    *reinterpret_cast<uint4*>(dst + 32 * c + 8 * q) = u;
                }
            };
            if (pc.j0 == 0 && pc.j1 == pc.ntiles) {
                // ---- a whole item: out = O / l ----
                const float inv = 1.f / l_run;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    float o[32];
                    load_o(c, o);
                    if (valid) store_out(c, o, inv);
                }
                release_o();
                continue;
            }
            if (kNarrow && threadIdx.x == 0) {
                CutItem& it = s_cut[*s_cuts];
                it.u = pc.u;
                it.row0 = pc.row0;
                it.nq = pc.nq;
                it.g = pc.g;
                it.ntiles = pc.ntiles;
                ++*s_cuts;
            }
            // ---- a piece of an item cut at a CTA boundary: its (m, l, O) go to the workspace ----
            uint8_t* part = part_of((int)blockIdx.x, pc.u <= u_lo ? 0 : 1, t);
            float4* po = reinterpret_cast<float4*>(part);        // [32 float4 of channels][lp rows]
            const int lp = (min(T, pc.nq - (kNarrow ? 0 : t * T)) * G + 7) & ~7;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                float o[32];
                load_o(c, o);
                if (valid) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        __stcg(po + (8 * c + q) * lp + r, make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]));
                }
            }
            if (valid) __stcg(reinterpret_cast<float2*>(part + 128 * 128 * 4) + r, make_float2(m_run, l_run));
            release_o();
            if constexpr (kNarrow) {                             // merged at the CTA's end, by bulk copies
                fence_proxy_async_global();
                continue;
            }
            // Wide: the warp's ticket for its 32 rows. The warp barrier orders every lane's stores before lane
            // 0's release-acquire; the loads of the last one, which merges, follow its acquire:
            // out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k, in the order of the pieces, whoever merges.
            // The other warps go on meanwhile. (Merged at the CTA's end as below, 512 tokens on 8 x 2048
            // contexts took 171 us instead of 160; narrow chunks have few rows, hence few warps, for this.)
            __syncwarp();
            const int c_first = cta_of(pc.u), c_last = cta_of(pc.u + pc.ntiles - 1);
            unsigned int* tick = p.tickets + ((int64_t)c_last * 2 + t) * 4 + quarter;
            unsigned int prev = 0;
            if (lane == 0) prev = atomic_add_acq_rel_gpu(tick, 1u);
            prev = __shfl_sync(0xffffffffu, prev, 0);
            __syncwarp();
            if (prev != (unsigned int)(c_last - c_first)) continue;
            if (lane == 0) *tick = 0u;                           // ready for the next call
            if (!valid) continue;
            const int first_slot = pc.u <= range_lo(c_first) ? 0 : 1;
            auto piece_at = [&](int c) { return part_of(c, c == c_first ? first_slot : 0, t); };
            auto ml_of = [&](int c) { return __ldcg(reinterpret_cast<const float2*>(piece_at(c) + 128 * 128 * 4) + r); };
            float M = kLogitFloor;
#pragma unroll 1
            for (int c = c_first; c <= c_last; ++c) M = fmaxf(M, ml_of(c).x);
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {                        // 32 channels at a time
                float o[32], den = 0.f;
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0.f;
#pragma unroll 1
                for (int c = c_first; c <= c_last; ++c) {
                    const float4* src = reinterpret_cast<const float4*>(piece_at(c)) + 8 * h * lp + r;
                    float4 v[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] = __ldcg(src + q * lp);
                    const float2 ml = ml_of(c);
                    const float w = fast_exp2(ml.x - M);         // 0 for a piece that saw no position of the row
                    den = fmaf(w, ml.y, den);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        o[4 * q] = fmaf(w, v[q].x, o[4 * q]);
                        o[4 * q + 1] = fmaf(w, v[q].y, o[4 * q + 1]);
                        o[4 * q + 2] = fmaf(w, v[q].z, o[4 * q + 2]);
                        o[4 * q + 3] = fmaf(w, v[q].w, o[4 * q + 3]);
                    }
                }
                store_out(h, o, 1.f / den);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == S::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, S::kTmemCols);
    }
    if (!kNarrow || *s_abort) return;                    // (uniform: the barrier lies between it and the last write)

    // ---- narrow: the items this CTA has a piece of (its first and its last one, at most). The CTA that takes an
    // item's last ticket merges its pieces, all threads together, through the shared memory that is free by now,
    // three pieces at a time by bulk copy. (Merged warp by warp as above, 4 tokens on one 2000-token context took
    // 28 us instead of 18.) The block's barrier orders the pieces' stores before the release-acquire ticket; the
    // copies behind its acquire come after the next barrier. The stores are the generic proxy's and the copies the
    // async proxy's: a proxy fence follows the stores, and another precedes the copies. ----
    const int n_cut = *s_cuts;
    if (n_cut == 0) return;
    if (warp < n_cut && lane == 0) {                             // an item is known by the last CTA it reaches
        const CutItem& it = s_cut[warp];
        const int c_last = cta_of(it.u + it.ntiles - 1), others = c_last - cta_of(it.u);
        const bool last = atomic_add_acq_rel_gpu(p.tickets + c_last, 1u) == (unsigned int)others;
        if (last) p.tickets[c_last] = 0u;                        // ready for the next call
        s_first[warp] = last ? 1 : 0;
    }
    __syncthreads();
    const bool won0 = s_first[0] != 0, won1 = n_cut > 1 && s_first[1] != 0;
    float* weight = reinterpret_cast<float*>(smem_raw + S::kOffScales);      // [slot][row], then 1 / sum
    long long* out_of_row = reinterpret_cast<long long*>(smem_raw + 3 * 65536);             // behind the three slots
    uint32_t phase = 0;
#pragma unroll 1
    for (int k = 0; k < n_cut; ++k) {
        if (!(k ? won1 : won0)) continue;
        const CutItem it = s_cut[k];
        const int live = it.nq * G;                              // rows
        const int lp = (live + 7) & ~7;
        const int c_first = cta_of(it.u), c_last = cta_of(it.u + it.ntiles - 1);
        const int first_slot = it.u <= range_lo(c_first) ? 0 : 1;
        if ((int)threadIdx.x < live) {                           // where row threadIdx.x goes
            const int ti = threadIdx.x / G;
            out_of_row[threadIdx.x] = ((long long)(it.row0 + ti) * p.Hq + it.g * G + threadIdx.x - ti * G) * kHeadDim;
        }
        float M = kLogitFloor, den = 0.f;                        // of row threadIdx.x, over the pieces so far
        // (the order of the pieces decides the result, not who merges)
        for (int c0 = c_first; c0 <= c_last;) {
            // a running result sits in slot 0 after the first round
            const int s0 = c0 == c_first ? 0 : 1, n_new = min(3 - s0, c_last - c0 + 1), n_all = s0 + n_new;
            auto piece_at = [&](int u) { return part_of(c0 + u, c0 + u == c_first ? first_slot : 0, 0); };
            if (threadIdx.x == 0) {
                fence_proxy_async_shared();
                fence_proxy_async_global();
                mbar_arrive_expect_tx(merge_bar, (uint32_t)(n_new * 512 * lp));
                for (int u = 0; u < n_new; ++u)
                    bulk_load(base + (uint32_t)(s0 + u) * 65536u, piece_at(u), (uint32_t)(512 * lp), merge_bar);
            }
            if ((int)threadIdx.x < live) {
                float m_new = M;
                float2 ml[3];
#pragma unroll
                for (int u = 0; u < 3; ++u) {
                    ml[u] = make_float2(-INFINITY, 0.f);         // (as is a piece that saw no position of the row)
                    if (u < n_new) ml[u] = __ldcg(reinterpret_cast<const float2*>(piece_at(u) + 128 * 128 * 4) + threadIdx.x);
                    m_new = fmaxf(m_new, ml[u].x);
                }
                const float a = fast_exp2(M - m_new);
                den *= a;
                if (s0) weight[threadIdx.x] = a;
#pragma unroll
                for (int u = 0; u < 3; ++u) {
                    const float w = fast_exp2(ml[u].x - m_new);
                    den = fmaf(w, ml[u].y, den);
                    if (u < n_new) weight[128 * (s0 + u) + threadIdx.x] = w;
                }
                weight[128 * 3 + threadIdx.x] = 1.f / den;
                M = m_new;
            }
            // all leave together when the copies do not come
            if (__syncthreads_or(!mbar_wait(merge_bar, phase))) return;
            phase ^= 1;
            c0 += n_new;
            const bool done = c0 > c_last;
            // a warp takes eight rows x four float4 of channels at a time (whole 32-byte sectors of the output)
            const int q_lane = lane >> 3, r_lane = lane & 7;
            const float4* slot = reinterpret_cast<const float4*>(smem_raw);
            auto combine = [&](int blk, int& r, int& q) -> float4 {
                r = 8 * (blk >> 3) + r_lane;
                q = 4 * (blk & 7) + q_lane;
                const int at = q * lp + r;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int u = 0; u < 3; ++u) {
                    if (u < n_all) {
                        const float4 v = slot[4096 * u + at];
                        const float w = weight[128 * u + r];
                        acc.x = fmaf(w, v.x, acc.x);
                        acc.y = fmaf(w, v.y, acc.y);
                        acc.z = fmaf(w, v.z, acc.z);
                        acc.w = fmaf(w, v.w, acc.w);
                    }
                }
                return acc;
            };
            if (done) {
#pragma unroll 2
                for (int blk = warp; blk < lp; blk += S::kThreads / 32) {
                    int r, q;
                    const float4 acc = combine(blk, r, q);
                    const float inv = weight[128 * 3 + r];
                    if (r < live)
                        reinterpret_cast<uint2*>(p.out + out_of_row[r])[q] =
                            make_uint2(pack_half2(acc.x * inv, acc.y * inv), pack_half2(acc.z * inv, acc.w * inv));
                }
            } else {
                for (int blk = warp; blk < lp; blk += S::kThreads / 32) {
                    int r, q;
                    const float4 acc = combine(blk, r, q);
                    reinterpret_cast<float4*>(smem_raw)[q * lp + r] = acc;
                }
            }
            __syncthreads();                                     // the slots and weights may be overwritten
        }
    }
}

}  // namespace pkv

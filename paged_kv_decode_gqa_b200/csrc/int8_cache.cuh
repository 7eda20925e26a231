// The 8-bit paged cache with a scale per token and KV head, and the write that
// rotates, quantises and stores in one launch.
//
// Format: code u8 = 128 + round(x / s), value = (code - 128) * s, with
// s = max(amax |x|, 2^-24) / 127 over the 128 channels of one (token, KV head)
// of K or of V. The offset of 128 lets a code become an f16 integer by one byte
// permute and one subtraction (0x6400 | code is 1024 + code). The scales are
// fp32 [num_blocks, Hkv, 2, 16]: the K and V scales of one page and head are
// one 128-byte line, read by one copy beside the page.
//
// rope_cache_write_kernel: eight threads hold one head row of 128 channels,
// thread i two 8-channel chunks chosen so that the two channels of every
// rotated pair meet in one thread (chunks i and i + R/16 of the rotated part R;
// two consecutive chunks of the part left as it is), so neither pairing style
// needs a shuffle, and the row's amax takes three. A warp holds rows of one
// token, four at a time: it computes the token's R/2 angles once (two a lane,
// exchanged through its own shared memory, while its first rows are in flight),
// and every thread keeps the eight it needs in registers for all its rows. No
// block-wide step exists. A token's rows are shared out over several warps only
// when there are too few tokens to fill the SMs.
// Angles: a fraction of a turn, from fp64 arithmetic in which the product of the
// position and the frequency and that with 1 / (2 pi) keep their low parts
// (turn_fraction), then the fp32 sincospi. In fp32 a position near 2^20 would
// leave the fastest angle off by 2^-4 radians; in plain fp64 one near 2^31 by
// 4e-7, several times the rounding of the reduced angle to fp32.
// Rounding: fp32 throughout, once to f16, to E4M3 (of x / scale, an IEEE
// division, as paged_kv_cache_write) or to the 8-bit code.
// Bound: HBM; every row is read and written once. Measured in a graph: f16, 16384
// tokens at 28 / 4 heads 52.6 us, 5.75 TB/s (0.88 of the measured copy rate), f16, 128
// tokens of them 2.8 us, and E4M3, 2049 tokens at 12 / 2 heads 5.8 us, where the launch
// and round trips to memory take most of it: one for the 128 tokens; two for the 2049,
// whose 4098 shares of rows (two warps a token) the 2368 warps that fit take in two turns.
#pragma once

#include "cache_write.cuh"

namespace pkv {

enum CacheKind { kCacheF16 = 0, kCacheFp8 = 1, kCacheInt8 = 2 };

constexpr int kRopeMaxAxes = 4;
constexpr int kMaxTokens = (1 << 30) - 1;                // of one call
constexpr float kInt8MinAmax = 5.9604644775390625e-8f;   // 2^-24, the smallest positive binary16

struct RopeWriteParams {
    __half* q_out;             // [T, Hq, 128]; may be q
    const __half* q;
    const __half* k_new;       // [T, Hkv, 128]
    const __half* v_new;
    void* k_cache;             // [NB, bs, Hkv, 128] f16 or u8
    void* v_cache;
    float* kv_scales;          // int8: [NB, Hkv, 2, 16]
    const int64_t* slot_mapping;
    const int64_t* positions;  // [axes, T]
    const float* inv_freq;     // [half]
    int64_t num_slots;
    int32_t num_tokens, Hq, Hkv;
    int32_t half;              // R / 2 rotated pairs; 0: nothing is rotated
    int32_t axes, cyclic, pairs;
    int32_t sections[kRopeMaxAxes];
    float k_scale, v_scale;    // FP8
    const float* k_scales;     // FP8 device scales or null
    const float* v_scales;
    int32_t scales_per_head;
    int32_t splits;            // warps that share a token's rows
};

// Four codes (low byte first) to two f16x2 of their exact values: 0x6400 | code
// is 1024 + code in f16, and 1152 is subtracted exactly.
__device__ __forceinline__ uint32_t sub_1152(uint32_t h) {
    const uint32_t bias = 0x64806480u;
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&bias));
    return *reinterpret_cast<const uint32_t*>(&d);
}
// bytes (0, 1) and (2, 3): consecutive channels of one token
__device__ __forceinline__ void codes_to_half2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
    lo = sub_1152(prmt(w, 0x64646464u, 0x5140u));
    hi = sub_1152(prmt(w, 0x64646464u, 0x5342u));
}
// bytes (0, 2) and (1, 3): one channel of two tokens each
__device__ __forceinline__ void codes_to_half2x2_cross(uint32_t w, uint32_t& even, uint32_t& odd) {
    even = sub_1152(prmt(w, 0x64646464u, 0x5240u));
    odd = sub_1152(prmt(w, 0x64646464u, 0x5341u));
}

// 16-byte load of data read once. Not through the read-only path: q may be
// rotated in place (each thread reads its channels before it writes them).
__device__ __forceinline__ uint4 ld_once_16(const uint4* src) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(src) : "memory");
    return v;
}

// Eight channels as fp32.
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        f[2 * k] = p.x;
        f[2 * k + 1] = p.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]),
                      pack_half2(f[6], f[7]));
}

// Eight fp32 values divided by `scale` (IEEE), to E4M3 (nearest even, saturating at 448).
__device__ __forceinline__ uint2 quantize8_e4m3_f32(const float (&f)[8], float scale) {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f[4 * k + 1] / scale), "f"(f[4 * k] / scale));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f[4 * k + 3] / scale), "f"(f[4 * k + 2] / scale));
        w[k] = (uint32_t)lo | ((uint32_t)hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

// Largest finite magnitude of 16 values (0 when none is finite). fmaxf ignores NaN; infinities are rare
// enough to be sorted out afterwards.
__device__ __forceinline__ float finite_amax16(const float (&a)[8], const float (&b)[8]) {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(fmaxf(m, fabsf(a[k])), fabsf(b[k]));
    if (m > 3.402823466e38f) {
        m = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            m = fabsf(a[k]) <= 3.402823466e38f ? fmaxf(m, fabsf(a[k])) : m;
            m = fabsf(b[k]) <= 3.402823466e38f ? fmaxf(m, fabsf(b[k])) : m;
        }
    }
    return m;
}

// Codes 128 + round(x / scale) of eight values: nearest even, infinities at
// +-127, NaN at 0; x / scale is the fp32 quotient, correctly rounded.
// x * inv, inv = 1 / scale, taken exactly by the multiply-add, is within 2^-16
// of that quotient (two roundings of a value of at most 127), so both round to
// the same integer unless the product lies within 2^-14 of a tie; only then
// (one value in 8000, and where x is not finite) is the division done.
__device__ __forceinline__ uint2 quantize8_int8(const float (&f)[8], float scale, float inv) {
    constexpr float kMagic = 12583040.f;                     // 1.5 x 2^23 + 128: the low byte of x + kMagic is the code
    uint32_t c[8];
    float worst = 0.f;
    bool finite = true;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float r = fmaf(f[k], inv, kMagic);
        c[k] = __float_as_uint(r);
        const float d = fabsf(fmaf(f[k], inv, kMagic - r));  // distance from the integer taken
        worst = fmaxf(worst, d);
        finite = finite && d < 1.f;                          // (false for NaN, which fmaxf would drop)
    }
    if (worst > 0.5f - 6.103515625e-5f || !finite) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            c[k] = (uint32_t)(min(127, max(-127, __float2int_rn(f[k] / scale))) + 128);   // NaN gives 0
    }
    return make_uint2(prmt(prmt(c[0], c[1], 0x0040u), prmt(c[2], c[3], 0x0040u), 0x5410u),
                      prmt(prmt(c[4], c[5], 0x0040u), prmt(c[6], c[7], 0x0040u), 0x5410u));
}

// pos * freq / (2 pi) less the nearest integer, to 2^-52 for |pos| up to 2^53 (a position past that is rounded to
// fp64 first). With c + c' = 1 / (2 pi) to 2^-109: the product a + a' is exact (multiply-adds keep what a product
// rounds off), t = a c has its low part kept as well, and t less its integer part is exact.
__device__ __forceinline__ double turn_fraction(double pos, double freq) {
    constexpr double c = 0.15915494309189535, c_low = -9.839338337591243e-18;
    const double a = pos * freq, a_low = fma(pos, freq, -a);
    const double t = a * c;
    return (t - rint(t)) + (fma(a, c, -t) + fma(a, c_low, a_low * c));
}

// Position axis of frequency j.
__device__ __forceinline__ int rope_axis(const RopeWriteParams& p, int j) {
    if (p.cyclic) {
        const int a = j % p.axes;
        return a > 0 && j < p.axes * p.sections[a] ? a : 0;
    }
    int a = 0, end = p.sections[0];
    while (j >= end && a + 1 < p.axes) end += p.sections[++a];
    return a;
}

constexpr int kRopeWarps = 4;       // warps of a block, each on its own
constexpr int kRopeBatch = 3;       // rows in flight per thread of the rotating write
constexpr int kRowBatch = 2;        // and of the plain write and the read

// Stores one head row's eight-thread share (chunks ca, cb as fp32 a, b; as read: ua, ub) of K or V.
template <int kKind, bool kPlain = false>
__device__ __forceinline__ void store_kv_row(const RopeWriteParams& p, int i, int ca, int cb, bool is_v, int h,
                                             int64_t slot, bool live, const float (&a)[8], const float (&b)[8],
                                             const uint4& ua, const uint4& ub) {
    float scale = 1.f;
    if constexpr (kKind == kCacheInt8) {             // amax of the row, over its eight threads
        float m = finite_amax16(a, b);
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        scale = fmaxf(m, kInt8MinAmax) / 127.f;
    }
    if (!live || slot < 0) return;                   // padding token
    if (slot >= p.num_slots) {
        if (i == 0 && h == 0) flag_error(PKV_DEVERR_SLOT);
        return;
    }
    const int64_t dst = (slot * p.Hkv + h) * 16;     // in chunks of 8 channels
    void* cache = is_v ? p.v_cache : p.k_cache;
    if constexpr (kKind == kCacheF16) {
        reinterpret_cast<uint4*>(cache)[dst + ca] = is_v ? ua : pack8(a);
        reinterpret_cast<uint4*>(cache)[dst + cb] = is_v ? ub : pack8(b);
    } else if constexpr (kKind == kCacheFp8) {
        float s = is_v ? p.v_scale : p.k_scale;
        if (p.k_scales) s = head_scale(is_v ? p.v_scales : p.k_scales, p.scales_per_head, h);
        reinterpret_cast<uint2*>(cache)[dst + ca] = quantize8_e4m3_f32(a, s);
        reinterpret_cast<uint2*>(cache)[dst + cb] = quantize8_e4m3_f32(b, s);
    } else {
        const float inv = 1.f / scale;
        const uint2 x = quantize8_int8(a, scale, inv), y = quantize8_int8(b, scale, inv);
        if (kPlain) {                                // neighbouring chunks
            *reinterpret_cast<uint4*>(reinterpret_cast<uint2*>(cache) + dst + ca) = make_uint4(x.x, x.y, y.x, y.y);
        } else {
            reinterpret_cast<uint2*>(cache)[dst + ca] = x;
            reinterpret_cast<uint2*>(cache)[dst + cb] = y;
        }
        if (i == 0) p.kv_scales[((slot / 16 * p.Hkv + h) * 2 + (is_v ? 1 : 0)) * 16 + slot % 16] = scale;
    }
}

template <int kKind>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_cache_write_kernel(const RopeWriteParams p) {
    __shared__ float2 s_turn[kRopeWarps][64];            // (cos, sin) of the warp's token
    const int lane = threadIdx.x & 31, i = lane & 7, sub = lane >> 3;
    const int warp = (int)blockIdx.x * kRopeWarps + (int)(threadIdx.x >> 5);
    const int step = (int)(gridDim.x * kRopeWarps) / p.splits;       // tokens between a warp's turns
    int tok = warp / p.splits;
    const int split = warp - tok * p.splits;
    const int rows = p.Hq + 2 * p.Hkv;                   // q heads, k heads, v heads
    const int rot = p.half >> 3;                         // threads of a row that hold rotated pairs
    const int ca = i < rot ? i : 2 * i, cb = i < rot ? i + rot : 2 * i + 1;   // this thread's chunks

    grid_dependency_wait();
    grid_dependents_launch();
    if (kKind == kCacheFp8 && p.k_scales && blockIdx.x == 0)
        check_scales(p.k_scales, p.v_scales, p.scales_per_head ? p.Hkv : 1, threadIdx.x, blockDim.x);
    if (tok >= p.num_tokens || tok >= step) return;      // (warps left over by an uneven split)

    // A token's rows of this warp: first + sub, first = 4 split, 4 split + stride, ..., in batches of
    // kRopeBatch. Every row's registers are refilled as soon as it is done, with the row a batch ahead:
    // of this token, or of the warp's next.
    const int stride = 4 * p.splits;
    uint4 ua[kRopeBatch], ub[kRopeBatch];
    auto load = [&](int u, int t, int row) {
        if (t < p.num_tokens && row < rows) {
            const __half* s = row < p.Hq ? p.q + ((int64_t)t * p.Hq + row) * 128
                              : row < p.Hq + p.Hkv ? p.k_new + ((int64_t)t * p.Hkv + (row - p.Hq)) * 128
                                                   : p.v_new + ((int64_t)t * p.Hkv + (row - p.Hq - p.Hkv)) * 128;
            ua[u] = ld_once_16(reinterpret_cast<const uint4*>(s) + ca);
            ub[u] = ld_once_16(reinterpret_cast<const uint4*>(s) + cb);
        }
    };
#pragma unroll
    for (int u = 0; u < kRopeBatch; ++u) load(u, tok, 4 * split + u * stride + sub);
    // this lane's frequencies and their axes
    double freq[2] = {0.0, 0.0};
    const int64_t* where[2] = {p.positions, p.positions};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int j = lane + 32 * e;
        if (j < p.half) {
            freq[e] = (double)__ldg(p.inv_freq + j);
            where[e] += (int64_t)rope_axis(p, j) * p.num_tokens;
        }
    }
    int64_t pos[2] = {__ldg(where[0] + tok), __ldg(where[1] + tok)};
    int64_t slot = __ldg(p.slot_mapping + tok);
    float2* turn = s_turn[threadIdx.x >> 5];
    while (tok < p.num_tokens) {
        const int next = p.num_tokens - tok > step ? tok + step : p.num_tokens;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int j = lane + 32 * e;
            if (j < p.half) {
                const float frac = (float)turn_fraction((double)pos[e], freq[e]);     // in [-1/2, 1/2]
                sincospif(2.f * frac, &turn[j].y, &turn[j].x);
            }
        }
        __syncwarp();
        // pair k of this thread: channels (2k, 2k + 1) of chunk a, then of chunk b; or channel k of both
        float2 cs[8];
        if (i < rot) {
#pragma unroll
            for (int k = 0; k < 8; ++k) cs[k] = turn[p.pairs ? (k < 4 ? 4 * ca + k : 4 * cb + k - 4) : 8 * i + k];
        }
        __syncwarp();                                    // before the next token's angles
        const int64_t this_slot = slot;
        if (next < p.num_tokens) {
            pos[0] = __ldg(where[0] + next);
            pos[1] = __ldg(where[1] + next);
            slot = __ldg(p.slot_mapping + next);
        }
        for (int first0 = 4 * split; first0 < rows; first0 += kRopeBatch * stride) {
            const bool more = first0 + kRopeBatch * stride < rows;       // batches left of this token
#pragma unroll
            for (int u = 0; u < kRopeBatch; ++u) {
                const int first = first0 + u * stride, row = first + sub;
                if (first < rows) {                      // (the whole warp)
                    const bool live = row < rows, is_q = row < p.Hq, is_v = row >= p.Hq + p.Hkv;
                    float a[8], b[8];
                    unpack8(ua[u], a);
                    unpack8(ub[u], b);
                    if (!is_v && i < rot) {
                        if (p.pairs) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float a0 = a[2 * k], a1 = a[2 * k + 1], b0 = b[2 * k], b1 = b[2 * k + 1];
                                a[2 * k] = fmaf(a0, cs[k].x, -a1 * cs[k].y);
                                a[2 * k + 1] = fmaf(a1, cs[k].x, a0 * cs[k].y);
                                b[2 * k] = fmaf(b0, cs[4 + k].x, -b1 * cs[4 + k].y);
                                b[2 * k + 1] = fmaf(b1, cs[4 + k].x, b0 * cs[4 + k].y);
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const float a0 = a[k], b0 = b[k];
                                a[k] = fmaf(a0, cs[k].x, -b0 * cs[k].y);
                                b[k] = fmaf(b0, cs[k].x, a0 * cs[k].y);
                            }
                        }
                    }
                    if (live && is_q) {
                        uint4* dst = reinterpret_cast<uint4*>(p.q_out + ((int64_t)tok * p.Hq + row) * 128);
                        dst[ca] = pack8(a);
                        dst[cb] = pack8(b);
                    }
                    if (first + 4 > p.Hq)                // (the whole warp: it takes the row's amax together)
                        store_kv_row<kKind>(p, i, ca, cb, is_v, is_v ? row - p.Hq - p.Hkv : row - p.Hq, this_slot,
                                            live && !is_q, a, b, ua[u], ub[u]);
                }
                if (more) load(u, tok, row + kRopeBatch * stride);
                else load(u, next, 4 * split + u * stride + sub);
            }
        }
        tok = next;
    }
}

// A walk over the K and V rows of all tokens (row < 2 Hkv of token tok), in steps of `items` rows:
// advanced by addition, because a division per row would cost as much as quantising it.
struct RowWalk {
    int tok, row, dtok, drow, rows;
    __device__ __forceinline__ RowWalk(int64_t first, int64_t items, int rows_) : rows(rows_) {
        tok = (int)(first / rows);
        row = (int)(first - (int64_t)tok * rows);
        dtok = (int)(items / rows);
        drow = (int)(items - (int64_t)dtok * rows);
    }
    __device__ __forceinline__ void next() {
        row += drow;
        const int carry = row >= rows ? 1 : 0;
        row -= carry ? rows : 0;
        tok = min(tok + dtok + carry, kMaxTokens);       // (stays past the last token)
    }
};

// The write without rotation into an 8-bit cache: the K and V rows of all tokens in one run; a thread
// keeps kRowBatch rows in flight and refills each as soon as it is done. Bound: HBM; 16411 tokens of 4 KV heads
// written and read back (two launches, 102 MB) take 26.7 us, 0.58 of the measured copy rate.
__global__ void __launch_bounds__(256, 4) cache_write_int8_kernel(const RopeWriteParams p) {
    const int i = threadIdx.x & 7;
    const int64_t groups = (int64_t)gridDim.x * 32;
    grid_dependency_wait();
    grid_dependents_launch();
    RowWalk walk((int64_t)blockIdx.x * 32 + (threadIdx.x >> 3), groups, 2 * p.Hkv);
    // the warp's first row decides when it ends, so that all of it reaches the row maxima
    RowWalk lead((int64_t)blockIdx.x * 32 + ((threadIdx.x >> 5) << 2), groups, 2 * p.Hkv);
    uint4 ua[kRowBatch], ub[kRowBatch];
    int64_t slot[kRowBatch];
    int row[kRowBatch];
    auto load = [&](int u) {
        slot[u] = -1;
        row[u] = walk.row;
        if (walk.tok < p.num_tokens) {
            const __half* src = walk.row < p.Hkv ? p.k_new + ((int64_t)walk.tok * p.Hkv + walk.row) * 128
                                                 : p.v_new + ((int64_t)walk.tok * p.Hkv + walk.row - p.Hkv) * 128;
            ua[u] = ld_stream_16(reinterpret_cast<const uint4*>(src) + 2 * i);
            ub[u] = ld_stream_16(reinterpret_cast<const uint4*>(src) + 2 * i + 1);
            slot[u] = __ldg(p.slot_mapping + walk.tok);
        }
        walk.next();
    };
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) {
        ua[u] = ub[u] = make_uint4(0, 0, 0, 0);
        load(u);
    }
    while (lead.tok < p.num_tokens) {
#pragma unroll
        for (int u = 0; u < kRowBatch; ++u) {
            float a[8], b[8];
            unpack8(ua[u], a);
            unpack8(ub[u], b);
            const bool is_v = row[u] >= p.Hkv;
            store_kv_row<kCacheInt8, true>(p, i, 2 * i, 2 * i + 1, is_v, is_v ? row[u] - p.Hkv : row[u], slot[u], true, a,
                                           b, ua[u], ub[u]);
            load(u);
            lead.next();
        }
    }
}

// paged_kv_cache_read: rows of the cache named by slots, back as dense f16.
struct CacheReadParams {
    __half* k_out;             // [T, Hkv, 128]
    __half* v_out;
    const void* k_cache;
    const void* v_cache;
    const float* kv_scales;
    const int64_t* slot_mapping;
    int64_t num_slots;
    int32_t num_tokens, Hkv;
    float k_scale, v_scale;
};

// Eight 8-bit codes times their scale, in fp32, rounded once to f16.
__device__ __forceinline__ uint4 dequantize8_int8(uint2 u, float s) {
    uint32_t h[4];
    codes_to_half2x2(u.x, h[0], h[1]);
    codes_to_half2x2(u.y, h[2], h[3]);
    float f[8];
    unpack8(make_uint4(h[0], h[1], h[2], h[3]), f);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] *= s;
    return pack8(f);
}

__device__ __forceinline__ uint4 dequantize8_e4m3(uint2 u, float s) {
    uint32_t h[4];
    e4m3x4_to_half2x2(u.x, h[0], h[1]);
    e4m3x4_to_half2x2(u.y, h[2], h[3]);
    float f[8];
    unpack8(make_uint4(h[0], h[1], h[2], h[3]), f);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] *= s;
    return pack8(f);
}

// Eight threads a row, two 8-channel chunks each; kRowBatch rows in flight per thread, each refilled as
// soon as it is done, and their slots one batch further ahead.
template <int kKind>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheReadParams p) {
    const int i = threadIdx.x & 7;
    const int64_t groups = (int64_t)gridDim.x * 32;
    grid_dependency_wait();
    grid_dependents_launch();
    const int64_t first = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
    RowWalk out(first, groups, 2 * p.Hkv), in = out, look = out;     // rows stored, loaded, looked up
    int64_t ahead[kRowBatch];                            // slots looked up
    uint4 x[kRowBatch], y[kRowBatch];
    float s[kRowBatch];
    bool live[kRowBatch];
    auto look_up = [&](int u) {
        ahead[u] = look.tok < p.num_tokens ? __ldg(p.slot_mapping + look.tok) : -1;
        look.next();
    };
    auto load = [&](int u) {
        const int64_t slot = ahead[u];
        live[u] = slot >= 0 && slot < p.num_slots;
        if (live[u]) {
            const bool is_v = in.row >= p.Hkv;
            const int h = is_v ? in.row - p.Hkv : in.row;
            const int64_t src = (slot * p.Hkv + h) * 16;
            const void* cache = is_v ? p.v_cache : p.k_cache;
            if constexpr (kKind == kCacheF16) {
                x[u] = ld_stream_16(reinterpret_cast<const uint4*>(cache) + src + 2 * i);
                y[u] = ld_stream_16(reinterpret_cast<const uint4*>(cache) + src + 2 * i + 1);
            } else {
                x[u] = ld_stream_16(reinterpret_cast<const uint4*>(reinterpret_cast<const uint2*>(cache) + src) + i);
                if constexpr (kKind == kCacheFp8) s[u] = is_v ? p.v_scale : p.k_scale;
                else s[u] = __ldg(p.kv_scales + ((slot / 16 * p.Hkv + h) * 2 + (is_v ? 1 : 0)) * 16 + slot % 16);
            }
        } else if (slot >= 0 && i == 0 && in.row == 0) {
            flag_error(PKV_DEVERR_SLOT);
        }
        in.next();
    };
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) look_up(u);
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) {
        load(u);
        look_up(u);
    }
    while (out.tok < p.num_tokens) {
#pragma unroll
        for (int u = 0; u < kRowBatch; ++u) {
            if (live[u]) {
                const bool is_v = out.row >= p.Hkv;
                const int h = is_v ? out.row - p.Hkv : out.row;
                uint4* dst = reinterpret_cast<uint4*>((is_v ? p.v_out : p.k_out) + ((int64_t)out.tok * p.Hkv + h) * 128) + 2 * i;
                const uint2 lo = make_uint2(x[u].x, x[u].y), hi = make_uint2(x[u].z, x[u].w);
                if constexpr (kKind == kCacheF16) {
                    dst[0] = x[u];
                    dst[1] = y[u];
                } else if constexpr (kKind == kCacheFp8) {
                    dst[0] = dequantize8_e4m3(lo, s[u]);
                    dst[1] = dequantize8_e4m3(hi, s[u]);
                } else {
                    dst[0] = dequantize8_int8(lo, s[u]);
                    dst[1] = dequantize8_int8(hi, s[u]);
                }
            }
            out.next();
            load(u);
            look_up(u);
        }
    }
}

}  // namespace pkv

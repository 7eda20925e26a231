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
// needs a shuffle, and the row's amax takes three. The angles of a token are
// computed once per block (R/2 of them, against up to Hq + Hkv rows that use
// them) while the rows' loads are in flight: pos * inv_freq in fp64 (exact: 24
// significant bits times an integer below 2^29, and within 2^-53 past it),
// reduced to a fraction of a turn, then the fp32 sincospi. In fp32 a position
// near 2^20 would leave the fastest angle off by 2^-4 radians.
// Rounding: fp32 throughout, once to f16, to E4M3 (of x / scale, an IEEE
// division, as paged_kv_cache_write) or to the 8-bit code.
#pragma once

#include "cache_write.cuh"

namespace pkv {

enum CacheKind { kCacheF16 = 0, kCacheFp8 = 1, kCacheInt8 = 2 };

constexpr int kRopeMaxAxes = 4;
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
    int32_t tokens_per_block;
};

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

// Largest finite magnitude of eight values (0 when none is finite).
__device__ __forceinline__ float finite_amax8(const float (&f)[8], float m) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float a = fabsf(f[k]);
        m = a <= 3.402823466e38f ? fmaxf(m, a) : m;
    }
    return m;
}

// Codes 128 + round(x / scale) of eight values: nearest even, infinities at
// +-127, NaN at 0. The division is IEEE, so that the code is the one its
// definition names, and not a neighbour at a tie.
__device__ __forceinline__ uint2 quantize8_int8(const float (&f)[8], float scale) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int c = __float2int_rn(f[k] / scale);          // NaN gives 0, infinities saturate
        w[k >> 2] |= (uint32_t)(min(127, max(-127, c)) + 128) << (8 * (k & 3));
    }
    return make_uint2(w[0], w[1]);
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

template <int kKind>
__global__ void __launch_bounds__(512) rope_cache_write_kernel(const RopeWriteParams p) {
    extern __shared__ float2 s_turn[];                   // [tokens_per_block][half] (cos, sin)
    const int i = threadIdx.x & 7, group = threadIdx.x >> 3, groups = blockDim.x >> 3;
    const int rows = p.Hq + 2 * p.Hkv;                   // q heads, k heads, v heads of one token
    const int t0 = (int)blockIdx.x * p.tokens_per_block;
    const int nt = min(p.tokens_per_block, p.num_tokens - t0);
    const int rot = p.half >> 3;                         // threads of a row that hold rotated pairs
    // this thread's two chunks of a rotated row
    const int ca = i < rot ? i : 2 * i, cb = i < rot ? i + rot : 2 * i + 1;

    grid_dependency_wait();
    grid_dependents_launch();
    if (kKind == kCacheFp8 && p.k_scales && blockIdx.x == 0)
        check_scales(p.k_scales, p.v_scales, p.scales_per_head ? p.Hkv : 1, threadIdx.x, blockDim.x);

    auto source = [&](int t, int row) -> const uint4* {
        const __half* s = row < p.Hq ? p.q + ((int64_t)t * p.Hq + row) * 128
                          : row < p.Hq + p.Hkv ? p.k_new + ((int64_t)t * p.Hkv + (row - p.Hq)) * 128
                                               : p.v_new + ((int64_t)t * p.Hkv + (row - p.Hq - p.Hkv)) * 128;
        return reinterpret_cast<const uint4*>(s);
    };
    uint4 ua, ub;
    auto load = [&](int item) {
        if (item < nt * rows) {
            const int t = item / rows;
            const uint4* s = source(t0 + t, item - t * rows);
            ua = ld_once_16(s + ca);
            ub = ld_once_16(s + cb);
        }
    };
    load(group);                                         // in flight while the angles are computed
    for (int k = threadIdx.x; k < nt * p.half; k += blockDim.x) {
        const int t = k / p.half, j = k - t * p.half;
        const int64_t pos = __ldg(p.positions + (int64_t)rope_axis(p, j) * p.num_tokens + t0 + t);
        const double turns = (double)pos * (double)__ldg(p.inv_freq + j) * 0.15915494309189533577;
        const float frac = (float)(turns - rint(turns));     // in [-1/2, 1/2]
        float2 cs;
        sincospif(2.f * frac, &cs.y, &cs.x);
        s_turn[k] = cs;
    }
    __syncthreads();

    const int last = (nt * rows + groups - 1) / groups * groups;    // whole warps reach the shuffles
    for (int item = group; item < last; item += groups) {
        const bool live = item < nt * rows;
        const int t = live ? item / rows : 0, row = live ? item - t * rows : 0;
        const int tok = t0 + t;
        float a[8], b[8];
        const uint4 va = ua, vb = ub;
        unpack8(va, a);
        unpack8(vb, b);
        load(item + groups);
        const bool is_q = row < p.Hq, is_v = row >= p.Hq + p.Hkv;
        if (live && !is_v && i < rot) {
            const float2* turn = s_turn + t * p.half;
            if (p.pairs) {                               // channels (2j, 2j + 1): both in one chunk
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 x = turn[4 * ca + k], y = turn[4 * cb + k];
                    const float a0 = a[2 * k], a1 = a[2 * k + 1], b0 = b[2 * k], b1 = b[2 * k + 1];
                    a[2 * k] = fmaf(a0, x.x, -a1 * x.y);
                    a[2 * k + 1] = fmaf(a1, x.x, a0 * x.y);
                    b[2 * k] = fmaf(b0, y.x, -b1 * y.y);
                    b[2 * k + 1] = fmaf(b1, y.x, b0 * y.y);
                }
            } else {                                     // channels (j, j + R/2): one in each chunk
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 x = turn[8 * i + k];
                    const float a0 = a[k], b0 = b[k];
                    a[k] = fmaf(a0, x.x, -b0 * x.y);
                    b[k] = fmaf(b0, x.x, a0 * x.y);
                }
            }
        }
        float scale = 1.f;
        if constexpr (kKind == kCacheInt8) {             // amax of the row, over its eight threads
            float m = finite_amax8(b, finite_amax8(a, 0.f));
#pragma unroll
            for (int off = 1; off < 8; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            scale = fmaxf(m, kInt8MinAmax) / 127.f;
        }
        if (!live) continue;
        if (is_q) {
            uint4* dst = reinterpret_cast<uint4*>(p.q_out + ((int64_t)tok * p.Hq + row) * 128);
            dst[ca] = pack8(a);
            dst[cb] = pack8(b);
            continue;
        }
        const int64_t slot = __ldg(p.slot_mapping + tok);
        if (slot < 0) continue;                          // padding token
        const int h = is_v ? row - p.Hq - p.Hkv : row - p.Hq;
        if (slot >= p.num_slots) {
            if (i == 0 && h == 0) flag_error(PKV_DEVERR_SLOT);
            continue;
        }
        const int64_t dst = (slot * p.Hkv + h) * 16;     // in chunks of 8 channels
        void* cache = is_v ? p.v_cache : p.k_cache;
        if constexpr (kKind == kCacheF16) {
            reinterpret_cast<uint4*>(cache)[dst + ca] = is_v ? va : pack8(a);
            reinterpret_cast<uint4*>(cache)[dst + cb] = is_v ? vb : pack8(b);
        } else if constexpr (kKind == kCacheFp8) {
            float s = is_v ? p.v_scale : p.k_scale;
            if (p.k_scales) s = head_scale(is_v ? p.v_scales : p.k_scales, p.scales_per_head, h);
            reinterpret_cast<uint2*>(cache)[dst + ca] = quantize8_e4m3_f32(a, s);
            reinterpret_cast<uint2*>(cache)[dst + cb] = quantize8_e4m3_f32(b, s);
        } else {
            reinterpret_cast<uint2*>(cache)[dst + ca] = quantize8_int8(a, scale);
            reinterpret_cast<uint2*>(cache)[dst + cb] = quantize8_int8(b, scale);
            if (i == 0) p.kv_scales[((slot / 16 * p.Hkv + h) * 2 + (is_v ? 1 : 0)) * 16 + slot % 16] = scale;
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
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = (float)((int)(((k < 4 ? u.x : u.y) >> (8 * (k & 3))) & 0xff) - 128) * s;
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

// Eight threads a row, two 8-channel chunks each, as in the write.
template <int kKind>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheReadParams p) {
    const int i = threadIdx.x & 7;
    const int64_t item = (int64_t)blockIdx.x * (blockDim.x >> 3) + (threadIdx.x >> 3);
    grid_dependency_wait();
    grid_dependents_launch();
    const int rows = 2 * p.Hkv;
    if (item >= (int64_t)p.num_tokens * rows) return;
    const int tok = (int)(item / rows), row = (int)(item - (int64_t)tok * rows);
    const int64_t slot = __ldg(p.slot_mapping + tok);
    if (slot < 0) return;
    const bool is_v = row >= p.Hkv;
    const int h = is_v ? row - p.Hkv : row;
    if (slot >= p.num_slots) {
        if (i == 0 && row == 0) flag_error(PKV_DEVERR_SLOT);
        return;
    }
    const int64_t src = (slot * p.Hkv + h) * 16;
    const void* cache = is_v ? p.v_cache : p.k_cache;
    uint4* dst = reinterpret_cast<uint4*>((is_v ? p.v_out : p.k_out) + ((int64_t)tok * p.Hkv + h) * 128);
    if constexpr (kKind == kCacheF16) {
        const uint4* s = reinterpret_cast<const uint4*>(cache) + src;
        const uint4 a = __ldg(s + i), b = __ldg(s + i + 8);
        dst[i] = a;
        dst[i + 8] = b;
    } else {
        // 16 codes of one chunk pair: chunks 2i and 2i + 1
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint2*>(cache) + src) + i);
        const uint2 lo = make_uint2(u.x, u.y), hi = make_uint2(u.z, u.w);
        if constexpr (kKind == kCacheFp8) {
            const float s = is_v ? p.v_scale : p.k_scale;
            dst[2 * i] = dequantize8_e4m3(lo, s);
            dst[2 * i + 1] = dequantize8_e4m3(hi, s);
        } else {
            const float s = __ldg(p.kv_scales + ((slot / 16 * p.Hkv + h) * 2 + (is_v ? 1 : 0)) * 16 + slot % 16);
            dst[2 * i] = dequantize8_int8(lo, s);
            dst[2 * i + 1] = dequantize8_int8(hi, s);
        }
    }
}

}  // namespace pkv

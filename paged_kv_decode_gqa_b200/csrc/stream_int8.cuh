// Attention over the 8-bit paged cache with a scale per token and KV head
// (int8_cache.cuh), load-balanced streaming form: decode (one query token per
// sequence), and chunks whose query tokens x heads fit eight columns.
//
// A unit is one page (16 tokens) of one KV head of one sequence; the units of
// the batch form a row, and every warp of the persistent grid takes an equal
// run of it and streams its pages through its own ring of TMA copies. A
// segment (sequence, KV head) that lies in one warp's run is written by that
// warp. The pieces of the others are merged at the end of the CTA's run: a
// warp leaves the piece its run ends in in its (then free) ring, the piece its
// run began in in the workspace, and after a barrier each chain of pieces of
// one segment is merged by one warp. A chain that is the whole segment is
// written; one that reaches into other CTAs becomes an item of a ticket tree
// of fan-in 16, whose last arrival at each node merges it, staging the items'
// 64 KiB through the ring in one round trip. Nothing waits on another CTA.
// (With the pieces merged through the workspace warp by warp instead, in a
// fan-in-32 tree as decode_balanced.cuh does, the 64-sequence decode took
// 24.1 us and the skewed one 30.2 us, most of it in the merges.)
//
// Columns: the N = 8 side of the tensor-core products (mma.sync m16n8k16,
// tokens on M) holds (query token, head of the KV head's group), column =
// token * G + head. Each column has its own causal limit.
//
// The mathematics, for a column with query vector q and a token t with codes
// ck_t, cv_t (exact in f16) and scales ks_t, vs_t:
//   x_t = softmax_scale log2(e) ks_t (q . ck_t)        logit, exp2 domain
//   y_t = x_t + log2(vs_t),  w_t = 2^(y_t - m)         weight of cv_t
//   O = sum w_t cv_t,  l = sum w_t / vs_t,  out = O / l
// Moving the value scale into the exponent keeps the weights that are rounded
// to f16 for the tensor cores (2^-12 each) in [0, 64] whatever the scales
// are, and leaves the codes exact; l is summed in fp32 from the unrounded
// weights. m follows the largest y only when that exceeds it by more than 6
// (so w <= 64): most pages then skip the rescaling of O and l.
// Codes are finite, so rows past the context need no zeroing: their weight is
// 0. A scale outside [0, 2^60] is flagged and counts as 0, a row of zeros
// (V: 2^-60 in its place, which rounds to zeros in any f16 output).
//
// Bound: HBM. Bytes of a unit: 2 x 16 x (128 + 4). Measured in a graph (called in a
// row in brackets): at 28 / 4 heads 128 sequences of 512 to 4096 tokens 58.9 us (63.1),
// 0.81 (0.76) of the measured copy rate; 64 sequences of 32 to 2048 tokens at 12 / 2
// heads (35.5 MB) 18.1 us (18.6), and 8 sequences, one of 32768 tokens, at 28 / 4 heads
// (39 MB) 21.7 us (22.2), where the launch, the scan of the lengths, the first loads
// and the merges, which no byte hides, take about two thirds: a batch of two short
// sequences, which has little else, takes 6.8 us, and the merges of many pieces by
// one warp each the rest.
#pragma once

#include <type_traits>

#include "decode_balanced.cuh"
#include "int8_cache.cuh"

namespace pkv {

struct StreamInt8Params {
    __half* out;                  // [B, Hq, 128], or [total, Hq, 128] with query_start
    const __half* q;
    const int32_t* block_tables;  // [B, max_blocks_per_seq]
    const int32_t* context_lens;  // [B]
    const int32_t* query_start;   // [B + 1], or null: one query per sequence (decode)
    // partial results: unnormalised O and (m, l) of columns 2c, 2c + 1, of the pieces that workers' runs
    // begin in, then of two items per CTA (a segment that began in an earlier CTA; one that began here)
    float4* ws_o;                 // [workers + 2 CTAs][8][32 lanes]
    float4* ws_ml;                // [workers + 2 CTAs][4]
    unsigned int* ws_count;       // [kTreeLevels][2 CTAs] tickets of the merge tree, zero between calls
    int32_t B, Hq, Hkv, G;
    int32_t total, max_query_len;
    int32_t max_blocks_per_seq, num_blocks, max_context_len;
    int32_t min_units_per_worker;
    float logit_scale_log2;       // softmax_scale * log2(e)
};

constexpr float kScaleMax = 1.152921504606846976e18f;      // 2^60
constexpr float kScaleMin = 8.673617379884035472e-19f;     // 2^-60
constexpr float kStreamRaise = 6.f;                        // log2 of the largest weight
constexpr float kLogitFloor = -1e30f;                      // stands in for a maximum of -inf
constexpr int kTreeFan = 16;                               // items a node of the cross-CTA tree merges
constexpr int kTreeLevels = 3;                             // 16^3 CTAs

template <int kWarps, int kStages>
struct StreamInt8Shape {
    static constexpr int kTileBytes = 2048;                 // one page of K (or V) codes, one head
    static constexpr int kSlotBytes = 2 * kTileBytes;
    static constexpr int kScaleBytes = 128;                 // K scales, V scales of the page
    static constexpr int kRingBytes = kWarps * kStages * kSlotBytes;
    static constexpr int kScaleRing = kWarps * kStages * kScaleBytes;
    static constexpr int kMergeFloats = 2 * 32 * 8 + 8;     // per warp: weights and weighted sums of 32 items x 8 columns, M
    static constexpr int kTailBytes = kWarps * 4 * 16;      // (m, l) of the pieces the warps' runs end in
    static constexpr int kSegBytes = kWarps * 2 * 4;        // segment of every warp's first and last piece, or -1
    static constexpr int kMergeBytes = (kWarps * kMergeFloats * 4 + kTailBytes + kSegBytes + 15) / 16 * 16;
    static constexpr int kStageItems = kRingBytes / 2 / 4096;   // items half the ring can hold
    static_assert(2 * kWarps <= 32 && kStageItems >= kTreeFan && kStages * kSlotBytes >= 3 * 4096, "chains and tree nodes fit one warp's lanes and staging");
    static constexpr int kBarBytes = kWarps * kStages * 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kFixed = 1024 + kRingBytes + kScaleRing + kMergeBytes + kBarBytes;
    static size_t smem_bytes(int B) { return (size_t)kFixed + ((size_t)(B + 1) * 4 + 15) / 16 * 16; }
};

__device__ __forceinline__ float fast_log2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Maximum over the warp (redux.sync takes fp32 on sm_100a; NaN is ignored).
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lds32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}
template <int kWarps, int kStages>
__global__ void __launch_bounds__(32 * kWarps)
stream_int8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ CUtensorMap tm_s, const StreamInt8Params p) {
    using S = StreamInt8Shape<kWarps, kStages>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_warp_sum[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int B = p.B, Hkv = p.Hkv, G = p.G;
    const bool chunked = p.query_start != nullptr;

    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t ring = (raw + 1023u) & ~1023u;
    const uint32_t scale_ring = ring + S::kRingBytes;
    uint8_t* after = smem_raw + (ring - raw) + S::kRingBytes + S::kScaleRing;
    float* wts = reinterpret_cast<float*>(after) + warp * S::kMergeFloats;   // [32 items][8 columns] x 2, M[8]
    float4* tail_ml = reinterpret_cast<float4*>(after + kWarps * S::kMergeFloats * 4);              // [warps][4]
    int* seg_of = reinterpret_cast<int*>(after + kWarps * S::kMergeFloats * 4 + S::kTailBytes);   // [warps][2]
    const uint32_t bars = scale_ring + S::kScaleRing + S::kMergeBytes;
    int* prefix = reinterpret_cast<int*>(after + S::kMergeBytes + S::kBarBytes);   // [B + 1]

    grid_dependency_wait();                       // inputs may come from the previous launch
    grid_dependents_launch();

    const int cap = min(p.max_context_len, p.max_blocks_per_seq * kPageRows);
    // context length and query count of sequence b (decode: clamped, one query; chunk: inconsistent
    // lengths give no queries); `flag`: report what was wrong
    auto sequence = [&](int b, int& L, int& nq, bool flag) {
        L = __ldg(p.context_lens + b);
        if (!chunked) {
            nq = 1;
            if (L < 0 || L > cap) {
                if (flag) flag_error(PKV_DEVERR_CONTEXT_LEN);
                L = L < 0 ? 0 : cap;
            }
            return;
        }
        const int q0 = __ldg(p.query_start + b), q1 = __ldg(p.query_start + b + 1);
        nq = q1 - q0;
        if (q0 < 0 || q1 < q0 || q1 > p.total || nq > p.max_query_len || L < nq || L > cap) {
            if (flag) flag_error(PKV_DEVERR_CONTEXT_LEN);
            nq = 0;
        }
    };
    auto units_of_seq = [&](int b, bool flag) -> int {
        int L, nq;
        sequence(b, L, nq, flag);
        return nq > 0 ? Hkv * ((L + kPageRows - 1) / kPageRows) : 0;
    };

    // ---- unit order: units of sequence b start at prefix[b], as (KV head, page) ----
    {
        const int per = (B + S::kThreads - 1) / S::kThreads;
        const int b_lo = min(B, (int)threadIdx.x * per), b_hi = min(B, b_lo + per);
        int local = 0;
        for (int b = b_lo; b < b_hi; ++b) local += units_of_seq(b, blockIdx.x == 0);
        int incl = local;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        if (lane == 31) s_warp_sum[warp] = incl;
        if (lane == 0)
            for (int s = 0; s < kStages; ++s) mbar_init(bars + 8u * (warp * kStages + s), 1);
        mbar_init_fence();
        __syncthreads();
        int run = incl - local;
        for (int w = 0; w < warp; ++w) run += s_warp_sum[w];
        for (int b = b_lo; b < b_hi; ++b) {
            prefix[b] = run;
            run += units_of_seq(b, false);
        }
        if (b_hi == B && b_lo < B) prefix[B] = run;
        __syncthreads();
    }
    const int U = prefix[B];
    const int W_total = gridDim.x * kWarps;
    const int worker = blockIdx.x * kWarps + warp;
    // decode: empty contexts get zero rows, spread over all warps
    if (!chunked) {
        for (int b = worker; b < B; b += W_total) {
            if (prefix[b + 1] != prefix[b]) continue;
            uint4* ob = reinterpret_cast<uint4*>(p.out + (int64_t)b * p.Hq * kHeadDim);
            for (int i = lane; i < p.Hq * kHeadDim / 8; i += 32) ob[i] = make_uint4(0, 0, 0, 0);
        }
    }
    const int want = (int)(((int64_t)U + p.min_units_per_worker - 1) / p.min_units_per_worker);
    const int W = min(W_total, max(1, want));
    const int u0 = U == 0 ? 0 : (int)range_start(worker, U, W);
    const int n = (U == 0 || worker >= W) ? 0 : (int)range_start(worker + 1, U, W) - u0;
    if (lane < 2) seg_of[2 * warp + lane] = -1;
    if (lane == 0) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        prefetch_tensormap(&tm_s);
    }

    auto full_bar = [&](int s) { return bars + 8u * (warp * kStages + s); };
    auto k_tile = [&](int s) { return ring + (warp * kStages + s) * S::kSlotBytes; };
    auto s_tile = [&](int s) { return scale_ring + (warp * kStages + s) * S::kScaleBytes; };
    auto pages_of = [&](int b) { return (min(max(__ldg(p.context_lens + b), 0), cap) + kPageRows - 1) / kPageRows; };

    // Block-table window: lane k holds (physical block, KV head) of unit 32 w + k.
    auto load_window = [&](int w, int& phys, int& head) {
        const int t = 32 * w + lane;
        phys = -1;
        head = 0;
        if (t < n) {
            const int u = u0 + t;
            const int b = seq_of_unit(prefix, B, u);
            const int nb = pages_of(b);
            const int rr = u - prefix[b];
            head = rr / nb;
            phys = __ldg(p.block_tables + (int64_t)b * p.max_blocks_per_seq + (rr - head * nb));
        }
    };
    int win_phys, win_head, nxt_phys, nxt_head, cur_win = 0;
    load_window(0, win_phys, win_head);
    nxt_phys = -1, nxt_head = 0;                 // (the next window is looked up behind the first copies)
    const uint64_t policy = l2_evict_first_policy();             // a page is read once
    int issued = 0;                              // units [0, issued) have their copies in flight or landed
    auto issue = [&](int t) {
        const int w = t >> 5;
        if (w != cur_win) {                      // windows are consumed in order
            win_phys = nxt_phys;
            win_head = nxt_head;
            cur_win = w;
            load_window(w + 1, nxt_phys, nxt_head);
        }
        int pb = __shfl_sync(0xffffffffu, win_phys, t & 31);
        const int hg = __shfl_sync(0xffffffffu, win_head, t & 31);
        issued = t + 1;
        if (lane == 0) {
            if (pb < 0 || pb >= p.num_blocks) {  // outside the pool: scales (and codes) read as zeros
                flag_error(PKV_DEVERR_BLOCK_ID);
                pb = -1;
            }
            const int s = t % kStages;
            fence_proxy_async_shared();          // earlier generic reads of the slot come first
            mbar_arrive_expect_tx(full_bar(s), S::kSlotBytes + S::kScaleBytes);
            tma_load_3d(s_tile(s), &tm_s, full_bar(s), 0, hg, pb, policy);
            tma_load_3d(k_tile(s), &tm_k, full_bar(s), 0, hg, pb * kPageRows, policy);
            tma_load_3d(k_tile(s) + S::kTileBytes, &tm_v, full_bar(s), 0, hg, pb * kPageRows, policy);
        }
    };
    for (int t = 0; t < min(n, kStages); ++t) issue(t);
    load_window(1, nxt_phys, nxt_head);

    // ---- the current segment: KV head g of sequence b; page j of nb ----
    const int r = lane >> 2, c = lane & 3;
    int b = n > 0 ? seq_of_unit(prefix, B, u0) : 0;
    int nb = n > 0 ? pages_of(b) : 1;
    int g = n > 0 ? (u0 - prefix[b]) / nb : 0;
    int j = n > 0 ? (u0 - prefix[b]) - g * nb : 0;
    int piece_j0 = j;
    int row0 = 0, ncols = 0;                     // the sequence's first row of q and out; live columns
    int lim_lo = 0, lim_hi = 0;                  // positions of its first and last query
    int lim[2];                                  // causal limits of this lane's columns 2c, 2c + 1
    uint32_t qf[8][2];                           // query vector of column r, as the B operand
    auto open_segment = [&]() {
        int L, nq;
        sequence(b, L, nq, false);
        row0 = chunked ? __ldg(p.query_start + b) : b;
        ncols = nq * G;
        lim_lo = L - nq;
        lim_hi = L - 1;
#pragma unroll
        for (int e = 0; e < 2; ++e) lim[e] = 2 * c + e < ncols ? lim_lo + (2 * c + e) / G : lim_hi;   // idle: as the last
        // channels 16 kk + 4c .. + 3, in the order the codes arrive
        const uint2* qrow = reinterpret_cast<const uint2*>(
            p.q + ((int64_t)(row0 + r / G) * p.Hq + (int64_t)g * G + r % G) * kHeadDim);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            const uint2 v = r < ncols ? __ldg(qrow + 4 * kk + c) : make_uint2(0u, 0u);
            qf[kk][0] = v.x;
            qf[kk][1] = v.y;
        }
    };
    if (n > 0) open_segment();

    float m[2], l[2], o[8][4];                   // columns 2c, 2c + 1: running maximum, sum, output
    auto reset = [&]() {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    };
    reset();
    const float sl = p.logit_scale_log2;

    // One online-softmax step over kPages consecutive pages (slots s0, s1) from page jp on.
    auto attend = [&](auto pages_tag, int s0, int s1, int jp) {
        constexpr int kPages = decltype(pages_tag)::value;
        float x[kPages][4], rv[kPages][2];
#pragma unroll
        for (int pg = 0; pg < kPages; ++pg) {
            const int s = pg ? s1 : s0;
            const uint32_t kt = k_tile(s), sc = s_tile(s);
            float ks[2], lv[2];
            const int t0 = (jp + pg) * kPageRows;               // position of the page's first token
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float kr = lds32(sc + 4 * (r + 8 * e)), vr = lds32(sc + 64 + 4 * (r + 8 * e));
                const bool k_ok = kr >= 0.f && kr <= kScaleMax, v_ok = vr >= 0.f && vr <= kScaleMax;
                if (t0 + r + 8 * e <= lim_hi && !(k_ok && v_ok)) flag_error(PKV_DEVERR_SCALE);
                ks[e] = k_ok ? kr * sl : 0.f;
                const float v = v_ok ? fmaxf(vr, kScaleMin) : kScaleMin;
                lv[e] = fast_log2(v);
                rv[pg][e] = fast_rcp(v);
            }
            // S^T (16 tokens x 8 columns) = K (16 x 128) . Q^T, in the codes' units, in two accumulators
            // (half the chain of dependent products)
            float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            const int row = lane & 15;
#pragma unroll
            for (int J = 0; J < 4; ++J) {
                const int chunk = 2 * J + (lane >> 4);
                uint32_t w0, w1, w2, w3;                        // 4 codes each: channels 16 chunk + 4c .. + 3
                ldsm_x4(kt + row * 128 + ((chunk ^ (row & 7)) << 4), w0, w1, w2, w3);
                uint32_t h[8];
                codes_to_half2x2(w0, h[0], h[1]);
                codes_to_half2x2(w1, h[2], h[3]);
                codes_to_half2x2(w2, h[4], h[5]);
                codes_to_half2x2(w3, h[6], h[7]);
                mma_16816(acc[0], h[0], h[2], h[1], h[3], qf[2 * J][0], qf[2 * J][1]);
                mma_16816(acc[1], h[4], h[6], h[5], h[7], qf[2 * J + 1][0], qf[2 * J + 1][1]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) x[pg][e] = fmaf(acc[0][e] + acc[1][e], ks[e >> 1], lv[e >> 1]);
            if (t0 + kPageRows - 1 > lim_lo) {                  // some row lies past some column's limit
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t0 + r + 8 * (e >> 1) > lim[e & 1]) x[pg][e] = -INFINITY;
            }
        }
        float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
        for (int pg = 0; pg < kPages; ++pg) {
            b0 = fmaxf(b0, fmaxf(x[pg][0], x[pg][2]));
            b1 = fmaxf(b1, fmaxf(x[pg][1], x[pg][3]));
        }
        if (__any_sync(0xffffffffu, b0 > m[0] + kStreamRaise || b1 > m[1] + kStreamRaise)) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, off));
                b1 = fmaxf(b1, __shfl_xor_sync(0xffffffffu, b1, off));
            }
            const float n0 = fmaxf(m[0], b0), n1 = fmaxf(m[1], b1);
            // (a column that has seen no live row keeps m = -inf, l = 0 and O = 0)
            const float a0 = fast_exp2(m[0] - fmaxf(n0, kLogitFloor)), a1 = fast_exp2(m[1] - fmaxf(n1, kLogitFloor));
            m[0] = n0;
            m[1] = n1;
            l[0] *= a0;
            l[1] *= a1;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i][0] *= a0; o[i][1] *= a1; o[i][2] *= a0; o[i][3] *= a1;
            }
        }
        const float m0 = fmaxf(m[0], kLogitFloor), m1 = fmaxf(m[1], kLogitFloor);
        uint32_t pb[kPages][2];
#pragma unroll
        for (int pg = 0; pg < kPages; ++pg) {
            const float p0 = fast_exp2(x[pg][0] - m0), p1 = fast_exp2(x[pg][1] - m1);
            const float p2 = fast_exp2(x[pg][2] - m0), p3 = fast_exp2(x[pg][3] - m1);
            l[0] = fmaf(p0, rv[pg][0], fmaf(p2, rv[pg][1], l[0]));
            l[1] = fmaf(p1, rv[pg][0], fmaf(p3, rv[pg][1], l[1]));
            // P^T as the B operand: transpose the (token x column) accumulator layout
            pb[pg][0] = movmatrix_trans(pack_half2(p0, p1));
            pb[pg][1] = movmatrix_trans(pack_half2(p2, p3));
        }
        // O^T (128 channels x 8 columns) += V^T . P^T: a transposing load of byte pairs gives lane
        // (r, c) channels 16 i + 2r, + 1 of tokens 2c, 2c + 1, so rows r and r + 8 of product tile i
        // are channels 16 i + 2r and 16 i + 2r + 1
#pragma unroll
        for (int pg = 0; pg < kPages; ++pg) {
            const uint32_t vt = k_tile(pg ? s1 : s0) + S::kTileBytes;
            const int row = lane & 15;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const int chunk = i + (lane >> 4);
                uint32_t w0, w1, w2, w3;
                ldsm_x4_trans(vt + row * 128 + ((chunk ^ (row & 7)) << 4), w0, w1, w2, w3);
                uint32_t h[8];
                codes_to_half2x2_cross(w0, h[0], h[1]);
                codes_to_half2x2_cross(w1, h[2], h[3]);
                codes_to_half2x2_cross(w2, h[4], h[5]);
                codes_to_half2x2_cross(w3, h[6], h[7]);
                mma_16816(o[i], h[0], h[1], h[2], h[3], pb[pg][0], pb[pg][1]);
                mma_16816(o[i + 1], h[4], h[5], h[6], h[7], pb[pg][0], pb[pg][1]);
            }
        }
    };

    // out[row, head of g], from fragment-order values times inv0, inv1
    auto write_out = [&](const float (&v)[8][4], float inv0, float inv1) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int col = 2 * c + e;
            if (col >= ncols) continue;
            __half2* dst = reinterpret_cast<__half2*>(
                p.out + ((int64_t)(row0 + col / G) * p.Hq + (int64_t)g * G + col % G) * kHeadDim);
            const float inv = e ? inv1 : inv0;
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[8 * i + r] = __floats2half2_rn(v[i][e] * inv, v[i][2 + e] * inv);
        }
    };
    // Writes or puts aside the piece of the current segment whose last page is j_last.
    auto finish_piece = [&](int j_last, bool at_end) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], off);
            l[1] += __shfl_xor_sync(0xffffffffu, l[1], off);
        }
        if (piece_j0 == 0 && j_last == nb - 1) {                // the whole segment
            write_out(o, 1.f / l[0], 1.f / l[1]);
            return;
        }
        // the piece a run ends in stays in the ring (free by now), the piece it began in goes to the workspace
        const float4 ml = make_float4(m[0], l[0], m[1], l[1]);
        if (at_end) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" :: "r"(k_tile(0) + 512 * i + 16 * lane),
                             "f"(o[i][0]), "f"(o[i][1]), "f"(o[i][2]), "f"(o[i][3]) : "memory");
            if (r == 0) tail_ml[4 * warp + c] = ml;
        } else {
            float4* dst = p.ws_o + (int64_t)worker * 256 + lane;
#pragma unroll
            for (int i = 0; i < 8; ++i) __stcg(dst + 32 * i, make_float4(o[i][0], o[i][1], o[i][2], o[i][3]));
            if (r == 0) __stcg(p.ws_ml + (int64_t)worker * 4 + c, ml);
        }
        if (lane == 0) seg_of[2 * warp + (at_end ? 1 : 0)] = b * Hkv + g;
    };

    // A wait that ran out (flagged) ends this worker's run, after the copies it issued have landed. Its
    // pieces are not merged; the workspace's tickets must be cleared.
    auto drain_after = [&](int lost) {
        for (int u = lost + 1; u < issued; ++u) mbar_wait(full_bar(u % kStages), (u / kStages) & 1);
    };
    for (int t = 0; t < n; ++t) {
        const int s = t % kStages;
        if (!__all_sync(0xffffffffu, mbar_wait(full_bar(s), (t / kStages) & 1))) {
            drain_after(t);
            break;
        }
        if (j + 1 < nb && t + 1 < n) {           // two pages of the segment in one softmax step
            const int s2 = (t + 1) % kStages;
            if (!__all_sync(0xffffffffu, mbar_wait(full_bar(s2), ((t + 1) / kStages) & 1))) {
                drain_after(t + 1);
                break;
            }
            attend(std::integral_constant<int, 2>(), s, s2, j);
            __syncwarp();
            if (t + kStages < n) issue(t + kStages);
            if (t + 1 + kStages < n) issue(t + 1 + kStages);
            ++t;                                  // the cursor moves to the second page
            ++j;
        } else {
            attend(std::integral_constant<int, 1>(), s, s, j);
            __syncwarp();
            if (t + kStages < n) issue(t + kStages);
        }
        const bool seg_end = j == nb - 1;
        if (seg_end || t == n - 1) {
            finish_piece(j, t == n - 1);
            if (t == n - 1) break;
            // (a run's last unit always closes a piece, so here the segment ended)
            j = 0;
            if (++g == Hkv) {
                g = 0;
                do { ++b; } while (prefix[b + 1] == prefix[b]);
                nb = pages_of(b);
            }
            open_segment();
            reset();
            piece_j0 = 0;
        } else {
            ++j;
        }
    }

    // ---- the CTA's pieces, in the order of its run: piece 2 w (the one warp w's run began in) and
    // 2 w + 1 (the one it ended in), where they exist; pieces of one segment are neighbours ----
    __syncthreads();
    const int my_seg = lane < 2 * kWarps ? seg_of[lane] : -1;
    const unsigned pieces = __ballot_sync(0xffffffffu, my_seg >= 0);
    const unsigned before = pieces & ((1u << lane) - 1u);
    const int prev_seg = __shfl_sync(0xffffffffu, my_seg, before ? 31 - __clz(before) : 0);
    unsigned starts = __ballot_sync(0xffffffffu, my_seg >= 0 && (before == 0 || prev_seg != my_seg));
    const int n_chains = __popc(starts);
    const int cta_lo = (int)range_start(min((int)blockIdx.x * kWarps, W), U, W);
    const int cta_hi = (int)range_start(min(((int)blockIdx.x + 1) * kWarps, W), U, W);
    float acc[8][4], L0, L1;                                    // a merge's O, and sums of columns 2c, 2c + 1
    // Starts a merge of n_it items, whose (m, l) of columns 2k, 2k + 1 lane q has for item q: their weights
    // 2^(m - M) go to wts.
    auto weigh = [&](int n_it, auto ml) {
        float mm[8], ll[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float4 a = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
            if (lane < n_it) a = ml(k);
            mm[2 * k] = a.x; ll[2 * k] = a.y; mm[2 * k + 1] = a.z; ll[2 * k + 1] = a.w;
        }
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            const float M = warp_max(mm[h]);
            const float w = fast_exp2(mm[h] - fmaxf(M, kLogitFloor));       // 0 for an item that saw nothing
            wts[lane * 8 + h] = w;
            wts[256 + lane * 8 + h] = w * ll[h];
            if (lane == 0) wts[512 + h] = M;
        }
        __syncwarp();
        L0 = L1 = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    };
    // adds item k, `v` being this lane's eight float4 of it
    auto add_item = [&](int k, const float4 (&v)[8]) {
        const float w0 = wts[k * 8 + 2 * c], w1 = wts[k * 8 + 2 * c + 1];
        L0 += wts[256 + k * 8 + 2 * c];
        L1 += wts[257 + k * 8 + 2 * c];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            acc[i][0] = fmaf(w0, v[i].x, acc[i][0]); acc[i][1] = fmaf(w1, v[i].y, acc[i][1]);
            acc[i][2] = fmaf(w0, v[i].z, acc[i][2]); acc[i][3] = fmaf(w1, v[i].w, acc[i][3]);
        }
    };
    auto load_shared_item = [&](uint32_t addr, float4 (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint4 u = lds128(addr + 512 * i + 16 * lane);
            v[i] = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
        }
    };
    const int item0 = gridDim.x * kWarps;                       // the CTAs' items lie behind the workers' pieces
    auto publish = [&](int slot) {
        float4* dst = p.ws_o + (int64_t)slot * 256 + lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) __stcg(dst + 32 * i, make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]));
        if (r == 0)
            __stcg(p.ws_ml + (int64_t)slot * 4 + c,
                   make_float4(wts[512 + 2 * c], L0, wts[513 + 2 * c], L1));
    };
    int half = -1, seg_first = 0;                               // this warp's item of the CTA: 0, 1 or none
    for (int k = 0; k < n_chains; ++k) {
        const int first = __ffs(starts) - 1;
        starts &= starts - 1;
        // a warp each; of kWarps + 1 chains (every boundary between warps cuts a segment) the last warp takes
        // two, of which the first lies inside the CTA
        if (min(k, kWarps - 1) != warp) continue;
        // the chain: the pieces from `first` up to the next chain
        const unsigned chain = pieces & ~((1u << first) - 1u) & (starts ? (1u << (__ffs(starts) - 1)) - 1u : 0xffffffffu);
        const int n_it = __popc(chain);
        const int seg = __shfl_sync(0xffffffffu, my_seg, first);
        b = seg / Hkv;
        g = seg - b * Hkv;
        nb = pages_of(b);
        open_segment();
        const int sf = prefix[b] + g * nb;
        // lane q's piece, 2 w or 2 w + 1: the q-th set bit of the chain
        unsigned rest = chain;
        for (int q = 0; q < lane && q < n_it; ++q) rest &= rest - 1;
        const int piece = lane < n_it ? __ffs(rest) - 1 : 0;
        weigh(n_it, [&](int e) {
            return (piece & 1) ? tail_ml[4 * (piece >> 1) + e]
                               : __ldcg(p.ws_ml + (int64_t)(blockIdx.x * kWarps + (piece >> 1)) * 4 + e);
        });
        for (int q = 0; q < n_it; ++q) {
            const int pq = __shfl_sync(0xffffffffu, piece, q), w = pq >> 1;
            float4 v[8];
            if (pq & 1) {
                load_shared_item(ring + w * kStages * S::kSlotBytes, v);
            } else {
                const float4* src = p.ws_o + (int64_t)(blockIdx.x * kWarps + w) * 256 + lane;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __ldcg(src + 32 * i);
            }
            add_item(q, v);
        }
        if (sf >= cta_lo && sf + nb <= cta_hi) {
            write_out(acc, 1.f / L0, 1.f / L1);
        } else {
            half = sf >= cta_lo ? 1 : 0;
            seg_first = sf;
            publish(item0 + 2 * blockIdx.x + half);
        }
        __syncwarp();
    }
    // A merge of more than two items stages them through the ring, once every warp is done with the pieces
    // in it; nobody else waits for that.
    bool arrived = false;
    auto leave_ring = [&]() {
        if (!arrived) asm volatile("bar.arrive 1, %0;" :: "n"(S::kThreads) : "memory");
        arrived = true;
    };
    auto take_ring = [&]() {
        if (!arrived) asm volatile("bar.sync 1, %0;" :: "n"(S::kThreads) : "memory");
        arrived = true;
    };
    if (half < 0) {
        leave_ring();
        return;
    }

    // ---- the ticket tree over the CTAs' items of this segment ----
    const int c_first = worker_of(seg_first, U, W) / kWarps;
    int n_items = worker_of(seg_first + nb - 1, U, W) / kWarps - c_first + 1;
    int item = blockIdx.x - c_first, span = 1;
    auto slot_of_item = [&](int q) {                             // 2 c + 1 where the segment began in CTA c
        const int cc = c_first + q;
        return 2 * cc + (range_start(cc * kWarps, U, W) <= seg_first ? 1 : 0);
    };
    bool whole_ring = false;                                    // the ring has been waited for
    for (int lvl = 0;; ++lvl) {
        const int first = item - item % kTreeFan, last = min(first + kTreeFan, n_items) - 1;
        const int cslot = slot_of_item(first * span);
        unsigned int* cnt = p.ws_count + (int64_t)lvl * 2 * gridDim.x + cslot;
        // the warp barrier orders every lane's stores before lane 0's release-acquire ticket; the
        // merger's loads follow its acquire
        __syncwarp();
        unsigned int prev = 0;
        if (lane == 0) prev = atomic_add_acq_rel_gpu(cnt, 1u);
        prev = __shfl_sync(0xffffffffu, prev, 0);
        __syncwarp();                           // the acquire is lane 0's: the shuffle orders no memory
        if (prev != (unsigned int)(last - first)) {             // another item merges the node
            leave_ring();
            return;
        }
        if (lane == 0) *cnt = 0u;                               // ready for the next call
        const int n_it = last - first + 1;
        // two items fit behind this warp's own piece in its share of the ring
        whole_ring = whole_ring || n_it > 2;
        if (whole_ring) take_ring();
        const uint32_t stage = whole_ring ? ring + half * (S::kStageItems * 4096) : k_tile(0) + 4096;
        const int my_slot = item0 + (lane < n_it ? slot_of_item((first + lane) * span) : 0);
        for (int q = 0; q < n_it; ++q) {
            const int slot = __shfl_sync(0xffffffffu, my_slot, q);
            const float4* src = p.ws_o + (int64_t)slot * 256 + lane;
#pragma unroll
            for (int i = 0; i < 8; ++i) cp_async16(stage + q * 4096 + 512 * i + 16 * lane, src + 32 * i);
        }
        cp_async_commit();
        weigh(n_it, [&](int e) { return __ldcg(p.ws_ml + (int64_t)my_slot * 4 + e); });
        cp_async_wait_all();
        __syncwarp();
        for (int q = 0; q < n_it; ++q) {
            float4 v[8];
            load_shared_item(stage + q * 4096, v);
            add_item(q, v);
        }
        const int n_next = (n_items + kTreeFan - 1) / kTreeFan;
        if (n_next == 1) {
            leave_ring();
            write_out(acc, 1.f / L0, 1.f / L1);
            return;
        }
        publish(item0 + cslot);                                 // the node is one item of the next level
        __syncwarp();
        item = first / kTreeFan;
        n_items = n_next;
        span *= kTreeFan;
    }
}

}  // namespace pkv

// Attention over the 8-bit paged cache with a scale per token and KV head
// (int8_cache.cuh), load-balanced streaming form: decode (one query token per
// sequence), and chunks whose query tokens x heads fit eight columns.
//
// Work is cut as in decode_balanced.cuh: a unit is one page (16 tokens) of one
// KV head of one sequence; the units of the batch form a row, every warp of
// the persistent grid takes an equal run of it, streams its pages through its
// own ring of TMA copies, and the pieces of a segment (sequence, KV head) that
// was cut between warps are merged by a fan-in-32 ticket tree. Nothing waits
// on another CTA.
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
// Bound: HBM. Bytes of a unit: 2 x 16 x (128 + 4).
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
    float4* ws_o;                 // [2 * workers][8][32 lanes]  pieces' unnormalised O
    float4* ws_ml;                // [2 * workers][4]  (m, l) of columns 2c, 2c + 1
    unsigned int* ws_count;       // tickets of the merge tree, zero between calls
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

template <int kWarps, int kStages>
struct StreamInt8Shape {
    static constexpr int kTileBytes = 2048;                 // one page of K (or V) codes, one head
    static constexpr int kSlotBytes = 2 * kTileBytes;
    static constexpr int kScaleBytes = 128;                 // K scales, V scales of the page
    static constexpr int kRingBytes = kWarps * kStages * kSlotBytes;
    static constexpr int kScaleRing = kWarps * kStages * kScaleBytes;
    static constexpr int kMergeBytes = kWarps * kMergeFloats * 4;
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
    float* wts = reinterpret_cast<float*>(after) + warp * kMergeFloats;    // [32 items][8 columns], M[8], L[8]
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
    if (n <= 0) return;
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
    load_window(1, nxt_phys, nxt_head);
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

    // ---- the current segment: KV head g of sequence b; page j of nb ----
    const int r = lane >> 2, c = lane & 3;
    int b = seq_of_unit(prefix, B, u0);
    int nb = pages_of(b);
    int g = (u0 - prefix[b]) / nb;
    int j = (u0 - prefix[b]) - g * nb;
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
    open_segment();

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
    // (m, l, O) of one partial result, in fragment order, at workspace slot `slot`
    auto store_item = [&](int slot, const float (&v)[8][4], float m0, float l0, float m1, float l1) {
        float4* dst = p.ws_o + (int64_t)slot * 256 + lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) __stcg(dst + 32 * i, make_float4(v[i][0], v[i][1], v[i][2], v[i][3]));
        if (r == 0) __stcg(p.ws_ml + (int64_t)slot * 4 + c, make_float4(m0, l0, m1, l1));
    };

    // Finishes the piece of the current segment whose last page is j_last.
    auto finish_piece = [&](int j_last) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], off);
            l[1] += __shfl_xor_sync(0xffffffffu, l[1], off);
        }
        if (piece_j0 == 0 && j_last == nb - 1) {                // the whole segment
            write_out(o, 1.f / l[0], 1.f / l[1]);
            return;
        }
        const int seg_first = prefix[b] + g * nb;
        const int k_first = worker_of(seg_first, U, W);
        const int k_last = worker_of(seg_first + nb - 1, U, W);
        auto slot_of_piece = [&](int q) {
            const int k = k_first + q;
            return 2 * k + (range_start(k, U, W) >= seg_first ? 0 : 1);
        };
        int item = worker - k_first, n_items = k_last - k_first + 1, span = 1;
        store_item(slot_of_piece(item), o, m[0], l[0], m[1], l[1]);
        for (int lvl = 0;; ++lvl) {
            const int first = item - item % kMergeFan, last = min(first + kMergeFan, n_items) - 1;
            const int cslot = slot_of_piece(first * span);
            unsigned int* cnt = p.ws_count + (int64_t)lvl * 2 * W_total + cslot;
            // the warp barrier orders every lane's stores before lane 0's release-acquire ticket;
            // the merger's loads follow its acquire
            __syncwarp();
            unsigned int prev = 0;
            if (lane == 0) prev = atomic_add_acq_rel_gpu(cnt, 1u);
            prev = __shfl_sync(0xffffffffu, prev, 0);
            if (prev != (unsigned int)(last - first)) return;   // another item merges the group
            const int n_it = last - first + 1;
            const int my_slot = lane < n_it ? slot_of_piece((first + lane) * span) : 0;
            const int n_next = (n_items + kMergeFan - 1) / kMergeFan;
            auto load_vals = [&](float4 (&dst)[2][8], int k) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (k + u < n_it) {
                        const int slot = __shfl_sync(0xffffffffu, my_slot, k + u);
                        const float4* src = p.ws_o + (int64_t)slot * 256 + lane;
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[u][i] = __ldcg(src + 32 * i);
                    }
            };
            float4 va[2][8];
            load_vals(va, 0);
            float mm[8], ll[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float4 a = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
                if (lane < n_it) a = __ldcg(p.ws_ml + (int64_t)my_slot * 4 + k);
                mm[2 * k] = a.x; ll[2 * k] = a.y; mm[2 * k + 1] = a.z; ll[2 * k + 1] = a.w;
            }
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                float M = mm[h];
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
                const float w = fast_exp2(mm[h] - fmaxf(M, kLogitFloor));   // 0 for an item that saw nothing
                float L = w * ll[h];
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
                wts[lane * 8 + h] = w;
                if (lane == 0) {
                    wts[256 + h] = M;
                    wts[264 + h] = L;
                }
            }
            __syncwarp();
            float acc[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll 1
            for (int k = 0; k < n_it; k += 2) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (k + u < n_it) {
                        const float w0 = wts[(k + u) * 8 + 2 * c], w1 = wts[(k + u) * 8 + 2 * c + 1];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            acc[i][0] += w0 * va[u][i].x; acc[i][1] += w1 * va[u][i].y;
                            acc[i][2] += w0 * va[u][i].z; acc[i][3] += w1 * va[u][i].w;
                        }
                    }
                if (k + 2 < n_it) load_vals(va, k + 2);
            }
            const float M0 = wts[256 + 2 * c], M1 = wts[256 + 2 * c + 1];
            const float L0 = wts[264 + 2 * c], L1 = wts[264 + 2 * c + 1];
            __syncwarp();
            if (lane == 0) *cnt = 0u;                             // ready for the next call
            if (n_next == 1) {
                write_out(acc, 1.f / L0, 1.f / L1);
                return;
            }
            store_item(cslot, acc, M0, L0, M1, L1);               // the group is one item of the next level
            item = first / kMergeFan;
            n_items = n_next;
            span *= kMergeFan;
        }
    };

    // A wait that ran out (flagged) ends this worker, after the copies it issued have landed.
    auto drain_after = [&](int lost) {
        for (int u = lost + 1; u < issued; ++u) mbar_wait(full_bar(u % kStages), (u / kStages) & 1);
    };
    for (int t = 0; t < n; ++t) {
        const int s = t % kStages;
        if (!__all_sync(0xffffffffu, mbar_wait(full_bar(s), (t / kStages) & 1))) {
            drain_after(t);
            return;
        }
        if (j + 1 < nb && t + 1 < n) {           // two pages of the segment in one softmax step
            const int s2 = (t + 1) % kStages;
            if (!__all_sync(0xffffffffu, mbar_wait(full_bar(s2), ((t + 1) / kStages) & 1))) {
                drain_after(t + 1);
                return;
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
            finish_piece(j);
            if (t == n - 1) break;
            // (a range's last unit always closes a piece, so here the segment ended)
            j = 0;
            if (++g == Hkv) {
                g = 0;
                do { ++b; } while (prefix[b + 1] == prefix[b]);
                nb = pages_of(b);
            }
            __syncwarp();
            open_segment();
            reset();
            piece_j0 = 0;
        } else {
            ++j;
        }
    }
}

}  // namespace pkv

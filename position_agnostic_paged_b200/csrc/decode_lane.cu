// decode_lane.cu -- decode attention over the bf16 pool that also accumulates each table word's
// attention weight.
//
// Per request, query head h on KV head k, key t with table offset o, local index j and position
// o + j <= p (the query's), as in decode.cu:
//   s_t = scale q_h^T R(-(p - o)) k_t,   w_t = 2^(s_t - M) / L,   out = sum_t w_t v_t,
//   block_mass[word] += sum_h sum_{t in word} w_t.
//
// Work split.  The words of all requests lie one after the other in `table`, so for one KV head
// they form one line of total_words items.  It is cut into equal pieces, one per resident warp
// (a single wave of CTAs: ragged batches balance by themselves, and no request waits for the
// longest).  A warp streams its piece; where a request ends it writes a partial result (m, l,
// acc) to the workspace slot (warp + request), which is unique because each new partial moves on
// to the next warp or the next request.  The second kernel joins a request's partials in order.
//
// Data path.  Each warp is its own producer: lane 0 loads the warp's next words by TMA (128-byte
// swizzle) into the warp's stages, so there are no barriers between warps.  (With cp.async the
// loads of table words, and spilled registers, waited in the L1's queue behind all copies in flight.)
// The K index order of an MMA is free as long as both operands use the same one, and so is the order
// of output rows; both are chosen to make a lane's share contiguous, and a quarter warp's 16-byte
// reads cover all banks:
//   K (rows = keys as the A operand): lane (rr, c) takes 16-byte pieces 2c, 2c + 1 of each half
//     row of 64 dims, key rows rr and rr + 8;
//   V^T (rows = head dims as the A operand): lane (rr, c) takes piece rr of key rows 2c, 2c+1,
//     2c+8, 2c+9 and pairs keys with byte permutes.
// The query is scaled by a power of two to [1, 2) and split into three bf16 parts, so that the
// accumulated fp32 weights are good to a few 2^-22; the weights of the V product are two bf16 parts (2^-16: with one
// the output is off by 0.0023 of itself in the 2-norm, with two by 0.0017, its bf16 rounding alone; 64 requests of 4161
// tokens take the same time, with 32 heads on one KV head 83 us instead of 78).  Scores, sums, maxima and
// outputs are fp32.
//
// What bounds it: HBM.  64 requests of 4161 tokens, 32 heads on 8, read 1.09 GB in 182 us from cold
// caches (6.0 TB/s), 193 us a call with the joining kernel; the two stages that fit a warp (12
// warps per SM, 196 KB in flight) leave it waiting for loads most of the time.  A KV head's wider group of
// query heads is taken by neighbouring warps, eight heads each: one warp with up to 32 heads spilled registers and held one
// CTA per SM (64 requests, 32 heads on one KV head: 177 us against 79 at the time).
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace lazy {

namespace {

constexpr int kMinWords = 2;       // least words per warp
constexpr float kSlack = 8.f;      // log2 units by which a score may pass its reference

__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float fast_log2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Words per warp of one KV head's line: the same on both kernels.
__device__ __forceinline__ int words_per_warp(int total, int warps) {
    return max(kMinWords, (total + warps - 1) / warps);
}

constexpr int kQParts = 3;
constexpr int kTileBytes = 2 * kBoxBytes;        // K (or V) of one word and head
constexpr int kStageBytes = 2 * kTileBytes;

constexpr int kWarps = 4, kOcc = 3;              // per CTA; CTAs per SM, by registers
constexpr int kExtra = 512 + 64;                 // angles, barriers of a warp
constexpr int kStages = ((227 * 1024 / kOcc - 2048) / kWarps - kExtra) / kStageBytes;
constexpr int kSmem = kWarps * (kStages * kStageBytes + kExtra) + 1024;   // stages 1 KiB aligned
static_assert(kStages >= 2 && kStages <= 8, "pipeline depth");

// Groups of 8 query heads of a KV head.
__host__ __device__ inline int head_groups(int group) { return (group + 7) / 8; }

// First of the four head dims of the query fragment's registers for k-step s: rows are two halves of 64 dims,
// lane c has dims 16c .. + 15 of each, and rotation pairs lie in k-steps s and s + 4.
__device__ __forceinline__ int qdim(int s, int c) { return 16 * c + 4 * (s & 3) + 64 * (s >> 2); }
// First head dim of output tile t's row pair (rows rr and rr + 8 hold odim and odim + 1).
__device__ __forceinline__ int odim(int t, int rr) { return 64 * (t >> 2) + 8 * rr + 2 * (t & 3); }

__global__ void __launch_bounds__(kWarps * 32, kOcc)
    decode_lane_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ LaneParams p) {
    pdl_trigger();
    constexpr int QP = kQParts, S = kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = lane & 3, rr = lane >> 2;
    const AttnParams &a = p.a;
    const int G = a.group, hkv = a.hkv, B = a.num_req;
    const int gw = blockIdx.x * kWarps + warp;
    // neighbouring warps take the head groups of one KV head: its words come from L2 for all but the first
    const int groups = head_groups(G), wi = gw / (hkv * groups), line = gw - wi * hkv * groups;
    const int kvh = line / groups, g0 = 8 * (line - kvh * groups);
    // the rotation frequencies: a per-lane read of the parameter table takes 32 turns
    __shared__ double theta[kHalfDim];
    for (int i = threadIdx.x; i < kHalfDim; i += kWarps * 32) theta[i] = a.rope.theta[i];
    __syncthreads();
    if (wi >= p.pieces) return;
    const int base = a.table_indptr[0];
    const int total = a.table_indptr[B] - base;
    if (total <= 0) return;
    const int per = words_per_warp(total, p.pieces);
    if (wi > (total - 1) / per) return;
    const int lo = wi * per, cnt = min(total - lo, per);

    uint8_t *stages = sm + warp * S * kStageBytes;
    uint8_t *extra = sm + kWarps * S * kStageBytes + warp * kExtra;
    float2 *cs = reinterpret_cast<float2 *>(extra);               // [64]
    uint64_t *bars = reinterpret_cast<uint64_t *>(extra + 512);   // [S]
    if (lane < S) mbar_init(&bars[lane], 1);
    fence_barrier_init();
    fence_proxy_async_smem();
    __syncwarp();

    // ---- the words of this warp, 32 at a time, one per lane; metadata is loaded a batch
    // ahead of their use and words two, so that no load is waited for
    uint32_t w_cur, m_cur, w_nxt, m_nxt, w_2nd;
    auto word_at = [&](int k) { return k < cnt ? a.table[base + lo + k] : 0u; };
    auto meta_at = [&](int k, uint32_t w) {
        if (k >= cnt) return 0u;
        const uint32_t b = word_block(w);
        if (b < static_cast<uint32_t>(a.num_blocks)) return a.blk_meta[b];
        set_status(a.d_status, LAZY_DSTATUS_BAD_BLOCK);
        return 0u;
    };
    w_cur = word_at(lane);
    w_nxt = word_at(32 + lane);
    w_2nd = word_at(64 + lane);
    m_cur = meta_at(lane, w_cur);
    m_nxt = meta_at(32 + lane, w_nxt);

    // copies of word k (of this warp) into stage sg, by the lane that holds the word.  A word without tokens, or
    // without a block, completes its phase with no data.
    auto issue = [&](int k, bool next_batch, int sg) {
        if (k < cnt && lane == (k & 31)) {
            const uint32_t w = next_batch ? w_nxt : w_cur, m = next_batch ? m_nxt : m_cur;
            uint64_t *bar = &bars[sg];
            if (meta_valid(m) > 0) {
                uint8_t *d = stages + sg * kStageBytes;
                const int row = (static_cast<int>(word_block(w)) * hkv + kvh) * kBlockTokens;
                mbar_arrive_expect_tx(bar, kStageBytes);
                tma_load_2d(d, &tmK, 0, row, bar);
                tma_load_2d(d + kBoxBytes, &tmK, kHalfDim, row, bar);
                tma_load_2d(d + kTileBytes, &tmV, 0, row, bar);
                tma_load_2d(d + kTileBytes + kBoxBytes, &tmV, kHalfDim, row, bar);
            } else {
                mbar_arrive(bar);
            }
        }
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) issue(k, false, k);

    // ---- the request of the first word: the largest r with table_indptr[r] <= its index
    int r = 0;
    {
        int hi = B;
        while (hi - r > 1) {
            const int step = (hi - r + 31) >> 5;
            const int x = r + step * lane;
            const bool below = x < hi && a.table_indptr[x] - base <= lo;
            const int k = __popc(__ballot_sync(0xffffffffu, below)) - 1;
            r += step * k;
            hi = min(hi, r + step);
        }
    }
    int r_beg = a.table_indptr[r] - base, r_end = a.table_indptr[r + 1] - base;
    int qpos = 0, cur_off = -1;
    uint32_t qb[QP][8][2];
    float qn;            // 2^-e of this lane's fragment head (g0 + rr)
    float hm[2];         // score factor of heads g0 + 2c, + 1: softmax scale * log2(e) * 2^e
    // per head, in log2 units: reference mu of the weights (0 and l_run 0 before the first visible key)
    float mu[2], l_run[2];
    float oacc[8][4];

    auto begin_request = [&]() {
        qpos = a.q_pos[r];
        cur_off = -1;
        if (lo <= r_beg && r_end - r_beg > a.max_words && line == 0 && lane == 0)
            set_status(a.d_status, LAZY_DSTATUS_BAD_TABLE);
        const int g = g0 + rr;
        const uint32_t *q = reinterpret_cast<const uint32_t *>(
            a.q_raw + (static_cast<size_t>(r) * a.hq + kvh * G + min(g, G - 1)) * kHeadDim);
        float am = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const int d = qdim(s, c);
            uint32_t w0 = 0u, w1 = 0u;
            if (g < G) {
                w0 = q[d >> 1];
                w1 = q[(d >> 1) + 1];
            }
            am = fmaxf(am, fmaxf(fmaxf(fabsf(bf16_lo(w0)), fabsf(bf16_hi(w0))),
                                 fmaxf(fabsf(bf16_lo(w1)), fabsf(bf16_hi(w1)))));
        }
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
        // q 2^-e in [1, 2); e = 0 for an all-zero or non-finite head
        int e = static_cast<int>(__float_as_uint(am) >> 23) - 127;
        e = (am == 0.f || e == 128) ? 0 : max(-126, min(126, e));
        qn = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const float q2 = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * a.scale_log2;
        hm[0] = __shfl_sync(0xffffffffu, q2, 8 * c);
        hm[1] = __shfl_sync(0xffffffffu, q2, 8 * c + 4);
#pragma unroll
        for (int j = 0; j < 2; ++j) mu[j] = l_run[j] = 0.f;
#pragma unroll
        for (int t = 0; t < 8; ++t) oacc[t][0] = oacc[t][1] = oacc[t][2] = oacc[t][3] = 0.f;
    };
    // the query turned by (qpos - off), as fragments: angles once per warp (two per lane), shared
    auto rotate = [&](int off) {
        cur_off = off;
        const int delta = a.alibi ? 0 : qpos - off;
        float2 z0, z1;
        rope_cos_sin(delta, theta[lane], z0.x, z0.y);
        rope_cos_sin(delta, theta[lane + 32], z1.x, z1.y);
        __syncwarp();
        cs[lane] = z0;
        cs[lane + 32] = z1;
        __syncwarp();
        const int g = g0 + rr;
        const uint32_t *q = reinterpret_cast<const uint32_t *>(
            a.q_raw + (static_cast<size_t>(r) * a.hq + kvh * G + min(g, G - 1)) * kHeadDim);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            // k-steps s and s + 4: dims d .. d + 3 and their pairs
            const int d = qdim(s, c);
            float x[8];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint32_t wa = g < G ? q[(d >> 1) + y] : 0u, wb = g < G ? q[(d >> 1) + 32 + y] : 0u;
                const float4 z = *reinterpret_cast<const float4 *>(&cs[d + 2 * y]);   // (cos, sin) of two pairs
                const float a0 = bf16_lo(wa) * qn, a1 = bf16_hi(wa) * qn;
                const float b0 = bf16_lo(wb) * qn, b1 = bf16_hi(wb) * qn;
                x[2 * y] = a0 * z.x - b0 * z.y;
                x[2 * y + 1] = a1 * z.z - b1 * z.w;
                x[4 + 2 * y] = b0 * z.x + a0 * z.y;
                x[5 + 2 * y] = b1 * z.z + a1 * z.w;
            }
#pragma unroll
            for (int part = 0; part < QP; ++part) {
                uint32_t w[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    w[y] = pack_bf16(x[2 * y], x[2 * y + 1]);
                    x[2 * y] -= bf16_lo(w[y]);
                    x[2 * y + 1] -= bf16_hi(w[y]);
                }
                qb[part][s][0] = w[0];
                qb[part][s][1] = w[1];
                qb[part][s + 4][0] = w[2];
                qb[part][s + 4][1] = w[3];
            }
        }
    };
    auto end_request = [&]() {
        const size_t slot = static_cast<size_t>(kvh) * (p.pieces + B) + wi + r;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int g = g0 + 2 * c + j;
            if (g < G) {
                float *o = a.ws_acc + (slot * G + g) * kHeadDim;
#pragma unroll
                for (int t = 0; t < 8; t += 2) {
                    // tiles t and t + 1: four consecutive head dims
                    *reinterpret_cast<float4 *>(o + odim(t, rr)) =
                        make_float4(oacc[t][j], oacc[t][j + 2], oacc[t + 1][j], oacc[t + 1][j + 2]);
                }
                if (rr == 0)
                    p.ws_ml[slot * G + g] = l_run[j] == 0.f ? make_float4(-INFINITY, 0.f, -INFINITY, 0.f)
                                                               : make_float4(mu[j], l_run[j], mu[j], 0.f);
            }
        }
    };
    begin_request();

    int sg = S - 1, before = S - 2;   // stages of words k and k - 1
    uint32_t phase = 1;               // of stage sg
    for (int k = 0; k < cnt; ++k) {
        before = sg;
        if (++sg == S) {
            sg = 0;
            phase ^= 1;
        }
        if (k > 0 && (k & 31) == 0) {
            w_cur = w_nxt;
            m_cur = m_nxt;
            w_nxt = w_2nd;
            w_2nd = word_at(k + 64 + lane);
            m_nxt = meta_at(k + 32 + lane, w_nxt);
        }
        __syncwarp();   // every lane has read the stage that is loaded next
        issue(k + S - 1, (k & 31) + S - 1 >= 32, before);
        if (!__all_sync(0xffffffffu, mbar_wait(&bars[sg], phase))) {
            set_status(a.d_status, LAZY_DSTATUS_TIMEOUT);
            for (int i = k; i < min(cnt, k + S); ++i) mbar_wait(&bars[i % S], (i / S) & 1);   // copies in flight
            break;
        }
        if (lo + k >= r_end) {
            end_request();
            do {
                ++r;
                r_beg = r_end;
                r_end = a.table_indptr[r + 1] - base;
            } while (lo + k >= r_end);
            begin_request();
        }
        const uint32_t w = __shfl_sync(0xffffffffu, w_cur, k & 31);
        const uint32_t meta = __shfl_sync(0xffffffffu, m_cur, k & 31);
        const int i_req = lo + k - r_beg;                       // index of the word in its request
        const int off = word_offset(w);
        const int pos0 = off + meta_j0(meta);
        // keys of this word that the query sees: slots 0 .. lim - 1
        const int lim = i_req < a.max_words ? seen_slots(meta_valid(meta), qpos, pos0) : 0;
        float *lse = p.ws_lse + (static_cast<size_t>(r) * a.max_words + i_req) * a.hq + kvh * G;
        if (lim <= 0) {
            if (i_req < a.max_words && lane < 8 && g0 + lane < G) lse[g0 + lane] = -INFINITY;
            continue;
        }
        if (cur_off < 0 || (off != cur_off && !a.alibi)) rotate(off);

        const uint32_t st = smem_u32(stages) + sg * kStageBytes;
        // ---- S^T [16 keys][8 heads] = K q^T
        float sa[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            // piece 2c + (m & 1) of half m >> 1 of key rows rr and rr + 8: two k-steps
            const uint32_t ka = st + (m >> 1) * kBoxBytes + rr * 128 + (((2 * c + (m & 1)) ^ rr) << 4);
            const uint4 ra = lds16(ka), rb = lds16(ka + 1024);
            const uint32_t aw[4] = {ra.x, ra.y, ra.z, ra.w}, bw[4] = {rb.x, rb.y, rb.z, rb.w};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int s = 2 * m + u;
                const uint32_t a0 = aw[2 * u], a1 = bw[2 * u], a2 = aw[2 * u + 1], a3 = bw[2 * u + 1];
#pragma unroll
                for (int part = 0; part < QP; ++part) mma_bf16(sa, a0, a1, a2, a3, qb[part][s][0], qb[part][s][1]);
            }
        }
        // ---- softmax over the word's keys (rr and rr + 8 in this lane).  A reference moves
        // only when some score passes it by kSlack: weights stay below 2^8 and most words need neither the
        // maxima nor rescaling.
        // scores relative to mu
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            sa[j] = fmaf(sa[j], hm[j], -mu[j]);
            sa[j + 2] = fmaf(sa[j + 2], hm[j], -mu[j]);
        }
        if (a.alibi) {
            const float d0 = static_cast<float>(pos0 + rr - qpos);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float sl = g0 + 2 * c + j < G ? a.alibi_log2[kvh * G + g0 + 2 * c + j] : 0.f;
                sa[j] = fmaf(sl, d0, sa[j]);
                sa[j + 2] = fmaf(sl, d0 + 8.f, sa[j + 2]);
            }
        }
        if (lim < kBlockTokens) {
            if (rr >= lim) sa[0] = sa[1] = -INFINITY;
            if (rr + 8 >= lim) sa[2] = sa[3] = -INFINITY;
        }
        bool past = false;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float top = fmaxf(sa[j], sa[j + 2]);
            past |= top > (l_run[j] == 0.f ? -INFINITY : kSlack);
        }
        if (__any_sync(0xffffffffu, past)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float bm = fmaxf(sa[j], sa[j + 2]);
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, x));
                if (bm == -INFINITY) continue;   // this head sees no key of the word
                const float up = l_run[j] == 0.f ? bm : fmaxf(bm, 0.f);
                if (l_run[j] != 0.f) {
                    const float sc = fast_exp2(-up);
                    l_run[j] *= sc;
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        oacc[t][j] *= sc;
                        oacc[t][j + 2] *= sc;
                    }
                }
                mu[j] += up;
                sa[j] -= up;
                sa[j + 2] -= up;
            }
        }
        float pr[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float p0 = fast_exp2(sa[j]), p1 = fast_exp2(sa[j + 2]);
            float ps = p0 + p1;
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) ps += __shfl_xor_sync(0xffffffffu, ps, x);
            const int g = g0 + 2 * c + j;
            if (rr == 0 && g < G) lse[g] = mu[j] + fast_log2(ps);
            l_run[j] += ps;
            pr[j] = p0;
            pr[j + 2] = p1;
        }
        // P^T (keys x heads) to the B fragment, as bf16 and what that leaves
        uint32_t pb[2][2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const uint32_t w = pack_bf16(pr[2 * y], pr[2 * y + 1]);
            pb[0][y] = movmatrix_t(w);
            pb[1][y] = movmatrix_t(pack_bf16(pr[2 * y] - bf16_lo(w), pr[2 * y + 1] - bf16_hi(w)));
        }
        // ---- O^T [128][8 heads] += V^T P^T
        const uint32_t sv = st + kTileBytes + 2 * c * 128;
        const uint32_t x0 = (rr ^ (2 * c)) << 4, x1 = (rr ^ (2 * c + 1)) << 4;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            uint4 v0 = lds16(sv + kBoxBytes * m + x0), v1 = lds16(sv + kBoxBytes * m + 128 + x1);
            uint4 v2 = lds16(sv + kBoxBytes * m + 1024 + x0), v3 = lds16(sv + kBoxBytes * m + 1152 + x1);
            if (lim < kBlockTokens) {
                // a weight of 0 does not undo a NaN in a slot that the query does not see
                const uint4 z = make_uint4(0, 0, 0, 0);
                if (2 * c >= lim) v0 = z;
                if (2 * c + 1 >= lim) v1 = z;
                if (2 * c + 8 >= lim) v2 = z;
                if (2 * c + 9 >= lim) v3 = z;
            }
            const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
            const uint32_t w2[4] = {v2.x, v2.y, v2.z, v2.w}, w3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t a0 = __byte_perm(w0[x], w1[x], 0x5410), a1 = __byte_perm(w0[x], w1[x], 0x7632);
                const uint32_t a2 = __byte_perm(w2[x], w3[x], 0x5410), a3 = __byte_perm(w2[x], w3[x], 0x7632);
                mma_bf16(oacc[4 * m + x], a0, a1, a2, a3, pb[0][0], pb[0][1]);
                mma_bf16(oacc[4 * m + x], a0, a1, a2, a3, pb[1][0], pb[1][1]);
            }
        }
    }
    end_request();
}

// ---------------------------------------------------------------------------- joining the partials
constexpr int kMassWords = 32;   // words per CTA of the mass part

// Maximum and sum of a head's partials: M = max m_i, L = sum l_i 2^(m_i - M), and the largest output reference; the
// whole warp, partials over its lanes.
__device__ __forceinline__ void join_head(const float4 *ml, int nw, int G, int lane, float &M, float &L, float &MO) {
    M = MO = -INFINITY;
    L = 0.f;
    // eight loads in flight per lane
    for (int i0 = 0; i0 < nw; i0 += 256) {
        float4 v[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int i = i0 + 32 * x + lane;
            v[x] = i < nw ? ml[static_cast<size_t>(i) * G] : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
        }
        float top = M;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            top = fmaxf(top, v[x].x);
            MO = fmaxf(MO, v[x].z);
        }
        const float mu = top == -INFINITY ? 0.f : top;
        L *= fast_exp2(M - mu);
        M = top;
#pragma unroll
        for (int x = 0; x < 8; ++x) L += v[x].y * fast_exp2(v[x].x - mu);
    }
    float all = M;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
        all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, x));
        MO = fmaxf(MO, __shfl_xor_sync(0xffffffffu, MO, x));
    }
    L *= fast_exp2(M - (all == -INFINITY ? 0.f : all));
    M = all;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
}

// Grid (request, y).  y < rows / rows per CTA: a row of the output from the request's partials, four head
// dims per lane; one row per warp, or (JOIN warps, where a request has many partials) one per CTA with every
// JOIN-th partial per warp.  y behind them: the word accumulators, mass[w] += sum_h 2^(lse[w][h] - z_h), z_h = M_h + log2 L_h.
// One warp per word.
template <int JOIN>
__global__ void __launch_bounds__(JOIN > 1 ? 32 * JOIN : 128) lane_combine_kernel(const __grid_constant__ LaneParams p, int min_words) {
    constexpr int kJoinWarps = JOIN > 1 ? JOIN : 4;
    pdl_wait();
    const AttnParams &a = p.a;
    const unsigned B = a.num_req, G = p.rows, hq = p.rows * a.hkv;   // rows per KV head, and of all
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned r = blockIdx.x, out_ctas = JOIN > 1 ? hq : (hq + 3) / 4;
    const int base = a.table_indptr[0];
    const unsigned total = a.table_indptr[B] - base;
    const unsigned beg = a.table_indptr[r] - base;
    const int n = min(a.table_indptr[r + 1] - base - static_cast<int>(beg), a.max_words);
    const unsigned per = max(static_cast<unsigned>(min_words), (total + p.pieces - 1) / static_cast<unsigned>(p.pieces));
    const unsigned w0 = n > 0 ? beg / per : 0;
    const int nw = n > 0 ? static_cast<int>((beg + n - 1) / per - w0 + 1) : 0;
    if (blockIdx.y < out_ctas) {
        const unsigned h = JOIN > 1 ? blockIdx.y : blockIdx.y * 4 + warp;
        if (h >= hq) return;
        const unsigned kvh = h / G, g = h - kvh * G;
        size_t row = static_cast<size_t>(r) * hq + h;
        if (a.cu_q) {
            // a request's few tokens: row g is (token, head of the group)
            const int q0 = a.cu_q[r], tokens = min(a.cu_q[r + 1] - q0, a.max_q), tok = g / a.group;
            if (tok >= tokens) return;
            row = static_cast<size_t>(q0 + tok) * a.hq + kvh * a.group + g - tok * a.group;
        }
        const size_t s0 = static_cast<size_t>(kvh) * (p.pieces + B) + w0 + r;
        const float4 *ml = p.ws_ml + s0 * G + g;
        float M, L, MO;
        join_head(ml, nw, G, lane, M, L, MO);
        const float mu = M == -INFINITY ? 0.f : M, mou = MO == -INFINITY ? 0.f : MO;
        const float4 *acc = reinterpret_cast<const float4 *>(a.ws_acc + (s0 * G + g) * kHeadDim) + lane;
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll (JOIN > 1 ? 8 : 2)
        for (int i = JOIN > 1 ? warp : 0; i < nw; i += JOIN) {
            const float w = fast_exp2(ml[static_cast<size_t>(i) * G].z - mou);
            if (w != 0.f) {   // (a partial without keys has no acc)
                const float4 v = acc[static_cast<size_t>(i) * G * (kHeadDim / 4)];
                A.x += w * v.x;
                A.y += w * v.y;
                A.z += w * v.z;
                A.w += w * v.w;
            }
        }
        if constexpr (JOIN > 1) {
            __shared__ float4 part[JOIN][32];
            part[warp][lane] = A;
            __syncthreads();
            if (warp != 0) return;
#pragma unroll
            for (int x = 1; x < JOIN; ++x) {
                const float4 v = part[x][lane];
                A.x += v.x;
                A.y += v.y;
                A.z += v.z;
                A.w += v.w;
            }
        }
        // A is relative to 2^MO, L to 2^M; 2^(MO - M) may pass the range of a float where the output does not: as a square
        const float f = fast_exp2(0.5f * fminf(fmaxf(mou - mu, -250.f), 250.f)), inv = L > 0.f || L != L ? 1.f / L : 0.f;
        auto value = [&](float x) { return x * inv * f * f; };
        reinterpret_cast<uint2 *>(a.out + row * kHeadDim)[lane] =
            make_uint2(pack_bf16(value(A.x), value(A.y)), pack_bf16(value(A.z), value(A.w)));
    } else {
        extern __shared__ float z[];   // [Hq]
        const int c0 = (blockIdx.y - out_ctas) * kMassWords;
        if (c0 >= n) return;
        for (unsigned h = JOIN > 1 ? warp : threadIdx.x; h < hq; h += JOIN > 1 ? kJoinWarps : 128) {
            const unsigned kvh = h / G, g = h - kvh * G;
            const float4 *ml = p.ws_ml + (static_cast<size_t>(kvh) * (p.pieces + B) + w0 + r) * G + g;
            float M = -INFINITY, L = 0.f, MO;
            if (JOIN > 1) {
                join_head(ml, nw, G, lane, M, L, MO);
            } else {
                // a few partials: one thread per head
                for (int i = 0; i < nw; ++i) M = fmaxf(M, ml[static_cast<size_t>(i) * G].x);
                for (int i = 0; i < nw; ++i) {
                    const float4 v = ml[static_cast<size_t>(i) * G];
                    L += v.y * fast_exp2(v.x - (M == -INFINITY ? 0.f : M));
                }
            }
            if (JOIN == 1 || lane == 0) z[h] = L > 0.f || L != L ? (M == -INFINITY ? 0.f : M) + fast_log2(L) : INFINITY;
        }
        __syncthreads();
#pragma unroll 4
        for (int i = c0 + warp; i < min(n, c0 + kMassWords); i += kJoinWarps) {
            const float *lse = p.ws_lse + (static_cast<size_t>(r) * a.max_words + i) * hq;
            float s = 0.f;
            for (unsigned h = lane; h < hq; h += 32) s += fast_exp2(lse[h] - z[h]);
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
            if (lane == 0) p.mass[base + beg + i] += s;
        }
    }
}

}  // namespace

LanePlan decode_mass_plan(int num_req, int hkv, int max_words, int group, int sms) {
    // one wave of resident warps, but at least kMinWords words each
    const int64_t words = static_cast<int64_t>(num_req) * max_words;
    const int64_t most = (words + kMinWords - 1) / kMinWords;
    const int64_t resident = static_cast<int64_t>(sms > 0 ? sms : 1) * kOcc * kWarps / (hkv * head_groups(group));
    LanePlan pl;
    pl.pieces = static_cast<int>(most < resident ? most : resident);
    if (pl.pieces < 1) pl.pieces = 1;
    pl.slots = static_cast<int64_t>(hkv) * (pl.pieces + num_req);
    return pl;
}

cudaError_t launch_lane_combine(const LaneParams &p, int min_words, cudaStream_t s) {
    const int rows = p.rows * p.a.hkv;
    const int chunks = p.mass ? (p.a.max_words + kMassWords - 1) / kMassWords : 0;
    const size_t smem = p.mass ? p.a.hq * sizeof(float) : 0;
    // a request has about pieces / requests partials
    if (p.pieces > 8 * p.a.num_req)
        return launch_dependent(lane_combine_kernel<8>, dim3(p.a.num_req, rows + chunks), 256, smem, s, p, min_words);
    return launch_dependent(lane_combine_kernel<1>, dim3(p.a.num_req, (rows + 3) / 4 + chunks), 128, smem, s, p, min_words);
}

cudaError_t launch_decode_mass(const CUtensorMap &tk, const CUtensorMap &tv, const LaneParams &p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(decode_lane_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const int ctas = (p.pieces * p.a.hkv * head_groups(p.a.group) + kWarps - 1) / kWarps;
    decode_lane_kernel<<<ctas, kWarps * 32, kSmem, s>>>(tk, tv, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_lane_combine(p, kMinWords, s);
}

}  // namespace lazy

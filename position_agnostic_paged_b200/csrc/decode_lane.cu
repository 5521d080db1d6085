// decode_lane.cu -- decode attention that also accumulates each table word's attention weight,
// and decode attention over the 8-bit pool.
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
// Data path.  Every lane copies with cp.async exactly the 16-byte pieces it will feed to the
// tensor cores itself, so a warp's stages are lane-private FIFOs: no barriers, no bank
// conflicts, no producer warp.  The K index order of an MMA is free as long as both operands use
// the same one, and so is the order of output rows; both are chosen to make a lane's share
// contiguous:
//   K (rows = keys as the A operand): lane (rr, c) takes 16-byte pieces c, c + 4, ... of key rows
//     rr and rr + 8, a full 32-byte sector per two lanes;
//   V^T (rows = head dims as the A operand): lane (rr, c) takes piece(s) rr of key rows 2c, 2c+1,
//     2c+8, 2c+9 and pairs keys with byte permutes.
// e4m3 codes become f16 (exact); the query is scaled by a power of two to [1, 2) and rounded to f16
// (2^-12 of its largest element); weights are f16 against a running reference that includes the
// block's V scale, so they neither overflow nor lose the small blocks.  Scores, sums, maxima and
// outputs are fp32.  With block mass the query is split into two f16 (8-bit pool) or three bf16
// parts (bf16 pool), which keeps the fp32 weights to a few 2^-22.
#include <cuda_fp16.h>

#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "q8.cuh"

namespace lazy {

namespace {

constexpr int kMinWords = 2;   // least words per warp

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool Q8>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    if (Q8)
        mma_f16(d, a0, a1, a2, a3, b0, b1);
    else
        mma_bf16(d, a0, a1, a2, a3, b0, b1);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
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

// NT: groups of 8 query heads per KV head.  QP: parts the query is split into.
template <bool Q8, int NT, bool MASS>
struct Cfg {
    static constexpr int QP = Q8 ? (MASS ? 2 : 1) : 3;
    static constexpr bool kRegQ = NT == 1;                     // query fragments in registers, else in shared memory
    static constexpr int kPieces = Q8 ? 4 : 8;                 // 16-byte pieces of K (and of V) per lane and word
    static constexpr int kStageBytes = 2 * kPieces * 512;
    static constexpr int kQBytes = kRegQ ? 0 : NT * QP * 8 * 32 * 8;      // query fragments per warp
    static constexpr int kLeast = 2 * kStageBytes + kQBytes + 512;        // shared memory per warp, two stages
    // CTAs per SM by registers (4 warps each); where the query fragments leave no room for two stages of so
    // many warps (bf16 with block mass, G > 8): one CTA of as many warps as fit
    static constexpr int kOcc0 = NT == 4 ? 2 : (NT == 2 || !Q8) ? 3 : 4;
    static constexpr bool kFits = kOcc0 * (4 * kLeast + 1024) <= 227 * 1024;
    static constexpr int kOcc = kFits ? kOcc0 : 1;
    static constexpr int kWarps = kFits ? 4 : 226 * 1024 / kLeast;
    static constexpr int kStages0 = ((227 * 1024 / kOcc - 1024) / kWarps - kQBytes - 512) / kStageBytes;
    static constexpr int kStages = kStages0 > 8 ? 8 : kStages0;
    static constexpr int kWarpBytes = kStages * kStageBytes + kQBytes + 512;
    static constexpr int kSmem = kWarps * kWarpBytes;
    static_assert(kStages >= 2 && kWarps <= 8, "pipeline depth");
};

// Head dims of the query fragment: register pair x of k-step s holds dims qdim(s) + {0, 1} and + {2, 3}
// (s < 4; k-step s + 4 the dims 64 above: the rotation pairs).
template <bool Q8>
__device__ __forceinline__ int qdim(int s, int c) {
    return Q8 ? 16 * c + 4 * s : 32 * (s >> 1) + 8 * c + 4 * (s & 1);
}
// First head dim of output tile t's row pair (rows rr and rr + 8 hold odim and odim + 1).
template <bool Q8>
__device__ __forceinline__ int odim(int t, int rr) {
    return Q8 ? 16 * rr + 2 * t : 64 * (t >> 2) + 8 * rr + 2 * (t & 3);
}

template <bool Q8, int NT, bool MASS>
__global__ void __launch_bounds__((Cfg<Q8, NT, MASS>::kWarps * 32), (Cfg<Q8, NT, MASS>::kOcc)) decode_lane_kernel(const LaneParams p) {
    using C = Cfg<Q8, NT, MASS>;
    constexpr int QP = C::QP, S = C::kStages, kWarps = C::kWarps;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = lane & 3, rr = lane >> 2;
    const AttnParams &a = p.a;
    const int G = a.group, hkv = a.hkv, B = a.num_req;
    const int gw = blockIdx.x * kWarps + warp;
    const int kvh = gw % hkv, wi = gw / hkv;
    if (wi >= p.warps_per_head) return;
    const int base = a.table_indptr[0];
    const int total = a.table_indptr[B] - base;
    if (total <= 0) return;
    const int per = words_per_warp(total, p.warps_per_head);
    if (wi > (total - 1) / per) return;
    const int lo = wi * per, cnt = min(total - lo, per);

    uint8_t *ws = smem_raw + warp * C::kWarpBytes;
    const uint32_t fifo = smem_u32(ws) + lane * 16;
    uint2 *qs = reinterpret_cast<uint2 *>(ws + S * C::kStageBytes);              // [NT][QP][8][32]
    float2 *cs = reinterpret_cast<float2 *>(ws + S * C::kStageBytes + C::kQBytes);   // [64]

    // ---- the words of this warp, 32 at a time, one per lane
    uint32_t w_cur = 0, m_cur = 0, w_nxt = 0, m_nxt = 0;
    float ks_cur = 0.f, lv_cur = 0.f, ks_nxt = 0.f, lv_nxt = 0.f;
    auto fetch = [&](int k0, uint32_t &w, uint32_t &m, float &ks, float &lv) {
        w = 0u;
        m = 0u;
        ks = 0.f;
        lv = 0.f;
        if (k0 + lane < cnt) {
            w = a.table[base + lo + k0 + lane];
            const uint32_t b = word_block(w);
            if (b < static_cast<uint32_t>(a.num_blocks)) {
                m = a.blk_meta[b];
                if (Q8) {
                    ks = p.k_scale[static_cast<size_t>(b) * hkv + kvh];
                    lv = fast_log2(p.v_scale[static_cast<size_t>(b) * hkv + kvh]);
                }
            } else {
                set_status(a.d_status, LAZY_DSTATUS_BAD_BLOCK);
            }
        }
    };
    fetch(0, w_cur, m_cur, ks_cur, lv_cur);
    fetch(32, w_nxt, m_nxt, ks_nxt, lv_nxt);

    const size_t k_lane = Q8 ? rr * 128 + c * 16 : rr * 256 + c * 16;
    const size_t v_lane = Q8 ? c * 256 + rr * 16 : c * 512 + rr * 16;
    constexpr size_t kTile = Q8 ? 2048 : 4096;
    // copies of word k (of this warp) into stage k % S; `kb` is the batch that w_cur holds
    auto issue = [&](int k, int kb) {
        if (k < cnt) {
            const bool nx = (k >> 5) != kb;
            const uint32_t w = __shfl_sync(0xffffffffu, nx ? w_nxt : w_cur, k & 31);
            const uint32_t m = __shfl_sync(0xffffffffu, nx ? m_nxt : m_cur, k & 31);
            if (meta_valid(m) > 0) {
                const size_t tile = (static_cast<size_t>(word_block(w)) * hkv + kvh) * kTile;
                const uint8_t *ks = p.k + tile + k_lane, *vs = p.v + tile + v_lane;
                const uint32_t d = fifo + (k % S) * C::kStageBytes;
                if (Q8) {
                    cp16(d, ks);
                    cp16(d + 512, ks + 64);
                    cp16(d + 1024, ks + 1024);
                    cp16(d + 1536, ks + 1088);
                    cp16(d + 2048, vs);
                    cp16(d + 2560, vs + 128);
                    cp16(d + 3072, vs + 1024);
                    cp16(d + 3584, vs + 1152);
                } else {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        cp16(d + 512 * x, ks + 64 * x);
                        cp16(d + 512 * (4 + x), ks + 2048 + 64 * x);
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int row = (x & 1) * 256 + (x >> 1) * 2048;   // key rows 2c, 2c+1, 2c+8, 2c+9
                        cp16(d + 4096 + 512 * x, vs + row);
                        cp16(d + 4096 + 512 * (4 + x), vs + row + 128);
                    }
                }
            }
        }
        cp_commit();
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) issue(k, 0);

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
    const double th0 = a.rope.theta[lane], th1 = a.rope.theta[lane + 32];

    int r_beg = a.table_indptr[r] - base, r_end = a.table_indptr[r + 1] - base;
    int qpos = 0, cur_off = -1;
    uint32_t qraw[C::kRegQ ? 8 : 1][2];
    uint32_t qb[C::kRegQ ? QP : 1][C::kRegQ ? 8 : 1][2];
    float qn[NT];            // 2^-e of this lane's fragment head (8 n + rr)
    float hm[NT][2];         // score factor of heads 8 n + 2c, + 1: softmax scale * log2(e) * 2^e
    float sl[NT][2];         // ALiBi slopes of those heads (log2 units)
    float m_run[NT][2], l_run[NT][2], mo[NT][2];
    float oacc[NT][8][4];

    auto begin_request = [&]() {
        qpos = a.q_pos[r];
        cur_off = -1;
        if (lo <= r_beg && r_end - r_beg > a.max_words && kvh == 0 && lane == 0)
            set_status(a.d_status, LAZY_DSTATUS_BAD_TABLE);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int g = 8 * n + rr;
            const uint32_t *q = reinterpret_cast<const uint32_t *>(
                a.q_raw + (static_cast<size_t>(r) * a.hq + kvh * G + min(g, G - 1)) * kHeadDim);
            float am = 0.f;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int d = qdim<Q8>(s & 3, c) + 64 * (s >> 2);
                uint32_t w0 = 0u, w1 = 0u;
                if (g < G) {
                    w0 = q[d >> 1];
                    w1 = q[(d >> 1) + 1];
                }
                if (C::kRegQ) {
                    qraw[s][0] = w0;
                    qraw[s][1] = w1;
                }
                am = fmaxf(am, fmaxf(fmaxf(fabsf(bf16_lo(w0)), fabsf(bf16_hi(w0))),
                                     fmaxf(fabsf(bf16_lo(w1)), fabsf(bf16_hi(w1)))));
            }
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
            // q 2^-e in [1, 2); e = 0 for an all-zero or non-finite head
            int e = static_cast<int>(__float_as_uint(am) >> 23) - 127;
            e = (am == 0.f || e == 128) ? 0 : max(-126, min(126, e));
            qn[n] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            const float q2 = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * a.scale_log2;
            hm[n][0] = __shfl_sync(0xffffffffu, q2, 8 * c);
            hm[n][1] = __shfl_sync(0xffffffffu, q2, 8 * c + 4);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int h = 8 * n + 2 * c + j;
                sl[n][j] = (a.alibi && h < G) ? a.alibi_log2[kvh * G + h] : 0.f;
                m_run[n][j] = mo[n][j] = -INFINITY;
                l_run[n][j] = 0.f;
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) oacc[n][t][0] = oacc[n][t][1] = oacc[n][t][2] = oacc[n][t][3] = 0.f;
        }
    };
    // the query turned by (qpos - off), as fragments: angles once per warp (two per lane), shared
    auto rotate = [&](int off) {
        cur_off = off;
        const int delta = a.alibi ? 0 : qpos - off;
        float2 z0, z1;
        rope_cos_sin(delta, th0, z0.x, z0.y);
        rope_cos_sin(delta, th1, z1.x, z1.y);
        __syncwarp();
        cs[lane] = z0;
        cs[lane + 32] = z1;
        __syncwarp();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int g = 8 * n + rr;
            const uint32_t *q = reinterpret_cast<const uint32_t *>(
                a.q_raw + (static_cast<size_t>(r) * a.hq + kvh * G + min(g, G - 1)) * kHeadDim);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int d = qdim<Q8>(s, c);
                float x[8];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t wa, wb;
                    if (C::kRegQ) {
                        wa = qraw[s][y];
                        wb = qraw[C::kRegQ ? s + 4 : 0][y];
                    } else {
                        wa = g < G ? q[(d >> 1) + y] : 0u;
                        wb = g < G ? q[(d >> 1) + y + 32] : 0u;
                    }
                    const float4 z = *reinterpret_cast<const float4 *>(&cs[d + 2 * y]);   // (cos, sin) of two pairs
                    const float a0 = bf16_lo(wa) * qn[n], a1 = bf16_hi(wa) * qn[n];
                    const float b0 = bf16_lo(wb) * qn[n], b1 = bf16_hi(wb) * qn[n];
                    x[2 * y] = a0 * z.x - b0 * z.y;
                    x[2 * y + 1] = a1 * z.z - b1 * z.w;
                    x[4 + 2 * y] = b0 * z.x + a0 * z.y;
                    x[4 + 2 * y + 1] = b1 * z.z + a1 * z.w;
                }
#pragma unroll
                for (int part = 0; part < QP; ++part) {
                    uint32_t w[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        if (Q8) {
                            w[y] = pack_f16(x[2 * y], x[2 * y + 1]);
                            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[y]));
                            x[2 * y] -= f.x;
                            x[2 * y + 1] -= f.y;
                        } else {
                            w[y] = pack_bf16(x[2 * y], x[2 * y + 1]);
                            x[2 * y] -= bf16_lo(w[y]);
                            x[2 * y + 1] -= bf16_hi(w[y]);
                        }
                    }
                    if (C::kRegQ) {
                        qb[part][s][0] = w[0];
                        qb[part][s][1] = w[1];
                        qb[part][C::kRegQ ? s + 4 : 0][0] = w[2];
                        qb[part][C::kRegQ ? s + 4 : 0][1] = w[3];
                    } else {
                        qs[((n * QP + part) * 8 + s) * 32 + lane] = make_uint2(w[0], w[1]);
                        qs[((n * QP + part) * 8 + s + 4) * 32 + lane] = make_uint2(w[2], w[3]);
                    }
                }
            }
        }
    };
    auto end_request = [&]() {
        const size_t slot = static_cast<size_t>(kvh) * (p.warps_per_head + B) + wi + r;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float l = l_run[n][j];
                if (!MASS) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
                }
                const int g = 8 * n + 2 * c + j;
                if (g < G) {
                    float *o = a.ws_acc + (slot * G + g) * kHeadDim;
#pragma unroll
                    for (int t = 0; t < 8; t += 2) {
                        // tiles t and t + 1: four consecutive head dims
                        *reinterpret_cast<float4 *>(o + odim<Q8>(t, rr)) =
                            make_float4(oacc[n][t][j], oacc[n][t][j + 2], oacc[n][t + 1][j], oacc[n][t + 1][j + 2]);
                    }
                    if (rr == 0) p.ws_ml[slot * G + g] = make_float4(m_run[n][j], l, Q8 ? mo[n][j] : m_run[n][j], 0.f);
                }
            }
    };
    begin_request();

    for (int k = 0; k < cnt; ++k) {
        if (k > 0 && (k & 31) == 0) {
            w_cur = w_nxt;
            m_cur = m_nxt;
            ks_cur = ks_nxt;
            lv_cur = lv_nxt;
            fetch(k + 32, w_nxt, m_nxt, ks_nxt, lv_nxt);
        }
        issue(k + S - 1, k >> 5);
        cp_wait<S - 1>();
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
        const float ksc = Q8 ? __shfl_sync(0xffffffffu, ks_cur, k & 31) : 1.f;
        const float lv = Q8 ? __shfl_sync(0xffffffffu, lv_cur, k & 31) : 0.f;
        const int i_req = lo + k - r_beg;                       // index of the word in its request
        const int off = word_offset(w);
        const int pos0 = off + meta_j0(meta);
        // keys of this word that the query sees: slots 0 .. lim - 1
        const int lim = i_req < a.max_words ? min(meta_valid(meta), qpos - pos0 + 1) : 0;
        float *lse = MASS ? p.ws_lse + (static_cast<size_t>(r) * a.max_words + i_req) * a.hq + kvh * G : nullptr;
        if (lim <= 0) {
            if (MASS && i_req < a.max_words && lane < G) lse[lane] = -INFINITY;
            continue;
        }
        if (cur_off < 0 || (off != cur_off && !a.alibi)) rotate(off);

        const uint32_t st = fifo + (k % S) * C::kStageBytes;
        // ---- S^T [16 keys][8 heads] = K q^T
        float sa[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) sa[n][0] = sa[n][1] = sa[n][2] = sa[n][3] = 0.f;
#pragma unroll
        for (int m = 0; m < C::kPieces / 2; ++m) {
            // piece m of key rows rr and rr + 8: two (bf16) or four (e4m3) k-steps
            const uint4 ra = lds16(st + 512 * m), rb = lds16(st + 512 * (C::kPieces / 2 + m));
            const uint32_t aw[4] = {ra.x, ra.y, ra.z, ra.w}, bw[4] = {rb.x, rb.y, rb.z, rb.w};
#pragma unroll
            for (int u = 0; u < (Q8 ? 4 : 2); ++u) {
                const int s = (Q8 ? 4 : 2) * m + u;
                uint32_t a0, a1, a2, a3;
                if (Q8) {
                    codes_to_f16(aw[u], a0, a2);
                    codes_to_f16(bw[u], a1, a3);
                } else {
                    a0 = aw[2 * (u & 1)];
                    a2 = aw[2 * (u & 1) + 1];
                    a1 = bw[2 * (u & 1)];
                    a3 = bw[2 * (u & 1) + 1];
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int part = 0; part < QP; ++part) {
                        uint2 b;
                        if (C::kRegQ)
                            b = make_uint2(qb[part][C::kRegQ ? s : 0][0], qb[part][C::kRegQ ? s : 0][1]);
                        else
                            b = qs[((n * QP + part) * 8 + s) * 32 + lane];
                        mma16<Q8>(sa[n], a0, a1, a2, a3, b.x, b.y);
                    }
            }
        }
        // ---- softmax over the word's keys (rr and rr + 8 in this lane)
        const bool vis0 = rr < lim, vis1 = rr + 8 < lim;
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float bm[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float f = hm[n][j] * ksc;
                float s0 = sa[n][j] * f, s1 = sa[n][j + 2] * f;
                if (a.alibi) {
                    const float d0 = static_cast<float>(pos0 + rr - qpos);
                    s0 = fmaf(sl[n][j], d0, s0);
                    s1 = fmaf(sl[n][j], d0 + 8.f, s1);
                }
                sa[n][j] = vis0 ? s0 : -INFINITY;
                sa[n][j + 2] = vis1 ? s1 : -INFINITY;
                bm[j] = fmaxf(sa[n][j], sa[n][j + 2]);
            }
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                bm[0] = fmaxf(bm[0], __shfl_xor_sync(0xffffffffu, bm[0], x));
                bm[1] = fmaxf(bm[1], __shfl_xor_sync(0xffffffffu, bm[1], x));
            }
            float pr[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float mn = fmaxf(m_run[n][j], bm[j]);
                const float mu = mn == -INFINITY ? 0.f : mn;
                if (mn != m_run[n][j]) {
                    const float sc = fast_exp2(m_run[n][j] - mu);
                    l_run[n][j] *= sc;
                    if (!Q8) {
#pragma unroll
                        for (int t = 0; t < 8; ++t) {
                            oacc[n][t][j] *= sc;
                            oacc[n][t][j + 2] *= sc;
                        }
                    }
                    m_run[n][j] = mn;
                }
                float p0 = fast_exp2(sa[n][j] - mu), p1 = fast_exp2(sa[n][j + 2] - mu);
                float ps = p0 + p1;
                if (MASS) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) ps += __shfl_xor_sync(0xffffffffu, ps, x);
                    const int g = 8 * n + 2 * c + j;
                    if (rr == 0 && g < G) lse[g] = mu + fast_log2(ps);
                }
                l_run[n][j] += ps;
                if (Q8) {
                    // weights for the V product, against the running maximum of score + log2(V scale)
                    const float mon = fmaxf(mo[n][j], bm[j] + lv);
                    const float mou = mon == -INFINITY ? 0.f : mon;
                    if (mon != mo[n][j]) {
                        const float sc = fast_exp2(mo[n][j] - mou);
#pragma unroll
                        for (int t = 0; t < 8; ++t) {
                            oacc[n][t][j] *= sc;
                            oacc[n][t][j + 2] *= sc;
                        }
                        mo[n][j] = mon;
                    }
                    const float f = fast_exp2(fminf(mu + lv - mou, 126.f));
                    p0 *= f;
                    p1 *= f;
                }
                pr[j] = p0;
                pr[j + 2] = p1;
            }
            // P^T (keys x heads) to the B fragment
            pb[n][0] = movmatrix_t(Q8 ? pack_f16(pr[0], pr[1]) : pack_bf16(pr[0], pr[1]));
            pb[n][1] = movmatrix_t(Q8 ? pack_f16(pr[2], pr[3]) : pack_bf16(pr[2], pr[3]));
        }
        // ---- O^T [128][8 heads] += V^T P^T
        const uint32_t sv = st + C::kStageBytes / 2;
#pragma unroll
        for (int m = 0; m < C::kPieces / 4; ++m) {
            uint4 v0 = lds16(sv + 2048 * m), v1 = lds16(sv + 2048 * m + 512);
            uint4 v2 = lds16(sv + 2048 * m + 1024), v3 = lds16(sv + 2048 * m + 1536);
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
                if (Q8) {
                    uint32_t a0, a1, a2, a3;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t sel = u ? 0x7362 : 0x5140;   // codes of keys 2c, 2c+1 side by side, two dims
                        codes_to_f16(__byte_perm(w0[x], w1[x], sel), a0, a1);
                        codes_to_f16(__byte_perm(w2[x], w3[x], sel), a2, a3);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16<Q8>(oacc[n][2 * x + u], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                    }
                } else {
                    const uint32_t a0 = __byte_perm(w0[x], w1[x], 0x5410), a1 = __byte_perm(w0[x], w1[x], 0x7632);
                    const uint32_t a2 = __byte_perm(w2[x], w3[x], 0x5410), a3 = __byte_perm(w2[x], w3[x], 0x7632);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16<Q8>(oacc[n][4 * m + x], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                }
            }
        }
    }
    end_request();
    cp_wait<0>();
}

// ---------------------------------------------------------------------------- joining the partials
constexpr int kMassWords = 32;   // words per CTA of the mass part

// CTAs 0 .. num_req * Hq - 1: out[r][h] from the request's partials.  The CTAs behind them: the
// word accumulators, mass[w] += sum_h 2^(lse[w][h] - z_h), z_h = M_h + log2 L_h, one warp per word.
__global__ void __launch_bounds__(128) lane_combine_kernel(const LaneParams p) {
    const AttnParams &a = p.a;
    const int B = a.num_req, G = a.group, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool for_out = static_cast<int>(blockIdx.x) < B * a.hq;
    const int chunks = (a.max_words + kMassWords - 1) / kMassWords;
    const int mi = blockIdx.x - B * a.hq;
    const int r = for_out ? blockIdx.x / a.hq : mi / chunks;
    const int base = a.table_indptr[0];
    const int total = a.table_indptr[B] - base;
    const int beg = a.table_indptr[r] - base;
    const int n = min(a.table_indptr[r + 1] - base - beg, a.max_words);
    const int per = words_per_warp(total, p.warps_per_head);
    const int w0 = n > 0 ? beg / per : 0, nw = n > 0 ? (beg + n - 1) / per - w0 + 1 : 0;
    if (for_out) {
        __shared__ float red[4][2], wgt[128], lsum[4];
        const int h = blockIdx.x % a.hq, kvh = h / G, g = h % G;
        const size_t s0 = static_cast<size_t>(kvh) * (p.warps_per_head + B) + w0 + r;
        float M = -INFINITY, MO = -INFINITY;
        for (int i = tid; i < nw; i += 128) {
            const float4 ml = p.ws_ml[(s0 + i) * G + g];
            M = fmaxf(M, ml.x);
            MO = fmaxf(MO, ml.z);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) {
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
            MO = fmaxf(MO, __shfl_xor_sync(0xffffffffu, MO, x));
        }
        if (lane == 0) {
            red[warp][0] = M;
            red[warp][1] = MO;
        }
        __syncthreads();
        M = fmaxf(fmaxf(red[0][0], red[1][0]), fmaxf(red[2][0], red[3][0]));
        MO = fmaxf(fmaxf(red[0][1], red[1][1]), fmaxf(red[2][1], red[3][1]));
        const float mu = M == -INFINITY ? 0.f : M, mou = MO == -INFINITY ? 0.f : MO;
        float L = 0.f, A = 0.f;
        for (int i0 = 0; i0 < nw; i0 += 128) {
            if (i0 > 0) __syncthreads();
            if (i0 + tid < nw) {
                const float4 ml = p.ws_ml[(s0 + i0 + tid) * G + g];
                L += ml.y * fast_exp2(ml.x - mu);
                wgt[tid] = fast_exp2(ml.z - mou);
            }
            __syncthreads();
            const int m = min(128, nw - i0);
            const float *acc = a.ws_acc + ((s0 + i0) * G + g) * kHeadDim + tid;
#pragma unroll 8
            for (int i = 0; i < m; ++i) A += wgt[i] * acc[static_cast<size_t>(i) * G * kHeadDim];
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
        if (lane == 0) lsum[warp] = L;
        __syncthreads();
        L = (lsum[0] + lsum[1]) + (lsum[2] + lsum[3]);
        // A is relative to 2^MO, L to 2^M (fminf only keeps an overflow of the factor from making 0 * inf)
        const float o = L > 0.f || L != L ? A / L * fast_exp2(fminf(mou - mu, 126.f)) : 0.f;
        const __nv_bfloat16 ob = __float2bfloat16_rn(o);
        a.out[(static_cast<size_t>(r) * a.hq + h) * kHeadDim + tid] = *reinterpret_cast<const uint16_t *>(&ob);
    } else {
        extern __shared__ float z[];   // [Hq]
        const int c0 = (mi % chunks) * kMassWords;
        if (c0 >= n) return;
        for (int h = tid; h < a.hq; h += 128) {
            const int kvh = h / G, g = h % G;
            const float4 *ml = p.ws_ml + (static_cast<size_t>(kvh) * (p.warps_per_head + B) + w0 + r) * G + g;
            float M = -INFINITY, L = 0.f;
            for (int i = 0; i < nw; ++i) M = fmaxf(M, ml[static_cast<size_t>(i) * G].x);
            const float mu = M == -INFINITY ? 0.f : M;
            for (int i = 0; i < nw; ++i) {
                const float4 v = ml[static_cast<size_t>(i) * G];
                L += v.y * fast_exp2(v.x - mu);
            }
            z[h] = L > 0.f || L != L ? mu + fast_log2(L) : INFINITY;
        }
        __syncthreads();
        for (int i = c0 + warp; i < min(n, c0 + kMassWords); i += 4) {
            const float *lse = p.ws_lse + (static_cast<size_t>(r) * a.max_words + i) * a.hq;
            float s = 0.f;
            for (int h = lane; h < a.hq; h += 32) s += fast_exp2(lse[h] - z[h]);
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
            if (lane == 0) p.mass[base + beg + i] += s;
        }
    }
}

template <bool Q8, int NT, bool MASS>
cudaError_t launch_t(const LaneParams &p, cudaStream_t s) {
    using C = Cfg<Q8, NT, MASS>;
    auto kern = decode_lane_kernel<Q8, NT, MASS>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int ctas = (p.warps_per_head * p.a.hkv + C::kWarps - 1) / C::kWarps;
    kern<<<ctas, C::kWarps * 32, C::kSmem, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int chunks = (p.a.max_words + kMassWords - 1) / kMassWords;
    lane_combine_kernel<<<p.a.num_req * (p.a.hq + (p.mass ? chunks : 0)), 128, p.mass ? p.a.hq * sizeof(float) : 0, s>>>(p);
    return cudaGetLastError();
}

template <bool Q8, bool MASS>
cudaError_t launch_g(const LaneParams &p, cudaStream_t s) {
    if (p.a.group <= 8) return launch_t<Q8, 1, MASS>(p, s);
    return p.a.group <= 16 ? launch_t<Q8, 2, MASS>(p, s) : launch_t<Q8, 4, MASS>(p, s);
}

}  // namespace

template <bool Q8, bool MASS>
static int resident_warps(int group) {
    if (group <= 8) return Cfg<Q8, 1, MASS>::kOcc * Cfg<Q8, 1, MASS>::kWarps;
    return group <= 16 ? Cfg<Q8, 2, MASS>::kOcc * Cfg<Q8, 2, MASS>::kWarps : Cfg<Q8, 4, MASS>::kOcc * Cfg<Q8, 4, MASS>::kWarps;
}

LanePlan lane_plan(int num_req, int hkv, int max_words, int group, bool q8, bool mass, int sms) {
    // one wave of resident warps, but at least kMinWords words each
    const int per_sm = !q8 ? resident_warps<false, true>(group)
                           : mass ? resident_warps<true, true>(group) : resident_warps<true, false>(group);
    const int64_t words = static_cast<int64_t>(num_req) * max_words;
    const int64_t most = (words + kMinWords - 1) / kMinWords;
    const int64_t resident = static_cast<int64_t>(sms > 0 ? sms : 1) * per_sm / hkv;
    LanePlan pl;
    pl.warps_per_head = static_cast<int>(most < resident ? most : resident);
    if (pl.warps_per_head < 1) pl.warps_per_head = 1;
    pl.slots = static_cast<int64_t>(hkv) * (pl.warps_per_head + num_req);
    return pl;
}

cudaError_t launch_decode_lane(const LaneParams &p, bool q8, cudaStream_t s) {
    if (!q8) return launch_g<false, true>(p, s);
    return p.mass ? launch_g<true, true>(p, s) : launch_g<true, false>(p, s);
}

}  // namespace lazy

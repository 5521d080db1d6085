// prefill_q8.cu -- causal prefill attention over the 8-bit pool on tcgen05 tensor cores.
//
// For query row i (token at position p_i, head h on KV head kvh) and key t of block b at offset o,
// local index j, with codes k_t, v_t and the block's scales s_k, s_v:
//   s_it = scale q_i^T R(-(p_i - o)) (s_k k_t),  w_it = 2^(s_it - m) / l,  out_i = sum_t w_it s_v v_t.
//
// A CTA takes 256 query rows (two 128-row MMA tiles; rows are (token, head of the group) pairs) of
// one KV head of one request and walks the request's words in tiles of up to 8 words (128 keys) that
// share one offset.  Words that no row of the CTA sees are not visited: a long prompt's first rows
// skip its later keys.  All MMA operands are f16:
//   Q'  R(p_i - P0) q_i 2^-e_i, the row's largest element in [1, 2) (P0: the CTA's first position):
//       prepared by a kernel before, in rows already laid out as the tensor core reads them;
//   K'  R(o - P0) k_t: codes rotated without their scale, which multiplies the scores instead (one
//       factor per 16 columns, in the instruction that subtracts the maximum);
//   P'  w 2^(log2 s_v - r) with a running reference r >= max(s + log2 s_v) - 8, so that neither
//       a large nor a small V scale over- or underflows f16;
//   V'  the codes themselves (exact).
// f16 keeps an operand to 2^-11 of its largest element where bf16 would keep 2^-8; K' is rotated in f16
// (cos and sin, one product and the sum rounded: 3 x 2^-11), which halves its cost and moves the
// output's error by less than its bf16 rounding.  Sums, maxima and outputs are fp32.
//
// 16 warps by role:
//   warp 0      table walk: per tile the words' metadata and scales into a ring of records, and the
//               blocks' codes (2 KiB per block, contiguous) into shared memory by bulk copies
//   warps 2, 1  MMA issuers of row tiles 0 and 1 (warp 2 owns tensor memory)
//   warp 3      the query tiles, then each tile's angles
//   warps 4-7, 8-11   softmax of row tile 0 and 1, one row per thread
//   warps 12-15 codes to f16: K rotated, V with the slots that no row sees as zeros, into the
//               128-byte-swizzled operand tiles (two stages each; codes have one)
// Tensor memory (512 columns): per row tile two score buffers of 64 columns (P over their first
// halves), then O0, O1 of 128 columns.
//
// What bounds it: shared memory's data pipe, which the tensor cores' operands take half of and the conversions
// with their stores about a third: 16 requests of 256 tokens over 4161, 32 heads on 8, 352 GFLOP in 385 us alone
// (0.91 PFLOP/s), 407 us in a graph, 445 to 458 us in a row of calls.
#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "pdl.cuh"
#include "q8.cuh"
#include "tc.cuh"

namespace lazy {

namespace {

constexpr int kTileRows = 128, kRows = 2 * kTileRows, kTileBlocks = 8;
constexpr int kTileBytes = kTileRows * kHeadDim * 2, kHalfPlane = kTileBytes / 2;
constexpr int kCodeBlock = kBlockTokens * kHeadDim, kCodeBytes = kTileBlocks * kCodeBlock;
constexpr int kStages = 2, kInfoStages = 4, kThreads = 512;
static_assert(kRows == kPrefillRows, "rows per CTA");

// One tile of the walk; n = 0 ends it.
struct TileInfo {
    uint32_t meta[kTileBlocks];
    float ks[kTileBlocks];    // K scales
    float lv[kTileBlocks];    // log2 of the V scales
    int n, off, full, pad;    // full: every key of 8 blocks is visible to every row
};

constexpr int kOffQ = 0;                                     // 2 row tiles
constexpr int kOffK = kOffQ + 2 * kTileBytes;
constexpr int kOffV = kOffK + kStages * kTileBytes;
constexpr int kOffKC = kOffV + kStages * kTileBytes;         // codes: one stage each
constexpr int kOffVC = kOffKC + kCodeBytes;
constexpr int kOffInfo = kOffVC + kCodeBytes;
constexpr int kOffBar = kOffInfo + kInfoStages * static_cast<int>(sizeof(TileInfo));
// barriers: codes landed / converted; per stage operand tile written / read, angles; records; per row tile
// and score buffer scores / weights / product done
constexpr int B_KCFULL = 0, B_KCEMPTY = 1, B_VCFULL = 2, B_VCEMPTY = 3, B_KFULL = 4, B_KEMPTY = B_KFULL + kStages,
              B_VFULL = B_KEMPTY + kStages, B_VEMPTY = B_VFULL + kStages, B_AFULL = B_VEMPTY + kStages,
              B_IFULL = B_AFULL + kStages, B_IEMPTY = B_IFULL + kInfoStages, B_SFULL = B_IEMPTY + kInfoStages,
              B_PFULL = B_SFULL + 4, B_ODONE = B_PFULL + 4, B_QFULL = B_ODONE + 4, B_DRAIN = B_QFULL + 1,
              kNumBars = B_DRAIN + 2;
constexpr int kOffAngle = (kOffBar + kNumBars * 8 + 15) / 16 * 16;   // two tables of f16 cos [64], sin [64]
constexpr int kOffMisc = kOffAngle + 2 * 256;
constexpr int kOffSlope = kOffMisc + 16;
constexpr size_t kSmem = kOffSlope + 32 * 4 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr int kColO = 256;                  // tensor memory columns of O (S from 0)
constexpr int kInfoConsumers = 15;          // 8 softmax, 2 MMA, 4 conversion warps, the angle warp
constexpr float kSlack = 8.0f;   // log2 units by which a maximum may pass its reference

// kind::f16 with f16 A/B and fp32 accumulation, M = 128.
constexpr uint32_t idesc_f16(int n, bool b_mn_major) {
    return (1u << 4) | (b_mn_major ? (1u << 16) : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

// size bytes (a multiple of 16), both addresses 16-byte aligned
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t size, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(size), "r"(smem_u32(bar))
                 : "memory");
}
// Out of line: the roles' loops together have to fit the instruction cache.
__device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *d_status) {
    return wait_or_abort(bar, parity, abort_flag, d_status);
}
// Same decision for every lane of the warp.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *d_status) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_long(bar, parity, abort_flag, d_status));
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ float log2_of(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^d as a product of two factors, so that |d| up to 250 neither overflows nor flushes on the way
__device__ __forceinline__ float half_exp2(float d) { return fast_exp2(0.5f * fmaxf(-250.f, fminf(d, 250.f))); }

// Work unit of CTA order s: long m-tiles first (their rows see the most keys), then KV head, request.
__device__ __forceinline__ void unit_of(const AttnParams &a, int s, int &mt, int &kvh, int &r) {
    const int per = a.hkv * a.num_req;
    mt = a.pf_mtiles - 1 - s / per;
    kvh = s % per % a.hkv;
    r = s % per / a.hkv;
}
// Index of a unit's 256 rows in the prepared query buffer.
__device__ __forceinline__ int64_t unit_rows(const AttnParams &a, int mt, int kvh, int r) {
    return ((static_cast<int64_t>(r) * a.hkv + kvh) * a.pf_mtiles + mt) * kRows;
}

// TILES: row tiles with rows; with one the other's issuer and softmax warps have nothing to do.
template <bool ALIBI, int TILES>
__global__ void __launch_bounds__(kThreads, 1) prefill_q8_kernel(const __grid_constant__ Q8PrefillParams P) {
    const AttnParams &p = P.a;
    pdl_trigger();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + kOffBar);
    float *slope_s = reinterpret_cast<float *>(sm + kOffSlope);
    TileInfo *info = reinterpret_cast<TileInfo *>(sm + kOffInfo);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + kOffMisc + 4);

    int order = static_cast<int>(blockIdx.x), part = -1;
    if (order >= p.pf_base) {
        const int k = order - p.pf_base;
        order = p.pf_base + k / P.parts;
        part = k % P.parts;
    }
    int mt, kvh, r;
    unit_of(p, order, mt, kvh, r);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.group;
    const int q0 = p.cu_q[r];
    const int T = p.cu_q[r + 1] - q0;
    const int R0 = mt * kRows;
    if (R0 >= T * G) {   // uniform: no rows
        pdl_wait();      // (what follows on the stream waits for this kernel, and so for the query kernel, in every case)
        return;
    }
    const int wbase = p.table_indptr[r];
    const int n_all = p.table_indptr[r + 1] - wbase, n_words = min(n_all, p.max_words);
    int wbeg = 0, wend = n_words;
    if (part >= 0) {
        const int per = ((n_words + P.parts - 1) / P.parts + kTileBlocks - 1) / kTileBlocks * kTileBlocks;
        wbeg = min(n_words, part * per);
        wend = min(n_words, wbeg + per);
    }
    const int pos0 = p.q_pos0[r];
    const int tok_first = R0 / G, tok_last = min(T - 1, (R0 + kRows - 1) / G);
    const int Pbase = pos0 + tok_first, Plast = pos0 + tok_last;

    if (threadIdx.x == 0) {
        mbar_init(&bars[B_KCFULL], 1);
        mbar_init(&bars[B_KCEMPTY], 4);
        mbar_init(&bars[B_VCFULL], 1);
        mbar_init(&bars[B_VCEMPTY], 4);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars[B_KFULL + i], 4);
            mbar_init(&bars[B_KEMPTY + i], TILES);
            mbar_init(&bars[B_VFULL + i], 4);
            mbar_init(&bars[B_VEMPTY + i], TILES);
            mbar_init(&bars[B_AFULL + i], 1);
        }
        for (int i = 0; i < kInfoStages; ++i) {
            mbar_init(&bars[B_IFULL + i], 1);
            mbar_init(&bars[B_IEMPTY + i], TILES == 2 ? kInfoConsumers : kInfoConsumers - 5);
        }
        for (int t = 0; t < 4; ++t) {
            mbar_init(&bars[B_SFULL + t], 1);
            mbar_init(&bars[B_PFULL + t], 4);
            mbar_init(&bars[B_ODONE + t], 1);
        }
        mbar_init(&bars[B_QFULL], 1);
        mbar_init(&bars[B_DRAIN], 1);
        mbar_init(&bars[B_DRAIN + 1], 1);
        *abort_flag = 0;
        if (mt == 0 && kvh == 0 && n_all > p.max_words) set_status(p.d_status, LAZY_DSTATUS_BAD_TABLE);
        fence_barrier_init();
    }
    if (ALIBI && threadIdx.x < G) slope_s[threadIdx.x] = p.alibi_log2[kvh * G + threadIdx.x];
    if (warp == 2) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = *tmem_slot;
    pdl_wait();   // the prepared query

    const int role = TILES == 1 && (warp == 1 || (warp >= 8 && warp < 12)) ? 16 : warp;
    if (role < 4) {
        const bool leader = tc::elect_one();
        if (warp == 0) {
            // ======================================================== table walk and code copies
            int j = 0, n_kc = 0;   // tiles whose V, K copies were issued
            bool ok = true;
            // 32 words at a time, one per lane, with their blocks' metadata and scales: three dependent loads
            // serve up to four tiles
            uint32_t wl = 0u, mt_l = 0u, seen = 0u;
            float ks_l = 0.f, lv_l = 0.f;
            int w0 = INT_MIN / 2;
            for (int w = wbeg; w < wend;) {
                if (w - w0 + kTileBlocks > 32 && w0 + 32 < wend) {
                    w0 = w;
                    wl = mt_l = 0u;
                    bool vis = false;
                    if (w + lane < wend) {
                        wl = p.table[wbase + w + lane];
                        const uint32_t b = word_block(wl);
                        if (b < static_cast<uint32_t>(p.num_blocks)) {
                            const size_t bh = static_cast<size_t>(b) * p.hkv + kvh;
                            mt_l = p.blk_meta[b];
                            ks_l = P.k_scale[bh];
                            lv_l = log2_of(P.v_scale[bh]);
                            vis = meta_valid(mt_l) > 0 && word_offset(wl) + meta_j0(mt_l) <= Plast;
                        } else {
                            set_status(p.d_status, LAZY_DSTATUS_BAD_BLOCK);
                        }
                    }
                    seen = __ballot_sync(0xffffffffu, vis);
                }
                const int i = w - w0;
                const uint32_t rest = seen >> i;
                if (rest == 0u) {
                    w = w0 + 32;
                    continue;
                }
                const int skip = __ffs(rest) - 1;
                if (skip > 0) {
                    w += skip;
                    continue;
                }
                // the tile: up to 8 visible words that share an offset; lane k < 8 holds word w + k
                const int src = (i + lane) & 31;
                const uint32_t wk = __shfl_sync(0xffffffffu, wl, src);
                const uint32_t mt = __shfl_sync(0xffffffffu, mt_l, src);
                const float ks = __shfl_sync(0xffffffffu, ks_l, src), lv = __shfl_sync(0xffffffffu, lv_l, src);
                const int off = word_offset(__shfl_sync(0xffffffffu, wl, i));
                const bool same = lane < kTileBlocks && i + lane < 32 && ((seen >> src) & 1u) && word_offset(wk) == off;
                const int n = __ffs(~__ballot_sync(0xffffffffu, same)) - 1;
                const size_t bh = static_cast<size_t>(word_block(wk)) * p.hkv + kvh;
                const bool full =
                    n == kTileBlocks && __all_sync(0xffffffffu, lane >= n || (meta_valid(mt) == kBlockTokens &&
                                                                              off + meta_j0(mt) + kBlockTokens - 1 <= Pbase));
                const int is = j % kInfoStages;
                ok = warp_wait(&bars[B_IEMPTY + is], ((j / kInfoStages) & 1) ^ 1, abort_flag, p.d_status);
                if (!ok) break;
                TileInfo &ti = info[is];
                if (lane < kTileBlocks) {
                    ti.meta[lane] = lane < n ? mt : 0u;
                    ti.ks[lane] = lane < n ? ks : 0.f;
                    ti.lv[lane] = lane < n ? lv : 0.f;
                }
                if (leader) {
                    ti.n = n;
                    ti.off = off;
                    ti.full = full;
                }
                __syncwarp();
                if (leader) mbar_arrive(&bars[B_IFULL + is]);
                ok = warp_wait(&bars[B_KCEMPTY], (j & 1) ^ 1, abort_flag, p.d_status);
                if (!ok) break;
                if (leader) mbar_arrive_expect_tx(&bars[B_KCFULL], n * kCodeBlock);
                __syncwarp();
                if (lane < n) bulk_load(sm + kOffKC + lane * kCodeBlock, P.k_codes + bh * kCodeBlock, kCodeBlock, &bars[B_KCFULL]);
                ++n_kc;
                ok = warp_wait(&bars[B_VCEMPTY], (j & 1) ^ 1, abort_flag, p.d_status);
                if (!ok) break;
                if (leader) mbar_arrive_expect_tx(&bars[B_VCFULL], n * kCodeBlock);
                __syncwarp();
                if (lane < n) bulk_load(sm + kOffVC + lane * kCodeBlock, P.v_codes + bh * kCodeBlock, kCodeBlock, &bars[B_VCFULL]);
                ++j;
                w += n;
            }
            if (ok) {
                const int is = j % kInfoStages;
                if (warp_wait(&bars[B_IEMPTY + is], ((j / kInfoStages) & 1) ^ 1, abort_flag, p.d_status)) {
                    if (leader) {
                        info[is].n = 0;
                        mbar_arrive(&bars[B_IFULL + is]);
                    }
                    __syncwarp();
                }
            }
            // every copy lands before the kernel can end, whatever stopped the walk
            if (n_kc > 0) mbar_wait(&bars[B_KCFULL], (n_kc - 1) & 1);
            if (j > 0) mbar_wait(&bars[B_VCFULL], (j - 1) & 1);
        } else if (warp < 3) {
            // ======================================================== MMA issuers (warp 2: row tile 0, warp 1: row tile 1)
            // Step i is half a tile (64 keys), its scores in buffer i & 1:
            //   QK(0) QK(1) | PV(0) QK(2) | PV(1) QK(3) | ...
            // Scores are a step ahead of the softmax, so that neither it nor the tensor core waits for a round
            // trip.  QK(i + 2) follows PV(i) in issue order, which lets P(i) live in S(i).  One warp per row
            // tile: a step's waits and issues take one warp longer than the products themselves.
            const int t = warp == 2 ? 0 : 1;
            constexpr uint32_t idq = idesc_f16(64, false), idv = idesc_f16(128, true);
            const uint64_t dQ = tc::smem_desc(smem_u32(sm + kOffQ + t * kTileBytes), 16, 1024);
            const uint64_t dK0 = tc::smem_desc(smem_u32(sm + kOffK), 16, 1024);
            const uint64_t dV0 = tc::smem_desc(smem_u32(sm + kOffV), kHalfPlane, 1024);
            const uint32_t tS = tbase + 128 * t, tO = tbase + kColO + 128 * t;
            // a step: blocks (0 ends the walk), and stage | half << 1 | (last of its tile) << 2
            struct Step {
                int n, at;
            };
            int tj = -1, tn = 0, th = 0;
            bool ok = true;
            auto fetch = [&]() {
                if (tn > 4 * (th + 1)) {
                    ++th;
                } else {
                    ++tj;
                    th = 0;
                    // the conversion warps have read the tile's record before they signal its keys
                    ok = warp_wait(&bars[B_KFULL + tj % kStages], (tj / kStages) & 1, abort_flag, p.d_status);
                    const int is = tj % kInfoStages;
                    tn = ok ? info[is].n : 0;
                    __syncwarp();
                    if (leader) mbar_arrive(&bars[B_IEMPTY + is]);
                    tc::fence_after_sync();
                }
                return Step{min(4, tn - 4 * th), (tj % kStages) | th << 1 | (tn <= 4 * (th + 1) ? 4 : 0)};
            };
            auto qk = [&](int buf, const Step &st) {
                const uint64_t kb = dK0 + static_cast<uint64_t>(((st.at & 1) * kTileBytes + ((st.at >> 1) & 1) * 64 * 128) >> 4);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint64_t o = static_cast<uint64_t>(((kk >> 2) * kHalfPlane + (kk & 3) * 32) >> 4);
                    tc::mma_ss(tS + 64 * buf, dQ + o, kb + o, idq, kk > 0 ? 1u : 0u);
                }
                tc::commit(&bars[B_SFULL + 2 * t + buf]);
                if (st.at & 4) tc::commit(&bars[B_KEMPTY + (st.at & 1)]);
            };
            Step s0 = {0, 0}, s1 = {0, 0};
            if (warp_wait(&bars[B_QFULL], 0, abort_flag, p.d_status)) {
                s0 = fetch();
                if (s0.n > 0) {
                    if (leader) qk(0, s0);
                    __syncwarp();
                    s1 = fetch();
                    if (leader && s1.n > 0) qk(1, s1);
                    __syncwarp();
                }
            }
            int vj = 0;   // tile of step s0
            for (int i = 0; s0.n > 0; ++i) {
                const int buf = i & 1, vs = s0.at & 1, half = (s0.at >> 1) & 1;
                if (half == 0 && !warp_wait(&bars[B_VFULL + vs], (vj / kStages) & 1, abort_flag, p.d_status)) break;
                if (!warp_wait(&bars[B_PFULL + 2 * t + buf], (i >> 1) & 1, abort_flag, p.d_status)) break;
                tc::fence_after_sync();
                if (leader) {
                    const uint64_t vb = dV0 + static_cast<uint64_t>((vs * kTileBytes + half * 4 * kBoxBytes) >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < s0.n)
                            tc::mma_ts(tO, tS + 64 * buf + 8 * k, vb + static_cast<uint64_t>((k * kBoxBytes) >> 4), idv,
                                       (i > 0 || k > 0) ? 1u : 0u);
                    // one barrier per buffer: S(i) full says that PV(i - 2) is done, so a wait for PV(i - 1)
                    // meets a barrier at most one phase behind
                    tc::commit(&bars[B_ODONE + 2 * t + buf]);
                    if (s0.at & 4) tc::commit(&bars[B_VEMPTY + vs]);
                }
                __syncwarp();
                if (s0.at & 4) ++vj;
                s0 = s1;
                if (s1.n > 0) {
                    s1 = fetch();
                    if (!ok) break;
                    if (leader && s1.n > 0) qk(buf, s1);
                    __syncwarp();
                }
            }
            // every MMA has completed before tensor memory is freed
            if (leader) tc::commit(&bars[B_DRAIN + t]);
            __syncwarp();
            mbar_wait(&bars[B_DRAIN + t], 0);
        } else {
            // ======================================================== query tiles and angles
            if (leader) {
                mbar_arrive_expect_tx(&bars[B_QFULL], TILES * kTileBytes);
                const uint16_t *q = p.q_prep + unit_rows(p, mt, kvh, r) * kHeadDim;
#pragma unroll
                for (int t = 0; t < 2 * TILES; ++t)
                    bulk_load(sm + kOffQ + t * kHalfPlane, q + t * (kHalfPlane / 2), kHalfPlane, &bars[B_QFULL]);
            }
            __syncwarp();
            // tile j's angles into table j & 1, free since the K of tile j - 2 is done
            const double th0 = p.rope.theta[lane], th1 = p.rope.theta[lane + 32];
            int cur = INT_MIN;
            float c0 = 1.f, s0 = 0.f, c1 = 1.f, s1 = 0.f;
            for (int j = 0;; ++j) {
                const int is = j % kInfoStages, st = j % kStages;
                if (!warp_wait(&bars[B_IFULL + is], (j / kInfoStages) & 1, abort_flag, p.d_status)) break;
                const int n = info[is].n, off = info[is].off;
                if (n == 0) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_IEMPTY + is]);
                if (off != cur) {
                    cur = off;
                    rope_cos_sin(off - Pbase, th0, c0, s0);
                    rope_cos_sin(off - Pbase, th1, c1, s1);
                }
                if (!warp_wait(&bars[B_KFULL + st], ((j / kStages) & 1) ^ 1, abort_flag, p.d_status)) break;
                __half *tab = reinterpret_cast<__half *>(sm + kOffAngle + st * 256);
                tab[lane] = __float2half_rn(c0);
                tab[lane + 32] = __float2half_rn(c1);
                tab[kHalfDim + lane] = __float2half_rn(s0);
                tab[kHalfDim + lane + 32] = __float2half_rn(s1);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_AFULL + st]);
            }
            mbar_wait(&bars[B_QFULL], 0);   // landed before the kernel can end
        }
    } else if (role < 12) {
        // ============================================================ softmax (one row per thread)
        const int t = (warp - 4) >> 2;
        const int row = threadIdx.x - 128 - 128 * t;
        const int R = R0 + kTileRows * t + row;
        const bool row_ok = R < T * G;
        const int tok = row_ok ? R / G : tok_first;
        const int g = R % G;
        const int prow = pos0 + tok;
        const float slope = ALIBI ? slope_s[g] : 0.f;
        const float hm = P.row_scale[unit_rows(p, mt, kvh, r) + kTileRows * t + row];   // softmax scale log2(e) 2^e
        const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t tS = tbase + 128 * t + lane_off, tO = tbase + kColO + 128 * t + lane_off;
        float m_run = -INFINITY, l_run = 0.f, mo = -INFINITY;
        int i = 0;   // steps of 64 keys
        bool ok = true;
        for (int j = 0; ok; ++j) {
            const int is = j % kInfoStages;
            ok = warp_wait(&bars[B_IFULL + is], (j / kInfoStages) & 1, abort_flag, p.d_status);
            if (!ok) break;
            const TileInfo &ti = info[is];
            const int n = ti.n;
            if (n == 0) break;
#pragma unroll 1
            for (int k0 = 0; k0 < n; k0 += 4, ++i) {
                const int buf = i & 1;
                ok = warp_wait(&bars[B_SFULL + 2 * t + buf], (i >> 1) & 1, abort_flag, p.d_status);
                if (!ok) break;
                tc::fence_after_sync();
                uint32_t sv[64];
                tc::ld32(tS + 64 * buf, *reinterpret_cast<uint32_t(*)[32]>(sv));
                tc::ld32(tS + 64 * buf + 32, *reinterpret_cast<uint32_t(*)[32]>(sv + 32));
                const float4 ks4 = *reinterpret_cast<const float4 *>(&ti.ks[k0]), lv4 = *reinterpret_cast<const float4 *>(&ti.lv[k0]);
                const float ks[4] = {ks4.x, ks4.y, ks4.z, ks4.w}, lv[4] = {lv4.x, lv4.y, lv4.z, lv4.w};
                tc::wait_ld();
                auto f = [&sv](int c) { return __uint_as_float(sv[c]); };
                if (ALIBI) {
                    // scores with the in-block part of the bias; the block part joins the maxima and offsets
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float fk = ks[k] * hm;
#pragma unroll
                        for (int c = 16 * k; c < 16 * k + 16; ++c)
                            sv[c] = __float_as_uint(fmaf(f(c), fk, slope * static_cast<float>(c & 15)));
                    }
                }
                if (!ti.full) {
                    // slots that this row sees of each block; blocks behind the tile's last have none
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t m = ti.meta[k0 + k];
                        // (a tile's keys are not all behind the last query, so the difference does not overflow)
                        const int lim = min(meta_valid(m) - 1, prow - ti.off - meta_j0(m)) + 1;
#pragma unroll
                        for (int c = 16 * k; c < 16 * k + 16; ++c) sv[c] = (c & 15) < lim ? sv[c] : 0xFF800000u;
                    }
                }
                // factor of a block's scores; at least the smallest normal number, so that -inf stays -inf
                auto factor = [&](int k) { return ALIBI ? 1.f : fmaxf(ks[k] * hm, 0x1p-126f); };
                auto bias = [&](int k) {
                    return ALIBI ? slope * static_cast<float>(ti.off + meta_j0(ti.meta[k0 + k]) - prow) : 0.f;
                };
                float m_new = -INFINITY, mo_new = -INFINITY;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float a = max3(f(16 * k), f(16 * k + 1), f(16 * k + 2)), b = f(16 * k + 15);
#pragma unroll
                    for (int c = 3; c < 15; c += 4) {
                        a = max3(a, f(16 * k + c), f(16 * k + c + 1));
                        b = max3(b, f(16 * k + c + 2), f(16 * k + c + 3));
                    }
                    const float s = fmaf(fmaxf(a, b), factor(k), bias(k));
                    m_new = fmaxf(m_new, s);
                    mo_new = fmaxf(mo_new, s + lv[k]);
                }
                // References move only when the maxima pass them by kSlack (log2 units): weights stay below 2^8,
                // and most steps need no rescaling.
                const bool need = mo_new > mo + kSlack;
                float scale = 1.f;
                if (__any_sync(0xffffffffu, need || m_new > m_run + kSlack)) {
                    m_new = fmaxf(m_new, m_run);
                    if (m_new > m_run) {
                        l_run *= fast_exp2(m_run - m_new);
                        m_run = m_new;
                    }
                    if (need) {
                        scale = fast_exp2(mo - mo_new);
                        mo = mo_new;
                    }
                }
                const float mu = m_run == -INFINITY ? 0.f : m_run, mou = mo == -INFINITY ? 0.f : mo;
                // Weights for the products, w' = 2^(s - m + e) with e = m + log2 s_v - r; the row sum takes a block's
                // sum times 2^-e.  e is kept above -40, where w' is 0 in f16 either way: the sum of a block
                // whose values are that much smaller than others still counts its weights.
                float ls = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float e = fmaxf(mu + lv[k] - mou, -40.f);
                    const float fk = factor(k), nm = bias(k) - mu + e;
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int c = 8 * k; c < 8 * k + 8; ++c) {
                        float x0, x1;
                        fma2v(x0, x1, f(2 * c), f(2 * c + 1), fk, fk, nm, nm);
                        x0 = fast_exp2(x0);
                        x1 = fast_exp2(x1);
                        add2(s0, s1, x0, x1);
                        sv[c] = pack_h2(x0, x1);
                    }
                    ls = fmaf(s0 + s1, fast_exp2(-e), ls);
                }
                l_run += ls;
                tc::st32(tS + 64 * buf, *reinterpret_cast<uint32_t(*)[32]>(sv));
                if (i > 0 && __any_sync(0xffffffffu, need)) {
                    ok = warp_wait(&bars[B_ODONE + 2 * t + (buf ^ 1)], ((i - 1) >> 1) & 1, abort_flag, p.d_status);
                    if (!ok) break;
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[32];
                        tc::ld32(tO + 32 * c, o);
                        tc::wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * scale);
                        tc::st32(tO + 32 * c, o);
                    }
                }
                tc::wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_PFULL + 2 * t + buf]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_IEMPTY + is]);
        }
        // ------------------------------------------------------------ epilogue: O 2^(mo - m) / l
        bool have = ok && i > 0;
        if (have) have = warp_wait(&bars[B_ODONE + 2 * t + ((i - 1) & 1)], ((i - 1) >> 1) & 1, abort_flag, p.d_status);
        have = __all_sync(0xffffffffu, have);
        if (have) tc::fence_after_sync();
        const bool some = have && m_run != -INFINITY;
        const float hf = some ? half_exp2(mo - m_run) : (have && l_run != l_run ? 1.f : 0.f);
        const float inv = part >= 0 ? hf : (have && (l_run > 0.f || l_run != l_run)) ? hf / l_run : 0.f;
        float *po = nullptr;
        uint4 *o = nullptr;
        if (part >= 0) {
            const size_t srow = (static_cast<size_t>(order - p.pf_base) * P.parts + part) * kRows + kTileRows * t + row;
            po = p.ws_acc + srow * kHeadDim;
            p.ws_ml[2 * srow] = have ? m_run : -INFINITY;
            p.ws_ml[2 * srow + 1] = have ? l_run : 0.f;
        } else if (row_ok) {
            o = reinterpret_cast<uint4 *>(p.out + (static_cast<size_t>(q0 + tok) * p.hq + kvh * G + g) * kHeadDim);
        }
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            uint32_t ob[32];
            if (have) {
                tc::ld32(tO + 32 * c, ob);
                tc::wait_ld();
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) ob[e] = inv != 0.f ? __float_as_uint(__uint_as_float(ob[e]) * hf * inv) : 0u;
            if (po) {
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    reinterpret_cast<uint4 *>(po)[8 * c + v] = make_uint4(ob[4 * v], ob[4 * v + 1], ob[4 * v + 2], ob[4 * v + 3]);
            } else if (o) {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    uint4 u;
                    u.x = pack_bf16(__uint_as_float(ob[8 * v + 0]), __uint_as_float(ob[8 * v + 1]));
                    u.y = pack_bf16(__uint_as_float(ob[8 * v + 2]), __uint_as_float(ob[8 * v + 3]));
                    u.z = pack_bf16(__uint_as_float(ob[8 * v + 4]), __uint_as_float(ob[8 * v + 5]));
                    u.w = pack_bf16(__uint_as_float(ob[8 * v + 6]), __uint_as_float(ob[8 * v + 7]));
                    o[4 * c + v] = u;
                }
            }
        }
    } else if (role < 16) {
        // ============================================================ codes to f16 operand tiles
        // Thread (ch, rb) takes elements 8 ch .. + 7 (a) and 64 above (b) of slot rb of every block.  Where rb is
        // odd b is loaded first: two rows' 8-byte loads then cover all banks.  K: (a, b) -> (a c - b s, b c + a s);
        // with b in a's place the same formulas with -s give b c + a s first.
        const int tid = threadIdx.x - 384;
        const int ch = tid & 7, rb = tid >> 3, up = rb & 1;
        const uint32_t at = rb * kHeadDim + 8 * ch;                        // in a block's codes
        const uint32_t sw = rb * 128 + ((ch ^ (rb & 7)) << 4);             // in a half plane of its operand tile
        const uint32_t flip = up ? 0x80008000u : 0u;
        const uint8_t *kc = sm + kOffKC + at, *vc = sm + kOffVC + at;
        const int first = up * kHalfDim, second = kHalfDim - first;
        for (int j = 0;; ++j) {
            const int is = j % kInfoStages, st = j % kStages;
            if (!warp_wait(&bars[B_IFULL + is], (j / kInfoStages) & 1, abort_flag, p.d_status)) break;
            const TileInfo &ti = info[is];
            if (ti.n == 0) {
                // The end, for the MMA issuers.  As before a tile's keys: they have seen the stage's last phase, so
                // that none of them waits for one that is two phases back (a walk of two tiles could end before
                // the query lets them see the first).
                if (!warp_wait(&bars[B_KEMPTY + st], ((j / kStages) & 1) ^ 1, abort_flag, p.d_status)) break;
                if (lane == 0) mbar_arrive(&bars[B_KFULL + st]);
                break;
            }
            uint32_t keep = 0u;   // bit k: some row may see slot rb of block k
#pragma unroll
            for (int k = 0; k < kTileBlocks; ++k)
                keep |= (rb <= min(meta_valid(ti.meta[k]) - 1, Plast - ti.off - meta_j0(ti.meta[k])) ? 1u : 0u) << k;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_IEMPTY + is]);
            if (!warp_wait(&bars[B_AFULL + st], (j / kStages) & 1, abort_flag, p.d_status)) break;
            const uint4 c4 = *reinterpret_cast<const uint4 *>(sm + kOffAngle + st * 256 + 16 * ch);
            const uint4 s4 = *reinterpret_cast<const uint4 *>(sm + kOffAngle + st * 256 + 128 + 16 * ch);
            const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x ^ flip, s4.y ^ flip, s4.z ^ flip, s4.w ^ flip};
            if (!warp_wait(&bars[B_KCFULL], j & 1, abort_flag, p.d_status)) break;
            if (!warp_wait(&bars[B_KEMPTY + st], ((j / kStages) & 1) ^ 1, abort_flag, p.d_status)) break;
            uint8_t *kt = sm + kOffK + st * kTileBytes + sw;
            // all 8 blocks (those behind the tile's last hold old codes, whose scores are masked), loads
            // ahead of the stores they could otherwise not pass
#pragma unroll
            for (int k0 = 0; k0 < kTileBlocks; k0 += 4) {
                uint2 x[4], y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[k] = *reinterpret_cast<const uint2 *>(kc + (k0 + k) * kCodeBlock + first);
                    y[k] = *reinterpret_cast<const uint2 *>(kc + (k0 + k) * kCodeBlock + second);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t a[4], b[4], oa[4], ob[4];
                    codes_to_f16(x[k].x, a[0], a[1]);
                    codes_to_f16(x[k].y, a[2], a[3]);
                    codes_to_f16(y[k].x, b[0], b[1]);
                    codes_to_f16(y[k].y, b[2], b[3]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        oa[u] = h2_fma(b[u], s[u] ^ 0x80008000u, h2_mul(a[u], c[u]));
                        ob[u] = h2_fma(a[u], s[u], h2_mul(b[u], c[u]));
                    }
                    uint8_t *kd = kt + (k0 + k) * kBoxBytes;
                    *reinterpret_cast<uint4 *>(kd + up * kHalfPlane) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
                    *reinterpret_cast<uint4 *>(kd + (up ^ 1) * kHalfPlane) = make_uint4(ob[0], ob[1], ob[2], ob[3]);
                }
            }
            fence_proxy_async_smem();   // generic writes become visible to the tensor core
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars[B_KCEMPTY]);
                mbar_arrive(&bars[B_KFULL + st]);
            }
            if (!warp_wait(&bars[B_VCFULL], j & 1, abort_flag, p.d_status)) break;
            if (!warp_wait(&bars[B_VEMPTY + st], ((j / kStages) & 1) ^ 1, abort_flag, p.d_status)) break;
            uint8_t *vt = sm + kOffV + st * kTileBytes + sw;
            // (blocks behind the tile's last hold old codes that no MMA reads)
#pragma unroll
            for (int k0 = 0; k0 < kTileBlocks; k0 += 4) {
                uint2 x[4][2];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[k][0] = *reinterpret_cast<const uint2 *>(vc + (k0 + k) * kCodeBlock + first);
                    x[k][1] = *reinterpret_cast<const uint2 *>(vc + (k0 + k) * kCodeBlock + second);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint2 w = x[k][h];
                        if (!((keep >> (k0 + k)) & 1u)) w = make_uint2(0u, 0u);   // a weight of 0 does not undo a NaN
                        uint4 o;
                        codes_to_f16(w.x, o.x, o.y);
                        codes_to_f16(w.y, o.z, o.w);
                        *reinterpret_cast<uint4 *>(vt + (k0 + k) * kBoxBytes + (up ^ h) * kHalfPlane) = o;
                    }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars[B_VCEMPTY]);
                mbar_arrive(&bars[B_VFULL + st]);
            }
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == 2) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tbase, 512);
    }
}

// Joins the parts of each split unit: O = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.  One warp per
// query row, 4 head dims per lane.
__global__ void __launch_bounds__(256) prefill_q8_join_kernel(const __grid_constant__ Q8PrefillParams P) {
    pdl_wait();
    const AttnParams &p = P.a;
    const int row_in = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    int mt, kvh, r;
    unit_of(p, p.pf_base + blockIdx.x, mt, kvh, r);
    const int G = p.group, q0 = p.cu_q[r], T = p.cu_q[r + 1] - q0;
    const int R = mt * kRows + row_in;
    if (R >= T * G) return;
    const size_t s0 = static_cast<size_t>(blockIdx.x) * P.parts * kRows + row_in;
    float M = -INFINITY;
    for (int i = 0; i < P.parts; ++i) M = fmaxf(M, p.ws_ml[2 * (s0 + static_cast<size_t>(i) * kRows)]);
    const float mu = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < P.parts; ++i) {
        const size_t s = s0 + static_cast<size_t>(i) * kRows;
        const float w = fast_exp2(p.ws_ml[2 * s] - mu);
        L += w * p.ws_ml[2 * s + 1];
        const float4 a = reinterpret_cast<const float4 *>(p.ws_acc + s * kHeadDim)[lane];
        A.x += w * a.x;
        A.y += w * a.y;
        A.z += w * a.z;
        A.w += w * a.w;
    }
    const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
    const int tok = R / G, g = R % G;
    reinterpret_cast<uint2 *>(p.out + (static_cast<size_t>(q0 + tok) * p.hq + kvh * G + g) * kHeadDim)[lane] =
        make_uint2(pack_bf16(A.x * inv, A.y * inv), pack_bf16(A.z * inv, A.w * inv));
}

// The query tiles of every unit: row R (token R / G, head R % G of the group) becomes
// Q' = R(p - P0) q 2^-e in f16, laid out as the kernel's shared memory holds it (two row tiles of two
// half planes, 128-byte swizzled), and row_scale = scale log2(e) 2^e.  Rows behind the request's last
// are zero.  Half a warp per row, its angles evaluated once for all KV heads.
__global__ void __launch_bounds__(256) prefill_q8_query_kernel(const __grid_constant__ Q8PrefillParams P) {
    const AttnParams &p = P.a;
    const int r = blockIdx.y, lane = threadIdx.x & 31, c = lane & 15;
    const int R = blockIdx.x * 16 + (threadIdx.x >> 4);
    const int G = p.group, q0 = p.cu_q[r], T = p.cu_q[r + 1] - q0;
    const int mt = R / kRows, row = R % kRows;
    pdl_trigger();
    // uniform for the 16 rows of the block; a second row tile is read where some request has rows for it
    if (mt >= p.pf_mtiles || mt * kRows >= T * G || (row >= kTileRows && p.max_q * G <= kTileRows)) return;
    const bool live = R < T * G;
    const int tok = live ? R / G : 0, g = R % G;
    float cs[4], sn[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) rope_cos_sin(live ? tok - (mt * kRows) / G : 0, p.rope.theta[4 * c + u], cs[u], sn[u]);
    // byte offset of dims 4 c .. + 3 of this row in its half plane
    const uint32_t at = (row / kTileRows) * kTileBytes + (row % kTileRows) * 128 + (((c >> 1) ^ (row & 7)) << 4) + (c & 1) * 8;
    for (int kvh = blockIdx.z; kvh < p.hkv; kvh += gridDim.z) {
        uint2 lo = make_uint2(0u, 0u), hi = lo;
        if (live) {
            const uint2 *q = reinterpret_cast<const uint2 *>(p.q_raw + (static_cast<size_t>(q0 + tok) * p.hq + kvh * G + g) * kHeadDim);
            lo = __ldg(q + c);
            hi = __ldg(q + 16 + c);
        }
        const float a[4] = {bf16_lo(lo.x), bf16_hi(lo.x), bf16_lo(lo.y), bf16_hi(lo.y)};
        const float b[4] = {bf16_lo(hi.x), bf16_hi(hi.x), bf16_lo(hi.y), bf16_hi(hi.y)};
        float am = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) am = fmaxf(am, fmaxf(fabsf(a[u]), fabsf(b[u])));
#pragma unroll
        for (int x = 1; x < 16; x <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, x));
        // q 2^-e in [1, 2); e = 0 for an all-zero row.  A row with an infinite element becomes NaN, as its softmax
        // is (scores of -infinity alone would read as keys that it does not see).
        const bool inf = am > FLT_MAX;
        int e = static_cast<int>(__float_as_uint(am) >> 23) - 127;
        e = (am == 0.f || inf) ? 0 : max(-126, min(126, e));
        const float dn = inf ? NAN : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        float x[4], y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float av = a[u] * dn, bv = b[u] * dn;
            x[u] = av * cs[u] - bv * sn[u];
            y[u] = bv * cs[u] + av * sn[u];
        }
        const int64_t unit = unit_rows(p, mt, kvh, r);
        uint8_t *dst = reinterpret_cast<uint8_t *>(p.q_prep + unit * kHeadDim) + at;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_h2(x[0], x[1]), pack_h2(x[2], x[3]));
        *reinterpret_cast<uint2 *>(dst + kHalfPlane) = make_uint2(pack_h2(y[0], y[1]), pack_h2(y[2], y[3]));
        if (c == 0) P.row_scale[unit + row] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * p.scale_log2;
    }
}

// Zeros for the rows of all requests (one after the other from the first one's), and for no others.
constexpr int kZeroCtas = 148;
__global__ void __launch_bounds__(256) zero_prefill_kernel(const __grid_constant__ AttnParams p) {
    const int64_t per = static_cast<int64_t>(p.hq) * (kHeadDim / 8), end = p.cu_q[p.num_req] * per;
    uint4 *out = reinterpret_cast<uint4 *>(p.out);
    for (int64_t i = p.cu_q[0] * per + blockIdx.x * 256 + threadIdx.x; i < end; i += kZeroCtas * 256) out[i] = make_uint4(0, 0, 0, 0);
}

constexpr int kQuerySplit = 512;   // CTAs of the query kernel up to which it takes a CTA per KV head

template <bool ALIBI, int TILES>
cudaError_t launch_t(const Q8PrefillParams &p, cudaStream_t s) {
    auto kern = prefill_q8_kernel<ALIBI, TILES>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    // with few rows a CTA per KV head, which evaluates the angles again (8 requests of 12 tokens, 8 heads,
    // with the launches overlapped: 47 us -> 39 in all)
    const int64_t ctas = static_cast<int64_t>(p.a.pf_mtiles) * (kRows / 16) * p.a.num_req;
    const dim3 grid(p.a.pf_mtiles * (kRows / 16), p.a.num_req, ctas <= kQuerySplit ? p.a.hkv : 1);
    prefill_q8_query_kernel<<<grid, 256, 0, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_dependent(kern, dim3(p.a.pf_base + p.parts * p.a.pf_nsplit), kThreads, kSmem, s, p);
    if (e != cudaSuccess || p.a.pf_nsplit == 0) return e;
    return launch_dependent(prefill_q8_join_kernel, dim3(p.a.pf_nsplit, kRows / 8), 256, 0, s, p);
}

}  // namespace

Q8PrefillPlan q8_prefill_plan(int64_t units, int max_words, int sms) {
    // Units of a last wave that leaves at least half of the SMs idle are split over their words, at
    // least two tiles a part.
    Q8PrefillPlan pl = {0, 1};
    if (units <= 0 || sms <= 0) return pl;
    const int64_t rem = units % sms;
    if (rem == 0 || 2 * rem > sms) return pl;
    const int64_t parts = std::min<int64_t>(std::min<int64_t>(sms / rem, 16), (int64_t(max_words) + 2 * kTileBlocks - 1) / (2 * kTileBlocks));
    if (parts < 2) return pl;
    pl.nsplit = static_cast<int>(rem);
    pl.parts = static_cast<int>(parts);
    return pl;
}

size_t q8_prefill_ws_bytes(int64_t units, int max_words, int sms) {
    const Q8PrefillPlan pl = q8_prefill_plan(units, max_words, sms);
    return static_cast<size_t>(units) * kRows * (kHeadDim * 2 + 4) +
           static_cast<size_t>(pl.nsplit) * pl.parts * (pl.nsplit ? kRows * (kHeadDim + 2) * 4 : 0);
}

cudaError_t launch_zero_prefill(const AttnParams &p, cudaStream_t s) {
    zero_prefill_kernel<<<kZeroCtas, 256, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_prefill_q8(Q8PrefillParams &p, void *workspace, int64_t units, int sms, cudaStream_t s) {
    const Q8PrefillPlan pl = q8_prefill_plan(units, p.a.max_words, sms);
    p.parts = pl.parts;
    p.a.pf_nsplit = pl.nsplit;
    p.a.pf_base = static_cast<int>(units) - pl.nsplit;
    p.a.q_prep = static_cast<uint16_t *>(workspace);
    p.a.ws_acc = reinterpret_cast<float *>(p.a.q_prep + units * kRows * kHeadDim);
    p.a.ws_ml = p.a.ws_acc + (pl.nsplit ? static_cast<size_t>(pl.nsplit) * pl.parts * kRows * kHeadDim : 0);
    p.row_scale = p.a.ws_ml + (pl.nsplit ? static_cast<size_t>(pl.nsplit) * pl.parts * kRows * 2 : 0);
    // One row tile where no request has rows for two (64 requests of 261 words, 12 tokens, 32 heads on 8: 393 us ->
    // 302).  A choice per CTA cost the long prompts 2 % (registers).
    if (static_cast<int64_t>(p.a.max_q) * p.a.group <= kTileRows)
        return p.a.alibi ? launch_t<true, 1>(p, s) : launch_t<false, 1>(p, s);
    return p.a.alibi ? launch_t<true, 2>(p, s) : launch_t<false, 2>(p, s);
}

}  // namespace lazy

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
//       prepared by a kernel before, so that the attention kernel loads it with plain bulk copies of
//       rows already laid out as the tensor core reads them;
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
//   warp 2      MMA issuer (and owner of tensor memory)
//   warps 4-7, 8-11   softmax of row tile 0 and 1, one row per thread
//   warps 12-15 K codes to rotated f16; warps 1 and 3 (after loading the query tiles) the angles of the
//               next tile, and V codes to f16, slots that no row sees as zeros.  Operand tiles are
//               128-byte swizzled, two stages each; codes have one stage each
// Tensor memory (512 columns): S0, S1 (P over their first halves), O0, O1, 128 columns each.
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>

#include "common.cuh"
#include "kernels.h"
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

constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + 2 * kTileBytes;
constexpr int kOffV = kOffK + kStages * kTileBytes;
constexpr int kOffKC = kOffV + kStages * kTileBytes;
constexpr int kOffVC = kOffKC + kCodeBytes;
constexpr int kOffInfo = kOffVC + kCodeBytes;
constexpr int kOffBar = kOffInfo + kInfoStages * static_cast<int>(sizeof(TileInfo));
constexpr int B_KCFULL = 0, B_KCEMPTY = 1, B_VCFULL = 2, B_VCEMPTY = 3, B_KFULL = 4, B_KEMPTY = B_KFULL + kStages,
              B_VFULL = B_KEMPTY + kStages, B_VEMPTY = B_VFULL + kStages, B_IFULL = B_VEMPTY + kStages,
              B_IEMPTY = B_IFULL + kInfoStages, B_SFULL = B_IEMPTY + kInfoStages, B_PFULL = B_SFULL + 2,
              B_ODONE = B_PFULL + 2, B_QFULL = B_ODONE + 2, B_DRAIN = B_QFULL + 1, B_AFULL = B_DRAIN + 1,
              kNumBars = B_AFULL + 2;
constexpr int kOffAngle = (kOffBar + kNumBars * 8 + 15) / 16 * 16;   // two tables of f16 cos [64], sin [64]
constexpr int kOffMisc = kOffAngle + 2 * 256;
constexpr int kOffSlope = kOffMisc + 16;
constexpr size_t kSmem = kOffSlope + 32 * 4 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr int kInfoConsumers = 15;          // 8 softmax warps, the MMA warp, 4 + 2 conversion warps
constexpr float kRescaleThreshold = 8.0f;   // log2 units: P' stays below 2^8 between rescales of O

// kind::f16 with f16 A/B and fp32 accumulation, 128 x 128.
constexpr uint32_t idesc_f16(bool b_mn_major) {
    return (1u << 4) | (b_mn_major ? (1u << 16) : 0u) | (16u << 17) | (8u << 24);
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

template <bool ALIBI>
__global__ void __launch_bounds__(kThreads, 1) prefill_q8_kernel(const __grid_constant__ Q8PrefillParams P) {
    const AttnParams &p = P.a;
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
    if (R0 >= T * G) return;   // uniform: no rows
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
        mbar_init(&bars[B_VCEMPTY], 2);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars[B_KFULL + i], 4);
            mbar_init(&bars[B_KEMPTY + i], 1);
            mbar_init(&bars[B_VFULL + i], 2);
            mbar_init(&bars[B_AFULL + i], 2);
            mbar_init(&bars[B_VEMPTY + i], 1);
        }
        for (int i = 0; i < kInfoStages; ++i) {
            mbar_init(&bars[B_IFULL + i], 1);
            mbar_init(&bars[B_IEMPTY + i], kInfoConsumers);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars[B_SFULL + t], 1);
            mbar_init(&bars[B_PFULL + t], 4);
            mbar_init(&bars[B_ODONE + t], 1);
        }
        mbar_init(&bars[B_QFULL], 1);
        mbar_init(&bars[B_DRAIN], 1);
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

    if (warp < 4) {
        const bool leader = tc::elect_one();
        if (warp == 0) {
            // ======================================================== table walk and code copies
            int j = 0, n_kc = 0, n_vc = 0;   // tiles, K and V copies issued
            bool ok = true;
            int n_v = 0;        // tile n_vc: its blocks, and this lane's block
            size_t bh_v = 0;
            auto load_v = [&]() {
                if (!warp_wait(&bars[B_VCEMPTY], (n_vc & 1) ^ 1, abort_flag, p.d_status)) return false;
                if (leader) mbar_arrive_expect_tx(&bars[B_VCFULL], n_v * kCodeBlock);
                __syncwarp();
                if (lane < n_v) bulk_load(sm + kOffVC + lane * kCodeBlock, P.v_codes + bh_v * kCodeBlock, kCodeBlock, &bars[B_VCFULL]);
                ++n_vc;
                return true;
            };
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
                // V one tile behind, so that the record of tile j never waits for the V of tile j - 2
                if (j > 0 && !(ok = load_v())) break;
                n_v = n;
                bh_v = bh;
                ++j;
                w += n;
            }
            if (ok && j > 0) ok = load_v();
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
            if (n_vc > 0) mbar_wait(&bars[B_VCFULL], (n_vc - 1) & 1);
        } else if (warp == 2) {
            // ======================================================== MMA issuer
            // Order: QK_0(0) QK_1(0) | PV_0(0) QK_0(1) | PV_1(0) QK_1(1) | PV_0(1) QK_0(2) | ...
            // One row tile's softmax runs while the tensor core works on the other's MMAs;
            // QK_t(j + 1) follows PV_t(j) in issue order, which is what lets P_t live in S_t.
            constexpr uint32_t idq = idesc_f16(false), idv = idesc_f16(true);
            const uint64_t dQ = tc::smem_desc(smem_u32(sm + kOffQ), 16, 1024), dK0 = tc::smem_desc(smem_u32(sm + kOffK), 16, 1024);
            const uint64_t dV0 = tc::smem_desc(smem_u32(sm + kOffV), kHalfPlane, 1024);
            auto qk = [&](int t, int stage) {
                const uint64_t qb = dQ + static_cast<uint64_t>((t * kTileBytes) >> 4);
                const uint64_t kb = dK0 + static_cast<uint64_t>((stage * kTileBytes) >> 4);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint64_t o = static_cast<uint64_t>(((kk >> 2) * kHalfPlane + (kk & 3) * 32) >> 4);
                    tc::mma_ss(tbase + 128 * t, qb + o, kb + o, idq, kk > 0 ? 1u : 0u);
                }
                tc::commit(&bars[B_SFULL + t]);
                if (t == 1) tc::commit(&bars[B_KEMPTY + stage]);
            };
            int n = 0;
            bool ok = warp_wait(&bars[B_QFULL], 0, abort_flag, p.d_status) && warp_wait(&bars[B_IFULL], 0, abort_flag, p.d_status);
            if (ok) {
                n = info[0].n;
                __syncwarp();
                if (leader) mbar_arrive(&bars[B_IEMPTY]);
                if (n > 0) {
                    ok = warp_wait(&bars[B_KFULL], 0, abort_flag, p.d_status);
                    tc::fence_after_sync();
                    if (ok && leader) {
                        qk(0, 0);
                        qk(1, 0);
                    }
                    __syncwarp();
                }
            }
            for (int j = 0; ok && n > 0; ++j) {
                const int is = (j + 1) % kInfoStages, ksn = (j + 1) % kStages, vs = j % kStages;
                if (!warp_wait(&bars[B_IFULL + is], ((j + 1) / kInfoStages) & 1, abort_flag, p.d_status)) break;
                const int n_next = info[is].n;
                __syncwarp();
                if (leader) mbar_arrive(&bars[B_IEMPTY + is]);
                if (n_next > 0 && !warp_wait(&bars[B_KFULL + ksn], ((j + 1) / kStages) & 1, abort_flag, p.d_status)) break;
                if (!warp_wait(&bars[B_VFULL + vs], (j / kStages) & 1, abort_flag, p.d_status)) break;
                const uint64_t vb = dV0 + static_cast<uint64_t>((vs * kTileBytes) >> 4);
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    ok = warp_wait(&bars[B_PFULL + t], j & 1, abort_flag, p.d_status);
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (leader) {
                        for (int k = 0; k < n; ++k)
                            tc::mma_ts(tbase + 256 + 128 * t, tbase + 128 * t + 8 * k,
                                       vb + static_cast<uint64_t>((k * kBoxBytes) >> 4), idv, (j > 0 || k > 0) ? 1u : 0u);
                        tc::commit(&bars[B_ODONE + t]);
                        if (t == 1) tc::commit(&bars[B_VEMPTY + vs]);
                        if (n_next > 0) qk(t, ksn);
                    }
                    __syncwarp();
                }
                n = n_next;
            }
            // every MMA has completed before tensor memory is freed
            if (leader) tc::commit(&bars[B_DRAIN]);
            __syncwarp();
            mbar_wait(&bars[B_DRAIN], 0);
        } else {
            // ======================================================== query tiles, angles, V codes (warps 1 and 3)
            if (warp == 3 && leader) {
                mbar_arrive_expect_tx(&bars[B_QFULL], 2 * kTileBytes);
                const uint16_t *q = p.q_prep + unit_rows(p, mt, kvh, r) * kHeadDim;
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    bulk_load(sm + kOffQ + t * kHalfPlane, q + t * (kHalfPlane / 2), kHalfPlane, &bars[B_QFULL]);
            }
            __syncwarp();
            const int pair = (warp == 3 ? 32 : 0) + lane;
            const double th = p.rope.theta[pair];
            int cur = INT_MIN;
            float c = 1.f, s = 0.f;
            // angles of tile j (this warp's 32 pairs) into table j & 1, free since the K of tile j - 2 is done;
            // returns the tile's blocks, -1 if a wait gave up
            auto angles = [&](int j) -> int {
                const int is = j % kInfoStages, st = j % kStages;
                if (!warp_wait(&bars[B_IFULL + is], (j / kInfoStages) & 1, abort_flag, p.d_status)) return -1;
                const int n = info[is].n, off = info[is].off;
                if (n == 0) return 0;
                if (off != cur) {
                    cur = off;
                    rope_cos_sin(off - Pbase, th, c, s);
                }
                if (!warp_wait(&bars[B_KFULL + st], ((j / kStages) & 1) ^ 1, abort_flag, p.d_status)) return -1;
                __half *tab = reinterpret_cast<__half *>(sm + kOffAngle + st * 256);
                tab[pair] = __float2half_rn(c);
                tab[kHalfDim + pair] = __float2half_rn(s);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_AFULL + st]);
                return n;
            };
            // V: thread (ch, rb) takes dims 16 ch .. + 15 of slots rb and rb + 8 of every block
            const int ch = lane & 7, rb = (lane >> 3) + (warp == 3 ? 4 : 0);
            const uint8_t *vc = sm + kOffVC + rb * kHeadDim + 16 * ch;
            const uint32_t vrow = (ch >> 2) * kHalfPlane + rb * 128;
            const uint32_t v0 = vrow + (((2 * (ch & 3)) ^ rb) << 4), v1 = vrow + (((2 * (ch & 3) + 1) ^ rb) << 4);
            int n = angles(0);
            for (int j = 0; n > 0; ++j) {
                const int is = j % kInfoStages, st = j % kStages;
                const int n_next = angles(j + 1);
                const TileInfo &ti = info[is];
                uint32_t keep = 0u;   // bit k, bit 8 + k: some row may see slot rb, rb + 8 of block k
#pragma unroll
                for (int k = 0; k < kTileBlocks; ++k) {
                    const int lim = min(meta_valid(ti.meta[k]), Plast - ti.off - meta_j0(ti.meta[k]) + 1);
                    keep |= (rb < lim ? 1u << k : 0u) | (rb + 8 < lim ? 256u << k : 0u);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_IEMPTY + is]);
                if (!warp_wait(&bars[B_VCFULL], j & 1, abort_flag, p.d_status)) break;
                if (!warp_wait(&bars[B_VEMPTY + st], ((j / kStages) & 1) ^ 1, abort_flag, p.d_status)) break;
                uint8_t *vt = sm + kOffV + st * kTileBytes;
                // blocks behind the tile's last hold old codes that no MMA reads
#pragma unroll
                for (int k0 = 0; k0 < kTileBlocks; k0 += 2) {
                    uint4 w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = *reinterpret_cast<const uint4 *>(vc + (k0 + (k >> 1)) * kCodeBlock + (k & 1) * 8 * kHeadDim);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (!((keep >> (k0 + (k >> 1) + 8 * (k & 1))) & 1u)) w[k] = make_uint4(0, 0, 0, 0);   // 0 * NaN
                        uint4 x, y;
                        codes_to_f16(w[k].x, x.x, x.y);
                        codes_to_f16(w[k].y, x.z, x.w);
                        codes_to_f16(w[k].z, y.x, y.y);
                        codes_to_f16(w[k].w, y.z, y.w);
                        uint8_t *vd = vt + (k0 + (k >> 1)) * kBoxBytes + (k & 1) * 1024;
                        *reinterpret_cast<uint4 *>(vd + v0) = x;
                        *reinterpret_cast<uint4 *>(vd + v1) = y;
                    }
                }
                fence_proxy_async_smem();   // generic writes become visible to the tensor core
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars[B_VCEMPTY]);
                    mbar_arrive(&bars[B_VFULL + st]);
                }
                n = n_next;
            }
            if (warp == 3) mbar_wait(&bars[B_QFULL], 0);   // landed before the kernel can end
        }
    } else if (warp < 12) {
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
        const uint32_t tS = tbase + 128 * t, tO = tbase + 256 + 128 * t;
        float m_run = -INFINITY, l_run = 0.f, mo = -INFINITY;
        int j = 0;
        bool ok = true;
        for (;; ++j) {
            const int is = j % kInfoStages;
            ok = warp_wait(&bars[B_IFULL + is], (j / kInfoStages) & 1, abort_flag, p.d_status);
            if (!ok) break;
            const TileInfo &ti = info[is];
            const int n = ti.n;
            if (n == 0) break;
            // visible keys of each block for this row, five bits per block
            uint64_t limp = 0;
            if (!ti.full) {
#pragma unroll
                for (int k = 0; k < kTileBlocks; ++k) {
                    const int nv = k < n ? meta_valid(ti.meta[k]) : 0;
                    limp |= static_cast<uint64_t>(max(0, min(nv, prow - ti.off - meta_j0(ti.meta[k]) + 1))) << (5 * k);
                }
            }
            ok = warp_wait(&bars[B_SFULL + t], j & 1, abort_flag, p.d_status);
            if (!ok) break;
            tc::fence_after_sync();
            // The row in two halves of 64 columns, first for its maxima and again for the weights: tensor
            // memory is read twice, but the loop is a quarter of the code of one over all 128 columns in
            // registers, whose instructions did not fit the cache beside the other roles'.
            uint32_t sv[64];
            auto f = [&](int c) { return __uint_as_float(sv[c]); };
            auto load = [&](int h) {
                tc::ld32(tS + lane_off + 64 * h, *reinterpret_cast<uint32_t(*)[32]>(sv));
                tc::ld32(tS + lane_off + 64 * h + 32, *reinterpret_cast<uint32_t(*)[32]>(sv + 32));
                tc::wait_ld();
                if (ALIBI) {
                    // scores with the in-block part of the bias; the block part joins the maxima and offsets
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float fk = ti.ks[4 * h + k] * hm;
#pragma unroll
                        for (int c = 16 * k; c < 16 * k + 16; ++c)
                            sv[c] = __float_as_uint(fmaf(f(c), fk, slope * static_cast<float>(c & 15)));
                    }
                }
                if (!ti.full) {
                    const uint32_t l4 = static_cast<uint32_t>(limp >> (20 * h));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int lim = static_cast<int>((l4 >> (5 * k)) & 31u);
#pragma unroll
                        for (int c = 16 * k; c < 16 * k + 16; ++c) sv[c] = (c & 15) < lim ? sv[c] : 0xFF800000u;
                    }
                }
            };
            // factor of a block's scores; at least the smallest normal number, so that -inf stays -inf
            auto factor = [&](int k) { return ALIBI ? 1.f : fmaxf(ti.ks[k] * hm, 0x1p-126f); };
            auto bias = [&](int k) { return ALIBI ? slope * static_cast<float>(ti.off + meta_j0(ti.meta[k]) - prow) : 0.f; };
            float m_new = m_run, mo_new = -INFINITY;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                load(h);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float a = max3(f(16 * k), f(16 * k + 1), f(16 * k + 2)), b = f(16 * k + 15);
#pragma unroll
                    for (int c = 3; c < 15; c += 4) {
                        a = max3(a, f(16 * k + c), f(16 * k + c + 1));
                        b = max3(b, f(16 * k + c + 2), f(16 * k + c + 3));
                    }
                    const float s = fmaf(fmaxf(a, b), factor(4 * h + k), bias(4 * h + k));
                    m_new = fmaxf(m_new, s);
                    mo_new = fmaxf(mo_new, s + ti.lv[4 * h + k]);
                }
            }
            const float mu = m_new == -INFINITY ? 0.f : m_new;
            if (m_new != m_run) {
                l_run *= fast_exp2(m_run - mu);
                m_run = m_new;
            }
            const bool need = mo_new > mo + kRescaleThreshold;
            float scale = 1.f;
            if (need) {
                scale = fast_exp2(mo - mo_new);
                mo = mo_new;
            }
            const float mou = mo == -INFINITY ? 0.f : mo;
            float ls0 = 0.f, ls1 = 0.f;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                load(h);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float fk = factor(4 * h + k), nm = bias(4 * h + k) - mu;
                    const float F = fast_exp2(fminf(mu + ti.lv[4 * h + k] - mou, 126.f));
#pragma unroll
                    for (int e = 8 * k; e < 8 * k + 8; ++e) {
                        float x0, x1;
                        fma2v(x0, x1, f(2 * e), f(2 * e + 1), fk, fk, nm, nm);
                        float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                        add2(ls0, ls1, p0, p1);
                        mul2(p0, p1, p0, p1, F, F);
                        sv[e] = pack_h2(p0, p1);
                    }
                }
                // P over columns of S that have been read
                tc::st32(tS + lane_off + 32 * h, *reinterpret_cast<uint32_t(*)[32]>(sv));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_IEMPTY + is]);
            l_run += ls0 + ls1;
            if (j > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[32];
                    tc::ld32(tO + lane_off + 32 * c, o);
                    tc::wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * scale);
                    tc::st32(tO + lane_off + 32 * c, o);
                }
            }
            tc::wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_PFULL + t]);
        }
        // ------------------------------------------------------------ epilogue: O 2^(mo - m) / l
        bool have = ok && j > 0;
        if (have) have = warp_wait(&bars[B_ODONE + t], (j - 1) & 1, abort_flag, p.d_status);
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
                tc::ld32(tO + lane_off + 32 * c, ob);
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
    } else {
        // ============================================================ K codes to rotated f16 tiles
        // thread (ch, rb): pairs 8 ch .. + 7 of slot rb of every block.  (a, b) -> (a c - b s, b c + a s) in f16
        const int tid = threadIdx.x - 384;
        const int ch = tid & 7, rb = tid >> 3;
        const uint8_t *kc = sm + kOffKC + rb * kHeadDim + 8 * ch;
        const uint32_t ksw = rb * 128 + ((ch ^ (rb & 7)) << 4);
        for (int j = 0;; ++j) {
            const int is = j % kInfoStages, st = j % kStages;
            if (!warp_wait(&bars[B_IFULL + is], (j / kInfoStages) & 1, abort_flag, p.d_status)) break;
            const int n = info[is].n;
            if (n == 0) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_IEMPTY + is]);
            if (!warp_wait(&bars[B_AFULL + st], (j / kStages) & 1, abort_flag, p.d_status)) break;
            const uint4 c4 = *reinterpret_cast<const uint4 *>(sm + kOffAngle + st * 256 + 16 * ch);
            const uint4 s4 = *reinterpret_cast<const uint4 *>(sm + kOffAngle + st * 256 + 128 + 16 * ch);
            const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
            if (!warp_wait(&bars[B_KCFULL], j & 1, abort_flag, p.d_status)) break;
            if (!warp_wait(&bars[B_KEMPTY + st], ((j / kStages) & 1) ^ 1, abort_flag, p.d_status)) break;
            uint8_t *kt = sm + kOffK + st * kTileBytes;
            // all 8 blocks (those behind the tile's last hold old codes, whose scores are masked), loads
            // ahead of the stores they could otherwise not pass
#pragma unroll
            for (int k0 = 0; k0 < kTileBlocks; k0 += 4) {
                uint2 lo[4], hi[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    lo[k] = *reinterpret_cast<const uint2 *>(kc + (k0 + k) * kCodeBlock);
                    hi[k] = *reinterpret_cast<const uint2 *>(kc + (k0 + k) * kCodeBlock + kHalfDim);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t a[4], b[4], ol[4], oh[4];
                    codes_to_f16(lo[k].x, a[0], a[1]);
                    codes_to_f16(lo[k].y, a[2], a[3]);
                    codes_to_f16(hi[k].x, b[0], b[1]);
                    codes_to_f16(hi[k].y, b[2], b[3]);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        ol[x] = h2_fma(b[x], s[x] ^ 0x80008000u, h2_mul(a[x], c[x]));
                        oh[x] = h2_fma(a[x], s[x], h2_mul(b[x], c[x]));
                    }
                    uint8_t *kd = kt + (k0 + k) * kBoxBytes + ksw;
                    *reinterpret_cast<uint4 *>(kd) = make_uint4(ol[0], ol[1], ol[2], ol[3]);
                    *reinterpret_cast<uint4 *>(kd + kHalfPlane) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars[B_KCEMPTY]);
                mbar_arrive(&bars[B_KFULL + st]);
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
    if (mt >= p.pf_mtiles || mt * kRows >= T * G) return;   // uniform for the 16 rows of the block
    const bool live = R < T * G;
    const int tok = live ? R / G : 0, g = R % G;
    float cs[4], sn[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) rope_cos_sin(live ? tok - (mt * kRows) / G : 0, p.rope.theta[4 * c + u], cs[u], sn[u]);
    // byte offset of dims 4 c .. + 3 of this row in its half plane
    const uint32_t at = (row / kTileRows) * kTileBytes + (row % kTileRows) * 128 + (((c >> 1) ^ (row & 7)) << 4) + (c & 1) * 8;
    for (int kvh = 0; kvh < p.hkv; ++kvh) {
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
        // q 2^-e in [1, 2); e = 0 for an all-zero or non-finite row
        int e = static_cast<int>(__float_as_uint(am) >> 23) - 127;
        e = (am == 0.f || e == 128) ? 0 : max(-126, min(126, e));
        const float dn = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
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

template <bool ALIBI>
cudaError_t launch_t(const Q8PrefillParams &p, cudaStream_t s) {
    auto kern = prefill_q8_kernel<ALIBI>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    prefill_q8_query_kernel<<<dim3(p.a.pf_mtiles * (kRows / 16), p.a.num_req), 256, 0, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    kern<<<p.a.pf_base + p.parts * p.a.pf_nsplit, kThreads, kSmem, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.a.pf_nsplit == 0) return e;
    prefill_q8_join_kernel<<<dim3(p.a.pf_nsplit, kRows / 8), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

Q8PrefillPlan q8_prefill_plan(int64_t units, int max_words, int sms) {
    // Units of a last wave that leaves at least half of the SMs idle are split over their words, at
    // least two tiles a part.
    Q8PrefillPlan pl = {0, 1};
    if (units <= 0 || sms <= 0) return pl;
    const int64_t rem = units % sms;
    if (rem == 0 || 2 * rem > sms) return pl;
    const int64_t parts = std::min<int64_t>(std::min<int64_t>(sms / rem, 16), (max_words + 2 * kTileBlocks - 1) / (2 * kTileBlocks));
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

cudaError_t launch_prefill_q8(Q8PrefillParams &p, void *workspace, int64_t units, int sms, cudaStream_t s) {
    const Q8PrefillPlan pl = q8_prefill_plan(units, p.a.max_words, sms);
    p.parts = pl.parts;
    p.a.pf_nsplit = pl.nsplit;
    p.a.pf_base = static_cast<int>(units) - pl.nsplit;
    p.a.q_prep = static_cast<uint16_t *>(workspace);
    p.a.ws_acc = reinterpret_cast<float *>(p.a.q_prep + units * kRows * kHeadDim);
    p.a.ws_ml = p.a.ws_acc + (pl.nsplit ? static_cast<size_t>(pl.nsplit) * pl.parts * kRows * kHeadDim : 0);
    p.row_scale = p.a.ws_ml + (pl.nsplit ? static_cast<size_t>(pl.nsplit) * pl.parts * kRows * 2 : 0);
    return p.a.alibi ? launch_t<true>(p, s) : launch_t<false>(p, s);
}

}  // namespace lazy

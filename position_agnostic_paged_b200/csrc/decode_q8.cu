// decode_q8.cu -- decode attention over the 8-bit pool on tcgen05 tensor cores, codes used as they are.
//
// Per request, query head h on KV head k, key t (code k_t, v_t) of a block with scales s_k, s_v, table
// offset o, local index j and position o + j <= p (the query's):
//   s_t = scale s_k q_h^T R(-(p - o)) k_t,   w_t = 2^(s_t - M) / L,   out = sum_t w_t s_v v_t,
//   block_mass[word] += sum_h sum_{t in word} w_t.
//
// Both products take e4m3 operands (kind::f8f6f4), so no code is ever converted.  The other operand, a
// rotated query or a weight x <= 448, becomes a sum of e4m3 parts with steps of 2^-4 (e4m3 rounds to 2^-4 of
// a value, so 2^4 times the rest is at most 256):
//   x = x_0 + 2^-4 x_1 + 2^-8 x_2,   x_0 = e4m3(x), x_1 = e4m3(2^4 (x - x_0)), x_2 = e4m3(2^4 (...)):
// three parts (the query, its largest element at least 128) are off by 2^-6 at most, 2^-13 of 128 (f16 would keep
// 2^-11); four (the weights) by 2^-11, and reach down to 2^-21.  Each
// part is a row group of the B operand with accumulator columns of its own; the sum is taken in fp32
// when they are read.  With block mass, whose fp32 sums are the result, the query has five parts (2^-16, fp32's own
// rounding of such numbers).
//
//   S^T [128 keys][parts x heads] = K [128 keys][128] Q^T      A: the K codes of 8 words as they lie in the pool
//   O^T [128 dims][parts x heads] += V^T [128 dims][keys] P^T  A: the V codes, keys as rows (MN-major)
//
// A block's K scale multiplies the scores of its 16 lanes of S^T; its V scale joins the weights.
//
// Work split.  The words of all requests lie one after the other in `table`, so for one KV head they
// form one line; it is cut into equal pieces, one per resident CTA: ragged batches balance by
// themselves and no request waits for the longest.  Where a request ends inside a piece the CTA writes a
// partial result (m, l, acc) to workspace slot (piece + request), unique because each new partial moves
// on to the next piece or the next request.  A second kernel joins a request's partials in order.
//
// A CTA takes up to 16 query rows of a KV head; a wider group of heads is taken by neighbouring CTAs, two per
// SM, whose barriers and waits overlap (32 heads on one KV head with block mass, with the operand's rows as they were
// before kKeyRows: one CTA of 32 rows 136 us, two of 16 131).  A prefill of a few tokens runs here too, its rows (token, head) pairs: 128 keys cost a CTA of the
// prefill's kernel about 3 us however few its rows, here under 2.
//
// Warps: four per group of 8 query rows (or 4) for the softmax (thread t of a group: key t of the tile, later
// head dim t), one for the table walk and the TMA loads, one for MMA issue.  A tile is up to 8 words of one
// request with one offset; K and V of a tile (32 KiB) share a stage.  Scores are double-buffered; QK of tile
// i + 1 runs under the weights of tile i.  (Making tile i + 1's query before the scores of tile i, to run QK
// under all of it: 107 -> 111 us; with block mass and 32 heads, before kKeyRows, 131 -> 137.)
//
// What bounds it: HBM for long tables with few rows (64 requests of 4161 tokens, 32 heads on 8: 548 MB in 106 us
// with the joining kernel, 5.2 TB/s, 79 % of the copy rate), the chain of a tile (scores, references, weights'
// parts, about 1900 cycles with 4 rows) and its instructions where rows are many (32 heads with block mass:
// 118 us, 56 % of issue slots).
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

constexpr int kTileWords = 8;
constexpr int kCodeBlock = kBlockTokens * kHeadDim;              // codes of one block of one head
constexpr int kHalfStage = kTileWords * kCodeBlock, kStageBytes = 2 * kHalfStage;
constexpr int kRecords = 4;
// A reference is set kMargin above the largest score seen, and moves when a score passes it by kSlack (log2
// units): weights times 2^7 stay below 448, the largest is 2^2 or more, and few tiles move a reference
// (32 heads, margin 3 against 5: up to 15 against 4 of 38 tiles, 3 us each).  Four parts of the weights reach
// down to 2^-23 of the largest.
constexpr float kSlack = 1.75f, kMargin = 5.f;
constexpr float kPartStep = 16.f;     // between parts
constexpr int kPP = 4;                // parts of the weights

// One tile of the walk; n = 0 ends it.
struct Tile {
    int n, off, req, word;            // words, offset, request, index of the first word in the request
    int rows, qpos;                   // query rows of the request here; position of its first query
    int lim[kTileWords];              // visible slots of each word
    int pos[kTileWords];              // position of its slot 0
    float ks[kTileWords], vs[kTileWords];
};

constexpr int kCtaRows = 16;         // query rows of a CTA
// CTAs that share a KV head's query rows.
__host__ __device__ inline int row_groups(int rows) { return (rows + kCtaRows - 1) / kCtaRows; }

// NG: query heads of a CTA, rounded up to 4, 8 or 16.  QP: parts of the query.
template <int NG, int QP>
struct Cfg {
    static constexpr int kHT = NG < 8 ? NG : 8, kGroups = NG / kHT;          // heads per softmax thread, groups of 128 threads
    static constexpr int kSoft = 128 * kGroups, kThreads = kSoft + 64;
    static constexpr int kQRows = QP * NG, kQN = (kQRows + 15) / 16 * 16;    // rows of the Q operand, N of the S product
    static constexpr int kPRows = kPP * NG, kPN = (kPRows + 15) / 16 * 16;
    // The P operand: keys as rows of kPN bytes (MN-major), which a thread writes eight heads at a time; with 4
    // heads too narrow for that, rows of 128 keys (K-major), a byte per store (32 heads on one KV head with block mass: 131 us
    // with it, 117 without)
    static constexpr bool kKeyRows = NG >= 8;
    static constexpr int kQBytes = (kQN + 7) / 8 * 1024, kPBytes = (kPN + 7) / 8 * 1024;
    static constexpr int kFixed = 2 * kQBytes + 2 * kPBytes + 4096 + 1024;   // buffers, small state, alignment
    static constexpr int kOcc = 2 * (kFixed + 2 * kStageBytes + 1024) <= 227 * 1024 ? 2 : 1;
    static constexpr int kStages0 = (227 * 1024 / kOcc - 1024 - kFixed) / kStageBytes;
    static constexpr int kStages = kStages0 > 4 ? 4 : kStages0;
    static constexpr int kSmem = kFixed + kStages * kStageBytes;
    static constexpr int kCols0 = 2 * kQN + kPN;
    static constexpr int kCols = kCols0 <= 64 ? 64 : kCols0 <= 128 ? 128 : kCols0 <= 256 ? 256 : 512;   // tensor memory
    static_assert(!kKeyRows || kPN == 32 || kPN == 64, "swizzle");
    static_assert(kStages >= 2 && kOcc * kCols <= 512 && kSoft / 16 >= NG, "resources");
    // shared memory, from a 1 KiB boundary
    static constexpr int kOffQ = kStages * kStageBytes, kOffP = kOffQ + 2 * kQBytes, kOffState = kOffP + 2 * kPBytes;
};
// small state, from kOffState
constexpr int kOffTile = 0;                                      // records
constexpr int kOffBars = kOffTile + kRecords * static_cast<int>(sizeof(Tile));
constexpr int kOffHead = kOffBars + 256;                         // mu, dm, step of O, hm of two Q buffers, slope, token: [32] each
constexpr int kOffRed = kOffHead + 7 * 128;                      // [2][4][32] reductions
constexpr int kOffAngle = kOffRed + 1024;                        // [64] float2, or [64] double
constexpr int kOffMisc = kOffAngle + 512;
static_assert(kOffMisc + 16 <= 4096, "state");

// kind::f8f6f4 with e4m3 A/B and fp32 accumulation, M = 128.
constexpr uint32_t idesc_e4m3(int n, bool a_mn_major, bool b_mn_major) {
    return (1u << 4) | (a_mn_major ? (1u << 15) : 0u) | (b_mn_major ? (1u << 16) : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t *r) {
    static_assert(N == 4 || N == 8, "columns");
    if constexpr (N == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(taddr));
}
__device__ __forceinline__ void tmem_store4(uint32_t taddr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *d_status) {
    return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, d_status));
}
__device__ __forceinline__ float log2_of(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// the softmax warps
template <int N>
__device__ __forceinline__ void sync_softmax() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(N) : "memory"); }
template <int N>
__device__ __forceinline__ bool any_softmax(bool x) {
    uint32_t y;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(y)
                 : "r"(x ? 1u : 0u), "n"(N)
                 : "memory");
    return y != 0;
}
// maximum over the warp (NaN ignored)
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
// Four values as the codes of their next part, each value replaced by 2^4 times what is left of it.
__device__ __forceinline__ uint32_t take_part(float (&x)[4]) {
    const uint32_t w = f32_to_codes(x[0], x[1], x[2], x[3]);
    uint32_t h0, h1;
    float y[4];
    codes_to_f16(w, h0, h1);
    f16x2_to_f32(h0, y[0], y[1]);
    f16x2_to_f32(h1, y[2], y[3]);
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        mul2(x[i], x[i + 1], x[i], x[i + 1], kPartStep, kPartStep);
        fma2v(x[i], x[i + 1], y[i], y[i + 1], -kPartStep, -kPartStep, x[i], x[i + 1]);
    }
    return w;
}
// byte offset of column `col` of row `row` in an operand of 128-byte rows, 128-byte swizzled
__device__ __forceinline__ uint32_t swz8(int row, int col) {
    return row * 128 + (((col >> 4) ^ (row & 7)) << 4) + (col & 15);
}
// Words per piece: the same on both kernels.
__device__ __forceinline__ int words_per_piece(int total, int pieces) {
    return max(kLineMinWordsQ8, (total + pieces - 1) / pieces);
}

// CHUNK: a row is a (token, head of the group) pair of a request's few tokens, with a position and visible keys
// of its own, else one of the request's one token's heads.
template <int NG, int QP, bool MASS, bool CHUNK>
__global__ void __launch_bounds__((Cfg<NG, QP>::kThreads), (Cfg<NG, QP>::kOcc)) decode_q8_kernel(const __grid_constant__ CUtensorMap tmK,
                                                                                  const __grid_constant__ CUtensorMap tmV,
                                                                                  const __grid_constant__ LaneParams p) {
    using C = Cfg<NG, QP>;
    pdl_trigger();   // (one wave of CTAs: the join's do not take places from this kernel's)
    constexpr int S = C::kStages, HT = C::kHT, kWalk = C::kSoft / 32, kIssue = kWalk + 1;   // warps
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *state = sm + C::kOffState;
    Tile *tiles = reinterpret_cast<Tile *>(state + kOffTile);
    uint64_t *bars = reinterpret_cast<uint64_t *>(state + kOffBars);
    uint64_t *full = bars, *empty = bars + 4, *ifull = bars + 8, *iempty = bars + 12, *qready = bars + 16, *sfull = bars + 18,
             *pready = bars + 20, *odone = bars + 22, *drain = bars + 24;
    float *h_mu = reinterpret_cast<float *>(state + kOffHead), *h_dm = h_mu + 32, *h_step = h_mu + 64,
          *h_hm = h_mu + 96, *h_slope = h_mu + 160, *h_tok = h_mu + 192;
    float(*red)[32] = reinterpret_cast<float(*)[32]>(state + kOffRed), (*red_o)[32] = red + 4;
    float2 *angle = reinterpret_cast<float2 *>(state + kOffAngle);
    double *theta = reinterpret_cast<double *>(state + kOffAngle);   // CHUNK
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(state + kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(state + kOffMisc + 4);

    const AttnParams &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hkv = a.hkv, B = a.num_req;
    // neighbouring CTAs take the row groups of one KV head: its words come from L2 for all but the first
    const int groups = row_groups(p.rows), wi = blockIdx.x / (hkv * groups), line = blockIdx.x - wi * hkv * groups;
    const int kvh = line / groups, hg = kCtaRows * (line - kvh * groups);   // hg: the first row here
    // rows of request r here
    auto rows_of = [&](int r) {
        if (!CHUNK) return min(kCtaRows, a.group - hg);
        const int tokens = max(0, min(a.cu_q[r + 1] - a.cu_q[r], a.max_q));
        return max(0, min(kCtaRows, tokens * a.group - hg));
    };
    const int base = a.table_indptr[0];
    const int total = a.table_indptr[B] - base;
    if (total <= 0) return;
    const int per = words_per_piece(total, p.pieces);
    if (wi > (total - 1) / per) return;
    const int lo = wi * per, cnt = min(total - lo, per);

    // the walk's first loads, while the others set up: the request of the first word (the largest r with
    // table_indptr[r] <= its index), its bounds, and 32 words, one per lane
    int r = 0, r_beg = 0, r_end = 0;
    uint32_t wl = 0u;
    if (warp == kWalk) {
        if (lane < cnt) wl = a.table[base + lo + lane];
        int hi = B;
        while (hi - r > 1) {
            const int step = (hi - r + 31) >> 5, x = r + step * lane;
            const bool below = x < hi && a.table_indptr[x] - base <= lo;
            const int k = __popc(__ballot_sync(0xffffffffu, below)) - 1;
            r += step * k;
            hi = min(hi, r + step);
        }
        r_beg = a.table_indptr[r] - base;
        r_end = a.table_indptr[r + 1] - base;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kRecords; ++i) {
            mbar_init(&ifull[i], 1);
            mbar_init(&iempty[i], kWalk + 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qready[i], kWalk);
            mbar_init(&sfull[i], 1);
            mbar_init(&pready[i], kWalk);
            mbar_init(&odone[i], 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    // rows of the operands that hold no head stay zero
    for (int i = threadIdx.x; i < (2 * C::kQBytes + 2 * C::kPBytes) / 16; i += C::kThreads)
        reinterpret_cast<uint4 *>(sm + C::kOffQ)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x < 32) {
        const int row = hg + threadIdx.x, tok = CHUNK ? row / a.group : 0;
        if (a.alibi) h_slope[threadIdx.x] = row < p.rows ? a.alibi_log2[kvh * a.group + row - tok * a.group] : 0.f;
        if (CHUNK) h_tok[threadIdx.x] = static_cast<float>(tok);
    }
    if (CHUNK)
        for (int i = threadIdx.x; i < kHalfDim; i += C::kThreads) theta[i] = a.rope.theta[i];
    if (warp == kIssue) {
        tc::tmem_alloc(tmem_slot, C::kCols);
        tc::tmem_relinquish();
    }
    fence_proxy_async_smem();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = *tmem_slot;
    const uint32_t tO = tbase + 2 * C::kQN;

    if (warp == kWalk) {
        // ============================================================ table walk and loads
        const bool leader = tc::elect_one();
        if (leader) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        int rows, qpos, last;     // of the request: rows here, positions of its first and last query
        int j = 0, first = 0;     // tiles; the first tile of the request
        bool ok = true;
        auto enter = [&]() {
            rows = rows_of(r);
            qpos = CHUNK ? a.q_pos0[r] : a.q_pos[r];
            last = !CHUNK ? qpos : rows > 0 ? qpos + (hg + rows - 1) / a.group : -1;
            if (lo <= r_beg && r_end - r_beg > a.max_words && line == 0 && lane == 0) set_status(a.d_status, LAZY_DSTATUS_BAD_TABLE);
        };
        // a request none of whose words here is visible has no tile to write its partial result
        auto leave = [&]() {
            if (j == first && lane < rows)
                p.ws_ml[((static_cast<size_t>(kvh) * (p.pieces + B)) + wi + r) * p.rows + hg + lane] =
                    make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
            first = j;
        };
        enter();
        uint32_t ml = 0u;
        float ksl = 1.f, vsl = 1.f;
        int b0 = INT_MIN / 2;
        for (int k = 0; k < cnt;) {
            if (lo + k >= r_end) {
                leave();
                do {
                    ++r;
                    r_beg = r_end;
                    r_end = a.table_indptr[r + 1] - base;
                } while (lo + k >= r_end);
                enter();
            }
            if (k - b0 + kTileWords > 32 && b0 + 32 < cnt) {
                // 32 words, one per lane, with their blocks' metadata and scales
                b0 = k;
                ml = 0u;
                if (k > 0) wl = k + lane < cnt ? a.table[base + lo + k + lane] : 0u;
                if (k + lane < cnt) {
                    const uint32_t b = word_block(wl);
                    if (b < static_cast<uint32_t>(a.num_blocks)) {
                        const size_t bh = static_cast<size_t>(b) * hkv + kvh;
                        ml = a.blk_meta[b];
                        ksl = p.k_scale[bh];
                        vsl = p.v_scale[bh];
                    } else {
                        set_status(a.d_status, LAZY_DSTATUS_BAD_BLOCK);
                    }
                }
            }
            const int i = k - b0, x = b0 + lane;             // lane `lane` holds word x
            const int pos = word_offset(wl) + meta_j0(ml);
            const bool mine = x >= k && x < cnt && lo + x < r_end;
            const int lim = mine && lo + x - r_beg < a.max_words ? seen_slots(meta_valid(ml), last, pos) : 0;
            const uint32_t seen = __ballot_sync(0xffffffffu, lim > 0);
            const int here = __popc(__ballot_sync(0xffffffffu, mine));      // words of the request from k on, in this batch
            if (!((seen >> i) & 1u)) {
                const int skip = min(here, seen ? __ffs(seen) - 1 - i : 32);
                if (MASS)
                    for (int y = k; y < k + skip; ++y)
                        if (lo + y - r_beg < a.max_words && lane < rows)
                            p.ws_lse[(static_cast<size_t>(r) * a.max_words + lo + y - r_beg) * a.hq + kvh * a.group + hg + lane] = -INFINITY;
                k += skip;
                continue;
            }
            const int src = (i + lane) & 31;
            const uint32_t wk = __shfl_sync(0xffffffffu, wl, src);
            const int lim_k = __shfl_sync(0xffffffffu, lim, src), pos_k = __shfl_sync(0xffffffffu, pos, src);
            const float ks = __shfl_sync(0xffffffffu, ksl, src), vs = __shfl_sync(0xffffffffu, vsl, src);
            const int off = word_offset(__shfl_sync(0xffffffffu, wl, i));
            const bool same = lane < kTileWords && i + lane < 32 && lim_k > 0 && (a.alibi || word_offset(wk) == off);
            const int n = __ffs(~__ballot_sync(0xffffffffu, same)) - 1;
            const int is = j % kRecords, st = j % S;
            ok = warp_wait(&iempty[is], ((j / kRecords) & 1) ^ 1, abort_flag, a.d_status);
            if (!ok) break;
            Tile &t = tiles[is];
            if (lane < kTileWords) {
                t.lim[lane] = lane < n ? lim_k : 0;
                t.pos[lane] = lane < n ? pos_k : 0;
                t.ks[lane] = lane < n ? ks : 1.f;
                t.vs[lane] = lane < n ? vs : 1.f;
            }
            if (leader) {
                t.n = n;
                t.off = off;
                t.req = r;
                t.rows = rows;
                t.qpos = qpos;
                t.word = lo + k - r_beg;
            }
            __syncwarp();
            if (leader) mbar_arrive(&ifull[is]);
            ok = warp_wait(&empty[st], ((j / S) & 1) ^ 1, abort_flag, a.d_status);
            if (!ok) break;
            if (leader) mbar_arrive_expect_tx(&full[st], n * 2 * kCodeBlock);
            __syncwarp();
            if (lane < n) {
                const int row = (static_cast<int>(word_block(wk)) * hkv + kvh) * kBlockTokens;
                uint8_t *d = sm + st * kStageBytes + lane * kCodeBlock;
                tma_load_2d(d, &tmK, 0, row, &full[st]);
                tma_load_2d(d + kHalfStage, &tmV, 0, row, &full[st]);
            }
            __syncwarp();
            ++j;
            k += n;
        }
        if (ok) {
            leave();
            const int is = j % kRecords;
            if (warp_wait(&iempty[is], ((j / kRecords) & 1) ^ 1, abort_flag, a.d_status)) {
                if (leader) {
                    tiles[is].n = 0;
                    mbar_arrive(&ifull[is]);
                }
                __syncwarp();
            }
        }
        // every copy lands before the kernel can end, whatever stopped the walk
        for (int i = max(0, j - S); i < j; ++i) mbar_wait(&full[i % S], (i / S) & 1);
    } else if (warp == kIssue) {
        // ============================================================ MMA issue
        //   QK(0) | QK(1) PV(0) | QK(2) PV(1) | ...; PV(i) goes first where tile i + 1 has not landed
        const bool leader = tc::elect_one();
        constexpr uint32_t idq = idesc_e4m3(C::kQN, false, false), idp = idesc_e4m3(C::kPN, true, C::kKeyRows);
        const uint64_t dA = tc::smem_desc(smem_u32(sm), 16, 1024);
        const uint64_t dQ = tc::smem_desc(smem_u32(sm + C::kOffQ), 16, 1024), dP0 = tc::smem_desc(smem_u32(sm + C::kOffP), 16, C::kKeyRows ? 8 * C::kPN : 1024);
        // rows of 64 bytes: 64-byte swizzle (4), of 32 bytes: 32-byte swizzle (6), in place of 128-byte (2)
        const uint64_t dP = C::kKeyRows ? (dP0 & ~(7ull << 61)) | (C::kPN == 64 ? 4ull : 6ull) << 61 : dP0;
        constexpr int kPStep = (C::kKeyRows ? 32 * C::kPN : 32) >> 4;   // 32 keys
        bool ok = true;
        int off = 0, req = -1, qbuf = 1;       // of the tile whose QK was issued last
        // record of tile i: words, and whether it opens a request
        auto read = [&](int i, int &n, bool &opens) {
            const int is = i % kRecords;
            ok = warp_wait(&ifull[is], (i / kRecords) & 1, abort_flag, a.d_status);
            n = ok ? tiles[is].n : 0;
            if (n > 0) {
                const int o = tiles[is].off, q = tiles[is].req;
                opens = q != req;
                if (opens || (o != off && !a.alibi)) qbuf ^= 1;   // the softmax warps count the same changes
                off = o;
                req = q;
            }
            __syncwarp();
            if (leader) mbar_arrive(&iempty[is]);
        };
        auto qk = [&](int i) {
            const int st = i % S;
            if (!warp_wait(&full[st], (i / S) & 1, abort_flag, a.d_status) ||
                !warp_wait(&qready[i & 1], (i >> 1) & 1, abort_flag, a.d_status)) {
                ok = false;
                return;
            }
            tc::fence_after_sync();
            if (leader) {
                const uint64_t ka = dA + static_cast<uint64_t>((st * kStageBytes) >> 4);
                const uint64_t qb = dQ + static_cast<uint64_t>((qbuf * C::kQBytes) >> 4);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    mma_e4m3(tbase + (i & 1) * C::kQN, ka + 2 * s, qb + 2 * s, idq, s > 0 ? 1u : 0u);
                tc::commit(&sfull[i & 1]);
            }
            __syncwarp();
        };
        int n = 0, n1 = 0;
        bool opens = true, opens1 = true;
        read(0, n, opens);
        if (n > 0) qk(0);
        for (int i = 0; ok && n > 0; ++i) {
            read(i + 1, n1, opens1);
            if (!ok) break;
            const bool early = n1 > 0 && __all_sync(0xffffffffu, mbar_test_wait(&full[(i + 1) % S], ((i + 1) / S) & 1));
            if (early) {
                qk(i + 1);
                if (!ok) break;
            }
            if (!warp_wait(&pready[i & 1], (i >> 1) & 1, abort_flag, a.d_status)) break;
            tc::fence_after_sync();
            if (leader) {
                const int st = i % S;
                const uint64_t va = dA + static_cast<uint64_t>((st * kStageBytes + kHalfStage) >> 4);
                const uint64_t pb = dP + static_cast<uint64_t>(((i & 1) * C::kPBytes) >> 4);
                for (int s = 0; 2 * s < n; ++s)
                    mma_e4m3(tO, va + static_cast<uint64_t>((s * 32 * 128) >> 4), pb + kPStep * s, idp, (opens && s == 0) ? 0u : 1u);
                tc::commit(&empty[st]);
                tc::commit(&odone[i & 1]);
            }
            __syncwarp();
            if (n1 > 0 && !early) qk(i + 1);
            n = n1;
            opens = opens1;
        }
        if (leader) tc::commit(drain);
        __syncwarp();
        mbar_wait(drain, 0);
    } else {
        // ============================================================ softmax
        const int t = threadIdx.x & 127, wq = warp & 3;   // key of the tile, later head dim; warp of the group
        const int g0 = (threadIdx.x >> 7) * HT;           // first head of this thread
        const uint32_t lane_off = static_cast<uint32_t>(32 * wq) << 16;
        // (read once: a per-lane read of the parameter table takes 32 turns)
        const double my_theta = !CHUNK && threadIdx.x < kHalfDim ? a.rope.theta[threadIdx.x] : 0.0;
        float l[HT];
        int qbuf = 1, cur_req = -1, cur_off = 0;   // of the Q operand made last
        // the query of tile `tl` as e4m3 parts, if it is not the one made last
        auto query = [&](const Tile &tl) {
            const int off = tl.off, r = tl.req, rows = tl.rows;
            if (r == cur_req && (off == cur_off || a.alibi)) return;
            qbuf ^= 1;
            cur_req = r;
            cur_off = off;
            // 16 threads per row: dims 4c .. + 3 and 64 above
            const int c = threadIdx.x & 15, h = threadIdx.x >> 4;
            const int tok = CHUNK ? (hg + h) / a.group : 0, head = kvh * a.group + hg + h - tok * a.group;
            uint2 lo2 = make_uint2(0u, 0u), hi2 = lo2;
            if (h < rows) {
                const uint2 *q = reinterpret_cast<const uint2 *>(
                    a.q_raw + (static_cast<size_t>(CHUNK ? a.cu_q[r] + tok : r) * a.hq + head) * kHeadDim);
                lo2 = __ldg(q + c);
                hi2 = __ldg(q + 16 + c);
            }
            if (!CHUNK) {
                if (threadIdx.x < kHalfDim)
                    rope_cos_sin(a.alibi ? 0 : tl.qpos - off, my_theta, angle[threadIdx.x].x, angle[threadIdx.x].y);
                sync_softmax<C::kSoft>();
            }
            uint8_t *qd = sm + C::kOffQ + qbuf * C::kQBytes;
            const float av[4] = {bf16_lo(lo2.x), bf16_hi(lo2.x), bf16_lo(lo2.y), bf16_hi(lo2.y)};
            const float bv[4] = {bf16_lo(hi2.x), bf16_hi(hi2.x), bf16_lo(hi2.y), bf16_hi(hi2.y)};
            float am = 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u) am = fmaxf(am, fmaxf(fabsf(av[u]), fabsf(bv[u])));
#pragma unroll
            for (int x = 1; x < 16; x <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, x));
            // largest element in [128, 256): a rotation keeps it below 363; e = 0 for an all-zero head.  A head with an
            // infinite element becomes NaN (codes have no infinity, its parts would be finite).
            const bool inf = am > FLT_MAX;
            int e = static_cast<int>(__float_as_uint(am) >> 23) - 127;
            e = (am == 0.f || inf) ? 0 : max(-119, e);
            const float dn = inf ? NAN : __uint_as_float(static_cast<uint32_t>(134 - e) << 23);   // 2^(7 - e)
            float x[4], y[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float2 z;
                if (CHUNK)
                    rope_cos_sin(a.alibi ? 0 : tl.qpos + tok - off, theta[4 * c + u], z.x, z.y);
                else
                    z = angle[4 * c + u];
                const float xa = av[u] * dn, xb = bv[u] * dn;
                x[u] = xa * z.x - xb * z.y;
                y[u] = xb * z.x + xa * z.y;
            }
            if (h < rows) {
#pragma unroll
                for (int part = 0; part < QP; ++part) {
                    const int row = part * NG + h;
                    *reinterpret_cast<uint32_t *>(qd + swz8(row, 4 * c)) = take_part(x);
                    *reinterpret_cast<uint32_t *>(qd + swz8(row, 64 + 4 * c)) = take_part(y);
                }
                if (c == 0) h_hm[32 * qbuf + h] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * (a.scale_log2 * 0x1p-7f);
            }
            if (threadIdx.x >= rows && threadIdx.x < 32) h_hm[32 * qbuf + threadIdx.x] = 0.f;
            fence_proxy_async_smem();
            sync_softmax<C::kSoft>();   // hm and the angles' next use
        };
        auto open = [&]() {
#pragma unroll
            for (int h = 0; h < HT; ++h) l[h] = 0.f;
            if (threadIdx.x < 32) {
                h_mu[threadIdx.x] = 0.f;
                h_dm[threadIdx.x] = INFINITY;
            }
        };
        open();
        // (the softmax warps take one decision on waits, as they meet at barriers)
        bool ok = !any_softmax<C::kSoft>(!warp_wait(&ifull[0], 0, abort_flag, a.d_status));
        int n = ok ? tiles[0].n : 0;
        if (n > 0) {
            query(tiles[0]);
            if (lane == 0) mbar_arrive(&qready[0]);
        }
        bool opens = true;
        for (int i = 0; ok && n > 0; ++i) {
            const Tile &tl = tiles[i % kRecords], &nx = tiles[(i + 1) % kRecords];
            const int buf = i & 1, my_q = qbuf, r = tl.req, rows = tl.rows;
            // ---- scores
            const int blk = t >> 4, slot = t & 15;
            const int lim = tl.lim[blk];
            const bool vis = slot < lim;
            // the first row here, from g0 on, that sees the key
            const int seer = CHUNK ? min(max(tl.pos[blk] + slot - tl.qpos, 0), kFewRows) * a.group - hg - g0 : 0;
            const float ks = tl.ks[blk], lv = log2_of(tl.vs[blk]);
            const float dpos = a.alibi ? static_cast<float>(tl.pos[blk] + slot - tl.qpos) : 0.f;
            const bool got = warp_wait(&sfull[buf], (i >> 1) & 1, abort_flag, a.d_status) &&
                             warp_wait(&ifull[(i + 1) % kRecords], ((i + 1) / kRecords) & 1, abort_flag, a.d_status);
            tc::fence_after_sync();
            float x[HT];
            {
                uint32_t sv[QP][HT];
#pragma unroll
                for (int part = 0; part < QP; ++part) tmem_load<HT>(tbase + lane_off + buf * C::kQN + part * NG + g0, sv[part]);
                tc::wait_ld();
#pragma unroll
                for (int h = 0; h < HT; h += 4) {
                    const float4 hm = *reinterpret_cast<const float4 *>(&h_hm[32 * my_q + g0 + h]);
                    const float4 mu = *reinterpret_cast<const float4 *>(&h_mu[g0 + h]);
                    const float hm4[4] = {hm.x, hm.y, hm.z, hm.w}, mu4[4] = {mu.x, mu.y, mu.z, mu.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        float s = __uint_as_float(sv[QP - 1][h + y]);
#pragma unroll
                        for (int part = QP - 2; part >= 0; --part)
                            s = fmaf(s, 1.f / kPartStep, __uint_as_float(sv[part][h + y]));
                        x[h + y] = fmaf(s, ks * hm4[y], -mu4[y]);
                        if (a.alibi) x[h + y] = fmaf(h_slope[g0 + h + y], CHUNK ? dpos - h_tok[g0 + h + y] : dpos, x[h + y]);
                        if (!vis || (CHUNK && h + y < seer)) x[h + y] = -INFINITY;
                    }
                }
            }
            bool past = !got;
            float dm[HT];
#pragma unroll
            for (int h = 0; h < HT; h += 4) {
                const float4 d = *reinterpret_cast<const float4 *>(&h_dm[g0 + h]);
                dm[h] = d.x;
                dm[h + 1] = d.y;
                dm[h + 2] = d.z;
                dm[h + 3] = d.w;
#pragma unroll
                for (int y = h; y < h + 4; ++y) past |= x[y] + fmaxf(lv + dm[y], 0.f) > kSlack;
            }
            if (any_softmax<C::kSoft>(past)) {
                ok = !any_softmax<C::kSoft>(!got);
                if (!ok) break;
                // ---- references (mu for the row sums, mo for score + log2 of the V scale) move to the new maxima
                float top[HT];
#pragma unroll
                for (int h = 0; h < HT; ++h) {
                    const float m = warp_max(x[h]), m_o = warp_max(x[h] + lv);
                    if (lane == 0) {
                        red[wq][g0 + h] = m;
                        red_o[wq][g0 + h] = m_o;
                    }
                }
                sync_softmax<C::kSoft>();
#pragma unroll
                for (int h = 0; h < HT; ++h) {
                    const int gh = g0 + h;
                    const float m = fmaxf(fmaxf(red[0][gh], red[1][gh]), fmaxf(red[2][gh], red[3][gh]));
                    const bool none = m == -INFINITY, fresh = dm[h] == INFINITY;
                    top[h] = !none && (fresh || m > kSlack) ? m + kMargin : 0.f;   // how far mu moves
                    if (t == h) {
                        const float m_o = fmaxf(fmaxf(red_o[0][gh], red_o[1][gh]), fmaxf(red_o[2][gh], red_o[3][gh]));
                        const float mu = h_mu[gh], mo_old = mu - dm[h], mo_new = mu + m_o;
                        const float mo = fresh || mo_new > mo_old + kSlack ? mo_new + kMargin : mo_old;
                        h_step[gh] = none || fresh ? 1.f : fast_exp2(mo_old - mo);
                        if (!none) {
                            h_mu[gh] = mu + top[h];
                            h_dm[gh] = mu + top[h] - mo;
                        }
                    }
                }
                sync_softmax<C::kSoft>();
#pragma unroll
                for (int h = 0; h < HT; ++h) {
                    x[h] -= top[h];
                    if (top[h] > 0.f) l[h] *= fast_exp2(-top[h]);   // (at the first maximum l is 0)
                }
                if (!opens) {
                    // O of the tiles before, once the last product is done
                    ok = !any_softmax<C::kSoft>(!warp_wait(&odone[buf ^ 1], ((i - 1) >> 1) & 1, abort_flag, a.d_status));
                    if (!ok) break;
                    tc::fence_after_sync();
                    uint32_t o[kPP][HT];
#pragma unroll
                    for (int part = 0; part < kPP; ++part) tmem_load<HT>(tO + lane_off + part * NG + g0, o[part]);
                    tc::wait_ld();
#pragma unroll
                    for (int part = 0; part < kPP; ++part)
#pragma unroll
                        for (int h = 0; h < HT; h += 4) {
#pragma unroll
                            for (int y = h; y < h + 4; ++y) o[part][y] = __float_as_uint(__uint_as_float(o[part][y]) * h_step[g0 + y]);
                            tmem_store4(tO + lane_off + part * NG + g0 + h, &o[part][h]);
                        }
                    tc::wait_st();
                    tc::fence_before_sync();
                }
            }
            // ---- the next tile's query, so that its scores are computed meanwhile
            const int n_next = nx.n;
            const bool closes = n_next == 0 || nx.req != r;
            if (n_next > 0) {
                query(nx);
                __syncwarp();
                if (lane == 0) mbar_arrive(&qready[buf ^ 1]);
            }
            // ---- weights, their sums, and their parts as the P operand: 2^7 2^(s + log2 s_v - mo).  The V scale joins in
            // the exponent: as factors, a scale and the references' difference over- or underflow each for itself where
            // scales span the range of a float.
            uint8_t *pd = sm + C::kOffP + buf * C::kPBytes;
            float w[HT / 4][4];
#pragma unroll
            for (int h = 0; h < HT; h += 4) {
                const float4 d = *reinterpret_cast<const float4 *>(&h_dm[g0 + h]);
                const float dm4[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    // (a key that no row sees before the first that one sees: dm is infinite, the score -infinity)
                    w[h / 4][y] = vis && !(CHUNK && h + y < seer) ? fast_exp2(x[h + y] + (lv + 7.f + dm4[y])) : 0.f;
                    x[h + y] = fast_exp2(x[h + y]);
                    l[h + y] += x[h + y];
                }
            }
#pragma unroll
            for (int part = 0; part < kPP; ++part) {
                if constexpr (C::kKeyRows) {
                    // columns part * NG + head; 16-byte pieces swizzled by the row's bits above 128 bytes
                    const int at = t * C::kPN + part * NG + g0;
                    const uint32_t lo4 = take_part(w[0]), hi4 = take_part(w[1]);
                    *reinterpret_cast<uint2 *>(pd + (at ^ (((at >> 7) & (C::kPN / 16 - 1)) << 4))) = make_uint2(lo4, hi4);
                } else {
                    const uint32_t codes = take_part(w[0]);
#pragma unroll
                    for (int y = 0; y < 4; ++y) pd[swz8(part * NG + g0 + y, t)] = static_cast<uint8_t>(codes >> (8 * y));
                }
            }
            // a weight of 0 does not undo a NaN in a slot that the query does not see
            if (!vis && g0 == 0 && t < ((n + 1) & ~1) * kBlockTokens) {
                mbar_wait(&full[i % S], (i / S) & 1);
                uint4 *row = reinterpret_cast<uint4 *>(sm + (i % S) * kStageBytes + kHalfStage + t * 128);
#pragma unroll
                for (int y = 0; y < 8; ++y) row[y] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pready[buf]);
            if (MASS) {
                // sum over the 16 lanes of a word, the heads spread over the lanes on the way
                float v[HT];
#pragma unroll
                for (int h = 0; h < HT; ++h) v[h] = x[h];
                int head = 0, left = HT;
#pragma unroll
                for (int bit = 8; bit > 0; bit >>= 1) {
                    if (left > 1) {
                        left >>= 1;
                        const bool up = (lane & bit) != 0;
                        if (up) head += left;
#pragma unroll
                        for (int h = 0; h < HT / 2; ++h)
                            if (h < left) {
                                const float keep = up ? v[h + left] : v[h], send = up ? v[h] : v[h + left];
                                v[h] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
                            }
                    } else {
                        v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
                    }
                }
                // HT lanes of the word hold a head each
                if (blk < n && (slot & (16 / HT - 1)) == 0 && g0 + head < rows)
                    p.ws_lse[(static_cast<size_t>(r) * a.max_words + tl.word + blk) * a.hq + kvh * a.group + hg + g0 + head] =
                        h_mu[g0 + head] + log2_of(v[0]);
            }
            if (closes) {
                // ---- the request's partial result
                ok = !any_softmax<C::kSoft>(!warp_wait(&odone[buf], (i >> 1) & 1, abort_flag, a.d_status));
                if (!ok) break;
                tc::fence_after_sync();
                const size_t slot_g = (static_cast<size_t>(kvh) * (p.pieces + B) + wi + r) * p.rows + hg;
#pragma unroll
                for (int h = 0; h < HT; ++h) {
                    float s = l[h];
#pragma unroll
                    for (int y = 16; y > 0; y >>= 1) s += __shfl_xor_sync(0xffffffffu, s, y);
                    if (lane == 0) red[wq][g0 + h] = s;
                }
                sync_softmax<C::kSoft>();
                if (threadIdx.x < rows) {
                    const int h = threadIdx.x;
                    const float s = (red[0][h] + red[1][h]) + (red[2][h] + red[3][h]);
                    const bool none = h_dm[h] == INFINITY && s == s;
                    p.ws_ml[slot_g + h] = none ? make_float4(-INFINITY, 0.f, -INFINITY, 0.f)
                                               : make_float4(h_mu[h], s, h_mu[h] - h_dm[h], 0.f);
                }
#pragma unroll
                for (int h = 0; h < HT; h += 4) {
                    uint32_t o[kPP][4];
#pragma unroll
                    for (int part = 0; part < kPP; ++part) tmem_load<4>(tO + lane_off + part * NG + g0 + h, o[part]);
                    tc::wait_ld();
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        if (g0 + h + y < rows) {
                            float v = __uint_as_float(o[kPP - 1][y]);
#pragma unroll
                            for (int part = kPP - 2; part >= 0; --part) v = fmaf(v, 1.f / kPartStep, __uint_as_float(o[part][y]));
                            a.ws_acc[(slot_g + g0 + h + y) * kHeadDim + t] = v * 0x1p-7f;
                        }
                }
                tc::fence_before_sync();
                sync_softmax<C::kSoft>();
                open();
                sync_softmax<C::kSoft>();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&iempty[i % kRecords]);
            opens = closes;
            n = n_next;
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == kIssue) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tbase, C::kCols);
    }
}

template <int NG, int QP, bool MASS, bool CHUNK>
cudaError_t launch_t(const CUtensorMap &tk, const CUtensorMap &tv, const LaneParams &p, cudaStream_t s) {
    using C = Cfg<NG, QP>;
    auto kern = decode_q8_kernel<NG, QP, MASS, CHUNK>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    kern<<<p.pieces * p.a.hkv * row_groups(p.rows), C::kThreads, C::kSmem, s>>>(tk, tv, p);
    return cudaGetLastError();
}
template <int NG>
cudaError_t launch_g(const CUtensorMap &tk, const CUtensorMap &tv, const LaneParams &p, cudaStream_t s) {
    if (p.a.cu_q) return launch_t<NG, 3, false, true>(tk, tv, p, s);
    return p.mass ? launch_t<NG, 5, true, false>(tk, tv, p, s) : launch_t<NG, 3, false, false>(tk, tv, p, s);
}
template <int QP>
int occupancy(int rows) {
    return rows <= 4 ? Cfg<4, QP>::kOcc : rows <= 8 ? Cfg<8, QP>::kOcc : Cfg<16, QP>::kOcc;
}

}  // namespace

LanePlan decode_q8_plan(int num_req, int hkv, int max_words, int rows, bool mass, int sms) {
    // one wave of resident CTAs, at least one tile of words each
    const int64_t words = static_cast<int64_t>(num_req) * max_words;
    const int64_t most = (words + kLineMinWordsQ8 - 1) / kLineMinWordsQ8;
    const int64_t resident = static_cast<int64_t>(sms > 0 ? sms : 1) * (mass ? occupancy<5>(rows) : occupancy<3>(rows)) /
                             (hkv * row_groups(rows));
    LanePlan pl;
    pl.pieces = static_cast<int>(most < resident ? most : resident);
    if (pl.pieces < 1) pl.pieces = 1;
    pl.slots = static_cast<int64_t>(hkv) * (pl.pieces + num_req);
    return pl;
}

cudaError_t launch_decode_q8(const CUtensorMap &tk, const CUtensorMap &tv, const LaneParams &p, cudaStream_t s) {
    const cudaError_t e = p.rows <= 4   ? launch_g<4>(tk, tv, p, s)
                          : p.rows <= 8 ? launch_g<8>(tk, tv, p, s)
                                        : launch_g<16>(tk, tv, p, s);
    return e == cudaSuccess ? launch_lane_combine(p, kLineMinWordsQ8, s) : e;
}

}  // namespace lazy

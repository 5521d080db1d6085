// write_q8.cu -- new tokens into the 8-bit pool.
//
// Per (block, KV head) that the call writes to, with x = RoPE(k, j) or v over the call's tokens there:
//   s = max(s_old if the block holds tokens, least 2^e >= 2^-126 with max |x| <= 448 2^e),
//   code = e4m3_rne(float_rne(x / s)),  earlier tokens' codes = e4m3_rne(code s_old / s) where s grew.
//
// One owner (a CTA or a warp) writes all of a block's tokens, so scales, rescaled codes and metadata need
// no atomics on the pool and no order of execution enters the result.
//
// Up to kQ8ScanTokens tokens (the decode step's append, where latency counts): CTA t owns token t's block if
// t is the call's first token there, found by reading all slots of the call; one launch, no
// workspace.  The block's angles are evaluated once and shared by its heads, one head per warp.
//
// More tokens: token indices are scattered to a row of 16 per block; then a CTA owns the blocks whose first
// stored token is one of 16 consecutive ones.  Angles are those of the block's first position, one per
// pair, times a table of the 16 slots' (one per call), shared by the heads.  A warp takes every fourth
// head; its rows come by bulk copies into shared memory, values while keys are worked on and the next
// head's keys while values are.  Loops over rows stay rolled: unrolled, the code missed the instruction
// cache (32768 tokens x 8 heads: 118 us, now 79; 202 MB, 2.5 TB/s).  37.2 M instructions take half the
// issue slots, a third each for angles and rotation, scales, and codes with their error intervals; the rest are waits that
// 28 % occupancy does not hide (loads, two barriers and 64 fp64 angles per block ahead of its rows).  Ownership by the
// first token puts up to 16 blocks into one CTA where the call's tokens are not in slot order: 20000 tokens 64 us in
// order, 215 permuted.
// Half a warp per token row, 8 elements per lane.  Rotations run in fp32.  Where a code or a scale could
// depend on the rotation's rounding (the error interval holds a rounding border: some elements in 10^5) it is
// computed again in fp64.  A code is e4m3_rne(float_rne(x / s)): the quotient is rounded to fp32 first, here as there.
#include <cfloat>

#include "common.cuh"
#include "kernels.h"
#include "pdl.cuh"
#include "q8.cuh"

namespace lazy {

namespace {

constexpr int kThreads = 256;           // small calls
constexpr int kGroup = 16;              // large calls: tokens per CTA
constexpr int kBulkWarps = 4;
// Bounds of |x in fp32 - x| relative to |x0| + |x1| >= r = sqrt(a^2 + b^2) of the rotated pair; u = 2^-24 is half an ulp
// relative to the least value of its binade, so a rounding is off by up to u |value|.
// Large calls: cos and sin rounded from fp64 (below 1, so u / 2 absolute each: u / 2 (|a| + |b|) <= 0.71 u r), a
// product and a sum of at most r (u r each): 2.71 u r = 1.62e-7 r; 1.45e-7 was met.  The interval's ends
// y -+ e are rounded as well, but monotonically: the float next to x / scale lies between them.
// Small calls: cos and sin to 2.4e-7 (angle rounded to fp32, sincosf to 2 ulp): 3.4e-7 r, and 2 u r: 4.6e-7 r.
constexpr float kErrSmall = 7.1e-7f, kErrLarge = 1.7e-7f;
// Where product or sum are below the smallest normal number each is off by up to 2^-150 instead.
constexpr float kErrTiny = 0x1p-148f;
constexpr float kAmaxErr = 1.5e-6f;     // relative: twice the larger of them, and its own rounding

// biased fp32 exponent of the least power of two s >= 2^-126 with amax <= 448 s
__device__ __forceinline__ int scale_exp(double amax) {
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(amax));
    const int e = static_cast<int>(u >> 52) - 1023 - 8 + ((u & 0xFFFFFFFFFFFFFull) > 0xC000000000000ull ? 1 : 0);
    return max(e + 127, 1);
}
__device__ __noinline__ double2 rotate_f64(double a, double b, int j, double theta) {
    double s, c;
    sincos(static_cast<double>(j) * theta, &s, &c);
    return make_double2(a * c - b * s, b * c + a * s);
}
__device__ __forceinline__ double bits_f64(uint16_t b) { return static_cast<double>(bits_to_float(b)); }

// max |x| over the finite elements of the block's new rows of one head, in fp64; the whole warp calls it
template <bool KEY>
__device__ __noinline__ double amax_f64(const Q8WriteParams &p, const int *tok, const int *pos, int h, int lane) {
    double am = 0.0;
    for (int row = 0; row < kBlockTokens; ++row) {
        if (tok[row] < 0) continue;
        const uint16_t *x = (KEY ? p.k_raw : p.v_raw) + (static_cast<size_t>(tok[row]) * p.hkv + h) * kHeadDim;
        for (int i = lane; i < kHalfDim; i += 32) {
            double2 z = make_double2(bits_f64(x[i]), bits_f64(x[i + kHalfDim]));
            if (KEY) z = rotate_f64(z.x, z.y, pos[row], p.rope.theta[i]);
            if (fabs(z.x) <= DBL_MAX) am = fmax(am, fabs(z.x));
            if (fabs(z.y) <= DBL_MAX) am = fmax(am, fabs(z.y));
        }
    }
    for (int o = 16; o > 0; o >>= 1) am = fmax(am, __shfl_xor_sync(0xffffffffu, am, o));
    return am;
}
// The codes of elements 4 c .. + 3 (up = 0) or 64 above of one row, by fp64.
template <bool KEY>
__device__ __noinline__ uint32_t codes_f64(const Q8WriteParams &p, int t, int j, int h, int c, int up, float scale) {
    const uint16_t *x = (KEY ? p.k_raw : p.v_raw) + (static_cast<size_t>(t) * p.hkv + h) * kHeadDim + 4 * c;
    float y[4];
#pragma unroll 1
    for (int u = 0; u < 4; ++u) {
        double2 z = make_double2(bits_f64(x[u]), bits_f64(x[u + kHalfDim]));
        if (KEY) z = rotate_f64(z.x, z.y, j, p.rope.theta[4 * c + u]);
        y[u] = static_cast<float>((up ? z.y : z.x) / static_cast<double>(scale));
    }
    return f32_to_codes(y[0], y[1], y[2], y[3]);
}

// Eight bf16 as floats: elements 4 c .. + 3 and 64 above of a row.
__device__ __forceinline__ void unpack_row(uint2 lo, uint2 hi, float (&x)[8]) {
    x[0] = bf16_lo(lo.x), x[1] = bf16_hi(lo.x), x[2] = bf16_lo(lo.y), x[3] = bf16_hi(lo.y);
    x[4] = bf16_lo(hi.x), x[5] = bf16_hi(hi.x), x[6] = bf16_lo(hi.y), x[7] = bf16_hi(hi.y);
}
// x (four pairs: u and u + 4) turned by the angles with cosines c and sines s.  (Scalar: negations and absolute values
// are free there, and paired fp32 instructions would spend more on moves.)
__device__ __forceinline__ void turn(float (&x)[8], const float4 c, const float4 s) {
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const float a = x[u], b = x[u + 4];
        x[u] = fmaf(-b, ss[u], a * cc[u]);
        x[u + 4] = fmaf(a, ss[u], b * cc[u]);
    }
}
// largest |x| so far; NaN does not enter
__device__ __forceinline__ float max_abs(float am, const float (&x)[8]) {
#pragma unroll
    for (int u = 0; u < 8; ++u) am = fmaxf(am, fabsf(x[u]));
    return am;
}

// The codes of the elements x (0 .. 3 of row t at dims 4 c, 4 .. 7 64 above) for the scale 1 / inv.
template <bool KEY>
__device__ __forceinline__ uint2 code_row(const Q8WriteParams &p, const float (&x)[8], float inv, float err, float scale, int t, int j,
                                          int h, int c) {
    float y[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) y[u] = x[u] * inv;
    uint2 code;
    if (KEY || err != 0.f) {
        // Codes of both ends of the error interval: they differ where it holds a rounding border.  A key's error is
        // that of its pair; a value's is its own (its partner may be NaN or infinite).
        float e[8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            e[u] = KEY ? fmaf(fabsf(y[u]) + fabsf(y[u + 4]), err, inv * kErrTiny) : fabsf(y[u]) * err;
            e[u + 4] = KEY ? e[u] : fabsf(y[u + 4]) * err;
        }
        code.x = f32_to_codes(y[0] + e[0], y[1] + e[1], y[2] + e[2], y[3] + e[3]);
        code.y = f32_to_codes(y[4] + e[4], y[5] + e[5], y[6] + e[6], y[7] + e[7]);
        if (code.x != f32_to_codes(y[0] - e[0], y[1] - e[1], y[2] - e[2], y[3] - e[3]))
            code.x = codes_f64<KEY>(p, t, j, h, c, 0, scale);
        if (code.y != f32_to_codes(y[4] - e[4], y[5] - e[5], y[6] - e[6], y[7] - e[7]))
            code.y = codes_f64<KEY>(p, t, j, h, c, 1, scale);
    } else {
        code.x = f32_to_codes(y[0], y[1], y[2], y[3]);
        code.y = f32_to_codes(y[4], y[5], y[6], y[7]);
    }
    return code;
}

// One head's scale from max |x| in fp32 over the lanes, and its rows' codes; row(r, x) gives row r (x in fp32) to its
// half warp.  tok, pos: token index (-1: none) and local index per slot, have: bit mask of the slots with
// one; nv: slots that held tokens before.
template <bool KEY, typename Row>
__device__ __forceinline__ void code_head(const Q8WriteParams &p, int blk, int h, int nv, const int *tok, const int *pos,
                                          uint32_t have, int lane, float am, float key_err, Row &&row) {
    const int hl = lane >> 4, c = lane & 15;
    float *scale_p = (KEY ? p.k_scale : p.v_scale) + static_cast<size_t>(blk) * p.hkv + h;
    const float before = nv > 0 ? *scale_p : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
    float fresh = q8_scale_for(fminf(am, FLT_MAX));
    // an infinity (or an overflow of fp32) among the elements, or a border of the scales within the error
    if (am > FLT_MAX || (KEY && q8_scale_for(am * (1.f - kAmaxErr)) != q8_scale_for(fminf(am * (1.f + kAmaxErr), FLT_MAX))))
        fresh = __uint_as_float(static_cast<uint32_t>(scale_exp(amax_f64<KEY>(p, tok, pos, h, lane))) << 23);
    const float scale = nv > 0 ? fmaxf(before, fresh) : fresh;
    const bool pow2 = (__float_as_uint(scale) & 0x7FFFFFu) == 0;   // then x / scale = x * inv exactly
    const float inv = 1.f / scale;
    const bool grew = nv > 0 && scale != before;
    const float err = (KEY ? key_err : 0.f) + (pow2 ? 0.f : 0x1p-22f);   // of x * inv, relative to |x0| + |x1|
    uint8_t *codes = (KEY ? p.k_codes : p.v_codes) + (static_cast<size_t>(blk) * p.hkv + h) * kBlockTokens * kHeadDim;
    uint32_t *dst = reinterpret_cast<uint32_t *>(codes + hl * kHeadDim) + c;
    if (have == 0xFFFFu) {
#pragma unroll 2
        for (int i = 0; i < 8; ++i, dst += 2 * kHeadDim / 4) {
            float x[8];
            row(2 * i + hl, x);
            const uint2 code = code_row<KEY>(p, x, inv, err, scale, tok[2 * i + hl], pos[2 * i + hl], h, c);
            dst[0] = code.x;
            dst[16] = code.y;
        }
    } else {
        const float ratio = before / scale;
#pragma unroll 1
        for (int i = 0; i < 8; ++i, dst += 2 * kHeadDim / 4) {
            const int r = 2 * i + hl;
            if (!((have >> (2 * i)) & 3u) && !(grew && 2 * i < nv)) continue;   // neither row of the pair
            if ((have >> r) & 1u) {
                float x[8];
                row(r, x);
                const uint2 code = code_row<KEY>(p, x, inv, err, scale, tok[r], pos[r], h, c);
                dst[0] = code.x;
                dst[16] = code.y;
            } else if (r < nv && grew) {
#pragma unroll 1
                for (int s = 0; s < 2; ++s) {
                    uint32_t h0, h1;
                    float y[4];
                    codes_to_f16(dst[16 * s], h0, h1);
                    f16x2_to_f32(h0, y[0], y[1]);
                    f16x2_to_f32(h1, y[2], y[3]);
                    dst[16 * s] = f32_to_codes(y[0] * ratio, y[1] * ratio, y[2] * ratio, y[3] * ratio);
                }
            }
        }
    }
    if (lane == 0) *scale_p = scale;
}

// 0: good; else the status bit of a token that is skipped
__device__ __forceinline__ int token_fault(const Q8WriteParams &p, int slot, int j) {
    if (slot < 0 || static_cast<int64_t>(slot) >= static_cast<int64_t>(p.num_blocks) * kBlockTokens) return LAZY_DSTATUS_BAD_SLOT;
    return j < 0 || (j & (kBlockTokens - 1)) != (slot & (kBlockTokens - 1)) ? LAZY_DSTATUS_BAD_ALIGN : 0;
}
__device__ __forceinline__ uint32_t meta_of(int slot, int j) {
    return (static_cast<uint32_t>(j / kBlockTokens) << 8) | static_cast<uint32_t>(slot % kBlockTokens + 1);
}

// The workspace of a large call: rows[b][s] = 1 + the last token of the call in slot s of block b; one word per
// block, the largest metadata word of the call's tokens there; (cos, sin) of s theta_i as [16][64] in fp64.
__device__ __forceinline__ uint32_t *ws_metas(const Q8WriteParams &p) {
    return p.rows + static_cast<size_t>(p.num_blocks) * kBlockTokens;
}
__device__ __forceinline__ double2 *ws_angles(const Q8WriteParams &p) {
    return reinterpret_cast<double2 *>(ws_metas(p) + (static_cast<size_t>(p.num_blocks) + 3) / 4 * 4);
}
__global__ void __launch_bounds__(256) q8_rows_kernel(const __grid_constant__ Q8WriteParams p) {
    pdl_trigger();
    const int t = blockIdx.x * 256 + threadIdx.x;
    if (t < kBlockTokens * kHalfDim) {   // (a large call has more tokens than this)
        const int s = t / kHalfDim, i = t % kHalfDim;
        ws_angles(p)[t] = rotate_f64(1.0, 0.0, s, p.rope.theta[i]);   // (cos, sin)
    }
    if (t >= p.n_tok) return;
    const int slot = p.slot[t], j = p.local_j[t];
    if (const int f = token_fault(p, slot, j)) {
        set_status(p.d_status, f);
        return;
    }
    atomicMax(&p.rows[slot], static_cast<uint32_t>(t + 1));
    atomicMax(&ws_metas(p)[slot / kBlockTokens], meta_of(slot, j));
}

constexpr int kRawBytes = kBlockTokens * kHeadDim * 2;                              // rows of one head
constexpr int kAngleBytes = kBlockTokens * 2 * kHalfDim * 4;
constexpr int kBulkSmem = kAngleBytes + kBulkWarps * 2 * kRawBytes;

__global__ void __launch_bounds__(kBulkWarps * 32, 5) kv_write_q8_bulk_kernel(const __grid_constant__ Q8WriteParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    float(*cs)[2][kHalfDim] = reinterpret_cast<float(*)[2][kHalfDim]>(smem);           // [16][2][64]
    __shared__ int toks[kGroup][kBlockTokens], pos[kBlockTokens];
    __shared__ int owned[kGroup], n_owned;
    __shared__ double2 base_cs[kHalfDim];
    __shared__ uint64_t bars[kBulkWarps][2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hl = lane >> 4, c = lane & 15;
    uint8_t *raw[2] = {smem + kAngleBytes + warp * 2 * kRawBytes, smem + kAngleBytes + (warp * 2 + 1) * kRawBytes};   // K, V
    if (lane < 2) mbar_init(&bars[warp][lane], 1);
    fence_barrier_init();
    pdl_wait();
    if (warp == 0) {
        const int t = blockIdx.x * kGroup + lane;
        int b = -1;
        if (lane < kGroup && t < p.n_tok) {
            const int slot = p.slot[t], j = p.local_j[t];
            if (!token_fault(p, slot, j)) {
                b = slot / kBlockTokens;
                uint32_t first = 0xFFFFFFFFu;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 row = reinterpret_cast<const uint4 *>(p.rows + static_cast<size_t>(b) * kBlockTokens)[i];
                    // 0 (no token) wraps to the largest value
                    first = min(first, min(min(row.x - 1u, row.y - 1u), min(row.z - 1u, row.w - 1u)));
                }
                if (first != static_cast<uint32_t>(t)) b = -1;
            }
        }
        const uint32_t m = __ballot_sync(0xffffffffu, b >= 0);
        const int n = __popc(m);
        if (b >= 0) owned[__popc(m & ((1u << lane) - 1u))] = b;
        if (lane == 0) n_owned = n;
        __syncwarp();
        for (int i = lane; i < n * kBlockTokens; i += 32)
            toks[i / kBlockTokens][i % kBlockTokens] =
                static_cast<int>(p.rows[static_cast<size_t>(owned[i / kBlockTokens]) * kBlockTokens + i % kBlockTokens]) - 1;
    }
    __syncthreads();
    uint32_t phase[2] = {0u, 0u};
    bool ok = true, flying[2] = {false, false};   // copies that have not landed
    for (int k = 0; k < n_owned; ++k) {
        const int blk = owned[k], *tok = toks[k];
        const int my = lane < kBlockTokens ? tok[lane] : -1;
        const uint32_t have = __ballot_sync(0xffffffffu, my >= 0);
        // rows of K (0) or V (1) of head h; lane r copies row r
        auto fetch = [&](int which, int h) {
            __syncwarp();   // the last head's rows are read
            flying[which] = true;
            if (lane == 0) mbar_arrive_expect_tx(&bars[warp][which], __popc(have) * 256);
            __syncwarp();
            if (my >= 0) {
                const uint16_t *src = (which ? p.v_raw : p.k_raw) + (static_cast<size_t>(my) * p.hkv + h) * kHeadDim;
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], 256, [%2];" ::"r"(
                                 smem_u32(raw[which] + lane * 256)),
                             "l"(src), "r"(smem_u32(&bars[warp][which]))
                             : "memory");
            }
        };
        auto landed = [&](int which) {
            const bool got = __all_sync(0xffffffffu, mbar_wait(&bars[warp][which], phase[which]));
            if (!got) {
                set_status(p.d_status, LAZY_DSTATUS_TIMEOUT);
                return false;
            }
            phase[which] ^= 1;
            flying[which] = false;
            return true;
        };
        if (warp < p.hkv) {
            fetch(0, warp);
            fetch(1, warp);
        }
        // position of slot 0 by any of the tokens; all the same but in a call that contradicts itself
        const int j = my >= 0 ? p.local_j[my] : 0;
        const int j0 = __shfl_sync(0xffffffffu, j - lane, __ffs(have) - 1);
        const bool one = __all_sync(0xffffffffu, my < 0 || j - lane == j0);
        const uint32_t meta = p.blk_meta[blk];
        const int nv = meta_valid(meta);
        if (tid < kBlockTokens) pos[tid] = j;
        if (tid < kHalfDim) base_cs[tid] = rotate_f64(1.0, 0.0, j0, p.rope.theta[tid]);
        __syncthreads();
        const double2 *table = ws_angles(p);
        for (int i = tid; i < kBlockTokens * kHalfDim; i += kBulkWarps * 32) {
            const int r = i / kHalfDim, d = i % kHalfDim;
            double2 z = make_double2(0.0, 0.0);
            if (one) {
                // cos(a + b) = cos a cos b - sin a sin b, sin(a + b) = sin a cos b + cos a sin b
                const double2 x = base_cs[d], y = table[i];
                z = make_double2(x.x * y.x - x.y * y.y, x.y * y.x + x.x * y.y);
            } else if (tok[r] >= 0) {
                z = rotate_f64(1.0, 0.0, pos[r], p.rope.theta[d]);
            }
            cs[r][0][d] = static_cast<float>(z.x);
            cs[r][1][d] = static_cast<float>(z.y);
        }
        __syncthreads();
#pragma unroll 1
        for (int h = warp; h < p.hkv && ok; h += kBulkWarps) {
            auto key_row = [&](int r, float(&x)[8]) {
                const uint2 *q = reinterpret_cast<const uint2 *>(raw[0] + r * 256);
                unpack_row(q[c], q[16 + c], x);
                turn(x, *reinterpret_cast<const float4 *>(&cs[r][0][4 * c]), *reinterpret_cast<const float4 *>(&cs[r][1][4 * c]));
            };
            auto val_row = [&](int r, float(&x)[8]) {
                const uint2 *q = reinterpret_cast<const uint2 *>(raw[1] + r * 256);
                unpack_row(q[c], q[16 + c], x);
            };
            ok = landed(0);
            if (!ok) break;
            float am = 0.f;
            if (have == 0xFFFFu) {
#pragma unroll 2
                for (int r = hl; r < kBlockTokens; r += 2) {
                    float x[8];
                    key_row(r, x);
                    am = max_abs(am, x);
                }
            } else {
#pragma unroll 1
                for (int r = hl; r < kBlockTokens; r += 2) {
                    float x[8];
                    if (!((have >> r) & 1u)) continue;
                    key_row(r, x);
                    am = max_abs(am, x);
                }
            }
            __syncwarp();
            code_head<true>(p, blk, h, nv, tok, pos, have, lane, am, kErrLarge, key_row);
            if (h + kBulkWarps < p.hkv) fetch(0, h + kBulkWarps);
            ok = landed(1);
            if (!ok) break;
            // max |v| as bf16 pairs (a NaN does not enter)
            __nv_bfloat162 v2 = __float2bfloat162_rn(0.f);
#pragma unroll 2
            for (int r = hl; r < kBlockTokens; r += 2) {
                const uint4 *q = reinterpret_cast<const uint4 *>(raw[1] + r * 256);
                const uint4 w = q[c];
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
                if ((have >> r) & 1u)
#pragma unroll
                    for (int u = 0; u < 4; ++u) v2 = __hmax2(v2, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&ws[u])));
            }
            const float vm = fmaxf(__low2float(v2), __high2float(v2));
            __syncwarp();
            code_head<false>(p, blk, h, nv, tok, pos, have, lane, vm, 0.f, val_row);
            if (h + kBulkWarps < p.hkv) fetch(1, h + kBulkWarps);
        }
        const bool stop = __syncthreads_or(!ok);
        if (tid == 0) p.blk_meta[blk] = max(meta, ws_metas(p)[blk]);
        if (stop) break;
    }
    // a wait that ran out: no copy may land in the memory of a CTA that is gone
#pragma unroll
    for (int which = 0; which < 2; ++which)
        if (flying[which]) mbar_wait(&bars[warp][which], phase[which]);
}

// A small call: CTA t owns token t's block if t is the call's first token there.
__global__ void __launch_bounds__(kThreads) kv_write_q8_kernel(const __grid_constant__ Q8WriteParams p) {
    __shared__ __align__(16) float cs[kBlockTokens][2][kHalfDim];
    __shared__ int tok[kBlockTokens], pos[kBlockTokens];
    __shared__ uint32_t meta_new;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hl = lane >> 4, c = lane & 15;
    const int t = blockIdx.x;
    const int slot = p.slot[t], j = p.local_j[t];
    if (const int f = token_fault(p, slot, j)) {
        if (tid == 0) set_status(p.d_status, f);
        return;
    }
    const int b = slot / kBlockTokens;
    if (tid < kBlockTokens) tok[tid] = -1;
    if (tid == 0) meta_new = 0u;
    const uint32_t meta = p.blk_meta[b];
    __syncthreads();
    bool later = false;   // an earlier token of the call lies in the same block
    for (int i = tid; i < p.n_tok; i += kThreads) {
        const int si = p.slot[i], ji = p.local_j[i];
        if (si < 0 || si / kBlockTokens != b || token_fault(p, si, ji)) continue;
        later |= i < t;
        atomicMax(&tok[si % kBlockTokens], i);
        atomicMax(&meta_new, meta_of(si, ji));
    }
    if (__syncthreads_or(later)) return;
    uint32_t have = 0u;
#pragma unroll
    for (int i = 0; i < kBlockTokens; ++i) have |= (tok[i] >= 0 ? 1u : 0u) << i;
    if (tid < kBlockTokens) pos[tid] = tok[tid] >= 0 ? p.local_j[tok[tid]] : 0;
    __syncthreads();
    for (int i = tid; i < kBlockTokens * kHalfDim; i += kThreads) {
        const int row = i / kHalfDim, d = i % kHalfDim;
        if (tok[row] >= 0) rope_cos_sin(pos[row], p.rope.theta[d], cs[row][0][d], cs[row][1][d]);
    }
    __syncthreads();
    const int nv = meta_valid(meta);
    for (int h = warp; h < p.hkv; h += kThreads / 32) {
        auto val_row = [&](const uint16_t *raw, int r, float(&x)[8]) {
            const uint2 *src = reinterpret_cast<const uint2 *>(raw + (static_cast<size_t>(tok[r]) * p.hkv + h) * kHeadDim);
            unpack_row(__ldg(src + c), __ldg(src + 16 + c), x);
        };
        auto key_row = [&](int r, float(&x)[8]) {
            val_row(p.k_raw, r, x);
            turn(x, *reinterpret_cast<const float4 *>(&cs[r][0][4 * c]), *reinterpret_cast<const float4 *>(&cs[r][1][4 * c]));
        };
        float am = 0.f, vm = 0.f;
#pragma unroll 2
        for (int i = 0; i < 8; ++i) {
            const int r = 2 * i + hl;
            if (!((have >> r) & 1u)) continue;
            float x[8];
            key_row(r, x);
            am = max_abs(am, x);
            val_row(p.v_raw, r, x);
            vm = max_abs(vm, x);
        }
        __syncwarp();
        code_head<true>(p, b, h, nv, tok, pos, have, lane, am, kErrSmall, key_row);
        code_head<false>(p, b, h, nv, tok, pos, have, lane, vm, 0.f, [&](int r, float(&x)[8]) { val_row(p.v_raw, r, x); });
    }
    __syncthreads();
    if (tid == 0) p.blk_meta[b] = max(meta, meta_new);
}

}  // namespace

cudaError_t launch_kv_write_q8(const Q8WriteParams &p, cudaStream_t s) {
    if (!p.rows) {
        kv_write_q8_kernel<<<p.n_tok, kThreads, 0, s>>>(p);
        return cudaGetLastError();
    }
    cudaError_t e = cudaMemsetAsync(p.rows, 0, static_cast<size_t>(p.num_blocks) * (kBlockTokens + 1) * 4, s);
    if (e != cudaSuccess) return e;
    q8_rows_kernel<<<(p.n_tok + 255) / 256, 256, 0, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kv_write_q8_bulk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBulkSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kv_write_q8_bulk_kernel, (p.n_tok + kGroup - 1) / kGroup, kBulkWarps * 32, kBulkSmem, s, p);
}

}  // namespace lazy

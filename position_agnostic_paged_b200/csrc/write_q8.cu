// write_q8.cu -- new tokens into the 8-bit pool.
//
// Per (block, KV head) that the call writes to, with x = RoPE(k, j) or v over the call's tokens there:
//   s = max(s_old if the block holds tokens, least 2^e >= 2^-126 with max |x| <= 448 2^e),
//   code = e4m3_rne(x / s),  earlier tokens' codes = e4m3_rne(code s_old / s) where s grew.
//
// One CTA owns a block and writes all of its tokens, so scales, rescaled codes and metadata need no
// atomics on the pool and no order of execution enters the result.  A call of up to kQ8ScanTokens
// tokens finds a block's tokens by reading all slots of the call (one launch, no workspace: the
// decode step's append, where latency counts); a larger one first scatters token indices to a
// row of 16 per block.  The angles of a block's tokens are evaluated once and shared by its heads.
// A warp takes one head: half a warp per token row, 8 elements per lane.
//
// Rotations run in fp32.  Where a code or a scale could depend on fp32 rounding (the error bound
// straddles a rounding border: about one element in 10^5) it is computed again in fp64.
#include <cfloat>

#include "common.cuh"
#include "kernels.h"
#include "q8.cuh"

namespace lazy {

namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 16;              // tokens per CTA of a large call
// |x in fp32 - x| <= kErr (|a| + |b|): cos and sin to 2.4e-7 (angle rounded to fp32, sincosf to 2 ulp),
// two products and a sum of half an ulp (6e-8) each
constexpr float kErr = 5e-7f;
constexpr float kAmaxErr = 1.2e-6f;     // relative: |a| + |b| <= 2 max(|x0|, |x1|), and its own rounding

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

// max |x| (finite elements) of the block's new keys of one head, in fp64; the whole warp calls it
__device__ __noinline__ double key_amax_f64(const Q8WriteParams &p, const int *tok, const int *pos, int h, int lane) {
    double am = 0.0;
    for (int row = 0; row < kBlockTokens; ++row) {
        if (tok[row] < 0) continue;
        const uint16_t *k = p.k_raw + (static_cast<size_t>(tok[row]) * p.hkv + h) * kHeadDim;
        for (int i = lane; i < kHalfDim; i += 32) {
            const double2 x = rotate_f64(bits_f64(k[i]), bits_f64(k[i + kHalfDim]), pos[row], p.rope.theta[i]);
            if (fabs(x.x) <= DBL_MAX) am = fmax(am, fabs(x.x));
            if (fabs(x.y) <= DBL_MAX) am = fmax(am, fabs(x.y));
        }
    }
    for (int o = 16; o > 0; o >>= 1) am = fmax(am, __shfl_xor_sync(0xffffffffu, am, o));
    return am;
}

// One head's K (KEY) or V of a block.  tok, pos: token index (-1: none) and local index per slot;
// cs: their angles; nv: slots that held tokens before the call.
template <bool KEY>
__device__ __forceinline__ void write_head(const Q8WriteParams &p, int blk, int h, int nv, const int *tok,
                                           const int *pos, const float2 (*cs)[kHalfDim], int lane) {
    const int hl = lane >> 4, c = lane & 15;
    const uint16_t *raw = KEY ? p.k_raw : p.v_raw;
    uint2 lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int t = tok[2 * i + hl];
        lo[i] = hi[i] = make_uint2(0u, 0u);
        if (t >= 0) {
            const uint2 *src = reinterpret_cast<const uint2 *>(raw + (static_cast<size_t>(t) * p.hkv + h) * kHeadDim);
            lo[i] = __ldg(src + c);
            hi[i] = __ldg(src + 16 + c);
        }
    }
    // the 8 elements of row i that this lane holds (4 c .. + 3 and 64 above), and |a| + |b| of each pair
    auto row_x = [&](int i, float (&x)[8], float (&mag)[4]) {
        const float a[4] = {bf16_lo(lo[i].x), bf16_hi(lo[i].x), bf16_lo(lo[i].y), bf16_hi(lo[i].y)};
        const float b[4] = {bf16_lo(hi[i].x), bf16_hi(hi[i].x), bf16_lo(hi[i].y), bf16_hi(hi[i].y)};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (KEY) {
                const float2 z = cs[2 * i + hl][4 * c + u];
                x[u] = a[u] * z.x - b[u] * z.y;
                x[u + 4] = b[u] * z.x + a[u] * z.y;
                mag[u] = fabsf(a[u]) + fabsf(b[u]);
            } else {
                x[u] = a[u];
                x[u + 4] = b[u];
                mag[u] = 0.f;
            }
        }
    };
    float am = 0.f;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (tok[2 * i + hl] < 0) continue;
        float x[8], mag[4];
        row_x(i, x, mag);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const bool fin = fabsf(x[u]) <= FLT_MAX;
            am = fmaxf(am, fin ? fabsf(x[u]) : 0.f);
            odd |= !fin;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
    float fresh = q8_scale_for(am);
    if (KEY) {
        const float below = q8_scale_for(am * (1.f - kAmaxErr)), above = q8_scale_for(fminf(am * (1.f + kAmaxErr), FLT_MAX));
        if (__any_sync(0xffffffffu, odd) || below != above)   // fp32 may decide wrongly, or overflow
            fresh = __uint_as_float(static_cast<uint32_t>(scale_exp(key_amax_f64(p, tok, pos, h, lane))) << 23);
    }
    float *scale_p = (KEY ? p.k_scale : p.v_scale) + static_cast<size_t>(blk) * p.hkv + h;
    const float before = *scale_p;
    const float scale = nv > 0 ? fmaxf(before, fresh) : fresh;
    const bool pow2 = (__float_as_uint(scale) & 0x7FFFFFu) == 0;   // then x / scale = x * inv exactly
    const float inv = 1.f / scale;
    const bool grew = nv > 0 && scale != before;
    const float ratio = before / scale;
    uint8_t *codes = (KEY ? p.k_codes : p.v_codes) + (static_cast<size_t>(blk) * p.hkv + h) * kBlockTokens * kHeadDim;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = 2 * i + hl;
        uint32_t *dst = reinterpret_cast<uint32_t *>(codes + row * kHeadDim) + c;
        if (tok[row] >= 0) {
            float x[8], mag[4];
            row_x(i, x, mag);
            uint32_t code[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                float y[4], e[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    y[u] = x[4 * s + u] * inv;
                    e[u] = (KEY ? kErr * mag[u] * inv : 0.f) + (pow2 ? 0.f : fabsf(y[u]) * 0x1p-22f);
                }
                code[s] = f32_to_codes(y[0], y[1], y[2], y[3]);
                if (KEY || !pow2) {
                    const uint32_t up = f32_to_codes(y[0] + e[0], y[1] + e[1], y[2] + e[2], y[3] + e[3]);
                    const uint32_t dn = f32_to_codes(y[0] - e[0], y[1] - e[1], y[2] - e[2], y[3] - e[3]);
                    if (up != dn) {
                        // some element lies within the error bound of a rounding border
                        const uint32_t wl[2] = {lo[i].x, lo[i].y}, wh[2] = {hi[i].x, hi[i].y};
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const double a = (u & 1) ? bf16_hi(wl[u >> 1]) : bf16_lo(wl[u >> 1]);
                            const double b = (u & 1) ? bf16_hi(wh[u >> 1]) : bf16_lo(wh[u >> 1]);
                            double2 z = make_double2(a, b);
                            if (KEY) z = rotate_f64(a, b, pos[row], p.rope.theta[4 * c + u]);
                            y[u] = static_cast<float>((s ? z.y : z.x) / static_cast<double>(scale));
                        }
                        code[s] = f32_to_codes(y[0], y[1], y[2], y[3]);
                    }
                }
            }
            dst[0] = code[0];
            dst[16] = code[1];
        } else if (row < nv && grew) {
#pragma unroll
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

// rows[b][s] = 1 + the last token of the call in slot s of block b; behind the rows one word per
// block, the largest metadata word of the call's tokens there.
__global__ void __launch_bounds__(256) q8_rows_kernel(const Q8WriteParams p) {
    const int t = blockIdx.x * 256 + threadIdx.x;
    if (t >= p.n_tok) return;
    const int slot = p.slot[t], j = p.local_j[t];
    if (const int f = token_fault(p, slot, j)) {
        set_status(p.d_status, f);
        return;
    }
    atomicMax(&p.rows[slot], static_cast<uint32_t>(t + 1));
    atomicMax(&p.rows[static_cast<size_t>(p.num_blocks) * kBlockTokens + slot / kBlockTokens], meta_of(slot, j));
}

// SCAN: CTA t owns token t's block if t is the call's first token there.  Otherwise: CTA g owns the
// blocks whose first stored token is one of tokens 16 g .. 16 g + 15.
template <bool SCAN>
__global__ void __launch_bounds__(kThreads) kv_write_q8_kernel(const __grid_constant__ Q8WriteParams p) {
    __shared__ float2 cs[kBlockTokens][kHalfDim];
    __shared__ int tok[kBlockTokens], pos[kBlockTokens];
    __shared__ int owned[kGroup], n_owned;
    __shared__ uint32_t meta_new;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (SCAN) {
        const int t = blockIdx.x;
        const int slot = p.slot[t], j = p.local_j[t];
        if (const int f = token_fault(p, slot, j)) {
            if (tid == 0) set_status(p.d_status, f);
            return;
        }
        const int b = slot / kBlockTokens;
        if (tid < kBlockTokens) tok[tid] = -1;
        if (tid == 0) meta_new = 0u;
        __syncthreads();
        bool later = false;   // an earlier token of the call lies in the same block
        for (int i = tid; i < p.n_tok; i += kThreads) {
            const int si = p.slot[i];
            if (si < 0 || si / kBlockTokens != b) continue;
            const int ji = p.local_j[i];
            if (token_fault(p, si, ji)) continue;
            later |= i < t;
            atomicMax(&tok[si % kBlockTokens], i);
            atomicMax(&meta_new, meta_of(si, ji));
        }
        if (__syncthreads_or(later)) return;
        if (tid == 0) {
            owned[0] = b;
            n_owned = 1;
        }
    } else {
        if (tid < 32) {
            const int t = blockIdx.x * kGroup + tid;
            int b = -1;
            if (tid < kGroup && t < p.n_tok) {
                const int slot = p.slot[t], j = p.local_j[t];
                if (!token_fault(p, slot, j)) {
                    b = slot / kBlockTokens;
                    uint32_t first = 0xFFFFFFFFu;
                    const uint4 *row = reinterpret_cast<const uint4 *>(p.rows + static_cast<size_t>(b) * kBlockTokens);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 v = row[i];
                        // 0 (no token) wraps to the largest value
                        first = min(first, min(min(v.x - 1u, v.y - 1u), min(v.z - 1u, v.w - 1u)));
                    }
                    if (first != static_cast<uint32_t>(t)) b = -1;
                }
            }
            const uint32_t m = __ballot_sync(0xffffffffu, b >= 0);
            if (b >= 0) owned[__popc(m & ((1u << tid) - 1u))] = b;
            if (tid == 0) n_owned = __popc(m);
        }
    }
    __syncthreads();
    for (int k = 0; k < n_owned; ++k) {
        const int b = owned[k];
        if (!SCAN && tid < kBlockTokens) tok[tid] = static_cast<int>(p.rows[static_cast<size_t>(b) * kBlockTokens + tid]) - 1;
        if (!SCAN && tid == 0) meta_new = p.rows[static_cast<size_t>(p.num_blocks) * kBlockTokens + b];
        __syncthreads();
        if (tid < kBlockTokens) pos[tid] = tok[tid] >= 0 ? p.local_j[tok[tid]] : 0;
        __syncthreads();
        for (int i = tid; i < kBlockTokens * kHalfDim; i += kThreads) {
            const int row = i / kHalfDim, d = i % kHalfDim;
            if (tok[row] >= 0) rope_cos_sin(pos[row], p.rope.theta[d], cs[row][d].x, cs[row][d].y);
        }
        const uint32_t meta = p.blk_meta[b];
        const int nv = meta_valid(meta);
        __syncthreads();
        for (int h = warp; h < p.hkv; h += kThreads / 32) {
            write_head<true>(p, b, h, nv, tok, pos, cs, lane);
            write_head<false>(p, b, h, nv, tok, pos, cs, lane);
        }
        __syncthreads();
        if (tid == 0) p.blk_meta[b] = max(meta, meta_new);
    }
}

}  // namespace

cudaError_t launch_kv_write_q8(const Q8WriteParams &p, cudaStream_t s) {
    if (!p.rows) {
        kv_write_q8_kernel<true><<<p.n_tok, kThreads, 0, s>>>(p);
        return cudaGetLastError();
    }
    cudaError_t e = cudaMemsetAsync(p.rows, 0, q8_write_ws_bytes(p.num_blocks), s);
    if (e != cudaSuccess) return e;
    q8_rows_kernel<<<(p.n_tok + 255) / 256, 256, 0, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    kv_write_q8_kernel<false><<<(p.n_tok + kGroup - 1) / kGroup, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace lazy

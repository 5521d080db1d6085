// stage_q8.cu -- the table words of a prefill over the 8-bit pool as bf16 keys and values.
//
// Word i of request r becomes row prefix(r) + i of the staging buffers: K rotated to absolute
// positions, R(offset) (s_k code) rounded to bf16 as the prefill's own K rotation rounds, V = s_v code
// (exact in bf16 for scales that are powers of two).  Slots that no query of the request sees are
// zero.  A table and metadata that name the rows follow.
#include "common.cuh"
#include "kernels.h"
#include "q8.cuh"

namespace lazy {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) q8_stage_kernel(const Q8StageParams p) {
    __shared__ float2 cs[kHalfDim];
    __shared__ int red[kThreads / 32];
    const int r = blockIdx.y, i = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const int beg = p.table_indptr[r];
    const int n_all = p.table_indptr[r + 1] - beg, n = min(n_all, p.max_words);
    if (i > 0 && i >= n) return;
    int before = 0;
    for (int q = tid; q < r; q += kThreads) before += max(0, min(p.table_indptr[q + 1] - p.table_indptr[q], p.max_words));
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) before += __shfl_xor_sync(0xffffffffu, before, x);
    if (lane == 0) red[tid >> 5] = before;
    uint32_t word = 0u, meta = 0u, blk = 0u;
    if (i < n) {
        word = p.table[beg + i];
        blk = word_block(word);
        if (blk < static_cast<uint32_t>(p.num_blocks))
            meta = p.blk_meta[blk];
        else if (tid == 0)
            set_status(p.d_status, LAZY_DSTATUS_BAD_BLOCK);
    }
    const int off = word_offset(word);
    if (tid < kHalfDim) rope_cos_sin(off, p.rope.theta[tid], cs[tid].x, cs[tid].y);
    __syncthreads();
    before = 0;
#pragma unroll
    for (int x = 0; x < kThreads / 32; ++x) before += red[x];
    if (tid == 0) {
        if (n_all > p.max_words && i == 0) set_status(p.d_status, LAZY_DSTATUS_BAD_TABLE);
        if (r == 0 && i == 0) p.indptr_out[0] = 0;
        if (i == 0) p.indptr_out[r + 1] = min(before + max(n, 0), p.cap_words);
    }
    const int row = before + i;
    if (i >= n) return;
    if (row >= p.cap_words) {
        if (tid == 0) set_status(p.d_status, LAZY_DSTATUS_BAD_TABLE);
        return;
    }
    const int last = p.q_pos0[r] + p.cu_q[r + 1] - p.cu_q[r] - 1;
    const int lim = p.cu_q[r + 1] > p.cu_q[r] ? max(0, min(meta_valid(meta), last - off - meta_j0(meta) + 1)) : 0;
    if (tid == 0) {
        p.table_out[row] = (static_cast<uint32_t>(off) << LAZY_BLOCK_BITS) | static_cast<uint32_t>(row);
        p.meta_out[row] = (meta & ~255u) | static_cast<uint32_t>(lim);
    }
    for (int it = tid; it < p.hkv * kBlockTokens * 16; it += kThreads) {
        const int c = it & 15, s = (it >> 4) & 15, h = it >> 8;   // dims 4 c .. + 3 and 64 above
        uint2 kl = make_uint2(0u, 0u), kh = kl, vl = kl, vh = kl;
        if (s < lim) {
            const size_t bh = static_cast<size_t>(blk) * p.hkv + h;
            const float ks = p.k_scale[bh], vs = p.v_scale[bh];
            const uint32_t *kc = reinterpret_cast<const uint32_t *>(p.k_codes + (bh * kBlockTokens + s) * kHeadDim) + c;
            const uint32_t *vc = reinterpret_cast<const uint32_t *>(p.v_codes + (bh * kBlockTokens + s) * kHeadDim) + c;
            auto dec = [](uint32_t w, float f, float (&x)[4]) {
                uint32_t h0, h1;
                codes_to_f16(w, h0, h1);
                f16x2_to_f32(h0, x[0], x[1]);
                f16x2_to_f32(h1, x[2], x[3]);
#pragma unroll
                for (int u = 0; u < 4; ++u) x[u] *= f;
            };
            float a[4], b[4], x[4], y[4];
            dec(kc[0], ks, a);
            dec(kc[16], ks, b);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float2 z = cs[4 * c + u];
                x[u] = a[u] * z.x - b[u] * z.y;
                y[u] = b[u] * z.x + a[u] * z.y;
            }
            kl = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
            kh = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
            dec(vc[0], vs, a);
            dec(vc[16], vs, b);
            vl = make_uint2(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]));
            vh = make_uint2(pack_bf16(b[0], b[1]), pack_bf16(b[2], b[3]));
        }
        const size_t dst = ((static_cast<size_t>(row) * p.hkv + h) * kBlockTokens + s) * kHeadDim;
        uint2 *ko = reinterpret_cast<uint2 *>(p.k_out + dst) + c, *vo = reinterpret_cast<uint2 *>(p.v_out + dst) + c;
        ko[0] = kl;
        ko[16] = kh;
        vo[0] = vl;
        vo[16] = vh;
    }
}

}  // namespace

cudaError_t launch_q8_stage(const Q8StageParams &p, cudaStream_t s) {
    q8_stage_kernel<<<dim3(p.max_words, p.num_req), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace lazy

// evict.cu -- each request's table cut to its words of largest accumulated attention weight.
//
// Order of request r's n words: protected ones (the first n_first and last n_last) before all
// others, then by weight, then by index; the first k = min(n, max(keep, 0)) stay, in table order.
// Weights become 32-bit keys of the same order; the k-th key is found by radix selection (8 bits a
// pass, stopping as soon as the bin that holds it is taken whole), ties at that key go to the lowest
// indices, and one ordered compaction writes survivors and evicted words.
//
// A cluster of CTAs takes one request, each a run of its words with the keys in shared memory; the CTAs add up
// their histograms and counts over distributed shared memory.  Latency is the bound: 8 requests of 32768
// words move 2.5 MB (0.4 us at the copy rate) in 15 us, most of it the four passes' barriers and the atomics
// of the histograms; one CTA per request took 48 us for them.  About 16 clusters of such CTAs run at once, so
// that many requests are better off with a CTA each (64 of 8192 words: 15 us, in clusters
// 48; but 32 of 32768: 48 us, in clusters 39 to 45).
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace lazy {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kSmemKeys = 49152;     // words of a CTA whose keys stay in shared memory
constexpr int kCluster = 8;          // CTAs of a cluster
// In clusters where tables of more than kLongWords words (measured for 8 requests: 4096 words 9.4 us in one CTA
// each, 4100 in clusters 9.4, 8192 in one 15.7, in clusters 11.6) and the calls' waves of clusters are few:
// each wave costs about what kWaveWords words cost one CTA.
constexpr int kLongWords = 4096, kWaveWords = 16384, kWave = 16;

// Each request's CTA adds up the words that stay of the requests before it, work that grows with their square; above
// kScanRequests requests a kernel before writes the row pointers (1024 requests 31.7 us without it, 32.6 with; 2048
// 58.5, 58.3; 4096 115, 112; 16384 493, 431; 65536 2619, 1704).
constexpr int kScanRequests = 2048;

__device__ __forceinline__ uint32_t key_of(float m) {
    if (m != m) m = INFINITY;
    m += 0.f;   // -0 as 0
    const uint32_t u = __float_as_uint(m);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Words of request q that stay.
__device__ __forceinline__ int kept_of(const EvictParams &p, int q) {
    const int m = p.table_indptr[q + 1] - p.table_indptr[q];
    return max(0, min(min(m, p.max_words), p.keep[q]));
}
// Sum over the CTA, in all threads; red: [kWarps].
__device__ __forceinline__ int sum_cta(int x, int *red, int warp, int lane) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (lane == 0) red[warp] = x;
    __syncthreads();
    x = red[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The new row pointers, kScanChunk requests a CTA: each adds up the requests before its own, which is read work of
// num_req^2 / (2 kScanChunk) counts in all, and scans its own.
constexpr int kScanPer = 4, kScanChunk = kScanPer * kThreads;
__global__ void __launch_bounds__(kThreads) evict_offsets_kernel(const EvictParams p) {
    __shared__ int red[kWarps], wsum[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r0 = blockIdx.x * kScanChunk;
    int before = 0;
#pragma unroll 8
    for (int q = tid; q < r0; q += kThreads) before += kept_of(p, q);
    before = sum_cta(before, red, warp, lane);
    int k[kScanPer], s = 0;
#pragma unroll
    for (int i = 0; i < kScanPer; ++i) {
        const int q = r0 + tid * kScanPer + i;
        k[i] = q < p.num_req ? kept_of(p, q) : 0;
        s += k[i];
    }
    int inc = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += wsum[w];
    int at = before + inc - s;
    if (blockIdx.x == 0 && tid == 0) p.indptr_out[0] = 0;
#pragma unroll
    for (int i = 0; i < kScanPer; ++i) {
        const int q = r0 + tid * kScanPer + i;
        at += k[i];
        if (q < p.num_req) p.indptr_out[q + 1] = at;
    }
}

// CL: CTAs per request (a cluster).
template <int CL>
__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictParams p, int smem_keys) {
    extern __shared__ uint32_t keys[];
    __shared__ int total[CL > 1 ? 256 : 1];
    __shared__ int hist[2][256];          // of this CTA; two, so that a pass need not wait for readers of the last one
    __shared__ int red[kWarps], cnt_gt[kWarps], cnt_eq[kWarps], cta_cnt[2];
    __shared__ int sel_bin, sel_above, sel_count;
    const int r = blockIdx.x / CL, rank = blockIdx.x % CL;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto sync_request = [&]() {
        if constexpr (CL > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
    };
    // the same shared variable of CTA q of the request
    auto of_rank = [&](int *x, int q) -> int * {
        if constexpr (CL > 1)
            return cg::this_cluster().map_shared_rank(x, q);
        else
            return x;
    };
    const int base = p.table_indptr[0];
    const int beg = p.table_indptr[r], n_all = p.table_indptr[r + 1] - beg;
    const int n = max(0, min(n_all, p.max_words));
    if (tid == 0 && rank == 0 && n_all > p.max_words) set_status(p.d_status, LAZY_DSTATUS_BAD_TABLE);
    const int k = kept_of(p, r);
    // ---- this CTA's words; where the request's survivors go
    const int run = ((n + CL - 1) / CL + 31) / 32 * 32;
    const int lo = min(n, rank * run), hi = min(n, lo + run);
    int before = 0;
    if (p.scanned)
        before = tid == 0 ? p.indptr_out[r] : 0;
    else
        for (int q = tid; q < r; q += kThreads) before += kept_of(p, q);
    const float *mass = p.mass + beg;
    for (int i = lo + tid; i < min(hi, lo + smem_keys); i += kThreads) keys[i - lo] = key_of(mass[i]);
    if (tid < 256) hist[0][tid] = 0;
    const int out = sum_cta(before, red, warp, lane);
    if (tid == 0 && rank == 0 && !p.scanned) {
        if (r == 0) p.indptr_out[0] = 0;
        p.indptr_out[r + 1] = out + k;
    }
    auto key = [&](int i) { return i - lo < smem_keys ? keys[i - lo] : key_of(mass[i]); };
    // ---- the class that the cut goes through: the protected words if they alone are too many, else the others
    const int nf = min(p.n_first, n), nl = min(p.n_last, n - nf), n_prot = nf + nl;
    auto is_prot = [&](int i) { return i < nf || i >= n - nl; };
    const bool cut_prot = k < n_prot;
    int need = cut_prot ? k : k - n_prot;
    const int n_class = cut_prot ? n_prot : n - n_prot;
    const bool none = need == 0, all = need == n_class;
    uint32_t prefix = 0u, mask = 0u;
    bool whole = false;   // every key of the class with (key & mask) == prefix stays
    if (!none && !all) {   // (the same for all CTAs of the request)
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass, buf = pass & 1;
            for (int i = lo + tid; i < hi; i += kThreads) {
                const uint32_t u = key(i);
                if (is_prot(i) == cut_prot && (u & mask) == prefix) atomicAdd(&hist[buf][(u >> shift) & 255u], 1);
            }
            sync_request();
            if (tid < 256) {
                hist[buf ^ 1][tid] = 0;   // read last before the sync
                if constexpr (CL > 1) {
                    int c = 0;
#pragma unroll
                    for (int q = 0; q < CL; ++q) c += of_rank(hist[buf], q)[tid];
                    total[tid] = c;
                }
            }
            if constexpr (CL > 1) __syncthreads();
            if (warp == 0) {
                // lane l: bins 255 - 8 l downwards
                const int *h = CL > 1 ? total : hist[buf];
                int c[8], s = 0;
#pragma unroll
                for (int x = 0; x < 8; ++x) s += c[x] = h[255 - 8 * lane - x];
                int inc = s;
#pragma unroll
                for (int x = 1; x < 32; x <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, inc, x);
                    if (lane >= x) inc += y;
                }
                int above = inc - s;
                if (above < need && need <= inc) {
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        if (above < need && need <= above + c[x]) {
                            sel_bin = 255 - 8 * lane - x;
                            sel_above = above;
                            sel_count = c[x];
                        }
                        above += c[x];
                    }
                }
            }
            __syncthreads();
            prefix |= static_cast<uint32_t>(sel_bin) << shift;
            mask |= 255u << shift;
            need -= sel_above;
            whole = need == sel_count;
            if (whole) break;
            __syncthreads();   // sel_* are read before the next pass writes them
        }
    }
    // 2: stays, 1: stays if among the first `need` of its kind, 0: goes
    auto verdict = [&](int i) {
        if (is_prot(i) != cut_prot) return cut_prot ? 0 : 2;
        if (none || all) return all ? 2 : 0;
        const uint32_t u = key(i) & mask;
        return u > prefix ? 2 : u < prefix ? 0 : whole ? 2 : 1;
    };
    // ---- ordered compaction: a warp takes a run of words
    const int seg = ((hi - lo + kThreads - 1) / kThreads) * 32;
    const int w0 = min(hi, lo + warp * seg), w1 = min(hi, w0 + seg);
    int gt = 0, eq = 0;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int v = i0 + lane < w1 ? verdict(i0 + lane) : 0;
        gt += __popc(__ballot_sync(0xffffffffu, v == 2));
        eq += __popc(__ballot_sync(0xffffffffu, v == 1));
    }
    if (lane == 0) {
        cnt_gt[warp] = gt;
        cnt_eq[warp] = eq;
    }
    __syncthreads();
    int gt_before = lane < warp ? cnt_gt[lane] : 0, eq_before = lane < warp ? cnt_eq[lane] : 0;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
        gt_before += __shfl_xor_sync(0xffffffffu, gt_before, x);
        eq_before += __shfl_xor_sync(0xffffffffu, eq_before, x);
    }
    if constexpr (CL > 1) {
        if (tid == kThreads - 32) {   // the last warp's totals include all warps
            cta_cnt[0] = gt_before + gt;
            cta_cnt[1] = eq_before + eq;
        }
        sync_request();
        for (int q = 0; q < rank; ++q) {
            const int *c = of_rank(cta_cnt, q);
            gt_before += c[0];
            eq_before += c[1];
        }
    }
    int stay = gt_before + min(eq_before, need);   // survivors before this position
    const uint32_t lower = (1u << lane) - 1u;
    const int gone0 = beg - base - out;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const bool in = i < w1;
        const int v = in ? verdict(i) : 0;
        const uint32_t em = __ballot_sync(0xffffffffu, v == 1);
        const bool st = v == 2 || (v == 1 && eq_before + __popc(em & lower) < need);
        const uint32_t sm = __ballot_sync(0xffffffffu, st);
        if (in) {
            const uint32_t w = p.table[beg + i];
            const int pos = stay + __popc(sm & lower);
            if (st) {
                p.table_out[out + pos] = w;
                p.mass_out[out + pos] = mass[i];
            } else if (p.evicted) {
                p.evicted[gone0 + i - pos] = w;
            }
        }
        stay += __popc(sm);
        eq_before += __popc(em);
    }
    if (p.evicted)
        for (int i = n + rank * kThreads + tid; i < n_all; i += CL * kThreads) p.evicted[gone0 + i - k] = p.table[beg + i];
    if constexpr (CL > 1) sync_request();   // shared memory lives until the other CTAs have read it
}

}  // namespace

cudaError_t launch_evict(EvictParams p, cudaStream_t s) {
    p.scanned = p.num_req > kScanRequests;
    if (p.scanned) {
        evict_offsets_kernel<<<(p.num_req + kScanChunk - 1) / kScanChunk, kThreads, 0, s>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const long long waves = (p.num_req + kWave - 1) / kWave;
    const bool cluster = p.max_words > kLongWords + kWaveWords * (waves - 1);
    const int per_cta = cluster ? p.max_words / kCluster + 64 : p.max_words;
    const int smem_keys = per_cta < kSmemKeys ? per_cta : kSmemKeys;
    auto kern = cluster ? evict_kernel<kCluster> : evict_kernel<1>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemKeys * 4);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster ? kCluster : 1;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.num_req * (cluster ? kCluster : 1));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_keys * 4;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p, smem_keys);
}

}  // namespace lazy

// Thinning caches out by accumulated attention: per (layer, sequence) row, find the n lowest-scored
// pages among those that may go, and close the row's table and scores up over them.
#include "kv_device.h"

namespace lorapool {

constexpr int EV_THREADS = 1024;

// A key whose unsigned order is the score's: negative values inverted, NaN above everything, -0 as 0.
__device__ __forceinline__ uint32_t score_key(float v) {
    if (v != v) return 0xffffffffu;
    const uint32_t u = __float_as_uint(v + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t score_key(double v) {
    if (v != v) return ~0ull;
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return u >> 63 ? ~u : u | (1ull << 63);
}

// Key of a page: its token's score, or the float64 sum of its tokens' scores in token order.
__device__ __forceinline__ uint32_t page_key(const float *sc, int32_t page, int32_t, uint32_t) { return score_key(sc[page]); }
__device__ __forceinline__ uint64_t page_key(const float *sc, int32_t page, int32_t tpp, uint64_t) {
    double sum = sc[(int64_t)page * tpp];
    for (int32_t i = 1; i < tpp; ++i) sum += (double)sc[(int64_t)page * tpp + i];
    return score_key(sum);
}

// Exclusive sum over the workgroup of one value per thread, and the total; every thread must call.
__device__ __forceinline__ int block_excl(int v, int *waves, int *total) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int incl = wave_incl_scan(v, lane);
    if (lane == 63) waves[w] = incl;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < EV_THREADS / 64; ++i) {
        const int x = waves[i];
        before += i < w ? x : 0;
        all += x;
    }
    __syncthreads();
    *total = all;
    return before + incl - v;
}

// One workgroup per (sequence, layer).  KEY: uint32_t where a page is one token, else uint64_t.
template <typename KEY>
__global__ __launch_bounds__(EV_THREADS) void k_kv_evict(KvEvict e) {
    __shared__ int hist[256], waves[EV_THREADS / 64], pick[2];
    __shared__ int32_t list[EV_THREADS];
    const int32_t b = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x, tpp = e.tpp;
    const int64_t row = (int64_t)layer * e.n_seq + b, width = (int64_t)e.max_pages * tpp;
    const int32_t *kt = e.table + row * 2 * e.max_pages, *vt = kt + e.max_pages;
    int32_t *ko = e.table_out + row * 2 * e.max_pages, *vo = ko + e.max_pages;
    const float *sc = e.scores + row * width;
    float *so = e.scores_out + row * width;
    int32_t *kd = e.dropped + row * 2 * e.max_drop, *vd = kd + e.max_drop;
    const int32_t len = e.lens[b];
    if (len < 0 || len > width) {   // left as it is
        if (e.table_out != e.table)
            for (int32_t i = tid; i < 2 * e.max_pages; i += EV_THREADS) ko[i] = kt[i];
        if (e.scores_out != e.scores)
            for (int64_t i = tid; i < width; i += EV_THREADS) so[i] = sc[i];
        for (int32_t i = tid; i < 2 * e.max_drop; i += EV_THREADS) kd[i] = -1;
        if (tid == 0 && layer == 0) {
            atomicOr(e.err, DEV_ERR_LEN);
            e.lens_out[b] = len;
            e.n_dropped[b] = 0;
        }
        return;
    }
    const int32_t n_pages = (len + tpp - 1) / tpp;
    const int32_t lo = (e.keep_first + tpp - 1) / tpp, hi = max(lo, (len - e.keep_last) < 0 ? 0 : (len - e.keep_last) / tpp);
    const int32_t over = len > e.budget ? (len - e.budget + tpp - 1) / tpp : 0;
    const int32_t n_drop = min(min(e.max_drop, hi - lo), over);

    // the n_drop-th lowest key, a byte at a time from the top; `left`: how many of that very key go
    KEY prefix = 0, mask = 0;
    int left = n_drop;
    if (n_drop > 0) {
        for (int shift = (int)sizeof(KEY) * 8 - 8; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int32_t p = lo + tid; p < hi; p += EV_THREADS) {
                const KEY k = page_key(sc, p, tpp, KEY(0));
                if ((k & mask) == prefix) atomicAdd(&hist[(int)(k >> shift) & 255], 1);
            }
            __syncthreads();
            if (tid < 64) {   // the bin in which the count reaches `left`
                int h[4], sum = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) sum += h[i] = hist[tid * 4 + i];
                int before = wave_incl_scan(sum, tid) - sum;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (before < left && left <= before + h[i]) { pick[0] = tid * 4 + i; pick[1] = left - before; }
                    before += h[i];
                }
            }
            __syncthreads();
            prefix |= (KEY)pick[0] << shift;
            mask |= (KEY)255 << shift;
            left = pick[1];
            __syncthreads();
        }
    }

    // close the rows up, EV_THREADS pages at a time; what a step writes lies before what later steps
    // read, so the rows may be changed in place
    const int32_t new_len = len - n_drop * tpp;
    int32_t kept0 = 0, gone0 = 0, ties0 = 0;
    for (int32_t p0 = 0; p0 < n_pages; p0 += EV_THREADS) {
        const int32_t p = p0 + tid;
        const bool held = p < n_pages;
        int32_t kp = -1, vp = -1;
        KEY key = 0;
        bool below = false, tie = false;
        if (held) {
            kp = kt[p];
            vp = vt[p];
            if (n_drop > 0 && p >= lo && p < hi) {
                key = page_key(sc, p, tpp, KEY(0));
                below = key < prefix;
                tie = key == prefix;
            }
        }
        int n_ties, n_kept;
        const int tie_rank = ties0 + block_excl(tie, waves, &n_ties);
        const bool go = below || (tie && tie_rank < left);
        const bool stay = held && !go;
        const int my = block_excl(stay, waves, &n_kept);
        if (stay) {
            ko[kept0 + my] = kp;
            vo[kept0 + my] = vp;
            list[my] = p;
        } else if (held) {
            const int32_t d = gone0 + (tid - my);
            kd[d] = kp;
            vd[d] = vp;
        }
        __syncthreads();
        const int64_t n_tok = (int64_t)n_kept * tpp;
        for (int64_t i0 = 0; i0 < n_tok; i0 += EV_THREADS) {
            const int64_t i = i0 + tid;
            float v = 0.f;
            if (i < n_tok) {
                const int32_t l = (int32_t)(i / tpp);
                v = sc[(int64_t)list[l] * tpp + (i - (int64_t)l * tpp)];
            }
            __syncthreads();
            const int64_t dst = (int64_t)kept0 * tpp + i;
            if (i < n_tok && dst < new_len) so[dst] = v;
        }
        __syncthreads();
        kept0 += n_kept;
        gone0 += min((int32_t)EV_THREADS, n_pages - p0) - n_kept;
        ties0 += n_ties;
    }
    for (int32_t i = kept0 + tid; i < e.max_pages; i += EV_THREADS) ko[i] = vo[i] = -1;
    for (int64_t i = new_len + tid; i < width; i += EV_THREADS) so[i] = 0.f;
    for (int32_t i = n_drop + tid; i < e.max_drop; i += EV_THREADS) kd[i] = vd[i] = -1;
    if (tid == 0 && layer == 0) {
        e.lens_out[b] = new_len;
        e.n_dropped[b] = n_drop;
    }
}

hipError_t launch_kv_evict(const KvEvict &e, hipStream_t s) {
    const dim3 grid(e.n_seq, e.layers);
    if (e.tpp == 1) hipLaunchKernelGGL(k_kv_evict<uint32_t>, grid, dim3(EV_THREADS), 0, s, e);
    else hipLaunchKernelGGL(k_kv_evict<uint64_t>, grid, dim3(EV_THREADS), 0, s, e);
    return hipGetLastError();
}

}  // namespace lorapool

// New tokens' K and V rows into their pages.  A copy: bound by the bytes moved, each row read and
// written once, 16 bytes per lane; for few tokens by the two look-ups before it (sequence and length, then page).
// 8 x 512 tokens of 8 KiB rows (134 MB moved): 25.3 - 26.8 us, 5.0 - 5.3 TB/s, a plain copy of 1 GiB reaches 5.5;
// 64 tokens (2 MB): 4.4 us.
#include <algorithm>

#include "kv_device.h"

namespace lorapool {

// A workgroup takes `per` neighbouring tokens: looks their sequences, positions and pages up together, then copies
// their K and V rows, eight pieces of a thread on their way at a time.
constexpr int WRITE_MOST = 2;
__global__ __launch_bounds__(256) void k_kv_write(KvArgs a, const char *__restrict__ k, int64_t ldk_bytes,
                                                  const char *__restrict__ v, int64_t ldv_bytes, int32_t per) {
    __shared__ int32_t seq[WRITE_MOST];
    __shared__ int64_t to[2 * WRITE_MOST];                  // where a token's K and V go; -1: nowhere
    const int32_t t0 = blockIdx.x * per, n = min(per, a.T - t0), tid = threadIdx.x;
    if (blockIdx.x == 0) check_seqs(a);
    if (a.q_start) {
        if (tid < WRITE_MOST) seq[tid] = -1;
        __syncthreads();
        for (int32_t b = tid; b < a.n_seq; b += 256) {      // the rows of this workgroup that are sequence b's
            const int32_t s0 = a.q_start[b], s1 = a.q_start[b + 1];
            if (s0 < 0 || s1 > a.T) continue;
            for (int32_t t = max(s0, t0); t < min(s1, t0 + n); ++t) atomicMax(&seq[t - t0], b);
        }
        __syncthreads();
    }
    if (tid < n) {
        const int32_t t = t0 + tid, b = a.q_start ? seq[tid] : t < a.n_seq ? t : -1;
        int64_t ko = -1, vo = -1;
        if (b >= 0) {
            const SeqRows s = seq_rows(a, b);
            if (s.n > 0) {
                const int32_t *row = a.table + (int64_t)b * 2 * a.max_pages, pos = s.n - s.m + (t - s.first);
                ko = token_offset(a, row, pos);
                vo = token_offset(a, row + a.max_pages, pos);
                if (ko < 0 || vo < 0) {
                    record(a, DEV_ERR_PAGE);
                    ko = vo = -1;
                }
            }
        }
        to[2 * tid] = ko;
        to[2 * tid + 1] = vo;
    }
    __syncthreads();
    const int32_t units = a.tok_bytes / 16;
    int32_t row = 0, u = tid;                               // K of the first token, V of it, K of the second, ...
    while (u >= units) { u -= units; ++row; }
    while (row < 2 * n) {
        u32x4_t piece[8];
        char *dst[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dst[i] = nullptr;
            if (row < 2 * n) {
                const int64_t at = to[row];
                const char *src = row & 1 ? v + (t0 + row / 2) * ldv_bytes : k + (t0 + row / 2) * ldk_bytes;
                if (at >= 0) {
                    dst[i] = a.pages + at + 16 * u;
                    piece[i] = load16(src + 16 * u);
                }
                u += 256;
                while (u >= units) { u -= units; ++row; }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (dst[i]) store16(dst[i], piece[i]);
    }
}

hipError_t launch_kv_write(int dtype, const KvArgs &a, const void *k, int64_t ldk, const void *v, int64_t ldv,
                           hipStream_t s) {
    const int64_t elem = dtype == LORA_F32 ? 4 : 2;
    // Two tokens a workgroup once there are 1024 such workgroups (8 x 512 tokens of 8 KiB: 25.4 us, one token each 28.6, eight
    // 30.0); one below that (64 tokens: 4.4 us, two each 5.5).
    const int32_t per = std::max(1, std::min(WRITE_MOST, a.T / 1024));
    hipLaunchKernelGGL(k_kv_write, dim3((unsigned)((a.T + per - 1) / per)), dim3(256), 0, s, a, (const char *)k, ldk * elem,
                       (const char *)v, ldv * elem, per);
    return hipGetLastError();
}

}  // namespace lorapool

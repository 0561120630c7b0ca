// New tokens' K and V rows into their pages.  A copy: bound by the bytes moved, each row read and
// written once, 16 bytes per lane.
#include "kv_device.h"

namespace lorapool {

// One workgroup per new token: find its sequence and position, copy its K row and its V row.
__global__ __launch_bounds__(256) void k_kv_write(KvArgs a, const char *__restrict__ k, int64_t ldk_bytes,
                                                  const char *__restrict__ v, int64_t ldv_bytes) {
    __shared__ int32_t sh;
    const int32_t t = blockIdx.x;
    if (t == 0) check_seqs(a);
    const int32_t b = find_seq(a, t, &sh);
    if (b < 0) return;
    const SeqRows s = seq_rows(a, b);
    if (s.n == 0) return;
    const int32_t pos = s.n - s.m + (t - s.first);
    const int32_t *row = a.table + (int64_t)b * 2 * a.max_pages;
    const int64_t ko = token_offset(a, row, pos), vo = token_offset(a, row + a.max_pages, pos);
    if (ko < 0 || vo < 0) {
        if (threadIdx.x == 0) record(a, DEV_ERR_PAGE);
        return;
    }
    const int32_t units = a.tok_bytes / 16;
    for (int32_t i = threadIdx.x; i < 2 * units; i += blockDim.x) {
        const bool is_v = i >= units;
        const int32_t u = is_v ? i - units : i;
        const int64_t dst = is_v ? vo : ko;
        const char *src = is_v ? v + t * ldv_bytes : k + t * ldk_bytes;
        store16(a.pages + dst + 16 * u, load16(src + 16 * u));
    }
}

hipError_t launch_kv_write(int dtype, const KvArgs &a, const void *k, int64_t ldk, const void *v, int64_t ldv,
                           hipStream_t s) {
    const int64_t elem = dtype == LORA_F32 ? 4 : 2;
    hipLaunchKernelGGL(k_kv_write, dim3((unsigned)a.T), dim3(256), 0, s, a, (const char *)k, ldk * elem,
                       (const char *)v, ldv * elem);
    return hipGetLastError();
}

}  // namespace lorapool

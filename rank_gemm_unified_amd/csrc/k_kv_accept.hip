// Which drafted nodes the model agrees with, and their K and V closed up behind the tokens before.
//
// From the root the path goes on to the first child whose token is the one the model chose at its parent: a wave
// compares all nodes with the current one at once.  Every workgroup walks by itself (the chain of a few compares is
// shorter than a second launch) and then moves the path's K and V rows in one layer.  Node path[i] goes to place i, and
// path[i] >= i and rises, so no move overwrites what a later one reads; a thread reads eight rows' pieces before it
// writes the first, and each thread has its own 16 bytes of every row.  64 trees of 16 nodes in 32 layers of 32 heads: a call
// takes 17 to 18 us on several cards for 69 MB (its kernel in traces 16.5 and 17.1, 4.1 TB/s), two rounds of workgroups, each the
// chain rows -> walk -> pages -> move (on a card where it takes 17.0: by 128 threads a workgroup, in one round, 17.7, by 512 19.8);
// one tree: 4 us, that chain.
#include "kv_device.h"

namespace lorapool {

__global__ __launch_bounds__(256) void k_kv_accept(KvAccept c) {
    __shared__ int32_t target[LORA_MAX_TREE], path[LORA_MAX_TREE];
    __shared__ int64_t src[LORA_MAX_TREE], dst[LORA_MAX_TREE];
    __shared__ int32_t steps;
    const KvArgs &a = c.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t b = blockIdx.y, which = blockIdx.x;       // layer which / 2, K or V
    SeqRows sq = seq_rows(a, b);
    if (sq.m > c.max_nodes) {
        sq.m = 0;
        sq.err = DEV_ERR_LEN;
    }
    if (which == 0 && tid == 0) record(a, sq.err);
    if (sq.m == 0 || sq.n == 0) {                           // nothing drafted
        if (which == 0) {
            for (int32_t i = tid; i < c.max_nodes; i += 256) c.path[(int64_t)b * c.max_nodes + i] = -1;
            if (tid == 0) {
                c.n_path[b] = 0;
                c.next[b] = -1;
            }
        }
        return;
    }
    for (int32_t i = tid; i < sq.m; i += 256) target[i] = c.targets[sq.first + i];
    __syncthreads();
    if (wave == 0) {
        int32_t parent[LORA_MAX_TREE / 64], token[LORA_MAX_TREE / 64];
#pragma unroll
        for (int x = 0; x < LORA_MAX_TREE / 64; ++x) {
            const int32_t i = 64 * x + lane;
            parent[x] = i > 0 && i < sq.m ? c.parents[sq.first + i] : -1;
            token[x] = i > 0 && i < sq.m ? c.tokens[sq.first + i] : 0;
        }
        int32_t node = 0, k = 0;
        for (;;) {
            if (lane == 0) path[k] = node;
            ++k;
            const int32_t want = target[node];
            int32_t next = -1;
#pragma unroll
            for (int x = 0; x < LORA_MAX_TREE / 64; ++x) {
                const uint64_t hit = __ballot(parent[x] == node && token[x] == want && 64 * x + lane > node);
                if (next < 0 && hit) next = 64 * x + __ffsll((long long)hit) - 1;
            }
            if (next < 0) break;
            node = uniform(next);
        }
        if (lane == 0) steps = k;
    }
    __syncthreads();
    const int32_t k = steps, old = sq.n - sq.m;
    if (which == 0) {
        for (int32_t i = tid; i < c.max_nodes; i += 256) c.path[(int64_t)b * c.max_nodes + i] = i < k ? path[i] : -1;
        if (tid == 0) {
            c.lens_out[b] = old + k;
            c.n_path[b] = k;
            c.next[b] = target[path[k - 1]];
        }
    }
    const int32_t *row = a.table + (((int64_t)(which >> 1) * a.n_seq + b) * 2 + (which & 1)) * a.max_pages;
    for (int32_t i = tid; i < k; i += 256) {
        int64_t s = -1, d = -1;
        if (path[i] != i) {
            s = token_offset(a, row, old + path[i]);
            d = token_offset(a, row, old + i);
            if (s < 0 || d < 0) {
                record(a, DEV_ERR_PAGE);
                s = d = -1;
            }
        }
        src[i] = s;
        dst[i] = d;
    }
    __syncthreads();
    for (int32_t u = tid; u < a.tok_bytes / 16; u += 256)
        for (int32_t i0 = 1; i0 < k; i0 += 8) {
            u32x4_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + i < k && src[i0 + i] >= 0) v[i] = load16(a.pages + src[i0 + i] + 16 * u);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + i < k && src[i0 + i] >= 0) store16(a.pages + dst[i0 + i] + 16 * u, v[i]);
        }
}

hipError_t launch_kv_accept(const KvAccept &c, hipStream_t s) {
    hipLaunchKernelGGL(k_kv_accept, dim3((unsigned)(2 * c.layers), (unsigned)c.a.n_seq), dim3(256), 0, s, c);
    return hipGetLastError();
}

}  // namespace lorapool

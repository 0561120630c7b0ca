// Attention over the paged cache: one row of queries at a time.
#include "kv_device.h"

namespace lorapool {

// One workgroup per (row, head): its four waves take the tokens in turn, each with a running maximum
// and sum of its own; the four are joined in LDS.
template <typename E, int HD>
__global__ __launch_bounds__(256) void k_kv_rows(KvArgs a, KvAttend at, float2 *__restrict__ stats) {
    constexpr int PER = HD / 64;
    __shared__ int32_t sh;
    __shared__ float part[4][HD], pm[4], pl[4];
    const int32_t t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (t == 0 && h == 0) check_seqs(a);
    const int32_t b = find_seq(a, t, &sh);
    if (b < 0) return;
    const SeqRows s = seq_rows(a, b);
    const int32_t seen = s.n == 0 ? 0 : s.n - s.m + (t - s.first) + 1;   // tokens this row reads
    const int32_t *krow = a.table + (int64_t)b * 2 * a.max_pages, *vrow = krow + a.max_pages;
    const int64_t head_bytes = (int64_t)(h / a.group) * HD * sizeof(E);
    const E *q = (const E *)at.q + t * at.ldq + (int64_t)h * HD;
    float qf[PER], acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        qf[i] = to_f32(q[lane * PER + i]);
        acc[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    int bad = 0;
    for (int32_t j = wave; j < seen; j += 4) {
        const int64_t ko = token_offset(a, krow, j), vo = token_offset(a, vrow, j);
        if (ko < 0 || vo < 0) { bad = DEV_ERR_PAGE; continue; }
        const E *kp = (const E *)(a.pages + ko + head_bytes), *vp = (const E *)(a.pages + vo + head_bytes);
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) d += qf[i] * to_f32(kp[lane * PER + i]);
        const float x = wave_sum(d) * at.scale;
        const float mn = fmaxf(m, x), ms = mn == -INFINITY ? 0.f : mn;
        const float c = __expf(m - ms), p = __expf(x - ms);
        l = l * c + p;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = acc[i] * c + p * to_f32(vp[lane * PER + i]);
        m = mn;
    }
    if (bad && lane == 0) record(a, bad);
#pragma unroll
    for (int i = 0; i < PER; ++i) part[wave][lane * PER + i] = acc[i];
    if (lane == 0) { pm[wave] = m; pl[wave] = l; }
    __syncthreads();
    float M = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
    const float Ms = M == -INFINITY ? 0.f : M;
    float L = 0.f, w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = __expf(pm[i] - Ms);
        L += pl[i] * w[i];
    }
    E *o = (E *)at.out + t * at.ldo + (int64_t)h * HD;
    for (int32_t d = threadIdx.x; d < HD; d += 256) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) v += part[i][d] * w[i];
        from_f32(o + d, L == 0.f ? 0.f : v / L);
    }
    if (stats && threadIdx.x == 0) stats[(int64_t)t * a.n_heads + h] = make_float2(Ms, L == 0.f ? 0.f : 1.f / L);
}

// scores[b][t] = prior + sum over the sequence's new rows and heads of the weight of token t.  One wave
// per token; the weights are computed again from the rows' statistics.
template <typename E, int HD>
__global__ __launch_bounds__(256) void k_kv_scores(KvArgs a, KvAttend at, const float2 *__restrict__ stats) {
    constexpr int PER = HD / 64;
    const int32_t b = blockIdx.y, lane = threadIdx.x & 63, j = blockIdx.x * 4 + (threadIdx.x >> 6);
    const SeqRows s = seq_rows(a, b);
    if (j >= s.n) return;
    const int32_t *krow = a.table + (int64_t)b * 2 * a.max_pages;
    const int64_t ko = token_offset(a, krow, j), vo = token_offset(a, krow + a.max_pages, j);
    float sum = 0.f;
    if (ko >= 0 && vo >= 0) {
        const int32_t r0 = max(0, j - (s.n - s.m));   // the first new row that sees token j
        for (int32_t h = 0; h < a.n_heads; ++h) {
            const E *kp = (const E *)(a.pages + ko) + (h / a.group) * HD;
            float kf[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) kf[i] = to_f32(kp[lane * PER + i]);
            for (int32_t r = r0; r < s.m; ++r) {
                const int64_t t = s.first + r;
                const E *q = (const E *)at.q + t * at.ldq + (int64_t)h * HD;
                float d = 0.f;
#pragma unroll
                for (int i = 0; i < PER; ++i) d += to_f32(q[lane * PER + i]) * kf[i];
                const float2 st = stats[t * a.n_heads + h];
                sum += __expf(wave_sum(d) * at.scale - st.x) * st.y;
            }
        }
    }
    const int64_t at_ = (int64_t)b * at.score_ld + j;
    if (lane == 0) at.scores[at_] = (at.prior ? at.prior[at_] : 0.f) + sum;
}

size_t kv_chunk_ws_bytes(int, const lora_kv_layout_t &l, int32_t, int64_t T, int64_t, bool scores) {
    return scores ? (size_t)T * l.n_heads * 8 : 0;
}

template <typename E, int HD>
static hipError_t rows(const KvArgs &a, const KvAttend &at, hipStream_t s) {
    float2 *stats = at.scores ? (float2 *)at.ws : nullptr;
    hipLaunchKernelGGL((k_kv_rows<E, HD>), dim3(a.T, a.n_heads), dim3(256), 0, s, a, at, stats);
    if (at.scores)
        hipLaunchKernelGGL((k_kv_scores<E, HD>), dim3((a.cap + 3) / 4, a.n_seq), dim3(256), 0, s, a, at, stats);
    return hipGetLastError();
}

template <typename E>
static hipError_t by_dim(const KvArgs &a, const KvAttend &at, hipStream_t s) {
    return a.head_dim == 64 ? rows<E, 64>(a, at, s) : a.head_dim == 128 ? rows<E, 128>(a, at, s) : rows<E, 256>(a, at, s);
}

hipError_t launch_kv_chunk(int dtype, const KvArgs &a, const KvAttend &at, hipStream_t s) {
    return dtype == LORA_F32 ? by_dim<float>(a, at, s) : by_dim<uint16_t>(a, at, s);
}

}  // namespace lorapool

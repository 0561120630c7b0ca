// Thinning caches out by accumulated attention: per (layer, sequence) row, find the n lowest-scored
// pages among those that may go, and close the row's table and scores up over them.
// The bytes are few (a row is read and written once); what costs is the chain: read, select 11 bits at a time
// (three passes for float32 keys, six at most for float64), place, close up.  32 layers of 16 sequences of up to 4096
// one-token pages (37 MB): 17.0 us, 2.2 TB/s, two workgroups a CU and one round of them; 4 sequences of up to 2003 tokens,
// five a page: 6.4 us.  The rows read from memory at every pass: 32.5 and 17.4 us.  Rows over 8192 pages do that still:
// one of 32768 one-token pages 89.0 us, 64 of them (8 layers, 50 MB) 98.0.
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

// What a row is to lose.
struct Plan1 {
    int32_t n_pages, lo, hi, n_drop;   // pages it holds; those that may go are [lo, hi); how many go
    int32_t new_len;
};
__device__ __forceinline__ Plan1 plan_row(const KvEvict &e, int32_t len) {
    Plan1 p;
    p.n_pages = (len + e.tpp - 1) / e.tpp;
    p.lo = (e.keep_first + e.tpp - 1) / e.tpp;
    p.hi = max(p.lo, len < e.keep_last ? 0 : (len - e.keep_last) / e.tpp);
    const int32_t over = len > e.budget ? (len - e.budget + e.tpp - 1) / e.tpp : 0;
    p.n_drop = min(min(e.max_drop, p.hi - p.lo), over);
    p.new_len = len - p.n_drop * e.tpp;
    return p;
}

// A row whose length is out of range is left as it is.
__device__ __forceinline__ bool left_alone(const KvEvict &e, int32_t len, int64_t width, const int32_t *kt, int32_t *ko,
                                           const float *sc, float *so, int32_t *kd, int threads) {
    if (len >= 0 && len <= width) return false;
    if (e.table_out != e.table)
        for (int32_t i = threadIdx.x; i < 2 * e.max_pages; i += threads) ko[i] = kt[i];
    if (e.scores_out != e.scores)
        for (int64_t i = threadIdx.x; i < width; i += threads) so[i] = sc[i];
    for (int32_t i = threadIdx.x; i < 2 * e.max_drop; i += threads) kd[i] = -1;
    if (threadIdx.x == 0 && blockIdx.y == 0) {
        atomicOr(e.err, DEV_ERR_LEN);
        e.lens_out[blockIdx.x] = len;
        e.n_dropped[blockIdx.x] = 0;
    }
    return true;
}

// Behind what stayed and what left.
__device__ __forceinline__ void finish_row(const KvEvict &e, int32_t b, int32_t layer, const Plan1 &p, int64_t width, int32_t *ko,
                                           int32_t *vo, float *so, int32_t *kd, int32_t *vd, int threads) {
    for (int32_t i = p.n_pages - p.n_drop + threadIdx.x; i < e.max_pages; i += threads) ko[i] = vo[i] = -1;
    for (int64_t i = p.new_len + (int32_t)threadIdx.x; i < width; i += threads) so[i] = 0.f;
    for (int32_t i = p.n_drop + threadIdx.x; i < e.max_drop; i += threads) kd[i] = vd[i] = -1;
    if (threadIdx.x == 0 && layer == 0) {
        e.lens_out[b] = p.new_len;
        e.n_dropped[b] = p.n_drop;
    }
}

// Rows of up to THREADS * I pages: a thread keeps I neighbouring pages in registers, keys, table entries and (where a
// page is one token) scores, all loaded at once, so that the selection and the closing up need no second look.
// Bins of 11 bits, two copies: scores lie close together, and equal bins of a wave are counted one after the other.
constexpr int RG_THREADS = 512, RG_BINS = 2048;
typedef u32x4_t any16 __attribute__((aligned(4)));

// Exclusive sums over the workgroup of two counts (at most 16 bits each) at once.
__device__ __forceinline__ uint32_t regs_excl(uint32_t v, uint32_t *waves) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const uint32_t incl = (uint32_t)wave_incl_scan((int)v, lane);
    if (lane == 63) waves[w] = incl;
    __syncthreads();
    uint32_t before = 0;
#pragma unroll
    for (int i = 0; i < RG_THREADS / 64; ++i) before += i < w ? waves[i] : 0;
    __syncthreads();
    return before + incl - v;
}

template <typename KEY, int I>
__global__ __launch_bounds__(RG_THREADS) void k_kv_evict_regs(KvEvict e) {
    constexpr bool ONE = sizeof(KEY) == 4;
    constexpr int WORDS = RG_THREADS * I > 2 * RG_BINS ? RG_THREADS * I : 2 * RG_BINS;
    __shared__ uint32_t buf[WORDS], waves[RG_THREADS / 64], pick[3];
    const int32_t b = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x, tpp = e.tpp;
    const int64_t row = (int64_t)layer * e.n_seq + b, width = (int64_t)e.max_pages * tpp;
    const int32_t *kt = e.table + row * 2 * e.max_pages, *vt = kt + e.max_pages;
    int32_t *ko = e.table_out + row * 2 * e.max_pages, *vo = ko + e.max_pages;
    const float *sc = e.scores + row * width;
    float *so = e.scores_out + row * width;
    int32_t *kd = e.dropped + row * 2 * e.max_drop, *vd = kd + e.max_drop;
    const int32_t len = e.lens[b];
    if (left_alone(e, len, width, kt, ko, sc, so, kd, RG_THREADS)) return;
    const Plan1 pl = plan_row(e, len);
    const int32_t p0 = tid * I;
    int32_t kid[I], vid[I];
    float tok[I];
    KEY key[I];
    if (I % 4 == 0 && p0 + I <= pl.n_pages) {               // 16 bytes at a time, from any 4-byte boundary
#pragma unroll
        for (int i = 0; i + 4 <= I; i += 4) {
            const any16 k = *(const any16 *)(kt + p0 + i), v = *(const any16 *)(vt + p0 + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                kid[i + j] = (int32_t)k[j];
                vid[i + j] = (int32_t)v[j];
            }
            if constexpr (ONE) {
                const any16 t = *(const any16 *)(sc + p0 + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) tok[i + j] = __uint_as_float(t[j]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int32_t p = p0 + i;
            const bool held = p < pl.n_pages;
            kid[i] = held ? kt[p] : -1;
            vid[i] = held ? vt[p] : -1;
            if constexpr (ONE) tok[i] = held ? sc[p] : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int32_t p = p0 + i;
        if constexpr (ONE) key[i] = score_key(tok[i]);
        else key[i] = p >= pl.lo && p < pl.hi ? page_key(sc, p, tpp, KEY(0)) : KEY(0);
    }
    // the n_drop-th lowest key, 11 bits at a time from the top, until every key with these bits goes
    int shift = sizeof(KEY) * 8;
    KEY prefix = 0;                                         // the bits from `shift` up
    uint32_t left = pl.n_drop;                              // how many of the keys with them go
    if (pl.n_drop > 0) {
        for (;;) {
            const int bits = shift < 11 ? shift : 11, at = shift - bits;
            for (int i = tid; i < 2 * RG_BINS; i += RG_THREADS) buf[i] = 0;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < I; ++i) {
                const int32_t p = p0 + i;
                const bool in = p >= pl.lo && p < pl.hi && (shift == sizeof(KEY) * 8 || key[i] >> shift == prefix);
                if (in) atomicAdd(&buf[(tid & 1) * RG_BINS + ((uint32_t)(key[i] >> at) & ((1u << bits) - 1))], 1u);
            }
            __syncthreads();
            constexpr int PB = RG_BINS / RG_THREADS;        // bins a thread looks at
            uint32_t h[PB], sum = 0;
#pragma unroll
            for (int i = 0; i < PB; ++i) sum += h[i] = buf[tid * PB + i] + buf[RG_BINS + tid * PB + i];
            uint32_t before = regs_excl(sum, waves);
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                if (before < left && left <= before + h[i]) { pick[0] = tid * PB + i; pick[1] = left - before; pick[2] = h[i]; }
                before += h[i];
            }
            __syncthreads();
            prefix = (shift == sizeof(KEY) * 8 ? KEY(0) : prefix << bits) | pick[0];
            left = pick[1];
            shift = at;
            const bool all = pick[2] == left;
            __syncthreads();
            if (shift == 0 || all) break;
        }
    }
    // places: what goes is below the threshold, or one of the first `left` at it
    uint32_t below = 0, ties = 0;
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int32_t p = p0 + i;
        if (pl.n_drop > 0 && p >= pl.lo && p < pl.hi) {
            below += key[i] >> shift < prefix ? 1 : 0;
            ties += key[i] >> shift == prefix ? 1 : 0;
        }
    }
    const uint32_t excl = regs_excl(below | ties << 16, waves);
    uint32_t gone = (excl & 0xffff) + min(excl >> 16, left), tie = excl >> 16;
    const uint32_t n_kept = pl.n_pages - pl.n_drop;
    uint32_t to[I];                                         // place among those that stay, then those that go
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int32_t p = p0 + i;
        bool go = false;
        if (pl.n_drop > 0 && p >= pl.lo && p < pl.hi) {
            if (key[i] >> shift < prefix) go = true;
            else if (key[i] >> shift == prefix) go = tie++ < left;
        }
        to[i] = go ? n_kept + gone : p - gone;
        gone += go;
    }
    // through LDS, so that whole lines leave; everything has been read, so the rows may be changed in place
    auto move = [&](auto value, uint32_t *out, uint32_t *out_gone) {
#pragma unroll
        for (int i = 0; i < I; ++i)
            if (p0 + i < pl.n_pages) buf[to[i]] = value(i);
        __syncthreads();
        for (int32_t x = tid; x < pl.n_pages; x += RG_THREADS) {
            if (x < (int32_t)n_kept) out[x] = buf[x];
            else if (out_gone) out_gone[x - n_kept] = buf[x];
        }
        __syncthreads();
    };
    move([&](int i) { return (uint32_t)kid[i]; }, (uint32_t *)ko, (uint32_t *)kd);
    move([&](int i) { return (uint32_t)vid[i]; }, (uint32_t *)vo, (uint32_t *)vd);
    if constexpr (ONE) {
        move([&](int i) { return __float_as_uint(tok[i]); }, (uint32_t *)so, nullptr);
    } else {
        // tokens: so many at a time, read before they are written
#pragma unroll
        for (int i = 0; i < I; ++i)
            if (p0 + i < pl.n_pages) buf[to[i]] = p0 + i;
        __syncthreads();
        const int64_t n_tok = (int64_t)n_kept * tpp;
        for (int64_t x0 = 0; x0 < n_tok; x0 += 4 * RG_THREADS) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t x = x0 + i * RG_THREADS + tid;
                if (x < n_tok) {
                    const int32_t p = (int32_t)x / tpp;
                    v[i] = sc[(int64_t)buf[p] * tpp + ((int32_t)x - p * tpp)];
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t x = x0 + i * RG_THREADS + tid;
                if (x < pl.new_len) so[x] = v[i];
            }
            __syncthreads();
        }
    }
    finish_row(e, b, layer, pl, width, ko, vo, so, kd, vd, RG_THREADS);
}

// Longer rows.
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
    if (left_alone(e, len, width, kt, ko, sc, so, kd, EV_THREADS)) return;
    const Plan1 pl = plan_row(e, len);
    const int32_t n_pages = pl.n_pages, lo = pl.lo, hi = pl.hi, n_drop = pl.n_drop, new_len = pl.new_len;

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
    finish_row(e, b, layer, pl, width, ko, vo, so, kd, vd, EV_THREADS);
}

template <typename KEY>
static void launch_rows(const KvEvict &e, hipStream_t s) {
    const dim3 grid(e.n_seq, e.layers);
    const int32_t per = (e.max_pages + RG_THREADS - 1) / RG_THREADS;
    if (per <= 1) hipLaunchKernelGGL((k_kv_evict_regs<KEY, 1>), grid, dim3(RG_THREADS), 0, s, e);
    else if (per <= 4) hipLaunchKernelGGL((k_kv_evict_regs<KEY, 4>), grid, dim3(RG_THREADS), 0, s, e);
    else if (per <= 8) hipLaunchKernelGGL((k_kv_evict_regs<KEY, 8>), grid, dim3(RG_THREADS), 0, s, e);
    else if (per <= 16) hipLaunchKernelGGL((k_kv_evict_regs<KEY, 16>), grid, dim3(RG_THREADS), 0, s, e);
    else hipLaunchKernelGGL(k_kv_evict<KEY>, grid, dim3(EV_THREADS), 0, s, e);
}

hipError_t launch_kv_evict(const KvEvict &e, hipStream_t s) {
    if (e.tpp == 1) launch_rows<uint32_t>(e, s);
    else launch_rows<uint64_t>(e, s);
    return hipGetLastError();
}

}  // namespace lorapool

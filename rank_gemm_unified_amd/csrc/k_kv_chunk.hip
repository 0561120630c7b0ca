// Causal attention of many new tokens per sequence over the paged cache (a prompt, or its next part).
//
// Matrix products bound it: 4 * head_dim operations for every (query row, token) pair that the mask lets
// through.  One workgroup takes 128 query rows of one K/V head -- 128 tokens of one head, or 64 or 32 of
// two or four heads that share it -- and walks the sequence's tokens NT at a time with a running maximum
// and sum.  K and V go from their pages straight to LDS (16 bytes a lane, gathered row by row, double
// buffered); a wave's 32 rows stay in registers, as columns:
//     S^T = K Q^T   (rows tokens, columns query rows)       out^T += V^T P^T   (rows dims)
// so that a lane holds one query row's logits, and the products of the first are, after the softmax,
// in place as the right operand of the second: the weights never leave their registers.  V^T comes out of
// LDS through the transposing read.  Two workgroups a CU: one's softmax runs under the other's products.
//
// bfloat16, head_dim 128, 32 heads: the last 2048 of 16384 tokens on 8 K/V heads (515 GFLOP) 558 - 577 us on several cards,
// 890 - 925 TFLOP/s, where a large matrix product reaches 1220; one prompt of 4096 tokens (137 GFLOP) 181 us; eight of 512
// (17 GFLOP, 134 MB) 45 - 48 us.  A long cache is bound by one wave's chain of LDS reads, products and softmax with two waves
// a SIMD; short prompts by what a workgroup does around its steps (8 us: its sequence, its page ids, the first K, the rows'
// way out; 2 us a step).  Few rows on a long cache are cut along it: 512 tokens behind 15872 173 us, 781 TFLOP/s.  float32,
// head_dim 64, 5 x 201 tokens behind 130: 30.5 us.  There a step of 32 tokens is 64 products of 64 cycles in one wave,
// 1.7 us; the 11 steps of the longest rows are 19 us, on fewer waves (640 at most) than the GPU has SIMDs.
#include <algorithm>
#include <type_traits>

#include "kv_tile.h"

namespace lorapool {

struct KvChunk {
    int32_t hpw;              // query heads of one K/V head a workgroup takes: 1, 2 or 4
    int32_t slots_x;          // query tiles (pairs of them) of one row of the grid
    int32_t ranges;           // ranges of tokens a tile's are cut into, at most; 1: not cut
    float *piece_o;           // [ranges][T][n_heads][head_dim]: sums of a range, not divided
    float2 *piece_ml;         // [ranges][T][n_heads]: its maximum (base-2 logits) and sum
    float2 *stats;            // [n_heads][T]: maximum (base-2 logits) and 1 / sum of each row, for the scores; or null
    int32_t hs;               // workgroups that share the query heads of a K/V head, for the scores; divides group
    float *part;              // [n_seq][n_kv * hs][cap_ld]: their shares of the scores
    int64_t cap_ld;
};

// Page ids to addresses, in units of 128 bytes (every token row starts on one): token tok of a sequence of n,
// one per lane; which tokens are there.
__device__ __forceinline__ void lane_ids(const KvArgs &a, const int32_t *row, int32_t tok, int32_t n, int32_t *kid, int32_t *vid) {
    int32_t e, slot;
    page_of(a, tok, &e, &slot);
    *kid = *vid = -1;
    if (tok < n) { *kid = row[e]; *vid = row[a.max_pages + e]; }
}
__device__ __forceinline__ uint64_t lane_units(const KvArgs &a, int32_t tok, int32_t n, int32_t kid, int32_t vid, uint32_t *ku,
                                               uint32_t *vu, int *bad) {
    int32_t e, slot;
    page_of(a, tok, &e, &slot);
    const bool ok = kid >= 0 && vid >= 0 && kid < a.num_pages && vid < a.num_pages;
    if (tok < n && !ok) *bad = DEV_ERR_PAGE;
    const uint32_t pu = (uint32_t)(a.page_bytes >> 7), tu = (uint32_t)(a.tok_bytes >> 7);
    *ku = ok ? (uint32_t)kid * pu + (uint32_t)slot * tu : 0u;
    *vu = ok ? (uint32_t)vid * pu + (uint32_t)slot * tu : 0u;
    return __ballot(ok);
}

// What a slot stands for: sequence and tile, or pair of tiles, in it; -1 behind the last.  Slots count those of all
// sequences from the end, so that the longest rows of a sequence start first.  All 256 threads call.
template <bool PAIR>
__device__ __forceinline__ int32_t slots_of(int32_t m, int32_t tq) { return ((m + tq - 1) / tq + PAIR) / (1 + PAIR); }
template <bool PAIR>
__device__ __forceinline__ int32_t find_tile(const KvArgs &a, int32_t slot, int32_t tq, int32_t *tile, SeqRows *rows, int32_t *sh) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t per = (a.n_seq + 255) / 256, b0 = min(a.n_seq, tid * per), b1 = min(a.n_seq, b0 + per);
    int32_t mine = 0;
    for (int32_t b = b0; b < b1; ++b) mine += slots_of<PAIR>(seq_rows(a, b).m, tq);
    const int32_t incl = wave_incl_scan(mine, lane);
    if (lane == 63) sh[wave] = incl;
    if (tid == 0) sh[4] = -1;
    __syncthreads();
    int32_t excl = incl - mine, total = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        excl += i < wave ? sh[i] : 0;
        total += sh[i];
    }
    const int32_t want = total - 1 - slot;
    if (want >= excl && want < excl + mine) {
        int32_t at = excl;
        for (int32_t b = b0; b < b1; ++b) {
            const int32_t t = slots_of<PAIR>(seq_rows(a, b).m, tq);
            if (want < at + t) {
                const SeqRows q = seq_rows(a, b);
                sh[4] = b;
                sh[5] = want - at;
                sh[6] = q.first;
                sh[7] = q.m;
                sh[8] = q.n;
                break;
            }
            at += t;
        }
    }
    __syncthreads();
    *tile = uniform(sh[5]);
    rows->first = uniform(sh[6]);
    rows->m = uniform(sh[7]);
    rows->n = uniform(sh[8]);
    return uniform(sh[4]);
}

// Steps of one of a tile's ranges: whole runs of the tokens whose addresses are looked up together.
constexpr int PH = 256;
__device__ __forceinline__ int32_t range_steps(int32_t steps, int32_t ranges, int32_t run) {
    return ((steps + ranges - 1) / ranges + run - 1) / run * run;
}

// PAIR: a workgroup takes two tiles of a sequence, one from each end, one after the other: as much work for every pair,
// and its start is paid once.  SPLIT: it takes one range (blockIdx.z) of the tile's tokens, and k_kv_chunk_join puts the
// ranges together.
template <typename E, int HD, bool PAIR, bool SPLIT>
__global__ __launch_bounds__(256, (Chunk<E, HD>::WAVES)) void k_kv_chunk(KvArgs a, KvAttend at, KvChunk ck) {
    using C = Chunk<E, HD>;
    constexpr int NT = C::NT, NB = C::NB, RB = C::RB, CH = C::CH, KQ = C::KQ, ND = HD / 32;
    constexpr bool BF = C::BF;
    extern __shared__ __align__(256) char smem[];
    __shared__ int32_t sh[9];
    __shared__ unsigned long long sh_flag;
    const int wave = uniform((int)threadIdx.x >> 6);
    const int32_t groups = a.n_heads / ck.hpw, hg = blockIdx.x % groups, slot = blockIdx.y * ck.slots_x + blockIdx.x / groups;
    if (blockIdx.x == 0 && blockIdx.y == 0 && (!SPLIT || blockIdx.z == 0)) check_seqs(a);
    const int32_t tq = 128 / ck.hpw;
    int32_t tile;
    SeqRows sq;
    const int32_t b = find_tile<PAIR>(a, slot, tq, &tile, &sq, sh), tiles = (sq.m + tq - 1) / tq;
    if (b < 0 || tile < 0 || tile >= slots_of<PAIR>(sq.m, tq)) return;   // (ranges that overlap can have more than counted)
    int32_t second = -1;
    if constexpr (PAIR) {
        const int32_t first = tiles - 1 - tile;
        if (tile < first) second = tile;
        tile = first;
    }
    const int32_t head = hg * ck.hpw + (wave & (ck.hpw - 1)), in_tile = (wave / ck.hpw) * 32;
    const int32_t old = sq.n - sq.m;                        // tokens before the new ones
    const int32_t *trow = a.table + (int64_t)b * 2 * a.max_pages;
    const char *base = a.pages + (int64_t)(head / a.group) * RB;
    const float scale2 = at.scale * 1.4426950408889634f;
    bool placed = false;                                    // the addresses of the first tokens are in LDS
    for (;;) {
    int tid = threadIdx.x;
    if constexpr (PAIR) asm volatile("" : "+v"(tid));       // what hangs on it is worked out for each tile, not kept over both
    const int lane = tid & 63, col = lane & 31, hh = lane >> 5;
    const int32_t q0 = tile * tq + in_tile;
    const int32_t qi = q0 + col;
    const bool row_ok = qi < sq.m;
    const int64_t row = sq.first + (row_ok ? qi : sq.m - 1);
    E *orow = (E *)at.out + row * at.ldo + (int64_t)head * HD;
    if (SPLIT && sq.n == 0) return;
    if (sq.n == 0) {                                        // no tokens: zero rows
        if (row_ok)
            for (int d = hh * (HD / 2); d < (hh + 1) * (HD / 2); ++d) from_f32(orow + d, 0.f);
        if (ck.stats && row_ok && hh == 0) ck.stats[(int64_t)head * a.T + row] = make_float2(0.f, 0.f);
        if (!PAIR || second < 0) return;
        tile = second;
        second = -1;
        continue;
    }
    const int32_t pos = old + (row_ok ? qi : sq.m - 1);     // this lane's row sees tokens 0 .. pos
    const int32_t wave_lo = old + min(q0, sq.m - 1), wave_hi = old + min(q0 + 31, sq.m - 1);
    const int32_t wg_lo = old + tile * tq, wg_hi = old + min(tile * tq + tq, sq.m) - 1;
    constexpr int SP = PH / NT;                             // steps that one look-up of addresses lasts for
    int32_t begin = 0, steps = wg_hi / NT + 1;              // the first step, and the one behind the last
    if constexpr (SPLIT) {
        const int32_t per = range_steps(steps, ck.ranges, SP);
        begin = (int32_t)blockIdx.z * per;
        if (begin >= steps) return;
        steps = min(steps, begin + per);
    }
    u32x4_t Q[KQ];
    {
        const char *p = (const char *)((const E *)at.q + row * at.ldq + (int64_t)head * HD) + 16 * hh;
#pragma unroll
        for (int i = 0; i < KQ; ++i) Q[i] = load16(p + 32 * i);
    }
    // Where the tokens' rows lie, PH tokens at a time: a thread looks one token's pages up and leaves the addresses in
    // LDS, in units of 128 bytes (every token row starts on one); tokens that are not there get the pool's first page.
    uint32_t *units = (uint32_t *)(smem + 4 * C::BUF);           // [2][K, V][PH]
    int32_t *raw = (int32_t *)(units + 4 * PH) + 64 * wave;             // [K, V][PH]: page ids, this wave's 64 tokens
    uint64_t *masks = (uint64_t *)((uint32_t *)(smem + 4 * C::BUF) + 6 * PH);   // [2][PH / 64]: which tokens are there
    int bad = 0;
    auto look_up = [&](int32_t ph) {                        // page ids on their way to LDS (from the table's first entry
        const int32_t tok = ph * PH + tid;                  // where no token is)
        int32_t e, slot;
        page_of(a, tok, &e, &slot);
        const int32_t *p = trow + (tok < sq.n ? e : 0);
        lds_gload4(p, (lds_void *)raw);
        lds_gload4(p + a.max_pages, (lds_void *)(raw + PH));
    };
    auto place = [&](int32_t ph) {
        const int32_t tok = ph * PH + tid, kid = raw[lane], vid = raw[PH + lane];
        int32_t e, slot;
        page_of(a, tok, &e, &slot);
        const bool token = tok < sq.n && tok < steps * NT;
        const bool ok = token && kid >= 0 && vid >= 0 && kid < a.num_pages && vid < a.num_pages;
        if (token && !ok) bad = DEV_ERR_PAGE;
        const uint32_t pu = (uint32_t)(a.page_bytes >> 7), at0 = (uint32_t)slot * (uint32_t)(a.tok_bytes >> 7);
        uint32_t *u = units + (ph & 1) * 2 * PH + tid;
        u[0] = ok ? (uint32_t)kid * pu + at0 : 0u;
        u[PH] = ok ? (uint32_t)vid * pu + at0 : 0u;
        const uint64_t there = __ballot(ok);
        if (lane == 0) masks[(ph & 1) * (PH / 64) + wave] = there;
    };
    // K and V of step j to LDS: every lane brings 16 bytes to where they are read from.
    auto fetch = [&](int32_t j) {
        const uint32_t *uk = units + (j / SP & 1) * 2 * PH + j % SP * NT, *uv = uk + PH;
        char *kb = smem + (j & 1) * C::BUF, *vb = smem + (2 + (j & 1)) * C::BUF;
#pragma unroll
        for (int x = 0; x < C::PER; ++x) {
            const int at0 = (wave * C::PER + x) * 1024, byte = at0 + lane * 16, t = byte / RB, c = (byte % RB) / 16;
            lds_gload16(base + ((uint64_t)uk[t] << 7) + 16 * C::k_swz(t, c), (lds_void *)(kb + at0));
            lds_gload16(base + ((uint64_t)uv[t] << 7) + 16 * C::v_swz(t, c), (lds_void *)(vb + at0));
        }
    };
    auto other_half = [](float x) {                          // the value of the lane 32 further, or before
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        return __uint_as_float(threadIdx.x & 32 ? r[0] : r[1]);
    };

    f32x16_t acc[ND], S[NB];
    float m, l;
    // S^T = K Q^T of one step
    auto logits = [&](const char *kb, f32x16_t (&x)[NB]) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 16; ++i) x[nb][i] = 0.f;
#pragma unroll
        for (int k = 0; k < KQ; ++k)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const u32x4_t f = load16(kb + (32 * nb + col) * RB + 16 * C::k_swz(col, 2 * k + hh));
                if constexpr (BF) {
                    x[nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, f), __builtin_bit_cast(bf16x8_t, Q[k]), x[nb], 0, 0, 0);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[nb] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(f[e]), __uint_as_float(Q[k][e]), x[nb], 0, 0, 0);
                }
            }
    };
    // Two passes at most.  The first lets tokens behind a row's own position into the products with weight 0, which
    // is right unless their V holds an infinity or NaN; then a row comes out not finite, and the second
    // pass takes such values out of the products and adds them to the rows that see them.
    auto pass = [&](auto careful) {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
        m = -INFINITY;
        l = 0.f;
        if (!PAIR || !placed) {
            look_up(begin / SP);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            place(begin / SP);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        fetch(begin);
        for (int32_t j = begin; j < steps; ++j) {
            const int32_t t0 = j * NT;
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");   // this step's K and V are in
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            fetch(j + 1);
            if ((j + 2) % SP == 0) place((j + 2) / SP);     // before the first fetch from there, at the next step
            if ((j + 3) % SP == 0) look_up((j + 3) / SP);
            const int32_t at64 = t0 % (2 * PH) / 64;
            const uint64_t word = (uint64_t)(uint32_t)uniform((int32_t)(masks[at64] >> 32)) << 32 | (uint32_t)uniform((int32_t)masks[at64]);
            const uint64_t there = NT == 64 ? word : word >> (t0 & 32) & 0xffffffffu;
            constexpr uint64_t ALL = NT == 64 ? ~0ull : 0xffffffffu;
            char *vb = smem + (2 + (j & 1)) * C::BUF;
            if (there != ALL) {                             // rows of tokens that are not there must not reach the products
                for (int x = tid; x < NT * CH; x += 256)
                    if (!((there >> (x / CH)) & 1)) store16(vb + 16 * x, u32x4_t{0, 0, 0, 0});
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_s_barrier();
            }
            if (careful.value && t0 + NT - 1 > wg_lo) {     // some row does not see all of these tokens
                if (tid == 0) sh_flag = 0;
                __syncthreads();
                auto odd = [&](uint32_t w) {                // non-finite parts of a dword, the rest zero
                    if constexpr (!BF) return (w & 0x7f800000u) == 0x7f800000u ? w : 0u;
                    else return ((w & 0x7f80u) == 0x7f80u ? w & 0xffffu : 0u) | ((w & 0x7f800000u) == 0x7f800000u ? w & 0xffff0000u : 0u);
                };
                for (int x = tid; x < NT * CH; x += 256) {
                    const u32x4_t w = load16(vb + 16 * x);
                    if (odd(w[0]) | odd(w[1]) | odd(w[2]) | odd(w[3])) atomicOr(&sh_flag, 1ull << (x / CH));
                }
                __syncthreads();
                if (const unsigned long long flags = sh_flag) {
                    for (unsigned long long f = flags; f; f &= f - 1) {
                        const int t = __ffsll((long long)f) - 1;
                        if (t0 + t <= pos) {
#pragma unroll
                            for (int d = 0; d < ND; ++d)
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const int byte = (32 * d + 8 * (i / 4) + 4 * hh + (i & 3)) * (int)sizeof(E);
                                    const float x = to_f32(*(const E *)(vb + t * RB + 16 * C::v_swz(t, byte / 16) + byte % 16));
                                    if (x - x != 0.f) acc[d][i] += x;
                                }
                        }
                    }
                    __syncthreads();
                    for (int x = tid; x < NT * CH; x += 256) {
                        u32x4_t w = load16(vb + 16 * x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] ^= odd(w[i]);
                        store16(vb + 16 * x, w);
                    }
                    __syncthreads();
                }
            }
            if (t0 > wave_hi) continue;
            __builtin_amdgcn_sched_barrier(0);
            logits(smem + (j & 1) * C::BUF, S);
            // K pieces come out of LDS three products ahead
            __builtin_amdgcn_sched_group_barrier(0x100, 3 * NB, 0);
#pragma unroll
            for (int k = 0; k < KQ; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x008, NB * (BF ? 1 : 4), 0);
                if (k + 3 < KQ) __builtin_amdgcn_sched_group_barrier(0x100, NB, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            float sc = scale2;
            if (!(scale2 > 0.f)) {                          // the largest logit need not be the largest product's
                sc = 1.f;
                float by = scale2;
                asm volatile("" : "+v"(by));                // keeps the products inside the branch
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) S[nb][i] *= by;
            }
            if (there != ALL || t0 + NT - 1 > wave_lo) {    // tokens counted from this lane half's first
                const int32_t last = pos - t0 - 4 * hh;
                const uint64_t in = there >> (4 * hh);
                const uint32_t in0 = (uint32_t)in, in1 = (uint32_t)(in >> 32);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int t = 8 * (i / 4) + (i & 3);
                        if (32 * nb + t > last || !((nb ? in1 : in0) & (1u << t))) S[nb][i] = -INFINITY;
                    }
            }
            float mt = -INFINITY;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 16; ++i) mt = fmaxf(mt, S[nb][i]);
            mt = fmaxf(mt, other_half(mt)) * sc;
            // bfloat16: the running maximum follows at once, so that a row's largest weight is one and its rounding, the
            // one that counts most, is none (weights of up to 2^8 instead would double the variance of the weights' part of
            // the error: 0.0023 against 0.0020 from float64, behind 14336 tokens).  It costs 3% there, 1.4% at 8 x 512.
            // float32 rounds no weights: there the maximum moves only when a logit passes it by 8, to rescale less often.
            if (__any(mt > m + (BF ? 0.f : 8.f))) {
                const float mn = fmaxf(m, mt), ms = mn == -INFINITY ? 0.f : mn;
                // (before a row's first weight the accumulators hold zeros, or infinities that the second pass added)
                const float c = careful.value && m == -INFINITY ? 1.f : exp2_hw(m - ms);
                m = mn;
                l *= c;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[d][i] *= c;
            }
            __builtin_amdgcn_sched_barrier(0);
            const float ms = m == -INFINITY ? 0.f : m;
            float ps = 0.f;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    S[nb][i] = exp2_hw(S[nb][i] * sc - ms);
                    ps += S[nb][i];
                }
            l += ps;
            if constexpr (BF) {
                // Weights rounded once to bfloat16, the type that V comes and the output goes in.  With the rest of each as a
                // second product, as for one token, the error is the output's own rounding (0.0017 from float64 instead of
                // 0.0020 behind 14336 tokens, 0.0016 instead of 0.0018 at 8 x 512), but these products are what bounds the call:
                // 567 us would be 734, one prompt of 4096 tokens 181 and 229, 8 x 512 45 and 53.
                const int i16 = lane & 15;
#pragma unroll
                for (int s = 0; s < NT / 16; ++s) {
                    u32x4_t p;                              // this lane's eight weights: tokens 16 s + 4 hh + 0..3 and 8 on
#pragma unroll
                    for (int x = 0; x < 4; ++x) p[x] = pack2(S[s / 2][8 * (s & 1) + 2 * x], S[s / 2][8 * (s & 1) + 2 * x + 1]);
                    const int t = 16 * s + 4 * hh + (i16 >> 2);
#pragma unroll
                    for (int d = 0; d < ND; ++d) {
                        const int c = 4 * d + 2 * ((lane >> 4) & 1) + ((i16 & 3) >> 1);
                        const char *ad = vb + t * RB + 16 * C::v_swz(t, c) + 8 * (i16 & 1);
                        const s16x4_t v0 = read_tr((lds_s16x4 *)ad);
                        const s16x4_t v1 = read_tr((lds_s16x4 *)(ad + 8 * RB));
                        typedef short s16x8_t __attribute__((ext_vector_type(8)));
                        const s16x8_t v = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
                        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, v),
                                                                         __builtin_bit_cast(bf16x8_t, p), acc[d], 0, 0, 0);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int t = 8 * (i / 4) + 4 * hh + (i & 3);
#pragma unroll
                    for (int d = 0; d < ND; ++d)
                        acc[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(*(const float *)(vb + t * RB + 4 * (32 * d + col)), S[0][i], acc[d], 0, 0, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");    // no load is on its way to LDS any more
        __syncthreads();
    };
    pass(std::false_type{});
    float chk = 0.f;                                        // 0, or NaN where a sum is not finite
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) chk += acc[d][i] * 0.f;
    if (__syncthreads_or(chk != 0.f)) pass(std::true_type{});
    if (bad) record(a, bad);
    if constexpr (SPLIT) {
        const float sum = l + other_half(l);
        if (row_ok) {
            const int64_t at_piece = ((int64_t)blockIdx.z * a.T + row) * a.n_heads + head;
            if (hh == 0) ck.piece_ml[at_piece] = make_float2(m, sum);
            float *o = ck.piece_o + at_piece * HD;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    *(float4 *)(o + 32 * d + 8 * x + 4 * hh) = make_float4(acc[d][4 * x], acc[d][4 * x + 1], acc[d][4 * x + 2], acc[d][4 * x + 3]);
        }
        return;
    }
    const float L = l + other_half(l), inv = L == 0.f ? 0.f : 1.f / L;
    if (L == 0.f)                                           // no weight: zero, also where a value is not finite
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
    if (ck.stats && row_ok && hh == 0) ck.stats[(int64_t)head * a.T + row] = make_float2(m == -INFINITY ? 0.f : m, inv);
    if constexpr (BF) {
        // rows through LDS, so that a row leaves in one piece
        constexpr int OB = RB + 16;
        char *o = smem + wave * 32 * OB;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint2 w = make_uint2(pack2(acc[d][4 * x] * inv, acc[d][4 * x + 1] * inv),
                                     pack2(acc[d][4 * x + 2] * inv, acc[d][4 * x + 3] * inv));
                *(uint2 *)(o + col * OB + (32 * d + 8 * x + 4 * hh) * 2) = w;
            }
        __builtin_amdgcn_wave_barrier();
        E *out = (E *)at.out + (sq.first + (int64_t)q0) * at.ldo + (int64_t)head * HD;
        for (int x = lane; x < 32 * CH; x += 64) {
            const int r = x / CH, c = x % CH;
            if (q0 + r < sq.m) store16(out + r * at.ldo + 8 * c, load16(o + r * OB + 16 * c));
        }
    } else if (row_ok) {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *(float4 *)(orow + 32 * d + 8 * x + 4 * hh) = make_float4(acc[d][4 * x] * inv, acc[d][4 * x + 1] * inv,
                                                                        acc[d][4 * x + 2] * inv, acc[d][4 * x + 3] * inv);
    }
    if (!PAIR || second < 0) return;
    placed = steps <= 2 * SP - 2;                           // nothing has been put over them
    tile = second;
    second = -1;
    }
}

// Put the ranges of a row (blockIdx.x) together: a wave to a head.  out = sum 2^(m_s - M) o_s / sum 2^(m_s - M) l_s; the
// bytes are the ranges' sums once, at most 128 rows of each workgroup there was (32 MiB at head_dim 128), from the caches.
constexpr int RANGES = 512;
template <typename E, int HD>
__global__ __launch_bounds__(256) void k_kv_chunk_join(KvArgs a, KvAttend at, KvChunk ck) {
    __shared__ int32_t seq;
    __shared__ float weight[4][RANGES];
    const int32_t t = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, head = blockIdx.y * 4 + wave;
    if (tid == 0) seq = -1;
    __syncthreads();
    for (int32_t b = tid; b < a.n_seq; b += 256) {
        const SeqRows q = seq_rows(a, b);
        if (t >= q.first && t < q.first + q.m) atomicMax(&seq, b);
    }
    __syncthreads();
    if (seq < 0 || head >= a.n_heads) return;
    const SeqRows sq = seq_rows(a, seq);
    constexpr int W = HD / 64;                              // dims of a lane
    E *out = (E *)at.out + (int64_t)t * at.ldo + (int64_t)head * HD + W * lane;
    const int32_t tq = 128 / ck.hpw, tile = (t - sq.first) / tq, last = sq.n - sq.m + min(tile * tq + tq, sq.m) - 1;
    constexpr int NT = Chunk<E, HD>::NT;
    const int32_t steps = last / NT + 1, per = range_steps(steps, ck.ranges, PH / NT);
    const int32_t used = sq.n ? (steps + per - 1) / per : 0;
    const int64_t first = (int64_t)t * a.n_heads + head, next = (int64_t)a.T * a.n_heads;
    float M = -INFINITY;
    for (int32_t s = lane; s < used; s += 64) M = fmaxf(M, ck.piece_ml[first + s * next].x);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor(M, o, 64));
    const float Ms = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    for (int32_t s = lane; s < used; s += 64) {
        const float2 ml = ck.piece_ml[first + s * next];
        const float w = exp2_hw(ml.x - Ms);
        weight[wave][s] = w;
        L += ml.y * w;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) L += __shfl_xor(L, o, 64);
    __builtin_amdgcn_wave_barrier();
    float v[W];
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = 0.f;
#pragma unroll 8
    for (int32_t s = 0; s < used; ++s) {
        const float *o = ck.piece_o + (first + s * next) * HD + W * lane;
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] += o[i] * weight[wave][s];
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int i = 0; i < W; ++i) from_f32(out + i, L == 0.f ? 0.f : v[i] * inv);
    if (ck.stats && lane == 0) ck.stats[(int64_t)head * a.T + t] = make_float2(Ms, inv);
}

// ---- scores: the weights once more, summed over the rows ---------------------------------------------
// A token's weights can be summed only when its rows' maxima and sums are known.  One workgroup takes 128
// tokens of one K/V head, K in registers, and walks the query rows of the heads that share it; the logits are
// multiplied again (half of the attention's products), and a lane sums its query rows' weights for each of its tokens.
// 8 x 512 tokens, 32 heads of 128 (one to a K/V head): 28.0 us (two blocks of rows at a time; one: 36; 64 tokens a workgroup and rows
// summed one exchange a token: 44), and 4.1 for the sum over the K/V heads.
template <typename E, int HD>
struct Scores {
    static constexpr bool BF = sizeof(E) == 2;
    static constexpr int RB = HD * (int)sizeof(E);
    static constexpr int TOK = 4 * 32;
    static constexpr int NQ = RB > 256 ? 32 : 64;           // query rows of a step
    static constexpr int BUF = NQ * RB;
    static constexpr int WAVES = RB > 512 ? 1 : RB > 256 ? 2 : 4;
};

template <typename E, int HD>
__global__ __launch_bounds__(256, (Scores<E, HD>::WAVES)) void k_kv_chunk_scores(KvArgs a, KvAttend at, KvChunk ck) {
    using P = Scores<E, HD>;
    using C = Chunk<E, HD>;
    constexpr int RB = P::RB, KQ = C::KQ, NQ = P::NQ;
    constexpr bool BF = P::BF;
    __shared__ __align__(256) char smem[2 * P::BUF];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), col = lane & 31, hh = lane >> 5;
    const int32_t b = blockIdx.z, kvh = blockIdx.x / ck.hs, heads = a.group / ck.hs, t0 = blockIdx.y * P::TOK;
    const SeqRows sq = seq_rows(a, b);
    if (t0 >= sq.n) return;
    const int32_t old = sq.n - sq.m, tw = t0 + wave * 32;
    const float scale2 = at.scale * 1.4426950408889634f;
    const int32_t *trow = a.table + (int64_t)b * 2 * a.max_pages;

    u32x4_t K[KQ];
    int32_t kid, vid;
    uint32_t ku, vu;
    int bad = 0;
    lane_ids(a, trow, tw + col, sq.n, &kid, &vid);
    const uint32_t there = (uint32_t)lane_units(a, tw + col, sq.n, kid, vid, &ku, &vu, &bad);
    {
        const char *p = a.pages + ((uint64_t)ku << 7) + (int64_t)kvh * RB + 16 * hh;
#pragma unroll
        for (int k = 0; k < KQ; ++k) K[k] = load16(p + 32 * k);
    }
    f32x16_t sum;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum[i] = 0.f;

    // steps: for each head of the group, NQ query rows at a time from the first that sees token t0.  (fh, fr): the
    // next step to fetch, off: its distance in bytes from the first one's rows, where this lane's pieces lie.
    const int32_t r0 = max(0, t0 - old) / NQ * NQ, per = sq.m > r0 ? (sq.m - r0 + NQ - 1) / NQ : 0;
    const int32_t steps = per * heads, h0 = blockIdx.x * heads;
    constexpr int PER = P::BUF / 4096;
    const int64_t row_bytes = at.ldq * (int64_t)sizeof(E);
    const char *piece[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int byte = (wave * PER + j) * 1024 + lane * 16, x = byte / RB, c = (byte % RB) / 16;
        piece[j] = (const char *)at.q + (sq.first + r0 + x) * row_bytes + (int64_t)h0 * RB + 16 * C::k_swz(x, c);
    }
    int32_t fh = 0, fr = r0;
    int64_t off = 0;
    float2 st[NQ / 32], st1[NQ / 32];
    auto fetch = [&](char *to) {
        const int32_t over = fr + NQ - sq.m;                // rows of the step behind the last one: it comes again
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int at0 = (wave * PER + j) * 1024, x = (at0 + lane * 16) / RB;
            const char *p = piece[j] + off;
            if (over > 0) p -= max(0, x + over - NQ + 1) * row_bytes;
            lds_gload16(p, (lds_void *)(to + at0));
        }
#pragma unroll
        for (int qb = 0; qb < NQ / 32; ++qb) {
            const int32_t r = fr + 32 * qb + col;
            st1[qb] = ck.stats[(int64_t)(h0 + fh) * a.T + sq.first + min(r, sq.m - 1)];
            if (r >= sq.m) st1[qb].y = 0.f;
        }
        fr += NQ;
        off += NQ * row_bytes;
        if (fr >= sq.m) {
            fr = r0;
            ++fh;
            off = (int64_t)fh * RB;
        }
    };
    if (steps) fetch(smem);
    // K is waited for here: the compiler would put the wait into the loop, where it would also wait for the rows ahead
#pragma unroll
    for (int k = 0; k < KQ; ++k) asm volatile("" : "+v"(K[k]));
    int32_t r = r0;
    for (int32_t it = 0; it < steps; ++it) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int qb = 0; qb < NQ / 32; ++qb) st[qb] = st1[qb];
        if (it + 1 < steps) fetch(smem + (~it & 1) * P::BUF);
        const char *q = smem + (it & 1) * P::BUF;
        if (tw <= old + min(r + NQ, sq.m) - 1) {            // else no row of the step sees the wave's tokens
            constexpr int NB = NQ / 32;
            f32x16_t S[NB];
#pragma unroll
            for (int qb = 0; qb < NB; ++qb)
#pragma unroll
                for (int i = 0; i < 16; ++i) S[qb][i] = 0.f;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < KQ; ++k)
#pragma unroll
                for (int qb = 0; qb < NB; ++qb) {
                    const u32x4_t f = load16(q + (32 * qb + col) * RB + 16 * C::k_swz(col, 2 * k + hh));
                    if constexpr (BF) {
                        S[qb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, K[k]), __builtin_bit_cast(bf16x8_t, f), S[qb], 0, 0, 0);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            S[qb] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(K[k][e]), __uint_as_float(f[e]), S[qb], 0, 0, 0);
                    }
                }
            // the rows come out of LDS three products ahead
            __builtin_amdgcn_sched_group_barrier(0x100, 3 * NB, 0);
#pragma unroll
            for (int k = 0; k < KQ; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x008, NB * (BF ? 1 : 4), 0);
                if (k + 3 < KQ) __builtin_amdgcn_sched_group_barrier(0x100, NB, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (tw + 31 > old + r || r + NQ > sq.m) {       // some row does not see all of the wave's tokens, or is none
#pragma unroll
                for (int qb = 0; qb < NB; ++qb) {
                    const int32_t last = old + r + 32 * qb + col - tw - 4 * hh;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float w = exp2_hw(S[qb][i] * scale2 - st[qb].x) * st[qb].y;
                        sum[i] += 8 * (i / 4) + (i & 3) > last ? 0.f : w;
                    }
                }
            } else {
#pragma unroll
                for (int qb = 0; qb < NB; ++qb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum[i] += exp2_hw(S[qb][i] * scale2 - st[qb].x) * st[qb].y;
            }
        }
        r += NQ;
        if (r >= sq.m) r = r0;
    }
    if (bad) record(a, bad);
    // Sum over the 32 query rows, which are the lanes: at each exchange a lane hands half of its tokens over and keeps
    // the other half's sums, until one token is left to it.
    float v[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) v[x] = sum[x];
#pragma unroll
    for (int o = 16; o > 1; o >>= 1)
#pragma unroll
        for (int x = 0; x < o / 2; ++x) {
            const bool up = col & o;
            v[x] = (up ? v[x + o / 2] : v[x]) + __shfl_xor(up ? v[x] : v[x + o / 2], o, 64);
        }
    v[0] += __shfl_xor(v[0], 1, 64);
    const int x = col >> 1, t = 8 * (x / 4) + 4 * hh + (x & 3);
    if (!(col & 1) && tw + t < sq.n) ck.part[((int64_t)b * gridDim.x + blockIdx.x) * ck.cap_ld + tw + t] = (there >> t) & 1 ? v[0] : 0.f;
}

__global__ __launch_bounds__(256) void k_kv_chunk_sum(KvArgs a, KvAttend at, KvChunk ck) {
    const int32_t b = blockIdx.y, t = blockIdx.x * 256 + threadIdx.x;
    const SeqRows sq = seq_rows(a, b);
    if (t >= sq.n) return;
    float s = 0.f;
    const int32_t shares = a.n_kv * ck.hs;
    const float *p = ck.part + (int64_t)b * shares * ck.cap_ld + t;
#pragma unroll 8
    for (int32_t h = 0; h < shares; ++h) s += p[(int64_t)h * ck.cap_ld];
    const int64_t i = (int64_t)b * at.score_ld + t;
    at.scores[i] = (at.prior ? at.prior[i] : 0.f) + s;
}

// ---- host ------------------------------------------------------------------------------------------
namespace {

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

// More than 64 KiB of LDS has to be asked for, on each device.
hipError_t big_lds(const void *kernel, int bytes) {
    return bytes <= 64 * 1024 ? hipSuccess : hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

struct ChunkPlan {
    int32_t hpw, groups, tiles, ranges, hs;
    int64_t cap_ld;
    size_t off_part, off_o, off_ml, total;
};
ChunkPlan chunk_plan(int n_heads, int n_kv, int hd, int32_t n_seq, int64_t T, int64_t max_len, bool scores) {
    ChunkPlan p;
    const int group = n_heads / n_kv;
    p.hpw = group % 4 == 0 ? 4 : group % 2 == 0 ? 2 : 1;
    p.groups = n_heads / p.hpw;
    const int32_t tq = 128 / p.hpw;
    p.tiles = (int32_t)((T + std::min<int64_t>(n_seq, T) * (tq - 1)) / tq);   // at most
    // A tile's tokens are cut into ranges of 256 or more where the tiles alone do not fill the GPU, two workgroups a CU (one,
    // head_dim 256).  Whole calls: bfloat16, 32 heads of 128 on 8: 2 x 12 tokens behind 12652 295 us whole, 42 in ranges,
    // 512 behind 15872 387 and 173; float32, 4 heads of 64 on 2, 4 x 1 behind 12897: 962 and 50.  Below 512 tokens it goes
    // either way, and they are left whole: 4 x 64 behind 300, 32 heads of 128 on 8, 17.9 us whole, 24.8 in two, 1 x 8 behind
    // 480 19.7 and 17.4; float32, 16 heads of 64 35.7 and 30.7; 16 heads of 256 on 4, 2 x 40 behind 400, 38.1 and 32.1, in
    // float32 161 and 103.
    const int64_t wgs = (int64_t)p.groups * p.tiles, most = std::min<int64_t>(max_len / PH, RANGES);
    const int slots = hd == 256 ? 256 : 512;
    p.ranges = (int32_t)std::max<int64_t>(1, std::min(slots / std::max<int64_t>(wgs, 1), most));
    p.cap_ld = (max_len + 63) / 64 * 64;
    // The size grows with T and max_len, so that what serves the largest call serves them all: ranges * T * n_heads is
    // at most 128 rows for each of the GPU's workgroups.
    const int64_t rows = most < 2 ? 0 : std::min<int64_t>(most * T * n_heads, 128 * slots);
    p.off_part = scores ? up256((size_t)T * n_heads * 8) : 0;
    // Query heads of a K/V head go to more workgroups while the GPU has room, four a CU (the whole call, float32, 8 heads of
    // 128 on one, 6 x 377 tokens: 316 us -> 102; bfloat16, 32 on 8, 2 x 1184: 141 -> 88).
    const int64_t one = (int64_t)n_kv * n_seq * ((max_len + 127) / 128);
    p.hs = (int32_t)std::max<int64_t>(1, std::min<int64_t>(group, 1024 / std::max<int64_t>(one, 1)));
    while (group % p.hs) --p.hs;
    const int64_t shares = std::min<int64_t>((int64_t)n_seq * n_heads * p.cap_ld,
                                             std::max<int64_t>((int64_t)n_seq * n_kv * p.cap_ld, 1024 * 128));   // never less for a larger call
    p.off_o = p.off_part + (scores ? up256((size_t)shares * 4) : 0);
    p.off_ml = p.off_o + up256((size_t)rows * hd * 4);
    p.total = p.off_ml + up256((size_t)rows * 8);
    return p;
}

template <typename E, int HD>
hipError_t run(const KvArgs &a, const KvAttend &at, hipStream_t s) {
    using C = Chunk<E, HD>;
    const ChunkPlan pl = chunk_plan(a.n_heads, a.n_kv, HD, a.n_seq, a.T, a.cap, at.scores != nullptr);
    char *ws = (char *)at.ws;
    KvChunk ck;
    ck.hpw = pl.hpw;
    ck.ranges = pl.ranges;
    ck.hs = pl.hs;
    ck.cap_ld = pl.cap_ld;
    ck.stats = at.scores ? (float2 *)ws : nullptr;
    ck.part = (float *)(ws + pl.off_part);
    ck.piece_o = (float *)(ws + pl.off_o);
    ck.piece_ml = (float2 *)(ws + pl.off_ml);
    const int32_t tq = 128 / ck.hpw, groups = pl.groups;
    constexpr int OUT = C::BF ? 4 * 32 * (C::RB + 16) : 0, LDS = std::max(C::LDS, OUT);
    auto launch = [&](auto kernel, int32_t slots) {
        const hipError_t e = big_lds((const void *)kernel, LDS);
        if (e != hipSuccess) return e;
        ck.slots_x = std::min(slots, (1 << 22) / groups);   // a row of the grid has less than 2^32 threads
        const dim3 grid((unsigned)(groups * ck.slots_x), (unsigned)((slots + ck.slots_x - 1) / ck.slots_x), (unsigned)ck.ranges);
        hipLaunchKernelGGL(kernel, grid, dim3(256), LDS, s, a, at, ck);
        return hipSuccess;
    };
    const int32_t seqs = std::min(a.n_seq, a.T);
    // Pairs where they fill the GPU, two workgroups a CU, and sequences are so short that starts count (32 heads of 128:
    // 8 x 512 tokens 55.6 us one by one, 49.1 in pairs, 4 x 1024 75.9 and 71.3, 2 x 2048 125.6 and 124.4, kernels alone from
    // a profile's colder clocks).  Not for float32 and head_dim 256, which products and registers bind.
    constexpr bool CAN = C::BF && HD <= 128;
    hipError_t e;
    if (ck.ranges > 1) {
        e = launch(k_kv_chunk<E, HD, false, true>, pl.tiles);
        if (e == hipSuccess)
            hipLaunchKernelGGL((k_kv_chunk_join<E, HD>), dim3(a.T, (a.n_heads + 3) / 4), dim3(256), 0, s, a, at, ck);
    } else if (CAN && (int64_t)groups * (a.T / tq) >= 2 * 512 && a.cap <= 1024) {
        e = launch(k_kv_chunk<E, HD, CAN, false>, (pl.tiles + seqs + 1) / 2);
    } else {
        e = launch(k_kv_chunk<E, HD, false, false>, pl.tiles);
    }
    if (e != hipSuccess) return e;
    if (at.scores) {
        constexpr int TOK = Scores<E, HD>::TOK;
        hipLaunchKernelGGL((k_kv_chunk_scores<E, HD>), dim3(a.n_kv * ck.hs, (a.cap + TOK - 1) / TOK, a.n_seq), dim3(256), 0, s, a, at, ck);
        hipLaunchKernelGGL(k_kv_chunk_sum, dim3((a.cap + 255) / 256, a.n_seq), dim3(256), 0, s, a, at, ck);
    }
    return hipGetLastError();
}

template <typename E>
hipError_t by_dim(const KvArgs &a, const KvAttend &at, hipStream_t s) {
    return a.head_dim == 64 ? run<E, 64>(a, at, s) : a.head_dim == 128 ? run<E, 128>(a, at, s) : run<E, 256>(a, at, s);
}

}  // namespace

size_t kv_chunk_ws_bytes(int, const lora_kv_layout_t &l, int32_t n_seq, int64_t T, int64_t max_len, bool scores) {
    return chunk_plan(l.n_heads, l.n_kv_heads, l.head_dim, n_seq, T, max_len, scores).total;
}

hipError_t launch_kv_chunk(int dtype, const KvArgs &a, const KvAttend &at, hipStream_t s) {
    return dtype == LORA_F32 ? by_dim<float>(a, at, s) : by_dim<uint16_t>(a, at, s);
}

}  // namespace lorapool

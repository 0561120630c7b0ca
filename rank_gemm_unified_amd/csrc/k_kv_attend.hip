// Attention of one new token per sequence over the paged cache (the decode step).
//
// The work is reading K and V once: 4 * len * n_heads * head_dim operations on 2 * len * n_kv * head_dim
// elements, a few operations a byte, so HBM bounds it.  The tiles (TT tokens) of all sequences, one
// sequence behind the other, are cut into R equal ranges whatever the lengths; one wave takes one range
// of one K/V head, so every wave reads the same amount, and waves next to each other read neighbouring
// heads of the same pages.  A range ends inside a sequence as a rule: what a wave has of a sequence it
// did not see whole goes to the workspace with its maximum and sum, and k_kv_join puts the pieces
// together (split and joined, no atomics: results do not change from call to call).
//
// The logits go through the matrix units although a decode step leaves most of their columns empty (16 query heads of a
// K/V head, one where none is shared): a first kernel on the vector units, whose sums cross lanes, took 680 us for the
// 64 sequences below.  bfloat16, head_dim 128, 32 heads, with scores: 64 sequences of up to 1031 tokens (637 MB of K, V
// and scores): 116 - 121 us (5.3 - 5.5 TB/s), and 11.6 us for the join, which reads the logits; 8 of up to 32768 on
// 8 K/V heads (748 MB): 138 - 146 us (5.1 - 5.4 TB/s), and 15.7.  float32, 16 sequences of up to 777 tokens, 16 heads
// of 64, in one launch: 18.1 - 20.7 us (3.3 - 3.7 TB/s: few tiles a wave); with scores 19.4 and 6.8 for the join.  A copy of
// 1 GiB reaches 5.5 TB/s.
#include <algorithm>

#include "kv_ranges.h"

namespace lorapool {

struct KvSplit {
    int32_t R;                // ranges
    int32_t ncb;              // blocks of 16 query heads of one K/V head
    int32_t hu;               // K/V heads * ncb
    int32_t jh;               // heads a workgroup of the join takes: 4, or 1
    float *part_o;            // [R][2][n_heads][head_dim]: slot 0 a range's first piece, 1 its last
    float2 *part_ml;          // [R][2][n_heads]: maximum (base-2 logits), sum
    float2 *done_ml;          // [n_seq][n_heads]: of the sequences one range saw whole
    int32_t cols;             // query heads of a block, at most
    int64_t tiles;            // at most
    float *logits;            // [hu][tiles][cols][TT] base-2 logits, for the scores
};

template <typename E, int HD> struct Tile;   // tokens per step
template <int HD> struct Tile<uint16_t, HD> { static constexpr int TT = 32; };
template <int HD> struct Tile<float, HD> { static constexpr int TT = HD == 64 ? 32 : 16; };


// Tiles of sequence b.
template <int TT>
__device__ __forceinline__ int32_t seq_tiles(const KvArgs &a, int32_t b) {
    const int32_t n = a.lens[b];
    return n <= 0 || n > a.cap ? 0 : (n + TT - 1) / TT;
}

// Sum over the sequences before `upto` (and over all) of their tiles, by a workgroup of 256.
template <int TT>
__device__ __forceinline__ int64_t tiles_before(const KvArgs &a, int32_t upto, int64_t *sh, int64_t *total) {
    int64_t before = 0, all = 0;
    for (int32_t b = threadIdx.x; b < a.n_seq; b += 256) {
        const int32_t t = seq_tiles<TT>(a, b);
        all += t;
        before += b < upto ? t : 0;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        all += __shfl_xor(all, o, 64);
        before += __shfl_xor(before, o, 64);
    }
    if ((threadIdx.x & 63) == 0) {
        sh[threadIdx.x >> 6] = all;
        sh[4 + (threadIdx.x >> 6)] = before;
    }
    __syncthreads();
    *total = sh[0] + sh[1] + sh[2] + sh[3];
    const int64_t r = sh[4] + sh[5] + sh[6] + sh[7];
    __syncthreads();
    return r;
}

// waves a SIMD holds: what the registers of K, two V tiles, the accumulators and the queries leave room for
constexpr int split_waves(int hd) { return hd == 256 ? 1 : 2; }

// LOCAL: one workgroup per (sequence, K/V head), its waves sharing the sequence's tiles, joined in LDS: no second
// launch.  For short caches of few sequences, where launches and round trips are the time.
template <typename E, int HD, bool SCORES, bool LOCAL>
__global__ __launch_bounds__(LOCAL ? 256 * split_waves(HD) : 256, split_waves(HD)) void k_kv_split(KvArgs a, KvAttend at, KvSplit sp) {
    constexpr int TT = Tile<E, HD>::TT, NS = TT / 16;
    constexpr bool BF = sizeof(E) == 2;
    constexpr int KS = HD * (int)sizeof(E) / 64;           // 16-byte loads of a lane per token row of K
    constexpr int NV = BF ? (TT / 32) * 8 : NS * 4;        // tokens of V a lane holds parts of
    constexpr int VC = BF ? (HD == 64 ? 1 : HD / 128) : HD / 64;   // 16-byte (bf16, 64: 8-byte) parts of each
    constexpr int NA = HD / 16;                            // accumulators: 16 dims x 16 heads each
    __shared__ int64_t sh_sum[4];
    __shared__ int64_t sh_total;
    __shared__ int32_t sh_b[4], sh_j[4];
    // logits on their way to memory.  Stores are waited for in their turn with the loads around them, and take
    // longest where loads fill the queues, so a wave gathers what it can hold first (whole calls, 8 sequences of 32768 tokens
    // each, 32 heads on 8 K/V heads, 1.08 GB: 243 us stored tile by tile, 231 gathered in 4 KiB, 216 in 15 KiB; without
    // scores, and so without logits, 194).
    __shared__ __align__(16) float sh_log[4][SCORES ? 3840 : 4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;

    if (blockIdx.x == 0 && (!LOCAL || blockIdx.y == 0)) check_seqs(a);
    // ---- where this workgroup's waves begin ----
    if constexpr (!LOCAL) {
        if (tid < 4) sh_b[tid] = sh_j[tid] = 0;
        const int32_t per = (a.n_seq + 255) / 256, b0 = tid * per, b1 = min(a.n_seq, b0 + per);
        int64_t mine = 0;
        for (int32_t b = b0; b < b1; ++b) mine += seq_tiles<TT>(a, b);
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int64_t x = __shfl_up(incl, o, 64);
            if (lane >= o) incl += x;
        }
        if (lane == 63) sh_sum[wave] = incl;
        __syncthreads();
        int64_t excl = incl - mine;
#pragma unroll
        for (int i = 0; i < 4; ++i) excl += i < wave ? sh_sum[i] : 0;
        const int64_t total = sh_sum[0] + sh_sum[1] + sh_sum[2] + sh_sum[3];
        if (tid == 0) sh_total = total;
        const Ranges rg = ranges_of(total, sp.R);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int32_t r = (blockIdx.x * 4 + w) / sp.hu;
            const int64_t s = rg.start(r);
            if (r < rg.R && mine > 0 && s >= excl && s < excl + mine) {   // one thread at most
                int64_t at0 = excl;
                int32_t b = b0;
                for (; b < b1; ++b) {
                    const int32_t t = seq_tiles<TT>(a, b);
                    if (s < at0 + t) break;
                    at0 += t;
                }
                sh_b[w] = b;
                sh_j[w] = (int32_t)(s - at0);
            }
        }
        __syncthreads();
    }
    int32_t range, hu, count, b0, j0;
    int64_t gtile = 0;
    if constexpr (LOCAL) {
        constexpr int NW = 4 * split_waves(HD);
        hu = blockIdx.x;
        b0 = blockIdx.y;
        range = 0;
        const int32_t nt = seq_tiles<TT>(a, b0);
        j0 = uniform(wave * nt / NW);
        count = uniform((wave + 1) * nt / NW) - j0;
    } else {
        const int32_t job = blockIdx.x * 4 + wave;
        range = job / sp.hu;
        hu = job - range * sp.hu;
        const Ranges rg = ranges_of(sh_total, sp.R);
        if (range >= rg.R) return;
        gtile = rg.start(range);
        count = uniform((int32_t)(rg.start(range + 1) - gtile));
        b0 = uniform(sh_b[wave]);
        j0 = uniform(sh_j[wave]);
    }

    const int32_t kvh = uniform(hu / sp.ncb), cb = uniform(hu - kvh * sp.ncb);
    const int32_t head = kvh * a.group + cb * 16 + col;
    const bool mine = cb * 16 + col < a.group;             // this lane's column is a query head
    const int64_t head_bytes = (int64_t)kvh * HD * sizeof(E);
    const uint32_t page_units = (uint32_t)(a.page_bytes >> 7), tok_units = (uint32_t)(a.tok_bytes >> 7);
    const float scale2 = at.scale * 1.4426950408889634f;

    struct Pos { int32_t b, j, n; };
    auto len_of = [&](int32_t b) { const int32_t n = a.lens[b]; return n <= 0 || n > a.cap ? 0 : n; };
    auto next = [&](Pos p) {                               // only called while there is a next tile
        p.j++;
        if (p.j * TT >= p.n) {
            p.j = 0;
            do { p.b++; p.n = len_of(p.b); } while (p.n == 0 && p.b + 1 < a.n_seq);
        }
        return p;
    };
    // page ids of a tile's tokens, each lane those of token lane % TT; -1 behind the sequence's end
    auto load_ids = [&](const Pos &p, int32_t *kid, int32_t *vid) {
        const int32_t t = p.j * TT + (lane & (TT - 1));
        int32_t e, slot;
        page_of(a, t, &e, &slot);
        const int32_t *row = a.table + (int64_t)p.b * 2 * a.max_pages + e;
        *kid = *vid = -1;
        if (t < p.n) { *kid = row[0]; *vid = row[a.max_pages]; }
    };
    int bad = 0;
    // addresses in units of 128 bytes (every token row starts on one), and which tokens are there
    auto to_units = [&](const Pos &p, int32_t kid, int32_t vid, uint32_t *ku, uint32_t *vu) -> uint64_t {
        const int32_t t = p.j * TT + (lane & (TT - 1));
        int32_t e, slot;
        page_of(a, t, &e, &slot);
        const bool ok = kid >= 0 && vid >= 0 && kid < a.num_pages && vid < a.num_pages;
        if (t < p.n && !ok) bad = DEV_ERR_PAGE;
        *ku = ok ? (uint32_t)kid * page_units + (uint32_t)slot * tok_units : 0u;
        *vu = ok ? (uint32_t)vid * page_units + (uint32_t)slot * tok_units : 0u;
        return __ballot(ok);
    };
    const char *base = a.pages + head_bytes;
    u32x4_t K[NS][KS], V0[NV][VC], V1[NV][VC];   // V of this tile and of the next
    auto load_k = [&](uint32_t ku) {
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const uint32_t u = __shfl(ku, 16 * s + col, 64);
            const char *p = base + ((uint64_t)u << 7) + 16 * g;
#pragma unroll
            for (int i = 0; i < KS; ++i) K[s][i] = load16(p + 64 * i);
        }
    };
    auto v_token = [&](int j) { return BF ? 32 * (j >> 3) + 16 * ((j >> 2) & 1) + 4 * g + (j & 3) : 16 * (j >> 2) + 4 * g + (j & 3); };
    auto load_v = [&](u32x4_t (&Vr)[NV][VC], uint32_t vu) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t u = __shfl(vu, v_token(j), 64);
            const char *p = base + ((uint64_t)u << 7);
            if constexpr (BF && HD == 64) {
                const uint2 x = *(const uint2 *)(p + 8 * col);
                Vr[j][0][0] = x.x;
                Vr[j][0][1] = x.y;
            } else {
#pragma unroll
                for (int c = 0; c < VC; ++c) Vr[j][c] = load16(p + 16 * col + 256 * c);
            }
        }
    };

    u32x4_t Q[KS];
    f32x4_t acc[NA];
    float m = -INFINITY, l = 0.f;
    // query rows of sequence b; lanes without a head take the first one's (their columns are never stored)
    auto load_q = [&](int32_t b) {
        const char *p = (const char *)at.q + ((int64_t)b * at.ldq + (int64_t)(mine ? head : 0) * HD) * sizeof(E) + 16 * g;
#pragma unroll
        for (int i = 0; i < KS; ++i) Q[i] = load16(p + 64 * i);
    };
    auto reset = [&]() {
#pragma unroll
        for (int i = 0; i < NA; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        m = -INFINITY;
        l = 0.f;
    };
    auto finish = [&](const Pos &p, bool whole, int slot) {
        float L = l + __shfl_xor(l, 16, 64);
        L += __shfl_xor(L, 32, 64);
        if (!mine) return;
        const int64_t pl = ((int64_t)range * 2 + slot) * a.n_heads + head;
        if (g == 0) (whole ? sp.done_ml[(int64_t)p.b * a.n_heads + head] : sp.part_ml[pl]) = make_float2(m, L);
        const float inv = whole ? 1.f / L : 1.f;
        const bool none = whole && L == 0.f;               // no weight: zero, also where a value is not finite
        float *po = sp.part_o + pl * HD;
        E *o = (E *)at.out + (int64_t)p.b * at.ldo + (int64_t)head * HD;
        constexpr int W = BF && HD >= 128 ? 8 : 4;         // consecutive dims of one row of the accumulators
#pragma unroll
        for (int c = 0; c < NA / W; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = 16 * W * c + W * (4 * g + r);
                float v[W];
#pragma unroll
                for (int i = 0; i < W; ++i) v[i] = none ? 0.f : acc[W * c + i][r] * inv;
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < W; i += 4) *(float4 *)(po + d + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                } else if constexpr (BF && W == 8) {
                    store16(o + d, u32x4_t{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])});
                } else if constexpr (BF) {
                    *(uint2 *)(o + d) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
                } else {
                    *(float4 *)(o + d) = make_float4(v[0], v[1], v[2], v[3]);
                }
            }
    };

    // ---- the pipeline: page ids two tiles ahead, K and V one tile ahead ----
    // The loads of the next tile are issued whether there is one or not (behind the last tile they read the
    // pool's first page): a load under a condition would make every later wait a wait for all.
    Pos p0{b0, j0, len_of(b0)};
    Pos p1 = p0, p2;
    int32_t kid, vid;
    uint32_t ku, vu;
    uint64_t there, there1;
    load_ids(p0, &kid, &vid);
    load_q(p0.b);
    reset();
    there = to_units(p0, kid, vid, &ku, &vu);
    if (count > 1) p1 = next(p0);
    load_ids(p1, &kid, &vid);
    p2 = p1;
    load_k(ku);
    load_v(V0, vu);
    const int32_t hold = max(3840 / (sp.cols * TT), 1);
    int32_t held = 0;
    int32_t first_j = p0.j;      // the tile this wave began the sequence at
    bool first_piece = true;
    auto step = [&](int32_t i, u32x4_t (&Vr)[NV][VC], u32x4_t (&Vn)[NV][VC]) {
        // logits: rows are tokens, columns heads
        f32x4_t S[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            S[s] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                if constexpr (BF) {
                    S[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, K[s][k]),
                                                                   __builtin_bit_cast(bf16x8_t, Q[k]), S[s], 0, 0, 0);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        S[s] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(K[s][k][e]), __uint_as_float(Q[k][e]), S[s], 0, 0, 0);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        const bool more = i + 1 < count;
        if (more && p1.j == 0) load_q(p1.b);
        uint32_t ku1, vu1;
        there1 = to_units(p1, kid, vid, &ku1, &vu1);
        if (i + 2 < count) p2 = next(p1);
        load_ids(p2, &kid, &vid);
        load_k(more ? ku1 : 0u);
        load_v(Vn, more ? vu1 : 0u);
        __builtin_amdgcn_sched_barrier(0);
        // softmax statistics of this lane's head; the four lane groups hold different tokens
        const bool full = (~there & ((1ull << TT) - 1)) == 0;
        float mt = -INFINITY;
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float x = S[s][r] * scale2;
                if (!full && !((there >> (16 * s + 4 * g + r)) & 1)) x = -INFINITY;
                S[s][r] = x;
                mt = fmaxf(mt, x);
            }
        if constexpr (SCORES) {
            float *lg = sh_log[wave] + (held * sp.cols + col) * TT + 4 * g;
            if (mine)
#pragma unroll
                for (int s = 0; s < NS; ++s) *(f32x4_t *)(lg + 16 * s) = S[s];
            if (++held == hold || !more) {                 // what is held, in one go
                __builtin_amdgcn_wave_barrier();
                float *dst = sp.logits + (hu * sp.tiles + gtile + 1 - held) * sp.cols * TT;
                for (int32_t x = 4 * lane; x < held * sp.cols * TT; x += 256)
                    *(f32x4_t *)(dst + x) = *(const f32x4_t *)(sh_log[wave] + x);
                held = 0;
                __builtin_amdgcn_wave_barrier();
            }
        }
        mt = fmaxf(mt, __shfl_xor(mt, 16, 64));
        mt = fmaxf(mt, __shfl_xor(mt, 32, 64));
        const float mn = fmaxf(m, mt), ms = mn == -INFINITY ? 0.f : mn;
        const float c = exp2_hw(m - ms);
        m = mn;
        float ps = 0.f;
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                S[s][r] = exp2_hw(S[s][r] - ms);
                ps += S[s][r];
            }
        l = l * c + ps;
#pragma unroll
        for (int x = 0; x < NA; ++x) acc[x] *= c;
        if (!full) {                                       // what lies where no token is must not reach the products
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (!((there >> v_token(j)) & 1))
#pragma unroll
                    for (int cc = 0; cc < VC; ++cc) Vr[j][cc] = u32x4_t{0, 0, 0, 0};
        }
        // out^T += V^T P^T: rows are dims, columns heads
        if constexpr (BF) {
#pragma unroll
            for (int q = 0; q < TT / 32; ++q) {
                // weights as the sum of two bfloat16 numbers, so that they are off by at most 2^-15: the
                // first their leading bits, cut off, the second the rest, rounded.  The second is raised to 2^-126 where
                // the rest is less, unless the weight itself is: an infinite value times a weight stays that infinity,
                // and a weight of zero stays zero.  (Below 2^-111 a weight is off by up to 2^-126, not by 2^-15 of itself.)
                u32x4_t hi, lo;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float a0 = S[2 * q + x / 2][2 * (x & 1)], a1 = S[2 * q + x / 2][2 * (x & 1) + 1];
                    const uint32_t h0 = __float_as_uint(a0) & 0xffff0000u, h1 = __float_as_uint(a1) & 0xffff0000u;
                    hi[x] = h0 >> 16 | h1;
                    const float f0 = __uint_as_float(h0), f1 = __uint_as_float(h1);
                    lo[x] = pack2(__builtin_amdgcn_fmed3f(a0 - f0, f0, 0x1p-126f), __builtin_amdgcn_fmed3f(a1 - f1, f1, 0x1p-126f));
                }
                constexpr int W = HD == 64 ? 4 : 8;
#pragma unroll
                for (int cc = 0; cc < VC; ++cc)
#pragma unroll
                    for (int x = 0; x < W; ++x) {
                        u32x4_t f;
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            f[y] = __builtin_amdgcn_perm(Vr[8 * q + 2 * y + 1][cc][x / 2], Vr[8 * q + 2 * y][cc][x / 2],
                                                         x & 1 ? 0x07060302u : 0x05040100u);
                        acc[W * cc + x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8_t, f), __builtin_bit_cast(bf16x8_t, lo), acc[W * cc + x], 0, 0, 0);
                        acc[W * cc + x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8_t, f), __builtin_bit_cast(bf16x8_t, hi), acc[W * cc + x], 0, 0, 0);
                    }
            }
        } else {
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int cc = 0; cc < VC; ++cc)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[4 * cc + e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(Vr[4 * s + r][cc][e]), S[s][r],
                                                                                   acc[4 * cc + e], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        const bool ends = (p0.j + 1) * TT >= p0.n;
        if (!LOCAL && (ends || i + 1 == count)) {
            finish(p0, ends && first_j == 0, first_piece ? 0 : 1);
            first_piece = false;
            reset();
            first_j = 0;
        }
        p0 = p1;
        p1 = p2;
        there = there1;
        ++gtile;
    };
    for (int32_t i = 0; i < count;) {
        step(i, V0, V1);
        if (++i >= count) break;
        step(i, V1, V0);
        ++i;
    }
    if (bad) record(a, bad);
    if constexpr (LOCAL) {
        constexpr int NW = 4 * split_waves(HD), W = BF && HD >= 128 ? 8 : 4;
        extern __shared__ __align__(16) float sh_o[];       // [NW][cols][HD], then maxima and sums [NW][cols]
        float2 *sh_s = (float2 *)(sh_o + NW * sp.cols * HD);
        float L = l + __shfl_xor(l, 16, 64);
        L += __shfl_xor(L, 32, 64);
        if (mine) {
            float *o = sh_o + (wave * sp.cols + col) * HD;
#pragma unroll
            for (int c = 0; c < NA / W; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int i = 0; i < W; ++i) o[16 * W * c + W * (4 * g + r) + i] = acc[W * c + i][r];
            if (g == 0) sh_s[wave * sp.cols + col] = make_float2(m, L);
        }
        __syncthreads();
        const int32_t nc = min(16, a.group - 16 * cb);
        for (int32_t x = tid; x < nc * HD; x += 64 * NW) {
            const int32_t c = x / HD, d = x % HD;
            float M = -INFINITY, sum = 0.f, v = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) M = fmaxf(M, sh_s[w * sp.cols + c].x);
            const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float2 ml = sh_s[w * sp.cols + c];
                const float f = exp2_hw(ml.x - Ms);
                sum += ml.y * f;
                v += sh_o[(w * sp.cols + c) * HD + d] * f;
            }
            from_f32((E *)at.out + (int64_t)b0 * at.ldo + (int64_t)(kvh * a.group + cb * 16 + c) * HD + d, sum == 0.f ? 0.f : v / sum);
        }
    }
}

// Put the pieces of a sequence (blockIdx.y) together, and form its scores.  The first workgroups take jh heads
// each: a wave to a head where the pieces are few, else all four waves a part of the pieces of one head after the
// other, joined in LDS.  The others take 256 tokens' scores.
template <typename E, int HD>
__global__ __launch_bounds__(256) void k_kv_join(KvArgs a, KvAttend at, KvSplit sp) {
    constexpr int TT = Tile<E, HD>::TT;
    extern __shared__ float2 sh_ml[];
    __shared__ int64_t sh[8];
    __shared__ float sh_o[4][HD], sh_m[4], sh_l[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t join_wgs = (a.n_heads + sp.jh - 1) / sp.jh, b = blockIdx.y, first = ((int32_t)blockIdx.x - join_wgs) * 256;
    const int32_t n = a.lens[b], nt = seq_tiles<TT>(a, b);
    if (first >= 0 && (nt == 0 || first >= n)) return;
    int64_t total;
    const int64_t t0 = tiles_before<TT>(a, b, sh, &total);
    if (first < 0) {
        const int32_t h0 = blockIdx.x * sp.jh;
        constexpr int PER = HD / 64;
        E *out = (E *)at.out + (int64_t)b * at.ldo;
        if (nt == 0) {
            if (wave < sp.jh && h0 + wave < a.n_heads)
#pragma unroll
                for (int i = 0; i < PER; ++i) from_f32(out + (int64_t)(h0 + wave) * HD + 64 * i + lane, 0.f);
            return;
        }
        const Pieces p = pieces_of(t0, t0 + nt, ranges_of(total, sp.R));
        if (p.r0 == p.r1) return;
        // pieces r, r + by, ... of head h: a lane's dims, and the maximum and sum they go by; four loads at once
        float m, l, acc[PER];
        auto gather = [&](int32_t h, int32_t r, int32_t by) {
            m = -INFINITY;
            l = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] = 0.f;
            for (; r <= p.r1; r += 4 * by) {
                float2 ml[4];
                float v[4][PER];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int32_t ru = min(r + by * u, p.r1);
                    const int64_t pl = ((int64_t)ru * 2 + (ru == p.r0 ? p.s0 : 0)) * a.n_heads + h;
                    ml[u] = sp.part_ml[pl];
#pragma unroll
                    for (int i = 0; i < PER; ++i) v[u][i] = sp.part_o[pl * HD + 64 * i + lane];
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (r + by * u > p.r1) break;
                    const float mn = fmaxf(m, ml[u].x), ms = mn == -INFINITY ? 0.f : mn;
                    const float c = exp2_hw(m - ms), w = exp2_hw(ml[u].x - ms);
                    l = l * c + ml[u].y * w;
#pragma unroll
                    for (int i = 0; i < PER; ++i) acc[i] = acc[i] * c + v[u][i] * w;
                    m = mn;
                }
            }
        };
        if (sp.jh == 4 && p.r1 - p.r0 < 8) {                // few pieces: a wave to a head
            if (h0 + wave < a.n_heads) {
                gather(h0 + wave, p.r0, 1);
                const float inv = 1.f / l;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    from_f32(out + (int64_t)(h0 + wave) * HD + 64 * i + lane, l == 0.f ? 0.f : acc[i] * inv);
            }
            return;
        }
        for (int32_t h = h0; h < min(h0 + sp.jh, a.n_heads); ++h) {
            gather(h, p.r0 + wave, 4);
#pragma unroll
            for (int i = 0; i < PER; ++i) sh_o[wave][64 * i + lane] = acc[i];
            if (lane == 0) { sh_m[wave] = m; sh_l[wave] = l; }
            __syncthreads();
            const float M = fmaxf(fmaxf(sh_m[0], sh_m[1]), fmaxf(sh_m[2], sh_m[3])), Ms = M == -INFINITY ? 0.f : M;
            float L = 0.f, w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = exp2_hw(sh_m[i] - Ms);
                L += sh_l[i] * w[i];
            }
            const float inv = 1.f / L;
            for (int d = tid; d < HD; d += 256) {
                float v = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) v += sh_o[i][d] * w[i];
                from_f32(out + (int64_t)h * HD + d, L == 0.f ? 0.f : v * inv);
            }
            __syncthreads();
        }
        return;
    }
    // The first heads' logits are on their way while the statistics are formed.
    const int32_t t = first + tid;
    const float *lg = sp.logits + (t0 + t / TT) * sp.cols * TT + (t & (TT - 1));
    const int64_t plane = sp.tiles * sp.cols * TT;
    int32_t cb = 0, col = 0;
    constexpr int AHEAD = 32;
    float x[AHEAD], sum = 0.f;
    auto fetch = [&](int32_t heads) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (i >= heads) break;
            x[i] = t < n ? lg[col * TT] : 0.f;
            if (++col == min(16, a.group - 16 * cb)) {
                col = 0;
                cb = cb + 1 == sp.ncb ? 0 : cb + 1;
                lg += plane;
            }
        }
    };
    fetch(a.n_heads);
    const int64_t si = (int64_t)b * at.score_ld + t;
    const float prior = at.prior && t < n ? at.prior[si] : 0.f;
    // each head's final maximum and 1 / sum, by as many threads a head as there are
    const Pieces p = pieces_of(t0, t0 + nt, ranges_of(total, sp.R));
    const int32_t per = max(1, 256 / a.n_heads);
    for (int32_t x = tid; x < a.n_heads * per; x += 256) {
        const int32_t hh = per == 1 ? x : x % a.n_heads, k = per == 1 ? 0 : x / a.n_heads;
        float m = -INFINITY, l = 0.f;
        if (p.r0 == p.r1) {
            if (k == 0) {
                const float2 ml = sp.done_ml[(int64_t)b * a.n_heads + hh];
                m = ml.x;
                l = ml.y;
            }
        } else {
#pragma unroll 4
            for (int32_t r = p.r0 + k; r <= p.r1; r += per) {
                const float2 ml = sp.part_ml[((int64_t)r * 2 + (r == p.r0 ? p.s0 : 0)) * a.n_heads + hh];
                const float mn = fmaxf(m, ml.x), ms = mn == -INFINITY ? 0.f : mn;
                l = l * exp2_hw(m - ms) + ml.y * exp2_hw(ml.x - ms);
                m = mn;
            }
        }
        sh_ml[k * a.n_heads + hh] = make_float2(m, l);
    }
    __syncthreads();
    for (int32_t hh = tid; hh < a.n_heads; hh += 256) {
        float m = -INFINITY, l = 0.f;
        for (int32_t k = 0; k < per; ++k) {
            const float2 ml = sh_ml[k * a.n_heads + hh];
            const float mn = fmaxf(m, ml.x), ms = mn == -INFINITY ? 0.f : mn;
            l = l * exp2_hw(m - ms) + ml.y * exp2_hw(ml.x - ms);
            m = mn;
        }
        sh_ml[hh] = make_float2(m == -INFINITY ? 0.f : m, l == 0.f ? 0.f : 1.f / l);   // this thread alone reads head hh
    }
    __syncthreads();
    for (int32_t hh = 0; hh < a.n_heads; hh += AHEAD) {
        if (hh) fetch(a.n_heads - hh);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (i >= a.n_heads - hh) break;
            const float2 ml = sh_ml[hh + i];
            sum += exp2_hw(x[i] - ml.x) * ml.y;
        }
    }
    if (t < n) at.scores[si] = prior + sum;
}

// ---- host ----------------------------------------------------------------------------------------
namespace {

int tile_tokens(int dtype, int hd) { return dtype == LORA_F32 && hd > 64 ? 16 : 32; }

struct SplitPlan {
    int32_t R, ncb, hu, cols;
    int64_t tiles;
    bool local;
    size_t off_ml, off_done, off_logits;
    size_t need, ask;         // bytes of workspace that the call uses, and that it asks for
};
SplitPlan split_plan(int dtype, int n_heads, int n_kv, int hd, int32_t n_seq, int64_t max_len, bool scores) {
    SplitPlan s;
    const int tt = tile_tokens(dtype, hd), group = n_heads / n_kv;
    const int64_t tiles = s.tiles = (max_len + tt - 1) / tt * n_seq;
    s.cols = std::min(group, 16);
    s.ncb = (group + 15) / 16;
    s.hu = n_kv * s.ncb;
    // One workgroup per (sequence, head), all of them on the chip at once, where none of their waves gets more than a few
    // tiles.  Whole calls, 32 heads of 128: one sequence of 203 tokens 8.5 us (ranges and join: 12.5), of 768 12.5 (13.9),
    // eight of 1024 28.0 (33.4).  With fewer than 64 workgroups three tiles a wave are the most, for float32: one sequence
    // of 400 tokens would take 17.0 (15.0), of 512 19.0 (16.4).  (bfloat16 keeps to the same, though four would do: one of
    // 1024 14.8 (15.8), 16 heads of 64 10.5 (13.8), 16 of 256 on 4, 512 tokens, 15.8 (15.4).)  Behind that the ranges are as
    // fast, and lengths that differ leave none of their waves idle.  Scores need every head's sums, so they keep the second
    // launch.
    const int64_t wgs = (int64_t)n_seq * s.hu;
    auto few = [&](int64_t w) { return (max_len + tt - 1) / tt <= (w < 64 ? 3 : 4) * 4 * split_waves(hd); };
    s.local = !scores && wgs <= 256 && few(wgs);
    // as many waves as the chip holds; no more ranges than tiles
    s.R = (int32_t)std::max<int64_t>(1, std::min<int64_t>(tiles, 1024 * split_waves(hd) / s.hu));
    auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
    s.off_ml = up((size_t)s.R * 2 * n_heads * hd * 4);
    s.off_done = s.off_ml + up((size_t)s.R * 2 * n_heads * 8);
    s.off_logits = s.off_done + up((size_t)n_seq * n_heads * 8);
    const size_t ranges = s.off_logits + (scores ? up((size_t)s.hu * tiles * s.cols * tt * 4) : 0);
    s.need = s.local ? 0 : ranges;
    // What serves the largest call has to serve them all, and of a length at which 64 workgroups take one launch fewer may
    // take two: nothing is asked for only where one sequence alone would take one launch too.
    s.ask = s.local && few(s.hu) ? 0 : ranges;
    return s;
}

template <typename E, int HD>
hipError_t run(int dtype, const KvArgs &a, const KvAttend &at, hipStream_t s) {
    const SplitPlan pl = split_plan(dtype, a.n_heads, a.n_kv, HD, a.n_seq, a.cap, at.scores != nullptr);
    char *ws = (char *)at.ws;
    // a wave to a head where a sequence has a few pieces on average (64 sequences, 64 ranges: 14.3 -> 11.6 us with
    // scores); all four waves to one where it has many (8 sequences, 256 ranges: 15.5 us, one wave 26.8)
    const int32_t jh = pl.R <= 4 * a.n_seq ? 4 : 1;
    const KvSplit sp{pl.R, pl.ncb, pl.hu, jh, (float *)ws, (float2 *)(ws + pl.off_ml), (float2 *)(ws + pl.off_done),
                     pl.cols, pl.tiles, (float *)(ws + pl.off_logits)};
    if (pl.local) {
        constexpr int NW = 4 * split_waves(HD);
        const int lds = NW * pl.cols * (HD * 4 + 8);
        if (lds > 64 * 1024) {                              // asked for on each device
            const hipError_t e = hipFuncSetAttribute((const void *)k_kv_split<E, HD, false, true>,
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds);
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL((k_kv_split<E, HD, false, true>), dim3(pl.hu, a.n_seq), dim3(64 * NW), lds, s, a, at, sp);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)(((int64_t)pl.R * pl.hu + 3) / 4));
    if (at.scores) hipLaunchKernelGGL((k_kv_split<E, HD, true, false>), grid, dim3(256), 0, s, a, at, sp);
    else hipLaunchKernelGGL((k_kv_split<E, HD, false, false>), grid, dim3(256), 0, s, a, at, sp);
    const int32_t sb = at.scores ? (a.cap + 255) / 256 : 0;
    hipLaunchKernelGGL((k_kv_join<E, HD>), dim3((a.n_heads + sp.jh - 1) / sp.jh + sb, a.n_seq), dim3(256),
                       at.scores ? std::max(a.n_heads, 256) * sizeof(float2) : 0, s, a, at, sp);
    return hipGetLastError();
}

template <typename E>
hipError_t by_dim(int dtype, const KvArgs &a, const KvAttend &at, hipStream_t s) {
    return a.head_dim == 64 ? run<E, 64>(dtype, a, at, s) : a.head_dim == 128 ? run<E, 128>(dtype, a, at, s)
                                                                              : run<E, 256>(dtype, a, at, s);
}

}  // namespace

size_t kv_attend_ws_bytes(int dtype, const lora_kv_layout_t &l, int32_t n_seq, int64_t max_len, bool scores) {
    return split_plan(dtype, l.n_heads, l.n_kv_heads, l.head_dim, n_seq, max_len, scores).ask;
}

size_t kv_attend_ws_need(int dtype, const lora_kv_layout_t &l, int32_t n_seq, int64_t max_len, bool scores) {
    return split_plan(dtype, l.n_heads, l.n_kv_heads, l.head_dim, n_seq, max_len, scores).need;
}

hipError_t launch_kv_attend(int dtype, const KvArgs &a, const KvAttend &at, hipStream_t s) {
    return dtype == LORA_F32 ? by_dim<float>(dtype, a, at, s) : by_dim<uint16_t>(dtype, a, at, s);
}

}  // namespace lorapool

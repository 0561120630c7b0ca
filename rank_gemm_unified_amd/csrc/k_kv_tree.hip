// Attention of a tree of new tokens per sequence over the paged cache (the verification of drafted tokens): up to 16 rows of a
// K/V head, and the pieces' joining for all; more rows are k_kv_tree_wide.hip's.
//
// A sequence's m nodes times the query heads that share a K/V head are the rows of a matrix product with the K/V
// head's tokens, node by node: row r is head r % group of node r / group.  4 * rows * head_dim operations for 2 *
// head_dim elements of K and V: up to a hundred rows or so HBM bounds it.  The tiles (TT tokens) of all sequences, one
// sequence behind the other, are cut into equal ranges whatever the lengths; one workgroup takes one range of one K/V
// head and up to 16 NB rows, or of up to four neighbouring heads, whose pieces of a page are then read at one time; its waves
// an equal part of the range each, K and V of the next tile in flight.  Where a sequence ends the waves' sums are joined in
// LDS, so that only what a range has of a sequence it did not see whole goes to the workspace (rows * head_dim numbers of 32
// bits, once a workgroup and not once a wave); k_kv_tree_join puts those pieces together.  No atomics: results do not change
// from call to call.  Weights of bfloat16 pools are two bfloat16 numbers (off by 2^-15 of themselves at most): the second
// product is nearly free beside the reads.
// 64 trees of 16 nodes behind up to 1031 tokens, 32 heads of 128: 133 to 152 us on several cards for 648 MB (4.3 to 4.9 TB/s); in a
// trace the kernel here takes 133 to 136 of them, and the join 8.  One tree behind 203 tokens: 9.5 us, the
// chain length -> page ids -> K -> softmax -> V -> join in LDS.
#include <algorithm>

#include "kv_tree.h"

namespace lorapool {

template <typename E, int HD, int NB>
struct TreeTile {
    static constexpr bool BF = sizeof(E) == 2;
    static constexpr int TT = BF || HD == 64 ? 32 : 16;    // tokens per step
    static constexpr int WAVES = HD == 256 || (!BF && HD == 128 && NB == 2) ? 1 : 2;   // a SIMD holds: registers
    static constexpr bool AHEAD = NB == 1;                 // V of the next tile has registers of its own
    static constexpr int NW = 4 * WAVES;                   // waves of a workgroup; one workgroup a CU
    static constexpr int CW = 16 * NB;
    static constexpr int LDW = HD + 4;                     // floats between rows in LDS: columns in other banks
    static constexpr int LDS = NW * CW * (LDW * 4 + 8);
};

// LOCAL: a workgroup takes one whole sequence (blockIdx.y) of a K/V head: no second launch.  For few or short ones.
template <typename E, int HD, int NB, bool LOCAL>
__global__ __launch_bounds__((64 * TreeTile<E, HD, NB>::NW), (TreeTile<E, HD, NB>::WAVES)) void k_kv_tree(KvArgs a, KvAttend at, KvTreeSplit tr) {
    using C = TreeTile<E, HD, NB>;
    constexpr int TT = C::TT, NS = TT / 16, NW = C::NW, CW = C::CW, LDW = C::LDW, THREADS = 64 * NW;
    constexpr bool BF = C::BF;
    constexpr int KS = HD * (int)sizeof(E) / 64;           // 16-byte loads of a lane per token row of K
    constexpr int NV = BF ? (TT / 32) * 8 : NS * 4;        // tokens of V a lane holds parts of
    constexpr int VC = BF ? (HD == 64 ? 1 : HD / 128) : HD / 64;   // 16-byte (bf16, 64: 8-byte) parts of each
    constexpr int NA = HD / 16;                            // accumulators: 16 dims x 16 rows each
    constexpr int W = BF && HD >= 128 ? 8 : 4;             // consecutive dims of one row of the accumulators
    constexpr int SLOTS = LOCAL ? 1 : 2;
    extern __shared__ __align__(16) float sh_o[];          // [NW][SLOTS][CW][LDW], then maxima and sums [NW][SLOTS][CW]
    float2 *sh_s = (float2 *)(sh_o + NW * SLOTS * CW * LDW);
    __shared__ int32_t piece_b[NW * SLOTS], piece_at[NW * SLOTS];   // of each: its sequence, or -1, and where in the range that begins
    __shared__ TreeBegin parts[NW];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), col = lane & 15, g = lane >> 4;

    // LOCAL: all waves take one head.  Else `hw` neighbouring ones, so that neighbouring pieces of a page are read at the same
    // time, and each head's waves a part of the range each.
    const int32_t hw = LOCAL ? 1 : tr.hw, head0 = blockIdx.x % (a.n_kv / hw) * hw, rest = blockIdx.x / (a.n_kv / hw);
    const int32_t kvh = head0 + wave % hw, part = wave / hw, n_parts = NW / hw, r0 = rest % tr.ncb * CW, range = rest / tr.ncb;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        int bits = 0;
        for (int32_t b = tid; b < a.n_seq; b += THREADS) bits |= tree_rows(a, tr, b).err;
        record(a, bits);
    }
    int32_t total, begin, count, from = 0, b0 = blockIdx.y, range_b = b0;
    if constexpr (LOCAL) {
        total = count = tree_tiles<TT>(a, tree_rows_scalar(a, tr, b0), r0);
        begin = 0;
    } else {
        total = tree_begin<E, TT, THREADS>(a, at, tr, r0, CW, head0, hw, range, n_parts, parts);
        if (total == 0) return;
        range_b = uniform(parts[0].b);
        b0 = uniform(parts[part].b);
        from = uniform(parts[part].j);
        begin = uniform(part_of(total, part, n_parts));    // this wave's tiles [begin, count) of the range
        count = uniform(part_of(total, part + 1, n_parts));
    }

    const int64_t head_bytes = (int64_t)kvh * HD * sizeof(E);
    const uint32_t page_units = (uint32_t)(a.page_bytes >> 7), tok_units = (uint32_t)(a.tok_bytes >> 7);
    const float scale2 = at.scale * 1.4426950408889634f;

    // page ids of a tile's tokens, each lane those of token lane % TT
    auto load_ids = [&](const TreePos &p, int32_t *kid, int32_t *vid) {
        const int32_t t = p.j * TT + (lane & (TT - 1));
        int32_t e, slot;
        page_of(a, t, &e, &slot);
        const int32_t *row = a.table + (int64_t)p.b * 2 * a.max_pages + (t < p.n ? e : 0);   // (there is a first entry)
        *kid = row[0];
        *vid = row[a.max_pages];
    };
    int bad = 0;
    auto to_units = [&](const TreePos &p, int32_t kid, int32_t vid, uint32_t *ku, uint32_t *vu) -> uint64_t {
        const int32_t t = p.j * TT + (lane & (TT - 1));
        int32_t e, slot;
        page_of(a, t, &e, &slot);
        const bool ok = t < p.n && kid >= 0 && vid >= 0 && kid < a.num_pages && vid < a.num_pages;
        if (t < p.n && !ok) bad = DEV_ERR_PAGE;
        *ku = ok ? (uint32_t)kid * page_units + (uint32_t)slot * tok_units : 0u;
        *vu = ok ? (uint32_t)vid * page_units + (uint32_t)slot * tok_units : 0u;
        return __ballot(ok);
    };
    const char *base = a.pages + head_bytes;
    u32x4_t K[NS][KS], V0[NV][VC], V1[NV][VC];
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
    auto load_v = [&](u32x4_t (&V)[NV][VC], uint32_t vu) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t u = __shfl(vu, v_token(j), 64);
            const char *p = base + ((uint64_t)u << 7);
            if constexpr (BF && HD == 64) {
                const uint2 x = *(const uint2 *)(p + 8 * col);
                V[j][0][0] = x.x;
                V[j][0][1] = x.y;
            } else {
#pragma unroll
                for (int c = 0; c < VC; ++c) V[j][c] = load16(p + 16 * col + 256 * c);
            }
        }
    };
    // Rows of this lane's columns: r0 + 16 x + col.  Columns without a row take the sequence's first (they are
    // never stored).
    auto row_of = [&](const TreePos &p, int x) {
        const int32_t r = r0 + 16 * x + col;
        return r < p.m * a.group ? r : 0;
    };
    u32x4_t Q[NB][KS];
    auto load_q = [&](const TreePos &p) {
#pragma unroll
        for (int x = 0; x < NB; ++x) {
            const int32_t r = row_of(p, x), node = node_of(a, tr, r);
            const char *q = (const char *)at.q + ((int64_t)(p.first + node) * at.ldq + (int64_t)(kvh * a.group + r - node * a.group) * HD) * sizeof(E) + 16 * g;
#pragma unroll
            for (int i = 0; i < KS; ++i) Q[x][i] = load16(q + 64 * i);
        }
    };
    uint64_t mlo[NB], mhi[NB];
    auto load_mask = [&](const TreePos &p) {
#pragma unroll
        for (int x = 0; x < NB; ++x) mask_at(tr, p.first + node_of(a, tr, row_of(p, x)), p.j * TT - (p.n - p.m), &mlo[x], &mhi[x]);
    };

    f32x4_t acc[NB][NA];
    float m[NB], l[NB];
    bool odd = false;                                      // some node's V holds an infinity or NaN
    auto reset = [&]() {
#pragma unroll
        for (int x = 0; x < NB; ++x) {
#pragma unroll
            for (int i = 0; i < NA; ++i) acc[x][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            m[x] = -INFINITY;
            l[x] = 0.f;
        }
        odd = false;
    };

    // The segment: what the wave has of one sequence, its tiles [begin, end) of the range, the sequence's from `from` on.
    TreePos seg = tree_pos<TT>(a, tr, r0, b0, from);
    if (LOCAL && r0 >= seg.m * a.group) return;            // no rows in this block
    int32_t end = min(count, begin + seg.tiles - from);
    if (lane < SLOTS) piece_b[wave * SLOTS + lane] = -1;
    // Infinities and NaN of nodes' V, which the products leave out, to the rows that see them: into this wave's sums in LDS.
    auto put_odd = [&](float *so) {
        const int32_t old = seg.n - seg.m;
        const int32_t *row = a.table + (int64_t)seg.b * 2 * a.max_pages;
#pragma unroll 1
        for (int32_t t = old; t < seg.n; ++t) {
            const int32_t j = t - old;
            if (t / TT < from || (LOCAL ? t / TT % NW != wave : begin + t / TT - from >= end) || token_offset(a, row, t) < 0) continue;
            const int64_t off = token_offset(a, row + a.max_pages, t);
            if (off < 0) continue;
            const E *v = (const E *)(base + off);
#pragma unroll 1
            for (int32_t d = lane; d < HD; d += 64) {
                const float y = to_f32(v[d]);
                if (y - y == 0.f) continue;
#pragma unroll 1
                for (int32_t c = 0; c < CW; ++c) {
                    const int32_t r = r0 + c;
                    if (r >= seg.m * a.group) break;
                    const uint64_t *w = tr.mask + (int64_t)(seg.first + node_of(a, tr, r)) * tr.words;
                    if (w[j >> 6] >> (j & 63) & 1) so[c * LDW + d] += y;
                }
            }
        }
    };
    auto out_at = [&](int32_t first, int32_t kvh, int32_t r, int32_t d) {
        const int32_t node = node_of(a, tr, r0 + r);
        return (E *)at.out + (int64_t)(first + node) * at.ldo + (int64_t)(kvh * a.group + r0 + r - node * a.group) * HD + d;
    };
    auto put_out = [&](E *o, f32x4_t v, float sum) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (sum == 0.f) v = f32x4_t{0.f, 0.f, 0.f, 0.f};   // no weight: zero, also where a value is not finite
        if constexpr (BF) *(uint2 *)o = make_uint2(pack2(v[0] * inv, v[1] * inv), pack2(v[2] * inv, v[3] * inv));
        else *(f32x4_t *)o = v * inv;
    };
    // The segment's sums to LDS, and out if the wave saw the sequence whole: a wave waits for no other while it has tiles.
    bool first_piece = true;
    auto flush = [&]() {
        const bool whole = !LOCAL && from == 0 && end - begin == seg.tiles;
        const int slot = wave * SLOTS + (LOCAL || (first_piece && !whole) ? 0 : 1);
        float *so = sh_o + slot * CW * LDW;
        float2 *ss = sh_s + slot * CW;
#pragma unroll
        for (int x = 0; x < NB; ++x) {
            float L = l[x] + __shfl_xor(l[x], 16, 64);
            L += __shfl_xor(L, 32, 64);
            float *o = so + (16 * x + col) * LDW;
#pragma unroll
            for (int c = 0; c < NA / W; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int i = 0; i < W; i += 4)
                        *(f32x4_t *)(o + 16 * W * c + W * (4 * g + r) + i) =
                            f32x4_t{acc[x][W * c + i][r], acc[x][W * c + i + 1][r], acc[x][W * c + i + 2][r], acc[x][W * c + i + 3][r]};
            if (g == 0) ss[16 * x + col] = make_float2(m[x], L);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (__any(odd)) {
            put_odd(so);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        if (whole) {
            const int32_t rows = min(CW, seg.m * a.group - r0);
            for (int32_t x = lane; x < rows * (HD / 4); x += 64) {
                const int32_t r = x / (HD / 4), d = 4 * (x % (HD / 4));
                put_out(out_at(seg.first, kvh, r, d), *(const f32x4_t *)(so + r * LDW + d), ss[r].y);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        } else if (lane == 0) {
            piece_b[slot] = seg.b;
            piece_at[slot] = begin - from;
        }
    };

    // ---- the pipeline: page ids two tiles ahead, K and V one ----
    // The loads of the next tile are issued whether there is one or not (behind the last tile they read the
    // pool's first page): a load under a condition would make every later wait a wait for all.
    constexpr int STEP = LOCAL ? NW : 1;                   // whole sequences: every NW-th tile
    int32_t i = begin + (LOCAL ? wave : 0);                // tile of the range
    TreePos p0 = seg, p1, p2;
    if constexpr (LOCAL) p0.j = wave;
    int32_t kid, vid;
    uint32_t ku, vu;
    uint64_t there;
    load_ids(p0, &kid, &vid);
    load_q(p0);
    load_mask(p0);
    reset();
    p1 = p0;
    if (i + STEP < count) p1 = tree_next<TT>(a, tr, r0, p0, STEP);
    there = to_units(p0, kid, vid, &ku, &vu);
    load_ids(p1, &kid, &vid);
    __builtin_amdgcn_sched_barrier(0);                     // loads in the order in which they are waited for
    load_k(i < count ? ku : 0u);
    __builtin_amdgcn_sched_barrier(0);
    load_v(V0, i < count ? vu : 0u);
    auto step = [&](u32x4_t (&V)[NV][VC], u32x4_t (&Vn)[NV][VC]) {
        // logits: rows are tokens, columns the query rows
        f32x4_t S[NB][NS];
#pragma unroll
        for (int x = 0; x < NB; ++x)
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                S[x][s] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    if constexpr (BF) {
                        S[x][s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, K[s][k]),
                                                                          __builtin_bit_cast(bf16x8_t, Q[x][k]), S[x][s], 0, 0, 0);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            S[x][s] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(K[s][k][e]), __uint_as_float(Q[x][k][e]), S[x][s], 0, 0, 0);
                    }
                }
            }
        __builtin_amdgcn_sched_barrier(0);
        const bool more = i + STEP < count;
        const int32_t s0 = p0.j * TT - (p0.n - p0.m);      // the tile's first token as a node; below 0: cached before
        uint32_t sees[NB];
#pragma unroll
        for (int x = 0; x < NB; ++x) sees[x] = (uint32_t)(mask_window(tr, s0, mlo[x], mhi[x]) & there);
        if (more && p1.b != p0.b) load_q(p1);
        uint32_t ku1, vu1;
        const uint64_t there1 = to_units(p1, kid, vid, &ku1, &vu1);
        p2 = p1;
        if (i + 2 * STEP < count) p2 = tree_next<TT>(a, tr, r0, p1, STEP);
        load_ids(p2, &kid, &vid);
        load_mask(p1);
        __builtin_amdgcn_sched_barrier(0);
        load_k(more ? ku1 : 0u);
        __builtin_amdgcn_sched_barrier(0);
        if (C::AHEAD) load_v(Vn, more ? vu1 : 0u);
        __builtin_amdgcn_sched_barrier(0);
        const bool nodes = s0 + TT > 0;
        const bool full = (~there & ((1ull << TT) - 1)) == 0;
        if (!full) {                                       // what lies where no token is must not reach the products
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (!((there >> v_token(j)) & 1))
#pragma unroll
                    for (int c = 0; c < VC; ++c) V[j][c] = u32x4_t{0, 0, 0, 0};
        }
        if (nodes) {                                       // infinities and NaN of nodes: not by the products
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (s0 + v_token(j) >= 0)
#pragma unroll
                    for (int c = 0; c < VC; ++c)
#pragma unroll
                        for (int y = 0; y < (BF && HD == 64 ? 2 : 4); ++y) {
                            const uint32_t w = V[j][c][y];
                            const uint32_t out = not_finite<E>(w);
                            if (out) odd = true;
                            V[j][c][y] = w ^ out;
                        }
        }
        // weights; statistics of this lane's rows: the four lane groups hold different tokens
#pragma unroll
        for (int x = 0; x < NB; ++x) {
            float mt = -INFINITY;
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float y = S[x][s][r] * scale2;
                    if ((nodes || !full) && !(sees[x] >> (16 * s + 4 * g + r) & 1)) y = -INFINITY;
                    S[x][s][r] = y;
                    mt = fmaxf(mt, y);
                }
            mt = fmaxf(mt, __shfl_xor(mt, 16, 64));
            mt = fmaxf(mt, __shfl_xor(mt, 32, 64));
            const float mn = fmaxf(m[x], mt), ms = mn == -INFINITY ? 0.f : mn;
            const float c = exp2_hw(m[x] - ms);
            m[x] = mn;
            float ps = 0.f;
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    S[x][s][r] = exp2_hw(S[x][s][r] - ms);
                    ps += S[x][s][r];
                }
            l[x] = l[x] * c + ps;
#pragma unroll
            for (int y = 0; y < NA; ++y) acc[x][y] *= c;
        }
        // out^T += V^T P^T: rows are dims, columns the query rows
        if constexpr (BF) {
#pragma unroll
            for (int q = 0; q < TT / 32; ++q) {
                u32x4_t hi[NB], lo[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint2 w = split2(S[b][2 * q + x / 2][2 * (x & 1)], S[b][2 * q + x / 2][2 * (x & 1) + 1]);
                        hi[b][x] = w.x;
                        lo[b][x] = w.y;
                    }
                constexpr int WV = HD == 64 ? 4 : 8;
#pragma unroll
                for (int c = 0; c < VC; ++c)
#pragma unroll
                    for (int x = 0; x < WV; ++x) {
                        u32x4_t f;
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            f[y] = __builtin_amdgcn_perm(V[8 * q + 2 * y + 1][c][x / 2], V[8 * q + 2 * y][c][x / 2],
                                                         x & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            acc[b][WV * c + x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(bf16x8_t, f), __builtin_bit_cast(bf16x8_t, lo[b]), acc[b][WV * c + x], 0, 0, 0);
                            acc[b][WV * c + x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(bf16x8_t, f), __builtin_bit_cast(bf16x8_t, hi[b]), acc[b][WV * c + x], 0, 0, 0);
                        }
                    }
            }
        } else {
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int c = 0; c < VC; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int b = 0; b < NB; ++b)
                                acc[b][4 * c + e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(V[4 * s + r][c][e]), S[b][s][r],
                                                                                        acc[b][4 * c + e], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (!C::AHEAD) load_v(V, more ? vu1 : 0u);
        p0 = p1;
        p1 = p2;
        there = there1;
        i += STEP;
        if (i >= end) {
            flush();
            if (i < count) {
                first_piece = false;
                reset();
                begin = i;
                seg = p0;
                from = 0;
                end = min(count, begin + seg.tiles);
            }
        }
    };
    while (i < count) {
        step(V0, V1);
        if (C::AHEAD && i < count) step(V1, V0);
    }
    if (bad) record(a, bad);
    // ---- the waves' sums of the sequence, or of those that no wave saw whole, put together ----
    __syncthreads();
    const int32_t mine = lane < NW * SLOTS ? piece_b[lane] : -1;
    auto held = [&](int32_t y) { return __builtin_amdgcn_readlane(mine, y); };   // the sequence of piece y, or -1
    auto join = [&](int32_t x, int32_t b, int32_t y0, int32_t y1, int32_t by, f32x4_t *v, float *sum) {   // of y0, y0 + by, ... < y1
        const int32_t r = x / (HD / 4), d = 4 * (x % (HD / 4));
        float M = -INFINITY;
        for (int32_t y = y0; y < y1; y += by)
            if (held(y) == b) M = fmaxf(M, sh_s[y * CW + r].x);
        const float Ms = M == -INFINITY ? 0.f : M;
        *sum = 0.f;
        *v = f32x4_t{0.f, 0.f, 0.f, 0.f};
        for (int32_t y = y0; y < y1; y += by)
            if (held(y) == b) {
                const float2 ml = sh_s[y * CW + r];
                const float f = exp2_hw(ml.x - Ms);
                *sum += ml.y * f;
                // (a wave that saw none of the row's tokens holds zeros, or infinities of nodes whose weights are zero)
                *v += *(const f32x4_t *)(sh_o + (y * CW + r) * LDW + d) * f;
            }
        return M;
    };
    f32x4_t v;
    float sum;
    if constexpr (LOCAL) {
        const int32_t rows = min(CW, seg.m * a.group - r0);
        for (int32_t x = tid; x < rows * (HD / 4); x += THREADS) {
            join(x, seg.b, 0, NW, 1, &v, &sum);
            put_out(out_at(seg.first, kvh, x / (HD / 4), 4 * (x % (HD / 4))), v, sum);
        }
        return;
    }
    // A sequence is put together by the wave that holds its first piece; the others lie in the first slots of its head's next
    // waves (some of which may have no piece: no tiles, or whole sequences alone).
    for (int s = 0; s < SLOTS; ++s) {
        const int32_t y0 = wave * SLOTS + s, b = held(y0);
        if (b < 0) continue;
        if (s == 0) {                                      // not the first, if a wave before ended inside the sequence
            int32_t w = wave - hw;
            while (w >= 0 && held(w * SLOTS) < 0 && held(w * SLOTS + 1) < 0) w -= hw;
            if (w >= 0 && (held(w * SLOTS) == b || held(w * SLOTS + 1) == b)) continue;
        }
        const int32_t at0 = uniform(piece_at[y0]);
        const SeqRows sq = tree_rows_scalar(a, tr, b);
        const int32_t rows = min(CW, sq.m * a.group - r0), tiles = tree_tiles<TT>(a, sq, r0);
        const bool whole = at0 >= 0 && at0 + tiles <= total;
        const int64_t piece = (((int64_t)range * 2 + (b == range_b ? 0 : 1)) * a.n_kv + kvh) * tr.rows_ld + r0;
        for (int32_t x = lane; x < rows * (HD / 4); x += 64) {
            const int32_t r = x / (HD / 4), d = 4 * (x % (HD / 4));
            f32x4_t v1;
            float sum1;
            const float M1 = join(x, b, (wave + hw) * SLOTS, NW * SLOTS, hw * SLOTS, &v1, &sum1);
            const float2 ml = sh_s[y0 * CW + r];
            const float M = fmaxf(M1, ml.x), Ms = M == -INFINITY ? 0.f : M, f = exp2_hw(ml.x - Ms), f1 = exp2_hw(M1 - Ms);
            sum = ml.y * f + sum1 * f1;
            v = *(const f32x4_t *)(sh_o + (y0 * CW + r) * LDW + d) * f + v1 * f1;
            if (whole) {
                put_out(out_at(sq.first, kvh, r, d), v, sum);
            } else {
                if (d == 0) tr.part_ml[piece + r] = make_float2(M, sum);
                *(f32x4_t *)(tr.part_o + (piece + r) * HD + d) = v;
            }
        }
    }
}

// Put the pieces of a sequence (blockIdx.y) together: out = sum 2^(m_s - M) o_s / sum 2^(m_s - M) l_s.  A thread takes
// four dims of a row; G groups of threads take every G-th piece of the same row each, and are joined in LDS: where a sequence has
// many pieces, a row's thread would read them one behind the other (one sequence in 32 pieces, 16 rows of 32 heads: 15.4 us).
// blockIdx.x: a K/V head and some of its rows, which lie in one block of CW.  blockIdx.y: a sequence, or, where the sequences are
// more than the places between two ranges, one of those: the first that lies inside the sequence.
template <int HD> constexpr int join_slots() { return 1024 / HD; }   // rows that 256 threads take
template <typename E, int HD, int G>
__global__ __launch_bounds__(256) void k_kv_tree_join(KvArgs a, KvAttend at, KvTreeSplit tr, int32_t tt_log, int32_t cw, int by_range) {
    constexpr int ROWS = join_slots<HD>() / G;
    __shared__ int64_t sh[4], sh_before;
    __shared__ int32_t sh_seq;
    __shared__ float2 sh_ml[G > 1 ? 256 : 1];
    __shared__ f32x4_t sh_v[G > 1 ? 256 : 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int32_t kvh = blockIdx.x % a.n_kv, first = blockIdx.x / a.n_kv * ROWS, r0 = first / cw * cw;
    const int32_t per = (a.n_seq + 255) / 256, f0 = min(a.n_seq, tid * per), f1 = min(a.n_seq, f0 + per);
    auto tiles_of = [&](const SeqRows &s) { return s.m * a.group > r0 ? (s.n + (1 << tt_log) - 1) >> tt_log : 0; };
    int64_t before = 0, total = 0;
    for (int32_t b = f0; b < f1; ++b) before += tiles_of(tree_rows(a, tr, b));
    int64_t incl = before;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t y = __shfl_up(incl, o, 64);
        if (lane >= o) incl += y;
    }
    if (lane == 63) sh[wave] = incl;
    if (tid == 0) sh_seq = -1;
    __syncthreads();
    before = incl - before;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        before += i < wave ? sh[i] : 0;
        total += sh[i];
    }
    const Ranges rg = ranges_of(total, tr.R);
    // the sequence, by the thread that has it, if more than one range has a piece of it
    const int64_t place = by_range && (int32_t)blockIdx.y + 1 < rg.R ? rg.start(blockIdx.y + 1) : -1;
    for (int32_t b = f0; b < f1; ++b) {
        const int32_t t = tiles_of(tree_rows(a, tr, b));
        if (by_range ? place > before && place < before + t && rg.start(blockIdx.y) <= before : b == (int32_t)blockIdx.y && t > 0) {
            sh_seq = b;
            sh_before = before;
        }
        before += t;
    }
    __syncthreads();
    const int32_t b = uniform(sh_seq);
    if (b < 0) return;
    const SeqRows sq = tree_rows_scalar(a, tr, b);
    const int32_t rows = sq.m * a.group, nt = tiles_of(sq);
    const Pieces p = pieces_of(sh_before, sh_before + nt, rg);
    if (first >= rows || p.r0 == p.r1) return;             // one range saw it whole
    const int32_t r = first + tid / (HD / 4) % ROWS, d = 4 * (tid % (HD / 4)), g = tid / (HD / 4) / ROWS;
    float m = -INFINITY, l = 0.f;
    f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto add = [&](float2 ml, f32x4_t v) {
        const float mn = fmaxf(m, ml.x), ms = mn == -INFINITY ? 0.f : mn;
        const float c = exp2_hw(m - ms), w = exp2_hw(ml.x - ms);
        l = l * c + ml.y * w;
        acc = acc * c + v * w;
        m = mn;
    };
    if (r < rows)
        for (int32_t s = p.r0 + g; s <= p.r1; s += 8 * G) {   // eight loads at once
            float2 ml[8];
            f32x4_t v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int32_t su = min(s + u * G, p.r1);
                const int64_t pl = (((int64_t)su * 2 + (su == p.r0 ? p.s0 : 0)) * a.n_kv + kvh) * tr.rows_ld + r;
                ml[u] = tr.part_ml[pl];
                v[u] = *(const f32x4_t *)(tr.part_o + pl * HD + d);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (s + u * G > p.r1) break;
                add(ml[u], v[u]);
            }
        }
    if constexpr (G > 1) {
        sh_ml[tid] = make_float2(m, l);
        sh_v[tid] = acc;
        __syncthreads();
        if (g > 0) return;
#pragma unroll
        for (int u = 1; u < G; ++u) add(sh_ml[tid + u * ROWS * (HD / 4)], sh_v[tid + u * ROWS * (HD / 4)]);
    }
    if (r >= rows) return;
    const int32_t node = node_of(a, tr, r);
    E *o = (E *)at.out + (int64_t)(sq.first + node) * at.ldo + (int64_t)(kvh * a.group + r - node * a.group) * HD + d;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (l == 0.f) acc = f32x4_t{0.f, 0.f, 0.f, 0.f};       // no weight: zero, also where a value is not finite
    if constexpr (sizeof(E) == 2) *(uint2 *)o = make_uint2(pack2(acc[0] * inv, acc[1] * inv), pack2(acc[2] * inv, acc[3] * inv));
    else *(f32x4_t *)o = acc * inv;
}

// ---- host ----------------------------------------------------------------------------------------
namespace {

struct TreePlan {
    int32_t nb, cw, ncb, R, tt, hw;   // nb: blocks of 16 rows; 0: the kernel for many rows
    bool local;
    size_t off_ml, total;
};
TreePlan tree_plan(int dtype, int n_heads, int n_kv, int hd, int32_t n_seq, int32_t max_nodes, int64_t max_len) {
    TreePlan p;
    const int group = n_heads / n_kv;
    const int64_t rows = (int64_t)max_nodes * group;
    const int64_t blocks = (rows + WIDE_ROWS - 1) / WIDE_ROWS;
    // Up to 16 rows in one block of the kernel for few rows, float32 up to 32 in two: bfloat16 of 32 rows took 172 us so, by the
    // other kernel 139, with weights of one number then (float32, 32 trees of 32 nodes, 16 heads of 64 behind up to 500 tokens: 41 and 53).
    p.nb = rows <= 16 ? 1 : rows <= 32 && hd < 256 && dtype == LORA_F32 ? 2 : 0;
    // Whole sequences, one workgroup each of a head and block of rows, need no pieces and no second launch, but their longest has
    // to be a small part of a workgroup's share.  `whole` workgroups against ranges, us:
    //   few rows, one a CU: 32 of 1000 tokens 18 and 21.5, of 2000 29 and 22.6; 256 of 1900 51 and 60; 512 of up to 500 25 and 32,
    //   of up to 2000 86 and 80; 1024 of up to 500 54.5 and 53; 2048 of up to 1031 150 and 135
    //   many rows, two a CU: 8 of 500 24 and 16; 64 of 500 24 and 22 (heads of 256: 44.5 and 39); 128 of up to 1000 40.5 and 34;
    //   256 of up to 1000 43 and 43, of up to 2000 76 and 60; 512 of up to 2000 101 and 103 (32 heads on 8: 119 and 124); 2048 of up
    //   to 300 72 and 95, of up to 1000 159 and 186; 1024 of up to 4000 289 and 289
    //   many rows, float32: 32 of 500 47 and 23; 512 of 190 38 and 43, of up to 500 77 and 71
    const int64_t whole = (int64_t)n_seq * n_kv * (p.nb ? 1 : blocks);
    if (p.nb) p.local = whole <= 512 && max_len <= (whole >= 128 && whole <= 256 ? 2048 : 1024);
    else if (dtype == LORA_F32) p.local = max_len <= std::max<int64_t>(64, std::min<int64_t>(2048, whole / 2));
    else p.local = max_len <= std::max<int64_t>(whole >= 64 && hd < 256 ? 512 : 256, std::min<int64_t>(2048, 4 * whole));
    // No workspace: where every smaller call takes its sequences whole too, so that what serves a larger call serves it.
    const bool none = whole <= 512 && max_len <= (p.nb ? 1024 : dtype == LORA_F32 ? 64 : 256);
    // Neighbouring heads a workgroup: four of the kernel for few rows (64 trees of 16 nodes, 32 heads, in ranges: 8, 4, 2, 1 of them
    // 140, 138, 140, 149).  Two of the kernel for many rows where 64 are enough and the call keeps every workgroup busy for several
    // steps: in ranges (16 trees of 32 nodes, 32 heads, behind up to 2000 tokens: 87, one head each 90; 64 of 16, 16 heads of 256 on
    // 4, behind up to 1000 72 and 77, but 8 of 16, 32 heads on 8, behind up to 9000 72 and 65; one tree of 16, 32 heads on 8, behind
    // 1000: 19 and 14.5), and whole where two a CU are left (1024 whole of up to 500 tokens 57, one head each 68; 512 of up to 2000
    // 106 and 104, of 32 nodes 103 and 89).
    const bool two = rows <= WIDE_ROWS / 2 && n_kv % 2 == 0 && dtype != LORA_F32 && (p.local ? whole >= 1024 : (max_len + 63) / 64 * n_seq * n_kv >= 4 * 512);
    p.hw = p.nb ? (n_kv % 4 == 0 ? 4 : n_kv % 2 == 0 ? 2 : 1) : two ? 2 : 1;
    p.cw = p.nb ? 16 * p.nb : WIDE_ROWS / p.hw;
    p.tt = p.nb ? (dtype == LORA_F32 && hd > 64 ? 16 : 32) : (dtype == LORA_F32 ? 32 : 64) / p.hw;
    const int64_t tiles = (max_len + p.tt - 1) / p.tt * n_seq;
    p.ncb = (int32_t)((rows + p.cw - 1) / p.cw);
    const int64_t hu = (int64_t)n_kv * p.ncb, slots = p.nb || hd == 256 ? 256 : 512;
    // A workgroup a CU, two of the kernel for many rows; but ranges of four tiles at least, where that leaves 64 (one
    // sequence of 20000 tokens, 8 heads on one, 16 nodes: 24.7 us, without the limit 38.6; of 6000, 32 heads on 8, 4 nodes 24.6 and 27.8).
    p.R = (int32_t)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(tiles, std::max<int64_t>(64, tiles / 4)), slots * p.hw / hu));
    // Room for at least `slots` workgroups' pieces, so that what serves the largest call serves them all: the ranges of more rows
    // are fewer.  For many rows by blocks and steps of one head a workgroup, which two heads need no more than: the sizes for which
    // `two` holds begin anywhere.
    const int64_t cw = p.nb ? p.cw : WIDE_ROWS, step = p.tt * (p.nb ? 1 : p.hw), block_rows = (int64_t)n_kv * ((rows + cw - 1) / cw) * cw;
    const size_t pieces = 2 * (size_t)std::min<int64_t>((max_len + step - 1) / step * n_seq * block_rows,
                                                        std::max<int64_t>(slots * p.hw * p.cw, block_rows));
    p.off_ml = (pieces * hd * 4 + 255) & ~size_t(255);
    p.total = none ? 0 : p.off_ml + ((pieces * 8 + 255) & ~size_t(255));
    return p;
}

template <typename E, int HD, int NB>
hipError_t few(const KvArgs &a, const KvAttend &at, const KvTreeSplit &tr, bool local, hipStream_t s) {
    using C = TreeTile<E, HD, NB>;
    const unsigned hu = (unsigned)(a.n_kv * tr.ncb);
    auto launch = [&](auto kernel, dim3 grid) {
        const int lds = (local ? 1 : 2) * C::LDS;
        if (lds > 64 * 1024) {                             // has to be asked for, on each device
            const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL(kernel, grid, dim3(64 * C::NW), lds, s, a, at, tr);
        return hipGetLastError();
    };
    return local ? launch(k_kv_tree<E, HD, NB, true>, dim3(hu, (unsigned)a.n_seq)) : launch(k_kv_tree<E, HD, NB, false>, dim3(hu / tr.hw * tr.R));
}

template <typename E, int HD>
hipError_t run(int dtype, const KvArgs &a, const KvAttend &at, const KvTreeArgs &ta, hipStream_t s) {
    const TreePlan pl = tree_plan(dtype, a.n_heads, a.n_kv, HD, a.n_seq, ta.max_nodes, a.cap);
    KvTreeSplit tr{};
    tr.R = pl.R;
    tr.hw = pl.hw;
    tr.ncb = pl.ncb;
    tr.rows_ld = pl.ncb * pl.cw;
    tr.max_nodes = ta.max_nodes;
    tr.words = (ta.max_nodes + 63) / 64;
    tr.group_magic = a.group == 1 ? 0 : (uint32_t)(((uint64_t(1) << 32) + a.group - 1) / a.group);
    tr.mask = ta.mask;
    tr.part_o = (float *)at.ws;
    tr.part_ml = (float2 *)((char *)at.ws + pl.off_ml);
    hipError_t e = hipErrorInvalidValue;
    if (pl.nb == 0) e = launch_tree_wide(dtype, a, at, tr, pl.local, s);
    else if (pl.nb == 1) e = few<E, HD, 1>(a, at, tr, pl.local, s);
    else if constexpr (HD < 256 && sizeof(E) == 4) e = few<E, HD, 2>(a, at, tr, pl.local, s);
    if (e != hipSuccess || pl.local) return e;
    // All threads of a workgroup to one row where a sequence is in more than eight pieces on average (one of 30000 tokens, 8 heads,
    // 4 nodes: 43 us, by one thread 83; 8 of 1000, 32 nodes, in four pieces each: 42 and 29.7).
    constexpr int SLOTS = join_slots<HD>();
    if (pl.R == 1) return e;                               // one range sees every sequence whole
    const int64_t rows = (int64_t)ta.max_nodes * a.group;
    const int by_range = pl.R - 1 < a.n_seq, tt_log = __builtin_ctz(pl.tt);
    const unsigned y = (unsigned)(by_range ? pl.R - 1 : a.n_seq);
    if (pl.R > 8 * a.n_seq)
        hipLaunchKernelGGL((k_kv_tree_join<E, HD, SLOTS>), dim3((unsigned)(rows * a.n_kv), y), dim3(256), 0, s, a, at, tr, tt_log, pl.cw, by_range);
    else
        hipLaunchKernelGGL((k_kv_tree_join<E, HD, 1>), dim3((unsigned)((rows + SLOTS - 1) / SLOTS * a.n_kv), y), dim3(256), 0, s, a, at, tr, tt_log,
                           pl.cw, by_range);
    return hipGetLastError();
}

template <typename E>
hipError_t by_dim(int dtype, const KvArgs &a, const KvAttend &at, const KvTreeArgs &ta, hipStream_t s) {
    return a.head_dim == 64 ? run<E, 64>(dtype, a, at, ta, s) : a.head_dim == 128 ? run<E, 128>(dtype, a, at, ta, s)
                                                                                  : run<E, 256>(dtype, a, at, ta, s);
}

}  // namespace

size_t kv_tree_ws_bytes(int dtype, const lora_kv_layout_t &l, int32_t n_seq, int32_t max_nodes, int64_t max_len) {
    return tree_plan(dtype, l.n_heads, l.n_kv_heads, l.head_dim, n_seq, max_nodes, max_len).total;
}

hipError_t launch_kv_tree(int dtype, const KvArgs &a, const KvAttend &at, const KvTreeArgs &ta, hipStream_t s) {
    return dtype == LORA_F32 ? by_dim<float>(dtype, a, at, ta, s) : by_dim<uint16_t>(dtype, a, at, ta, s);
}

}  // namespace lorapool

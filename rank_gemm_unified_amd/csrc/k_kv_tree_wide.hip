// Attention of trees of new tokens where a K/V head has many rows (k_kv_tree.hip has the formulas and the few rows).
//
// A hundred operations a byte and more: the matrix units and HBM are both near their limits.  One workgroup takes 128 rows
// of one K/V head, 32 a wave, and one of the equal ranges of all sequences' steps of NT tokens.  K and V go from their
// pages straight to LDS (16 bytes a lane, gathered row by row, the next step's while this one's are used); a wave's rows
// stay in registers, as columns:
//     S^T = K Q^T   (rows tokens, columns query rows)       out^T += V^T P^T   (rows dims)
// so that the weights are in place as the right operand of the second product, bfloat16 ones as two numbers (split2), as for the few
// rows: what a row comes out as does not hang on how many rows the call may have.  Rounded to one number they would be off by
// 2^-8 of themselves, and the call would take 185 us instead of 208 below, 97 instead of 105 for 16 trees of 64 nodes behind up to
// 2000 tokens and 32 heads, 90 instead of 92 for 32 nodes, 103 instead of 121 for 64 of 32 nodes, 32 heads on 8.  Two workgroups
// a CU: one's softmax runs under the other's products and loads (one a CU with four stages in LDS took half as long again).
// 8 trees of 32 nodes behind up to 32768 tokens, 32 heads of 128 on 8: 192 to 210 us on several cards for 750 MB (3.6 to
// 3.9 TB/s) and 125 Gflop of products (102 us at the rate of a large one); in a trace 192 of 209 in here, 14 in the pieces' join.  The
// loads alone took 150 on a card where the call with one number took 185.
#include "kv_tile.h"
#include "kv_tree.h"

namespace lorapool {

// LOCAL: one whole sequence (blockIdx.y), no pieces.  HEADS: two neighbouring heads share the workgroup where 64 rows are enough
// for each: two waves a head, steps of half the tokens, and pieces of the pages twice as long that are read at one time.
template <typename E, int HD, int HEADS, bool LOCAL>
__global__ __launch_bounds__(256, (Chunk<E, HD>::WAVES)) void k_kv_tree_wide(KvArgs a, KvAttend at, KvTreeSplit tr) {
    using C = Chunk<E, HD>;
    constexpr int TILE = C::NT, NT = TILE / HEADS, NB = NT / 32;   // rows of a tile in LDS, head by head; tokens of a step
    constexpr int RB = C::RB, CH = C::CH, KQ = C::KQ, ND = HD / 32, WPH = 4 / HEADS, ROWS = 32 * WPH;
    constexpr bool BF = C::BF;
    extern __shared__ __align__(256) char smem[];
    __shared__ unsigned long long sh_flag;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), col = lane & 31, hh = lane >> 5;
    const int32_t head0 = blockIdx.x % (a.n_kv / HEADS) * HEADS, rest = blockIdx.x / (a.n_kv / HEADS), mine = wave / WPH, kvh = head0 + mine;
    const int32_t r0 = rest % tr.ncb * ROWS, rw = r0 + 32 * (wave % WPH), range = rest / tr.ncb;   // rw: the wave's first row
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        int bits = 0;
        for (int32_t b = tid; b < a.n_seq; b += 256) bits |= tree_rows(a, tr, b).err;
        record(a, bits);
    }
    __shared__ TreeBegin w;
    int32_t count, from = 0, b0 = blockIdx.y;
    if constexpr (LOCAL) {
        count = tree_tiles<NT>(a, tree_rows(a, tr, b0), r0);
    } else {
        count = tree_begin<E, NT, 256>(a, at, tr, r0, ROWS, head0, HEADS, range, 1, &w);
        if (count == 0) return;
        b0 = uniform(w.b);
        from = uniform(w.j);
    }
    TreePos seg = tree_pos<NT>(a, tr, r0, b0, from);
    if (LOCAL && r0 >= seg.m * a.group) return;
    int32_t begin = 0, end = min(count, seg.tiles - from);
    bool first_piece = true;

    const char *base = a.pages + (int64_t)head0 * RB;
    const uint32_t page_units = (uint32_t)(a.page_bytes >> 7), tok_units = (uint32_t)(a.tok_bytes >> 7);
    const float scale2 = at.scale * 1.4426950408889634f;
    const int32_t r = rw + col;                // this lane's row
    int bad = 0;
    // LDS as it stands for every wave; loads that are on their way to it are not waited for
    auto meet = [] {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    auto load_ids = [&](const TreePos &p, int32_t *kid, int32_t *vid) {
        const int32_t t = p.j * NT + (lane & (NT - 1));
        int32_t e, slot;
        page_of(a, t, &e, &slot);
        const int32_t *row = a.table + (int64_t)p.b * 2 * a.max_pages + (t < p.n ? e : 0);   // (there is a first entry)
        *kid = row[0];
        *vid = row[a.max_pages];
    };
    auto to_units = [&](const TreePos &p, int32_t kid, int32_t vid, uint32_t *ku, uint32_t *vu) -> uint64_t {
        const int32_t t = p.j * NT + (lane & (NT - 1));
        int32_t e, slot;
        page_of(a, t, &e, &slot);
        const bool ok = t < p.n && kid >= 0 && vid >= 0 && kid < a.num_pages && vid < a.num_pages;
        if (t < p.n && !ok) bad = DEV_ERR_PAGE;
        *ku = ok ? (uint32_t)kid * page_units + (uint32_t)slot * tok_units : 0u;
        *vu = ok ? (uint32_t)vid * page_units + (uint32_t)slot * tok_units : 0u;
        return __ballot(ok) & (NT == 64 ? ~0ull : 0xffffffffull);
    };
    auto fetch = [&](int32_t buf, uint32_t ku, uint32_t vu) {
        char *kb = smem + buf * C::BUF, *vb = smem + (2 + buf) * C::BUF;
#pragma unroll
        for (int x = 0; x < C::PER; ++x) {
            const int at0 = (wave * C::PER + x) * 1024, byte = at0 + lane * 16, t = byte / RB, c = (byte % RB) / 16;
            const uint32_t k = __shfl(ku, t % NT, 64), v = __shfl(vu, t % NT, 64);
            const char *of = base + t / NT * RB;
            lds_gload16(of + ((uint64_t)k << 7) + 16 * C::k_swz(t, c), (lds_void *)(kb + at0));
            lds_gload16(of + ((uint64_t)v << 7) + 16 * C::v_swz(t, c), (lds_void *)(vb + at0));
        }
    };
    auto row_of = [&](const TreePos &p) { return p.first + node_of(a, tr, r < p.m * a.group ? r : r0); };
    auto head_of = [&](const TreePos &p) {                 // rows behind the last take the block's first
        const int32_t x = r < p.m * a.group ? r : r0;
        return kvh * a.group + x - node_of(a, tr, x) * a.group;
    };
    u32x4_t Q[KQ];
    auto load_q = [&](const TreePos &p) {
        const char *q = (const char *)((const E *)at.q + (int64_t)row_of(p) * at.ldq + (int64_t)head_of(p) * HD) + 16 * hh;
#pragma unroll
        for (int i = 0; i < KQ; ++i) Q[i] = load16(q + 32 * i);
    };
    auto other_half = [](float x) {                        // the value of the lane 32 further, or before
        const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        return __uint_as_float(threadIdx.x & 32 ? y[0] : y[1]);
    };
    f32x16_t acc[ND], S[NB];
    float m, l;
    auto reset = [&]() {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
        m = -INFINITY;
        l = 0.f;
    };
    // The rows' way out: divided, or as a piece.
    auto flush = [&]() {
        const float L = l + other_half(l);
        if (r >= seg.m * a.group) return;
        if (from == 0 && end - begin == seg.tiles) {
            const float inv = L == 0.f ? 0.f : 1.f / L;
            E *o = (E *)at.out + (int64_t)row_of(seg) * at.ldo + (int64_t)head_of(seg) * HD;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    f32x4_t v;
#pragma unroll
                    for (int y = 0; y < 4; ++y) v[y] = L == 0.f ? 0.f : acc[d][4 * x + y] * inv;   // no weight: zero
                    E *to = o + 32 * d + 8 * x + 4 * hh;
                    if constexpr (BF) *(uint2 *)to = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
                    else *(f32x4_t *)to = v;
                }
            return;
        }
        const int64_t piece = (((int64_t)range * 2 + (first_piece ? 0 : 1)) * a.n_kv + kvh) * tr.rows_ld + r;
        if (hh == 0) tr.part_ml[piece] = make_float2(m, L);
        float *o = tr.part_o + piece * HD;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *(f32x4_t *)(o + 32 * d + 8 * x + 4 * hh) = f32x4_t{acc[d][4 * x], acc[d][4 * x + 1], acc[d][4 * x + 2], acc[d][4 * x + 3]};
    };

    TreePos p0 = seg, p1 = seg, p2;
    int32_t kid, vid;
    uint32_t ku, vu;
    uint64_t there, mlo = 0, mhi = 0;
    reset();
    load_ids(p0, &kid, &vid);
    if (count > 1) p1 = tree_next<NT>(a, tr, r0, p0, 1);
    there = to_units(p0, kid, vid, &ku, &vu);
    load_ids(p1, &kid, &vid);
    load_q(seg);
    mask_at(tr, row_of(p0), p0.j * NT - (p0.n - p0.m), &mlo, &mhi);
    fetch(0, ku, vu);
    for (int32_t i = 0; i < count; ++i) {
        // this step's K and V are in; by a builtin, so that the compiler knows that what else was loaded is in too, and
        // does not wait for it once more behind the next step's loads
        __builtin_amdgcn_s_waitcnt(0x0070);                // vmcnt(0) lgkmcnt(0)
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        const int32_t s0 = p0.j * NT - (p0.n - p0.m);      // the step's first token as a node
        const bool nodes = s0 + NT > 0;
        const uint64_t sees = mask_window(tr, s0, mlo, mhi) & there;
        const uint64_t there1 = to_units(p1, kid, vid, &ku, &vu);
        const bool more = i + 1 < count;
        fetch(~i & 1, more ? ku : 0u, more ? vu : 0u);
        p2 = p1;
        if (i + 2 < count) p2 = tree_next<NT>(a, tr, r0, p1, 1);
        load_ids(p2, &kid, &vid);
        {
            const int32_t s1 = p1.j * NT - (p1.n - p1.m);
            if (s1 + NT > 0) mask_at(tr, row_of(p1), s1, &mlo, &mhi);
        }
        constexpr uint64_t ALL = NT == 64 ? ~0ull : 0xffffffffull;
        char *v_tile = smem + (2 + (i & 1)) * C::BUF;
        const char *kb = smem + (i & 1) * C::BUF + mine * (NT * RB), *vb = v_tile + mine * (NT * RB);   // this wave's head's
        if (there != ALL) {                                // rows of tokens that are not there must not reach the products
            for (int x = tid; x < TILE * CH; x += 256)
                if (!((there >> (x / CH % NT)) & 1)) store16(v_tile + 16 * x, u32x4_t{0, 0, 0, 0});
            meet();
        }
        if (nodes) {                                       // infinities and NaN of nodes: not by the products, but to the
            if (tid == 0) sh_flag = 0;                     // rows that see them
            meet();
            for (int x = tid; x < TILE * CH; x += 256) {
                const u32x4_t y = load16(v_tile + 16 * x);
                if (s0 + x / CH % NT >= 0 && (not_finite<E>(y[0]) | not_finite<E>(y[1]) | not_finite<E>(y[2]) | not_finite<E>(y[3])))
                    atomicOr(&sh_flag, 1ull << (x / CH));
            }
            meet();
            if (const unsigned long long flags = sh_flag) {
                for (unsigned long long f = flags; f; f &= f - 1) {
                    const int t = __ffsll((long long)f) - 1;
                    if (t / NT == mine && sees >> (t % NT) & 1) {
#pragma unroll
                        for (int d = 0; d < ND; ++d)
#pragma unroll
                            for (int x = 0; x < 16; ++x) {
                                const int byte = (32 * d + 8 * (x / 4) + 4 * hh + (x & 3)) * (int)sizeof(E);
                                const float y = to_f32(*(const E *)(v_tile + t * RB + 16 * C::v_swz(t, byte / 16) + byte % 16));
                                if (y - y != 0.f) acc[d][x] += y;
                            }
                    }
                }
                meet();
                for (int x = tid; x < TILE * CH; x += 256)
                    if (flags >> (x / CH) & 1) {
                        u32x4_t y = load16(v_tile + 16 * x);
#pragma unroll
                        for (int z = 0; z < 4; ++z) y[z] ^= not_finite<E>(y[z]);
                        store16(v_tile + 16 * x, y);
                    }
                meet();
            }
        }
        if (rw < seg.m * a.group) {                         // else the wave has no rows
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int x = 0; x < 16; ++x) S[nb][x] = 0.f;
#pragma unroll
            for (int k = 0; k < KQ; ++k)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const u32x4_t f = load16(kb + (32 * nb + col) * RB + 16 * C::k_swz(col, 2 * k + hh));
                    if constexpr (BF) {
                        S[nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, f), __builtin_bit_cast(bf16x8_t, Q[k]), S[nb], 0, 0, 0);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            S[nb] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(f[e]), __uint_as_float(Q[k][e]), S[nb], 0, 0, 0);
                    }
                }
            // K pieces come out of LDS three products ahead
            __builtin_amdgcn_sched_group_barrier(0x100, 3 * NB, 0);
#pragma unroll
            for (int k = 0; k < KQ; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x008, NB * (BF ? 1 : 4), 0);
                if (k + 3 < KQ) __builtin_amdgcn_sched_group_barrier(0x100, NB, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            float sc = scale2;
            if (!(scale2 > 0.f)) {                         // the largest logit need not be the largest product's
                sc = 1.f;
                float by = scale2;
                asm volatile("" : "+v"(by));               // keeps the products inside the branch
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int x = 0; x < 16; ++x) S[nb][x] *= by;
            }
            if (there != ALL || nodes) {                   // tokens counted from this lane half's first
                const uint64_t in = sees >> (4 * hh);
                const uint32_t in0 = (uint32_t)in, in1 = (uint32_t)(in >> 32);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const int t = 8 * (x / 4) + (x & 3);
                        if (!((nb ? in1 : in0) & (1u << t))) S[nb][x] = -INFINITY;
                    }
            }
            float mt = -INFINITY;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int x = 0; x < 16; ++x) mt = fmaxf(mt, S[nb][x]);
            mt = fmaxf(mt, other_half(mt)) * sc;
            if (__any(mt > m + 8.f)) {                     // (weights of up to 2^8 do no harm)
                const float mn = fmaxf(m, mt), ms = mn == -INFINITY ? 0.f : mn;
                // (before a row's first weight the accumulators hold zeros, or infinities of nodes)
                const float c = m == -INFINITY ? 1.f : exp2_hw(m - ms);
                m = mn;
                l *= c;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int x = 0; x < 16; ++x) acc[d][x] *= c;
            }
            __builtin_amdgcn_sched_barrier(0);
            const float ms = m == -INFINITY ? 0.f : m;
            float ps = 0.f;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    S[nb][x] = exp2_hw(S[nb][x] * sc - ms);
                    ps += S[nb][x];
                }
            l += ps;
            if constexpr (BF) {
                const int i16 = lane & 15;
                typedef short s16x8_t __attribute__((ext_vector_type(8)));
#pragma unroll
                for (int s = 0; s < NT / 16; ++s) {
                    u32x4_t hi, lo;                        // this lane's eight weights: tokens 16 s + 4 hh + 0..3 and 8 on
                    const int t = 16 * s + 4 * hh + (i16 >> 2);
                    s16x8_t v[ND];
#pragma unroll
                    for (int d = 0; d < ND; ++d) {
                        const int c = 4 * d + 2 * ((lane >> 4) & 1) + ((i16 & 3) >> 1);
                        const char *ad = vb + t * RB + 16 * C::v_swz(t, c) + 8 * (i16 & 1);
                        const s16x4_t v0 = read_tr((lds_s16x4 *)ad);
                        const s16x4_t v1 = read_tr((lds_s16x4 *)(ad + 8 * RB));
                        v[d] = s16x8_t{v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint2 w = split2(S[s / 2][8 * (s & 1) + 2 * x], S[s / 2][8 * (s & 1) + 2 * x + 1]);
                        hi[x] = w.x;
                        lo[x] = w.y;
                    }
#pragma unroll
                    for (int d = 0; d < ND; ++d)
                        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, v[d]),
                                                                         __builtin_bit_cast(bf16x8_t, hi), acc[d], 0, 0, 0);
#pragma unroll
                    for (int d = 0; d < ND; ++d)
                        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, v[d]),
                                                                         __builtin_bit_cast(bf16x8_t, lo), acc[d], 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const int t = 8 * (x / 4) + 4 * hh + (x & 3);
#pragma unroll
                    for (int d = 0; d < ND; ++d)
                        acc[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(*(const float *)(vb + t * RB + 4 * (32 * d + col)), S[0][x], acc[d], 0, 0, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (i + 1 == end && more) load_q(p1);              // the next sequence's
        p0 = p1;
        p1 = p2;
        there = there1;
        if (i + 1 == end) {
            flush();
            if (end < count) {
                first_piece = false;
                begin = end;
                seg = p0;
                from = 0;
                end = min(count, begin + seg.tiles);
                reset();
            }
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // no load is on its way to LDS any more
    if (LOCAL && count == 0) flush();                      // no tokens: zero rows
    if (bad) record(a, bad);
}

namespace {

template <typename E, int HD>
hipError_t run(const KvArgs &a, const KvAttend &at, const KvTreeSplit &tr, bool local, hipStream_t s) {
    constexpr int LDS = 4 * Chunk<E, HD>::BUF;
    auto launch = [&](auto kernel, dim3 grid) {
        if (LDS > 64 * 1024) {
            const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL(kernel, grid, dim3(256), LDS, s, a, at, tr);
        return hipGetLastError();
    };
    const unsigned hu = (unsigned)(a.n_kv / tr.hw * tr.ncb);
    if constexpr (sizeof(E) == 2)
        if (tr.hw == 2)
            return local ? launch(k_kv_tree_wide<E, HD, 2, true>, dim3(hu, (unsigned)a.n_seq)) : launch(k_kv_tree_wide<E, HD, 2, false>, dim3(hu * tr.R));
    if (local) return launch(k_kv_tree_wide<E, HD, 1, true>, dim3(hu, (unsigned)a.n_seq));
    return launch(k_kv_tree_wide<E, HD, 1, false>, dim3(hu * tr.R));
}

template <typename E>
hipError_t by_dim(const KvArgs &a, const KvAttend &at, const KvTreeSplit &tr, bool local, hipStream_t s) {
    return a.head_dim == 64 ? run<E, 64>(a, at, tr, local, s) : a.head_dim == 128 ? run<E, 128>(a, at, tr, local, s)
                                                                                  : run<E, 256>(a, at, tr, local, s);
}

}  // namespace

hipError_t launch_tree_wide(int dtype, const KvArgs &a, const KvAttend &at, const KvTreeSplit &tr, bool local, hipStream_t s) {
    return dtype == LORA_F32 ? by_dim<float>(a, at, tr, local, s) : by_dim<uint16_t>(a, at, tr, local, s);
}

}  // namespace lorapool

// What the kernels over trees of new tokens share: rows, the ranges of a block of rows, masks.
//
// The rows of a K/V head are its sequence's nodes times the query heads that share it, node by node: row r is head
// r % group of node r / group.  A workgroup takes one block of CW rows, and one range of the tiles (TT tokens) of all the
// sequences that have rows in that block.
#pragma once

#include "kv_ranges.h"

namespace lorapool {

struct KvTreeSplit {
    int32_t R;                // ranges of a block's tiles, at most
    int32_t hw;               // heads of a workgroup's waves
    int32_t ncb;              // blocks of CW rows of one K/V head
    int32_t rows_ld;          // rows of a piece: ncb * CW
    int32_t max_nodes, words; // 64-bit words of a row's mask
    uint32_t group_magic;     // ceil(2^32 / group): r / group = mulhi(r, magic) for r < 2^18, group in 2..1024
    const uint64_t *mask;     // [T][words]
    float *part_o;            // [R][2][n_kv][rows_ld][head_dim]: slot 0 a range's first piece, 1 its last
    float2 *part_ml;          // [R][2][n_kv][rows_ld]: maximum (base-2 logits), sum
};

// Sequence b's rows and length; more new tokens than a tree may have count as none.
__device__ __forceinline__ SeqRows tree_rows(const KvTreeSplit &tr, SeqRows s) {
    if (s.m > tr.max_nodes) {
        s.m = 0;
        s.err = DEV_ERR_LEN;
    }
    return s;
}
__device__ __forceinline__ SeqRows tree_rows(const KvArgs &a, const KvTreeSplit &tr, int32_t b) { return tree_rows(tr, seq_rows(a, b)); }

// The same for a sequence that is the same in every lane, by scalar loads: a vector load amid those of K and V would have
// to wait for all of them.
typedef const __attribute__((address_space(4))) int32_t *scalar_ptr;
__device__ __forceinline__ SeqRows tree_rows_scalar(const KvArgs &a, const KvTreeSplit &tr, int32_t b) {
    const scalar_ptr starts = (scalar_ptr)(uintptr_t)a.q_start, lens = (scalar_ptr)(uintptr_t)a.lens;
    return tree_rows(tr, seq_rows(a, starts[b], starts[b + 1], lens[b]));
}
// Tiles of a sequence in the block of rows that begins at row r0.
template <int TT>
__device__ __forceinline__ int32_t tree_tiles(const KvArgs &a, const SeqRows &s, int32_t r0) {
    return s.m * a.group > r0 ? (s.n + TT - 1) / TT : 0;
}

__device__ __forceinline__ int32_t node_of(const KvArgs &a, const KvTreeSplit &tr, int32_t r) {
    return a.group == 1 ? r : (int32_t)__umulhi((uint32_t)r, tr.group_magic);
}

// Zero rows of a sequence without tokens, by one thread: nothing else comes by (a program's step has few, if any).
template <typename E>
__device__ __forceinline__ void zero_rows(const KvArgs &a, const KvAttend &at, const KvTreeSplit &tr, const SeqRows &s, int32_t r0, int32_t cw,
                                          int32_t head0, int32_t heads) {
    for (int32_t r = r0; r < min(r0 + cw, s.m * a.group); ++r) {
        const int32_t node = node_of(a, tr, r);
        for (int32_t h = head0; h < head0 + heads; ++h) {
            E *o = (E *)at.out + (int64_t)(s.first + node) * at.ldo + (int64_t)(h * a.group + r - node * a.group) * a.head_dim;
            for (int32_t d = 0; d < a.head_dim; d += 16 / (int)sizeof(E)) store16(o + d, u32x4_t{0, 0, 0, 0});
        }
    }
}

// Where `n` equal parts of a range begin: sequence and tile of it.  Returns the range's tiles (0: there is no such range).
// The first range's workgroups also write the rows of sequences without tokens.  All threads call.
struct TreeBegin { int32_t b, j; };
__device__ __forceinline__ int32_t part_of(int32_t count, int32_t i, int32_t n) { return (int32_t)(((int64_t)count * i) / n); }
template <typename E, int TT, int THREADS>
__device__ __forceinline__ int32_t tree_begin(const KvArgs &a, const KvAttend &att, const KvTreeSplit &tr, int32_t r0, int32_t cw, int32_t head0,
                                              int32_t heads, int32_t range, int32_t n, TreeBegin *at) {
    __shared__ int64_t sum[THREADS / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t per = (a.n_seq + THREADS - 1) / THREADS, f0 = min(a.n_seq, tid * per), f1 = min(a.n_seq, f0 + per);
    int64_t mine = 0;
    for (int32_t b = f0; b < f1; ++b) {
        const SeqRows s = tree_rows(a, tr, b);
        mine += tree_tiles<TT>(a, s, r0);
        if (range == 0 && s.n == 0 && s.m > 0) zero_rows<E>(a, att, tr, s, r0, cw, head0, heads);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t x = __shfl_up(incl, o, 64);
        if (lane >= o) incl += x;
    }
    if (lane == 63) sum[wave] = incl;
    __syncthreads();
    int64_t excl = incl - mine, total = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) {
        excl += i < wave ? sum[i] : 0;
        total += sum[i];
    }
    const Ranges rg = ranges_of(total, tr.R);
    if (range >= rg.R) return 0;
    const int64_t s = rg.start(range);
    const int32_t count = uniform((int32_t)(rg.start(range + 1) - s));
    for (int32_t i = 0; i < n; ++i) {
        const int64_t x = s + part_of(count, i, n);        // (inside the range: i < n)
        if (mine > 0 && x >= excl && x < excl + mine) {    // one thread
            int64_t to = excl;
            int32_t b = f0;
            for (; b < f1; ++b) {
                const int32_t t = tree_tiles<TT>(a, tree_rows(a, tr, b), r0);
                if (x < to + t) break;
                to += t;
            }
            at[i] = TreeBegin{b, (int32_t)(x - to)};
        }
    }
    __syncthreads();
    return count;
}

struct TreePos { int32_t b, j, n, m, first, tiles; };      // a sequence and a tile of it
template <int TT>
__device__ __forceinline__ TreePos tree_pos(const KvArgs &a, const KvTreeSplit &tr, int32_t r0, int32_t b, int32_t j) {
    const SeqRows s = tree_rows_scalar(a, tr, b);
    return TreePos{b, j, uniform(s.n), uniform(s.m), uniform(s.first), uniform(tree_tiles<TT>(a, s, r0))};
}
template <int TT>
__device__ __forceinline__ TreePos tree_next(const KvArgs &a, const KvTreeSplit &tr, int32_t r0, TreePos p, int32_t by) {
    p.j += by;                                             // only called while there is such a tile
    while (p.j >= p.tiles && p.b + 1 < a.n_seq) p = tree_pos<TT>(a, tr, r0, p.b + 1, p.j - p.tiles);
    return p;
}

// Two neighbouring words of a row's mask, from the one that the tile's first node lies in (s: the tile's first token as a
// node; below 0: cached before), and which of the tile's up to 64 tokens, cached or nodes, the row sees by them.
__device__ __forceinline__ void mask_at(const KvTreeSplit &tr, int32_t row, int32_t s, uint64_t *lo, uint64_t *hi) {
    const uint64_t *w = tr.mask + (int64_t)row * tr.words;
    const int32_t d = max(s, 0) >> 6;
    *lo = w[min(d, tr.words - 1)];
    *hi = w[min(d + 1, tr.words - 1)];
}
__device__ __forceinline__ uint64_t mask_window(const KvTreeSplit &tr, int32_t s, uint64_t lo, uint64_t hi) {
    if (s <= -64) return ~0ull;
    if (s < 0) return lo << -s | ((1ull << -s) - 1);
    const int32_t k = s & 63;
    return k == 0 ? lo : lo >> k | ((s >> 6) + 1 < tr.words ? hi << (64 - k) : 0);
}

template <typename E>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {   // the parts of a dword that are infinite or NaN, the rest zero
    if constexpr (sizeof(E) == 4) return (w & 0x7f800000u) == 0x7f800000u ? w : 0u;
    else return ((w & 0x7f80u) == 0x7f80u ? w & 0xffffu : 0u) | ((w & 0x7f800000u) == 0x7f800000u ? w & 0xffff0000u : 0u);
}

// Two weights as the sums of two bfloat16 numbers each, off by at most 2^-15: x the first ones, their leading bits, cut off; y the
// second, the rest, rounded, and raised to 2^-126 where it is less, unless the weight itself is: an infinite value times a
// weight stays that infinity, and a weight of zero stays zero.
__device__ __forceinline__ uint2 split2(float a0, float a1) {
    const uint32_t u0 = __float_as_uint(a0), u1 = __float_as_uint(a1);
    const float f0 = __uint_as_float(u0 & 0xffff0000u), f1 = __uint_as_float(u1 & 0xffff0000u);
    return make_uint2(__builtin_amdgcn_perm(u1, u0, 0x07060302u),
                      pack2(__builtin_amdgcn_fmed3f(a0 - f0, f0, 0x1p-126f), __builtin_amdgcn_fmed3f(a1 - f1, f1, 0x1p-126f)));
}

// More than 16 rows, float32 also heads of up to 128 more than 32 (k_kv_tree_wide.hip)
constexpr int WIDE_ROWS = 128;
hipError_t launch_tree_wide(int dtype, const KvArgs &a, const KvAttend &at, const KvTreeSplit &tr, bool local, hipStream_t s);

}  // namespace lorapool

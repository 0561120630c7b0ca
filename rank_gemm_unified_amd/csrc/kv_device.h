// Device-side helpers of the KV-cache kernels: a sequence's rows and length, checked, and the address
// of a token's K or V row.
#pragma once

#include "device_common.h"
#include "kv.h"

namespace lorapool {

struct SeqRows {
    int32_t first;   // first new row
    int32_t m;       // new rows (0 for a bad range)
    int32_t n;       // tokens in the cache, the new ones included (0 for a bad length)
    int err;
};

// Sequence b's rows and length.  A range outside [0, T] counts as empty; a length below 0, above the
// capacity or (when not 0) below the number of new rows counts as 0.
__device__ __forceinline__ SeqRows seq_rows(const KvArgs &a, int32_t s0, int32_t s1, int32_t n) {
    SeqRows s;
    bool bad = s0 < 0 || s1 < s0 || s1 > a.T;
    s.first = bad ? 0 : s0;
    s.m = bad ? 0 : s1 - s0;
    s.err = bad ? DEV_ERR_LEN : 0;
    bad = n < 0 || n > a.cap || (n > 0 && n < s.m);
    s.n = bad ? 0 : n;
    if (bad) s.err = DEV_ERR_LEN;
    return s;
}
__device__ __forceinline__ SeqRows seq_rows(const KvArgs &a, int32_t b) {
    return a.q_start ? seq_rows(a, a.q_start[b], a.q_start[b + 1], a.lens[b]) : seq_rows(a, b, b + 1, a.lens[b]);
}

// Page index of token t, and t's place in that page.
__device__ __forceinline__ void page_of(const KvArgs &a, int32_t t, int32_t *page, int32_t *slot) {
    const int32_t p = a.tpp == 1 ? t : (int32_t)__umulhi((uint32_t)t, a.tpp_magic);
    *page = p;
    *slot = t - p * a.tpp;
}

// Byte offset of token t's row inside the pool, or -1 for a page id outside the pool.
__device__ __forceinline__ int64_t token_offset(const KvArgs &a, const int32_t *row, int32_t t) {
    int32_t e, slot;
    page_of(a, t, &e, &slot);
    const int32_t pg = row[e];
    if (pg < 0 || (int64_t)pg >= a.num_pages) return -1;
    return (int64_t)pg * a.page_bytes + (int64_t)slot * a.tok_bytes;
}

__device__ __forceinline__ void record(const KvArgs &a, int bits) {
    if (bits) atomicOr(a.err, bits);
}

// Record every sequence whose rows or length are out of bounds, by the threads of one workgroup.
__device__ __forceinline__ void check_seqs(const KvArgs &a) {
    int bits = 0;
    for (int32_t b = threadIdx.x; b < a.n_seq; b += blockDim.x) bits |= seq_rows(a, b).err;
    record(a, bits);
}

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack2(float a, float b) {   // two floats to bfloat16, round to nearest even
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
// A value that is the same in every lane of the wave, as a scalar.
__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_bits_to_f32(v); }
__device__ __forceinline__ void from_f32(float *p, float v) { *p = v; }
__device__ __forceinline__ void from_f32(uint16_t *p, float v) { *p = (uint16_t)f32_to_bf16_bits(v); }

}  // namespace lorapool

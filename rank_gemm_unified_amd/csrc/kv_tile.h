// K and V tiles in LDS, as the kernels over many query rows lay them out: steps of NT tokens, double buffered.
#pragma once

#include "kv_device.h"

namespace lorapool {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

// The transposing read.  (Behind a restrict pointer: the compiler else takes it for a reader of the loads to LDS that
// are in flight, and waits for them.  The waits that are needed are written out.)
__device__ __forceinline__ s16x4_t read_tr(lds_s16x4 *__restrict__ p) { return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p); }

template <typename E, int HD>
struct Chunk {
    static constexpr bool BF = sizeof(E) == 2;
    static constexpr int NT = BF ? 64 : 32;                 // tokens of a step
    static constexpr int NB = NT / 32;
    static constexpr int RB = HD * (int)sizeof(E);          // bytes of a token's row
    static constexpr int CH = RB / 16;                      // 16-byte pieces of it
    static constexpr int BUF = NT * RB;
    static constexpr int LDS = 4 * BUF + 6 * 1024 + 64;     // two steps of K and of V; addresses, page ids, a bit of 512 tokens
    static constexpr int WAVES = HD == 256 ? 1 : 2;         // workgroups a CU (registers)
    static constexpr int KQ = BF ? HD / 16 : HD / 8;        // 16-byte pieces of a query row a lane holds
    static constexpr int PER = BUF / 4096;                  // 1 KiB pieces of a step's K a wave brings
    // Where piece c of row t lies in LDS.  What one cycle reads has to lie in different banks (256 bytes of them): of
    // K one piece of 16 rows, of V (bfloat16, transposing read) two neighbouring pairs of pieces of four rows.
    static __device__ __forceinline__ int k_swz(int t, int c) { return c ^ (CH == 8 ? t >> 1 & 7 : t & 15); }
    static __device__ __forceinline__ int v_swz(int t, int c) { return !BF ? c : c ^ (CH == 8 ? (t >> 1 & 1) << 2 : (t & 3) << 2); }
};

}  // namespace lorapool

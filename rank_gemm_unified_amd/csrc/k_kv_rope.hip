// New tokens' rows after the projections: q and k turned by their positions (rotary embedding), K and V to their slots.
//
// A pair (a, b) of a head's elements becomes (a c - b s, a s + b c), c and s from the caller's table.  A copy with three
// multiplications an element: bound by the bytes moved, 16 bytes a lane and load (8 x 512 tokens of 32 heads of 128: 41.5 us
// for 202 MB, 4.9 TB/s); for few tokens by the chain position -> table -> store (64 of them 3.5 us).
#include <algorithm>

#include "kv_device.h"

namespace lorapool {

struct RopeUnits {            // pieces of 16 bytes a thread takes at a time
    int32_t per_head;         // of a q or k head: pairs of pieces that turn (halves) or pieces (neighbours), and the rest
    int32_t turn;             // of them turn
    uint32_t magic;           // u / per_head = mulhi(u, magic) for u < 2^17; per_head 1: 0
    int32_t q, k, total;      // units of q, of q and k, of a token
    uint32_t total_magic;     // as magic, of total; for items below 2^17
};

// MANY: a workgroup takes `per` tokens, their units one behind the other; else one (8 x 512 tokens of 32 heads: 41.8 us, by
// the other form 45.2; 8192 of 8 heads on one: 17.8, by the other 11.2).
template <typename E, bool MANY>
__global__ __launch_bounds__(256) void k_kv_rope(KvRope r, RopeUnits ru, int32_t per) {
    constexpr int VE = 16 / (int)sizeof(E);                // elements of a piece
    // One unit u of row t: its slots' places kd and vd in the pages, its position's cosines and sines.
    auto unit = [&](int32_t t, int32_t u, char *kd, char *vd, const float *turn) {
        if (u >= ru.k) {
            const int32_t x = u - ru.k;
            store16(vd + 16 * (int64_t)x, load16((const char *)r.v + t * r.ldv * (int64_t)sizeof(E) + 16 * (int64_t)x));
            return;
        }
        const bool is_q = u < ru.q;
        const int32_t x = is_q ? u : u - ru.q, head = ru.magic ? (int32_t)__umulhi((uint32_t)x, ru.magic) : x, y = x - head * ru.per_head;
        const E *src = (is_q ? (const E *)r.q + t * r.ldq : (const E *)r.k + t * r.ldk) + (int64_t)head * r.head_dim;
        E *dst = (is_q ? (E *)r.q_out + t * r.ldqo : (E *)kd) + (int64_t)head * r.head_dim;
        if (y >= ru.turn) {                            // what does not turn
            const int32_t d = r.rot + (y - ru.turn) * VE;
            store16(dst + d, load16(src + d));
            return;
        }
        float a[VE], b[VE], c[2 * VE];
        if (r.pairs) {                                 // neighbours: VE / 2 pairs in a piece
            const u32x4_t w = load16(src + y * VE);
#pragma unroll
            for (int i = 0; i < VE / 2; i += 2) *(f32x4_t *)(c + 2 * i) = *(const f32x4_t *)(turn + y * VE + 2 * i);
            if constexpr (VE == 8) unpack_bf16x8(w, a);
            else
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = __uint_as_float(w[i]);
#pragma unroll
            for (int i = 0; i < VE; i += 2) {
                b[i] = a[i] * c[i] - a[i + 1] * c[i + 1];
                b[i + 1] = a[i] * c[i + 1] + a[i + 1] * c[i];
            }
            if constexpr (VE == 8) store16(dst + y * VE, u32x4_t{pack2(b[0], b[1]), pack2(b[2], b[3]), pack2(b[4], b[5]), pack2(b[6], b[7])});
            else store16(dst + y * VE, u32x4_t{__float_as_uint(b[0]), __float_as_uint(b[1]), __float_as_uint(b[2]), __float_as_uint(b[3])});
            return;
        }
        const int32_t d = y * VE, d2 = d + r.rot / 2;
        const u32x4_t w = load16(src + d), w2 = load16(src + d2);
#pragma unroll
        for (int i = 0; i < VE; i += 2) *(f32x4_t *)(c + 2 * i) = *(const f32x4_t *)(turn + 2 * d + 2 * i);
        if constexpr (VE == 8) {
            unpack_bf16x8(w, a);
            unpack_bf16x8(w2, b);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = __uint_as_float(w[i]);
                b[i] = __uint_as_float(w2[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const float p = a[i] * c[2 * i] - b[i] * c[2 * i + 1], q = a[i] * c[2 * i + 1] + b[i] * c[2 * i];
            a[i] = p;
            b[i] = q;
        }
        if constexpr (VE == 8) {
            store16(dst + d, u32x4_t{pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(a[4], a[5]), pack2(a[6], a[7])});
            store16(dst + d2, u32x4_t{pack2(b[0], b[1]), pack2(b[2], b[3]), pack2(b[4], b[5]), pack2(b[6], b[7])});
        } else {
            store16(dst + d, u32x4_t{__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]), __float_as_uint(a[3])});
            store16(dst + d2, u32x4_t{__float_as_uint(b[0]), __float_as_uint(b[1]), __float_as_uint(b[2]), __float_as_uint(b[3])});
        }
    };
    // Where row t's K and V go, and its cosines and sines; false: nowhere.
    auto row = [&](int32_t t, bool say, char **kd, char **vd, const float **turn) {
        const int64_t ks = r.slots[t], vs = r.slots[(int64_t)r.T + t], most = r.num_pages * r.tpp;
        const int32_t pos = r.positions[t];
        if (ks < 0 && vs < 0) return false;                // a row of no sequence
        if (ks < 0 || vs < 0 || ks >= most || vs >= most || pos < 0 || pos >= r.n_positions) {
            if (say) atomicOr(r.err, pos < 0 || pos >= r.n_positions ? DEV_ERR_LEN : DEV_ERR_PAGE);
            return false;
        }
        auto place = [&](int64_t slot) {                   // slots are below 2^32: a pool of 512 GiB, token rows of 128 bytes
            const uint32_t page = (uint32_t)slot / (uint32_t)r.tpp;
            return r.pages + (int64_t)page * r.page_bytes + (int64_t)((uint32_t)slot - page * r.tpp) * r.tok_bytes;
        };
        *kd = place(ks);
        *vd = place(vs);
        *turn = r.table + (int64_t)pos * r.rot;
        return true;
    };
    const int32_t first = blockIdx.y * 256 + threadIdx.x, step = gridDim.y * 256;
    char *kd, *vd;
    const float *turn;
    if constexpr (MANY) {
        const int32_t t0 = blockIdx.x * per, items = min(per, r.T - t0) * ru.total;
        for (int32_t item = first; item < items; item += step) {
            const int32_t local = (int32_t)__umulhi((uint32_t)item, ru.total_magic), u = item - local * ru.total;
            if (row(t0 + local, u == 0, &kd, &vd, &turn)) unit(t0 + local, u, kd, vd, turn);
        }
    } else if (row(blockIdx.x, first == 0, &kd, &vd, &turn)) {
        for (int32_t u = first; u < ru.total; u += step) unit(blockIdx.x, u, kd, vd, turn);
    }
}

template <typename E>
static hipError_t rope(const KvRope &r, hipStream_t s) {
    constexpr int VE = 16 / (int)sizeof(E);
    RopeUnits u;
    u.turn = r.rot / (r.pairs ? VE : 2 * VE);
    u.per_head = u.turn + (r.head_dim - r.rot) / VE;
    u.magic = u.per_head == 1 ? 0 : (uint32_t)(((uint64_t(1) << 32) + u.per_head - 1) / u.per_head);
    u.q = r.q ? r.n_heads * u.per_head : 0;
    u.k = u.q + r.n_kv * u.per_head;
    u.total = u.k + r.n_kv * (r.head_dim / VE);
    // Few tokens: one unit a thread, a token's over several workgroups; many small ones: several a workgroup.
    const int32_t most = (u.total + 255) / 256, gy = std::min(most, std::max(1, 1024 / r.T));
    const int32_t per = std::max(1, std::min(1024 / u.total, r.T / 1024));
    u.total_magic = (uint32_t)(((uint64_t(1) << 32) + u.total - 1) / u.total);
    const dim3 grid((unsigned)((r.T + per - 1) / per), (unsigned)gy);
    if (per > 1) hipLaunchKernelGGL((k_kv_rope<E, true>), grid, dim3(256), 0, s, r, u, per);
    else hipLaunchKernelGGL((k_kv_rope<E, false>), grid, dim3(256), 0, s, r, u, per);
    return hipGetLastError();
}

hipError_t launch_kv_rope(int dtype, const KvRope &r, hipStream_t s) {
    return dtype == LORA_F32 ? rope<float>(r, s) : rope<uint16_t>(r, s);
}

}  // namespace lorapool

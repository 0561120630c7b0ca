// A step's plan from its lengths: rows, pages, slots, positions and tree masks, on the GPU.
//
// Everything is a prefix sum over the sequences: of new tokens (the rows), of pages that come and of pages that go.  A
// row's slot is then page * tokens_per_page + place, its page from the table or, if it is new, from the ring of free
// page groups, where the prefix sum says.  8 bytes written for each (layer, K/V, row) and a few read: the time is the
// chain lengths -> sums -> page -> slot, so it is one launch: each workgroup takes 256 rows of some layers and forms
// the sums over all sequences by itself.  In place the lengths are written by the workgroup that comes last, when
// nobody reads them any more.  64 sequences of a token in 32 layers 7.4 to 7.7 us, with trees of 16 nodes 8.0, 8 prompts of 512 7.2
// (4.2 MB); in place, one behind the other in a replayed graph, 9.5 and, chains of 16 nodes, 13.5.
#include <algorithm>

#include "kv_device.h"

namespace lorapool {

namespace {

struct Want {                 // what a sequence asks for
    int32_t n, h;             // tokens cached, pages held
    int32_t c;                // rows
    int32_t take, give;       // pages that come, and that go
    bool valid;               // it may take part
    int err;
};

__device__ __forceinline__ int32_t pages_of(const KvPlan &p, int32_t tokens) {
    const int32_t t = tokens + p.tpp - 1;
    return p.tpp == 1 ? tokens : (int32_t)__umulhi((uint32_t)t, p.tpp_magic);
}

__device__ __forceinline__ int32_t rows_of(const KvPlan &p, int32_t b, int *err) {
    const int32_t c = p.counts[b];
    const bool bad = c < 0 || c > (p.parents ? p.max_nodes : p.T);
    if (bad) *err = DEV_ERR_LEN;
    return bad ? 0 : c;
}
// `end`: rows up to this sequence's last; behind T it has no room, takes nothing and gives nothing.
__device__ __forceinline__ Want want_of(const KvPlan &p, int32_t b, int64_t end) {
    Want w;
    w.err = 0;
    w.c = rows_of(p, b, &w.err);
    w.n = p.lens[b];
    w.h = p.held[b];
    w.take = w.give = 0;
    w.valid = w.n >= 0 && w.n <= p.cap && w.h >= 0 && w.h <= p.max_pages && pages_of(p, w.n) <= w.h;
    if (!w.valid) {
        w.err = DEV_ERR_LEN;
        return w;
    }
    if (w.c > 0 && (end > p.T || w.c > p.cap - w.n)) {     // refused: its pages stay, those it has too much too
        w.err = DEV_ERR_LEN;
        w.valid = false;
        return w;
    }
    const int32_t pages = pages_of(p, w.n + w.c);
    w.take = max(0, pages - w.h);
    w.give = max(0, w.h - pages);
    return w;
}

struct Sums { int64_t rows, take, give; };

}  // namespace

__global__ __launch_bounds__(256) void k_kv_plan(KvPlan p, int32_t per_layers, int in_place) {
    __shared__ int64_t sh[4][3];
    __shared__ int32_t mark[256], top[4], parent[512];
    __shared__ struct { int32_t b, i, n, h, ok; int64_t before; } at[256];
    __shared__ int last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t per = (p.n_seq + 255) / 256, b0 = min(p.n_seq, tid * per), b1 = min(p.n_seq, b0 + per);
    int err = 0;

    // ---- sums over the sequences: this thread's begin at `mine` ----
    // All three at once, as if every row had room; where they have not (T says fewer) the sequences behind T take nothing,
    // and the sums are formed again.
    Sums mine{0, 0, 0}, all;
    auto sum_up = [&](Sums &x) {                           // exclusive; returns the totals
        int64_t v[3] = {x.rows, x.take, x.give}, total[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            int64_t incl = v[k];
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int64_t y = __shfl_up(incl, o, 64);
                if (lane >= o) incl += y;
            }
            if (lane == 63) sh[wave][k] = incl;
            v[k] = incl - v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            total[k] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[k] += i < wave ? sh[i][k] : 0;
                total[k] += sh[i][k];
            }
        }
        x = Sums{v[0], v[1], v[2]};
        return Sums{total[0], total[1], total[2]};
    };
    for (int32_t b = b0; b < b1; ++b) {
        const Want w = want_of(p, b, 0);
        mine.rows += w.c;
        mine.take += w.take;
        mine.give += w.give;
        err |= w.err;
    }
    all = sum_up(mine);
    if (all.rows > p.T) {
        int64_t end = mine.rows;
        const int64_t first = end;
        mine.take = mine.give = 0;
        for (int32_t b = b0; b < b1; ++b) {
            int e = 0;
            end += rows_of(p, b, &e);
            const Want w = want_of(p, b, end);
            mine.take += w.take;
            mine.give += w.give;
            err |= w.err;
        }
        mine.rows = 0;
        __syncthreads();
        all.take = all.give = 0;
        const Sums again = sum_up(mine);
        mine.rows = first;
        all.take = again.take;
        all.give = again.give;
    }
    const int64_t rows = all.rows, given = all.give;
    int32_t head = p.state[0], free = p.state[1];
    const bool ring = head >= 0 && head < p.groups && free >= 0 && free <= p.groups;
    if (!ring) {
        err |= DEV_ERR_LEN;
        head = free = 0;
    }
    const int64_t room = ring ? p.groups - free : 0;       // groups that can come back
    auto ring_at = [&](int64_t x) { return x >= p.groups ? x - p.groups : x; };
    // this thread's sequences: f(b, what it wants, sums before it, whether it is served, whether its pages go)
    auto each = [&](auto f) {
        Sums s = mine;
        for (int32_t b = b0; b < b1; ++b) {
            int e = 0;
            const int32_t c = rows_of(p, b, &e);
            const Want w = want_of(p, b, s.rows + c);
            f(b, w, s, w.valid && (w.take == 0 || s.take + w.take <= free), s.give + w.give <= room);
            s.rows += c;
            s.take += w.take;
            s.give += w.give;
        }
    };
    // the last marked place up to this thread's
    auto marked = [&]() {
        int32_t m = mark[tid];
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int32_t y = __shfl_up(m, o, 64);
            if (lane >= o) m = max(m, y);
        }
        if (lane == 63) top[wave] = m;
        __syncthreads();
        for (int i = 0; i < wave; ++i) m = max(m, top[i]);
        return m;
    };

    // ---- rows ----
    const int32_t t0 = blockIdx.x * 256, t = t0 + tid, l0 = blockIdx.y * per_layers, l1 = min(p.layers, l0 + per_layers);
    mark[tid] = -1;
    if (p.parents && blockIdx.y == 0)
        for (int x = tid; x < 512; x += 256) {
            const int32_t r = t0 - 256 + x;
            parent[x] = r >= 0 && r < p.T ? p.parents[r] : -1;
        }
    __syncthreads();
    each([&](int32_t b, const Want &w, const Sums &s, bool ok, bool) {
        if (w.c == 0 || s.rows >= t0 + 256 || s.rows + w.c <= t0) return;
        const int32_t place = max(0, (int32_t)(s.rows - t0));
        mark[place] = place;
        at[place].b = b;
        at[place].i = (int32_t)(t0 + place - s.rows);
        at[place].n = w.n;
        at[place].h = w.h;
        at[place].ok = ok;
        at[place].before = s.take;
    });
    __syncthreads();
    const int32_t from = marked();
    if (t < p.T) {
        const bool row = from >= 0 && t < rows && at[max(from, 0)].ok;
        int32_t b = 0, i = 0, pos = 0, e = 0, h = 0;
        int64_t group = 0;
        if (row) {
            b = at[from].b;
            i = at[from].i + tid - from;
            pos = at[from].n + i;
            h = at[from].h;
            e = p.tpp == 1 ? pos : (int32_t)__umulhi((uint32_t)pos, p.tpp_magic);
            group = ring_at(head + at[from].before + max(0, e - h));
        }
        const int32_t place = pos - e * p.tpp;
        if (blockIdx.y == 0) {
            int32_t depth = i;
            if (p.parents) {
                uint64_t word[LORA_MAX_TREE / 64];
#pragma unroll
                for (int w = 0; w < LORA_MAX_TREE / 64; ++w) word[w] = row && i >> 6 == w ? 1ull << (i & 63) : 0;
                depth = 0;
                for (int32_t j = i; row && j > 0; ++depth) {
                    const int32_t up = parent[256 + tid - i + j];
                    if (up < 0 || up >= j) { err |= DEV_ERR_TREE; break; }
                    j = up;
#pragma unroll
                    for (int w = 0; w < LORA_MAX_TREE / 64; ++w) word[w] |= j >> 6 == w ? 1ull << (j & 63) : 0;
                }
#pragma unroll
                for (int w = 0; w < LORA_MAX_TREE / 64; ++w)
                    if (w < p.words) p.mask[(int64_t)t * p.words + w] = word[w];
            }
            p.positions[t] = row ? pos - i + depth : 0;
        }
        for (int32_t x = 2 * l0; x < 2 * l1; ++x) {        // layer x / 2, K or V
            int32_t page = -1;
            if (row) {
                int32_t *entry = p.table + (((int64_t)(x >> 1) * p.n_seq + b) * 2 + (x & 1)) * p.max_pages + e;
                if (e < h) {
                    page = *entry;
                } else {
                    page = p.stock[group * 2 * p.layers + x];
                    if (place == 0) *entry = page;
                }
                if (page < 0 || page >= p.num_pages) err |= DEV_ERR_PAGE, page = -1;
            }
            p.slots[(int64_t)x * p.T + t] = page < 0 ? -1 : (int64_t)page * p.tpp + place;
        }
    }

    // ---- pages that go, behind the free ones ----
    for (int64_t x0 = (int64_t)blockIdx.x * 256; x0 < given; x0 += (int64_t)gridDim.x * 256) {
        __syncthreads();
        mark[tid] = -1;
        __syncthreads();
        each([&](int32_t b, const Want &w, const Sums &s, bool, bool fits) {
            if (w.give == 0 || s.give >= x0 + 256 || s.give + w.give <= x0) return;
            const int32_t place = (int32_t)max((int64_t)0, s.give - x0);
            mark[place] = place;
            at[place].b = b;
            at[place].i = w.h - w.give + (int32_t)(x0 + place - s.give);
            at[place].ok = fits;
        });
        __syncthreads();
        const int32_t f = marked();
        if (f >= 0 && x0 + tid < given && at[max(f, 0)].ok) {
            const int32_t b = at[f].b, e = at[f].i + tid - f;
            const int64_t group = ring_at(ring_at(head + free) + x0 + tid);
            for (int32_t x = 2 * l0; x < 2 * l1; ++x)
                p.stock[group * 2 * p.layers + x] = p.table[(((int64_t)(x >> 1) * p.n_seq + b) * 2 + (x & 1)) * p.max_pages + e];
        }
    }
    if (err) atomicOr(p.err, err);

    // ---- lengths ----
    if (in_place && gridDim.x * gridDim.y > 1) {
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            last = atomicAdd((int32_t *)&p.state[3], 1) == (int)(gridDim.x * gridDim.y) - 1;
            __threadfence();
        }
        __syncthreads();
        if (!last) return;
    } else if (blockIdx.x || blockIdx.y) {
        return;
    }
    int64_t taken = 0, back = 0, refused = 0;
    each([&](int32_t b, const Want &w, const Sums &s, bool ok, bool fits) {
        if (ok && w.take) taken = s.take + w.take;
        if (w.give && fits) back = s.give + w.give;
        if (w.give && !fits) atomicOr(p.err, DEV_ERR_LEN);
        refused += w.c > 0 && !ok;
        p.q_start[b] = (int32_t)min(s.rows, (int64_t)p.T);
        if (b == p.n_seq - 1) p.q_start[b + 1] = (int32_t)min(s.rows + w.c, (int64_t)p.T);
        p.step_lens[b] = ok && w.c ? w.n + w.c : 0;
        p.lens_out[b] = ok ? w.n + w.c : w.n;
        p.held_out[b] = w.h + (ok ? w.take : 0) - (fits ? w.give : 0);
    });
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        taken = max(taken, __shfl_xor(taken, o, 64));
        back = max(back, __shfl_xor(back, o, 64));
        refused += __shfl_xor(refused, o, 64);
    }
    __syncthreads();
    if (lane == 0) {
        sh[wave][0] = taken;
        sh[wave][1] = back;
        sh[wave][2] = refused;
    }
    __syncthreads();
    if (tid == 0) {
        if (p.n_seq == 0) p.q_start[0] = 0;
        taken = back = refused = 0;
        for (int i = 0; i < 4; ++i) {
            taken = max(taken, sh[i][0]);
            back = max(back, sh[i][1]);
            refused += sh[i][2];
        }
        p.state_out[0] = ring ? (int32_t)ring_at(head + taken) : p.state[0];
        p.state_out[1] = ring ? (int32_t)(free - taken + back) : p.state[1];
        p.state_out[2] = (int32_t)refused;
        p.state_out[3] = 0;
        if (in_place && p.state_out != p.state) ((int32_t *)p.state)[3] = 0;
    }
}

hipError_t launch_kv_plan(const KvPlan &p, hipStream_t s) {
    const int32_t gx = std::max(1, (p.T + 255) / 256), gy = std::min(p.layers, std::max(1, 512 / gx));
    const int32_t per = (p.layers + gy - 1) / gy;
    const bool in_place = p.lens_out == p.lens || p.held_out == p.held || p.state_out == p.state;
    hipLaunchKernelGGL(k_kv_plan, dim3((unsigned)gx, (unsigned)((p.layers + per - 1) / per)), dim3(256), 0, s, p, per, (int)in_place);
    return hipGetLastError();
}

}  // namespace lorapool

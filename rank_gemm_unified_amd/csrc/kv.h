// Declarations shared by the host code and the kernels of the KV-cache calls (lora_kv_*).
#pragma once

#include "internal.h"

namespace lorapool {

// One call's view of the cache: what every KV kernel needs to find a sequence's rows, its length and
// its tokens' addresses.  Passed to the kernels by value.
struct KvArgs {
    char *pages;
    int64_t num_pages;
    int64_t page_bytes;       // hidden * element
    const int32_t *table;     // [n_seq][2][max_pages]
    const int32_t *q_start;   // [n_seq + 1], or null: row b is sequence b's one new token
    const int32_t *lens;      // [n_seq]
    int *err;                 // the pool's device error word
    int32_t max_pages;
    int32_t n_seq;
    int32_t T;                // rows of q, k, v, out
    int32_t cap;              // largest length a sequence may have in this call
    int32_t n_heads, n_kv, head_dim, group;   // group = n_heads / n_kv
    int32_t tpp;              // tokens a page
    uint32_t tpp_magic;       // ceil(2^32 / tpp): t / tpp = mulhi(t, magic) for t < 2^24, tpp in 2..256
    int32_t tok_bytes;        // n_kv * head_dim * element
};

struct KvAttend {
    const void *q;
    void *out;
    int64_t ldq, ldo;         // elements
    float scale;
    const float *prior;       // [n_seq][score_ld] or null
    float *scores;            // ... or null
    int64_t score_ld;
    void *ws;
};

struct KvTreeArgs {
    const uint64_t *mask;     // [T][(max_nodes + 63) / 64]: bit j of row i: it sees node j of its sequence
    int32_t max_nodes;        // new tokens of a sequence, at most
};

struct KvPlan {
    int64_t num_pages;
    int32_t layers, n_seq, max_pages, tpp, T;
    uint32_t tpp_magic;       // as in KvArgs
    int32_t cap;              // largest length a sequence may reach
    const int32_t *counts, *lens, *held, *state;
    int32_t *table, *stock;   // [layers][n_seq][2][max_pages]; [groups][layers][2]
    int32_t groups;
    int32_t *step_lens, *q_start, *positions, *lens_out, *held_out, *state_out;
    int64_t *slots;           // [layers][2][T]
    const int32_t *parents;   // [T] or null
    uint64_t *mask;           // [T][words]
    int32_t max_nodes, words;
    int *err;
};

struct KvRope {
    char *pages;
    int64_t num_pages, page_bytes;
    int32_t tpp, T;
    int32_t n_heads, n_kv, head_dim, tok_bytes;
    const float *table;       // [n_positions][rot / 2][2]
    int32_t n_positions, rot, pairs;
    const void *q, *k, *v;
    void *q_out;
    int64_t ldq, ldqo, ldk, ldv;
    const int64_t *slots;     // [2][T]
    const int32_t *positions;
    int *err;
};

struct KvAccept {
    KvArgs a;                 // table: [layers][n_seq][2][max_pages]
    int32_t layers, max_nodes;
    const int32_t *tokens, *targets, *parents;
    int32_t *lens_out, *path, *n_path, *next;
};

struct KvEvict {
    int32_t layers, n_seq, max_pages, tpp;
    const int32_t *table;
    int32_t *table_out;
    const float *scores;
    float *scores_out;
    const int32_t *lens;
    int32_t *lens_out;
    int32_t budget, keep_first, keep_last, max_drop;
    int32_t *dropped, *n_dropped;
    int *err;
};

// Workspace to have (never less for a larger call), and what the call itself uses.
size_t kv_attend_ws_bytes(int dtype, const lora_kv_layout_t &l, int32_t n_seq, int64_t max_len, bool scores);
size_t kv_attend_ws_need(int dtype, const lora_kv_layout_t &l, int32_t n_seq, int64_t max_len, bool scores);
size_t kv_chunk_ws_bytes(int dtype, const lora_kv_layout_t &l, int32_t n_seq, int64_t T, int64_t max_len, bool scores);
size_t kv_tree_ws_bytes(int dtype, const lora_kv_layout_t &l, int32_t n_seq, int32_t max_nodes, int64_t max_len);

hipError_t launch_kv_write(int dtype, const KvArgs &a, const void *k, int64_t ldk, const void *v, int64_t ldv,
                           hipStream_t s);
hipError_t launch_kv_attend(int dtype, const KvArgs &a, const KvAttend &at, hipStream_t s);
hipError_t launch_kv_chunk(int dtype, const KvArgs &a, const KvAttend &at, hipStream_t s);
hipError_t launch_kv_tree(int dtype, const KvArgs &a, const KvAttend &at, const KvTreeArgs &ta, hipStream_t s);
hipError_t launch_kv_plan(const KvPlan &p, hipStream_t s);
hipError_t launch_kv_rope(int dtype, const KvRope &r, hipStream_t s);
hipError_t launch_kv_accept(const KvAccept &c, hipStream_t s);
hipError_t launch_kv_evict(const KvEvict &e, hipStream_t s);

}  // namespace lorapool

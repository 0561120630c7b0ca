/*
 * lorapool.h -- unmerged multi-LoRA projection over a unified page pool, for AMD Instinct MI355X
 * (gfx950).  Plain C ABI: opaque pool handle, plain pointers and sizes, int status codes.
 *
 * What it computes ("S-LoRA, in depth", section "Merge or keep adapters separate"): a LoRA adapter
 * turns an h-by-h weight W into W + AB with A h-by-r and B r-by-h; a token with activation x gets
 * xW + (xA)B.  Unmerged serving keeps W shared, batches xW over every token whatever its adapter,
 * and adds the low-rank term per token.  This library computes, for T tokens in one call,
 *
 *     y[t] = x[t] W + s[a] * (x[t] A_a) B_a        a = adapter_ids[t]
 *
 * and y[t] = x[t] W when a == -1 or the adapter has rank 0 (the weightless "identity" adapter of
 * "Switch Adapters by Routing Requests Through Resident, Verified State", its adapter registry).
 * The per-adapter float scale s[a] is this library's reading of the usual LoRA scaling; s = 1
 * gives the page's formula.
 *
 * Where A and B live ("S-LoRA, in depth", section "Unified paging: adapters and KV cache in one
 * pool"): a pool of pages, each one vector of H elements, shared by KV cache and adapters through
 * one free list.  An adapter of rank r on one projection takes 2r pages: the r columns of A and
 * the r rows of B.  Pages need not be contiguous or in order; a per-projection page table maps
 * (adapter, j) to a page, and the projection's gather fetches each token's pages from wherever the
 * pool placed them (same page, section "The architecture").
 *
 * Conventions for every function returning int:
 *   0 = LORA_OK, negative = error (below).  No C++ exception crosses this boundary.  On error,
 *   lora_last_error() returns a message for the calling thread, valid until its next call.
 *   Arguments are validated on the host before any device work; an invalid call leaves every
 *   caller buffer untouched.
 * Streams: `stream` arguments are hipStream_t values passed as void* (NULL = the null stream).
 *   All device work of a call is enqueued on that stream, in call order, so a load followed by a
 *   projection on the same stream sees the new weights.  Ordering across streams is the caller's
 *   job (events).
 * Memory ownership: the caller owns every device buffer (pool pages, page table, x, W, y, ids,
 *   ranks, scales, workspace).  The library owns only host bookkeeping plus two small device
 *   buffers it allocates at pool creation (a staging buffer for loads and a device error word),
 *   freed by lora_pool_free.
 * Threads: calls that change a pool (load, release, evict, KV) take the pool's mutex.
 *   lora_project changes no pool state and holds no "active adapter": adapter choice is per token,
 *   carried by adapter_ids (the routing page's warning against a shared mutable active adapter).
 */
#ifndef LORAPOOL_H
#define LORAPOOL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum lora_status {
    LORA_OK = 0,
    LORA_EINVAL = -1,   /* bad argument: null/misaligned pointer, size, dtype, range            */
    LORA_ENOMEM = -2,   /* not enough free pages (or a library allocation failed)              */
    LORA_ENOENT = -3,   /* unknown adapter / request id                                        */
    LORA_ERANK = -4,    /* rank out of range, or not the rank the adapter was loaded at        */
    LORA_EBUSY = -5,    /* adapter still has users                                             */
    LORA_EEXIST = -6,   /* adapter already resident at another rank                            */
    LORA_EHIP = -7,     /* a HIP runtime call failed (message has the HIP error string)        */
    LORA_EDEVICE = -8   /* earlier work found bad ids/ranks/pages/lengths on the device            */
};

enum lora_dtype {
    LORA_F32 = 0,       /* pages, x, W, A, B, y in IEEE float32                                 */
    LORA_BF16 = 1       /* ... in bfloat16; products accumulate in float32                      */
};

enum lora_victim_rule {         /* which idle adapter a load that is short of pages evicts first */
    LORA_VICTIM_LOAD_ORDER = 0, /* oldest load first: the pool sketch's rule (the default)        */
    LORA_VICTIM_LRU = 1,        /* least recently admitted first                                  */
    LORA_VICTIM_FARTHEST = 2    /* next request in the lookahead farthest first (Belady's rule);
                                   adapters beyond the lookahead last-admitted-longest-ago first  */
};

#define LORA_MAX_RANK 64        /* largest rank a pool can be created for                       */
#define LORA_MAX_ADAPTERS 8192  /* largest adapter id + 1                                       */
#define LORA_MAX_TOKENS (1 << 22) /* most tokens (T) one projection call takes                  */

typedef struct lora_pool lora_pool;

typedef struct lora_pool_stats {
    int64_t num_pages;          /* pool size                                                    */
    int64_t free_pages;         /* on the free list                                             */
    int64_t kv_pages;           /* held by KV requests                                          */
    int64_t adapter_pages;      /* held by resident adapters                                    */
    int32_t resident_adapters;  /* adapters holding pages (rank-0 adapters count, with 0 pages) */
    int32_t idle_adapters;      /* resident adapters with no users                              */
    int64_t kv_requests;        /* requests holding KV pages                                    */
    int64_t loads;              /* adapter loads that allocated pages (not refcount bumps)      */
    int64_t evictions;          /* adapters whose pages were reclaimed                          */
    int64_t bytes_loaded;       /* bytes copied into pages by loads                             */
} lora_pool_stats_t;

/* ---- pool lifecycle ("Unified paging" section and its pool sketch) ------------------------- */

/*
 * Create a pool over caller-owned device memory.
 *   pages        device, num_pages * hidden elements of `dtype`, 16-byte aligned.  Page p is the
 *                hidden-element vector at pages + p * hidden.
 *   num_pages    >= 1.
 *   hidden       H, the page length and the projection's input and output width; a multiple of
 *                64, 64 <= H <= 65536.
 *   dtype        LORA_F32 or LORA_BF16.
 *   max_rank     1..LORA_MAX_RANK; every adapter's rank must be <= max_rank.
 *   n_slots      projections per adapter (layers * projections, e.g. 32 * 4 for q/k/v/o of a
 *                7B model); each slot has its own page-table block.
 *   max_adapters adapter ids are 0..max_adapters-1 (<= LORA_MAX_ADAPTERS).
 *   page_table   device int32 [n_slots][max_adapters][2*max_rank], caller-owned, 4-byte aligned.
 *                Row (slot, a) lists adapter a's pages for that slot: entries 0..r-1 the columns
 *                of A, r..2r-1 the rows of B, -1 after that.  The library writes it (set to -1
 *                here, synchronously); callers only read it.
 *   free_order   host int64 [num_pages], a permutation of 0..num_pages-1 giving the initial free
 *                list, or NULL for 0..num_pages-1.  Allocation takes pages from the END of the
 *                list and frees append to it (the sketch's pop and extend), so the default hands
 *                out num_pages-1 first.
 *   out          receives the handle.
 * pages and page_table may both be NULL: a bookkeeping-only pool that allocates and accounts
 * pages but touches no device memory (loads copy nothing; projections are refused).
 * Errors: LORA_EINVAL (bad argument, free_order not a permutation), LORA_EHIP.
 */
int lora_pool_create(void *pages, int64_t num_pages, int32_t hidden, int32_t dtype,
                     int32_t max_rank, int32_t n_slots, int32_t max_adapters, int32_t *page_table,
                     const int64_t *free_order, lora_pool **out);

/* Destroy the pool's bookkeeping and library-owned device buffers; waits for the pool's pending
 * loads first.  Caller buffers are untouched.  NULL is accepted.  Returns LORA_OK or LORA_EHIP. */
int lora_pool_free(lora_pool *pool);

/*
 * Make adapter `adapter_id` resident at `rank` (0..max_rank), as the sketch's ensure_adapter:
 *   - already resident at the same rank: one more user (refcount + 1); nothing is copied;
 *   - already resident at another rank: LORA_EEXIST;
 *   - otherwise it needs 2 * rank * n_slots pages; if fewer are free, idle adapters (no users)
 *     are evicted oldest-load first until enough are free; if even that is not enough the call
 *     returns LORA_ENOMEM with no pages taken (idle adapters evicted on the way stay evicted,
 *     as in the sketch).  On success the adapter has one user.
 * The adapter's page list takes pages from the free list in order; list entry i belongs to slot
 * i / (2r), entry i % (2r) of that slot's table row.
 *   A_t  [n_slots][rank][hidden] of the pool dtype: row j of slot s is column j of that slot's A.
 *   B    [n_slots][rank][hidden]: row j of slot s is row j of that slot's B.
 * A_t and B may be host (pageable or pinned) or device memory; they are read during the call
 * for pageable memory and, otherwise, by work on `stream`: keep them alive and unchanged until
 * the stream has passed this call.  Both may be NULL when rank == 0 or the pool is
 * bookkeeping-only.  The copies and the page-table update are enqueued on `stream`, so with
 * pinned memory and a stream of its own a load overlaps projections on other streams (section
 * "Scheduling: prefetch, clustering and early abort"); make the first projection that uses the
 * adapter wait for `stream` (an event).  Host rows are staged through one of two load buffers per
 * pool: the call waits on the host only while the load two calls earlier is still queued.
 * Errors: LORA_EINVAL, LORA_ERANK (rank > max_rank), LORA_EEXIST, LORA_ENOMEM, LORA_EHIP.
 */
int lora_pool_load_adapter(lora_pool *pool, int32_t adapter_id, int32_t rank, const void *A_t,
                           const void *B, void *stream);

/* Choose the victim rule for idle-adapter eviction (enum lora_victim_rule).  The pool sketch of
 * "S-LoRA, in depth" (section "Unified paging") evicts idle adapters in load order; the MoE-offload
 * page ("Cache the Experts You Will Need", sections "A better eviction rule cuts transfers without
 * changing routing" and "Limited foresight") compares least-recently-used eviction with evicting the
 * entry whose next request lies farthest ahead, given a window of upcoming requests.  A "use" is a
 * call of lora_pool_load_adapter that names the adapter (resident or not).  Errors: LORA_EINVAL. */
int lora_pool_set_victim_rule(lora_pool *pool, int32_t rule);

/* The upcoming adapter requests the farthest-future rule looks at: `n` host ids, soonest first (for
 * a scheduler, its waiting queue).  Copied; n == 0 clears it.  Adapters that do not occur count as
 * needed after every one that does.  Errors: LORA_EINVAL (n < 0, or ids NULL with n > 0). */
int lora_pool_set_lookahead(lora_pool *pool, const int32_t *adapter_ids, int64_t n);

/* One user of the adapter finished (refcount - 1).  At zero users it stays resident but idle and
 * becomes evictable.  Errors: LORA_ENOENT (not resident), LORA_EINVAL (already idle). */
int lora_pool_release_adapter(lora_pool *pool, int32_t adapter_id);

/* Reclaim an idle adapter's pages (section "The architecture": an adapter that no active request
 * uses may give its pages back): they return to the end of the free list in page-list
 * order, and the adapter's page-table rows are reset to -1 on `stream`.  The caller must not
 * evict an adapter that queued, unfinished projections still read.
 * Errors: LORA_ENOENT, LORA_EBUSY (has users). */
int lora_pool_evict_adapter(lora_pool *pool, int32_t adapter_id, void *stream);

/* Grow request `request_id`'s KV cache by one token: 2 * layers pages (K and V per layer), as the
 * sketch's grow_kv.  If page_ids_out is not NULL it receives the 2*layers page ids (host int64).
 * Errors: LORA_ENOMEM (no room: the caller has to stop or cut short some request to make room),
 * LORA_EINVAL. */
int lora_pool_grow_kv(lora_pool *pool, int64_t request_id, int32_t layers, int64_t *page_ids_out);

/* Request finished: its KV pages return to the end of the free list.  The caller must not give back
 * pages that queued, unfinished work still reads.  Errors: LORA_ENOENT. */
int lora_pool_free_kv(lora_pool *pool, int64_t request_id);

/* ---- queries (host only, no device work) ----------------------------------------------------- */

/* Pages for an adapter of `rank` on `projections` projections of `layers` layers:
 * rank * 2 * projections * layers (A and B per projection).  Negative input gives -1. */
int64_t lora_pool_pages_for(int32_t rank, int32_t projections, int32_t layers);

/* KV pages one token takes: 2 * layers (K and V per layer).  Negative input gives -1. */
int64_t lora_kv_pages_per_token(int32_t layers);

int lora_pool_stats(const lora_pool *pool, lora_pool_stats_t *out);

/* Device pointer to `slot`'s page-table block [max_adapters][2*max_rank] and its row stride in
 * elements (2*max_rank).  Errors: LORA_EINVAL (slot out of range, bookkeeping-only pool). */
int lora_pool_page_table(const lora_pool *pool, int32_t slot, const int32_t **table,
                         int32_t *row_stride);

/* Copy adapter `adapter_id`'s page list (2 * rank * n_slots ids, in list order) into out[cap];
 * *n_out = its length, *rank_out = its rank, *users_out = its refcount (each may be NULL).
 * Errors: LORA_ENOENT, LORA_EINVAL (cap too small: *n_out still set). */
int lora_pool_adapter_pages(const lora_pool *pool, int32_t adapter_id, int64_t *out, int64_t cap,
                            int64_t *n_out, int32_t *rank_out, int32_t *users_out);

/* Copy request `request_id`'s KV page list into out[cap]; *n_out = its length.
 * Errors: LORA_ENOENT, LORA_EINVAL (cap too small). */
int lora_pool_kv_pages(const lora_pool *pool, int64_t request_id, int64_t *out, int64_t cap,
                       int64_t *n_out);

/* Copy the free list (front to end; allocation takes from the end) into out[cap]. */
int lora_pool_free_list(const lora_pool *pool, int64_t *out, int64_t cap, int64_t *n_out);

/* Resident adapter ids in load order (oldest first), the order idle eviction follows. */
int lora_pool_resident(const lora_pool *pool, int32_t *out, int32_t cap, int32_t *n_out);

/* ---- the projection --------------------------------------------------------------------------- */

/* Bytes of device workspace lora_project needs for T tokens on this pool (256-byte aligned). */
size_t lora_project_workspace_size(const lora_pool *pool, int64_t T);

/*
 * y = x W + s * (x A) B for T tokens, each on its own adapter (sections "Merge or keep adapters
 * separate" and "The architecture" of "S-LoRA, in depth").
 *   x            device [T][H], pool dtype, row-major, 16-byte aligned.
 *   W            device [H][H], pool dtype, OUT-MAJOR: element (k, n) of W (input k, output n)
 *                is W[n * H + k] -- the layout of a linear layer's weight matrix.  16-byte aligned.
 *   page_table   device: one slot's block [max_adapters][2*max_rank] (lora_pool_page_table).
 *   adapter_ids  device int32 [T]: adapter per token, -1 = none.
 *   ranks        device int32 [max_adapters]: rank per adapter; must equal the loaded rank for
 *                every adapter a token uses (entries of unused adapters are not read).
 *   scale        device float32 [max_adapters]: s per adapter.
 *   y            device [T][H], pool dtype, 16-byte aligned; must not overlap x.  Each element is
 *                accumulated in float32 (base and low-rank parts together) and rounded once to the
 *                pool dtype (round to nearest even).
 *   workspace    device, >= lora_project_workspace_size(pool, T) bytes, 256-byte aligned; its
 *                contents on entry do not matter.  Calls that share a workspace must be ordered
 *                (same stream, or events).
 * T == 0 is a no-op; T above LORA_MAX_TOKENS is LORA_EINVAL.  Ids, ranks and page ids are checked on the device: a token whose adapter id
 * is out of range, whose rank is out of range or differs from the page table, or whose page ids
 * are out of range gets the base product only, and the pool's device error word records the
 * fault; lora_check_device_errors() reports and clears it.
 * Errors (host-side, before any device work): LORA_EINVAL, LORA_EHIP.
 */
int lora_project(lora_pool *pool, const void *x, const void *W, const int32_t *page_table,
                 const int32_t *adapter_ids, const int32_t *ranks, const float *scale, int64_t T,
                 void *y, void *workspace, size_t workspace_bytes, void *stream);

#define LORA_MAX_CALL_SLOTS 4   /* most slots one lora_project_slots call takes                    */

/* Bytes of device workspace lora_project_slots needs for n slots and T tokens (0 if n is out of
 * range): n times lora_project_workspace_size. */
size_t lora_project_slots_workspace_size(const lora_pool *pool, int32_t n, int64_t T);

/*
 * The projection for n (1..LORA_MAX_CALL_SLOTS) slots that share the same tokens: the q, k and v
 * projections of a layer read one x ("S-LoRA, in depth": an adapter has A and B for each of the
 * projections of each layer, and the base product is batched over all tokens).  For each z < n,
 *     y[z][t] = x[t] W[z] + s[a] * (x[t] A_{slots[z],a}) B_{slots[z],a},    a = adapter_ids[t],
 * exactly what lora_project gives for that slot (bit for bit: every sum runs in the same order).
 * One call groups the tokens once and launches each stage once for all n slots, so the base
 * GEMM's tiles of the n slots share the chip (better load balance than n calls).
 *   slots        host int32 [n], distinct or not, each in [0, n_slots); page tables are the pool's
 *   W, y         host arrays of n device pointers, as lora_project's W and y; no two outputs may
 *                overlap each other or x
 *   workspace    >= lora_project_slots_workspace_size(pool, n, T) bytes, 256-byte aligned: n regions
 *                of lora_project_workspace_size(pool, T) bytes, region z for the z-th slot
 * The rest as lora_project.  Float32 pools run the slots one after another.
 * Errors (host-side, before any device work): LORA_EINVAL, LORA_EHIP.  Device checks as
 * lora_project, with one difference for T > 256 (the prefill path, whose grouping serves every
 * slot): an adapter whose page-table row is bad in any slot of the call gets the base product
 * only, in every slot of the call.
 */
int lora_project_slots(lora_pool *pool, int32_t n, const int32_t *slots, const void *x,
                       const void *const *W, const int32_t *adapter_ids, const int32_t *ranks,
                       const float *scale, int64_t T, void *const *y, void *workspace,
                       size_t workspace_bytes, void *stream);

/*
 * lora_project_slots where each slot reads its own input rows: x is a host array of n device
 * pointers (each as lora_project's x; slots may share one).  The q, k, v and o projections of a layer
 * act on the same tokens but o reads the attention output, not the layer input ("S-LoRA, in depth":
 * an adapter has A and B for each of the projections of each layer); with this call all four go in
 * one launch per stage, so their tiles share the chip.  For each z < n,
 *     y[z][t] = x[z][t] W[z] + s[a] * (x[z][t] A_{slots[z],a}) B_{slots[z],a},   a = adapter_ids[t],
 * bit for bit what lora_project gives for that slot.  No output may overlap any input or another
 * output.  Workspace, errors and device checks as lora_project_slots.
 */
int lora_project_slots_x(lora_pool *pool, int32_t n, const int32_t *slots, const void *const *x,
                         const void *const *W, const int32_t *adapter_ids, const int32_t *ranks,
                         const float *scale, int64_t T, void *const *y, void *workspace,
                         size_t workspace_bytes, void *stream);

/*
 * The projection with its own indices exposed ("S-LoRA, in depth", section "The architecture": the
 * gather fetches each request's A and B pages from wherever the pool placed them).  Runs exactly the
 * kernels lora_project runs for these arguments -- in instantiations that also record the indices
 * they use -- and writes y bit for bit as lora_project does.  In addition (device int32, caller-owned,
 * 4-byte aligned, filled with -1 by the call first):
 *   gather_out   [T][2*max_rank], input token order: entry j < r is the page whose A column the
 *                shrink multiplied into token t's v[j]; entry r + j the page whose B row the expand
 *                multiplied into token t's y; -1 elsewhere (no adapter, rank 0, past the rank).  An
 *                entry that two workgroups or kernels filled with different pages reads -2.
 *   order_out    [T][2], per sorted position q (the grouping the kernels consumed): the token at q
 *                and the adapter of its segment.  T <= 256 (bfloat16): every token, the ones with a
 *                low-rank term first, grouped by adapter (segments by ceil(r / 16) from 4 down to 1,
 *                then by first token), then the others with adapter -1.  Otherwise: positions
 *                [0, n) hold the n tokens with a low-rank term, grouped by adapter in adapter
 *                order; the rest stay (-1, -1).
 * Other arguments, checks and errors as lora_project.  For tests and debugging; not a fast path.
 */
int lora_debug_project(lora_pool *pool, const void *x, const void *W, const int32_t *page_table,
                       const int32_t *adapter_ids, const int32_t *ranks, const float *scale, int64_t T,
                       void *y, void *workspace, size_t workspace_bytes, int32_t *gather_out,
                       int32_t *order_out, void *stream);

/*
 * Page-table view of the gather (no projection): for every token t (input order) writes the table
 * entries its adapter owns into page_ids_out[t][0..2*max_rank) (device int32): entries 0..r-1 its A
 * columns, r..2r-1 its B rows, -1 elsewhere and for tokens with no adapter or rank 0.  Same inputs
 * and device checks as lora_project (an invalid token gets all -1).  Enqueued on `stream`.  The
 * pages the projection's kernels themselves read come from lora_debug_project.
 */
int lora_debug_gather(lora_pool *pool, const int32_t *page_table, const int32_t *adapter_ids,
                      const int32_t *ranks, int64_t T, int32_t *page_ids_out, void *stream);

/*
 * lora_project for callers that cannot allocate device memory: code under HIP graph capture, tight
 * serving loops, harnesses that forbid allocation.  No workspace argument: the call uses a scratch
 * array of LORA_NOALLOC_SCRATCH_MB MiB that the library holds on each GPU it runs on until the
 * process ends (its address is taken at pool creation).  It allocates nothing and writes y exactly as
 * lora_project does.  Calls that need more scratch than that (lora_project_workspace_size) are refused
 * with LORA_EINVAL before any device work: at H = 4096 every decode batch (T <= 256) and prefill
 * batches up to about 25k tokens fit.  Every call on a GPU shares that GPU's array: calls that overlap
 * on one GPU (several streams or threads without ordering between them) race and may produce wrong
 * results; order them.  Other arguments, checks and errors as lora_project.
 */
#define LORA_NOALLOC_SCRATCH_MB 32
int lora_project_noalloc(lora_pool *pool, const void *x, const void *W, const int32_t *page_table,
                         const int32_t *adapter_ids, const int32_t *ranks, const float *scale, int64_t T,
                         void *y, void *stream);

/* ---- the KV cache: writing it, reading it, thinning it out -------------------------------------- */

/*
 * "S-LoRA, in depth", section "Unified paging": KV cache and adapters share one pool; a token takes
 * one K and one V vector per layer.  The calls below put the K and V rows of new tokens into the
 * pages lora_pool_grow_kv handed out, attend over them, and thin a cache out by the attention its
 * tokens received, so that its pages go back to the free list the adapters also draw from.
 *
 * One call serves one layer (lora_kv_evict: several) and n_seq sequences.
 *   layout       how heads lie in a page (lora_kv_layout_t).
 *   table        device int32 [n_seq][2][max_pages], 4-byte aligned, caller-owned: row (b, 0) lists
 *                sequence b's K pages of this layer in token order, row (b, 1) its V pages.  Token t
 *                of a sequence is the (t % tokens_per_page)-th of the page in entry
 *                t / tokens_per_page; entries behind the last token's are not read.  Sequences may
 *                share pages (a common prefix).  lora_pool_grow_kv's ids come in (K, V) pairs, layer
 *                by layer: entry 2 l is layer l's K page, 2 l + 1 its V page.
 *   lens         device int32 [n_seq]: tokens of each sequence in the cache, the new ones included.
 *                0 = an unused row of a padded batch: nothing is written for it, its output is zero.
 *   q_start      device int32 [n_seq + 1]: sequence b's new tokens are the rows q_start[b] up to (not
 *                with) q_start[b + 1] of k, v, q and out, and the LAST tokens of its cache.  Rows
 *                outside every sequence (behind q_start[n_seq]) are neither read nor written.
 * Page ids, lengths and row ranges are checked on the device, as the projection's ids are: a page id
 * outside the pool hides its tokens (they are not written, and get no weight); a length that is
 * negative, above the capacity or below the number of new tokens counts as 0; a q_start range that
 * does not lie in [0, T] counts as empty.  Each is recorded in the pool's device error word
 * (lora_check_device_errors).
 * Pool dtype throughout (k, v, q, out); products are summed, and softmax statistics and scores held,
 * in float32.  Rows are `ld` elements apart (a column range of a wider matrix, such as the output of
 * one projection for q, k and v, is fine); every row starts on a 16-byte boundary.  What a call writes
 * may overlap nothing else that it is given, unless it says so below; rows count from the first one's
 * begin to the last one's end, with what lies between them.
 * Row counts up to LORA_MAX_TOKENS, n_seq up to LORA_MAX_SEQS, max_pages * tokens_per_page up to
 * LORA_MAX_KV_TOKENS, and n_seq times the longest length up to 2^34.  n_seq == 0 or no rows: nothing is done.
 */
#define LORA_MAX_SEQS 65535
#define LORA_MAX_KV_TOKENS (1 << 22)
#define LORA_MAX_TOKENS_PER_PAGE 256
#define LORA_MAX_HEADS 1024

typedef struct lora_kv_layout {
    int32_t n_heads;            /* query heads                                                  */
    int32_t n_kv_heads;         /* K/V heads; divides n_heads.  Query head h reads K/V head
                                   h / (n_heads / n_kv_heads)                                   */
    int32_t head_dim;           /* 64, 128 or 256                                               */
    int32_t tokens_per_page;    /* >= 1: tokens one page holds, one behind the other, each
                                   n_kv_heads * head_dim elements; what is left of the page's
                                   `hidden` elements stays unused                               */
} lora_kv_layout_t;

/*
 * Put the new tokens' K and V rows into their pages: token i of sequence b goes to position
 * lens[b] - (q_start[b + 1] - q_start[b]) + i.
 *   k, v         device [T][n_kv_heads * head_dim], rows ldk (ldv) elements apart; outside the pool's pages
 *   q_start      NULL: one new token per sequence (T == n_seq), as in a decode step
 * Two new tokens for one place (sequences that share the page they write) is the caller's error.
 * Errors: LORA_EINVAL, LORA_EHIP.
 */
int lora_kv_write(lora_pool *pool, const lora_kv_layout_t *layout, const void *k, int64_t ldk,
                  const void *v, int64_t ldv, const int32_t *table, int32_t max_pages,
                  const int32_t *q_start, const int32_t *lens, int32_t n_seq, int64_t T, void *stream);

/* Bytes of device workspace (256-byte aligned) lora_kv_attend needs; 0 if an argument is out of
 * range, or if neither this call nor a smaller one uses any.  with_scores: whether the call collects
 * scores.  Never less for more sequences or tokens, or with scores: a workspace of the largest call serves them all. */
size_t lora_kv_attend_workspace_size(const lora_pool *pool, const lora_kv_layout_t *layout,
                                     int32_t n_seq, int64_t max_len, int32_t with_scores);

/*
 * Attention of one new token per sequence over its cached tokens (the decode step), each head h with
 * its K/V head's vectors:
 *     p_t = softmax over t < lens[b] of (scale * q_h . k_t),   out_h = sum_t p_t v_t
 * The new token's own K and V are in the cache already (lora_kv_write first).
 *   q, out       device [n_seq][n_heads * head_dim], rows ldq (ldo) elements apart; row b belongs to
 *                sequence b; they may not overlap each other or the pool's pages
 *   max_len      no length in this call is above it (1 .. max_pages * tokens_per_page): the call's
 *                work is split, and its workspace sized, for it.  It fixes nothing else, so a
 *                captured call may be replayed with any lengths up to it.
 *   scores       device float32 [n_seq][max_pages * tokens_per_page] or NULL: scores[b][t] = prior[b][t]
 *                + the sum over the heads of p_t, for t < lens[b]; the other entries stay as they were
 *   prior        the same shape; NULL: zeros.  May be `scores` itself (accumulate in place); must not
 *                overlap it otherwise
 *   workspace    as lora_project's
 * The out element is rounded once from float32; bfloat16 pools: the weights enter the product with V
 * as the sum of two bfloat16 numbers, off by at most 2^-15 of themselves, or by 2^-126 of the row's largest where that
 * is more; a weight of zero stays zero.  Where every weight is zero (no token, or each product is -inf) the output is
 * zero.  Results do not change from call to call of the same shape.
 * Errors: LORA_EINVAL, LORA_EHIP.
 */
int lora_kv_attend(lora_pool *pool, const lora_kv_layout_t *layout, const void *q, int64_t ldq,
                   const int32_t *table, int32_t max_pages, const int32_t *lens, int32_t n_seq,
                   int64_t max_len, float scale, void *out, int64_t ldo, const float *prior,
                   float *scores, void *workspace, size_t workspace_bytes, void *stream);

/* As lora_kv_attend_workspace_size, for lora_kv_attend_chunk with T rows.  Never less for more rows,
 * sequences or tokens: a workspace of the largest call serves them all. */
size_t lora_kv_attend_chunk_workspace_size(const lora_pool *pool, const lora_kv_layout_t *layout,
                                           int32_t n_seq, int64_t T, int64_t max_len,
                                           int32_t with_scores);

/*
 * Attention of many new tokens per sequence (a prompt, or the next part of one) over its cached
 * tokens, causal: the new token at position p reads the tokens at positions 0 .. p.  A token's K and V
 * reach no row before it, whatever they hold (infinities and NaN included).
 *   q, out       device [T][n_heads * head_dim]; sequence b's rows as q_start says
 *   scores       as lora_kv_attend's, summed over the sequence's new tokens too
 * bfloat16 pools: the weights are rounded to bfloat16 for the product with V, off by at most 2^-8 of
 * themselves, the largest not at all (scores take them unrounded).  An infinite value whose weight is
 * zero makes a row NaN or that infinity.  The rest as lora_kv_attend.  Errors: LORA_EINVAL, LORA_EHIP.
 */
int lora_kv_attend_chunk(lora_pool *pool, const lora_kv_layout_t *layout, const void *q, int64_t ldq,
                         const int32_t *table, int32_t max_pages, const int32_t *q_start,
                         const int32_t *lens, int32_t n_seq, int64_t T, int64_t max_len, float scale,
                         void *out, int64_t ldo, const float *prior, float *scores, void *workspace,
                         size_t workspace_bytes, void *stream);

/*
 * Thin the caches of n_seq sequences out, in `layers` layers at once, to about `budget` tokens each:
 * in every layer the pages whose tokens received the least attention leave the table.  Only pages
 * that lie wholly in [keep_first, lens[b] - keep_last) can go (the first tokens and the latest ones
 * stay).  From a sequence go, in every layer,
 *     n_dropped[b] = min(max_drop, pages that can go, ceil((lens[b] - budget) / tokens_per_page)),
 * (0 if lens[b] <= budget): the ones with the lowest sums of their tokens' scores, added in token
 * order in float64; of equal sums the earlier page goes, and NaN counts as the highest.  The tokens that stay keep their
 * order: nothing is moved in the pages, the tables close up.
 *   table        device int32 [layers][n_seq][2][max_pages]; table_out the same shape: the entries
 *                that stay, -1 behind them.  It may be `table` itself (in place).
 *   scores       device float32 [layers][n_seq][max_pages * tokens_per_page]; scores_out the same: the scores of
 *                the tokens that stay, 0 behind them.  It may be `scores` itself.
 *   lens_out     device int32 [n_seq]: lens[b] - n_dropped[b] * tokens_per_page; must not be `lens`
 *   dropped      device int32 [layers][n_seq][2][max_drop]: the K and V pages that left, in token
 *                order, -1 behind them; copy them to the host and give them to lora_pool_drop_kv
 *   n_dropped    device int32 [n_seq]
 * A sequence whose length is out of range is recorded as above and left as it is.  The
 * table's entries are not checked here.  Errors: LORA_EINVAL, LORA_EHIP.
 */
int lora_kv_evict(lora_pool *pool, const lora_kv_layout_t *layout, int32_t layers, int32_t n_seq,
                  const int32_t *table, int32_t *table_out, int32_t max_pages, const float *scores,
                  float *scores_out, const int32_t *lens, int32_t *lens_out, int32_t budget,
                  int32_t keep_first, int32_t keep_last, int32_t *dropped, int32_t max_drop,
                  int32_t *n_dropped, void *stream);

/* Give `n` of request `request_id`'s KV pages back: they leave its page list (the others keep their
 * order) and go to the end of the free list in the order given.  page_ids: host int64 [n].  All or
 * none: a page that the request does not hold, or that is named twice, is LORA_EINVAL.  A request
 * without pages stays known until lora_pool_free_kv.  The caller must not give back pages that
 * queued, unfinished work still reads.  Errors: LORA_ENOENT, LORA_EINVAL. */
int lora_pool_drop_kv(lora_pool *pool, int64_t request_id, const int64_t *page_ids, int64_t n);

/* ---- steps of drafted tokens: planned, written, attended and accepted on the GPU ------------------ */

/*
 * A step of speculative decoding: each sequence gets a few drafted tokens, a tree of them, the model takes them all at
 * once, and the path that it agrees with stays.  The calls above serve a step whose lengths the host knows; here the
 * lengths, the page tables and the free pages live on the GPU, so that a step follows another without the host:
 *     lora_kv_plan        rows, pages, slots, positions and masks of the step, from each sequence's new tokens
 *     lora_kv_write_rope  per layer: q and k turned by the positions, K and V to their slots
 *     lora_kv_attend_tree per layer: attention of the tree's nodes (lora_kv_attend[_chunk] serve steps without trees)
 *     lora_kv_accept      the agreed path, its K and V closed up in every layer, the new lengths
 * A sequence's m new tokens are the nodes 0 .. m - 1 of its tree, in the order of its rows; node 0 is the root (the token
 * chosen last), and parents[row] names each other node's parent, a node before it in the same sequence.
 * table, lens, q_start, rows and errors as above.  Every buffer is the caller's, on the pool's device.
 */
#define LORA_MAX_TREE 256       /* new tokens of a sequence in a step with trees */

/*
 * Plan a step.  Sequence b, which holds lens[b] tokens in held[b] pages a layer, gets counts[b] >= 0 new ones:
 *   rows       q_start: prefix sums of the counts; step_lens[b]: its length with the new ones, 0 where counts[b] is 0 or
 *              the sequence is refused (the calls of the step then leave it alone, its output is zero)
 *   pages      it holds ceil(length / tokens_per_page) pages of each layer's K and V afterwards.  What it lacks comes from
 *              the stock, what it has too much (lens[b] shrunk since the last plan) goes back there, behind what can be
 *              taken in this call: a finished request is lens[b] = 0, counts[b] = 0
 *   slots      [layers][2][T]: where each row's K and V go: page * tokens_per_page + place in the page; -1 for rows of
 *              refused sequences and rows behind the last
 *   positions  [T]: the row's place in its sequence, or, with parents, lens[b] + its depth in the tree; 0 where slots are -1
 *   mask       [T][(max_nodes + 63) / 64]: bit j of word j / 64: the row sees its sequence's node j (itself and the nodes it
 *              descends from); 0 where slots are -1.  parents and mask are both given or both NULL
 *   table      device int32 [layers][n_seq][2][max_pages], as lora_kv_evict's: entries of pages that come are written; those
 *              of pages that went stay behind the last token's, unread
 *   stock      device int32 [stock_groups][layers][2]: a ring of page groups, one page of each layer's K and V (what
 *              lora_pool_grow_kv hands out).  It has room for every group that exists, free or held
 *   state      device int32 [4]: first free group's place in the ring; free groups; sequences that this call refused
 *              although they have new tokens (state_out alone); 0 (the call counts its workgroups there)
 * Sequences are served in order: the first that the free groups do not suffice for, and every later one that needs any, is
 * refused: its length and pages stay.  So is one that would grow over max_len (recorded in the error word, as are counts
 * below 0, over T or, with parents, over max_nodes, which count as 0; lengths over max_len or not covered by held; rows
 * behind T; a parent that is no earlier node, where the walk to the root ends; page ids outside the pool, whose slots
 * are -1).  No page is taken or given twice as long as held, table, stock and state come from one another.
 * lens_out [n_seq], held_out [n_seq] and state_out [4] may be lens, held and state themselves.  T == 0 plans a step without
 * rows (pages may go back), n_seq == 0 one without sequences: every slot is -1, q_start is 0.  Errors: LORA_EINVAL, LORA_EHIP.
 */
int lora_kv_plan(lora_pool *pool, const lora_kv_layout_t *layout, int32_t layers, int32_t n_seq, const int32_t *counts,
                 const int32_t *lens, const int32_t *held, int32_t *table, int32_t max_pages, int64_t max_len,
                 int32_t *stock, int32_t stock_groups, int32_t *state, int64_t T, const int32_t *parents,
                 int32_t max_nodes, int32_t *step_lens, int32_t *q_start, int64_t *slots, int32_t *positions,
                 uint64_t *mask, int32_t *lens_out, int32_t *held_out, int32_t *state_out, void *stream);

#define LORA_ROPE_HALVES 0      /* element i of the part that turns pairs with element i + rot_dim / 2 */
#define LORA_ROPE_NEIGHBOURS 1  /* element 2 i pairs with element 2 i + 1                              */

typedef struct lora_rope {
    const float *table;         /* device [n_positions][rot_dim / 2][2], 16-byte aligned: cosine and sine of each pair's angle */
    int32_t n_positions;
    int32_t rot_dim;            /* a head's first rot_dim elements turn, the rest stay: a multiple of 16 up to head_dim */
    int32_t pairing;            /* LORA_ROPE_HALVES or LORA_ROPE_NEIGHBOURS */
} lora_rope_t;

/*
 * One layer's rows of a step: each pair (a, b) of a q or k head becomes (a c - b s, a s + b c), c and s from the table's
 * row positions[t], in float32 and rounded once; k and v go to their slots, q to q_out.
 *   q, q_out     device [T][n_heads * head_dim], rows ldq (ldqo) elements apart; both NULL: k and v alone.  q_out may be q
 *                (and ldqo ldq), and q, k and v may be column ranges of one matrix; it overlaps nothing else
 *   k, v         device [T][n_kv_heads * head_dim], rows ldk (ldv) elements apart; outside the pool's pages
 *   slots        device int64 [2][T], 8-byte aligned: one layer of lora_kv_plan's
 *   positions    device int32 [T]
 * A row whose two slots are negative is left alone (q_out too).  So is one with one negative slot, a slot outside the pool
 * or a position outside the table, and it is recorded in the pool's error word.  Two rows for one slot are the caller's
 * error.  Errors: LORA_EINVAL, LORA_EHIP.
 */
int lora_kv_write_rope(lora_pool *pool, const lora_kv_layout_t *layout, const lora_rope_t *rope, const void *q, int64_t ldq,
                       void *q_out, int64_t ldqo, const void *k, int64_t ldk, const void *v, int64_t ldv,
                       const int64_t *slots, const int32_t *positions, int64_t T, void *stream);

/* As lora_kv_attend_workspace_size, for lora_kv_attend_tree.  Never less for more sequences, nodes or tokens. */
size_t lora_kv_attend_tree_workspace_size(const lora_pool *pool, const lora_kv_layout_t *layout, int32_t n_seq,
                                          int32_t max_nodes, int64_t max_len);

/*
 * Attention of trees of new tokens: node i of a sequence reads the tokens cached before its tree, and the nodes whose bits
 * its mask row has (its own among them, if it is to read itself), whatever any other token's K and V hold.
 *   q, out       device [T][n_heads * head_dim]; sequence b's rows as q_start says
 *   mask         device uint64 [T][(max_nodes + 63) / 64], as lora_kv_plan writes it; any other set of nodes will do.
 *                Bits of nodes that a sequence does not have are not looked at
 *   max_nodes    no sequence has more new tokens (1 .. LORA_MAX_TREE): one that does counts as empty, and is recorded
 * A row that sees nothing comes out as zero.  bfloat16 pools: the weights enter the product with V as lora_kv_attend's.  An
 * infinite value of a node whose weight is zero makes a row that sees it NaN or that infinity.  The rest as lora_kv_attend.
 * Errors: LORA_EINVAL, LORA_EHIP.
 */
int lora_kv_attend_tree(lora_pool *pool, const lora_kv_layout_t *layout, const void *q, int64_t ldq,
                        const int32_t *table, int32_t max_pages, const int32_t *q_start, const int32_t *lens,
                        int32_t n_seq, int64_t T, const uint64_t *mask, int32_t max_nodes, int64_t max_len, float scale,
                        void *out, int64_t ldo, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Keep the drafted tokens that the model agrees with.  tokens[row] is the token a node stands for, targets[row] the one
 * the model chose behind it.  The path starts at node 0; from node i it goes on to the first child of i whose token is
 * targets[i].  Node path[k]'s K and V move to place k of the tree, in `layers` layers, and the rest of the tree leaves.
 *   table        device int32 [layers][n_seq][2][max_pages]; lens, q_start: the step's (step_lens)
 *   lens_out     device int32 [n_seq]: the tokens before the tree and the path's; of sequences without new tokens or with a
 *                length of 0 the entry stays as it was.  Must not be lens (it may be what lora_kv_plan next takes as lens)
 *   path         device int32 [n_seq][max_nodes]: the path's nodes, -1 behind them; n_path [n_seq]: how many, 0 for
 *                sequences without new tokens
 *   next         device int32 [n_seq]: targets of the path's last node: the next tree's root; -1 where the path is empty
 * Pages that hold moved tokens belong to one sequence alone.  A token on a bad page does not move, and is recorded; a
 * parent that is no earlier node makes its node nobody's child.  A step's path is kept once: a second call would move what
 * has moved.  T == 0: every path is empty; tokens, targets and parents may be NULL.  Errors: LORA_EINVAL, LORA_EHIP.
 */
int lora_kv_accept(lora_pool *pool, const lora_kv_layout_t *layout, int32_t layers, int32_t n_seq, const int32_t *table,
                   int32_t max_pages, const int32_t *q_start, const int32_t *lens, int64_t T, const int32_t *tokens,
                   const int32_t *targets, const int32_t *parents, int32_t max_nodes, int32_t *lens_out, int32_t *path,
                   int32_t *n_path, int32_t *next, void *stream);

/* Wait for all device work, then report and clear the pool's device error word:
 * LORA_OK, or LORA_EDEVICE with a message naming the kinds of fault seen. */
int lora_check_device_errors(lora_pool *pool);

/* ---- per-kernel timing (opt-in, for measurement) ---------------------------------------------- */

typedef struct lora_profile {
    int64_t calls;              /* projections recorded                                          */
    double ms_group;            /* summed device time of the token-grouping kernel (prefill and
                                   float32 paths; the decode path groups inside its first kernel) */
    double ms_first;            /* ... of the first compute launch: decode = shrink + base GEMM
                                   partials; prefill and float32 = shrink                          */
    double ms_second;           /* ... of the second: decode = partial sum + expand + rounding;
                                   prefill and float32 = base GEMM + fused expand                  */
} lora_profile_t;

/* Start recording HIP events around each kernel of the next `max_calls` projections on this
 * pool, on the stream each kernel is launched on.  Recording adds event records between the
 * kernels; time the throughput without it.  Errors: LORA_EINVAL, LORA_EHIP. */
int lora_profile_start(lora_pool *pool, int32_t max_calls);

/* Wait for the recorded work, fill *out with per-kernel sums, and stop recording. */
int lora_profile_stop(lora_pool *pool, lora_profile_t *out);

/* Message for the calling thread's last error ("" if none). */
const char *lora_last_error(void);

/* Library version string. */
const char *lora_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LORAPOOL_H */

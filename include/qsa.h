/*
 * qsa.h -- C ABI of libqsa.so: selected-cell (QSA union) prompt attention over a
 * paged INT8 KV cache, on GB300 (sm_103a).
 *
 * Source: "sycl: prompt attention over 8-query selection unions on XMX" (Strata
 * PR #2808).  Section Summary: every prompt position attends only to its own
 * sorted selection of at most 2,051 K/V cells; for every 8 neighbouring
 * positions a first kernel builds the sorted union of their selections with each
 * cell marked by the positions that chose it, and a second kernel dequantises the
 * INT8 K/V of 64-cell chunks of that union once and runs S = Q K^T and O += P V
 * for all 96 rows (8 positions x 12 heads) with FP32 sums, setting a cell to
 * -inf for the positions that did not select it.  Section Extra Notes: a union
 * cell is an int32 with its 8-position mask in a separate byte; non-resident
 * pages are masked.  Section "What changed": the entry point carries the prompt
 * attention contract (query, paged K/V and scales, page table, per-position
 * selection lists and counts).
 *
 * Conventions shared by every entry point below
 *   - Device pointers point to CUDA global memory of the current device; host
 *     pointers are marked "host".  The caller owns all memory; the library
 *     allocates nothing, keeps no state between calls and never synchronises.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *     stream).  Work is enqueued on it; the call returns before it runs.
 *   - Shapes are fixed by the method: head dim d = 128, 12 query heads per KV
 *     head, 64-cell pages, groups of 8 consecutive queries starting at query 0
 *     (the last group may be ragged).
 *   - Layouts (row-major, no padding unless a stride is given):
 *       q          bf16  [n_q][n_kv*12][128]
 *       k_pool     int8  [n_ppages][n_kv][64][128]      (one KV head's page = 8 KB)
 *       v_pool     int8  [n_ppages][n_kv][64][128]
 *       k_scale    fp16  [n_ppages][n_kv][64]           per-cell per-KV-head scale
 *       v_scale    fp16  [n_ppages][n_kv][64]
 *       page_table int32 [n_lpages]   physical page of logical page c>>6; < 0 = not resident
 *       sel        int32 [n_q][sel_stride]   strictly increasing cell ids >= 0
 *       sel_count  int32 [n_q]               0 <= count <= sel_stride
 *       union_cells int32 [n_groups][union_stride], union_mask uint8 [..], union_count int32 [n_groups]
 *       out        fp32  [n_q][n_kv*12][128]
 *     with n_groups = ceil(n_q / 8).  K/V value of cell c for KV head h is
 *     int8 * scale at [page_table[c>>6]][h][c&63]; query head i uses KV head i/12.
 *   - bf16 / fp16 tensors are passed as uint16_t bit patterns.
 *   - Pointers to q, k_pool, v_pool and out must be 16-byte aligned.
 *   - Errors: a non-zero qsa_status is returned before anything is enqueued when
 *     an argument is invalid; QSA_ERR_CUDA reports a launch failure.  Problems that
 *     only the device can see (a bad count, cell or page-table entry, a union that
 *     does not fit, a device wait that ran out) never cause an out-of-bounds
 *     access: the offending cell is masked or the count clamped, and the matching
 *     QSA_DEV_* bit is OR-ed into *dev_status when dev_status is not NULL.
 */
#ifndef QSA_H
#define QSA_H
#include <stddef.h>
#include <stdint.h>
#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    QSA_OK = 0,
    QSA_ERR_ARG = 1,          /* null pointer, negative size, bad alignment or stride */
    QSA_ERR_UNSUPPORTED = 2,  /* shape outside what the kernels are built for */
    QSA_ERR_CAPACITY = 3,     /* workspace too small */
    QSA_ERR_CUDA = 4,         /* a CUDA launch or device query failed */
    QSA_ERR_DEVICE_CHECK = 5  /* reserved for callers decoding *dev_status */
} qsa_status;

/* Bits OR-ed into the optional device status word (int32 in device memory). */
enum {
    QSA_DEV_BAD_SEL_COUNT = 1,     /* a selection count outside [0, sel_stride] (clamped) */
    QSA_DEV_UNION_OVERFLOW = 2,    /* a union longer than union_stride (truncated) */
    QSA_DEV_BAD_CELL = 4,          /* a cell < 0 or on a page >= n_lpages (masked) */
    QSA_DEV_BAD_PAGE = 8,          /* a page-table entry >= n_ppages (masked) */
    QSA_DEV_BAD_UNION_COUNT = 16,  /* a union count outside [0, union_stride] (clamped) */
    QSA_DEV_WAIT_TIMEOUT = 32,     /* a pipelined kernel gave up waiting; its output is invalid */
    QSA_DEV_BAD_SEQ_LEN = 64,      /* a length that is negative or longer than its page table (clamped) */
    QSA_DEV_NO_PAGE = 128,         /* the free list ran out, or a token's page is not resident (slot -1) */
    QSA_DEV_TOKEN_OVERFLOW = 256,  /* more new tokens than the token arrays hold (the rest is not mapped) */
    QSA_DEV_BAD_AXIS = 512,        /* a pair's axis outside [0, n_axes) (axis 0 is used) */
    QSA_DEV_BAD_STATE = 1024       /* a state slot past the pool (its sequence is left out) */
};

/* Element types of the 16- and 32-bit tensors that more than one type is allowed for. */
enum {
    QSA_BF16 = 0,
    QSA_F16 = 1,
    QSA_F32 = 2
};

/* Attention kernel variants (all sm_103a).  QSA_ATTN_DEFAULT picks the fastest. */
enum {
    QSA_ATTN_DEFAULT = 0,
    QSA_ATTN_TCGEN05 = 1,   /* tcgen05.mma with TMEM accumulators, warp-specialised pipeline,
                               one CTA per (group, KV head), 64-cell chunks, two CTAs per SM */
    QSA_ATTN_TCGEN05_SM = 2 /* tcgen05, one CTA per (group, KV head) and per SM: Q, an O per
                               softmax set and three S/P buffers in TMEM, two softmax warp sets
                               on alternating chunks, combined at the end (the kernel
                               qsa_fused_attn runs with the union built in-CTA) */
};

/* The variant QSA_ATTN_DEFAULT resolves to in this build (one of the values above). */
int qsa_attn_default_variant(void);

/* Human-readable name of a qsa_status value.  Never NULL. */
const char* qsa_status_str(int status);

/* Bytes of one workspace holding the union arrays for n_q queries:
 * union_cells, then union_mask, then union_count, each 256-byte aligned.
 * Returns 0 for n_q < 0 or union_stride <= 0. */
size_t qsa_union_workspace_bytes(int32_t n_q, int32_t union_stride);

/* Union build (first kernel).  Defined by "sycl: prompt attention over 8-query
 * selection unions on XMX" (Strata PR #2808), section Summary (the sorted union of
 * 8 neighbouring positions' selections, each cell marked by the positions that
 * chose it) and section Extra Notes (a union cell is an int32 with its 8-position
 * mask in a separate byte).  For each group g of up to 8 consecutive queries:
 * union_cells[g][0:union_count[g]] = the sorted set union of their selection lists,
 * union_mask[g][u] bit j = query 8g+j selected union_cells[g][u] (bits of absent
 * ragged queries are 0).  Entries past union_count[g] are left unspecified.
 * Bit-exact and deterministic (no order-dependent atomics).
 * Requires union_stride % 64 == 0 and sel_stride >= 1; union_stride >= 8*sel_stride
 * guarantees that every union fits.  n_q == 0 returns QSA_OK with no launch. */
int qsa_union_build(const int32_t* sel, const int32_t* sel_count, int32_t n_q, int32_t sel_stride,
                    int32_t* union_cells, uint8_t* union_mask, int32_t* union_count,
                    int32_t union_stride, int32_t* dev_status, void* stream);

/* Union attention (second kernel).  Defined by "sycl: prompt attention over
 * 8-query selection unions on XMX" (Strata PR #2808), section Summary: for
 * query i (group g = i/8, j = i%8) and query head hq, out[i][hq][:] = sum over
 * union cells c with bit j of the mask set and a resident page of
 * softmax(q . k_c * sm_scale) * v_c, with k_c, v_c the dequantised K/V of KV
 * head hq/12; zeros when no such cell exists (our reading for the empty case).
 * One CTA per (group, KV head) covers 96 rows; K/V chunks of 64 union cells are
 * gathered through the page table and dequantised once.  Both variants compute
 * S = Q K^T on FP16 operands (Q converted from BF16, exact, with an exact
 * power-of-two row scale for rows outside FP16's comfortable range; K as the
 * exact INT8 integers, its scale applied to the score column in FP32) and
 * O += P V with FP32 accumulation (QSA_ATTN_TCGEN05: P = p * v_scale rounded to
 * BF16 against exact BF16 V; QSA_ATTN_TCGEN05_SM: P rounded to FP16 against exact
 * FP16 V, the V scale carried by a per-chunk power of two).  Typically
 * sm_scale = 1/sqrt(128).  `variant` is one of the QSA_ATTN_* values.
 * n_q == 0 returns QSA_OK. */
int qsa_union_attn(const uint16_t* q, const int8_t* k_pool, const int8_t* v_pool,
                   const uint16_t* k_scale, const uint16_t* v_scale,
                   const int32_t* page_table, int32_t n_lpages, int32_t n_ppages, int32_t n_kv,
                   const int32_t* union_cells, const uint8_t* union_mask, const int32_t* union_count,
                   int32_t union_stride, int32_t n_q, float sm_scale, float* out,
                   int32_t variant, int32_t* dev_status, void* stream);

/* Whole prompt-attention step: qsa_union_build into `workspace` (device memory
 * of at least qsa_union_workspace_bytes(n_q, union_stride) bytes, 256-byte
 * aligned, owned by the caller) followed by qsa_union_attn, both on `stream`.
 * Returns QSA_ERR_CAPACITY when workspace_bytes is too small. */
int qsa_prompt_attn(const uint16_t* q, const int8_t* k_pool, const int8_t* v_pool,
                    const uint16_t* k_scale, const uint16_t* v_scale,
                    const int32_t* page_table, int32_t n_lpages, int32_t n_ppages, int32_t n_kv,
                    const int32_t* sel, const int32_t* sel_count, int32_t sel_stride, int32_t n_q,
                    float sm_scale, float* out, void* workspace, size_t workspace_bytes,
                    int32_t union_stride, int32_t variant, int32_t* dev_status, void* stream);

/* The whole prompt-attention step in one launch, with each group's union built
 * inside the attention CTA ("sycl: prompt attention over 8-query selection unions
 * on XMX", Strata PR #2808, section Summary: the union of 8 neighbouring
 * positions' sorted selections; section What changed: there the union and the
 * attention run as a launch pair).  No union arrays reach global memory and no
 * workspace is needed.  The result is that of qsa_prompt_attn with
 * variant = QSA_ATTN_TCGEN05_SM, bit for bit: each CTA first builds its group's
 * union in shared memory with the union kernel's own algorithm, then runs that
 * variant's attention pipeline on it.
 *   - Arguments and layouts are those of qsa_prompt_attn without the workspace,
 *     union stride and variant.  Lists must be strictly increasing (the union
 *     build's precondition); counts outside [0, sel_stride] are clamped and
 *     reported as QSA_DEV_BAD_SEL_COUNT.  Device checks as in qsa_union_attn.
 *   - The union of 8 lists (up to 8 x sel_stride entries, 5 bytes each) must fit
 *     the CTA's shared memory next to the pipeline's (sm_103's per-block limit
 *     of 227 KB): sel_stride up to about 2,800 (2,056 holds the method's
 *     2,051-cell cap); QSA_ERR_UNSUPPORTED, before any CUDA call, above that,
 *     and for more than 65,535 groups (n_q > 524,280).
 *   - n_q == 0 returns QSA_OK with no launch. */
int qsa_fused_attn(const uint16_t* q, const int8_t* k_pool, const int8_t* v_pool,
                   const uint16_t* k_scale, const uint16_t* v_scale,
                   const int32_t* page_table, int32_t n_lpages, int32_t n_ppages, int32_t n_kv,
                   const int32_t* sel, const int32_t* sel_count, int32_t sel_stride, int32_t n_q,
                   float sm_scale, float* out, int32_t* dev_status, void* stream);

/* Per-position selected-cell attention without unions: out[i][hq][:] is the same
 * softmax over query i's own resident selected cells as qsa_union_attn computes,
 * but every position gathers its own cells ("sycl: prompt attention over 8-query
 * selection unions on XMX", Strata PR #2808, section Summary: the prompt path's
 * default, each position gathering its own ~2,051 cells; section Extra Notes
 * times it against the union kernel).  It is the baseline the union path
 * replaces, built on the warp-level tensor path (mma.sync, FP32 sums): S on FP16
 * operands (Q converted from BF16 with the union kernel's exact power-of-two row
 * scaling, K as the exact INT8 integers, its scale on the score column in FP32),
 * P V on BF16 operands (V exact, P = p * v_scale rounded to BF16 once).  Each
 * (query, KV head) list is split
 * over four warps whose partial softmax states are merged at the end, so the
 * summation order differs from a single walk of the list (results agree within
 * BF16 rounding of the weights).  Arguments and layouts are those of
 * qsa_prompt_attn (sel: [n_q][sel_stride] cells, sel_count: [n_q]); no workspace.
 * The lists need not be sorted.  Device checks as in qsa_union_attn
 * (QSA_DEV_BAD_SEL_COUNT, QSA_DEV_BAD_CELL, QSA_DEV_BAD_PAGE into *dev_status).
 * n_q == 0 returns QSA_OK with no launch. */
int qsa_select_attn(const uint16_t* q, const int8_t* k_pool, const int8_t* v_pool,
                    const uint16_t* k_scale, const uint16_t* v_scale,
                    const int32_t* page_table, int32_t n_lpages, int32_t n_ppages, int32_t n_kv,
                    const int32_t* sel, const int32_t* sel_count, int32_t sel_stride, int32_t n_q,
                    float sm_scale, float* out, int32_t* dev_status, void* stream);

/* Decode-time selected-cell attention over a batch of sequences: query i is the
 * current position of sequence i and attends to its own selected cells through
 * its own page table.  The union pages leave decode untouched ("sycl: prompt
 * attention over 8-query selection unions on XMX", Strata PR #2808, section
 * Summary: the decode kernel gathers each position's own cells); this is that
 * computation -- the softmax of qsa_select_attn, per query -- with one page table
 * per query instead of one for the whole chunk.
 *   - q: [n_q][n_kv*12][128] BF16; out: [n_q][n_kv*12][128] FP32, written for
 *     every query (zeros when no selected cell is resident).
 *   - page_tables: query i's table is page_tables[i * pt_stride ...], n_lpages
 *     entries (logical page -> physical page in the shared pools, < 0 = not
 *     resident).  pt_stride == 0 gives every query one shared table (then this
 *     is qsa_select_attn); otherwise pt_stride >= n_lpages.
 *   - Pools, scales, sel / sel_count / sel_stride, sm_scale, dev_status and
 *     stream as in qsa_select_attn; lists need not be sorted.
 *   - Returns QSA_ERR_ARG for a negative pt_stride or 0 < pt_stride < n_lpages,
 *     otherwise as qsa_select_attn.  n_q == 0 returns QSA_OK with no launch. */
int qsa_decode_attn(const uint16_t* q, const int8_t* k_pool, const int8_t* v_pool,
                    const uint16_t* k_scale, const uint16_t* v_scale,
                    const int32_t* page_tables, int32_t pt_stride, int32_t n_lpages, int32_t n_ppages,
                    int32_t n_kv, const int32_t* sel, const int32_t* sel_count, int32_t sel_stride,
                    int32_t n_q, float sm_scale, float* out, int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * Serving a cache: the operators around the paged INT8 cache that the attention
 * calls above read.  None of them is part of the selected-cell method; they use
 * its cache (pools, scales, page tables, 64-cell pages, d = 128, non-resident
 * pages masked) and its conventions.  A step of a serving loop is
 *     qsa_extend_tables -> qsa_rope_append -> qsa_paged_attn or qsa_decode_attn
 * on one stream, with nothing read back by the host in between.  Here the query
 * heads of a KV head are n_heads / n_kv, any whole number (not only 12).
 * Scale arrays, like pools, must be 16-byte aligned; a pool whose rows (n_ppages *
 * n_kv * 64) exceed 2^31 - 64 is QSA_ERR_UNSUPPORTED.
 * ------------------------------------------------------------------------ */

/* Attention of one new token per sequence over its whole paged cache: for
 * sequence s and query head i, with n = seq_lens[s] and KV head i / (n_heads / n_kv),
 *     out[s][i][:] = sum over cells c of softmax(q . k_c * sm_scale) * v_c,
 * c running over the cells max(0, n - window) .. n-1 (window = 0: over 0 .. n-1)
 * whose page is resident.  Zeros when no such cell exists.  Where lse is not
 * NULL, lse[s][i] = log(sum over the same cells of exp(q . k_c * sm_scale)),
 * natural logarithm, -infinity when no such cell exists.
 *   - q: [n_seq][n_heads][128] of q_type (QSA_BF16 or QSA_F16); out: the same
 *     shape of out_type (QSA_BF16, QSA_F16 or QSA_F32); lse: FP32 [n_seq][n_heads].
 *     n_heads is a multiple of n_kv.  out and lse must not overlap an input.
 *   - page_tables: sequence s's table is page_tables[s * pt_stride ...], n_lpages
 *     entries; pt_stride == 0 gives every sequence one shared table, otherwise
 *     pt_stride >= n_lpages.  Entries past the sequence's last cell, and cells
 *     outside the window, are never read; nor are the contents of cells past n in
 *     the last page used (they may hold anything).
 *   - A length outside [0, n_lpages * 64] is clamped and reported
 *     (QSA_DEV_BAD_SEQ_LEN); an entry >= n_ppages is masked and reported
 *     (QSA_DEV_BAD_PAGE).
 *   - Only the device knows the lengths; the kernels are chosen by n_seq, the head counts
 *     and n_lpages.  A batch of a few short sequences is fastest when n_lpages is no
 *     larger than they need, whatever the tables' width pt_stride (one sequence of
 *     1,021 cells: 6.9 us with 16, 11.1 with 512).
 *   - The cache's length is split over the GPU and the parts joined in a fixed
 *     order: the same call gives the same bits.
 *   - Scores: Q rounded to FP16 after an exact power-of-two scaling of each row
 *     (exact for elements within 2^26 of the row's largest), K as the exact
 *     INT8 integers, FP32 sums (of q (k + 128), from -128 times the sum of q).
 *     Weights times V scales are rounded to FP16 once (relative 2^-11, whatever the
 *     type of out; a power of two per row keeps them in FP16's range, and what is
 *     below 2^-32 of the row's largest product, or 2^-78 of its largest weight, loses
 *     bits), V exact, FP32 sums.
 *   - workspace: device memory of at least qsa_paged_attn_workspace_bytes(n_kv,
 *     n_heads) bytes, 256-byte aligned; its contents need not be set and are
 *     not kept.  Two calls that can overlap on the device need one each.
 *   - QSA_ERR_UNSUPPORTED when n_seq * (n_lpages + 1) * n_kv * ceil(n_heads / n_kv /
 *     16) exceeds 2^30; QSA_ERR_CAPACITY for too small a workspace.  n_seq == 0 returns QSA_OK with no launch. */
int qsa_paged_attn(const void* q, int32_t q_type, const int8_t* k_pool, const int8_t* v_pool,
                   const uint16_t* k_scale, const uint16_t* v_scale, const int32_t* page_tables,
                   int32_t pt_stride, int32_t n_lpages, int32_t n_ppages, int32_t n_kv, int32_t n_heads,
                   const int32_t* seq_lens, int32_t n_seq, int32_t window, float sm_scale,
                   void* out, int32_t out_type, float* lse, void* workspace, size_t workspace_bytes,
                   int32_t* dev_status, void* stream);

/* Workspace of qsa_paged_attn (independent of lengths and of n_seq); 0 for
 * n_kv <= 0 or n_heads not a positive multiple of n_kv. */
size_t qsa_paged_attn_workspace_bytes(int32_t n_kv, int32_t n_heads);

/* Rotary positions, and the cache's write.  For each of n_tok tokens: pair j of
 * every query and key head is turned by the angle positions[pair_axis[j]][t] *
 * inv_freq[j] (radians), (a, b) -> (a cos - b sin, b cos + a sin); then each key
 * and value row is quantised and written to the cell slots[t].
 *   - q: [n_tok][n_heads][128], k, v: [n_tok][n_kv][128] of `type` (QSA_BF16 or
 *     QSA_F16), tokens q_stride, k_stride, v_stride elements apart (multiples of
 *     8; slices of one projection's output), 16-byte aligned.  q may be NULL
 *     (then q_out is not written).
 *   - positions: int32 [n_axes][pos_stride], pos_stride >= n_tok, n_axes 1 to 4
 *     (time, height, width, ...); any int32 value.  inv_freq: FP64 [n_pairs],
 *     finite.  pair_axis: int32 [n_pairs] or NULL (every pair on axis 0).
 *     n_pairs is a multiple of 8 up to 64, or 0 for no rotation at all (then the
 *     three pointers may be NULL).  Pair j is dims (j, j + n_pairs), or (2j, 2j + 1)
 *     when interleaved; dims from 2 n_pairs on pass through.  The angle is formed
 *     as a 64-bit fixed-point fraction of a turn, so positions far out lose nothing.
 *   - q_out: as q, q_out_stride elements between tokens; the rotated queries,
 *     rounded once.  q_out == q with equal strides is allowed; otherwise q_out
 *     must not overlap an input.
 *   - Rotated keys are quantised from FP32, not rounded to 16 bits before.  A
 *     row's scale is max |x| / 127 rounded up to FP16 (at most 65504), its
 *     integers round(x / scale), ties to even, within [-127, 127].  A row that
 *     holds an infinity or NaN gets a NaN scale.
 *   - slots: int32 [n_tok], physical cell (page * 64 + cell of the page) or < 0:
 *     the token is not written.  A slot past the pool is not written and
 *     reported (QSA_DEV_BAD_CELL).  Slots >= 0 must be distinct: two tokens of one
 *     call with the same slot leave that cell a mixture of the two.
 *   - Nothing but the named cells and q_out is written.  n_tok == 0 returns QSA_OK. */
int qsa_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                    int64_t v_stride, int32_t type, const int32_t* positions, int32_t n_axes, int32_t pos_stride,
                    const double* inv_freq, const int32_t* pair_axis, int32_t n_pairs, int32_t interleaved,
                    void* q_out, int64_t q_out_stride, int8_t* k_pool, int8_t* v_pool, uint16_t* k_scale,
                    uint16_t* v_scale, const int32_t* slots, int32_t n_ppages, int32_t n_heads, int32_t n_kv,
                    int32_t n_tok, int32_t* dev_status, void* stream);

/* The rotation of qsa_rope_append alone: x [n_tok][n_heads][128] -> out, tokens
 * x_stride and out_stride elements apart (queries or keys of a layer that keeps no
 * cache, such as an image encoder's).  Arguments as there; out == x is allowed with
 * equal strides. */
int qsa_rope(const void* x, int64_t x_stride, int32_t type, const int32_t* positions, int32_t n_axes,
             int32_t pos_stride, const double* inv_freq, const int32_t* pair_axis, int32_t n_pairs,
             int32_t interleaved, void* out, int64_t out_stride, int32_t n_heads, int32_t n_tok,
             int32_t* dev_status, void* stream);

/* Cells read back as the values they stand for: k_out[i][h][:] = int8 * scale of
 * cell slots[i] for KV head h, and v_out likewise, computed in FP32 and rounded
 * once to out_type (QSA_BF16, QSA_F16 or QSA_F32); [n_cell][n_kv][128], 16-byte
 * aligned.  For a consumer of plain keys and values: a prefix handed to another
 * attention, a cache moved or checked.  A slot < 0 gives zeros, a slot past the
 * pool zeros and QSA_DEV_BAD_CELL; a slot may be named more than once.
 * n_cell == 0 returns QSA_OK. */
int qsa_cache_gather(const int8_t* k_pool, const int8_t* v_pool, const uint16_t* k_scale,
                     const uint16_t* v_scale, const int32_t* slots, int32_t n_cell, int32_t n_ppages,
                     int32_t n_kv, void* k_out, void* v_out, int32_t out_type, int32_t* dev_status, void* stream);

/* Page tables extended and slots mapped for a step's new tokens.  Sequence s
 * holds seq_lens[s] cells and gets new_lens[s] more; its pages beyond
 * ceil(seq_lens[s] / 64) are taken from the free list, sequences in order, and
 * written to its page table.  The new tokens of all sequences, in order, are
 * numbered t = 0, 1, ...:
 *     positions[t] = the token's cell in its sequence, token_seq[t] = s,
 *     slots[t] = its physical cell (page * 64 + cell of the page), or -1,
 * and for t from the total on, up to n_tok: slot -1, position 0, sequence -1.
 *   - page_tables: int32 [n_seq][pt_stride], n_lpages <= pt_stride entries in
 *     use; only the entries of new pages are written.
 *   - free_pages: int32 [n_free] physical pages; *free_head (NULL: 0) of them are
 *     already taken.  *free_head_out = that plus the pages taken now (at most
 *     n_free).  It must not be the same word as *free_head: keep two and swap.
 *     n_free, n_seq and n_tok are at most 2^30.
 *   - seq_lens_out [n_seq] = lengths after the step; cu_tokens [n_seq + 1] = first
 *     token of each sequence, then the total.  seq_lens_out must be neither seq_lens
 *     nor new_lens.
 *   - Reported, never faulting: lengths that are negative or do not fit n_lpages
 *     pages (clamped, QSA_DEV_BAD_SEQ_LEN); more new tokens than n_tok (the tokens
 *     from n_tok on are not added to their sequences, QSA_DEV_TOKEN_OVERFLOW); a
 *     head outside [0, n_free] (clamped), a free list that ran out (entry and slots
 *     -1) or a token on a page that is not resident (slot -1), QSA_DEV_NO_PAGE; a
 *     page outside [0, n_ppages) taken from the list (as if run out) or >= n_ppages
 *     in the table (slot -1), QSA_DEV_BAD_PAGE.
 *   - slots, positions and token_seq must be 16-byte aligned.  One launch, no
 *     atomics on results, no workspace; n_seq == 0 fills the padding. */
int qsa_extend_tables(const int32_t* seq_lens, const int32_t* new_lens, int32_t n_seq, int32_t* page_tables,
                      int32_t pt_stride, int32_t n_lpages, int32_t n_ppages, const int32_t* free_pages,
                      int32_t n_free, const int32_t* free_head, int32_t n_tok, int32_t* slots,
                      int32_t* positions, int32_t* token_seq, int32_t* seq_lens_out, int32_t* cu_tokens,
                      int32_t* free_head_out, int32_t* dev_status, void* stream);

/* ---------------------------------------------------------------- layers with a state
 * Models that select cells in some layers have layers of another kind between them,
 * which keep a state of fixed size per sequence in place of a cache: a short
 * convolution, the gated delta rule, and a norm of its heads.  The calls below are
 * those layers' step.  They share the serving calls' conventions, and
 *   - the step's new tokens of all sequences lie end to end, sequence s holding
 *     tokens cu_tokens[s] .. cu_tokens[s + 1] - 1 (int32 [n_seq + 1], from 0 up and
 *     nowhere falling; qsa_extend_tables writes it).  n_tok is what the token arrays
 *     hold; tokens from cu_tokens[n_seq] on belong to nobody: nothing of theirs is
 *     used, and their rows of the outputs stay as they are.  Bounds that fall or lie
 *     outside [0, n_tok] are clamped and reported (QSA_DEV_BAD_SEQ_LEN).  Where they
 *     fall, sequences may come to share tokens: what their rows and states end as is
 *     not specified, and qsa_delta_prompt leaves out those of more than 32 tokens whose
 *     bounds are out of order with another's.
 *   - state_slots: int32 [n_seq], the sequence's place in the state pool, or < 0: the
 *     sequence is left out, nothing of it is used and its rows of the outputs stay
 *     as they are (padding of a batch; its tokens' rows exist all the same and may be
 *     read).  A slot past the pool is treated alike and reported (QSA_DEV_BAD_STATE).
 *     Slots >= 0 must be distinct.
 *   - old_lens: int32 [n_seq], how many tokens the sequence had before this step
 *     (qsa_extend_tables' seq_lens).  Where it is <= 0 the state starts from zeros
 *     and the pool's contents are not read.  NULL: every sequence goes on.
 *   - After the call the pool holds each sequence's state after its last token;
 *     other slots are not touched. */

/* Activations. */
enum { QSA_ACT_NONE = 0, QSA_ACT_SILU = 1 };

/* Causal depthwise convolution over the last `width` inputs of a sequence:
 *     out[t][c] = act(bias[c] + sum_j weight[c][j] x[t - (width - 1) + j][c]),
 * inputs from before the step taken from the state, FP32 sums, rounded once.
 *   - x: [n_tok][n_ch] of `type` (QSA_BF16 or QSA_F16), tokens x_stride elements
 *     apart; out likewise, out_stride; both strides multiples of 8, >= n_ch, both
 *     16-byte aligned.  n_ch is a multiple of 8, width 2 to 4.  out must not overlap x.
 *   - weight [n_ch][width], bias [n_ch] or NULL, of w_type: `type` or QSA_F32,
 *     16-byte aligned.
 *   - state: [n_slots][width - 1][n_ch] of `type`, the last inputs, oldest first;
 *     16-byte aligned; must not overlap any other argument.
 *   - cu_tokens NULL: one token to every sequence (n_seq == n_tok). */
int qsa_short_conv(const void* x, int64_t x_stride, int32_t type, const void* weight, const void* bias,
                   int32_t w_type, int32_t width, int32_t activation, void* state, const int32_t* state_slots,
                   int32_t n_slots, const int32_t* old_lens, const int32_t* cu_tokens, int32_t n_seq,
                   int32_t n_tok, int32_t n_ch, void* out, int64_t out_stride, int32_t* dev_status,
                   void* stream);

/* The gated delta rule over a step's tokens.  For value head h, with the key head
 * h / (n_v / n_k), a state S (128 x 128, value by key) and token t:
 *     g = -exp(a_log[h]) softplus(a[t][h] + dt_bias[h]),  beta = sigmoid(b[t][h]),
 *     k = k_t / sqrt(|k_t|^2 + eps),  q = q_t scale / sqrt(|q_t|^2 + eps),
 *     S = exp(g) S,  S = S + beta (v_t - S k) k^T,  out[t][h] = S q.
 *   - q, k: [n_tok][n_k][128], v: [n_tok][n_v][128] of `type` (QSA_BF16 or QSA_F16),
 *     tokens q_stride, k_stride, v_stride elements apart (multiples of 8; slices of
 *     the convolution's output), 16-byte aligned; out as v, out_stride; out must
 *     not overlap an input.  n_v is a multiple of n_k.
 *   - a, b: [n_tok][n_v] of `type`, tokens a_stride and b_stride elements apart.
 *     a_log, dt_bias: FP32 [n_v].  a_log = -infinity: no decay; b = infinity: beta = 1.
 *   - eps >= 0; scale is finite.
 *   - state: FP32 [n_slots][n_v][128][128], the key dim innermost, 16-byte aligned.
 *   - Sequences of more than 32 tokens go by chunks of 64 on the tensor cores; the
 *     state and all sums in FP32, the state's and the new values' operands as pairs of
 *     FP16 (22 bits, with a power of two per value dim), and so are the other factors
 *     of the products that end in `out`.  Shorter ones go token by token,
 *     in FP32 throughout (in a step of one sequence, if n_tok <= 32).  Where the step
 *     has few heads (n_seq n_v below half the SMs) and many tokens, long sequences are
 *     cut into segments that run at once and are put together afterwards.
 *   - The same call gives the same bits, and no sequence's results depend on the
 *     contents of others; how a sequence is split into steps, and the step's n_seq,
 *     n_tok and n_v where they decide on segments, change the last bits.
 *   - Range: any finite values and states of magnitudes from 2^-90 to 2^120 or zero.
 *     By chunks, keys and queries likewise (their rows are scaled by powers of two;
 *     elements below 2^-24 of their row's largest lose bits; rows 2^54 and more below
 *     sqrt(eps) count as zeros, and what short ones add to the state is lost below
 *     2^-28 of their chunk's values).  Token by token their squares are summed in FP32 as
 *     they are (lengths from 2^-60 to 2^60).  A row of zeros needs eps > 0.  NaN and
 *     infinities stay in their sequence; by chunks they spoil all of their chunk of 64
 *     tokens, earlier ones too (a value's own value dim alone).
 *   - By chunks, a value dim's new values of a chunk of 64 tokens share a power of two
 *     with the largest value in the chunk and with the state row that its first token
 *     leaves.  That largest leaves errors of 2^-30 of it in the outputs of all of the
 *     chunk's tokens and of 2^-34 in the state, beside FP32's: they show where it is
 *     some 2^16 times what others of them are made of, those before it or behind a
 *     gate that has forgotten it.  What the gates have forgotten at the chunk's end or
 *     by its first token leaves none.
 *   - state and workspace must not overlap any other argument.
 *   - workspace: device memory of at least qsa_delta_prompt_workspace_bytes(n_tok,
 *     n_seq, n_k, n_v) bytes, 256-byte aligned, contents neither set nor kept:
 *     32,768 n_k + 25,600 n_v bytes for each of n_tok / 64 + n_seq chunks, or for each of
 *     n_tok / 32 in a step of several sequences if those are fewer; where segments may
 *     be cut 1,024 n_v bytes a token and 1 MB n_seq n_v more; 256 bytes for up to 32
 *     tokens.
 *     Two calls that can overlap on the device need one each, captured ones too.
 *   - n_seq == 0 returns QSA_OK with no launch. */
int qsa_delta_prompt(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                     int64_t v_stride, int32_t type, const void* a, int64_t a_stride, const void* b,
                     int64_t b_stride, const float* a_log, const float* dt_bias, float* state,
                     const int32_t* state_slots, int32_t n_slots, const int32_t* old_lens,
                     const int32_t* cu_tokens, int32_t n_seq, int32_t n_tok, int32_t n_k, int32_t n_v,
                     float eps, float scale, void* out, int64_t out_stride, void* workspace,
                     size_t workspace_bytes, int32_t* dev_status, void* stream);

/* Workspace of qsa_delta_prompt; 0 for sizes that it refuses. */
size_t qsa_delta_prompt_workspace_bytes(int32_t n_tok, int32_t n_seq, int32_t n_k, int32_t n_v);

/* The same for one token of every sequence (token s is sequence s's), FP32
 * throughout: the decode step, one launch, no workspace.  Keys and queries as token by
 * token above. */
int qsa_delta_step(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                   int64_t v_stride, int32_t type, const void* a, int64_t a_stride, const void* b,
                   int64_t b_stride, const float* a_log, const float* dt_bias, float* state,
                   const int32_t* state_slots, int32_t n_slots, const int32_t* old_lens, int32_t n_seq,
                   int32_t n_k, int32_t n_v, float eps, float scale, void* out, int64_t out_stride,
                   int32_t* dev_status, void* stream);

/* Each group of `size` channels of each token normalised over itself, channels last:
 *     y = (x - m) / sqrt(mean((x - m)^2) + eps) weight + bias,
 * m the group's mean when centred, else 0; then out = y act(gate), or act(y) without a
 * gate.  Statistics in FP32 (the mean first, then the squares), rounded once.
 *   - x, gate (or NULL), out: [n_tok][n_groups][size] of `type` (QSA_BF16 or QSA_F16),
 *     tokens x_stride, gate_stride, out_stride elements apart (multiples of 8),
 *     16-byte aligned.  size is a multiple of 8 up to 8192.  out may be x or gate, with
 *     equal strides; otherwise it must not overlap them.
 *   - weight, bias: [size], or [n_groups][size] when per_group, or NULL (ones,
 *     zeros), of w_type: `type` or QSA_F32, 16-byte aligned.
 *   - eps >= 0.  Squares are summed in FP32 as they are: x - m of magnitudes up to 2^57;
 *     without an eps that outweighs them, their root mean square no less than 2^-60. */
int qsa_group_norm(const void* x, int64_t x_stride, const void* gate, int64_t gate_stride, int32_t type,
                   const void* weight, const void* bias, int32_t w_type, int32_t per_group, int32_t n_tok,
                   int32_t n_groups, int32_t size, float eps, int32_t centred, int32_t activation, void* out,
                   int64_t out_stride, void* stream);

/* The same calls with their arguments in one struct, in the order of the
 * parameters, for callers to whom converting each argument costs more than the call
 * (interpreters).  Statuses and results are those of the calls; NULL is QSA_ERR_ARG. */
typedef struct {
    const void* q;
    int32_t q_type;
    const int8_t *k_pool, *v_pool;
    const uint16_t *k_scale, *v_scale;
    const int32_t* page_tables;
    int32_t pt_stride, n_lpages, n_ppages, n_kv, n_heads;
    const int32_t* seq_lens;
    int32_t n_seq, window;
    float sm_scale;
    void* out;
    int32_t out_type;
    float* lse;
    void* workspace;
    size_t workspace_bytes;
    int32_t* dev_status;
    void* stream;
} qsa_paged_attn_args;
int qsa_paged_attn_packed(const qsa_paged_attn_args* args);

typedef struct {
    const void* q;
    int64_t q_stride;
    const void* k;
    int64_t k_stride;
    const void* v;
    int64_t v_stride;
    int32_t type;
    const int32_t* positions;
    int32_t n_axes, pos_stride;
    const double* inv_freq;
    const int32_t* pair_axis;
    int32_t n_pairs, interleaved;
    void* q_out;
    int64_t q_out_stride;
    int8_t *k_pool, *v_pool;
    uint16_t *k_scale, *v_scale;
    const int32_t* slots;
    int32_t n_ppages, n_heads, n_kv, n_tok;
    int32_t* dev_status;
    void* stream;
} qsa_rope_append_args;
int qsa_rope_append_packed(const qsa_rope_append_args* args);

typedef struct {
    const int8_t *k_pool, *v_pool;
    const uint16_t *k_scale, *v_scale;
    const int32_t* slots;
    int32_t n_cell, n_ppages, n_kv;
    void *k_out, *v_out;
    int32_t out_type;
    int32_t* dev_status;
    void* stream;
} qsa_cache_gather_args;
int qsa_cache_gather_packed(const qsa_cache_gather_args* args);

typedef struct {
    const int32_t *seq_lens, *new_lens;
    int32_t n_seq;
    int32_t* page_tables;
    int32_t pt_stride, n_lpages, n_ppages;
    const int32_t* free_pages;
    int32_t n_free;
    const int32_t* free_head;
    int32_t n_tok;
    int32_t *slots, *positions, *token_seq, *seq_lens_out, *cu_tokens, *free_head_out, *dev_status;
    void* stream;
} qsa_extend_tables_args;
int qsa_extend_tables_packed(const qsa_extend_tables_args* args);

typedef struct {
    const void* x;
    int64_t x_stride;
    int32_t type;
    const void *weight, *bias;
    int32_t w_type, width, activation;
    void* state;
    const int32_t* state_slots;
    int32_t n_slots;
    const int32_t *old_lens, *cu_tokens;
    int32_t n_seq, n_tok, n_ch;
    void* out;
    int64_t out_stride;
    int32_t* dev_status;
    void* stream;
} qsa_short_conv_args;
int qsa_short_conv_packed(const qsa_short_conv_args* args);

typedef struct {
    const void* q;
    int64_t q_stride;
    const void* k;
    int64_t k_stride;
    const void* v;
    int64_t v_stride;
    int32_t type;
    const void* a;
    int64_t a_stride;
    const void* b;
    int64_t b_stride;
    const float *a_log, *dt_bias;
    float* state;
    const int32_t* state_slots;
    int32_t n_slots;
    const int32_t *old_lens, *cu_tokens;
    int32_t n_seq, n_tok, n_k, n_v;
    float eps, scale;
    void* out;
    int64_t out_stride;
    void* workspace;
    size_t workspace_bytes;
    int32_t* dev_status;
    void* stream;
} qsa_delta_prompt_args;
int qsa_delta_prompt_packed(const qsa_delta_prompt_args* args);

typedef struct {
    const void* q;
    int64_t q_stride;
    const void* k;
    int64_t k_stride;
    const void* v;
    int64_t v_stride;
    int32_t type;
    const void* a;
    int64_t a_stride;
    const void* b;
    int64_t b_stride;
    const float *a_log, *dt_bias;
    float* state;
    const int32_t* state_slots;
    int32_t n_slots;
    const int32_t* old_lens;
    int32_t n_seq, n_k, n_v;
    float eps, scale;
    void* out;
    int64_t out_stride;
    int32_t* dev_status;
    void* stream;
} qsa_delta_step_args;
int qsa_delta_step_packed(const qsa_delta_step_args* args);

typedef struct {
    const void* x;
    int64_t x_stride;
    const void* gate;
    int64_t gate_stride;
    int32_t type;
    const void *weight, *bias;
    int32_t w_type, per_group, n_tok, n_groups, size;
    float eps;
    int32_t centred, activation;
    void* out;
    int64_t out_stride;
    void* stream;
} qsa_group_norm_args;
int qsa_group_norm_packed(const qsa_group_norm_args* args);

/* Self-test of the bounded waits (not part of the method: the pages have no
 * counterpart).  Every pipelined kernel here waits on mbarriers with a wall-time
 * limit and, when one runs out, records QSA_DEV_WAIT_TIMEOUT in *dev_status and
 * returns instead of hanging.  This launches one warp that waits on an mbarrier
 * nothing arrives on, for limit_us microseconds, then records that bit: a test
 * can see the whole path -- the wait ending by time, the device status reaching
 * the host, the context staying usable -- without faulting anything.
 *   - limit_us in (0, 10^7]; dev_status: device int32, OR-ed into, required.
 *   - Returns QSA_ERR_ARG otherwise, QSA_ERR_CUDA if the launch fails. */
int qsa_wait_selftest(int32_t limit_us, int32_t* dev_status, void* stream);

/* Bytes of the static device scratch behind qsa_prompt_attn_static (32 MiB):
 * room for n_q <= 3256 queries at union_stride 16448, more at smaller strides. */
#define QSA_STATIC_SCRATCH_BYTES (32u << 20)

/* qsa_prompt_attn without a workspace argument and without any allocation.
 * The method's description has no counterpart of this call: it exists for
 * callers that cannot hand over device memory -- a plain C host with no device
 * allocator of its own, for which cudaMalloc / cudaFree around each step would
 * synchronise the device, or a caller inside a framework whose allocator it
 * cannot reach.  The union arrays go to a scratch of QSA_STATIC_SCRATCH_BYTES
 * in this library's static device memory (one per device), and the result is
 * that of qsa_prompt_attn on a workspace of that size.
 *   - Arguments, layouts and ownership are those of qsa_prompt_attn; the
 *     stream must belong to the current device (QSA_ERR_ARG otherwise).
 *   - Checks that need no CUDA call come first, in this order: sizes, shape
 *     arguments and variant (QSA_ERR_ARG), then capacity: QSA_ERR_CAPACITY when
 *     qsa_union_workspace_bytes(n_q, union_stride) > QSA_STATIC_SCRATCH_BYTES,
 *     then null pointers (QSA_ERR_ARG).  QSA_ERR_CUDA when the scratch's
 *     address cannot be resolved.
 *   - The first call on each device resolves the scratch's address with
 *     cudaGetSymbolAddress (this may load the library's device code on that
 *     device) and caches it for the life of the process; make that first call
 *     before any stream capture begins.  The cached address is not valid after
 *     cudaDeviceReset (the module is loaded again and the scratch may move):
 *     a process that resets a device must not call this entry point on that
 *     device afterwards.
 *   - Nothing in the scratch must start at zero (the union build writes all
 *     that the attention kernel reads), so no call clears it.
 *   - All calls on one device share the one scratch: two calls whose work can
 *     overlap on the device (different streams, or different host threads
 *     without ordering between their streams) race on it.  Order them. */
int qsa_prompt_attn_static(const uint16_t* q, const int8_t* k_pool, const int8_t* v_pool,
                           const uint16_t* k_scale, const uint16_t* v_scale,
                           const int32_t* page_table, int32_t n_lpages, int32_t n_ppages, int32_t n_kv,
                           const int32_t* sel, const int32_t* sel_count, int32_t sel_stride, int32_t n_q,
                           float sm_scale, float* out, int32_t union_stride, int32_t variant,
                           int32_t* dev_status, void* stream);

#ifdef __cplusplus
}
#endif
#endif

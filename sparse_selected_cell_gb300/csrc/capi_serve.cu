// capi_serve.cu -- the extern "C" boundary of the serving operators around the
// paged INT8 cache (declared in include/qsa.h): argument validation and launches.
// No allocation, no synchronisation, no host fallback.
#include <cstdint>
#include <cuda_runtime.h>

#include "serve.cuh"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA; }

bool type16(int t) { return t == QSA_BF16 || t == QSA_F16; }

// A slot (page * 64 + cell) is an int32; as everywhere in this library, so are the rows
// of one pool, n_ppages * n_kv * 64.
bool pool_fits(int32_t n_ppages, int32_t n_kv) {
    return (long long)n_ppages * n_kv <= ((1LL << 31) - 64) / qsa::kPage;
}

int check_pool(const int8_t* k_pool, const int8_t* v_pool, const uint16_t* k_scale, const uint16_t* v_scale,
               int32_t n_ppages, int32_t n_kv) {
    if (n_ppages > 0 && (!k_pool || !v_pool || !k_scale || !v_scale)) return QSA_ERR_ARG;
    if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(k_scale, 16) || !aligned(v_scale, 16))
        return QSA_ERR_ARG;
    return pool_fits(n_ppages, n_kv) ? QSA_OK : QSA_ERR_UNSUPPORTED;
}

// The rotation's arguments (n_pairs > 0), shared by qsa_rope and qsa_rope_append.
int check_rotation(const int32_t* positions, int32_t n_axes, int32_t pos_stride, const double* inv_freq,
                   int32_t n_pairs, int32_t n_tok) {
    if (n_pairs < 0 || n_pairs > qsa::kHeadDim / 2 || n_pairs % 8 != 0) return QSA_ERR_ARG;
    if (n_pairs == 0) return QSA_OK;
    if (n_axes < 1 || n_axes > 4 || pos_stride < n_tok) return QSA_ERR_ARG;
    if (n_tok > 0 && (!positions || !inv_freq || !aligned(inv_freq, 8))) return QSA_ERR_ARG;
    return QSA_OK;
}

// A [n_tok][heads][128] tensor of 16-bit elements with `stride` elements between tokens.
bool rows_ok(const void* p, int64_t stride, int32_t heads) {
    return p && aligned(p, 16) && stride % 8 == 0 && stride >= (int64_t)heads * qsa::kHeadDim;
}

constexpr int32_t kMaxHeads = 1 << 16;   // heads * 128 * tokens stays well inside 64-bit offsets

}  // namespace

extern "C" {

size_t qsa_paged_attn_workspace_bytes(int32_t n_kv, int32_t n_heads) {
    if (n_kv <= 0 || n_heads <= 0 || n_heads % n_kv != 0) return 0;
    return qsa::paged_attn_workspace(n_kv, n_heads);
}

int qsa_paged_attn(const void* q, int32_t q_type, const int8_t* k_pool, const int8_t* v_pool,
                   const uint16_t* k_scale, const uint16_t* v_scale, const int32_t* page_tables,
                   int32_t pt_stride, int32_t n_lpages, int32_t n_ppages, int32_t n_kv, int32_t n_heads,
                   const int32_t* seq_lens, int32_t n_seq, int32_t window, float sm_scale, void* out,
                   int32_t out_type, float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                   void* stream) {
    if (n_seq < 0 || n_lpages < 0 || n_ppages < 0 || n_kv <= 0 || n_heads <= 0 || n_heads % n_kv != 0 || window < 0)
        return QSA_ERR_ARG;
    if (!type16(q_type) || (!type16(out_type) && out_type != QSA_F32)) return QSA_ERR_ARG;
    if (pt_stride < 0 || (pt_stride > 0 && pt_stride < n_lpages)) return QSA_ERR_ARG;
    if (n_heads > kMaxHeads) return QSA_ERR_UNSUPPORTED;
    if (n_seq == 0) return QSA_OK;
    if (!q || !out || !seq_lens || !workspace || (n_lpages > 0 && !page_tables)) return QSA_ERR_ARG;
    if (out == q) return QSA_ERR_ARG;   // rows are read by several blocks, at any time
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256)) return QSA_ERR_ARG;
    const int rc = check_pool(k_pool, v_pool, k_scale, v_scale, n_ppages, n_kv);
    if (rc != QSA_OK) return rc;
    const long long tiles = (n_heads / n_kv + 15) / 16;
    if ((long long)n_lpages * qsa::kPage > (1LL << 31) - 64) return QSA_ERR_UNSUPPORTED;
    // pages of all (sequence, KV head, row tile) items and a place for each item: the kernel numbers them in int32
    if (n_lpages > 0 && (long long)n_seq * (n_lpages + 1LL) > (1LL << 30) / (n_kv * tiles)) return QSA_ERR_UNSUPPORTED;
    if (workspace_bytes < qsa::paged_attn_workspace(n_kv, n_heads)) return QSA_ERR_CAPACITY;
    const qsa::PagedArgs a{q, q_type, k_pool, v_pool, k_scale, v_scale, page_tables, pt_stride, n_lpages, n_ppages,
                           n_kv, n_heads, seq_lens, n_seq, window, sm_scale, out, out_type, lse,
                           static_cast<uint8_t*>(workspace), dev_status};
    return cuda_status(qsa::launch_paged_attn(a, static_cast<cudaStream_t>(stream)));
}

int qsa_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                    int64_t v_stride, int32_t type, const int32_t* positions, int32_t n_axes, int32_t pos_stride,
                    const double* inv_freq, const int32_t* pair_axis, int32_t n_pairs, int32_t interleaved,
                    void* q_out, int64_t q_out_stride, int8_t* k_pool, int8_t* v_pool, uint16_t* k_scale,
                    uint16_t* v_scale, const int32_t* slots, int32_t n_ppages, int32_t n_heads, int32_t n_kv,
                    int32_t n_tok, int32_t* dev_status, void* stream) {
    if (n_tok < 0 || n_ppages < 0 || n_kv <= 0 || n_heads < 0 || !type16(type)) return QSA_ERR_ARG;
    int rc = check_rotation(positions, n_axes, pos_stride, inv_freq, n_pairs, n_tok);
    if (rc != QSA_OK) return rc;
    if (n_heads > kMaxHeads || n_kv > kMaxHeads) return QSA_ERR_UNSUPPORTED;
    if (n_tok == 0) return QSA_OK;
    if (q && (!rows_ok(q, q_stride, n_heads) || !rows_ok(q_out, q_out_stride, n_heads) || n_heads == 0))
        return QSA_ERR_ARG;
    if (q && q_out == q && q_out_stride != q_stride) return QSA_ERR_ARG;
    if (!rows_ok(k, k_stride, n_kv) || !rows_ok(v, v_stride, n_kv) || !slots) return QSA_ERR_ARG;
    rc = check_pool(k_pool, v_pool, k_scale, v_scale, n_ppages, n_kv);
    if (rc != QSA_OK) return rc;
    const qsa::RopeArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                          static_cast<const uint16_t*>(v), q_stride, k_stride, v_stride, type, positions, n_axes,
                          pos_stride, inv_freq, pair_axis, n_pairs, interleaved, static_cast<uint16_t*>(q_out),
                          q_out_stride, k_pool, v_pool, k_scale, v_scale, slots, n_ppages, q ? n_heads : 0, n_kv,
                          n_tok, dev_status};
    return cuda_status(qsa::launch_rope_append(a, static_cast<cudaStream_t>(stream)));
}

int qsa_rope(const void* x, int64_t x_stride, int32_t type, const int32_t* positions, int32_t n_axes,
             int32_t pos_stride, const double* inv_freq, const int32_t* pair_axis, int32_t n_pairs,
             int32_t interleaved, void* out, int64_t out_stride, int32_t n_heads, int32_t n_tok,
             int32_t* dev_status, void* stream) {
    if (n_tok < 0 || n_heads <= 0 || !type16(type)) return QSA_ERR_ARG;
    const int rc = check_rotation(positions, n_axes, pos_stride, inv_freq, n_pairs, n_tok);
    if (rc != QSA_OK) return rc;
    if (n_heads > kMaxHeads) return QSA_ERR_UNSUPPORTED;
    if (n_tok == 0) return QSA_OK;
    if (!rows_ok(x, x_stride, n_heads) || !rows_ok(out, out_stride, n_heads)) return QSA_ERR_ARG;
    if (out == x && out_stride != x_stride) return QSA_ERR_ARG;
    const qsa::RopeArgs a{static_cast<const uint16_t*>(x), nullptr, nullptr, x_stride, 0, 0, type, positions, n_axes,
                          pos_stride, inv_freq, pair_axis, n_pairs, interleaved, static_cast<uint16_t*>(out),
                          out_stride, nullptr, nullptr, nullptr, nullptr, nullptr, 0, n_heads, 0, n_tok, dev_status};
    return cuda_status(qsa::launch_rope_append(a, static_cast<cudaStream_t>(stream)));
}

int qsa_cache_gather(const int8_t* k_pool, const int8_t* v_pool, const uint16_t* k_scale, const uint16_t* v_scale,
                     const int32_t* slots, int32_t n_cell, int32_t n_ppages, int32_t n_kv, void* k_out, void* v_out,
                     int32_t out_type, int32_t* dev_status, void* stream) {
    if (n_cell < 0 || n_ppages < 0 || n_kv <= 0 || (!type16(out_type) && out_type != QSA_F32)) return QSA_ERR_ARG;
    if (n_kv > kMaxHeads) return QSA_ERR_UNSUPPORTED;
    if (n_cell == 0) return QSA_OK;
    if (!slots || !k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16)) return QSA_ERR_ARG;
    const int rc = check_pool(k_pool, v_pool, k_scale, v_scale, n_ppages, n_kv);
    if (rc != QSA_OK) return rc;
    const qsa::GatherArgs a{k_pool, v_pool, k_scale, v_scale, slots, n_cell, n_ppages, n_kv, k_out, v_out, out_type,
                            dev_status};
    return cuda_status(qsa::launch_cache_gather(a, static_cast<cudaStream_t>(stream)));
}

int qsa_extend_tables(const int32_t* seq_lens, const int32_t* new_lens, int32_t n_seq, int32_t* page_tables,
                      int32_t pt_stride, int32_t n_lpages, int32_t n_ppages, const int32_t* free_pages,
                      int32_t n_free, const int32_t* free_head, int32_t n_tok, int32_t* slots, int32_t* positions,
                      int32_t* token_seq, int32_t* seq_lens_out, int32_t* cu_tokens, int32_t* free_head_out,
                      int32_t* dev_status, void* stream) {
    if (n_seq < 0 || n_lpages < 0 || pt_stride < n_lpages || n_ppages < 0 || n_free < 0 || n_tok < 0)
        return QSA_ERR_ARG;
    if ((long long)n_lpages * qsa::kPage > (1LL << 31) - 64 || !pool_fits(n_ppages, 1)) return QSA_ERR_UNSUPPORTED;
    if (n_seq > (1 << 30) || n_tok > (1 << 30) || n_free > (1 << 30)) return QSA_ERR_UNSUPPORTED;
    if (!cu_tokens || !free_head_out || free_head_out == free_head) return QSA_ERR_ARG;
    if (n_seq > 0 && (!seq_lens || !new_lens || !seq_lens_out || seq_lens_out == seq_lens ||
                      seq_lens_out == new_lens || (n_lpages > 0 && !page_tables)))
        return QSA_ERR_ARG;
    if (n_free > 0 && !free_pages) return QSA_ERR_ARG;
    if (n_tok > 0 && (!slots || !positions || !token_seq || !aligned(slots, 16) || !aligned(positions, 16) ||
                      !aligned(token_seq, 16)))
        return QSA_ERR_ARG;
    const qsa::TablesArgs a{seq_lens, new_lens, n_seq, page_tables, pt_stride, n_lpages, n_ppages, free_pages, n_free,
                            free_head, n_tok, slots, positions, token_seq, seq_lens_out, cu_tokens, free_head_out,
                            dev_status};
    return cuda_status(qsa::launch_extend_tables(a, static_cast<cudaStream_t>(stream)));
}

int qsa_paged_attn_packed(const qsa_paged_attn_args* a) {
    if (!a) return QSA_ERR_ARG;
    return qsa_paged_attn(a->q, a->q_type, a->k_pool, a->v_pool, a->k_scale, a->v_scale, a->page_tables, a->pt_stride,
                          a->n_lpages, a->n_ppages, a->n_kv, a->n_heads, a->seq_lens, a->n_seq, a->window, a->sm_scale,
                          a->out, a->out_type, a->lse, a->workspace, a->workspace_bytes, a->dev_status, a->stream);
}

int qsa_rope_append_packed(const qsa_rope_append_args* a) {
    if (!a) return QSA_ERR_ARG;
    return qsa_rope_append(a->q, a->q_stride, a->k, a->k_stride, a->v, a->v_stride, a->type, a->positions, a->n_axes,
                           a->pos_stride, a->inv_freq, a->pair_axis, a->n_pairs, a->interleaved, a->q_out,
                           a->q_out_stride, a->k_pool, a->v_pool, a->k_scale, a->v_scale, a->slots, a->n_ppages,
                           a->n_heads, a->n_kv, a->n_tok, a->dev_status, a->stream);
}

int qsa_cache_gather_packed(const qsa_cache_gather_args* a) {
    if (!a) return QSA_ERR_ARG;
    return qsa_cache_gather(a->k_pool, a->v_pool, a->k_scale, a->v_scale, a->slots, a->n_cell, a->n_ppages, a->n_kv,
                            a->k_out, a->v_out, a->out_type, a->dev_status, a->stream);
}

int qsa_extend_tables_packed(const qsa_extend_tables_args* a) {
    if (!a) return QSA_ERR_ARG;
    return qsa_extend_tables(a->seq_lens, a->new_lens, a->n_seq, a->page_tables, a->pt_stride, a->n_lpages, a->n_ppages,
                             a->free_pages, a->n_free, a->free_head, a->n_tok, a->slots, a->positions, a->token_seq,
                             a->seq_lens_out, a->cu_tokens, a->free_head_out, a->dev_status, a->stream);
}

}  // extern "C"

// capi_linear.cu -- the extern "C" boundary of the layers that keep a state per sequence
// (declared in include/qsa.h): argument validation and launches.  No allocation, no
// synchronisation, no host fallback.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "linear.cuh"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA; }

bool type16(int t) { return t == QSA_BF16 || t == QSA_F16; }

bool act_ok(int act) { return act == QSA_ACT_NONE || act == QSA_ACT_SILU; }

// Tokens of `width` 16-bit elements each, `stride` elements apart.
bool rows_ok(const void* p, int64_t stride, int64_t width) {
    return p && aligned(p, 16) && stride % 8 == 0 && stride >= width;
}

constexpr int32_t kMaxHeads = 1 << 16;
constexpr int32_t kMaxTokens = 1 << 30;

// Blocks of a launch: two to a sequence and value head, one to a chunk (at most n_tok / 64 + n_seq) and key head.
bool sizes_fit(int32_t n_tok, int32_t n_seq, int32_t n_k, int32_t n_v) {
    return n_v <= kMaxHeads && n_tok <= kMaxTokens && (long long)n_seq * n_v <= kMaxTokens / 2 &&
           (n_tok / 64 + (long long)n_seq) * n_k <= kMaxTokens;
}

// Whether two arrays of n tokens, `width` 16-bit elements of each in use, share a byte (strides in elements).  Rows
// interleave where both are slices of one wider array: equal strides, and offsets that keep them apart.
bool overlap(const void* p, int64_t ps, int64_t pw, const void* q, int64_t qs, int64_t qw, int64_t n) {
    const intptr_t a = reinterpret_cast<intptr_t>(p) / 2, b = reinterpret_cast<intptr_t>(q) / 2;
    if (n <= 0) return false;
    if (a >= b + (n - 1) * qs + qw || b >= a + (n - 1) * ps + pw) return false;
    if (ps != qs || n == 1) return true;
    const intptr_t off = ((a - b) % ps + ps) % ps;        // p's row begins `off` behind one of q's
    return off < qw || off + pw > ps;
}

// The heads and gates of the delta rule, shared by its two calls.
int check_delta(const qsa::DeltaArgs& a) {
    if (a.n_seq < 0 || a.n_tok < 0 || a.n_slots < 0 || a.n_k <= 0 || a.n_v <= 0 || a.n_v % a.n_k != 0 || !type16(a.type))
        return QSA_ERR_ARG;
    if (!(a.eps >= 0.f) || !std::isfinite(a.eps) || !std::isfinite(a.scale)) return QSA_ERR_ARG;
    if (!sizes_fit(a.n_tok, a.n_seq, a.n_k, a.n_v)) return QSA_ERR_UNSUPPORTED;
    if (a.n_seq == 0) return QSA_OK;
    if (!a.state_slots || !a.a_log || !a.dt_bias || !aligned(a.state, 16) || (a.n_slots > 0 && !a.state)) return QSA_ERR_ARG;
    if (a.n_tok == 0) return QSA_OK;
    const int64_t kw = (int64_t)a.n_k * qsa::kHeadDim, vw = (int64_t)a.n_v * qsa::kHeadDim;
    if (!rows_ok(a.q, a.q_stride, kw) || !rows_ok(a.k, a.k_stride, kw) || !rows_ok(a.v, a.v_stride, vw) ||
        !rows_ok(a.out, a.out_stride, vw) || !a.a || !a.b || a.a_stride < a.n_v || a.b_stride < a.n_v)
        return QSA_ERR_ARG;
    if (!aligned(a.a, 2) || !aligned(a.b, 2)) return QSA_ERR_ARG;
    if (overlap(a.out, a.out_stride, vw, a.q, a.q_stride, kw, a.n_tok) ||
        overlap(a.out, a.out_stride, vw, a.k, a.k_stride, kw, a.n_tok) ||
        overlap(a.out, a.out_stride, vw, a.v, a.v_stride, vw, a.n_tok) ||
        overlap(a.out, a.out_stride, vw, a.a, a.a_stride, a.n_v, a.n_tok) ||
        overlap(a.out, a.out_stride, vw, a.b, a.b_stride, a.n_v, a.n_tok))
        return QSA_ERR_ARG;
    return QSA_OK;
}

}  // namespace

extern "C" {

int qsa_short_conv(const void* x, int64_t x_stride, int32_t type, const void* weight, const void* bias,
                   int32_t w_type, int32_t width, int32_t activation, void* state, const int32_t* state_slots,
                   int32_t n_slots, const int32_t* old_lens, const int32_t* cu_tokens, int32_t n_seq,
                   int32_t n_tok, int32_t n_ch, void* out, int64_t out_stride, int32_t* dev_status,
                   void* stream) {
    if (n_seq < 0 || n_tok < 0 || n_slots < 0 || n_ch <= 0 || n_ch % 8 != 0 || width < 2 || width > 4 || !type16(type) ||
        (w_type != type && w_type != QSA_F32) || !act_ok(activation))
        return QSA_ERR_ARG;
    if (!cu_tokens && n_seq != n_tok) return QSA_ERR_ARG;
    if (n_tok > kMaxTokens || n_seq > kMaxTokens || n_ch > kMaxHeads * qsa::kHeadDim || !qsa::short_conv_fits(n_tok, n_ch))
        return QSA_ERR_UNSUPPORTED;
    if (n_seq == 0) return QSA_OK;
    if (!weight || !state_slots || !aligned(weight, 16) || !aligned(bias, 16) || !aligned(state, 16) ||
        (n_slots > 0 && !state))
        return QSA_ERR_ARG;
    if (n_tok > 0) {
        if (!rows_ok(x, x_stride, n_ch) || !rows_ok(out, out_stride, n_ch)) return QSA_ERR_ARG;
        if (overlap(out, out_stride, n_ch, x, x_stride, n_ch, n_tok)) return QSA_ERR_ARG;
    }
    const qsa::ConvArgs a{static_cast<const uint16_t*>(x), x_stride, type, weight, bias, w_type, width, activation,
                          static_cast<uint16_t*>(state), state_slots, n_slots, old_lens, cu_tokens, n_seq, n_tok, n_ch,
                          static_cast<uint16_t*>(out), out_stride, dev_status};
    return cuda_status(qsa::launch_short_conv(a, static_cast<cudaStream_t>(stream)));
}

size_t qsa_delta_prompt_workspace_bytes(int32_t n_tok, int32_t n_seq, int32_t n_k, int32_t n_v) {
    if (n_tok < 0 || n_seq < 0 || n_k <= 0 || n_v <= 0 || n_v % n_k != 0 || !sizes_fit(n_tok, n_seq, n_k, n_v)) return 0;
    return qsa::delta_prompt_workspace(n_tok, n_seq, n_k, n_v);
}

int qsa_delta_prompt(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                     int64_t v_stride, int32_t type, const void* a, int64_t a_stride, const void* b,
                     int64_t b_stride, const float* a_log, const float* dt_bias, float* state,
                     const int32_t* state_slots, int32_t n_slots, const int32_t* old_lens,
                     const int32_t* cu_tokens, int32_t n_seq, int32_t n_tok, int32_t n_k, int32_t n_v,
                     float eps, float scale, void* out, int64_t out_stride, void* workspace,
                     size_t workspace_bytes, int32_t* dev_status, void* stream) {
    const qsa::DeltaArgs d{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                           static_cast<const uint16_t*>(v), q_stride, k_stride, v_stride, type,
                           static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(b), a_stride, b_stride, a_log,
                           dt_bias, state, state_slots, n_slots, old_lens, cu_tokens, n_seq, n_tok, n_k, n_v, eps, scale,
                           static_cast<uint16_t*>(out), out_stride, static_cast<uint8_t*>(workspace), dev_status, 0, 1};
    const int rc = check_delta(d);
    if (rc != QSA_OK || n_seq == 0) return rc;
    if (!cu_tokens || !workspace || !aligned(workspace, 256)) return QSA_ERR_ARG;
    if (workspace_bytes < qsa::delta_prompt_workspace(n_tok, n_seq, n_k, n_v)) return QSA_ERR_CAPACITY;
    return cuda_status(qsa::launch_delta_prompt(d, static_cast<cudaStream_t>(stream)));
}

int qsa_delta_step(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                   int64_t v_stride, int32_t type, const void* a, int64_t a_stride, const void* b,
                   int64_t b_stride, const float* a_log, const float* dt_bias, float* state,
                   const int32_t* state_slots, int32_t n_slots, const int32_t* old_lens, int32_t n_seq,
                   int32_t n_k, int32_t n_v, float eps, float scale, void* out, int64_t out_stride,
                   int32_t* dev_status, void* stream) {
    const qsa::DeltaArgs d{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                           static_cast<const uint16_t*>(v), q_stride, k_stride, v_stride, type,
                           static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(b), a_stride, b_stride, a_log,
                           dt_bias, state, state_slots, n_slots, old_lens, nullptr, n_seq, n_seq, n_k, n_v, eps, scale,
                           static_cast<uint16_t*>(out), out_stride, nullptr, dev_status, 0, 1};
    const int rc = check_delta(d);
    if (rc != QSA_OK || n_seq == 0) return rc;
    return cuda_status(qsa::launch_delta_step(d, static_cast<cudaStream_t>(stream)));
}

int qsa_group_norm(const void* x, int64_t x_stride, const void* gate, int64_t gate_stride, int32_t type,
                   const void* weight, const void* bias, int32_t w_type, int32_t per_group, int32_t n_tok,
                   int32_t n_groups, int32_t size, float eps, int32_t centred, int32_t activation, void* out,
                   int64_t out_stride, void* stream) {
    if (n_tok < 0 || n_groups <= 0 || size <= 0 || size % 8 != 0 || !type16(type) ||
        (w_type != type && w_type != QSA_F32) || !act_ok(activation) || !(eps >= 0.f) || !std::isfinite(eps))
        return QSA_ERR_ARG;
    if (size > 8192 || n_groups > kMaxHeads || n_tok > kMaxTokens || !qsa::group_norm_fits(n_tok, n_groups, size))
        return QSA_ERR_UNSUPPORTED;
    if (n_tok == 0) return QSA_OK;
    const int64_t row = (int64_t)n_groups * size;
    if (!rows_ok(x, x_stride, row) || !rows_ok(out, out_stride, row) || (gate && !rows_ok(gate, gate_stride, row)))
        return QSA_ERR_ARG;
    if (!aligned(weight, 16) || !aligned(bias, 16)) return QSA_ERR_ARG;
    if (out == x ? out_stride != x_stride : overlap(out, out_stride, row, x, x_stride, row, n_tok)) return QSA_ERR_ARG;
    if (gate && (out == gate ? out_stride != gate_stride : overlap(out, out_stride, row, gate, gate_stride, row, n_tok)))
        return QSA_ERR_ARG;
    const qsa::NormArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(gate), x_stride, gate_stride, type,
                          weight, bias, w_type, per_group, n_tok, n_groups, size, eps, centred, activation,
                          static_cast<uint16_t*>(out), out_stride};
    return cuda_status(qsa::launch_group_norm(a, static_cast<cudaStream_t>(stream)));
}

int qsa_short_conv_packed(const qsa_short_conv_args* a) {
    if (!a) return QSA_ERR_ARG;
    return qsa_short_conv(a->x, a->x_stride, a->type, a->weight, a->bias, a->w_type, a->width, a->activation, a->state,
                          a->state_slots, a->n_slots, a->old_lens, a->cu_tokens, a->n_seq, a->n_tok, a->n_ch, a->out,
                          a->out_stride, a->dev_status, a->stream);
}

int qsa_delta_prompt_packed(const qsa_delta_prompt_args* a) {
    if (!a) return QSA_ERR_ARG;
    return qsa_delta_prompt(a->q, a->q_stride, a->k, a->k_stride, a->v, a->v_stride, a->type, a->a, a->a_stride, a->b,
                            a->b_stride, a->a_log, a->dt_bias, a->state, a->state_slots, a->n_slots, a->old_lens,
                            a->cu_tokens, a->n_seq, a->n_tok, a->n_k, a->n_v, a->eps, a->scale, a->out, a->out_stride,
                            a->workspace, a->workspace_bytes, a->dev_status, a->stream);
}

int qsa_delta_step_packed(const qsa_delta_step_args* a) {
    if (!a) return QSA_ERR_ARG;
    return qsa_delta_step(a->q, a->q_stride, a->k, a->k_stride, a->v, a->v_stride, a->type, a->a, a->a_stride, a->b,
                          a->b_stride, a->a_log, a->dt_bias, a->state, a->state_slots, a->n_slots, a->old_lens, a->n_seq,
                          a->n_k, a->n_v, a->eps, a->scale, a->out, a->out_stride, a->dev_status, a->stream);
}

int qsa_group_norm_packed(const qsa_group_norm_args* a) {
    if (!a) return QSA_ERR_ARG;
    return qsa_group_norm(a->x, a->x_stride, a->gate, a->gate_stride, a->type, a->weight, a->bias, a->w_type, a->per_group,
                          a->n_tok, a->n_groups, a->size, a->eps, a->centred, a->activation, a->out, a->out_stride,
                          a->stream);
}

}  // extern "C"

// linear.cuh -- arguments and launchers of the layers that keep a state per sequence: the
// short convolution (short_conv.cu), the gated delta rule over prompts (delta_prompt.cu)
// and per token (delta_step.cu), and the group norm (group_norm.cu).  Called by
// capi_linear.cu after argument validation.
#pragma once
#include "serve.cuh"

namespace qsa {

struct ConvArgs {
    const uint16_t* x;
    long long x_stride;           // elements from one token to the next
    int type;
    const void* weight;           // [n_ch][width]
    const void* bias;             // [n_ch], or null
    int w_type, width, activation;
    uint16_t* state;              // [n_slots][width - 1][n_ch]
    const int32_t* state_slots;
    int n_slots;
    const int32_t* old_lens;      // or null: every sequence goes on
    const int32_t* cu_tokens;     // or null: one token to every sequence
    int n_seq, n_tok, n_ch;
    uint16_t* out;
    long long out_stride;
    int32_t* dev_status;
};

bool short_conv_fits(long long n_tok, long long n_ch);   // into one launch
cudaError_t launch_short_conv(const ConvArgs& a, cudaStream_t stream);

struct DeltaArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    long long q_stride, k_stride, v_stride;
    int type;
    const uint16_t* a;
    const uint16_t* b;
    long long a_stride, b_stride;
    const float* a_log;           // [n_v]
    const float* dt_bias;         // [n_v]
    float* state;                 // [n_slots][n_v][128 value][128 key]
    const int32_t* state_slots;
    int n_slots;
    const int32_t* old_lens;      // or null
    const int32_t* cu_tokens;     // null for launch_delta_step: one token to every sequence
    int n_seq, n_tok, n_k, n_v;
    float eps, scale;
    uint16_t* out;
    long long out_stride;
    uint8_t* workspace;
    int32_t* dev_status;
    int chunked_from;             // delta_prompt.cu: the fewest tokens of a sequence that goes by chunks
    int n_split;                  // delta_prompt.cu: the most segments a sequence's chunks are cut into
};

cudaError_t launch_delta_step(const DeltaArgs& a, cudaStream_t stream);
// Of a step's sequences (cu_tokens) those of up to kDeltaShort tokens, token by token: a chunk of any length takes its SM for as
// long as a full one.  With 32 value heads, in a graph, token by token and by chunks: 1 sequence x 16 tokens 6.9 and 17.4 us,
// 1 x 32 11.6 and 17.5, 8 x 24 30.0 and 34.2, 64 x 24 182 and 218, 8 x 32 37.6 and 34.4, 64 x 32 235 and 220; 1 x 40 14.4 and
// 17.5, 8 x 40 45.5 and 34.5.  The border lies at some 45 tokens for one sequence and near 28 for many; this is one number for both.
constexpr int kDeltaShort = 32;
cudaError_t launch_delta_short(const DeltaArgs& a, cudaStream_t stream);
size_t delta_prompt_workspace(int n_tok, int n_seq, int n_k, int n_v);
cudaError_t launch_delta_prompt(const DeltaArgs& a, cudaStream_t stream);

struct NormArgs {
    const uint16_t* x;
    const uint16_t* gate;         // or null
    long long x_stride, gate_stride;
    int type;
    const void* weight;           // [size] or [n_groups][size], or null
    const void* bias;
    int w_type, per_group, n_tok, n_groups, size;
    float eps;
    int centred, activation;
    uint16_t* out;
    long long out_stride;
};

bool group_norm_fits(long long n_tok, long long n_groups, int size);   // into one launch
cudaError_t launch_group_norm(const NormArgs& a, cudaStream_t stream);

// ---------------------------------------------------------------- device helpers
__device__ __forceinline__ float to_f32(uint16_t v, int type) {
    return type == QSA_F16 ? __half2float(__ushort_as_half(v)) : __uint_as_float((uint32_t)v << 16);
}

// Eight consecutive elements of a 16-byte aligned array of `type` (16 bits) or FP32.
__device__ __forceinline__ void load8(const void* p, size_t at, int type, float (&x)[8]) {
    if (type == QSA_F32) {
        const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        const float4 u = src[0], v = src[1];
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
    } else {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at), type, x);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8], int type) {
    return make_uint4(pack2(x[0], x[1], type), pack2(x[2], x[3], type), pack2(x[4], x[5], type), pack2(x[6], x[7], type));
}

// ---------------------------------------------------------------- two FP32 at a time
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float x, float y) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpair(f2 p, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Eight consecutive 16-bit elements as four pairs, and back.
__device__ __forceinline__ void unpack_pairs(const uint4& w, int type, f2 (&x)[4]) {
    float f[8];
    unpack8(w, type, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = pair(f[2 * j], f[2 * j + 1]);
}
__device__ __forceinline__ uint4 pack_pairs(const f2 (&x)[4], int type) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) unpair(x[j], f[2 * j], f[2 * j + 1]);
    return pack8(f, type);
}
__device__ __forceinline__ void load_pairs(const void* p, size_t at, int type, f2 (&x)[4]) {
    float f[8];
    load8(p, at, type, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = pair(f[2 * j], f[2 * j + 1]);
}

// x / (1 + e^-x), good to a few 2^-22 (the results are rounded to 16 bits).
__device__ __forceinline__ f2 silu2(f2 x) {
    float a, b;
    unpair(mul2(x, pair(-kLog2e, -kLog2e)), a, b);
    unpair(add2(pair(fast_exp2(a), fast_exp2(b)), pair(1.f, 1.f)), a, b);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
    return mul2(x, pair(a, b));
}

// The decay's logarithm and the new value's weight, from the layer's two gate inputs.
__device__ __forceinline__ float log_decay(float a, float dt_bias, float a_log) {
    const float u = a + dt_bias, soft = fmaxf(u, 0.f) + log1pf(expf(-fabsf(u)));
    return -expf(a_log) * soft;
}
__device__ __forceinline__ float sigmoid(float b) { return __fdiv_rn(1.f, 1.f + expf(-b)); }

// First and last (exclusive) token of sequence s; bounds that fall or lie outside the arrays are clamped.
__device__ __forceinline__ int2 tokens_of(const int32_t* cu_tokens, int s, int n_tok) {
    if (!cu_tokens) return make_int2(s, s + 1);
    const int lo = min(max(cu_tokens[s], 0), n_tok);
    return make_int2(lo, min(max(cu_tokens[s + 1], lo), n_tok));
}
__device__ __forceinline__ bool tokens_bad(const int32_t* cu_tokens, int s, int n_tok) {
    if (!cu_tokens) return false;
    const int lo = cu_tokens[s], hi = cu_tokens[s + 1];
    return lo < 0 || hi < lo || hi > n_tok || (s == 0 && lo != 0);
}

}  // namespace qsa

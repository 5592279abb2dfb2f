// delta_step.cu -- the gated delta rule token by token (qsa_delta_step, and a prompt step's shortest sequences).
//
// With S the state (value by key), one pass over it gives S k and S q of the old state, and
//     new = beta (v - alpha S k),  out = alpha S q + new (k . q),  S = alpha S + new k^T:
// 7 flops for 8 bytes, so bytes are all: each state is read and written once, in FP32.
//
// Eight threads take a state row (one value dim), each the 16-byte pieces l, l + 8, l + 16,
// l + 24 of its 128 key dims, so that a warp's loads and stores are four whole 128-byte
// lines; S k and S q are summed over the eight by three exchanges.  A warp has kStepRows rows,
// all of whose loads are on their way before the first is used.
#include "linear.cuh"

namespace qsa {
namespace {

constexpr int kStepWarps = 4;
constexpr int kStepPasses = 4;                       // of four rows each, to a warp
constexpr int kStepRows = kStepWarps * kStepPasses * 4;   // state rows (value dims) to a block

__device__ __forceinline__ float sum8(float x) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// What a token brings: this thread's 16 key dims of its key and query, 4 (l + 8 i) .. + 3, its value dims, the gates' inputs.
struct Token {
    uint2 k[4], q[4];
    uint16_t v[kStepPasses], a, b;
};
template <int TYPE>
__device__ __forceinline__ void two_words(const uint2& w, float* x) {
    float f[8];
    unpack8(make_uint4(w.x, w.y, 0u, 0u), TYPE, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = f[j];
}

// SHORT: the sequences of up to kDeltaShort tokens of a step, their bounds from cu_tokens; otherwise one token each.
template <int TYPE, bool SHORT>
__global__ void __launch_bounds__(32 * kStepWarps) delta_step_kernel(const __grid_constant__ DeltaArgs a) {
    constexpr int kParts = kHeadDim / kStepRows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7;
    const unsigned item = blockIdx.x / kParts, s = item / (unsigned)a.n_v, h = item - s * (unsigned)a.n_v;
    const int row0 = (int)(blockIdx.x % kParts) * kStepRows + warp * (kStepPasses * 4) + (lane >> 3);
    const int kh = (int)h / (a.n_v / a.n_k);
    wait_for_stream();
    const int slot = a.state_slots[s];
    int2 span = make_int2((int)s, (int)s + 1);
    if (SHORT) {
        span = tokens_of(a.cu_tokens, (int)s, a.n_tok);
        if (span.y - span.x > kDeltaShort) return;   // the chunks' kernels have it, and report what is wrong with it
    }
    auto ask = [&](int t) {
        Token x;
        const uint16_t* k = a.k + (long long)t * a.k_stride + (size_t)kh * kHeadDim + 4 * l;
        const uint16_t* q = a.q + (long long)t * a.q_stride + (size_t)kh * kHeadDim + 4 * l;
        const uint16_t* v = a.v + (long long)t * a.v_stride + (size_t)h * kHeadDim + row0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x.k[i] = *reinterpret_cast<const uint2*>(k + 32 * i);
            x.q[i] = *reinterpret_cast<const uint2*>(q + 32 * i);
        }
#pragma unroll
        for (int p = 0; p < kStepPasses; ++p) x.v[p] = v[4 * p];
        x.a = a.a[(long long)t * a.a_stride + h], x.b = a.b[(long long)t * a.b_stride + h];
        return x;
    };
    Token next;
    if (!SHORT || span.x < span.y) next = ask(span.x);
    if (threadIdx.x == 0 && h == 0 && blockIdx.x % kParts == 0) {
        if (slot >= a.n_slots) report(a.dev_status, QSA_DEV_BAD_STATE);
        if (SHORT && tokens_bad(a.cu_tokens, (int)s, a.n_tok)) report(a.dev_status, QSA_DEV_BAD_SEQ_LEN);
    }
    if (slot < 0 || slot >= a.n_slots) return;
    const bool fresh = a.old_lens && a.old_lens[s] <= 0;
    if (SHORT && span.x == span.y && !fresh) return;
    float4* state = reinterpret_cast<float4*>(a.state + ((size_t)slot * a.n_v + h) * kHeadDim * kHeadDim) + row0 * (kHeadDim / 4) + l;
    float4 st[kStepPasses][4];
#pragma unroll
    for (int p = 0; p < kStepPasses; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            st[p][i] = fresh ? make_float4(0.f, 0.f, 0.f, 0.f) : state[4 * p * (kHeadDim / 4) + 8 * i];
    const float dt_bias = a.dt_bias[h], a_log = a.a_log[h];
#pragma unroll 1
    for (int t = span.x; t < span.y; ++t) {
        const Token x = next;
        if (SHORT && t + 1 < span.y) next = ask(t + 1);
        float k[16], q[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            two_words<TYPE>(x.k[i], k + 4 * i);
            two_words<TYPE>(x.q[i], q + 4 * i);
        }
        float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            kk = fmaf(k[j], k[j], kk);
            qq = fmaf(q[j], q[j], qq);
            kq = fmaf(k[j], q[j], kq);
        }
        const float rk = __frsqrt_rn(sum8(kk) + a.eps), rq = __frsqrt_rn(sum8(qq) + a.eps) * a.scale;
        kq = sum8(kq) * rk * rq;
#pragma unroll
        for (int j = 0; j < 16; ++j) k[j] *= rk;
        const float alpha = expf(log_decay(to_f32(x.a, TYPE), dt_bias, a_log)), beta = sigmoid(to_f32(x.b, TYPE));
#pragma unroll
        for (int p = 0; p < kStepPasses; ++p) {
            float sk = 0.f, sq = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                st[p][i].x *= alpha, st[p][i].y *= alpha, st[p][i].z *= alpha, st[p][i].w *= alpha;
                sk = fmaf(st[p][i].x, k[4 * i], sk), sk = fmaf(st[p][i].y, k[4 * i + 1], sk);
                sk = fmaf(st[p][i].z, k[4 * i + 2], sk), sk = fmaf(st[p][i].w, k[4 * i + 3], sk);
                sq = fmaf(st[p][i].x, q[4 * i], sq), sq = fmaf(st[p][i].y, q[4 * i + 1], sq);
                sq = fmaf(st[p][i].z, q[4 * i + 2], sq), sq = fmaf(st[p][i].w, q[4 * i + 3], sq);
            }
            sk = sum8(sk), sq = sum8(sq) * rq;
            const float added = beta * (to_f32(x.v[p], TYPE) - sk);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                st[p][i].x = fmaf(added, k[4 * i], st[p][i].x), st[p][i].y = fmaf(added, k[4 * i + 1], st[p][i].y);
                st[p][i].z = fmaf(added, k[4 * i + 2], st[p][i].z), st[p][i].w = fmaf(added, k[4 * i + 3], st[p][i].w);
                if (!SHORT) state[4 * p * (kHeadDim / 4) + 8 * i] = st[p][i];
            }
            if (l == 0)
                a.out[(long long)t * a.out_stride + (size_t)h * kHeadDim + row0 + 4 * p] = (uint16_t)pack2(fmaf(added, kq, sq), 0.f, TYPE);
        }
    }
    if (SHORT) {
#pragma unroll
        for (int p = 0; p < kStepPasses; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i) state[4 * p * (kHeadDim / 4) + 8 * i] = st[p][i];
    }
}

template <int TYPE, bool SHORT>
cudaError_t launch_tokens(const DeltaArgs& a, cudaStream_t stream) {
    const long long grid = (long long)a.n_seq * a.n_v * (kHeadDim / kStepRows);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_overlapped(delta_step_kernel<TYPE, SHORT>, dim3((unsigned)grid), 32 * kStepWarps, 0, stream, a);
}

}  // namespace

cudaError_t launch_delta_step(const DeltaArgs& a, cudaStream_t stream) {
    return a.type == QSA_F16 ? launch_tokens<QSA_F16, false>(a, stream) : launch_tokens<QSA_BF16, false>(a, stream);
}

cudaError_t launch_delta_short(const DeltaArgs& a, cudaStream_t stream) {
    return a.type == QSA_F16 ? launch_tokens<QSA_F16, true>(a, stream) : launch_tokens<QSA_BF16, true>(a, stream);
}

}  // namespace qsa

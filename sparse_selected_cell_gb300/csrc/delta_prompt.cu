// delta_prompt.cu -- the gated delta rule over the new tokens of several sequences (qsa_delta_prompt).
//
// The simplest form: a block to (sequence, value head, quarter of the value dims) holds its
// part of the state in registers and goes through the tokens one by one,
//     new = beta (v - alpha S k),  S = alpha S + new k^T,  out = S q.
// Eight threads to a state row, 16 key dims each.  Bound by the chain of tokens.
#include "linear.cuh"

namespace qsa {
namespace {

__device__ __forceinline__ float sum8(float x) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

constexpr int kWarps = 4, kRows = 32;

template <int TYPE>
__global__ void __launch_bounds__(32 * kWarps) delta_prompt_kernel(const __grid_constant__ DeltaArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7;
    const unsigned item = blockIdx.x / 4, s = item / (unsigned)a.n_v, h = item - s * (unsigned)a.n_v;
    const int row0 = (int)(blockIdx.x & 3) * kRows + warp * 8 + (lane >> 3);
    wait_for_stream();
    const int slot = a.state_slots[s];
    const int2 span = tokens_of(a.cu_tokens, (int)s, a.n_tok);
    if (h == 0 && (blockIdx.x & 3) == 0 && threadIdx.x == 0) {
        if (tokens_bad(a.cu_tokens, (int)s, a.n_tok)) report(a.dev_status, QSA_DEV_BAD_SEQ_LEN);
        if (slot >= a.n_slots) report(a.dev_status, QSA_DEV_BAD_STATE);
    }
    if (slot < 0 || slot >= a.n_slots) return;
    const bool fresh = a.old_lens && a.old_lens[s] <= 0;
    const int kh = (int)h / (a.n_v / a.n_k);
    float* state = a.state + ((size_t)slot * a.n_v + h) * kHeadDim * kHeadDim;
    float st[2][16];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < 16; ++i) st[p][i] = fresh ? 0.f : state[(row0 + 4 * p) * kHeadDim + 16 * l + i];
    for (long long t = span.x; t < span.y; ++t) {
        float k[16], q[16], kk = 0.f, qq = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            k[i] = to_f32(a.k[t * a.k_stride + (size_t)kh * kHeadDim + 16 * l + i], TYPE);
            q[i] = to_f32(a.q[t * a.q_stride + (size_t)kh * kHeadDim + 16 * l + i], TYPE);
            kk = fmaf(k[i], k[i], kk);
            qq = fmaf(q[i], q[i], qq);
        }
        const float rk = __frsqrt_rn(sum8(kk) + a.eps), rq = __frsqrt_rn(sum8(qq) + a.eps) * a.scale;
        const float alpha = expf(log_decay(to_f32(a.a[t * a.a_stride + h], TYPE), a.dt_bias[h], a.a_log[h]));
        const float beta = sigmoid(to_f32(a.b[t * a.b_stride + h], TYPE));
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            float sk = 0.f, sq = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                st[p][i] *= alpha;
                sk = fmaf(st[p][i], k[i], sk);
            }
            const float v = to_f32(a.v[t * a.v_stride + (size_t)h * kHeadDim + row0 + 4 * p], TYPE);
            const float fresh_v = beta * (v - sum8(sk) * rk) * rk;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                st[p][i] = fmaf(fresh_v, k[i], st[p][i]);
                sq = fmaf(st[p][i], q[i], sq);
            }
            sq = sum8(sq) * rq;
            if (l == 0) a.out[t * a.out_stride + (size_t)h * kHeadDim + row0 + 4 * p] = (uint16_t)pack2(sq, 0.f, TYPE);
        }
    }
    if (span.x == span.y && !fresh) return;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < 16; ++i) state[(row0 + 4 * p) * kHeadDim + 16 * l + i] = st[p][i];
}

}  // namespace

size_t delta_prompt_workspace(int n_tok, int n_seq, int n_k, int n_v) {
    const size_t chunks = (size_t)n_tok / 64 + n_seq + 1;
    return chunks * ((size_t)n_k * 32768 + (size_t)n_v * 28672) + 256;
}

cudaError_t launch_delta_prompt(const DeltaArgs& a, cudaStream_t stream) {
    const long long grid = (long long)a.n_seq * a.n_v * 4;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (a.type == QSA_F16)
        return launch_overlapped(delta_prompt_kernel<QSA_F16>, dim3((unsigned)grid), 32 * kWarps, 0, stream, a);
    return launch_overlapped(delta_prompt_kernel<QSA_BF16>, dim3((unsigned)grid), 32 * kWarps, 0, stream, a);
}

}  // namespace qsa

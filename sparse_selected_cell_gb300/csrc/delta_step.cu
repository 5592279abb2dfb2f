// delta_step.cu -- the gated delta rule token by token (qsa_delta_step).
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

// This thread's 16 key dims of a row: 4 (l + 8 i) .. + 3.
__device__ __forceinline__ void load_dims(const uint16_t* row, int l, int type, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint2 w = *reinterpret_cast<const uint2*>(row + 4 * (l + 8 * i));
        float f[8];
        unpack8(make_uint4(w.x, w.y, 0u, 0u), type, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * i + j] = f[j];
    }
}

template <int TYPE>
__global__ void __launch_bounds__(32 * kStepWarps) delta_step_kernel(const __grid_constant__ DeltaArgs a) {
    constexpr int kParts = kHeadDim / kStepRows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7;
    const unsigned item = blockIdx.x / kParts, s = item / (unsigned)a.n_v, h = item - s * (unsigned)a.n_v;
    const int row0 = (int)(blockIdx.x % kParts) * kStepRows + warp * (kStepPasses * 4) + (lane >> 3);
    wait_for_stream();
    const int slot = a.state_slots[s];
    const long long t = (long long)s;
    const int kh = (int)h / (a.n_v / a.n_k);
    float k[16], q[16];
    load_dims(a.k + t * a.k_stride + (size_t)kh * kHeadDim, l, TYPE, k);
    load_dims(a.q + t * a.q_stride + (size_t)kh * kHeadDim, l, TYPE, q);
    const float ga = to_f32(a.a[t * a.a_stride + h], TYPE), gb = to_f32(a.b[t * a.b_stride + h], TYPE);
    if (slot < 0 || slot >= a.n_slots) {
        if (slot >= 0 && h == 0 && blockIdx.x % kParts == 0 && threadIdx.x == 0) report(a.dev_status, QSA_DEV_BAD_STATE);
        return;
    }
    const bool fresh = a.old_lens && a.old_lens[s] <= 0;
    float4* state = reinterpret_cast<float4*>(a.state + ((size_t)slot * a.n_v + h) * kHeadDim * kHeadDim);
    float4 st[kStepPasses][4];
#pragma unroll
    for (int p = 0; p < kStepPasses; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            st[p][i] = fresh ? make_float4(0.f, 0.f, 0.f, 0.f) : state[(row0 + 4 * p) * (kHeadDim / 4) + l + 8 * i];
    float v[kStepPasses];
#pragma unroll
    for (int p = 0; p < kStepPasses; ++p) v[p] = to_f32(a.v[t * a.v_stride + (size_t)h * kHeadDim + row0 + 4 * p], TYPE);

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
    const float alpha = expf(log_decay(ga, a.dt_bias[h], a.a_log[h])), beta = sigmoid(gb);
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
        const float fresh_v = beta * (v[p] - sk);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            st[p][i].x = fmaf(fresh_v, k[4 * i], st[p][i].x), st[p][i].y = fmaf(fresh_v, k[4 * i + 1], st[p][i].y);
            st[p][i].z = fmaf(fresh_v, k[4 * i + 2], st[p][i].z), st[p][i].w = fmaf(fresh_v, k[4 * i + 3], st[p][i].w);
            state[(row0 + 4 * p) * (kHeadDim / 4) + l + 8 * i] = st[p][i];
        }
        if (l == 0) {
            const float o = fmaf(fresh_v, kq, sq);
            a.out[t * a.out_stride + (size_t)h * kHeadDim + row0 + 4 * p] = (uint16_t)pack2(o, 0.f, TYPE);
        }
    }
}

}  // namespace

cudaError_t launch_delta_step(const DeltaArgs& a, cudaStream_t stream) {
    const long long grid = (long long)a.n_seq * a.n_v * (kHeadDim / kStepRows);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (a.type == QSA_F16)
        return launch_overlapped(delta_step_kernel<QSA_F16>, dim3((unsigned)grid), 32 * kStepWarps, 0, stream, a);
    return launch_overlapped(delta_step_kernel<QSA_BF16>, dim3((unsigned)grid), 32 * kStepWarps, 0, stream, a);
}

}  // namespace qsa

// delta_step.cu -- the gated delta rule token by token (qsa_delta_step, and a prompt step's shortest sequences).
//
// With S the state (value by key), one pass over it gives S k and S q of the old state, and
//     new = beta (v - alpha S k),  out = alpha S q + new (k . q),  S = alpha S + new k^T:
// 7 flops for 8 bytes, so bytes are all: each state is read and written once, in FP32.
//
// Eight threads take a state row (one value dim), each the 16-byte pieces l, l + 8, l + 16,
// l + 24 of its 128 key dims, so that a warp's loads and stores are four whole 128-byte
// lines; S k and S q are summed over the eight by three exchanges.  A warp has 16 rows, all of
// whose loads are on their way before the first is used.
//
// With 32 value heads, 61 sequences (257 MB) take 39.6 us, 6.49 TB/s, 0.96 of what a plain copy
// reaches; 768 (3.2 GB) 460 us, 7.05 TB/s (reads and writes of the same lines suit HBM better
// than a copy's); one 2.4 us in a graph, launch and two loads behind one another.
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

template <int TYPE>
__device__ __forceinline__ void two_words(const uint2& w, float* x) {
    float f[8];
    unpack8(make_uint4(w.x, w.y, 0u, 0u), TYPE, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = f[j];
}

// A token's factors, from its key and query (16 elements of each to each of eight threads), which are brought to their
// lengths, the query's with the scale.
struct Token {
    float alpha, beta, kq;
};
__device__ __forceinline__ Token token_of(float (&k)[16], float (&q)[16], float log_alpha, float beta, float eps, float scale) {
    float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        kk = fmaf(k[j], k[j], kk);
        qq = fmaf(q[j], q[j], qq);
        kq = fmaf(k[j], q[j], kq);
    }
    const float rk = __frsqrt_rn(sum8(kk) + eps), rq = __frsqrt_rn(sum8(qq) + eps) * scale;
#pragma unroll
    for (int j = 0; j < 16; ++j) k[j] *= rk, q[j] *= rq;
    return Token{expf(log_alpha), beta, sum8(kq) * rk * rq};
}

template <int TYPE>
__global__ void __launch_bounds__(32 * kStepWarps) delta_step_kernel(const __grid_constant__ DeltaArgs a) {
    constexpr int kParts = kHeadDim / kStepRows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7;
    const unsigned item = blockIdx.x / kParts, s = item / (unsigned)a.n_v, h = item - s * (unsigned)a.n_v;
    const int row0 = (int)(blockIdx.x % kParts) * kStepRows + warp * (kStepPasses * 4) + (lane >> 3);
    const int kh = (int)h / (a.n_v / a.n_k);
    wait_for_stream();
    const int slot = a.state_slots[s];
    const uint16_t* key = a.k + (long long)s * a.k_stride + (size_t)kh * kHeadDim + 4 * l;
    const uint16_t* query = a.q + (long long)s * a.q_stride + (size_t)kh * kHeadDim + 4 * l;
    const uint16_t* value = a.v + (long long)s * a.v_stride + (size_t)h * kHeadDim + row0;
    uint2 rk[4], rq[4];
    uint16_t rv[kStepPasses];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        rk[i] = *reinterpret_cast<const uint2*>(key + 32 * i);
        rq[i] = *reinterpret_cast<const uint2*>(query + 32 * i);
    }
#pragma unroll
    for (int p = 0; p < kStepPasses; ++p) rv[p] = value[4 * p];
    const uint16_t ra = a.a[(long long)s * a.a_stride + h], rb = a.b[(long long)s * a.b_stride + h];
    if (threadIdx.x == 0 && h == 0 && blockIdx.x % kParts == 0 && slot >= a.n_slots) report(a.dev_status, QSA_DEV_BAD_STATE);
    if (slot < 0 || slot >= a.n_slots) return;
    const bool fresh = a.old_lens && a.old_lens[s] <= 0;
    float4* state = reinterpret_cast<float4*>(a.state + ((size_t)slot * a.n_v + h) * kHeadDim * kHeadDim) + row0 * (kHeadDim / 4) + l;
    float4 st[kStepPasses][4];
#pragma unroll
    for (int p = 0; p < kStepPasses; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            st[p][i] = fresh ? make_float4(0.f, 0.f, 0.f, 0.f) : state[4 * p * (kHeadDim / 4) + 8 * i];
    float k[16], q[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        two_words<TYPE>(rk[i], k + 4 * i);
        two_words<TYPE>(rq[i], q + 4 * i);
    }
    const Token t = token_of(k, q, log_decay(to_f32(ra, TYPE), a.dt_bias[h], a.a_log[h]), sigmoid(to_f32(rb, TYPE)), a.eps, a.scale);
#pragma unroll
    for (int p = 0; p < kStepPasses; ++p) {
        float sk = 0.f, sq = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            st[p][i].x *= t.alpha, st[p][i].y *= t.alpha, st[p][i].z *= t.alpha, st[p][i].w *= t.alpha;
            sk = fmaf(st[p][i].x, k[4 * i], sk), sk = fmaf(st[p][i].y, k[4 * i + 1], sk);
            sk = fmaf(st[p][i].z, k[4 * i + 2], sk), sk = fmaf(st[p][i].w, k[4 * i + 3], sk);
            sq = fmaf(st[p][i].x, q[4 * i], sq), sq = fmaf(st[p][i].y, q[4 * i + 1], sq);
            sq = fmaf(st[p][i].z, q[4 * i + 2], sq), sq = fmaf(st[p][i].w, q[4 * i + 3], sq);
        }
        sk = sum8(sk), sq = sum8(sq);
        const float added = t.beta * (to_f32(rv[p], TYPE) - sk);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            st[p][i].x = fmaf(added, k[4 * i], st[p][i].x), st[p][i].y = fmaf(added, k[4 * i + 1], st[p][i].y);
            st[p][i].z = fmaf(added, k[4 * i + 2], st[p][i].z), st[p][i].w = fmaf(added, k[4 * i + 3], st[p][i].w);
            state[4 * p * (kHeadDim / 4) + 8 * i] = st[p][i];
        }
        if (l == 0)
            a.out[(long long)s * a.out_stride + (size_t)h * kHeadDim + row0 + 4 * p] = (uint16_t)pack2(fmaf(added, t.kq, sq), 0.f, TYPE);
    }
}

// A prompt step's sequences of up to kDeltaShort tokens.  What a token brings that does not need the state (its key and
// query with their factors, the gates) is formed for all tokens at once, eight threads to a token, and kept in shared memory;
// the chain from token to token is then S k, S q and the update, on pairs of FP32: 0.3 us a token (0.8 when each token's
// factors were formed in the chain).  Many sequences are bound by FP32 operations, four to a state element and token:
// 64 x 16 tokens x 32 heads take 112 us (126 with the chunks' kernels, which end at once), of which the states' bytes would need 40.
template <int TYPE>
__global__ void __launch_bounds__(32 * kStepWarps) delta_short_kernel(const __grid_constant__ DeltaArgs a) {
    constexpr int kParts = kHeadDim / kStepRows;
    static_assert(kStepRows == 64, "eight values to each thread of a token");
    __shared__ __align__(16) float s_k[kDeltaShort][kHeadDim], s_q[kDeltaShort][kHeadDim];
    __shared__ __align__(16) uint16_t s_v[kDeltaShort][kStepRows];   // values, then outputs
    __shared__ float4 s_t[kDeltaShort];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7;
    const unsigned item = blockIdx.x / kParts, s = item / (unsigned)a.n_v, h = item - s * (unsigned)a.n_v;
    const int part = (int)(blockIdx.x % kParts) * kStepRows, own = warp * (kStepPasses * 4) + (lane >> 3);   // its first row of the part's
    const int kh = (int)h / (a.n_v / a.n_k);
    wait_for_stream();
    const int slot = a.state_slots[s];
    const int2 span = tokens_of(a.cu_tokens, (int)s, a.n_tok);
    const int n = span.y - span.x;
    if (n > kDeltaShort) return;                     // the chunks' kernels have it, and report what is wrong with it
    if (threadIdx.x == 0 && h == 0 && part == 0) {
        if (slot >= a.n_slots) report(a.dev_status, QSA_DEV_BAD_STATE);
        if (tokens_bad(a.cu_tokens, (int)s, a.n_tok)) report(a.dev_status, QSA_DEV_BAD_SEQ_LEN);
    }
    const bool fresh = a.old_lens && a.old_lens[s] <= 0;
    if (slot < 0 || slot >= a.n_slots || (n == 0 && !fresh)) return;
    ulonglong2* state = reinterpret_cast<ulonglong2*>(a.state + ((size_t)slot * a.n_v + h) * kHeadDim * kHeadDim) + (part + own) * (kHeadDim / 4) + l;
    ulonglong2 st[kStepPasses][4];
#pragma unroll
    for (int p = 0; p < kStepPasses; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) st[p][i] = fresh ? make_ulonglong2(0ull, 0ull) : state[4 * p * (kHeadDim / 4) + 8 * i];
    const float dt_bias = a.dt_bias[h], a_log = a.a_log[h];
#pragma unroll 1
    for (int t0 = 0; t0 < n; t0 += 4 * kStepWarps) {
        const int t = t0 + 4 * warp + (lane >> 3);
        const long long at = span.x + min(t, n - 1);
        float k[16], q[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            two_words<TYPE>(*reinterpret_cast<const uint2*>(a.k + at * a.k_stride + (size_t)kh * kHeadDim + 4 * l + 32 * i), k + 4 * i);
            two_words<TYPE>(*reinterpret_cast<const uint2*>(a.q + at * a.q_stride + (size_t)kh * kHeadDim + 4 * l + 32 * i), q + 4 * i);
        }
        const uint4 v = *reinterpret_cast<const uint4*>(a.v + at * a.v_stride + (size_t)h * kHeadDim + part + 8 * l);
        const float ga = to_f32(a.a[at * a.a_stride + h], TYPE), gb = to_f32(a.b[at * a.b_stride + h], TYPE);
        const Token x = token_of(k, q, log_decay(ga, dt_bias, a_log), sigmoid(gb), a.eps, a.scale);
        if (t >= n) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            *reinterpret_cast<float4*>(&s_k[t][4 * l + 32 * i]) = make_float4(k[4 * i], k[4 * i + 1], k[4 * i + 2], k[4 * i + 3]);
            *reinterpret_cast<float4*>(&s_q[t][4 * l + 32 * i]) = make_float4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
        }
        *reinterpret_cast<uint4*>(&s_v[t][8 * l]) = v;
        if (l == 0) s_t[t] = make_float4(x.alpha, x.beta, x.kq, 0.f);
    }
    __syncthreads();
#pragma unroll 1
    for (int t = 0; t < n; ++t) {
        const float4 x = s_t[t];
        const f2 alpha = pair(x.x, x.x);
        ulonglong2 k[4], q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            k[i] = *reinterpret_cast<const ulonglong2*>(&s_k[t][4 * l + 32 * i]);
            q[i] = *reinterpret_cast<const ulonglong2*>(&s_q[t][4 * l + 32 * i]);
        }
        float sk[kStepPasses], sq[kStepPasses];
#pragma unroll
        for (int p = 0; p < kStepPasses; ++p) {
            f2 uk = 0ull, uq = 0ull;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                st[p][i].x = mul2(st[p][i].x, alpha), st[p][i].y = mul2(st[p][i].y, alpha);
                uk = fma2(st[p][i].x, k[i].x, uk), uk = fma2(st[p][i].y, k[i].y, uk);
                uq = fma2(st[p][i].x, q[i].x, uq), uq = fma2(st[p][i].y, q[i].y, uq);
            }
            float u, v;
            unpair(uk, u, v);
            sk[p] = u + v;
            unpair(uq, u, v);
            sq[p] = u + v;
        }
#pragma unroll
        for (int p = 0; p < kStepPasses; ++p) {
            sk[p] = sum8(sk[p]), sq[p] = sum8(sq[p]);
            const float added = x.y * (to_f32(s_v[t][own + 4 * p], TYPE) - sk[p]);
            const f2 a2 = pair(added, added);
#pragma unroll
            for (int i = 0; i < 4; ++i) st[p][i].x = fma2(a2, k[i].x, st[p][i].x), st[p][i].y = fma2(a2, k[i].y, st[p][i].y);
            __syncwarp();                            // the value has been read by all eight
            if (l == 0) s_v[t][own + 4 * p] = (uint16_t)pack2(fmaf(added, x.z, sq[p]), 0.f, TYPE);
        }
    }
#pragma unroll
    for (int p = 0; p < kStepPasses; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) state[4 * p * (kHeadDim / 4) + 8 * i] = st[p][i];
    __syncthreads();
    for (int i = threadIdx.x; i < 8 * n; i += 32 * kStepWarps)
        *reinterpret_cast<uint4*>(a.out + (long long)(span.x + (i >> 3)) * a.out_stride + (size_t)h * kHeadDim + part + 8 * (i & 7)) =
            *reinterpret_cast<const uint4*>(&s_v[i >> 3][8 * (i & 7)]);
}

template <class Kernel>
cudaError_t launch_tokens(Kernel kernel, const DeltaArgs& a, cudaStream_t stream) {
    const long long grid = (long long)a.n_seq * a.n_v * (kHeadDim / kStepRows);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_overlapped(kernel, dim3((unsigned)grid), 32 * kStepWarps, 0, stream, a);
}

}  // namespace

cudaError_t launch_delta_step(const DeltaArgs& a, cudaStream_t stream) {
    return a.type == QSA_F16 ? launch_tokens(delta_step_kernel<QSA_F16>, a, stream) : launch_tokens(delta_step_kernel<QSA_BF16>, a, stream);
}

cudaError_t launch_delta_short(const DeltaArgs& a, cudaStream_t stream) {
    return a.type == QSA_F16 ? launch_tokens(delta_short_kernel<QSA_F16>, a, stream) : launch_tokens(delta_short_kernel<QSA_BF16>, a, stream);
}

}  // namespace qsa

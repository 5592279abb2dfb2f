// group_norm.cu -- groups of a token's channels normalised, weighted and gated (qsa_group_norm).
//
// Bytes are all: x and the gate read once, out written once.  A group is held in registers
// by as many threads as it has 16-byte words, up to a warp (LANES, a power of two), each with
// PIECES words, or by a block's eight warps where it has more than 128 words; so the mean is
// taken first and the squares of what is left after it, in FP32, without a second read.
#include "linear.cuh"

namespace qsa {
namespace {

constexpr int kNormThreads = 256;

template <int LANES>
__device__ __forceinline__ float sum_over(float x, float* s_part) {
#pragma unroll
    for (int o = 1; o < (LANES < 32 ? LANES : 32); o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (LANES <= 32) return x;
    __syncthreads();                                 // the sums of the round before have been read
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < kNormThreads / 32; ++i) x += s_part[i];
    return x;
}

// A thread has words l, l + LANES, .. (PIECES of them) of ITEMS groups, kNormThreads / LANES apart, all asked for at once.
template <int TYPE, int LANES, int PIECES, int ITEMS>
__global__ void __launch_bounds__(kNormThreads) group_norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kRow = kNormThreads / LANES;       // groups side by side in a block
    __shared__ float s_part[kNormThreads / 32];
    const int l = threadIdx.x % LANES, words = a.size / 8;
    const unsigned groups = (unsigned)a.n_groups;
    const long long items = (long long)a.n_tok * a.n_groups, item0 = (long long)blockIdx.x * (kRow * ITEMS);
    // the block's first token by one wide division, its threads' from there in 32 bits
    const unsigned t0 = (unsigned)(item0 / groups), g0 = (unsigned)(item0 - (long long)t0 * groups) + threadIdx.x / LANES;
    wait_for_stream();
    uint4 rx[ITEMS][PIECES], rz[ITEMS][PIECES];
    long long tok[ITEMS];
    unsigned grp[ITEMS];
    bool live[ITEMS];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const unsigned from = g0 + k * kRow, more = from / groups;
        live[k] = item0 + threadIdx.x / LANES + k * kRow < items;
        tok[k] = (long long)t0 + more;
        grp[k] = from - more * groups;
        const uint16_t* x = a.x + tok[k] * a.x_stride + (size_t)grp[k] * a.size;
        const uint16_t* z = a.gate + tok[k] * a.gate_stride + (size_t)grp[k] * a.size;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int w = l + i * LANES;
            rx[k][i] = rz[k][i] = make_uint4(0, 0, 0, 0);
            if (live[k] && w < words) {
                rx[k][i] = *reinterpret_cast<const uint4*>(x + 8 * w);
                if (a.gate) rz[k][i] = *reinterpret_cast<const uint4*>(z + 8 * w);
            }
        }
    }
    const float inv = 1.f / (float)a.size;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        float mean = 0.f, sq = 0.f;
        if (a.centred) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                float f[8];
                unpack8(rx[k][i], TYPE, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) mean += f[j];
            }
            mean = sum_over<LANES>(mean, s_part) * inv;
        }
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            float f[8];
            unpack8(rx[k][i], TYPE, f);
            if (l + i * LANES < words) {
#pragma unroll
                for (int j = 0; j < 8; ++j) sq = fmaf(f[j] - mean, f[j] - mean, sq);
            }
        }
        const float r = __frsqrt_rn(fmaf(sum_over<LANES>(sq, s_part), inv, a.eps));
        uint16_t* out = a.out + tok[k] * a.out_stride + (size_t)grp[k] * a.size;
        const size_t w0 = a.per_group ? (size_t)grp[k] * a.size : 0;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int w = l + i * LANES;
            if (!live[k] || w >= words) continue;
            float y[8], p[8];
            unpack8(rx[k][i], TYPE, y);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = (y[j] - mean) * r;
            if (a.weight) {
                load8(a.weight, w0 + 8 * w, a.w_type, p);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] *= p[j];
            }
            if (a.bias) {
                load8(a.bias, w0 + 8 * w, a.w_type, p);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] += p[j];
            }
            if (a.gate) {
                unpack8(rz[k][i], TYPE, p);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] *= a.activation == QSA_ACT_SILU ? silu(p[j]) : p[j];
            } else if (a.activation == QSA_ACT_SILU) {
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = silu(y[j]);
            }
            *reinterpret_cast<uint4*>(out + 8 * w) = pack8(y, TYPE);
        }
    }
}

template <int TYPE, int LANES, int PIECES, int ITEMS>
cudaError_t launch_items(const NormArgs& a, cudaStream_t stream) {
    const long long items = (long long)a.n_tok * a.n_groups, per = (long long)kNormThreads / LANES * ITEMS, grid = (items + per - 1) / per;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_overlapped(group_norm_kernel<TYPE, LANES, PIECES, ITEMS>, dim3((unsigned)grid), kNormThreads, 0, stream, a);
}

// Two words to a thread, or four groups, once that still gives every SM a few blocks; below that one group a thread, for
// the shortest way through.
template <int TYPE, int LANES, int PIECES>
cudaError_t launch_lanes(const NormArgs& a, cudaStream_t stream) {
    constexpr int kItems = PIECES >= 4 ? 1 : PIECES == 2 ? 2 : 4;
    if (kItems > 1 && (long long)a.n_tok * a.n_groups * LANES >= 4LL * kNormThreads * kItems * 152)
        return launch_items<TYPE, LANES, PIECES, kItems>(a, stream);
    return launch_items<TYPE, LANES, PIECES, 1>(a, stream);
}

template <int TYPE>
cudaError_t launch_type(const NormArgs& a, cudaStream_t stream) {
    const int words = a.size / 8;
    if (words <= 1) return launch_lanes<TYPE, 1, 1>(a, stream);
    if (words <= 2) return launch_lanes<TYPE, 2, 1>(a, stream);
    if (words <= 4) return launch_lanes<TYPE, 4, 1>(a, stream);
    if (words <= 8) return launch_lanes<TYPE, 8, 1>(a, stream);
    if (words <= 16) return launch_lanes<TYPE, 16, 1>(a, stream);
    if (words <= 32) return launch_lanes<TYPE, 32, 1>(a, stream);
    if (words <= 64) return launch_lanes<TYPE, 32, 2>(a, stream);
    if (words <= 128) return launch_lanes<TYPE, 32, 4>(a, stream);
    if (words <= 512) return launch_lanes<TYPE, kNormThreads, 2>(a, stream);
    return launch_lanes<TYPE, kNormThreads, 4>(a, stream);
}

}  // namespace

cudaError_t launch_group_norm(const NormArgs& a, cudaStream_t stream) {
    return a.type == QSA_F16 ? launch_type<QSA_F16>(a, stream) : launch_type<QSA_BF16>(a, stream);
}

}  // namespace qsa

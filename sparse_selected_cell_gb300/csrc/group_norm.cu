// group_norm.cu -- groups of a token's channels normalised, weighted and gated (qsa_group_norm).
//
// Bytes are all: x and the gate read once, out written once.  A group is held in registers
// by as many threads as it has 16-byte words, up to a warp (LANES, a power of two), each with
// PIECES words, or by a block's eight warps where it has more than 128 words; so the mean is
// taken first and the squares of what is left after it, in FP32, without a second read.
//
// 8,192 tokens x 32 groups x 128 with a gate (201 MB) take 34.1 us, 5.9 TB/s, 0.87 of what a
// plain copy reaches: 70 % of the issue slots are taken (unpacking, SiLU's two special functions an
// element, packing), so the loads do not queue up as a copy's do.
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
__global__ void __launch_bounds__(kNormThreads, ITEMS == 2 ? 6 : 1) group_norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kRow = kNormThreads / LANES;       // groups side by side in a block
    __shared__ float s_part[kNormThreads / 32];
    const int l = threadIdx.x % LANES, words = a.size / 8;
    const unsigned groups = (unsigned)a.n_groups;
    const long long item0 = (long long)blockIdx.x * (kRow * ITEMS);
    // the block's first token by one wide division, its threads' from there in 32 bits
    const unsigned t0 = (unsigned)(item0 / groups), g0 = (unsigned)(item0 - (long long)t0 * groups) + threadIdx.x / LANES;
    wait_for_stream();
    uint4 rx[ITEMS][PIECES], rz[ITEMS][PIECES];
    unsigned tok[ITEMS], grp[ITEMS];
    bool live[ITEMS];
    tok[0] = g0 / groups, grp[0] = g0 - tok[0] * groups, tok[0] += t0;
    const unsigned more = kRow / groups, rest = kRow - more * groups;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        if (k > 0) {
            const bool over = grp[k - 1] + rest >= groups;
            tok[k] = tok[k - 1] + more + (over ? 1u : 0u), grp[k] = grp[k - 1] + rest - (over ? groups : 0u);
        }
        live[k] = tok[k] < (unsigned)a.n_tok;
        const uint16_t* x = a.x + (long long)tok[k] * a.x_stride + (size_t)grp[k] * a.size;
        const uint16_t* z = a.gate + (long long)tok[k] * a.gate_stride + (size_t)grp[k] * a.size;
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
    const bool silu = a.activation == QSA_ACT_SILU;
    // weights that all groups share are read once; conditions that all threads share stay outside the elements' loops
    constexpr bool kKeep = PIECES == 1;
    f2 weight[4], bias[4];
    auto shift = [&](int w, size_t w0) {
        if (a.weight) load_pairs(a.weight, w0 + 8 * w, a.w_type, weight);
        if (a.bias) load_pairs(a.bias, w0 + 8 * w, a.w_type, bias);
    };
    if (kKeep && !a.per_group && l < words) shift(l, 0);
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        float mean = 0.f;
        if (a.centred) {
            f2 sum = 0ull;
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                f2 x[4];
                unpack_pairs(rx[k][i], TYPE, x);
                sum = add2(sum, add2(add2(x[0], x[1]), add2(x[2], x[3])));
            }
            float u, v;
            unpair(sum, u, v);
            mean = sum_over<LANES>(u + v, s_part) * inv;
        }
        const f2 less = pair(-mean, -mean);
        f2 sq = 0ull;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            if (l + i * LANES >= words) continue;
            f2 x[4];
            unpack_pairs(rx[k][i], TYPE, x);
            if (a.centred) {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = add2(x[j], less);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) sq = fma2(x[j], x[j], sq);
        }
        float u, v;
        unpair(sq, u, v);
        const float r = rsqrtf(fmaf(sum_over<LANES>(u + v, s_part), inv, a.eps));
        const f2 r2 = pair(r, r);
        uint16_t* out = a.out + (long long)tok[k] * a.out_stride + (size_t)grp[k] * a.size;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int w = l + i * LANES;
            if (!live[k] || w >= words) continue;
            f2 y[4];
            unpack_pairs(rx[k][i], TYPE, y);
            if (a.centred) {
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = add2(y[j], less);
            }
            if (!kKeep || a.per_group) shift(w, a.per_group ? (size_t)grp[k] * a.size : 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], r2);
            if (a.weight) {
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], weight[j]);
            }
            if (a.bias) {
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = add2(y[j], bias[j]);
            }
            if (a.gate) {
                f2 z[4];
                unpack_pairs(rz[k][i], TYPE, z);
                if (silu) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) z[j] = silu2(z[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], z[j]);
            } else if (silu) {
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = silu2(y[j]);
            }
            *reinterpret_cast<uint4*>(out + 8 * w) = pack_pairs(y, TYPE);
        }
    }
}

template <int TYPE, int LANES, int PIECES, int ITEMS>
cudaError_t launch_items(const NormArgs& a, cudaStream_t stream) {
    const long long items = (long long)a.n_tok * a.n_groups, per = (long long)kNormThreads / LANES * ITEMS, grid = (items + per - 1) / per;
    return launch_overlapped(group_norm_kernel<TYPE, LANES, PIECES, ITEMS>, dim3((unsigned)grid), kNormThreads, 0, stream, a);
}

// Two groups to a thread, six blocks to an SM (40 registers, some of them spilled), once that still gives every SM a few blocks: 8,192 tokens x 32 x 128 with a gate
// 33.8 us instead of 38.0 (four groups in as many registers as they take: 37.8; in 40 registers: 42.4).  Below that one group a
// thread, for the shortest way through: 512 x 32 x 128 3.5 us instead of 3.9.
template <int TYPE, int LANES, int PIECES>
cudaError_t launch_lanes(const NormArgs& a, cudaStream_t stream) {
    constexpr int kItems = PIECES == 1 ? 2 : 1;
    if (kItems > 1) {
        int dev = 0, sms = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        if ((long long)a.n_tok * a.n_groups * LANES >= 4LL * kNormThreads * kItems * sms)
            return launch_items<TYPE, LANES, PIECES, kItems>(a, stream);
    }
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

// A block has one group of more than 128 words, eight of more than 32; of shorter ones, being many, two to every thread group.
bool group_norm_fits(long long n_tok, long long n_groups, int size) {
    const int words = size / 8;
    int lanes = 1;
    while (lanes < words && lanes < 32) lanes *= 2;
    const long long each = words > 128 ? 1 : words > 32 ? kNormThreads / 32 : kNormThreads / lanes * 2;
    return (n_tok * n_groups + each - 1) / each <= 0x7fffffffLL;
}

cudaError_t launch_group_norm(const NormArgs& a, cudaStream_t stream) {
    return a.type == QSA_F16 ? launch_type<QSA_F16>(a, stream) : launch_type<QSA_BF16>(a, stream);
}

}  // namespace qsa

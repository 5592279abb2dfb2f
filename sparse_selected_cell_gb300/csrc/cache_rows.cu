// cache_rows.cu -- rows on their way into and out of the paged INT8 cache: rotary
// positions with the quantising write (qsa_rope, qsa_rope_append) and the
// dequantising read (qsa_cache_gather).
//
// Rotation: pair j of a token's query or key row is turned by positions[axis_j] *
// inv_freq[j].  The angle is kept as a fraction of a turn in 64-bit fixed point:
// f = frac(inv_freq / 2 pi) * 2^64, and position * f modulo 2^64 IS the fraction
// of the turn that is left, whatever the position's size or sign; no range
// reduction loses bits.  Its top 32 bits go to sincospif.  f comes from the frequency's
// 53 bits by one integer product (FP64 arithmetic is slow on this GPU).
//
// Layout: one CTA per token, eight threads per 128-element row, so the token's 64
// sines and cosines are formed once, into shared memory, and a thread keeps the
// eight pairs it always works on in registers for all its rows.  Thread l of a row's
// eight holds the 16-byte pieces l and l + n_pairs / 8 of the row, which are the two
// halves of pairs 8l .. 8l + 7 (of interleaved pairs pieces l and l + 8, pairs 4l .. and
// 4l + 32 ..): every load and store is 16 bytes wide and eight threads' are 128
// consecutive bytes, and no value crosses threads but for the row's largest |x|.  Both
// kernels here are bound by HBM; the rows of two passes are on their way before the
// sines are formed.
#include "serve.cuh"

namespace qsa {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRowThreads = 8;                              // threads per row
constexpr int kRowsPerPass = kRopeThreads / kRowThreads;    // 16

// frac(x / 2 pi) * 2^64 of a finite double (0 for what is not finite): x = m 2^(e - 52)
// with m < 2^53, and m / 2 pi * 2^66 is one 64 x 64-bit product.
__device__ __forceinline__ unsigned long long turn_fraction(double x) {
    const unsigned long long bits = (unsigned long long)__double_as_longlong(x);
    const int field = (int)((bits >> 52) & 0x7FF);
    const unsigned long long m = (bits & 0xFFFFFFFFFFFFFull) | (field ? 1ull << 52 : 0ull);
    const unsigned __int128 p = (unsigned __int128)m * 0xA2F9836E4E44152Aull;   // round(2^66 / 2 pi)
    const int down = 54 - (field ? field - 1023 : -1022);                       // f = p 2^(e - 54)
    unsigned long long f;
    if (down >= 0) f = down < 128 ? (unsigned long long)(p >> down) : 0ull;
    else f = down > -64 ? (unsigned long long)p << -down : 0ull;
    return field == 0x7FF ? 0ull : (bits >> 63) ? 0ull - f : f;
}

__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ __align__(16) float s_cos[kHeadDim / 2], s_sin[kHeadDim / 2];
    const int t = blockIdx.x, tid = threadIdx.x;
    const int l = tid & (kRowThreads - 1);
    // the thread's two 16-byte pieces of any row, and whether they are turned
    const bool turned = a.interleaved || 8 * l < a.n_pairs;
    const int p0 = turned ? l : 2 * l;
    const int p1 = a.interleaved ? l + 8 : turned ? l + a.n_pairs / 8 : 2 * l + 1;
    wait_for_stream();

    // the token's cell, for its key and value rows
    long long cell_row = -1;
    if (a.k_pool) {
        const int slot = __ldg(a.slots + t);
        if (slot >= 0) {
            const int page = slot >> 6;
            if (page < a.n_ppages) cell_row = (long long)page * a.n_kv * kPage + (slot & (kPage - 1));
            else if (tid == 0) report(a.dev_status, QSA_DEV_BAD_CELL);
        }
    }
    const int n_rows = a.n_heads + (cell_row >= 0 ? 2 * a.n_kv : 0);
    const int r0 = tid >> 3;                         // rows r0, r0 + 16, ...: query, key, value rows
    auto load = [&](int r, uint4 (&w)[2]) {
        w[0] = w[1] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= n_rows) return;
        const int kv = r - a.n_heads;
        const uint16_t* src = kv < 0 ? a.q + t * a.q_stride + (size_t)r * kHeadDim
                              : kv < a.n_kv ? a.k + t * a.k_stride + (size_t)kv * kHeadDim
                                            : a.v + t * a.v_stride + (size_t)(kv - a.n_kv) * kHeadDim;
        w[0] = reinterpret_cast<const uint4*>(src)[p0];   // plain loads: q_out may be q itself
        w[1] = reinterpret_cast<const uint4*>(src)[p1];
    };
    uint4 next[2][2];
    load(r0, next[0]);
    load(r0 + kRowsPerPass, next[1]);

    if (tid < a.n_pairs) {
        int axis = a.pair_axis ? __ldg(a.pair_axis + tid) : 0;
        if (axis < 0 || axis >= a.n_axes) {
            report(a.dev_status, QSA_DEV_BAD_AXIS);
            axis = 0;
        }
        const long long pos = __ldg(a.positions + (size_t)axis * a.pos_stride + t);
        const unsigned long long f = turn_fraction(__ldg(a.inv_freq + tid));
        const int turn = (int)(((unsigned long long)pos * f) >> 32);     // [-1/2, 1/2) turns, 2^-32 each
        float sn, cs;
        sincospif((float)turn * 0x1p-31f, &sn, &cs);
        s_sin[tid] = sn;
        s_cos[tid] = cs;
    }
    __syncthreads();
    float cs[8], sn[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int pair = a.interleaved ? 4 * l + (j & 3) + 32 * (j >> 2) : 8 * l + j;
        cs[j] = pair < a.n_pairs ? s_cos[pair] : 1.f;
        sn[j] = pair < a.n_pairs ? s_sin[pair] : 0.f;
    }

    // one row; the row maximum shuffles, so a warp's four rows go together
    auto work = [&](int r, const uint4 (&w)[2]) {
        const int kv = r - a.n_heads;                // >= 0: key rows, then value rows
        const bool live = r < n_rows, is_v = kv >= a.n_kv;
        const int h = is_v ? kv - a.n_kv : kv;
        float x[2][8];
        unpack8(w[0], a.type, x[0]);
        unpack8(w[1], a.type, x[1]);
        if (kv < 0 || !is_v) {
            if (a.interleaved) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {        // pair j: elements 2j, 2j + 1 of the 16; a piece is turned whole
                    if (4 * l + 32 * (j >> 2) >= a.n_pairs) continue;
                    float& u = x[j >> 2][2 * (j & 3)];
                    float& z = x[j >> 2][2 * (j & 3) + 1];
                    const float p = u * cs[j] - z * sn[j];
                    z = z * cs[j] + u * sn[j];
                    u = p;
                }
            } else if (turned) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float u = x[0][j], z = x[1][j];
                    x[0][j] = u * cs[j] - z * sn[j];
                    x[1][j] = z * cs[j] + u * sn[j];
                }
            }
        }
        if (live && kv < 0) {
            uint4* dst = reinterpret_cast<uint4*>(a.q_out + t * a.q_out_stride + (size_t)r * kHeadDim);
            dst[p0] = make_uint4(pack2(x[0][0], x[0][1], a.type), pack2(x[0][2], x[0][3], a.type),
                                 pack2(x[0][4], x[0][5], a.type), pack2(x[0][6], x[0][7], a.type));
            dst[p1] = make_uint4(pack2(x[1][0], x[1][1], a.type), pack2(x[1][2], x[1][3], a.type),
                                 pack2(x[1][4], x[1][5], a.type), pack2(x[1][6], x[1][7], a.type));
        }
        if ((r & ~3) + 3 < a.n_heads) return;        // warp-uniform: four query rows
        // ---- key and value rows: scale = max |x| / 127 rounded up to FP16, so |x / scale| <= 127
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {                // NaN counts as infinite (fmaxf would drop it)
            const float u = fabsf(x[0][j]), z = fabsf(x[1][j]);
            amax = fmaxf(amax, fmaxf(u <= 3.402823466e38f ? u : INFINITY, z <= 3.402823466e38f ? z : INFINITY));
        }
#pragma unroll
        for (int o = 1; o < kRowThreads; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (live && kv >= 0) {
            const bool finite = amax < INFINITY;
            uint16_t sb = __half_as_ushort(__float2half_ru(__fdiv_rn(amax, 127.f)));
            if (sb > 0x7BFFu) sb = finite ? 0x7BFFu : 0x7FFFu;   // past FP16: the largest finite scale; not finite: NaN
            const float scale = __half2float(__ushort_as_half(sb));
            const float div = finite && sb != 0 ? scale : 1.f;
            const long long row = cell_row + (long long)h * kPage;
            int8_t* dst = (is_v ? a.v_pool : a.k_pool) + row * kHeadDim;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t b[2] = {0u, 0u};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    int i = __float2int_rn(__fdiv_rn(x[e][j], div));
                    i = finite ? min(127, max(-127, i)) : 0;
                    b[j >> 2] |= (uint32_t)(i & 0xFF) << (8 * (j & 3));
                }
                *reinterpret_cast<uint2*>(dst + 8 * (e ? p1 : p0)) = make_uint2(b[0], b[1]);
            }
            if (l == 0) (is_v ? a.v_scale : a.k_scale)[row] = sb;
        }
    };
    // warp-uniform trips (a warp's rows r .. r + 3): two passes at a time, the next two on their way
    for (int r = r0; (r & ~3) < n_rows; r += 2 * kRowsPerPass) {
        uint4 w[2][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            w[e][0] = next[e][0];
            w[e][1] = next[e][1];
            load(r + (2 + e) * kRowsPerPass, next[e]);
        }
        work(r, w[0]);
        if ((r & ~3) + kRowsPerPass < n_rows) work(r + kRowsPerPass, w[1]);
    }
}

// Read back: a row's threads take as many elements each as fill a 16-byte store (8, or 4
// of FP32), so that a warp's stores are consecutive; kGatherItems (cell, KV head) items
// per thread, whose loads are all on their way before the first is used.
constexpr int kGatherThreads = 256;
constexpr int kGatherItems = 2;

template <int TYPE>
__device__ __forceinline__ void put_row(void* out, size_t at, const uint2& w, float scale) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = (float)(int8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3))) * scale;
    if (TYPE == QSA_F32)
        *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(f[0], f[1], f[2], f[3]);
    else
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
            make_uint4(pack2(f[0], f[1], TYPE), pack2(f[2], f[3], TYPE), pack2(f[4], f[5], TYPE), pack2(f[6], f[7], TYPE));
}

template <int TYPE>
__global__ void __launch_bounds__(kGatherThreads) cache_gather_kernel(const __grid_constant__ GatherArgs a) {
    constexpr int kElems = TYPE == QSA_F32 ? 4 : 8, kLanes = kHeadDim / kElems, kRows = kGatherThreads / kLanes;
    const int l = threadIdx.x % kLanes;
    const long long items = (long long)a.n_cell * a.n_kv;
    const long long item0 = (long long)blockIdx.x * (kRows * kGatherItems) + threadIdx.x / kLanes;
    wait_for_stream();
    uint2 k[kGatherItems], v[kGatherItems];
    float ks[kGatherItems], vs[kGatherItems];
#pragma unroll
    for (int j = 0; j < kGatherItems; ++j) {
        const long long item = item0 + j * kRows;
        k[j] = v[j] = make_uint2(0u, 0u);
        ks[j] = vs[j] = 0.f;
        if (item >= items) continue;
        const int i = (int)(item / a.n_kv), h = (int)(item - (long long)i * a.n_kv);
        const int slot = __ldg(a.slots + i), page = slot >> 6;
        if (slot >= 0 && page < a.n_ppages) {
            const long long row = ((long long)page * a.n_kv + h) * kPage + (slot & (kPage - 1));
            if (TYPE == QSA_F32) {
                k[j].x = __ldg(reinterpret_cast<const uint32_t*>(a.k_pool + row * kHeadDim) + l);
                v[j].x = __ldg(reinterpret_cast<const uint32_t*>(a.v_pool + row * kHeadDim) + l);
            } else {
                k[j] = __ldg(reinterpret_cast<const uint2*>(a.k_pool + row * kHeadDim) + l);
                v[j] = __ldg(reinterpret_cast<const uint2*>(a.v_pool + row * kHeadDim) + l);
            }
            ks[j] = __half2float(__ushort_as_half(__ldg(a.k_scale + row)));
            vs[j] = __half2float(__ushort_as_half(__ldg(a.v_scale + row)));
        } else if (slot >= 0 && l == 0) {
            report(a.dev_status, QSA_DEV_BAD_CELL);
        }
    }
#pragma unroll
    for (int j = 0; j < kGatherItems; ++j) {
        const long long item = item0 + j * kRows;
        if (item >= items) continue;
        const size_t at = (size_t)item * kHeadDim + kElems * l;
        put_row<TYPE>(a.k_out, at, k[j], ks[j]);
        put_row<TYPE>(a.v_out, at, v[j], vs[j]);
    }
}

template <int TYPE>
cudaError_t launch_gather(const GatherArgs& a, cudaStream_t stream) {
    constexpr int kElems = TYPE == QSA_F32 ? 4 : 8;
    constexpr long long kBlock = (long long)kGatherThreads / (kHeadDim / kElems) * kGatherItems;
    const long long grid = ((long long)a.n_cell * a.n_kv + kBlock - 1) / kBlock;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_overlapped(cache_gather_kernel<TYPE>, dim3((unsigned)grid), kGatherThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t stream) {
    return launch_overlapped(rope_append_kernel, dim3((unsigned)a.n_tok), kRopeThreads, 0, stream, a);
}

cudaError_t launch_cache_gather(const GatherArgs& a, cudaStream_t stream) {
    if (a.out_type == QSA_F32) return launch_gather<QSA_F32>(a, stream);
    if (a.out_type == QSA_F16) return launch_gather<QSA_F16>(a, stream);
    return launch_gather<QSA_BF16>(a, stream);
}

}  // namespace qsa

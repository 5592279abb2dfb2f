// cache_rows.cu -- rows on their way into and out of the paged INT8 cache: rotary
// positions with the quantising write (qsa_rope, qsa_rope_append) and the
// dequantising read (qsa_cache_gather).
//
// Rotation: pair j of a token's query or key row is turned by positions[axis_j] *
// inv_freq[j].  The angle is kept as a fraction of a turn in 64-bit fixed point:
// f = frac(inv_freq / 2 pi) * 2^64, and position * f modulo 2^64 IS the fraction
// of the turn that is left, whatever the position's size or sign; no range
// reduction loses bits.  Its top 32 bits go to sincospif.
//
// Layout: one CTA per token, eight threads per 128-element row, so the token's 64
// sines and cosines are formed once, into shared memory, and a thread keeps the
// eight pairs it always works on in registers for all its rows.  Thread l of a
// row's eight holds pairs 8l .. 8l+7: the 16-byte pieces l and l + n_pairs/8 of
// the row (pieces 2l and 2l+1 when pairs are interleaved, and for the pieces that
// pass through), so every load and store is 16 bytes wide and no value crosses
// threads but for the row's largest |x|.
#include "serve.cuh"

namespace qsa {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRowThreads = 8;                              // threads per row
constexpr int kRowsPerPass = kRopeThreads / kRowThreads;    // 16

__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeArgs a) {
    __shared__ __align__(16) float s_cos[kHeadDim / 2], s_sin[kHeadDim / 2];
    const int t = blockIdx.x, tid = threadIdx.x;
    const int l = tid & (kRowThreads - 1);
    const bool turned = 8 * l < a.n_pairs;
    // the thread's two 16-byte pieces of any row
    const int p0 = turned && !a.interleaved ? l : 2 * l;
    const int p1 = turned && !a.interleaved ? l + a.n_pairs / 8 : 2 * l + 1;

    if (tid < a.n_pairs) {
        int axis = a.pair_axis ? __ldg(a.pair_axis + tid) : 0;
        if (axis < 0 || axis >= a.n_axes) {
            report(a.dev_status, QSA_DEV_BAD_AXIS);
            axis = 0;
        }
        const long long pos = __ldg(a.positions + (size_t)axis * a.pos_stride + t);
        double x = __ldg(a.inv_freq + tid) * 0.15915494309189533577;   // turns per position
        x -= floor(x);
        const unsigned long long f = __double2ull_rd(x * 18446744073709551616.0);
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
        cs[j] = turned ? s_cos[8 * l + j] : 1.f;
        sn[j] = turned ? s_sin[8 * l + j] : 0.f;
    }

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
    // warp-uniform trips: a warp's four rows r .. r+3 leave together (the row maximum shuffles)
    for (int r0 = (tid >> 5) * 4; r0 < n_rows; r0 += kRowsPerPass) {
        const int r = r0 + ((tid & 31) >> 3);
        const int kv = r - a.n_heads;                // >= 0: key rows, then value rows
        const bool is_v = kv >= a.n_kv;
        const int h = is_v ? kv - a.n_kv : kv;
        float x[2][8];
        if (r < n_rows) {
            const uint16_t* src = kv < 0 ? a.q + t * a.q_stride + (size_t)r * kHeadDim
                                         : (is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) + (size_t)h * kHeadDim;
            // plain loads: q_out may be q itself
            unpack8(reinterpret_cast<const uint4*>(src)[p0], a.type, x[0]);
            unpack8(reinterpret_cast<const uint4*>(src)[p1], a.type, x[1]);
            if (turned && !(kv >= 0 && is_v)) {
                if (a.interleaved) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {   // pair j: elements 2j, 2j + 1 of the 16
                        float& u = x[j >> 2][2 * (j & 3)];
                        float& w = x[j >> 2][2 * (j & 3) + 1];
                        const float p = u * cs[j] - w * sn[j];
                        w = w * cs[j] + u * sn[j];
                        u = p;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float u = x[0][j], w = x[1][j];
                        x[0][j] = u * cs[j] - w * sn[j];
                        x[1][j] = w * cs[j] + u * sn[j];
                    }
                }
            }
            if (kv < 0) {
                uint4* dst = reinterpret_cast<uint4*>(a.q_out + t * a.q_out_stride + (size_t)r * kHeadDim);
                dst[p0] = make_uint4(pack2(x[0][0], x[0][1], a.type), pack2(x[0][2], x[0][3], a.type),
                                     pack2(x[0][4], x[0][5], a.type), pack2(x[0][6], x[0][7], a.type));
                dst[p1] = make_uint4(pack2(x[1][0], x[1][1], a.type), pack2(x[1][2], x[1][3], a.type),
                                     pack2(x[1][4], x[1][5], a.type), pack2(x[1][6], x[1][7], a.type));
            }
        }
        if (r0 + 3 < a.n_heads) continue;            // warp-uniform: four query rows
        // ---- key and value rows: scale = max |x| / 127 rounded up to FP16, so |x / scale| <= 127
        float amax = 0.f;
        if (r < n_rows && kv >= 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {            // NaN counts as infinite (fmaxf would drop it)
                const float u = fabsf(x[0][j]), w = fabsf(x[1][j]);
                amax = fmaxf(amax, fmaxf(u <= 3.402823466e38f ? u : INFINITY, w <= 3.402823466e38f ? w : INFINITY));
            }
        }
#pragma unroll
        for (int o = 1; o < kRowThreads; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (r < n_rows && kv >= 0) {
            const bool finite = amax < INFINITY;
            uint16_t sb = __half_as_ushort(__float2half_ru(__fdiv_rn(amax, 127.f)));
            if (sb > 0x7BFFu) sb = finite ? 0x7BFFu : 0x7FFFu;   // past FP16: the largest finite scale; not finite: NaN
            const float scale = __half2float(__ushort_as_half(sb));
            const float div = finite && sb != 0 ? scale : 1.f;
            const long long row = cell_row + (long long)h * kPage;
            int8_t* dst = (is_v ? a.v_pool : a.k_pool) + row * kHeadDim;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t w[2] = {0u, 0u};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    int i = __float2int_rn(__fdiv_rn(x[e][j], div));
                    i = finite ? min(127, max(-127, i)) : 0;
                    w[j >> 2] |= (uint32_t)(i & 0xFF) << (8 * (j & 3));
                }
                *reinterpret_cast<uint2*>(dst + 8 * (e ? p1 : p0)) = make_uint2(w[0], w[1]);
            }
            if (l == 0) (is_v ? a.v_scale : a.k_scale)[row] = sb;
        }
    }
}

// Read back: eight threads per (cell, KV head), 16 bytes of the key row and of the
// value row each.
constexpr int kGatherThreads = 256;

template <int TYPE>
__device__ __forceinline__ void put16(void* out, size_t at, const uint4& w, float scale) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    float f[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) f[j] = (float)(int8_t)(v[j >> 2] >> (8 * (j & 3))) * scale;
    if (TYPE == QSA_F32) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
    } else {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            dst[j] = make_uint4(pack2(f[8 * j], f[8 * j + 1], TYPE), pack2(f[8 * j + 2], f[8 * j + 3], TYPE),
                                pack2(f[8 * j + 4], f[8 * j + 5], TYPE), pack2(f[8 * j + 6], f[8 * j + 7], TYPE));
    }
}

template <int TYPE>
__global__ void __launch_bounds__(kGatherThreads) cache_gather_kernel(const GatherArgs a) {
    const long long item = ((long long)blockIdx.x * kGatherThreads + threadIdx.x) >> 3;   // (cell, KV head)
    if (item >= (long long)a.n_cell * a.n_kv) return;
    const int l = threadIdx.x & 7;
    const int i = (int)(item / a.n_kv), h = (int)(item - (long long)i * a.n_kv);
    const int slot = __ldg(a.slots + i), page = slot >> 6;
    uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
    float ks = 0.f, vs = 0.f;
    if (slot >= 0 && page < a.n_ppages) {
        const long long row = ((long long)page * a.n_kv + h) * kPage + (slot & (kPage - 1));
        k = __ldg(reinterpret_cast<const uint4*>(a.k_pool + row * kHeadDim) + l);
        v = __ldg(reinterpret_cast<const uint4*>(a.v_pool + row * kHeadDim) + l);
        ks = __half2float(__ushort_as_half(__ldg(a.k_scale + row)));
        vs = __half2float(__ushort_as_half(__ldg(a.v_scale + row)));
    } else if (slot >= 0 && l == 0) {
        report(a.dev_status, QSA_DEV_BAD_CELL);
    }
    const size_t at = (size_t)item * kHeadDim + 16 * l;
    put16<TYPE>(a.k_out, at, k, ks);
    put16<TYPE>(a.v_out, at, v, vs);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t stream) {
    rope_append_kernel<<<(unsigned)a.n_tok, kRopeThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_cache_gather(const GatherArgs& a, cudaStream_t stream) {
    const long long threads = (long long)a.n_cell * a.n_kv * kRowThreads;
    const long long grid = (threads + kGatherThreads - 1) / kGatherThreads;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const unsigned g = (unsigned)grid;
    if (a.out_type == QSA_F32) cache_gather_kernel<QSA_F32><<<g, kGatherThreads, 0, stream>>>(a);
    else if (a.out_type == QSA_F16) cache_gather_kernel<QSA_F16><<<g, kGatherThreads, 0, stream>>>(a);
    else cache_gather_kernel<QSA_BF16><<<g, kGatherThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace qsa

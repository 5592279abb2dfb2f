// paged_attn.cu -- attention of one new token per sequence over its whole paged
// INT8 cache (qsa_paged_attn).
//
// out[s][i] = sum_c softmax_c(q . k_c * sm_scale) v_c over the resident cells c of
// the sequence (the last `window` of them), k_c = int8 * FP16 scale.
//
// The simplest form: one CTA of 128 threads per (sequence, query head), walking
// the cells in steps of 128.  In a step each thread scores one cell (a dot product
// of 128 in FP32), the block updates the running maximum, and each thread then
// adds the step's weighted values of its own dim.
#include "serve.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float block_max(float v, float* scratch) {
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    return fmaxf(fmaxf(scratch[0], scratch[1]), fmaxf(scratch[2], scratch[3]));
}

__global__ void __launch_bounds__(kThreads) paged_attn_kernel(const PagedArgs a) {
    __shared__ float s_q[kHeadDim], s_p[kThreads], s_red[4];
    __shared__ long long s_row[kThreads];
    const int tid = threadIdx.x;
    const int head = blockIdx.x % a.n_heads, s = blockIdx.x / a.n_heads;
    const int h = head / (a.n_heads / a.n_kv);
    const size_t row0 = (size_t)s * a.n_heads + head;
    const uint16_t qb = static_cast<const uint16_t*>(a.q)[row0 * kHeadDim + tid];
    s_q[tid] = a.q_type == QSA_F16 ? __half2float(__ushort_as_half(qb)) : bf16_lo(qb);
    int n = a.seq_lens[s];
    if (n < 0 || n > a.n_lpages * kPage) {
        if (tid == 0) report(a.dev_status, QSA_DEV_BAD_SEQ_LEN);
        n = n < 0 ? 0 : a.n_lpages * kPage;
    }
    const int first = a.window > 0 && a.window < n ? n - a.window : 0;
    const int32_t* table = a.page_tables + (size_t)s * a.pt_stride;
    float m = -INFINITY, l = 0.f, o = 0.f;
    __syncthreads();
    for (long long c0 = first; c0 < n; c0 += kThreads) {
        const long long c = c0 + tid;
        long long row = -1;
        if (c < n) {
            const int page = table[c >> 6];
            if (page >= a.n_ppages) report(a.dev_status, QSA_DEV_BAD_PAGE);
            else if (page >= 0) row = ((long long)page * a.n_kv + h) * kPage + (c & (kPage - 1));
        }
        float sc = -INFINITY;
        if (row >= 0) {
            const int8_t* k = a.k_pool + row * kHeadDim;
            float dot = 0.f;
            for (int d = 0; d < kHeadDim; ++d) dot += s_q[d] * (float)k[d];
            sc = dot * __half2float(__ushort_as_half(a.k_scale[row])) * a.sm_scale;
        }
        const float mn = fmaxf(m, block_max(sc, s_red));
        if (mn == -INFINITY) continue;   // uniform: nothing resident so far
        const float al = expf(m - mn);   // 0 while m is -inf
        m = mn;
        s_p[tid] = row >= 0 ? expf(sc - m) : 0.f;
        s_row[tid] = row;
        __syncthreads();
        float lb = 0.f, ob = 0.f;        // the step's own sums: chains stay short
        for (int j = 0; j < kThreads; ++j) {
            if (s_row[j] < 0) continue;
            lb += s_p[j];
            ob += s_p[j] * __half2float(__ushort_as_half(a.v_scale[s_row[j]])) * (float)a.v_pool[s_row[j] * kHeadDim + tid];
        }
        l = l * al + lb;
        o = o * al + ob;
        __syncthreads();
    }
    const float r = m == -INFINITY ? 0.f : o / l;
    const size_t at = row0 * kHeadDim + tid;
    if (a.out_type == QSA_F32) static_cast<float*>(a.out)[at] = r;
    else if (a.out_type == QSA_F16) static_cast<__half*>(a.out)[at] = __float2half_rn(r);
    else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(r);
    if (a.lse && tid == 0) a.lse[row0] = m == -INFINITY ? -INFINITY : m + logf(l);
}

}  // namespace

size_t paged_attn_workspace(int, int) { return 256; }

cudaError_t launch_paged_attn(const PagedArgs& a, cudaStream_t stream) {
    paged_attn_kernel<<<(unsigned)(a.n_seq * a.n_heads), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace qsa

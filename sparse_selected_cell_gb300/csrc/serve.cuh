// serve.cuh -- arguments and launchers of the serving operators around the paged
// INT8 cache: whole-cache decode attention (paged_attn.cu), rotary positions and
// the cache's INT8 write and read (cache_rows.cu), table extension
// (extend_tables.cu).  Called by capi_serve.cu after argument validation.
#pragma once
#include "qsa_common.cuh"

namespace qsa {

// ---------------------------------------------------------------- element types
// Eight consecutive 16-bit elements (one 16-byte word) to FP32 and back; `type`
// is QSA_BF16 or QSA_F16 and uniform over the launch.
__device__ __forceinline__ void unpack8(const uint4& w, int type, float (&x)[8]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (type == QSA_F16) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[j]));
            x[2 * j] = f.x;
            x[2 * j + 1] = f.y;
        } else {
            x[2 * j] = bf16_lo(v[j]);
            x[2 * j + 1] = bf16_hi(v[j]);
        }
    }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, int type) {
    return type == QSA_F16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}

// ---------------------------------------------------------------- launch overlap
// These kernels are launched so that their blocks may be set up while the kernel before
// them in the stream still drains; each waits here, before its first read, until that
// kernel has finished and its writes are visible.  Whatever was launched before, and
// whatever follows, sees plain stream order.  What they read may be written while they are
// already resident, so they read it by ordinary loads, which stay behind this wait, and
// never by non-coherent ones, which are for data that nothing writes in a kernel's lifetime
// and may be moved.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const A&... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// ---------------------------------------------------------------- launchers
struct PagedArgs {
    const void* q;
    int q_type;
    const int8_t* k_pool;
    const int8_t* v_pool;
    const uint16_t* k_scale;
    const uint16_t* v_scale;
    const int32_t* page_tables;   // sequence s: page_tables + s * pt_stride
    int pt_stride, n_lpages, n_ppages, n_kv, n_heads;
    const int32_t* seq_lens;
    int n_seq, window;
    float sm_scale;
    void* out;
    int out_type;
    float* lse;                   // or null
    uint8_t* workspace;
    int32_t* dev_status;
};

// Bytes of workspace the launch needs (host arithmetic only).
size_t paged_attn_workspace(int n_kv, int n_heads);
cudaError_t launch_paged_attn(const PagedArgs& a, cudaStream_t stream);

struct RopeArgs {
    const uint16_t* q;            // or null
    const uint16_t* k;            // or null
    const uint16_t* v;            // or null
    long long q_stride, k_stride, v_stride;   // elements from one token to the next
    int type;
    const int32_t* positions;     // [n_axes][pos_stride]
    int n_axes, pos_stride;
    const double* inv_freq;       // [n_pairs]
    const int32_t* pair_axis;     // [n_pairs], or null (axis 0)
    int n_pairs, interleaved;
    uint16_t* q_out;
    long long q_out_stride;
    int8_t* k_pool;
    int8_t* v_pool;
    uint16_t* k_scale;
    uint16_t* v_scale;
    const int32_t* slots;         // null: no keys and values, nothing is written to a cache
    int n_ppages, n_heads, n_kv, n_tok;
    int32_t* dev_status;
};

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t stream);

struct GatherArgs {
    const int8_t* k_pool;
    const int8_t* v_pool;
    const uint16_t* k_scale;
    const uint16_t* v_scale;
    const int32_t* slots;
    int n_cell, n_ppages, n_kv;
    void* k_out;
    void* v_out;
    int out_type;
    int32_t* dev_status;
};

cudaError_t launch_cache_gather(const GatherArgs& a, cudaStream_t stream);

struct TablesArgs {
    const int32_t* seq_lens;
    const int32_t* new_lens;
    int n_seq;
    int32_t* page_tables;
    int pt_stride, n_lpages, n_ppages;
    const int32_t* free_pages;
    int n_free;
    const int32_t* free_head;     // or null (0)
    int n_tok;
    int32_t* slots;
    int32_t* positions;
    int32_t* token_seq;
    int32_t* seq_lens_out;
    int32_t* cu_tokens;
    int32_t* free_head_out;
    int32_t* dev_status;
};

cudaError_t launch_extend_tables(const TablesArgs& a, cudaStream_t stream);

}  // namespace qsa

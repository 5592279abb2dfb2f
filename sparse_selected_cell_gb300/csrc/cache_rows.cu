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
// Layout: a block takes every gridDim-th token, a warp four rows of it at a time, eight
// threads per 128-element row.  Thread l of a row's eight holds the 16-byte pieces l and
// l + n_pairs / 8 of the row, which are the two halves of pairs 8l .. 8l + 7 (of
// interleaved pairs pieces l and l + 8, pairs 4l .. and 4l + 32 ..): every load and store
// is 16 bytes wide and eight threads' are 128 consecutive bytes, no value crosses threads
// but for the row's largest |x|, and a thread reads the sines of its eight pairs once per
// token.  The next rows, of this token and the next, are on their way by asynchronous
// copies, and the next token's sines are formed beside this one's rows.  Bound by HBM; a
// token's rows are read and written by one block at about the same time because that is
// what DRAM pages like (a token to a warp, every warp in a page of its own, copied at 5.2
// of the 6.5 TB/s of a plain copy).
//
// Measured (4 KV heads x 12, BF16, calls in a row): 8,192 tokens on three axes, written and
// read back, 243 MB in 43.4 us, 5.6 TB/s; written alone, 227 MB in 37.7 (interleaved pairs
// 38.1, FP16 37.9); 40,960 cells of 8 KV heads read back alone, 253 MB in 42.3 us, 6.0 TB/s
// (FP32 421 MB in 71.9).  Small steps are latency: inside a captured graph one token's write
// and read take 3.8 us, 256 tokens' 5.7.
#include "serve.cuh"

namespace qsa {
namespace {

constexpr int kRopeWarps = 4;                                // of a block; kRopeWide where tokens are few
constexpr int kRopeWide = 8;
constexpr int kRopeDepth = 3;                                // turns (four rows) of a warp on their way
constexpr int kRopeBlocks = 5;                               // of kRopeWarps warps, per SM

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

// round(x / scale), ties to even, within [-127, 127], of 16 values, as bytes; amax: the
// row's largest |x|.  x times the reciprocal is within 2^-16 of a quotient up to 127, so it
// rounds alike unless it lies next to a half; rows with such a value, and those beyond
// 127 (a scale that FP16 does not hold), are divided out.
__device__ __forceinline__ void quantise16(const float (&x)[2][8], float scale, float amax, uint32_t (&b)[2][2]) {
    constexpr float kMagic = 12582912.f;             // 1.5 * 2^23: adding it rounds to an integer, in the low bits
    const float inv = __fdiv_rn(1.f, scale);
    uint32_t t[2][8];
    float off = amax * inv < 127.4f ? 0.f : 1.f;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float y = x[e][j] * inv, m = __fadd_rn(y, kMagic);
            off = fmaxf(off, fabsf(y - __fadd_rn(m, -kMagic)));
            t[e][j] = __float_as_uint(m);
        }
    if (!(off < 0.4999f)) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                t[e][j] = (uint32_t)min(127, max(-127, __float2int_rn(__fdiv_rn(x[e][j], scale))));
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            b[e][j] = __byte_perm(__byte_perm(t[e][4 * j], t[e][4 * j + 1], 0x0040),
                                  __byte_perm(t[e][4 * j + 2], t[e][4 * j + 3], 0x0040), 0x5410);
}

template <int TYPE, bool INTERLEAVED, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, kRopeBlocks * kRopeWarps / WARPS)
rope_append_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ uint4 s_ring[WARPS][kRopeDepth][2][32];       // each thread's own pieces of the rows to come
    __shared__ __align__(16) float s_cos[2][kHeadDim / 2], s_sin[2][kHeadDim / 2];   // this token's and the next's
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned n_tok = (unsigned)a.n_tok, stride = gridDim.x;
    const int l = lane & 7;
    // the thread's two 16-byte pieces of any row, and whether they are turned
    const bool turned = INTERLEAVED || 8 * l < a.n_pairs;
    const int p0 = turned ? l : l + a.n_pairs / 8;
    const int p1 = INTERLEAVED || !turned ? l + 8 : l + a.n_pairs / 8;
    const int n_rows = a.n_heads + (a.slots ? 2 * a.n_kv : 0);   // query, key, value rows
    constexpr int kTurn = 4 * WARPS;                 // a warp's turns: rows 4 warp .. 4 warp + 3, then kTurn further
    wait_for_stream();

    // asynchronous copies of the next turn's pieces, a group a turn, running ahead of the work over all tokens
    unsigned l_tok = blockIdx.x;
    int l_row = 4 * warp, l_slot = 0;
    auto load = [&]() {
        if (l_tok < n_tok && l_row < n_rows) {
            const long long t = l_tok;
            const int r = l_row + (lane >> 3), kv = r - a.n_heads;
            if (r < n_rows) {
                const uint16_t* src = kv < 0 ? a.q + t * a.q_stride + (size_t)r * kHeadDim
                                      : kv < a.n_kv ? a.k + t * a.k_stride + (size_t)kv * kHeadDim
                                                    : a.v + t * a.v_stride + (size_t)(kv - a.n_kv) * kHeadDim;
                const uint32_t dst = smem_u32(&s_ring[warp][l_slot][0][lane]);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src + 8 * p0) : "memory");
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 512), "l"(src + 8 * p1) : "memory");
            }
            l_slot = (l_slot + 1) % kRopeDepth;
            l_row += kTurn;
            if (l_row >= n_rows) {
                l_tok += stride;
                l_row = 4 * warp;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int k = 0; k < kRopeDepth; ++k) load();

    // this thread's pair: its position and its turns per position
    const int pair = threadIdx.x;
    const bool has = pair < a.n_pairs;
    const int32_t* pos_at = a.positions;
    unsigned long long f = 0;
    int pos = 0, cell = a.slots ? a.slots[blockIdx.x] : -1;
    if (has) {
        int axis = a.pair_axis ? a.pair_axis[pair] : 0;
        f = turn_fraction(a.inv_freq[pair]);
        if (axis < 0 || axis >= a.n_axes) {
            report(a.dev_status, QSA_DEV_BAD_AXIS);
            axis = 0;
        }
        pos_at += (size_t)axis * a.pos_stride;
        pos = pos_at[blockIdx.x];
    }
    auto form = [&](int buf, unsigned next) {        // the sines of the token that pos is of; then the next one's position
        if (!has) return;
        const int turn = (int)(((unsigned long long)(long long)pos * f) >> 32);   // [-1/2, 1/2) turns, 2^-32 each
        sincospif((float)turn * 0x1p-31f, &s_sin[buf][pair], &s_cos[buf][pair]);
        if (next < n_tok) pos = pos_at[next];
    };
    form(0, blockIdx.x + stride);

    int slot = 0, buf = 0;
#pragma unroll 1
    for (unsigned tok = blockIdx.x; tok < n_tok; tok += stride, buf ^= 1) {
        const long long t = tok;
        __syncthreads();                             // this token's sines are there, the one before's have been read
        if (tok + stride < n_tok) form(buf ^ 1, tok + 2 * stride);
        long long cell_row = -1;
        if (cell >= 0) {
            const int page = cell >> 6;
            if (page < a.n_ppages) cell_row = (long long)page * a.n_kv * kPage + (cell & (kPage - 1));
            else if (threadIdx.x == 0) report(a.dev_status, QSA_DEV_BAD_CELL);
        }
        if (a.slots && tok + stride < n_tok) cell = a.slots[tok + stride];
        float cs[8], sn[8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int first = INTERLEAVED ? 4 * l + 32 * e : 8 * l + 4 * e;   // pair of elements 4 e .. 4 e + 3 here
            const float4 c = *reinterpret_cast<const float4*>(&s_cos[buf][first]);
            const float4 z = *reinterpret_cast<const float4*>(&s_sin[buf][first]);
            cs[4 * e] = c.x, cs[4 * e + 1] = c.y, cs[4 * e + 2] = c.z, cs[4 * e + 3] = c.w;
            sn[4 * e] = z.x, sn[4 * e + 1] = z.y, sn[4 * e + 2] = z.z, sn[4 * e + 3] = z.w;
        }
        // ---- its rows, four to a warp at a time
#pragma unroll 1
        for (int r4 = 4 * warp; r4 < n_rows; r4 += kTurn) {
            float x[2][8];
            asm volatile("cp.async.wait_group %0;" ::"n"(kRopeDepth - 1) : "memory");
            unpack8(s_ring[warp][slot][0][lane], TYPE, x[0]);   // the thread's own copies: no other has to wait
            unpack8(s_ring[warp][slot][1][lane], TYPE, x[1]);
            load();
            slot = (slot + 1) % kRopeDepth;
            const int r = r4 + (lane >> 3), kv = r - a.n_heads;   // kv >= 0: key rows, then value rows
            const bool is_v = kv >= a.n_kv;
            if (kv < 0 || !is_v) {
                if (INTERLEAVED) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {    // pair j: elements 2j, 2j + 1 of the 16; a piece is turned whole
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
            if (kv < 0) {
                uint4* dst = reinterpret_cast<uint4*>(a.q_out + t * a.q_out_stride + (size_t)r * kHeadDim);
                dst[p0] = make_uint4(pack2(x[0][0], x[0][1], TYPE), pack2(x[0][2], x[0][3], TYPE),
                                     pack2(x[0][4], x[0][5], TYPE), pack2(x[0][6], x[0][7], TYPE));
                dst[p1] = make_uint4(pack2(x[1][0], x[1][1], TYPE), pack2(x[1][2], x[1][3], TYPE),
                                     pack2(x[1][4], x[1][5], TYPE), pack2(x[1][6], x[1][7], TYPE));
            }
            if (r4 + 3 < a.n_heads || cell_row < 0) continue;   // warp-uniform: query rows only, or no cell
            // ---- key and value rows: scale = max |x| / 127 rounded up to FP16, so |x / scale| <= 127
            float amax = 0.f;
            uint32_t odd = 0u;                       // an infinity or NaN somewhere
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                amax = fmax3(amax, fabsf(x[0][j]), fabsf(x[1][j]));
                odd |= (fabsf(x[0][j]) <= 3.402823466e38f && fabsf(x[1][j]) <= 3.402823466e38f) ? 0u : 1u;
            }
            if (odd) amax = INFINITY;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            if (kv >= 0 && r < n_rows) {
                const bool finite = amax < INFINITY;
                uint16_t sb = __half_as_ushort(__float2half_ru(__fdiv_rn(amax, 127.f)));
                if (sb > 0x7BFFu) sb = finite ? 0x7BFFu : 0x7FFFu;   // past FP16: the largest finite scale; not finite: NaN
                uint32_t b[2][2] = {{0u, 0u}, {0u, 0u}};
                if (finite && sb != 0) quantise16(x, __half2float(__ushort_as_half(sb)), amax, b);
                const long long row = cell_row + (long long)(is_v ? kv - a.n_kv : kv) * kPage;
                int8_t* dst = (is_v ? a.v_pool : a.k_pool) + row * kHeadDim;
                *reinterpret_cast<uint2*>(dst + 8 * p0) = make_uint2(b[0][0], b[0][1]);
                *reinterpret_cast<uint2*>(dst + 8 * p1) = make_uint2(b[1][0], b[1][1]);
                if (l == 0) (is_v ? a.v_scale : a.k_scale)[row] = sb;
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int TYPE, bool INTERLEAVED>
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // Few tokens: eight warps to a token while all blocks run at once, two per SM.  Measured, us, eight warps against four:
    // 4 KV heads x 12, 256 tokens 3.7 / 4.0, 304 3.8 / 4.0, 305 4.8 / 4.0, 320 5.4 / 4.2, 380 5.7 / 4.2; 8 x 12, 304 tokens
    // 4.5 / 5.0, 320 6.6 / 5.5.
    const int rows = a.n_heads + (a.slots ? 2 * a.n_kv : 0), wide = sms * (kRopeBlocks * kRopeWarps / kRopeWide);
    if (a.n_tok <= wide && rows > 4 * kRopeWarps)
        return launch_overlapped(rope_append_kernel<TYPE, INTERLEAVED, kRopeWide>, dim3((unsigned)a.n_tok), 32 * kRopeWide, 0,
                                 stream, a);
    const int grid = a.n_tok < sms * kRopeBlocks ? a.n_tok : sms * kRopeBlocks;
    return launch_overlapped(rope_append_kernel<TYPE, INTERLEAVED, kRopeWarps>, dim3((unsigned)grid), 32 * kRopeWarps, 0, stream,
                             a);
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
    const long long items = (long long)a.n_cell * a.n_kv, block0 = (long long)blockIdx.x * (kRows * kGatherItems);
    // the block's first item by one wide division, its threads' from there in 32 bits
    const unsigned cell0 = (unsigned)(block0 / a.n_kv), head0 = (unsigned)(block0 - (long long)cell0 * a.n_kv);
    const unsigned local = threadIdx.x / kLanes;
    wait_for_stream();
    uint2 k[kGatherItems], v[kGatherItems];
    float ks[kGatherItems], vs[kGatherItems];
#pragma unroll
    for (int j = 0; j < kGatherItems; ++j) {
        k[j] = v[j] = make_uint2(0u, 0u);
        ks[j] = vs[j] = 0.f;
        if (block0 + local + j * kRows >= items) continue;
        const unsigned from = head0 + local + j * kRows, more = from / (unsigned)a.n_kv, h = from - more * (unsigned)a.n_kv;
        const int slot = a.slots[cell0 + more], page = slot >> 6;
        if (slot >= 0 && page < a.n_ppages) {
            const long long row = ((long long)page * a.n_kv + h) * kPage + (slot & (kPage - 1));
            if (TYPE == QSA_F32) {
                k[j].x = reinterpret_cast<const uint32_t*>(a.k_pool + row * kHeadDim)[l];
                v[j].x = reinterpret_cast<const uint32_t*>(a.v_pool + row * kHeadDim)[l];
            } else {
                k[j] = reinterpret_cast<const uint2*>(a.k_pool + row * kHeadDim)[l];
                v[j] = reinterpret_cast<const uint2*>(a.v_pool + row * kHeadDim)[l];
            }
            ks[j] = __half2float(__ushort_as_half(a.k_scale[row]));
            vs[j] = __half2float(__ushort_as_half(a.v_scale[row]));
        } else if (slot >= 0 && l == 0) {
            report(a.dev_status, QSA_DEV_BAD_CELL);
        }
    }
#pragma unroll
    for (int j = 0; j < kGatherItems; ++j) {
        const long long item = block0 + local + j * kRows;
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
    if (a.type == QSA_F16) return a.interleaved ? launch_rope<QSA_F16, true>(a, stream) : launch_rope<QSA_F16, false>(a, stream);
    return a.interleaved ? launch_rope<QSA_BF16, true>(a, stream) : launch_rope<QSA_BF16, false>(a, stream);
}

cudaError_t launch_cache_gather(const GatherArgs& a, cudaStream_t stream) {
    if (a.out_type == QSA_F32) return launch_gather<QSA_F32>(a, stream);
    if (a.out_type == QSA_F16) return launch_gather<QSA_F16>(a, stream);
    return launch_gather<QSA_BF16>(a, stream);
}

}  // namespace qsa

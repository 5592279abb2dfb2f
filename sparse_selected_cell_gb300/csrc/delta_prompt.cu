// delta_prompt.cu -- the gated delta rule over the new tokens of several sequences (qsa_delta_prompt).
//
// The rule token by token,
//     S_t = alpha_t S_{t-1} + v'_t k_t^T,  v'_t = beta_t (v_t - alpha_t S_{t-1} k_t),  o_t = S_t q_t,
// solved for chunks of C = 64 tokens.  With G_i the sum of log alpha over the chunk's tokens up
// to i, D_ij = exp(G_i - G_j) for i >= j (never above 1), and rows of V', V, K, Q by token,
//     V' = (I + A)^-1 diag(beta) X,   X = V - exp(G) (K S^T),   A_ij = beta_i D_ij k_i.k_j (i > j),
//     O  = exp(G) (Q S^T) + P V',     P_ij = D_ij q_i.k_j (i >= j),
//     S' = exp(G_C) S + sum_j exp(G_C - G_j) v'_j k_j^T.
// The first kernel (delta_prep_kernel) forms what does not need the state, for all chunks at
// once: T = (I + A)^-1 diag(beta), P, the keys and queries as FP16 operands, and the factors
// of each token.  The second (delta_chunk_kernel) goes through a sequence's chunks.
//
// Numbers.  Keys and queries enter as their FP16 selves times a power of two for each row
// (exact but for elements below 2^-24 of the row's largest, which lose bits); their lengths, 1 / |k|, are factors of
// columns and rows in FP32.  The state, X, V', T and P are pairs of FP16, hi + lo (22 bits), in
// products of which lo lo is left out; the state itself stays in FP32.  All products
// are summed in FP32.  The pairs of a value dim and chunk share a power of two (S, X, V' and V'
// as it is left at the chunk's end each their own), chosen from bounds that the rule gives (a
// chunk lengthens a state row by its values' sum at most) with the decays of the gates, so that
// nothing passes FP16's range and what counts stays in its upper bits.  (Products that end in outputs of
// single FP16, S Q^T without the state's lo, cost outputs 2^-12 of their row's length: 12 x 4,096
// 782 us instead of 825, 1 x 8,192 292 instead of 327.)
//
// Times (BF16, 16 key and 32 value heads; the first kernel's and the second's): 12 sequences x
// 4,096 tokens 329 + 504 us, 1 x 61 12 + 14 (the second begins beside the first: 18 in all);
// 1 x 8,192, cut into segments, 62 + 186, and 21 + 71 to put them together.  FP16, 8 and 16 heads,
// 24 x 1-2,000: 98 + 159.  Neither bytes nor products bound them (12 x 4,096: 183 us of bytes):
// the first is bound by shared memory (60 % of its cycles) and by waiting on it, the second by a
// chain of dependent steps, see there.
#include <type_traits>

#include "linear.cuh"
#include "tc_ptx.cuh"

namespace qsa {
namespace {

constexpr int kC = 64;                               // tokens of a chunk

// ---------------------------------------------------------------- workspace
// Chunk c of sequence s has place first / 64 + s + c, first being the sequence's first token:
// places never meet, and none passes n_tok / 64 + n_seq.  In a step of several sequences only
// those of more than 32 tokens have chunks; there first / 32 + c will do as well, which ends at
// n_tok / 32: the smaller of the two is taken.
constexpr uint32_t kKqBytes = 2 * kC * kHeadDim * 2; // keys, then queries: two 64-dim halves of 128 rows, 128-byte swizzle
// T and P are lower triangular, pairs of FP16, as tiles of 32 rows of 128 bytes, 128-byte swizzle: rows 0 to 31, whose second
// half is zero, one tile for both, hi and lo side by side; rows 32 to 63 a tile for hi and one for lo.
constexpr uint32_t kTileBytes = kC / 2 * 128, kTriBytes = 3 * kTileBytes;
constexpr uint32_t kOffP = kTriBytes, kOffScal = 2 * kTriBytes;
constexpr uint32_t kHeadBytes = kOffScal + 1024;     // T, P, the factors of each token
constexpr float kTriUnit = 16384.f;                  // T's and P's elements, 1 at most, are stored times this
// -exp(G) / |k|, exp(G_C - G) / |k| times the chunk's key unit, exp(G) / |q|, of 64 tokens each; then exp(G_C), the key unit and
// exp(G) of the first token; then exp(G_C - G) of 64 tokens in the call's type, rounded up
constexpr int kScalF = 0, kScalD = kC, kScalO = 2 * kC, kScalG = 3 * kC, kScalU = kScalG + 1, kScalFirst = kScalG + 2, kScalE = kScalG + 4;
static_assert((kScalE + kC / 2) * 4 <= 1024, "the factors' place");

static_assert(kDeltaShort >= kC / 2, "places that do not meet");
__host__ __device__ __forceinline__ bool by_tokens(int n_tok, int n_seq) { return n_seq > 1 && n_tok / (kC / 2) < n_tok / kC + n_seq; }
__device__ __forceinline__ int place_of(const DeltaArgs& a, int first, int s) {
    return by_tokens(a.n_tok, a.n_seq) ? first / (kC / 2) : first / kC + s;
}

struct Blobs {
    uint8_t* kq;                                     // [place][n_k][kKqBytes]
    uint8_t* head;                                   // [place][n_v][kHeadBytes]
};
__host__ __device__ __forceinline__ size_t places(int n_tok, int n_seq) {
    return by_tokens(n_tok, n_seq) ? (size_t)n_tok / (kC / 2) : (size_t)n_tok / kC + n_seq;
}
__device__ __forceinline__ Blobs blobs_of(const DeltaArgs& a) {
    return Blobs{a.workspace, a.workspace + places(a.n_tok, a.n_seq) * a.n_k * kKqBytes};
}

// Whether sequence s, of tokens [span.x, span.y), lies behind all earlier sequences' bounds and before all later ones' (by the
// whole block).  Where bounds fall, sequences can share tokens and places; those that pass here share none, and are the ones
// that delta_prep_kernel finds for their places.  The others are left out.
__device__ __forceinline__ bool in_order(const DeltaArgs& a, int s, int2 span) {
    if (a.n_seq == 1) return true;
    bool off = false;
    for (int i = threadIdx.x; i <= a.n_seq; i += blockDim.x) {
        const int b = min(max(a.cu_tokens[i], 0), a.n_tok);
        off = off || (i < s ? b > span.x : i > s + 1 && b < span.y);
    }
    return !__syncthreads_or(off);
}

// ---------------------------------------------------------------- segments
// A state row's way through a chunk is linear in the row: S' = S R + (what the chunk's values add).  Where there are fewer
// chains (sequences times value heads) than SMs, a long sequence is cut into segments that run at once: the first as it is;
// each other one from a state of zeros, and once more without values from the identity, which gives its R and, as outputs,
// R_t q_t.  delta_join_kernel then takes the states from segment to segment, and delta_add_kernel adds S R_t q_t to the
// segments' outputs, which are FP32 until then.  Cut and in one piece: 1 x 8,192 tokens 328 and 385 us with 32 value heads, 202
// and 340 with 8; 1 x 4,096 180 and 200 with 32, 128 and 175 with 8; 1 x 2,560 140 and 132 with 32, 132 and 126 with 16, 109 and
// 116 with 8; 1 x 2,048 122 and 105, 103 and 100, 96 and 93.  The border lies at 46 chunks with 32 heads, 44 with 16 and 36 with 8:
// 40 chunks in a step is what the rule asks for.  Segments of 8 chunks took 1 x 1,024 86 us instead of 59.
constexpr int kSplitMost = 8, kSplitChunks = 16, kSplitFrom = 40;   // segments of a sequence; chunks of a segment, of a step at least
constexpr int kStateFloats = kHeadDim * kHeadDim;
__host__ __device__ __forceinline__ int most_segments(int n_tok, int n_seq, int n_v, int sms) {
    if (n_tok < kC * kSplitFrom) return 1;
    const long long heads = (long long)n_seq * n_v;
    const long long room = heads > 0 ? (sms / heads + 1) / 2 : 0;   // n segments take 2 n - 1 blocks
    const int most = (int)min((long long)kSplitMost, min(room, (long long)n_tok / (kC * kSplitChunks)));
    return most < 2 ? 1 : most;
}
__device__ __forceinline__ int segments_of(int chunks, int most) { return max(1, min(most, chunks / kSplitChunks)); }
constexpr int kSplitSms = 160;                       // the SMs that the workspace's size reckons with

struct Split {
    float* plain;                                    // [0: from zeros, 1: from the identity][token][n_v][128]
    float* ends;                                     // [sequence, head][kSplitMost]: states at segments' ends; then before the next ones
    float* turns;                                    // [sequence, head][kSplitMost]: the segments' R
};
__device__ __forceinline__ Split split_of(const DeltaArgs& a) {
    const size_t at = places(a.n_tok, a.n_seq) * ((size_t)a.n_k * kKqBytes + (size_t)a.n_v * kHeadBytes);
    Split w;
    w.plain = reinterpret_cast<float*>(a.workspace + at);
    w.ends = w.plain + 2 * (size_t)a.n_tok * a.n_v * kHeadDim;
    w.turns = w.ends + (size_t)a.n_seq * a.n_v * kSplitMost * kStateFloats;
    return w;
}

// ---------------------------------------------------------------- PTX
// The next kernel's blocks may come in as soon as all of this one's have been here.
__device__ __forceinline__ void release_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}

// D (+)= A B^T, A in Tensor Memory, issued by the lane that has `leader` set (one of a converged warp).
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t add, uint32_t leader) {
    asm volatile("{\n .reg .pred e, t;\n setp.ne.b32 e, %4, 0;\n setp.ne.b32 t, %5, 0;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, t;\n}"
                 ::"r"(d), "r"(a), "l"(b), "r"(id), "r"(leader), "r"(add) : "memory");
}

// A factor of at most 1 in the call's type, nowhere below what it was (FP16's smallest for what is below that).
template <int TYPE>
__device__ __forceinline__ uint16_t rounded_up(float x) {
    if (TYPE == QSA_F16) return max(__half_as_ushort(__float2half_ru(x)), (unsigned short)1);
    return __bfloat16_as_ushort(__float2bfloat16_ru(x));
}
// Two values of the call's type at once: the one of larger magnitude (the sign is of no use), and products.
template <int TYPE>
__device__ __forceinline__ uint32_t larger2(uint32_t x, uint32_t y) {
    uint32_t r;
    if (TYPE == QSA_F16) asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    else asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}
template <int TYPE>
__device__ __forceinline__ uint32_t times2(uint32_t x, uint32_t y) {
    uint32_t r;
    if (TYPE == QSA_F16) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    else asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}

// x and y as FP16 pairs: hi the nearest, lo the nearest of what is left (x - hi is exact).
__device__ __forceinline__ void split2(f2 p, uint32_t& hi, uint32_t& lo) {
    float x, y;
    unpair(p, x, y);
    hi = pack_f16x2(x, y);
    asm("{\n .reg .b16 h, l, m;\n mov.b32 {l, h}, %2;\n mov.b16 m, 0xBC00;\n"
        " fma.rn.f32.f16 %0, l, m, %3;\n fma.rn.f32.f16 %1, h, m, %4;\n}"
        : "=f"(x), "=f"(y) : "r"(hi), "f"(x), "f"(y));
    lo = pack_f16x2(x, y);
}
__device__ __forceinline__ f2 pair_of(uint32_t x, uint32_t y) { return pair(__uint_as_float(x), __uint_as_float(y)); }

// Byte offset of 16-byte word j of row r in a tile of 128-byte rows, 128-byte swizzle.
__device__ __forceinline__ uint32_t swz(int r, int j) { return (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4)); }

// ================================================================ what does not need the state
//
// A block has a chunk of a key head and all its value heads, two at a time.  K K^T and Q K^T come from mma.sync over the FP16
// rows (their diagonals give the lengths); (I + A)^-1 by halves of halves: the four 16 x 16 blocks on the diagonal by
// substitution, a column to a thread, then [T11, 0; -T22 A21 T11, T22] for pairs of 16 and of 32, as products of FP16 pairs
// (a column to a thread over all 64 rows took five times as long).  Four blocks to an SM hide one another's waits; 256 threads
// to a block, with the products and rows halved, had a single chunk through 7 % sooner and took 45 % longer for many;
// five blocks in 96 registers took 2 % longer, three 17 %; rows of Q K^T from the other end, so that all warps have ten blocks, 7 %.
constexpr int kPrepThreads = 128;
// A's blocks of 32 x 32: rows and columns 0 to 31, rows 32 to 63 of the same columns, rows and columns 32 to 63.
constexpr int kAStride = 36, kABlock = kC / 2 * kAStride;   // floats to a row of a block, to a block
// Shared memory: keys and queries; in their place two heads' A, then their T in A's place, and P; the tokens' factors.
constexpr uint32_t kABytes = 3 * kABlock * 4, kPrepP = 2 * kABytes, kPrepVec = kPrepP + 2 * kTriBytes;
static_assert(kPrepVec >= kKqBytes && kPrepP % 1024 == 0 && kTriBytes <= kABytes, "A's place");
constexpr int kVecs = 5;                             // of a value head: G's hi and lo in powers of two, beta, exp(G), exp(G_C - G)
constexpr uint32_t kPrepBytes = kPrepVec + (4 * kC + 2 * kVecs * kC) * 4 + 4 * 8 + 1024;

// Column `col` of (I + A)^-1 of an N x N block of A (strictly lower, rows kAStride apart), by substitution.
template <int N>
__device__ __forceinline__ void solve(const float* A, int col, float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < i; j += 4) {
            const float4 w = *reinterpret_cast<const float4*>(A + i * kAStride + j);
            const float e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (j + u < i) acc[u] = fmaf(e[u], x[j + u], acc[u]);
        }
        x[i] = (i == col ? 1.f : 0.f) - ((acc[0] + acc[1]) + (acc[2] + acc[3]));
    }
}

// Operands of m16n8k16 as FP16 pairs from FP32 rows kAStride apart: A of 16 x 16 at M; B of 16 (k) x 8 (n) at M, M[k][n].
struct Frag4 { uint32_t hi[4], lo[4]; };
struct Frag2 { uint32_t hi[2], lo[2]; };
__device__ __forceinline__ Frag4 frag_a(const float* M, int lane) {
    Frag4 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {                    // rows lane / 4 and + 8, columns 2 (lane % 4) and + 8
        const float2 x = *reinterpret_cast<const float2*>(M + ((lane >> 2) + 8 * (i & 1)) * kAStride + 2 * (lane & 3) + 8 * (i >> 1));
        split2(pair(x.x, x.y), f.hi[i], f.lo[i]);
    }
    return f;
}
__device__ __forceinline__ Frag2 frag_b(const float* M, int lane) {
    Frag2 f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float* x = M + (2 * (lane & 3) + 8 * i) * kAStride + (lane >> 2);
        split2(pair(x[0], x[kAStride]), f.hi[i], f.lo[i]);
    }
    return f;
}
__device__ __forceinline__ void mma_pairs(float (&c)[4], const Frag4& a, const Frag2& b) {
    mma16816(c, a.hi, b.hi[0], b.hi[1]);
    mma16816(c, a.lo, b.hi[0], b.hi[1]);
    mma16816(c, a.hi, b.lo[0], b.lo[1]);
}
__device__ __forceinline__ void put_tile(float* M, const float (&c)[4], float sign, int lane) {
    float* at = M + (lane >> 2) * kAStride + 2 * (lane & 3);
    *reinterpret_cast<float2*>(at) = make_float2(sign * c[0], sign * c[1]);
    *reinterpret_cast<float2*>(at + 8 * kAStride) = make_float2(sign * c[2], sign * c[3]);
}

// MORE: more than two value heads to a key head, so that the Gram matrices outlive the first two's inverses.
template <int TYPE, bool MORE>
__global__ void __launch_bounds__(kPrepThreads, MORE ? 3 : 4) delta_prep_kernel(const __grid_constant__ DeltaArgs a) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u = smem_u32(smem_raw), base_u = (raw_u + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (base_u - raw_u);
    float* s_A = reinterpret_cast<float*>(base);
    float* s_r = reinterpret_cast<float*>(base + kPrepVec);          // 1 / |k|, 1 / |q| of the FP16 rows
    int* s_e = reinterpret_cast<int*>(s_r + 2 * kC);                 // the rows' powers of two
    float* s_g = s_r + 4 * kC;                                       // [head of the pair][kVecs][kC]
    double* s_sum = reinterpret_cast<double*>(s_g + 2 * kVecs * kC); // of the warps' decays
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int place = (int)(blockIdx.x / (unsigned)a.n_k), kh = (int)(blockIdx.x - (unsigned)place * (unsigned)a.n_k);
    wait_for_stream();
    // From here on, once all blocks run, the chunks' kernel may set itself up beside this one: whatever was before this one is
    // done, and it waits for this one before it reads what this one writes (1 x 61 tokens 18 us instead of 22).
    release_next();
    // the last sequence whose places begin here or before (every warp for itself)
    int s = 0;
    if (a.n_seq > 1) {
        int lo = 0, len = a.n_seq;                   // the first sequence whose places begin behind this one: in [lo, lo + len]
        while (len > 0) {
            const int step = (len + 31) / 32, at = lo + (lane + 1) * step - 1;
            const bool behind = at >= lo + len || place_of(a, min(max(a.cu_tokens[at], 0), a.n_tok), at) > place;
            const unsigned there = __ballot_sync(0xffffffffu, behind);
            const int f = there ? __ffs(there) - 1 : 32;
            const int from = min(lo + f * step, lo + len);
            len = min(lo + f * step + step - 1, lo + len) - from;
            lo = from;
        }
        s = lo - 1;
    }
    if (s < 0) return;
    const int slot = a.state_slots[s];
    if (slot < 0 || slot >= a.n_slots) return;
    const int2 span = tokens_of(a.cu_tokens, s, a.n_tok);
    const int first = span.x + (place - place_of(a, span.x, s)) * kC, n = min(kC, span.y - first);
    if (first < span.x || n <= 0 || span.y - span.x < a.chunked_from) return;
    const Blobs w = blobs_of(a);
    uint8_t* kq = w.kq + ((size_t)place * a.n_k + kh) * kKqBytes;

    // ---- the decays of two value heads, two warps each, a token to a thread: G in powers of two, summed in FP64, clamped
    // where a factor is long zero; first within a warp
    const int rep = a.n_v / a.n_k, tt = tid & (kC - 1);
    uint16_t gate_a = 0, gate_b = 0;
    float gate_dt = 0.f, gate_log = 0.f;
    auto ask_gates = [&](int h0) {
        const int h = kh * rep + h0 + (warp >> 1);
        if (h0 + (warp >> 1) >= rep || tt >= n) return;
        gate_a = a.a[(long long)(first + tt) * a.a_stride + h], gate_b = a.b[(long long)(first + tt) * a.b_stride + h];
        gate_dt = a.dt_bias[h], gate_log = a.a_log[h];
    };
    double sum = 0.0;
    float* vec = s_g + (warp >> 1) * kVecs * kC;
    auto scan_gates = [&](int h0) {
        sum = 0.0;
        float beta = 0.f;
        if (h0 + (warp >> 1) < rep && tt < n) {
            const float x = log_decay(to_f32(gate_a, TYPE), gate_dt, gate_log);
            sum = x < -700.f ? -1010.0 : (double)x * 1.4426950408889634;
            beta = sigmoid(to_f32(gate_b, TYPE));
        }
        vec[2 * kC + tt] = beta;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += up;
        }
        if (lane == 31) s_sum[warp] = sum;
    };
    auto join_gates = [&]() {                        // behind a barrier
        const double half = s_sum[warp & 2], last = half + s_sum[warp | 1];
        const double G = (warp & 1) ? half + sum : sum;
        const float hi = (float)G, lo = (float)(G - (double)hi);
        vec[tt] = hi, vec[kC + tt] = lo;
        vec[3 * kC + tt] = exp2f(hi) * (1.f + lo * 0.69314718f);
        vec[4 * kC + tt] = exp2f((float)(last - G));
    };
    ask_gates(0);
    // rows into their places as they are: a thread's own 16-byte words, rows 8 p + r0 of 64 keys, then of 64 queries
    const int l = lane & 15, r0 = 2 * warp + (lane >> 4);
    const uint32_t own = (uint32_t)(l >> 3) * (kKqBytes / 2) + swz(r0, l & 7);
    auto ask_rows = [&](const uint16_t* from, long long stride, uint32_t to) {
        const uint16_t* src = from + (long long)(first + r0) * stride + (size_t)kh * kHeadDim + 8 * l;
        const uint16_t* some = from + (long long)first * stride;     // (any address that may be read, where there is no token)
#pragma unroll
        for (int p = 0; p < kC / 8; ++p) {
            const bool there = 8 * p + r0 < n;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                         ::"r"(to + 1024 * p), "l"(there ? src : some), "r"(there ? 16 : 0) : "memory");
            src += 8 * stride;
        }
    };
    ask_rows(a.k, a.k_stride, base_u + own);
    ask_rows(a.q, a.q_stride, base_u + own + kC * 128);
    scan_gates(0);
    // ---- keys and queries to FP16 rows, each times the power of two that puts its largest element in [2^10, 2^11)
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 4
    for (int p = 0; p < 16; ++p) {
        const int r = 8 * p + r0;
        const uint32_t at = own + 1024 * p;
        float x[8];
        unpack8(*reinterpret_cast<const uint4*>(base + at), TYPE, x);
        float m = fmax3(fmax3(fabsf(x[0]), fabsf(x[1]), fabsf(x[2])), fmax3(fabsf(x[3]), fabsf(x[4]), fabsf(x[5])), fmaxf(fabsf(x[6]), fabsf(x[7])));
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        // a row of zeros is any power of two of itself: one that leaves 1 / |k| small
        const int e = m > 0.f ? min(10 - f32_exponent(m), 126) : 90;
        const f2 up = pair(exp2i(e), exp2i(e));
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float u, w2;
            unpair(mul2(pair(x[2 * j], x[2 * j + 1]), up), u, w2);
            h[j] = pack_f16x2(u, w2);
        }
        *reinterpret_cast<uint4*>(base + at) = make_uint4(h[0], h[1], h[2], h[3]);
        if (l == 0) s_e[r] = e;
    }
    tc::fence_proxy_async();
    __syncthreads();
    if (tid == 0) {
        bulk_store(kq, base_u, kKqBytes);
        bulk_commit();
    }
    join_gates();
    // ---- K K^T and Q K^T: a warp has rows 16 warp .. + 15 of both, columns up to the diagonal; of Q Q^T the diagonal's block
    float kk[8][4], qk[8][4], qq[2][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) kk[i][j] = qk[i][j] = qq[i & 1][j] = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t tile = base_u + (uint32_t)(k >> 2) * (kKqBytes / 2);
        const int brow = (lane & 7) + ((lane >> 4) << 3), bword = 2 * (k & 3) + ((lane >> 3) & 1);
        uint32_t ak[4], aq[4], b[4];
        ldmatrix4(tile + swz(16 * warp + (lane & 15), 2 * (k & 3) + (lane >> 4)), ak);
        ldmatrix4(tile + swz(kC + 16 * warp + (lane & 15), 2 * (k & 3) + (lane >> 4)), aq);
        ldmatrix4(tile + swz(kC + 16 * warp + brow, bword), b);
        mma16816(qq[0], aq, b[0], b[1]);
        mma16816(qq[1], aq, b[2], b[3]);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            if (p > warp) continue;
            ldmatrix4(tile + swz(16 * p + brow, bword), b);
            mma16816(kk[2 * p], ak, b[0], b[1]);
            mma16816(kk[2 * p + 1], ak, b[2], b[3]);
            mma16816(qk[2 * p], aq, b[0], b[1]);
            mma16816(qk[2 * p + 1], aq, b[2], b[3]);
        }
    }
    // the diagonals: element (i, i) of a 16 x 16 block lies with lane 4 (i % 8) + (i % 8) / 2
    if ((lane & 3) == (lane >> 3)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 16 * warp + (lane >> 2) + 8 * e;
            float k2 = 0.f;
#pragma unroll
            for (int p = 0; p < 4; ++p)
                if (p == warp) k2 = (lane >> 2) & 1 ? kk[2 * p + e][2 * e + 1] : kk[2 * p + e][2 * e];
            const float q2 = (lane >> 2) & 1 ? qq[e][2 * e + 1] : qq[e][2 * e];
            s_r[i] = i < n ? __frsqrt_rn(k2 + ldexpf(a.eps, 2 * s_e[i])) : 0.f;
            s_r[kC + i] = i < n ? __frsqrt_rn(q2 + ldexpf(a.eps, 2 * s_e[kC + i])) : 0.f;
        }
    }
    if (tid == 0) bulk_wait_read();                  // the rows have left, A may come in their place
    __syncthreads();
    // the power of two that brings the largest 1 / |k| of a stored key into [1/2, 1): the chunk's key unit
    float key_unit = fmaxf(s_r[lane], s_r[lane + 32]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) key_unit = fmaxf(key_unit, __shfl_xor_sync(0xffffffffu, key_unit, o));
    key_unit = exp2i(min(max(-1 - f32_exponent(key_unit), 9), 16));   // (of lengths from 2^10 to 2^14.5, or of rows that eps outweighs)
    // ---- two value heads at a time: warps 0, 1 and 2, 3
    for (int h0 = 0; h0 < (MORE ? rep : 1); h0 += 2) {
        const int mine = h0 + (warp >> 1), h = kh * rep + mine;
        const bool has = mine < rep;
        uint8_t* blob = w.head + ((size_t)place * a.n_v + h) * kHeadBytes;
        if (MORE && h0 > 0) {
            ask_gates(h0);
            scan_gates(h0);
            __syncthreads();
            join_gates();
            __syncthreads();
        }
        if (has) {                                   // each token's factors
            float* scal = reinterpret_cast<float*>(blob + kOffScal);
            scal[kScalF + tt] = -vec[3 * kC + tt] * s_r[tt];
            scal[kScalD + tt] = vec[4 * kC + tt] * (s_r[tt] * key_unit);
            scal[kScalO + tt] = vec[3 * kC + tt] * s_r[kC + tt];
            if (tt == kC - 1) scal[kScalG] = vec[3 * kC + tt], scal[kScalU] = key_unit, scal[kScalFirst] = vec[3 * kC];
            reinterpret_cast<uint16_t*>(scal + kScalE)[tt] = rounded_up<TYPE>(vec[4 * kC + tt]);
        }
#pragma unroll 1
        for (int hh = 0; hh < 2; ++hh) {
            if (h0 + hh >= rep) continue;
            const float* ve = s_g + hh * kVecs * kC;
            float* A = s_A + hh * 3 * kABlock;
            f2 ghi[2], glo[2], ka[2], qa[2];
            const f2 less = pair(-1.f, -1.f);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 16 * warp + (lane >> 2) + 8 * e;
                const float k1 = ve[2 * kC + i] * s_r[i], q1 = s_r[kC + i] * kTriUnit;
                ghi[e] = pair(ve[i], ve[i]), glo[e] = pair(ve[kC + i], ve[kC + i]), ka[e] = pair(k1, k1), qa[e] = pair(q1, q1);
            }
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                if (p > (warp | 1)) continue;        // (zeros above the diagonal's blocks, too, up to the tile's end)
#pragma unroll
                for (int t = 2 * p; t < 2 * p + 2; ++t) {
                    const int j = 8 * t + 2 * (lane & 3);
                    const f2 gj = *reinterpret_cast<const f2*>(ve + j), lj = *reinterpret_cast<const f2*>(ve + kC + j), rj = *reinterpret_cast<const f2*>(s_r + j);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int i = 16 * warp + (lane >> 2) + 8 * e;
                        float x, y;
                        unpair(add2(fma2(less, gj, ghi[e]), fma2(less, lj, glo[e])), x, y);
                        const f2 d = mul2(pair(fast_exp2(x), fast_exp2(y)), rj);
                        unpair(mul2(mul2(pair(kk[t][2 * e], kk[t][2 * e + 1]), ka[e]), d), x, y);
                        *reinterpret_cast<float2*>(A + (warp < 2 ? 0 : 1 + (p >> 1)) * kABlock + (i & 31) * kAStride + (j & 31)) =
                            make_float2(j < i ? x : 0.f, j + 1 < i ? y : 0.f);
                        unpair(mul2(mul2(pair(qk[t][2 * e], qk[t][2 * e + 1]), qa[e]), d), x, y);
                        uint32_t hi, lo;
                        split2(pair(j <= i ? x : 0.f, j + 1 <= i ? y : 0.f), hi, lo);
                        uint8_t* P = base + kPrepP + hh * kTriBytes + 4 * (lane & 3);
                        *reinterpret_cast<uint32_t*>(P + swz(i, t)) = hi;
                        *reinterpret_cast<uint32_t*>(P + (warp < 2 ? swz(i, t + 4) : kTileBytes + swz(i, t))) = lo;
                    }
                }
            }
        }
        tc::fence_proxy_async();
        __syncthreads();
        if (tid == 0) {
            for (int hh = 0; hh < 2 && h0 + hh < rep; ++hh)
                bulk_store(w.head + ((size_t)place * a.n_v + kh * rep + h0 + hh) * kHeadBytes + kOffP, base_u + kPrepP + hh * kTriBytes, kTriBytes);
            bulk_commit();
        }
        // ---- (I + A)^-1 of the warp pair's head, in A's place
        float* A = s_A + (warp >> 1) * 3 * kABlock;
        const int side = warp & 1;
        if (has) {
            // the diagonal's blocks 2 side and 2 side + 1, a column to a thread
            float* D = A + 2 * side * kABlock + (lane & 16) * (kAStride + 1);
            float x[16];
            solve<16>(D, lane & 15, x);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) D[i * kAStride + (lane & 15)] = x[i];
            __syncwarp();
            // the pair of them: T21 = -T22 (A21 T11)
            D = A + 2 * side * kABlock;
            float* A21 = D + 16 * kAStride;
            const float* T22 = A21 + 16;
            float y[2][4] = {}, z[2][4] = {};
            const Frag4 fa = frag_a(A21, lane);
#pragma unroll
            for (int t = 0; t < 2; ++t) mma_pairs(y[t], fa, frag_b(D + 8 * t, lane));
            __syncwarp();
#pragma unroll
            for (int t = 0; t < 2; ++t) put_tile(A21 + 8 * t, y[t], 1.f, lane);
            __syncwarp();
            const Frag4 ft = frag_a(T22, lane);
#pragma unroll
            for (int t = 0; t < 2; ++t) mma_pairs(z[t], ft, frag_b(A21 + 8 * t, lane));
            __syncwarp();
#pragma unroll
            for (int t = 0; t < 2; ++t) put_tile(A21 + 8 * t, z[t], -1.f, lane);
        }
        __syncthreads();
        {
            // the halves: rows 32 + 16 side .. of A21 T11 (T11's block above the diagonal is zero), then of -T22 times that
            float* A21 = A + kABlock + 16 * side * kAStride;
            const float* T22 = A21 + kABlock;
            float y[4][4] = {};
            if (has) {
                const Frag4 f0 = frag_a(A21, lane), f1 = frag_a(A21 + 16, lane);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (t < 2) mma_pairs(y[t], f0, frag_b(A + 8 * t, lane));
                    mma_pairs(y[t], f1, frag_b(A + 16 * kAStride + 8 * t, lane));
                }
                __syncwarp();
#pragma unroll
                for (int t = 0; t < 4; ++t) put_tile(A21 + 8 * t, y[t], 1.f, lane);
            }
            __syncthreads();
            float z[4][4] = {};
            if (has) {
                const Frag4 f0 = frag_a(T22, lane);
#pragma unroll
                for (int t = 0; t < 4; ++t) mma_pairs(z[t], f0, frag_b(A + kABlock + 8 * t, lane));
                if (side) {
                    const Frag4 f1 = frag_a(T22 + 16, lane);
#pragma unroll
                    for (int t = 0; t < 4; ++t) mma_pairs(z[t], f1, frag_b(A + kABlock + 16 * kAStride + 8 * t, lane));
                }
            }
            __syncthreads();                         // both warps have read the product
            if (has) {
#pragma unroll
                for (int t = 0; t < 4; ++t) put_tile(A21 + 8 * t, z[t], -1.f, lane);
            }
        }
        __syncthreads();
        {
            // times beta of the column, as pairs, in A's place: a thread has row tid % 64, eight columns at a time up to its
            // tile's end (zeros above the diagonal, as A has them there)
            const int i = tid & (kC - 1);
            uint4 hi[8], lo[8];
            if (has) {
                const f2 u = pair(kTriUnit, kTriUnit);
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    if (t > 4 * side + 3) continue;
                    const float* row = A + (side + (t >> 2)) * kABlock + (i & 31) * kAStride + 8 * (t & 3);
                    const float4 x = *reinterpret_cast<const float4*>(row), y = *reinterpret_cast<const float4*>(row + 4);
                    const float4 b0 = *reinterpret_cast<const float4*>(vec + 2 * kC + 8 * t), b1 = *reinterpret_cast<const float4*>(vec + 2 * kC + 8 * t + 4);
                    split2(mul2(mul2(pair(x.x, x.y), pair(b0.x, b0.y)), u), hi[t].x, lo[t].x);
                    split2(mul2(mul2(pair(x.z, x.w), pair(b0.z, b0.w)), u), hi[t].y, lo[t].y);
                    split2(mul2(mul2(pair(y.x, y.y), pair(b1.x, b1.y)), u), hi[t].z, lo[t].z);
                    split2(mul2(mul2(pair(y.z, y.w), pair(b1.z, b1.w)), u), hi[t].w, lo[t].w);
                }
            }
            __syncthreads();
            if (has) {
                uint8_t* T = base + (warp >> 1) * kTriBytes;
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    if (t > 4 * side + 3) continue;
                    *reinterpret_cast<uint4*>(T + swz(i, t)) = hi[t];
                    *reinterpret_cast<uint4*>(T + (side ? kTileBytes + swz(i, t) : swz(i, t + 4))) = lo[t];
                }
            }
        }
        tc::fence_proxy_async();
        __syncthreads();
        if (tid == 0) {
            for (int hh = 0; hh < 2 && h0 + hh < rep; ++hh)
                bulk_store(w.head + ((size_t)place * a.n_v + kh * rep + h0 + hh) * kHeadBytes, base_u + hh * kTriBytes, kTriBytes);
            bulk_commit();
            if (h0 + 2 < rep) bulk_wait_read();
        }
        if (h0 + 2 < rep) __syncthreads();           // P and T have left, the gates have been read
    }
    if (tid == 0) bulk_wait();
}

// ================================================================ the chunks of a sequence
//
// A block has one sequence and value head.  Everything is transposed: the 128 value dims are
// the tensor core's rows (Tensor Memory's lanes), tokens or key dims its columns, so that a
// thread of the state warps owns a value dim: its state row stays in its lane, in FP32,
// and whatever passes from one product to the next is a thread's own row, read from the
// accumulator and written back as the next one's A operand, with no exchange at all.
//   state warps (0-7)     two warps to 32 value dims, each with half the key dims and half the tokens:
//                         S -> pair;  X^T = V^T - (S K^T) f -> pair;
//                         V'^T -> pair with each token's decay, and pair without;  S = g S + D
//   output warps (8-11)   O^T = (S Q^T) o + V'^T P^T, to the type, to rows of tokens
//   warp 12               issues all products:  S K^T (hi, lo), S Q^T (hi, lo), V'^T = X^T T^T (hi hi, lo hi, hi lo),
//                         D = V'^T K (hi, lo), V'^T P^T (hi hi, lo hi, hi lo)
//   warps 13, 14          copy a chunk's operands and values ahead
// The chain of one chunk is S K^T -> X -> V' -> D -> S; each of its products begins as soon as
// the first half of its operand is there, and S Q^T is issued behind V', while its pairs are
// formed.  A chunk takes some 5,100 cycles: 750 until a warp has S as pairs, 850 until K S^T is there (the units are
// chosen and the values brought to theirs meanwhile), 600 for X, 1,050 for V' (the state is scaled meanwhile), 750 for its
// pairs with and without decays, then 1,250 for D, beside which the next values are read.  The tensor pipe is busy for 1,850
// of them, and the issue slots for two fifths; conversions to pairs and the outputs' share them.
// (The next values read while K S^T is formed took 5 % longer, the outputs of the chunk before are written then; V' without
// decays as pairs by the output warps 6 %; S Q^T's hi before V', and the largest values with their decays found by a warp of
// its own or by the output warps, the same.)
constexpr int kChunkThreads = 512;
constexpr int kStages = 3, kVStages = 2;
constexpr uint32_t kStageBytes = kKqBytes + kHeadBytes, kVBytes = kC * kHeadDim * 2;
constexpr uint32_t kOffV = kStages * kStageBytes;
constexpr uint32_t kOffOut = kOffV + kVStages * kVBytes;             // [output warp][token][32 dims]
constexpr uint32_t kOffPow = kOffOut + 4 * kC * 64;                  // [chunk & 1][value dim]: 1 / the units of S Q^T and of V' P^T
constexpr uint32_t kOffTop = kOffPow + 2 * kHeadDim * 8;             // [chunk & 1][half][value dim]: largest value; then largest of S
constexpr uint32_t kOffDec = kOffTop + 2 * 2 * 2 * kHeadDim * 4;     // [half][value dim], the call's type: largest value with its decay
constexpr uint32_t kOffBar = kOffDec + 2 * kHeadDim * 2;
enum { BAR_FULL = 0, BAR_EMPTY = BAR_FULL + kStages, BAR_VFULL = BAR_EMPTY + kStages, BAR_VEMPTY = BAR_VFULL + kVStages,
       BAR_S = BAR_VEMPTY + kVStages, BAR_X = BAR_S + 2, BAR_D = BAR_X + 2, BAR_TOP = BAR_D + 2, BAR_KS = BAR_TOP + 4,
       BAR_V, BAR_U, BAR_H, BAR_O, BAR_OFREE, BAR_DRAIN, BAR_DEC, NUM_BARS = BAR_DEC + 4 };
constexpr uint32_t kOffMisc = kOffBar + NUM_BARS * 8;
constexpr uint32_t kChunkBytes = kOffMisc + 16 + 1024;
static_assert(kStageBytes % 1024 == 0 && kChunkBytes <= 227 * 1024, "shared memory");
constexpr int kRanked = 256;                         // sequences, at most, whose blocks go by length (24 x 1-2,000: 249 us instead of 279)
// Sequences that the chunks' kernel has blocks for: by length, no more than can have more than kDeltaShort tokens (64 sequences x
// 16 tokens x 32 heads 126 us instead of 138); delta_short_kernel has looked at the others' bounds and slots.
__host__ __device__ __forceinline__ int ranks(int n_tok, int n_seq) {
    return n_seq > 1 && n_seq <= kRanked ? min(n_seq, n_tok / (kDeltaShort + 1)) : n_seq;
}
static_assert(kSplitSms <= kRanked, "where sequences are cut, their order is looked at with their lengths");
constexpr uint64_t kWaitNs = 1000000000ull;
// Tensor Memory columns.  S: for each 16 key dims 8 columns of hi and 8 of lo.  D: FP32, the decayed state, to which the chunk's
// products are added.  X and, after V' is formed, V' with decays: hi, lo.  V' without lies where S K^T was, V' P^T
// where V' was.
constexpr uint32_t kTmS = 0, kTmKs = 128, kTmH = 128, kTmQs = 192, kTmX = 256, kTmV = 320, kTmPv = 320, kTmD = 384;
// The quarters of an operand in the order in which they are there: each half's first, each half's second.  Two of them have a
// barrier (one each took 1 to 3 % longer: what counts is the issuing warp's time).
__device__ __forceinline__ constexpr int quarter(int i) { return ((i & 1) << 1) | (i >> 1); }

struct Block {
    const DeltaArgs* a;
    uint8_t* base;
    uint32_t base_u, tmem;
    volatile int* abort_flag;
    int s, h, slot, n_tok, n_chunks;                 // of the block's part of the sequence
    int first, chunk0;                               // its first token, and chunk of the sequence
    int kind;                                        // 0: from the sequence's state; 1: from zeros; 2: from the identity, without values
    float* plain;                                    // outputs in FP32 (kinds 1 and 2), or null
    const float* state_in;                           // the pool's state (kind 0)
    float* state_out;
    bool fresh;
};
__device__ __forceinline__ uint32_t bar(const Block& c, int i) { return c.base_u + kOffBar + 8u * i; }
// (without a time to suspend for: the warps wait some ten times a chunk, and wake later with one: 12 x 4,096 tokens 856 us
// instead of 828)
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait(const Block& c, int i, int parity) {
    // inline, without a call (the groups of warps have registers of their own number), and short: the loops of all roles
    // together have to stay in the instruction caches, which neighbouring SMs share
    uint64_t since = 0;
#pragma unroll 1
    while (!try_wait(bar(c, i), (uint32_t)parity)) {
        const uint64_t now = tc::globaltimer_ns();
        if (since == 0) since = now;
        if (*c.abort_flag || now - since > kWaitNs) {
            *c.abort_flag = 1;                       // reported at the block's end
            return false;
        }
    }
    return true;
}
// The warp's stores to Tensor Memory, and its loads from it, are done: tell whoever waits on `i`.
__device__ __forceinline__ void tell(const Block& c, int i) {
    tc::fence_before_sync();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar(c, i));
}

__device__ void copy_role(const Block& c, int lane) {
    const DeltaArgs& a = *c.a;
    const int kh = c.h / (a.n_v / a.n_k), place0 = place_of(a, c.first - c.chunk0 * kC, c.s) + c.chunk0;
    const Blobs w = blobs_of(a);
    wait_for_stream();
    int done = 0;
    for (int i = 0; i < c.n_chunks; ++i, ++done) {
        const int st = i % kStages;
        if (i >= kStages && !wait(c, BAR_EMPTY + st, (i / kStages - 1) & 1)) break;
        if (lane == 0) {
            const uint32_t to = c.base_u + st * kStageBytes;
            mbar_expect(bar(c, BAR_FULL + st), kStageBytes);
            bulk_load(to, w.kq + ((size_t)(place0 + i) * a.n_k + kh) * kKqBytes, kKqBytes, bar(c, BAR_FULL + st));
            bulk_load(to + kKqBytes, w.head + ((size_t)(place0 + i) * a.n_v + c.h) * kHeadBytes, kHeadBytes, bar(c, BAR_FULL + st));
        }
        __syncwarp();
    }
    // no copy may be on its way into shared memory when the block ends
    for (int i = max(0, done - kStages); i < done; ++i)
        if (!tc::mbar_wait_drain(bar(c, BAR_FULL + i % kStages), (uint32_t)(i / kStages) & 1u, kWaitNs)) report(a.dev_status, QSA_DEV_WAIT_TIMEOUT);
}

// The values' rows lie a token's stride apart, 256 bytes each: by a warp's 16-byte copies (as 64 bulk copies a chunk they were
// what the chain waited for, 6,000 instead of 4,000 cycles a chunk).
__device__ void value_role(const Block& c, int lane) {
    const DeltaArgs& a = *c.a;
    const uint16_t* v = a.v + (long long)c.first * a.v_stride + (size_t)c.h * kHeadDim + 8 * (lane & 15);
    for (int i = 0; i < c.n_chunks; ++i) {
        const int vs = i % kVStages;
        if (i >= kVStages && !wait(c, BAR_VEMPTY + vs, (i / kVStages - 1) & 1)) break;
        const uint32_t to = c.base_u + kOffV + vs * kVBytes + lane * 16;
#pragma unroll 4
        for (int p = 0; p < kC / 2; ++p) {
            // tokens that the last chunk does not have are filled with zeros (their factors are zero, but what lies there might be no number)
            const int t = i * kC + 2 * p + (lane >> 4);
            const bool there = t < c.n_tok;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                         ::"r"(to + p * 512), "l"(v + (long long)(there ? t : 0) * a.v_stride), "r"(there ? 16 : 0) : "memory");
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(c, BAR_VFULL + vs)) : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// The whole warp runs this, and one elected lane issues, so that descriptors and addresses stay in uniform registers: a
// 64-column product then takes 35 cycles; issued by a thread alone, 53, whatever its columns.
__device__ void product_role(const Block& c) {
    // FP16 operands: the type fields (bits 7 to 12) zero
    constexpr uint32_t kTypes = ~((7u << 7) | (7u << 10));
    constexpr uint32_t id64 = tc::idesc_bf16(128, 64, false, false) & kTypes;
    constexpr uint32_t id32 = tc::idesc_bf16(128, kC / 2, false, false) & kTypes;
    constexpr uint32_t idD = tc::idesc_bf16(128, kHeadDim, false, true) & kTypes;       // B = keys, key dims along the row
    const uint64_t dkq0 = tc::smem_desc(c.base_u, 16, 1024, 2), dkt0 = tc::smem_desc(c.base_u, kKqBytes / 2, 1024, 2);
    bool ok = true;
    uint32_t leader;
    asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}" : "=r"(leader));
    auto with_queries = [&](uint64_t stage, int lo) {       // S Q^T, of the hi or the lo
#pragma unroll 1
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                product(c.tmem + kTmQs, c.tmem + kTmS + 64 * half + 16 * k + lo,
                        dkq0 + stage + ((half * (kKqBytes / 2) + kC * 128 + k * 32) >> 4), id64, half | k | lo, leader);
    };
    for (int i = 0; i < c.n_chunks && ok; ++i) {
        const int st = i % kStages, par = i & 1;
        const uint64_t stage = (uint64_t)(st * kStageBytes) >> 4, tri = stage + (kKqBytes >> 4);
        if (!(ok = wait(c, BAR_FULL + st, (i / kStages) & 1))) break;
        // V' P^T of the chunk before reads columns that S K^T writes, and products of different accumulators may pass one another
        if (i > 0 && !(ok = wait(c, BAR_O, par ^ 1))) break;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int q = quarter(n);
            if (!(n & 1)) {
                if (!(ok = wait(c, BAR_S + n / 2, par))) break;
                tc::fence_after_sync();
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint64_t d = dkq0 + stage + (((q >> 1) * (kKqBytes / 2) + (q & 1) * 64 + k * 32) >> 4);
                product(c.tmem + kTmKs, c.tmem + kTmS + 32 * q + 16 * k, d, id64, q | k, leader);
                product(c.tmem + kTmKs, c.tmem + kTmS + 32 * q + 16 * k + 8, d, id64, 1, leader);
            }
        }
        if (!ok) break;
        tc::commit_elect(bar(c, BAR_KS));
        if (i > 0 && !(ok = wait(c, BAR_OFREE, par ^ 1))) break;
        tc::fence_after_sync();
#pragma unroll
        for (int n = 0; n < 4; ++n) {                // T is lower triangular: tokens 0 to 31 take tokens 0 to 31 only
            const int b = quarter(n);
            if (!(n & 1)) {
                if (!(ok = wait(c, BAR_X + n / 2, par))) break;
                tc::fence_after_sync();
            }
            const uint32_t at = c.tmem + kTmX + 8 * b;
            const uint64_t d = dkq0 + tri + ((b * 32) >> 4);
            if (b < 2) {
                product(c.tmem + kTmV, at, d, id32, b, leader);
                product(c.tmem + kTmV, at + 32, d, id32, 1, leader);
                product(c.tmem + kTmV, at, d + (64 >> 4), id32, 1, leader);
            }
            product(c.tmem + kTmV + 32, at, d + (kTileBytes >> 4), id32, b, leader);
            product(c.tmem + kTmV + 32, at + 32, d + (kTileBytes >> 4), id32, 1, leader);
            product(c.tmem + kTmV + 32, at, d + (2 * kTileBytes >> 4), id32, 1, leader);
        }
        if (!ok) break;
        tc::commit_elect(bar(c, BAR_V));
        with_queries(stage, 0);
        with_queries(stage, 8);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int b = quarter(n);
            if (!(n & 1)) {
                if (!(ok = wait(c, BAR_D + n / 2, par))) break;
                tc::fence_after_sync();
            }
            const uint64_t d = dkt0 + stage + ((b * 2048) >> 4);
            product(c.tmem + kTmD, c.tmem + kTmX + 8 * b, d, idD, 1, leader);
            product(c.tmem + kTmD, c.tmem + kTmX + 32 + 8 * b, d, idD, 1, leader);
        }
        if (!ok) break;
        tc::commit_elect(bar(c, BAR_U));
        if (!(ok = wait(c, BAR_H, par))) break;
        tc::fence_after_sync();
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint32_t at = c.tmem + kTmH + 8 * b;
            const uint64_t d = dkq0 + tri + ((kOffP + b * 32) >> 4);
            if (b < 2) {
                product(c.tmem + kTmPv, at, d, id32, b, leader);
                product(c.tmem + kTmPv, at + 32, d, id32, 1, leader);
                product(c.tmem + kTmPv, at, d + (64 >> 4), id32, 1, leader);
            }
            product(c.tmem + kTmPv + 32, at, d + (kTileBytes >> 4), id32, b, leader);
            product(c.tmem + kTmPv + 32, at + 32, d + (kTileBytes >> 4), id32, 1, leader);
            product(c.tmem + kTmPv + 32, at, d + (2 * kTileBytes >> 4), id32, 1, leader);
        }
        tc::commit_elect(bar(c, BAR_O));
        tc::commit_elect(bar(c, BAR_EMPTY + st));
    }
    // every product issued above must be complete before Tensor Memory is released
    tc::commit_elect(bar(c, BAR_DRAIN));
    if (!tc::mbar_wait_drain(bar(c, BAR_DRAIN), 0, kWaitNs)) report(c.a->dev_status, QSA_DEV_WAIT_TIMEOUT);
}

template <int TYPE>
__device__ __forceinline__ void both(uint32_t w, float& x, float& y) {
    x = to_f32((uint16_t)(w & 0xFFFFu), TYPE);
    y = to_f32((uint16_t)(w >> 16), TYPE);
}
template <int TYPE>
__device__ __forceinline__ float larger_of(uint32_t w) {
    float x, y;
    both<TYPE>(w, x, y);
    return fmaxf(fabsf(x), fabsf(y));
}
// This thread's value dim of half a chunk's values, two tokens to a word, and the largest of them.
template <int TYPE>
__device__ __forceinline__ float read_values(const uint8_t* values, int half, int r, uint32_t (&v)[16]) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(values) + half * (kC / 2) * kHeadDim + r;
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint32_t x = p[(2 * j) * kHeadDim], y = p[(2 * j + 1) * kHeadDim];
        v[j] = x | (y << 16);
        m = larger2<TYPE>(m, v[j]);
    }
    return larger_of<TYPE>(m);
}

// 2^(14 - e) for x in [2^e, 2^(e+1)): what brings x below 2^15.
__device__ __forceinline__ float unit_of(float x) { return exp2i(14 - max(f32_exponent(x), -80)); }
// 1 / x for a power of two from 2^-126 to 2^126.
__device__ __forceinline__ float inverse(float x) { return __uint_as_float(0x7F000000u - __float_as_uint(x)); }

template <int TYPE, bool SPLIT>
__device__ void state_role(const Block& c, int half, int r, uint32_t lanes) {
    const float4* row = reinterpret_cast<const float4*>(c.state_in + (size_t)r * kHeadDim + half * (kHeadDim / 2));
    float2* pows = reinterpret_cast<float2*>(c.base + kOffPow) + r;
    float* top_v = reinterpret_cast<float*>(c.base + kOffTop) + r;           // + 256 (chunk & 1) + 128 half
    float* top_s = top_v + 4 * kHeadDim;
    const int q = (int)(lanes >> 21);
    const uint32_t tm = c.tmem + lanes, tmS = tm + kTmS + 64 * half, tmD = tm + kTmD + 64 * half, tmT = tm + 32 * half;
    float sm = 0.f;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        uint32_t d[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if ((!SPLIT || c.kind == 0) && !c.fresh) x = row[8 * b + j];
            if (SPLIT && c.kind == 2) {
                const int k = 64 * half + 32 * b + 4 * j;
                x = make_float4(r == k ? 1.f : 0.f, r == k + 1 ? 1.f : 0.f, r == k + 2 ? 1.f : 0.f, r == k + 3 ? 1.f : 0.f);
            }
            d[4 * j] = __float_as_uint(x.x), d[4 * j + 1] = __float_as_uint(x.y);
            d[4 * j + 2] = __float_as_uint(x.z), d[4 * j + 3] = __float_as_uint(x.w);
            sm = fmax3(sm, fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
        }
        tc::tmem_st32(tmD + 32 * b, d);
    }
    tc::tmem_wait_st();
    uint32_t v[16];
    float vm = 0.f;
    auto values = [&](int i) {                       // of chunk i
        if (SPLIT && c.kind == 2) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0u;
            vm = 0.f;
            return true;
        }
        if (!wait(c, BAR_VFULL + i % kVStages, (i / kVStages) & 1)) return false;
        vm = read_values<TYPE>(c.base + kOffV + (i % kVStages) * kVBytes, half, r, v);
        return true;
    };
    if (!values(0)) return;
    // both halves' largest value of the chunk to come, and of the state before the chunk in hand
    auto publish = [&](int i) {
        top_v[(i & 1) * 256 + half * 128] = vm;
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            tc::mbar_arrive(bar(c, BAR_VEMPTY + i % kVStages));
            tc::mbar_arrive(bar(c, BAR_TOP + q));
        }
    };
    // The powers of two of chunk i, one each for S, X, V' and D, from bounds, all with the decays that the gates give: the state
    // row's length before the chunk by its largest element one chunk earlier (12) and that chunk's values, both as far as they
    // are left at that chunk's end; |x| <= |v| + |S|, the state from its first token on; |v'| <= that + the values before it; with
    // its decay to the chunk's end, |S| and values as they are left there.  (What the gates have forgotten has no say from the next
    // chunk on; within the chunk that forgets it X and V' hold what is below 2^-14 of it with fewer bits, below 2^-38 with none.
    // With one unit for S and X, from bounds without decays, 12 x 4,096 tokens took 810 us instead of 854, and what was forgotten
    // cost the chunk behind it its bits.)
    float d_up = 1.f;                                // 1 / the unit of D
    float len = 0.f, s_unit = 1.f;                   // of the state row before the chunk
    float g_tot = 1.f, v_dec = 0.f;                  // of the chunk before: the decay of all of it, the largest value with its decay
    // (units no more than 2^100 finer than what they come from: factors from one to the next stay finite, 2^116 at
    // most with the key unit; from 1, where the first chunk's state is, nothing is cut)
    auto settle = [&](int i) {
        const int par = i & 1;
        if (!wait(c, BAR_TOP + q, par)) return false;
        vm = fmaxf(vm, top_v[par * 256 + (half ^ 1) * 128]);
        sm = fmaxf(sm, top_s[(par ^ 1) * 256 + (half ^ 1) * 128]);
        len = fmaf(12.f * g_tot, sm, 66.f * v_dec);
        s_unit = fminf(unit_of(len), 0x1p100f * inverse(d_up));
        return true;
    };
    uint16_t* dec = reinterpret_cast<uint16_t*>(c.base + kOffDec) + r;       // + 128 half
    top_s[256 + half * 128] = sm;
    publish(0);
    if (!settle(0)) return;
    for (int i = 0; i < c.n_chunks; ++i) {
        const int st = i % kStages, par = i & 1;
        const float* scal = reinterpret_cast<const float*>(c.base + st * kStageBytes + kKqBytes + kOffScal) + 32 * half;
        // ---- the state as the next operand
        const f2 s2 = pair(s_unit * d_up, s_unit * d_up);
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {
            uint32_t d[32];
            tc::tmem_ld32(tmD + 32 * b, d);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t w[16];                      // 8 columns of hi, 8 of lo
#pragma unroll
                for (int j = 0; j < 8; ++j) split2(mul2(s2, pair_of(d[16 * e + 2 * j], d[16 * e + 2 * j + 1])), w[j], w[8 + j]);
                tc::tmem_st16(tmS + 32 * b + 16 * e, w);
            }
            tc::tmem_wait_st();
            tell(c, BAR_S + b);
        }
        // ---- while S K^T is formed: the units of X and V', the values in X's, and the largest of them with its decay
        if (!wait(c, BAR_FULL + st, (i / kStages) & 1)) return;
        g_tot = scal[kScalG - 32 * half];
        const float seen = scal[kScalFirst - 32 * half] * len;
        const float unit = fminf(unit_of(vm + seen), 0x1p100f * s_unit), v_unit = fminf(unit_of(fmaf(66.f, vm, seen)), unit);
        if (half == 0) pows[par * kHeadDim] = make_float2(inverse(s_unit), inverse(v_unit * kTriUnit));
        f2 x2[16];
        uint32_t md = 0u;
        {
            const uint4* decays = reinterpret_cast<const uint4*>(scal + kScalE - 16 * half);
            const f2 unit2 = pair(unit, unit);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const uint4 w = decays[b];
                const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float x, y;
                    both<TYPE>(v[4 * b + j], x, y);
                    x2[4 * b + j] = mul2(pair(x, y), unit2);
                    md = larger2<TYPE>(md, times2<TYPE>(v[4 * b + j], e[j]));
                }
            }
        }
        md = larger2<TYPE>(md, md >> 16);
        dec[half * kHeadDim] = (uint16_t)(md & 0x7FFFu);
        __syncwarp();
        if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar(c, BAR_DEC + q));
        // ---- X = V - f (S K^T)
        const float up = unit * inverse(s_unit);
        const f2 up2 = pair(up, up);
        if (!wait(c, BAR_KS, par)) return;
        tc::fence_after_sync();
        {
            uint32_t ks[32];
            tc::tmem_ld32(tmT + kTmKs, ks);
            tc::tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(scal + kScalF + 16 * b + 2 * j);
                    const uint32_t* k = ks + 16 * b + 2 * j;
                    split2(fma2(mul2(f.x, up2), pair_of(k[0], k[1]), x2[8 * b + j]), hi[j], lo[j]);
                    split2(fma2(mul2(f.y, up2), pair_of(k[2], k[3]), x2[8 * b + j + 1]), hi[j + 1], lo[j + 1]);
                }
                tmem_st8(tm + kTmX + 16 * half + 8 * b, hi);
                tmem_st8(tm + kTmX + 32 + 16 * half + 8 * b, lo);
                tc::tmem_wait_st();
                tell(c, BAR_X + b);
            }
        }
        // ---- while V' is formed: the decayed state for D, and its largest element
        if (!wait(c, BAR_DEC + q, par)) return;
        // (FP16 products round to 2^-25 at the nearest)
        v_dec = larger_of<TYPE>(md & 0x7FFFu | (uint32_t)dec[(half ^ 1) * kHeadDim] << 16) + (TYPE == QSA_F16 ? 0x1p-24f : 0.f);
        const float dv_unit = fminf(unit_of(fmaf(g_tot, len, 66.f * v_dec)), 0x1p100f * fminf(unit, inverse(d_up)));
        const float d_unit = dv_unit * scal[kScalU - 32 * half], gd = g_tot * (d_unit * d_up);
        const f2 g2 = pair(gd, gd);
        sm = 0.f;
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {
            uint32_t d[32];
            tc::tmem_ld32(tmD + 32 * b, d);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                sm = fmax3(sm, fabsf(__uint_as_float(d[2 * j])), fabsf(__uint_as_float(d[2 * j + 1])));
                float gx, gy;
                unpair(mul2(g2, pair_of(d[2 * j], d[2 * j + 1])), gx, gy);
                d[2 * j] = __float_as_uint(gx), d[2 * j + 1] = __float_as_uint(gy);
            }
            tc::tmem_st32(tmD + 32 * b, d);
        }
        sm *= d_up;
        top_s[par * 256 + half * 128] = sm;
        d_up = inverse(d_unit);
        const float down = inverse(unit) * (1.f / kTriUnit), vx = v_unit * down, dx = dv_unit * down;
        // ---- V', with each token's decay to the chunk's end
        if (!wait(c, BAR_V, par)) return;
        tc::fence_after_sync();
        const f2 vx2 = pair(vx, vx), dx2 = pair(dx, dx);
        {
            uint32_t w[32];
            tc::tmem_ld32(tmT + kTmV, w);
            tc::tmem_wait_ld();
            // with decays first: the chain waits for them
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(scal + kScalD + 16 * b + 2 * j);
                    const uint32_t* k = w + 16 * b + 2 * j;
                    split2(mul2(mul2(dx2, pair_of(k[0], k[1])), f.x), hi[j], lo[j]);
                    split2(mul2(mul2(dx2, pair_of(k[2], k[3])), f.y), hi[j + 1], lo[j + 1]);
                }
                tmem_st8(tm + kTmX + 16 * half + 8 * b, hi);
                tmem_st8(tm + kTmX + 32 + 16 * half + 8 * b, lo);
                tc::tmem_wait_st();
                tell(c, BAR_D + b);
            }
            uint32_t one[16], rest[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) split2(mul2(vx2, pair_of(w[2 * j], w[2 * j + 1])), one[j], rest[j]);
            tc::tmem_st16(tm + kTmH + 16 * half, one);
            tc::tmem_st16(tm + kTmH + 32 + 16 * half, rest);
            tc::tmem_wait_st();
        }
        tell(c, BAR_H);
        if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar(c, BAR_EMPTY + st));   // this chunk's factors have been read
        // ---- the next chunk's values, while the products run
        if (i + 1 < c.n_chunks) {
            if (!values(i + 1)) return;
            publish(i + 1);
            if (!settle(i + 1)) return;
        }
        if (!wait(c, BAR_U, par)) return;
        tc::fence_after_sync();
    }
    const f2 up2 = pair(d_up, d_up);
    float4* row_out = reinterpret_cast<float4*>(c.state_out + (size_t)r * kHeadDim + half * (kHeadDim / 2));
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        uint32_t d[32];
        tc::tmem_ld32(tmD + 32 * b, d);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float4 o;
            unpair(mul2(up2, pair_of(d[4 * j], d[4 * j + 1])), o.x, o.y);
            unpair(mul2(up2, pair_of(d[4 * j + 2], d[4 * j + 3])), o.z, o.w);
            row_out[8 * b + j] = o;
        }
    }
}

// Registers that a load from Tensor Memory has filled: nothing that uses them moves before this.
__device__ __forceinline__ void arrived(uint32_t (&x)[16], uint32_t (&y)[16]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) asm volatile("" : "+r"(x[j]), "+r"(y[j]));
}
// 16 lanes x 32 columns as m16n8 accumulators lie: r[4 k + 2 e + u] is lane lane / 4 + 8 e, column 8 k + 2 (lane % 4) + u.
__device__ __forceinline__ void tmem_ld_tiles(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr) : "memory");
}
// Four 8 x 8 tiles of pairs along a column, transposed into rows of 16 bytes, whose addresses the lanes give, eight to a tile.
__device__ __forceinline__ void stmatrix4t(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

__device__ __forceinline__ void stmatrix4(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

// Value dims by tokens become tokens by value dims: accumulators as matrix tiles, so that a transposing store takes 16 tokens x
// 16 dims at once (a token's 16 bits at a time, a lane to a dim, it is twice the instructions, which the state warps pay for).
// PLAIN: segments' FP32 outputs.
template <int TYPE, bool PLAIN>
__device__ void output_role(const Block& c, int q, int lane) {
    const DeltaArgs& a = *c.a;
    const uint32_t mine_u = c.base_u + kOffOut + q * kC * 64;        // a token's 32 dims: four 16-byte words, word w at w ^ (token / 2) % 4
    uint8_t* mine = c.base + kOffOut + q * kC * 64;
    float* whole = reinterpret_cast<float*>(mine);                   // FP32 outputs, 32 tokens at a time: dim d at d ^ 8 ((token / 2) % 4)
    const float2* pows = reinterpret_cast<const float2*>(c.base + kOffPow) + 32 * q + (lane >> 2);
    const uint32_t tm = c.tmem + ((uint32_t)q << 21);
    const int col = 2 * (lane & 3);
    // where this lane's row of the tiles goes: token (lane % 8) + 8 (lane / 16) of 16, word (lane / 8) % 2 of two
    const int row = (lane & 7) + 8 * (lane >> 4), word = (lane >> 3) & 1;
    for (int i = 0; i < c.n_chunks; ++i) {
        const int st = i % kStages, par = i & 1;
        const float* scal = reinterpret_cast<const float*>(c.base + st * kStageBytes + kKqBytes + kOffScal) + kScalO;
        if (!wait(c, BAR_FULL + st, (i / kStages) & 1) || !wait(c, BAR_H, par) || !wait(c, BAR_O, par)) return;
        tc::fence_after_sync();
        // 1 / the units of dims 16 h + 8 e + lane / 4, read before BAR_OFREE: two chunks on they are overwritten
        const float scale = PLAIN && c.kind == 2 ? 1.f : a.scale;
        float2 unit[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                unit[h][e] = pows[(i & 1) * kHeadDim + 16 * h + 8 * e];
                unit[h][e].x *= scale, unit[h][e].y *= scale;
            }
        const int n = min(kC, c.n_tok - i * kC);
        // the next 16 dims' or 32 tokens' accumulators are on their way while the ones before are written
        uint32_t qs[2][16], pv[2][16];
        auto ask = [&](int half, int h) {            // 32 tokens of 16 dims
            tmem_ld_tiles(tm + ((uint32_t)h << 20) + kTmQs + 32 * half, qs[h]);
            tmem_ld_tiles(tm + ((uint32_t)h << 20) + kTmPv + 32 * half, pv[h]);
        };
        auto put = [&](int half, int h) {
            uint32_t w[4];
            f2 us[2], uv[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                us[e] = pair(unit[h][e].x, unit[h][e].x), uv[e] = pair(unit[h][e].y, unit[h][e].y);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const f2 o = *reinterpret_cast<const f2*>(scal + 32 * half + 8 * k + col);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 4 * k + 2 * e;
                    float x, y;
                    unpair(fma2(mul2(o, us[e]), pair_of(qs[h][r], qs[h][r + 1]), mul2(uv[e], pair_of(pv[h][r], pv[h][r + 1]))), x, y);
                    if (PLAIN) {
                        float* to = whole + (8 * k + col) * 32 + ((16 * h + 8 * e + (lane >> 2)) ^ (4 * col));
                        to[0] = x, to[32] = y;
                    } else {
                        w[2 * (k & 1) + e] = pack2(x, y, TYPE);
                    }
                }
                if (!PLAIN && (k & 1)) {
                    const int t = 32 * half + 8 * (k - 1) + row;
                    stmatrix4t(mine_u + t * 64 + (((2 * h + word) ^ ((t >> 1) & 3)) << 4), w);
                }
            }
        };
        ask(0, 0);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            tc::tmem_wait_ld();
            arrived(qs[0], pv[0]);
            ask(half, 1);
            put(half, 0);
            tc::tmem_wait_ld();
            arrived(qs[1], pv[1]);
            if (half == 0) ask(1, 0);
            else tell(c, BAR_OFREE);
            put(half, 1);
            if (PLAIN) {
                __syncwarp();
                float* to = c.plain + ((size_t)(c.first + i * kC + 32 * half) * a.n_v + c.h) * kHeadDim + 32 * q + 4 * (lane & 7);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int t = (lane >> 3) + 4 * j;
                    if (32 * half + t < n)
                        *reinterpret_cast<float4*>(to + (size_t)t * a.n_v * kHeadDim) =
                            *reinterpret_cast<const float4*>(whole + t * 32 + ((4 * (lane & 7)) ^ (8 * ((t >> 1) & 3))));
                }
                __syncwarp();
            }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(c, BAR_EMPTY + st));
        if (PLAIN) continue;
        uint16_t* to = a.out + (long long)(c.first + i * kC) * a.out_stride + (size_t)c.h * kHeadDim + 32 * q + 8 * (lane & 3);
#pragma unroll 2
        for (int t = lane >> 2; t < n; t += 8)
            *reinterpret_cast<uint4*>(to + (long long)t * a.out_stride) =
                *reinterpret_cast<const uint4*>(mine + t * 64 + (((lane & 3) ^ ((t >> 1) & 3)) << 4));
        __syncwarp();
    }
}

// SPLIT: sequences may be cut into segments (see above).
template <int TYPE, bool SPLIT>
__global__ void __launch_bounds__(kChunkThreads, 1) delta_chunk_kernel(const __grid_constant__ DeltaArgs a) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u = smem_u32(smem_raw), base_u = (raw_u + 1023u) & ~1023u;
    Block c;
    c.a = &a;
    c.base = smem_raw + (base_u - raw_u);
    c.base_u = base_u;
    c.abort_flag = reinterpret_cast<volatile int*>(c.base + kOffMisc + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const unsigned heads = (unsigned)ranks(a.n_tok, a.n_seq) * (unsigned)a.n_v, part = SPLIT ? blockIdx.x / heads : 0u, item = blockIdx.x - part * heads;
    c.s = (int)(item / (unsigned)a.n_v);
    c.h = (int)(item - (unsigned)c.s * (unsigned)a.n_v);
    bool ordered = true;
    if (a.n_seq > 1 && a.n_seq <= kRanked) {
        // the longest sequences first: block b's is the one of which c.s are longer (or as long, and before it); and whether it is
        // in order with all others, as in_order has it
        int* bounds = reinterpret_cast<int*>(c.base + kOffOut);       // (no bulk copy ever writes there)
        for (int i = tid; i <= a.n_seq; i += kChunkThreads) bounds[i] = min(max(a.cu_tokens[i], 0), a.n_tok);
        __syncthreads();
        for (int i = tid; i < a.n_seq; i += kChunkThreads) {
            const int first = bounds[i], end = max(bounds[i + 1], first);
            int rank = 0, off = 0;
            for (int j = 0, at = bounds[0]; j < a.n_seq; ++j) {
                const int next = bounds[j + 1], len = max(next - at, 0);
                rank += len > end - first || (len == end - first && j < i) ? 1 : 0;
                off += j < i ? at > first : j > i && next < end;
                at = next;
            }
            if (rank == c.s) bounds[kRanked + 1] = off ? -1 - i : i;
        }
        __syncthreads();
        c.s = bounds[kRanked + 1];
        ordered = c.s >= 0;
        c.s = ordered ? c.s : -1 - c.s;
        __syncthreads();
    }
    // Behind delta_prep_kernel this kernel is released when all of that one's blocks have passed their own
    // wait, so that everything before it is there already: only the copies of its results wait for it here, and every block
    // does before it ends, so that this kernel's end means that one's too.
    c.slot = a.state_slots[c.s];
    const int2 span = tokens_of(a.cu_tokens, c.s, a.n_tok);
    if (c.h == 0 && part == 0 && tid == 0) {
        if (tokens_bad(a.cu_tokens, c.s, a.n_tok)) report(a.dev_status, QSA_DEV_BAD_SEQ_LEN);
        if (c.slot >= a.n_slots) report(a.dev_status, QSA_DEV_BAD_STATE);
    }
    if (c.slot < 0 || c.slot >= a.n_slots || span.y - span.x < a.chunked_from || !ordered ||
        (!SPLIT && a.n_seq > kRanked && !in_order(a, c.s, span))) {      // (segments: fewer sequences than SMs)
        wait_for_stream();
        return;
    }
    c.fresh = a.old_lens && a.old_lens[c.s] <= 0;
    float* pool = a.state + ((size_t)c.slot * a.n_v + c.h) * kStateFloats;
    const int chunks = (span.y - span.x + kC - 1) / kC;
    c.kind = c.chunk0 = 0;
    c.n_chunks = chunks;
    c.first = span.x;
    c.n_tok = span.y - span.x;
    c.state_in = c.state_out = pool;
    c.plain = nullptr;
    if (SPLIT) {
        // parts 0 .. n_split - 1 are the segments, from zeros but the first; then all but the first from the identity
        const int segments = segments_of(chunks, a.n_split), segment = (int)part < a.n_split ? (int)part : (int)part - a.n_split + 1;
        if (segment >= segments) {
            wait_for_stream();
            return;
        }
        const int each = (chunks + segments - 1) / segments;
        c.kind = (int)part >= a.n_split ? 2 : part > 0 ? 1 : 0;
        c.chunk0 = segment * each;
        c.n_chunks = min(each, chunks - c.chunk0);
        c.first = span.x + c.chunk0 * kC;
        c.n_tok = min(c.n_chunks * kC, span.y - c.first);
        if (segments > 1) {
            const Split w = split_of(a);
            c.state_out = (c.kind == 2 ? w.turns : w.ends) + (((size_t)c.s * a.n_v + c.h) * kSplitMost + segment) * kStateFloats;
            if (c.kind) c.plain = w.plain + (c.kind - 1) * (size_t)a.n_tok * a.n_v * kHeadDim;
        }
    }
    if (c.n_chunks == 0) {
        if (c.fresh) {
            float4* st = reinterpret_cast<float4*>(pool);
            for (int i = tid; i < kHeadDim * kHeadDim / 4; i += kChunkThreads) st[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        wait_for_stream();
        return;
    }
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(c.base + kOffMisc);
    if (tid == 0) {
        for (int st = 0; st < kStages; ++st) {
            tc::mbar_init(bar(c, BAR_FULL + st), 1);
            tc::mbar_init(bar(c, BAR_EMPTY + st), 13);         // the products', the state warps' and the output warps' last use
        }
        for (int st = 0; st < kVStages; ++st) {
            tc::mbar_init(bar(c, BAR_VFULL + st), 32);
            tc::mbar_init(bar(c, BAR_VEMPTY + st), 8);
        }
        for (int b = 0; b < 4; ++b) {
            if (b < 2) {
                tc::mbar_init(bar(c, BAR_S + b), 8);
                tc::mbar_init(bar(c, BAR_X + b), 8);
                tc::mbar_init(bar(c, BAR_D + b), 8);
            }
            tc::mbar_init(bar(c, BAR_TOP + b), 2);
            tc::mbar_init(bar(c, BAR_DEC + b), 2);
        }
        tc::mbar_init(bar(c, BAR_KS), 1);
        tc::mbar_init(bar(c, BAR_V), 1);
        tc::mbar_init(bar(c, BAR_U), 1);
        tc::mbar_init(bar(c, BAR_H), 8);
        tc::mbar_init(bar(c, BAR_O), 1);
        tc::mbar_init(bar(c, BAR_OFREE), 4);
        tc::mbar_init(bar(c, BAR_DRAIN), 1);
        *c.abort_flag = 0;
        tc::fence_mbar_init();
    }
    if (warp == 12) {
        tc::tmem_alloc(smem_u32(tmem_holder), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    c.tmem = *tmem_holder;
    // registers: the launch's 512 x 128 as 168 + 168 + 96 + 80 for the four groups of four warps
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        state_role<TYPE, SPLIT>(c, warp >> 2, tid & 127, (uint32_t)(warp & 3) << 21);
        tc::tmem_wait_st();                          // (of a chunk that a wait running out has ended)
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        if (SPLIT && c.plain) output_role<TYPE, true>(c, warp - 8, lane);
        else output_role<TYPE, false>(c, warp - 8, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == 12) product_role(c);
        else if (warp == 13) copy_role(c, lane);
        else if (warp == 14 && !(SPLIT && c.kind == 2)) value_role(c, lane);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (tid == 0 && *c.abort_flag) report(a.dev_status, QSA_DEV_WAIT_TIMEOUT);
    if (warp == 12) {
        tc::fence_after_sync();
        tc::tmem_dealloc(c.tmem, 512);
    }
}

// ================================================================ segments put together
// States from segment to segment: S before segment g + 1 = (S before g) R_g + (segment g's from zeros), a block to a sequence
// and head.  A warp has 16 state rows, as accumulators of m16n8k16, which are the next product's A operand as they lie.
constexpr int kJoinThreads = 256;
constexpr uint32_t kRBytes = kHeadDim * kHeadDim * 2, kJoinBytes = 2 * kRBytes + 64 + 1024;
static_assert(2 * kRBytes == kStateFloats * 4, "a state as pairs in its own place");
// 1 / the units of the rows of S before segment g, of a sequence and head: where the first segment's R would be, which has none.
__device__ __forceinline__ float* units_of(const Split& w, size_t item, int g) { return w.turns + item * kSplitMost * kStateFloats + g * kHeadDim; }
static_assert(kSplitMost * kHeadDim <= kStateFloats, "the units' place");

__global__ void __launch_bounds__(kJoinThreads) delta_join_kernel(const __grid_constant__ DeltaArgs a) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u = smem_u32(smem_raw), base_u = (raw_u + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (base_u - raw_u);         // R as FP16 pairs: hi, then lo, two halves of 64 columns each
    float* s_top = reinterpret_cast<float*>(base + 2 * kRBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int sq = (int)(blockIdx.x / (unsigned)a.n_v), h = (int)(blockIdx.x - (unsigned)sq * (unsigned)a.n_v);
    wait_for_stream();
    const int slot = a.state_slots[sq];
    const int2 span = tokens_of(a.cu_tokens, sq, a.n_tok);
    const int chunks = (span.y - span.x + kC - 1) / kC, segments = segments_of(chunks, a.n_split);
    if (slot < 0 || slot >= a.n_slots || segments < 2 || span.y - span.x < a.chunked_from || !in_order(a, sq, span)) return;
    const Split w = split_of(a);
    const size_t item = (size_t)blockIdx.x * kSplitMost;
    const int row = 16 * warp + (lane >> 2), col = 2 * (lane & 3);
    float s[16][4];
    auto place = [&](float* m, int t, int e) { return reinterpret_cast<float2*>(m + (row + 8 * e) * kHeadDim + 8 * t + col); };
#pragma unroll
    for (int t = 0; t < 16; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float2 x = *place(w.ends + item * kStateFloats, t, e);
            s[t][2 * e] = x.x, s[t][2 * e + 1] = x.y;
        }
    for (int g = 1; g < segments; ++g) {
        const float4* turn = reinterpret_cast<const float4*>(w.turns + (item + g) * kStateFloats);
        constexpr int kEach = kStateFloats / 4 / kJoinThreads;
        float4 rows[kEach];                          // four columns of R's rows warp, warp + 8, ..
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) rows[i] = turn[tid + i * kJoinThreads];
#pragma unroll
        for (int i = 0; i < kEach; ++i) top = fmax3(top, fmaxf(fabsf(rows[i].x), fabsf(rows[i].y)), fmaxf(fabsf(rows[i].z), fabsf(rows[i].w)));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) s_top[warp] = top;
        __syncthreads();                             // (the products of the segment before are done, too)
#pragma unroll
        for (int i = 0; i < kJoinThreads / 32; ++i) top = fmaxf(top, s_top[i]);
        // powers of two: one for R, one for each state row
        const float r_unit = unit_of(top);
        float unit[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float m = 0.f;
#pragma unroll
            for (int t = 0; t < 16; ++t) m = fmax3(m, fabsf(s[t][2 * e]), fabsf(s[t][2 * e + 1]));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            unit[e] = unit_of(m);
        }
        // S before segment g for delta_add_kernel, in its place: pairs of FP16 in units as that one's tiles, hi, then lo
        uint8_t* image = reinterpret_cast<uint8_t*>(w.ends + (item + g - 1) * kStateFloats);
#pragma unroll
        for (int t = 0; t < 16; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e)
            {
                uint32_t hi, lo;
                split2(mul2(pair(s[t][2 * e], s[t][2 * e + 1]), pair(unit[e], unit[e])), hi, lo);
                uint32_t* at = reinterpret_cast<uint32_t*>(image + (t >> 3) * (kHeadDim * 128) + swz(row + 8 * e, t & 7) + 4 * (lane & 3));
                at[0] = hi, at[kRBytes / 4] = lo;
            }
        if ((lane & 3) == 0) {
            float* units = units_of(w, blockIdx.x, g);
            units[row] = 1.f / unit[0], units[row + 8] = 1.f / unit[1];
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            uint2 hi, lo;
            split2(mul2(pair(rows[i].x, rows[i].y), pair(r_unit, r_unit)), hi.x, lo.x);
            split2(mul2(pair(rows[i].z, rows[i].w), pair(r_unit, r_unit)), hi.y, lo.y);
            uint8_t* at = base + (lane >> 4) * (kHeadDim * 128) + swz(warp + 8 * i, (lane & 15) >> 1) + 8 * (lane & 1);
            *reinterpret_cast<uint2*>(at) = hi;
            *reinterpret_cast<uint2*>(at + kRBytes) = lo;
        }
        __syncthreads();
        float n[16][4];
#pragma unroll
        for (int t = 0; t < 16; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) n[t][j] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            Frag4 f;
#pragma unroll
            for (int j = 0; j < 4; ++j)              // rows lane / 4 and + 8 of tiles 2 k and 2 k + 1
                split2(mul2(pair(s[2 * k + (j >> 1)][2 * (j & 1)], s[2 * k + (j >> 1)][2 * (j & 1) + 1]), pair(unit[j & 1], unit[j & 1])), f.hi[j], f.lo[j]);
#pragma unroll
            for (int t = 0; t < 8; ++t) {            // columns 16 t .. + 15: R's rows 16 k .. + 15 as they lie, transposed
                uint32_t hi[4], lo[4];
                const uint32_t at = base_u + (t >> 2) * (kHeadDim * 128) + swz(16 * k + (lane & 15), 2 * (t & 3) + (lane >> 4));
                ldmatrix4t(at, hi);
                ldmatrix4t(at + kRBytes, lo);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    mma16816(n[2 * t + u], f.hi, hi[2 * u], hi[2 * u + 1]);
                    mma16816(n[2 * t + u], f.lo, hi[2 * u], hi[2 * u + 1]);
                    mma16816(n[2 * t + u], f.hi, lo[2 * u], lo[2 * u + 1]);
                }
            }
        }
        float* add = w.ends + (item + g) * kStateFloats;
        float* pool = a.state + ((size_t)slot * a.n_v + h) * kStateFloats;
        const float up[2] = {1.f / unit[0] / r_unit, 1.f / unit[1] / r_unit};
#pragma unroll
        for (int t = 0; t < 16; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 x = *place(add, t, e);
                s[t][2 * e] = fmaf(n[t][2 * e], up[e], x.x), s[t][2 * e + 1] = fmaf(n[t][2 * e + 1], up[e], x.y);
                if (g + 1 == segments) *place(pool, t, e) = make_float2(s[t][2 * e], s[t][2 * e + 1]);
            }
    }
}

// The outputs of segments behind the first: from zeros, plus scale (S before the segment) (R_t q_t).  A block takes
// kAddChunks consecutive chunks of a sequence and head: tokens by value dims, S in shared memory as pairs of FP16 with a power
// of two for each row (as delta_join_kernel left it), the tokens' R_t q_t likewise.
constexpr int kAddThreads = 256, kAddChunks = 4;
constexpr uint32_t kAddS = 0, kAddT = 2 * kRBytes, kAddTlo = kC * kHeadDim * 2, kAddUnit = kAddT + 2 * kAddTlo;
constexpr uint32_t kAddBytes = kAddUnit + (kHeadDim + kC) * 4 + 1024;

template <int TYPE>
__global__ void __launch_bounds__(kAddThreads, 2) delta_add_kernel(const __grid_constant__ DeltaArgs a, const int groups) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u = smem_u32(smem_raw), base_u = (raw_u + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (base_u - raw_u);
    float* s_unit = reinterpret_cast<float*>(base + kAddUnit);       // 1 / the units of S's rows, then of the tokens
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const unsigned item = blockIdx.x / (unsigned)groups;
    const int group = (int)(blockIdx.x - item * (unsigned)groups);
    const int sq = (int)(item / (unsigned)a.n_v), h = (int)(item - (unsigned)sq * (unsigned)a.n_v);
    wait_for_stream();
    const int slot = a.state_slots[sq];
    const int2 span = tokens_of(a.cu_tokens, sq, a.n_tok);
    const int chunks = (span.y - span.x + kC - 1) / kC, segments = segments_of(chunks, a.n_split);
    if (slot < 0 || slot >= a.n_slots || segments < 2 || span.y - span.x < a.chunked_from || !in_order(a, sq, span)) return;
    const int each = (chunks + segments - 1) / segments;
    const Split w = split_of(a);
    const size_t apart = (size_t)a.n_v * kHeadDim;
    int held = 0;
    for (int c = max(group * kAddChunks, each); c < min(chunks, (group + 1) * kAddChunks); ++c) {
        const int g = c / each;
        const int first = span.x + c * kC, n = min(kC, span.y - first);
        __syncthreads();                             // the tiles of the chunk before have been read
        if (g != held) {
            held = g;
            const uint8_t* S = reinterpret_cast<const uint8_t*>(w.ends + ((size_t)item * kSplitMost + g - 1) * kStateFloats);
#pragma unroll
            for (int i = 0; i < (int)(kAddT / 16) / kAddThreads; ++i) {
                const uint32_t at = 16 * (tid + i * kAddThreads);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(base_u + kAddS + at), "l"(S + at) : "memory");
            }
            if (tid < kHeadDim) s_unit[tid] = units_of(w, item, g)[tid];
        }
        // R_t q_t of eight tokens of a warp (every eighth), a lane's four elements of each: the largest, the unit, FP16; zeros
        // from the sequence's end on
        const float* turned = w.plain + (size_t)a.n_tok * apart + (size_t)first * apart + h * kHeadDim;
        float4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = warp + 8 * i < n ? reinterpret_cast<const float4*>(turned + (warp + 8 * i) * apart)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = warp + 8 * i;
            float m = fmaxf(fmaxf(fabsf(x[i].x), fabsf(x[i].y)), fmaxf(fabsf(x[i].z), fabsf(x[i].w)));
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float unit = unit_of(m);
            uint2 hi, lo;
            split2(mul2(pair(x[i].x, x[i].y), pair(unit, unit)), hi.x, lo.x);
            split2(mul2(pair(x[i].z, x[i].w), pair(unit, unit)), hi.y, lo.y);
            uint8_t* at = base + kAddT + (lane >> 4) * (kC * 128) + swz(r, (lane & 15) >> 1) + 8 * (lane & 1);
            *reinterpret_cast<uint2*>(at) = hi;
            *reinterpret_cast<uint2*>(at + kAddTlo) = lo;
            if (lane == 0) s_unit[kHeadDim + r] = 1.f / unit;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        // the outputs so far, on their way meanwhile
        const float* from = w.plain + ((size_t)first * a.n_v + h) * kHeadDim;
        float2 so_far[2][8];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int t = 16 * (warp & 3) + (lane >> 2) + 8 * e;
                so_far[e][j] = t < n ? *reinterpret_cast<const float2*>(from + t * apart + 64 * (warp >> 2) + 8 * j + 2 * (lane & 3))
                                     : make_float2(0.f, 0.f);
            }
        __syncthreads();
        const int m0 = 16 * (warp & 3), n0 = 64 * (warp >> 2);       // tokens m0 .. + 15, value dims n0 .. + 63
        float acc[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[t][j] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t f[4], fl[4], b[4], bl[4];
            const uint32_t at = base_u + kAddT + (k >> 2) * (kC * 128) + swz(m0 + (lane & 15), 2 * (k & 3) + (lane >> 4));
            ldmatrix4(at, f);
            ldmatrix4(at + kAddTlo, fl);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint32_t rows = base_u + kAddS + (k >> 2) * (kHeadDim * 128) + swz(n0 + 16 * t + (lane & 7) + ((lane >> 4) << 3), 2 * (k & 3) + ((lane >> 3) & 1));
                ldmatrix4(rows, b);
                ldmatrix4(rows + kRBytes, bl);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    mma16816(acc[2 * t + u], f, b[2 * u], b[2 * u + 1]);
                    mma16816(acc[2 * t + u], fl, b[2 * u], b[2 * u + 1]);
                    mma16816(acc[2 * t + u], f, bl[2 * u], bl[2 * u + 1]);
                }
            }
        }
        __syncthreads();                             // R_t q_t has been read: the outputs in its place, then out by rows
#pragma unroll
        for (int j = 0; j < 8; j += 2) {             // tiles: tokens 0-7 and 8-15 of dims 8 j, then of dims 8 (j + 1)
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float up = s_unit[kHeadDim + m0 + (lane >> 2) + 8 * e] * a.scale;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float2 unit = *reinterpret_cast<const float2*>(s_unit + n0 + 8 * (j + u) + 2 * (lane & 3)), x = so_far[e][j + u];
                    w[2 * u + e] = pack2(fmaf(acc[j + u][2 * e], up * unit.x, x.x), fmaf(acc[j + u][2 * e + 1], up * unit.y, x.y), TYPE);
                }
            }
            stmatrix4(base_u + kAddT + (warp >> 2) * (kC * 128) + swz(m0 + (lane & 15), j + (lane >> 4)), w);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = tid + i * kAddThreads, t = at >> 4, word = at & 15;
            if (t < n)
                *reinterpret_cast<uint4*>(a.out + (long long)(first + t) * a.out_stride + (size_t)h * kHeadDim + 8 * word) =
                    *reinterpret_cast<const uint4*>(base + kAddT + (word >> 3) * (kC * 128) + swz(t, word & 7));
        }
    }
}

template <int TYPE>
cudaError_t launch(DeltaArgs a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    a.n_split = most_segments(a.n_tok, a.n_seq, a.n_v, sms < kSplitSms ? sms : kSplitSms);
    const long long prep = (long long)places(a.n_tok, a.n_seq) * a.n_k, heads = (long long)a.n_seq * a.n_v,
                    chunks = (long long)ranks(a.n_tok, a.n_seq) * a.n_v * (2 * a.n_split - 1);
    if (prep > 0x7fffffffLL || chunks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    // Lengths are device data.  Few tokens in all: every sequence is short.  Several sequences: some may be.
    if (a.n_tok <= kDeltaShort || a.n_seq > 1) {
        e = launch_delta_short(a, stream);
        if (e != cudaSuccess || a.n_tok <= kDeltaShort) return e;
        a.chunked_from = kDeltaShort + 1;
    }
    auto* kernel = a.n_v > 2 * a.n_k ? delta_prep_kernel<TYPE, true> : delta_prep_kernel<TYPE, false>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPrepBytes);
    auto* chunk_kernel = a.n_split > 1 ? delta_chunk_kernel<TYPE, true> : delta_chunk_kernel<TYPE, false>;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kChunkBytes);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(kernel, dim3((unsigned)prep), kPrepThreads, kPrepBytes, stream, a);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(chunk_kernel, dim3((unsigned)chunks), kChunkThreads, kChunkBytes, stream, a);
    if (e != cudaSuccess || a.n_split < 2) return e;
    e = cudaFuncSetAttribute(delta_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kJoinBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(delta_add_kernel<TYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kAddBytes);
    if (e == cudaSuccess) e = launch_overlapped(delta_join_kernel, dim3((unsigned)heads), kJoinThreads, kJoinBytes, stream, a);
    if (e != cudaSuccess) return e;
    const int groups = (a.n_tok / kC + 1 + kAddChunks - 1) / kAddChunks;
    return launch_overlapped(delta_add_kernel<TYPE>, dim3((unsigned)(heads * groups)), kAddThreads, kAddBytes, stream, a, groups);
}

}  // namespace

size_t delta_prompt_workspace(int n_tok, int n_seq, int n_k, int n_v) {
    if (n_tok <= kDeltaShort) return 256;            // (token by token, without)
    size_t bytes = places(n_tok, n_seq) * ((size_t)n_k * kKqBytes + (size_t)n_v * kHeadBytes) + 256;
    if (most_segments(n_tok, n_seq, n_v, kSplitSms) > 1)
        bytes += ((size_t)n_tok * kHeadDim + (size_t)n_seq * kSplitMost * kStateFloats) * 2 * n_v * 4;
    return bytes;
}

cudaError_t launch_delta_prompt(const DeltaArgs& a, cudaStream_t stream) {
    return a.type == QSA_F16 ? launch<QSA_F16>(a, stream) : launch<QSA_BF16>(a, stream);
}

}  // namespace qsa

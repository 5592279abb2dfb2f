// paged_attn.cu -- attention of one new token per sequence over its whole paged
// INT8 cache (qsa_paged_attn), split over the cache's length and joined.
//
// out[s][i] = sum_c softmax_c(q . k_c * sm_scale) v_c over the resident cells c of
// the sequence (the last `window` of them), k_c = int8 * FP16 scale.
//
// Bound by HBM: a cell costs 260 bytes per KV head and 4 * 128 * group flops (24
// flops per byte at 12 query heads), so what matters is that every SM always has
// enough copies in flight, and that the arithmetic per byte fits beside them.
//
// Split.  The pages of all (sequence, KV head, 16-row tile) items, laid end to end,
// are cut into equal runs of pages, one per CTA of a grid of two per SM: ragged
// batches, one long sequence and many short ones all give every SM the same number
// of bytes.  Each CTA sums the page counts itself (the lengths are device data; no
// host value is needed, so a captured graph follows the lengths).  A run touches at
// most two items that it does not hold whole, its first and its last: their partial
// (max, sum, O) go to the workspace and paged_join_kernel, launched beside this
// kernel and waiting for it on the device, joins them in the order of the CTAs.
//
// A CTA: a producer warp copies whole pages of one KV head (8 KB of K, 8 KB of V by
// TMA in the 128-byte swizzle, 128-byte scale rows by bulk copy) into a ring; four
// consumer warps take pages in turn, each page by one warp with its own running
// softmax, and merge at the end of each item.  The tensor work is mma.sync
// m16n8k16: 16 rows per tile (12 query heads) would fill an eighth of a
// tcgen05.mma's 128 rows, whose operands would also have to be written back to
// shared memory in 16 bits, twice the traffic of the INT8 rows; here they are
// converted in registers, exactly.
//   * S = Q K^T on FP16 operands.  Q is scaled per row by a power of two (its
//     largest element in [2^12, 2^13)) and held in registers; within each 64-dim
//     half the dims are permuted (Q and K alike) so that a lane's K operands of four
//     k steps are one 16-byte piece of the INT8 row.  Column g of a score tile is
//     cell perm(g) = g / 2 + 4 (g & 1) of its eight: the 16-byte reads of eight lanes
//     then fall in eight different bank groups of the swizzled page.
//   * The K scale, sm_scale and log2 e multiply the score column in FP32, the row's
//     power of two enters with the exponent's multiply-add.
//   * P = p * v_scale * 2^f in FP16, f per row such that the row's largest |p *
//     v_scale| so far is 2^7 to 2^15: P keeps FP16's 11 bits however scores and V
//     scales lie, and what is below 2^-32 of the largest vanishes (2^20 such cells
//     weigh 2^-12).  The running maximum moves only when a score passes it by 7 in
//     log2; O follows it and f.  V goes from the INT8 page to the B operands by
//     ldmatrix.trans on byte pairs.
#include <cuda.h>

#include <atomic>

#include "serve.cuh"
#include "tc_ptx.cuh"

namespace qsa {
namespace {

constexpr int kWarps = 4;                          // consumer warps
constexpr int kThreads = 32 * (kWarps + 1);        // and one producer
constexpr int kRowsTile = 16;                      // rows of a tile (query heads of one KV head)
constexpr int kPageBytes = kPage * kHeadDim;       // one KV head's page of K or V
constexpr int kScaleBytes = kPage * 2;
constexpr int kStageBytes = 2 * kPageBytes + 2 * kScaleBytes;
constexpr int kMaxStages = 8;
constexpr int kMaxCtas = 320;                      // two per SM of 152, with room
constexpr int kMinPages = 4;                       // pages of a run at least: one per consumer warp
constexpr float kLazy = 7.f;
constexpr int kPBits = 7;                          // a row's largest |p v_scale| becomes 2^7 to 2^8 (2^15 at most) in P
constexpr uint64_t kWaitNs = 1000000000ull;

// Workspace: a record per CTA for the join, then two partial results per CTA (0: the
// item its run begins inside, 1: the item its run ends inside).
struct Rec {
    int item, last;      // the item cut at this run's end and the last CTA that holds a part of it; item < 0: none
    int seq, hk;
};
struct Part {
    float o[kRowsTile][kHeadDim];
    float m[kRowsTile], l[kRowsTile];
};

struct Ws {
    Rec* rec;
    Part* part;
};
__host__ __device__ __forceinline__ Ws workspace_of(uint8_t* p) {
    return Ws{reinterpret_cast<Rec*>(p), reinterpret_cast<Part*>(p + kMaxCtas * sizeof(Rec))};
}

// ---------------------------------------------------------------- small device helpers
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float lds_half(uint32_t addr) {
    uint16_t b;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b) : "r"(addr) : "memory");
    return __half2float(__ushort_as_half(b));
}
// Largest over the four lanes that share rows g and g + 8.
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// INT8 bytes (0, 2) and (1, 3) of a word as FP16 pairs, exactly (as int8x4_to_f16).
__device__ __forceinline__ void int8x4_to_f16_even_odd(uint32_t w, uint32_t& out02, uint32_t& out13) {
    const uint32_t u = w ^ 0x80808080u;
    out02 = f16x2_sub(__byte_perm(u, 0x64646464u, 0x4240), 0x64806480u);
    out13 = f16x2_sub(__byte_perm(u, 0x64646464u, 0x4341), 0x64806480u);
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// One KV head's page (64 rows of 128 bytes) into a 1,024-byte aligned buffer, 16-byte
// pieces XOR-swizzled by (row & 7).  x = 0; row is a multiple of 64 inside the pool.
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(0), "r"(row), "r"(bar) : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

// Four consecutive elements of the output.
__device__ __forceinline__ void store4(void* out, int type, size_t at, float a, float b, float c, float d) {
    if (type == QSA_F32) *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(a, b, c, d);
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(pack2(a, b, type), pack2(c, d, type));
}
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}
// Weight of a partial state with running maximum m (log2) and sum l in a merge around
// M.  m = -inf: nothing was summed (l = 0), or only NaN (l = NaN, which must show).
__device__ __forceinline__ float merge_weight(float m, float l, float M) {
    return m == -INFINITY ? l : fast_exp2(m - M);
}

// ---------------------------------------------------------------- the runs of pages
// The pages of one sequence: first page, count, and the cells' limits.
struct Seq {
    int n, first;    // cells first .. n-1
    int p0, np;      // pages p0 .. p0 + np - 1
};
__device__ __forceinline__ Seq seq_of(const PagedArgs& a, int s, bool tell) {
    int n = __ldg(a.seq_lens + s);
    const int cap = a.n_lpages * kPage;
    if (n < 0 || n > cap) {
        if (tell) report(a.dev_status, QSA_DEV_BAD_SEQ_LEN);
        n = n < 0 ? 0 : cap;
    }
    Seq q;
    q.n = n;
    q.first = a.window > 0 && a.window < n ? n - a.window : 0;
    q.p0 = q.first / kPage;
    q.np = (n + kPage - 1) / kPage - q.p0;
    return q;
}

// A place in the laid-out pages: sequence, item within it, page within the item.
struct Walk {
    int s, hk, off;
    Seq q;
    __device__ __forceinline__ void next_item(const PagedArgs& a, int n_hk) {
        off = 0;
        if (++hk < n_hk) return;
        hk = 0;
        do {
            ++s;
            if (s >= a.n_seq) return;   // behind the last page: the caller stops by its page count
            q = seq_of(a, s, false);
        } while (q.np == 0);
    }
};

struct Ctx {
    uint32_t ring, scales, full, empty;   // shared-memory addresses
    uint32_t* resident;                   // per stage: the page is there
    float* merge;                         // [kWarps][rows][128], 16-float pieces swapped in odd rows
    float* merge_m;                       // [kWarps][16] running maxima, then sums
    volatile int* abort_flag;
    int stages, rows;                     // rows: rows of the widest tile
    int begin, end, chunk;                // this CTA's pages
    int n_hk, tiles, group;
};

// ---------------------------------------------------------------- producer warp
__device__ __noinline__ void produce(const PagedArgs& a, const Ctx& c, Walk w, const CUtensorMap* kmap,
                                     const CUtensorMap* vmap) {
    const int lane = threadIdx.x & 31;
    int st = 0, uses = 0;                 // stage, times round the ring
    bool ok = true;
    for (int pos = c.begin; pos < c.end && ok;) {
        const int n = min(w.q.np - w.off, c.end - pos), h = w.hk / c.tiles;
        const int32_t* table = a.page_tables + (size_t)w.s * a.pt_stride + w.q.p0 + w.off;
        for (int i0 = 0; i0 < n && ok; i0 += 32) {
            int entry = -1;
            if (i0 + lane < n) {
                entry = __ldg(table + i0 + lane);
                if (entry >= a.n_ppages) {
                    report(a.dev_status, QSA_DEV_BAD_PAGE);
                    entry = -1;
                }
            }
            for (int i = i0; i < min(n, i0 + 32); ++i) {
                const int page = __shfl_sync(0xffffffffu, entry, i - i0);
                const uint32_t full = c.full + 8 * st;
                if (uses > 0) {
                    ok = tc::mbar_wait(c.empty + 8 * st, (uint32_t)(uses - 1) & 1u, c.abort_flag, kWaitNs);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                if (lane == 0) {
                    c.resident[st] = page >= 0;
                    if (page >= 0) {
                        const long long block = (long long)page * a.n_kv + h;
                        const uint32_t dst = c.ring + st * 2 * kPageBytes, sdst = c.scales + st * 2 * kScaleBytes;
                        mbar_expect_tx(full, kStageBytes);
                        tma_page(dst, kmap, (int)(block * kPage), full);
                        bulk_copy(sdst, a.k_scale + block * kPage, kScaleBytes, full);
                        tma_page(dst + kPageBytes, vmap, (int)(block * kPage), full);
                        bulk_copy(sdst + kScaleBytes, a.v_scale + block * kPage, kScaleBytes, full);
                    } else {
                        tc::mbar_arrive(full);
                    }
                }
                __syncwarp();
                if (++st == c.stages) {
                    st = 0;
                    ++uses;
                }
            }
        }
        pos += n;
        w.next_item(a, c.n_hk);
    }
    if (!ok) {                            // gave up: wait for the copies in flight before the CTA may leave
        if (lane == 0) report(a.dev_status, QSA_DEV_WAIT_TIMEOUT);
        for (int k = 0; k < c.stages; ++k) {
            // stage k was filled uses + (k < st) times; its last fill has parity (fills - 1) & 1
            const int fills = uses + (k < st);
            if (fills > 0) tc::mbar_wait_drain(c.full + 8 * k, (uint32_t)(fills - 1) & 1u, kWaitNs);
        }
    }
    // rows of the sequences that have no page at all
    for (int s = blockIdx.x; s < a.n_seq; s += gridDim.x) {
        if (seq_of(a, s, false).np > 0) continue;
        const size_t row = (size_t)s * a.n_heads;
        for (int e = lane; e < a.n_heads * (kHeadDim / 4); e += 32)
            store4(a.out, a.out_type, row * kHeadDim + 4 * e, 0.f, 0.f, 0.f, 0.f);
        if (a.lse)
            for (int e = lane; e < a.n_heads; e += 32) a.lse[row + e] = -INFINITY;
    }
}

// ---------------------------------------------------------------- consumer warps
// Running state of one warp over the pages of one item: rows g and g + 8 of lane
// (g, t) = (lane / 4, lane % 4).
struct State {
    float o[16][4];
    float m0, m1, l0, l1;                 // maxima in log2; l per lane, over the lane's own columns
    float top0, top1;                     // largest |p v_scale| when f was last set
    int f0, f1;                           // P and O carry 2^f
};

__device__ __forceinline__ void page_step(State& s, const uint32_t (&qa)[8][4], float rs0, float rs1, float kmul,
                                          uint32_t k_base, uint32_t sc_base, int lo, int hi, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int pg = (g >> 1) | ((g & 1) << 2);            // cell (of eight) of this lane's K column
    // ---- S = Q K^T
    float sc[8][4];
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
        const uint32_t row = k_base + (uint32_t)(8 * nt + pg) * kHeadDim;
        const uint4 w0 = lds128(row + (uint32_t)((t ^ pg) << 4)), w1 = lds128(row + (uint32_t)(((4 + t) ^ pg) << 4));
        const uint32_t kw[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
        sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            uint32_t b0, b1;
            int8x4_to_f16(kw[kk], b0, b1);
            mma_f16(sc[nt], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b0, b1);
        }
    }
    // ---- scales of the lane's columns: cells 8 nt + t and 8 nt + t + 4 of columns 2t, 2t + 1
    const bool whole = lo == 0 && hi == kPage;           // warp-uniform
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
        float ks[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) ks[e] = lds_half(sc_base + 2 * (8 * nt + t + 4 * e)) * kmul;
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt][e] *= ks[e & 1];
        if (!whole) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c = 8 * nt + t + 4 * e;
                if (c < lo || c >= hi) sc[nt][e] = sc[nt][e + 2] = -INFINITY;
            }
        }
        mx0 = fmax3(mx0, sc[nt][0], sc[nt][1]);
        mx1 = fmax3(mx1, sc[nt][2], sc[nt][3]);
    }
    // ---- running maxima (lazily moved)
    mx0 *= rs0;
    mx1 *= rs1;
    float al0 = 1.f, al1 = 1.f;
    const bool moved = __any_sync(0xffffffffu, mx0 > s.m0 + kLazy || mx1 > s.m1 + kLazy);
    if (moved) {
        mx0 = quad_max(mx0);
        mx1 = quad_max(mx1);
        if (mx0 > s.m0 + kLazy) {                        // from -inf: O and l are zero, the factor does not matter
            al0 = s.m0 == -INFINITY ? 1.f : fast_exp2(s.m0 - mx0);
            s.m0 = mx0;
        }
        if (mx1 > s.m1 + kLazy) {
            al1 = s.m1 == -INFINITY ? 1.f : fast_exp2(s.m1 - mx1);
            s.m1 = mx1;
        }
    }
    // ---- p, the row sums, and p * v_scale in place of the scores
    const float mu0 = s.m0 == -INFINITY ? 0.f : s.m0, mu1 = s.m1 == -INFINITY ? 0.f : s.m1;
    float ps0 = 0.f, ps1 = 0.f, pm0 = 0.f, pm1 = 0.f;
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
        float vs[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int c = 8 * nt + t + 4 * e;
            vs[e] = lds_half(sc_base + kScaleBytes + 2 * c);
            if (!whole && (c < lo || c >= hi)) vs[e] = 0.f;   // its scale may be anything
        }
        const float e0 = fast_exp2(fmaf(sc[nt][0], rs0, -mu0)), e1 = fast_exp2(fmaf(sc[nt][1], rs0, -mu0));
        const float e2 = fast_exp2(fmaf(sc[nt][2], rs1, -mu1)), e3 = fast_exp2(fmaf(sc[nt][3], rs1, -mu1));
        ps0 += e0 + e1;
        ps1 += e2 + e3;
        sc[nt][0] = e0 * vs[0];
        sc[nt][1] = e1 * vs[1];
        sc[nt][2] = e2 * vs[0];
        sc[nt][3] = e3 * vs[1];
        pm0 = fmax3(pm0, fabsf(sc[nt][0]), fabsf(sc[nt][1]));
        pm1 = fmax3(pm1, fabsf(sc[nt][2]), fabsf(sc[nt][3]));
    }
    s.l0 = s.l0 * al0 + ps0;
    s.l1 = s.l1 * al1 + ps1;
    // ---- the rows' powers of two for P: moved when P would pass 2^15, or when the maximum moved
    if (__any_sync(0xffffffffu, moved || pm0 * exp2i(s.f0) > 32768.f || pm1 * exp2i(s.f1) > 32768.f)) {
        s.top0 = fmaxf(s.top0 * al0, quad_max(pm0));
        s.top1 = fmaxf(s.top1 * al1, quad_max(pm1));
        const int n0 = s.top0 > 0.f ? kPBits - min(max(f32_exponent(s.top0), -100), 24) : s.f0;
        const int n1 = s.top1 > 0.f ? kPBits - min(max(f32_exponent(s.top1), -100), 24) : s.f1;
        al0 *= exp2i(n0 - s.f0);
        al1 *= exp2i(n1 - s.f1);
        s.f0 = n0;
        s.f1 = n1;
#pragma unroll
        for (int d = 0; d < 16; ++d) {
            s.o[d][0] *= al0;
            s.o[d][1] *= al0;
            s.o[d][2] *= al1;
            s.o[d][3] *= al1;
        }
    }
    const float f0 = exp2i(s.f0), f1 = exp2i(s.f1);
    // ---- O += P V, 16 cells at a time
    const int vr = lane & 7;
    const int vcell = ((vr >> 1) | ((vr & 1) << 2)) + 8 * ((lane >> 3) & 1);
    const uint32_t v_base = k_base + kPageBytes + (uint32_t)vcell * kHeadDim;
#pragma unroll
    for (int ks16 = 0; ks16 < 4; ++ks16) {
        uint32_t af[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float* p = sc[2 * ks16 + j];
            af[2 * j] = pack_f16x2(p[0] * f0, p[1] * f0);
            af[2 * j + 1] = pack_f16x2(p[2] * f1, p[3] * f1);
        }
        // byte pairs by ldmatrix.trans: of the 32 dims 32q .. 32q + 31, lane (g, t) gets, of cells
        // perm(2t), perm(2t + 1) (and those + 8), dims 32q + 2g, + 1 and 32q + 16 + 2g, + 1.  O tile
        // 4q + 2h + e holds dims 32q + 16h + 2n + e at column n.
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t r[4];
            ldsm_x4_t(v_base + ks16 * 16 * kHeadDim + (uint32_t)(((2 * q + (lane >> 4)) ^ (vcell & 7)) << 4), r[0], r[1], r[2],
                      r[3]);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                uint32_t e0, d0, e1, d1;
                int8x4_to_f16_even_odd(r[2 * hh], e0, d0);
                int8x4_to_f16_even_odd(r[2 * hh + 1], e1, d1);
                mma_f16(s.o[4 * q + 2 * hh], af[0], af[1], af[2], af[3], e0, e1);
                mma_f16(s.o[4 * q + 2 * hh + 1], af[0], af[1], af[2], af[3], d0, d1);
            }
        }
    }
}

// The tile's query rows g and g + 8 as FP16 A operands, each row times a power of two
// 2^-e that puts its largest element in [2^12, 2^13); rs = 2^e.
__device__ __forceinline__ void load_q(const PagedArgs& a, size_t row0, int rows, int lane, uint32_t (&qa)[8][4], float& rs0,
                                       float& rs1) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int r = g + 8 * half;
        uint4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {     // dims 64 (j / 2) + 16 t + 8 (j & 1) .. + 7
            w[j] = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows)
                w[j] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (row0 + r) * kHeadDim +
                                                            64 * (j >> 1) + 16 * t + 8 * (j & 1)));
        }
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x[8];
            unpack8(w[j], a.q_type, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = amax > 0.f ? min(max(f32_exponent(amax) - 12, -114), 114) : 0;
        const float down = exp2i(-e);
        (half ? rs1 : rs0) = exp2i(e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x[8];
            unpack8(w[j], a.q_type, x);
#pragma unroll
            for (int k = 0; k < 2; ++k) {   // k step 4 (j / 2) + 2 (j & 1) + k: four dims
                const int kk = 4 * (j >> 1) + 2 * (j & 1) + k;
                qa[kk][half] = pack_f16x2(x[4 * k] * down, x[4 * k + 1] * down);
                qa[kk][2 + half] = pack_f16x2(x[4 * k + 2] * down, x[4 * k + 3] * down);
            }
        }
    }
}

__device__ __forceinline__ void consume(const PagedArgs& a, const Ctx& c, Walk w) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const Ws ws = workspace_of(a.workspace);
    const float kmul = a.sm_scale * kLog2e;
    int next = c.begin + warp;            // this warp's next page
    int st = warp, uses = 0;              // its stage (warp < stages) and the times round the ring
    bool dead = false;                    // a wait ran out: go through the motions, so that no barrier is left waiting
    for (int pos = c.begin; pos < c.end; w.next_item(a, c.n_hk)) {
        const int n = min(w.q.np - w.off, c.end - pos);
        const int h = w.hk / c.tiles, tile = w.hk - h * c.tiles;
        const int rows = min(kRowsTile, c.group - kRowsTile * tile);
        const size_t row0 = (size_t)w.s * a.n_heads + h * c.group + kRowsTile * tile;
        const bool complete = w.off == 0 && n == w.q.np;
        const int seg_end = pos + n;
        const bool mine = next < seg_end;
        State s;
        float rs0 = 1.f, rs1 = 1.f;
#pragma unroll
        for (int d = 0; d < 16; ++d) s.o[d][0] = s.o[d][1] = s.o[d][2] = s.o[d][3] = 0.f;
        s.m0 = s.m1 = -INFINITY;
        s.l0 = s.l1 = 0.f;
        s.top0 = s.top1 = 0.f;
        s.f0 = s.f1 = 0;
        if (mine) {
            uint32_t qa[8][4];
            load_q(a, row0, rows, lane, qa, rs0, rs1);
#pragma unroll 1
            for (; next < seg_end; next += kWarps) {
                if (!dead) {
                    const bool ok = tc::mbar_wait(c.full + 8 * st, (uint32_t)uses & 1u, c.abort_flag, kWaitNs);
                    dead = __any_sync(0xffffffffu, !ok);
                    if (dead && lane == 0) report(a.dev_status, QSA_DEV_WAIT_TIMEOUT);
                }
                if (!dead) {
                    if (c.resident[st]) {
                        const int cell0 = (w.q.p0 + w.off + (next - pos)) * kPage;
                        page_step(s, qa, rs0, rs1, kmul, c.ring + st * 2 * kPageBytes, c.scales + st * 2 * kScaleBytes,
                                  max(w.q.first - cell0, 0), min(w.q.n - cell0, kPage), lane);
                    }
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(c.empty + 8 * st);
                }
                st += kWarps;
                if (st >= c.stages) {     // kWarps <= stages
                    st -= c.stages;
                    ++uses;
                }
            }
            s.l0 += __shfl_xor_sync(0xffffffffu, s.l0, 1);
            s.l0 += __shfl_xor_sync(0xffffffffu, s.l0, 2);
            s.l1 += __shfl_xor_sync(0xffffffffu, s.l1, 1);
            s.l1 += __shfl_xor_sync(0xffffffffu, s.l1, 2);
            const float back0 = exp2i(-s.f0), back1 = exp2i(-s.f1);
#pragma unroll
            for (int d = 0; d < 16; ++d) {
                s.o[d][0] *= back0;
                s.o[d][1] *= back0;
                s.o[d][2] *= back1;
                s.o[d][3] *= back1;
            }
        }
        Part* part = ws.part + 2 * blockIdx.x + (w.off == 0 ? 1 : 0);
        if (n == 1) {
            // one page, one warp: straight from the registers
            if (mine) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int r = g + 8 * half;
                    if (r >= rows) continue;
                    const float l = half ? s.l1 : s.l0, m = half ? s.m1 : s.m0;
                    const float inv = complete ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const int d = 16 * q + 4 * t, e = 2 * q, v = 2 * half;
                        const float x0 = s.o[e][v] * inv, x1 = s.o[e + 1][v] * inv, x2 = s.o[e][v + 1] * inv,
                                    x3 = s.o[e + 1][v + 1] * inv;
                        if (complete) store4(a.out, a.out_type, (row0 + r) * kHeadDim + d, x0, x1, x2, x3);
                        else *reinterpret_cast<float4*>(&part->o[r][d]) = make_float4(x0, x1, x2, x3);
                    }
                    if (t == 0) {
                        if (!complete) {
                            part->m[r] = m;
                            part->l[r] = l;
                        } else if (a.lse) {
                            a.lse[row0 + r] = lse_of(m, l);
                        }
                    }
                }
            }
        } else {
            // merge the warps that had pages: (pos - begin) % kWarps is the first of them
            consumers_sync();             // the last merge has been read
            if (mine) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int r = g + 8 * half;
                    if (r < rows) {
                        float* dst = c.merge + ((size_t)warp * c.rows + r) * kHeadDim;
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const int d = (16 * q + 4 * t) ^ ((r & 1) << 4), e = 2 * q, v = 2 * half;
                            *reinterpret_cast<float4*>(dst + d) =
                                make_float4(s.o[e][v], s.o[e + 1][v], s.o[e][v + 1], s.o[e + 1][v + 1]);
                        }
                        if (t == 0) {
                            c.merge_m[warp * kRowsTile + r] = half ? s.m1 : s.m0;
                            c.merge_m[(kWarps + warp) * kRowsTile + r] = half ? s.l1 : s.l0;
                        }
                    }
                }
            }
            consumers_sync();
            const int lead = (pos - c.begin) % kWarps;
            for (int r = warp; r < rows; r += kWarps) {
                float m[kWarps], l[kWarps], M = -INFINITY;
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    const bool had = ((k - lead + kWarps) % kWarps) < n;
                    m[k] = had ? c.merge_m[k * kRowsTile + r] : -INFINITY;
                    l[k] = had ? c.merge_m[(kWarps + k) * kRowsTile + r] : 0.f;
                    M = fmaxf(M, m[k]);
                }
                float L = 0.f, x0 = 0.f, x1 = 0.f, x2 = 0.f, x3 = 0.f;
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    if (((k - lead + kWarps) % kWarps) >= n) continue;
                    const float wt = merge_weight(m[k], l[k], M);
                    const float4 o = *reinterpret_cast<const float4*>(c.merge + ((size_t)k * c.rows + r) * kHeadDim +
                                                                      ((4 * lane) ^ ((r & 1) << 4)));
                    L += wt * l[k];
                    x0 += wt * o.x;
                    x1 += wt * o.y;
                    x2 += wt * o.z;
                    x3 += wt * o.w;
                }
                if (complete) {
                    const float inv = L == 0.f ? 0.f : 1.f / L;
                    store4(a.out, a.out_type, (row0 + r) * kHeadDim + 4 * lane, x0 * inv, x1 * inv, x2 * inv, x3 * inv);
                    if (lane == 0 && a.lse) a.lse[row0 + r] = lse_of(M, L);
                } else {
                    *reinterpret_cast<float4*>(&part->o[r][4 * lane]) = make_float4(x0, x1, x2, x3);
                    if (lane == 0) {
                        part->m[r] = M;
                        part->l[r] = L;
                    }
                }
            }
        }
        if (threadIdx.x == 0 && seg_end == c.end) {
            // the run's last item: cut here, and begun here, if pages of it are left
            Rec rec{-1, 0, w.s, w.hk};
            if (w.off == 0 && n < w.q.np) {
                rec.item = 0;
                rec.last = (pos + w.q.np - 1) / c.chunk;
            }
            ws.rec[blockIdx.x] = rec;
        }
        pos = seg_end;
    }
}

// Sum over the block of each thread's count and the sum before this thread.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int& before) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int total = 0;
    before = inc - v;
#pragma unroll
    for (int k = 0; k <= kWarps; ++k) {
        if (k < warp) before += s_warp[k];
        total += s_warp[k];
    }
    return total;
}

__global__ void __launch_bounds__(kThreads, 2)
paged_attn_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  int stages, int rows) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_bars[2 * kMaxStages];
    __shared__ uint32_t s_resident[kMaxStages];
    __shared__ float s_ml[2 * kWarps * kRowsTile];
    __shared__ int s_warp[kWarps + 1], s_abort, s_start[3];
    const int tid = threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;");   // the join may be set up now; it waits for this grid's end

    Ctx c;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    c.ring = base;
    c.scales = base + stages * 2 * kPageBytes;
    c.merge = reinterpret_cast<float*>(smem_raw + (base - raw) + stages * kStageBytes);
    c.merge_m = s_ml;
    c.full = smem_u32(s_bars);
    c.empty = c.full + 8 * kMaxStages;
    c.resident = s_resident;
    c.abort_flag = &s_abort;
    c.stages = stages;
    c.rows = rows;
    c.group = a.n_heads / a.n_kv;
    c.tiles = (c.group + kRowsTile - 1) / kRowsTile;
    c.n_hk = a.n_kv * c.tiles;
    if (tid == 0) {
        for (int k = 0; k < stages; ++k) {
            tc::mbar_init(c.full + 8 * k, 1);
            tc::mbar_init(c.empty + 8 * k, 1);
        }
        s_abort = 0;
        tc::fence_mbar_init();
    }

    // ---- this CTA's run of the pages of all items
    const int per = (a.n_seq + kThreads - 1) / kThreads;   // consecutive sequences per thread
    const int s_lo = min(tid * per, a.n_seq), s_hi = min(s_lo + per, a.n_seq);
    int sum = 0, before;
    for (int s = s_lo; s < s_hi; ++s) sum += seq_of(a, s, blockIdx.x == 0).np;
    const int total = block_scan(sum, s_warp, before) * c.n_hk;   // at most 2^30, checked on the host
    c.chunk = max((total + (int)gridDim.x - 1) / (int)gridDim.x, kMinPages);
    c.begin = (int)min((long long)blockIdx.x * c.chunk, (long long)total);
    c.end = (int)min((long long)c.begin + c.chunk, (long long)total);
    if (c.begin < c.end && c.begin >= before * c.n_hk && c.begin < (before + sum) * c.n_hk) {
        int at = before, s = s_lo;                         // the one thread whose sequences hold the first page
        for (;; ++s) {
            const int np = seq_of(a, s, false).np;
            if (c.begin < (at + np) * c.n_hk) break;
            at += np;
        }
        s_start[0] = s;
        s_start[1] = c.begin - at * c.n_hk;
    }
    if (tid == 0 && c.begin >= c.end) workspace_of(a.workspace).rec[blockIdx.x] = Rec{-1, 0, 0, 0};
    __syncthreads();
    Walk w;
    w.s = w.hk = w.off = 0;
    w.q = Seq{0, 0, 0, 1};
    if (c.begin < c.end) {
        w.s = s_start[0];
        w.q = seq_of(a, w.s, false);
        w.hk = s_start[1] / w.q.np;
        w.off = s_start[1] - w.hk * w.q.np;
    }
    if (tid >= 32 * kWarps) produce(a, c, w, &kmap, &vmap);
    else consume(a, c, w);
}

// Joins the parts of the item that run blockIdx.x begins and others end: row
// blockIdx.y of it.  Warps take parts in turn, a lane four dims.
__global__ void __launch_bounds__(128) paged_join_kernel(const PagedArgs a) {
    __shared__ float s_o[4][kHeadDim], s_l[4];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Ws ws = workspace_of(a.workspace);
    const int c0 = blockIdx.x, r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Rec rec = ws.rec[c0];
    if (rec.item < 0) return;
    const int group = a.n_heads / a.n_kv, tiles = (group + kRowsTile - 1) / kRowsTile;
    const int h = rec.hk / tiles, tile = rec.hk - h * tiles;
    if (r >= min(kRowsTile, group - kRowsTile * tile)) return;
    const int n = rec.last - c0 + 1;      // part 0 is run c0's last item, part i the first of run c0 + i
    const Part* part = ws.part + 2 * c0;
    auto at = [&](int i) { return part + (i == 0 ? 1 : 2 * i); };
    float M = -INFINITY;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, at(i)->m[r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f, x0 = 0.f, x1 = 0.f, x2 = 0.f, x3 = 0.f;
#pragma unroll 4
    for (int i = warp; i < n; i += 4) {
        const Part* p = at(i);
        const float l = p->l[r], wt = merge_weight(p->m[r], l, M);
        const float4 o = *reinterpret_cast<const float4*>(&p->o[r][4 * lane]);
        L += wt * l;
        x0 += wt * o.x;
        x1 += wt * o.y;
        x2 += wt * o.z;
        x3 += wt * o.w;
    }
    *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = make_float4(x0, x1, x2, x3);
    if (lane == 0) s_l[warp] = L;
    __syncthreads();
    if (warp != 0) return;
    L = s_l[0] + s_l[1] + s_l[2] + s_l[3];
    const float inv = L == 0.f ? 0.f : 1.f / L;
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        x[e] = (s_o[0][4 * lane + e] + s_o[1][4 * lane + e] + s_o[2][4 * lane + e] + s_o[3][4 * lane + e]) * inv;
    const size_t row = (size_t)rec.seq * a.n_heads + h * group + kRowsTile * tile + r;
    store4(a.out, a.out_type, row * kHeadDim + 4 * lane, x[0], x[1], x[2], x[3]);
    if (lane == 0 && a.lse) a.lse[row] = lse_of(M, L);
}

// ---------------------------------------------------------------- host side
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder (a host function without state), looked up once.
EncodeTiled encoder() {
    static std::atomic<void*> found{nullptr};
    void* p = found.load(std::memory_order_acquire);
    if (!p) {
        cudaDriverEntryPointQueryResult st;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &st) != cudaSuccess ||
            st != cudaDriverEntryPointSuccess)
            return nullptr;
        found.store(p, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(p);
}

bool page_map(CUtensorMap* map, const int8_t* pool, long long rows) {
    const EncodeTiled encode = encoder();
    if (!encode) return false;
    const cuuint64_t dims[2] = {kHeadDim, (cuuint64_t)rows}, strides[1] = {kHeadDim};
    const cuuint32_t box[2] = {kHeadDim, kPage}, steps[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(pool), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t paged_attn_workspace(int, int) { return kMaxCtas * (sizeof(Rec) + 2 * sizeof(Part)); }

cudaError_t launch_paged_attn(const PagedArgs& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    CUtensorMap kmap{}, vmap{};
    if (a.n_ppages > 0) {                 // an empty pool: every page is masked and no copy is made
        const long long rows = (long long)a.n_ppages * a.n_kv * kPage;
        if (!page_map(&kmap, a.k_pool, rows) || !page_map(&vmap, a.v_pool, rows)) return cudaErrorInvalidValue;
    }
    // two CTAs share an SM's shared memory: 113 KB each, the merge's rows first, the ring from the rest
    const int rows = a.n_heads / a.n_kv < kRowsTile ? a.n_heads / a.n_kv : kRowsTile;
    const int merge = kWarps * rows * kHeadDim * 4;
    int stages = (112 * 1024 - 3072 - merge) / kStageBytes;
    stages = stages > kMaxStages ? kMaxStages : stages;
    const int smem = 1024 + stages * kStageBytes + merge;
    e = cudaFuncSetAttribute(paged_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int grid = 2 * sms < kMaxCtas ? 2 * sms : kMaxCtas;
    paged_attn_kernel<<<grid, kThreads, smem, stream>>>(a, kmap, vmap, stages, rows);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid, (unsigned)rows);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_join_kernel, a);
}

}  // namespace qsa

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
// are cut into equal runs (an item's start counts as a page), one per warp of a grid of two
// CTAs per SM: ragged batches, one long sequence and many short ones all give every SM as
// much to do, and a warp keeps an item's running softmax to itself, so that short items
// (most of a chat batch) need no merge at all.  The CTA sums the page counts itself
// (the lengths are device data; no host value is needed, so a captured graph follows
// the lengths).  An item cut between warps leaves parts (max, sum, O): those of one CTA
// are merged once, when its run is done, in the shared memory its copies have left;
// what is cut between CTAs goes to the workspace, at most two parts a CTA, and
// paged_join_kernel, launched beside this kernel and waiting for it on the device,
// joins them in the order of the CTAs.
//
// Few and short items (a small batch of short conversations) take paged_small_kernel
// instead: a cluster of eight CTAs per item, whose parts are merged through distributed
// shared memory; one launch, no sum over the lengths, no workspace.
//
// A warp has a ring of two 32-cell steps (4 KB of K, 4 KB of V, two 64-byte rows of
// scales), filled by 16-byte asynchronous copies, 512 consecutive bytes an instruction,
// 16-byte pieces XOR-swizzled by (row & 7) as they land (a bulk copy would leave every
// row on the same banks, eightfold conflicts for V).  It computes on one step while the
// other is in flight and refills it when it is used: 67 to 133 KB per SM are on the way
// at any time (a third step measured 1 to 3 % slower).  A page's table entry is looked
// up a page ahead, an item's queries an item ahead.
//
// Measured (12 heads to a KV head, BF16, calls in a row): 96 sequences of 16,000 to
// 20,000 cells, 4 KV heads, 1.81 GB: 271 us, 6.69 TB/s, the rate of a plain copy; one of
// 262,149, 8 KV heads, 545 MB: 90 us, 6.05 TB/s; 64 of 1 to 8,192, 4 KV heads, 316 MB:
// 60.6 us, 5.2 TB/s.  Beside the bytes there are 2 us until the lengths are summed, 3 until the
// first rows are there, 4 to 8 in which some runs are over and others not (they hold as
// many bytes, DRAM does not serve them alike; next pages prefetched into L2 made it 1 to 2
// % slower), 1 to 3 for the merge and 3 for the join.
//
// The tensor work is mma.sync m16n8k16: 16 rows per tile (12 query heads) would fill an
// eighth of a tcgen05.mma's 128 rows, whose operands would also have to be written back
// to shared memory in 16 bits, twice the traffic of the INT8 rows; here they are
// converted in registers, exactly.
//   * S = Q K^T on FP16 operands.  Q is scaled per row by a power of two (its
//     largest element in [2^12, 2^13)) and held in registers.  K enters as K + 128, an
//     unsigned byte in the low bits of an FP16 word, which is the subnormal (K + 128) *
//     2^-24: three instructions for four values; the accumulators start at -128 sum(Q).
//     Within each 64-dim half the dims are permuted (Q and K alike) so that a lane's K
//     operands of four k steps are one 16-byte piece of the INT8 row.  Column g of a
//     score tile is cell perm(g) = g / 2 + 4 (g & 1) of its eight: the 16-byte reads of
//     eight lanes then fall in eight different bank groups of the swizzled rows.
//   * The K scale, sm_scale and log2 e multiply the score column in FP32, the row's
//     power of two enters with the exponent's multiply-add: p = 2^(score - R).
//   * The row's reference R is not the running maximum of the scores but that of
//     score + log2 |v_scale|, less 7 to 15: the product p * v_scale, which enters O += P V
//     in FP16, then is at most 2^15 and its largest so far at least 2^7, so P keeps
//     FP16's 11 bits however scores and V scales lie, and what is below 2^-32 of the
//     largest product vanishes (2^20 such cells weigh 2^-12).  Where cells without values (V
//     scales of zero, or close to it) take nearly all of the weight, R stays 64 below their
//     scores: p is FP32, and products down to 2^-78 of the largest weight are normal in FP16.
//     R moves, and O and the row sum with it, only when a product would pass 2^15 (or the
//     sum 2^76): one vote a step.  V goes from the INT8 rows to the B operands by
//     ldmatrix.trans on byte pairs.
#include <cooperative_groups.h>

#include "serve.cuh"

namespace qsa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRowsTile = 16;                      // rows of a tile (query heads of one KV head)
constexpr int kStep = 32;                          // cells of a step
constexpr int kDepth = 2;                          // steps of a warp's ring
constexpr int kStepBytes = kStep * kHeadDim;       // of K, and of V
constexpr int kStepScales = kStep * 2;             // bytes of K scales, and of V scales
constexpr int kWarpBytes = kDepth * 2 * (kStepBytes + kStepScales);
constexpr int kRings = kWarps * kWarpBytes;
constexpr int kMaxCtas = 320;                      // two per SM of 152, with room
constexpr int kPBits = 7;                          // a row's largest |p v_scale| is set to 2^7 .. 2^8 when R moves
constexpr int kPMost = 64;                         // and no weight p above 2^64 then, whatever its v_scale is
// A run's 2^21 steps at most (2^30 pages over the warps) then sum to 2^99; what a change of reference or a merge flushes
// (factors below 2^-126) is below 2^-27, beside sums of 2^-9 or more.
constexpr float kPTop = 32768.f, kSumTop = 0x1p76f;

// A part of an item's result: rows relative to their reference m (log2).  The
// 16-float pieces of odd rows are swapped in pairs (see col()).
struct Part {
    float o[kRowsTile][kHeadDim];
    float m[kRowsTile], l[kRowsTile];
};
__device__ __forceinline__ int col(int r, int d) { return d ^ ((r & 1) << 4); }
static_assert(sizeof(Part) <= kDepth * 2 * kStepBytes, "a part fits a warp's ring");
// Shared memory: the warps' rings, then for each warp the part of an item that its run
// begins inside and ends.  What a run ends with lies in its ring.
constexpr int kSmem = kRings + kWarps * (int)sizeof(Part);

// Workspace, per CTA: a record for the join, and two parts (0: of the item its run
// begins inside, 1: of the item its run ends inside).
struct Rec {
    int last;            // last CTA with a part of the item that this CTA begins and does not end; < 0: there is none
    int seq, hk, pad;
};
struct CtaSpace {
    Part cta[2];
};
struct Ws {
    Rec* rec;
    CtaSpace* cta;
};
__host__ __device__ __forceinline__ Ws workspace_of(uint8_t* p) {
    return Ws{reinterpret_cast<Rec*>(p), reinterpret_cast<CtaSpace*>(p + kMaxCtas * sizeof(Rec))};
}

// ---------------------------------------------------------------- small device helpers
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(addr) : "memory");
}
// Largest over the four lanes that share rows g and g + 8.
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// INT8 bytes of a word plus 128, as FP16 pairs (bytes 0, 2) and (1, 3), times 2^-24:
// an integer in FP16's low bits is a subnormal of just that value, exact to the tensor
// core, and takes no conversion.
__device__ __forceinline__ void biased_pairs(uint32_t w, uint32_t& out02, uint32_t& out13) {
    const uint32_t u = w ^ 0x80808080u;
    out02 = u & 0x00FF00FFu;
    out13 = __byte_perm(u, 0u, 0x4341);
}
// INT8 bytes (0, 2) and (1, 3) of a word as FP16 pairs, exactly (as int8x4_to_f16).
__device__ __forceinline__ void int8x4_to_f16_even_odd(uint32_t w, uint32_t& out02, uint32_t& out13) {
    const uint32_t u = w ^ 0x80808080u;
    out02 = f16x2_sub(__byte_perm(u, 0x64646464u, 0x4240), 0x64806480u);
    out13 = f16x2_sub(__byte_perm(u, 0x64646464u, 0x4341), 0x64806480u);
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Four consecutive elements of the output.
__device__ __forceinline__ void store4(void* out, int type, size_t at, float a, float b, float c, float d) {
    if (type == QSA_F32) *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(a, b, c, d);
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(pack2(a, b, type), pack2(c, d, type));
}
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}
// Weight of a partial state with reference m (log2) and sum l in a merge around M.
// m = -inf: nothing was summed (l = 0), or only NaN (l = NaN, which must show).
__device__ __forceinline__ float merge_weight(float m, float l, float M) {
    return m == -INFINITY ? l : fast_exp2(m - M);
}

// ---------------------------------------------------------------- the runs of pages
// The pages of one sequence: first page, count, and the cells' limits.
struct Seq {
    int n, first;    // cells first .. n-1
    int p0, np;      // pages p0 .. p0 + np - 1
};
__device__ __forceinline__ Seq seq_from(const PagedArgs& a, int n, bool tell) {
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
__device__ __forceinline__ Seq seq_of(const PagedArgs& a, int s, bool tell) { return seq_from(a, a.seq_lens[s], tell); }

// Places are counted with kItemPlaces before every item's first page, which stand for the
// time that a warp takes from one item to the next (64 sequences of 1 to 8,192 cells 59.2
// us without, 55.7 with one, 55.4 with two; 512 of a 1,000-cell window 91.9, 89.0, 88.9;
// 64 of 4,096 cells 53.8, 53.6, 53.2).
constexpr int kItemPlaces = 1;
__device__ __forceinline__ int places(int np) { return np > 0 ? np + kItemPlaces : 0; }

// The runs: run i of `runs` begins at place total i / runs, so that any two differ by a
// place at most (a run may hold no page, but not inside an item); and the CTA whose runs
// hold a place.
__device__ __forceinline__ int run_begin(int total, int i, int runs) {
    i = min(i, runs);                     // total i / runs, in 32 bits: runs^2 < 2^31
    const int q = total / runs, r = total - q * runs;
    return q * i + r * i / runs;
}
__device__ __forceinline__ int cta_of(int total, int place, int runs) {
    return (int)((((long long)place + 1) * runs - 1) / total) / kWarps;
}
__device__ __forceinline__ int run_count(int total, int ctas) { return max(1, min(ctas * kWarps, total)); }

// Where a run begins: the sequence, the place among its items' places, the sequence's
// pages and the pages of one KV head's items before it.
struct Start {
    int s, place, np, pages;
};
// A page on the way: sequence, item within it, page within the item.
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
    // `pages` further; the place must exist.
    __device__ __forceinline__ void advance(const PagedArgs& a, int n_hk, int pages) {
        off += pages;
        while (off >= q.np) {
            const int rest = off - q.np;
            next_item(a, n_hk);
            if (s >= a.n_seq) return;
            off = rest;
        }
    }
};

struct Ctx {
    uint8_t* ring;                        // this warp's steps in shared memory, 2 * kStepBytes each
    Part* ended;                          // this warp's part of an item that ends inside its run
    uint8_t* scales;                      // and their scales, 2 * kStepScales each
    float* cols;                          // this warp's [2][32]: the step's K and V scales as the lanes need them
    int n;                                // this warp's pages
    int n_hk, tiles, group;
};

// ---------------------------------------------------------------- copies
// A warp's copies, step by step over its pages.  The table entry of the page after the
// current one is already on its way.
struct Fetch {
    Walk w;                               // on the page looked up last
    int idx, at;                          // that page's place in the run; where w stands
    int entry;
    bool second;                          // the next step is its page's second one
    uint32_t resident;                    // per slot: its step's page is there
    bool ok;                              // the current page is there
    int lo, hi;                           // its cells' limits, from the next step's first one
    const int8_t* ksrc;                   // the next step, for this lane
    const int8_t* vsrc;
    const uint16_t* ssrc;

    __device__ __forceinline__ void look(const PagedArgs& a, const Ctx& c, int page) {
        idx = page;
        if (idx >= c.n) return;
        w.advance(a, c.n_hk, idx - at);
        at = idx;
        entry = a.page_tables[(size_t)w.s * a.pt_stride + w.q.p0 + w.off];
    }
    // The next step into slot `slot` of the ring; one group, empty behind the run's end.
    __device__ __forceinline__ void put(const PagedArgs& a, const Ctx& c, int slot) {
        const int lane = threadIdx.x & 31;
        if (!second) {                    // a new page
            ok = idx < c.n && entry >= 0;
            if (ok && entry >= a.n_ppages) {
                if (lane == 0) report(a.dev_status, QSA_DEV_BAD_PAGE);
                ok = false;
            }
            if (ok) {
                const long long row = ((long long)entry * a.n_kv + (c.tiles == 1 ? w.hk : w.hk / c.tiles)) * kPage;
                ksrc = a.k_pool + row * kHeadDim + 16 * lane;
                vsrc = a.v_pool + row * kHeadDim + 16 * lane;
                ssrc = (lane < 4 ? a.k_scale : a.v_scale) + row + 8 * (lane & 3);
            }
            const int cell0 = (w.q.p0 + w.off) * kPage;
            lo = w.q.first - cell0;
            hi = w.q.n - cell0;
            if (idx < c.n) look(a, c, idx + 1);
        }
        second = !second;
        resident = ok ? resident | (1u << slot) : resident & ~(1u << slot);
        if (ok && hi > 0 && lo < kStep) {
            // lane l copies piece l & 7 of rows l / 8 + 4 j; for odd j, (row & 7) flips bit 2 of the piece
            const uint32_t dst = smem_u32(c.ring) + slot * 2 * kStepBytes + (uint32_t)(lane >> 3) * kHeadDim +
                                 (uint32_t)(((lane & 7) ^ (lane >> 3)) << 4);
            const uint32_t sdst = smem_u32(c.scales) + slot * 2 * kStepScales + 16 * lane;
            if (hi >= kStep) {
#pragma unroll
                for (int j = 0; j < kStep / 4; ++j) copy16((dst ^ ((j & 1) << 6)) + 512 * j, ksrc + 512 * j);
                if (lane < 8) copy16(sdst, ssrc);   // 64 bytes of K scales, 64 of V scales
#pragma unroll
                for (int j = 0; j < kStep / 4; ++j) copy16((dst ^ ((j & 1) << 6)) + kStepBytes + 512 * j, vsrc + 512 * j);
            } else {                      // the sequence's end: its rows only, four at a time
                if (lane < 8) copy16(sdst, ssrc);
                for (int j = 0; 4 * j < hi; ++j) {
                    copy16((dst ^ ((j & 1) << 6)) + 512 * j, ksrc + 512 * j);
                    copy16((dst ^ ((j & 1) << 6)) + kStepBytes + 512 * j, vsrc + 512 * j);
                }
            }
        }
        copies_commit();
        ksrc += kStepBytes;
        vsrc += kStepBytes;
        ssrc += kStep;
        lo -= kStep;
        hi -= kStep;
    }
};

// ---------------------------------------------------------------- a step
// Running state of one warp over the pages of one item: rows g and g + 8 of lane
// (g, t) = (lane / 4, lane % 4).
struct State {
    float o[16][4];
    float r0, r1;                         // references R (log2); -inf: nothing yet
    float l0, l1;                         // row sums, per lane, over the lane's own columns
};

// A tile's query rows g and g + 8 as FP16 A operands: each row times a power of two 2^-e
// that puts its largest element in [2^12, 2^13).  Within each 64-dim half the dims are
// permuted: k step 4 h + k holds dims 64 h + 16 t + 4 k + (0, 2 | 1, 3) of lane column t,
// in the order in which biased_pairs takes a word's bytes.
struct Query {
    uint32_t a[8][4];
    float rs0, rs1;                       // 2^e
    float bias0, bias1;                   // -128 * (sum of the row) * 2^-24
};

// p = 2^(score - R) of the lane's columns, with their sums, and p * v_scale in place.
__device__ __forceinline__ void weigh(const float (&sc)[4][4], float (&pv)[4][4], const float (&vs)[8], float rs0, float rs1,
                                      float r0, float r1, float& sum0, float& sum1, float& top0, float& top1) {
    sum0 = sum1 = top0 = top1 = 0.f;
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
        const float e0 = fast_exp2(fmaf(sc[nt][0], rs0, -r0)), e1 = fast_exp2(fmaf(sc[nt][1], rs0, -r0));
        const float e2 = fast_exp2(fmaf(sc[nt][2], rs1, -r1)), e3 = fast_exp2(fmaf(sc[nt][3], rs1, -r1));
        sum0 += e0 + e1;
        sum1 += e2 + e3;
        pv[nt][0] = e0 * vs[2 * nt];
        pv[nt][1] = e1 * vs[2 * nt + 1];
        pv[nt][2] = e2 * vs[2 * nt];
        pv[nt][3] = e3 * vs[2 * nt + 1];
        top0 = fmax3(top0, fabsf(pv[nt][0]), fabsf(pv[nt][1]));
        top1 = fmax3(top1, fabsf(pv[nt][2]), fabsf(pv[nt][3]));
    }
}

// A new reference for a row: the largest score mx of the step (log2), and the largest
// |2^(score - mx) * v_scale|, both over the row.  R never falls, so a step without values
// (top = 0) must not put it near mx: the products that come later may lie far below.
__device__ __forceinline__ float new_reference(float r, float mx, float top) {
    const int least = kPBits - kPMost, e = top > 0.f ? max(f32_exponent(top), least) : least;
    return fmaxf(r, mx + (float)(e - kPBits));
}

// The 32 cells of slot x; cells lo .. hi - 1 of them count (hi > 0, lo < 32).
__device__ __forceinline__ void step32(State& s, const Query& q, float kmul, const Ctx& c, int x, int lo, int hi, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int pg = (g >> 1) | ((g & 1) << 2);            // cell (of eight) of this lane's K column
    const uint8_t* kst = c.ring + x * 2 * kStepBytes;
    const bool whole = lo <= 0 && hi >= kStep;           // warp-uniform
    // ---- the columns' scales, each converted once: lane (g, t) will need cells 8 nt + t + 4 e, in that order
    {
        const __half* sp = reinterpret_cast<const __half*>(c.scales + x * 2 * kStepScales) + lane;
        const int at = 8 * (lane & 3) + 2 * (lane >> 3) + ((lane >> 2) & 1);
        float ks = __half2float(sp[0]) * kmul, vs = __half2float(sp[kStep]);
        if (!whole && (lane < lo || lane >= hi)) ks = vs = 0.f;   // they may be anything
        c.cols[at] = ks;
        c.cols[kStep + at] = vs;
        __syncwarp();
    }
    // ---- S = Q K^T: Q (K + 128) from the accumulators' start at -128 sum(Q), in units of 2^-24
    float sc[4][4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
        sc[nt][0] = sc[nt][1] = q.bias0;
        sc[nt][2] = sc[nt][3] = q.bias1;
    }
#pragma unroll
    for (int hk = 0; hk < 2; ++hk) {
        uint4 w[4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
            w[nt] = *reinterpret_cast<const uint4*>(kst + (8 * nt + pg) * kHeadDim + (((4 * hk + t) ^ pg) << 4));
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {             // four independent chains
                uint32_t b0, b1;
                biased_pairs(k == 0 ? w[nt].x : k == 1 ? w[nt].y : k == 2 ? w[nt].z : w[nt].w, b0, b1);
                const uint32_t(&a)[4] = q.a[4 * hk + k];
                mma_f16(sc[nt], a[0], a[1], a[2], a[3], b0, b1);
            }
    }
    float vs[8];
    {
        const float4* cp = reinterpret_cast<const float4*>(c.cols + 8 * t);
        const float4 k0 = cp[0], k1 = cp[1], v0 = cp[kStep / 4], v1 = cp[kStep / 4 + 1];
        const float ks[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
        vs[0] = v0.x, vs[1] = v0.y, vs[2] = v0.z, vs[3] = v0.w, vs[4] = v1.x, vs[5] = v1.y, vs[6] = v1.z, vs[7] = v1.w;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[nt][e] *= ks[2 * nt + (e & 1)];
    }
    if (!whole) {
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int cell = 8 * nt + t + 4 * e;
                if (cell < lo || cell >= hi) sc[nt][e] = sc[nt][e + 2] = -INFINITY;
            }
    }
    // ---- weights; the reference moves when a product or a sum passes its limit
    float pv[4][4], sum0, sum1, top0, top1;
    bool move = __any_sync(0xffffffffu, s.r0 == -INFINITY || s.r1 == -INFINITY);   // an item's first step
    if (!move) {
        weigh(sc, pv, vs, q.rs0, q.rs1, s.r0, s.r1, sum0, sum1, top0, top1);
        move = __any_sync(0xffffffffu, top0 > kPTop || top1 > kPTop || sum0 > kSumTop || sum1 > kSumTop);
    }
    if (move) {
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            mx0 = fmax3(mx0, sc[nt][0], sc[nt][1]);
            mx1 = fmax3(mx1, sc[nt][2], sc[nt][3]);
        }
        mx0 = quad_max(mx0 * q.rs0);
        mx1 = quad_max(mx1 * q.rs1);
        weigh(sc, pv, vs, q.rs0, q.rs1, mx0, mx1, sum0, sum1, top0, top1);
        const float n0 = new_reference(s.r0, mx0, quad_max(top0)), n1 = new_reference(s.r1, mx1, quad_max(top1));
        const float al0 = s.r0 == -INFINITY ? 1.f : fast_exp2(s.r0 - n0), al1 = s.r1 == -INFINITY ? 1.f : fast_exp2(s.r1 - n1);
        s.r0 = n0;
        s.r1 = n1;
        s.l0 *= al0;
        s.l1 *= al1;
#pragma unroll
        for (int d = 0; d < 16; ++d) {
            s.o[d][0] *= al0;
            s.o[d][1] *= al0;
            s.o[d][2] *= al1;
            s.o[d][3] *= al1;
        }
        weigh(sc, pv, vs, q.rs0, q.rs1, n0, n1, sum0, sum1, top0, top1);
    }
    s.l0 += sum0;
    s.l1 += sum1;
    // ---- O += P V, 16 cells at a time
    const int vr = lane & 7;
    const int vcell = ((vr >> 1) | ((vr & 1) << 2)) + 8 * ((lane >> 3) & 1);
    const uint32_t v_base = smem_u32(kst) + kStepBytes + (uint32_t)vcell * kHeadDim;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t af[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            af[2 * e] = pack_f16x2(pv[2 * j + e][0], pv[2 * j + e][1]);
            af[2 * e + 1] = pack_f16x2(pv[2 * j + e][2], pv[2 * j + e][3]);
        }
        // byte pairs by ldmatrix.trans: of the 32 dims 32 d4 .. + 31, lane (g, t) gets, of cells
        // perm(2t), perm(2t + 1) (and those + 8), dims 32 d4 + 2g, + 1 and 32 d4 + 16 + 2g, + 1.
        // O tile 4 d4 + 2h + e holds dims 32 d4 + 16h + 2n + e at column n.
#pragma unroll
        for (int d4 = 0; d4 < 4; ++d4) {
            uint32_t r[4];
            ldsm_x4_t(v_base + j * 16 * kHeadDim + (uint32_t)(((2 * d4 + (lane >> 4)) ^ (vcell & 7)) << 4), r[0], r[1], r[2],
                      r[3]);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                uint32_t e0, d0, e1, d1;
                int8x4_to_f16_even_odd(r[2 * hh], e0, d0);
                int8x4_to_f16_even_odd(r[2 * hh + 1], e1, d1);
                mma_f16(s.o[4 * d4 + 2 * hh], af[0], af[1], af[2], af[3], e0, e1);
                mma_f16(s.o[4 * d4 + 2 * hh + 1], af[0], af[1], af[2], af[3], d0, d1);
            }
        }
    }
}

struct RawQuery {
    uint4 w[2][4];                        // rows g and g + 8: dims 64 (j / 2) + 16 t + 8 (j & 1) .. + 7
};
__device__ __forceinline__ void load_q(const PagedArgs& a, size_t row0, int rows, int lane, RawQuery& raw) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            raw.w[half][j] = make_uint4(0u, 0u, 0u, 0u);
            if (g + 8 * half < rows)
                raw.w[half][j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                                 (row0 + g + 8 * half) * kHeadDim + 64 * (j >> 1) + 16 * t +
                                                                 8 * (j & 1));
        }
}
// Largest |x| of packed 16-bit pairs, still packed.
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t w, int type) {
    if (type == QSA_F16) {
        const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&m), __habs2(*reinterpret_cast<const __half2*>(&w)));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    const __nv_bfloat162 r =
        __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&m), __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void convert_q(const RawQuery& raw, int type, Query& q) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t top = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4& w = raw.w[half][j];
            top = max_abs2(max_abs2(max_abs2(max_abs2(top, w.x, type), w.y, type), w.z, type), w.w, type);
        }
        const float lo = type == QSA_F16 ? __half2float(__ushort_as_half((uint16_t)top)) : bf16_lo(top);
        const float hi = type == QSA_F16 ? __half2float(__ushort_as_half((uint16_t)(top >> 16))) : bf16_hi(top);
        const float amax = quad_max(fmaxf(lo, hi));
        const int e = amax > 0.f ? min(max(f32_exponent(amax) - 12, -114), 114) : 0;
        const float down = exp2i(-e);
        (half ? q.rs1 : q.rs0) = exp2i(e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x[8];
            unpack8(raw.w[half][j], type, x);
#pragma unroll
            for (int k = 0; k < 2; ++k) {   // k step 4 (j / 2) + 2 (j & 1) + k: four dims
                const int kk = 4 * (j >> 1) + 2 * (j & 1) + k;
                q.a[kk][half] = pack_f16x2(x[4 * k] * down, x[4 * k + 2] * down);
                q.a[kk][2 + half] = pack_f16x2(x[4 * k + 1] * down, x[4 * k + 3] * down);
            }
        }
    }
    // the rows' sums times 128 * 2^-24, by the same products: every K + 128 = 128
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) mma_f16(sum, q.a[kk][0], q.a[kk][1], q.a[kk][2], q.a[kk][3], 0x00800080u, 0x00800080u);
    q.bias0 = -sum[0];
    q.bias1 = -sum[2];
}

// Rows of an item: the first one's number in q and out, and how many.
__device__ __forceinline__ size_t first_row(const PagedArgs& a, const Ctx& c, int seq, int hk, int& rows) {
    const int h = c.tiles == 1 ? hk : hk / c.tiles, tile = hk - h * c.tiles;
    rows = min(kRowsTile, c.group - kRowsTile * tile);
    return (size_t)seq * a.n_heads + h * c.group + kRowsTile * tile;
}

// What a warp leaves for the CTA's merge.
struct Left {
    int first;           // its run begins inside an item (seq, hk), and that: 1 = ends in the run (part in
    int seq, hk;         // `ended`), 2 = goes on behind it, 3 = ends with it (part in the ring); 0: no such item
    int open;            // its run ends inside an item begun in it (part in the ring): that item, and how many of its
    int oseq, ohk, rest; // pages are behind the run
};

// One warp's pages, from place w on.  SMALL: they are all one item's, and what comes of
// them stays in the ring.
template <bool SMALL>
__device__ __forceinline__ void walk_run(const PagedArgs& a, const Ctx& c, Walk w, Left& left) {
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const float kmul = a.sm_scale * kLog2e * 0x1p24f;   // scores come in units of 2^-24
    left = Left{0, w.s, w.hk, 0, 0, 0, 0};
    Fetch f;
    f.w = w;
    f.at = 0;
    f.entry = -1;
    f.resident = 0;
    f.ok = f.second = false;
    f.ksrc = a.k_pool;
    f.vsrc = a.v_pool;
    f.ssrc = a.k_scale;
    f.look(a, c, 0);
    int rows;
    size_t row0 = first_row(a, c, w.s, w.hk, rows);
    RawQuery raw;
    load_q(a, row0, rows, lane, raw);
#pragma unroll 1
    for (int k = 0; k < kDepth; ++k) f.put(a, c, k);
    int slot = 0;                         // where the next step is
#pragma unroll 1
    for (int pos = 0; pos < c.n;) {
        const int n = min(w.q.np - w.off, c.n - pos);
        Query query;
        convert_q(raw, a.q_type, query);
        // the item after this one: its queries are on their way while this one is worked on
        const Walk here = w;
        const size_t here0 = row0;
        const int here_rows = rows;
        if (pos + n < c.n) {
            w.next_item(a, c.n_hk);
            row0 = first_row(a, c, w.s, w.hk, rows);
            load_q(a, row0, rows, lane, raw);
        }
        State s;
#pragma unroll
        for (int d = 0; d < 16; ++d) s.o[d][0] = s.o[d][1] = s.o[d][2] = s.o[d][3] = 0.f;
        s.r0 = s.r1 = -INFINITY;
        s.l0 = s.l1 = 0.f;
        const int cell0 = (here.q.p0 + here.off) * kPage;
        int lo = here.q.first - cell0, hi = here.q.n - cell0;   // the item's cells, from the step's first one
#pragma unroll 1
        for (int step = 0; step < n * (kPage / kStep); ++step) {
            copies_wait<kDepth - 1>();    // one group a step: all but the youngest ones have landed
            __syncwarp();
            if (((f.resident >> slot) & 1u) && hi > 0 && lo < kStep) step32(s, query, kmul, c, slot, lo, hi, lane);
            __syncwarp();                 // every lane has read the step
            f.put(a, c, slot);
            slot = slot + 1 == kDepth ? 0 : slot + 1;
            lo -= kStep;
            hi -= kStep;
        }
        pos += n;
        // ---- the item's end, or the run's
        s.l0 += __shfl_xor_sync(0xffffffffu, s.l0, 1);
        s.l0 += __shfl_xor_sync(0xffffffffu, s.l0, 2);
        s.l1 += __shfl_xor_sync(0xffffffffu, s.l1, 1);
        s.l1 += __shfl_xor_sync(0xffffffffu, s.l1, 2);
        const bool ends = here.off + n == here.q.np;
        const bool complete = !SMALL && here.off == 0 && ends;
        Part* part = nullptr;
        if (!complete) {
            if (SMALL || here.off == 0) {
                left.open = 1;
                left.oseq = here.s;
                left.ohk = here.hk;
                left.rest = here.q.np - n;
            } else {
                left.first = !ends ? 2 : pos < c.n ? 1 : 3;
            }
            if (SMALL || pos == c.n) {  // the run is over: its ring is free
                copies_wait<0>();
                __syncwarp();
                part = reinterpret_cast<Part*>(c.ring);
            } else {
                part = c.ended;
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = g + 8 * half;
            if (r >= here_rows) continue;
            const float l = half ? s.l1 : s.l0, m = half ? s.r1 : s.r0;
            const float back = complete ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int d = 16 * k + 4 * t, e = 2 * k, v = 2 * half;
                const float x0 = s.o[e][v] * back, x1 = s.o[e + 1][v] * back, x2 = s.o[e][v + 1] * back,
                            x3 = s.o[e + 1][v + 1] * back;
                if (complete) store4(a.out, a.out_type, (here0 + r) * kHeadDim + d, x0, x1, x2, x3);
                else *reinterpret_cast<float4*>(&part->o[r][col(r, d)]) = make_float4(x0, x1, x2, x3);
            }
            if (t == 0) {
                if (!complete) {
                    part->m[r] = m;
                    part->l[r] = l;
                } else if (a.lse) {
                    a.lse[here0 + r] = lse_of(m, l);
                }
            }
        }
    }
    copies_wait<0>();                     // nothing in flight when a warp leaves
}

// Merges the parts that the CTA's warps have left, item by item, a row to a warp.  The
// warps' runs follow one another, so an item's parts are those of consecutive warps.
__device__ __forceinline__ void merge_cta(const PagedArgs& a, const Ctx& c, const Left* s_left, const uint8_t* smem,
                                          int total, int runs) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Ws ws = workspace_of(a.workspace);
    Rec rec{-1, 0, 0, 0};
    for (int w0 = 0, skip_first = 0; w0 < kWarps;) {
        // a chain of parts: from warp w0's first part, or from its open one
        const Left& x = s_left[w0];
        const bool from_before = !skip_first && x.first != 0;   // only in warp 0: elsewhere the chain before took it
        const bool open = x.open != 0;
        if (!from_before && !open) {
            ++w0;
            skip_first = 0;
            continue;
        }
        const int seq = from_before ? x.seq : x.oseq, hk = from_before ? x.hk : x.ohk;
        int w1 = w0;
        bool closed = from_before && x.first != 2;
        while (!closed && w1 + 1 < kWarps && s_left[w1 + 1].first != 0) {
            ++w1;
            closed = s_left[w1].first != 2;
        }
        const bool complete = closed && !from_before;
        int rows;
        const size_t row0 = first_row(a, c, seq, hk, rows);
        Part* to = &ws.cta[blockIdx.x].cta[from_before ? 0 : 1];
        if (!complete && !from_before)
            rec = Rec{cta_of(total, run_begin(total, blockIdx.x * kWarps + w0 + 1, runs) + x.rest - 1, runs), seq, hk, 0};
        auto part_of = [&](int w) {       // w0's ring where the chain begins with an open part
            const bool ended = (w > w0 || from_before) && s_left[w].first == 1;
            return reinterpret_cast<const Part*>(ended ? smem + kRings + w * sizeof(Part) : smem + w * kDepth * 2 * kStepBytes);
        };
        // rows warp, warp + 4, ..; those from `rows` on hold anything and are not written
        constexpr int kMine = kRowsTile / kWarps;
        float M[kMine], L[kMine];
        float4 o[kMine];
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            M[j] = -INFINITY;
            L[j] = 0.f;
            o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 1
        for (int w = w0; w <= w1; ++w)
#pragma unroll
            for (int j = 0; j < kMine; ++j) M[j] = fmaxf(M[j], part_of(w)->m[warp + j * kWarps]);
#pragma unroll 1
        for (int w = w0; w <= w1; ++w) {
            const Part* p = part_of(w);
#pragma unroll
            for (int j = 0; j < kMine; ++j) {
                const int r = warp + j * kWarps;
                const float l = p->l[r], wt = merge_weight(p->m[r], l, M[j]);
                const float4 v = *reinterpret_cast<const float4*>(&p->o[r][col(r, 4 * lane)]);
                L[j] += wt * l;
                o[j].x += wt * v.x;
                o[j].y += wt * v.y;
                o[j].z += wt * v.z;
                o[j].w += wt * v.w;
            }
        }
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int r = warp + j * kWarps;
            if (r >= rows) break;
            if (complete) {
                const float inv = L[j] == 0.f ? 0.f : 1.f / L[j];
                store4(a.out, a.out_type, (row0 + r) * kHeadDim + 4 * lane, o[j].x * inv, o[j].y * inv, o[j].z * inv, o[j].w * inv);
                if (lane == 0 && a.lse) a.lse[row0 + r] = lse_of(M[j], L[j]);
            } else {
                *reinterpret_cast<float4*>(&to->o[r][col(r, 4 * lane)]) = o[j];
                if (lane == 0) {
                    to->m[r] = M[j];
                    to->l[r] = L[j];
                }
            }
        }
        // go on behind the chain: with the open part of the warp that it ended in, if that is another item's
        skip_first = 1;
        if (w1 == w0 && !from_before) {
            ++w0;
            skip_first = 0;
        } else {
            w0 = w1;
            if (!closed) break;           // the chain reaches the run's end
        }
    }
    if (threadIdx.x == 0) ws.rec[blockIdx.x] = rec;
}

__device__ __forceinline__ Ctx context(const PagedArgs& a, uint8_t* smem, float* cols, int warp) {
    Ctx c;
    c.ring = smem + warp * kDepth * 2 * kStepBytes;
    c.scales = smem + kWarps * kDepth * 2 * kStepBytes + warp * kDepth * 2 * kStepScales;
    c.ended = reinterpret_cast<Part*>(smem + kRings) + warp;
    c.cols = cols;
    c.group = a.n_heads / a.n_kv;
    c.tiles = (c.group + kRowsTile - 1) / kRowsTile;
    c.n_hk = a.n_kv * c.tiles;
    c.n = 0;
    return c;
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
    for (int k = 0; k < kWarps; ++k) {
        if (k < warp) before += s_warp[k];
        total += s_warp[k];
    }
    return total;
}

__global__ void __launch_bounds__(kThreads, 2) paged_attn_kernel(const __grid_constant__ PagedArgs a) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ int s_warp[2][kWarps];
    __shared__ Start s_start[kWarps + 1];
    __shared__ Left s_left[kWarps];
    __shared__ __align__(16) float s_cols[kWarps][2 * kStep];
    const int tid = threadIdx.x, warp = tid >> 5;
    wait_for_stream();
    asm volatile("griddepcontrol.launch_dependents;");   // the join may be set up now; it waits for this grid's end

    Ctx c = context(a, smem_raw, s_cols[warp], warp);

    // ---- the warps' runs of the pages of all items
    const int per = (a.n_seq + kThreads - 1) / kThreads;   // consecutive sequences per thread
    const int s_lo = min(tid * per, a.n_seq), s_hi = min(s_lo + per, a.n_seq);
    int pages = 0, sum = 0, pages_before, before;
    for (int s = s_lo; s < s_hi; ++s) {
        const int np = seq_of(a, s, blockIdx.x == 0).np;
        pages += np;
        sum += places(np);
    }
    const int all_pages = block_scan(pages, s_warp[0], pages_before);
    const int total = block_scan(sum, s_warp[1], before) * c.n_hk;   // at most 2^30, checked on the host
    const int runs = run_count(total, (int)gridDim.x);
    {
        int at = before, at_page = pages_before, s = s_lo, np = -1;
#pragma unroll
        for (int k = 0; k <= kWarps; ++k) {
            // the one thread whose sequences hold the place where warp k begins
            const int first = run_begin(total, blockIdx.x * kWarps + k, runs);
            if (first >= total && tid == 0) s_start[k] = Start{0, 0, 1, all_pages};
            if (first < before * c.n_hk || first >= (before + sum) * c.n_hk) continue;
            for (;;) {
                if (np < 0) np = seq_of(a, s, false).np;
                if (first < (at + places(np)) * c.n_hk) break;
                at += places(np);
                at_page += np;
                ++s;
                np = -1;
            }
            s_start[k] = Start{s, first - at * c.n_hk, np, at_page};
        }
    }
    __syncthreads();
    Left left{0, 0, 0, 0, 0, 0, 0};
    Walk w;
    {
        // even lanes: where this warp begins, odd ones: where the next does
        const Start st = s_start[warp + (tid & 1)];
        const int hk = st.place / places(st.np), off = max(st.place - hk * places(st.np) - kItemPlaces, 0);
        const int page = st.pages * c.n_hk + hk * st.np + off;
        c.n = __shfl_sync(0xffffffffu, page, 1) - __shfl_sync(0xffffffffu, page, 0);
        w.s = __shfl_sync(0xffffffffu, st.s, 0);
        w.hk = __shfl_sync(0xffffffffu, hk, 0);
        w.off = __shfl_sync(0xffffffffu, off, 0);
    }
    if (c.n > 0) {
        w.q = seq_of(a, w.s, false);
        walk_run<false>(a, c, w, left);
    }
    if ((tid & 31) == 0) s_left[warp] = left;
    __syncthreads();
    merge_cta(a, c, s_left, smem_raw, total, runs);
    // rows of the sequences that have no page at all
    for (int s = blockIdx.x; s < a.n_seq; s += gridDim.x) {
        if (seq_of(a, s, false).np > 0) continue;
        const size_t row = (size_t)s * a.n_heads;
        for (int e = tid; e < a.n_heads * (kHeadDim / 4); e += kThreads)
            store4(a.out, a.out_type, row * kHeadDim + 4 * e, 0.f, 0.f, 0.f, 0.f);
        if (a.lse)
            for (int e = tid; e < a.n_heads; e += kThreads) a.lse[row + e] = -INFINITY;
    }
}

// One item per cluster: warp i of its 32 takes pages i np / 32 .. (i + 1) np / 32.  Each
// CTA merges its warps' parts into one, then CTA r of the cluster joins all eight CTAs'
// rows r and r + 8.
constexpr int kCluster = 8;
// As many clusters as run at once: two CTAs per SM, but a cluster stays within one of the GPU's processing clusters, and 152
// SMs of them hold between 32 (each a cluster short of 2 n / 8) and 38; beyond 32 the occupancy query says (0.8 us).
constexpr int kSmallItems = 38, kSmallSure = 32;

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 2)
paged_small_kernel(const __grid_constant__ PagedArgs a) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ Part s_part;               // of this CTA; m = -inf and l = 0 where it has none
    __shared__ int s_has[kWarps];
    __shared__ __align__(16) float s_cols[kWarps][2 * kStep];
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    wait_for_stream();
    const int rank = (int)cluster.block_rank(), item = blockIdx.x / kCluster;
    Ctx c = context(a, smem_raw, s_cols[warp], warp);
    Walk w;
    w.s = item / c.n_hk;
    w.hk = item - w.s * c.n_hk;
    w.q = seq_of(a, w.s, rank == 0 && tid == 0 && w.hk == 0);
    const int i = rank * kWarps + warp, all = kCluster * kWarps;
    w.off = (int)((long long)w.q.np * i / all);
    c.n = (int)((long long)w.q.np * (i + 1) / all) - w.off;
    Left left{0, 0, 0, 0, 0, 0, 0};
    if (c.n > 0) walk_run<true>(a, c, w, left);
    if (lane == 0) s_has[warp] = left.open;
    int rows;
    const size_t row0 = first_row(a, c, w.s, w.hk, rows);
    __syncthreads();
    for (int r = warp; r < rows; r += kWarps) {
        float m[kWarps], l[kWarps], M = -INFINITY;
        const Part* part[kWarps];
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            part[k] = reinterpret_cast<const Part*>(smem_raw + k * kDepth * 2 * kStepBytes);
            m[k] = s_has[k] ? part[k]->m[r] : -INFINITY;
            l[k] = s_has[k] ? part[k]->l[r] : 0.f;
            M = fmaxf(M, m[k]);
        }
        float L = 0.f, x0 = 0.f, x1 = 0.f, x2 = 0.f, x3 = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            if (!s_has[k]) continue;
            const float wt = merge_weight(m[k], l[k], M);
            const float4 o = *reinterpret_cast<const float4*>(&part[k]->o[r][col(r, 4 * lane)]);
            L += wt * l[k];
            x0 += wt * o.x;
            x1 += wt * o.y;
            x2 += wt * o.z;
            x3 += wt * o.w;
        }
        *reinterpret_cast<float4*>(&s_part.o[r][col(r, 4 * lane)]) = make_float4(x0, x1, x2, x3);
        if (lane == 0) {
            s_part.m[r] = M;
            s_part.l[r] = L;
        }
    }
    cluster.sync();
    const int r = rank + kCluster * warp; // warps 0 and 1
    if (r < rows) {
        float m[kCluster], l[kCluster], M = -INFINITY;
        float4 o[kCluster];
#pragma unroll
        for (int k = 0; k < kCluster; ++k) {
            const Part* p = cluster.map_shared_rank(&s_part, k);
            m[k] = p->m[r];
            l[k] = p->l[r];
            o[k] = *reinterpret_cast<const float4*>(&p->o[r][col(r, 4 * lane)]);
            M = fmaxf(M, m[k]);
        }
        float L = 0.f, x0 = 0.f, x1 = 0.f, x2 = 0.f, x3 = 0.f;
#pragma unroll
        for (int k = 0; k < kCluster; ++k) {
            const float wt = merge_weight(m[k], l[k], M);
            L += wt * l[k];
            x0 += wt * o[k].x;
            x1 += wt * o[k].y;
            x2 += wt * o[k].z;
            x3 += wt * o[k].w;
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        store4(a.out, a.out_type, (row0 + r) * kHeadDim + 4 * lane, x0 * inv, x1 * inv, x2 * inv, x3 * inv);
        if (lane == 0 && a.lse) a.lse[row0 + r] = lse_of(M, L);
    }
    cluster.sync();                       // no CTA leaves while its part is being read
}

// Joins the parts of items that are cut between CTAs.  SPLIT (few items, many parts
// each): block (k, r) takes row r of item k, whose place among the runs it works out
// from the lengths while the kernel before still runs; its warps share the parts.
// Otherwise (many items, a few parts each): block (k, r) takes the item that CTA k begins
// and does not end, rows 4 r .. 4 r + 3, one to a warp.
constexpr int kJoinThreads = 128;
constexpr int kJoinItems = 64;            // most items for SPLIT
constexpr int kJoinLoads = 8;             // parts on their way at a time

template <bool SPLIT>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedArgs a, int ctas) {
    __shared__ float s_o[4][kHeadDim], s_m[4], s_l[4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Ws ws = workspace_of(a.workspace);
    const int group = a.n_heads / a.n_kv, tiles = (group + kRowsTile - 1) / kRowsTile;
    int c0, last, seq, hk;
    if (SPLIT) {
        const int n_hk = a.n_kv * tiles;
        seq = blockIdx.x / n_hk;
        hk = blockIdx.x - seq * n_hk;
        // two sequences per lane: at most 64 items.  The lengths are final although this is before the wait: the attention
        // lets this grid start only after its own wait, behind all that came before it, and does not write them.
        const int n0 = 2 * lane < a.n_seq ? seq_from(a, __ldcg(a.seq_lens + 2 * lane), false).np : 0;
        const int n1 = 2 * lane + 1 < a.n_seq ? seq_from(a, __ldcg(a.seq_lens + 2 * lane + 1), false).np : 0;
        int before = (2 * lane < seq ? places(n0) : 0) + (2 * lane + 1 < seq ? places(n1) : 0);
        int total = places(n0) + places(n1);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            before += __shfl_xor_sync(0xffffffffu, before, o);
            total += __shfl_xor_sync(0xffffffffu, total, o);
        }
        const int np = __shfl_sync(0xffffffffu, seq & 1 ? n1 : n0, seq >> 1);
        const int start = before * n_hk + hk * places(np) + kItemPlaces;   // its first page
        c0 = last = 0;
        if (np > 0) {
            total *= n_hk;
            const int runs = run_count(total, ctas);
            c0 = cta_of(total, start, runs);
            last = cta_of(total, start + np - 1, runs);
        }
        wait_for_stream();                // every block: this grid's end has to mean the end of the one before
        if (last == c0) return;           // no page, or all in one CTA: done there
    } else {
        wait_for_stream();
        c0 = blockIdx.x;
        const Rec rec = ws.rec[c0];
        last = rec.last;
        seq = rec.seq;
        hk = rec.hk;
        if (last < 0) return;
    }
    const int h = hk / tiles, tile = hk - h * tiles;
    const int r = SPLIT ? blockIdx.y : 4 * blockIdx.y + warp;
    if (r >= min(kRowsTile, group - kRowsTile * tile)) return;
    // part 0 is CTA c0's second, part i the first of CTA c0 + i
    const int n = last - c0 + 1, step = SPLIT ? 4 : 1;
    float M = -INFINITY, L = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = SPLIT ? warp : 0; i0 < n; i0 += step * kJoinLoads) {
        float m[kJoinLoads], l[kJoinLoads], top = M;
        float4 o[kJoinLoads];
#pragma unroll
        for (int j = 0; j < kJoinLoads; ++j) {
            const int i = i0 + step * j;
            m[j] = -INFINITY;
            l[j] = 0.f;
            o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < n) {
                const Part* p = &ws.cta[c0 + i].cta[i == 0 ? 1 : 0];
                m[j] = p->m[r];
                l[j] = p->l[r];
                o[j] = *reinterpret_cast<const float4*>(&p->o[r][col(r, 4 * lane)]);
            }
        }
#pragma unroll
        for (int j = 0; j < kJoinLoads; ++j) top = fmaxf(top, m[j]);
        const float keep = merge_weight(M, L, top);
        M = top;
        L *= keep;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] *= keep;
#pragma unroll
        for (int j = 0; j < kJoinLoads; ++j) {
            const float wt = merge_weight(m[j], l[j], M);
            L += wt * l[j];
            x[0] += wt * o[j].x;
            x[1] += wt * o[j].y;
            x[2] += wt * o[j].z;
            x[3] += wt * o[j].w;
        }
    }
    if (SPLIT) {
        *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = make_float4(x[0], x[1], x[2], x[3]);
        if (lane == 0) {
            s_m[warp] = M;
            s_l[warp] = L;
        }
        __syncthreads();
        if (warp != 0) return;
        M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
        L = x[0] = x[1] = x[2] = x[3] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float wt = merge_weight(s_m[k], s_l[k], M);
            const float4 o = *reinterpret_cast<const float4*>(&s_o[k][4 * lane]);
            L += wt * s_l[k];
            x[0] += wt * o.x;
            x[1] += wt * o.y;
            x[2] += wt * o.z;
            x[3] += wt * o.w;
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const size_t row = (size_t)seq * a.n_heads + h * group + kRowsTile * tile + r;
    store4(a.out, a.out_type, row * kHeadDim + 4 * lane, x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    if (lane == 0 && a.lse) a.lse[row] = lse_of(M, L);
}

}  // namespace

size_t paged_attn_workspace(int, int) { return kMaxCtas * (sizeof(Rec) + sizeof(CtaSpace)); }

cudaError_t launch_paged_attn(const PagedArgs& a, cudaStream_t stream) {
    const int group = a.n_heads / a.n_kv, rows = group < kRowsTile ? group : kRowsTile;
    const long long items = (long long)a.n_seq * a.n_kv * ((group + kRowsTile - 1) / kRowsTile);
    cudaError_t e;
    // A cluster per item while all of them run at once and tables are not too wide: up to 64 pages, and two more for each
    // item that keeps the GPU busy beside it.  The width stands for the lengths, which only the device knows: a short
    // sequence under a wide table takes the runs (1 x 1,021 cells, 4 KV heads: 6.9 us under 16 entries, 11.1 under 512).
    // Measured, us, cluster against runs and join: 4 items of 1,024 cells 7.1 / 10.6, of 4,096 9.4 / 11.4, of 8,192 13.5 /
    // 12.6; 32 items of 1,024 7.9 / 12.1, of 8,192 16.5 / 20.4; 36 items (the most at once here) of 1,021 8.1 / 12.4, of
    // 4,096 11.6 / 16.2; 37 items (two waves) of 1,021 13.2 / 11.8; 38 of 4,096 19.6 / 17.0.
    if (items <= kSmallItems && a.n_lpages <= 64 + 2 * items) {
        e = cudaFuncSetAttribute(paged_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRings);
        int at_once = kSmallSure;
        if (e == cudaSuccess && items > kSmallSure) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3((unsigned)items * kCluster);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = kRings;
            e = cudaOccupancyMaxActiveClusters(&at_once, paged_small_kernel, &cfg);
        }
        if (e != cudaSuccess) return e;
        if (items <= at_once)
            return launch_overlapped(paged_small_kernel, dim3((unsigned)items * kCluster), kThreads, kRings, stream, a);
    }
    int dev = 0, sms = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(paged_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const int grid = 2 * sms < kMaxCtas ? 2 * sms : kMaxCtas;
    e = launch_overlapped(paged_attn_kernel, dim3((unsigned)grid), kThreads, kSmem, stream, a);
    if (e != cudaSuccess) return e;
    if (items <= kJoinItems)
        return launch_overlapped(paged_join_kernel<true>, dim3((unsigned)items, (unsigned)rows), kJoinThreads, 0, stream, a, grid);
    return launch_overlapped(paged_join_kernel<false>, dim3((unsigned)grid, (unsigned)(rows + 3) / 4), kJoinThreads, 0, stream,
                             a, grid);
}

}  // namespace qsa

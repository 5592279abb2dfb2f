// extend_tables.cu -- page tables extended and slots mapped for a step's new tokens
// (qsa_extend_tables).
//
// With old_s, new_s the lengths of sequence s: its tokens start at the exclusive
// sum of the earlier new lengths, and its new pages at the exclusive sum of the
// earlier page counts ceil((old + new) / 64) - ceil(old / 64), in the free list
// from its head on.  Everything else is per token.
//
// One launch: a CTA owns kTile consecutive tokens and scans all sequences itself
// (1,024 per step: a batch is one step, and reading 8 KB of lengths from L2 costs
// less than a second launch), leaving a mark at the first of its tokens of every
// sequence that has some; a running maximum over the marks gives each token its
// sequence.  The token on a new page's first cell writes the page's table entry,
// so each entry has one writer and no CTA reads what another writes.
//
// Bound by latency: a launch, one load of the lengths, two block sums, one load of a page
// and one store.  Inside a captured graph 1,024 sequences with a token each take 4.0 us, 300
// with up to 2,000 each (600,000 places, 7.2 MB) 5.1 us.
#include "serve.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;                    // consecutive sequences (in the scan) and tokens of a thread
constexpr int kTile = kThreads * kPer;     // tokens per CTA, sequences per scan step
constexpr unsigned kTop = 0x7fffffffu;     // sums stop here (tokens past n_tok are cut off anyway)

__device__ __forceinline__ unsigned add_top(unsigned x, unsigned y) { return min(x + y, kTop); }

struct Mark {                              // of a sequence, at the first of its tokens in the CTA's tile
    int seq, old, pos, base;               // pos: that token's cell; base: place in the free list of logical page 0
};

__global__ void __launch_bounds__(kThreads) extend_tables_kernel(const TablesArgs a) {
    __shared__ Mark s_mark[kTile];
    __shared__ int s_at[kTile];            // the place itself where a mark is, else -1
    __shared__ unsigned s_tok[8], s_pg[8];
    __shared__ int s_max[8];
    __shared__ unsigned s_taken;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned n_tok = (unsigned)a.n_tok;
    wait_for_stream();
    const unsigned lo = blockIdx.x * (unsigned)kTile, hi = min(lo + kTile, n_tok);
    int head = a.free_head ? a.free_head[0] : 0;
    if (head < 0 || head > a.n_free) {
        if (blockIdx.x == 0 && tid == 0) report(a.dev_status, QSA_DEV_NO_PAGE);
        head = head < 0 ? 0 : a.n_free;
    }
    const int cap = a.n_lpages * kPage;
#pragma unroll
    for (int j = 0; j < kPer; ++j) s_at[tid + j * kThreads] = -1;
    if (tid == 0) s_taken = 0;

    // ---- all sequences: where their tokens and new pages start
    unsigned tok0 = 0, pg0 = 0;            // of the sequences scanned so far
    for (int base = 0, step = 0; base < a.n_seq; base += kTile, ++step) {
        const bool mine = step % (int)gridDim.x == (int)blockIdx.x;   // this CTA writes the step's lengths
        int old[kPer], add[kPer];
        unsigned tok = 0, pg = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int s = base + tid * kPer + j;
            old[j] = add[j] = 0;
            if (s < a.n_seq) {
                old[j] = a.seq_lens[s];
                add[j] = a.new_lens[s];
            }
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int o = min(max(old[j], 0), cap), n = min(max(add[j], 0), cap - o);
            if (mine && (o != old[j] || n != add[j])) report(a.dev_status, QSA_DEV_BAD_SEQ_LEN);
            old[j] = o;
            add[j] = n;
            tok = add_top(tok, (unsigned)n);
            pg = add_top(pg, (unsigned)((o + n + kPage - 1) / kPage - (o + kPage - 1) / kPage));
        }
        unsigned itok = tok, ipg = pg;     // inclusive sums over the warp, then the block
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned t = __shfl_up_sync(0xffffffffu, itok, o), p = __shfl_up_sync(0xffffffffu, ipg, o);
            if (lane >= o) {
                itok = add_top(itok, t);
                ipg = add_top(ipg, p);
            }
        }
        __syncthreads();                   // the previous step's sums are read
        if (lane == 31) {
            s_tok[warp] = itok;
            s_pg[warp] = ipg;
        }
        __syncthreads();
        unsigned wtok = tok0, wpg = pg0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (w < warp) {
                wtok = add_top(wtok, s_tok[w]);
                wpg = add_top(wpg, s_pg[w]);
            }
            tok0 = add_top(tok0, s_tok[w]);
            pg0 = add_top(pg0, s_pg[w]);
        }
        // exclusive sum of the thread: the lane before's inclusive one (a stopped sum cannot be subtracted from)
        const unsigned ptok = __shfl_up_sync(0xffffffffu, itok, 1), ppg = __shfl_up_sync(0xffffffffu, ipg, 1);
        unsigned start = lane ? add_top(wtok, ptok) : wtok, pgs = lane ? add_top(wpg, ppg) : wpg;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int s = base + tid * kPer + j;
            if (s >= a.n_seq) break;
            const int o = old[j], held = (o + kPage - 1) / kPage;
            const int full = (o + add[j] + kPage - 1) / kPage - held;
            const unsigned first = min(start, n_tok);
            const int n = (int)min((unsigned)add[j], n_tok - first);   // the tokens that the arrays hold
            const int need = (o + n + kPage - 1) / kPage - held;
            if (mine) {
                a.seq_lens_out[s] = o + n;
                a.cu_tokens[s] = (int)first;
                if (n != add[j]) report(a.dev_status, QSA_DEV_TOKEN_OVERFLOW);
            }
            if (n > 0) {
                // pages of all sequences up to here; later ones only add (a sequence that is cut off
                // has none behind it)
                if (blockIdx.x == 0) atomicMax(&s_taken, pgs + (unsigned)need);
                const unsigned from = max(first, lo);
                if (from < min(first + (unsigned)n, hi)) {
                    const int place = (int)(from - lo);
                    s_at[place] = place;
                    s_mark[place] = Mark{s, o, o + (int)(from - first), head + (int)pgs - held};
                }
            }
            start = add_top(start, (unsigned)add[j]);
            pgs = add_top(pgs, (unsigned)full);
        }
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) {
        a.cu_tokens[a.n_seq] = (int)min(tok0, n_tok);
        a.free_head_out[0] = (int)min((unsigned)head + s_taken, (unsigned)a.n_free);
    }
    if (lo >= n_tok) return;

    // ---- the tile's tokens: the last mark at or before each
    int at[kPer], run = -1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        run = max(run, s_at[tid * kPer + j]);
        at[j] = run;
    }
    int inc = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc = max(inc, t);
    }
    if (lane == 31) s_max[warp] = inc;
    __syncthreads();
    int before = __shfl_up_sync(0xffffffffu, inc, 1);
    if (lane == 0) before = -1;
#pragma unroll
    for (int w = 0; w < 8; ++w)
        if (w < warp) before = max(before, s_max[w]);
    const unsigned total = min(tok0, n_tok);
    int slot[kPer], pos[kPer], seq[kPer], page[kPer];
    bool held[kPer], listed[kPer];         // on a page that the sequence had, or on one that the free list holds
    int32_t* entry[kPer];                  // where a new page's number goes, from the token on its first cell
#pragma unroll
    for (int j = 0; j < kPer; ++j) {       // all loads before the first store: entries read are not those written
        const int place = tid * kPer + j;
        pos[j] = 0;
        seq[j] = page[j] = -1;
        held[j] = listed[j] = false;
        entry[j] = nullptr;
        const int m = max(at[j], before);
        if (lo + place >= total || m < 0) continue;
        const Mark mk = s_mark[m];
        pos[j] = mk.pos + (place - m);
        seq[j] = mk.seq;
        const int lp = pos[j] >> 6, idx = mk.base + lp;
        int32_t* at_table = a.page_tables + (size_t)mk.seq * a.pt_stride + lp;
        held[j] = lp < (mk.old + kPage - 1) / kPage;
        listed[j] = !held[j] && idx < a.n_free;
        if (held[j]) page[j] = *at_table;
        else if (listed[j]) page[j] = a.free_pages[idx];
        if (!held[j] && (pos[j] & (kPage - 1)) == 0) entry[j] = at_table;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        slot[j] = -1;
        if (seq[j] < 0) continue;
        if (held[j] ? page[j] < 0 : !listed[j]) {
            report(a.dev_status, QSA_DEV_NO_PAGE);
        } else if (page[j] < 0 || page[j] >= a.n_ppages) {
            report(a.dev_status, QSA_DEV_BAD_PAGE);
            page[j] = -1;
        }
        if (entry[j]) *entry[j] = page[j];
        if (page[j] >= 0) slot[j] = page[j] * kPage + (pos[j] & (kPage - 1));
    }
    const unsigned t0 = lo + tid * kPer;
    if (t0 + kPer <= hi) {
        *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        *reinterpret_cast<int4*>(a.token_seq + t0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (t0 + j < hi) {
                a.slots[t0 + j] = slot[j];
                a.positions[t0 + j] = pos[j];
                a.token_seq[t0 + j] = seq[j];
            }
    }
}

}  // namespace

cudaError_t launch_extend_tables(const TablesArgs& a, cudaStream_t stream) {
    const unsigned grid = a.n_tok > 0 ? (unsigned)((a.n_tok + kTile - 1) / kTile) : 1u;
    return launch_overlapped(extend_tables_kernel, dim3(grid), kThreads, 0, stream, a);
}

}  // namespace qsa

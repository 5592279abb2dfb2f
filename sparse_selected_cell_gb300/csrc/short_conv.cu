// short_conv.cu -- the causal depthwise convolution of layers with a state (qsa_short_conv).
//
// out[t][c] = act(bias[c] + sum_j w[c][j] x[t - (W - 1) + j][c]): 2 W flops an element, so
// bytes are all: x read once, out written once, and the states of the sequences that go on.
//
// With 8,192 channels, 9 sequences of 1 to 2,000 tokens (8,600 in all, 235 MB) take 46 us, 5.1 TB/s,
// 0.75 of what a plain copy reaches (warps wait for DRAM: 166 registers a thread, weights and a
// window of inputs, leave 12 to an SM); one token to each of 512 (67 MB) 13.6 us, 0.73.
//
// A thread owns eight channels (one 16-byte word a token) and a run of consecutive tokens,
// the last W - 1 inputs in registers; a warp's accesses are 512 consecutive bytes.  Runs cut
// sequences anywhere.  Inside a sequence a run's loads go out together; where sequences
// begin, the tokens are taken one by one.
//
// States are updated in place without a block that waits for another: the block whose run
// holds a sequence's first token (the last run, for sequences that begin behind it and so
// have none) is the only one that touches its state.  It reads the old one, writes the new
// one, whose inputs it reads again where they lie in another run, and computes the first
// W - 1 tokens, the only ones that need the old state, even those past its run's end; the
// next run leaves them out.
#include "linear.cuh"

namespace qsa {
namespace {

constexpr int kConvThreads = 128;

// Weights [channel][tap] of eight channels (8 W consecutive values) as pairs of channels to a tap.
template <int W>
__device__ __forceinline__ void load_taps(const void* weight, size_t c, int type, f2 (&w)[W][4]) {
    float flat[8 * W];
#pragma unroll
    for (int i = 0; i < W; ++i) load8(weight, c * W + 8 * i, type, *reinterpret_cast<float(*)[8]>(flat + 8 * i));
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) w[i][j] = pair(flat[2 * j * W + i], flat[(2 * j + 1) * W + i]);
}

// The first sequence that begins at token t or later (n_seq: none), by the whole warp.
__device__ __forceinline__ int first_from(const int32_t* cu_tokens, int n_seq, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n_seq;                         // the answer is in [lo, lo + len]
    while (len > 0) {
        const int step = (len + 31) / 32, at = lo + (lane + 1) * step - 1;
        const unsigned there = __ballot_sync(0xffffffffu, at >= lo + len || cu_tokens[at] >= t);
        const int f = there ? __ffs(there) - 1 : 32;
        const int from = min(lo + f * step, lo + len);
        len = min(lo + f * step + step - 1, lo + len) - from;
        lo = from;
    }
    return lo;
}

template <int TYPE, int W, int RUN>
__global__ void __launch_bounds__(kConvThreads, 3) short_conv_kernel(const __grid_constant__ ConvArgs a, const unsigned cols) {
    const unsigned run = blockIdx.x / cols;          // the columns of one run side by side
    const int c = (int)((blockIdx.x - run * cols) * kConvThreads + threadIdx.x) * 8;
    const int t0 = (int)run * RUN, t1 = min(t0 + RUN, a.n_tok);
    const bool live = c < a.n_ch, last = blockIdx.x >= gridDim.x - cols;
    wait_for_stream();
    const uint16_t* x = a.x + c;
    uint16_t* out = a.out + c;
    auto input = [&](int t) { return *reinterpret_cast<const uint4*>(x + (long long)t * a.x_stride); };
    // the run's first inputs and the ones before it, whoever's they are
    constexpr int kAhead = 8;
    uint4 raw[kAhead], before[W - 1];
    if (live && t1 == t0 + RUN) {
#pragma unroll
        for (int i = 0; i < W - 1; ++i) before[i] = input(max(t0 - (W - 1) + i, 0));
#pragma unroll
        for (int i = 0; i < kAhead; ++i) raw[i] = input(t0 + i);
    }
    f2 w[W][4], bias[4] = {0ull, 0ull, 0ull, 0ull};
    if (live) {
        load_taps<W>(a.weight, (size_t)c, a.w_type, w);
        if (a.bias) load_pairs(a.bias, (size_t)c, a.w_type, bias);
    }
    f2 win[W - 1][4];                                // inputs t - (W - 1) .. t - 1
    auto token = [&](int t, const uint4& raw, bool write) {
        f2 in[4];
        unpack_pairs(raw, TYPE, in);
        if (write) {
            f2 y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[j] = bias[j];
#pragma unroll
                for (int i = 0; i < W - 1; ++i) y[j] = fma2(w[i][j], win[i][j], y[j]);
                y[j] = fma2(w[W - 1][j], in[j], y[j]);
            }
            if (a.activation == QSA_ACT_SILU) {
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = silu2(y[j]);
            }
            *reinterpret_cast<uint4*>(out + (long long)t * a.out_stride) = pack_pairs(y, TYPE);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int i = 0; i < W - 2; ++i) win[i][j] = win[i + 1][j];
            win[W - 2][j] = in[j];
        }
    };

    // the first sequence that begins here or later
    const int owned = t0 == 0 ? 0 : first_from(a.cu_tokens, a.n_seq, t0);
    if (blockIdx.x == 0 && a.dev_status)
        for (int i = threadIdx.x; i < a.n_seq; i += kConvThreads)
            if (tokens_bad(a.cu_tokens, i, a.n_tok)) report(a.dev_status, QSA_DEV_BAD_SEQ_LEN);
    if (!live) return;
    int s = owned - 1, begin = 0, end = t0;          // the sequence that the run begins in
    bool skip = true;
    auto look = [&]() {
        const int2 span = tokens_of(a.cu_tokens, s, a.n_tok);
        const int slot = a.state_slots[s];
        begin = span.x, end = span.y;
        skip = slot < 0 || slot >= a.n_slots;
        return slot;
    };
    if (s >= 0) look();
    const int following = owned < a.n_seq ? a.cu_tokens[owned] : a.n_tok;
    if (t0 - begin >= W - 1 && end >= t1 && following >= t1 && t1 == t0 + RUN && !last) {
        if (skip) return;                            // the whole run inside one sequence
#pragma unroll
        for (int i = 0; i < W - 1; ++i) unpack_pairs(before[i], TYPE, win[i]);
#pragma unroll 1
        for (int t = t0; t < t1; t += kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const uint4 now = raw[i];
                if (t + kAhead < t1) raw[i] = input(t + kAhead + i);
                token(t + i, now, true);
            }
        }
        return;
    }

    // Sequence s begins in this run: its state in, and out again as its tokens leave it.
    auto enter = [&]() {
        const int slot = look();
        if (c == 0 && slot >= a.n_slots) report(a.dev_status, QSA_DEV_BAD_STATE);
        if (skip) return;
        const bool fresh = a.old_lens && a.old_lens[s] <= 0;
        uint16_t* held = a.state + (size_t)slot * (W - 1) * a.n_ch + c;
        const int n = end - begin;
        uint4 old[W - 1], now[W - 1];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            old[i] = fresh ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(held + (size_t)i * a.n_ch);
            unpack_pairs(old[i], TYPE, win[i]);
        }
        if (n == 0 && !fresh) return;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {            // place i holds input n - (W - 1) + i: below 0, the old state's place i + n
            if (n - (W - 1) + i >= 0) {
                now[i] = input(begin + n - (W - 1) + i);
            } else {
                now[i] = old[i];
#pragma unroll
                for (int m = i + 1; m < W - 1; ++m)
                    if (m == i + n) now[i] = old[m];
            }
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i) *reinterpret_cast<uint4*>(held + (size_t)i * a.n_ch) = now[i];
    };
    // Up to W - 2 tokens past the run's end belong to a sequence that begins in it.
    const int reach = min(t1 + W - 2, a.n_tok);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {                // the inputs before the run, as far as they are the sequence's own
        const int t = t0 - (W - 1) + i;
        unpack_pairs(!skip && t >= begin && t < end ? input(t) : make_uint4(0, 0, 0, 0), TYPE, win[i]);
    }
    // from one sequence's first token to the next one's, eight inputs at a time
    int t = t0;
    while (t < reach) {
        int stop;
        if (t < t1) {
            while (s + 1 < a.n_seq && a.cu_tokens[s + 1] <= t) {
                ++s;
                enter();
            }
            stop = min(t1, s + 1 < a.n_seq ? max(a.cu_tokens[s + 1], t + 1) : a.n_tok);
        } else {
            if (skip || begin < t0) break;
            stop = min(reach, min(end, begin + W - 1));
            if (t >= stop) break;
        }
        const int from = skip ? stop : begin < t0 ? begin + W - 1 : t;   // tokens that are this run's to write
        const int to = min(stop, end);
        for (; t < stop; t += 8) {
            uint4 some[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) some[i] = t + i < stop ? input(t + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (t + i < stop) token(t + i, some[i], t + i >= from && t + i < to);
        }
        t = stop;
    }
    if (last)
        while (s + 1 < a.n_seq) {
            ++s;
            enter();
        }
}

// One token to every sequence: a thread keeps its channels' weights and goes through every gridDim.y-th sequence, the next
// one's state and input on their way while this one's are used.
template <int TYPE, int W>
__global__ void __launch_bounds__(kConvThreads) short_conv_step_kernel(const __grid_constant__ ConvArgs a) {
    const int c = (int)(blockIdx.x * kConvThreads + threadIdx.x) * 8;
    const bool live = c < a.n_ch;
    wait_for_stream();
    if (!live) return;
    f2 w[W][4], bias[4] = {0ull, 0ull, 0ull, 0ull};
    // slots and lengths two sequences ahead, states and inputs one
    const int stride = (int)gridDim.y;
    int slot = -1, slot_next = -1;
    bool fresh = false, fresh_next = false;
    uint4 held[W - 1], in = make_uint4(0, 0, 0, 0);
    auto ask_slot = [&](int s) {
        slot_next = -1;
        if (s >= a.n_seq) return;
        slot_next = a.state_slots[s];
        fresh_next = a.old_lens && a.old_lens[s] <= 0;
    };
    auto ask = [&](int s) {
        slot = slot_next, fresh = fresh_next;
        ask_slot(s + stride);
        if (slot >= a.n_slots) {
            if (c == 0) report(a.dev_status, QSA_DEV_BAD_STATE);
            slot = -1;
        }
        if (slot < 0) return;
        in = *reinterpret_cast<const uint4*>(a.x + (long long)s * a.x_stride + c);
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
            held[i] = fresh ? make_uint4(0, 0, 0, 0)
                            : *reinterpret_cast<const uint4*>(a.state + ((size_t)slot * (W - 1) + i) * a.n_ch + c);
    };
    ask_slot((int)blockIdx.y);
    ask((int)blockIdx.y);
    load_taps<W>(a.weight, (size_t)c, a.w_type, w);
    if (a.bias) load_pairs(a.bias, (size_t)c, a.w_type, bias);
#pragma unroll 1
    for (int s = (int)blockIdx.y; s < a.n_seq; s += stride) {
        const int at = slot;
        uint4 now[W];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) now[i] = held[i];
        now[W - 1] = in;
        if (s + stride < a.n_seq) ask(s + stride);
        if (at < 0) continue;
        f2 y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = bias[j];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            f2 x[4];
            unpack_pairs(now[i], TYPE, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = fma2(w[i][j], x[j], y[j]);
            if (i > 0) *reinterpret_cast<uint4*>(a.state + ((size_t)at * (W - 1) + i - 1) * a.n_ch + c) = now[i];
        }
        if (a.activation == QSA_ACT_SILU) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = silu2(y[j]);
        }
        *reinterpret_cast<uint4*>(a.out + (long long)s * a.out_stride + c) = pack_pairs(y, TYPE);
    }
}

constexpr int kStepBlocks = 5;                       // of kConvThreads, per SM

template <int TYPE, int W>
cudaError_t launch_step(const ConvArgs& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int cols = (a.n_ch / 8 + kConvThreads - 1) / kConvThreads;
    int rows = sms * kStepBlocks / cols;             // as many as run at once
    rows = rows < 1 ? 1 : rows > 65535 ? 65535 : rows;
    if (rows > a.n_seq) rows = a.n_seq;
    return launch_overlapped(short_conv_step_kernel<TYPE, W>, dim3((unsigned)cols, (unsigned)rows), kConvThreads, 0, stream, a);
}

template <int TYPE, int W, int RUN>
cudaError_t launch_run(const ConvArgs& a, cudaStream_t stream) {
    const long long cols = (a.n_ch / 8 + kConvThreads - 1) / kConvThreads;
    const long long runs = a.n_tok > 0 ? (a.n_tok + RUN - 1LL) / RUN : 1;
    return launch_overlapped(short_conv_kernel<TYPE, W, RUN>, dim3((unsigned)(cols * runs)), kConvThreads, 0, stream, a,
                             (unsigned)cols);
}

// Runs of 32 tokens where they are many; runs of 8 as long as there are no more than kShortRuns blocks of these to an SM: then
// what counts is how soon a run is through, the more so the more sequences begin in it.  Of 8,192 channels, runs of 8 and of 32:
// 64 sequences x 2 tokens 7.4 and 23.9 us, 512 x 4 36.6 and 43.2, 1 x 256 4.4 and 8.6, 1 x 2,048 13.8 and 15.4; 9 x 1-2,000
// (8,600 tokens) 51.5 and 45.9.  Runs of 1 take 58.2 us instead of 26.6 for 512 x 2, and win nowhere by more than half a us.
constexpr int kShortRuns = 32;

template <int TYPE, int W>
cudaError_t launch_width(const ConvArgs& a, cudaStream_t stream) {
    if (!a.cu_tokens) return launch_step<TYPE, W>(a, stream);
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const long long cols = (a.n_ch / 8 + kConvThreads - 1) / kConvThreads;
    if (a.n_tok / 8 * cols <= (long long)kShortRuns * sms) return launch_run<TYPE, W, 8>(a, stream);
    return launch_run<TYPE, W, 32>(a, stream);
}

template <int TYPE>
cudaError_t launch_type(const ConvArgs& a, cudaStream_t stream) {
    return a.width == 4 ? launch_width<TYPE, 4>(a, stream) : a.width == 3 ? launch_width<TYPE, 3>(a, stream)
                                                                          : launch_width<TYPE, 2>(a, stream);
}

}  // namespace

// Blocks of the runs of 32 tokens, which many tokens are cut into.
bool short_conv_fits(long long n_tok, long long n_ch) {
    return (n_tok + 31) / 32 * ((n_ch / 8 + kConvThreads - 1) / kConvThreads) <= 0x7fffffffLL;
}

cudaError_t launch_short_conv(const ConvArgs& a, cudaStream_t stream) {
    return a.type == QSA_F16 ? launch_type<QSA_F16>(a, stream) : launch_type<QSA_BF16>(a, stream);
}

}  // namespace qsa

// short_conv.cu -- short causal depthwise convolution over packed sequences,
// and its single-token step (gdn_short_conv, gdn_short_conv_step).
//
//   out[t, c] = act(bias[c] + sum_{j < K} w[c, j] x[t - K + 1 + j, c])
//
// with the K - 1 inputs before a sequence's first taken from its state.  Each
// input is read once and each output written once: 2 e bytes (e bytes per
// element) against 2 K flops, so both kernels are bound by HBM bandwidth and,
// for few tokens, by the latency of one load and one store.
//
// Over packed sequences a thread takes one word of four channels (two 16-bit
// elements or one element where the rows' alignment allows no more) through a
// run of consecutive tokens.  The last K - 1 inputs stay in registers, so only
// a run's start reads rows again (K - 1 rows per run, from L2).  The run's rows
// come through a ring in shared memory by asynchronous copies, 16 tokens ahead
// (8 with 16-byte words): 16 KB in flight per block without a register.
// Channels go in pairs through the packed fp32 instructions.
//
// Measured: 4000 tokens of 10240 bf16 channels, width 4, SiLU, 30 us, 82 % of
// the copy bandwidth.  What was tried beside it at this size: bf16 in words of
// 16 bytes, five blocks per SM, 8 tokens ahead, 35 us (98 registers a thread
// leave too few warps to cover a group's wait); 8-byte words with five, four
// and three blocks 33, 35 and 37; rows loaded into registers four ahead 49;
// runs of up to 96 tokens in place of 64, 33 (a longer last wave); weights
// staged in single floats 31.
// The step keeps 16-byte words: 256 sequences take 11 us for 42 MB, half of it
// the launch, the weights and the first loads.
#include <type_traits>

#include "block.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kStep = 4;   // tokens per group of copies
// Groups in flight: 24 KB of ring per block with 16-byte words, 20 KB with
// 8-byte ones, so that six blocks' rings stay on an SM.
template <int Bytes> constexpr int kAhead = Bytes == 16 ? 2 : 4;
template <int Bytes> constexpr int kRing = (kAhead<Bytes> + 1) * kStep;
// Blocks per SM that the registers are kept low for.  Above width 4 weights and
// inputs of all taps take too many for six: two, three and four took the same
// time at width 8 (4000 x 10240 bf16, 38 us now), short calls the least with two.
template <int K> constexpr int kBlocks = K <= 4 ? 6 : 2;

template <typename T> struct ConvArgs {
    const T *x;
    const float *weight, *bias;
    const int32_t *cu;
    const T *init;
    T *out, *fin;
    int N, T_, C;
    int64_t xs, os;
    int tx;          // threads along the channels (a power of two)
    int n_chan;      // blocks along the channels
    int run;         // tokens per thread
    int n_main;      // blocks of the convolution; the rest write states
    int first;       // number of this launch's first block
    bool act;
};

// The weights of this block's channels as [K][channels] in shared memory:
// read from [C, K] in order, so that the threads' own columns are not a
// strided walk over global memory, eight loads before their stores: all of
// them up to 32 weights a thread in 16-byte words.
template <int K, int V>
__device__ __forceinline__ void stage_words(float *sw, const float *from, int i0, int n, int width) {
    using Word = Vec<float, V>;
    for (i0 += threadIdx.x * V; i0 < n; i0 += 8 * kThreads * V) {
        Word w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i0 + k * kThreads * V < n) w[k] = Word::load(from + i0 + k * kThreads * V);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + k * kThreads * V;
            float v[V];
            w[k].to(v);
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (i < n) sw[(i + e) % K * width + (i + e) / K] = v[e];
        }
    }
}
template <int K>
__device__ __forceinline__ void stage_weights(float *sw, const float *w, int c0, int C, int width) {
    const int n = min(width, C - c0) * K;
    const float *from = w + (int64_t)c0 * K;
    const int whole = reinterpret_cast<uintptr_t>(from) % 16 == 0 ? n & ~3 : 0;
    stage_words<K, 4>(sw, from, 0, whole, width);
    if (whole < n) stage_words<K, 1>(sw, from, whole, n, width);
    __syncthreads();
}

// Input `pos` of the sequence that starts at token `start`: from the tokens,
// or from its state (positions start - K + 1 .. start - 1).
template <typename T, int V, int K>
__device__ __forceinline__ Vec<T, V> tap(const ConvArgs<T> &a, int n, int start, int pos, int c) {
    if (pos >= start) return Vec<T, V>::load(a.x + pos * a.xs + c);
    const int r = K - 1 + pos - start;
    if (!a.init || r < 0) return Vec<T, V>::zero();
    return Vec<T, V>::load(a.init + ((int64_t)n * (K - 1) + r) * a.C + c);
}

// The states after the sequences' last tokens.  One thread per sequence and
// word of channels reads all K - 1 rows before it writes the first, so that
// the new state may replace the old one.
template <typename T, int V, int K>
__device__ __forceinline__ void write_state(const ConvArgs<T> &a, int64_t i) {
    const int nv = a.C / V;
    if (i >= (int64_t)a.N * nv) return;
    const int n = (int)(i / nv), c = (int)(i % nv) * V;
    const int start = min(max(a.cu[n], 0), a.T_), end = min(max(a.cu[n + 1], start), a.T_);
    Vec<T, V> rows[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
        rows[j] = tap<T, V, K>(a, n, start, end - (K - 1) + j, c);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) rows[j].store(a.fin + ((int64_t)n * (K - 1) + j) * a.C + c);
}

template <typename T, int V, int K>
__global__ void __launch_bounds__(kThreads, kBlocks<K>) gdn_short_conv_kernel(const ConvArgs<T> a) {
    constexpr int P = (V + 1) / 2;  // pairs of channels
    extern __shared__ __align__(16) float sw[];
    const int blk = blockIdx.x + a.first;
    if (blk >= a.n_main) {
        write_state<T, V, K>(a, (int64_t)(blk - a.n_main) * kThreads + threadIdx.x);
        return;
    }
    const int tx = threadIdx.x & (a.tx - 1), ty = threadIdx.x / a.tx;
    const int c0 = (blk % a.n_chan) * a.tx * V, c = c0 + tx * V;
    const int64_t first = ((int64_t)(blk / a.n_chan) * (kThreads / a.tx) + ty) * a.run;
    const bool live = c < a.C && first < a.T_;
    const int t0 = live ? (int)first : 0;
    const int t1 = live ? (int)min(first + a.run, (int64_t)a.T_) : 0;

    // A ring of this thread's words: kGroups groups of kStep tokens on their
    // way while one is computed.  A thread reads only what it copied itself,
    // so its own wait is all the synchronisation needed.  (A single 16-bit
    // element comes as the aligned 4-byte word that holds it, without the
    // upper half where that is not needed.)
    using Word = Vec<T, V>;
    using Slot = std::conditional_t<sizeof(Word) == 2, uint32_t, Word>;
    constexpr int kGroups = kAhead<sizeof(Slot)>, kSlots = kRing<sizeof(Slot)>;
    Slot *ring = reinterpret_cast<Slot *>(sw + a.tx * V * K) + threadIdx.x;
    const T *ahead = a.x + t0 * a.xs + c;  // where copies go on
    int ahead_t = t0, ahead_slot = 0;
    auto issue = [&](bool first) {
        Slot *to = ring + ahead_slot * kThreads;
        auto copy = [&](int u) {
            if constexpr (sizeof(Word) == 2)
                copy_async_element(to + u * kThreads, ahead, odd(ahead), first && u == 0);
            else
                copy_async<sizeof(Word)>(to + u * kThreads, ahead);
            ahead += a.xs;
        };
#pragma unroll
        for (int u = 0; u < kStep; ++u)
            if (ahead_t + u < t1) copy(u);
        ahead_t += kStep;
        ahead_slot = ahead_slot + kStep == kSlots ? 0 : ahead_slot + kStep;
        copies_commit();
    };
    auto arrived = [&](int t, int slot) {
        const Slot v = ring[slot * kThreads];
        if constexpr (sizeof(Word) == 2) {
            const T *from = a.x + t * a.xs + c;
            const uint16_t half = (uint16_t)(odd(from) ? v >> 16 : v);
            return *reinterpret_cast<const Word *>(&half);
        } else {
            return v;
        }
    };
#pragma unroll
    for (int g = 0; g < kGroups; ++g) issue(g == 0 && t0 == 0 && c == 0);

    // Then, while they come: the sequence, the inputs before the run, the weights.
    Span s{};
    uint64_t in[K][P];  // the K - 1 inputs before a token, and the token's
    if (live) {
        s = locate(a.cu, a.N, a.T_, t0);
        Word word[K - 1];
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            word[j] = tap<T, V, K>(a, s.n, s.start, t0 - (K - 1) + j, c);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) to_pairs<V>(word[j], in[j]);
    }
    stage_weights<K>(sw, a.weight, c0, a.C, a.tx * V);
    if (!live) return;
    uint64_t w[K][P], b[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const float *wj = sw + j * a.tx * V + tx * V;
            w[j][i] = pack2f(wj[2 * i], V > 1 ? wj[2 * i + 1] : 0.f);
        }
        b[i] = a.bias ? pack2f(a.bias[c + 2 * i], V > 1 ? a.bias[c + 2 * i + 1] : 0.f) : 0;
    }
    T *to = a.out + t0 * a.os + c;
    auto token = [&](int t, int slot) {
        to_pairs<V>(arrived(t, slot), in[K - 1]);
        uint64_t sum[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            sum[i] = b[i];
#pragma unroll
            for (int j = 0; j < K; ++j) sum[i] = ffma2(w[j][i], in[j][i], sum[i]);
            if (a.act) sum[i] = silu2(sum[i]);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) in[j][i] = in[j + 1][i];
        }
        float y[V];
        from_pairs<V>(sum, y);
        Word::from(y).store(to);
        to += a.os;
    };
    if (sizeof(Word) == 2 && t0 == 0 && c == 0) load_first(ring, a.x);
    int slot = 0;
    for (int t = t0; t < t1; t += kStep) {
        copies_wait<kGroups - 1>();
        if (t + kStep <= min(s.end, t1)) {
#pragma unroll
            for (int u = 0; u < kStep; ++u) token(t + u, slot + u);
        } else {
            const int te = min(t + kStep, t1);
#pragma unroll 1
            for (int tok = t; tok < te; ++tok) {
                if (tok >= s.end) {  // the next sequence: its state comes before its tokens
                    s = next_span(a.cu, a.N, a.T_, s);
#pragma unroll
                    for (int j = 0; j < K - 1; ++j)
                        to_pairs<V>(tap<T, V, K>(a, s.n, s.start, tok - (K - 1) + j, c), in[j]);
                }
                token(tok, slot + tok - t);
            }
        }
        slot = slot + kStep == kSlots ? 0 : slot + kStep;
        issue(false);
    }
}

template <typename T> struct StepArgs {
    const T *x;
    const float *weight, *bias;
    const T *state;
    T *out, *next;
    int N, C;
    int64_t xs, os;
    int tx, n_chan, run;
    bool act;
};

template <typename T, int V, int K>
__global__ void __launch_bounds__(kThreads) gdn_short_conv_step_kernel(const StepArgs<T> a) {
    extern __shared__ float sw[];
    const int tx = threadIdx.x & (a.tx - 1), ty = threadIdx.x / a.tx;
    const int c0 = (blockIdx.x % a.n_chan) * a.tx * V, c = c0 + tx * V;
    const int64_t first = ((int64_t)(blockIdx.x / a.n_chan) * (kThreads / a.tx) + ty) * a.run;
    const int last = c < a.C ? (int)min(first + a.run, (int64_t)a.N) : 0;
    // The next sequence's rows are loaded before the one at hand is computed,
    // the first one's before the weights.
    using Word = Vec<T, V>;
    Word rows[K];
    auto fetch = [&](Word (&into)[K], int64_t n) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            into[j] = Word::load(a.state + (n * (K - 1) + j) * a.C + c);
        into[K - 1] = Word::load(a.x + n * a.xs + c);
    };
    if (first < last) fetch(rows, first);
    float bias[V];
#pragma unroll
    for (int v = 0; v < V; ++v) bias[v] = a.bias && first < last ? a.bias[c + v] : 0.f;
    stage_weights<K>(sw, a.weight, c0, a.C, a.tx * V);
    for (int n = (int)first; n < last; ++n) {
        Word ahead[K];
        if (n + 1 < last) fetch(ahead, n + 1);
        float y[V];
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = bias[v];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            float r[V];
            rows[j].to(r);
#pragma unroll
            for (int v = 0; v < V; ++v)
                y[v] = fmaf(sw[j * a.tx * V + tx * V + v], r[v], y[v]);
        }
        if (a.act)
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] = silu(y[v]);
        Word::from(y).store(a.out + n * a.os + c);
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            rows[j + 1].store(a.next + ((int64_t)n * (K - 1) + j) * a.C + c);
        if (n + 1 < last)
#pragma unroll
            for (int j = 0; j < K; ++j) rows[j] = ahead[j];
    }
}

// Threads along the channels: the words of a row, up to `most`.
int threads_along(int words, int most) {
    int tx = 1;
    while (tx < words && tx < most) tx *= 2;
    return tx;
}

template <typename T, int V, int K>
gdn_status run_conv(const gdn_conv_problem &p, const void *x, const float *weight,
                    const float *bias, const int32_t *cu, const void *init, void *out, void *fin,
                    cudaStream_t stream) {
    ConvArgs<T> a;
    a.x = static_cast<const T *>(x);
    a.weight = weight;
    a.bias = bias;
    a.cu = cu;
    a.init = static_cast<const T *>(init);
    a.out = static_cast<T *>(out);
    a.fin = static_cast<T *>(fin);
    a.N = p.num_seqs;
    a.T_ = (int)p.total_tokens;
    a.C = p.channels;
    a.xs = p.x_stride;
    a.os = p.out_stride;
    a.act = p.activation == GDN_ACT_SILU;
    const int words = p.channels / V;
    a.tx = threads_along(words, kThreads);
    a.n_chan = (words + a.tx - 1) / a.tx;
    const int ty = kThreads / a.tx;
    // Tokens per thread: long runs read fewer rows twice (K - 1 of each
    // run), short ones make enough blocks for the GPU.
    auto blocks = [&](int run) {
        return (int64_t)a.n_chan * ((p.total_tokens + (int64_t)run * ty - 1) / ((int64_t)run * ty));
    };
    // One wave of blocks with runs of up to 64 tokens, or so many full waves.
    const int64_t slots = kBlocks<K> * kGridSms;
    const int64_t each = (p.total_tokens * a.n_chan + slots * ty - 1) / (slots * ty);
    const int64_t waves = (each + 63) / 64;
    a.run = (int)((each + waves - 1) / (waves > 0 ? waves : 1));
    a.run = a.run < 1 ? 1 : a.run;
    const int64_t n_main = blocks(a.run);
    const int64_t n_state =
        fin ? ((int64_t)p.num_seqs * words + kThreads - 1) / kThreads : 0;
    if (n_main + n_state > INT32_MAX) return GDN_ERR_UNSUPPORTED;
    a.n_main = (int)n_main;
    // (40 KB at most, in fp32 at width 8: 16 of weights and 24 of ring.)
    constexpr int kSlot = sizeof(T) * V < 4 ? 4 : sizeof(T) * V;
    static_assert((kThreads * V * K * 4 + kRing<kSlot> * kThreads * kSlot) <= 48 * 1024);
    const size_t smem = (size_t)a.tx * V * K * sizeof(float) + kRing<kSlot> * kThreads * kSlot;
    // A state written in place must not replace what another block still
    // reads: its blocks then run as a launch of their own.
    const bool apart = fin && fin == init;
    a.first = 0;
    const int64_t together = n_main + (apart ? 0 : n_state);
    if (together > 0) gdn_short_conv_kernel<T, V, K><<<(unsigned)together, kThreads, smem, stream>>>(a);
    if (apart && n_state > 0) {
        a.first = a.n_main;
        gdn_short_conv_kernel<T, V, K><<<(unsigned)n_state, kThreads, smem, stream>>>(a);
    }
    return launch_status();
}

template <typename T, int V, int K>
gdn_status run_step(const gdn_conv_problem &p, const void *x, const float *weight,
                    const float *bias, const void *state, void *out, void *next,
                    cudaStream_t stream) {
    StepArgs<T> a;
    a.x = static_cast<const T *>(x);
    a.weight = weight;
    a.bias = bias;
    a.state = static_cast<const T *>(state);
    a.out = static_cast<T *>(out);
    a.next = static_cast<T *>(next);
    a.N = p.num_seqs;
    a.C = p.channels;
    a.xs = p.x_stride;
    a.os = p.out_stride;
    a.act = p.activation == GDN_ACT_SILU;
    const int words = p.channels / V;
    a.tx = threads_along(words, kThreads);
    a.n_chan = (words + a.tx - 1) / a.tx;
    const int ty = kThreads / a.tx;
    auto blocks = [&](int run) {
        return (int64_t)a.n_chan * ((p.num_seqs + (int64_t)run * ty - 1) / ((int64_t)run * ty));
    };
    // Sequences per thread: as many, up to 8, as leave four blocks per SM, or
    // hardly fewer.  (300 sequences of 6144: 2 8.2 us, 3 6.6, 4 7.0, 8 8.7;
    // 256 of 10240: 2 11.3, 4 10.3, 6 11.0; 512 of 8192: 4 16.2, 6 14.5, 8 15.5.)
    a.run = 8;
    while (a.run > 1 && blocks(a.run) * 50 < 4 * kGridSms * 49) --a.run;
    if (blocks(a.run) > INT32_MAX) return GDN_ERR_UNSUPPORTED;
    gdn_short_conv_step_kernel<T, V, K>
        <<<(unsigned)blocks(a.run), kThreads, (size_t)a.tx * V * K * sizeof(float), stream>>>(a);
    return launch_status();
}

// run<T, V, K>: the word by the rows' alignment, K by the width.
#define GDN_CONV_WIDTHS(run, T, V)                        \
    switch (p.width) {                                    \
        case 2: return run<T, V, 2>(GDN_CONV_ARGS);       \
        case 3: return run<T, V, 3>(GDN_CONV_ARGS);       \
        case 4: return run<T, V, 4>(GDN_CONV_ARGS);       \
        case 5: return run<T, V, 5>(GDN_CONV_ARGS);       \
        case 6: return run<T, V, 6>(GDN_CONV_ARGS);       \
        case 7: return run<T, V, 7>(GDN_CONV_ARGS);       \
        case 8: return run<T, V, 8>(GDN_CONV_ARGS);       \
    }                                                     \
    return GDN_ERR_UNSUPPORTED;
#define GDN_CONV_DISPATCH(run, T, wide, word)             \
    if (word == wide) {                                   \
        GDN_CONV_WIDTHS(run, T, wide)                     \
    }                                                     \
    if constexpr (sizeof(T) == 2)                         \
        if (word == 2) {                                  \
            GDN_CONV_WIDTHS(run, T, 2)                    \
        }                                                 \
    GDN_CONV_WIDTHS(run, T, 1)

// The word of rows of x and out, and of contiguous states: `wide` elements
// where the alignment allows, two 16-bit elements, or one element.
template <typename T>
int conv_word(int wide, const gdn_conv_problem &p, const void *x, const void *out, const void *a,
              const void *b) {
    const uint64_t bits = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out) |
                          reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |
                          (uint64_t)p.x_stride * sizeof(T) | (uint64_t)p.out_stride * sizeof(T) |
                          (uint64_t)p.channels * sizeof(T);
    return bits % (wide * sizeof(T)) == 0 ? wide : sizeof(T) == 2 && bits % 4 == 0 ? 2 : 1;
}

template <typename T>
gdn_status conv_typed(const gdn_conv_problem &p, const void *x, const float *weight,
                      const float *bias, const int32_t *cu, const void *init, void *out,
                      void *fin, cudaStream_t stream) {
    // Four elements, so 8 bytes of bf16: their few registers let six blocks
    // stay on an SM.
    const int word = conv_word<T>(4, p, x, out, init, fin);
#define GDN_CONV_ARGS p, x, weight, bias, cu, init, out, fin, stream
    GDN_CONV_DISPATCH(run_conv, T, 4, word)
#undef GDN_CONV_ARGS
}

template <typename T>
gdn_status step_typed(const gdn_conv_problem &p, const void *x, const float *weight,
                      const float *bias, const void *state, void *out, void *next,
                      cudaStream_t stream) {
    const int word = conv_word<T>(kWide<T>, p, x, out, state, next);
#define GDN_CONV_ARGS p, x, weight, bias, state, out, next, stream
    GDN_CONV_DISPATCH(run_step, T, kWide<T>, word)
#undef GDN_CONV_ARGS
}

}  // namespace

gdn_status launch_short_conv(const gdn_conv_problem &p, const void *x, const float *weight,
                             const float *bias, const int32_t *cu, const void *init, void *out,
                             void *fin, cudaStream_t stream) {
    return p.dtype == GDN_BF16
               ? conv_typed<__nv_bfloat16>(p, x, weight, bias, cu, init, out, fin, stream)
               : conv_typed<float>(p, x, weight, bias, cu, init, out, fin, stream);
}

gdn_status launch_short_conv_step(const gdn_conv_problem &p, const void *x, const float *weight,
                                  const float *bias, const void *state, void *out, void *next,
                                  cudaStream_t stream) {
    return p.dtype == GDN_BF16
               ? step_typed<__nv_bfloat16>(p, x, weight, bias, state, out, next, stream)
               : step_typed<float>(p, x, weight, bias, state, out, next, stream);
}

}  // namespace gdn

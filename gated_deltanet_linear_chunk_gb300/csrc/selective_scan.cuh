// selective_scan.cuh -- selective state space scan over packed sequences, and
// its single-token step (gdn_selective_scan, gdn_selective_scan_step): the
// kernels of one element type, instantiated in selective_scan_bf16.cu and
// selective_scan_f32.cu.
//
// Per sequence and channel d, with S states and s_t = softplus(dt_t + bias):
//
//   h_t = exp(s_t A) h_{t-1} + s_t x_t B_t,   y_t = C_t . h_t + skip x_t
//   out_t = y_t silu(z_t)
//
// The decay differs per channel and state, so no matrix product carries the
// recurrence: each (token, channel, state) costs one exponential and four
// fp32 operations (s A, (s x) B, the update of h, the sum with C), against
// 8 / S bytes of bf16 x, dt, z and out.  At S = 16 the arithmetic takes
// longer than the memory traffic.
//
// A thread walks the tokens in order with CH channels and all their states in
// registers, so the sums over the states need no exchange between lanes, and
// each B and C read from shared memory serves CH channels.  States go in
// pairs through the packed fp32 instructions.  B and C, the same for all
// channels of a group, are staged in shared memory as fp32; x, dt, z and the
// raw B and C arrive by asynchronous copies one tile of tokens ahead.
//
// D channels fill few threads, so the packed tokens are cut into W windows of
// equal length, whatever sequences they hold:
//   1. every window but the last: the state that its last sequence reaches at
//      the window's end, if that sequence goes on, starting from zero (or from
//      the sequence's own initial state if it starts in the window), and the
//      sum of its steps there;
//   2. the states entering the windows, in order: c <- exp(A sum s) c + h
//      (one exponential per state for a whole window, because the decays of
//      successive tokens multiply);
//   3. the outputs of every window.
// Windows of a fixed length balance exactly, and a window whose end falls
// between two sequences skips step 1.
//
// Infinities and NaN: with fewer states than registers for them, or without a
// skip, zeros that stand for what is not there would meet them.  A thread whose
// states show that one has passed takes its window's tokens again (scan_again).
//
// Measured, 4000 tokens of 6144 channels and 16 states in bf16: 74 us for step 1,
// 10 for step 2, 108 for step 3, 181 in all (they overlap at their ends): 393 M
// (token, channel, state) elements at 11.6 per clock and SM in step 3.  Issue
// slots are 58 % busy, the fp32 pipe 55 %, the exponentials' pipe 59 and 45 %
// (it takes 32 per clock and SM, fp32 128), memory 21 %: 199 instructions per
// token of two channels, 96 of them the recurrence.  The bytes alone would
// take 29 us, step 3's fp32 operations 42.
#pragma once

#include "block.cuh"
#include "sm103.cuh"

namespace gdn {
namespace {

constexpr int kMaxThreads = 128;
constexpr int kUnroll = 4;      // tokens in flight per thread

// NS: the states padded to a power of two (A = B = 0 beyond S: those states
// stay zero).  Two channels per thread, one where a channel's states and
// decay rates alone take 128 registers.  (4000 x 6144, 16 states, output pass:
// two channels in three blocks per SM 113 us, four in two blocks 143, one in
// six 176, where B and C are read twice as often.  1536 channels, 8 states:
// two channels 42 us the whole call, four 54.)
template <int NS> constexpr int kChannels = NS <= 32 ? 2 : 1;
// Blocks of kMaxThreads per SM.  Three leave 168 registers, with which the
// four tokens of a run overlap; four blocks (128 registers) took 8 % longer,
// two 10 %.
template <int NS> constexpr int kResident = NS <= 16 ? 3 : 2;
// Tokens per shared-memory tile, and tiles: one is computed, the others are on
// their way.
template <typename T, int CH> constexpr int kTileOf = sizeof(T) * CH <= 4 ? 16 : 8;
template <typename T, int CH> constexpr int kTilesOf = CH == 2 ? 2 : 3;

template <typename T> struct ScanArgs {
    const T *x, *dt, *B, *C, *z;
    const float *A, *skip, *bias;
    const int32_t *cu;
    const float *init;
    T *out;
    float *fin;
    float *carry;   // [W - 1, D, S]: state at each window's end, then entering the next
    float *steps;   // [W - 1, D]: sum of steps up to the window's end
    int N, T_, D, S, G;
    int per_group, tiles;  // channels per group, blocks per group
    int W, len;            // windows, tokens per window
    int64_t xs, dts, bs, cs, zs, os;
    int bc_word;  // CopyWord of B and C
    bool softplus, defer;
    bool out_own;      // out's rows are aligned to a thread's channels
    bool state_words;  // A, the states and the workspace allow 16-byte words
};

// A thread's channels and all their states.
template <typename T, int NS> struct ScanThread {
    static constexpr int CH = kChannels<NS>;
    static constexpr int NP = NS / 2;
    uint64_t A[CH][NP], h[CH][NP];
    uint64_t bias, skip, sum;  // of both channels; of one and zero where CH = 1
    int d, col;  // first channel: in the tensors, in the block
    int valid;   // channels that exist

    __device__ __forceinline__ void setup(const ScanArgs<T> &a, int group, int in_group0) {
        col = threadIdx.x * CH;
        d = group * a.per_group + in_group0 + col;
        valid = min(max(a.per_group - in_group0 - col, 0), CH);
        auto both = [&](const float *p) {
            return pack2f(p && valid > 0 ? p[d] : 0.f, p && valid > 1 ? p[d + 1] : 0.f);
        };
        bias = both(a.bias);
        skip = both(a.skip);
        sum = 0;
        read(a, a.A, 0, kLog2e, A);
    }
    // This thread's part of row `row` of a [rows, D, S] array (zeros where it
    // has none), in 16-byte words where the array allows.
    __device__ __forceinline__ void read(const ScanArgs<T> &a, const float *from, int64_t row,
                                         float scale, uint64_t (&to)[CH][NP]) const {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const float *p0 = from + (row * a.D + d + c) * a.S;
#pragma unroll
            for (int k = 0; k < NS; k += 4) {
                float v[4] = {0.f, 0.f, 0.f, 0.f};
                if (a.state_words) {
                    if (from && c < valid && k < a.S) Vec<float, 4>::load(p0 + k).to(v);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (from && c < valid && k + i < a.S) v[i] = p0[k + i];
                }
                to[c][k / 2] = pack2f(scale * v[0], scale * v[1]);
                to[c][k / 2 + 1] = pack2f(scale * v[2], scale * v[3]);
            }
        }
    }
    __device__ __forceinline__ void load(const ScanArgs<T> &a, const float *from, int64_t row) {
        read(a, from, row, 1.f, h);
    }
    __device__ __forceinline__ void store(const ScanArgs<T> &a, float *to, int64_t row) const {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float *p0 = to + (row * a.D + d + c) * a.S;
            if (c >= valid) continue;
#pragma unroll
            for (int k = 0; k < NS; k += 4) {
                const float2 u = unpack2f(h[c][k / 2]), w = unpack2f(h[c][k / 2 + 1]);
                const float v[4] = {u.x, u.y, w.x, w.y};
                if (a.state_words) {
                    if (k < a.S) Vec<float, 4>::from(v).store(p0 + k);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (k + i < a.S) p0[k + i] = v[i];
                }
            }
        }
    }
    // The state after sequence n's last token in window w.  A final state written
    // over the initial one must wait for the windows that read it: it takes the
    // place of the state that entered this window, copied by a last launch.
    __device__ __forceinline__ void finish(const ScanArgs<T> &a, int n, bool from_carry,
                                           int w) const {
        if (a.fin && from_carry && a.defer) store(a, a.carry, w - 1);
        else if (a.fin) store(a, a.fin, n);
    }
    // Whether a step times x that was not finite has passed: a padding state (of
    // S < NS states the last) is then NaN, a state infinite or NaN, and stays so.
    __device__ __forceinline__ bool spoiled(int S) const {
        bool r = false;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const float first = unpack2f(h[c][0]).x, last = unpack2f(h[c][NP - 1]).y;
            r |= c < valid && !((S < NS ? last : 0.f * first) == 0.f);
        }
        return r;
    }
    // One token: x and dt of the channels, B and C of the group; returns C . h.
    // EXACT: the padding states are kept at zero whatever x and dt are.
    template <bool OUT, bool EXACT = false>
    __device__ __forceinline__ uint64_t token(bool softplus_on, uint64_t x, uint64_t dt,
                                              const float *sB, const float *sC, int S = NS) {
        // (A choice, not a branch: the tokens of a run are one basic block,
        // which the compiler can interleave.)
        const uint64_t v = fadd2(dt, bias), sp = softplus2(v), s = softplus_on ? sp : v;
        if (!OUT) sum = fadd2(sum, s);
        const float2 s1 = unpack2f(s), u1 = unpack2f(fmul2(s, x));
        uint64_t s2[CH], u2[CH], y2[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            s2[c] = c ? pack2f(s1.y, s1.y) : pack2f(s1.x, s1.x);
            u2[c] = c ? pack2f(u1.y, u1.y) : pack2f(u1.x, u1.x);
            y2[c] = 0;
        }
#pragma unroll
        for (int k = 0; k < NS; k += 4) {
            const ulonglong2 b4 = *reinterpret_cast<const ulonglong2 *>(sB + k);
            ulonglong2 c4 = {0, 0};
            if (OUT) c4 = *reinterpret_cast<const ulonglong2 *>(sC + k);
            const uint64_t b[2] = {b4.x, b4.y}, cc[2] = {c4.x, c4.y};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const int p = k / 2 + i;
                    const float2 e = unpack2f(fmul2(s2[c], A[c][p]));
                    h[c][p] = ffma2(pack2f(ex2(e.x), ex2(e.y)), h[c][p], fmul2(u2[c], b[i]));
                    if (EXACT) {
                        const float2 f = unpack2f(h[c][p]);
                        h[c][p] = pack2f(2 * p < S ? f.x : 0.f, 2 * p + 1 < S ? f.y : 0.f);
                    }
                    if (OUT) y2[c] = ffma2(cc[i], h[c][p], y2[c]);
                }
        }
        const float2 y0 = unpack2f(y2[0]), y1 = unpack2f(y2[CH - 1]);
        return pack2f(y0.x + y0.y, CH > 1 ? y1.x + y1.y : 0.f);
    }
};

// How rows may be copied into shared memory: whole 16-byte words, 4-byte
// words, or element by element (16-bit rows at odd elements).
enum CopyWord : int { kCopy16 = 16, kCopy4 = 4, kCopyElement = 0 };

// Lanes that share a row of `words` copies: a power of two, as its logarithm.
__device__ __forceinline__ int row_lanes(int words) { return words > 16 ? 5 : 32 - __clz(words - 1); }

// `rows` rows of `cols` elements from `src` (rows `stride` apart) to `dst`
// (rows `pitch` apart): 2^lg lanes take a row's words.
template <typename T>
__device__ __forceinline__ void copy_rows(T *dst, int pitch, const T *src, int64_t stride,
                                          int rows, int cols, int word, int lg) {
    const int lane = threadIdx.x & ((1 << lg) - 1), first = threadIdx.x >> lg;
    const int apart = blockDim.x >> lg;
    if (word == kCopyElement) {
        // Four rows' loads before the first store.
        for (int c = lane; c < cols; c += 1 << lg)
            for (int r0 = first; r0 < rows; r0 += 4 * apart) {
                T v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (r0 + k * apart < rows) v[k] = src[(r0 + k * apart) * stride + c];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (r0 + k * apart < rows) dst[(r0 + k * apart) * pitch + c] = v[k];
            }
        return;
    }
    const int step = word == kCopy16 ? kWide<T> : 4 / (int)sizeof(T);
    for (int c = lane * step; c < cols; c += step << lg) {
        int r = first;
        const T *from = src + r * stride + c;
        T *to = dst + r * pitch + c;
        const int64_t next = apart * stride;
#pragma unroll 4
        for (; r < rows; r += apart, from += next, to += apart * pitch) {
            if (word == kCopy16) copy_async<16>(to, from);
            else copy_async<4>(to, from);
        }
    }
}

// Elements between p and the 16-byte word that holds it.
template <typename T> __device__ __forceinline__ int shift_of(const T *p) {
    return (int)(reinterpret_cast<uintptr_t>(p) / sizeof(T)) & (kWide<T> - 1);
}

// The same for rows at any alignment: element c of a row goes to place
// c + shift_of(row).  Whole 16-byte words from the one that holds the row's
// first element on, the last one's first bytes: what comes before the row is
// in the tensor too, the row before it or its own earlier columns.
template <typename T>
__device__ __forceinline__ void copy_rows_over(T *dst, int pitch, const T *src, int64_t stride,
                                               int rows, int cols, int lg) {
    constexpr int V = kWide<T>;
    const int lane = threadIdx.x & ((1 << lg) - 1), apart = blockDim.x >> lg;
    int r = threadIdx.x >> lg;
    const T *from = src + r * stride;
    T *to = dst + r * pitch;
    const int64_t next = apart * stride;
#pragma unroll 4
    for (; r < rows; r += apart, from += next, to += apart * pitch) {
        const int o = shift_of(from), n = o + cols;
        for (int k = lane * V; k < n; k += V << lg)
            copy_async_head(to + k, from - o + k, min(16, (n - k) * (int)sizeof(T)));
    }
}

// The same for a tensor's first tokens and channels, where nothing comes before:
// all but the row's ends in whole 16-byte words, the ends in 4-byte ones.  (A
// first 16-bit element in the upper half of its 4-byte word is left to
// copy_first.)
template <typename T>
__device__ __forceinline__ void copy_rows_shifted(T *dst, int pitch, const T *src, int64_t stride,
                                                  int rows, int cols) {
    constexpr int V = kWide<T>, E = 4 / (int)sizeof(T);  // elements per word
    const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
    for (int r = threadIdx.x / 32; r < rows; r += warps) {
        const T *from = src + r * stride;
        const int o = shift_of(from), lead = min((V - o) % V, cols);
        T *to = dst + r * pitch + o;
        const int words = (cols - lead) / V, tail = lead + words * V;
        for (int k = lane; k < words; k += 32)
            copy_async<16>(to + lead + k * V, from + lead + k * V);
        // Lanes 0 to 3 take the row's start, 4 to 7 its end.
        const int c = lane < 4 ? o % E + lane * E : tail + (lane - 4) * E;
        if (lane < 8 && c < (lane < 4 ? lead : cols)) {
            if constexpr (E == 1) copy_async<4>(to + c, from + c);
            else copy_async_part(to + c, from + c, c + 1 < cols ? 4 : 2);
        }
    }
}
template <typename T, int K>
__device__ __forceinline__ void copy_first(T *const (&dst)[K], int pitch, const T *const (&src)[K],
                                           const int64_t (&stride)[K], int rows) {
    for (int r = threadIdx.x; r < rows; r += blockDim.x) {
        T v[K];
        bool is[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            is[k] = src[k] && odd(src[k] + r * stride[k]);
            if (is[k]) v[k] = src[k][r * stride[k]];
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (is[k]) dst[k][r * pitch + shift_of(src[k] + r * stride[k])] = v[k];
    }
}

// Shared memory of a block: kTiles tiles of x, dt (and z) and of B (and C) as
// they lie in global memory, and one of B (and C) as fp32, zero past the last
// state.  SHIFT: rows of x, dt and z start anywhere.
template <typename T, int NS, bool OUT, bool SHIFT> struct ScanTiles {
    static constexpr int CH = kChannels<NS>;
    static constexpr int kTile = kTileOf<T, CH>, kTiles = kTilesOf<T, CH>;
    static constexpr int kIn = OUT ? 3 : 2, kBC = OUT ? 2 : 1;
    float *bc;     // [B, C][token][state]
    T *raws;       // the same, as loaded, of every tile
    T *ins;        // [x, dt, z][token][channel], of every tile
    int width;     // channels per block
    int pitch;     // elements between rows of `ins`
    int in_lanes, bc_lanes;  // that share a row, as logarithms
    __device__ ScanTiles(char *smem, int threads, int cols, int states, int bc_word)
        : width(threads * CH) {
        pitch = width + (SHIFT ? kWide<T> : 0);
        in_lanes = row_lanes((cols - 1 + (SHIFT ? kWide<T> - 1 : 0)) / kWide<T> + 1);
        bc_lanes = row_lanes(bc_word == kCopyElement ? states
                             : bc_word == kCopy16    ? (states - 1) / kWide<T> + 1
                                                     : (states - 1) / (4 / (int)sizeof(T)) + 1);
        bc = reinterpret_cast<float *>(smem);
        raws = reinterpret_cast<T *>(bc + kBC * kTile * NS);
        ins = raws + kTiles * kBC * kTile * NS;
    }
    // Tile `buf` (an offset, not an array of pointers: those would lose the
    // knowledge that they point to shared memory).
    __device__ __forceinline__ T *raw(int buf) const { return raws + buf * (kBC * kTile * NS); }
    __device__ __forceinline__ T *in(int buf) const { return ins + buf * (kIn * kTile * pitch); }
    static size_t bytes(int threads) {
        return kBC * kTile * NS * (sizeof(float) + kTiles * sizeof(T)) +
               kTiles * kIn * kTile * (threads * CH + (SHIFT ? kWide<T> : 0)) * sizeof(T);
    }
    // Starts the copies of tokens [t, te) (one tile at most) of the block's
    // channels, d the first of `cols`.
    __device__ __forceinline__ void load(const ScanArgs<T> &a, int buf, int t, int te, int d,
                                         int cols, int group) const {
        const int rows = min(te - t, kTile);
        const T *const src[3] = {a.x + t * a.xs + d, a.dt + t * a.dts + d,
                                 OUT && a.z ? a.z + t * a.zs + d : nullptr};
        const int64_t stride[3] = {a.xs, a.dts, a.zs};
        T *const dst[3] = {in(buf), in(buf) + kTile * pitch, in(buf) + 2 * kTile * pitch};
        // Whether a word that holds a row's first element may begin before the tensor.
        const bool start =
            t * min(min(a.xs, a.dts), OUT && a.z ? a.zs : a.xs) + d < kWide<T> - 1;
#pragma unroll
        for (int k = 0; k < kIn; ++k) {
            if (k == 2 && !a.z) break;
            if (!SHIFT) copy_rows(dst[k], pitch, src[k], stride[k], rows, cols, kCopy16, in_lanes);
            else if (!start) copy_rows_over(dst[k], pitch, src[k], stride[k], rows, cols, in_lanes);
            else copy_rows_shifted(dst[k], pitch, src[k], stride[k], rows, cols);
        }
        copy_rows(raw(buf), NS, a.B + t * a.bs + group * a.S, a.bs, rows, a.S, a.bc_word, bc_lanes);
        if (OUT)
            copy_rows(raw(buf) + kTile * NS, NS, a.C + t * a.cs + group * a.S, a.cs, rows, a.S,
                      a.bc_word, bc_lanes);
        if (SHIFT && start && sizeof(T) == 2) copy_first(dst, pitch, src, stride, rows);
    }
    // B and C of the tile that has arrived, to fp32.
    __device__ __forceinline__ void widen(const ScanArgs<T> &a, int buf) const {
        for (int i = threadIdx.x; i < kBC * kTile * NS; i += blockDim.x)
            bc[i] = i % NS < a.S ? to_f32(raw(buf)[i]) : 0.f;
    }
};

// U tokens from t of tile `buf`, whose first token is t0.  A byte each for x,
// dt and z: how far the tile's first row is shifted, and what a row adds.
template <typename T, int NS, bool OUT, bool SHIFT, int U>
__device__ __forceinline__ void scan_run(const ScanArgs<T> &a, ScanThread<T, NS> &th,
                                         const ScanTiles<T, NS, OUT, SHIFT> &tl, int buf, int t0,
                                         int t, uint32_t shifts, uint32_t steps) {
    constexpr int CH = kChannels<NS>, kTile = kTileOf<T, CH>;
    float y[U][CH];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = t - t0 + u;
        const T *in = tl.in(buf) + r * tl.pitch + th.col;
        const uint32_t o = SHIFT ? shifts + r * steps : 0;
        auto own = [&](int k) {
            const T *p = in + k * kTile * tl.pitch;
            float v[2] = {0.f, 0.f};
            if (SHIFT) {
#pragma unroll
                for (int c = 0; c < CH; ++c) v[c] = to_f32(p[c + (o >> (8 * k) & (kWide<T> - 1))]);
            } else {
                Vec<T, CH>::load(p).to(v);
            }
            return pack2f(v[0], v[1]);
        };
        const uint64_t x = own(0);
        const uint64_t sums = th.template token<OUT>(a.softplus, x, own(1), tl.bc + r * NS,
                                                     tl.bc + (kTile + r) * NS);
        if (OUT) {
            const uint64_t gate = silu2(own(2)), v = ffma2(th.skip, x, sums);
            const float2 f = unpack2f(a.z ? fmul2(v, gate) : v);
            y[u][0] = f.x;
            if (CH > 1) y[u][CH - 1] = f.y;
        }
    }
    if (!OUT) return;
    T *out = a.out + t * a.os + th.d;
    if (!SHIFT && a.out_own) {
#pragma unroll
        for (int u = 0; u < U; ++u, out += a.os)
            if (th.valid) Vec<T, CH>::from(y[u]).store(out);
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u, out += a.os)
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (c < th.valid) out[c] = from_f32<T>(y[u][c]);
    }
}

// Final states of empty sequences are their initial ones: rows of blocks of
// their own copy them, each every kEmptyRows-th sequence.
constexpr int kEmptyRows = 64;

template <typename T>
__device__ void copy_empty(const ScanArgs<T> &a, int first, int step, int d0, int cols) {
    for (int n = first; n < a.N; n += step) {
        if (a.cu[n + 1] > a.cu[n]) continue;
        const int64_t at = ((int64_t)n * a.D + d0) * a.S;
        for (int i = threadIdx.x; i < cols * a.S; i += blockDim.x)
            a.fin[at + i] = a.init ? a.init[at + i] : 0.f;
    }
}

// This thread's channels of window w once more, from the first token `t` of a
// sequence's part in it, straight from global memory: the padding states are
// kept at zero and a missing skip is left out, so that tokens that are not
// finite give the definition's infinities; all others what scan_run gave.
// (A function of its own, called when a window is done: inside the loop over the
// tiles it cost the tokens that are finite 2 to 10 %, here 0 to 2.4; a check of
// every tile before its tokens 2 to 10.)
template <typename T, int NS>
__device__ __noinline__ void scan_again(const ScanArgs<T> &a, int w, int t, int group,
                                        int in_group0) {
    ScanThread<T, NS> th;
    const int t0 = w * a.len, t1 = min(t0 + a.len, a.T_);
    auto both = [&](const T *p, int64_t stride) {
        p += t * stride + th.d;
        return pack2f(to_f32(p[0]), th.valid > 1 ? to_f32(p[1]) : 0.f);
    };
    th.setup(a, group, in_group0);
    Span s = locate(a.cu, a.N, a.T_, t);
#pragma unroll 1
    while (true) {
        const bool from_carry = s.start < t0;
        th.load(a, from_carry ? a.carry : a.init, from_carry ? w - 1 : s.n);
#pragma unroll 1
        for (const int te = min(s.end, t1); t < te; ++t) {
            alignas(16) float b[NS], c[NS];
#pragma unroll 1  // (in local memory: the registers are the states')
            for (int k = 0; k < NS; ++k) {
                b[k] = k < a.S ? to_f32(a.B[t * a.bs + group * a.S + k]) : 0.f;
                c[k] = k < a.S ? to_f32(a.C[t * a.cs + group * a.S + k]) : 0.f;
            }
            const uint64_t x = both(a.x, a.xs);
            const uint64_t sums =
                th.template token<true, true>(a.softplus, x, both(a.dt, a.dts), b, c, a.S);
            const uint64_t v = a.skip ? ffma2(th.skip, x, sums) : sums;
            const float2 f = unpack2f(a.z ? fmul2(v, silu2(both(a.z, a.zs))) : v);
            T *out = a.out + t * a.os + th.d;
            out[0] = from_f32<T>(f.x);
            if (th.valid > 1) out[1] = from_f32<T>(f.y);
        }
        if (s.end <= t1) th.finish(a, s.n, from_carry, w);
        if (t >= t1) break;
        s = next_span(a.cu, a.N, a.T_, s);
    }
}

// GUARD: there are padding states, or there is no skip, whose zeros times an
// infinity are NaN: tokens with any are taken again without them.
template <typename T, int NS, bool OUT, bool SHIFT, bool GUARD>
__global__ void __launch_bounds__(kMaxThreads, kResident<NS>) gdn_scan_kernel(const __grid_constant__ ScanArgs<T> a) {
    constexpr int CH = kChannels<NS>, kTile = kTileOf<T, CH>, kTiles = kTilesOf<T, CH>;
    extern __shared__ __align__(16) char smem[];
    const int group = blockIdx.x / a.tiles;
    const int in_group0 = (blockIdx.x % a.tiles) * (int)blockDim.x * CH;
    const int w = blockIdx.y, d0 = group * a.per_group + in_group0;
    const int cols = min((int)blockDim.x * CH, a.per_group - in_group0);
    const ScanTiles<T, NS, OUT, SHIFT> tl(smem, blockDim.x, cols, a.S, a.bc_word);
    if (OUT && w >= a.W) {
        copy_empty(a, w - a.W, gridDim.y - a.W, d0, cols);
        return;
    }
    int t0 = w * a.len;
    const int t1 = min(t0 + a.len, a.T_);
    Span s;
    bool from_carry = false;
    if (OUT) {
        s = locate_by_warp(a.cu, a.N, a.T_, t0);
        from_carry = s.start < t0;
    } else {
        // The sequence that goes on past this window's end.
        s = locate_by_warp(a.cu, a.N, a.T_, t1 - 1);
        if (s.end <= t1) return;
        from_carry = s.start < t0;
        t0 = max(t0, s.start);
    }
    auto fetch = [&](int tile) {
        const int t = t0 + tile * kTile;
        if (t < t1) tl.load(a, tile % kTiles, t, t1, d0, cols, group);
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k < kTiles - 1; ++k) fetch(k);
    ScanThread<T, NS> th;
    th.setup(a, group, in_group0);
    if (OUT) ptx::griddep_wait();  // the carries: all above is input to the whole call
    if (from_carry) th.load(a, OUT ? a.carry : nullptr, w - 1);
    else th.load(a, a.init, s.n);
    // Before a sequence's state is left: whether its tokens here have to be taken
    // again, at the end.  From there on the thread writes nothing.
    int again = -1;
    auto leave = [&] {
        if (!GUARD || !th.spoiled(a.S)) return;
        again = max(t0, s.start);
        th.valid = 0;
    };
    Span next = OUT && s.end < t1 ? next_span(a.cu, a.N, a.T_, s) : s;

    for (int tile = 0, tt = t0; tt < t1; ++tile, tt += kTile) {
        const int te = min(tt + kTile, t1), buf = tile % kTiles;
        copies_wait<kTiles - 2>();
        __syncthreads();  // the tile has arrived, and the one before is done with
        tl.widen(a, buf);
        fetch(tile + kTiles - 1);
        uint32_t shifts = 0, steps = 0;
        if (SHIFT) {
            constexpr int M = kWide<T> - 1;
            shifts = shift_of(a.x + tt * a.xs + d0) | shift_of(a.dt + tt * a.dts + d0) << 8 |
                     shift_of(a.z + tt * a.zs + d0) << 16;
            steps = (a.xs & M) | (a.dts & M) << 8 | (a.zs & M) << 16;
        }
        __syncthreads();
        int t = tt;
        while (t < te) {
            const int e = min(te, s.end);
            for (; t + kUnroll <= e; t += kUnroll)
                scan_run<T, NS, OUT, SHIFT, kUnroll>(a, th, tl, buf, tt, t, shifts, steps);
            for (; t < e; ++t) scan_run<T, NS, OUT, SHIFT, 1>(a, th, tl, buf, tt, t, shifts, steps);
            if (OUT && t == s.end) {
                leave();
                th.finish(a, s.n, from_carry, w);
                if (t < t1) {
                    s = next;
                    th.load(a, a.init, s.n);
                    from_carry = false;
                    if (s.end < t1) next = next_span(a.cu, a.N, a.T_, s);
                }
            }
        }
    }
    if (OUT && s.end > t1) leave();
    if (GUARD && again >= 0) scan_again<T, NS>(a, w, again, group, in_group0);
    if (!OUT) {
        ptx::griddep_launch_dependents();
        th.store(a, a.carry, w);
        const float2 sum = unpack2f(th.sum);
        float *steps = a.steps + (int64_t)w * a.D + th.d;
        if (th.valid > 0) steps[0] = sum.x;
        if (th.valid > 1) steps[1] = sum.y;
    }
}

constexpr int kCombineThreads = 256;

// 2^(x / 2), the factor that a window or run multiplies a state by twice.  Whole
// windows of growing states (A or the steps may have any sign) pass what one
// fp32 factor holds while the state does not, above all a state that is still
// zero.  Within 2^-126 .. 2^127 neither factor is zero or infinite: a zero state
// stays zero and an infinite one infinite, and the two take any fp32 state past
// either end of the range.
__device__ __forceinline__ float half_factor(float x) {
    return ex2(fminf(fmaxf(0.5f * x, -126.f), 127.f));
}

// States entering the windows: in window order, c <- exp(A sum s) c + h, from
// the window's own state alone where its last sequence starts inside it.  The
// steps compose, (h, k) then (h', k') being (k' h + h', k k'), so a block cuts
// many windows into SEG runs, walks all runs at once from zero, joins them in
// shared memory and walks them again from the states that enter them.
template <typename T, int SEG>
__global__ void __launch_bounds__(kCombineThreads) gdn_scan_combine_kernel(const ScanArgs<T> a) {
    constexpr int E = kCombineThreads / SEG;  // states per block
    __shared__ float end[SEG][E], kept[SEG][E];
    extern __shared__ char inside[];  // [W - 1]
    ptx::griddep_launch_dependents();
    const int n = a.W - 1;
    for (int w = threadIdx.x; w < n; w += blockDim.x)
        inside[w] = locate(a.cu, a.N, a.T_, (w + 1) * a.len - 1).start >= w * a.len;
    const int e = threadIdx.x % E, seg = threadIdx.x / E, run = (n + SEG - 1) / SEG;
    const int64_t ds = (int64_t)a.D * a.S, i = (int64_t)blockIdx.x * E + e;
    const bool ok = i < ds;
    const float rate = ok ? kLog2e * a.A[i] : 0.f;
    const int d = (int)(i / a.S);
    const int w0 = seg * run, w1 = min(w0 + run, n);
    __syncthreads();
    ptx::griddep_wait();
    constexpr int kAhead = 8;  // windows loaded at once: only the products are sequential
    auto walk = [&](float c, bool write, float &steps, bool &fresh) {
        for (int w = w0; w < w1; w += kAhead) {
            float h[kAhead], s[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int at = min(w + k, w1 - 1);
                h[k] = ok ? a.carry[at * ds + i] : 0.f;
                s[k] = ok ? a.steps[(int64_t)at * a.D + d] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (w + k >= w1) break;
                if (inside[w + k]) fresh = true;
                steps += s[k];
                const float f = half_factor(rate * s[k]);
                c = inside[w + k] ? h[k] : fmaf(f, f * c, h[k]);
                if (write && ok) a.carry[(w + k) * ds + i] = c;
            }
        }
        return c;
    };
    float steps = 0.f, c = 0.f;
    bool fresh = false;  // a sequence starts in this run: nothing enters past it
    if (SEG > 1) {
        end[seg][e] = walk(0.f, false, steps, fresh);
        kept[seg][e] = fresh ? -1.f : half_factor(rate * steps);
        __syncthreads();
        for (int k = 0; k < seg; ++k)
            c = kept[k][e] < 0.f ? end[k][e] : fmaf(kept[k][e], kept[k][e] * c, end[k][e]);
    }
    walk(c, true, steps, fresh);
}

// In place: the final states that gdn_scan_kernel left in the carries.
template <typename T>
__global__ void __launch_bounds__(kCombineThreads) gdn_scan_deferred_kernel(const ScanArgs<T> a) {
    const int w = blockIdx.y + 1, t0 = w * a.len;
    const Span s = locate(a.cu, a.N, a.T_, t0);
    if (s.start >= t0 || s.end > min(t0 + a.len, a.T_)) return;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, ds = (int64_t)a.D * a.S;
    if (i < ds) a.fin[s.n * ds + i] = a.carry[(w - 1) * ds + i];
}

// ------------------------------------------------------------ single tokens
// One step reads and writes 8 bytes per state for one exponential and four
// fp32 operations: bound by HBM bandwidth.  A block takes tiles of 128
// channels, a thread per channel, and walks (tile, sequence) pairs; a pair's
// states are contiguous in memory whatever S is.  They come into a ring in
// shared memory by asynchronous copies, some pairs ahead and without
// registers; each thread updates its channel's states there, and the block
// writes them back in order.  The decay rates stay in registers while the tile
// does.  Every block of one wave takes the same number of pairs.
//
// Measured: 256 sequences of 6144 channels and 16 states, 42 us, 75 % of the
// copy bandwidth; 13 states 40 us (65 %), where lanes sharing a channel took 131.
constexpr int kStepThreads = 128;

template <typename T> struct ScanStepArgs {
    const T *x, *dt, *B, *C, *z;
    const float *A, *skip, *bias, *state;
    T *out;
    float *next;
    int N, D, S, per_group;
    int tiles;               // of kStepThreads channels per group
    int64_t pairs, run;      // (tile, sequence) pairs, and how many per block
    int64_t xs, dts, bs, cs, zs, os;
    bool softplus, words;    // words: every pair's states are whole 16-byte words
};

// NS: the states padded to a power of two, at least 4.
// Stages of the ring, and blocks per SM: 48 KB in flight or more.  (256 x 6144,
// 16 states: four stages of six blocks 42 us, three of eight 46, six of four
// 48, two of ten 45; 32 states: three of four 41, four of three 44; 64
// states: two of three 41, three of two 47.)
template <int NS> constexpr int kStepStages = NS <= 16 ? 4 : NS == 32 ? 3 : 2;
template <int NS> constexpr int kStepBlocks = NS <= 8 ? 8 : NS == 16 ? 6 : NS == 32 ? 4 : 3;
template <int NS> constexpr size_t step_bytes() {
    return (size_t)kStepStages<NS> * kStepThreads * NS * sizeof(float) + 4 * NS * sizeof(float);
}

// QUADS: S is a multiple of four, A aligned to it: states four at a time.
template <typename T, int NS, bool QUADS>
__global__ void __launch_bounds__(kStepThreads, kStepBlocks<NS>)
gdn_scan_step_kernel(const ScanStepArgs<T> a) {
    constexpr int STAGES = kStepStages<NS>;
    extern __shared__ __align__(16) float ring[];  // [stage][channel][S]
    float *bc = ring + STAGES * kStepThreads * NS;  // [pair parity][B, C][NS]
    const int t = threadIdx.x;
    const int64_t first = (int64_t)blockIdx.x * a.run, last = min(first + a.run, a.pairs);

    // A pair's place: pairs go through all sequences of a tile in turn.
    struct Place {
        int64_t n;
        int tile, g, d0, count;
    };
    auto place = [&](int64_t n, int tile) {
        const int in_group = (tile % a.tiles) * kStepThreads, g = tile / a.tiles;
        return Place{n, tile, g, g * a.per_group + in_group,
                     min(kStepThreads, a.per_group - in_group)};
    };
    auto after = [&](Place p) {
        if (p.n + 1 == a.N) return place(0, p.tile + 1);
        ++p.n;
        return p;
    };
    // The states of pair i, at p, on their way to its stage.  (They are read
    // and written once: neither should push anything out of L2.  Without the
    // hint 256 x 6144 x 16 52 us in place of 42, 128 sequences with 32 states 43
    // for 41, 64 with 64 45 for 41.)
    const uint64_t once = evict_first_policy();
    auto copy = [&](int64_t i, const Place &p) {
        if (i < last) {
            const float *from = a.state + (p.n * a.D + p.d0) * a.S;
            float *to = ring + (i % STAGES) * (kStepThreads * NS);
            const int n = p.count * a.S;
            if (a.words) {
                for (int k = 4 * t; k < n; k += 4 * kStepThreads)
                    copy_async_once(to + k, from + k, once);
            } else {
                for (int k = t; k < n; k += kStepThreads) copy_async<4>(to + k, from + k);
            }
        }
        copies_commit();
    };
    // A pair's other inputs: this thread's channel's, and one B or C.
    struct Inputs {
        float dt, x, z, bc;
    };
    auto fetch = [&](Inputs &f, const Place &p) {
        const int d = p.d0 + min(t, p.count - 1);
        f.dt = to_f32(a.dt[p.n * a.dts + d]);
        f.x = to_f32(a.x[p.n * a.xs + d]);
        f.z = a.z ? to_f32(a.z[p.n * a.zs + d]) : 0.f;
        // Threads 0 .. NS - 1 take B, the next NS take C.
        const int k = t % NS;
        f.bc = 0.f;
        if (t < 2 * NS && k < a.S)
            f.bc = to_f32(t < NS ? a.B[p.n * a.bs + p.g * a.S + k]
                                    : a.C[p.n * a.cs + p.g * a.S + k]);
    };

    Place at = place(first % a.N, (int)(first / a.N)), ahead = at;
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) {
        copy(first + k, ahead);
        ahead = after(ahead);
    }
    Inputs in;
    fetch(in, at);
    const int quads = a.S / 4;
    // Where a thread starts in its channel's quads, so that the eight threads
    // of a 16-byte access phase hit distinct banks whatever power of two
    // divides the channels' distance.
    const int share = min(quads & -quads, 8);
    const int turn = QUADS ? t / (8 / share) % share : 0;
    auto quad = [&](int j) { return j + turn < quads ? j + turn : j + turn - quads; };
    float A[NS], bias = 0.f, skip = 0.f;
    int tile = -1;
    for (int64_t i = first; i < last; ++i) {
        const bool mine = t < at.count;
        if (at.tile != tile) {
            tile = at.tile;
            const int d = at.d0 + min(t, at.count - 1);
            const float *from = a.A + (int64_t)d * a.S;
            bias = a.bias ? a.bias[d] : 0.f;
            skip = a.skip ? a.skip[d] : 0.f;
            if (QUADS) {
#pragma unroll
                for (int j = 0; j < NS / 4; ++j)
                    if (j < quads) Vec<float, 4>::load(from + 4 * quad(j)).to(A + 4 * j);
#pragma unroll
                for (int k = 0; k < NS; ++k) A[k] *= kLog2e;
            } else {
#pragma unroll
                for (int k = 0; k < NS; ++k) A[k] = k < a.S ? kLog2e * from[k] : 0.f;
            }
        }
        float *both = bc + (i & 1) * (2 * NS);
        if (t < 2 * NS) both[t] = in.bc;
        const Inputs now = in;
        copies_wait<STAGES - 2>();
        __syncthreads();  // the pair's states are here, the pair before is written back
        copy(i + STAGES - 1, ahead);
        ahead = after(ahead);
        const Place next = after(at);
        if (i + 1 < last) fetch(in, next);

        float s = now.dt + bias;
        if (a.softplus) s = softplus(s);
        const float u = s * now.x;
        float y = 0.f;
        float *stage = ring + (i % STAGES) * (kStepThreads * NS);
        float *own = stage + t * a.S;
        if (mine) {
            if (QUADS) {
#pragma unroll
                for (int j = 0; j < NS / 4; ++j) {
                    if (j >= quads) break;
                    const int k = 4 * quad(j);
                    float h[4], b[4], c[4];
                    Vec<float, 4>::load(own + k).to(h);
                    Vec<float, 4>::load(both + k).to(b);
                    Vec<float, 4>::load(both + NS + k).to(c);
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        h[v] = fmaf(ex2(s * A[4 * j + v]), h[v], u * b[v]);
                        y = fmaf(c[v], h[v], y);
                    }
                    Vec<float, 4>::from(h).store(own + k);
                }
            } else {
#pragma unroll
                for (int k = 0; k < NS; ++k) {
                    if (k >= a.S) break;
                    const float h = fmaf(ex2(s * A[k]), own[k], u * both[k]);
                    y = fmaf(both[NS + k], h, y);
                    own[k] = h;
                }
            }
            if (a.skip) y = fmaf(skip, now.x, y);
            if (a.z) y *= silu(now.z);
            a.out[at.n * a.os + at.d0 + t] = from_f32<T>(y);
        }
        __syncthreads();
        float *to = a.next + (at.n * a.D + at.d0) * a.S;
        const int n = at.count * a.S;
        if (a.words) {
            for (int k = 4 * t; k < n; k += 4 * kStepThreads)
                __stcs(reinterpret_cast<float4 *>(to + k), Vec<float, 4>::load(stage + k).w);
        } else {
            for (int k = t; k < n; k += kStepThreads) __stcs(to + k, stage[k]);
        }
        at = next;
    }
}

// ------------------------------------------------------------------ sizes
// How a problem is cut: the states' padded count, threads per block, blocks
// per group, windows and their length.
struct ScanPlan {
    int ns, threads, tiles, W, len;
};

// The shortest window.  (128 tokens of 1024 channels, us by windows: 1 35, 4 21,
// 8 14, 16 12.5, 24 12.2, 48 18; 64 tokens of 6144: 1 19.5, 4 21, 8 18, 24 24.)
constexpr int kMinWindow = 8;
// Windows whose states are joined in one run.  Up to twice as many windows of
// less than 16 tokens are not worth the runs: 512 tokens of 2048 channels, 33
// windows 25 us, 57 26; 512 of 1024, 33 windows 18.4, 64 20; 400 of 512 15, 50 17.
constexpr int kFewWindows = 33;

// kChannels and kResident of the variant that runs.
inline int channels_per_thread(int ns) { return ns <= 32 ? 2 : 1; }
inline int resident_blocks(int ns) { return ns <= 16 ? 3 : 2; }

inline ScanPlan scan_plan(const gdn_ssm_problem &p) {
    ScanPlan s;
    s.ns = 4;
    while (s.ns < p.state_dim) s.ns *= 2;
    const int ch = channels_per_thread(s.ns), resident = resident_blocks(s.ns);
    const int per_group = p.channels / p.num_groups;
    const int warps = (per_group + 32 * ch - 1) / (32 * ch);
    const int64_t short_enough = p.total_tokens / kMinWindow;
    // One wave of blocks of up to `most` warps.
    auto cut = [&](int most) {
        s.threads = 32 * (warps < most ? warps : most);
        s.tiles = (per_group + s.threads * ch - 1) / (s.threads * ch);
        return (int64_t)resident * kGridSms * (kMaxThreads / s.threads) /
               ((int64_t)p.num_groups * s.tiles);
    };
    int64_t W = cut(kMaxThreads / 32);
    // Two warps where that leaves fewer channels' threads idle and so gives
    // more windows: 35879 x 1246 in 2 groups, 91 windows for 76, 441 us for
    // 492; 48014 x 3232 in 4, 32 for 28, 815 for 919.  (Elsewhere they read B
    // and C more often: 60 x 3496 19 for 20.5; with 64 states 847 for 955
    // although 13 windows for 12.)
    if (s.ns <= 16 && W < short_enough) {
        const int64_t narrow = cut(2);
        if (narrow > W) W = narrow;
        else W = cut(kMaxThreads / 32);
    }
    W = W < short_enough ? W : short_enough;
    if (W > kFewWindows && W <= 2 * kFewWindows && p.total_tokens < 16 * W) W = kFewWindows;
    // Two windows do 1.4 times the work of one for twice the blocks, with two
    // more launches: not worth it (2000 x 128: 440 us against 538, 128 x 1024
    // 33 against 35, 4000 x 6144 1249 against 987).
    W = W < 3 ? 1 : W;
    const int64_t len = (p.total_tokens + W - 1) / W;
    s.len = (int)(len > 0 ? len : 1);
    s.W = (int)((p.total_tokens + s.len - 1) / s.len);
    return s;
}

template <typename T> ScanArgs<T> scan_args(const gdn_ssm_problem &p, const ScanPlan &pl) {
    ScanArgs<T> a{};
    a.N = p.num_seqs;
    a.T_ = (int)p.total_tokens;
    a.D = p.channels;
    a.S = p.state_dim;
    a.G = p.num_groups;
    a.per_group = p.channels / p.num_groups;
    a.tiles = pl.tiles;
    a.W = pl.W;
    a.len = pl.len;
    a.xs = p.x_stride;
    a.dts = p.dt_stride;
    a.bs = p.b_stride;
    a.cs = p.c_stride;
    a.zs = p.z_stride;
    a.os = p.out_stride;
    a.softplus = p.dt_softplus != 0;
    a.carry = static_cast<float *>(p.workspace);
    a.steps = a.carry + (int64_t)(pl.W > 1 ? pl.W - 1 : 0) * a.D * a.S;
    return a;
}

template <typename T, int NS, bool SHIFT, bool GUARD>
gdn_status run_scan(const ScanPlan &pl, const ScanArgs<T> &a, bool empties, cudaStream_t stream) {
    const unsigned blocks = (unsigned)(a.G * pl.tiles);
    const int64_t ds = (int64_t)a.D * a.S;
    const size_t in_bytes = ScanTiles<T, NS, false, SHIFT>::bytes(pl.threads);
    const size_t out_bytes = ScanTiles<T, NS, true, SHIFT>::bytes(pl.threads);
    static std::atomic<bool> done[kMaxDevices];
    if (!raise_shared_memory(
            done,
            {reinterpret_cast<const void *>(gdn_scan_kernel<T, NS, false, SHIFT, false>),
             reinterpret_cast<const void *>(gdn_scan_kernel<T, NS, true, SHIFT, GUARD>)},
            {ScanTiles<T, NS, false, SHIFT>::bytes(kMaxThreads),
             ScanTiles<T, NS, true, SHIFT>::bytes(kMaxThreads)}))
        return GDN_ERR_CUDA;
    // With several windows the second and third launch may start while the
    // one before ends; they wait for it before they touch the carries.
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = pl.W > 1 ? 1 : 0;
    if (pl.W > 1) {
        gdn_scan_kernel<T, NS, false, SHIFT, false>
            <<<dim3(blocks, pl.W - 1), pl.threads, in_bytes, stream>>>(a);
        if (launch_status() != GDN_OK) return GDN_ERR_CUDA;
        // Eight windows are loaded at once: more than a few rounds of them
        // are cut into runs.  (512 tokens of 2048 channels in 57 windows, the
        // whole call: 16 runs 29 us, 4 runs 26; 8000 of 256 in 128 windows: 35
        // and 33 us, 2000 of 128 in 128: 18.5 and 19.)
        const int runs = pl.W <= kFewWindows ? 1 : pl.W <= 2 * kFewWindows ? 4 : 16;
        const int64_t each = kCombineThreads / runs;
        cfg.gridDim = dim3((unsigned)((ds + each - 1) / each));
        cfg.blockDim = dim3(kCombineThreads);
        cfg.dynamicSmemBytes = pl.W - 1;
        if (cudaLaunchKernelEx(&cfg, runs == 16  ? gdn_scan_combine_kernel<T, 16>
                                     : runs == 4 ? gdn_scan_combine_kernel<T, 4>
                                                 : gdn_scan_combine_kernel<T, 1>, a) != cudaSuccess)
            return GDN_ERR_CUDA;
    }
    const unsigned rows = (unsigned)(pl.W + (empties ? (a.N < kEmptyRows ? a.N : kEmptyRows) : 0));
    if (rows > 0) {
        cfg.gridDim = dim3(blocks, rows);
        cfg.blockDim = dim3(pl.threads);
        cfg.dynamicSmemBytes = out_bytes;
        if (cudaLaunchKernelEx(&cfg, gdn_scan_kernel<T, NS, true, SHIFT, GUARD>, a) != cudaSuccess)
            return GDN_ERR_CUDA;
    }
    if (a.defer && pl.W > 1)
        gdn_scan_deferred_kernel<T>
            <<<dim3((unsigned)((ds + kCombineThreads - 1) / kCombineThreads), pl.W - 1),
               kCombineThreads, 0, stream>>>(a);
    return launch_status();
}

template <typename T, int NS>
gdn_status run_scan(const ScanPlan &pl, const ScanArgs<T> &a, bool shifted, bool empties,
                    cudaStream_t stream) {
    if (a.S < NS || !a.skip)
        return shifted ? run_scan<T, NS, true, true>(pl, a, empties, stream)
                       : run_scan<T, NS, false, true>(pl, a, empties, stream);
    return shifted ? run_scan<T, NS, true, false>(pl, a, empties, stream)
                   : run_scan<T, NS, false, false>(pl, a, empties, stream);
}

template <typename T>
gdn_status scan_typed(const gdn_ssm_problem &p, const void *x, const void *dt, const float *A,
                      const void *B, const void *C, const float *skip, const void *z,
                      const float *bias, const int32_t *cu, const float *init, void *out,
                      float *fin, cudaStream_t stream) {
    const ScanPlan pl = scan_plan(p);
    ScanArgs<T> a = scan_args<T>(p, pl);
    if ((int64_t)a.G * pl.tiles > INT32_MAX) return GDN_ERR_UNSUPPORTED;
    a.x = static_cast<const T *>(x);
    a.dt = static_cast<const T *>(dt);
    a.B = static_cast<const T *>(B);
    a.C = static_cast<const T *>(C);
    a.z = static_cast<const T *>(z);
    a.A = A;
    a.skip = skip;
    a.bias = bias;
    a.cu = cu;
    a.init = init;
    a.out = static_cast<T *>(out);
    a.fin = fin;
    a.defer = fin && fin == init;
    // The widest word that all of these rows allow.
    auto word = [](std::initializer_list<const void *> ptrs, std::initializer_list<int64_t> sizes) {
        uint64_t bits = 0;
        for (const void *q : ptrs) bits |= reinterpret_cast<uintptr_t>(q);
        for (int64_t n : sizes) bits |= (uint64_t)n * sizeof(T);
        return bits % 16 == 0 ? kCopy16 : bits % 4 == 0 ? kCopy4 : kCopyElement;
    };
    const bool shifted =
        word({x, dt, z}, {p.x_stride, p.dt_stride, z ? p.z_stride : 0, a.per_group}) != kCopy16;
    a.bc_word = word({B, C}, {p.b_stride, p.c_stride, p.state_dim});
    a.state_words = p.state_dim % 4 == 0 && aligned16(A) && aligned16(init) && aligned16(fin);
    const int ch = channels_per_thread(pl.ns);
    a.out_own = (reinterpret_cast<uintptr_t>(out) | (uint64_t)p.out_stride * sizeof(T)) %
                        (ch * sizeof(T)) == 0 && a.per_group % ch == 0;
    // Only a batch of several sequences (or of no tokens) has empty ones.
    const bool empties = fin && fin != init && (p.num_seqs > 1 || p.total_tokens == 0);
    switch (pl.ns) {
        case 4: return run_scan<T, 4>(pl, a, shifted, empties, stream);
        case 8: return run_scan<T, 8>(pl, a, shifted, empties, stream);
        case 16: return run_scan<T, 16>(pl, a, shifted, empties, stream);
        case 32: return run_scan<T, 32>(pl, a, shifted, empties, stream);
        case 64: return run_scan<T, 64>(pl, a, shifted, empties, stream);
    }
    return GDN_ERR_UNSUPPORTED;
}

template <typename T, int NS, bool QUADS>
gdn_status run_scan_step(ScanStepArgs<T> &a, cudaStream_t stream) {
    static std::atomic<bool> done[kMaxDevices];
    if (!raise_shared_memory(done, {reinterpret_cast<const void *>(
                                       gdn_scan_step_kernel<T, NS, QUADS>)},
                             {step_bytes<NS>()}))
        return GDN_ERR_CUDA;
    a.tiles = (a.per_group + kStepThreads - 1) / kStepThreads;
    a.pairs = (int64_t)a.tiles * (a.D / a.per_group) * a.N;
    const int64_t blocks = kStepBlocks<NS> * kGridSms;
    a.run = (a.pairs + blocks - 1) / blocks;
    gdn_scan_step_kernel<T, NS, QUADS>
        <<<(unsigned)((a.pairs + a.run - 1) / a.run), kStepThreads, step_bytes<NS>(), stream>>>(a);
    return launch_status();
}

template <typename T, int NS> gdn_status run_scan_step(ScanStepArgs<T> &a, cudaStream_t stream) {
    return a.S % 4 == 0 && aligned16(a.A) ? run_scan_step<T, NS, true>(a, stream)
                                          : run_scan_step<T, NS, false>(a, stream);
}

template <typename T>
gdn_status scan_step_typed(const gdn_ssm_problem &p, const void *x, const void *dt,
                           const float *A, const void *B, const void *C, const float *skip,
                           const void *z, const float *bias, const float *state, void *out,
                           float *next, cudaStream_t stream) {
    ScanStepArgs<T> a;
    a.x = static_cast<const T *>(x);
    a.dt = static_cast<const T *>(dt);
    a.B = static_cast<const T *>(B);
    a.C = static_cast<const T *>(C);
    a.z = static_cast<const T *>(z);
    a.A = A;
    a.skip = skip;
    a.bias = bias;
    a.state = state;
    a.out = static_cast<T *>(out);
    a.next = next;
    a.N = p.num_seqs;
    a.D = p.channels;
    a.S = p.state_dim;
    a.per_group = p.channels / p.num_groups;
    a.xs = p.x_stride;
    a.dts = p.dt_stride;
    a.bs = p.b_stride;
    a.cs = p.c_stride;
    a.zs = p.z_stride;
    a.os = p.out_stride;
    a.softplus = p.dt_softplus != 0;
    // Tiles start at multiples of 128 channels in a group: whole words where
    // a group's states are.
    a.words = (int64_t)a.per_group * a.S % 4 == 0 && aligned16(state) && aligned16(next);
    const int S = p.state_dim;
    if (S <= 4) return run_scan_step<T, 4>(a, stream);
    if (S <= 8) return run_scan_step<T, 8>(a, stream);
    if (S <= 16) return run_scan_step<T, 16>(a, stream);
    if (S <= 32) return run_scan_step<T, 32>(a, stream);
    return run_scan_step<T, 64>(a, stream);
}

}  // namespace
}  // namespace gdn

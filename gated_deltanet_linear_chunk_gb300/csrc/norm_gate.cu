// norm_gate.cu -- the norm after a block with its gate and scaled residual,
// and the norm before the next block, in one pass (gdn_norm_gate_residual).
//
//   m = weight rms(y) act(gate)   (or weight rms(y act(gate)))
//   out = residual + scale m,     next = next_weight rms(out)
//
// with rms(v) = v / sqrt(mean(v^2) + eps).  Every input is read once and every
// output written once, about 10 flops per element: bound by HBM bandwidth,
// and for a few rows by the latency of a load, two reductions and a store.
//
// A row stays in registers from its loads to its stores: the second norm works
// on the fp32 sum of the first's result and the residual, before that sum is
// rounded to out's type.  Rows of up to 32 lanes' words share a warp (a
// power of two of lanes each, reduced by shuffles); longer rows take a block.
// The grid is one wave that walks the rows, so the weights are read once per
// block and a row's loads are on their way while the row before is reduced:
// in registers, or for long rows in shared memory.
//
// Measured: 4000 rows of 6144, bf16 y and gate, fp32 residual, both norms, 58 us,
// 87 % of the copy bandwidth (a block per row, weights read again for each: 90
// us); 192000 rows of 128 with a SiLU gate 28 us, 77 % (39 us with a block per
// eight rows: half of its instructions were addresses and weights).
#include "block.cuh"

namespace gdn {
namespace {

constexpr int kWarpThreads = 128;  // block of the rows that share warps
constexpr int64_t kRingBudget = 220 * 1024;  // of an SM's shared memory, for the rings

template <typename T, typename R> struct NormArgs {
    const T *y, *gate;
    const R *residual;
    const float *weight, *next_weight;
    R *out;
    T *next;
    int64_t rows;
    int dim, lanes, act;
    int ahead, row_bytes;  // rows in the ring, and the size of one
    bool staged;   // the weights are in shared memory
    bool gate_first;
    float eps, scale, inv_dim;
    int64_t ys, gs, rs, os, ns;
};

// V elements: in words of up to 16 bytes.
template <typename T, int V> struct Words {
    static constexpr int W = V < kWide<T> ? V : kWide<T>;
    Vec<T, W> w[V / W];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < V / W; ++i) w[i] = Vec<T, W>::load(p + i * W);
    }
    __device__ __forceinline__ void to(float *r) const {
#pragma unroll
        for (int i = 0; i < V / W; ++i) w[i].to(r + i * W);
    }
};
template <int V, typename T> __device__ __forceinline__ void load_f(const T *p, float *r) {
    Words<T, V> w;
    w.load(p);
    w.to(r);
}
template <int V, typename T> __device__ __forceinline__ void store_f(T *p, const float *r) {
    constexpr int W = Words<T, V>::W;
#pragma unroll
    for (int i = 0; i < V; i += W) Vec<T, W>::from(r + i).store(p + i);
}

// Sum over the lanes of a row.
template <bool BLOCK> __device__ __forceinline__ float row_sum(float v, int lanes, float *smem) {
    if (!BLOCK) {
        for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) smem[threadIdx.x / 32] = v;
    __syncthreads();
    const int warps = blockDim.x / 32;
    v = (threadIdx.x & 31) < warps ? smem[threadIdx.x & 31] : 0.f;
    return warp_sum(v);
}

// Where a lane's next rows wait.  In registers, one row ahead, or (RING) in a
// ring in shared memory, up to four rows ahead, through asynchronous copies:
//  - Long rows, a lane's 16 elements, with the weights and another row's words
//    leave no registers (us without rows ahead and with the ring: 2436 rows of
//    10088 46 and 31, 2590 of 9488 53 and 35, 791 of 11624 in fp32 42 and 22,
//    2552 of 9629 163 and 123).
//  - Words of four elements ahead in registers are few bytes in flight (in
//    registers and in the ring: 20617 rows of 1192 in fp32 57 and 36, 23630 of
//    1040 80 and 73), if a block takes several rows (31 rows of 2016 2.6 and 2.9).
//  - Words of eight are enough in registers (12047 rows of 2040 36.5 and 38),
//    and narrower ones are bound by their instructions (9965 of 2466 38 and 50).
template <int V, int I> constexpr bool kLongRow = V * I > 8 || I > 4;
// Blocks per SM of the rows that share warps, by the elements of a lane.
template <int N> constexpr int kWarpBlocks = N <= 8 ? 8 : 4;
// A block that shares one row has at most this many threads.
constexpr int kRowThreads = 1024;

// A lane's part of one row in the ring: I words of V elements in pieces of up
// to 16 bytes, a single 16-bit element in the 4-byte word that holds it.
template <typename E, int V, int I> struct RowSlots {
    static constexpr int kWord = V * (int)sizeof(E) < 4 ? 4 : V * (int)sizeof(E);
    static constexpr int kPiece = kWord < 16 ? kWord : 16, kPieces = kWord / kPiece;
    static constexpr int kBytes = I * kWord;  // per thread
    __device__ __forceinline__ static char *piece(char *base, int threads, int i, int k) {
        return base + ((i * kPieces + k) * threads + threadIdx.x) * kPiece;
    }
    // high: whether a single 16-bit element lies in its 4-byte word's upper half;
    // first: whether it is its tensor's first.
    __device__ __forceinline__ static void copy(char *base, int threads, int i, const E *from,
                                                int high, bool first) {
        if constexpr (V * sizeof(E) == 2) {
            copy_async_element(piece(base, threads, i, 0), from, high, first);
        } else {
#pragma unroll
            for (int k = 0; k < kPieces; ++k)
                copy_async<kPiece, (kPieces > 1)>(piece(base, threads, i, k),
                                                  from + k * (kPiece / sizeof(E)));
        }
    }
    __device__ __forceinline__ static void read(char *base, int threads, int i, int high,
                                                float *to) {
        if constexpr (V * sizeof(E) == 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(piece(base, threads, i, 0));
            const uint16_t half = (uint16_t)(high ? w >> 16 : w);
            to[0] = to_f32(*reinterpret_cast<const E *>(&half));
        } else {
            constexpr int W = kPiece / (int)sizeof(E);
#pragma unroll
            for (int k = 0; k < kPieces; ++k)
                Vec<E, W>::load(reinterpret_cast<const E *>(piece(base, threads, i, k))).to(to + k * W);
        }
    }
};


// I words of V elements per lane.  BLOCK: the block's threads share a row;
// otherwise a.lanes lanes do.  Each walks rows a grid apart, the weights in
// registers or shared memory, and starts the loads of the next rows before the
// first reduction of the one at hand.  Words past the row's end hold anything
// and are left out of sums and stores.  The gate commutes with the norm's
// factor, so a lane keeps only y times the gate and the residual.
template <typename T, typename R, int V, int I, bool BLOCK, bool RING>
__global__ void __launch_bounds__(BLOCK ? kRowThreads : kWarpThreads)
gdn_norm_kernel(const NormArgs<T, R> a) {
    constexpr bool HELD = !BLOCK || !kLongRow<V, I>;  // the weights are in registers
    using SlotT = RowSlots<T, V, I>;
    using SlotR = RowSlots<R, V, I>;
    using SlotW = RowSlots<float, V, I>;
    extern __shared__ __align__(16) char ring[];  // [row ahead][y, gate, residual], weights
    // Two sums per pass, in turn for odd and even passes: with only one of
    // them there is one barrier between a pass's reads and the next's writes.
    __shared__ float sums[2][2][32];
    int turn = 0;
    const int lanes = BLOCK ? blockDim.x : a.lanes;
    const int lane = BLOCK ? threadIdx.x : threadIdx.x & (lanes - 1);
    const int groups = BLOCK ? 1 : kWarpThreads / lanes;
    int64_t row = (int64_t)blockIdx.x * groups + (BLOCK ? 0 : threadIdx.x / lanes);
    const int64_t step = (int64_t)gridDim.x * groups;

    // Whether the row has word i of this lane, and its first element (of a word
    // that it has not, the row's first: the words held in registers are loaded
    // all).  Many words' places are computed each time, a few are kept.
    const int c0 = lane * V, span = lanes * V;
    int column[RING ? 1 : I];
    bool exists[RING ? 1 : I];
    auto ok = [&](int i) { return RING ? c0 + i * span < a.dim : exists[RING ? 0 : i]; };
    auto c = [&](int i) { return RING ? c0 + i * span : column[RING ? 0 : i]; };
    if (!RING)
#pragma unroll
        for (int i = 0; i < I; ++i) {
            exists[RING ? 0 : i] = c0 + i * span < a.dim;
            column[RING ? 0 : i] = exists[RING ? 0 : i] ? c0 + i * span : 0;
        }
    // Whether word i of a row is in the upper half of 4 bytes (a block's words
    // lie an even number of elements apart).
    auto high = [&](const auto *r, int i) { return odd(r + c0) ^ (BLOCK ? 0 : i & span & 1); };
    const int threads = blockDim.x;
    auto in_gate = [&](char *stage) { return stage + SlotT::kBytes * threads; };
    auto in_residual = [&](char *stage) {
        return stage + (a.gate ? 2 : 1) * SlotT::kBytes * threads;
    };
    char *const staged = ring + a.ahead * a.row_bytes;  // weights
    Words<T, V> yw[I], gw[I];
    Words<R, V> rw[I];
    // Row r's loads; in the ring's place `stage`, if it exists.  first: this
    // lane's first words there are the tensors' first.
    auto fetch = [&](int64_t r, char *stage, bool first) {
        if (!RING) {
            r = min(r, a.rows - 1);
#pragma unroll
            for (int i = 0; i < I; ++i) {
                yw[i].load(a.y + r * a.ys + c(i));
                if (a.gate) gw[i].load(a.gate + r * a.gs + c(i));
                if (a.residual) rw[i].load(a.residual + r * a.rs + c(i));
            }
            return;
        }
        if (r < a.rows) {
#pragma unroll
            for (int i = 0; i < I; ++i) {
                if (!ok(i)) break;
                const bool head = first && i == 0;
                SlotT::copy(stage, threads, i, a.y + r * a.ys + c(i), high(a.y + r * a.ys, i), head);
                if (a.gate)
                    SlotT::copy(in_gate(stage), threads, i, a.gate + r * a.gs + c(i),
                                high(a.gate + r * a.gs, i), head);
                if (a.residual)
                    SlotR::copy(in_residual(stage), threads, i, a.residual + r * a.rs + c(i),
                                high(a.residual + r * a.rs, i), head);
            }
        }
        copies_commit();
    };
    float w[HELD ? I : 1][V], nw[HELD ? I : 1][V];
    if (!HELD && a.staged)
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (!ok(i)) break;
            if (a.weight) SlotW::copy(staged, threads, i, a.weight + c(i), 0, false);
            if (a.next_weight)
                SlotW::copy(staged + SlotW::kBytes * threads, threads, i, a.next_weight + c(i), 0,
                            false);
        }
    if (RING)
        for (int k = 0; k < a.ahead; ++k)
            fetch(row + k * step, ring + k * a.row_bytes, k == 0 && row == 0 && lane == 0);
    else
        fetch(row, nullptr, false);
    if (HELD)
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int at = ok(i) ? c(i) : 0;
            if (a.weight) load_f<V>(a.weight + at, w[i]);
            if (a.next_weight) load_f<V>(a.next_weight + at, nw[i]);
        }
    if (RING && V * sizeof(T) == 2 && row == 0 && lane == 0) {
        load_first(SlotT::piece(ring, threads, 0, 0), a.y);
        if (a.gate) load_first(SlotT::piece(in_gate(ring), threads, 0, 0), a.gate);
        if (sizeof(R) == 2 && a.residual)
            load_first(SlotR::piece(in_residual(ring), threads, 0, 0), a.residual);
    }
    auto weight = [&](const float *all, int second, int i, float *to) {
        if (a.staged)
            SlotW::read(staged + second * SlotW::kBytes * threads, threads, i, 0, to);
        else
            load_f<V>(all + (ok(i) ? c(i) : 0), to);
    };
    // All groups of a block make the same number of passes: the sums need
    // every lane of a warp.
    int place = 0;  // of this row in the ring
    for (int64_t first = (int64_t)blockIdx.x * groups; first < a.rows;
         first += step, row += step, turn ^= 1) {
        const bool live = row < a.rows;
        char *const stage = ring + place * a.row_bytes;
        if (RING) {
            if (a.ahead == 1) copies_wait<0>();
            else if (a.ahead == 2) copies_wait<1>();
            else copies_wait<3>();
            place = place + 1 == a.ahead ? 0 : place + 1;
        }
        float m[I][V], r[I][V], sum = 0.f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (RING) SlotT::read(stage, threads, i, high(a.y + row * a.ys, i), m[i]);
            else yw[i].to(m[i]);
            float part = 0.f;
            if (!a.gate_first)
#pragma unroll
                for (int v = 0; v < V; ++v) part = fmaf(m[i][v], m[i][v], part);
            if (a.gate) {
                float g[V];
                if (RING) SlotT::read(in_gate(stage), threads, i, high(a.gate + row * a.gs, i), g);
                else gw[i].to(g);
                if (a.act == GDN_ACT_SILU) {
#pragma unroll
                    for (int v = 0; v < V; ++v) m[i][v] *= silu(g[v]);
                } else if (a.act == GDN_ACT_SIGMOID) {
#pragma unroll
                    for (int v = 0; v < V; ++v) m[i][v] *= sigmoid(g[v]);
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) m[i][v] *= g[v];
                }
            }
            if (a.gate_first)
#pragma unroll
                for (int v = 0; v < V; ++v) part = fmaf(m[i][v], m[i][v], part);
            if (ok(i)) sum += part;
            if (!a.residual) {
#pragma unroll
                for (int v = 0; v < V; ++v) r[i][v] = 0.f;
            } else if (RING) {
                SlotR::read(in_residual(stage), threads, i, high(a.residual + row * a.rs, i), r[i]);
            } else {
                rw[i].to(r[i]);
            }
        }
        fetch(row + (RING ? a.ahead : 1) * step, stage, false);
        float inv = a.scale;
        if (a.weight)
            inv *= rsqrtf(fmaf(row_sum<BLOCK>(sum, lanes, sums[turn][0]), a.inv_dim, a.eps));
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (a.weight) {
                float u[V];
                if (!HELD) weight(a.weight, 0, i, u);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    r[i][v] = fmaf(m[i][v] * inv, HELD ? w[HELD ? i : 0][v] : u[v], r[i][v]);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) r[i][v] = fmaf(m[i][v], inv, r[i][v]);
            }
            if (live && ok(i)) store_f<V>(a.out + row * a.os + c(i), r[i]);
            if (a.next_weight) {
                float part = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v) part = fmaf(r[i][v], r[i][v], part);
                if (ok(i)) sum += part;
            }
        }
        if (a.next_weight) {
            inv = rsqrtf(fmaf(row_sum<BLOCK>(sum, lanes, sums[turn][1]), a.inv_dim, a.eps));
#pragma unroll
            for (int i = 0; i < I; ++i) {
                float u[V];
                if (!HELD) weight(a.next_weight, 1, i, u);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    r[i][v] *= inv * (HELD ? nw[HELD ? i : 0][v] : u[v]);
                if (live && ok(i)) store_f<V>(a.next + row * a.ns + c(i), r[i]);
            }
        }
    }
    if (RING) copies_wait<0>();
}

// The grid holds what is resident at once (64 registers per thread, 128 in
// blocks of few words): more blocks would load the weights again.  Measured
// on 24000 rows of 1024 (128 threads): 6 blocks per SM 55 us, 4 61, 8 59.

// Starts blocks of `threads` for rows of `per` each, `resident` of them on an
// SM as far as registers go.
template <typename T, typename R, int V, int I, bool BLOCK, bool RING>
gdn_status launch_norm(NormArgs<T, R> &a, int threads, int64_t per, int resident,
                       cudaStream_t stream) {
    const int64_t blocks = (a.rows + per - 1) / per, most = (int64_t)resident * kGridSms;
    const int64_t grid = blocks < most ? blocks : most;
    int64_t bytes = 0;
    a.ahead = 0;
    a.staged = false;
    if (RING) {
        // As many rows ahead as the passes can use and an SM's shared memory
        // holds for its blocks, after the weights where one row fits beside them.
        const int64_t budget = kRingBudget / resident;
        const int64_t row = (int64_t)threads * ((a.gate ? 2 : 1) * RowSlots<T, V, I>::kBytes +
                                                (a.residual ? RowSlots<R, V, I>::kBytes : 0));
        const int64_t weights = (int64_t)threads * 2 * RowSlots<float, V, I>::kBytes;
        a.row_bytes = (int)row;
        a.staged = kLongRow<V, I> && weights + row <= budget;
        bytes = a.staged ? weights : 0;
        const int64_t passes = (blocks + grid - 1) / grid;
        a.ahead = 4;
        while (a.ahead > 1 && (a.ahead > passes || bytes + a.ahead * row > budget)) a.ahead /= 2;
        bytes += a.ahead * row;
        static std::atomic<bool> done[kMaxDevices];
        if (!raise_shared_memory(
                done, {reinterpret_cast<const void *>(gdn_norm_kernel<T, R, V, I, BLOCK, RING>)},
                {(size_t)kRingBudget}))
            return GDN_ERR_CUDA;
    }
    gdn_norm_kernel<T, R, V, I, BLOCK, RING>
        <<<(unsigned)grid, threads, (size_t)bytes, stream>>>(a);
    return launch_status();
}

// Rows that share warps.
template <typename T, typename R, int V, int I>
gdn_status run_norm_warps(NormArgs<T, R> &a, int words, cudaStream_t stream) {
    a.lanes = 1;
    while (a.lanes * I < words) a.lanes *= 2;
    return launch_norm<T, R, V, I, false, false>(a, kWarpThreads, kWarpThreads / a.lanes,
                                                 kWarpBlocks<V * I>, stream);
}

// Blocks that share a row.
template <typename T, typename R, int V, int I>
gdn_status run_norm_block(NormArgs<T, R> &a, int words, cudaStream_t stream) {
    const int threads = 32 * ((words + 32 * I - 1) / (32 * I));
    // Blocks per SM with a ring (64 registers a thread), and without.
    const int ring = 1024 / threads, held = threads <= 768 ? 768 / threads : 1;
    if constexpr (kLongRow<V, I>) {
        return launch_norm<T, R, V, I, true, true>(a, threads, 1, ring, stream);
    } else {
        if constexpr (V == 4)
            if (a.rows > ring * kGridSms)
                return launch_norm<T, R, V, I, true, true>(a, threads, 1, ring, stream);
        return launch_norm<T, R, V, I, true, false>(a, threads, 1, held, stream);
    }
}

// Rows in words of four or eight elements.
template <typename T, typename R, int V>
gdn_status run_norm(NormArgs<T, R> &a, cudaStream_t stream) {
    const int words = a.dim / V;
    if (words <= 32) return run_norm_warps<T, R, V, 1>(a, words, stream);
    if (words <= 64) return run_norm_warps<T, R, V, 2>(a, words, stream);
    if (words <= (V == 8 ? 1024 : 768)) return run_norm_block<T, R, V, 1>(a, words, stream);
    return run_norm_block<T, R, V, 16 / V>(a, words, stream);
}

template <typename T, typename R>
gdn_status norm_typed(const gdn_norm_problem &p, const void *y, const float *weight,
                      const void *gate, const void *residual, const float *next_weight, void *out,
                      void *next, cudaStream_t stream) {
    NormArgs<T, R> a;
    a.y = static_cast<const T *>(y);
    a.gate = static_cast<const T *>(gate);
    a.residual = static_cast<const R *>(residual);
    a.weight = weight;
    a.next_weight = next_weight;
    a.out = static_cast<R *>(out);
    a.next = static_cast<T *>(next);
    a.rows = p.rows;
    a.dim = p.dim;
    a.lanes = 0;
    a.act = p.activation;
    a.gate_first = p.gate_first != 0;
    a.eps = p.eps;
    a.scale = p.scale;
    a.inv_dim = 1.f / (float)p.dim;
    a.ys = p.y_stride;
    a.gs = p.gate_stride;
    a.rs = p.residual_stride;
    a.os = p.out_stride;
    a.ns = p.next_stride;
    auto whole = [&](auto bytes, const void *q, int64_t stride, size_t size) {
        return (reinterpret_cast<uintptr_t>(q) | (q ? (uint64_t)stride * size : 0)) % bytes == 0;
    };
    // Whether every row can be read V elements at a time.
    auto words_of = [&](int v) {
        const size_t e = sizeof(T), f = sizeof(R);
        const size_t b = v * e < 16 ? v * e : 16, c = v * f < 16 ? v * f : 16,
                     d = v * 4 < 16 ? v * 4 : 16;
        return p.dim % v == 0 && whole(b, y, p.y_stride, e) && whole(b, gate, p.gate_stride, e) &&
               whole(b, next, p.next_stride, e) && whole(c, residual, p.residual_stride, f) &&
               whole(c, out, p.out_stride, f) && whole(d, weight, 0, 4) &&
               whole(d, next_weight, 0, 4);
    };
    constexpr int V = kWide<T>;
    if (words_of(V)) return run_norm<T, R, V>(a, stream);
    if constexpr (V == 8)
        if (words_of(4)) return run_norm<T, R, 4>(a, stream);
    if constexpr (sizeof(T) == 2) {
        const int words = p.dim / 2;
        if (words_of(2)) {
            if (words <= 128) return run_norm_warps<T, R, 2, 4>(a, words, stream);
            if (words <= 4096) return run_norm_block<T, R, 2, 4>(a, words, stream);
            return run_norm_block<T, R, 2, 8>(a, words, stream);
        }
    }
    if (p.dim <= 128) return run_norm_warps<T, R, 1, 4>(a, p.dim, stream);
    if (p.dim <= 4096) return run_norm_block<T, R, 1, 4>(a, p.dim, stream);
    if (p.dim <= 8192) return run_norm_block<T, R, 1, 8>(a, p.dim, stream);
    return run_norm_block<T, R, 1, 16>(a, p.dim, stream);
}

}  // namespace

gdn_status launch_norm_gate_residual(const gdn_norm_problem &p, const void *y,
                                     const float *weight, const void *gate, const void *residual,
                                     const float *next_weight, void *out, void *next,
                                     cudaStream_t stream) {
    if (p.dtype == GDN_F32)
        return norm_typed<float, float>(p, y, weight, gate, residual, next_weight, out, next,
                                        stream);
    if (p.residual_dtype == GDN_F32)
        return norm_typed<__nv_bfloat16, float>(p, y, weight, gate, residual, next_weight, out,
                                                next, stream);
    return norm_typed<__nv_bfloat16, __nv_bfloat16>(p, y, weight, gate, residual, next_weight,
                                                    out, next, stream);
}

}  // namespace gdn

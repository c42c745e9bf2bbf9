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
// block and a row's loads are on their way while the row before is reduced.
//
// Measured: 4000 rows of 6144, bf16 y and gate, fp32 residual, both norms, 58 us,
// 87 % of the copy bandwidth (a block per row, weights read again for each: 90
// us); 192000 rows of 128 with a SiLU gate 28 us, 77 % (39 us with a block per
// eight rows: half of its instructions were addresses and weights).
#include "block.cuh"

namespace gdn {
namespace {

constexpr int kWarpThreads = 128;  // block of the rows that share warps

template <typename T, typename R> struct NormArgs {
    const T *y, *gate;
    const R *residual;
    const float *weight, *next_weight;
    R *out;
    T *next;
    int64_t rows;
    int dim, lanes, act;
    bool gate_first;
    float eps, scale, inv_dim;
    int64_t ys, gs, rs, os, ns;
};

// V elements: one, two, or whole 16-byte words.
template <typename T, int V> struct Words {
    static constexpr int W = V <= 2 ? V : kWide<T>;
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

// Elements of a row that a lane may hold with the weights and the next row's
// words beside them.
template <int V, int I> constexpr bool kAhead = V <= 2 ? I <= 4 : V * I <= 16;
// Threads of a block that shares one row: as many as leave a thread those
// registers.
template <int V, int I> constexpr int kRowThreads = V <= 2 || V * I <= 8 ? 1024 : 512;

// I words of V elements per lane.  BLOCK: the block's threads share a row;
// otherwise a.lanes lanes do.  Each walks rows a grid apart with the weights
// in registers, and starts the next row's loads before the first reduction
// of the one at hand.  Lanes past the row's end load its first word and leave
// it out of sums and stores.  The gate commutes with the norm's factor, so a
// lane keeps only y times the gate and the residual.
template <typename T, typename R, int V, int I, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kRowThreads<V, I> : kWarpThreads)
gdn_norm_kernel(const NormArgs<T, R> a) {
    constexpr bool AHEAD = kAhead<V, I>;
    // Two sums per pass, in turn for odd and even passes: with only one of
    // them there is one barrier between a pass's reads and the next's writes.
    __shared__ float sums[2][2][32];
    int turn = 0;
    const int lanes = BLOCK ? blockDim.x : a.lanes;
    const int lane = BLOCK ? threadIdx.x : threadIdx.x & (lanes - 1);
    const int groups = BLOCK ? 1 : kWarpThreads / lanes;
    int64_t row = (int64_t)blockIdx.x * groups + (BLOCK ? 0 : threadIdx.x / lanes);
    const int64_t step = (int64_t)gridDim.x * groups;

    int c[I];
    bool ok[I];
    float w[AHEAD ? I : 1][V], nw[AHEAD ? I : 1][V];
#pragma unroll
    for (int i = 0; i < I; ++i) {
        c[i] = (lane + i * lanes) * V;
        ok[i] = c[i] < a.dim;
        if (!ok[i]) c[i] = 0;
    }
    Words<T, V> yw[I], gw[I];
    Words<R, V> rw[I];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            yw[i].load(a.y + r * a.ys + c[i]);
            if (a.gate) gw[i].load(a.gate + r * a.gs + c[i]);
            if (a.residual) rw[i].load(a.residual + r * a.rs + c[i]);
        }
    };
    fetch(min(row, a.rows - 1));
    if (AHEAD)
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (a.weight) load_f<V>(a.weight + c[i], w[i]);
            if (a.next_weight) load_f<V>(a.next_weight + c[i], nw[i]);
        }
    // All groups of a block make the same number of passes: the sums need
    // every lane of a warp.
    for (int64_t first = (int64_t)blockIdx.x * groups; first < a.rows;
         first += step, row += step, turn ^= 1) {
        const bool live = row < a.rows;
        float m[I][V], r[I][V], sum = 0.f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            yw[i].to(m[i]);
            float part = 0.f;
            if (!a.gate_first)
#pragma unroll
                for (int v = 0; v < V; ++v) part = fmaf(m[i][v], m[i][v], part);
            if (a.gate) {
                float g[V];
                gw[i].to(g);
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
            if (ok[i]) sum += part;
            if (a.residual) {
                rw[i].to(r[i]);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) r[i][v] = 0.f;
            }
        }
        if (AHEAD) fetch(min(row + step, a.rows - 1));
        float inv = a.scale;
        if (a.weight)
            inv *= rsqrtf(fmaf(row_sum<BLOCK>(sum, lanes, sums[turn][0]), a.inv_dim, a.eps));
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (a.weight) {
                float u[V];
                if (!AHEAD) load_f<V>(a.weight + c[i], u);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    r[i][v] = fmaf(m[i][v] * inv, AHEAD ? w[AHEAD ? i : 0][v] : u[v], r[i][v]);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) r[i][v] = fmaf(m[i][v], inv, r[i][v]);
            }
            if (live && ok[i]) store_f<V>(a.out + row * a.os + c[i], r[i]);
            if (a.next_weight) {
                float part = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v) part = fmaf(r[i][v], r[i][v], part);
                if (ok[i]) sum += part;
            }
        }
        if (a.next_weight) {
            inv = rsqrtf(fmaf(row_sum<BLOCK>(sum, lanes, sums[turn][1]), a.inv_dim, a.eps));
#pragma unroll
            for (int i = 0; i < I; ++i) {
                float u[V];
                if (!AHEAD) load_f<V>(a.next_weight + c[i], u);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    r[i][v] *= inv * (AHEAD ? nw[AHEAD ? i : 0][v] : u[v]);
                if (live && ok[i]) store_f<V>(a.next + row * a.ns + c[i], r[i]);
            }
        }
        if (!AHEAD) fetch(min(row + step, a.rows - 1));
    }
}

// The grid holds what is resident at once (64 registers per thread, 128 in
// blocks of few words): more blocks would load the weights again.  Measured
// on 24000 rows of 1024 (128 threads): 6 blocks per SM 55 us, 4 61, 8 59.

// Rows that share warps.
template <typename T, typename R, int V, int I>
gdn_status run_norm_warps(NormArgs<T, R> &a, int words, cudaStream_t stream) {
    a.lanes = 1;
    while (a.lanes * I < words) a.lanes *= 2;
    const int64_t per = kWarpThreads / a.lanes, blocks = (a.rows + per - 1) / per;
    const int64_t most = (V * I <= 8 ? 8 : 4) * kGridSms;
    gdn_norm_kernel<T, R, V, I, false>
        <<<(unsigned)(blocks < most ? blocks : most), kWarpThreads, 0, stream>>>(a);
    return launch_status();
}

// Blocks that share a row.
template <typename T, typename R, int V, int I>
gdn_status run_norm_block(NormArgs<T, R> &a, int words, cudaStream_t stream) {
    const int threads = 32 * ((words + 32 * I - 1) / (32 * I));
    const int64_t most = (threads <= 384 ? 768 / threads : 1) * kGridSms;
    gdn_norm_kernel<T, R, V, I, true>
        <<<(unsigned)(a.rows < most ? a.rows : most), threads, 0, stream>>>(a);
    return launch_status();
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
    if (words_of(V)) {
        const int words = p.dim / V;
        if (words <= 32) return run_norm_warps<T, R, V, 1>(a, words, stream);
        if (words <= 64) return run_norm_warps<T, R, V, 2>(a, words, stream);
        if (words <= (V == 8 ? 1024 : 768)) return run_norm_block<T, R, V, 1>(a, words, stream);
        if (words <= 2048) return run_norm_block<T, R, V, 4>(a, words, stream);
        if constexpr (V == 4) return run_norm_block<T, R, V, 8>(a, words, stream);
    }
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

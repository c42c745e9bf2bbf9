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

// V elements as fp32: one element, or whole 16-byte words.
template <int V, typename T> __device__ __forceinline__ void load_f(const T *p, float *r) {
    constexpr int W = V == 1 ? 1 : kWide<T>;
#pragma unroll
    for (int i = 0; i < V; i += W) Vec<T, W>::load(p + i).to(r + i);
}
template <int V, typename T> __device__ __forceinline__ void store_f(T *p, const float *r) {
    constexpr int W = V == 1 ? 1 : kWide<T>;
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

// Threads of a block that shares one row: as many as leave a thread the
// registers for its part of the row.
template <int V, int I> constexpr int kRowThreads = V * I >= 32 ? 512 : 1024;

// I words of V elements per lane; BLOCK: the block's threads share one row.
// The gate commutes with the norm's factor, so a lane keeps only y times the
// gate and the residual.
template <typename T, typename R, int V, int I, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kRowThreads<V, I> : kWarpThreads)
gdn_norm_kernel(const NormArgs<T, R> a) {
    __shared__ float sums[2][32];
    const int lanes = BLOCK ? blockDim.x : a.lanes;
    const int lane = BLOCK ? threadIdx.x : threadIdx.x & (lanes - 1);
    const int64_t row = BLOCK ? blockIdx.x
                              : (int64_t)blockIdx.x * (kWarpThreads / lanes) + threadIdx.x / lanes;
    float m[I][V], r[I][V];
    bool ok[I];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int c = (lane + i * lanes) * V;
        ok[i] = row < a.rows && c < a.dim;
#pragma unroll
        for (int v = 0; v < V; ++v) m[i][v] = r[i][v] = 0.f;
        if (ok[i]) {
            load_f<V>(a.y + row * a.ys + c, m[i]);
            if (a.residual) load_f<V>(a.residual + row * a.rs + c, r[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
        float g[V];
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] = 1.f;
        if (a.gate && ok[i]) {
            load_f<V>(a.gate + row * a.gs + (lane + i * lanes) * V, g);
            if (a.act != GDN_ACT_NONE)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    g[v] = sigmoid(g[v]) * (a.act == GDN_ACT_SILU ? g[v] : 1.f);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float gated = m[i][v] * g[v];
            const float normed = a.gate_first ? gated : m[i][v];
            sum = fmaf(normed, normed, sum);
            m[i][v] = gated;
        }
    }
    float inv = a.scale;
    if (a.weight)
        inv *= rsqrtf(fmaf(row_sum<BLOCK>(sum, lanes, sums[0]), a.inv_dim, a.eps));
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int c = (lane + i * lanes) * V;
        if (!ok[i]) continue;
        float w[V];
#pragma unroll
        for (int v = 0; v < V; ++v) w[v] = 1.f;
        if (a.weight) load_f<V>(a.weight + c, w);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            r[i][v] = fmaf(m[i][v] * inv, w[v], r[i][v]);
            sum = fmaf(r[i][v], r[i][v], sum);
        }
        store_f<V>(a.out + row * a.os + c, r[i]);
    }
    if (!a.next_weight) return;
    inv = rsqrtf(fmaf(row_sum<BLOCK>(sum, lanes, sums[1]), a.inv_dim, a.eps));
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int c = (lane + i * lanes) * V;
        if (!ok[i]) continue;
        float w[V];
        load_f<V>(a.next_weight + c, w);
#pragma unroll
        for (int v = 0; v < V; ++v) w[v] *= r[i][v] * inv;
        store_f<V>(a.next + row * a.ns + c, w);
    }
}

template <typename T, typename R, int V, int I>
gdn_status run_norm(NormArgs<T, R> &a, int words, cudaStream_t stream) {
    if (words <= 32 * I) {
        a.lanes = 1;
        while (a.lanes * I < words) a.lanes *= 2;
        const int64_t per = kWarpThreads / a.lanes, blocks = (a.rows + per - 1) / per;
        if (blocks > INT32_MAX) return GDN_ERR_UNSUPPORTED;
        gdn_norm_kernel<T, R, V, I, false><<<(unsigned)blocks, kWarpThreads, 0, stream>>>(a);
    } else {
        if (a.rows > INT32_MAX) return GDN_ERR_UNSUPPORTED;
        const int threads = 32 * ((words + 32 * I - 1) / (32 * I));
        gdn_norm_kernel<T, R, V, I, true><<<(unsigned)a.rows, threads, 0, stream>>>(a);
    }
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
    const bool wide = p.dim % kWide<T> == 0 && rows_aligned16<T>(y, p.y_stride) &&
                      rows_aligned16<T>(gate, p.gate_stride) &&
                      rows_aligned16<R>(residual, p.residual_stride) &&
                      rows_aligned16<R>(out, p.out_stride) &&
                      rows_aligned16<T>(next, p.next_stride) &&
                      rows_aligned16<float>(weight, 0) && rows_aligned16<float>(next_weight, 0);
    constexpr int V = kWide<T>;
    if (wide) {
        const int words = p.dim / V;
        if (words <= 32) return run_norm<T, R, V, 1>(a, words, stream);
        if (words <= 512) return run_norm<T, R, V, 2>(a, words, stream);
        return run_norm<T, R, V, 4>(a, words, stream);
    }
    if (p.dim <= 32) return run_norm<T, R, 1, 1>(a, p.dim, stream);
    if (p.dim <= 2048) return run_norm<T, R, 1, 8>(a, p.dim, stream);
    return run_norm<T, R, 1, 16>(a, p.dim, stream);
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

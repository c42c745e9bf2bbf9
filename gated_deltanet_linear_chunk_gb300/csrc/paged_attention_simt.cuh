// paged_attention_simt.cuh -- the attention of paged_attention.cuh in fp32
// arithmetic.
//
// A warp takes eight tokens at a time: four lanes share a token's scores, each
// with a quarter of its key, then every lane sums its own elements of the
// values.
#pragma once

#include "paged_attention.cuh"

namespace gdn {

constexpr int kSimtWarps = 4, kSimtTokens = 8, kSimtChunk = 64;

// RR rows at a time, TC in the cache.
template <typename T, typename TC, int D, int RR>
__global__ void __launch_bounds__(kSimtWarps * 32)
gdn_attention_simt_kernel(const __grid_constant__ AttentionArgs a) {
    constexpr int W = 16 / (int)sizeof(TC), WORDS = D / W, E = D / 32;
    constexpr float kNone = -__builtin_huge_valf();
    extern __shared__ __align__(16) float smem[];
    float *qs = smem;                                // [RR][D]
    float *ps = qs + RR * D;                         // [warps][RR][tokens]
    float *os = ps + kSimtWarps * RR * kSimtTokens;  // [warps][RR][D]
    __shared__ float2 ml[kSimtWarps][RR];
    __shared__ int lims[RR];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int tok = lane / 4, s = lane % 4;
    float *pw = ps + warp * RR * kSimtTokens;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const Range range = find_range<kSimtChunk, 1, kSimtWarps * 32, 1>(a, a.Hkv * a.row_blocks, 0);
    for_pieces<kSimtChunk, 1, RR>(a, range, [&](const Unit &u, const Piece &piece) {
        const int t0 = piece.first_token<kSimtChunk, 1>(u.len), t1 = piece.last_token<kSimtChunk, 1>(u.len);
        const int slot = piece.whole() ? -1 : piece.slot(range.group);
        __syncthreads();  // the last piece's rows
        for (int i = threadIdx.x; i < RR * D; i += kSimtWarps * 32) {
            const int r = i / D;
            float v = 0.f;
            if (r < u.rows) {
                const RowPlace p = row_place(a, u, r);
                v = to_f32(((const T *)a.q)[p.token * a.qs + p.head * a.qh + i % D]);
            }
            qs[i] = v;
        }
        if (threadIdx.x < RR)
            lims[threadIdx.x] = threadIdx.x < u.rows ? seen_by(a, u, threadIdx.x) : 0;
        __syncthreads();
        const float scale = a.scale_log2 * (a.k_scale ? a.k_scale[u.head] : 1.f);
        float m[RR], l[RR], o[RR][E];
#pragma unroll
        for (int r = 0; r < RR; ++r) {
            m[r] = kNone, l[r] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[r][e] = 0.f;
        }
        bool bad = false;
        for (int j0 = t0 + warp * kSimtTokens; j0 < t1; j0 += kSimtWarps * kSimtTokens) {
            const int j = j0 + tok;
            int64_t page = -1;
            if (j < t1) {
                page = a.table[u.n * a.table_stride + j / a.page_size];
                if (page < 0 || page >= a.num_pages) page = -1, bad = true;
            }
            const int place = j % a.page_size;
            const TC *k = (const TC *)((const char *)a.k + page * a.kps + place * a.kts + u.head * a.khs);
            const int64_t v_at = page * a.vps + place * a.vts + u.head * a.vhs;
            float acc[RR];
#pragma unroll
            for (int r = 0; r < RR; ++r) acc[r] = 0.f;
            for (int i = s; i < WORDS; i += 4) {
                float x[W];
                if (page < 0) {
#pragma unroll
                    for (int e = 0; e < W; ++e) x[e] = 0.f;
                } else {
                    load_cached(k + i * W, x);
                }
#pragma unroll
                for (int r = 0; r < RR; ++r)
#pragma unroll
                    for (int e = 0; e < W; ++e) acc[r] = fmaf(qs[r * D + i * W + e], x[e], acc[r]);
            }
            float fade[RR];
#pragma unroll
            for (int r = 0; r < RR; ++r) {
                float x = acc[r];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                x = j < t1 && j < lims[r] ? x * scale : kNone;
                float top = x;
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                top = fmaxf(top, m[r]);
                const float p = ex2(x - against(top));
                fade[r] = ex2(m[r] - against(top));
                m[r] = top;
                l[r] = l[r] * fade[r] + p;
                if (s == 0) pw[r * kSimtTokens + tok] = p;
            }
            __syncwarp();
#pragma unroll
            for (int r = 0; r < RR; ++r)
#pragma unroll
                for (int e = 0; e < E; ++e) o[r][e] *= fade[r];
            for (int t = 0; t < kSimtTokens && j0 + t < t1; ++t) {
                const int64_t at = __shfl_sync(0xffffffffu, v_at, t * 4);
                if (__shfl_sync(0xffffffffu, (int)(page < 0), t * 4)) continue;
                float x[E];
                load_cached((const TC *)((const char *)a.v + at) + lane * E, x);
#pragma unroll
                for (int r = 0; r < RR; ++r) {
                    if (j0 + t >= lims[r]) continue;
                    const float p = pw[r * kSimtTokens + t];
#pragma unroll
                    for (int e = 0; e < E; ++e) o[r][e] = fmaf(p, x[e], o[r][e]);
                }
            }
            __syncwarp();
        }
        bad = __any_sync(0xffffffffu, bad);
        // The warps' sums, joined.
#pragma unroll
        for (int r = 0; r < RR; ++r) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
            if (bad) l[r] = __int_as_float(0x7fffffff);
            if (lane == 0) ml[warp][r] = make_float2(m[r], l[r]);
#pragma unroll
            for (int e = 0; e < E; ++e) os[(warp * RR + r) * D + lane * E + e] = o[r][e];
        }
        __syncthreads();
        const float v_scale = a.v_scale ? a.v_scale[u.head] : 1.f;
        for (int i = threadIdx.x; i < u.rows * D; i += kSimtWarps * 32) {
            const int r = i / D, e = i % D;
            float top = kNone, sum = 0.f, y = 0.f;
#pragma unroll
            for (int w = 0; w < kSimtWarps; ++w) top = fmaxf(top, ml[w][r].x);
#pragma unroll
            for (int w = 0; w < kSimtWarps; ++w) {
                const float f = ex2(ml[w][r].x - against(top));
                sum += ml[w][r].y * f;
                y += os[(w * RR + r) * D + e] * f;
            }
            y *= v_scale;
            if (slot < 0) {
                const RowPlace p = row_place(a, u, r);
                const T *gate = a.gate ? (const T *)a.gate + p.token * a.gs + p.head * a.gh + e : nullptr;
                ((T *)a.out)[p.token * a.os + p.head * a.oh + e] =
                    from_f32<T>(finish(y, inverse(sum), gate));
                if (e == 0) store_lse(a, p, top, sum);
            } else {
                a.sums[((int64_t)slot * RR + r) * D + e] = y;
                if (e == 0) a.stats[slot * RR + r] = make_float2(top, sum);
            }
        }
    });
}

// Rows at a time: those of a unit, up to 16.
inline AttentionShape simt_shape(int R) {
    return {R <= 4 ? 4 : R <= 8 ? 8 : 16, kSimtChunk, 1, 1, 2 * kGridSms};
}

template <typename T, typename TC, int D, int RR>
gdn_status simt_run(int blocks, const AttentionArgs &a, cudaStream_t stream) {
    constexpr size_t bytes =
        sizeof(float) * RR * (D + kSimtWarps * kSimtTokens + kSimtWarps * D);
    static std::atomic<bool> done[kMaxDevices];
    const auto kernel = gdn_attention_simt_kernel<T, TC, D, RR>;
    if (!raise_shared_memory(done, {reinterpret_cast<const void *>(kernel)}, {bytes}))
        return GDN_ERR_CUDA;
    return launch_programmatic(kernel, dim3(blocks), kSimtWarps * 32, bytes, stream, a);
}

template <typename T, typename TC, int D>
gdn_status simt_rows(int blocks, const AttentionArgs &a, cudaStream_t stream) {
    if (a.R <= 4) return simt_run<T, TC, D, 4>(blocks, a, stream);
    if (a.R <= 8) return simt_run<T, TC, D, 8>(blocks, a, stream);
    return simt_run<T, TC, D, 16>(blocks, a, stream);
}

template <typename T, typename TC>
gdn_status simt_attention(int D, int blocks, const AttentionArgs &a, cudaStream_t stream) {
    if (D == 64) return simt_rows<T, TC, 64>(blocks, a, stream);
    if (D == 128) return simt_rows<T, TC, 128>(blocks, a, stream);
    return simt_rows<T, TC, 256>(blocks, a, stream);
}

}  // namespace gdn

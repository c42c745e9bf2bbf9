// paged_attention_simt.cuh -- the attention of paged_attention.cuh in fp32.
//
// A warp takes eight tokens at a time, whose keys and then values asynchronous
// copies bring to shared memory: the values while the scores are computed, the
// next keys while the values are added.  Four lanes share a token's scores, each
// with every fourth word of its key; then every lane sums its own elements of
// the values.  A row or four are bound by memory: 4096 units of 1024 tokens, one row
// of 128, 687 us (6.3 TB/s), four 709.  More are by reads of shared memory, where a
// lane gets every row's query word and weight again for its token: six rows of 128
// (taken as eight) 1070 us, its shared memory 70 % busy and the fp32 units 26 %; six
// of 256 1452 us for 512 tokens (3.0 TB/s), shared memory 44 %, fp32 18 %, memory 34
// %: there the two warps of a scheduler wait for those reads, and for the copies of
// a tile that nothing but the other half's arithmetic covers.  (Sixteen rows of 256
// spill 132 bytes of stores and 152 of loads.)
#pragma once

#include "paged_attention.cuh"

namespace gdn {

constexpr int kSimtWarps = 4, kSimtTokens = 8, kSimtChunk = 64;
// Blocks per SM: as registers and shared memory allow.
constexpr int simt_blocks(int D, int rows) { return rows > 8 || D > 128 ? 2 : 3; }

// RR rows at a time.
template <int D, int RR> struct Simt {
    static constexpr int kPitch = D + 16;  // floats: eight tokens' words on different banks
    static constexpr int kHalf = kSimtTokens * kPitch;
    static constexpr int kQueries = RR * D, kWeights = kSimtWarps * RR * kSimtTokens;
    static constexpr int kTiles = kSimtWarps * 2 * kHalf, kSums = kSimtWarps * RR * D;
    // The warps' sums lie over the tiles at a piece's end.
    static constexpr int kBytes = 4 * (kQueries + kWeights + (kTiles > kSums ? kTiles : kSums));
    static_assert(kBytes <= 233472 / simt_blocks(D, RR) - 2048, "");
};

template <int D, int RR>
__global__ void __launch_bounds__(kSimtWarps * 32, simt_blocks(D, RR))
gdn_attention_simt_kernel(const __grid_constant__ AttentionArgs a) {
    using S = Simt<D, RR>;
    constexpr int WORDS = D / 4, E = D / 32, PER = E < 4 ? E : 4;
    constexpr float kNone = -__builtin_huge_valf();
    extern __shared__ __align__(16) float smem[];
    float *qs = smem;                // [RR][D]
    float *ps = qs + S::kQueries;    // [warps][RR][tokens]
    float *tiles = ps + S::kWeights;
    float *os = tiles;               // [warps][RR][D]
    __shared__ float2 ml[kSimtWarps][RR];
    __shared__ int lims[RR];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int tok = lane / 4, s = lane % 4;
    float *pw = ps + warp * RR * kSimtTokens;
    float *keys = tiles + warp * 2 * S::kHalf, *values = keys + S::kHalf;
    // Element e of a lane's part of a row.
    auto element = [&](int e) { return e / PER * 32 * PER + lane * PER + e % PER; };
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const Range range = find_range<kSimtChunk, 1, kSimtWarps * 32, 1>(a, a.Hkv * a.row_blocks, 0);
    for_pieces<kSimtChunk, 1, RR>(a, range, [&](const Unit &u, const Piece &piece) {
        const int t0 = piece.first_token<kSimtChunk, 1>(u.len), t1 = piece.last_token<kSimtChunk, 1>(u.len);
        const int slot = piece.whole() ? -1 : piece.slot(range.group);
        const int32_t *table = a.table + u.n * a.table_stride;
        bool bad = false;
        int64_t k_at = -1, v_at = -1;  // of this lane's token in the tile that is copied
        int entry = -1;                // and of the next one, its page
        auto look_up = [&](int j0) {
            const int j = j0 + tok;
            entry = j < t1 ? table[a.by_page.of(j)] : -1;
        };
        auto place = [&](int j0) {
            const int j = j0 + tok;
            k_at = v_at = -1;
            if (j >= t1) return;
            if (entry < 0 || entry >= a.num_pages) {
                bad = true;
                return;
            }
            const int at = j - a.by_page.of(j) * a.page_size;
            k_at = (uint32_t)entry * a.kps + (uint32_t)at * a.kts + (uint32_t)u.head * a.khs;
            v_at = (uint32_t)entry * a.vps + (uint32_t)at * a.vts + (uint32_t)u.head * a.vhs;
        };
        // Rows that do not exist become zeros.
        auto copy = [&](float *to, const void *from, int64_t at) {
#pragma unroll
            for (int w0 = 0; w0 < kSimtTokens * WORDS; w0 += 32) {
                const int r = (w0 + lane) / WORDS, w = (w0 + lane) % WORDS;
                const int64_t off = __shfl_sync(0xffffffffu, at, r * 4);
                copy_async_head(to + r * S::kPitch + w * 4,
                                static_cast<const char *>(from) + (off < 0 ? 0 : off + w * 16), off < 0 ? 0 : 16);
            }
            copies_commit();
        };
        constexpr int kStep = kSimtWarps * kSimtTokens;
        const int first = t0 + warp * kSimtTokens;
        __syncthreads();  // the last piece's sums and rows
        look_up(first);
        for (int i = threadIdx.x; i < RR * D; i += kSimtWarps * 32) {
            const int r = i / D;
            float v = 0.f;
            if (r < u.rows) {
                const RowPlace p = row_place(a, u, r);
                v = ((const float *)a.q)[p.token * a.qs + p.head * a.qh + i % D];
            }
            qs[i] = v;
        }
        if (threadIdx.x < RR)
            lims[threadIdx.x] = threadIdx.x < u.rows ? seen_by(a, u, threadIdx.x) : 0;
        if (first < t1) {
            place(first);
            copy(keys, a.k, k_at);
            look_up(first + kStep);
        }
        __syncthreads();
        float m[RR], l[RR], o[RR][E];
#pragma unroll
        for (int r = 0; r < RR; ++r) {
            m[r] = kNone, l[r] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[r][e] = 0.f;
        }
        const int all_see = u.len - a.L + 1;  // from here on not every row sees a token
#pragma unroll 1
        for (int j0 = first; j0 < t1; j0 += kStep) {
            const int j = j0 + tok;
            copies_wait<0>();
            __syncwarp();
            copy(values, a.v, v_at);
            float acc[RR];
#pragma unroll
            for (int r = 0; r < RR; ++r) acc[r] = 0.f;
#pragma unroll 4
            for (int i = s; i < WORDS; i += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(keys + tok * S::kPitch + i * 4);
#pragma unroll
                for (int r = 0; r < RR; ++r) {
                    const float4 y = *reinterpret_cast<const float4 *>(qs + r * D + i * 4);
                    acc[r] = fmaf(y.x, x.x, acc[r]);
                    acc[r] = fmaf(y.y, x.y, acc[r]);
                    acc[r] = fmaf(y.z, x.z, acc[r]);
                    acc[r] = fmaf(y.w, x.w, acc[r]);
                }
            }
            float fade[RR];
#pragma unroll
            for (int r = 0; r < RR; ++r) {
                float x = acc[r];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                x = j < t1 && j < lims[r] ? x * a.scale_log2 : kNone;
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
#pragma unroll
            for (int r = 0; r < RR; ++r)
#pragma unroll
                for (int e = 0; e < E; ++e) o[r][e] *= fade[r];
            copies_wait<0>();
            __syncwarp();
            if (j0 + kStep < t1) {
                place(j0 + kStep);
                copy(keys, a.k, k_at);
                look_up(j0 + 2 * kStep);
            }
            // Not every row sees the newest tokens, and what it does not see may
            // be infinite or NaN.
            const bool edge = j0 + kSimtTokens > all_see;
#pragma unroll
            for (int t = 0; t < kSimtTokens; ++t) {
                float x[E];
#pragma unroll
                for (int e = 0; e < E; e += PER)
                    Vec<float, PER>::load(values + t * S::kPitch + element(e)).to(x + e);
#pragma unroll
                for (int r = 0; r < RR; ++r) {
                    if (edge && j0 + t >= lims[r]) continue;
                    const float p = pw[r * kSimtTokens + t];
#pragma unroll
                    for (int e = 0; e < E; ++e) o[r][e] = fmaf(p, x[e], o[r][e]);
                }
            }
            __syncwarp();
        }
        bad = __any_sync(0xffffffffu, bad);
        __syncthreads();  // the tiles
        // The warps' sums, joined.
#pragma unroll
        for (int r = 0; r < RR; ++r) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
            if (bad) l[r] = __int_as_float(0x7fffffff);
            if (lane == 0) ml[warp][r] = make_float2(m[r], l[r]);
#pragma unroll
            for (int e = 0; e < E; ++e) os[(warp * RR + r) * D + element(e)] = o[r][e];
        }
        __syncthreads();
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
            if (slot < 0) {
                const RowPlace p = row_place(a, u, r);
                const float *gate =
                    a.gate ? (const float *)a.gate + p.token * a.gs + p.head * a.gh + e : nullptr;
                y *= inverse(sum);
                if (gate) y *= sigmoid(*gate);
                ((float *)a.out)[p.token * a.os + p.head * a.oh + e] = y;
                if (e == 0) store_lse(a, p, top, sum);
            } else {
                a.sums[((int64_t)slot * RR + r) * D + e] = y;
                if (e == 0) a.stats[slot * RR + r] = make_float2(top, sum);
            }
        }
    });
}

// Rows at a time: those of a unit, up to 16.
inline AttentionShape simt_shape(int R, int D) {
    const int rows = R <= 4 ? 4 : R <= 8 ? 8 : 16;
    return {rows, kSimtChunk, 1, 1, simt_blocks(D, rows) * kGridSms};
}

template <int D, int RR>
gdn_status simt_run(int blocks, const AttentionArgs &a, cudaStream_t stream) {
    constexpr size_t bytes = Simt<D, RR>::kBytes;
    static std::atomic<bool> done[kMaxDevices];
    const auto kernel = gdn_attention_simt_kernel<D, RR>;
    if (!raise_shared_memory(done, {reinterpret_cast<const void *>(kernel)}, {bytes}))
        return GDN_ERR_CUDA;
    return launch_programmatic(kernel, dim3(blocks), kSimtWarps * 32, bytes, stream, a);
}

template <int D> gdn_status simt_rows(int blocks, const AttentionArgs &a, cudaStream_t stream) {
    if (a.R <= 4) return simt_run<D, 4>(blocks, a, stream);
    if (a.R <= 8) return simt_run<D, 8>(blocks, a, stream);
    return simt_run<D, 16>(blocks, a, stream);
}

}  // namespace gdn

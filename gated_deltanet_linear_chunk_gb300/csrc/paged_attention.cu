// paged_attention.cu -- the join of paged_attention.cuh's pieces, the
// workspace and the choice of a kernel.
#include "paged_attention.cuh"

namespace gdn {
namespace {

constexpr int kJoinThreads = 256, kJoinBlocks = 16 * kGridSms;

// The pieces of one unit: block x is the block that left the first, y its rows,
// every gridDim.y-th.  Threads are four elements of a row each, several pieces
// at a time.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads)
gdn_attention_join_kernel(const __grid_constant__ AttentionArgs a, int rows) {
    constexpr int WORDS = D / 4, TEAMS = kJoinThreads / WORDS;
    constexpr float kNone = -__builtin_huge_valf();
    __shared__ float weight[kAttentionBlocks + 1];
    __shared__ float tops[kJoinThreads / 32], totals[kJoinThreads / 32];
    __shared__ float4 parts[kJoinThreads];
    ptx::griddep_wait();
    const int block = blockIdx.x;
    const int4 join = a.joins[block];
    Unit u;
    u.n = join.x;
    if (u.n < 0) return;
    u.head = join.y / a.row_blocks;
    u.first_row = join.y % a.row_blocks * rows;
    u.rows = min(rows, a.R - u.first_row);
    const int pieces = join.z + 1;
    // The first piece ends its block's range, the others begin theirs.
    auto slot = [&](int i) { return i == 0 ? 2 * block + 1 : 2 * (block + i); };
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int team = threadIdx.x / WORDS, word = threadIdx.x % WORDS;
    for (int r = blockIdx.y; r < u.rows; r += gridDim.y) {
        float top = kNone;
        for (int i = threadIdx.x; i < pieces; i += kJoinThreads)
            top = fmaxf(top, a.stats[slot(i) * rows + r].x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        if (lane == 0) tops[warp] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kJoinThreads / 32; ++w) top = fmaxf(top, tops[w]);
        float total = 0.f;
        for (int i = threadIdx.x; i < pieces; i += kJoinThreads) {
            const float2 s = a.stats[slot(i) * rows + r];
            const float f = ex2(s.x - against(top));
            weight[i] = f;
            total += s.y * f;
        }
        total = warp_sum(total);
        if (lane == 0) totals[warp] = total;
        __syncthreads();
        total = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinThreads / 32; ++w) total += totals[w];

        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int i = team; i < pieces; i += TEAMS) {
            const float4 x = reinterpret_cast<const float4 *>(
                a.sums)[((int64_t)slot(i) * rows + r) * WORDS + word];
            const float f = weight[i];
            y.x = fmaf(f, x.x, y.x);
            y.y = fmaf(f, x.y, y.y);
            y.z = fmaf(f, x.z, y.z);
            y.w = fmaf(f, x.w, y.w);
        }
        parts[threadIdx.x] = y;
        __syncthreads();
        const RowPlace p = row_place(a, u, r);
        const float inv = inverse(total);
        for (int e = threadIdx.x; e < D; e += kJoinThreads) {
            float sum = 0.f;
#pragma unroll
            for (int t = 0; t < TEAMS; ++t)
                sum += reinterpret_cast<const float *>(&parts[t * WORDS])[e];
            const T *gate = a.gate ? (const T *)a.gate + p.token * a.gs + p.head * a.gh + e : nullptr;
            ((T *)a.out)[p.token * a.os + p.head * a.oh + e] = from_f32<T>(finish(sum, inv, gate));
        }
        if (threadIdx.x == 0) store_lse(a, p, top, total);
    }
}

struct Plan {
    int rows, blocks, chunk;
    bool split;
    size_t joins, stats, sums;  // bytes
};

Plan plan(const gdn_attention_problem &p, const gdn_paged_cache &c) {
    Plan pl;
    const int R = p.new_tokens * (p.q_heads / p.kv_heads);
    const AttentionShape s = p.dtype == GDN_F32        ? shape_f32(R, p.head_dim)
                             : c.dtype == GDN_E4M3 ? shape_e4m3(R, p.head_dim)
                                                   : shape_bf16(R, p.head_dim);
    pl.rows = s.rows;
    pl.chunk = s.chunk;
    const int64_t units = (int64_t)c.num_seqs * p.kv_heads * ((R + s.rows - 1) / s.rows);
    const int64_t chunks =
        ((int64_t)c.max_pages * c.page_size + s.chunk - 1) / s.chunk;  // of a unit, at most
    const int64_t all = units * (chunks > 1 ? chunks : 1);
    pl.blocks = (int)(all < s.blocks ? all : s.blocks);
    pl.split = chunks > 1;
    pl.joins = pl.split ? (size_t)pl.blocks * sizeof(int4) : 0;
    pl.stats = pl.split ? (size_t)pl.blocks * 2 * s.rows * sizeof(float2) : 0;
    pl.sums = pl.split ? (size_t)pl.blocks * 2 * s.rows * p.head_dim * sizeof(float) : 0;
    return pl;
}

template <typename T, int D>
gdn_status join(const AttentionArgs &a, const Plan &pl, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const int rows = pl.rows < a.R ? pl.rows : a.R, fit = kJoinBlocks / pl.blocks;
    cfg.gridDim = dim3(pl.blocks, rows < fit ? rows : fit);
    cfg.blockDim = dim3(kJoinThreads);
    return cudaLaunchKernelEx(&cfg, gdn_attention_join_kernel<T, D>, a, pl.rows) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
}

}  // namespace

size_t paged_attention_workspace(const gdn_attention_problem &p, const gdn_paged_cache &c) {
    if (c.num_seqs == 0) return 0;
    const Plan pl = plan(p, c);
    return pl.joins + pl.stats + pl.sums;
}

gdn_status launch_paged_attention(const gdn_attention_problem &p, const gdn_paged_cache &c,
                                  const void *q, const void *gate, void *out, float *lse,
                                  cudaStream_t stream) {
    const Plan pl = plan(p, c);
    AttentionArgs a = {};
    a.q = q, a.gate = gate, a.out = out, a.lse = lse;
    a.k = c.k, a.v = c.v, a.k_scale = c.k_scale, a.v_scale = c.v_scale;
    a.table = c.page_table, a.lens = c.seq_lens;
    a.qs = p.q_stride, a.qh = p.q_head_stride;
    a.gs = p.gate_stride, a.gh = p.gate_head_stride;
    a.os = p.out_stride, a.oh = p.out_head_stride;
    a.kps = c.k_page_stride, a.kts = c.k_token_stride, a.khs = c.k_head_stride;
    a.vps = c.v_page_stride, a.vts = c.v_token_stride, a.vhs = c.v_head_stride;
    a.table_stride = c.table_stride, a.num_pages = c.num_pages;
    a.N = c.num_seqs, a.L = p.new_tokens, a.Hkv = p.kv_heads;
    a.G = p.q_heads / p.kv_heads;
    a.R = a.L * a.G;
    a.row_blocks = (a.R + pl.rows - 1) / pl.rows;
    a.page_size = c.page_size;
    a.capacity = c.max_pages * c.page_size;
    a.scale_log2 = p.scale * kLog2e;
    auto words = [&](const void *x, int64_t stride, int64_t head_stride) {
        const uint64_t size = p.dtype == GDN_F32 ? 4 : 2;
        return aligned16(x) && (((a.N * a.L > 1 ? stride : 0) | (p.q_heads > 1 ? head_stride : 0)) * size) % 16 == 0;
    };
    a.q_words = words(q, p.q_stride, p.q_head_stride);
    a.gate_words = words(gate, p.gate_stride, p.gate_head_stride);
    a.out_words = words(out, p.out_stride, p.out_head_stride);
    if (pl.split) {
        // The sums first: they are read in 16-byte words.
        char *w = static_cast<char *>(p.workspace);
        a.sums = reinterpret_cast<float *>(w);
        a.joins = reinterpret_cast<int4 *>(w + pl.sums);
        a.stats = reinterpret_cast<float2 *>(w + pl.sums + pl.joins);
    }
    const gdn_status st = p.dtype == GDN_F32      ? attention_f32(p.head_dim, pl.blocks, a, stream)
                          : c.dtype == GDN_E4M3 ? attention_e4m3(p.head_dim, pl.blocks, a, stream)
                                                : attention_bf16(p.head_dim, pl.blocks, a, stream);
    if (st != GDN_OK || !pl.split) return st;
    const bool f32 = p.dtype == GDN_F32;
    switch (p.head_dim) {
        case 64: return f32 ? join<float, 64>(a, pl, stream) : join<__nv_bfloat16, 64>(a, pl, stream);
        case 128: return f32 ? join<float, 128>(a, pl, stream) : join<__nv_bfloat16, 128>(a, pl, stream);
        default: return f32 ? join<float, 256>(a, pl, stream) : join<__nv_bfloat16, 256>(a, pl, stream);
    }
}

}  // namespace gdn

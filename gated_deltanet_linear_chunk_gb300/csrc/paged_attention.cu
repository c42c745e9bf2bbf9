// paged_attention.cu -- the join of paged_attention.cuh's pieces, the
// workspace and the choice of a kernel.
#include "paged_attention.cuh"

namespace gdn {
namespace {

constexpr int kJoinThreads = 256, kJoinBlocks = 8 * kGridSms, kJoinAlone = 12;
// Pieces that a thread looks over, at most.
constexpr int kJoinEach = (kAttentionGroups + kJoinThreads) / kJoinThreads;

// The join of a unit: four elements of the sums of piece i, times f.
template <int D>
__device__ __forceinline__ void add_piece(const AttentionArgs &a, float4 &y, int slot, int rows, int r,
                                          int word, float f) {
    const float4 x =
        reinterpret_cast<const float4 *>(a.sums)[((int64_t)slot * rows + r) * (D / 4) + word];
    y.x = fmaf(f, x.x, y.x);
    y.y = fmaf(f, x.y, y.y);
    y.z = fmaf(f, x.z, y.z);
    y.w = fmaf(f, x.w, y.w);
}
template <typename T>
__device__ __forceinline__ void store_joined(const AttentionArgs &a, const RowPlace &p, int e, float inv,
                                             const float4 &y) {
    const float x[4] = {y.x, y.y, y.z, y.w};
    const T *gate = a.gate ? (const T *)a.gate + p.token * a.gs + p.head * a.gh + e : nullptr;
    T *out = (T *)a.out + p.token * a.os + p.head * a.oh + e;
    float by[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) by[i] = gate ? to_f32(gate[i]) : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = from_f32<T>(gate ? x[i] * inv * sigmoid(by[i]) : x[i] * inv);
}

// Joins the pieces of one unit: block x of the units, y of its rows (every
// gridDim.y-th).  Few pieces are a warp's work, a row each; many are a block's:
// threads take four elements of a row, several pieces at a time.  Its loads
// depend on one another three deep (join, statistics, sums), which is its time:
// 10 us alone with a cold cache, for 24 rows of 76 pieces as for 1536 rows of a
// few; part of that is beside the end of the attention.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads)
gdn_attention_join_kernel(const __grid_constant__ AttentionArgs a, int rows) {
    constexpr int WORDS = D / 4, TEAMS = kJoinThreads / WORDS, WARPS = kJoinThreads / 32;
    constexpr float kNone = -__builtin_huge_valf();
    __shared__ float weight[kAttentionGroups + 1];
    __shared__ int slots[kAttentionGroups + 1], counts[kJoinEach * (kJoinThreads / 32)];
    __shared__ float tops[WARPS], totals[WARPS];
    __shared__ float4 parts[kJoinThreads];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int per_seq = a.Hkv * a.row_blocks, unit = blockIdx.x % per_seq;
    Unit u;
    u.n = blockIdx.x / per_seq;
    u.head = unit / a.row_blocks;
    u.first_row = unit % a.row_blocks * rows;
    u.rows = min(rows, a.R - u.first_row);
    u.len = 0;
    ptx::griddep_wait();
    const int2 join = a.joins[blockIdx.x];
    const int group = join.x;
    if (group < 0) return;
    const int pieces = join.y + 1;
    // The first piece ends its group's range, the others begin theirs.
    auto slot = [&](int i) { return i == 0 ? 2 * group + 1 : 2 * (group + i); };

    if (pieces <= kJoinAlone) {
        for (int r = blockIdx.y * WARPS + warp; r < u.rows; r += gridDim.y * WARPS) {
            const float2 s = lane < pieces ? a.stats[slot(lane) * rows + r] : make_float2(kNone, 0.f);
            float top = s.x;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float f = ex2(s.x - against(top));
            const float total = warp_sum(s.y * f);
            const bool some = s.x != kNone || s.y != 0.f;
            const unsigned have = __ballot_sync(0xffffffffu, some);
            const RowPlace p = row_place(a, u, r);
#pragma unroll
            for (int w0 = 0; w0 < WORDS; w0 += 32) {  // all lanes take part in the shuffles
                const int w = w0 + lane;
                const bool mine = WORDS >= 32 || w < WORDS;
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int i = 0; i < pieces; ++i) {
                    const float fi = __shfl_sync(0xffffffffu, f, i);
                    if (mine && (have >> i & 1)) add_piece<D>(a, y, slot(i), rows, r, w, fi);
                }
                if (mine) store_joined<T>(a, p, w * 4, inverse(total), y);
            }
            if (lane == 0) store_lse(a, p, top, total);
        }
        return;
    }

    const int team = threadIdx.x / WORDS, word = threadIdx.x % WORDS;
    for (int r = blockIdx.y; r < u.rows; r += gridDim.y) {
        float2 s[kJoinEach];
        float top = kNone;
#pragma unroll
        for (int k = 0; k < kJoinEach; ++k) {
            const int i = k * kJoinThreads + threadIdx.x;
            s[k] = i < pieces ? a.stats[slot(i) * rows + r] : make_float2(kNone, 0.f);
            top = fmaxf(top, s[k].x);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        if (lane == 0) tops[warp] = top;
        // The pieces that have sums, in their order.
#pragma unroll
        for (int k = 0; k < kJoinEach; ++k) {
            const unsigned have = __ballot_sync(0xffffffffu, s[k].x != kNone || s[k].y != 0.f);
            if (lane == 0) counts[k * WARPS + warp] = __popc(have);
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WARPS; ++w) top = fmaxf(top, tops[w]);
        float total = 0.f;
        int some = 0;
#pragma unroll
        for (int k = 0; k < kJoinEach; ++k) {
            const float f = ex2(s[k].x - against(top));
            total += s[k].y * f;
            const bool has = s[k].x != kNone || s[k].y != 0.f;
            const unsigned have = __ballot_sync(0xffffffffu, has);
            int before = some;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                if (w < warp) before += counts[k * WARPS + w];
                some += counts[k * WARPS + w];
            }
            if (has) {
                const int to = before + __popc(have & ((1u << lane) - 1));
                weight[to] = f;
                slots[to] = slot(k * kJoinThreads + threadIdx.x);
            }
        }
        total = warp_sum(total);
        if (lane == 0) totals[warp] = total;
        __syncthreads();
        total = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) total += totals[w];
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int i = team; i < some; i += TEAMS) add_piece<D>(a, y, slots[i], rows, r, word, weight[i]);
        parts[threadIdx.x] = y;
        __syncthreads();
        const RowPlace p = row_place(a, u, r);
        if (threadIdx.x < WORDS) {
#pragma unroll
            for (int t = 1; t < TEAMS; ++t) {
                const float4 x = parts[t * WORDS + threadIdx.x];
                y.x += x.x, y.y += x.y, y.z += x.z, y.w += x.w;
            }
            store_joined<T>(a, p, threadIdx.x * 4, inverse(total), y);
        }
        if (threadIdx.x == 0) store_lse(a, p, top, total);
    }
}

struct Plan {
    int rows, blocks, groups;
    int64_t units;
    size_t joins, stats, sums;  // bytes
};

Plan plan(const gdn_attention_problem &p, const gdn_paged_cache &c) {
    Plan pl;
    const int R = p.new_tokens * (p.q_heads / p.kv_heads);
    const AttentionShape s = p.dtype == GDN_F32        ? shape_f32(R, p.head_dim)
                             : c.dtype == GDN_E4M3 ? shape_e4m3(R, p.head_dim)
                                                   : shape_bf16(R, p.head_dim);
    pl.rows = s.rows;
    pl.units = (int64_t)c.num_seqs * p.kv_heads * ((R + s.rows - 1) / s.rows);
    const int64_t tiles = s.setup + ((int64_t)c.max_pages * c.page_size + s.tokens - 1) / s.tokens;
    const int64_t need = (pl.units * tiles + s.groups - 1) / s.groups;  // blocks, at most
    pl.blocks = (int)(need < s.blocks ? need : s.blocks);
    pl.groups = pl.blocks * s.groups;
    // Any unit can be cut, also one without tokens.
    pl.joins = ((size_t)pl.units * sizeof(int2) + 15) / 16 * 16;
    pl.stats = (size_t)pl.groups * 2 * s.rows * sizeof(float2);
    pl.sums = (size_t)pl.groups * 2 * s.rows * p.head_dim * sizeof(float);
    return pl;
}

template <typename T, int D>
gdn_status join(const AttentionArgs &a, const Plan &pl, cudaStream_t stream) {
    const int rows = pl.rows < a.R ? pl.rows : a.R;
    const int fit = kJoinBlocks > pl.units ? (int)(kJoinBlocks / pl.units) : 1;
    return launch_programmatic(gdn_attention_join_kernel<T, D>, dim3((unsigned)pl.units, rows < fit ? rows : fit),
                               kJoinThreads, 0, stream, a, pl.rows);
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
    const int64_t e = c.dtype == GDN_F32 ? 4 : c.dtype == GDN_E4M3 ? 1 : 2;
    a.kps = c.k_page_stride * e, a.kts = c.k_token_stride * e, a.khs = c.k_head_stride * e;
    a.vps = c.v_page_stride * e, a.vts = c.v_token_stride * e, a.vhs = c.v_head_stride * e;
    a.table_stride = c.table_stride, a.num_pages = c.num_pages;
    a.N = c.num_seqs, a.L = p.new_tokens, a.Hkv = p.kv_heads;
    a.G = p.q_heads / p.kv_heads;
    a.R = a.L * a.G;
    a.row_blocks = (a.R + pl.rows - 1) / pl.rows;
    a.inv_group = 1.f / (float)a.G;
    a.page_size = c.page_size;
    a.by_page = Division::by(c.page_size);
    a.capacity = c.max_pages * c.page_size;
    a.scale_log2 = p.scale * kLog2e;
    auto words = [&](const void *x, int64_t stride, int64_t head_stride) {
        const uint64_t size = p.dtype == GDN_F32 ? 4 : 2;
        return aligned16(x) && (((a.N * a.L > 1 ? stride : 0) | (p.q_heads > 1 ? head_stride : 0)) * size) % 16 == 0;
    };
    a.q_words = words(q, p.q_stride, p.q_head_stride);
    a.gate_words = words(gate, p.gate_stride, p.gate_head_stride);
    a.out_words = words(out, p.out_stride, p.out_head_stride);
    // Multiples of 16 bytes first: they are read in such words.
    char *w = static_cast<char *>(p.workspace);
    a.sums = reinterpret_cast<float *>(w);
    a.joins = reinterpret_cast<int2 *>(w + pl.sums);
    a.stats = reinterpret_cast<float2 *>(w + pl.sums + pl.joins);
    const gdn_status st = p.dtype == GDN_F32      ? attention_f32(p.head_dim, pl.blocks, a, stream)
                          : c.dtype == GDN_E4M3 ? attention_e4m3(p.head_dim, pl.blocks, a, stream)
                                                : attention_bf16(p.head_dim, pl.blocks, a, stream);
    if (st != GDN_OK) return st;
    const bool f32 = p.dtype == GDN_F32;
    switch (p.head_dim) {
        case 64: return f32 ? join<float, 64>(a, pl, stream) : join<__nv_bfloat16, 64>(a, pl, stream);
        case 128: return f32 ? join<float, 128>(a, pl, stream) : join<__nv_bfloat16, 128>(a, pl, stream);
        default: return f32 ? join<float, 256>(a, pl, stream) : join<__nv_bfloat16, 256>(a, pl, stream);
    }
}

}  // namespace gdn

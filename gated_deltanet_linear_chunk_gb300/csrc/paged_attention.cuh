// paged_attention.cuh -- attention of one to eight new tokens of each sequence
// over its paged cache: what its kernels share.
//
// A unit is one key head of one sequence and a block of the rows (new tokens
// times query heads of the group) that attend to it; the softmax runs in one
// pass over the unit's tokens with a running maximum and sum.  The cache is
// read once, which bounds the operator, and every SM has to read its share of
// it, whatever the lengths are: the chunks (of a fixed number of tokens) of all
// units, one unit after the other, are divided evenly among the blocks, which
// find their place from the lengths on the device.  A block's range begins and
// ends inside units: what it has of those goes to the workspace, one piece for
// the range's begin and one for its end, and a second launch joins the pieces
// in their order.
#pragma once

#include "attention.cuh"
#include "sm103.cuh"

namespace gdn {

constexpr float kLn2 = 0.6931471805599453f;

struct AttentionArgs {
    const void *q, *gate;
    void *out;
    float *lse;
    const void *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *table, *lens;
    int64_t qs, qh, gs, gh, os, oh;
    int64_t kps, kts, khs, vps, vts, vhs, table_stride;
    int64_t num_pages;
    int N, L, Hkv, G, R, row_blocks, page_size, capacity;
    bool q_words, gate_words, out_words;  // rows of q, gate and out in whole 16-byte words
    float scale_log2;  // scale log2 e: scores in powers of two
    // workspace
    int4 *joins;     // [blocks] the unit whose first piece the block left: n, unit, blocks after it
    float2 *stats;   // [blocks, 2, row block] maximum and sum
    float *sums;     // [blocks, 2, row block, D]
};

// Rows of a unit's row block: tokens t = r / G, heads h G + r % G.
struct Unit {
    int n, head, first_row, rows, len;
};

__device__ __forceinline__ int held_tokens(const AttentionArgs &a, int n) {
    return min(max(a.lens[n], 0), a.capacity);
}
template <int CHUNK> __device__ __forceinline__ int chunks_of(int len) {
    return max(1, (len + CHUNK - 1) / CHUNK);  // an empty sequence has its rows to write
}

// A block's range of chunks.  (No more blocks than chunks have one: pieces of a
// unit are those of blocks that follow one another.)
struct Range {
    int64_t begin, end, total;
    int block, blocks;
    int n;          // the sequence it begins in
    int64_t base;   // that sequence's first chunk
};

// The first chunk of block b, and the block of a chunk.
__device__ __forceinline__ int64_t first_chunk(int64_t total, int blocks, int b) {
    return total * b / blocks;
}
__device__ __forceinline__ int block_of(int64_t total, int blocks, int64_t chunk) {
    return (int)(((chunk + 1) * blocks - 1) / total);
}

// By all threads of a block: sums over the sequences, a run of them per thread.
template <int CHUNK, int THREADS>
__device__ Range find_range(const AttentionArgs &a, int per_seq) {
    __shared__ int64_t warp_sums[THREADS / 32], found_base;
    __shared__ int found;
    const int run = (a.N + THREADS - 1) / THREADS;
    const int n0 = min((int)threadIdx.x * run, a.N), n1 = min(n0 + run, a.N);
    int64_t mine = 0;
    for (int n = n0; n < n1; ++n) mine += chunks_of<CHUNK>(held_tokens(a, n));
    int64_t upto = mine;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t below = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += below;
    }
    if (lane == 31) warp_sums[warp] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) upto += warp_sums[w];
        total += warp_sums[w];
    }
    Range r;
    r.total = total * per_seq;
    r.block = blockIdx.x;
    r.blocks = (int)min((int64_t)gridDim.x, r.total);
    r.begin = r.block < r.blocks ? first_chunk(r.total, r.blocks, r.block) : r.total;
    r.end = r.block < r.blocks ? first_chunk(r.total, r.blocks, r.block + 1) : r.total;
    if (threadIdx.x == 0) found = 0;
    __syncthreads();
    int64_t base = (upto - mine) * per_seq;
    if (r.begin >= base && r.begin < upto * per_seq) {
        for (int n = n0; n < n1; ++n) {
            const int64_t next = base + (int64_t)chunks_of<CHUNK>(held_tokens(a, n)) * per_seq;
            if (r.begin < next) {
                found = n;
                found_base = base;
                break;
            }
            base = next;
        }
    }
    __syncthreads();
    r.n = found;
    r.base = found_base;
    return r;
}

// Where row r of a unit lies in q, gate, out (times its strides) and lse.
struct RowPlace {
    int64_t token;
    int head;
};
__device__ __forceinline__ RowPlace row_place(const AttentionArgs &a, const Unit &u, int r) {
    const int row = u.first_row + r;
    return {(int64_t)u.n * a.L + row / a.G, u.head * a.G + row % a.G};
}
// How many of the unit's tokens row r sees.
__device__ __forceinline__ int seen_by(const AttentionArgs &a, const Unit &u, int r) {
    return u.len - a.L + 1 + (u.first_row + r) / a.G;
}

// Runs `piece(unit, first token, last token, slot)` over a block's range; slot
// -1: the whole unit, else the workspace's.
template <int CHUNK, int ROWS, typename F>
__device__ __forceinline__ void for_pieces(const AttentionArgs &a, const Range &g, F &&piece) {
    const int per_seq = a.Hkv * a.row_blocks;
    int4 join = make_int4(-1, 0, 0, 0);
    if (g.begin >= g.end) {
        if (a.joins && threadIdx.x == 0) a.joins[g.block] = join;
        return;
    }
    int n = g.n, len = held_tokens(a, n), chunks = chunks_of<CHUNK>(len);
    int unit = (int)((g.begin - g.base) / chunks), c = (int)((g.begin - g.base) % chunks);
    for (int64_t pos = g.begin; pos < g.end;) {
        const int c1 = (int)min((int64_t)chunks, c + (g.end - pos));
        Unit u;
        u.n = n;
        u.head = unit / a.row_blocks;
        u.first_row = unit % a.row_blocks * ROWS;
        u.rows = min(ROWS, a.R - u.first_row);
        u.len = len;
        const bool first = c == 0, last = c1 == chunks;
        if (first && !last)  // the pieces after it: up to the block of the unit's last chunk
            join = make_int4(n, unit, block_of(g.total, g.blocks, pos + chunks - 1) - g.block, 0);
        piece(u, min(c * CHUNK, len), min(c1 * CHUNK, len),
              first && last ? -1 : 2 * g.block + (first ? 1 : 0));
        pos += c1 - c;
        c = 0;
        if (++unit == per_seq && pos < g.end) {
            unit = 0;
            len = held_tokens(a, ++n);
            chunks = chunks_of<CHUNK>(len);
        }
    }
    if (a.joins && threadIdx.x == 0) a.joins[g.block] = join;
}

// A row's element i, divided by the sum and gated.
template <typename T>
__device__ __forceinline__ float finish(float sum, float inv, const T *gate) {
    float y = sum * inv;
    if (gate) y *= sigmoid(to_f32(*gate));
    return y;
}
__device__ __forceinline__ void store_lse(const AttentionArgs &a, const RowPlace &p, float m,
                                          float l) {
    if (a.lse)
        a.lse[p.token * (a.Hkv * a.G) + p.head] =
            l == 0.f ? __int_as_float(0xff800000) : (m + log2f(l)) * kLn2;
}
// Zeros for a row without weights: its sums are zeros.
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

// The maximum that exponents are taken against: a finite one where there is
// none yet.
__device__ __forceinline__ float against(float m) {
    return m == __int_as_float(0xff800000) ? 0.f : m;
}

// E consecutive elements of the cache as fp32, in words of up to 16 bytes.
template <int E> __device__ __forceinline__ void load_cached(const float *p, float (&x)[E]) {
    constexpr int V = E < 4 ? E : 4;
#pragma unroll
    for (int i = 0; i < E; i += V) {
        float w[V];
        Vec<float, V>::load(p + i).to(w);
#pragma unroll
        for (int j = 0; j < V; ++j) x[i + j] = w[j];
    }
}
template <int E> __device__ __forceinline__ void load_cached(const __nv_bfloat16 *p, float (&x)[E]) {
    Vec<__nv_bfloat16, E>::load(p).to(x);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return __half22float2(__half2(h));
}
template <int E> __device__ __forceinline__ void load_cached(const __nv_fp8_e4m3 *p, float (&x)[E]) {
#pragma unroll
    for (int i = 0; i < E; i += 2) {
        const float2 v = from_e4m3x2(*reinterpret_cast<const uint16_t *>(p + i));
        x[i] = v.x, x[i + 1] = v.y;
    }
}

// What a kernel takes at a time, for units of R rows: rows, the chunk, and its
// blocks on a GB300.
struct AttentionShape {
    int rows, chunk, blocks;
};
constexpr int kAttentionBlocks = 2 * kGridSms;  // at most
AttentionShape shape_f32(int R, int D);
AttentionShape shape_bf16(int R, int D);
AttentionShape shape_e4m3(int R, int D);
gdn_status attention_f32(int D, int blocks, const AttentionArgs &a, cudaStream_t stream);
gdn_status attention_bf16(int D, int blocks, const AttentionArgs &a, cudaStream_t stream);
gdn_status attention_e4m3(int D, int blocks, const AttentionArgs &a, cudaStream_t stream);

}  // namespace gdn

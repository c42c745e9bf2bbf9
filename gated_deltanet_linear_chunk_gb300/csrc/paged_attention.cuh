// paged_attention.cuh -- attention of one to eight new tokens of each sequence
// over its paged cache: what its kernels share.
//
// A unit is one key head of one sequence and a block of the rows (new tokens
// times query heads of the group) that attend to it; the softmax runs in one
// pass over the unit's tokens with a running maximum and sum.  The cache is
// read once, which bounds the operator, and every SM has to read its share of
// it, whatever the lengths are: the tiles (of a fixed number of tokens) of all
// units, one unit after the other, are divided evenly among groups of warps,
// which find their place from the lengths on the device.  A unit counts a few
// tiles more than it has, for what its queries and results cost: its first
// tiles have no tokens.  A group's range begins and ends inside units: what it has of those
// goes to the workspace, one piece for the range's begin and one for its end,
// and a second launch joins the pieces in their order.
#pragma once

#include "attention.cuh"
#include "sm103.cuh"

namespace gdn {

constexpr float kLn2 = 0.6931471805599453f;

// x / d for 0 <= x < 2^30 and d up to 2^20, as one product: with s = ceil(log2 d)
// the factor 2^(30 + s) / d, rounded up, is off by less than one in d <= 2^s, so
// the quotient of x by less than x / 2^30 of a step.
struct Division {
    uint32_t factor;
    int shift;
    static Division by(int d) {
        int s = 0;
        while ((1 << s) < d) ++s;
        const uint64_t two = 1ull << (30 + s);
        return {(uint32_t)((two + d - 1) / d), 30 + s};
    }
    __host__ __device__ __forceinline__ int of(int x) const {
        return (int)((uint64_t)(uint32_t)x * factor >> shift);
    }
};

// Strides of q, gate and out are in elements, of the cache in bytes.
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
    float inv_group;         // 1 / G
    Division by_page;        // tokens by page_size
    bool q_words, gate_words, out_words;  // rows of q, gate and out in whole 16-byte words
    float scale_log2;  // scale log2 e: scores in powers of two
    // workspace
    int2 *joins;     // [units] where the unit was cut: its first piece's group, groups after it
    float2 *stats;   // [groups, 2, row block] maximum and sum; -infinity and 0: no sums
    float *sums;     // [groups, 2, row block, D]
};

// Rows of a unit's row block: tokens t = r / G, heads h G + r % G.
struct Unit {
    int n, head, first_row, rows, len;
};

__device__ __forceinline__ int held_tokens(const AttentionArgs &a, int n) {
    return min(max(a.lens[n], 0), a.capacity);
}
// SETUP of them, at least one, are without tokens and come first.
template <int TOKENS, int SETUP> __device__ __forceinline__ int tiles_of(int len) {
    return SETUP + (len + TOKENS - 1) / TOKENS;
}

// A group's range of tiles, and that of its block's groups together.  (No more
// groups than tiles have one: pieces of a unit are those of groups that follow
// one another.)
struct Range {
    int64_t begin, end, total, block_end;
    int group, groups;
    int n, len;     // the sequence it begins in, and its tokens
    int4 together;  // of the block, where it lies inside one unit: 1, n, the unit, and
                    // whether its first (1) and last tile (2) are among the block's
    int64_t base;   // that sequence's first tile
};

// The first tile of a group, and the group of a tile.
__host__ __device__ __forceinline__ int64_t first_tile(int64_t total, int groups, int group) {
    return group < groups ? total * group / groups : total;
}
__host__ __device__ __forceinline__ int group_of(int64_t total, int groups, int64_t tile) {
    return (int)(((tile + 1) * groups - 1) / total);
}

// By all threads of a block: sums over the sequences, a run of them per thread.
// `mine`: the thread's group in the block, of GROUPS.
template <int TOKENS, int SETUP, int THREADS, int GROUPS>
__device__ Range find_range(const AttentionArgs &a, int per_seq, int mine) {
    __shared__ int64_t warp_sums[THREADS / 32], found_base[GROUPS];
    __shared__ int found[GROUPS], found_len[GROUPS];
    __shared__ int4 together;
    const int run = (a.N + THREADS - 1) / THREADS;
    const int n0 = min((int)threadIdx.x * run, a.N), n1 = min(n0 + run, a.N);
    int64_t count = 0;
    for (int n = n0; n < n1; ++n) count += tiles_of<TOKENS, SETUP>(held_tokens(a, n));
    int64_t upto = count;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t below = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += below;
    }
    if (lane == 31) warp_sums[warp] = upto;
    if (threadIdx.x == 0) together = make_int4(0, 0, 0, 0);
    if (threadIdx.x < GROUPS) found[threadIdx.x] = found_len[threadIdx.x] = 0, found_base[threadIdx.x] = 0;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) upto += warp_sums[w];
        total += warp_sums[w];
    }
    Range r;
    r.total = total * per_seq;
    r.groups = (int)min((int64_t)gridDim.x * GROUPS, r.total);
    r.block_end = first_tile(r.total, r.groups, (blockIdx.x + 1) * GROUPS);
    const int64_t base = (upto - count) * per_seq;
#pragma unroll 1
    for (int g = 0; g < GROUPS; ++g) {
        const int64_t begin = first_tile(r.total, r.groups, blockIdx.x * GROUPS + g);
        if (begin < base || begin >= upto * per_seq) continue;
        int64_t at = base;
        for (int n = n0; n < n1; ++n) {
            const int len = held_tokens(a, n);
            const int64_t next = at + (int64_t)tiles_of<TOKENS, SETUP>(len) * per_seq;
            if (begin < next) {
                found[g] = n;
                found_len[g] = len;
                found_base[g] = at;
                if (GROUPS > 1 && g == 0) {
                    const int tiles = tiles_of<TOKENS, SETUP>(len);
                    const int unit = (int)((begin - at) / tiles), first = (int)((begin - at) % tiles);
                    const int64_t last = first + r.block_end - begin;
                    if (last <= tiles)
                        together = make_int4(1, n, unit, (first == 0 ? 1 : 0) | (last == tiles ? 2 : 0));
                }
                break;
            }
            at = next;
        }
    }
    __syncthreads();
    r.group = blockIdx.x * GROUPS + mine;
    r.begin = first_tile(r.total, r.groups, r.group);
    r.end = first_tile(r.total, r.groups, r.group + 1);
    r.together = together;
    r.n = found[mine];
    r.len = found_len[mine];
    r.base = found_base[mine];
    return r;
}

// The new token of a row, row / G: the quotient is at most 8 (and a block's
// rows beyond), so its rounding, some 2^-20, is far from the half step of at
// least 2^-13 that the sum begins with.
__device__ __forceinline__ int row_token(const AttentionArgs &a, int row) {
    return (int)(((float)row + 0.5f) * a.inv_group);
}
// Where row r of a unit lies in q, gate, out (times its strides) and lse.
struct RowPlace {
    int64_t token;
    int head;
};
__device__ __forceinline__ RowPlace row_place(const AttentionArgs &a, const Unit &u, int r) {
    const int row = u.first_row + r, t = row_token(a, row);
    return {(int64_t)u.n * a.L + t, u.head * a.G + row - t * a.G};
}
// How many of the unit's tokens row r sees.
__device__ __forceinline__ int seen_by(const AttentionArgs &a, const Unit &u, int r) {
    return u.len - a.L + 1 + row_token(a, u.first_row + r);
}

// What a group has of a unit: tiles [first, last) of `tiles`.
struct Piece {
    int unit, tiles, first, last;
    __device__ __forceinline__ bool whole() const { return first == 0 && last == tiles; }
    // The workspace's slot: the begin of a unit ends its group's range.
    __device__ __forceinline__ int slot(int group) const { return 2 * group + (first == 0 ? 1 : 0); }
    template <int TOKENS, int SETUP> __device__ __forceinline__ int first_token(int len) const {
        return min(max(first - SETUP, 0) * TOKENS, len);
    }
    template <int TOKENS, int SETUP> __device__ __forceinline__ int last_token(int len) const {
        return min(max(last - SETUP, 0) * TOKENS, len);
    }
};
template <int ROWS>
__device__ __forceinline__ Unit unit_of(const AttentionArgs &a, int n, int unit, int len) {
    Unit u;
    u.n = n;
    u.head = unit / a.row_blocks;
    u.first_row = unit % a.row_blocks * ROWS;
    u.rows = min(ROWS, a.R - u.first_row);
    u.len = len;
    return u;
}
// The join of a unit of `tiles` from `at` on, of which a group has the first
// `last`; {-1, 0} where that is all.
__device__ __forceinline__ int2 join_from(const Range &g, int group, int last, int tiles, int64_t at) {
    return last == tiles ? make_int2(-1, 0)
                         : make_int2(group, group_of(g.total, g.groups, at + tiles - 1) - group);
}

// Runs `work(unit, piece)` over a block's range, its only group's.
template <int TOKENS, int SETUP, int ROWS, typename F>
__device__ __forceinline__ void for_pieces(const AttentionArgs &a, const Range &g, F &&work) {
    const int per_seq = a.Hkv * a.row_blocks;
    if (g.begin >= g.end) return;
    int n = g.n, len = g.len;
    Piece p;
    p.tiles = tiles_of<TOKENS, SETUP>(len);
    p.unit = (int)((g.begin - g.base) / p.tiles);
    p.first = (int)((g.begin - g.base) % p.tiles);
    for (int64_t pos = g.begin; pos < g.end;) {
        p.last = (int)min((int64_t)p.tiles, p.first + (g.end - pos));
        if (p.first == 0 && threadIdx.x == 0)
            a.joins[(int64_t)n * per_seq + p.unit] = join_from(g, g.group, p.last, p.tiles, pos);
        work(unit_of<ROWS>(a, n, p.unit, len), p);
        pos += p.last - p.first;
        p.first = 0;
        if (++p.unit == per_seq && pos < g.end) {
            p.unit = 0;
            len = held_tokens(a, ++n);
            p.tiles = tiles_of<TOKENS, SETUP>(len);
        }
    }
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

__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return __half22float2(__half2(h));
}
// What a kernel takes at a time, for units of R rows: rows, the tokens of a
// tile, a unit's tiles without any, groups per block and its blocks on a GB300.
struct AttentionShape {
    int rows, tokens, setup, groups, blocks;
};
constexpr int kAttentionGroups = 8 * kGridSms;  // at most
AttentionShape shape_f32(int R, int D);
AttentionShape shape_bf16(int R, int D);
AttentionShape shape_e4m3(int R, int D);
gdn_status attention_f32(int D, int blocks, const AttentionArgs &a, cudaStream_t stream);
gdn_status attention_bf16(int D, int blocks, const AttentionArgs &a, cudaStream_t stream);
gdn_status attention_e4m3(int D, int blocks, const AttentionArgs &a, cudaStream_t stream);

}  // namespace gdn

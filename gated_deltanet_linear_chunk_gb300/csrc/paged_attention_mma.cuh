// paged_attention_mma.cuh -- the attention of paged_attention.cuh for bf16
// queries over a bf16 or an 8-bit cache.
//
// Every element of the cache takes part in as many products as there are rows
// (query heads that share a key head, times new tokens): far fewer than the 280
// per byte at which a GB300's tensor cores would bound the operator, and more
// than fp32 units do beside a stream at full bandwidth.  So the products are
// warp-wide ones (m16n8k16) straight from the tiles that the copies land in,
// which have no setup, and the design is about keeping copies in flight: a
// group of warps has a ring of half stages (a tile's keys, then its values) that
// asynchronous copies fill ahead, over the units' ends, and no barrier but that
// of the warps that share the ring.  Most groups are one warp.
//   keys     S^T = K Q^T: 16 tokens by 8 rows at a time, so that eight rows (the
//            usual group of query heads) leave no part of a product empty
//   softmax  a running maximum and sum per row; sums are scaled down only when a
//            maximum grows by more than 2^8, weights are up to that (times 2^7
//            beside an 8-bit cache: weight_lift)
//   values   O^T += V^T P^T: 16 elements by 8 rows, the weights in one or two
//            parts of 16 bits (weight_parts)
// Measured, 24 / 4 heads of 256 in bf16, whole calls: one sequence of 262144
// tokens 171 us (6.3 TB/s, 92 % of a copy's bandwidth), 64 of up to 8192 tokens
// 95 us (5.3), one of 4000 14 us (latency); eight drafted tokens of 32 sequences,
// 48 rows, 62 us (2.2), bound by what six warps read of each tile from shared
// memory and by waits between products; 128 sequences, 64 / 8 heads of 128 over 8
// bits, 101 us (5.2).
#pragma once

#include "paged_attention.cuh"

namespace gdn {

constexpr float kMinusInfinity = -__builtin_huge_valf();

__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void load_matrices_transposed(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
// A lane's elements (row lane / 4, two columns) of an 8 x 8 matrix, transposed.
__device__ __forceinline__ uint32_t transpose_matrix(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// c += a b, 16 x 8 x 16, of bf16 or fp16.
template <bool HALF>
__device__ __forceinline__ void multiply(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    if constexpr (HALF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                     "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
                     "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two as fp16, infinities as they are.
__device__ __forceinline__ uint32_t pack_halves(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// (fp16: 65504 at most.  Scores from 2^24 on are rounded to whole numbers, so a
// weight can pass the 2^15 that it is meant to have.)
template <bool HALF> __device__ __forceinline__ uint32_t pack_weights(float a, float b) {
    if constexpr (HALF) {
        uint32_t r;
        asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
        return r;
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
// The same in two parts, the second of what the first leaves.  In bf16 neither is
// negative, and neither zero for a weight of 2^-109 or more, so that infinite
// values stay infinite: the first is cut instead of rounded, and the second has
// 2^-24 of the weight besides, which is a rounding of fp32.  (An 8-bit cache has no
// infinities.)
template <bool HALF> __device__ __forceinline__ uint2 split_weights(float a, float b) {
    if constexpr (HALF) {
        const uint32_t two = pack_weights<true>(a, b);
        const float2 first = __half22float2(*reinterpret_cast<const __half2 *>(&two));
        return make_uint2(two, pack_weights<true>(a - first.x, b - first.y));
    } else {
        const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
        return make_uint2(__byte_perm(x, y, 0x7632),
                          pack_weights<false>(fmaf(a, 0x1p-24f, a - __uint_as_float(x & 0xffff0000u)),
                                              fmaf(b, 0x1p-24f, b - __uint_as_float(y & 0xffff0000u))));
    }
}
// Parts of 16 bits that a weight is the sum of in the products.  Two, where MT
// warps of a ring with NB blocks of 8 rows each have up to 16 rows: a weight is
// then off by 2^-16 of itself (2^-22 in fp16, beside an 8-bit cache), which a bf16
// result hardly shows, and the stream hides the products (4.3 GB of cache, one and
// two parts: 8 rows of 256 700 and 702 us, 16 rows 730 and 730; over 8 bits 717 and
// 710, 914 and 922; the most, 16 rows of 128 over 8 bits, 1044 and 1076).  More
// rows are bound by their products and reads of shared memory, of which a second
// part takes its own (24 rows of 256 843 and 883 us, 48 rows 1277 and 1376, 64 rows
// 1615 and 2200; 64 rows of 128 1077 and 1324): there a weight is rounded once, by up
// to 2^-8 of itself (fp16: 2^-11), which is the step of the bf16 results that it
// goes into.
__host__ __device__ constexpr int weight_parts(int nb, int mt) { return nb * mt > 2 ? 1 : 2; }
// Weights, and with them their sums, are taken against the maximum less this, and
// so stand in `m`, the statistics and the log-sum-exp: nothing else knows of it.
// fp16 holds no less than 2^-24 and up to 65504, so weights of 1 to 2^8 at their
// largest would lose what is below 2^-25 of it, which many tokens beside a dominant
// one add up to.  Up to 2^15 they lose 2^-32 each.  (bf16 has the exponents of fp32.)
__host__ __device__ constexpr float weight_lift(bool half) { return half ? 7.f : 0.f; }
// Two elements of 8 bits as two of fp16: exact.
__device__ __forceinline__ uint32_t widen(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}

// Eight elements, in one word where the rows allow it.
__device__ __forceinline__ Vec<__nv_bfloat16, 8> load8(const __nv_bfloat16 *p, bool words) {
    if (words) return Vec<__nv_bfloat16, 8>::load(p);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(p[i]);
    return Vec<__nv_bfloat16, 8>::from(x);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, bool words, const float (&x)[8]) {
    if (words) {
        Vec<__nv_bfloat16, 8>::from(x).store(p);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = from_f32<__nv_bfloat16>(x[i]);
    }
}

// The tokens of a tile: a half stage of 8 KB, or of 16 KB where warps share it.
__host__ __device__ constexpr int tile_tokens(int row_bytes, int mt) {
    return mt > 1 ? (16384 / row_bytes < 64 ? 16384 / row_bytes : 64) : (8192 / row_bytes < 64 ? 8192 / row_bytes : 64);
}
// What a unit costs beside its tokens, in tiles.
__host__ __device__ constexpr int setup_tiles(int nb, int mt) { return mt > 2 ? 4 : nb > 1 || mt > 1 ? 3 : 2; }

// What a variant keeps in shared memory.  EIGHT: an 8-bit cache; NB blocks of 8
// rows per warp, MT warps that share a ring, GR such groups.
template <bool EIGHT, int D, int NB, int MT, int GR> struct Tiles {
    static constexpr int kRowBytes = D * (EIGHT ? 1 : 2);
    static constexpr int kPitch = kRowBytes + 16;  // rows of a matrix on different banks
    static constexpr int kTokens = tile_tokens(kRowBytes, MT);
    static constexpr int kTile = kTokens * kPitch;
    static constexpr int kSetup = setup_tiles(NB, MT);
    static constexpr int kThreads = MT * GR * 32, kWarpRows = NB * 8, kRows = MT * kWarpRows;
    // Eight rows' sums, on their way out: in a stage that is free, or where
    // warps share a ring in a place of each warp's own.
    static constexpr int kSumPitch = D + 4;
    static constexpr int kSums = 8 * kSumPitch * 4;
    static constexpr int kOwn = MT > 1 ? MT * GR * kSums : 0;
    // Two blocks per SM, with some 64 KB of copies in flight: enough for the
    // memory's latency.  More only queue, and unfairly: the SMs of fuller GPCs
    // then end later (three stages per warp, 128 KB: 262144 tokens 179 us, two
    // stages 172; the last SM at 186 us of 162 on average).
    static constexpr int kBlocks = 2;
    static constexpr int kStages = MT > 2 ? 3 : 2;
    static constexpr int kRing = GR * kStages * kTile;
    static constexpr int kBytes = kRing + kOwn;
    static_assert(kBytes <= 233472 / kBlocks - 2048 && kSums <= kTile, "");
    static_assert(GR == 1 || GR * kRows * kSumPitch * 4 <= kBytes, "");
};

template <bool EIGHT, int D, int NB, int MT, int GR>
__global__ void __launch_bounds__(MT *GR * 32, Tiles<EIGHT, D, NB, MT, GR>::kBlocks)
gdn_attention_mma_kernel(const __grid_constant__ AttentionArgs a) {
    using S = Tiles<EIGHT, D, NB, MT, GR>;
    using T = __nv_bfloat16;
    constexpr int TK = S::kTokens, TT = TK / 16, ST = S::kStages, AHEAD = (ST - 1) / 2;
    constexpr int ES = EIGHT ? 1 : 2, DT = D / 16, SETUP = S::kSetup;
    constexpr int WORDS = S::kRowBytes / 16;  // of a token's row
    constexpr int PER = MT * 32 / WORDS;      // rows that a group copies at once
    constexpr int HOLD = (TK + 31) / 32;      // rows whose place a lane knows
    extern __shared__ __align__(16) char smem[];
    __shared__ float2 ml[GR][S::kRows];
    __shared__ float inverses[S::kRows];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int group = warp / MT, mt = warp % MT;
    const int g8 = lane / 4, c4 = lane % 4;
    char *ring = smem + group * ST * S::kTile;
    const uint32_t ring_at = ptx::smem_u32(ring);
    // A lane's address in a key tile and in a value tile (transposed).
    const uint32_t k_lane = ((lane & 7) + (lane >> 3 & 1) * 8) * S::kPitch + (lane >> 4) * 16;
    const uint32_t v_lane =
        EIGHT ? k_lane : ((lane & 7) + (lane >> 4) * 8) * S::kPitch + (lane >> 3 & 1) * 16;

    auto group_sync = [&] {
        if constexpr (MT == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(MT * 32) : "memory");
    };

    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int per_seq = a.Hkv * a.row_blocks;
    const Range range = find_range<TK, SETUP, S::kThreads, GR>(a, per_seq, group);
    const T *queries = static_cast<const T *>(a.q), *gates = static_cast<const T *>(a.gate);

    // ---- the copies, ahead of the products.  The cursor is at the tile whose
    // entries of the page table are on their way.
    struct {
        int64_t left;  // tiles of the range from this one on
        int n, unit, tile, tiles, len;
    } c;
    c.left = range.end - range.begin;
    c.n = range.n;
    c.len = range.len;
    c.tiles = tiles_of<TK, SETUP>(c.len);
    c.unit = (int)((range.begin - range.base) / c.tiles);
    c.tile = (int)((range.begin - range.base) % c.tiles);
    const int range_tiles = c.tiles;  // of the unit that the range begins in
    Piece piece;
    piece.unit = c.unit, piece.first = c.tile, piece.tiles = c.tiles;
    int n = c.n, len = c.len;

    // Sixteen tokens that follow one another share a page where the size allows
    // it: then a lane knows the places of a whole segment, else of one token.
    const bool segments = a.page_size % 16 == 0;
    const int step = segments ? 16 : 1;
    int entry[HOLD];
    auto token_of = [&](int h) { return (c.tile - SETUP) * TK + (h * 32 + lane) * step; };
    auto look_up = [&] {
        while (c.left > 0 && (c.tile < SETUP || c.tile == c.tiles)) {  // no tokens
            if (c.tile == c.tiles) {
                c.tile = 0;
                if (++c.unit == per_seq) {
                    c.unit = 0;
                    c.len = held_tokens(a, ++c.n);
                    c.tiles = tiles_of<TK, SETUP>(c.len);
                }
            }
            ++c.tile, --c.left;
        }
#pragma unroll
        for (int h = 0; h < HOLD; ++h) {
            const int j = token_of(h);
            entry[h] = -1;
            if (c.left > 0 && (h * 32 + lane) * step < TK && j < c.len)
                entry[h] = a.table[c.n * a.table_stride + a.by_page.of(j)];
        }
    };
    int64_t k_at[HOLD], v_at[HOLD];  // bytes from the cache's start; -1: none
    int held = 0;                    // of the tile's tokens
    uint32_t bad_tiles = 0;          // bit i: of the i-th tile ahead, a page out of range
    auto place = [&](int ahead) {
        const int head = a.row_blocks == 1 ? c.unit : c.unit / a.row_blocks;
        bool bad = false;
        held = c.left > 0 ? c.len - (c.tile - SETUP) * TK : 0;
#pragma unroll
        for (int h = 0; h < HOLD; ++h) {
            const int j = token_of(h), p = entry[h];
            k_at[h] = v_at[h] = -1;
            if (!((h * 32 + lane) * step < TK && (h * 32 + lane) * step < held)) continue;
            if (p < 0 || p >= a.num_pages) {
                bad = true;
                continue;
            }
            const int at = j - a.by_page.of(j) * a.page_size;
            k_at[h] = (uint32_t)p * a.kps + (uint32_t)at * a.kts + (uint32_t)head * a.khs;
            v_at[h] = (uint32_t)p * a.vps + (uint32_t)at * a.vts + (uint32_t)head * a.vhs;
        }
        if (__any_sync(0xffffffffu, bad)) bad_tiles |= 1u << ahead;
        if (c.left > 0) {
            ++c.tile, --c.left;
            look_up();
        }
    };
    // Copies a half stage: rows that do not exist become zeros.
    auto copy = [&](int stage, const void *from, int64_t token_stride, const int64_t (&at)[HOLD]) {
        const int sub = mt * 32 + lane, word = sub % WORDS, r_lane = sub / WORDS;
        char *to = ring + stage * S::kTile + r_lane * S::kPitch + word * 16;
        const char *base = static_cast<const char *>(from) + word * 16;
        if (segments) {
            int64_t place[TT];
#pragma unroll
            for (int t = 0; t < TT; ++t) place[t] = __shfl_sync(0xffffffffu, at[0], t);
            int64_t off = 0;
            const char *x = base;
#pragma unroll
            for (int r0 = 0; r0 < TK; r0 += PER) {
                const int r = r0 + r_lane;
                if (16 % PER != 0 || r0 % 16 == 0) {
                    off = place[0];
#pragma unroll
                    for (int t = 1; t < TT; ++t)
                        if (PER > 16 || 16 % PER != 0 ? r >> 4 == t : r0 / 16 == t) off = place[t];
                    x = base + (off < 0 ? 0 : off) + (r & 15) * token_stride;
                }
                if (TK % PER == 0 || r < TK)
                    copy_async_head(to + r0 * S::kPitch, x, off >= 0 && r < held ? 16 : 0);
                x += PER * token_stride;
            }
        } else {
#pragma unroll
            for (int r0 = 0; r0 < TK; r0 += PER) {
                const int r = r0 + r_lane;
                int64_t off = __shfl_sync(0xffffffffu, at[0], r & 31);
                if (HOLD > 1) {
                    const int64_t upper = __shfl_sync(0xffffffffu, at[HOLD - 1], r & 31);
                    off = r & 32 ? upper : off;
                }
                if (TK % PER == 0 || r < TK)
                    copy_async_head(to + r0 * S::kPitch, base + (off < 0 ? 0 : off), off < 0 ? 0 : 16);
            }
        }
        copies_commit();
    };
    int stage = 0;  // the next to be used; the one before it is free
    auto free_stage = [&] { return stage == 0 ? ST - 1 : stage - 1; };
    look_up();
    // Where a whole block lies inside one unit its groups' sums are joined here,
    // and it has one piece.
    const int4 joined = range.together;
    const bool together = joined.x != 0;

    // Sums of the piece's unit: element 16 d + g8 (and + 8; of 8-bit tiles 2 g8
    // and + 1) of rows 8 b + 2 c4 (and + 1).
    float o[DT][NB][4], m[NB][2], l[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int e = 0; e < 2; ++e) m[b][e] = kMinusInfinity, l[b][e] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][b][e] = 0.f;
    }
    // l of all tokens, from the lanes'.
    auto total_sums = [&](bool bad) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], d);
                if (bad) l[b][e] = __int_as_float(0x7fffffff);
            }
    };
    // Block b's sums times by[] as rows of D elements.
    auto lay_out = [&](float *to, int b, float by0, float by1) {
        to += c4 * 2 * S::kSumPitch;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            if constexpr (EIGHT) {
                float2 *x = reinterpret_cast<float2 *>(to + d * 16 + g8 * 2);
                x[0] = make_float2(o[d][b][0] * by0, o[d][b][2] * by0);
                x[S::kSumPitch / 2] = make_float2(o[d][b][1] * by1, o[d][b][3] * by1);
            } else {
                float *x = to + d * 16 + g8;
                x[0] = o[d][b][0] * by0;
                x[8] = o[d][b][2] * by0;
                x[S::kSumPitch] = o[d][b][1] * by1;
                x[S::kSumPitch + 8] = o[d][b][3] * by1;
            }
        }
    };

    // ---- the products, unit by unit
    const float sign = a.scale_log2 < 0.f ? -1.f : a.scale_log2 == 0.f ? 0.f : 1.f;
    const float magnitude = sign == 0.f ? 1.f : fabsf(a.scale_log2);
    for (int64_t pos = range.begin; pos < range.end;) {
        piece.last = (int)min((int64_t)piece.tiles, piece.first + (range.end - pos));
        const Unit u = unit_of<S::kRows>(a, n, piece.unit, len);
        const int t0 = piece.template first_token<TK, SETUP>(len), t1 = piece.template last_token<TK, SETUP>(len);

        // Queries, times the sign of the scale: rows 8 b + g8, elements 16 k + 2 c4
        // and + 8 (two each).  For an 8-bit cache elements 16 k + 4 c4 (four), in
        // fp16, each row over the power of two of its largest.
        uint32_t q[DT][NB][2];
        float scale[NB][2];
        int seen[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int r = mt * S::kWarpRows + b * 8 + g8;
            const bool live = r < u.rows;
            const RowPlace p = row_place(a, u, live ? r : 0);
            const T *from = queries + p.token * a.qs + p.head * a.qh;
#pragma unroll
            for (int k = 0; k < DT; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const T *x = from + k * 16 + (EIGHT ? c4 * 4 + h * 2 : c4 * 2 + h * 8);
                    if (!live) q[k][b][h] = 0;
                    else if (a.q_words) q[k][b][h] = *reinterpret_cast<const uint32_t *>(x);
                    else q[k][b][h] = (uint32_t) reinterpret_cast<const uint16_t *>(x)[0] |
                                      (uint32_t) reinterpret_cast<const uint16_t *>(x)[1] << 16;
                }
        }
        if (pos == range.begin) {  // the first copies, while the queries are on their way
            if constexpr (ST == 2) {
                place(0);
                copy(0, a.k, a.kts, k_at);
            } else {
#pragma unroll 1
                for (int i = 0; i < AHEAD; ++i) {
                    place(i);
                    copy(2 * i, a.k, a.kts, k_at);
                    copy(2 * i + 1, a.v, a.vts, v_at);
                }
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float up = 1.f;
            if constexpr (EIGHT) {
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < DT; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(q[k][b][h] << 16)),
                                               fabsf(__uint_as_float(q[k][b][h] & 0xffff0000u))));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^x <= top < 2^(x + 1), from the exponent's bits: as far as 2^x and
                // 2^-x are normal numbers, so that top 2^-x is below 4 for the largest
                // queries and below 1 for denormal ones.
                const int x = min(max((__float_as_int(top) >> 23) - 127, -126), 126);
                up = __int_as_float((127 + x) << 23);
                const float down = __int_as_float((127 - x) << 23) * sign;
#pragma unroll
                for (int k = 0; k < DT; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        q[k][b][h] = pack_halves(__uint_as_float(q[k][b][h] << 16) * down,
                                                 __uint_as_float(q[k][b][h] & 0xffff0000u) * down);
            } else if (sign != 1.f) {
#pragma unroll
                for (int k = 0; k < DT; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        q[k][b][h] = pack_weights<false>(__uint_as_float(q[k][b][h] << 16) * sign,
                                                         __uint_as_float(q[k][b][h] & 0xffff0000u) * sign);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                scale[b][e] = magnitude;
                if (EIGHT) scale[b][e] *= a.k_scale[u.head] * __shfl_sync(0xffffffffu, up, (c4 * 2 + e) * 4);
                seen[b][e] = min(t1, seen_by(a, u, mt * S::kWarpRows + b * 8 + c4 * 2 + e));
            }
        }
        // From here on not every row sees a token.
        const int all_see = min(t1, len - a.L + 1);
        bool bad = false;

#pragma unroll 1
        for (int j0 = t0; j0 < t1; j0 += TK) {
            // ---- keys
            copies_wait<ST - 2>();
            group_sync();
            if constexpr (ST > 2) place(AHEAD);
            bad |= bad_tiles & 1;
            bad_tiles >>= 1;
            if constexpr (ST > 2) copy(free_stage(), a.k, a.kts, k_at);
            else copy(free_stage(), a.v, a.vts, v_at);
            // Short chains of products: where they are few, even and odd steps
            // have sums of their own.
            constexpr int CHAINS = TT * NB < 4 ? 2 : 1;
            float s[TT][NB][4], odd[CHAINS == 2 ? TT : 1][CHAINS == 2 ? NB : 1][4];
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[t][b][e] = 0.f;
                        if constexpr (CHAINS == 2) odd[t][b][e] = 0.f;
                    }
            const uint32_t keys = ring_at + stage * S::kTile + k_lane;
#pragma unroll
            for (int k = 0; k < DT; k += EIGHT ? 2 : 1)
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    uint32_t x[4];
                    load_matrices(x, keys + t * 16 * S::kPitch + k * 16 * ES);
                    if constexpr (EIGHT) {
                        // A matrix is 8 tokens by 16 elements, of which a lane gets
                        // four that follow one another: two pairs, for both halves
                        // of k.
                        const uint32_t y0[4] = {widen(x[0]), widen(x[1]), widen(x[0] >> 16), widen(x[1] >> 16)};
                        const uint32_t y1[4] = {widen(x[2]), widen(x[3]), widen(x[2] >> 16), widen(x[3] >> 16)};
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            multiply<true>(s[t][b], y0, q[k][b][0], q[k][b][1]);
                            if constexpr (CHAINS == 2) multiply<true>(odd[t][b], y1, q[k + 1][b][0], q[k + 1][b][1]);
                            else multiply<true>(s[t][b], y1, q[k + 1][b][0], q[k + 1][b][1]);
                        }
                    } else {
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            if (CHAINS == 2 && k % 2)
                                multiply<false>(odd[CHAINS == 2 ? t : 0][CHAINS == 2 ? b : 0], x, q[k][b][0], q[k][b][1]);
                            else
                                multiply<false>(s[t][b], x, q[k][b][0], q[k][b][1]);
                        }
                    }
                }
            if constexpr (CHAINS == 2) {
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[t][b][e] += odd[t][b][e];
            }
            if (++stage == ST) stage = 0;

            // ---- softmax: token 16 t + g8 (e < 2, else + 8), row 8 b + 2 c4 + e % 2
            const bool edge = j0 + TK > all_see;
            if (edge) {
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (j0 + t * 16 + g8 + (e >> 1) * 8 >= seen[b][e & 1]) s[t][b][e] = kMinusInfinity;
            }
            float top[NB][2];
            bool grown = false;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(s[0][b][e], s[0][b][e + 2]);
#pragma unroll
                    for (int t = 1; t < TT; ++t) x = fmaxf(x, fmaxf(s[t][b][e], s[t][b][e + 2]));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                    top[b][e] = fmaf(x, scale[b][e], -weight_lift(EIGHT));
                    grown |= top[b][e] > m[b][e] + 8.f;
                }
            if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // Rows whose own maximum has not grown so far keep theirs: what
                        // the others see must not show in their last bits.
                        const float next = top[b][e] > m[b][e] + 8.f ? top[b][e] : m[b][e];
                        const float fade = ex2(m[b][e] - against(next));
                        m[b][e] = next;
                        l[b][e] *= fade;
#pragma unroll
                        for (int d = 0; d < DT; ++d) {
                            o[d][b][e] *= fade;
                            o[d][b][e + 2] *= fade;
                        }
                    }
            }
            constexpr int PARTS = weight_parts(NB, MT);
            uint32_t p[PARTS][TT][NB][2];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float low[2] = {against(m[b][0]), against(m[b][1])};
#pragma unroll
                for (int t = 0; t < TT; ++t) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[t][b][e] = ex2(fmaf(s[t][b][e], scale[b][e & 1], -low[e & 1]));
                        l[b][e & 1] += s[t][b][e];
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float w0 = s[t][b][h * 2], w1 = s[t][b][h * 2 + 1];
                        if constexpr (PARTS == 2) {
                            const uint2 parts = split_weights<EIGHT>(w0, w1);
                            p[0][t][b][h] = transpose_matrix(parts.x);
                            p[1][t][b][h] = transpose_matrix(parts.y);
                        } else {
                            p[0][t][b][h] = transpose_matrix(pack_weights<EIGHT>(w0, w1));
                        }
                    }
                }
            }

            // ---- values
            copies_wait<ST - 2>();
            group_sync();
            if constexpr (ST > 2) {
                copy(free_stage(), a.v, a.vts, v_at);
            } else {
                place(0);
                copy(free_stage(), a.k, a.kts, k_at);
            }
            const char *tile = ring + stage * S::kTile;
            const uint32_t values = ring_at + stage * S::kTile + v_lane;
            // The newest tokens' values may be infinite or NaN where some rows
            // do not see them: a weight of zero would not keep them out.
            bool apart = false;
            if (edge && a.L > 1) {
                for (int j = max(all_see, j0); j < min(t1, j0 + TK); ++j)
                    for (int w = lane; w < WORDS; w += 32) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(tile + (j - j0) * S::kPitch + w * 16);
                        const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if constexpr (EIGHT) {
#pragma unroll
                                for (int b = 0; b < 32; b += 8) apart |= (y[k] >> b & 0x7f) == 0x7f;
                            } else {
                                apart |= (y[k] & 0x7f80u) == 0x7f80u ||
                                         (y[k] & 0x7f800000u) == 0x7f800000u;
                            }
                        }
                    }
                apart = __any_sync(0xffffffffu, apart);
            }
            // Then the products take zeros instead, and the values follow one by one
            // for the rows that see them: the others keep every bit.
            const int keep = max(all_see - j0, 0);
            auto kept = [&](uint32_t two, int j) {  // fp16 or bf16 of tokens j, j + 1
                constexpr uint32_t kExponent = EIGHT ? 0x7c00u : 0x7f80u;
                if (j >= keep && (two & kExponent) == kExponent) two &= 0xffff0000u;
                if (j + 1 >= keep && (two >> 16 & kExponent) == kExponent) two &= 0xffffu;
                return two;
            };
            auto add_values = [&](auto masked) {
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const int j = t * 16 + c4 * 2;
#pragma unroll
                    for (int d = 0; d < DT; d += EIGHT ? 2 : 1) {
                        uint32_t x[4];
                        load_matrices_transposed(x, values + t * 16 * S::kPitch + d * 16 * ES);
                        if constexpr (EIGHT) {
                            // A matrix is 8 tokens by 16 elements, of which a lane gets
                            // two neighbours of two tokens: rows g8 and g8 + 8 of the
                            // product are even and odd elements.
                            uint32_t y[2][4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t even = widen(x[i]), next = widen(x[i] >> 16);
                                y[i / 2][i % 2 * 2] = __byte_perm(even, next, 0x5410);
                                y[i / 2][i % 2 * 2 + 1] = __byte_perm(even, next, 0x7632);
                            }
                            if (masked) {
#pragma unroll
                                for (int i = 0; i < 8; ++i) y[i / 4][i % 4] = kept(y[i / 4][i % 4], j + (i % 4 / 2) * 8);
                            }
#pragma unroll
                            for (int i = 0; i < PARTS; ++i)
#pragma unroll
                                for (int b = 0; b < NB; ++b) {
                                    multiply<true>(o[d][b], y[0], p[i][t][b][0], p[i][t][b][1]);
                                    multiply<true>(o[d + 1][b], y[1], p[i][t][b][0], p[i][t][b][1]);
                                }
                        } else {
                            if (masked) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) x[i] = kept(x[i], j + (i / 2) * 8);
                            }
#pragma unroll
                            for (int i = 0; i < PARTS; ++i)
#pragma unroll
                                for (int b = 0; b < NB; ++b)
                                    multiply<false>(o[d][b], x, p[i][t][b][0], p[i][t][b][1]);
                        }
                    }
                }
            };
            if (!apart) {
                add_values(std::false_type());
            } else {
                add_values(std::true_type());
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll 1
                        for (int i = 0; i < 8; ++i) {
                            const int j = t * 16 + h * 8 + i;
                            float w[NB][2];
#pragma unroll
                            for (int b = 0; b < NB; ++b)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    w[b][e] = __shfl_sync(0xffffffffu, s[t][b][h * 2 + e], i * 4 + c4);
                            if (j < keep || j0 + j >= t1) continue;
                            const char *row = tile + j * S::kPitch;
#pragma unroll
                            for (int d = 0; d < DT; ++d)
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const int at = d * 16 + (EIGHT ? g8 * 2 + k : g8 + k * 8);
                                    float v;
                                    if constexpr (EIGHT) v = from_e4m3x2((uint8_t)row[at]).x;
                                    else v = to_f32(reinterpret_cast<const T *>(row)[at]);
                                    if (isfinite(v)) continue;
#pragma unroll
                                    for (int b = 0; b < NB; ++b)
#pragma unroll
                                        for (int e = 0; e < 2; ++e)
                                            if (j0 + j < seen[b][e])
                                                o[d][b][k * 2 + e] = fmaf(w[b][e], v, o[d][b][k * 2 + e]);
                                }
                        }
            }
            if (++stage == ST) stage = 0;
        }
        total_sums(bad);

        if (!together) {
            // ---- the unit's rows, or the piece of them, eight at a time
            const bool whole = piece.whole();
            const int slot = piece.slot(range.group);
            const float v_scale = EIGHT ? a.v_scale[u.head] : 1.f;
            float *sums = reinterpret_cast<float *>(
                MT > 1 ? smem + S::kRing + warp * S::kSums : ring + free_stage() * S::kTile);
            if (piece.first == 0 && mt == 0 && lane == 0)
                a.joins[(int64_t)n * per_seq + piece.unit] = join_from(range, range.group, piece.last, piece.tiles, pos);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int r0 = mt * S::kWarpRows + b * 8;
                constexpr int Q8 = D / 8, EACH = 8 * Q8 / 32;
                // Rows and their places: of row lane % 8 by each lane, from there by
                // those that have its elements.
                const RowPlace p = row_place(a, u, min(r0 + lane % 8, u.rows - 1));
                const int64_t out_at = p.token * a.os + p.head * a.oh, gate_at = p.token * a.gs + p.head * a.gh;
                auto gate_of = [&](int i) {
                    const int at = i * 32 + lane, r = at / Q8;
                    const int64_t from = __shfl_sync(0xffffffffu, gate_at, r);
                    return r0 + r < u.rows ? load8(gates + from + at % Q8 * 8, a.gate_words) : Vec<T, 8>::zero();
                };
                Vec<T, 8> gate = Vec<T, 8>::zero();
                const bool gated = whole && a.gate;
                if (gated) gate = gate_of(0);
                lay_out(sums, b, whole ? inverse(l[b][0]) * v_scale : v_scale,
                        whole ? inverse(l[b][1]) * v_scale : v_scale);
                if (g8 == 0) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = r0 + c4 * 2 + e;
                        if (r >= u.rows) continue;
                        if (whole) store_lse(a, row_place(a, u, r), m[b][e], l[b][e]);
                        else a.stats[slot * S::kRows + r] = make_float2(m[b][e], l[b][e]);
                    }
                }
                __syncwarp();
#pragma unroll 1  // little code: a unit's end is where instructions are not at hand
                for (int i = 0; i < EACH; ++i) {
                    const Vec<T, 8> now = gate;
                    if (gated && i + 1 < EACH) gate = gate_of(i + 1);
                    const int at = i * 32 + lane, r = at / Q8, e = at % Q8 * 8;
                    const float4 *x = reinterpret_cast<const float4 *>(sums + r * S::kSumPitch + e);
                    const float4 x0 = x[0], x1 = x[1];
                    const int64_t to = __shfl_sync(0xffffffffu, out_at, r);
                    if (r0 + r >= u.rows) continue;
                    if (whole) {
                        float y[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                        if (gated) {
                            float by[8];
                            now.to(by);
#pragma unroll
                            for (int k = 0; k < 8; ++k) y[k] *= sigmoid(by[k]);
                        }
                        store8((T *)a.out + to + e, a.out_words, y);
                    } else {
                        float4 *sum = reinterpret_cast<float4 *>(a.sums + ((int64_t)slot * S::kRows + r0 + r) * D + e);
                        sum[0] = x0;
                        sum[1] = x1;
                    }
                }
                __syncwarp();
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int e = 0; e < 2; ++e) m[b][e] = kMinusInfinity, l[b][e] = 0.f;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[d][b][e] = 0.f;
            }
        }
        pos += piece.last - piece.first;
        piece.first = 0;
        if (++piece.unit == per_seq && pos < range.end) {
            piece.unit = 0;
            len = held_tokens(a, ++n);
            piece.tiles = tiles_of<TK, SETUP>(len);
        }
    }
    copies_wait<0>();
    if (!together) return;

    // ---- the groups' sums, joined
    if constexpr (GR > 1) {
        const Unit u = unit_of<S::kRows>(a, joined.y, joined.z, 0);
        const bool whole = joined.w == 3;
        const int group0 = blockIdx.x * GR, slot = 2 * group0 + (joined.w & 1);
        float *sums = reinterpret_cast<float *>(smem);
        __syncthreads();
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int r0 = mt * S::kWarpRows + b * 8;
            lay_out(sums + (group * S::kRows + r0) * S::kSumPitch, b, 1.f, 1.f);
            if (g8 == 0)
#pragma unroll
                for (int e = 0; e < 2; ++e) ml[group][r0 + c4 * 2 + e] = make_float2(m[b][e], l[b][e]);
        }
        __syncthreads();
        // Each row's factors for the groups' sums, the values' scale among them.
        if (threadIdx.x < u.rows) {
            const int r = threadIdx.x;
            const float v_scale = EIGHT ? a.v_scale[u.head] : 1.f;
            float top = kMinusInfinity, sum = 0.f;
#pragma unroll
            for (int w = 0; w < GR; ++w) top = fmaxf(top, ml[w][r].x);
#pragma unroll
            for (int w = 0; w < GR; ++w) {
                const float f = ex2(ml[w][r].x - against(top));
                sum += ml[w][r].y * f;
                ml[w][r].x = f * v_scale;
                if (w > 0 && !whole) a.stats[2 * (group0 + w) * S::kRows + r] = make_float2(kMinusInfinity, 0.f);
            }
            if (whole) store_lse(a, row_place(a, u, r), top, sum);
            else a.stats[slot * S::kRows + r] = make_float2(top, sum);
            inverses[r] = whole ? inverse(sum) : 1.f;
        }
        if (threadIdx.x == 0 && joined.w & 1)
            a.joins[(int64_t)joined.y * per_seq + joined.z] =
                join_from(range, group0, whole ? range_tiles : 0, range_tiles, range.begin);
        __syncthreads();
        constexpr int Q8 = D / 8;
        const int words = u.rows * Q8;
#pragma unroll 2
        for (int i = threadIdx.x; i < words; i += S::kThreads) {
            const int r = i / Q8, e = i % Q8 * 8;
            const RowPlace p = row_place(a, u, r);
            Vec<T, 8> gate = Vec<T, 8>::zero();
            if (whole && a.gate)
                gate = load8(gates + p.token * a.gs + p.head * a.gh + e, a.gate_words);
            float y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = 0.f;
#pragma unroll
            for (int w = 0; w < GR; ++w) {
                const float f = ml[w][r].x;
                const float4 *x = reinterpret_cast<const float4 *>(sums + (w * S::kRows + r) * S::kSumPitch + e);
                const float4 x0 = x[0], x1 = x[1];
                y[0] = fmaf(f, x0.x, y[0]), y[1] = fmaf(f, x0.y, y[1]);
                y[2] = fmaf(f, x0.z, y[2]), y[3] = fmaf(f, x0.w, y[3]);
                y[4] = fmaf(f, x1.x, y[4]), y[5] = fmaf(f, x1.y, y[5]);
                y[6] = fmaf(f, x1.z, y[6]), y[7] = fmaf(f, x1.w, y[7]);
            }
            if (whole) {
                float by[8];
                gate.to(by);
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] *= a.gate ? inverses[r] * sigmoid(by[k]) : inverses[r];
                store8((T *)a.out + p.token * a.os + p.head * a.oh + e, a.out_words, y);
            } else {
                float4 *to = reinterpret_cast<float4 *>(a.sums + ((int64_t)slot * S::kRows + r) * D + e);
                to[0] = make_float4(y[0], y[1], y[2], y[3]);
                to[1] = make_float4(y[4], y[5], y[6], y[7]);
            }
        }
    }
}

template <bool EIGHT, int D, int NB, int MT, int GR>
gdn_status mma_run(int blocks, const AttentionArgs &a, cudaStream_t stream) {
    using S = Tiles<EIGHT, D, NB, MT, GR>;
    static std::atomic<bool> done[kMaxDevices];
    const auto kernel = gdn_attention_mma_kernel<EIGHT, D, NB, MT, GR>;
    if (!raise_shared_memory(done, {reinterpret_cast<const void *>(kernel)}, {(size_t)S::kBytes}))
        return GDN_ERR_CUDA;
    return launch_programmatic(kernel, dim3(blocks), S::kThreads, S::kBytes, stream, a);
}

// Up to 64 rows of a unit at a time.  Eight per warp leave registers for two
// blocks of six warps; sixteen read a tile's matrices half as often, which heads of
// up to 128 have the registers for.  Not all do without spills (bytes of stores and
// loads per thread, an 8-bit cache's in brackets): six warps of heads of 256 116 and
// 152 (196 and 272), four of sixteen rows 512 and 428 (800 and 604), four of eight
// none (12 and 12), two 4 and 4 (none); heads of 128, three warps of sixteen rows, 64
// and 76 (96 and 124), two none (24 and 20).  One warp per ring has none.  (8 x 24 / 4 heads of 256, 48
// rows, 1024 tokens each: 3380 GB/s of cache with six warps of 8 rows, 2710 with
// three of 16.  Heads of 128: 32 rows 4890 with four of 8, 5830 with two of 16;
// 64 rows 2150 and 4060, heads of 256 2290 and 2690.)
struct Warps {
    int nb, mt;
};
constexpr Warps warps_of(int R, int D) {
    if (R <= 8) return {1, 1};
    if (R <= 16) return {1, 2};
    if (R <= 24) return {1, 3};
    if (R <= 32) return D > 128 ? Warps{1, 4} : Warps{2, 2};
    if (R <= 48) return D > 128 ? Warps{1, 6} : Warps{2, 3};
    return {2, 4};
}
constexpr int groups_of(Warps w) { return w.mt == 1 ? 4 : w.mt == 2 ? 2 : 1; }
inline AttentionShape mma_shape(bool eight, int R, int D) {
    const Warps w = warps_of(R, D);
    return {w.nb * w.mt * 8, tile_tokens(D * (eight ? 1 : 2), w.mt), setup_tiles(w.nb, w.mt), groups_of(w),
            2 * kGridSms};
}
template <bool EIGHT, int D, int R>
gdn_status mma_rows(int blocks, const AttentionArgs &a, cudaStream_t stream) {
    constexpr Warps w = warps_of(R, D);
    return mma_run<EIGHT, D, w.nb, w.mt, groups_of(w)>(blocks, a, stream);
}

template <bool EIGHT, int D>
gdn_status mma_rows(int blocks, const AttentionArgs &a, cudaStream_t stream) {
    if (a.R <= 8) return mma_rows<EIGHT, D, 8>(blocks, a, stream);
    if (a.R <= 16) return mma_rows<EIGHT, D, 16>(blocks, a, stream);
    if (a.R <= 24) return mma_rows<EIGHT, D, 24>(blocks, a, stream);
    if (a.R <= 32) return mma_rows<EIGHT, D, 32>(blocks, a, stream);
    if (a.R <= 48) return mma_rows<EIGHT, D, 48>(blocks, a, stream);
    return mma_rows<EIGHT, D, 64>(blocks, a, stream);
}

template <bool EIGHT> gdn_status mma_attention(int D, int blocks, const AttentionArgs &a, cudaStream_t stream) {
    if (D == 64) return mma_rows<EIGHT, 64>(blocks, a, stream);
    if (D == 128) return mma_rows<EIGHT, 128>(blocks, a, stream);
    return mma_rows<EIGHT, 256>(blocks, a, stream);
}

}  // namespace gdn

// paged_attention_mma.cuh -- the attention of paged_attention.cuh for bf16
// queries over a bf16 or an 8-bit cache.
//
// The rows of a unit (query heads that share a key head, times new tokens)
// are the rows of small matrix products with the unit's tokens, so every
// element of the cache takes part in as many products as there are rows: far
// fewer than the 256 or so per byte at which a GB300's tensor cores would bound the
// operator, and more than fp32 units do beside a stream at full bandwidth.  So
// the products are warp-wide ones (m16n8k16) straight from the tiles that the
// copies land in, which have no setup, and the design is about keeping copies
// in flight: every group of warps has a ring of half stages (a tile's keys, then
// its values) that asynchronous copies fill ahead, and no barrier but those of
// the warps that share the ring.
//   keys     S = Q K^T: a warp has 16 rows, and the scores of a tile's tokens
//   softmax  a running maximum and sum per row; sums are scaled down only when a
//            maximum grows by more than 2^8, weights are up to that
//   values   O += P V: 16 rows of D sums in registers
// Groups take the tiles of a block's piece in turn and are joined at its end.
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
template <bool HALF> __device__ __forceinline__ uint32_t pack_weights(float a, float b) {
    if constexpr (HALF) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
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

// What a variant keeps in shared memory.  EIGHT: an 8-bit cache; MT tiles of 16
// rows, each of one warp, share a ring; GR such groups.
template <bool EIGHT, int D, int MT, int GR> struct Tiles {
    static constexpr int kRowBytes = D * (EIGHT ? 1 : 2);
    static constexpr int kPitch = kRowBytes + 16;  // rows of a matrix on different banks
    static constexpr int kTokens = 8192 / kRowBytes < 64 ? 8192 / kRowBytes : 64;
    static constexpr int kTile = kTokens * kPitch;
    static constexpr int kThreads = MT * GR * 32, kRows = MT * 16;
    static constexpr int kQueryPitch = D * 2 + 16;
    static constexpr int kQueries = kRows * kQueryPitch;
    static constexpr int kRoom = 115712 - 512;  // of two blocks per SM, each
    static constexpr int kFit = (kRoom - kQueries) / (GR * kTile);
    static constexpr int kStages = kFit >= 9 ? 9 : kFit % 2 ? kFit : kFit - 1;  // odd
    static constexpr int kSumPitch = D + (EIGHT ? 16 : 8);
    static constexpr int kRing = GR * kStages * kTile;
    static constexpr int kBytes = kQueries + kRing;
    static constexpr int kChunk = 4 * kTokens;
    static_assert(kStages >= 3, "");
    static_assert(GR * kRows * kSumPitch * 4 <= kRing, "");
    static_assert(kChunk % (GR * kTokens) == 0, "");
};

template <bool EIGHT, int D, int MT, int GR>
__global__ void __launch_bounds__(MT *GR * 32, 2)
gdn_attention_mma_kernel(const __grid_constant__ AttentionArgs a) {
    using S = Tiles<EIGHT, D, MT, GR>;
    using T = __nv_bfloat16;
    constexpr int TK = S::kTokens, NT = TK / 8, ST = S::kStages, AHEAD = (ST - 1) / 2;
    constexpr int WORDS = S::kRowBytes / 16;           // of a token's row
    constexpr int PER = MT * 32 / WORDS;               // rows that a group copies at once
    constexpr int HOLD = (TK + 31) / 32;               // rows whose place a lane knows
    extern __shared__ __align__(16) char smem[];
    __shared__ float2 ml[GR][S::kRows];
    __shared__ float row_scale[S::kRows], inverses[S::kRows];
    char *queries = smem, *ring = smem + S::kQueries;
    float *sums = reinterpret_cast<float *>(ring);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int group = warp / MT, mt = warp % MT;
    const int g8 = lane / 4, c4 = lane % 4;
    const uint32_t mine = ptx::smem_u32(ring + group * ST * S::kTile);
    // A lane's address in a key tile (tokens by elements) and in a value tile.
    const uint32_t k_lane = EIGHT ? ((lane & 7) + (lane >> 3 & 1) * 8) * S::kPitch + (lane >> 4) * 16
                                  : ((lane & 7) + (lane >> 4) * 8) * S::kPitch + (lane >> 3 & 1) * 16;
    const uint32_t v_lane = ((lane & 7) + (lane >> 3 & 1) * 8) * S::kPitch + (lane >> 4) * 16;

    auto group_sync = [&] {
        if constexpr (MT == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(MT * 32) : "memory");
    };

    ptx::griddep_launch_dependents();
    const Range range = find_range<S::kChunk, S::kThreads>(a, a.Hkv * a.row_blocks);
    for_pieces<S::kChunk, S::kRows>(a, range, [&](const Unit &u, int t0, int t1, int slot) {
        const int tiles = (t1 - t0 + TK - 1) / TK;
        const int own = tiles > group ? (tiles - group + GR - 1) / GR : 0;  // this group's
        auto first_token = [&](int i) { return t0 + (i * GR + group) * TK; };
        const int32_t *table = a.table + u.n * a.table_stride;
        bool bad = false;

        // The entries of tile i's rows, loaded a tile before they are needed.
        int entry[HOLD];
        auto look_up = [&](int i) {
#pragma unroll
            for (int h = 0; h < HOLD; ++h) {
                const int j = first_token(i) + h * 32 + lane;
                entry[h] = i < own && h * 32 + lane < TK && j < t1 ? table[j / a.page_size] : -1;
            }
        };
        int64_t k_at[HOLD], v_at[HOLD];  // bytes from the cache's start; -1: none
        auto place = [&](int i) {
#pragma unroll
            for (int h = 0; h < HOLD; ++h) {
                const int j = first_token(i) + h * 32 + lane, p = entry[h];
                k_at[h] = v_at[h] = -1;
                if (!(i < own && h * 32 + lane < TK && j < t1)) continue;
                if (p < 0 || p >= a.num_pages) {
                    bad = true;
                    continue;
                }
                const int at = j % a.page_size;
                k_at[h] = (p * a.kps + at * a.kts + u.head * a.khs) * (EIGHT ? 1 : 2);
                v_at[h] = (p * a.vps + at * a.vts + u.head * a.vhs) * (EIGHT ? 1 : 2);
            }
        };
        // Copies a half stage: rows that do not exist become zeros.
        auto copy = [&](int stage, const void *from, const int64_t (&at)[HOLD]) {
            const int sub = mt * 32 + lane, word = sub % WORDS;
            char *to = ring + (group * ST + stage) * S::kTile + word * 16;
#pragma unroll
            for (int r0 = 0; r0 < TK; r0 += PER) {
                const int r = r0 + sub / WORDS;
                int64_t off = at[0];
                off = __shfl_sync(0xffffffffu, at[0], r & 31);
                if (HOLD > 1) {
                    const int64_t upper = __shfl_sync(0xffffffffu, at[HOLD - 1], r & 31);
                    off = r & 32 ? upper : off;
                }
                if (TK % PER == 0 || r < TK)
                    copy_async_head(to + r * S::kPitch,
                                    static_cast<const char *>(from) + (off < 0 ? 0 : off + word * 16),
                                    off < 0 ? 0 : 16);
            }
            copies_commit();
        };

        __syncthreads();  // the last piece's sums
        int stage = 0;
        look_up(0);
#pragma unroll 1
        for (int i = 0; i < AHEAD; ++i) {
            place(i);
            look_up(i + 1);
            copy(2 * i, a.k, k_at);
            copy(2 * i + 1, a.v, v_at);
        }

        // Queries, times the sign of the scale; for fp16 products each row over
        // the power of two of its largest, in the order of an 8-bit key's
        // elements (see below).  A thread has eight elements at a time, and all
        // it takes are loaded together.
        const float sign = a.scale_log2 < 0.f ? -1.f : a.scale_log2 == 0.f ? 0.f : 1.f;
        {
            constexpr int Q8 = D / 8, EACH = S::kRows * Q8 / S::kThreads, BATCH = EACH < 4 ? EACH : 4;
#pragma unroll 1
            for (int i0 = 0; i0 < EACH; i0 += BATCH) {
                Vec<T, 8> x[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int at = (i0 + i) * S::kThreads + threadIdx.x, r = at / Q8, e = at % Q8 * 8;
                    x[i] = Vec<T, 8>::zero();
                    if (r >= u.rows) continue;
                    const RowPlace p = row_place(a, u, r);
                    x[i] = load8(static_cast<const T *>(a.q) + p.token * a.qs + p.head * a.qh + e, a.q_words);
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int at = (i0 + i) * S::kThreads + threadIdx.x, r = at / Q8, e = at % Q8 * 8;
                    char *to = queries + r * S::kQueryPitch;
                    float y[8];
                    x[i].to(y);
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[k] *= sign;
                    if constexpr (EIGHT) {
                        float top = 0.f;
#pragma unroll
                        for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(y[k]));
#pragma unroll
                        for (int d = Q8 / 2; d > 0; d >>= 1)
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        // 2^n <= top < 2^(n + 1), from the exponent's bits.
                        const int n = top > 0x1p-120f && top < 0x1p120f ? (__float_as_int(top) >> 23) - 127 : 0;
                        const float down = __int_as_float((127 - n) << 23);
                        if (e == 0) row_scale[r] = __int_as_float((127 + n) << 23);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            y[k] *= down;
                            if (fabsf(y[k]) < __builtin_huge_valf()) y[k] = fminf(fmaxf(y[k], -65504.f), 65504.f);
                        }
                        // Elements 4 c + j of 16: pairs of j < 2 first.
                        uint32_t *half = reinterpret_cast<uint32_t *>(to + (e & ~15) * 2) + (e & 8) / 4;
                        half[0] = pack_weights<true>(y[0], y[1]);
                        half[4] = pack_weights<true>(y[2], y[3]);
                        half[1] = pack_weights<true>(y[4], y[5]);
                        half[5] = pack_weights<true>(y[6], y[7]);
                    } else {
                        Vec<T, 8>::from(y).store(reinterpret_cast<T *>(to) + e);
                    }
                }
            }
        }
        __syncthreads();
        uint32_t qf[D / 16][4];
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            load_matrices(qf[k], ptx::smem_u32(queries) + (mt * 16 + (lane & 15)) * S::kQueryPitch +
                                     k * 32 + (lane >> 4) * 16);
        // Rows g8 and g8 + 8 of the tile.
        const int row0 = mt * 16 + g8;
        float scale[2];
        int seen[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = row0 + e * 8;
            scale[e] = (sign == 0.f ? 1.f : fabsf(a.scale_log2)) * (EIGHT ? row_scale[r] * a.k_scale[u.head] : 1.f);
            seen[e] = min(t1, seen_by(a, u, r));
        }
        // From here on not every row sees a token.
        const int all_see = min(t1, u.len - a.L + 1);

        float o[D / 8][4], m[2] = {kMinusInfinity, kMinusInfinity}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;

#pragma unroll 1
        for (int i = 0; i < own; ++i) {
            const int j0 = first_token(i);
            // ---- keys
            copies_wait<ST - 2>();
            group_sync();
            {
                const int to = stage + ST - 1;
                place(i + AHEAD);
                look_up(i + AHEAD + 1);
                copy(to >= ST ? to - ST : to, a.k, k_at);
            }
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
            const uint32_t keys = mine + stage * S::kTile + k_lane;
            if constexpr (EIGHT) {
                // A matrix is 8 tokens by 16 elements, of which a lane gets four
                // that follow one another: two pairs, for both halves of k.
#pragma unroll
                for (int k = 0; k < D / 16; k += 2)
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        uint32_t b[4];
                        load_matrices(b, keys + n * 8 * S::kPitch + k * 16);
                        multiply<true>(s[n], qf[k], widen(b[0]), widen(b[0] >> 16));
                        multiply<true>(s[n + 1], qf[k], widen(b[1]), widen(b[1] >> 16));
                        multiply<true>(s[n], qf[k + 1], widen(b[2]), widen(b[2] >> 16));
                        multiply<true>(s[n + 1], qf[k + 1], widen(b[3]), widen(b[3] >> 16));
                    }
            } else {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        uint32_t b[4];
                        load_matrices(b, keys + n * 8 * S::kPitch + k * 32);
                        multiply<false>(s[n], qf[k], b[0], b[1]);
                        multiply<false>(s[n + 1], qf[k], b[2], b[3]);
                    }
            }
            if (++stage == ST) stage = 0;

            // ---- softmax
            const bool edge = j0 + TK > all_see;
            if (edge) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j0 + n * 8 + c4 * 2 + (e & 1) >= seen[e >> 1]) s[n][e] = kMinusInfinity;
            }
            float top[2] = {kMinusInfinity, kMinusInfinity};
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[n][e]);
            bool grown = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
                top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
                top[e] *= scale[e];
                grown |= top[e] > m[e] + 8.f;
            }
            if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float next = fmaxf(m[e], top[e]), fade = ex2(m[e] - against(next));
                    m[e] = next;
                    l[e] *= fade;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][2 * e] *= fade;
                        o[n][2 * e + 1] *= fade;
                    }
                }
            }
            uint32_t p[NT / 2][4];
            {
                const float low[2] = {against(m[0]), against(m[1])};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[n][e] = ex2(fmaf(s[n][e], scale[e >> 1], -low[e >> 1]));
                        l[e >> 1] += s[n][e];
                    }
                    p[n / 2][n % 2 * 2] = pack_weights<EIGHT>(s[n][0], s[n][1]);
                    p[n / 2][n % 2 * 2 + 1] = pack_weights<EIGHT>(s[n][2], s[n][3]);
                }
            }

            // ---- values
            copies_wait<ST - 2>();
            group_sync();
            {
                const int to = stage + ST - 1;
                copy(to >= ST ? to - ST : to, a.v, v_at);
            }
            const char *tile = ring + (group * ST + stage) * S::kTile;
            const uint32_t values = mine + stage * S::kTile + v_lane;
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
                for (int k = 0; k < NT / 2; ++k) {
                    const int j = k * 16 + c4 * 2;
#pragma unroll
                    for (int n = 0; n < D / 8; n += EIGHT ? 4 : 2) {
                        uint32_t b[4];
                        load_matrices_transposed(b, values + k * 16 * S::kPitch + n * (EIGHT ? 8 : 16));
                        if constexpr (EIGHT) {
                            // A matrix is 8 tokens by 16 elements, of which a lane
                            // gets two neighbours of two tokens: one for each of
                            // two products, whose columns are even and odd elements.
                            uint32_t lo[4], hi[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t x = widen(b[i]), y = widen(b[i] >> 16);
                                lo[i] = __byte_perm(x, y, 0x5410);
                                hi[i] = __byte_perm(x, y, 0x7632);
                                if (masked) {
                                    lo[i] = kept(lo[i], j + (i & 1) * 8);
                                    hi[i] = kept(hi[i], j + (i & 1) * 8);
                                }
                            }
                            multiply<true>(o[n], p[k], lo[0], lo[1]);
                            multiply<true>(o[n + 1], p[k], hi[0], hi[1]);
                            multiply<true>(o[n + 2], p[k], lo[2], lo[3]);
                            multiply<true>(o[n + 3], p[k], hi[2], hi[3]);
                        } else {
                            if (masked) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) b[i] = kept(b[i], j + (i & 1) * 8);
                            }
                            multiply<false>(o[n], p[k], b[0], b[1]);
                            multiply<false>(o[n + 1], p[k], b[2], b[3]);
                        }
                    }
                }
            };
            if (!apart) {
                add_values(std::false_type());
            } else {
                add_values(std::true_type());
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            const int j = n * 8 + c * 2 + b;
                            const float w0 = __shfl_sync(0xffffffffu, s[n][b], (lane & ~3) + c);
                            const float w1 = __shfl_sync(0xffffffffu, s[n][2 + b], (lane & ~3) + c);
                            if (j < keep || j0 + j >= t1) continue;
                            const bool see0 = j0 + j < seen[0], see1 = j0 + j < seen[1];
                            const char *row = tile + j * S::kPitch;
                            auto add = [&](float &x0, float &x1, float v) {
                                if (isfinite(v)) return;
                                if (see0) x0 = fmaf(w0, v, x0);
                                if (see1) x1 = fmaf(w1, v, x1);
                            };
                            if constexpr (EIGHT) {
#pragma unroll
                                for (int q = 0; q < D / 8; q += 2) {
                                    const uint32_t x = *reinterpret_cast<const uint32_t *>(row + q * 8 + c4 * 4);
                                    const float2 v = from_e4m3x2(x & 0xffff), y = from_e4m3x2(x >> 16);
                                    add(o[q][0], o[q][2], v.x);
                                    add(o[q + 1][0], o[q + 1][2], v.y);
                                    add(o[q][1], o[q][3], y.x);
                                    add(o[q + 1][1], o[q + 1][3], y.y);
                                }
                            } else {
#pragma unroll
                                for (int q = 0; q < D / 8; ++q) {
                                    const uint32_t x = *reinterpret_cast<const uint32_t *>(row + q * 16 + c4 * 4);
                                    add(o[q][0], o[q][2], __uint_as_float(x << 16));
                                    add(o[q][1], o[q][3], __uint_as_float(x & 0xffff0000u));
                                }
                            }
                        }
            }
            if (++stage == ST) stage = 0;
        }
        copies_wait<0>();
        bad = __any_sync(0xffffffffu, bad);

        // ---- the groups' sums, joined
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            const int r = row0 + e * 8;
            if (r >= u.rows) continue;
            if (c4 == 0) ml[group][r] = make_float2(m[e], bad ? __int_as_float(0x7fffffff) : l[e]);
            float *to = sums + (group * S::kRows + r) * S::kSumPitch;
#pragma unroll
            for (int n = 0; n < D / 8; n += 2) {
                if constexpr (EIGHT) {
                    *reinterpret_cast<float4 *>(to + n * 8 + c4 * 4) =
                        make_float4(o[n][2 * e], o[n + 1][2 * e], o[n][2 * e + 1], o[n + 1][2 * e + 1]);
                } else {
                    *reinterpret_cast<float2 *>(to + n * 8 + c4 * 2) = make_float2(o[n][2 * e], o[n][2 * e + 1]);
                    *reinterpret_cast<float2 *>(to + n * 8 + 8 + c4 * 2) =
                        make_float2(o[n + 1][2 * e], o[n + 1][2 * e + 1]);
                }
            }
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
            }
            if (slot < 0) {
                store_lse(a, row_place(a, u, r), top, sum);
                inverses[r] = inverse(sum);
            } else {
                a.stats[slot * S::kRows + r] = make_float2(top, sum);
            }
        }
        __syncthreads();
        const int words = u.rows * (D / 8);
        constexpr int BATCH = 4;
#pragma unroll 1
        for (int i0 = threadIdx.x; i0 < words; i0 += BATCH * S::kThreads) {
            Vec<T, 8> gate[BATCH];
            if (slot < 0 && a.gate) {
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int i = i0 + k * S::kThreads;
                    if (i >= words) continue;
                    const RowPlace p = row_place(a, u, i / (D / 8));
                    gate[k] = load8((const T *)a.gate + p.token * a.gs + p.head * a.gh + i % (D / 8) * 8,
                                    a.gate_words);
                }
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int i = i0 + k * S::kThreads, r = i / (D / 8), e = i % (D / 8) * 8;
                if (i >= words) continue;
                float y[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) y[q] = 0.f;
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
                if (slot < 0) {
                    const float inv = inverses[r];
                    float by[8];
                    if (a.gate) gate[k].to(by);
#pragma unroll
                    for (int q = 0; q < 8; ++q) y[q] *= a.gate ? inv * sigmoid(by[q]) : inv;
                    const RowPlace p = row_place(a, u, r);
                    store8((T *)a.out + p.token * a.os + p.head * a.oh + e, a.out_words, y);
                } else {
                    float4 *to = reinterpret_cast<float4 *>(a.sums + ((int64_t)slot * S::kRows + r) * D + e);
                    to[0] = make_float4(y[0], y[1], y[2], y[3]);
                    to[1] = make_float4(y[4], y[5], y[6], y[7]);
                }
            }
        }
    });
}

template <bool EIGHT, int D, int MT, int GR>
gdn_status mma_run(int blocks, const AttentionArgs &a, cudaStream_t stream) {
    using S = Tiles<EIGHT, D, MT, GR>;
    static std::atomic<bool> done[kMaxDevices];
    const auto kernel = gdn_attention_mma_kernel<EIGHT, D, MT, GR>;
    if (!raise_shared_memory(done, {reinterpret_cast<const void *>(kernel)}, {(size_t)S::kBytes}))
        return GDN_ERR_CUDA;
    kernel<<<blocks, S::kThreads, S::kBytes, stream>>>(a);
    return launch_status();
}

// Rows of a unit in whole tiles of 16, up to four of them at a time.
inline AttentionShape mma_shape(bool eight, int R, int D) {
    const int bytes = D * (eight ? 1 : 2), tokens = 8192 / bytes < 64 ? 8192 / bytes : 64;
    return {R > 48 ? 64 : (R + 15) / 16 * 16, 4 * tokens, 2 * kGridSms};
}

template <bool EIGHT, int D>
gdn_status mma_rows(int blocks, const AttentionArgs &a, cudaStream_t stream) {
    if (a.R <= 16) return mma_run<EIGHT, D, 1, 4>(blocks, a, stream);
    if (a.R <= 32) return mma_run<EIGHT, D, 2, 2>(blocks, a, stream);
    if (a.R <= 48) return mma_run<EIGHT, D, 3, 1>(blocks, a, stream);
    return mma_run<EIGHT, D, 4, 1>(blocks, a, stream);
}

template <bool EIGHT> gdn_status mma_attention(int D, int blocks, const AttentionArgs &a, cudaStream_t stream) {
    if (D == 64) return mma_rows<EIGHT, 64>(blocks, a, stream);
    if (D == 128) return mma_rows<EIGHT, 128>(blocks, a, stream);
    return mma_rows<EIGHT, 256>(blocks, a, stream);
}

}  // namespace gdn

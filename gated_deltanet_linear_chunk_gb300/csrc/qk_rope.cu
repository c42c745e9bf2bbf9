// qk_rope.cu -- norms of queries and keys for each head with their rotation by
// position, in one pass, to tensors (gdn_qk_norm_rope) or with keys and values
// on their way into a paged cache (gdn_paged_append).
//
// Per head one read and one write of D elements and some ten operations on each:
// bound by memory.  Every warp takes an equal share of all heads, token by token,
// so the sines and cosines of a token's angles are computed once for its heads,
// one per lane.  With a weight w and x' the partner of x, norm and rotation are
//     y = (x (w cos) + x' (-+ w' sin)) / sqrt(mean(x^2) + eps)
// with factors that all heads share: a lane keeps those of its elements in
// registers, loads its words of several heads at once, and gets the partners by a
// shuffle.  Measured in bf16: 4000 tokens of 28 heads of 256, 64 of them rotated,
// 24 us (4.8 TB/s, 70 % of a copy's bandwidth), 20480 of 40 heads of 128 76 us (81
// %), 8192 of 32 heads of 256 into an 8-bit cache 61 us (60 %): issue slots are 60
// to 66 % busy, with 60 to 130 instructions per head and some 400 where a share or
// a token begins.
#include "attention.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;  // per block
constexpr int kSetup = 6;  // what a token costs beside its heads, in groups of them
// Blocks per SM, by a lane's words of a head: all blocks run at once.  (Six leave 80
// registers, of which the append of heads of up to 128 into 8 bits spills 24 bytes of
// stores and 32 of loads, and nothing else any.)
__host__ __device__ constexpr int blocks_per_sm(int words) { return words <= 1 ? 6 : words <= 4 ? 4 : 3; }

// Strides are in elements: between tokens (s), heads (h) and the cache's pages,
// places and heads.
struct RopeArgs {
    const void *q, *k, *v;
    void *q_out, *k_out;
    const float *q_weight, *k_weight, *inv_freq;
    const int32_t *positions;
    int64_t qs, qh, ks, kh, vs, vh, qos, qoh, kos, koh, axis_stride;
    int T, Hq, Hk, D, half, interleaved, warps, setup;
    float eps, inv_dim;
    // the append's
    void *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int32_t *cu, *table, *lens;
    int64_t kps, kts, khs, vps, vts, vhs, table_stride, pages;
    int N, page_size, capacity;
    uint8_t axis[kMaxRotary / 2];
};

// A turn's fraction as 64 bits: angles are positions times it, modulo 2^64,
// which is exact in the position.  inv_freq = m 2^e is multiplied by the first 64
// bits of 1 / 2 pi = 0.159.. (from its third binary place on), so the angle of
// position p is off by 2^-64 of itself and |p| 2^-63 turns.  Odd: not a number,
// for an infinite or NaN inv_freq.  (In integers: a double has eleven bits less,
// and its arithmetic runs at a 64th of fp32's rate.)
__device__ __forceinline__ uint64_t turn_of(float inv_freq) {
    constexpr uint64_t kInverse = 0xa2f9836e4e441529;  // 2^66 / 2 pi
    const uint32_t bits = __float_as_uint(inv_freq);
    int e = bits >> 23 & 255;
    if (e == 255) return 1;
    uint64_t m = bits & 0x7fffff;
    if (e > 0) m |= 0x800000;
    else e = 1;
    const uint64_t low = m * kInverse, high = __umul64hi(m, kInverse);
    const int down = 152 - e;  // the product is 2^(150 - e + 2) of 2^64 turns
    uint64_t t;
    if (down >= 64) t = down < 88 ? high >> (down - 64) : 0;
    else if (down > 0) t = low >> down | high << (64 - down);
    else t = down > -64 ? low << -down : 0;
    return (bits >> 31 ? 0 - t : t) & ~1ull;
}
// cos and sin of position times turn.  The upper 32 bits, in half turns, round
// to fp32's 24: half a step is 2^-25 half turns, 9e-8 radians.
__device__ __forceinline__ float2 angle_of(int32_t position, uint64_t turn) {
    const int32_t top = (int32_t)(((uint64_t)(int64_t)position * turn) >> 32);
    float2 r;
    sincospif((float)top * 0x1p-31f, &r.y, &r.x);
    if (turn & 1) r.x = r.y = __int_as_float(0x7fffffff);
    return r;
}

// V elements as they are stored in the cache, over its scale.
template <typename TC, int V> struct Stored {
    static __device__ __forceinline__ void store(TC *p, float (&y)[V], float) {
        Vec<TC, V>::from(y).store(p);
    }
};
template <int V> struct Stored<__nv_fp8_e4m3, V> {
    static __device__ __forceinline__ void store(__nv_fp8_e4m3 *p, float (&y)[V], float scale) {
        if constexpr (V == 8) {
            uint32_t two[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)  // a quotient, as the definition has it: no reciprocal
                two[i] = __nv_cvt_float2_to_fp8x2(
                    make_float2(__fdiv_rn(y[2 * i], scale), __fdiv_rn(y[2 * i + 1], scale)),
                    __NV_SATFINITE, __NV_E4M3);
            *reinterpret_cast<uint2 *>(p) = make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
        } else {
            static_assert(V == 1, "");
            *reinterpret_cast<uint8_t *>(p) =
                __nv_cvt_float_to_fp8(__fdiv_rn(y[0], scale), __NV_SATFINITE, __NV_E4M3);
        }
    }
};

// Where an appended token goes.
struct Placed {
    bool live;           // whether it belongs to a sequence
    int index;           // in it
    int64_t k_at, v_at;  // in the cache; -1: nowhere
};
__device__ __forceinline__ Placed place_of(const RopeArgs &a, int t) {
    Placed r = {false, 0, -1, -1};
    int n, after;  // the sequence, and its tokens from this one on
    if (a.cu) {
        if (t < a.cu[0] || t >= a.cu[a.N]) return r;
        const Span s = locate_by_warp(a.cu, a.N, a.T, t);
        n = s.n, after = s.end - t;
    } else {
        const int each = a.T / a.N;
        n = t / each, after = each - t % each;
    }
    r.live = true;
    r.index = min(max(a.lens[n], 0), a.capacity) - after;
    if (r.index < 0) return r;
    const int page = a.table[n * a.table_stride + r.index / a.page_size];
    if (page < 0 || page >= a.pages) return r;
    const int place = r.index % a.page_size;
    r.k_at = page * a.kps + place * a.kts;
    r.v_at = page * a.vps + place * a.vts;
    return r;
}
// The token's cosines and sines, pair by pair.
__device__ __forceinline__ void find_angles(const RopeArgs &a, int t, int index, const uint64_t *turn,
                                            float2 *cs, int lane) {
    for (int i = lane; i < a.half; i += 32) {
        const int32_t p = a.positions ? a.positions[a.axis[i] * a.axis_stride + t] : index;
        cs[i] = angle_of(p, turn[i]);
    }
}
// V floats from a 16-byte boundary of shared memory.
template <int V> __device__ __forceinline__ void words_of(const float *p, float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float4 w = *reinterpret_cast<const float4 *>(p + i);
        x[i] = w.x, x[i + 1] = w.y, x[i + 2] = w.z, x[i + 3] = w.w;
    }
}
// Another lane's word.
template <typename T, int V> __device__ __forceinline__ Vec<T, V> shuffle_word(const Vec<T, V> &w, int from) {
    uint32_t r[sizeof(w) / 4];
    memcpy(r, &w, sizeof(w));
#pragma unroll
    for (int i = 0; i < (int)(sizeof(w) / 4); ++i) r[i] = __shfl_sync(0xffffffffu, r[i], from);
    Vec<T, V> x;
    memcpy(&x, r, sizeof(w));
    return x;
}


// A warp's share of all tokens' groups of heads, one token after the other.  A
// token counts a few groups more than it has, for its angles and factors: the
// first ones, which are nothing.
struct Share {
    int64_t begin, end;
    __device__ __forceinline__ Share(const RopeArgs &a, int groups, int warp) {
        const int64_t all = (int64_t)a.T * (groups + a.setup), w = (int64_t)blockIdx.x * kWarps + warp;
        begin = w < a.warps ? all * w / a.warps : all;
        end = w < a.warps ? all * (w + 1) / a.warps : all;
    }
    // The token of `at` and what the share has of its groups; where the next begins.
    __device__ __forceinline__ int64_t next(const RopeArgs &a, int64_t at, int groups, int &t, int &first,
                                            int &last) const {
        const int each = groups + a.setup;
        t = (int)(at / each);
        const int from = (int)(at - (int64_t)t * each), to = (int)min((int64_t)each, from + (end - at));
        first = max(from - a.setup, 0);
        last = max(to - a.setup, 0);
        return at + (to - from);
    }
};

// Words of V elements, NW for each of a head's LANES lanes: all rows start on
// their boundaries, and a
// word's elements are rotated, with partners in one other word or its own, or not
// at all.  T: of the tensors, TC: of the cache.
template <typename T, typename TC, int V, int LANES, int NW, bool APPEND>
__global__ void __launch_bounds__(kWarps * 32, blocks_per_sm(NW)) gdn_qk_rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int U = NW == 1 ? 4 : NW == 2 ? 2 : 1;  // heads that a lane loads at once
    __shared__ float2 angles[kWarps][kMaxRotary / 2];
    __shared__ uint64_t turns[kMaxRotary / 2];
    __shared__ __align__(16) float weights[2][NW * 32 * V];  // ones where there are none
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    constexpr int ROWS = 32 / LANES;          // heads of a warp at once
    const int row = lane / LANES, mine = lane % LANES;
    bool in[NW], turned[NW];  // whether a word is in the head, and rotated
#pragma unroll
    for (int j = 0; j < NW; ++j) {
        in[j] = (mine + j * LANES) * V < a.D;
        turned[j] = (mine + j * LANES) * V < 2 * a.half;
    }
    for (int i = threadIdx.x; i < a.half; i += kWarps * 32) turns[i] = turn_of(a.inv_freq[i]);
    for (int i = threadIdx.x; i < NW * 32 * V; i += kWarps * 32) {
        weights[0][i] = a.q_weight && i < a.D ? a.q_weight[i] : 1.f;
        weights[1][i] = a.k_weight && i < a.D ? a.k_weight[i] : 1.f;
    }
    __syncthreads();
    const int heads = a.Hq + (APPEND ? 2 : 1) * a.Hk, groups = (heads + ROWS - 1) / ROWS;
    float2 *cs = angles[warp];
    const Share share(a, groups, warp);
    for (int64_t at = share.begin; at < share.end;) {
        int t, begin, end;
        at = share.next(a, at, groups, t, begin, end);
        if (begin == end) continue;
        // The token's place and angles, found while its first heads are on their way.
        Placed place = {true, 0, -1, -1};
        bool ready = false;
        auto prepare = [&] {
            if (ready) return;
            ready = true;
            if (APPEND) place = place_of(a, t);
            __syncwarp();
            find_angles(a, t, place.index, turns, cs, lane);
            __syncwarp();
        };

        // Heads [first, last) of x to `out`.
        auto norm_and_turn = [&](const T *x, int64_t hs, const float *weight, bool normed, int first,
                                 int last, auto *out, int64_t ohs, const float *scales) {
            using TO = std::remove_pointer_t<decltype(out)>;
            x += (first + row) * hs + mine * V;
            Vec<T, V> w[U][NW];
            [[maybe_unused]] Vec<T, V> v[U][NW];  // partners
            auto load = [&](int h) {  // heads from h on
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool live = h + u * ROWS < last;
#pragma unroll
                    for (int j = 0; j < NW; ++j) {
                        w[u][j] = Vec<T, V>::zero();
                        if (live && in[j]) w[u][j] = Vec<T, V>::load(x + j * LANES * V);
                        if constexpr (NW > 1) {
                            const int e = (mine + j * LANES) * V;
                            v[u][j] = Vec<T, V>::zero();
                            if (live && turned[j] && !a.interleaved)
                                v[u][j] = Vec<T, V>::load(x + j * LANES * V + (e < a.half ? a.half : -a.half));
                        }
                    }
                    x += ROWS * hs;
                }
            };
            load(first + row);
            prepare();
            if (APPEND && !place.live) return;
            uint64_t own[NW][V / 2], other[NW][V / 2];  // factors of x and x', in pairs
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                const int e0 = (mine + j * LANES) * V;
                const bool second = e0 >= a.half;
                float f[V], g[V], c[V], d[V];  // w, w', cosine and sine
                words_of<V>(weight + e0, f);
                if (a.interleaved) {
#pragma unroll
                    for (int i = 0; i < V; i += 2) {
                        const float2 q = turned[j] ? cs[(e0 + i) / 2] : make_float2(1.f, 0.f);
                        c[i] = c[i + 1] = q.x;
                        d[i] = -q.y, d[i + 1] = q.y;
                        g[i] = f[i + 1], g[i + 1] = f[i];
                    }
                } else {
                    const int partner = !turned[j] ? e0 : second ? e0 - a.half : e0 + a.half;
                    words_of<V>(weight + partner, g);
                    const float2 *pairs = cs + (turned[j] ? second ? partner : e0 : 0);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float2 q = turned[j] ? pairs[i] : make_float2(1.f, 0.f);
                        c[i] = q.x;
                        d[i] = second ? q.y : -q.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    own[j][i / 2] = pack2f(f[i] * c[i], f[i + 1] * c[i + 1]);
                    other[j][i / 2] = pack2f(g[i] * d[i], g[i + 1] * d[i + 1]);
                }
            }
            // Where a lane's partner word is, for one word per lane.
            [[maybe_unused]] const int from = !turned[0] ? lane : mine * V < a.half ? lane + a.half / V : lane - a.half / V;
            out += (first + row) * ohs + mine * V;
            for (int h = first + row; h - row < last; h += ROWS * U) {
                float inv[U];
                if (normed) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        uint64_t sums = 0;
#pragma unroll
                        for (int j = 0; j < NW; ++j) {
                            uint64_t y[V / 2];
                            to_pairs<V>(w[u][j], y);
#pragma unroll
                            for (int i = 0; i < V / 2; ++i) sums = ffma2(y[i], y[i], sums);
                        }
                        const float2 two = unpack2f(sums);
                        inv[u] = two.x + two.y;
                    }
#pragma unroll
                    for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
                        for (int u = 0; u < U; ++u) inv[u] += __shfl_xor_sync(0xffffffffu, inv[u], o);
#pragma unroll
                    for (int u = 0; u < U; ++u) inv[u] = rsqrtf(fmaf(inv[u], a.inv_dim, a.eps));
                } else {
#pragma unroll
                    for (int u = 0; u < U; ++u) inv[u] = 1.f;
                }
                if constexpr (NW > 1) __syncwarp();  // rows in place: partners have been read
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint64_t by = pack2f(inv[u], inv[u]);
                    float scale = 1.f;
                    if constexpr (sizeof(TO) == 1) scale = h + u * ROWS < last ? scales[h + u * ROWS] : 1.f;
#pragma unroll
                    for (int j = 0; j < NW; ++j) {
                        uint64_t y[V / 2], z[V / 2];
                        to_pairs<V>(w[u][j], y);
                        if (a.interleaved) {
#pragma unroll
                            for (int i = 0; i < V / 2; ++i) {
                                const float2 q = unpack2f(y[i]);
                                z[i] = pack2f(q.y, q.x);
                            }
                        } else if constexpr (NW > 1) {
                            to_pairs<V>(v[u][j], z);
                        } else {
                            to_pairs<V>(shuffle_word(w[u][0], from), z);
                        }
                        float r[V];
#pragma unroll
                        for (int i = 0; i < V / 2; ++i) {
                            // What is not rotated has no partner: not one of zero, which
                            // would spread infinities.
                            uint64_t q = fmul2(y[i], own[j][i]);
                            if (turned[j]) q = ffma2(z[i], other[j][i], q);
                            const float2 two = unpack2f(fmul2(q, by));
                            r[2 * i] = two.x, r[2 * i + 1] = two.y;
                        }
                        if (h + u * ROWS < last && in[j]) Stored<TO, V>::store(out + j * LANES * V, r, scale);
                    }
                    out += ROWS * ohs;
                }
                if (h - row + ROWS * U < last) load(h + ROWS * U);
            }
        };

        // The share's heads, of queries, keys and values counted together.
        begin *= ROWS, end *= ROWS;
        if (begin < a.Hq)
            norm_and_turn((const T *)a.q + t * a.qs, a.qh, weights[0], a.q_weight, begin, min(end, a.Hq),
                          (T *)a.q_out + t * a.qos, a.qoh, nullptr);
        const int k0 = max(begin - a.Hq, 0), k1 = min(end - a.Hq, a.Hk);
        const T *keys = (const T *)a.k + t * a.ks;
        if (!APPEND && k0 < k1)
            norm_and_turn(keys, a.kh, weights[1], a.k_weight, k0, k1, (T *)a.k_out + t * a.kos, a.koh,
                          nullptr);
        if (APPEND) prepare();
        if (APPEND && k0 < k1 && place.k_at >= 0)
            norm_and_turn(keys, a.kh, weights[1], a.k_weight, k0, k1, (TC *)a.k_cache + place.k_at, a.khs,
                          a.k_scale);
        if (APPEND && place.v_at >= 0) {
            const T *x = (const T *)a.v + t * a.vs;
            TC *to = (TC *)a.v_cache + place.v_at;
            const int v0 = max(begin - a.Hq - a.Hk, 0), v1 = min(end - a.Hq - a.Hk, a.Hk);
            for (int h0 = v0; h0 < v1; h0 += ROWS * U) {
                Vec<T, V> w[U][NW];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int j = 0; j < NW; ++j) {
                        const int h = h0 + u * ROWS + row, e = (mine + j * LANES) * V;
                        w[u][j] = Vec<T, V>::zero();
                        if (h < v1 && e < a.D) w[u][j] = Vec<T, V>::load(x + (int64_t)h * a.vh + e);
                    }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int j = 0; j < NW; ++j) {
                        const int h = h0 + u * ROWS + row, e = (mine + j * LANES) * V;
                        if (h >= v1 || e >= a.D) continue;
                        float y[V];
                        w[u][j].to(y);
                        Stored<TC, V>::store(to + h * a.vhs + e, y, a.v_scale ? a.v_scale[h] : 1.f);
                    }
            }
        }
    }
}

// The same element by element, for any alignment and sizes: lanes take every
// 32nd element of a head, NW of them.
template <typename T, typename TC, int NW, bool APPEND>
__global__ void __launch_bounds__(kWarps * 32, blocks_per_sm(NW))
gdn_qk_rope_elements_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ float2 angles[kWarps][kMaxRotary / 2];
    __shared__ uint64_t turns[kMaxRotary / 2];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int i = threadIdx.x; i < a.half; i += kWarps * 32) turns[i] = turn_of(a.inv_freq[i]);
    __syncthreads();
    const int heads = a.Hq + (APPEND ? 2 : 1) * a.Hk;
    float2 *cs = angles[warp];
    const Share share(a, heads, warp);
    for (int64_t at = share.begin; at < share.end;) {
        int t, begin, end;
        at = share.next(a, at, heads, t, begin, end);
        if (begin == end) continue;
        Placed place = {true, 0, -1, -1};
        if (APPEND) {
            place = place_of(a, t);
            if (!place.live) continue;
        }
        __syncwarp();
        find_angles(a, t, place.index, turns, cs, lane);
        __syncwarp();
        for (int i = begin; i < end; ++i) {
            const bool is_q = i < a.Hq, is_k = !is_q && i < a.Hq + a.Hk;
            const int h = is_q ? i : is_k ? i - a.Hq : i - a.Hq - a.Hk;
            const T *x = is_q   ? (const T *)a.q + t * a.qs + h * a.qh
                         : is_k ? (const T *)a.k + t * a.ks + h * a.kh
                                : (const T *)a.v + t * a.vs + h * a.vh;
            const float *weight = is_q ? a.q_weight : is_k ? a.k_weight : nullptr;
            float y[NW], z[NW], sum = 0.f;
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                const int e = lane + j * 32;
                y[j] = z[j] = 0.f;
                if (e < a.D) y[j] = to_f32(x[e]);
                if (e < 2 * a.half && (is_q || is_k))
                    z[j] = to_f32(x[a.interleaved ? e ^ 1 : e < a.half ? e + a.half : e - a.half]);
                sum = fmaf(y[j], y[j], sum);
            }
            const float inv = weight ? rsqrtf(fmaf(warp_sum(sum), a.inv_dim, a.eps)) : 1.f;
            __syncwarp();  // every lane has read before any writes: rows may be in place
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                const int e = lane + j * 32;
                if (e >= a.D) continue;
                float r = y[j] * (weight ? weight[e] : 1.f);
                if (e < 2 * a.half && (is_q || is_k)) {
                    const bool second = a.interleaved ? e & 1 : e >= a.half;
                    const int partner = a.interleaved ? e ^ 1 : second ? e - a.half : e + a.half;
                    const float2 c = cs[a.interleaved ? e / 2 : second ? partner : e];
                    const float p = z[j] * (weight ? weight[partner] : 1.f);
                    r = fmaf(second ? p : -p, c.y, r * c.x);
                }
                r *= inv;
                float one[1] = {r};
                if (is_q)
                    ((T *)a.q_out)[t * a.qos + h * a.qoh + e] = from_f32<T>(r);
                else if (!APPEND)
                    ((T *)a.k_out)[t * a.kos + h * a.koh + e] = from_f32<T>(r);
                else if (is_k && place.k_at >= 0)
                    Stored<TC, 1>::store((TC *)a.k_cache + place.k_at + h * a.khs + e, one,
                                         a.k_scale ? a.k_scale[h] : 1.f);
                else if (!is_k && place.v_at >= 0)
                    Stored<TC, 1>::store((TC *)a.v_cache + place.v_at + h * a.vhs + e, one,
                                         a.v_scale ? a.v_scale[h] : 1.f);
            }
        }
    }
}

// LANES 0: element by element.
template <typename T, typename TC, int V, int LANES, int NW, bool APPEND>
gdn_status run(RopeArgs &a, cudaStream_t stream) {
    constexpr int ROWS = LANES > 0 ? 32 / LANES : 1;
    const int heads = a.Hq + (APPEND ? 2 : 1) * a.Hk, groups = (heads + ROWS - 1) / ROWS;
    // Every SM has its warps; of few heads each warp has one group.
    constexpr int most = kGridSms * blocks_per_sm(NW) * kWarps;
    const int64_t all = (int64_t)a.T * groups;
    a.warps = (int)(all < most ? all : most);
    a.setup = all < most ? 0 : kSetup;
    const unsigned grid = (unsigned)((a.warps + kWarps - 1) / kWarps);
    if constexpr (LANES > 0)
        return launch_programmatic(gdn_qk_rope_kernel<T, TC, V, LANES, NW, APPEND>, dim3(grid), kWarps * 32,
                                   0, stream, a);
    else
        return launch_programmatic(gdn_qk_rope_elements_kernel<T, TC, NW, APPEND>, dim3(grid), kWarps * 32,
                                   0, stream, a);
}

template <typename T, typename TC, bool APPEND>
gdn_status sized(RopeArgs &a, cudaStream_t stream) {
    constexpr int V = kWide<T>;
    // Words of V elements, if all rows start on their boundaries and no word
    // holds rotated elements beside others, or pairs of two partners.
    auto rows = [](const void *p, size_t bytes, std::initializer_list<int64_t> strides) {
        if (!p) return true;
        uintptr_t all = reinterpret_cast<uintptr_t>(p);
        for (int64_t s : strides) all |= (uintptr_t)s * (bytes / V);
        return all % bytes == 0;
    };
    const size_t e = V * sizeof(T), c = V * sizeof(TC);
    const bool wide =
        a.D % V == 0 && (a.interleaved ? 2 * a.half : a.half) % V == 0 &&
        rows(a.q, e, {a.qs, a.qh}) && rows(a.k, e, {a.ks, a.kh}) &&
        rows(a.q_out, e, {a.qos, a.qoh}) &&
        (APPEND ? rows(a.v, e, {a.vs, a.vh}) && rows(a.k_cache, c, {a.kps, a.kts, a.khs}) &&
                      rows(a.v_cache, c, {a.vps, a.vts, a.vhs})
                : rows(a.k_out, e, {a.kos, a.koh}));
    if (wide) {
        const int words = a.D / V;
        if (words <= 8) return run<T, TC, V, 8, 1, APPEND>(a, stream);
        if (words <= 16) return run<T, TC, V, 16, 1, APPEND>(a, stream);
        if (words <= 32) return run<T, TC, V, 32, 1, APPEND>(a, stream);
        if (V == 8 || words <= 64) return run<T, TC, V, 32, 2, APPEND>(a, stream);
        if constexpr (V < 8) return run<T, TC, V, 32, 4, APPEND>(a, stream);
    }
    if (a.D <= 64) return run<T, TC, 1, 0, 2, APPEND>(a, stream);
    if (a.D <= 128) return run<T, TC, 1, 0, 4, APPEND>(a, stream);
    if (a.D <= 256) return run<T, TC, 1, 0, 8, APPEND>(a, stream);
    return run<T, TC, 1, 0, 16, APPEND>(a, stream);
}

}  // namespace

gdn_status launch_qk_rope(const gdn_rope_problem &p, const gdn_paged_cache *cache, const void *q,
                          const void *k, const void *v, const float *q_weight,
                          const float *k_weight, const int32_t *positions, const float *inv_freq,
                          const int32_t *cu, void *q_out, void *k_out, cudaStream_t stream) {
    RopeArgs a = {};
    a.q = q, a.k = k, a.v = v, a.q_out = q_out, a.k_out = k_out;
    a.q_weight = q_weight, a.k_weight = k_weight;
    a.positions = positions, a.inv_freq = inv_freq;
    a.qs = p.q_stride, a.qh = p.q_head_stride, a.ks = p.k_stride, a.kh = p.k_head_stride;
    a.vs = p.v_stride, a.vh = p.v_head_stride;
    a.qos = p.q_out_stride, a.qoh = p.q_out_head_stride;
    a.kos = p.k_out_stride, a.koh = p.k_out_head_stride;
    a.axis_stride = p.axis_stride;
    a.T = (int)p.total_tokens, a.Hq = p.q_heads, a.Hk = p.kv_heads, a.D = p.head_dim;
    a.half = p.rotary_dim / 2, a.interleaved = p.interleaved != 0;
    a.eps = p.eps, a.inv_dim = 1.f / (float)p.head_dim;
    if (p.freq_axis)
        for (int i = 0; i < a.half; ++i) a.axis[i] = p.freq_axis[i];
    if (!cache)
        return p.dtype == GDN_F32 ? sized<float, float, false>(a, stream)
                                  : sized<__nv_bfloat16, __nv_bfloat16, false>(a, stream);
    a.k_cache = cache->k, a.v_cache = cache->v;
    a.k_scale = cache->k_scale, a.v_scale = cache->v_scale;
    a.kps = cache->k_page_stride, a.kts = cache->k_token_stride, a.khs = cache->k_head_stride;
    a.vps = cache->v_page_stride, a.vts = cache->v_token_stride, a.vhs = cache->v_head_stride;
    a.cu = cu, a.table = cache->page_table, a.lens = cache->seq_lens;
    a.table_stride = cache->table_stride, a.pages = cache->num_pages;
    a.N = cache->num_seqs, a.page_size = cache->page_size;
    a.capacity = cache->max_pages * cache->page_size;
    if (cache->dtype == GDN_E4M3)
        return sized<__nv_bfloat16, __nv_fp8_e4m3, true>(a, stream);
    return p.dtype == GDN_F32 ? sized<float, float, true>(a, stream)
                              : sized<__nv_bfloat16, __nv_bfloat16, true>(a, stream);
}

}  // namespace gdn

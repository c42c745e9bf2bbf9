// qk_rope.cu -- norms of queries and keys for each head with their rotation by
// position, in one pass, to tensors (gdn_qk_norm_rope) or with keys and values
// on their way into a paged cache (gdn_paged_append).
//
// Per head one read and one write of D elements and some ten operations on
// each: bound by memory.  A warp takes a token, or a part of its heads where
// there are few tokens, so the sines and cosines of the token's angles are
// computed once for all its heads, one per lane, and kept in shared memory.
#include "attention.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;  // per block

// The head's elements of one tensor: from, to (null: nothing is stored) and
// the strides between heads.
struct RopeArgs {
    const void *q, *k, *v;
    void *q_out, *k_out;
    const float *q_weight, *k_weight, *inv_freq;
    const int32_t *positions;
    int64_t qs, qh, ks, kh, vs, vh, qos, qoh, kos, koh, axis_stride;
    int T, Hq, Hk, D, half, interleaved, lanes, parts;
    float eps;
    // the append's
    void *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int32_t *cu, *table, *lens;
    int64_t kps, kts, khs, vps, vts, vhs, table_stride, pages;
    int N, page_size, capacity;
    uint8_t axis[kMaxRotary / 2];
};

// A turn's fraction as 64 bits: angles are positions times it, modulo 2^64,
// which is exact in the position.  inv_freq / 2 pi is rounded to double's 53
// bits, so the angle of position p is off by |p| 2^-53 of inv_freq: 1e-7 radians
// at 2^29 and one radian per position.  (One double product per pair and warp;
// the positions' products are of integers.)
__device__ __forceinline__ uint64_t turn_of(float inv_freq) {
    double t = (double)inv_freq * 0.15915494309189533577;  // 1 / 2 pi
    t -= floor(t);
    return (uint64_t)(t * 18446744073709551616.0);
}
// cos and sin of position times turn.  The upper 32 bits, in half turns, round
// to fp32's 24: half a step is 2^-25 half turns, 9e-8 radians.
__device__ __forceinline__ float2 angle_of(int32_t position, uint64_t turn) {
    const int32_t top = (int32_t)(((uint64_t)(int64_t)position * turn) >> 32);
    float2 r;
    sincospif((float)top * 0x1p-31f, &r.y, &r.x);
    return r;
}

// V elements as they are stored in the cache, times 1 / scale of it.
template <typename TC, int V> struct Stored {
    static __device__ __forceinline__ void store(TC *p, float (&y)[V], float) {
        Vec<TC, V>::from(y).store(p);
    }
};
template <int V> struct Stored<__nv_fp8_e4m3, V> {
    static __device__ __forceinline__ void store(__nv_fp8_e4m3 *p, float (&y)[V], float scale) {
        uint8_t b[V];
#pragma unroll
        for (int i = 0; i < V; ++i)  // a quotient, as the definition has it: no reciprocal
            b[i] = __nv_cvt_float_to_fp8(__fdiv_rn(y[i], scale), __NV_SATFINITE, __NV_E4M3);
        if constexpr (V == 8) {
            uint2 w;
            w.x = b[0] | b[1] << 8 | b[2] << 16 | (uint32_t)b[3] << 24;
            w.y = b[4] | b[5] << 8 | b[6] << 16 | (uint32_t)b[7] << 24;
            *reinterpret_cast<uint2 *>(p) = w;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) reinterpret_cast<uint8_t *>(p)[i] = b[i];
        }
    }
};

// What a lane does with its j-th word of a head: its first element, whether it
// lies in the head, and for rotated ones the partner's element and the pair.
struct Word {
    int e, partner, pair;
    float sign;  // of the sine's term: -1 for a pair's first element
    bool in, turned;
};

// T: of the tensors, TC: of the cache.  V elements per word, NW words per lane.
template <typename T, typename TC, int V, int NW, bool APPEND>
__global__ void __launch_bounds__(kWarps * 32) gdn_qk_rope_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ float2 turns[kWarps][kMaxRotary / 2];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t at = (int64_t)blockIdx.x * kWarps + warp;
    const int t = (int)(at / a.parts), part = (int)(at % a.parts);
    if (t >= a.T) return;
    float2 *cs = turns[warp];

    // The token's place.
    int index = 0;
    int64_t k_at = -1, v_at = -1;
    if (APPEND) {
        int n, after;  // the sequence, and its tokens from this one on
        if (a.cu) {
            if (t < a.cu[0] || t >= a.cu[a.N]) return;
            const Span s = locate_by_warp(a.cu, a.N, a.T, t);
            n = s.n, after = s.end - t;
        } else {
            const int each = a.T / a.N;
            n = t / each, after = each - t % each;
        }
        index = min(max(a.lens[n], 0), a.capacity) - after;
        if (index >= 0) {
            const int page = a.table[n * a.table_stride + index / a.page_size];
            if (page >= 0 && page < a.pages) {
                const int place = index % a.page_size;
                k_at = page * a.kps + place * a.kts;
                v_at = page * a.vps + place * a.vts;
            }
        }
    }
    for (int i = lane; i < a.half; i += 32) {
        const float f = a.inv_freq[i];
        const int32_t p = a.positions ? a.positions[a.axis[i] * a.axis_stride + t] : index;
        float2 r = angle_of(p, turn_of(f));
        if (!isfinite(f)) r.x = r.y = __int_as_float(0x7fffffff);
        cs[i] = r;
    }
    __syncwarp();

    const int lanes = a.lanes, row = lane / lanes, mine = lane % lanes, rows = 32 / lanes;
    Word word[NW];
#pragma unroll
    for (int j = 0; j < NW; ++j) {
        Word &w = word[j];
        w.e = (mine + j * lanes) * V;
        w.in = w.e < a.D;
        w.turned = w.e < 2 * a.half;
        if (a.interleaved) {
            w.pair = w.e / 2;
            w.partner = w.e ^ 1;  // of one element; longer words hold both
            w.sign = w.e & 1 ? 1.f : -1.f;
        } else {
            const bool first = w.e < a.half;
            w.pair = first ? w.e : w.e - a.half;
            w.partner = first ? w.e + a.half : w.e - a.half;
            w.sign = first ? -1.f : 1.f;
        }
    }
    const bool beside = !(V > 1 && a.interleaved);  // whether partners are in other words

    // Heads [h0, h1) of x, `heads` in all, of which this warp takes every
    // parts-th group.
    auto norm_and_turn = [&](const T *x, int64_t hs, const float *weight, int first, int last,
                             auto &&put) {
        float w[NW][V], pw[NW][V];
        if (weight) {
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                if (!word[j].in) continue;
#pragma unroll
                for (int i = 0; i < V; ++i) w[j][i] = weight[word[j].e + i];
                if (beside && word[j].turned)
#pragma unroll
                    for (int i = 0; i < V; ++i) pw[j][i] = weight[word[j].partner + i];
            }
        }
        for (int h0 = first; h0 < last; h0 += rows) {
            const int h = h0 + row;
            const bool live = h < last;
            const T *from = x + (int64_t)h * hs;
            float y[NW][V], py[NW][V];
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < NW; ++j) {
#pragma unroll
                for (int i = 0; i < V; ++i) y[j][i] = py[j][i] = 0.f;
                if (!live || !word[j].in) continue;
                Vec<T, V>::load(from + word[j].e).to(y[j]);
                if (beside && word[j].turned) Vec<T, V>::load(from + word[j].partner).to(py[j]);
            }
            if (weight) {
#pragma unroll
                for (int j = 0; j < NW; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) sum = fmaf(y[j][i], y[j][i], sum);
                for (int o = lanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const float inv = rsqrtf(sum / (float)a.D + a.eps);
#pragma unroll
                for (int j = 0; j < NW; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        y[j][i] *= inv * w[j][i];
                        if (beside) py[j][i] *= inv * pw[j][i];
                    }
            }
            __syncwarp();  // every lane has read before any writes: rows may be in place
            if (!live) continue;
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                const Word &d = word[j];
                if (!d.in) continue;
                if (d.turned) {
                    if (beside) {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float2 c = cs[d.pair + i];
                            y[j][i] = fmaf(d.sign * py[j][i], c.y, y[j][i] * c.x);
                        }
                    } else if constexpr (V > 1) {
#pragma unroll
                        for (int i = 0; i < V; i += 2) {
                            const float2 c = cs[d.pair + i / 2];
                            const float b = y[j][i + 1];
                            y[j][i + 1] = fmaf(y[j][i], c.y, b * c.x);
                            y[j][i] = fmaf(-b, c.y, y[j][i] * c.x);
                        }
                    }
                }
                put(h, d.e, y[j]);
            }
        }
    };

    // The part's heads, of queries, keys and values counted together.
    const int all = a.Hq + (APPEND ? 2 : 1) * a.Hk;
    const int groups = (all + rows - 1) / rows;  // shares in whole groups of rows
    const int begin = (int)((int64_t)groups * part / a.parts) * rows,
              end = (int)((int64_t)groups * (part + 1) / a.parts) * rows;
    if (begin < a.Hq) {
        T *to = (T *)a.q_out + t * a.qos;
        norm_and_turn((const T *)a.q + t * a.qs, a.qh, a.q_weight, begin, min(end, a.Hq),
                      [&](int h, int e, float(&y)[V]) {
                          Vec<T, V>::from(y).store(to + (int64_t)h * a.qoh + e);
                      });
    }
    const int k0 = max(begin - a.Hq, 0), k1 = min(end - a.Hq, a.Hk);
    if (k0 < k1 && (!APPEND || k_at >= 0)) {
        const T *x = (const T *)a.k + t * a.ks;
        if (APPEND) {
            TC *to = (TC *)a.k_cache + k_at;
            norm_and_turn(x, a.kh, a.k_weight, k0, k1, [&](int h, int e, float(&y)[V]) {
                Stored<TC, V>::store(to + h * a.khs + e, y, a.k_scale ? a.k_scale[h] : 1.f);
            });
        } else {
            T *to = (T *)a.k_out + t * a.kos;
            norm_and_turn(x, a.kh, a.k_weight, k0, k1, [&](int h, int e, float(&y)[V]) {
                Vec<T, V>::from(y).store(to + (int64_t)h * a.koh + e);
            });
        }
    }
    if (APPEND && v_at >= 0) {
        const T *x = (const T *)a.v + t * a.vs;
        TC *to = (TC *)a.v_cache + v_at;
        const int v0 = max(begin - a.Hq - a.Hk, 0), v1 = min(end - a.Hq - a.Hk, a.Hk);
        for (int h = v0 + row; h < v1; h += rows) {
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                if (!word[j].in) continue;
                float y[V];
                Vec<T, V>::load(x + (int64_t)h * a.vh + word[j].e).to(y);
                Stored<TC, V>::store(to + h * a.vhs + word[j].e, y, a.v_scale ? a.v_scale[h] : 1.f);
            }
        }
    }
}

template <typename T, typename TC, int V, int NW, bool APPEND>
gdn_status run(RopeArgs &a, cudaStream_t stream) {
    const int words = (a.D + V - 1) / V;
    a.lanes = 32;
    while (NW == 1 && a.lanes / 2 >= words) a.lanes /= 2;
    const int rows = 32 / a.lanes, heads = a.Hq + (APPEND ? 2 : 1) * a.Hk;
    const int groups = (heads + rows - 1) / rows;
    // Few tokens are cut into parts until every SM has eight warps.
    const int want = (kGridSms * 8 + a.T - 1) / a.T;
    a.parts = want < 1 ? 1 : want < groups ? want : groups;
    const int64_t warps = (int64_t)a.T * a.parts;
    gdn_qk_rope_kernel<T, TC, V, NW, APPEND>
        <<<(unsigned)((warps + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(a);
    return launch_status();
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
    const int words = wide ? a.D / V : a.D;
    if (wide) {
        if (words <= 32) return run<T, TC, V, 1, APPEND>(a, stream);
        if (words <= 64) return run<T, TC, V, 2, APPEND>(a, stream);
        return run<T, TC, V, 4, APPEND>(a, stream);
    }
    if (words <= 64) return run<T, TC, 1, 2, APPEND>(a, stream);
    if (words <= 128) return run<T, TC, 1, 4, APPEND>(a, stream);
    if (words <= 256) return run<T, TC, 1, 8, APPEND>(a, stream);
    return run<T, TC, 1, 16, APPEND>(a, stream);
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
    a.eps = p.eps;
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

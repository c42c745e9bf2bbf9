// block.cuh -- shared pieces of the operators of include/gdn_block.h (not part
// of the ABI): vector loads, elementary functions, the sequence of a token.
#pragma once

#include <atomic>
#include <initializer_list>

#include "common.cuh"
#include "gdn_block.h"

namespace gdn {

constexpr int kGridSms = 152;  // SMs of a GB300: the grids are sized for it

// ------------------------------------------------------- elementary functions
// ex2.approx and rcp.approx: two ulp and one, flushing denormals.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + e^-v): e^-v overflows to infinity below -88, where the result is 0.
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + ex2(-kLog2e * v)); }
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }

// log(1 + e^v) = max(v, 0) + log1p(e) with e = e^-|v| in (0, 1].  log1p(e) / e
// is a polynomial of degree 8, fitted to the least largest relative error on
// [0, 1] (6.4e-8 with the coefficients rounded to fp32; 1.8e-7 in fp32 arithmetic,
// 4e-8 on average): relative accuracy is kept for the small steps of very negative v, where log1p(e) is e.  (NaN:
// e is NaN, and so is the result.)
__device__ __forceinline__ constexpr float softplus_coefficient(int power) {
    constexpr float c[9] = {0.9999999403953552f,  -0.4999949336051941f,  0.3331909775733948f,
                            -0.2484298199415207f, 0.19106008112430573f,  -0.13663247227668762f,
                            0.07822594791650772f, -0.029505232349038124f, 0.005232691299170256f};
    return c[power];
}
__device__ __forceinline__ float softplus(float v) {
    const float e = ex2(-kLog2e * fabsf(v));
    float p = softplus_coefficient(8);
#pragma unroll
    for (int k = 7; k >= 0; --k) p = fmaf(p, e, softplus_coefficient(k));
    return fmaf(p, e, fmaxf(v, 0.f));
}

// ------------------------------------------------------- pairs of fp32 values
// Two values in one 64-bit register pair, and the packed operations on them.
__device__ __forceinline__ uint64_t pack2f(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2f(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// softplus, sigmoid and silu of both.
__device__ __forceinline__ uint64_t softplus2(uint64_t v) {
    const float2 w = unpack2f(v);
    const uint64_t e = pack2f(ex2(-kLog2e * fabsf(w.x)), ex2(-kLog2e * fabsf(w.y)));
    uint64_t p = pack2f(softplus_coefficient(8), softplus_coefficient(8));
#pragma unroll
    for (int k = 7; k >= 0; --k)
        p = ffma2(p, e, pack2f(softplus_coefficient(k), softplus_coefficient(k)));
    return ffma2(p, e, pack2f(fmaxf(w.x, 0.f), fmaxf(w.y, 0.f)));
}
__device__ __forceinline__ uint64_t sigmoid2(uint64_t v) {
    const float2 e = unpack2f(fmul2(v, pack2f(-kLog2e, -kLog2e)));
    const float2 f = unpack2f(fadd2(pack2f(ex2(e.x), ex2(e.y)), pack2f(1.f, 1.f)));
    return pack2f(rcp(f.x), rcp(f.y));
}
__device__ __forceinline__ uint64_t silu2(uint64_t v) { return fmul2(v, sigmoid2(v)); }

// ------------------------------------------------------------- vector access
// V consecutive elements in one word of up to 16 bytes.
template <typename T, int V> struct Vec;
template <typename T> struct Vec<T, 1> {
    T w;
    __device__ __forceinline__ static Vec load(const T *p) { return Vec{*p}; }
    __device__ __forceinline__ void store(T *p) const { *p = w; }
    __device__ __forceinline__ static Vec zero() { return Vec{from_f32<T>(0.f)}; }
    __device__ __forceinline__ void to(float *r) const { r[0] = to_f32(w); }
    __device__ __forceinline__ static Vec from(const float *r) { return Vec{from_f32<T>(r[0])}; }
};
template <> struct Vec<float, 4> {
    float4 w;
    __device__ __forceinline__ static Vec load(const float *p) {
        return Vec{*reinterpret_cast<const float4 *>(p)};
    }
    __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float4 *>(p) = w; }
    __device__ __forceinline__ static Vec zero() { return Vec{make_float4(0.f, 0.f, 0.f, 0.f)}; }
    __device__ __forceinline__ void to(float *r) const {
        r[0] = w.x; r[1] = w.y; r[2] = w.z; r[3] = w.w;
    }
    __device__ __forceinline__ static Vec from(const float *r) {
        return Vec{make_float4(r[0], r[1], r[2], r[3])};
    }
};
template <> struct Vec<__nv_bfloat16, 8> {
    uint4 w;
    __device__ __forceinline__ static Vec load(const __nv_bfloat16 *p) {
        return Vec{*reinterpret_cast<const uint4 *>(p)};
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
        *reinterpret_cast<uint4 *>(p) = w;
    }
    __device__ __forceinline__ static Vec zero() { return Vec{make_uint4(0, 0, 0, 0)}; }
    __device__ __forceinline__ void to(float *r) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[2 * i] = __uint_as_float(u[i] << 16);
            r[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ static Vec from(const float *r) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(r[2 * i], r[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return Vec{make_uint4(u[0], u[1], u[2], u[3])};
    }
};
template <> struct Vec<__nv_bfloat16, 4> {
    uint2 w;
    __device__ __forceinline__ static Vec load(const __nv_bfloat16 *p) {
        return Vec{*reinterpret_cast<const uint2 *>(p)};
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
        *reinterpret_cast<uint2 *>(p) = w;
    }
    __device__ __forceinline__ static Vec zero() { return Vec{make_uint2(0, 0)}; }
    __device__ __forceinline__ void to(float *r) const {
        r[0] = __uint_as_float(w.x << 16);
        r[1] = __uint_as_float(w.x & 0xffff0000u);
        r[2] = __uint_as_float(w.y << 16);
        r[3] = __uint_as_float(w.y & 0xffff0000u);
    }
    __device__ __forceinline__ static Vec from(const float *r) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(r[0], r[1]);
        const __nv_bfloat162 g = __floats2bfloat162_rn(r[2], r[3]);
        return Vec{make_uint2(*reinterpret_cast<const uint32_t *>(&h),
                              *reinterpret_cast<const uint32_t *>(&g))};
    }
};
template <> struct Vec<__nv_bfloat16, 2> {
    uint32_t w;
    __device__ __forceinline__ static Vec load(const __nv_bfloat16 *p) {
        return Vec{*reinterpret_cast<const uint32_t *>(p)};
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
        *reinterpret_cast<uint32_t *>(p) = w;
    }
    __device__ __forceinline__ void to(float *r) const {
        r[0] = __uint_as_float(w << 16);
        r[1] = __uint_as_float(w & 0xffff0000u);
    }
    __device__ __forceinline__ static Vec from(const float *r) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(r[0], r[1]);
        return Vec{*reinterpret_cast<const uint32_t *>(&h)};
    }
    __device__ __forceinline__ static Vec zero() { return Vec{0u}; }
};
template <> struct Vec<float, 2> {
    float2 w;
    __device__ __forceinline__ static Vec load(const float *p) {
        return Vec{*reinterpret_cast<const float2 *>(p)};
    }
    __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float2 *>(p) = w; }
    __device__ __forceinline__ void to(float *r) const { r[0] = w.x; r[1] = w.y; }
    __device__ __forceinline__ static Vec from(const float *r) {
        return Vec{make_float2(r[0], r[1])};
    }
};
// Whether element p lies in the upper half of its 4-byte word.
template <typename T> __host__ __device__ __forceinline__ int odd(const T *p) {
    return (int)(reinterpret_cast<uintptr_t>(p) / sizeof(T)) & 1;
}
// V elements of a word as pairs (an element alone: with a zero), and back.
template <int V, typename Word>
__device__ __forceinline__ void to_pairs(const Word &w, uint64_t (&p)[(V + 1) / 2]) {
    float r[V + 1];
    r[V] = 0.f;
    w.to(r);
#pragma unroll
    for (int i = 0; i < V; i += 2) p[i / 2] = pack2f(r[i], r[i + 1]);
}
template <int V>
__device__ __forceinline__ void from_pairs(const uint64_t (&p)[(V + 1) / 2], float (&r)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        const float2 v = unpack2f(p[i / 2]);
        r[i] = v.x;
        if (i + 1 < V) r[i + 1] = v.y;
    }
}
template <typename T> constexpr int kWide = 16 / (int)sizeof(T);

// Whether rows at p, `stride` elements apart, start on 16-byte boundaries.
template <typename T> inline bool rows_aligned16(const void *p, int64_t stride) {
    return !p || (aligned16(p) && (stride * (int64_t)sizeof(T)) % 16 == 0);
}

// ------------------------------------------------------- asynchronous copies
// From global to shared memory, 4 or 16 bytes, both sides aligned to them.
// (PART: the rest of a 32-byte sector is copied by this thread's next copy, which
// finds it in L1.)
template <int BYTES, bool PART = false>
__device__ __forceinline__ void copy_async(void *smem, const void *gmem) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    if constexpr (BYTES == 16 && !PART)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(gmem) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(gmem), "n"(BYTES)
                     : "memory");
}
// The first `bytes` of 16; the rest becomes zero.
__device__ __forceinline__ void copy_async_head(void *smem, const void *gmem, int bytes) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(gmem), "r"(bytes)
                 : "memory");
}
// 16 bytes that are not read again soon.
__device__ __forceinline__ uint64_t evict_first_policy() {
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    return policy;
}
__device__ __forceinline__ void copy_async_once(void *smem, const void *gmem, uint64_t policy) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(to), "l"(gmem),
                 "l"(policy)
                 : "memory");
}
// The first `bytes` (2 or 4) of a 4-byte word; the rest of it becomes zero.
__device__ __forceinline__ void copy_async_part(void *smem, const void *gmem, int bytes) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(gmem), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N committed groups of this thread's copies are on their way.
template <int N> __device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// What a copy of the 16-bit element at p reads: its 4-byte word up to the
// element.  (high: odd(p).)  The element that begins its tensor (`first`) in the
// upper half of a word has nothing before it that is the tensor's: no bytes are
// read, and load_first brings it.
template <typename T> struct ElementWord {
    const T *from;
    int bytes;
};
template <typename T>
__host__ __device__ __forceinline__ ElementWord<T> element_word(const T *p, int high, bool first) {
    return {p - high, high ? first ? 0 : 4 : 2};
}
// The 16-bit element at p to its half of a 4-byte word.
template <typename T>
__device__ __forceinline__ void copy_async_element(void *smem, const T *p, int high, bool first) {
    const ElementWord<T> w = element_word(p, high, first);
    copy_async_part(smem, w.from, w.bytes);
}
// A tensor's first element to the place that copy_async_element gave it, once
// this thread's copies are there.
template <typename T> __device__ __forceinline__ void load_first(void *smem, const T *p) {
    if (!odd(p)) return;
    copies_wait<0>();
    *static_cast<uint32_t *>(smem) = (uint32_t)*reinterpret_cast<const uint16_t *>(p) << 16;
}

// A kernel has 48 KB of shared memory by default: for more the limit is raised
// once per device and variant.
constexpr int kMaxDevices = 64;
inline bool raise_shared_memory(std::atomic<bool> (&done)[kMaxDevices],
                                std::initializer_list<const void *> kernels,
                                std::initializer_list<size_t> bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
    if (done[dev].load(std::memory_order_acquire)) return true;
    auto size = bytes.begin();
    for (const void *k : kernels)
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)*size++) != cudaSuccess)
            return false;
    done[dev].store(true, std::memory_order_release);
    return true;
}

// ---------------------------------------------------- packed sequences
// Sequence n holds tokens [start, end).  Values read from cu_seqlens are
// clamped so that start <= t < end <= T for the token t asked for, whatever
// the array holds.
struct Span {
    int n, start, end;
};

__device__ __forceinline__ Span span_at(const int32_t *cu, int N, int T, int t, int n) {
    const int s = cu[n], e = cu[n + 1];
    return Span{n, min(max(s, 0), t), min(max(e, t + 1), T)};
}

// The sequence of token t (0 <= t < T): the last n with cu[n] <= t.
__device__ __forceinline__ Span locate(const int32_t *cu, int N, int T, int t) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return span_at(cu, N, T, t, lo);
}

// The same by all 32 lanes of a warp, for one t: a probe per lane and round.
__device__ __forceinline__ Span locate_by_warp(const int32_t *cu, int N, int T, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
        const int passed = __popc(__ballot_sync(0xffffffffu, at <= hi && cu[at] <= t));
        lo += passed * step;
        hi = min(hi, lo + step - 1);
    }
    return span_at(cu, N, T, t, lo);
}

// The sequence of token t = s.end: the next one that is not empty.
__device__ __forceinline__ Span next_span(const int32_t *cu, int N, int T, const Span &s) {
    int n = s.n;
    while (n < N - 1 && cu[n + 1] <= s.end) ++n;
    Span r = span_at(cu, N, T, s.end, n);
    r.start = s.end;
    return r;
}

// ------------------------------------------------------------------ launchers
gdn_status launch_short_conv(const gdn_conv_problem &p, const void *x, const float *weight,
                             const float *bias, const int32_t *cu, const void *init, void *out,
                             void *fin, cudaStream_t stream);
gdn_status launch_short_conv_step(const gdn_conv_problem &p, const void *x, const float *weight,
                                  const float *bias, const void *state, void *out, void *next,
                                  cudaStream_t stream);
size_t scan_workspace_size(const gdn_ssm_problem &p);
gdn_status launch_selective_scan_bf16(const gdn_ssm_problem &p, const void *x, const void *dt,
                                      const float *A, const void *B, const void *C,
                                      const float *skip, const void *z, const float *bias,
                                      const int32_t *cu, const float *init, void *out, float *fin,
                                      cudaStream_t stream);
gdn_status launch_selective_scan_f32(const gdn_ssm_problem &p, const void *x, const void *dt,
                                     const float *A, const void *B, const void *C,
                                     const float *skip, const void *z, const float *bias,
                                     const int32_t *cu, const float *init, void *out, float *fin,
                                     cudaStream_t stream);
gdn_status launch_selective_scan_step_bf16(const gdn_ssm_problem &p, const void *x,
                                           const void *dt, const float *A, const void *B,
                                           const void *C, const float *skip, const void *z,
                                           const float *bias, const float *state, void *out,
                                           float *next, cudaStream_t stream);
gdn_status launch_selective_scan_step_f32(const gdn_ssm_problem &p, const void *x, const void *dt,
                                          const float *A, const void *B, const void *C,
                                          const float *skip, const void *z, const float *bias,
                                          const float *state, void *out, float *next,
                                          cudaStream_t stream);
gdn_status launch_norm_gate_residual(const gdn_norm_problem &p, const void *y,
                                     const float *weight, const void *gate, const void *residual,
                                     const float *next_weight, void *out, void *next,
                                     cudaStream_t stream);

}  // namespace gdn

// token_common.cuh -- building blocks of the token operators (verify.cu,
// slots.cu, embed.cu, embed_grad.cu): element types, vector accesses and
// block-wide scans.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "drs_device.cuh"
#include "drs_internal.h"

namespace drs {

__host__ __device__ constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ------------------------------------------------------------- elements

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }

// Rounded to nearest even.
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// 16 bytes read once: not kept in L1.
__device__ __forceinline__ uint4 load16_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Eight consecutive elements as they lie in memory (16-byte aligned): one
// or two 16-byte words.
template <typename T> struct Raw8 {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
            w[i] = load16_stream(reinterpret_cast<const char*>(p) + 16 * i);
    }
    __device__ __forceinline__ void unpack(float (&v)[8]) const;
};
template <> __device__ __forceinline__ void Raw8<float>::unpack(float (&v)[8]) const {
    v[0] = __uint_as_float(w[0].x), v[1] = __uint_as_float(w[0].y);
    v[2] = __uint_as_float(w[0].z), v[3] = __uint_as_float(w[0].w);
    v[4] = __uint_as_float(w[1].x), v[5] = __uint_as_float(w[1].y);
    v[6] = __uint_as_float(w[1].z), v[7] = __uint_as_float(w[1].w);
}
template <> __device__ __forceinline__ void Raw8<__nv_bfloat16>::unpack(float (&v)[8]) const {
    const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // a bf16 is the upper half of its fp32
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}
template <> __device__ __forceinline__ void Raw8<__half>::unpack(float (&v)[8]) const {
    const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = *reinterpret_cast<const __half2*>(&u[i]);
        const float2 f = __half22float2(h);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// The 16 bytes that begin `shift` bytes into the 32 bytes of lo and hi.
__device__ __forceinline__ uint4 joined(uint4 lo, uint4 hi, int shift) {
    uint32_t w[5] = {lo.x, lo.y, lo.z, lo.w, hi.x};
    if (shift >= 8) w[0] = lo.z, w[1] = lo.w, w[2] = hi.x, w[3] = hi.y, w[4] = hi.z;
    if (shift & 4) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = w[4], w[4] = shift >= 8 ? hi.w : hi.y;
    const int bits = (shift & 3) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// Eight consecutive elements that start anywhere inside a 16-byte word: the
// words that hold them, and one more where they reach into it.
template <typename T> struct Raw8Shifted {
    uint4 w[sizeof(T) / 2 + 1];
    // first: the start of the word that holds the first element, `shift`
    // bytes before it
    __device__ __forceinline__ void load(const T* first, int shift) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
            w[i] = load16_stream(reinterpret_cast<const char*>(first) + 16 * i);
        w[sizeof(T) / 2] = make_uint4(0, 0, 0, 0);
        if (shift) w[sizeof(T) / 2] = load16_stream(reinterpret_cast<const char*>(first) + 8 * sizeof(T));
    }
    __device__ __forceinline__ void unpack(int shift, float (&v)[8]) const {
        Raw8<T> r;
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.w[i] = joined(w[i], w[i + 1], shift);
        r.unpack(v);
    }
};

// ------------------------------------------------------------- scans

template <typename T> __device__ __forceinline__ T warp_scan_inclusive(T v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

template <typename T> __device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ------------------------------------------------------------- pairs

// A number as the sum s + c of two fp32, |c| at most half a step of s
// (about 48 bits). fp64 would hold more, but this GPU issues one fp64
// instruction per SM in 16 cycles, and these take one cycle each.
struct Pair {
    float s, c;
};

// s + c == a + b exactly (Knuth's two-sum).
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = a + b;
    const float z = s - a;
    return Pair{s, (a - (s - z)) + (b - z)};
}

__device__ __forceinline__ Pair normalized(float s, float c) {
    const float h = s + c;
    return Pair{h, c - (h - s)};
}

__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    const Pair t = two_sum(a.s, b.s);
    return normalized(t.s, t.c + (a.c + b.c));
}

__device__ __forceinline__ Pair operator*(float u, Pair a) {
    const float h = u * a.s;
    return normalized(h, fmaf(u, a.s, -h) + u * a.c);
}

__device__ __forceinline__ Pair shfl_up(Pair v, int o) {
    return Pair{__shfl_up_sync(0xffffffffu, v.s, o), __shfl_up_sync(0xffffffffu, v.c, o)};
}

__device__ __forceinline__ Pair shfl(Pair v, int lane) {
    return Pair{__shfl_sync(0xffffffffu, v.s, lane), __shfl_sync(0xffffffffu, v.c, lane)};
}

// Two fp32 at once: one instruction per operation on both.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}

__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Two running sums of fp32 values: the errors of the additions add up in c.
struct PairSum2 {
    uint64_t s = 0, c = 0;
    __device__ __forceinline__ void add(uint64_t w) {
        const uint64_t t = add2(s, w);
        const uint64_t z = sub2(t, s);
        c = add2(c, add2(sub2(s, sub2(t, z)), sub2(w, z)));
        s = t;
    }
    __device__ __forceinline__ Pair value() const {
        float s0, s1, c0, c1;
        unpack2(s, s0, s1);
        unpack2(c, c0, c1);
        return normalized(s0, c0) + normalized(s1, c1);
    }
};

// Inclusive scan over the first n lanes (n a power of two).
__device__ __forceinline__ Pair warp_scan_pair(Pair v, int lane, int n = 32) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        if (o >= n) break;
        const Pair u = shfl_up(v, o);
        if (lane >= o) v = u + v;
    }
    return v;
}

__device__ __forceinline__ Pair warp_sum_pair(Pair v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = v + Pair{__shfl_xor_sync(0xffffffffu, v.s, o), __shfl_xor_sync(0xffffffffu, v.c, o)};
    return v;
}

// ------------------------------------------------------------- clusters

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same barrier in two halves, which all threads call: past the wait every
// CTA of the cluster has started. Only then may a CTA reach into the shared
// memory of another; the halves stand apart so that work of the CTA's own hides
// the barrier. Nothing written before the arrival is handed over.
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Store 8 bytes into the same shared-memory variable of CTA `rank` of the
// cluster, which has to have started (a cluster barrier before the first call).
__device__ __forceinline__ void store_remote(void* local, uint32_t rank, uint64_t v) {
    uint32_t addr;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// ------------------------------------------------------------- host side

inline bool dtype_ok(drs_dtype t) { return t == DRS_DTYPE_FP32 || t == DRS_DTYPE_BF16 || t == DRS_DTYPE_FP16; }
inline size_t dtype_bytes(drs_dtype t) { return t == DRS_DTYPE_FP32 ? 4 : 2; }

// f(T{}) for the element type that `t` names.
template <typename F> auto with_dtype(drs_dtype t, F f) {
    if (t == DRS_DTYPE_FP32) return f(float{});
    if (t == DRS_DTYPE_BF16) return f(__nv_bfloat16{});
    return f(__half{});
}

}  // namespace drs

// dropout.cu -- dropout from the counter-based generator and its gradient
// (drs_dropout, drs_dropout_grad): out = residual + keep * x / (1 - q).
//
// The mask is a function of (seed, global row, column): 16 bits of
// Philox4x32-10 per element, eight elements to a counter. It is never stored;
// the gradient computes it again.
#include <cmath>

#include "token_common.cuh"

namespace drs {
namespace {

constexpr int kDropoutThreads = 128;
// The counter's second word, which is 0 in the sampler's noise: the two draw
// different numbers from one seed.
constexpr uint32_t kDropoutTag = 0x64726F70u;

struct DropoutParams {
    const void* x;  // NULL: everything is dropped
    const void* residual;
    void* out;
    const uint64_t* device_seed;
    uint64_t seed;
    int64_t rows, x_stride, residual_stride, out_stride, row0;
    int32_t width, columns;  // columns: CTAs (or, for odd rows, groups of lanes) along a row
    uint32_t limit;          // of 2^32: 16-bit numbers below its upper half are dropped
    float scale;
};

__device__ __forceinline__ PhiloxKey dropout_key(const DropoutParams& a) {
    const uint64_t seed = a.device_seed ? *a.device_seed : a.seed;
    return PhiloxKey{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32)};
}

// The eight elements' 16-bit numbers, two to a word, the lower half first, for
// n rows in step: they share the rounds' keys.
template <int n> __device__ __forceinline__ void dropout_words(PhiloxKey key, const uint64_t (&row)[n], uint32_t group,
                                                               uint4 (&w)[n]) {
#pragma unroll
    for (int i = 0; i < n; ++i)
        w[i] = make_uint4(group, kDropoutTag, static_cast<uint32_t>(row[i]), static_cast<uint32_t>(row[i] >> 32));
#pragma unroll
    for (int round = 0; round < 10; ++round) {
#pragma unroll
        for (int i = 0; i < n; ++i) w[i] = philox_round(w[i], key);
        key = philox_next(key);
    }
}

// The bits of the kept among eight elements.
__device__ __forceinline__ uint32_t kept_bits(const uint4& w, uint32_t limit) {
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = word_of(w, i);
        bits |= (u << 16 >= limit ? 1u : 0u) << (2 * i) | (u >= limit ? 1u : 0u) << (2 * i + 1);
    }
    return bits;
}

// v = residual + kept ? v scale : 0, in fp32.
template <bool kResidual>
__device__ __forceinline__ void dropped(float (&v)[8], const float (&residual)[8], const uint4& w, uint32_t limit,
                                        float scale) {
    const uint64_t scale2 = pack2(scale, scale);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const uint32_t u = word_of(w, e / 2);
        float v0, v1;
        const uint64_t x = pack2(v[e], v[e + 1]);
        unpack2(kResidual ? fma2(x, scale2, pack2(residual[e], residual[e + 1])) : mul2(x, scale2), v0, v1);
        v[e] = u << 16 >= limit ? v0 : kResidual ? residual[e] : 0.0f;
        v[e + 1] = u >= limit ? v1 : kResidual ? residual[e + 1] : 0.0f;
    }
}

// Rows of all arrays that start on 16-byte boundaries, widths that are multiples of 8.
// A thread has eight columns of kRows rows.
template <typename X, typename Y, bool kResidual, int kRows>
__global__ void __launch_bounds__(kDropoutThreads) dropout_kernel(const DropoutParams a) {
    const int group = static_cast<int>(blockIdx.x % a.columns) * blockDim.x + threadIdx.x;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x / a.columns) * (blockDim.y * kRows) + threadIdx.y;
    if (group * 8 >= a.width) return;
    Raw8<X> x[kRows];
    Raw8<Y> residual[kResidual ? kRows : 1];
    uint64_t row[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = r0 + i * static_cast<int64_t>(blockDim.y);
        row[i] = static_cast<uint64_t>(a.row0 + r);
        x[i] = Raw8<X>{};
        if (r >= a.rows) continue;
        if (a.x) x[i].load(static_cast<const X*>(a.x) + r * a.x_stride + group * 8);
        if constexpr (kResidual)
            residual[i].load(static_cast<const Y*>(a.residual) + r * a.residual_stride + group * 8);
    }
    uint4 w[kRows];
    dropout_words(dropout_key(a), row, static_cast<uint32_t>(group), w);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = r0 + i * static_cast<int64_t>(blockDim.y);
        if (r >= a.rows) break;
        float v[8], add[8];
        x[i].unpack(v);
        if constexpr (kResidual) residual[i].unpack(add);
        dropped<kResidual>(v, add, w[i], a.limit, a.scale);
        store8_stream(static_cast<Y*>(a.out) + r * a.out_stride + group * 8, v);
    }
}

// Other rows. A lane has the mask of eight columns from a multiple of 8 on, and
// writes eight from a 16-byte boundary of its row of `out` on: these reach into the
// next lane's mask. A group of `lanes` lanes (a power of two, 8 to 32) has lanes - 1
// such units of a row; the one behind the last whole unit is written
// element by element, like the columns before the first.
template <typename X, typename Y, bool kResidual>
__global__ void __launch_bounds__(kDropoutThreads) dropout_odd_kernel(const DropoutParams a, int lanes) {
    constexpr int kRows = 2;
    const int lane = threadIdx.x & (lanes - 1);
    const int64_t line = static_cast<int64_t>(blockIdx.x) * (kDropoutThreads / lanes) + threadIdx.x / lanes;
    const int64_t r0 = line / a.columns * kRows;
    const int unit = static_cast<int>(line % a.columns) * (lanes - 1) + lane;
    const bool writes = lane < lanes - 1;
    Any8<X> x[kRows];
    Any8<Y> residual[kResidual ? kRows : 1];
    uint64_t row[kRows];
    int head[kRows], left[kRows];  // columns before the first unit; columns from this unit's first to the row's end
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = r0 + i;
        row[i] = static_cast<uint64_t>(a.row0 + r);
        const Y* const out = static_cast<const Y*>(a.out) + r * a.out_stride;
        head[i] = min(static_cast<int>((-reinterpret_cast<uintptr_t>(out) & 15) / sizeof(Y)), a.width);
        left[i] = r < a.rows && writes ? a.width - head[i] - unit * 8 : 0;
        if (left[i] < 8) continue;
        const int col = a.width - left[i];
        if (a.x) x[i].load(static_cast<const X*>(a.x) + r * a.x_stride, col, a.width);
        else x[i] = Any8<X>{};
        if constexpr (kResidual)
            residual[i].load(static_cast<const Y*>(a.residual) + r * a.residual_stride, col, a.width);
    }
    uint4 w[kRows];
    dropout_words(dropout_key(a), row, static_cast<uint32_t>(unit), w);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = r0 + i;
        uint32_t bits = kept_bits(w[i], a.limit);
        const uint32_t own = bits;
        bits = (bits | __shfl_down_sync(0xffffffffu, bits, 1, lanes) << 8) >> head[i];
        const X* const from = static_cast<const X*>(a.x) + r * a.x_stride;
        const Y* const add = static_cast<const Y*>(a.residual) + r * a.residual_stride;
        Y* const out = static_cast<Y*>(a.out) + r * a.out_stride;
        const auto one = [&](int j, bool kept) {
            const float rest = kResidual ? to_f(add[j]) : 0.0f;
            out[j] = from_f<Y>(kept && a.x ? fmaf(to_f(from[j]), a.scale, rest) : rest);
        };
        if (left[i] >= 8) {
            float v[8], rest[8];
            x[i].unpack(v);
            if constexpr (kResidual) residual[i].unpack(rest);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float base = kResidual ? rest[e] : 0.0f;
                v[e] = bits >> e & 1 ? (kResidual ? fmaf(v[e], a.scale, base) : v[e] * a.scale) : base;
            }
            store8_stream(out + (a.width - left[i]), v);
        } else {
            for (int e = 0; e < left[i]; ++e) one(a.width - left[i] + e, bits >> e & 1);
        }
        if (unit == 0 && r < a.rows)
            for (int j = 0; j < head[i]; ++j) one(j, own >> j & 1);
    }
}

template <typename X, typename Y, bool kResidual>
drs_status launch_dropout(DropoutParams a, bool vec, cudaStream_t stream) {
    if (vec) {
        constexpr int kRows = 4;
        const int groups = a.width / 8;
        a.columns = static_cast<int32_t>(ceil_div(groups, kDropoutThreads));
        int x = static_cast<int>(ceil_div(groups, a.columns));
        if (x > 32) x = (x + 31) / 32 * 32;
        const dim3 block(x, kDropoutThreads / x);
        const int64_t blocks = ceil_div(a.rows, block.y * kRows) * a.columns;
        if (blocks > INT32_MAX) return DRS_ERR_UNSUPPORTED;
        dropout_kernel<X, Y, kResidual, kRows><<<static_cast<unsigned>(blocks), block, 0, stream>>>(a);
    } else {
        const int units = a.width / 8 + 1;  // a partial one among them
        const int lanes = units < 8 ? 8 : units < 16 ? 16 : 32;
        a.columns = static_cast<int32_t>(ceil_div(units, lanes - 1));
        const int64_t blocks = ceil_div(ceil_div(a.rows, 2) * a.columns, kDropoutThreads / lanes);
        if (blocks > INT32_MAX) return DRS_ERR_UNSUPPORTED;
        dropout_odd_kernel<X, Y, kResidual><<<static_cast<unsigned>(blocks), kDropoutThreads, 0, stream>>>(a, lanes);
    }
    return cuda_status(cudaGetLastError());
}

drs_status dropout(const void* x, drs_dtype dtype, int64_t rows, int64_t width, int64_t x_stride,
                   const void* residual, int64_t residual_stride, float p, uint64_t seed,
                   const uint64_t* device_seed, int64_t row0, void* out, drs_dtype out_dtype, int64_t out_stride,
                   cudaStream_t stream) {
    if (rows < 0 || width < 1 || row0 < 0 || row0 > INT64_MAX - rows || !dtype_ok(dtype) || !dtype_ok(out_dtype))
        return DRS_ERR_INVALID_ARG;
    if (!(p >= 0.0f && p <= 1.0f) || x_stride < width || out_stride < width || (residual && residual_stride < width))
        return DRS_ERR_INVALID_ARG;
    if (width > DRS_MAX_WIDTH || rows > int64_t{1} << 40) return DRS_ERR_UNSUPPORTED;
    if (rows == 0) return DRS_OK;
    if (!x || !out || !aligned(x, dtype_bytes(dtype)) || !aligned(out, dtype_bytes(out_dtype)) ||
        !aligned(residual, dtype_bytes(out_dtype)) || !aligned(device_seed, 8))
        return DRS_ERR_INVALID_ARG;
    if ((out == x && (dtype != out_dtype || x_stride != out_stride)) || (out == residual && residual_stride != out_stride))
        return DRS_ERR_INVALID_ARG;
    DropoutParams a{};
    a.x = x;
    a.residual = residual;
    a.out = out;
    a.device_seed = device_seed;
    a.seed = seed;
    a.rows = rows;
    a.x_stride = x_stride;
    a.residual_stride = residual_stride;
    a.out_stride = out_stride;
    a.row0 = row0;
    a.width = static_cast<int32_t>(width);
    const uint32_t dropped = static_cast<uint32_t>(std::floor(static_cast<double>(p) * 65536.0 + 0.5));
    if (dropped == 65536) a.x = nullptr;
    a.limit = dropped << 16;
    a.scale = dropped < 65536 ? static_cast<float>(65536.0 / (65536.0 - dropped)) : 0.0f;
    const auto on_boundaries = [&](const void* q, int64_t stride, drs_dtype t) {
        return aligned(q, 16) && stride * dtype_bytes(t) % 16 == 0;
    };
    const bool vec = width % 8 == 0 && on_boundaries(x, x_stride, dtype) && on_boundaries(out, out_stride, out_dtype) &&
                     (!residual || on_boundaries(residual, residual_stride, out_dtype));
    return with_dtype(dtype, [&](auto t) -> drs_status {
        return with_dtype(out_dtype, [&](auto o) -> drs_status {
            using X = decltype(t);
            using Y = decltype(o);
            return residual ? launch_dropout<X, Y, true>(a, vec, stream) : launch_dropout<X, Y, false>(a, vec, stream);
        });
    });
}

}  // namespace
}  // namespace drs

extern "C" drs_status drs_dropout(const void* x, drs_dtype dtype, int64_t rows, int64_t width, int64_t x_stride,
                                  const void* residual, int64_t residual_stride, float p, uint64_t seed,
                                  const uint64_t* device_seed, int64_t row0, void* out, drs_dtype out_dtype,
                                  int64_t out_stride, void* stream) {
    return drs::dropout(x, dtype, rows, width, x_stride, residual, residual_stride, p, seed, device_seed, row0, out,
                        out_dtype, out_stride, static_cast<cudaStream_t>(stream));
}

extern "C" drs_status drs_dropout_grad(const void* grad_out, drs_dtype grad_dtype, int64_t rows, int64_t width,
                                       int64_t grad_stride, float p, uint64_t seed, const uint64_t* device_seed,
                                       int64_t row0, void* grad_x, drs_dtype x_dtype, int64_t x_stride, void* stream) {
    return drs::dropout(grad_out, grad_dtype, rows, width, grad_stride, nullptr, 0, p, seed, device_seed, row0, grad_x,
                        x_dtype, x_stride, static_cast<cudaStream_t>(stream));
}

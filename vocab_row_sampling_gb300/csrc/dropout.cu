// dropout.cu -- dropout from the counter-based generator and its gradient
// (drs_dropout, drs_dropout_grad): out = residual + keep * x / (1 - q).
//
// The mask is a function of (seed, global row, column): 16 bits of
// Philox4x32-10 per element, eight elements to a counter. It is never stored;
// the gradient computes it again. 32 bits per element would take twice the
// rounds: about 15 integer instructions per element, which at 4 bytes moved per element
// is all that the SMs issue at the memory's rate; 16 bits leave q at multiples of
// 2^-16, and the scale is that of the rounded q.
//
// Bound by memory: x and the residual are read once, out is written once. Measured:
// 65536 x 4096 bf16 with a residual 224 us, 7.2 TB/s; 32768 x 4096 bf16 79 us, 6.8
// TB/s; 256 x 2048 2.1 us, the launch. Rows off 16-byte boundaries issue about
// 25 instructions per column and are bound by them: 30000 x 4095 122 us, 6.1 TB/s.
#include <cmath>
#include <type_traits>

#include "token_common.cuh"

namespace drs {
namespace {

constexpr int kDropoutThreads = 128;  // 65536 x 4096: 223 us with 64, 224 with 128, 223 with 256
// The counter's second word, which is 0 in the sampler's noise: the two draw
// different numbers from one seed.
constexpr uint32_t kDropoutTag = 0x64726F70u;

struct DropoutParams {
    const void* x;
    const void* residual;
    void* out;
    const uint64_t* device_seed;
    uint64_t seed;
    int64_t rows, x_stride, residual_stride, out_stride, row0;
    int32_t width, columns;  // columns: CTAs along a row
    uint32_t limit;          // of 2^32: 16-bit numbers below its upper half are dropped
    float scale;
};

__device__ __forceinline__ PhiloxKey dropout_key(const DropoutParams& a) {
    const uint64_t seed = a.device_seed ? *a.device_seed : a.seed;
    return PhiloxKey{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32)};
}

// The eight elements' 16-bit numbers, two to a word, the lower half first, for
// n counters in step: philox4x32_10 of each, whose rounds' keys they share.
template <int n>
__device__ __forceinline__ void dropout_words(PhiloxKey key, const uint64_t (&row)[n], const uint32_t (&group)[n], uint4 (&w)[n]) {
    constexpr uint32_t kMulA = 0xD2511F53u, kMulB = 0xCD9E8D57u;
    constexpr uint32_t kWeylA = 0x9E3779B9u, kWeylB = 0xBB67AE85u;
#pragma unroll
    for (int i = 0; i < n; ++i)
        w[i] = make_uint4(group[i], kDropoutTag, static_cast<uint32_t>(row[i]), static_cast<uint32_t>(row[i] >> 32));
#pragma unroll
    for (int round = 0; round < 10; ++round) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint64_t a = static_cast<uint64_t>(kMulA) * w[i].x, b = static_cast<uint64_t>(kMulB) * w[i].z;
            w[i] = make_uint4(static_cast<uint32_t>(b >> 32) ^ w[i].y ^ key.k0, static_cast<uint32_t>(b),
                              static_cast<uint32_t>(a >> 32) ^ w[i].w ^ key.k1, static_cast<uint32_t>(a));
        }
        key.k0 += kWeylA;
        key.k1 += kWeylB;
    }
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
    uint32_t groups[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = r0 + i * static_cast<int64_t>(blockDim.y);
        groups[i] = static_cast<uint32_t>(group);
        row[i] = static_cast<uint64_t>(a.row0 + r);
        if (r >= a.rows) continue;
        x[i].template load<true>(static_cast<const X*>(a.x) + r * a.x_stride + group * 8);
        if constexpr (kResidual)
            residual[i].template load<true>(static_cast<const Y*>(a.residual) + r * a.residual_stride + group * 8);
    }
    uint4 w[kRows];
    dropout_words(dropout_key(a), row, groups, w);
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

// The sixteen numbers from the head-th of those of a, b and c on, into a and b.
__device__ __forceinline__ void shift_numbers(uint4& a, uint4& b, const uint4& c, int head) {
    uint32_t w[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
    if (head & 4) {
#pragma unroll
        for (int i = 0; i < 10; ++i) w[i] = w[i + 2];
    }
    if (head & 2) {
#pragma unroll
        for (int i = 0; i < 9; ++i) w[i] = w[i + 1];
    }
    const int bits = (head & 1) * 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
}

// Where units of eight columns of `out` begin: on 16-byte boundaries, fp32 ones on 32-byte ones, so that
// a lane writes whole sectors.
template <typename Y> constexpr int kBoundary = sizeof(Y) == 4 ? 32 : 16;

// Columns before the first boundary of a row of `out`: at most 7.
template <typename Y> __device__ __forceinline__ int columns_before(const Y* out, int width) {
    return min(static_cast<int>((-reinterpret_cast<uintptr_t>(out) & (kBoundary<Y> - 1)) / sizeof(Y)), width);
}

// Other rows. A lane has the numbers of sixteen columns from a multiple of 16
// on, and writes sixteen from a 16-byte boundary of its row of `out` on, as two
// eights: their numbers are put together from its own and the next lane's. A
// group of `lanes` lanes (a power of two, 8 to 32) has lanes - 1 such units of a
// row. The columns before the first unit and behind the last whole eight, 14 at
// most, are written one by one by CTAs of their own behind the others.
// kAlike: the rows of all arrays lie alike within 16-byte words (such as
// contiguous ones of one type and odd width), so that a word of one meets a word
// of each other; else the words of x and residual are put together.
template <typename X, typename Y, bool kResidual, bool kAlike>
__global__ void __launch_bounds__(kDropoutThreads) dropout_odd_kernel(const DropoutParams a, int lanes, unsigned unit_blocks) {
    if (blockIdx.x >= unit_blocks) {
        const int64_t r = static_cast<int64_t>(blockIdx.x - unit_blocks) * (kDropoutThreads / 16) + threadIdx.x / 16;
        if (r >= a.rows) return;
        const int e = threadIdx.x % 16;
        Y* const out = static_cast<Y*>(a.out) + r * a.out_stride;
        const int head = columns_before(out, a.width), tail = head + (a.width - head) / 8 * 8;
        const int col = e < 8 ? e : tail + e - 8;
        if (e < 8 ? e >= head : col >= a.width) return;
        const float x = to_f((static_cast<const X*>(a.x) + r * a.x_stride)[col]);
        const float base = kResidual ? to_f((static_cast<const Y*>(a.residual) + r * a.residual_stride)[col]) : 0.0f;
        const uint64_t row[1] = {static_cast<uint64_t>(a.row0 + r)};
        const uint32_t group[1] = {static_cast<uint32_t>(col / 8)};
        uint4 w[1];
        dropout_words(dropout_key(a), row, group, w);
        const uint32_t u = word_of(w[0], col % 8 / 2);
        out[col] = from_f<Y>((col % 2 ? u : u << 16) >= a.limit ? fmaf(x, a.scale, base) : base);
        return;
    }
    const int lane = threadIdx.x & (lanes - 1);
    const int64_t r = static_cast<int64_t>(blockIdx.x / a.columns) * (kDropoutThreads / lanes) + threadIdx.x / lanes;
    const int unit = static_cast<int>(blockIdx.x % a.columns) * (lanes - 1) + lane;
    Y* const out = static_cast<Y*>(a.out) + r * a.out_stride;
    const int head = columns_before(out, a.width), col = head + unit * 16;
    const bool writes = r < a.rows && lane < lanes - 1;
    using Words = std::conditional_t<kAlike, Raw8<X>, Any8<X>>;
    using ResidualWords = std::conditional_t<kAlike, Raw8<Y>, Any8<Y>>;
    Words x[2];
    ResidualWords residual[kResidual ? 2 : 1];
    const X* const from = static_cast<const X*>(a.x) + r * a.x_stride;
    const Y* const rest = static_cast<const Y*>(a.residual) + r * a.residual_stride;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (!writes || col + 8 * h + 8 > a.width) continue;
        if constexpr (kAlike) {
            x[h].template load<true>(from + (col + 8 * h));
            if constexpr (kResidual) residual[h].template load<true>(rest + (col + 8 * h));
        } else {
            x[h].template load<true>(from, col + 8 * h, a.width);
            if constexpr (kResidual) residual[h].template load<true>(rest, col + 8 * h, a.width);
        }
    }
    const uint64_t row[2] = {static_cast<uint64_t>(a.row0 + r), static_cast<uint64_t>(a.row0 + r)};
    const uint32_t group[2] = {static_cast<uint32_t>(2 * unit), static_cast<uint32_t>(2 * unit + 1)};
    uint4 w[2];
    dropout_words(dropout_key(a), row, group, w);
    const uint4 next = make_uint4(__shfl_down_sync(0xffffffffu, w[0].x, 1, lanes), __shfl_down_sync(0xffffffffu, w[0].y, 1, lanes),
                                  __shfl_down_sync(0xffffffffu, w[0].z, 1, lanes), __shfl_down_sync(0xffffffffu, w[0].w, 1, lanes));
    shift_numbers(w[0], w[1], next, head);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (!writes || col + 8 * h + 8 > a.width) continue;
        float v[8], add[8];
        x[h].unpack(v);
        if constexpr (kResidual) residual[h].unpack(add);
        dropped<kResidual>(v, add, w[h], a.limit, a.scale);
        store8_stream(out + col + 8 * h, v);
    }
}

template <typename X, typename Y, bool kResidual, int kRows> drs_status launch_rows(DropoutParams a, cudaStream_t stream) {
    const int groups = a.width / 8;
    a.columns = static_cast<int32_t>(ceil_div(groups, kDropoutThreads));
    int x = static_cast<int>(ceil_div(groups, a.columns));
    if (x > 32) x = (x + 31) / 32 * 32;
    const dim3 block(x, kDropoutThreads / x);
    const int64_t blocks = ceil_div(a.rows, block.y * kRows) * a.columns;
    if (blocks > INT32_MAX) return DRS_ERR_UNSUPPORTED;
    dropout_kernel<X, Y, kResidual, kRows><<<static_cast<unsigned>(blocks), block, 0, stream>>>(a);
    return cuda_status(cudaGetLastError());
}

template <typename X, typename Y, bool kResidual>
drs_status launch_dropout(DropoutParams a, bool vec, cudaStream_t stream) {
    if (vec) {
        // us with two and four rows per thread (bf16): 256 x 2048 2.1, 2.3; 1000 x 1024 2.5, 2.7; 2048 x 1024 4.0, 4.0;
        // 32768 x 4096 84.2, 79.7.
        const bool many = a.rows * (a.width / 8) > int64_t{1} << 18;
        return many ? launch_rows<X, Y, kResidual, 4>(a, stream) : launch_rows<X, Y, kResidual, 2>(a, stream);
    }
    const int units = (a.width / 8 + 1) / 2;
    const int lanes = units < 8 ? 8 : units < 16 ? 16 : 32;
    a.columns = static_cast<int32_t>(ceil_div(units, lanes - 1));
    const int64_t unit_blocks = ceil_div(a.rows, kDropoutThreads / lanes) * a.columns;
    const int64_t blocks = unit_blocks + ceil_div(a.rows, kDropoutThreads / 16);
    if (blocks > INT32_MAX) return DRS_ERR_UNSUPPORTED;
    // us for 30000 x 4095 and 5003 x 1283 16-bit elements with a residual: 122 and 9.3 where the arrays lie alike, 148
    // and 10.7 by the words put together.
    auto kernel = dropout_odd_kernel<X, Y, kResidual, false>;
    if constexpr (std::is_same_v<X, Y>) {
        const auto alike = [&](const void* p, int64_t stride) {
            return (reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(a.out)) % 16 == 0 &&
                   (stride - a.out_stride) * static_cast<int64_t>(sizeof(Y)) % 16 == 0;
        };
        if (alike(a.x, a.x_stride) && (!kResidual || alike(a.residual, a.residual_stride)))
            kernel = dropout_odd_kernel<X, Y, kResidual, true>;
    }
    kernel<<<static_cast<unsigned>(blocks), kDropoutThreads, 0, stream>>>(a, lanes, static_cast<unsigned>(unit_blocks));
    return cuda_status(cudaGetLastError());
}

// Zeros in `rows` rows of `bytes` bytes. The runtime's pitched calls take pitches up to 2^31 - 1; an array of
// wider ones has few rows.
drs_status clear_rows(void* out, int64_t pitch, int64_t bytes, int64_t rows, cudaStream_t stream) {
    if (rows == 1 || pitch == bytes) return cuda_status(cudaMemsetAsync(out, 0, static_cast<size_t>(rows * bytes), stream));
    if (pitch <= INT32_MAX)
        return cuda_status(cudaMemset2DAsync(out, static_cast<size_t>(pitch), 0, static_cast<size_t>(bytes),
                                             static_cast<size_t>(rows), stream));
    for (int64_t r = 0; r < rows; ++r) {
        const drs_status st =
            cuda_status(cudaMemsetAsync(static_cast<char*>(out) + r * pitch, 0, static_cast<size_t>(bytes), stream));
        if (st != DRS_OK) return st;
    }
    return DRS_OK;
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
    if (dropped == 65536) {  // nothing of x is left
        if (!residual) return clear_rows(out, out_stride * dtype_bytes(out_dtype), width * dtype_bytes(out_dtype), rows, stream);
        return dropout(residual, out_dtype, rows, width, residual_stride, nullptr, 0, 0.0f, seed, device_seed, row0, out,
                       out_dtype, out_stride, stream);
    }
    a.limit = dropped << 16;
    a.scale = static_cast<float>(65536.0 / (65536.0 - dropped));
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

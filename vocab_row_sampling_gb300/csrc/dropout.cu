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

constexpr int kDropoutThreads = 256;
// The counter's second word, which is 0 in the sampler's noise: the two draw
// different numbers from one seed.
constexpr uint32_t kDropoutTag = 0x64726F70u;

struct DropoutParams {
    const void* x;
    const void* residual;
    void* out;
    const uint64_t* device_seed;
    uint64_t seed;
    int64_t rows, x_stride, residual_stride, out_stride, row0, groups;  // groups of 8 columns per row
    int32_t width;
    uint32_t dropped;  // of 65536
    float scale;
};

// The eight elements' 16 bits, two to a word, lower half first.
__device__ __forceinline__ uint4 dropout_words(PhiloxKey key, uint64_t row, uint32_t group) {
    return philox4x32_10(
        make_uint4(group, kDropoutTag, static_cast<uint32_t>(row), static_cast<uint32_t>(row >> 32)), key);
}

template <typename X, typename Y> __global__ void __launch_bounds__(kDropoutThreads) dropout_kernel(const DropoutParams a) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kDropoutThreads + threadIdx.x;
    const int64_t row = at / a.groups;
    const int group = static_cast<int>(at % a.groups);
    if (row >= a.rows) return;
    const uint64_t seed = a.device_seed ? *a.device_seed : a.seed;
    const uint4 w = dropout_words(PhiloxKey{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32)},
                                  static_cast<uint64_t>(a.row0 + row), static_cast<uint32_t>(group));
    const X* const x = static_cast<const X*>(a.x) + row * a.x_stride;
    const Y* const residual = static_cast<const Y*>(a.residual) + row * a.residual_stride;
    Y* const out = static_cast<Y*>(a.out) + row * a.out_stride;
    for (int e = 0; e < 8; ++e) {
        const int j = group * 8 + e;
        if (j >= a.width) break;
        const uint32_t half = word_of(w, e / 2) >> (16 * (e % 2)) & 0xFFFFu;
        float v = half >= a.dropped ? to_f(x[j]) * a.scale : 0.0f;
        if (a.residual) v += to_f(residual[j]);
        out[j] = from_f<Y>(v);
    }
}

drs_status dropout(const void* x, drs_dtype dtype, int64_t rows, int64_t width, int64_t x_stride,
                   const void* residual, int64_t residual_stride, float p, uint64_t seed,
                   const uint64_t* device_seed, int64_t row0, void* out, drs_dtype out_dtype, int64_t out_stride,
                   cudaStream_t stream) {
    if (rows < 0 || width < 1 || row0 < 0 || row0 > INT64_MAX - rows || !dtype_ok(dtype) || !dtype_ok(out_dtype))
        return DRS_ERR_INVALID_ARG;
    if (!(p >= 0.0f && p <= 1.0f) || x_stride < width || out_stride < width || (residual && residual_stride < width))
        return DRS_ERR_INVALID_ARG;
    if (width > DRS_MAX_WIDTH) return DRS_ERR_UNSUPPORTED;
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
    a.groups = ceil_div(width, 8);
    a.width = static_cast<int32_t>(width);
    a.dropped = static_cast<uint32_t>(std::floor(static_cast<double>(p) * 65536.0 + 0.5));
    a.scale = a.dropped < 65536 ? static_cast<float>(65536.0 / (65536.0 - a.dropped)) : 0.0f;
    if (rows > int64_t{INT32_MAX} * kDropoutThreads / a.groups) return DRS_ERR_UNSUPPORTED;
    const unsigned blocks = static_cast<unsigned>(ceil_div(rows * a.groups, kDropoutThreads));
    return with_dtype(dtype, [&](auto t) -> drs_status {
        return with_dtype(out_dtype, [&](auto o) -> drs_status {
            dropout_kernel<decltype(t), decltype(o)><<<blocks, kDropoutThreads, 0, stream>>>(a);
            return cuda_status(cudaGetLastError());
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

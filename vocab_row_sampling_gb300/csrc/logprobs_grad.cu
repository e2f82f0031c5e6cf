// logprobs_grad.cu -- the gradient of token logprobs and entropies with
// respect to the logits (drs_token_logprobs_grad).
//
// With p_j = e^((x_j - m) / T - L) from the forward call's (m, L), the
// entropy H, and the arriving gradients g of the logprob and h of the entropy:
//   dx_j = (1 / T) (g ([j == id] - p_j) - h p_j (ln p_j + H)).
//
// Bound by memory: the logits are read once and the gradient is written once,
// nothing in between is kept; about ten instructions per column beside them. p
// comes from the stored norm, so that no row has to be summed up again. Measured: 4096 x
// 262144 bf16 598 us, 7.1 TB/s; 777 x 50001 bf16 into fp32 (rows off 16-byte
// boundaries, with the entropy's part) 38 us, 6.1 TB/s; 128 x 8192 2.9 us, the launch.
#include "token_common.cuh"

namespace drs {
namespace {

constexpr int kGradThreads = 128;
// Units of eight columns per thread where rows are off 16-byte boundaries. us for 777 x 50001 bf16 into fp32 with 1,
// 2, 3 and 4 units: 39.7, 38.8, 48.2, 43.0; into bf16 36.3, 29.2, 35.2, 31.5.
constexpr int kOddUnits = 2;
constexpr float kLeastExponent = -200.0f;  // 2^-200 is 0 in fp32; -inf would give 0 times infinity

struct LogprobGradParams {
    const void* logits;
    const void* ids;
    const float* temps;
    const float* norm;
    const float* entropy;
    const float* grad_logprob;
    const float* grad_entropy;
    void* grad;
    int64_t row_stride, grad_stride, canvas_len;
    int32_t vocab, id_bits, chunks;  // chunks: CTAs along a row
};

// What a row's columns have in common. With l = log2 p_j:
//   dx_j = 2^l (a0 + a1 l), and g (1 - p) / T more in the token's column.
struct RowTerms {
    float top, scale, shift, a0, a1;
    float inverse, log_sum, g, h, entropy;
    int id;
    bool none;  // passed over, or without a distribution: zeros

    __device__ RowTerms(const LogprobGradParams& a, int64_t row) {
        const int64_t token =
            a.id_bits == 64 ? static_cast<const int64_t*>(a.ids)[row] : static_cast<const int32_t*>(a.ids)[row];
        top = a.norm[2 * row];
        log_sum = a.norm[2 * row + 1];
        none = token < 0 || token >= a.vocab || log_sum == -INFINITY;
        id = none ? -1 : static_cast<int>(token);
        inverse = a.temps ? 1.0f / fmaxf(a.temps[row / a.canvas_len], kTempFloor) : 1.0f;
        g = a.grad_logprob ? a.grad_logprob[row] : 0.0f;
        h = a.grad_entropy ? a.grad_entropy[row] : 0.0f;
        entropy = a.grad_entropy ? a.entropy[row] : 0.0f;
        scale = inverse * kLog2e;
        shift = log_sum * kLog2e;
        a0 = -(g + h * entropy) * inverse;
        a1 = -h * kLn2 * inverse;
    }

    // The token's column: g (1 - p) without the difference's cancellation.
    __device__ float own(float v) const {
        const float lp = (v - top) * inverse - log_sum;
        const float p = ex2_approx(max_nan((v - top) * scale - shift, kLeastExponent));
        return (h == 0.0f ? 0.0f : -h * p * (max_nan(lp, kLeastExponent) + entropy) * inverse) - g * expm1f(lp) * inverse;
    }

    __device__ float one(float v, int col) const {
        if (none) return 0.0f;
        if (col == id) return own(v);
        const float l = max_nan((v - top) * scale - shift, kLeastExponent);
        return ex2_approx(l) * fmaf(a1, l, a0);
    }

    // Columns col .. col+7.
    __device__ __forceinline__ void eight(float (&v)[8], int col) const {
        if (none) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.0f;
            return;
        }
        const bool here = static_cast<uint32_t>(id - col) < 8u;
        float at = 0.0f;
        if (here) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col + e == id) at = own(v[e]);
        }
        const uint64_t top2 = pack2(top, top), scale2 = pack2(scale, scale), shift2 = pack2(shift, shift);
        const uint64_t a02 = pack2(a0, a0), a12 = pack2(a1, a1);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            float l0, l1;
            unpack2(sub2(mul2(sub2(pack2(v[e], v[e + 1]), top2), scale2), shift2), l0, l1);
            l0 = max_nan(l0, kLeastExponent);
            l1 = max_nan(l1, kLeastExponent);
            unpack2(mul2(pack2(ex2_approx(l0), ex2_approx(l1)), fma2(a12, pack2(l0, l1), a02)), v[e], v[e + 1]);
        }
        if (here) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col + e == id) v[e] = at;
        }
    }
};

// Rows of both arrays that start on 16-byte boundaries. A thread has kUnits units
// of eight columns.
template <typename T, typename G, int kUnits>
__global__ void __launch_bounds__(kGradThreads) logprob_grad_kernel(const LogprobGradParams a) {
    const int64_t row = blockIdx.x / a.chunks;
    const int first = static_cast<int>(blockIdx.x % a.chunks) * (kGradThreads * kUnits * 8) + threadIdx.x * 8;
    const T* const x = static_cast<const T*>(a.logits) + row * a.row_stride;
    G* const out = static_cast<G*>(a.grad) + row * a.grad_stride;
    Raw8<T> raw[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int col = first + u * kGradThreads * 8;
        if (col + 8 <= a.vocab) raw[u].template load<true>(x + col);
    }
    const RowTerms terms(a, row);
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int col = first + u * kGradThreads * 8;
        if (col + 8 <= a.vocab) {
            float v[8];
            raw[u].unpack(v);
            terms.eight(v, col);
            store8_stream(out + col, v);
        } else {
            for (int j = col; j < a.vocab; ++j) out[j] = from_f<G>(terms.one(to_f(x[j]), j));
        }
    }
}

// Other rows: units of eight columns from a boundary of the gradient's row on,
// the logits of each put together from the words that hold them, and the
// columns before and after one by one.
template <typename T, typename G>
__global__ void __launch_bounds__(kGradThreads) logprob_grad_odd_kernel(const LogprobGradParams a) {
    const int64_t row = blockIdx.x / a.chunks;
    const int chunk = static_cast<int>(blockIdx.x % a.chunks);
    const T* const x = static_cast<const T*>(a.logits) + row * a.row_stride;
    G* const out = static_cast<G*>(a.grad) + row * a.grad_stride;
    constexpr int kBoundary = sizeof(G) == 4 ? 32 : 16;
    const int head = min(static_cast<int>((-reinterpret_cast<uintptr_t>(out) & (kBoundary - 1)) / sizeof(G)), a.vocab);
    const int tail = head + (a.vocab - head) / 8 * 8;  // the first column behind the units
    const int first = head + chunk * (kGradThreads * kOddUnits * 8) + threadIdx.x * 8;
    Any8<T> raw[kOddUnits];
#pragma unroll
    for (int u = 0; u < kOddUnits; ++u) {
        const int col = first + u * kGradThreads * 8;
        if (col < tail) raw[u].template load<true>(x, col, a.vocab);
    }
    const RowTerms terms(a, row);
#pragma unroll
    for (int u = 0; u < kOddUnits; ++u) {
        const int col = first + u * kGradThreads * 8;
        if (col >= tail) break;
        float v[8];
        raw[u].unpack(v);
        terms.eight(v, col);
        store8_stream(out + col, v);
    }
    if (chunk == 0 && threadIdx.x < head + a.vocab - tail) {
        const int j = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
        out[j] = from_f<G>(terms.one(to_f(x[j]), j));
    }
}

}  // namespace
}  // namespace drs

extern "C" drs_status drs_token_logprobs_grad(const void* logits, drs_dtype dtype, int64_t rows, int64_t vocab,
                                              int64_t row_stride, const void* ids, int32_t id_bits,
                                              const float* temps, int64_t canvas_len, const float* norm,
                                              const float* entropy, const float* grad_logprob,
                                              const float* grad_entropy, void* grad, drs_dtype grad_dtype,
                                              int64_t grad_stride, void* stream) {
    using namespace drs;
    if (rows < 0 || vocab < 1 || !dtype_ok(dtype) || !dtype_ok(grad_dtype) || (id_bits != 32 && id_bits != 64))
        return DRS_ERR_INVALID_ARG;
    if (row_stride < vocab || grad_stride < vocab || canvas_len < 1) return DRS_ERR_INVALID_ARG;
    if (vocab > DRS_MAX_VOCAB || rows > DRS_MAX_SCORE_ROWS) return DRS_ERR_UNSUPPORTED;
    if (rows == 0) return DRS_OK;
    if (!logits || !ids || !norm || !grad || (!grad_logprob && !grad_entropy) || (grad_entropy && !entropy))
        return DRS_ERR_INVALID_ARG;
    if (!aligned(logits, dtype_bytes(dtype)) || !aligned(grad, dtype_bytes(grad_dtype)) ||
        !aligned(ids, id_bits / 8) || !aligned(temps, 4) || !aligned(norm, 4) || !aligned(entropy, 4) ||
        !aligned(grad_logprob, 4) || !aligned(grad_entropy, 4))
        return DRS_ERR_INVALID_ARG;
    if (grad == logits && (grad_dtype != dtype || grad_stride != row_stride)) return DRS_ERR_INVALID_ARG;
    LogprobGradParams a{};
    a.logits = logits;
    a.ids = ids;
    a.temps = temps;
    a.norm = norm;
    a.entropy = entropy;
    a.grad_logprob = grad_logprob;
    a.grad_entropy = grad_entropy;
    a.grad = grad;
    a.row_stride = row_stride;
    a.grad_stride = grad_stride;
    a.canvas_len = canvas_len;
    a.vocab = static_cast<int32_t>(vocab);
    a.id_bits = id_bits;
    const bool vec = aligned(logits, 16) && aligned(grad, 16) && row_stride * dtype_bytes(dtype) % 16 == 0 &&
                     grad_stride * dtype_bytes(grad_dtype) % 16 == 0;
    return with_dtype(dtype, [&](auto t) -> drs_status {
        return with_dtype(grad_dtype, [&](auto o) -> drs_status {
            using T = decltype(t);
            using G = decltype(o);
            // us with two and four units: 4096 x 262144 bf16 666, 603; 777 x 50048 bf16 27.6, 25.8; 128 x 8192 bf16
            // 2.9, 3.3; 777 x 50048 into fp32 36.5, 38.2.
            const bool four = sizeof(T) == 2 && sizeof(G) == 2 && rows * vocab > int64_t{1} << 22;
            const int units = !vec ? kOddUnits : four ? 4 : 2;
            a.chunks = static_cast<int32_t>(ceil_div(vocab, kGradThreads * 8 * units));
            if (rows > INT32_MAX / a.chunks) return DRS_ERR_UNSUPPORTED;
            const auto kernel = !vec ? logprob_grad_odd_kernel<T, G> : four ? logprob_grad_kernel<T, G, 4> : logprob_grad_kernel<T, G, 2>;
            kernel<<<static_cast<unsigned>(rows * a.chunks), kGradThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
            return cuda_status(cudaGetLastError());
        });
    });
}

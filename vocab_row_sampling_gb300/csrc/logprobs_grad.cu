// logprobs_grad.cu -- the gradient of token logprobs and entropies with
// respect to the logits (drs_token_logprobs_grad).
//
// With p_j = e^((x_j - m) / T - L) from the forward call's (m, L), the
// entropy H, and the arriving gradients g of the logprob and h of the entropy:
//   dx_j = (1 / T) (g ([j == id] - p_j) - h p_j (ln p_j + H)).
#include "token_common.cuh"

namespace drs {
namespace {

constexpr int kGradThreads = 256;
constexpr float kLeastExponent = -200.0f;  // 2^-200 is 0 in fp32

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
    int32_t vocab;
};

template <typename T, typename G, typename I>
__global__ void __launch_bounds__(kGradThreads) logprob_grad_kernel(const LogprobGradParams a) {
    const int64_t row = blockIdx.x;
    const T* const x = static_cast<const T*>(a.logits) + row * a.row_stride;
    G* const out = static_cast<G*>(a.grad) + row * a.grad_stride;
    const int64_t id = static_cast<int64_t>(static_cast<const I*>(a.ids)[row]);
    const float top = a.norm[2 * row], log_sum = a.norm[2 * row + 1];
    if (id < 0 || id >= a.vocab || top == -INFINITY) {
        for (int j = threadIdx.x; j < a.vocab; j += kGradThreads) out[j] = from_f<G>(0.0f);
        return;
    }
    const float inverse = a.temps ? 1.0f / fmaxf(a.temps[row / a.canvas_len], kTempFloor) : 1.0f;
    const float g = a.grad_logprob ? a.grad_logprob[row] : 0.0f, h = a.grad_entropy ? a.grad_entropy[row] : 0.0f;
    const float entropy = a.grad_entropy ? a.entropy[row] : 0.0f;
    const float scale = inverse * kLog2e, shift = log_sum * kLog2e;
    const float a0 = -(g + h * entropy) * inverse, a1 = -h * kLn2 * inverse;
    for (int j = threadIdx.x; j < a.vocab; j += kGradThreads) {
        const float v = to_f(x[j]);
        const float l = fmaxf((v - top) * scale - shift, kLeastExponent);
        float d = ex2_approx(l) * fmaf(a1, l, a0);
        if (j == id) {  // g (1 - p) without the difference's cancellation
            const float lp = (v - top) * inverse - log_sum;
            d = (h == 0.0f ? 0.0f : -h * ex2_approx(l) * (fmaxf(lp, kLeastExponent) + entropy) * inverse) -
                g * expm1f(lp) * inverse;
        }
        out[j] = from_f<G>(d);
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
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return with_dtype(dtype, [&](auto t) -> drs_status {
        return with_dtype(grad_dtype, [&](auto o) -> drs_status {
            using T = decltype(t);
            using G = decltype(o);
            const unsigned grid = static_cast<unsigned>(rows);
            if (id_bits == 32) logprob_grad_kernel<T, G, int32_t><<<grid, kGradThreads, 0, st>>>(a);
            else logprob_grad_kernel<T, G, int64_t><<<grid, kGradThreads, 0, st>>>(a);
            return cuda_status(cudaGetLastError());
        });
    });
}

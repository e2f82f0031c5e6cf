// logprobs.cu -- log probabilities of given tokens with entropy, rank and top
// alternatives (drs_token_logprobs).
//
// s_j = x_j / T, m = max x, S = sum e^((x_j - m) / T):
//   logprob = (x_id - m) / T - ln S
//   entropy = ln S - (1 / S) sum e^((x_j - m) / T) (x_j - m) / T
//   rank    = 1 + the number of x_j > x_id
// The alternatives are the k largest x_j, equal ones in column order.
//
// A CTA takes a row: its largest logit, then the sums, then the alternatives
// one after the other, each as the largest key below the one before.
#include <climits>

#include "token_common.cuh"

namespace drs {
namespace {

constexpr int kThreadsPerRow = 256;
constexpr int kRowWarps = kThreadsPerRow / 32;
// Exponents (base 2) below this give 0; held there so that 0 times an
// infinite exponent does not arise in the entropy's sum.
constexpr float kLeastExponent = -200.0f;

struct LogprobParams {
    const void* logits;
    const void* ids;
    const float* temps;
    float* out_logprob;
    float* out_entropy;
    int32_t* out_rank;
    float* out_norm;
    int32_t* out_ids;
    float* out_logprobs;
    int64_t row_stride, canvas_len;
    int32_t vocab, k;
};

// Larger keys: larger values, then lower columns. NaN counts as -inf, -0 as 0.
__device__ __forceinline__ uint64_t key_of(float v, int column) {
    v = fmaxf(v, -INFINITY) + 0.0f;
    const uint32_t b = __float_as_uint(v);
    const uint32_t order = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    return static_cast<uint64_t>(order) << 32 | static_cast<uint32_t>(~column);
}

__device__ __forceinline__ float value_of(uint64_t key) {
    const uint32_t order = static_cast<uint32_t>(key >> 32);
    return __uint_as_float(order ^ (order >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ int column_of(uint64_t key) { return static_cast<int>(~static_cast<uint32_t>(key)); }

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <typename V, typename F> __device__ V block_reduce(V v, V* s_part, F f) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if (lane == 0) s_part[warp] = v;
    __syncthreads();
    v = s_part[0];
    for (int w = 1; w < kRowWarps; ++w) v = f(v, s_part[w]);
    return v;
}

template <typename T, typename I> __global__ void __launch_bounds__(kThreadsPerRow) logprob_kernel(const LogprobParams a) {
    __shared__ uint64_t s_key[kRowWarps];
    __shared__ float s_float[kRowWarps];
    __shared__ int s_int[kRowWarps];
    const int64_t row = blockIdx.x;
    const int64_t id = static_cast<int64_t>(static_cast<const I*>(a.ids)[row]);
    if (id < 0 || id >= a.vocab) {
        if (threadIdx.x == 0) {
            a.out_logprob[row] = 0.0f;
            if (a.out_entropy) a.out_entropy[row] = 0.0f;
            if (a.out_rank) a.out_rank[row] = 0;
            if (a.out_norm) a.out_norm[2 * row] = a.out_norm[2 * row + 1] = 0.0f;
        }
        for (int i = threadIdx.x; i < a.k; i += kThreadsPerRow) {
            a.out_ids[row * a.k + i] = -1;
            a.out_logprobs[row * a.k + i] = -INFINITY;
        }
        return;
    }
    const T* const x = static_cast<const T*>(a.logits) + row * a.row_stride;
    const float inverse = a.temps ? 1.0f / fmaxf(a.temps[row / a.canvas_len], kTempFloor) : 1.0f;
    const float own = to_f(x[id]);
    float top = -INFINITY;
    int above = 0;
    for (int j = threadIdx.x; j < a.vocab; j += kThreadsPerRow) {
        const float v = to_f(x[j]);
        top = fmaxf(top, v);
        above += v > own;
    }
    top = block_reduce(top, s_float, [](float p, float q) { return fmaxf(p, q); });
    above = block_reduce(above, s_int, [](int p, int q) { return p + q; });
    const float base = top == -INFINITY ? 0.0f : top, scale = inverse * kLog2e;
    float sum = 0.0f, weighted = 0.0f;
    for (int j = threadIdx.x; j < a.vocab; j += kThreadsPerRow) {
        const float t = max_nan((to_f(x[j]) - base) * scale, kLeastExponent);
        const float e = ex2_approx(t);
        sum += e;
        weighted = fmaf(e, t, weighted);
    }
    const auto add = [](float p, float q) { return p + q; };
    sum = block_reduce(sum, s_float, add);
    weighted = block_reduce(weighted, s_float, add);
    const float log_sum = top == -INFINITY && sum == 0.0f ? -INFINITY : logf(sum);
    const auto logprob = [&](float v) { return (v - top) * inverse - log_sum; };
    if (threadIdx.x == 0) {
        a.out_logprob[row] = logprob(own);
        if (a.out_entropy) a.out_entropy[row] = sum == 0.0f ? 0.0f : log_sum - weighted / sum * kLn2;
        if (a.out_rank) a.out_rank[row] = 1 + above;
        if (a.out_norm) a.out_norm[2 * row] = top, a.out_norm[2 * row + 1] = log_sum;
    }
    uint64_t last = ~0ull;
    for (int i = 0; i < a.k; ++i) {
        uint64_t best = 0;
        for (int j = threadIdx.x; j < a.vocab; j += kThreadsPerRow) {
            const uint64_t key = key_of(to_f(x[j]), j);
            if (key < last && key > best) best = key;
        }
        last = block_reduce(best, s_key, [](uint64_t p, uint64_t q) { return p > q ? p : q; });
        if (threadIdx.x == 0) {
            a.out_ids[row * a.k + i] = column_of(last);
            a.out_logprobs[row * a.k + i] = logprob(value_of(last));
        }
    }
}

}  // namespace
}  // namespace drs

extern "C" drs_status drs_token_logprobs(const void* logits, drs_dtype dtype, int64_t rows, int64_t vocab,
                                         int64_t row_stride, const void* ids, int32_t id_bits, const float* temps,
                                         int64_t canvas_len, int32_t k, float* out_logprob, float* out_entropy,
                                         int32_t* out_rank, float* out_norm, int32_t* out_ids, float* out_logprobs,
                                         void* stream) {
    using namespace drs;
    if (rows < 0 || vocab < 1 || !dtype_ok(dtype) || (id_bits != 32 && id_bits != 64)) return DRS_ERR_INVALID_ARG;
    if (row_stride < vocab || canvas_len < 1 || k < 0 || k > vocab) return DRS_ERR_INVALID_ARG;
    if (vocab > DRS_MAX_VOCAB || k > DRS_MAX_ALTERNATIVES || rows > DRS_MAX_SCORE_ROWS) return DRS_ERR_UNSUPPORTED;
    if (rows == 0) return DRS_OK;
    if (!logits || !ids || !out_logprob || (k > 0 && (!out_ids || !out_logprobs))) return DRS_ERR_INVALID_ARG;
    if (!aligned(logits, dtype_bytes(dtype)) || !aligned(ids, id_bits / 8) || !aligned(temps, 4) ||
        !aligned(out_logprob, 4) || !aligned(out_entropy, 4) || !aligned(out_rank, 4) || !aligned(out_norm, 4) ||
        !aligned(out_ids, 4) || !aligned(out_logprobs, 4))
        return DRS_ERR_INVALID_ARG;
    LogprobParams a{};
    a.logits = logits;
    a.ids = ids;
    a.temps = temps;
    a.out_logprob = out_logprob;
    a.out_entropy = out_entropy;
    a.out_rank = out_rank;
    a.out_norm = out_norm;
    a.out_ids = out_ids;
    a.out_logprobs = out_logprobs;
    a.row_stride = row_stride;
    a.canvas_len = canvas_len;
    a.vocab = static_cast<int32_t>(vocab);
    a.k = k;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return with_dtype(dtype, [&](auto t) -> drs_status {
        using T = decltype(t);
        const unsigned grid = static_cast<unsigned>(rows);
        if (id_bits == 32) logprob_kernel<T, int32_t><<<grid, kThreadsPerRow, 0, st>>>(a);
        else logprob_kernel<T, int64_t><<<grid, kThreadsPerRow, 0, st>>>(a);
        return cuda_status(cudaGetLastError());
    });
}

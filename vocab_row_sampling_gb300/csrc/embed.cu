// embed.cu -- the embedding lookup with scaling (drs_embed_tokens):
// out[t] = scale * table[ids[t]], rounded once.
//
// Bound by memory: one row read and one written per token. A block's threads
// lie along the columns, 16 bytes each, and take four tokens at once, so that
// each thread has four independent loads behind its four ids.
#include "token_common.cuh"

namespace drs {
namespace {

constexpr int kEmbedThreads = 256;
constexpr int kEmbedRows = 4;  // tokens a thread has in flight

struct EmbedParams {
    const void* table;
    const void* ids;
    void* out;
    int64_t tokens, vocab, table_stride, out_stride;
    int32_t width, columns;  // columns: of blockDim.x * kVec elements per block
    float scale;
};

// kVec: elements per access, 16 bytes or one element.
template <typename T, typename I, int kVec>
__global__ void __launch_bounds__(kEmbedThreads) embed_kernel(const EmbedParams a) {
    const T* const table = static_cast<const T*>(a.table);
    const I* const ids = static_cast<const I*>(a.ids);
    T* const out = static_cast<T*>(a.out);
    const int64_t block = blockIdx.x / a.columns;
    const int col = ((blockIdx.x % a.columns) * blockDim.x + threadIdx.x) * kVec;
    const int64_t t0 = block * (blockDim.y * kEmbedRows) + threadIdx.y;
    if (col >= a.width) return;
    int64_t id[kEmbedRows];
#pragma unroll
    for (int r = 0; r < kEmbedRows; ++r) {
        const int64_t t = t0 + r * blockDim.y;
        id[r] = t < a.tokens ? static_cast<int64_t>(ids[t]) : -1;
    }
    if constexpr (kVec > 1) {
        uint4 v[kEmbedRows];
#pragma unroll
        for (int r = 0; r < kEmbedRows; ++r) {
            v[r] = make_uint4(0, 0, 0, 0);
            if (id[r] >= 0 && id[r] < a.vocab)
                v[r] = __ldg(reinterpret_cast<const uint4*>(table + id[r] * a.table_stride + col));
        }
#pragma unroll
        for (int r = 0; r < kEmbedRows; ++r) {
            const int64_t t = t0 + r * blockDim.y;
            if (t >= a.tokens) continue;
            T* e = reinterpret_cast<T*>(&v[r]);
            if (id[r] >= 0 && id[r] < a.vocab) {
#pragma unroll
                for (int i = 0; i < kVec; ++i) e[i] = from_f<T>(to_f(e[i]) * a.scale);
            }
            __stcs(reinterpret_cast<uint4*>(out + t * a.out_stride + col), v[r]);
        }
    } else {
        T v[kEmbedRows];
#pragma unroll
        for (int r = 0; r < kEmbedRows; ++r) {
            v[r] = from_f<T>(0.0f);
            if (id[r] >= 0 && id[r] < a.vocab) v[r] = from_f<T>(to_f(table[id[r] * a.table_stride + col]) * a.scale);
        }
#pragma unroll
        for (int r = 0; r < kEmbedRows; ++r) {
            const int64_t t = t0 + r * blockDim.y;
            if (t < a.tokens) out[t * a.out_stride + col] = v[r];
        }
    }
}

template <typename T, typename I, int kVec> drs_status launch_embed(EmbedParams a, cudaStream_t stream) {
    int x = 1;
    const int64_t accesses = ceil_div(a.width, kVec);
    while (x < kEmbedThreads && x < accesses) x *= 2;
    const dim3 block(x, kEmbedThreads / x);
    a.columns = static_cast<int32_t>(ceil_div(accesses, x));
    const int64_t blocks = ceil_div(a.tokens, block.y * kEmbedRows) * a.columns;
    if (blocks > INT32_MAX) return DRS_ERR_UNSUPPORTED;
    embed_kernel<T, I, kVec><<<static_cast<unsigned>(blocks), block, 0, stream>>>(a);
    return cuda_status(cudaGetLastError());
}

}  // namespace
}  // namespace drs

extern "C" drs_status drs_embed_tokens(const void* table, drs_dtype dtype, int64_t vocab, int64_t width,
                                       int64_t table_stride, const void* ids, int32_t id_bits, int64_t tokens,
                                       float scale, void* out, int64_t out_stride, void* stream) {
    using namespace drs;
    if (tokens < 0 || vocab < 1 || width < 1 || !dtype_ok(dtype) || (id_bits != 32 && id_bits != 64))
        return DRS_ERR_INVALID_ARG;
    if (table_stride < width || out_stride < width) return DRS_ERR_INVALID_ARG;
    if (vocab > DRS_MAX_VOCAB || width > DRS_MAX_WIDTH) return DRS_ERR_UNSUPPORTED;
    if (tokens == 0) return DRS_OK;
    const size_t size = dtype_bytes(dtype);
    if (!table || !ids || !out || !aligned(table, size) || !aligned(out, size) || !aligned(ids, id_bits / 8))
        return DRS_ERR_INVALID_ARG;
    EmbedParams a{};
    a.table = table;
    a.ids = ids;
    a.out = out;
    a.tokens = tokens;
    a.vocab = vocab;
    a.table_stride = table_stride;
    a.out_stride = out_stride;
    a.width = static_cast<int32_t>(width);
    a.scale = scale;
    const bool vec = aligned(table, 16) && aligned(out, 16) && width * size % 16 == 0 &&
                     table_stride * size % 16 == 0 && out_stride * size % 16 == 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return with_dtype(dtype, [&](auto t) -> drs_status {
        using T = decltype(t);
        constexpr int kVec = 16 / sizeof(T);
        if (id_bits == 32) return vec ? launch_embed<T, int32_t, kVec>(a, st) : launch_embed<T, int32_t, 1>(a, st);
        return vec ? launch_embed<T, int64_t, kVec>(a, st) : launch_embed<T, int64_t, 1>(a, st);
    });
}

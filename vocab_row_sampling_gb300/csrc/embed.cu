// embed.cu -- the embedding lookup with scaling (drs_embed_tokens):
// out[t] = scale * table[ids[t]], rounded once.
//
// Bound by memory: one row read and one written per token. A block's threads
// lie along the columns, 16 bytes each, and take two or four tokens at once:
// that many independent loads per thread, behind as many ids. Rows that do
// not start on 16-byte boundaries (odd widths, strides or offsets) are
// written in aligned 16-byte words all the same, each put together from the
// two aligned words of the table that hold it: single elements took 12.1 us
// for 5003 x 1283 fp16, this 4.6. Measured: 65536 x 4096 bf16 117 us, 6.2 TB/s
// of the distinct rows and the output; 256 x 2048 2.1 us, the launch.
#include "token_common.cuh"

namespace drs {
namespace {

// Threads per CTA: 65536 x 4096 bf16 takes 117 us with 64 or 128, 120 with
// 256, 125 with 512.
constexpr int kAlignedThreads = 128;
// Rows off 16-byte boundaries: threads per CTA and words per thread. us for
// 30000 x 4095 and 5003 x 1283 16-bit elements: 57.5 and 4.7 with 128 and 4,
// 62.2 and 4.8 with 256 and 4, 64.9 and 5.4 with 128 and 2.
constexpr int kOddThreads = 128;
constexpr int kWords = 4;

struct EmbedParams {
    const void* table;
    const void* ids;
    void* out;
    int64_t tokens, vocab, table_stride, out_stride;
    int32_t width, columns;  // columns: CTAs along a row
    float scale;
};

__device__ __forceinline__ uint4 load16(const void* p) { return __ldg(static_cast<const uint4*>(p)); }

// 16 bytes of elements times scale.
template <typename T> __device__ __forceinline__ uint4 scaled(uint4 v, float scale) {
    T* const e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) e[i] = from_f<T>(to_f(e[i]) * scale);
    return v;
}

template <typename T, typename I, int kRows>
__global__ void __launch_bounds__(kAlignedThreads) embed_kernel(const EmbedParams a) {
    constexpr int kVec = 16 / sizeof(T);
    const T* const table = static_cast<const T*>(a.table);
    const I* const ids = static_cast<const I*>(a.ids);
    T* const out = static_cast<T*>(a.out);
    const int64_t block = blockIdx.x / a.columns;
    const int col = ((blockIdx.x % a.columns) * blockDim.x + threadIdx.x) * kVec;
    const int64_t t0 = block * (blockDim.y * kRows) + threadIdx.y;
    if (col >= a.width) return;
    int64_t id[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int64_t t = t0 + r * blockDim.y;
        const int64_t v = t < a.tokens ? static_cast<int64_t>(ids[t]) : -1;
        id[r] = v >= 0 && v < a.vocab ? v : -1;
    }
    uint4 v[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        v[r] = id[r] >= 0 ? load16(table + id[r] * a.table_stride + col) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int64_t t = t0 + r * blockDim.y;
        if (t >= a.tokens) continue;
        if (id[r] >= 0) v[r] = scaled<T>(v[r], a.scale);
        __stcs(reinterpret_cast<uint4*>(out + t * a.out_stride + col), v[r]);
    }
}

// Rows off 16-byte boundaries: a thread has up to kWords aligned words of one
// output row, and perhaps one element of the row's edges.
template <typename T, typename I> __global__ void __launch_bounds__(kOddThreads) embed_odd_kernel(const EmbedParams a) {
    constexpr int kVec = 16 / sizeof(T);
    const int64_t t = static_cast<int64_t>(blockIdx.x / a.columns) * blockDim.y + threadIdx.y;
    if (t >= a.tokens) return;
    const int c = (blockIdx.x % a.columns) * (blockDim.x * kWords) + threadIdx.x;
    const int64_t id = static_cast<int64_t>(static_cast<const I*>(a.ids)[t]);
    const bool have = id >= 0 && id < a.vocab;
    const T* const src = static_cast<const T*>(a.table) + (have ? id : 0) * a.table_stride;
    T* const dst = static_cast<T*>(a.out) + t * a.out_stride;
    const int head = min(static_cast<int>((-reinterpret_cast<uintptr_t>(dst) & 15) / sizeof(T)), a.width);
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(src + head) & 15);
    const int off = shift / static_cast<int>(sizeof(T));
    // words [w0, w1) of the row come from words that lie inside the table's
    // row; the elements before and after (at most 4 kVec - 2) one by one
    const int words = (a.width - head) / kVec;
    const int w0 = head < off ? 1 : 0;
    const int w1 = off && head - off + (words + 1) * kVec > a.width ? words - 1 : words;
    const T* const from = src + (head - off);
    uint4 lo[kWords], hi[kWords];
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
        const int w = c + k * blockDim.x;
        lo[k] = hi[k] = make_uint4(0, 0, 0, 0);
        if (have && w >= w0 && w < w1) {
            lo[k] = load16(from + w * kVec);
            if (off) hi[k] = load16(from + (w + 1) * kVec);
        }
    }
    const int lead = w0 < w1 ? head + w0 * kVec : a.width, trail = w0 < w1 ? head + w1 * kVec : a.width;
    if (c < lead + a.width - trail) {
        const int i = c < lead ? c : trail + c - lead;
        dst[i] = from_f<T>(have ? to_f(src[i]) * a.scale : 0.0f);
    }
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
        const int w = c + k * blockDim.x;
        if (w < w0 || w >= w1) continue;
        const uint4 v = joined(lo[k], hi[k], shift);
        __stcs(reinterpret_cast<uint4*>(dst + head + w * kVec), have ? scaled<T>(v, a.scale) : lo[k]);
    }
}

template <typename T, typename I, int kRows> drs_status launch_rows(EmbedParams a, cudaStream_t stream) {
    const int64_t places = a.width / (16 / sizeof(T));  // a word per thread along the columns
    a.columns = static_cast<int32_t>(ceil_div(places, kAlignedThreads));
    int x = static_cast<int>(ceil_div(places, a.columns));
    if (x > 32) x = (x + 31) / 32 * 32;
    const dim3 block(x, kAlignedThreads / x);
    const int64_t blocks = ceil_div(a.tokens, block.y * kRows) * a.columns;
    if (blocks > INT32_MAX) return DRS_ERR_UNSUPPORTED;
    embed_kernel<T, I, kRows><<<static_cast<unsigned>(blocks), block, 0, stream>>>(a);
    return cuda_status(cudaGetLastError());
}

template <typename T, typename I> drs_status launch_embed(EmbedParams a, bool vec, cudaStream_t stream) {
    constexpr int kVec = 16 / sizeof(T);
    const int64_t words = a.width / kVec;
    if (vec) {
        // us with one, two, four and eight tokens per thread (bf16): 256 x 2048
        // 1.9, 1.9, 2.1, 2.9; 512 x 4096 2.7, 2.4, 2.6, 3.2; at the border 2432 x 4096 7.3,
        // 6.0, 5.8, 6.4; 8192 x 4096 23.1, 18.5, 17.9, 18.7; 65536 x 4096 of 100000 rows
        // 159, 120, 114, 117.
        const bool many = a.tokens * words > int64_t{8192} * sm_count();
        return many ? launch_rows<T, I, 4>(a, stream) : launch_rows<T, I, 2>(a, stream);
    }
    a.columns = static_cast<int32_t>(ceil_div(words, kOddThreads * kWords));
    if (a.columns < 1) a.columns = 1;
    int x = static_cast<int>(ceil_div(words, int64_t{a.columns} * kWords));
    if (x < 32) x = 32;  // one for each of the elements of a row's edges
    const dim3 block(x, kOddThreads / x);
    const int64_t blocks = ceil_div(a.tokens, block.y) * a.columns;
    if (blocks > INT32_MAX) return DRS_ERR_UNSUPPORTED;
    embed_odd_kernel<T, I><<<static_cast<unsigned>(blocks), block, 0, stream>>>(a);
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
        return id_bits == 32 ? launch_embed<T, int32_t>(a, vec, st) : launch_embed<T, int64_t>(a, vec, st);
    });
}

// embed.cu -- the embedding lookup with scaling (drs_embed_tokens):
// out[t] = scale * table[ids[t]], rounded once.
//
// Bound by memory: one row read and one written per token. A block's threads
// lie along the columns, 16 bytes each, and take two or four tokens at once:
// that many independent loads per thread, behind as many ids. Rows that do
// not start on 16-byte boundaries (odd widths, strides or offsets) are
// written in aligned 16-byte words all the same, each put together from the
// two aligned words of the table that hold it: single elements took 12.1 us
// for 5003 x 1283 fp16.
#include "token_common.cuh"

namespace drs {
namespace {

// Threads per CTA, for rows off 16-byte boundaries and for aligned ones:
// 65536 x 4096 bf16 takes 117 us with 64 or 128, 120 with 256, 125 with 512.
constexpr int kThreadsOf[2] = {256, 128};

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

// The 16 bytes that begin `shift` bytes into the 32 bytes of lo and hi.
__device__ __forceinline__ uint4 joined(uint4 lo, uint4 hi, int shift) {
    uint32_t w[5] = {lo.x, lo.y, lo.z, lo.w, hi.x};
    if (shift >= 8) w[0] = lo.z, w[1] = lo.w, w[2] = hi.x, w[3] = hi.y, w[4] = hi.z;
    if (shift & 4) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = w[4], w[4] = shift >= 8 ? hi.w : hi.y;
    const int bits = (shift & 3) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// kAligned: every row of the table and of the output starts on 16 bytes. A
// thread has word `c` of its rows, and in rows that do not also an element of
// their edges.
template <typename T, typename I, bool kAligned, int kEmbedRows>
__global__ void __launch_bounds__(kThreadsOf[kAligned]) embed_kernel(const EmbedParams a) {
    constexpr int kVec = 16 / sizeof(T);
    const T* const table = static_cast<const T*>(a.table);
    const I* const ids = static_cast<const I*>(a.ids);
    T* const out = static_cast<T*>(a.out);
    const int64_t block = blockIdx.x / a.columns;
    const int c = (blockIdx.x % a.columns) * blockDim.x + threadIdx.x;
    const int64_t t0 = block * (blockDim.y * kEmbedRows) + threadIdx.y;
    if (kAligned && c * kVec >= a.width) return;
    int64_t id[kEmbedRows];
#pragma unroll
    for (int r = 0; r < kEmbedRows; ++r) {
        const int64_t t = t0 + r * blockDim.y;
        const int64_t v = t < a.tokens ? static_cast<int64_t>(ids[t]) : -1;
        id[r] = v >= 0 && v < a.vocab ? v : -1;
    }
    if constexpr (kAligned) {
        uint4 v[kEmbedRows];
#pragma unroll
        for (int r = 0; r < kEmbedRows; ++r)
            v[r] = id[r] >= 0 ? load16(table + id[r] * a.table_stride + c * kVec) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < kEmbedRows; ++r) {
            const int64_t t = t0 + r * blockDim.y;
            if (t >= a.tokens) continue;
            if (id[r] >= 0) v[r] = scaled<T>(v[r], a.scale);
            __stcs(reinterpret_cast<uint4*>(out + t * a.out_stride + c * kVec), v[r]);
        }
    } else {
        uint4 lo[kEmbedRows], hi[kEmbedRows];
        T edge[kEmbedRows];
        int at[kEmbedRows], shift[kEmbedRows], edge_at[kEmbedRows];  // -1: nothing here
#pragma unroll
        for (int r = 0; r < kEmbedRows; ++r) {
            const int64_t t = t0 + r * blockDim.y;
            at[r] = edge_at[r] = -1;
            lo[r] = hi[r] = make_uint4(0, 0, 0, 0);
            edge[r] = from_f<T>(0.0f);
            if (t >= a.tokens) continue;
            const T* const src = table + max(id[r], static_cast<int64_t>(0)) * a.table_stride;
            const int head = min(static_cast<int>((-reinterpret_cast<uintptr_t>(out + t * a.out_stride) & 15) / sizeof(T)), a.width);
            const int off = static_cast<int>(reinterpret_cast<uintptr_t>(src + head) & 15) / static_cast<int>(sizeof(T));
            // words [w0, w1) of the row come from words that lie inside the
            // table's row; the elements before and after (at most 4 kVec) one
            // by one
            const int words = (a.width - head) / kVec;
            const int w0 = head < off ? 1 : 0;
            const int w1 = off && head - off + (words + 1) * kVec > a.width ? words - 1 : words;
            const int lead = w0 < w1 ? head + w0 * kVec : a.width, trail = w0 < w1 ? head + w1 * kVec : a.width;
            if (c >= w0 && c < w1) {
                at[r] = head + c * kVec;
                shift[r] = off * static_cast<int>(sizeof(T));
                if (id[r] >= 0) {
                    lo[r] = load16(src + at[r] - off);
                    if (off) hi[r] = load16(src + at[r] - off + kVec);
                }
            }
            if (c < lead + a.width - trail) {
                edge_at[r] = c < lead ? c : trail + c - lead;
                if (id[r] >= 0) edge[r] = src[edge_at[r]];
            }
        }
#pragma unroll
        for (int r = 0; r < kEmbedRows; ++r) {
            T* const dst = out + (t0 + r * blockDim.y) * a.out_stride;
            if (at[r] >= 0) __stcs(reinterpret_cast<uint4*>(dst + at[r]), scaled<T>(joined(lo[r], hi[r], shift[r]), a.scale));
            if (edge_at[r] >= 0) dst[edge_at[r]] = id[r] >= 0 ? from_f<T>(to_f(edge[r]) * a.scale) : edge[r];
        }
    }
}

template <typename T, typename I, bool kAligned, int kRows>
drs_status launch_embed_rows(EmbedParams a, int64_t places, cudaStream_t stream) {
    constexpr int kThreads = kThreadsOf[kAligned];
    a.columns = static_cast<int32_t>(ceil_div(places, kThreads));
    int x = static_cast<int>(ceil_div(places, a.columns));
    if (x > 32) x = (x + 31) / 32 * 32;
    const dim3 block(x, kThreads / x);
    const int64_t blocks = ceil_div(a.tokens, block.y * kRows) * a.columns;
    if (blocks > INT32_MAX) return DRS_ERR_UNSUPPORTED;
    embed_kernel<T, I, kAligned, kRows><<<static_cast<unsigned>(blocks), block, 0, stream>>>(a);
    return cuda_status(cudaGetLastError());
}

template <typename T, typename I> drs_status launch_embed(const EmbedParams& a, bool vec, cudaStream_t stream) {
    constexpr int kVec = 16 / sizeof(T);
    // threads along the columns: a word each, and in rows off 16-byte
    // boundaries at least one for each of the (at most 4 kVec - 2) elements of
    // a row's edges
    int64_t places = a.width / kVec;
    if (!vec) return launch_embed_rows<T, I, false, 2>(a, places < 4 * kVec ? 4 * kVec : places, stream);
    // Tokens per thread, measured: 65536 x 4096 bf16 takes 164 us with one, 125
    // with two, 120 with four and 122 with eight; 256 x 2048 takes 1.9 us with
    // one or two, 2.2 with four, 3.0 with eight.
    const bool many = a.tokens * places > int64_t{8192} * sm_count();
    return many ? launch_embed_rows<T, I, true, 4>(a, places, stream) : launch_embed_rows<T, I, true, 2>(a, places, stream);
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

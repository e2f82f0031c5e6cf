// embed_grad.cu -- the gradient of the embedding lookup
// (drs_embed_tokens_grad): grad_table[v] = scale * sum of grad_out[t] over
// the tokens t with ids[t] == v.
//
// The tokens are sorted by id first (stable, so a row's tokens stay in
// order), and the sorted list is cut into pieces of kPiece tokens whatever
// the ids are: the work is even however often an id occurs. A piece's threads
// lie along the columns and add its tokens' rows in fp32 registers; an id
// that lies inside a piece is written at once, one that crosses a border
// leaves fp32 partial sums that a last kernel adds in order. No atomics
// touch a sum, so equal calls give equal bits. Rows without tokens are zeroed
// in the same launch (unless the call accumulates).
//
// Bound by memory: the gradients of the tokens are read once and the table's
// rows written once; the partial sums are at most 2 / kPiece of the former.
#include <climits>

#include "token_common.cuh"

namespace drs {
namespace {

// ------------------------------------------------------------- the sort
//
// Least significant digit first, one or two digits. A pass counts the digits
// of every tile and then places the tile's tokens: a CTA adds up the counts
// of the tiles before its own, and inside a tile a token's rank among equal
// digits comes from the warps' match masks, in order.

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortTiles = 148;  // at most: every CTA reads all tiles' counts
constexpr int kMaxDigit = 11;

struct SortParams {
    const void* ids;          // the first pass reads the ids themselves
    const uint32_t* keys_in;  // later passes the sorted keys and tokens
    const uint32_t* tokens_in;
    uint32_t* keys_out;
    uint32_t* tokens_out;
    uint32_t* counts;  // [tiles][bins]
    int64_t n;
    int32_t tile, tiles, bits, shift, vocab, id_bits;
};

// The key of a token: its id, `vocab` for one outside the vocabulary.
__device__ __forceinline__ uint32_t sort_key(const SortParams& a, int64_t i) {
    if (a.keys_in) return a.keys_in[i];
    const int64_t id = a.id_bits == 32 ? static_cast<int64_t>(static_cast<const int32_t*>(a.ids)[i])
                                       : static_cast<const int64_t*>(a.ids)[i];
    return static_cast<uint32_t>(id >= 0 && id < a.vocab ? id : a.vocab);
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortParams a) {
    extern __shared__ uint32_t s_count[];
    const int bins = 1 << a.bits;
    for (int i = threadIdx.x; i < bins; i += kSortThreads) s_count[i] = 0;
    __syncthreads();
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.tile;
    const int64_t hi = lo + a.tile < a.n ? lo + a.tile : a.n;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads)
        atomicAdd(&s_count[(sort_key(a, i) >> a.shift) & (bins - 1)], 1u);
    __syncthreads();
    for (int i = threadIdx.x; i < bins; i += kSortThreads) a.counts[static_cast<int64_t>(blockIdx.x) * bins + i] = s_count[i];
}

__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const SortParams a) {
    extern __shared__ uint32_t s_place[];  // [bins] next places, then uint16 [warps][bins] counts
    __shared__ uint32_t s_scan[kSortWarps];
    const int bins = 1 << a.bits, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint16_t* const s_warp = reinterpret_cast<uint16_t*>(s_place + bins);

    // a thread takes `per` consecutive digits: tokens with a lower digit, and
    // with this digit in earlier tiles, go first
    const int per = bins > kSortThreads ? bins / kSortThreads : 1;
    uint32_t earlier[1 << (kMaxDigit - 10)] = {}, total[1 << (kMaxDigit - 10)] = {}, sum = 0;
    if (tid * per < bins) {
        for (int t = 0; t < a.tiles; ++t)
            for (int k = 0; k < per; ++k) {
                const uint32_t c = a.counts[static_cast<int64_t>(t) * bins + tid * per + k];
                total[k] += c;
                if (t < static_cast<int>(blockIdx.x)) earlier[k] += c;
            }
        for (int k = 0; k < per; ++k) sum += total[k];
    }
    const uint32_t scan = warp_scan_inclusive(sum, lane);
    if (lane == 31) s_scan[warp] = scan;
    __syncthreads();
    uint32_t at = scan - sum;
    for (int w = 0; w < warp; ++w) at += s_scan[w];
    if (tid * per < bins)
        for (int k = 0; k < per; ++k) {
            s_place[tid * per + k] = at + earlier[k];
            at += total[k];
        }

    const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.tile;
    const int64_t hi = lo + a.tile < a.n ? lo + a.tile : a.n;
    for (int64_t base = lo; base < hi; base += kSortThreads) {
        for (int i = tid; i < bins * kSortWarps / 2; i += kSortThreads) reinterpret_cast<uint32_t*>(s_warp)[i] = 0;
        __syncthreads();
        const int64_t i = base + tid;
        const bool have = i < hi;
        const uint32_t key = have ? sort_key(a, i) : 0;
        const uint32_t token = !have ? 0 : a.tokens_in ? a.tokens_in[i] : static_cast<uint32_t>(i);
        const uint32_t digit = (key >> a.shift) & (bins - 1);
        const uint32_t same = __match_any_sync(0xffffffffu, have ? digit : 0xffffffffu);
        const int below = __popc(same & ((1u << lane) - 1));
        if (have && below == 0) s_warp[warp * bins + digit] = static_cast<uint16_t>(__popc(same));
        __syncthreads();
        for (int d = tid; d < bins; d += kSortThreads) {
            uint32_t run = 0;
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = s_warp[w * bins + d];
                s_warp[w * bins + d] = static_cast<uint16_t>(run);
                run += c;
            }
            // the counts of the sub-tile are added after its places are read
            earlier[d / kSortThreads] = run;
        }
        __syncthreads();
        if (have) {
            const uint32_t to = s_place[digit] + s_warp[warp * bins + digit] + below;
            a.keys_out[to] = key;
            a.tokens_out[to] = token;
        }
        __syncthreads();
        for (int d = tid; d < bins; d += kSortThreads) s_place[d] += earlier[d / kSortThreads];
    }
}

// ------------------------------------------------------------- the sums

constexpr int kPiece = 32;         // sorted tokens per piece
constexpr int kSumThreads = 256;
constexpr int kSumAhead = 8;       // rows a thread has in flight
constexpr int kZeroBytes = 65536;  // of the table per zeroing CTA, about

struct GradParams {
    const void* grad;
    void* table;
    const uint32_t* keys;  // sorted
    const uint32_t* tokens;
    float* partial;  // [pieces][2][width]
    int64_t n, pieces, grad_stride, table_stride;
    int64_t sum_blocks;  // the CTAs after these zero rows
    int32_t width, columns, vocab, zero_rows;
    float scale;
    bool accumulate;
};

template <typename G, int kVec> struct Row;  // kVec elements in flight
template <typename G> struct Row<G, 8> {
    Raw8<G> raw;
    __device__ __forceinline__ void load(const G* p) { raw.load(p); }
    __device__ __forceinline__ void unpack(float (&v)[8]) const { raw.unpack(v); }
};
template <typename G> struct Row<G, 1> {
    G raw;
    __device__ __forceinline__ void load(const G* p) { raw = __ldg(p); }
    __device__ __forceinline__ void unpack(float (&v)[1]) const { v[0] = to_f(raw); }
};

template <typename T, int kVec> __device__ __forceinline__ void store_row(T* p, const float (&v)[kVec]) {
    if constexpr (kVec == 1) {
        *p = from_f<T>(v[0]);
    } else {
        alignas(16) T e[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) e[i] = from_f<T>(v[i]);
#pragma unroll
        for (int i = 0; i < static_cast<int>(kVec * sizeof(T) / 16); ++i)
            __stcs(reinterpret_cast<uint4*>(p) + i, reinterpret_cast<const uint4*>(e)[i]);
    }
}

// The finished row of an id: scaled, added to what the table holds where
// the call accumulates, rounded once.
template <typename T, int kVec>
__device__ __forceinline__ void write_row(const GradParams& a, uint32_t key, int col, const float (&sum)[kVec]) {
    T* const p = static_cast<T*>(a.table) + static_cast<int64_t>(key) * a.table_stride + col;
    float v[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = a.accumulate ? to_f(p[i]) + sum[i] * a.scale : sum[i] * a.scale;
    store_row<T, kVec>(p, v);
}

template <typename T> __device__ void zero_rows(const GradParams& a, int64_t block) {
    __shared__ bool s_touched[kSumThreads];
    const int64_t v0 = block * a.zero_rows;
    const int n = static_cast<int>(v0 + a.zero_rows < a.vocab ? a.zero_rows : a.vocab - v0);
    for (int r = threadIdx.x; r < n; r += kSumThreads) {
        const uint32_t key = static_cast<uint32_t>(v0 + r);
        int64_t lo = 0, hi = a.n;  // the first token whose key is not below
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            if (a.keys[mid] < key) lo = mid + 1;
            else hi = mid;
        }
        s_touched[r] = lo < a.n && a.keys[lo] == key;
    }
    __syncthreads();
    for (int r = 0; r < n; ++r) {
        if (s_touched[r]) continue;
        T* const p = static_cast<T*>(a.table) + (v0 + r) * a.table_stride;
        // 16-byte stores between the row's ragged ends
        int lead = static_cast<int>((-reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
        lead = lead < a.width ? lead : a.width;
        const int words = (a.width - lead) / static_cast<int>(16 / sizeof(T));
        const int done = lead + words * static_cast<int>(16 / sizeof(T));
        for (int i = threadIdx.x; i < lead; i += kSumThreads) p[i] = from_f<T>(0.0f);
        for (int i = threadIdx.x; i < words; i += kSumThreads)
            __stcs(reinterpret_cast<uint4*>(p + lead) + i, make_uint4(0, 0, 0, 0));
        for (int i = done + threadIdx.x; i < a.width; i += kSumThreads) p[i] = from_f<T>(0.0f);
    }
}

template <typename G, typename T, int kVec>
__global__ void __launch_bounds__(kSumThreads) grad_sum_kernel(const GradParams a) {
    if (blockIdx.x >= a.sum_blocks) {
        zero_rows<T>(a, blockIdx.x - a.sum_blocks);
        return;
    }
    const int tx = threadIdx.x % a.columns, ty = threadIdx.x / a.columns;
    const int across = static_cast<int>(ceil_div(a.width, a.columns * kVec));  // CTAs along a row
    const int64_t piece = blockIdx.x / across * (kSumThreads / a.columns) + ty;
    const int col = static_cast<int>((blockIdx.x % across) * a.columns + tx) * kVec;
    if (piece >= a.pieces || col >= a.width) return;
    const uint32_t none = static_cast<uint32_t>(a.vocab);
    const int64_t p0 = piece * kPiece, p1 = p0 + kPiece < a.n ? p0 + kPiece : a.n;
    const G* const grad = static_cast<const G*>(a.grad) + col;
    float* const partial = a.partial + piece * 2 * a.width + col;

    float acc[kVec] = {};
    uint32_t cur = a.keys[p0];
    bool head = p0 > 0 && a.keys[p0 - 1] == cur;  // began in an earlier piece
    for (int64_t p = p0; p < p1; p += kSumAhead) {
        uint32_t key[kSumAhead];
        Row<G, kVec> row[kSumAhead];
#pragma unroll
        for (int k = 0; k < kSumAhead; ++k) {
            key[k] = p + k < p1 ? a.keys[p + k] : none;
            if (key[k] != none) row[k].load(grad + static_cast<int64_t>(a.tokens[p + k]) * a.grad_stride);
        }
#pragma unroll
        for (int k = 0; k < kSumAhead; ++k) {
            if (p + k >= p1) break;
            if (key[k] != cur) {
                if (head) store_row<float, kVec>(partial, acc);
                else write_row<T, kVec>(a, cur, col, acc);
#pragma unroll
                for (int i = 0; i < kVec; ++i) acc[i] = 0.0f;
                cur = key[k];
                head = false;
            }
            if (cur != none) {
                float v[kVec];
                row[k].unpack(v);
#pragma unroll
                for (int i = 0; i < kVec; ++i) acc[i] += v[i];
            }
        }
    }
    if (cur == none) return;
    const bool goes_on = p1 < a.n && a.keys[p1] == cur;
    if (head) store_row<float, kVec>(partial, acc);
    else if (goes_on) store_row<float, kVec>(partial + a.width, acc);
    else write_row<T, kVec>(a, cur, col, acc);
}

// The ids that cross borders: a CTA of the piece in which such an id begins
// adds its partial sums in order.
template <typename T, int kVec>
__global__ void __launch_bounds__(kSumThreads) grad_join_kernel(const GradParams a) {
    const int tx = threadIdx.x % a.columns, ty = threadIdx.x / a.columns;
    const int across = static_cast<int>(ceil_div(a.width, a.columns * kVec));
    const int64_t piece = blockIdx.x / across * (kSumThreads / a.columns) + ty;
    const int col = static_cast<int>((blockIdx.x % across) * a.columns + tx) * kVec;
    if (piece >= a.pieces || col >= a.width) return;
    const int64_t p0 = piece * kPiece, p1 = p0 + kPiece;
    if (p1 >= a.n) return;
    const uint32_t key = a.keys[p1 - 1];
    if (key == static_cast<uint32_t>(a.vocab) || a.keys[p1] != key) return;
    if (p0 > 0 && a.keys[p0 - 1] == key) return;  // began earlier
    int64_t lo = p1, hi = a.n;  // the end of the id's tokens
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (a.keys[mid] <= key) lo = mid + 1;
        else hi = mid;
    }
    const int64_t last = (lo - 1) / kPiece;
    float acc[kVec];
    Row<float, kVec> row;
    row.load(a.partial + (piece * 2 + 1) * a.width + col);
    row.unpack(acc);
    for (int64_t q = piece + 1; q <= last; ++q) {
        float v[kVec];
        row.load(a.partial + q * 2 * a.width + col);
        row.unpack(v);
#pragma unroll
        for (int i = 0; i < kVec; ++i) acc[i] += v[i];
    }
    write_row<T, kVec>(a, key, col, acc);
}

// ------------------------------------------------------------- the call

size_t rounded(size_t bytes) { return (bytes + kWorkspaceAlign - 1) / kWorkspaceAlign * kWorkspaceAlign; }

struct SortPlan {
    int passes, bits;
    int32_t tile, tiles;
    static SortPlan of(int64_t n, int64_t vocab) {
        int key = 1;
        while ((int64_t{1} << key) <= vocab) ++key;  // keys are 0 .. vocab
        SortPlan s;
        s.passes = key <= kMaxDigit ? 1 : 2;
        s.bits = (key + s.passes - 1) / s.passes;
        const int64_t tiles = ceil_div(n, kSortThreads) < kSortTiles ? ceil_div(n, kSortThreads) : kSortTiles;
        s.tile = static_cast<int32_t>(ceil_div(ceil_div(n, tiles), kSortThreads) * kSortThreads);
        s.tiles = static_cast<int32_t>(ceil_div(n, s.tile));
        return s;
    }
};

struct Workspace {
    uint32_t *keys[2], *tokens[2], *counts;
    float* partial;
    size_t bytes;
    static Workspace of(void* base, int64_t n, int64_t vocab, int64_t width) {
        Workspace w{};
        size_t at = 0;
        const auto take = [&](size_t bytes) {
            unsigned char* p = static_cast<unsigned char*>(base) + at;
            at += rounded(bytes);
            return p;
        };
        const SortPlan s = SortPlan::of(n, vocab);
        for (int i = 0; i < s.passes; ++i) {
            w.keys[i] = reinterpret_cast<uint32_t*>(take(static_cast<size_t>(n) * 4));
            w.tokens[i] = reinterpret_cast<uint32_t*>(take(static_cast<size_t>(n) * 4));
        }
        w.counts = reinterpret_cast<uint32_t*>(take((static_cast<size_t>(s.tiles) << s.bits) * 4));
        w.partial = reinterpret_cast<float*>(take(static_cast<size_t>(ceil_div(n, kPiece)) * 2 * width * 4));
        w.bytes = at;
        return w;
    }
};

drs_status sort_tokens(const SortPlan& s, const Workspace& w, const void* ids, int id_bits, int64_t n, int64_t vocab,
                       cudaStream_t stream) {
    const size_t bins = size_t{1} << s.bits;
    const size_t count_smem = bins * 4, place_smem = bins * 4 + bins * 2 * kSortWarps;
    if (cudaFuncSetAttribute(sort_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(place_smem)) != cudaSuccess)
        return DRS_ERR_CUDA;
    for (int pass = 0; pass < s.passes; ++pass) {
        SortParams a{};
        a.ids = ids;
        a.keys_in = pass ? w.keys[0] : nullptr;
        a.tokens_in = pass ? w.tokens[0] : nullptr;
        a.keys_out = w.keys[pass];
        a.tokens_out = w.tokens[pass];
        a.counts = w.counts;
        a.n = n;
        a.tile = s.tile;
        a.tiles = s.tiles;
        a.bits = s.bits;
        a.shift = pass * s.bits;
        a.vocab = static_cast<int32_t>(vocab);
        a.id_bits = id_bits;
        sort_count_kernel<<<s.tiles, kSortThreads, count_smem, stream>>>(a);
        sort_place_kernel<<<s.tiles, kSortThreads, place_smem, stream>>>(a);
    }
    return cuda_status(cudaGetLastError());
}

template <typename G, typename T, int kVec> drs_status launch_sums(GradParams a, cudaStream_t stream) {
    int x = 1;
    while (x < kSumThreads && x * kVec < a.width) x *= 2;
    a.columns = x;
    const int64_t across = ceil_div(a.width, static_cast<int64_t>(x) * kVec);
    a.sum_blocks = ceil_div(a.pieces, kSumThreads / x) * across;
    int64_t zero_blocks = 0;
    if (!a.accumulate) {
        const int64_t rows = kZeroBytes / (static_cast<int64_t>(a.width) * sizeof(T));
        a.zero_rows = static_cast<int32_t>(rows < 1 ? 1 : rows > kSumThreads ? kSumThreads : rows);
        zero_blocks = ceil_div(a.vocab, a.zero_rows);
    }
    if (a.sum_blocks + zero_blocks > INT_MAX) return DRS_ERR_UNSUPPORTED;
    if (a.sum_blocks + zero_blocks > 0)
        grad_sum_kernel<G, T, kVec>
            <<<static_cast<unsigned>(a.sum_blocks + zero_blocks), kSumThreads, 0, stream>>>(a);
    if (a.pieces > 1)
        grad_join_kernel<T, kVec><<<static_cast<unsigned>(a.sum_blocks), kSumThreads, 0, stream>>>(a);
    return cuda_status(cudaGetLastError());
}

bool grad_sizes_ok(int64_t tokens, int64_t vocab, int64_t width) {
    return tokens >= 0 && tokens <= DRS_MAX_TOKENS && vocab >= 1 && vocab <= DRS_MAX_VOCAB && width >= 1 &&
           width <= DRS_MAX_WIDTH;
}

}  // namespace
}  // namespace drs

extern "C" size_t drs_embed_tokens_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t width) {
    using namespace drs;
    if (!grad_sizes_ok(tokens, vocab, width) || tokens == 0) return 0;
    return Workspace::of(nullptr, tokens, vocab, width).bytes;
}

extern "C" drs_status drs_embed_tokens_grad(const void* grad_out, drs_dtype grad_dtype, int64_t tokens, int64_t width,
                                            int64_t grad_stride, const void* ids, int32_t id_bits, float scale,
                                            int accumulate, void* grad_table, drs_dtype table_dtype, int64_t vocab,
                                            int64_t table_stride, void* workspace, size_t workspace_bytes,
                                            void* stream) {
    using namespace drs;
    if (tokens < 0 || vocab < 1 || width < 1 || !dtype_ok(grad_dtype) || !dtype_ok(table_dtype) ||
        (id_bits != 32 && id_bits != 64))
        return DRS_ERR_INVALID_ARG;
    if (table_stride < width || grad_stride < width) return DRS_ERR_INVALID_ARG;
    if (!grad_sizes_ok(tokens, vocab, width)) return DRS_ERR_UNSUPPORTED;
    if (!grad_table || !aligned(grad_table, dtype_bytes(table_dtype))) return DRS_ERR_INVALID_ARG;
    if (tokens > 0) {
        if (!grad_out || !ids || !aligned(grad_out, dtype_bytes(grad_dtype)) || !aligned(ids, id_bits / 8))
            return DRS_ERR_INVALID_ARG;
        if (!workspace || !aligned(workspace, kWorkspaceAlign) ||
            workspace_bytes < drs_embed_tokens_grad_workspace_bytes(tokens, vocab, width))
            return DRS_ERR_INVALID_ARG;
    }
    if (tokens == 0 && accumulate) return DRS_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    GradParams a{};
    if (tokens > 0) {
        const SortPlan s = SortPlan::of(tokens, vocab);
        const Workspace w = Workspace::of(workspace, tokens, vocab, width);
        const drs_status status = sort_tokens(s, w, ids, id_bits, tokens, vocab, st);
        if (status != DRS_OK) return status;
        a.keys = w.keys[s.passes - 1];
        a.tokens = w.tokens[s.passes - 1];
        a.partial = w.partial;
    }
    a.grad = grad_out;
    a.table = grad_table;
    a.n = tokens;
    a.pieces = ceil_div(tokens, kPiece);
    a.grad_stride = grad_stride;
    a.table_stride = table_stride;
    a.width = static_cast<int32_t>(width);
    a.vocab = static_cast<int32_t>(vocab);
    a.scale = scale;
    a.accumulate = accumulate != 0;
    const bool vec = width % 8 == 0 && aligned(grad_out, 16) && aligned(grad_table, 16) &&
                     grad_stride * dtype_bytes(grad_dtype) % 16 == 0 &&
                     table_stride * dtype_bytes(table_dtype) % 16 == 0;
    return with_dtype(grad_dtype, [&](auto g) -> drs_status {
        return with_dtype(table_dtype, [&](auto t) -> drs_status {
            return vec ? launch_sums<decltype(g), decltype(t), 8>(a, st)
                       : launch_sums<decltype(g), decltype(t), 1>(a, st);
        });
    });
}

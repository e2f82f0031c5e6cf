// embed_grad.cu -- the gradient of the embedding lookup
// (drs_embed_tokens_grad): grad_table[v] = scale * sum of grad_out[t] over
// the tokens t with ids[t] == v.
//
// The tokens are sorted by id first (stable, so a row's tokens stay in
// order), and the sorted list is cut into pieces of equal length whatever
// the ids are: the work is even however often an id occurs. A piece's threads
// lie along the columns and add its tokens' rows in fp32 registers; an id
// that lies inside a piece is written at once, one that crosses a border
// leaves fp32 partial sums that the last of its pieces to finish adds in
// order. No atomics touch a sum, so equal calls give equal bits. Rows without
// tokens are zeroed in the same launch (unless the call accumulates).
//
// Bound by memory: the gradients of the tokens are read once and the table's
// rows written once. The partial sums are at most two rows of fp32 per piece,
// written and read again: 2 / piece of the elements of the gradients, twice that
// share of their bytes where those have 16 bits.
// Measured: 32768 x 2048 bf16 into 262144 fp32 rows 317 us, 7.2 TB/s (15 for the
// sort, the rest mostly stores, which alone reach 7.6 TB/s); 2048 x 1024 into
// 8192 rows 14.2 us, most of it latency.
#include <climits>

#include "token_common.cuh"

namespace drs {
namespace {

// The sums follow the sort as a programmatic dependent launch: their CTAs are
// in place when the sort ends.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------------- the sort
//
// By ranks, by one cluster or by tiles, as the number of tokens grows. The
// latter two go by digits, the least significant first, one or two of them. A
// pass of the tiles counts the digits of every tile and then places the tile's tokens: a CTA adds up the counts
// of the tiles before its own, and inside a tile a token's rank among equal
// digits comes from the warps' masks, in order.

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
    unsigned long long* clear;  // counters that the first kernel sets to 0
    int64_t n, clear_n;
    int32_t tile, tiles, bits, shift, vocab, id_bits;
};

// The key of a token: its id, `vocab` for one outside the vocabulary.
__device__ __forceinline__ uint32_t sort_key(const SortParams& a, int64_t i) {
    if (a.keys_in) return a.keys_in[i];
    const int64_t id = a.id_bits == 32 ? static_cast<int64_t>(static_cast<const int32_t*>(a.ids)[i])
                                       : static_cast<const int64_t*>(a.ids)[i];
    return static_cast<uint32_t>(id >= 0 && id < a.vocab ? id : a.vocab);
}

// The lanes of the warp with the same digit, for lanes that have one: a
// ballot per bit. __match_any_sync takes a turn per distinct digit, up to 32
// (2048 tokens: 18.3 us for the whole call with it, 17.2 so; 131072: 75, 72).
__device__ __forceinline__ uint32_t lanes_with(uint32_t digit, int bits, bool have) {
    uint32_t same = __ballot_sync(0xffffffffu, have);
#pragma unroll
    for (int b = 0; b < kMaxDigit; ++b) {
        if (b >= bits) break;
        const uint32_t set = __ballot_sync(0xffffffffu, digit >> b & 1);
        same &= digit >> b & 1 ? set : ~set;
    }
    return same;
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortParams a) {
    extern __shared__ uint32_t s_count[];
    const int bins = 1 << a.bits;
    for (int i = threadIdx.x; i < bins; i += kSortThreads) s_count[i] = 0;
    __syncthreads();
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.tile;
    const int64_t hi = lo + a.tile < a.n ? lo + a.tile : a.n;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kSortThreads + threadIdx.x; i < a.clear_n;
         i += static_cast<int64_t>(gridDim.x) * kSortThreads)
        a.clear[i] = 0;
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
#pragma unroll
        for (int k = 0; k < 1 << (kMaxDigit - 10); ++k) {
            if (k >= per) break;
            const uint32_t* const c = a.counts + tid * per + k;
#pragma unroll 16
            for (int t = 0; t < a.tiles; ++t) {
                const uint32_t n = c[t * bins];
                total[k] += n;
                if (t < static_cast<int>(blockIdx.x)) earlier[k] += n;
            }
            sum += total[k];
        }
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
        const uint32_t same = lanes_with(digit, a.bits, have);
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

// Up to kRankSort tokens: a token's place is the number of keys below its own,
// and of equal ones before it, counted by kPerKey threads per token over all
// keys in shared memory. No passes and no barriers between CTAs.
// us for the whole call of 2048 tokens (1024 columns), 4096, 6000 and 8192 (512
// columns) into 8192 rows so: 14.4, 18.2, 28.9, 35.2; sorted by a cluster: 18.3, 18.8,
// 19.5, 21.6 (the comparisons grow with the square).
constexpr int kRankThreads = 512;
constexpr int64_t kRankSort = 4096;

template <int kPerKey> __global__ void __launch_bounds__(kRankThreads) sort_rank_kernel(const SortParams a) {
    extern __shared__ uint4 s_keys4[];
    uint32_t* const s_keys = reinterpret_cast<uint32_t*>(s_keys4);
    const int tid = threadIdx.x, n = static_cast<int>(a.n), groups = (n + 3) / 4;
    launch_next();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRankThreads + tid; i < a.clear_n;
         i += static_cast<int64_t>(gridDim.x) * kRankThreads)
        a.clear[i] = 0;
#pragma unroll 8
    for (int i = tid; i < 4 * groups; i += kRankThreads) s_keys[i] = i < n ? sort_key(a, i) : 0xffffffffu;
    __syncthreads();
    const int i = blockIdx.x * (kRankThreads / kPerKey) + tid / kPerKey;
    const uint32_t key = i < n ? s_keys[i] : 0;
    int below = 0;
#pragma unroll 4
    for (int g = tid % kPerKey; g < groups; g += kPerKey) {
        const uint4 k = s_keys4[g];
        const int j = 4 * g;
        below += (k.x < key + (j < i)) + (k.y < key + (j + 1 < i)) + (k.z < key + (j + 2 < i)) + (k.w < key + (j + 3 < i));
    }
#pragma unroll
    for (int o = kPerKey / 2; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
    if (i < n && tid % kPerKey == 0) {
        a.keys_out[below] = key;
        a.tokens_out[below] = static_cast<uint32_t>(i);
    }
}

// More, up to kClusterSort, are sorted by one thread-block cluster (one
// launch; the tiles take two per digit). A warp owns 32 kItems consecutive
// items and ranks them 32 at a time with masks and counts of its own; the
// CTAs read each other's totals through distributed shared memory and send
// every item to the CTA that holds its place.
constexpr int kSortCluster = 16;
constexpr int kClusterThreads = 512;
constexpr int kClusterWarps = kClusterThreads / 32;
// Items per CTA until the cluster is full. us for the whole call of 4097, 8192, 10007,
// 16384 and 32768 tokens of 64 bf16 columns into 32768 fp32 rows, with 512: 18.8, 19.9,
// 20.8, 24.7, 28.6; 1024: 17.6, 19.2, 20.8, 24.7, 28.6; 2048: 17.6, 19.9, 19.9, 24.4, 28.6;
// 4096: 21.2, 24.0, 23.9, 28.5, 33.9.
constexpr int kClusterShare = 2048;
constexpr int kMaxShare = 8192;      // 16-bit counts, and room in shared memory
constexpr int64_t kClusterSort = int64_t{kSortCluster} * kMaxShare;

struct ClusterSortParams {
    SortParams s;  // ids, keys_out, tokens_out, n, bits, vocab, id_bits
    int32_t share;  // items per CTA
    int32_t passes, cluster;
};

// 16 bytes of the same shared-memory variable of CTA `rank`.
__device__ __forceinline__ uint4 load_remote(const void* local, uint32_t rank) {
    uint32_t addr;
    uint4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

template <int kItems> __global__ void __launch_bounds__(kClusterThreads) sort_cluster_kernel(const ClusterSortParams a) {
    extern __shared__ uint64_t s_item[];  // [share] key << 32 | token, then the counts
    __shared__ uint32_t s_scan[kClusterWarps];
    const int bins = 1 << a.s.bits, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int csize = a.cluster, rank = static_cast<int>(cluster_rank());
    // counts are 16-bit: a CTA has at most 8192 items
    uint16_t* const s_total = reinterpret_cast<uint16_t*>(s_item + (a.share + 1) / 2 * 2);  // [bins] this CTA's counts
    uint16_t* const s_counts = s_total + bins;                                             // [warps][bins]
    uint32_t* const s_place = reinterpret_cast<uint32_t*>(s_counts + kClusterWarps * bins);   // [bins] places of its first items
    uint16_t* const s_warp = s_counts + warp * bins;
    const int64_t base = static_cast<int64_t>(rank) * a.share;
    const int count = static_cast<int>(a.s.n - base < a.share ? (a.s.n > base ? a.s.n - base : 0) : a.share);
    const int mine = warp * 32 * kItems + lane;  // item i of this thread: mine + 32 i

    launch_next();
    for (int64_t i = static_cast<int64_t>(rank) * kClusterThreads + tid; i < a.s.clear_n; i += csize * kClusterThreads)
        a.s.clear[i] = 0;
    uint64_t item[kItems];  // key << 32 | token
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int at = mine + 32 * i;
        item[i] = at < count ? static_cast<uint64_t>(sort_key(a.s, base + at)) << 32 | static_cast<uint32_t>(base + at) : 0;
    }
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * a.s.bits;
        if (pass > 0) {
#pragma unroll
            for (int i = 0; i < kItems; ++i)
                if (mine + 32 * i < count) item[i] = s_item[mine + 32 * i];
        }
        // ranks inside the warp's items
        for (int d = lane; d < bins / 2; d += 32) reinterpret_cast<uint32_t*>(s_warp)[d] = 0;
        __syncwarp();
        uint32_t below[kItems];
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const bool have = mine + 32 * i < count;
            const uint32_t digit = static_cast<uint32_t>(item[i] >> (32 + shift)) & (bins - 1);
            const uint32_t same = lanes_with(digit, a.s.bits, have);
            const uint32_t before = have ? s_warp[digit] : 0, ahead = __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (have && ahead == 0) s_warp[digit] = static_cast<uint16_t>(before + __popc(same));
            __syncwarp();
            below[i] = before + ahead;
        }
        __syncthreads();
        // the warps' counts become the counts of the warps before, two digits
        // per thread
        for (int d = tid; d < bins / 2; d += kClusterThreads) {
            uint32_t* const c = reinterpret_cast<uint32_t*>(s_counts) + d;
            uint32_t n[kClusterWarps], run = 0;
#pragma unroll
            for (int w = 0; w < kClusterWarps; ++w) n[w] = c[w * (bins / 2)];
#pragma unroll
            for (int w = 0; w < kClusterWarps; ++w) {
                c[w * (bins / 2)] = run;
                run += n[w];
            }
            reinterpret_cast<uint32_t*>(s_total)[d] = run;
        }
        cluster_sync_all();
        // places: items with a lower digit, then those of the CTAs before.
        // A thread takes eight digits.
        uint32_t all[8] = {}, earlier[8] = {}, sum = 0;
        if (tid < bins / 8) {
#pragma unroll 8
            for (int i = 0; i < csize; ++i) {
                // each CTA begins with itself: a CTA answers one at a time
                const int c = (rank + i) & (csize - 1);
                const uint4 v = load_remote(s_total + 8 * tid, c);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t n = k % 2 ? w[k / 2] >> 16 : w[k / 2] & 0xffffu;
                    all[k] += n;
                    if (c < rank) earlier[k] += n;
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += all[k];
        }
        const uint32_t scan = warp_scan_inclusive(sum, lane);
        if (lane == 31) s_scan[warp] = scan;
        __syncthreads();
        uint32_t lower = warp_sum(lane < warp ? s_scan[lane] : 0u) + scan - sum;
        if (tid < bins / 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s_place[8 * tid + k] = lower + earlier[k];
                lower += all[k];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            if (mine + 32 * i >= count) continue;
            const uint32_t digit = static_cast<uint32_t>(item[i] >> (32 + shift)) & (bins - 1);
            const uint32_t to = s_place[digit] + s_warp[digit] + below[i];
            if (pass + 1 == a.passes) {
                a.s.keys_out[to] = static_cast<uint32_t>(item[i] >> 32);
                a.s.tokens_out[to] = static_cast<uint32_t>(item[i]);
            } else {
                store_remote(&s_item[to % a.share], to / a.share, item[i]);
            }
        }
        // all items sent and all totals read (the last pass reads totals too:
        // no CTA may leave while another reads its shared memory)
        cluster_sync_all();
    }
}

// ------------------------------------------------------------- the sums

constexpr int kSumThreads = 256;
constexpr int kMinColumns = 32;  // threads of a piece, at least: a warp has one piece
constexpr int64_t kZeroBytes = 65536;  // of the table per zeroing CTA, about
constexpr int kMaxZeroRows = 1024;

struct GradParams {
    const void* grad;
    void* table;
    const uint32_t* keys;  // sorted
    const uint32_t* tokens;
    float* partial;               // [pieces][2][width]
    unsigned long long* arrived;  // [pieces][across], 0 at the start
    int64_t n, pieces, grad_stride, table_stride;
    int64_t sum_blocks;  // the CTAs after these zero rows
    int32_t width, vocab, piece_bits, zero_rows;
    uint32_t columns, across;  // threads along the columns, CTAs along a row
    uint32_t zero_across;      // threads along a row that is zeroed
    float scale;
    bool accumulate;
};

// The number of sorted tokens with a key below `key`, by one warp: each step
// takes 32 probes.
__device__ __forceinline__ int64_t count_below(const GradParams& a, uint32_t key, int lane) {
    int64_t lo = 0, n = a.n;  // the answer is in [lo, lo + n]
    while (n > 0) {
        const int64_t step = (n + 31) / 32, at = lane * step;
        const bool below = at < n && a.keys[lo + at] < key;
        const int hit = __popc(__ballot_sync(0xffffffffu, below));
        if (hit == 0) return lo;
        const int64_t skip = (hit - 1) * step + 1;
        lo += skip;
        n = min(step - 1, n - skip);
    }
    return lo;
}

template <typename G, int kVec> struct Row;  // kVec elements in flight
template <typename G> struct Row<G, 8> {
    Raw8<G> raw;
    __device__ __forceinline__ void load(const G* p) { raw.load(p); }
    __device__ __forceinline__ void unpack(float (&v)[8]) const { raw.unpack(v); }
};
template <typename G> struct Row<G, 1> {
    G raw;
    __device__ __forceinline__ void load(const G* p) { raw = *p; }
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

// Partial sums, handed on between CTAs of one launch through L2.
template <int kVec> __device__ __forceinline__ void store_partial(float* p, const float (&v)[kVec]) {
    if constexpr (kVec == 8) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *p = v[0];
    }
}

template <int kVec> __device__ __forceinline__ void load_partial(const float* p, float (&v)[kVec]) {
    if constexpr (kVec == 8) {
        const float4 lo = __ldcg(reinterpret_cast<const float4*>(p)), hi = __ldcg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
    } else {
        v[0] = __ldcg(p);
    }
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// The finished row of an id: scaled, added to what the table holds where
// the call accumulates, rounded once.
template <typename T, int kVec>
__device__ __forceinline__ void write_row(const GradParams& a, uint32_t key, int col, const float (&sum)[kVec]) {
    T* const p = static_cast<T*>(a.table) + static_cast<int64_t>(key) * a.table_stride + col;
    float v[kVec] = {};
    if (a.accumulate) {
        if constexpr (kVec == 8) {
            Raw8<T> old;
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) old.w[i] = reinterpret_cast<const uint4*>(p)[i];
            old.unpack(v);
        } else {
            v[0] = to_f(*p);
        }
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = a.accumulate ? v[i] + sum[i] * a.scale : sum[i] * a.scale;
    store_row<T, kVec>(p, v);
}

// n elements from p on by `threads` threads (8 at least), in 16-byte stores
// between the ragged ends.
template <typename T> __device__ __forceinline__ void zero_range(T* p, int64_t n, int thread, int threads) {
    constexpr int kPer = 16 / sizeof(T);
    int64_t lead = static_cast<int64_t>((-reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    lead = lead < n ? lead : n;
    const int64_t words = (n - lead) / kPer, done = lead + words * kPer;
    if (thread < lead) p[thread] = from_f<T>(0.0f);
    if (thread < n - done) p[done + thread] = from_f<T>(0.0f);
    uint4* const w = reinterpret_cast<uint4*>(p + lead);
    for (int64_t i = thread; i < words; i += threads) __stcs(w + i, make_uint4(0, 0, 0, 0));
}

template <typename T> __device__ __forceinline__ void zero_rows(const GradParams& a, int64_t block) {
    __shared__ bool s_touched[kMaxZeroRows];
    __shared__ int64_t s_range[2];
    const int64_t v0 = block * a.zero_rows;
    const int n = static_cast<int>(v0 + a.zero_rows < a.vocab ? a.zero_rows : a.vocab - v0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int r = threadIdx.x; r < n; r += kSumThreads) s_touched[r] = false;
    if (warp < 2) {
        const int64_t at = count_below(a, static_cast<uint32_t>(v0 + warp * n), lane);
        if (lane == 0) s_range[warp] = at;
    }
    __syncthreads();
    for (int64_t p = s_range[0] + threadIdx.x; p < s_range[1]; p += kSumThreads) s_touched[a.keys[p] - v0] = true;
    __syncthreads();
    T* const table = static_cast<T*>(a.table) + v0 * a.table_stride;
    constexpr int kPer = 16 / sizeof(T);
    const uint4 zeros = make_uint4(0, 0, 0, 0);
    if (a.table_stride != a.width || a.width < kPer) {
        // rows apart from each other (or very short): some threads for each
        const int tx = threadIdx.x % a.zero_across, ny = kSumThreads / a.zero_across;
        for (int r = threadIdx.x / a.zero_across; r < n; r += ny)
            if (!s_touched[r]) zero_range(table + r * a.table_stride, a.width, tx, a.zero_across);
        return;
    }
    // Rows that follow each other: the 16-byte words of all of them in one loop.
    // A word belongs to the row(s) of its first and last element; the quotients
    // are exact below 2^21 elements.
    const float inv = 1.0f / static_cast<float>(a.width);
    const auto row_of = [&](int element) { return static_cast<int>((static_cast<float>(element) + 0.5f) * inv); };
    const int total = n * a.width;
    if (a.width % kPer == 0 && (reinterpret_cast<uintptr_t>(table) & 15) == 0) {
#pragma unroll 4
        for (int e = threadIdx.x * kPer; e < total; e += kSumThreads * kPer)
            if (!s_touched[row_of(e)]) __stcs(reinterpret_cast<uint4*>(table + e), zeros);
        return;
    }
    const int lead = static_cast<int>((-reinterpret_cast<uintptr_t>(table) & 15) / sizeof(T));
    const int done = lead + (total - lead) / kPer * kPer;
#pragma unroll 4
    for (int e = lead + threadIdx.x * kPer; e < done; e += kSumThreads * kPer) {
        const int last = row_of(e + kPer - 1), first = row_of(e);
        const bool head = !s_touched[first], tail = !s_touched[last];
        if (head && tail) {
            __stcs(reinterpret_cast<uint4*>(table + e), zeros);
        } else if (head || tail) {
            const int border = last * a.width;  // the last row's first element
            for (int i = head ? e : border; i < (head ? border : e + kPer); ++i) table[i] = from_f<T>(0.0f);
        }
    }
    // the elements before the first word, and after the last one
    const int edge = threadIdx.x < lead ? threadIdx.x : done + threadIdx.x - lead;
    if (edge < total && !s_touched[row_of(edge)]) table[edge] = from_f<T>(0.0f);
}

// One piece's tokens, summed by its threads. head: its first id began in an
// earlier piece; on: its last id goes on in the next one.
template <typename G, typename T, int kVec>
__device__ __forceinline__ void sum_piece(const GradParams& a, const uint32_t* keys, const uint32_t* tokens, int len,
                                          int64_t piece, int col, bool head, bool on) {
    constexpr int kAhead = kVec == 8 && sizeof(G) == 4 ? 4 : 8;  // rows a thread has in flight
    const uint32_t none = static_cast<uint32_t>(a.vocab);
    const G* const grad = static_cast<const G*>(a.grad) + col;
    float* const partial = a.partial + piece * 2 * a.width + col;
    float acc[kVec] = {};
    uint32_t cur = keys[0];
    for (int p = 0; p < len; p += kAhead) {
        Row<G, kVec> row[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (p + k >= len || keys[p + k] == none) continue;
            row[k].load(grad + static_cast<int64_t>(tokens[p + k]) * a.grad_stride);
            // the table's row that the id's sum will be added to (32768 x
            // 2048 into 262144 rows 86.5 -> 81.9 us)
            if (kVec == 8 && a.accumulate && (p + k + 1 == len || keys[p + k + 1] != keys[p + k]))
                prefetch_l2(static_cast<const T*>(a.table) + static_cast<int64_t>(keys[p + k]) * a.table_stride + col);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (p + k >= len) break;
            const uint32_t key = keys[p + k];
            if (key != cur) {
                if (head) store_partial<kVec>(partial, acc);
                else write_row<T, kVec>(a, cur, col, acc);
#pragma unroll
                for (int i = 0; i < kVec; ++i) acc[i] = 0.0f;
                cur = key;
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
    if (head) store_partial<kVec>(partial, acc);
    else if (on) store_partial<kVec>(partial + a.width, acc);
    else write_row<T, kVec>(a, cur, col, acc);
}

// An id that crosses borders: the partial sums of the pieces start ..
// start + n - 1, added in order.
template <typename T, int kVec>
__device__ __forceinline__ void join_pieces(const GradParams& a, uint32_t key, int64_t start, int n, int col) {
    constexpr int kAhead = kVec == 8 ? 4 : 8;
    const float* p = a.partial + start * 2 * a.width + a.width + col;  // the piece where it begins
    float acc[kVec];
    load_partial<kVec>(p, acc);
    p += a.width;  // the others' first ids
    for (int q = 1; q < n; q += kAhead) {
        float v[kAhead][kVec];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (q + k < n) load_partial<kVec>(p + static_cast<int64_t>(k) * 2 * a.width, v[k]);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (q + k >= n) break;
#pragma unroll
            for (int i = 0; i < kVec; ++i) acc[i] += v[k][i];
        }
        p += static_cast<int64_t>(kAhead) * 2 * a.width;
    }
    write_row<T, kVec>(a, key, col, acc);
}

// CTAs per SM that registers are held to. With one element per access 8 take 75.8 us
// for 10007 x 1283, 6 77.8, 5 and 4 80.0: more rows in flight are worth the 60 bytes
// per thread that 32 registers spill. With eight 4 take 317 us for 32768 x 2048 (82.2
// accumulating; 12 to 40 bytes spilled), 3 318 (83.8), 5 336 (105.7) and 2 350 (89.1).
template <typename G, typename T, int kVec>
__global__ void __launch_bounds__(kSumThreads, kVec == 1 ? 8 : 4) grad_sum_kernel(const GradParams a) {
    extern __shared__ uint32_t s_list[];  // keys, then tokens of the CTA's pieces
    __shared__ int64_t s_start[kSumThreads / kMinColumns][2];
    __shared__ int s_parts[kSumThreads / kMinColumns][2];
    wait_for_previous();
    if (blockIdx.x >= a.sum_blocks) {
        zero_rows<T>(a, blockIdx.x - a.sum_blocks);
        return;
    }
    const int tx = threadIdx.x % a.columns, ty = threadIdx.x / a.columns;
    const int per_cta = kSumThreads / a.columns;
    const uint32_t slab = blockIdx.x % a.across;
    const int64_t piece0 = static_cast<int64_t>(blockIdx.x / a.across) * per_cta, piece = piece0 + ty;
    const int col = static_cast<int>(slab * a.columns + tx) * kVec;
    const uint32_t none = static_cast<uint32_t>(a.vocab);
    const int listed = per_cta << a.piece_bits;
    for (int i = threadIdx.x; i < listed; i += kSumThreads) {
        const int64_t p = (piece0 << a.piece_bits) + i;
        s_list[i] = p < a.n ? a.keys[p] : none;
        s_list[listed + i] = p < a.n ? a.tokens[p] : 0;
    }
    __syncthreads();
    const bool have = piece < a.pieces;
    const int64_t p0 = piece << a.piece_bits;
    const int len = !have ? 0 : a.n - p0 < 1 << a.piece_bits ? static_cast<int>(a.n - p0) : 1 << a.piece_bits;
    const uint32_t* const keys = s_list + (ty << a.piece_bits);
    const uint32_t first = have ? keys[0] : none, last = have ? keys[len - 1] : none;
    const bool head = first != none && p0 > 0 && a.keys[p0 - 1] == first;
    const bool on = last != none && p0 + len < a.n && a.keys[p0 + len] == last;
    if (have && col < a.width) sum_piece<G, T, kVec>(a, keys, keys + listed, len, piece, col, head, on);

    // Ids that cross borders. Every piece with a part of such an id counts
    // itself in at the piece where the id begins, and the one where it ends
    // says how many there are: whoever makes the count whole adds the parts
    // up, in their order. Nobody waits.
    if (!__syncthreads_or(head || on)) return;
    const bool through = head && on && first == last;
    if (tx < 32) {  // the piece's first warp
        const int lane = threadIdx.x & 31;
        const int64_t start = head ? count_below(a, first, lane) >> a.piece_bits : 0;
        if (lane < 2) {
            const bool mine = lane == 0 ? head : on && !through;
            const int64_t at = lane == 0 ? start : piece;
            int parts = 0;
            if (mine) {
                unsigned long long add = 1;
                if (lane == 0 && !through) add |= static_cast<unsigned long long>(piece - start + 1) << 32;
                __threadfence();
                const unsigned long long now = atomicAdd(a.arrived + at * a.across + slab, add) + add;
                if (now >> 32 == (now & 0xffffffffu)) parts = static_cast<int>(now >> 32);
                __threadfence();
            }
            s_start[ty][lane] = at;
            s_parts[ty][lane] = parts;
        }
    }
    __syncthreads();
    if (col >= a.width) return;
    for (int side = 0; side < 2; ++side)
        if (s_parts[ty][side]) join_pieces<T, kVec>(a, side ? last : first, s_start[ty][side], s_parts[ty][side], col);
}

// ------------------------------------------------------------- the call

size_t rounded(size_t bytes) { return (bytes + kWorkspaceAlign - 1) / kWorkspaceAlign * kWorkspaceAlign; }

// Sorted tokens per piece, a power of two: short pieces spread few tokens over
// the GPU, long ones leave fewer partial sums of a frequent id.
int32_t piece_bits_of(int64_t n) { return n <= 4096 ? 3 : n <= 16384 ? 4 : n <= 65536 ? 5 : n <= 262144 ? 6 : 7; }
int64_t pieces_of(int64_t n) { return ceil_div(n, int64_t{1} << piece_bits_of(n)); }

struct SortPlan {
    int passes, bits;
    int32_t tile, tiles;    // where the tiles sort
    int32_t cluster, share; // where a cluster does (cluster > 0)
    bool ranks;             // where every token is ranked by itself
    static SortPlan of(int64_t n, int64_t vocab) {
        int key = 1;
        while ((int64_t{1} << key) <= vocab) ++key;  // keys are 0 .. vocab
        SortPlan s;
        s.passes = key <= kMaxDigit ? 1 : 2;
        s.bits = (key + s.passes - 1) / s.passes;
        if (s.bits < 4) s.bits = 4;  // eight digits are one 16-byte word
        s.cluster = 0;
        s.share = 0;
        s.ranks = n <= kRankSort;
        if (!s.ranks && n <= kClusterSort) {
            s.cluster = 2;
            while (s.cluster < kSortCluster && n > int64_t{kClusterShare} * s.cluster) s.cluster *= 2;
            s.share = static_cast<int32_t>(ceil_div(n, s.cluster));
        }
        const int64_t tiles = ceil_div(n, kSortThreads) < kSortTiles ? ceil_div(n, kSortThreads) : kSortTiles;
        s.tile = static_cast<int32_t>(ceil_div(ceil_div(n, tiles), kSortThreads) * kSortThreads);
        s.tiles = static_cast<int32_t>(ceil_div(n, s.tile));
        return s;
    }
};

struct Workspace {
    uint32_t *keys[2], *tokens[2], *counts, *sorted_keys, *sorted_tokens;
    float* partial;
    unsigned long long* arrived;
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
        const int copies = s.ranks || s.cluster ? 1 : s.passes;
        for (int i = 0; i < copies; ++i) {
            w.keys[i] = reinterpret_cast<uint32_t*>(take(static_cast<size_t>(n) * 4));
            w.tokens[i] = reinterpret_cast<uint32_t*>(take(static_cast<size_t>(n) * 4));
        }
        w.sorted_keys = w.keys[copies - 1];
        w.sorted_tokens = w.tokens[copies - 1];
        if (!s.ranks && !s.cluster) w.counts = reinterpret_cast<uint32_t*>(take((static_cast<size_t>(s.tiles) << s.bits) * 4));
        const size_t pieces = static_cast<size_t>(pieces_of(n));
        w.partial = reinterpret_cast<float*>(take(pieces * 2 * width * 4));
        // a CTA has 256 columns of a piece at least, or all of them
        w.arrived = reinterpret_cast<unsigned long long*>(take(pieces * ceil_div(width, kSumThreads) * 8));
        w.bytes = at;
        return w;
    }
};

template <int kItems> drs_status launch_cluster_sort(const ClusterSortParams& a, cudaStream_t stream) {
    const size_t bins = size_t{1} << a.s.bits;
    const size_t smem = static_cast<size_t>(a.share + 1) * 8 + bins * (2 + 2 * kClusterWarps + 4);
    const auto kernel = sort_cluster_kernel<kItems>;
    if (!prepare_kernel(reinterpret_cast<const void*>(kernel), smem, a.cluster > 8)) return DRS_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.cluster));
    cfg.blockDim = dim3(kClusterThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(a.cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, a));
}

drs_status sort_tokens(const SortPlan& s, const Workspace& w, const void* ids, int id_bits, int64_t n, int64_t vocab,
                       int64_t counters, cudaStream_t stream) {
    if (s.ranks) {
        SortParams a{};
        a.ids = ids;
        a.keys_out = w.sorted_keys;
        a.tokens_out = w.sorted_tokens;
        a.clear = w.arrived;
        a.n = n;
        a.clear_n = counters;
        a.vocab = static_cast<int32_t>(vocab);
        a.id_bits = id_bits;
        const size_t smem = static_cast<size_t>(ceil_div(n, 4)) * 16;
        // at most 128 CTAs
        if (n <= 2048)
            sort_rank_kernel<32><<<static_cast<unsigned>(ceil_div(n, kRankThreads / 32)), kRankThreads, smem, stream>>>(a);
        else
            sort_rank_kernel<16><<<static_cast<unsigned>(ceil_div(n, kRankThreads / 16)), kRankThreads, smem, stream>>>(a);
        return cuda_status(cudaGetLastError());
    }
    if (s.cluster) {
        ClusterSortParams a{};
        a.s.ids = ids;
        a.s.keys_out = w.sorted_keys;
        a.s.tokens_out = w.sorted_tokens;
        a.s.n = n;
        a.s.clear = w.arrived;
        a.s.clear_n = counters;
        a.s.bits = s.bits;
        a.s.vocab = static_cast<int32_t>(vocab);
        a.s.id_bits = id_bits;
        a.share = s.share;
        a.passes = s.passes;
        a.cluster = s.cluster;
        constexpr int kFew = kClusterShare / kClusterThreads;
        if (s.share <= kClusterShare) return launch_cluster_sort<kFew>(a, stream);
        if (s.share <= 2 * kClusterShare) return launch_cluster_sort<2 * kFew>(a, stream);
        return launch_cluster_sort<4 * kFew>(a, stream);
    }
    const size_t bins = size_t{1} << s.bits;
    const size_t count_smem = bins * 4, place_smem = bins * 4 + bins * 2 * kSortWarps;
    if (!prepare_kernel(reinterpret_cast<const void*>(sort_place_kernel), place_smem, false)) return DRS_ERR_CUDA;
    for (int pass = 0; pass < s.passes; ++pass) {
        SortParams a{};
        a.ids = ids;
        a.keys_in = pass ? w.keys[0] : nullptr;
        a.tokens_in = pass ? w.tokens[0] : nullptr;
        a.keys_out = w.keys[pass];
        a.tokens_out = w.tokens[pass];
        a.counts = w.counts;
        a.n = n;
        a.clear = w.arrived;
        a.clear_n = pass == 0 ? counters : 0;
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

// Threads of a CTA along the columns, CTAs along a row, and of all pieces.
void lay_out(GradParams& a, int vec) {
    int x = kMinColumns;
    while (x < kSumThreads && int64_t{x} * vec < a.width) x *= 2;
    a.columns = x;
    a.across = static_cast<uint32_t>(ceil_div(a.width, int64_t{x} * vec));
    a.sum_blocks = ceil_div(a.pieces, kSumThreads / x) * a.across;
}

template <typename G, typename T, int kVec> drs_status launch_sums(GradParams a, cudaStream_t stream) {
    const int sms = sm_count();
    if (sms <= 0) return DRS_ERR_CUDA;
    int64_t zero_blocks = 0;
    if (!a.accumulate) {
        // us with 64 KB, 256 KB and 1 MB per CTA: 32768 x 2048 bf16 into 262144
        // fp32 rows 317, 323, 337; 10007 x 1283 fp32 into 131072 bf16 rows 75.8,
        // 85.8, 86.3. Fewer rows where that would leave SMs idle.
        int64_t rows = kZeroBytes / (static_cast<int64_t>(a.width) * sizeof(T));
        const int64_t even = ceil_div(a.vocab, sms * 8);
        rows = rows < even ? rows : even;
        a.zero_rows = static_cast<int32_t>(rows < 1 ? 1 : rows > kMaxZeroRows ? kMaxZeroRows : rows);
        zero_blocks = ceil_div(a.vocab, a.zero_rows);
        a.zero_across = 8;
        while (a.zero_across < kSumThreads && a.zero_across * 16 < a.width * sizeof(T)) a.zero_across *= 2;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.sum_blocks + zero_blocks));
    cfg.blockDim = dim3(kSumThreads);
    cfg.dynamicSmemBytes = (static_cast<size_t>(kSumThreads / a.columns) << a.piece_bits) * 8;
    cfg.stream = stream;
    cudaLaunchAttribute dependent[1];
    dependent[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    dependent[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = dependent;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, grad_sum_kernel<G, T, kVec>, a));
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
    a.grad = grad_out;
    a.table = grad_table;
    a.n = tokens;
    a.grad_stride = grad_stride;
    a.table_stride = table_stride;
    a.width = static_cast<int32_t>(width);
    a.vocab = static_cast<int32_t>(vocab);
    a.scale = scale;
    a.accumulate = accumulate != 0;
    const bool vec = width % 8 == 0 && aligned(grad_out, 16) && aligned(grad_table, 16) &&
                     grad_stride * dtype_bytes(grad_dtype) % 16 == 0 &&
                     table_stride * dtype_bytes(table_dtype) % 16 == 0;
    // Single elements per access: pieces twice as long (10007 x 1283 fp32 81.1 ->
    // 75.6 us; 32768 x 64 in eights 29.5 -> 35.8, so not there).
    a.piece_bits = piece_bits_of(tokens) + (vec || tokens <= 4096 ? 0 : 1);
    a.pieces = ceil_div(tokens, int64_t{1} << a.piece_bits);
    lay_out(a, vec ? 8 : 1);
    if (a.sum_blocks + vocab > INT_MAX) return DRS_ERR_UNSUPPORTED;
    if (tokens > 0) {
        const SortPlan s = SortPlan::of(tokens, vocab);
        const Workspace w = Workspace::of(workspace, tokens, vocab, width);
        const drs_status status = sort_tokens(s, w, ids, id_bits, tokens, vocab, a.pieces * a.across, st);
        if (status != DRS_OK) return status;
        a.keys = w.sorted_keys;
        a.tokens = w.sorted_tokens;
        a.partial = w.partial;
        a.arrived = w.arrived;
    }
    return with_dtype(grad_dtype, [&](auto g) -> drs_status {
        return with_dtype(table_dtype, [&](auto t) -> drs_status {
            return vec ? launch_sums<decltype(g), decltype(t), 8>(a, st)
                       : launch_sums<decltype(g), decltype(t), 1>(a, st);
        });
    });
}

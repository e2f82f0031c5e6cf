// logprobs.cu -- log probabilities of given tokens with entropy, rank and top
// alternatives (drs_token_logprobs).
//
// With c = log2(e) / T and t_j = (x_j - M) c for any reference M:
//   S = sum 2^t_j, W = sum 2^t_j t_j
//   ln of the softmax's denominator relative to M: ln S
//   entropy = ln 2 (log2 S - W / S)
//   rank    = 1 + the number of x_j > x_id
// M is a warp's running reference, raised when a segment's largest logit
// passes it by more than 2^8 in the exponent; S and W then move along:
// S' = 2^d S, W' = 2^d (W + d S) with d = (M - M') c.
//
// One read of the row. Warps take blocks of two (fp32: one) segments of 256
// columns and keep each segment's largest logit in shared memory. The k
// largest logits lie in the k segments whose largest logits come first (by
// value, then by column): any logit of another segment has k before it, one in
// each of these. So only k segments are looked at again, from L2, and of these
// only what reaches the k-th segment's largest.
//
// Many rows: a team of 1 to 8 warps, a CTA, takes rows in turn; its next blocks,
// the next row's among them, come by asynchronous copies while it computes.
// Few rows: a cluster of up to 16 CTAs takes a row and its first CTA selects.
//
// Bound by memory for large batches, by instructions close behind: 16-bit rows
// take about 8 issued per column (an exponential, a product and three sums
// each), and 24 warps of 80 registers per SM do better than 32 of 64 (4096 x
// 262144 bf16 rows with 20 alternatives 329 us against 416). Measured: these
// 329 us, 6.4 TB/s (315, 6.7 TB/s, without alternatives); 256 x 262144 fp32 46 us,
// 5.7 TB/s; 1003 x 50001 fp16 with 5 alternatives 27 us, of which the rows' reading
// takes 15 to 20, the rest the launch, the first loads and the selection; one row
// of 262144 bf16 6.5 us with 20 alternatives, 3.9 without: launch, the read's
// latency, a cluster's barrier.
#include <algorithm>
#include <climits>

#include "token_common.cuh"

namespace drs {
namespace {

constexpr int kResident = 24;  // warps per SM
constexpr int kMaxRowCluster = 16;
constexpr int kListed = 256;       // candidates of the short way
constexpr int kSegment = 256;      // columns whose largest is kept: eight per lane of a warp
constexpr int kBlockBytes = 1024;  // what a warp takes at once: two 16-byte words per lane
// Blocks on their way to a warp. us with 2, 3, 4, 5 and 6: 4096 x 262144 bf16 rows with 20 alternatives 354, 334, 329, 332,
// 333, 2432 without alternatives 206, 195, 190, 194, 194; 256 x 262144 fp32 55.9, 48.6, 46.3, 45.6, 45.5; 1003 x 50001
// fp16 with 5 29.0, 27.0, 26.6, 27.5, 27.8; 4096 x 8192 fp32 46.5, 43.4, 41.6, 47.5, 47.2 (larger rings leave room for
// fewer teams).
constexpr int kDepth = 4;
// Exponents (base 2) below this give 0; held there so that 0 times an
// infinite exponent does not arise in W.
constexpr float kLeastExponent = -200.0f;
constexpr float kSlack = 8.0f;  // exponents above the reference before it moves

// Bytes that a warp of a team looks at again at once: four segments, two of fp32 in small teams, whose memory counts.
__host__ __device__ constexpr int stage_bytes(int warps, int element) { return element == 4 && warps >= 4 ? 4096 : 2048; }

// Segments in a block, and its columns.
template <typename T> constexpr int kParts = sizeof(T) == 2 ? 2 : 1;
template <typename T> constexpr int kBlock = kSegment * kParts<T>;

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
    int64_t rows, row_stride, canvas_len;
    int32_t vocab, k, id_bits;
    int32_t blocks, cluster, part;  // blocks: of a row, at most; part: of them a CTA's
};

// ------------------------------------------------------------- elements

// 2^x, results below the normal range 0: one instruction (ex2_approx takes
// four), in sums of terms relative to their largest.
__device__ __forceinline__ float ex2_flushed(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The largest of eight elements (NaN left out), and how many exceed a value. 16-bit elements are compared in
// pairs, whose results 0 or 0xFFFF in each half are added up as one number: with n_low and n_high of
// them it is 65536 (n_low - n_high) - n_low modulo 2^32, and holds up to 65535 of each.
template <typename T> struct Eight;
template <> struct Eight<float> {
    __device__ static float largest(const Raw8<float>& r) {
        float v[8];
        r.unpack(v);
        return fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
    }
    __device__ static void count(const Raw8<float>& r, float own, uint32_t& n) {
        float v[8];
        r.unpack(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) n += v[e] > own ? 1 : 0;
    }
    __device__ static int total(uint32_t n) { return static_cast<int>(n); }
};
template <typename T, typename T2> struct EightHalves {
    __device__ static T2 pair(uint32_t w) { return *reinterpret_cast<const T2*>(&w); }
    __device__ static float largest(const Raw8<T>& r) {
        const T2 m = __hmax2(__hmax2(pair(r.w[0].x), pair(r.w[0].y)), __hmax2(pair(r.w[0].z), pair(r.w[0].w)));
        return fmaxf(to_f(m.x), to_f(m.y));
    }
    __device__ static void count(const Raw8<T>& r, T own, uint32_t& n) {
        T2 o;
        o.x = o.y = own;
        n += __hgt2_mask(pair(r.w[0].x), o) + __hgt2_mask(pair(r.w[0].y), o);
        n += __hgt2_mask(pair(r.w[0].z), o) + __hgt2_mask(pair(r.w[0].w), o);
    }
    __device__ static int total(uint32_t n) {
        const uint32_t low = -n & 0xFFFFu;
        return static_cast<int>(low + (low - (n + low >> 16) & 0xFFFFu));
    }
};
template <> struct Eight<__nv_bfloat16> : EightHalves<__nv_bfloat16, __nv_bfloat162> {};
template <> struct Eight<__half> : EightHalves<__half, __half2> {};

template <typename T> __device__ T rounded_down(float v);
template <> __device__ __forceinline__ __nv_bfloat16 rounded_down<__nv_bfloat16>(float v) { return __float2bfloat16_rd(v); }
template <> __device__ __forceinline__ __half rounded_down<__half>(float v) { return __float2half_rd(v); }
template <typename T> __device__ constexpr float largest_finite();
template <> __device__ constexpr float largest_finite<__nv_bfloat16>() { return 0x1.FEp127f; }
template <> __device__ constexpr float largest_finite<__half>() { return 65504.0f; }

// The least logit that is told from smaller ones: it holds exponents at about
// kLeastExponent or below, finite. 16-bit elements are raised to it in pairs, before
// they are taken apart, fp32 exponents one by one.
template <typename T> struct Floor {
    static constexpr bool kPaired = false;
    __device__ bool set(float) { return true; }
    __device__ __forceinline__ const Raw8<T>& raise(const Raw8<T>& r) const { return r; }
};
template <typename T, typename T2> struct FloorHalves {
    static constexpr bool kPaired = true;
    T2 least;
    // false: below the type's range
    __device__ __forceinline__ bool set(float v) {
        least.x = least.y = rounded_down<T>(v);
        return v >= -largest_finite<T>();
    }
    __device__ __forceinline__ Raw8<T> raise(const Raw8<T>& r) const {
        Raw8<T> q;
        q.w[0] = make_uint4(one(r.w[0].x), one(r.w[0].y), one(r.w[0].z), one(r.w[0].w));
        return q;
    }
    __device__ __forceinline__ uint32_t one(uint32_t w) const {
        const T2 v = __hmax2_nan(*reinterpret_cast<const T2*>(&w), least);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
};
template <> struct Floor<__nv_bfloat16> : FloorHalves<__nv_bfloat16, __nv_bfloat162> {};
template <> struct Floor<__half> : FloorHalves<__half, __half2> {};

// A row as a line of aligned units of eight elements: column j stands at
// place j + lead, so that units start on 16-byte boundaries; places outside the
// row count as -inf and are not read.
template <typename T> struct Row {
    const T* first;  // place 0
    int lead, end;   // places of columns 0 and vocab

    __device__ Row(const T* x, int vocab) {
        lead = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
        first = x - lead;
        end = vocab + lead;
    }
    __device__ __forceinline__ bool whole(int place, int n) const { return place >= lead && place + n <= end; }
    __device__ __forceinline__ int blocks() const { return (end + kBlock<T> - 1) / kBlock<T>; }
    // Those wholly inside the row.
    __device__ __forceinline__ int whole_first() const { return lead > 0 ? 1 : 0; }
    __device__ __forceinline__ int whole_end() const { return end / kBlock<T>; }
    // The 16-byte word at a place.
    __device__ __forceinline__ uint4 word(int place) const {
        constexpr int kVec = 16 / sizeof(T);
        if (whole(place, kVec)) return load16_stream(first + place);
        uint4 w;
        T* const e = reinterpret_cast<T*>(&w);
#pragma unroll
        for (int i = 0; i < kVec; ++i) e[i] = place + i >= lead && place + i < end ? first[place + i] : from_f<T>(-INFINITY);
        return w;
    }
    // Eight columns from a place on.
    __device__ __forceinline__ Raw8<T> unit(int place) const {
        Raw8<T> r;
#pragma unroll
        for (int h = 0; h < static_cast<int>(sizeof(T) / 2); ++h) r.w[h] = word(place + 4 * h);
        return r;
    }
};

// ------------------------------------------------------------- keys

// Whole numbers in the order of the values: NaN counts as -inf, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float v) {
    const uint32_t b = __float_as_uint(fmaxf(v, -INFINITY) + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t order) {
    return __uint_as_float(order ^ (order >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

// Larger keys: larger values, then lower places. No key is 0.
__device__ __forceinline__ uint64_t key_of(uint32_t order, int place) {
    return static_cast<uint64_t>(order) << 32 | static_cast<uint32_t>(~place);
}

__device__ __forceinline__ int place_of(uint64_t key) { return static_cast<int>(~static_cast<uint32_t>(key)); }

// ------------------------------------------------------------- asynchronous copies

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// Two words, half a block apart.
__device__ __forceinline__ void copy_halves(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n\tcp.async.cg.shared.global [%0 + %2], [%1 + %2], 16;" ::"r"(to),
                 "l"(from), "n"(kBlockBytes / 2)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory"); }
template <int offset> __device__ __forceinline__ uint4 load_shared16(uint32_t from) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(from), "n"(offset)
                 : "memory");
    return v;
}
__device__ __forceinline__ void store_shared16(uint32_t to, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// The whole blocks of rows on their way to a warp: those first, first + step, ... of a row, and, when all of
// them are on their way, those of the next row. Each turn takes one block and fetches the one kDepth
// further into its slot; a lane reads what it has copied itself.
template <typename T, int kStep> struct Ring {
    uint32_t base, slot = 0;    // this lane's first word; the slot of the next block to take
    const char* from = nullptr;  // this lane's first word of the next block to fetch
    int left = 0;                // blocks to fetch at `from` and after it

    __device__ __forceinline__ explicit Ring(float* memory)
        : base(smem_u32(memory) + (threadIdx.x >> 5) * (kDepth * kBlockBytes) + (threadIdx.x & 31) * 16) {}

    __device__ __forceinline__ void point_at(const Row<T>& row, int first, int count) {
        from = reinterpret_cast<const char*>(row.first) + (first * kBlockBytes + (threadIdx.x & 31) * 16);
        left = count;
    }
    __device__ __forceinline__ void fetch(uint32_t to) {
        if (left > 0) {
            copy_halves(base + to, from);
            from += kStep * kBlockBytes;
            --left;
        }
        copies_commit();
    }
    // The first blocks of a row that nothing has been fetched of.
    __device__ __forceinline__ void fill() {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) fetch((slot + d * kBlockBytes) % (kDepth * kBlockBytes));
    }
    __device__ __forceinline__ void take(uint4 (&w)[2]) {
        copies_wait<kDepth - 1>();
        w[0] = load_shared16<0>(base + slot);
        w[1] = load_shared16<kBlockBytes / 2>(base + slot);
    }
    __device__ __forceinline__ void fetch_next() {
        fetch(slot);
        slot = (slot + kBlockBytes) % (kDepth * kBlockBytes);
    }
};

// A lane's eight elements of each of a block's segments, and the places of these in the segment.
template <typename T> __device__ __forceinline__ void segments_of(const uint4 (&w)[2], Raw8<T> (&raw)[kParts<T>]) {
    if constexpr (sizeof(T) == 2) raw[0].w[0] = w[0], raw[1].w[0] = w[1];
    else raw[0].w[0] = w[0], raw[0].w[1] = w[1];
}
template <typename T> __device__ __forceinline__ int place_in_segment(int lane, int e) {
    return sizeof(T) == 2 ? lane * 8 + e : lane * 4 + e % 4 + e / 4 * 128;
}

// ------------------------------------------------------------- selection

__device__ __forceinline__ float warp_min(float v) {
    float r;
    asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// A team's warps select together: kWarps of them, which are the CTA.
template <int kWarps> __device__ __forceinline__ void team_sync() {
    if constexpr (kWarps == 1) __syncwarp();
    else __syncthreads();
}

// A selection's memory: candidates' keys, segments chosen (and units), counters, and the segments that the
// warps look at (or the largest of units).
struct Selection {
    uint64_t* list;
    int* chosen;
    int* counts;
    uint32_t* stage;

    __host__ __device__ static constexpr size_t bytes(int warps, int k, int element) {
        const size_t stage = static_cast<size_t>(stage_bytes(warps, element)) * warps;
        const size_t units = size_t{128} * ((k + 3) / 4 * 4);  // those of k segments, in fours
        return kListed * 8 + 2 * DRS_MAX_ALTERNATIVES * 4 + 16 + (stage > units ? stage : units);
    }
    __device__ explicit Selection(float* memory) {
        list = reinterpret_cast<uint64_t*>(memory);
        chosen = reinterpret_cast<int*>(list + kListed);
        counts = chosen + 2 * DRS_MAX_ALTERNATIVES;
        stage = reinterpret_cast<uint32_t*>(counts + 4);
    }
};

// Dynamic shared memory: the warps' rings, a selection's (kTop), the segments' largest (kTop).
constexpr size_t kRingBytes = kDepth * kBlockBytes;
__host__ __device__ constexpr size_t shared_before(int warps, int k, int element) {
    return warps * kRingBytes + (k > 0 ? Selection::bytes(warps, k, element) : 0);
}
__host__ __device__ constexpr size_t shared_bytes(int warps, int k, int element, int segments) {
    return shared_before(warps, k, element) + (k > 0 ? static_cast<size_t>(segments + 127) / 128 * 512 : 0);
}

// Places for a thread's `mine` entries in a list that the team counts in `count`: the first. Their order differs from
// call to call; what comes of the list does not, as it goes by the keys' ranks. (With scans of the warps in its
// place, words that hold candidates listed before they are taken apart, and a lane to a key in the ranks: 4096 x 8192 with
// 20 alternatives 35.3 us, 32.4 now; fp32 47.1, 41.6.)
__device__ __forceinline__ int places_for(int mine, int* count) { return mine ? atomicAdd(count, mine) : 0; }

// f(key, how many keys exceed it) for each of the n keys of a list, by the team: up to eight lanes to a key (kAlone:
// eight).
template <int kWarps, bool kAlone, typename F> __device__ __forceinline__ void rank_keys(const uint64_t* list, int n, F f) {
    const ulonglong2* const pairs = reinterpret_cast<const ulonglong2*>(list);
    constexpr int kThreads = kWarps * 32;
    int shift = 3;
    if constexpr (!kAlone)
        while (shift > 0 && n << shift > kThreads) --shift;
    const int part = threadIdx.x & ((1 << shift) - 1);
    const uint64_t last = (n & 1) && part == 0 ? list[n - 1] : 0;
    for (int i0 = 0; i0 < n; i0 += kThreads >> shift) {
        const int i = i0 + (static_cast<int>(threadIdx.x) >> shift);
        const uint64_t key = i < n ? list[i] : 0;
        int above = last > key;
#pragma unroll(kAlone ? 2 : 4)
        for (int j = part; j < n / 2; j += 1 << shift) {
            const ulonglong2 p = pairs[j];
            above += (p.x > key) + (p.y > key);
        }
        for (int d = 1; d < 1 << shift; d <<= 1) above += __shfl_xor_sync(0xffffffffu, above, d);
        if (i < n && part == 0) f(key, above);
    }
}

// The k-th largest of the warp's 32 n values, -inf where there are fewer.
template <int n> __device__ __forceinline__ float kth_of(const float (&v)[n], int k) {
    int above[n] = {};
#pragma unroll
    for (int i = 0; i < 32; ++i) {
#pragma unroll
        for (int j = 0; j < n; ++j) {
            const float u = __shfl_sync(0xffffffffu, v[j], i);
#pragma unroll
            for (int h = 0; h < n; ++h) above[h] += u > v[h];
        }
    }
    float least = INFINITY;  // the smallest that fewer than k exceed
#pragma unroll
    for (int h = 0; h < n; ++h) least = fminf(least, above[h] < k ? v[h] : INFINITY);
    return warp_min(least);
}

// Apart for more than 20: unrolled, these would weigh on the registers of the reading.
__device__ __noinline__ float kth_of_64(float a, float b, int k) {
    const float v[2] = {a, b};
    return kth_of<2>(v, k);
}
__device__ __noinline__ float kth_of_128(float4 u, int k) {
    const float v[4] = {u.x, u.y, u.z, u.w};
    return kth_of<4>(v, k);
}

// A value that at least k of the 128 n values reach, or -inf (which NaN counts
// as): the k-th largest of the largest of 32, 64 or 128 groups of them. With 1.6 k
// groups or more not many more than k reach it: of 1024 about 31 for k = 20 and
// 43 for k = 32 (130 with 32 groups: the smallest of them all).
__device__ __forceinline__ float reached_by(const float4* value, int n, int k, int lane) {
    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const float4 u = value[i * 32 + lane];
        v = make_float4(fmaxf(v.x, u.x), fmaxf(v.y, u.y), fmaxf(v.z, u.z), fmaxf(v.w, u.w));
    }
    if (k > 40) return kth_of_128(v, k);
    const float a = fmaxf(v.x, v.y), b = fmaxf(v.z, v.w);
    if (k > 20) return kth_of_64(a, b, k);
    const float one[1] = {fmaxf(a, b)};
    return kth_of<1>(one, k);
}

// The same with 32 groups, by the team: each warp reads its share of the values, and the groups' largest are compared
// in memory (64 floats per warp). For a team that is alone: with it, and the segments' ranks left out where one go takes
// all listed, 16 x 262144 bf16 rows with 20 alternatives 10.2 us, 10.5 without; 16 x 46000 with 5 5.8, 6.1; but 4096 x
// 8192, whose teams share their SM, 33.6, 32.5.
template <int kWarps> __device__ __forceinline__ float reached_together(const float4* value, int n, int k, float* memory) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float v = -INFINITY;
#pragma unroll 4
    for (int i = warp; i < n; i += kWarps) {
        const float4 u = value[i * 32 + lane];
        v = fmaxf(v, fmaxf(fmaxf(u.x, u.y), fmaxf(u.z, u.w)));
    }
    if constexpr (kWarps > 1) {
        memory[threadIdx.x] = v;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v = fmaxf(v, memory[w * 32 + lane]);
    }
    float* const own = memory + (kWarps + warp) * 32;
    own[lane] = v;
    __syncwarp();
    int above = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 u = reinterpret_cast<const float4*>(own)[i];
        above += (u.x > v) + (u.y > v) + (u.z > v) + (u.w > v);
    }
    return warp_min(above < k ? v : INFINITY);
}

// The k largest of n numbers, equal ones by index, as indices in ascending
// order (all when n <= k): how many.
__device__ int select_exact(const uint32_t* value, int n, int k, int* chosen, int lane) {
    __syncwarp();
    uint32_t least = 0;  // the largest number that at least k reach, bit by bit
    if (n > k) {
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t next = least | 1u << bit;
            int reach = 0;
            for (int i = lane; i < n; i += 32) reach += value[i] >= next;
            reach = __reduce_add_sync(0xffffffffu, reach);
            if (reach >= k) least = next;
            if (reach == k) break;
        }
    }
    int above = 0;
    for (int i = lane; i < n; i += 32) above += value[i] > least;
    int ties = min(n, k) - __reduce_add_sync(0xffffffffu, above), at = 0;
    const uint32_t below = (1u << lane) - 1;
    for (int i = lane; i - lane < n; i += 32) {
        const uint32_t v = i < n ? value[i] : 0;
        const uint32_t same = __ballot_sync(0xffffffffu, i < n && v == least);
        const bool take = i < n && (v > least || (v == least && __popc(same & below) < ties));
        const uint32_t taken = __ballot_sync(0xffffffffu, take);
        if (take) chosen[at + __popc(taken & below)] = i;
        at += __popc(taken);
        ties -= min(ties, __popc(same));
    }
    __syncwarp();
    return at;
}

// For rows with many equal logits, or where they rise over long stretches: the k segments,
// then their k units of eight columns, then their k elements, by one warp. us for 4096 x 262144 bf16 with 20 (64)
// alternatives: sorted rows 465 (687), constant ones 500 (718), others 330 (373); one row 36, 42, 6.5 with 20; 4096 x 8192
// 131, 155, 32.6.
template <typename T> __device__ __noinline__ int select_slowly(const Row<T> row, float* segment, int n, int k, const Selection s) {
    const int lane = threadIdx.x & 31;
    uint32_t* const order = reinterpret_cast<uint32_t*>(segment);
    for (int i = lane; i < n; i += 32) order[i] = order_of(segment[i]);
    const int segments = select_exact(order, n, k, s.chosen, lane);
    for (int c = 0; c < segments; ++c) {
        float v[8];
        const int place = s.chosen[c] * kSegment + lane * 8;
        row.unit(place).unpack(v);
        uint32_t most = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (place + e >= row.lead && place + e < row.end) most = max(most, order_of(v[e]));
        s.stage[c * 32 + lane] = most;
    }
    int* const units = s.chosen + DRS_MAX_ALTERNATIVES;
    const int m = select_exact(s.stage, segments * 32, k, units, lane);
    for (int i = lane; i < m; i += 32) units[i] = s.chosen[units[i] / 32] * 32 + units[i] % 32;
    __syncwarp();
    for (int i = lane; i < m * 8; i += 32) {
        const int place = units[i >> 3] * 8 + (i & 7);
        s.stage[i] = place >= row.lead && place < row.end ? order_of(to_f(row.first[place])) : 0;
    }
    const int found = select_exact(s.stage, m * 8, k, s.chosen, lane);
    for (int i = lane; i < found; i += 32) {
        const int j = s.chosen[i];
        s.list[i] = s.stage[j] ? key_of(s.stage[j], units[j >> 3] * 8 + (j & 7)) : 0;
    }
    return found;
}

// The row's k largest logits into s.list, in no order: how many keys, at least k.
// segment: its n segments' largest, with -inf up to a multiple of 128. s.counts are 0 before. By the
// team, with a barrier at its end. kAlone: nothing else runs meanwhile, so that its steps' latencies count, not its
// instructions.
template <int kWarps, bool kAlone, typename T>
__device__ __forceinline__ int select_top(const Row<T>& row, float* segment, int n, int k, const Selection& s) {
    constexpr float kLowest = -0x1.fffffep127f;  // all but -inf and NaN reach it
    constexpr int kThreads = kWarps * 32;
    constexpr int kBytes = kSegment * static_cast<int>(sizeof(T)), kStage = stage_bytes(kWarps, sizeof(T)), kAtOnce = kStage / kBytes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int segments = n;       // looked at
    float least = kLowest;  // what reaches it is taken
    bool slowly = false;
    if (n > k) {
        const int quads = (n + 127) / 128;
        const float4* const quad = reinterpret_cast<const float4*>(segment);
        const float reached = kAlone && k <= 20
                                  ? reached_together<kWarps>(quad, quads, k, reinterpret_cast<float*>(s.stage))
                                  : reached_by(quad, quads, k, lane);
        const float bound = fmaxf(reached, kLowest);
        // 32 values per lane at a time: a bit for each that reaches the bound
        for (int i0 = warp; i0 < quads; i0 += 8 * kWarps) {
            uint32_t reach = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = i0 + i * kWarps;
                if (at >= quads) break;
                const float4 v = quad[at * 32 + lane];
                reach |= (v.x >= bound ? 1u : 0u) << (4 * i) | (v.y >= bound ? 2u : 0u) << (4 * i) |
                         (v.z >= bound ? 4u : 0u) << (4 * i) | (v.w >= bound ? 8u : 0u) << (4 * i);
            }
            int at = places_for(__popc(reach), &s.counts[0]);
            for (; reach; reach &= reach - 1, ++at) {
                const int bit = __ffs(reach) - 1, place = ((i0 + bit / 4 * kWarps) * 32 + lane) * 4 + bit % 4;
                if (kAlone && at < kAtOnce * kWarps) s.chosen[at] = place;
                if (at < kListed) s.list[at] = key_of(order_of(segment[place]), place);
            }
        }
        team_sync<kWarps>();
        const int listed = s.counts[0];
        slowly = listed > kListed;
        if (kAlone && listed <= kAtOnce * kWarps) {  // one go takes them all: no need of their ranks
            segments = listed;
            least = bound;
        } else if (!slowly) {
            rank_keys<kWarps, kAlone>(s.list, listed, [&](uint64_t key, int above) {
                if (above < k) s.chosen[above] = place_of(key);
            });
            segments = min(listed, k);
            team_sync<kWarps>();
            if (listed >= k) least = segment[s.chosen[k - 1]];
        }
    } else {
        for (int i = tid; i < n; i += kThreads) s.chosen[i] = i;
        float* const unit = reinterpret_cast<float*>(s.stage);
#pragma unroll 2
        for (int c = warp; c < (n + 3) / 4 * 4; c += kWarps)  // a lane's in its own float4s
            unit[(c / 4 * 32 + lane) * 4 + c % 4] = c < n ? Eight<T>::largest(row.unit(c * kSegment + lane * 8)) : -INFINITY;
        team_sync<kWarps>();
        if (n * 32 >= k) least = fmaxf(reached_by(reinterpret_cast<const float4*>(unit), (n + 3) / 4, k, lane), kLowest);
        team_sync<kWarps>();
    }
    if (!slowly) {
        // Each warp has its share of the segments, each lane of their words.
        constexpr int kHalves = sizeof(T) / 2;
        static_assert(kAtOnce * 8 <= 32, "bits");
        char* const stage = reinterpret_cast<char*>(s.stage) + warp * kStage;
        const uint32_t to = smem_u32(stage) + lane * 16;
        const auto word_at = [&](int c) {
            Raw8<T> raw;
#pragma unroll
            for (int h = 0; h < kHalves; ++h) raw.w[h] = reinterpret_cast<const uint4*>(stage)[(c * kHalves + h) * 32 + lane];
            return raw;
        };
        for (int c0 = warp; c0 < segments; c0 += kAtOnce * kWarps) {
            // this lane's of the segments at once
            const int own = lane < kAtOnce && c0 + lane * kWarps < segments ? s.chosen[c0 + lane * kWarps] : -1;
            const T* const line = row.first + lane * static_cast<int>(16 / sizeof(T));
            if (__all_sync(0xffffffffu, own < 0 || row.whole(own * kSegment, kSegment))) {
#pragma unroll
                for (int c = 0; c < kAtOnce; ++c) {
                    const int segment_at = __shfl_sync(0xffffffffu, own, c);
                    if (segment_at >= 0)
#pragma unroll
                        for (int h = 0; h < kHalves; ++h)
                            copy16(to + c * kBytes + h * 512, line + segment_at * kSegment + h * 128);
                }
            } else {
                for (int c = 0; c < kAtOnce; ++c) {
                    const int segment_at = __shfl_sync(0xffffffffu, own, c);
                    const int place = segment_at * kSegment + lane * static_cast<int>(16 / sizeof(T));
                    if (segment_at >= 0)
                        for (int h = 0; h < kHalves; ++h) store_shared16(to + c * kBytes + h * 512, row.word(place + h * 128));
                }
            }
            copies_commit();
            copies_wait<0>();  // a lane reads what it has copied itself
            uint32_t reach = 0;  // of this lane's words, eight bits for each segment
#pragma unroll
            for (int c = 0; c < kAtOnce; ++c) {
                float v[8];
                word_at(c).unpack(v);
                if (c0 + c * kWarps < segments)
#pragma unroll
                    for (int e = 0; e < 8; ++e) reach |= (v[e] >= least ? 1u : 0u) << (8 * c + e);
            }
            for (int at = places_for(__popc(reach), &s.counts[1]); reach; reach &= reach - 1, ++at) {
                const int bit = __ffs(reach) - 1, c = bit / 8, in = place_in_segment<T>(lane, bit % 8);
                const T x = reinterpret_cast<const T*>(stage)[c * kSegment + in];
                if (at < kListed) s.list[at] = key_of(order_of(to_f(x)), s.chosen[c0 + c * kWarps] * kSegment + in);
            }
        }
        team_sync<kWarps>();
        slowly = s.counts[1] > kListed;
    }
    if (slowly || s.counts[1] < k) {
        team_sync<kWarps>();  // everyone has read the counter
        if (warp == 0) {
            int found = s.counts[1];
            if (slowly) {
                found = select_slowly(row, segment, n, k, s);
            } else {
                // Fewer than k above -inf: the first columns at -inf (or NaN) follow.
                for (int place = row.lead + lane; found < k && place - lane < row.end; place += 32) {
                    const bool take = place < row.end && !(to_f(row.first[place]) > -INFINITY);
                    const uint32_t taken = __ballot_sync(0xffffffffu, take);
                    const int at = found + __popc(taken & ((1u << lane) - 1));
                    if (take && at < kListed) s.list[at] = key_of(order_of(-INFINITY), place);
                    found += __popc(taken);
                }
            }
            if (lane == 0) s.counts[1] = found;
        }
        team_sync<kWarps>();
    }
    return s.counts[1];
}

// What the outputs of a row's alternatives need.
struct TopOutputs {
    int32_t* ids;
    float* logprobs;
    float top, inverse, log_sum;
    int lead, k;
    __device__ __forceinline__ void write(uint64_t key, int above) const {
        if (above >= k) return;
        ids[above] = place_of(key) - lead;
        logprobs[above] = (value_of(static_cast<uint32_t>(key >> 32)) - top) * inverse - log_sum;
    }
};

// Apart from the reading, whose registers it would take: 4096 x 262144 bf16 348 us within, 336 apart (with scans in the
// lists). The outputs are written within by teams (329 us; apart as well 340), apart by clusters (one row of 262144 6.6 us
// within, 6.4 apart).
template <int kWarps, typename T>
__device__ __noinline__ int select_top_apart(const Row<T> row, float* segment, int n, int k, const Selection s) {
    return select_top<kWarps, false>(row, segment, n, k, s);
}
template <int kWarps, typename T>
__device__ __noinline__ void select_alone(const Row<T> row, float* segment, int n, const Selection s, const TopOutputs out) {
    const int found = select_top<kWarps, true>(row, segment, n, out.k, s);
    rank_keys<kWarps, true>(s.list, found, [&](uint64_t key, int above) { out.write(key, above); });
}

// ------------------------------------------------------------- sums

// S and W relative to `top`, and the number of columns above the token.
struct Sums {
    float top, sum, weighted;
    int above;
};

// The exponent by which sums relative to `from` are moved to `to`.
__device__ __forceinline__ float shift_of(float from, float to, float c) {
    return from == -INFINITY ? 0.0f : max_nan((from - to) * c, -1000.0f);
}

// The first n lanes' sums together, on every lane.
__device__ __forceinline__ Sums together(Sums s, bool have, float c) {
    if (!have) s = Sums{-INFINITY, 0.0f, 0.0f, 0};
    const float top = warp_max(s.top);
    const float d = shift_of(s.top, top, c), f = ex2_approx(d);
    return Sums{top, warp_sum(s.sum * f), warp_sum(f * fmaf(d, s.sum, s.weighted)), warp_sum(s.above)};
}

// The sums of a thread's part of a row; top and reference are the warp's. The
// reference is kept as an exponent, shift = M c rounded: t = x c - shift takes
// one rounding, and what shift is off by moves all exponents alike and is
// known (x c - shift at x = M). Where that is too much (shift above 2^24: tiny
// temperatures, huge logits) or the floor leaves the type's range, the warp
// begins again with kCareful: t is (x - M) c, held element by element.
template <typename T, bool kCareful> struct RunningSums {
    float top = -INFINITY, bound = -INFINITY;  // bound: where the reference moves
    float base = 0.0f;                         // careful: M, else M c rounded; 0 before there is one
    bool none = true;
    // Without a reference the floor may be -inf, by which add() multiplies 0: weighted then counts as sum, which is 0, or
    // NaN after a NaN.
    uint64_t sum = 0, weighted = 0;
    Floor<T> floor;

    __device__ __forceinline__ RunningSums(float c) { floor.set(kLeastExponent / c); }

    // The exponent by which the sums move to those relative to `to`.
    __device__ __forceinline__ float distance(float to, float c) const {
        if (none) return 0.0f;
        return max_nan(kCareful ? (base - to) * c : -fmaf(to, c, -base), -1000.0f);
    }

    // The reference moves to the largest so far; false: not without care.
    __device__ __forceinline__ bool move(float c) {
        const float next = kCareful ? top : top * c;
        if (!kCareful && !(fabsf(next) < 0x1p24f && floor.set(top + kLeastExponent / c))) return false;
        const float d = none ? 0.0f : max_nan(kCareful ? (base - next) * c : base - next, -1000.0f);
        const float f = ex2_approx(d);
        const uint64_t f2 = pack2(f, f);
        if (none) weighted = sum;
        weighted = mul2(f2, fma2(pack2(d, d), sum, weighted));
        sum = mul2(f2, sum);
        base = next;
        bound = top + kSlack / c;
        none = false;
        return true;
    }

    // A block: its own sums first, which keeps small terms that would be lost in the row's.
    __device__ __forceinline__ void add(const Raw8<T> (&raw)[kParts<T>], float c) {
        const uint64_t c2 = pack2(c, c), base2 = kCareful ? pack2(base, base) : pack2(-base, -base);
        uint64_t part = 0, weight = 0;
#pragma unroll
        for (int p = 0; p < kParts<T>; ++p) {
            float v[8];
            if constexpr (kCareful) raw[p].unpack(v);
            else floor.raise(raw[p]).unpack(v);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const uint64_t x = pack2(v[e], v[e + 1]);
                uint64_t t = kCareful ? mul2(sub2(x, base2), c2) : fma2(x, c2, base2);
                float t0, t1;
                unpack2(t, t0, t1);
                if constexpr (kCareful || !Floor<T>::kPaired) {
                    t0 = max_nan(t0, kLeastExponent);
                    t1 = max_nan(t1, kLeastExponent);
                    t = pack2(t0, t1);
                }
                const uint64_t q = pack2(ex2_flushed(t0), ex2_flushed(t1));
                part = p + e == 0 ? q : add2(part, q);
                weight = p + e == 0 ? mul2(q, t) : fma2(q, t, weight);
            }
        }
        sum = add2(sum, part);
        weighted = add2(weighted, weight);
    }

    // The warp's sums, on every lane.
    __device__ __forceinline__ Sums value(float c, int above) const {
        float s0, s1, w0, w1;
        unpack2(sum, s0, s1);
        unpack2(weighted, w0, w1);
        if (none) w0 = s0, w1 = s1;
        const float d = distance(top, c), f = ex2_approx(d);
        return Sums{top, warp_sum(f * (s0 + s1)), warp_sum(f * fmaf(d, s0 + s1, w0 + w1)), warp_sum(above)};
    }
};

// What a warp does with the blocks of a row that come to it: sums, the token's rank, and (kTop) the segments'
// largest into `segment`.
template <typename T, bool kTop, bool kCareful> struct RowReader {
    RunningSums<T, kCareful> sums;
    float c, own_value;
    T own;
    float* segment;
    uint32_t above = 0;

    __device__ __forceinline__ RowReader(float c, T own, float* segment)
        : sums(c), c(c), own_value(to_f(own)), own(own), segment(segment) {}

    // false: not without care
    __device__ __forceinline__ bool add(const Raw8<T> (&raw)[kParts<T>], int block) {
        float most = -INFINITY;
#pragma unroll
        for (int p = 0; p < kParts<T>; ++p) {
            const float largest = warp_max(Eight<T>::largest(raw[p]));
            if (kTop && (threadIdx.x & 31) == 0) segment[block * kParts<T> + p] = largest;
            most = fmaxf(most, largest);
        }
        sums.top = fmaxf(sums.top, most);
        if (most > sums.bound && !sums.move(c)) return false;
        sums.add(raw, c);
        if (most > own_value) {
#pragma unroll
            for (int p = 0; p < kParts<T>; ++p) Eight<T>::count(raw[p], own, above);
        }
        return true;
    }
    __device__ __forceinline__ Sums value() const { return sums.value(c, Eight<T>::total(above)); }
};

// ------------------------------------------------------------- the row's results

// What a row's warps need to know of it.
template <typename T> struct Task {
    Row<T> row;
    T own;
    float inverse, c;
    __device__ __forceinline__ Task(const LogprobParams& a, int r, int id)
        : row(static_cast<const T*>(a.logits) + r * a.row_stride, a.vocab), own(row.first[row.lead + max(id, 0)]) {
        inverse = a.temps ? 1.0f / fmaxf(a.temps[r / a.canvas_len], kTempFloor) : 1.0f;
        c = inverse * kLog2e;
    }
};

// The row's token, -1 where it is passed over.
__device__ __forceinline__ int id_of(const LogprobParams& a, int r) {
    const int64_t id = a.id_bits == 64 ? static_cast<const int64_t*>(a.ids)[r] : static_cast<const int32_t*>(a.ids)[r];
    return id >= 0 && id < a.vocab ? static_cast<int>(id) : -1;
}

// A block by plain loads.
template <typename T> __device__ __forceinline__ void load_block(const Row<T>& row, int block, Raw8<T> (&raw)[kParts<T>]) {
    uint4 w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        w[h] = row.word(block * kBlock<T> + h * (kBlock<T> / 2) + static_cast<int>(threadIdx.x & 31) * static_cast<int>(16 / sizeof(T)));
    segments_of(w, raw);
}

// Blocks first, first + step, ... below end of a row by plain loads, with care.
template <typename T, bool kTop>
__device__ __noinline__ Sums careful_sums(const Task<T> task, int first, int step, int end, float* segment) {
    RowReader<T, kTop, true> reader(task.c, task.own, segment);
    for (int i = first; i < end; i += step) {
        Raw8<T> raw[kParts<T>];
        load_block(task.row, i, raw);
        reader.add(raw, i);
    }
    return reader.value();
}

// Adds the blocks among [first, end) of a row that reach over its ends to a warp's sums.
// false: there are none.
template <bool kTop, typename T>
__device__ __forceinline__ bool add_edges(const Task<T>& task, int first, int end, float* segment, Sums& sums) {
    const int whole_first = max(task.row.whole_first(), first), whole_end = min(task.row.whole_end(), end);
    const int lane = threadIdx.x & 31;
    const bool before = first < whole_first, behind = whole_end < end && whole_end >= whole_first;
    if (before) sums = careful_sums<T, kTop>(task, first, 1, min(whole_first, end), segment);
    if (behind) {
        const Sums more = careful_sums<T, kTop>(task, whole_end, 1, end, segment);
        sums = before ? together(lane == 0 ? sums : more, lane < 2, task.c) : more;
    }
    return before || behind;
}

// The warp's blocks first, first + kStep, ... (count of them), which come through the ring; before the last kDepth
// of them all have been fetched, and `go_on` may point it at the next row's.
template <bool kTop, bool kCareful, typename T, int kStep, typename F>
__device__ __forceinline__ Sums ring_sums(Ring<T, kStep>& ring, const Task<T>& task, int first, int count, float* segment, F go_on) {
    RowReader<T, kTop, kCareful> reader(task.c, task.own, segment);
    bool fine = true;
    int n = 0;
    for (int end = max(count - kDepth, 0);; end = count) {
        for (; n < end; ++n) {
            uint4 w[2];
            Raw8<T> raw[kParts<T>];
            ring.take(w);
            segments_of(w, raw);
            if (!reader.add(raw, first + n * kStep) && !kCareful) {
                fine = false;
                break;
            }
            ring.fetch_next();
        }
        if (!fine || end == count) break;
        go_on(ring);
    }
    if (fine) return reader.value();
    for (;; ++n) {  // what is on its way, and the fetches ahead
        if (n == count) break;
        if (n == max(count - kDepth, 0)) go_on(ring);
        uint4 w[2];
        ring.take(w);
        ring.fetch_next();
    }
    return careful_sums<T, kTop>(task, first, kStep, first + (count - 1) * kStep + 1, segment);
}

// With care from the start where temperatures leave no doubt (0, say); beyond it only logits above 4096 do. us for 4096 x
// 262144 bf16 with 20 alternatives: 367 with care from the start, 330 without. A warp whose first blocks hold the
// type's lowest value throughout, as some masks do, finds out on the way and reads its share again by plain loads: 769
// for rows that begin so, 330 where they begin with -inf or hold the lowest value here and there.
constexpr float kCarefulFrom = 4096.0f;  // c
template <bool kTop, typename T, int kStep, typename F>
__device__ __forceinline__ Sums row_sums(Ring<T, kStep>& ring, const Task<T>& task, int first, int count, float* segment, F go_on) {
    if (task.c < kCarefulFrom) return ring_sums<kTop, false>(ring, task, first, count, segment, go_on);
    return ring_sums<kTop, true>(ring, task, first, count, segment, go_on);
}

// How many of the numbers first, first + step, ... lie below end.
__device__ __forceinline__ int steps_below(int first, int step, int end) { return max(0, (end - first + step - 1) / step); }

// A row that is passed over, by one warp.
template <bool kTop> __device__ __forceinline__ void pass_over(const LogprobParams& a, int64_t r) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
        a.out_logprob[r] = 0.0f;
        if (a.out_entropy) a.out_entropy[r] = 0.0f;
        if (a.out_rank) a.out_rank[r] = 0;
        if (a.out_norm) a.out_norm[2 * r] = a.out_norm[2 * r + 1] = 0.0f;
    }
    if (kTop)
        for (int i = lane; i < a.k; i += 32) {
            a.out_ids[r * a.k + i] = -1;
            a.out_logprobs[r * a.k + i] = -INFINITY;
        }
}

// Before a row is read: nothing is selected yet, and the line of segments ends in -inf.
template <int kWarps, typename T> __device__ __forceinline__ void prepare(const Row<T>& row, float* segment, const Selection& s) {
    const int n = row.blocks() * kParts<T>;
    for (int i = n + threadIdx.x; i < (n + 127) / 128 * 128; i += kWarps * 32) segment[i] = -INFINITY;
    if (threadIdx.x == 0) s.counts[0] = s.counts[1] = 0;
}

// The row's outputs from its sums and segments, by the team.
template <int kWarps, bool kTop, bool kAlone, typename T>
__device__ __forceinline__ void finish(const LogprobParams& a, int64_t r, const Task<T>& task, const Sums& sums, float* segment,
                                       const Selection& s) {
    int found = 0;
    if constexpr (kTop && !kAlone) found = select_top_apart<kWarps>(task.row, segment, task.row.blocks() * kParts<T>, a.k, s);
    // The largest logit's term is 1: a sum below that is off by the roundings of its exponent alone. No log
    // probability exceeds 0 and no entropy falls below it.
    const float log_sum = sums.sum == 0.0f ? -INFINITY : sums.sum < 1.0f ? 0.0f : logf(sums.sum);
    if (threadIdx.x == (kWarps - 1) * 32) {
        a.out_logprob[r] = (to_f(task.own) - sums.top) * task.inverse - log_sum;
        if (a.out_entropy) a.out_entropy[r] = sums.sum == 0.0f ? 0.0f : max_nan(log_sum - sums.weighted / sums.sum * kLn2, 0.0f);
        if (a.out_rank) a.out_rank[r] = 1 + sums.above;
        if (a.out_norm) a.out_norm[2 * r] = sums.top, a.out_norm[2 * r + 1] = log_sum;
    }
    if constexpr (kTop) {
        const TopOutputs out{a.out_ids + r * a.k, a.out_logprobs + r * a.k, sums.top, task.inverse, log_sum, task.row.lead, a.k};
        if constexpr (kAlone) select_alone<kWarps>(task.row, segment, task.row.blocks() * kParts<T>, s, out);
        else rank_keys<kWarps, false>(s.list, found, [&](uint64_t key, int above) { out.write(key, above); });
    }
}

// ------------------------------------------------------------- many rows

// A team of kWarps warps, a CTA, takes rows in turn.
template <int kWarps, bool kTop, typename T>
__global__ void __launch_bounds__(kWarps * 32, kResident / kWarps) logprob_kernel(const LogprobParams a) {
    extern __shared__ __align__(16) float s_memory[];
    __shared__ Sums s_warp[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Selection select(s_memory + kWarps * kRingBytes / 4);
    float* const segment = s_memory + shared_before(kWarps, kTop ? a.k : 0, sizeof(T)) / 4;
    const int rows = static_cast<int>(a.rows), step = static_cast<int>(gridDim.x);
    Ring<T, kWarps> ring(s_memory);
    bool fetched = true;  // the row's first blocks are on their way: here before its token is known
    {
        const Row<T> row(static_cast<const T*>(a.logits) + blockIdx.x * a.row_stride, a.vocab);
        const int first = row.whole_first() + warp;
        ring.point_at(row, first, steps_below(first, kWarps, row.whole_end()));
        ring.fill();
    }
    int id = id_of(a, blockIdx.x), next_id = rows - static_cast<int>(blockIdx.x) > step ? id_of(a, blockIdx.x + step) : -1;
    Task<T> task(a, blockIdx.x, id);
    for (int r = blockIdx.x; r < rows; r += step) {
        const Task<T> next(a, rows - r > step ? r + step : r, next_id);  // its loads come back while this row is read
        const int next_next_id = rows - r > 2 * step ? id_of(a, r + 2 * step) : -1;
        const int first = task.row.whole_first() + warp, next_first = next.row.whole_first() + warp;
        const int count = steps_below(first, kWarps, task.row.whole_end());
        const int next_count = steps_below(next_first, kWarps, next.row.whole_end());
        if (id >= 0) {
            if (!fetched) {
                ring.point_at(task.row, first, count);
                ring.fill();
            }
            fetched = false;
            if constexpr (kTop) prepare<kWarps>(task.row, segment, select);
            // what reaches over the row's ends, while the first blocks are on their way
            Sums edges{-INFINITY, 0.0f, 0.0f, 0};
            const bool edged = warp == kWarps - 1 && add_edges<kTop>(task, 0, task.row.blocks(), segment, edges);
            Sums sums = row_sums<kTop>(ring, task, first, count, segment, [&](Ring<T, kWarps>& g) {
                if (next_id >= 0 && count >= kDepth) {
                    g.point_at(next.row, next_first, next_count);
                    fetched = true;
                }
            });
            if (edged) sums = together(lane == 0 ? sums : edges, lane < 2, task.c);
            if constexpr (kWarps > 1) {
                if (lane == 0) s_warp[warp] = sums;
                __syncthreads();
                sums = together(s_warp[lane % kWarps], lane < kWarps, task.c);
            } else {
                __syncwarp();
            }
            finish<kWarps, kTop, false>(a, r, task, sums, segment, select);
            team_sync<kWarps>();
        } else {
            if (warp == 0) pass_over<kTop>(a, r);
            copies_wait<0>();
            fetched = false;
        }
        id = next_id;
        next_id = next_next_id;
        task = next;
    }
}

// ------------------------------------------------------------- few rows

// A cluster takes a row; its first CTA finishes it.
template <bool kTop, typename T>
__global__ void __launch_bounds__(256, kResident / 8) logprob_cluster_kernel(const LogprobParams a) {
    constexpr int kWarps = 8;
    extern __shared__ __align__(16) float s_memory[];
    __shared__ uint64_t s_cta[kMaxRowCluster][2];  // the CTAs' sums
    __shared__ Sums s_warp[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = static_cast<int>(cluster_rank());
    const Selection select(s_memory + kWarps * kRingBytes / 4);
    float* const segment = s_memory + shared_before(kWarps, kTop ? a.k : 0, sizeof(T)) / 4;
    const int r = static_cast<int>(blockIdx.x / a.cluster);
    cluster_arrive();
    // the first blocks are on their way before the token is known
    const Row<T> row(static_cast<const T*>(a.logits) + r * a.row_stride, a.vocab);
    const int first = min(rank * a.part, row.blocks()), end = min(first + a.part, row.blocks());
    Ring<T, kWarps> ring(s_memory);
    const int at = max(first, row.whole_first()) + warp, count = steps_below(at, kWarps, min(end, row.whole_end()));
    ring.point_at(row, at, count);
    ring.fill();
    const int id = id_of(a, r);
    if (id < 0) {  // the same for the whole cluster
        copies_wait<0>();
        if (rank == 0 && warp == 0) pass_over<kTop>(a, r);
        cluster_wait();
        return;
    }
    const Task<T> task(a, r, id);
    if constexpr (kTop) prepare<kWarps>(row, segment, select);
    Sums edges{-INFINITY, 0.0f, 0.0f, 0};
    const bool edged = warp == kWarps - 1 && add_edges<kTop>(task, first, end, segment, edges);
    Sums sums = row_sums<kTop>(ring, task, at, count, segment, [](Ring<T, kWarps>&) {});
    if (edged) sums = together(lane == 0 ? sums : edges, lane < 2, task.c);
    if (lane == 0) s_warp[warp] = sums;
    __syncthreads();
    cluster_wait();
    if (kTop && rank != 0)
        for (int i = first * kParts<T> + tid; i < end * kParts<T>; i += kWarps * 32)
            store_remote32(&segment[i], 0, __float_as_uint(segment[i]));
    if (warp == 0) {
        sums = together(s_warp[lane % kWarps], lane < kWarps, task.c);
        if (lane == 0) {
            store_remote(&s_cta[rank][0], 0, pack2(sums.top, sums.sum));
            store_remote(&s_cta[rank][1], 0, pack2(sums.weighted, __int_as_float(sums.above)));
        }
    }
    cluster_sync_all();
    if (rank != 0) return;
    const int from = lane % kMaxRowCluster;
    float above;
    unpack2(s_cta[from][0], sums.top, sums.sum);
    unpack2(s_cta[from][1], sums.weighted, above);
    sums.above = __float_as_int(above);
    sums = together(sums, lane < a.cluster, task.c);
    finish<kWarps, kTop, true>(a, r, task, sums, segment, select);
}

// ------------------------------------------------------------- launches

using LogprobKernel = void (*)(LogprobParams);

template <typename T> LogprobKernel logprob_kernel_of(int warps, bool top) {
    if (warps == 1) return top ? logprob_kernel<1, true, T> : logprob_kernel<1, false, T>;
    if (warps == 2) return top ? logprob_kernel<2, true, T> : logprob_kernel<2, false, T>;
    if (warps == 4) return top ? logprob_kernel<4, true, T> : logprob_kernel<4, false, T>;
    return top ? logprob_kernel<8, true, T> : logprob_kernel<8, false, T>;
}

template <typename T> drs_status launch_logprobs(LogprobParams a, bool vec, cudaStream_t stream) {
    const int sms = sm_count();
    if (sms <= 0) return DRS_ERR_CUDA;
    a.blocks = static_cast<int32_t>(ceil_div(a.vocab + (vec ? 0 : 16 / sizeof(T) - 1), kBlock<T>));
    const int segments = a.blocks * kParts<T>;
    const bool top = a.k > 0;
    const int64_t bytes = a.vocab * static_cast<int64_t>(sizeof(T));
    // CTAs per row: as many as are resident at once, with more than 4096 columns each; with alternatives, and more CTAs
    // than SMs, with 40 KB each, as the selection's CTA waits for all of them. us with one, 2, 4, 8 and 16 (20
    // alternatives, bf16): 1 x 262144 18.8, 12.7, 9.2, 7.2, 6.6; 16 x 262144 20.4, 14.0, 10.5, 9.6, 10.3; 50 x 131072
    // 13.6, 10.7, 10.2, 10.8; 100 x 20000 7.7, 8.6, 9.1; 64 x 46000 9.7, 9.1, 8.6 (without alternatives 6.5, 5.7, 5.0);
    // 110 x 262144 21.2, 19.4, 18.0; 225 x 262144 30.6, 26.8; a second wave costs more: 300 x 131072 19.4, 25.4.
    const int64_t resident = int64_t{sms} * kResident;
    int cluster = 1, warps = 8;
    while (cluster < kMaxRowCluster && a.vocab > 8192 * cluster && a.rows * cluster * 2 <= resident / 8 &&
           (!top || a.rows * cluster * 2 <= sms || bytes >= 80 * 1024 * cluster))
        cluster *= 2;
    const auto teams_of = [&](int w) {  // resident at once
        const size_t smem = shared_bytes(w, a.k, sizeof(T), segments);
        return int64_t{sms} * std::min<int64_t>(kSmemPerSm / (smem + kSmemReserved + 512), kResident / w);
    };
    // Warps per row: as many as leave every row a team at once, but no fewer than suit the row's bytes. us with
    // 8, 4, 2 and 1 (16-bit): 300 x 65536 13.8, 15.1, 20.4, 40.6; 600 x 65536 25.7, 20.4, 23.5, 40.9; 1003 x 50001
    // 37.0, 33.7, 31.7, 41.8; 4096 x 8192 62.1, 42.0, 32.6, 33.3; 2500 x 20000 51.9, 40.1, 35.6, 36.9; 3000 x 60000
    // 88.6, 77.2, 77.5, 101; 1024 x 262144 89.6, 99.9, 103, 149; 4096 x 262144 340, 327, 344, 414; fp32: 2048 x
    // 131072 161, 165, 198, 173; 1653 x 28800 50.4, 43.8, 44.4, 49.7. Longer rows take fewer warps too where all
    // rows then run at once, the first wave of larger teams leaving only a few: 600 x 262144 65.0, 55.8; fp32 500 x
    // 131072 53.8, 47.4; 1216 x 131072 67.2, 61.6, 57.5; fp32 1003 x 65536 51.4, 57.3, 49.3. And they take two where
    // one would leave a few rows over: 3200 x 4096 28.5 (four), 23.9, 29.6; fp32 33.6 (four), 28.9, 38.1.
    const int64_t one = teams_of(1);
    const int64_t most = sizeof(T) == 2 && a.rows * 2 > resident ? 512 * 1024 : 256 * 1024;  // of a row for four warps
    if (a.rows * 8 > resident && (bytes <= most || a.rows * 6 <= resident)) warps = 4;
    if (a.rows * 4 > resident && bytes <= (a.rows * 3 <= resident ? 256 * 1024 : 128 * 1024)) warps = 2;
    if (a.rows * 2 > resident && bytes <= 40 * 1024 && (a.rows <= one || a.rows * 5 > one * 7)) warps = 1;
    if (cluster > 1) warps = 8;
    a.cluster = cluster;
    a.part = static_cast<int32_t>(ceil_div(a.blocks, cluster));
    const size_t smem = shared_bytes(warps, a.k, sizeof(T), segments);
    const int64_t teams = teams_of(warps);
    const LogprobKernel kernel =
        cluster > 1 ? (top ? logprob_cluster_kernel<true, T> : logprob_cluster_kernel<false, T>) : logprob_kernel_of<T>(warps, top);
    const size_t large = smem > 46 * 1024 ? smem : 0;  // beyond what every launch may have, beside the static memory
    if ((large || cluster > 8) && !prepare_kernel(reinterpret_cast<const void*>(kernel), large, cluster > 8))
        return DRS_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster > 1 ? a.rows * cluster : a.rows < teams ? a.rows : teams));
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, a));
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
    a.rows = rows;
    a.row_stride = row_stride;
    a.canvas_len = canvas_len;
    a.vocab = static_cast<int32_t>(vocab);
    a.k = k;
    a.id_bits = id_bits;
    const bool vec = aligned(logits, 16) && row_stride * dtype_bytes(dtype) % 16 == 0;
    return with_dtype(dtype, [&](auto t) { return launch_logprobs<decltype(t)>(a, vec, static_cast<cudaStream_t>(stream)); });
}

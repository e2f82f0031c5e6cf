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
// One read of the row. A CTA (or a cluster of them) takes a row, its warps segments of
// 256 columns, and keep each segment's largest logit in shared memory. The k
// largest logits lie in the k segments whose largest logits come first (by
// value, then by column): any logit of another segment has k before it, one in
// each of these. So only k segments are looked at again, from L2, and of
// these only what reaches the k-th segment's largest.
#include <climits>

#include "token_common.cuh"

namespace drs {
namespace {

constexpr int kThreadsPerRow = 256;
constexpr int kRowWarps = kThreadsPerRow / 32;
constexpr int kMaxRowCluster = 16;
constexpr int kSegment = 256;   // columns a warp takes at once: 8 per lane
constexpr int kTile = 4;        // segments whose loads a warp has in flight
constexpr int kListed = 512;    // candidates of the short way
// Exponents (base 2) below this give 0; held there so that 0 times an
// infinite exponent does not arise in W.
constexpr float kLeastExponent = -200.0f;
constexpr float kSlack = 8.0f;  // exponents above the reference before it moves

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
    int32_t vocab, k, id_bits, cluster, part;  // part: segments of a CTA
};

// ------------------------------------------------------------- elements

// 2^x, results below the normal range 0: one instruction (ex2_approx takes
// four), in sums of terms relative to their largest.
__device__ __forceinline__ float ex2_flushed(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The largest of eight elements (NaN left out), and how many exceed a value,
// counted over a tile: 16-bit elements in pairs of 16-bit sums (whole numbers
// of at most 4 per segment in each half).
template <typename T> struct Eight;
template <> struct Eight<float> {
    using Count = int;
    __device__ static float largest(const Raw8<float>& r) {
        float v[8];
        r.unpack(v);
        return fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
    }
    __device__ static Count zero() { return 0; }
    __device__ static void count(const Raw8<float>& r, float own, Count& n) {
        float v[8];
        r.unpack(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) n += v[e] > own;
    }
    __device__ static int total(Count n) { return n; }
};
template <typename T, typename T2> struct EightHalves {
    using Count = T2;
    __device__ static T2 pair(uint32_t w) { return *reinterpret_cast<const T2*>(&w); }
    __device__ static float largest(const Raw8<T>& r) {
        const T2 m = __hmax2(__hmax2(pair(r.w[0].x), pair(r.w[0].y)), __hmax2(pair(r.w[0].z), pair(r.w[0].w)));
        return fmaxf(to_f(m.x), to_f(m.y));
    }
    __device__ static Count zero() { return pair(0); }
    __device__ static void count(const Raw8<T>& r, T own, Count& n) {
        T2 o;
        o.x = o.y = own;
        n = __hadd2(n, __hadd2(__hadd2(__hgt2(pair(r.w[0].x), o), __hgt2(pair(r.w[0].y), o)),
                               __hadd2(__hgt2(pair(r.w[0].z), o), __hgt2(pair(r.w[0].w), o))));
    }
    __device__ static int total(Count n) { return static_cast<int>(to_f(n.x) + to_f(n.y)); }
};
template <> struct Eight<__nv_bfloat16> : EightHalves<__nv_bfloat16, __nv_bfloat162> {};
template <> struct Eight<__half> : EightHalves<__half, __half2> {};

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
    __device__ __forceinline__ Raw8<T> unit(int place) const {
        Raw8<T> r;
        if (whole(place, 8)) {
            r.load(first + place);
        } else {
            T* const e = reinterpret_cast<T*>(&r);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                e[i] = place + i >= lead && place + i < end ? first[place + i] : from_f<T>(-INFINITY);
        }
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

// ------------------------------------------------------------- selection

struct Selection {
    __align__(16) uint64_t list[kListed];      // candidates: keys of segments, then of elements
    uint32_t unit[DRS_MAX_ALTERNATIVES * 32];  // orders of units' largest, then of elements
    int chosen[2][DRS_MAX_ALTERNATIVES];
    int counts[32];
    int n, m;
};

// How many of the n keys exceed this one. The list goes on with three zeros.
__device__ __forceinline__ int keys_above(const uint64_t* list, int n, uint64_t key) {
    int above = 0;
#pragma unroll 2
    for (int i = 0; i < n; i += 4) {
        const ulonglong2 p = *reinterpret_cast<const ulonglong2*>(list + i), q = *reinterpret_cast<const ulonglong2*>(list + i + 2);
        above += (p.x > key) + (p.y > key) + (q.x > key) + (q.y > key);
    }
    return above;
}

// A value that at least k of the n > k values reach, by every warp for itself: the
// k-th largest of the largest of 32 (k <= 32) or 64 groups of them.
__device__ __forceinline__ uint32_t reached_by(const uint32_t* value, int n, int k, int lane) {
    uint32_t a = 0, b = 0;  // below every order
    int above_a = 0, above_b = 0;
    if (k <= 32) {
        for (int i = lane; i < n; i += 32) a = max(a, value[i]);
#pragma unroll 8
        for (int i = 0; i < 32; ++i) above_a += __shfl_sync(0xffffffffu, a, i) > a;
        return __reduce_min_sync(0xffffffffu, above_a < k ? a : 0xffffffffu);  // the smallest that fewer than k exceed
    }
    for (int i = lane; i < n; i += 64) {
        a = max(a, value[i]);
        if (i + 32 < n) b = max(b, value[i + 32]);
    }
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
        const uint32_t u = __shfl_sync(0xffffffffu, a, i), v = __shfl_sync(0xffffffffu, b, i);
        above_a += (u > a) + (v > a);
        above_b += (u > b) + (v > b);
    }
    return __reduce_min_sync(0xffffffffu, min(above_a < k ? a : 0xffffffffu, above_b < k ? b : 0xffffffffu));
}

// The k largest of n values, equal ones by index, as indices in ascending
// order (all when n <= k): their number. By all threads; any values.
__device__ int select_exact(const uint32_t* value, int n, int k, int* chosen, Selection& s) {
    const int tid = threadIdx.x, lane = tid & 31;
    if (n <= k) {
        __syncthreads();
        for (int i = tid; i < n; i += kThreadsPerRow) chosen[i] = i;
        __syncthreads();
        return n;
    }
    __syncthreads();
    if (tid < 32) s.counts[tid] = 0;
    __syncthreads();
    uint32_t least = 0;  // the largest number that at least k values reach, bit by bit
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t next = least | 1u << bit;
        int reach = 0;
        for (int i = tid; i < n; i += kThreadsPerRow) reach += value[i] >= next;
        reach = __reduce_add_sync(0xffffffffu, reach);
        if (lane == 0) atomicAdd(&s.counts[bit], reach);
        __syncthreads();
        reach = s.counts[bit];
        if (reach >= k) least = next;
        if (reach == k) break;
    }
    if (tid < 32) {  // those above, and the first of the equal ones
        int above = 0;
        for (int i = lane; i < n; i += 32) above += value[i] > least;
        int ties = k - __reduce_add_sync(0xffffffffu, above), at = 0;
        for (int i = lane; i - lane < n && at < k; i += 32) {
            const uint32_t v = i < n ? value[i] : 0;
            const uint32_t more = __ballot_sync(0xffffffffu, v > least);
            const uint32_t same = __ballot_sync(0xffffffffu, i < n && v == least);
            const uint32_t below = (1u << lane) - 1;
            const int rank = __popc(same & below);
            const bool take = (more >> lane & 1) || ((same >> lane & 1) && rank < ties);
            const uint32_t taken = __ballot_sync(0xffffffffu, take);
            if (take) chosen[at + __popc(taken & below)] = i;
            at += __popc(taken);
            ties -= min(ties, __popc(same));
        }
    }
    __syncthreads();
    return k;
}

// The row's k largest logits into s.list, in no order: their number, at least k (keys of 0
// among them are places outside the row). segment: the orders of its n
// segments' largest.
template <typename T> __device__ int select_top(const Row<T>& row, const uint32_t* segment, int n, int k, Selection& s) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (n > k) {
        // The short way: segments that reach a bound, k of them, and what in
        // these reaches the k-th one's largest.
        const uint32_t bound = reached_by(segment, n, k, lane);
        for (int i = tid; i < n; i += kThreadsPerRow) {
            if (segment[i] >= bound) {
                const int at = atomicAdd(&s.n, 1);
                if (at < kListed) s.list[at] = key_of(segment[i], i);
            }
        }
        __syncthreads();
        const int listed = s.n;
        if (listed <= kListed - 4) {
            if (tid < 3) s.list[listed + tid] = 0;
            __syncthreads();
            for (int i = tid; i < listed; i += kThreadsPerRow) {
                const uint64_t key = s.list[i];
                const int above = keys_above(s.list, listed, key);
                if (above < k) s.chosen[0][above] = place_of(key);
            }
            __syncthreads();
            const uint32_t least = segment[s.chosen[0][k - 1]];
            constexpr int kAtOnce = 4;
            for (int c = warp; c < k; c += kRowWarps * kAtOnce) {
                Raw8<T> raw[kAtOnce];
                int place[kAtOnce];
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) {
                    const int at = c + u * kRowWarps;
                    place[u] = at < k ? s.chosen[0][at] * kSegment + lane * 8 : row.end;  // the row's end: none
                    raw[u] = row.unit(place[u]);
                }
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) {
                    float v[8];
                    raw[u].unpack(v);
                    uint32_t reach = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const bool inside = place[u] + e >= row.lead && place[u] + e < row.end;
                        reach |= (inside && order_of(v[e]) >= least ? 1u : 0u) << e;
                    }
                    if (reach) {
                        int at = atomicAdd(&s.m, __popc(reach));
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (reach >> e & 1) {
                                if (at < kListed) s.list[at] = key_of(order_of(v[e]), place[u] + e);
                                ++at;
                            }
                    }
                }
            }
            __syncthreads();
            if (s.m <= kListed - 4) return s.m;
        }
    }
    // The long way, for rows with many equal logits and for short ones: the k
    // segments, then their k units of eight, then their k elements.
    const int segments = select_exact(segment, n, k, s.chosen[0], s);
    for (int c = warp; c < segments; c += kRowWarps) {
        float v[8];
        const int place = s.chosen[0][c] * kSegment + lane * 8;
        row.unit(place).unpack(v);
        uint32_t most = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (place + e >= row.lead && place + e < row.end) most = max(most, order_of(v[e]));
        s.unit[c * 32 + lane] = most;
    }
    const int units = select_exact(s.unit, segments * 32, k, s.chosen[1], s);
    if (tid < units) s.chosen[1][tid] = s.chosen[0][s.chosen[1][tid] >> 5] * 32 + (s.chosen[1][tid] & 31);
    __syncthreads();
    for (int i = tid; i < units * 8; i += kThreadsPerRow) {
        const int place = s.chosen[1][i >> 3] * 8 + (i & 7);
        s.unit[i] = place >= row.lead && place < row.end ? order_of(to_f(row.first[place])) : 0;
    }
    const int found = select_exact(s.unit, units * 8, k, s.chosen[0], s);
    if (tid < found) {
        const int i = s.chosen[0][tid];
        s.list[tid] = s.unit[i] ? key_of(s.unit[i], s.chosen[1][i >> 3] * 8 + (i & 7)) : 0;
    }
    __syncthreads();
    return found;
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

// The sums of a thread's part of a row; top and reference are the warp's.
struct RunningSums {
    float top = -INFINITY, reference = -INFINITY, bound = -INFINITY;  // bound: where the reference moves
    float base = 0.0f;                                                // the reference, 0 before there is one
    uint64_t sum = 0, weighted = 0;

    // The reference moves to the largest so far.
    __device__ __forceinline__ void move(float c) {
        const float d = shift_of(reference, top, c), f = ex2_approx(d);
        const uint64_t f2 = pack2(f, f);
        weighted = mul2(f2, fma2(pack2(d, d), sum, weighted));
        sum = mul2(f2, sum);
        reference = base = top;
        bound = top + kSlack / c;
    }

    // Eight columns per lane; most: the warp's largest.
    template <typename T> __device__ __forceinline__ void add(const Raw8<T>& raw, float most, float c) {
        top = fmaxf(top, most);
        if (most > bound) move(c);
        const uint64_t base2 = pack2(base, base), c2 = pack2(c, c);
        float v[8];
        raw.unpack(v);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            float t0, t1;
            unpack2(mul2(sub2(pack2(v[e], v[e + 1]), base2), c2), t0, t1);
            t0 = max_nan(t0, kLeastExponent);
            t1 = max_nan(t1, kLeastExponent);
            const uint64_t p = pack2(ex2_flushed(t0), ex2_flushed(t1));
            sum = add2(sum, p);
            weighted = fma2(p, pack2(t0, t1), weighted);
        }
    }

    __device__ __forceinline__ Sums value(float c, int above) const {
        float s0, s1, w0, w1;
        unpack2(sum, s0, s1);
        unpack2(weighted, w0, w1);
        const float d = shift_of(reference, top, c), f = ex2_approx(d);
        return Sums{top, f * (s0 + s1), f * fmaf(d, s0 + s1, w0 + w1), above};
    }
};

// The sums of the row's segments [first, end). kTop: their largest go to `segment`.
template <typename T, bool kTop>
__device__ __forceinline__ Sums row_sums(const Row<T>& row, int first, int end, float c, T own, float* segment) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    RunningSums sums;
    int above = 0;
    for (int i = first + warp * kTile; i < end; i += kRowWarps * kTile) {
        typename Eight<T>::Count exceed = Eight<T>::zero();
        if (i + kTile <= end && row.whole(i * kSegment, kTile * kSegment)) {
            Raw8<T> raw[kTile];
            const T* const from = row.first + i * kSegment + lane * 8;
#pragma unroll
            for (int u = 0; u < kTile; ++u) raw[u].load(from + u * kSegment);
#pragma unroll
            for (int u = 0; u < kTile; ++u) {
                const float most = warp_max(Eight<T>::largest(raw[u]));
                if (kTop && lane == 0) segment[i + u] = most;
                sums.add(raw[u], most, c);
                Eight<T>::count(raw[u], own, exceed);
            }
        } else {
#pragma unroll 1
            for (int u = i; u < min(i + kTile, end); ++u) {
                const Raw8<T> raw = row.unit(u * kSegment + lane * 8);
                const float most = warp_max(Eight<T>::largest(raw));
                if (kTop && lane == 0) segment[u] = most;
                sums.add(raw, most, c);
                Eight<T>::count(raw, own, exceed);
            }
        }
        above += Eight<T>::total(exceed);
    }
    return sums.value(c, above);
}

// ------------------------------------------------------------- the kernel

template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreadsPerRow, 4) logprob_kernel(const LogprobParams a) {
    extern __shared__ uint32_t s_segment[];  // the row's segments' largest: values, then their orders
    __shared__ Selection s_select;
    __shared__ uint64_t s_cta[kMaxRowCluster][2];  // the cluster's CTAs' sums
    __shared__ Sums s_warp[kRowWarps];
    __shared__ float s_norm[2];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int csize = a.cluster, k = a.k;
    const int rank = csize > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int64_t r = blockIdx.x / csize;
    const int64_t id = a.id_bits == 64 ? static_cast<const int64_t*>(a.ids)[r] : static_cast<const int32_t*>(a.ids)[r];
    if (id < 0 || id >= a.vocab) {  // the same for the whole cluster
        if (rank == 0) {
            if (tid == 0) {
                a.out_logprob[r] = 0.0f;
                if (a.out_entropy) a.out_entropy[r] = 0.0f;
                if (a.out_rank) a.out_rank[r] = 0;
                if (a.out_norm) a.out_norm[2 * r] = a.out_norm[2 * r + 1] = 0.0f;
            }
            for (int i = tid; i < k; i += kThreadsPerRow) {
                a.out_ids[r * k + i] = -1;
                a.out_logprobs[r * k + i] = -INFINITY;
            }
        }
        return;
    }
    if (csize > 1) cluster_arrive();
    const T* const x = static_cast<const T*>(a.logits) + r * a.row_stride;
    const Row<T> row(x, a.vocab);
    const T own = x[id];
    const float inverse = a.temps ? 1.0f / fmaxf(a.temps[r / a.canvas_len], kTempFloor) : 1.0f;
    const float c = inverse * kLog2e;

    const int segments = (row.end + kSegment - 1) / kSegment;
    const int first = min(rank * a.part, segments), end = min(first + a.part, segments);
    Sums sums = row_sums<T, kTop>(row, first, end, c, own, reinterpret_cast<float*>(s_segment));
    sums.sum = warp_sum(sums.sum);
    sums.weighted = warp_sum(sums.weighted);
    sums.above = warp_sum(sums.above);
    if (lane == 0) s_warp[warp] = sums;
    if (kTop && tid == 0) s_select.n = s_select.m = 0;
    __syncthreads();
    if (kTop && rank == 0)
        for (int i = first + tid; i < end; i += kThreadsPerRow) s_segment[i] = order_of(__uint_as_float(s_segment[i]));
    if (csize > 1) {  // the first CTA takes it from here
        cluster_wait();
        if (rank != 0) {
            if (kTop)
                for (int i = first + tid; i < end; i += kThreadsPerRow)
                    store_remote32(&s_segment[i], 0, order_of(__uint_as_float(s_segment[i])));
        }
        if (warp == 0) {
            sums = together(s_warp[lane % kRowWarps], lane < kRowWarps, c);
            if (lane == 0) {
                store_remote(&s_cta[rank][0], 0, pack2(sums.top, sums.sum));
                store_remote(&s_cta[rank][1], 0, pack2(sums.weighted, __int_as_float(sums.above)));
            }
        }
        cluster_sync_all();
        if (rank != 0) return;
    } else if (kTop) {
        __syncthreads();
    }
    if (warp == 0) {
        if (csize > 1) {
            const int from = lane % kMaxRowCluster;
            unpack2(s_cta[from][0], sums.top, sums.sum);
            float above;
            unpack2(s_cta[from][1], sums.weighted, above);
            sums.above = __float_as_int(above);
            sums = together(sums, lane < csize, c);
        } else {
            sums = together(s_warp[lane % kRowWarps], lane < kRowWarps, c);
        }
        if (lane == 0) {
            const float log_sum = sums.sum == 0.0f ? -INFINITY : logf(sums.sum);
            a.out_logprob[r] = (to_f(own) - sums.top) * inverse - log_sum;
            if (a.out_entropy) a.out_entropy[r] = sums.sum == 0.0f ? 0.0f : log_sum - sums.weighted / sums.sum * kLn2;
            if (a.out_rank) a.out_rank[r] = 1 + sums.above;
            if (a.out_norm) a.out_norm[2 * r] = sums.top, a.out_norm[2 * r + 1] = log_sum;
            s_norm[0] = sums.top;
            s_norm[1] = log_sum;
        }
    }
    if (!kTop) return;
    const int found = select_top(row, s_segment, segments, k, s_select);  // a barrier comes before s_norm's use
    if (tid < 3) s_select.list[found + tid] = 0;
    __syncthreads();
    for (int i = tid; i < found; i += kThreadsPerRow) {
        const uint64_t key = s_select.list[i];
        const int above = keys_above(s_select.list, found, key);
        if (above < k && key) {
            a.out_ids[r * k + above] = place_of(key) - row.lead;
            a.out_logprobs[r * k + above] = (value_of(static_cast<uint32_t>(key >> 32)) - s_norm[0]) * inverse - s_norm[1];
        }
    }
}

template <typename T> drs_status launch_logprobs(LogprobParams a, int64_t rows, cudaStream_t stream) {
    const int sms = sm_count();
    if (sms <= 0) return DRS_ERR_CUDA;
    const int64_t segments = ceil_div(a.vocab + 16 / sizeof(T) - 1, kSegment);
    const int64_t resident = int64_t{sms} * 4;
    int cluster = 1;
    while (cluster < kMaxRowCluster &&
           segments > 32 * cluster && rows * cluster * 2 <= resident - (cluster < 8 ? sms / 2 : sms * 3 / 2))
        cluster *= 2;
    a.cluster = cluster;
    a.part = static_cast<int32_t>(ceil_div(segments, cluster));
    const auto kernel = a.k > 0 ? logprob_kernel<T, true> : logprob_kernel<T, false>;
    if (cluster > 8 && !prepare_kernel(reinterpret_cast<const void*>(kernel), 0, true)) return DRS_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * cluster));
    cfg.blockDim = dim3(kThreadsPerRow);
    cfg.dynamicSmemBytes = a.k > 0 ? segments * sizeof(uint32_t) : 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
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
    a.row_stride = row_stride;
    a.canvas_len = canvas_len;
    a.vocab = static_cast<int32_t>(vocab);
    a.k = k;
    a.id_bits = id_bits;
    return with_dtype(dtype, [&](auto t) { return launch_logprobs<decltype(t)>(a, rows, static_cast<cudaStream_t>(stream)); });
}

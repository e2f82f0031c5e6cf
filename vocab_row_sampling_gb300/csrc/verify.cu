// verify.cu -- verification of drafted tokens against the target's
// probabilities (drs_verify_drafts).
//
// Speculative sampling (Leviathan, Kalman and Matias, "Fast inference from
// transformers via speculative decoding", 2023): draft j of a request is
// kept while u_j q_j(x_j) < p_j(x_j); the token after the kept ones is drawn
// from max(p - q, 0) of the first refused position, or from p of the
// position after the last draft. The draw is by inversion: the lowest
// column whose running sum of weights exceeds u times their total.
//
// One launch. A thread-block cluster takes a request: every warp reads the
// request's few drafted probabilities itself (no barrier), then the cluster's
// CTAs sum a share of the one row (two with draft probabilities) that the
// draw needs, exchange their totals through distributed shared memory, and
// the CTA whose share holds the drawn column reads one warp's part of it
// again (from L2) to find the column. Bound by memory for large batches: each
// needed row is read once. Measured: 256 requests of 262144 bf16 and fp16
// columns 47.9 us, 4.9 TB/s of those rows (the same reads without the
// cluster's barrier and the draw 41 us); one request of 131072 columns 6.3 us,
// the latency of four dependent loads, a cluster's barrier and a second look.
// The CTAs arrive at a cluster barrier when they begin and wait for it before
// they store into each other's shared memory; the sums in between hide it.
//
// Sums. A drawn column moves when the running sums are off by more than the
// distance of u * total to a border, so they are held to about 2^-44 of the
// total: all sums are pairs of fp32 (the sum and the errors of the additions).
// Another column than that of 64-bit sums comes out in about one draw in
// 10^13 per column. fp64 sums took most of the kernel's time (162 us for 256
// requests of 262144 columns): this GPU issues one fp64 instruction per SM in 16
// cycles. The weight itself is the fp32 difference p - q, rounded once
// (relative 2^-24, exact between values of near exponents).
#include <climits>
#include <type_traits>

#include "token_common.cuh"

namespace drs {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kStep = 256;  // elements a warp takes at once: 8 per lane

struct NoDraft {};

// CTAs per SM that registers are held to: us for 256 requests of 262144 columns
// with 3, 4, 5, 6 and 8 (16-bit rows): 58.4, 50.9, 47.9, 47.5, 49.7. From 6 on
// (40 registers) every kernel spills, at 5 some do, by up to 24 bytes per thread,
// and those of fp32 rows with 16-bit ones by up to 16 at 4.
// bytes: of an element of both rows.
constexpr int resident_ctas(size_t bytes) { return bytes < 6 ? 5 : 4; }

struct VerifyParams {
    const void* target;
    const void* draft;
    const int64_t* tokens;
    const int32_t* cu;
    const float* accept_u;
    const float* sample_u;
    int64_t* out_tokens;
    int32_t* out_accepted;
    int64_t target_rows, target_stride, draft_rows, draft_stride;
    int32_t vocab, max_drafts, cluster, part;
};

// The row (or pair of rows) a request draws from. q is null where nothing
// is subtracted; `without` is a column whose weight is 0 (-1: none).
// kVec: the rows start 16-byte aligned.
template <typename P, typename Q, bool kVec> struct Weights {
    const P* p;
    const Q* q;
    int without, vocab;

    __device__ __forceinline__ float one(int i) const {
        float w = to_f(p[i]);
        if constexpr (!std::is_same<Q, NoDraft>::value) {
            if (q) w -= to_f(q[i]);
        }
        return i == without ? 0.0f : fmaxf(w, 0.0f);  // NaN counts as 0
    }

    // Eight columns from i on.
    template <bool kSub> __device__ __forceinline__ void finish(const Raw8<P>& rp, const float (&qv)[8], int i,
                                                                float (&w)[8]) const {
        rp.unpack(w);
        if constexpr (kSub) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) unpack2(sub2(pack2(w[e], w[e + 1]), pack2(qv[e], qv[e + 1])), w[e], w[e + 1]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = fmaxf(w[e], 0.0f);
        if (!kSub && static_cast<uint32_t>(without - i) < 8u) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (i + e == without) w[e] = 0.0f;
        }
    }

    // Columns i .. i+7, 0 from `end` on (with kVec i is a multiple of 8).
    __device__ __forceinline__ void load(int64_t i, int end, float (&w)[8]) const {
        if (kVec && i + 8 <= end) {
            Raw8<P> rp;
            rp.load(p + i);
            if constexpr (!std::is_same<Q, NoDraft>::value) {
                if (q) {
                    Raw8<Q> rq;
                    float qv[8];
                    rq.load(q + i);
                    rq.unpack(qv);
                    finish<true>(rp, qv, static_cast<int>(i), w);
                    return;
                }
            }
            finish<false>(rp, w, static_cast<int>(i), w);
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = i + e < end ? one(static_cast<int>(i) + e) : 0.0f;
    }
};

// What a running sum is held against: u times the total. Small totals
// are taken times 2^100 on both sides, which keeps the product's error clear of
// underflow (three weights of 2^-149 and u = 1/2: 1.5 steps).
struct Border {
    Pair t;
    float up;
    __device__ __forceinline__ Border(float u, Pair total) {
        up = total.s < 0x1p-20f ? 0x1p100f : 1.0f;
        t = u * Pair{total.s * up, total.c * up};
    }
    __device__ __forceinline__ bool below(Pair sum) const {
        return fmaf(sum.s, up, -t.s) + fmaf(sum.c, up, -t.c) > 0.0f;
    }
};

// The first of n shares (a power of two, one per lane) whose running sum
// from `before` on exceeds the border, and in `before` the sum before it; the last
// share with any mass where none does.
__device__ __forceinline__ int pick(const Pair* share, int n, int lane, const Border& border, Pair& before) {
    const Pair mine = lane < n ? share[lane] : Pair{0.0f, 0.0f};
    const Pair upto = before + warp_scan_pair(mine, lane, n);
    const bool some = lane < n && mine.s > 0.0f;
    const uint32_t over = __ballot_sync(0xffffffffu, some && border.below(upto)), any = __ballot_sync(0xffffffffu, some);
    const int found = over ? __ffs(over) - 1 : 31 - __clz(any);
    const Pair lower = shfl(upto, found > 0 ? found - 1 : 0);
    if (found > 0) before = lower;
    return found;
}

// The sum of the weights of columns [begin, end), begin a multiple of kStep,
// by one warp; every lane gets its own part.
template <bool kSub, typename P, typename Q, bool kVec>
__device__ __forceinline__ Pair lane_sum(const Weights<P, Q, kVec>& wt, int begin, int end, int lane) {
    PairSum2 sum;
    if constexpr (kVec) {
        constexpr int kUnroll = kSub || sizeof(P) == 4 ? 2 : 4;  // 2 KB of a warp's loads in flight
        int i = begin + 8 * lane;
        for (; i + (kUnroll - 1) * kStep + 8 <= end; i += kUnroll * kStep) {
            Raw8<P> rp[kUnroll];
            Raw8<typename std::conditional<kSub, Q, P>::type> rq[kSub ? kUnroll : 1];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                rp[k].load(wt.p + i + k * kStep);
                if constexpr (kSub) rq[k].load(wt.q + i + k * kStep);
            }
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                float qv[8], w[8];
                if constexpr (kSub) rq[k].unpack(qv);
                wt.template finish<kSub>(rp[k], qv, i + k * kStep, w);
#pragma unroll
                for (int e = 0; e < 8; e += 2) sum.add(pack2(w[e], w[e + 1]));
            }
        }
        for (; i < end; i += kStep) {
            if (i + 8 <= end) {
                Raw8<P> rp;
                float qv[8], w[8];
                rp.load(wt.p + i);
                if constexpr (kSub) {
                    Raw8<Q> rq;
                    rq.load(wt.q + i);
                    rq.unpack(qv);
                }
                wt.template finish<kSub>(rp, qv, i, w);
#pragma unroll
                for (int e = 0; e < 8; e += 2) sum.add(pack2(w[e], w[e + 1]));
            } else {
                for (int e = i; e < end; ++e) sum.add(pack2(wt.one(e), 0.0f));
            }
        }
    } else {
        // Rows off 16-byte boundaries: groups of 8 columns from a boundary of p
        // on, their q put together from the words that hold them; the columns
        // before and after (and those whose words would leave the row) one by
        // one. Single elements throughout took 58 us for 256 requests of 200001
        // columns.
        using R = typename std::conditional<kSub, Q, P>::type;
        [[maybe_unused]] constexpr int kWord = 16 / sizeof(R);
        int i0 = begin + static_cast<int>((-reinterpret_cast<uintptr_t>(wt.p + begin) & 15) / sizeof(P));
        int shift = 0, off = 0, most = end;
        if constexpr (kSub) {
            shift = static_cast<int>(reinterpret_cast<uintptr_t>(wt.q + i0) & 15);
            off = shift / static_cast<int>(sizeof(R));
            if (i0 < off) i0 += 8;
            if (off) most = min(end, wt.vocab - kWord + off);
        }
        const int groups = most > i0 ? (most - i0) / 8 : 0, i1 = groups ? i0 + 8 * groups : begin;
        if (!groups) i0 = begin;
        if constexpr (kSub) {
#pragma unroll 1
            for (int i = i0 + 8 * lane; i < i1; i += kStep) {
                Raw8<P> rp;
                Raw8Shifted<R> rq;
                rp.load(wt.p + i);
                rq.load(wt.q + i - off, shift);
                float qv[8], w[8];
                rq.unpack(shift, qv);
                wt.template finish<true>(rp, qv, i, w);
#pragma unroll
                for (int e = 0; e < 8; e += 2) sum.add(pack2(w[e], w[e + 1]));
            }
        } else {
#pragma unroll 2
            for (int i = i0 + 8 * lane; i < i1; i += kStep) {
                Raw8<P> rp;
                float w[8];
                rp.load(wt.p + i);
                wt.template finish<false>(rp, w, i, w);
#pragma unroll
                for (int e = 0; e < 8; e += 2) sum.add(pack2(w[e], w[e + 1]));
            }
        }
        for (int i = begin + lane; i < i0; i += 32) sum.add(pack2(wt.one(i), 0.0f));
        for (int i = i1 + lane; i < end; i += 32) sum.add(pack2(wt.one(i), 0.0f));
    }
    return sum.value();
}

template <typename P, typename Q, bool kVec>
__global__ void __launch_bounds__(kVerifyThreads, resident_ctas(sizeof(P) + sizeof(Q)))
    verify_kernel(const VerifyParams a) {
    constexpr bool kDraft = !std::is_same<Q, NoDraft>::value;
    __shared__ __align__(8) Pair s_cta[2][kMaxCluster];  // the CTAs' totals, by attempt
    __shared__ Pair s_warp[kVerifyWarps];                // this CTA's warps' totals
    __shared__ Pair s_scan[kVerifyWarps];
    __shared__ int s_first, s_last;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int csize = a.cluster;
    const int rank = csize > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int64_t b = blockIdx.x / csize;
    const int64_t first = a.cu[b];
    int64_t count = static_cast<int64_t>(a.cu[b + 1]) - first;
    count = count < 0 ? 0 : count > a.max_drafts ? a.max_drafts : count;
    int64_t* const out = a.out_tokens + b * (static_cast<int64_t>(a.max_drafts) + 1);
    // rows outside the arrays: nothing is read (the same for the whole cluster)
    if (first < 0 || first + count > a.draft_rows || first + b + count >= a.target_rows) {
        if (rank == 0) {
            for (int64_t k = tid; k <= a.max_drafts; k += kVerifyThreads) out[k] = -1;
            if (tid == 0) a.out_accepted[b] = -1;
        }
        return;
    }
    if (csize > 1) cluster_arrive();
    const P* const target = static_cast<const P*>(a.target) + (first + b) * a.target_stride;

    // The accepted drafts, by every warp for itself. u q < p is decided
    // exactly, from the product and its rounding error; both sides are taken
    // times 2^100, which keeps the error clear of underflow.
    int accepted = 0;
    for (int64_t base = 0; base < count; base += 32) {
        const int64_t j = base + lane;
        bool ok = false;
        if (j < count) {
            const int64_t x = a.tokens[first + j];
            if (x >= 0 && x < a.vocab) {
                const float p = to_f(target[j * a.target_stride + x]) * 0x1p100f;
                const float u = a.accept_u[first + j];
                float q = 0x1p100f;
                if constexpr (kDraft)
                    q = to_f(static_cast<const Q*>(a.draft)[(first + j) * a.draft_stride + x]) * 0x1p100f;
                const float h = u * q;
                ok = h < p || (h == p && fmaf(u, q, -h) < 0.0f);
            }
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, ok);
        const int n = mask == 0xffffffffu ? 32 : __ffs(~mask) - 1;
        accepted += n;
        if (n < 32) break;
    }
    const bool whole = accepted == count;
    if (rank == 0) {
        for (int64_t k = tid; k <= a.max_drafts; k += kVerifyThreads)
            if (k != accepted) out[k] = k < accepted ? a.tokens[first + k] : -1;
        if (tid == 0) a.out_accepted[b] = accepted;
    }

    Weights<P, Q, kVec> wt;
    wt.p = target + accepted * a.target_stride;
    wt.q = nullptr;
    wt.without = -1;
    wt.vocab = a.vocab;
    if (!whole) {
        if constexpr (kDraft) {
            wt.q = static_cast<const Q*>(a.draft) + (first + accepted) * a.draft_stride;
        } else {
            const int64_t x = a.tokens[first + accepted];
            if (x >= 0 && x < a.vocab) wt.without = static_cast<int>(x);
        }
    }

    // Each warp of the cluster owns `part` consecutive columns.
    const int part = a.part;
    Pair total{0.0f, 0.0f};
    int used = 0;  // the attempt whose totals count
    for (int attempt = 0; attempt < 2; ++attempt) {
        const int64_t begin64 = static_cast<int64_t>(rank * kVerifyWarps + warp) * part;
        const int begin = begin64 < a.vocab ? static_cast<int>(begin64) : a.vocab;
        const int end = begin64 + part < a.vocab ? static_cast<int>(begin64 + part) : a.vocab;
        Pair sum{0.0f, 0.0f};
        if (begin < end) {
            if (kDraft && wt.q) {
                if constexpr (kDraft) sum = lane_sum<true>(wt, begin, end, lane);
            } else {
                sum = lane_sum<false>(wt, begin, end, lane);
            }
        }
        sum = warp_sum_pair(sum);
        if (csize > 1 && attempt == 0) cluster_wait();  // the others' shared memory is there
        if (lane == 0) s_warp[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            const Pair cta = shfl(warp_scan_pair(lane < kVerifyWarps ? s_warp[lane] : Pair{0.0f, 0.0f}, lane, kVerifyWarps),
                                  kVerifyWarps - 1);
            const uint64_t bits = static_cast<uint64_t>(__float_as_uint(cta.c)) << 32 | __float_as_uint(cta.s);
            if (csize > 1) {
                if (lane < csize) store_remote(&s_cta[attempt][rank], lane, bits);
            } else if (lane == 0) {
                s_cta[attempt][0] = cta;
            }
        }
        if (csize > 1) cluster_sync_all();
        else __syncthreads();
        total = shfl(warp_scan_pair(lane < csize ? s_cta[attempt][lane] : Pair{0.0f, 0.0f}, lane, csize), csize - 1);
        // A refused draft whose p never exceeds its q (rounded
        // probabilities) draws from the target's own row.
        if (total.s > 0.0f || whole || attempt == 1) break;
        used = 1;
        wt.q = nullptr;
        wt.without = -1;
    }
    if (!(total.s > 0.0f)) {  // no mass anywhere
        if (rank == 0 && tid == 0) out[accepted] = -1;
        return;
    }

    // The share that holds the drawn column: the first whose running sum
    // exceeds the border; the last one with any mass where rounding (or u >= 1)
    // leaves none.
    const Border border(a.sample_u[b], total);
    Pair before{0.0f, 0.0f};
    const int cta = pick(s_cta[used], csize, lane, border, before);
    if (rank != cta) return;
    const int w = pick(s_warp, kVerifyWarps, lane, border, before);
    const int begin = (rank * kVerifyWarps + w) * part;
    const int end = begin + part < a.vocab ? begin + part : a.vocab;
    int last = -1;  // the last column with a weight that this thread saw
    for (int64_t at = begin; at < end; at += 8 * kVerifyThreads) {
        const int64_t i = at + 8 * tid;
        float v[8];
        wt.load(i, end, v);
        PairSum2 own;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e % 2) own.add(pack2(v[e - 1], v[e]));
            if (v[e] > 0.0f) last = static_cast<int>(i) + e;
        }
        const Pair sum = own.value(), scan = warp_scan_pair(sum, lane);
        if (lane == 31) s_scan[warp] = scan;
        if (tid == 0) s_first = INT_MAX;
        __syncthreads();
        Pair lower = before;
        for (int k = 0; k < warp; ++k) lower = lower + s_scan[k];
        if (sum.s > 0.0f && border.below(lower + scan)) atomicMin(&s_first, tid);
        const Pair left = shfl_up(scan, 1);
        __syncthreads();
        if (s_first == tid) {
            Pair run = lane > 0 ? lower + left : lower;
            int col = last;  // in this thread's eight, as its sum is positive
            for (int e = 0; e < 8; ++e) {
                run = run + Pair{v[e], 0.0f};
                if (v[e] > 0.0f && border.below(run)) {
                    col = static_cast<int>(i) + e;
                    break;
                }
            }
            out[accepted] = col;
        }
        if (s_first != INT_MAX) return;
        for (int k = 0; k < kVerifyWarps; ++k) before = before + s_scan[k];
        __syncthreads();
    }
    // The share's sum, added in another order, fell just short of the border.
    if (tid == 0) s_last = -1;
    __syncthreads();
    atomicMax(&s_last, last);
    __syncthreads();
    if (tid == 0) out[accepted] = s_last;
}

using VerifyKernel = void (*)(VerifyParams);

template <typename P, typename Q> VerifyKernel verify_kernel_of(bool vec) {
    return vec ? verify_kernel<P, Q, true> : verify_kernel<P, Q, false>;
}

template <typename P> VerifyKernel verify_kernel_for(bool draft, drs_dtype t, bool vec) {
    if (!draft) return verify_kernel_of<P, NoDraft>(vec);
    return with_dtype(t, [vec](auto q) -> VerifyKernel { return verify_kernel_of<P, decltype(q)>(vec); });
}

}  // namespace
}  // namespace drs

extern "C" drs_status drs_verify_drafts(const void* target, drs_dtype target_dtype, int64_t target_rows,
                                        int64_t target_stride, const void* draft, drs_dtype draft_dtype,
                                        int64_t draft_rows, int64_t draft_stride, int64_t vocab,
                                        const int64_t* draft_tokens, const int32_t* cu_drafts, int64_t requests,
                                        int32_t max_drafts, const float* accept_u, const float* sample_u,
                                        int64_t* out_tokens, int32_t* out_accepted, void* stream) {
    using namespace drs;
    if (requests < 0 || max_drafts < 0 || target_rows < 0 || draft_rows < 0) return DRS_ERR_INVALID_ARG;
    if (!dtype_ok(target_dtype) || (draft && !dtype_ok(draft_dtype))) return DRS_ERR_INVALID_ARG;
    if (vocab < 1 || target_stride < vocab || (draft && draft_stride < vocab)) return DRS_ERR_INVALID_ARG;
    if (vocab > DRS_MAX_VOCAB || requests > INT32_MAX / kMaxCluster) return DRS_ERR_UNSUPPORTED;
    if (requests == 0) return DRS_OK;
    if (!target || !cu_drafts || !sample_u || !out_tokens || !out_accepted) return DRS_ERR_INVALID_ARG;
    if (draft_rows > 0 && (!draft_tokens || !accept_u)) return DRS_ERR_INVALID_ARG;
    if (!aligned(target, dtype_bytes(target_dtype)) || (draft && !aligned(draft, dtype_bytes(draft_dtype))) ||
        !aligned(draft_tokens, 8) || !aligned(out_tokens, 8) || !aligned(cu_drafts, 4) || !aligned(accept_u, 4) ||
        !aligned(sample_u, 4) || !aligned(out_accepted, 4))
        return DRS_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms <= 0) return DRS_ERR_CUDA;

    VerifyParams a{};
    a.target = target;
    a.draft = draft;
    a.tokens = draft_tokens;
    a.cu = cu_drafts;
    a.accept_u = accept_u;
    a.sample_u = sample_u;
    a.out_tokens = out_tokens;
    a.out_accepted = out_accepted;
    a.target_rows = target_rows;
    a.target_stride = target_stride;
    a.draft_rows = draft_rows;
    a.draft_stride = draft_stride;
    a.vocab = static_cast<int32_t>(vocab);
    a.max_drafts = max_drafts;
    // CTAs per request: as many as are resident at once (about half an SM's
    // worth is lost to the grouping of clusters, more with 16), 8192 columns
    // (32 per thread) each at least. us at 262144 columns with 4, 8 and 16
    // CTAs: 32 requests 21.3, 14.1, 11.9; 64 requests 23.8, 17.7, 20.7;
    // 88 requests 26.2, 20.7, 26.6; 95 requests 26.9, 24.6, 27.7 (a second wave;
    // the rule takes 4 from 86 on).
    // Requests that fill several waves anyway: 32768 columns of 4 bytes per CTA
    // (256 requests 51.5, 48.0, 61.9 us; 55.6 with 2), or 65536 where that is
    // one wave (128 requests 29.4, 30.0).
    const size_t bytes = dtype_bytes(target_dtype) + (draft ? dtype_bytes(draft_dtype) : 1);
    const bool vec = aligned(target, 16) && target_stride * dtype_bytes(target_dtype) % 16 == 0 &&
                     (!draft || (aligned(draft, 16) && draft_stride * dtype_bytes(draft_dtype) % 16 == 0));
    const int64_t resident = int64_t{sms} * resident_ctas(bytes);
    int cluster = 1;
    while (cluster < kMaxCluster && vocab > 8192 * cluster &&
           requests * cluster * 2 <= resident - (cluster < 8 ? sms / 2 : sms * 3 / 2))
        cluster *= 2;
    const int64_t row = vocab * static_cast<int64_t>(draft ? bytes : bytes - 1);
    if (row > (int64_t{1} << 18) * cluster)
        while (cluster < 8 && row > (int64_t{1} << 17) * cluster) cluster *= 2;
    a.cluster = cluster;
    a.part = static_cast<int32_t>(ceil_div(ceil_div(vocab, cluster * kVerifyWarps), kStep) * kStep);

    const bool has_draft = draft != nullptr;
    const VerifyKernel kernel = with_dtype(target_dtype, [&](auto p) -> VerifyKernel {
        return verify_kernel_for<decltype(p)>(has_draft, draft_dtype, vec);
    });
    if (cluster > 8 && !prepare_kernel(reinterpret_cast<const void*>(kernel), 0, true)) return DRS_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(requests * cluster));
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, a));
}

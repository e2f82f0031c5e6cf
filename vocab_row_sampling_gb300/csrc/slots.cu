// slots.cu -- block tables and slot maps from request lengths
// (drs_map_slots).
//
// The requests are the work of one thread-block cluster: a few prefix sums,
// bound by latency, whose phases a cluster's barriers order without further
// launches or a workspace.
//   1. every CTA sums its share of the requests: new tokens, blocks to take
//      from the ring of free blocks, blocks to give back; the CTAs exchange
//      their sums through distributed shared memory;
//   2. every CTA writes its requests' offsets and counts and moves their
//      blocks between the table and the ring.
// The tokens then find their request in the offsets and look up their block:
// in the same launch where there are few, in a launch over all SMs (a
// programmatic dependent one) where there are many.
// Measured: 64 decoding requests 7.1 us, 32 canvases of 256 tokens 8.2, 4096
// requests with 262144 tokens 16.1 (11 for the requests, 5 for the tokens).
// The CTAs arrive at a cluster barrier when they begin and wait for it before
// they store into each other's shared memory; the first sums hide it.
// All sums are 64-bit integers in request order, so the blocks that a
// request gets do not depend on how the work is split.
#include <climits>

#include "token_common.cuh"

namespace drs {
namespace {

constexpr int kSlotThreads = 512;
constexpr int kSlotWarps = kSlotThreads / 32;
constexpr int kSlotCluster = 16;

struct SlotParams {
    const int32_t* lens;
    const int32_t* new_lens;
    const int32_t* held;
    int32_t* table;
    int32_t* ring;
    const int64_t* state;
    int32_t* out_cu;
    int32_t* out_request;
    int32_t* out_position;
    int64_t* out_slot;
    int32_t* out_held;
    int64_t* out_state;
    int32_t* out_lacking;
    int64_t table_stride, ring_size, capacity;
    int32_t requests, max_blocks, block, cluster;
};

// 64-bit divisions take about 100 instructions; almost every length fits 32.
__device__ __forceinline__ int64_t quotient(int64_t x, int32_t d) {
    if (static_cast<uint64_t>(x) >> 32) return x / d;
    return static_cast<uint32_t>(x) / static_cast<uint32_t>(d);
}

struct Sums {
    int64_t tokens, take, give;
    __device__ __forceinline__ Sums& operator+=(const Sums& o) {
        tokens += o.tokens, take += o.take, give += o.give;
        return *this;
    }
};

// What one request asks for. Negative lengths and counts are 0, a count
// of held blocks is at most the table's width.
struct Request {
    int64_t len, fresh;  // cached tokens, new tokens
    int32_t held, need;  // blocks; need is at most the table's width
    int64_t want;        // blocks the lengths ask for

    __device__ __forceinline__ static Request of(const SlotParams& a, int b) {
        Request r;
        r.len = max(a.lens[b], 0);
        r.fresh = max(a.new_lens[b], 0);
        r.held = min(max(a.held[b], 0), a.max_blocks);
        r.want = quotient(r.len + r.fresh + a.block - 1, a.block);
        r.need = static_cast<int32_t>(min(r.want, static_cast<int64_t>(a.max_blocks)));
        return r;
    }
    __device__ __forceinline__ Sums sums() const {
        return Sums{fresh, static_cast<int64_t>(max(need - held, 0)), static_cast<int64_t>(max(held - need, 0))};
    }
};

// A counter of the ring as a place in it.
__device__ __forceinline__ int64_t ring_start(int64_t counter, int64_t size) {
    const uint64_t c = static_cast<uint64_t>(counter), n = static_cast<uint64_t>(size);
    if ((c | n) >> 32) return static_cast<int64_t>(c % n);
    return static_cast<uint32_t>(c) % static_cast<uint32_t>(n);
}

// The place `offset` entries after `place` in the ring. Offsets are below
// the ring's size where its counters are consistent.
__device__ __forceinline__ int64_t ring_place(int64_t place, int64_t offset, int64_t size) {
    int64_t at = place + offset;
    if (at >= size) {
        at -= size;
        if (at >= size) at %= size;
    }
    return at;
}

constexpr int kOwnMoves = 4;    // blocks of a request that its thread moves by itself
constexpr int kMoveChunk = 128;  // further ones a warp moves at once, four per lane

// The blocks of a request past its first kOwnMoves.
struct LongMove {
    int32_t* row;  // the first block's place in the table
    int64_t from;  // its offset from the ring's head or tail
    int32_t n;
    bool take;
};

// The request, position and slot of token t of request b, whose first
// token is `first`.
__device__ __forceinline__ void map_token(const SlotParams& a, int64_t t, int b, int32_t first, int32_t len, int32_t now,
                                          const int32_t* row) {
    const int64_t at = max(len, 0) + (t - first);
    const int64_t col = quotient(at, a.block);
    int64_t slot = -1;
    if (col < now) slot = static_cast<int64_t>(__ldcg(row + col)) * a.block + (at - col * a.block);
    a.out_request[t] = b;
    a.out_position[t] = static_cast<int32_t>(min(at, static_cast<int64_t>(INT_MAX)));
    a.out_slot[t] = slot;
}

__device__ __forceinline__ void pad_token(const SlotParams& a, int64_t t) {
    a.out_request[t] = -1;
    a.out_position[t] = 0;
    a.out_slot[t] = -1;
}

// The tokens of warp `w` of `warps`: a run of groups of 32. kSame: the
// offsets were written by this launch and are read from L2; else by the one
// before, and L1 serves the probes that all warps share (from L2 they took
// 10 of 13 us at 262144 tokens: every warp asks for the same lines).
template <bool kSame> __device__ __forceinline__ void map_tokens(const SlotParams& a, int w, int warps, int lane) {
    const auto offset = [&](int b) { return kSame ? __ldcg(a.out_cu + b) : a.out_cu[b]; };
    const int groups = static_cast<int>(ceil_div(a.capacity, 32));
    const int per = groups / warps, rest = groups % warps;
    const int g0 = w * per + min(w, rest), g1 = g0 + per + (w < rest);
    if (g0 >= g1) return;
    const int32_t total = offset(a.requests);
    // the request of the first token, the last b with out_cu[b] <= t: each
    // step takes 32 probes
    int b = 0;
    for (int n = a.requests; n > 1;) {
        const int step = (n + 31) / 32;
        const int at = lane * step;
        const bool below = at < n && offset(b + at) <= g0 * 32;
        const int hit = __popc(__ballot_sync(0xffffffffu, below)) - 1;  // lane 0 is below
        b += hit * step;
        n = min(step, n - hit * step);
    }
    int32_t start = offset(b);
    for (int g = g0; g < g1; ++g) {
        const int64_t t = static_cast<int64_t>(g) * 32 + lane;
        if (static_cast<int64_t>(g) * 32 < total) {
            // the next 32 offsets; a token's request follows from how many
            // of them are not above it
            const int32_t next = b + 1 + lane <= a.requests ? offset(b + 1 + lane) : INT_MAX;
            int n = 0;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1)
                if (__shfl_sync(0xffffffffu, next, n + s - 1) <= t) n += s;
            int request = b + n;
            int32_t first = __shfl_sync(0xffffffffu, next, n > 0 ? n - 1 : 0);
            if (n == 0) first = start;
            if (__shfl_sync(0xffffffffu, next, 31) <= t && t < total) {
                // over 31 requests without tokens between two tokens
                int below = request, above = a.requests;
                while (above - below > 1) {
                    const int mid = below + (above - below) / 2;
                    if (offset(mid) <= t) below = mid;
                    else above = mid;
                }
                request = below;
                first = offset(below);
            }
            if (t < total) {
                const int32_t len = a.lens[request], now = kSame ? __ldcg(a.out_held + request) : a.out_held[request];
                map_token(a, t, request, first, len, now, a.table + request * a.table_stride);
            }
            b = __shfl_sync(0xffffffffu, request, 31);  // past the last token: not used again
            start = __shfl_sync(0xffffffffu, first, 31);
        }
        if (t >= total && t < a.capacity) pad_token(a, t);
    }
}

constexpr int kStage = 1024;  // requests whose offsets fit a CTA's shared memory

template <bool kTokens> __global__ void __launch_bounds__(kSlotThreads) slots_kernel(const SlotParams a) {
    __shared__ Sums s_warp[kSlotWarps];
    __shared__ Sums s_all;
    __shared__ int64_t s_cta[kSlotCluster][3];  // every CTA's sums
    __shared__ int64_t s_end[kSlotCluster][2];  // blocks taken and lacking, by CTA
    __shared__ unsigned long long s_taken, s_lacking;
    __shared__ LongMove s_move[kSlotThreads];
    __shared__ int s_moves;
    __shared__ int32_t s_cu[kTokens ? kStage + 1 : 1], s_len[kTokens ? kStage : 1], s_now[kTokens ? kStage : 1];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int csize = a.cluster, rank = csize > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int share = static_cast<int>(ceil_div(a.requests, csize));
    const int lo = min(rank * static_cast<int64_t>(share), static_cast<int64_t>(a.requests));
    const int hi = min(lo + static_cast<int64_t>(share), static_cast<int64_t>(a.requests));
    // a thread takes consecutive requests
    const int run = static_cast<int>(ceil_div(hi - lo, kSlotThreads));
    const int b0 = min(lo + static_cast<int64_t>(tid) * run, static_cast<int64_t>(hi));
    const int b1 = min(b0 + run, hi);

    if (csize > 1) cluster_arrive();
    if constexpr (!kTokens) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t head = a.state[0], tail = a.state[1];
    int64_t avail = tail - head;
    avail = avail < 0 ? 0 : avail > a.ring_size ? a.ring_size : avail;
    if (tid == 0) s_taken = 0, s_lacking = 0, s_moves = 0;

    // 1. sums before this thread's requests
    Sums mine{0, 0, 0};
    for (int b = b0; b < b1; ++b) mine += Request::of(a, b).sums();
    Sums at{warp_scan_inclusive(mine.tokens, lane), warp_scan_inclusive(mine.take, lane),
            warp_scan_inclusive(mine.give, lane)};
    if (csize > 1) cluster_wait();  // the others' shared memory is there
    if (lane == 31) s_warp[warp] = at;
    at.tokens -= mine.tokens, at.take -= mine.take, at.give -= mine.give;
    __syncthreads();
    if (warp == 0) {  // the warps' sums become the sums before them
        const Sums own = lane < kSlotWarps ? s_warp[lane] : Sums{0, 0, 0};
        const Sums upto{warp_scan_inclusive(own.tokens, lane), warp_scan_inclusive(own.take, lane),
                        warp_scan_inclusive(own.give, lane)};
        if (lane < kSlotWarps) s_warp[lane] = Sums{upto.tokens - own.tokens, upto.take - own.take, upto.give - own.give};
        if (csize > 1) {
            const Sums all{__shfl_sync(0xffffffffu, upto.tokens, 31), __shfl_sync(0xffffffffu, upto.take, 31),
                           __shfl_sync(0xffffffffu, upto.give, 31)};
            if (lane < csize) {
                store_remote(&s_cta[rank][0], lane, static_cast<uint64_t>(all.tokens));
                store_remote(&s_cta[rank][1], lane, static_cast<uint64_t>(all.take));
                store_remote(&s_cta[rank][2], lane, static_cast<uint64_t>(all.give));
            }
        } else if (lane == 31) {
            s_all = upto;
        }
    }
    if (csize > 1) {
        cluster_sync_all();
        if (warp == 0) {  // and the sums of the CTAs before this one
            const Sums own = lane < csize ? Sums{s_cta[lane][0], s_cta[lane][1], s_cta[lane][2]} : Sums{0, 0, 0};
            const Sums upto{warp_scan_inclusive(own.tokens, lane), warp_scan_inclusive(own.take, lane),
                            warp_scan_inclusive(own.give, lane)};
            Sums before{__shfl_up_sync(0xffffffffu, upto.tokens, 1), __shfl_up_sync(0xffffffffu, upto.take, 1),
                        __shfl_up_sync(0xffffffffu, upto.give, 1)};
            if (lane == 31) s_all = upto;
            if (lane == 0) before = Sums{0, 0, 0};
            const Sums add{__shfl_sync(0xffffffffu, before.tokens, rank), __shfl_sync(0xffffffffu, before.take, rank),
                           __shfl_sync(0xffffffffu, before.give, rank)};
            if (lane < kSlotWarps) s_warp[lane] += add;
        }
    }
    __syncthreads();
    at += s_warp[warp];
    const Sums all = s_all;

    // 2. the requests' outputs and the moves of blocks: a few by the
    // request's thread, longer ones by all warps (a request that ends gives
    // hundreds of blocks back).
    const int64_t head_at = ring_start(head, a.ring_size), tail_at = ring_start(tail, a.ring_size);
    int64_t taken = 0, lacking = 0;
    for (int k = 0; k < run; ++k) {
        const int b = b0 + k;
        const bool have = b < b1;
        Request r{};
        Sums s{0, 0, 0};
        int32_t now = 0;
        if (have) {
            r = Request::of(a, b);
            s = r.sums();
            const bool served = at.take + s.take <= avail;
            now = served ? r.need : min(r.need, r.held);
            if (served) taken += s.take;
            lacking += r.want - now;
            const int32_t cu = static_cast<int32_t>(min(at.tokens, a.capacity));
            a.out_cu[b] = cu;
            a.out_held[b] = now;
            if (kTokens && csize == 1 && a.requests <= kStage) s_cu[b] = cu, s_len[b] = static_cast<int32_t>(r.len), s_now[b] = now;
        }
        // blocks taken: ring -> columns [held, now); given: columns [need, held) -> ring
        const bool takes = now > r.held;
        const int32_t moves = have ? takes ? now - r.held : max(r.held - r.need, 0) : 0;
        const int32_t col = takes ? r.held : r.need;
        const int64_t from = takes ? at.take : at.give;
        int32_t* const row = a.table + b * a.table_stride + col;
        int32_t ids[kOwnMoves];
#pragma unroll
        for (int i = 0; i < kOwnMoves; ++i)
            if (i < moves) ids[i] = takes ? a.ring[ring_place(head_at, from + i, a.ring_size)] : row[i];
#pragma unroll
        for (int i = 0; i < kOwnMoves; ++i)
            if (i < moves) (takes ? row[i] : a.ring[ring_place(tail_at, from + i, a.ring_size)]) = ids[i];
        if (moves > kOwnMoves) s_move[atomicAdd(&s_moves, 1)] = LongMove{row, from, moves, takes};
        __syncthreads();
        // chunks of the long moves, dealt out to the warps
        const int n = s_moves;
        for (int m = 0; m < n; ++m) {
            const LongMove e = s_move[m];
            for (int64_t c = (warp - m) & (kSlotWarps - 1); kOwnMoves + c * kMoveChunk < e.n; c += kSlotWarps) {
                const int64_t i = kOwnMoves + c * kMoveChunk + lane;
                int32_t id[kMoveChunk / 32];
#pragma unroll
                for (int u = 0; u < kMoveChunk / 32; ++u)
                    if (i + 32 * u < e.n)
                        id[u] = e.take ? a.ring[ring_place(head_at, e.from + i + 32 * u, a.ring_size)] : e.row[i + 32 * u];
#pragma unroll
                for (int u = 0; u < kMoveChunk / 32; ++u)
                    if (i + 32 * u < e.n)
                        (e.take ? e.row[i + 32 * u] : a.ring[ring_place(tail_at, e.from + i + 32 * u, a.ring_size)]) = id[u];
            }
        }
        if (k + 1 < run) {  // the list is used again
            __syncthreads();
            if (tid == 0) s_moves = 0;
            __syncthreads();
        }
        at += s;
    }
    taken = warp_sum(taken), lacking = warp_sum(lacking);
    if (lane == 0) {
        if (taken) atomicAdd(&s_taken, static_cast<unsigned long long>(taken));
        if (lacking) atomicAdd(&s_lacking, static_cast<unsigned long long>(lacking));
    }
    if (rank == 0 && tid == 0) a.out_cu[a.requests] = static_cast<int32_t>(min(all.tokens, a.capacity));
    __syncthreads();
    if (tid < 2) {
        const uint64_t v = tid == 0 ? s_taken : s_lacking;
        if (csize > 1) store_remote(&s_end[rank][tid], 0, v);
        else s_end[0][tid] = static_cast<int64_t>(v);
    }
    if (csize > 1) cluster_sync_all();
    else __syncthreads();
    if (rank == 0 && tid == 0) {
        int64_t sum[2] = {0, 0};
        for (int c = 0; c < csize; ++c) sum[0] += s_end[c][0], sum[1] += s_end[c][1];
        a.out_state[0] = head + sum[0];
        a.out_state[1] = tail + all.give;
        *a.out_lacking = static_cast<int32_t>(min(sum[1], static_cast<int64_t>(INT_MAX)));
    }
    if constexpr (kTokens) {
        if (a.requests > kStage) {
            map_tokens<true>(a, rank * kSlotWarps + warp, csize * kSlotWarps, lane);
            return;
        }
        const int32_t total = static_cast<int32_t>(min(all.tokens, a.capacity));
        if (csize > 1) {
            for (int b = tid; b < a.requests; b += kSlotThreads) {
                s_cu[b] = __ldcg(a.out_cu + b);
                s_len[b] = a.lens[b];
                s_now[b] = __ldcg(a.out_held + b);
            }
            __syncthreads();
        }
        for (int64_t t = rank * kSlotThreads + tid; t < a.capacity; t += csize * kSlotThreads) {
            if (t >= total) {
                pad_token(a, t);
                continue;
            }
            int below = 0, above = a.requests;  // s_cu[below] <= t < s_cu[above]
            while (above - below > 1) {
                const int mid = (below + above) / 2;
                if (s_cu[mid] <= t) below = mid;
                else above = mid;
            }
            map_token(a, t, below, s_cu[below], s_len[below], s_now[below], a.table + below * a.table_stride);
        }
    }
}

constexpr int kTokenThreads = 256;
constexpr int kTokenWarps = kTokenThreads / 32;

__global__ void __launch_bounds__(kTokenThreads) slot_tokens_kernel(const SlotParams a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    map_tokens<false>(a, blockIdx.x * kTokenWarps + (threadIdx.x >> 5), gridDim.x * kTokenWarps, threadIdx.x & 31);
}

}  // namespace
}  // namespace drs

extern "C" drs_status drs_map_slots(const int32_t* lens, const int32_t* new_lens, const int32_t* held,
                                    int64_t requests, int32_t block_size, int32_t* block_table,
                                    int64_t table_stride, int32_t max_blocks, int32_t* free_ring, int64_t ring_size,
                                    const int64_t* ring_state, int64_t capacity, int32_t* out_cu,
                                    int32_t* out_request, int32_t* out_position, int64_t* out_slot,
                                    int32_t* out_held, int64_t* out_ring_state, int32_t* out_lacking, void* stream) {
    using namespace drs;
    if (requests < 0 || block_size < 1 || max_blocks < 1 || table_stride < max_blocks || ring_size < 1 || capacity < 0)
        return DRS_ERR_INVALID_ARG;
    if (requests > DRS_MAX_REQUESTS || capacity > INT32_MAX) return DRS_ERR_UNSUPPORTED;
    if (!ring_state || !out_cu || !out_ring_state || !out_lacking || !free_ring) return DRS_ERR_INVALID_ARG;
    if (requests > 0 && (!lens || !new_lens || !held || !block_table || !out_held)) return DRS_ERR_INVALID_ARG;
    if (capacity > 0 && (!out_request || !out_position || !out_slot)) return DRS_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(lens), static_cast<const void*>(new_lens),
                          static_cast<const void*>(held), static_cast<const void*>(block_table),
                          static_cast<const void*>(free_ring), static_cast<const void*>(out_cu),
                          static_cast<const void*>(out_request), static_cast<const void*>(out_position),
                          static_cast<const void*>(out_held), static_cast<const void*>(out_lacking)})
        if (!aligned(p, 4)) return DRS_ERR_INVALID_ARG;
    if (!aligned(ring_state, 8) || !aligned(out_slot, 8) || !aligned(out_ring_state, 8)) return DRS_ERR_INVALID_ARG;
    // out_held and out_ring_state may be held and ring_state themselves: a
    // request's count is read and written by one thread, the counters are read
    // at the start and written after the last barrier
    if (out_held && (out_held == lens || out_held == new_lens)) return DRS_ERR_INVALID_ARG;

    const int sms = sm_count();
    if (sms <= 0) return DRS_ERR_CUDA;

    SlotParams a{};
    a.lens = lens;
    a.new_lens = new_lens;
    a.held = held;
    a.table = block_table;
    a.ring = free_ring;
    a.state = ring_state;
    a.out_cu = out_cu;
    a.out_request = out_request;
    a.out_position = out_position;
    a.out_slot = out_slot;
    a.out_held = out_held;
    a.out_state = out_ring_state;
    a.out_lacking = out_lacking;
    a.table_stride = table_stride;
    a.ring_size = ring_size;
    a.capacity = capacity;
    a.requests = static_cast<int32_t>(requests);
    a.max_blocks = max_blocks;
    a.block = block_size;
    // Few tokens: one launch. Many: the cluster for the requests, then a launch
    // for the tokens. us in one and in two launches: 64 requests, 512 tokens
    // 6.7, 8.0; 512 requests, 2048 tokens 9.2, 10.1; 32 requests, 8192 tokens 8.1, 7.9;
    // 64 requests, 16384 tokens 9.6, 8.4; 128 requests, 32768 tokens 11.3, 8.7.
    const bool apart = capacity > kSlotCluster * kSlotThreads;
    // One CTA, or a cluster of 16, by the requests (256 per CTA), the tokens
    // that the cluster maps itself and, apart from them, the blocks that they
    // may take. us with 1, 4 and 16 CTAs: 64 requests, 512 tokens 6.7, 7.9, 7.9;
    // 512 requests, 2048 tokens 13.1, 9.6, 9.2; 4096 requests, 262144 tokens 63.7,
    // 25.3, 16.0; 128 requests, 32768 tokens (512 blocks) 8.7, 9.4, 9.6.
    int64_t work = requests * 2;
    if (!apart && capacity > work) work = capacity;
    if (apart && capacity / block_size > work) work = capacity / block_size;
    const int cluster = work <= kSlotThreads ? 1 : kSlotCluster;
    a.cluster = cluster;
    const auto kernel = apart ? slots_kernel<false> : slots_kernel<true>;
    if (cluster > 8 && !prepare_kernel(reinterpret_cast<const void*>(kernel), 0, true)) return DRS_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(kSlotThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return DRS_ERR_CUDA;
    if (!apart) return DRS_OK;
    // up to 8 CTAs per SM, a group of 32 tokens per warp at least
    const int64_t blocks = ceil_div(capacity, 32 * kTokenWarps);
    cudaLaunchConfig_t next{};
    next.gridDim = dim3(static_cast<unsigned>(blocks < sms * 8 ? blocks : sms * 8));
    next.blockDim = dim3(kTokenThreads);
    next.stream = cfg.stream;
    cudaLaunchAttribute dependent[1];
    dependent[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    dependent[0].val.programmaticStreamSerializationAllowed = 1;
    next.attrs = dependent;
    next.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&next, slot_tokens_kernel, a));
}

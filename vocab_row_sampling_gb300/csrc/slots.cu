// slots.cu -- block tables and slot maps from request lengths
// (drs_map_slots).
//
// One launch of one thread-block cluster: the call is a few prefix sums over
// the requests and one look-up per token, bound by latency, and a cluster's
// barriers order its phases without a second launch or a workspace.
//   1. every CTA sums its share of the requests: new tokens, blocks to take
//      from the ring of free blocks, blocks to give back; the CTAs exchange
//      their sums through distributed shared memory;
//   2. every CTA writes its requests' offsets and counts and moves their
//      blocks between the table and the ring;
//   3. every CTA finds the request of its share of the tokens by binary
//      search and looks up its block.
// All sums are 64-bit integers in request order, so the blocks that a
// request gets do not depend on how the work is split.
#include <climits>

#include "token_common.cuh"

namespace drs {
namespace {

constexpr int kSlotThreads = 1024;
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
        r.want = (r.len + r.fresh + a.block - 1) / a.block;
        r.need = static_cast<int32_t>(min(r.want, static_cast<int64_t>(a.max_blocks)));
        return r;
    }
    __device__ __forceinline__ Sums sums() const {
        return Sums{fresh, static_cast<int64_t>(max(need - held, 0)), static_cast<int64_t>(max(held - need, 0))};
    }
};

// A place of the ring, for any 64-bit counter.
__device__ __forceinline__ int64_t ring_place(int64_t counter, int64_t size) {
    return static_cast<int64_t>(static_cast<uint64_t>(counter) % static_cast<uint64_t>(size));
}

__global__ void __launch_bounds__(kSlotThreads) slots_kernel(const SlotParams a) {
    __shared__ Sums s_warp[kSlotWarps];
    __shared__ int64_t s_cta[kSlotCluster][3];  // every CTA's sums
    __shared__ int64_t s_end[kSlotCluster][2];  // blocks taken and lacking, by CTA
    __shared__ unsigned long long s_taken, s_lacking;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int csize = a.cluster, rank = csize > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int share = static_cast<int>(ceil_div(a.requests, csize));
    const int lo = min(rank * static_cast<int64_t>(share), static_cast<int64_t>(a.requests));
    const int hi = min(lo + static_cast<int64_t>(share), static_cast<int64_t>(a.requests));
    // a thread takes consecutive requests
    const int run = static_cast<int>(ceil_div(hi - lo, kSlotThreads));
    const int b0 = min(lo + static_cast<int64_t>(tid) * run, static_cast<int64_t>(hi));
    const int b1 = min(b0 + run, hi);

    const int64_t head = a.state[0], tail = a.state[1];
    int64_t avail = tail - head;
    avail = avail < 0 ? 0 : avail > a.ring_size ? a.ring_size : avail;
    if (tid == 0) s_taken = 0, s_lacking = 0;

    // 1. sums before this thread's requests
    Sums mine{0, 0, 0};
    for (int b = b0; b < b1; ++b) mine += Request::of(a, b).sums();
    Sums at{warp_scan_inclusive(mine.tokens, lane), warp_scan_inclusive(mine.take, lane),
            warp_scan_inclusive(mine.give, lane)};
    if (lane == 31) s_warp[warp] = at;
    __syncthreads();
    at.tokens -= mine.tokens, at.take -= mine.take, at.give -= mine.give;
    Sums all{0, 0, 0};
    for (int w = 0; w < kSlotWarps; ++w) {
        if (w < warp) at += s_warp[w];
        all += s_warp[w];
    }
    if (tid < csize) {
        const int64_t v[3] = {all.tokens, all.take, all.give};
        for (int i = 0; i < 3; ++i) {
            if (csize > 1) store_remote(&s_cta[rank][i], tid, static_cast<uint64_t>(v[i]));
            else s_cta[0][i] = v[i];
        }
    }
    if (csize > 1) cluster_sync_all();
    else __syncthreads();
    all = Sums{0, 0, 0};
    for (int c = 0; c < csize; ++c) {
        const Sums s{s_cta[c][0], s_cta[c][1], s_cta[c][2]};
        if (c < rank) at += s;
        all += s;
    }

    // 2. the requests' outputs and the moves of blocks. Warps stay whole:
    // long moves are made by all lanes.
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
            a.out_cu[b] = static_cast<int32_t>(min(at.tokens, a.capacity));
            a.out_held[b] = now;
        }
        const int32_t moves = have ? max(now - r.held, 0) + max(r.held - r.need, 0) : 0;
        for (uint32_t todo = __ballot_sync(0xffffffffu, moves > 0); todo; todo &= todo - 1) {
            const int src = __ffs(todo) - 1;
            const int32_t n = __shfl_sync(0xffffffffu, moves, src);
            const int32_t held = __shfl_sync(0xffffffffu, r.held, src);
            const int32_t need = __shfl_sync(0xffffffffu, r.need, src);
            const int64_t from = head + __shfl_sync(0xffffffffu, at.take, src);
            const int64_t to = tail + __shfl_sync(0xffffffffu, at.give, src);
            int32_t* const row = a.table + __shfl_sync(0xffffffffu, b, src) * a.table_stride;
            for (int32_t i = lane; i < n; i += 32) {
                if (need > held) row[held + i] = a.ring[ring_place(from + i, a.ring_size)];
                else a.ring[ring_place(to + i, a.ring_size)] = row[need + i];
            }
        }
        at += s;
    }
    if (taken) atomicAdd(&s_taken, static_cast<unsigned long long>(taken));
    if (lacking) atomicAdd(&s_lacking, static_cast<unsigned long long>(lacking));
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

    // 3. the tokens. What the cluster wrote is read from L2.
    const int64_t total = min(all.tokens, a.capacity);
    const int64_t step = static_cast<int64_t>(csize) * kSlotThreads;
    for (int64_t t = static_cast<int64_t>(rank) * kSlotThreads + tid; t < a.capacity; t += step) {
        int32_t request = -1, position = 0;
        int64_t slot = -1;
        if (t < total) {
            int below = 0, above = a.requests;  // out_cu[below] <= t < out_cu[above]
            while (above - below > 1) {
                const int mid = below + (above - below) / 2;
                if (__ldcg(a.out_cu + mid) <= t) below = mid;
                else above = mid;
            }
            request = below;
            const int64_t at_token = max(a.lens[below], 0) + (t - __ldcg(a.out_cu + below));
            position = static_cast<int32_t>(min(at_token, static_cast<int64_t>(INT_MAX)));
            const int64_t col = at_token / a.block;
            if (col < __ldcg(a.out_held + below))
                slot = static_cast<int64_t>(__ldcg(a.table + below * a.table_stride + col)) * a.block + at_token % a.block;
        }
        a.out_request[t] = request;
        a.out_position[t] = position;
        a.out_slot[t] = slot;
    }
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
    // out_held and out_ring_state may be held and ring_state themselves (read
    // before the cluster's first barrier, written after it)
    if (out_held && (out_held == lens || out_held == new_lens)) return DRS_ERR_INVALID_ARG;

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
    const int64_t work = capacity > requests ? capacity : requests;
    int cluster = 1;
    while (cluster < kSlotCluster && work > static_cast<int64_t>(cluster) * kSlotThreads) cluster *= 2;
    a.cluster = cluster;
    if (cluster > 8 &&
        cudaFuncSetAttribute(reinterpret_cast<const void*>(slots_kernel),
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return DRS_ERR_CUDA;
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
    return cuda_status(cudaLaunchKernelEx(&cfg, slots_kernel, a));
}

// Eviction from a paged cache by accumulated attention weight.
//
// Two kernels. The first, a CTA for each (request, key/value head), selects: of the tokens between the first
// `sinks` and the newest `recent` the K = budget - sinks - recent heaviest stay. Weights are >= 0, so their
// bits order as whole numbers; a radix selection over digits of 11, 11 and 10 bits finds the
// K-th largest key and how many of its equals are needed (the lower places). One ordered pass then writes
// the places that stay, ascending, to `kept`. Chains of barriers and shared-memory atomics bound it: 20 us for up to
// 8192 places of 192 (request, head) pairs. Grouping a warp's equal digits before the atomics took 53 us.
//
// The second moves rows: place kept[i] -> i. kept[i] >= i and ascending, so a CTA that walks the places in
// blocks may write block b once every thread has read it: the sources of later blocks lie at or behind their own
// destinations, past everything written so far. Blocks depend on each other only within a (request, head, array,
// slice of the row), so keys, values, weights and slices of a row are CTAs of their own. Its bytes bound it where there
// are many requests: 96 of 8192 places to 4096, 816 MB, both kernels in 138 to 142 us a call among calls on other caches, 179
// to 197 us on the same cache again and again (25 of them the selection). Loads of the block after next held in registers left
// room for fewer CTAs (286 us of the latter kind), a ring of bulk copies in shared memory 314 us.
#include "kv_cache.cuh"

namespace sala {
namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kCached = 8192;    // keys held in shared memory; those behind are read again

struct EvictArgs {
    int budget, sinks, recent;
    int32_t *new_lens, *kept;
};

__device__ __forceinline__ uint32_t key_of(float w) { return w > 0.f ? __float_as_uint(w) : 0u; }

// Exclusive prefix of two counts (16 bits would not hold them: a pair of words) over the block.
__device__ __forceinline__ int2 block_prefix(bool a, bool b, int2 *warp_sums, int2 *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned ma = __ballot_sync(0xffffffffu, a), mb = __ballot_sync(0xffffffffu, b);
    const unsigned below = (1u << lane) - 1u;
    __syncthreads();   // the sums of the pass before are read
    if (lane == 0) warp_sums[warp] = make_int2(__popc(ma), __popc(mb));
    __syncthreads();
    int2 mine = warp_sums[lane], sum = mine;   // kSelWarps == 32
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum.x, o), y = __shfl_up_sync(0xffffffffu, sum.y, o);
        if (lane >= o) sum.x += x, sum.y += y;
    }
    total->x = __shfl_sync(0xffffffffu, sum.x, 31);
    total->y = __shfl_sync(0xffffffffu, sum.y, 31);
    const int px = __shfl_sync(0xffffffffu, sum.x - mine.x, warp), py = __shfl_sync(0xffffffffu, sum.y - mine.y, warp);
    return make_int2(px + __popc(ma & below), py + __popc(mb & below));
}
static_assert(kSelWarps == 32, "one lane for each warp's sum");

__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(const KvArgs c, const EvictArgs a) {
    __shared__ uint32_t keys[kCached];
    __shared__ int hist[kBins];
    __shared__ int2 warp_sums[32];
    __shared__ int found_bin, found_rank;
    dependent_start();
    const int64_t n = blockIdx.x / c.H;
    const int h = static_cast<int>(blockIdx.x - n * c.H), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = kv::request_len(c, n);
    int32_t *kept = a.kept + static_cast<int64_t>(blockIdx.x) * a.budget;
    if (h == 0 && tid == 0 && a.new_lens) a.new_lens[n] = min(len, a.budget);
    if (len <= a.budget) {
        for (int i = tid; i < a.budget; i += kSelThreads) kept[i] = i < len ? i : -1;
        return;
    }
    const int s = a.sinks, e = len - a.recent, K = a.budget - a.sinks - a.recent;
    auto load = [&](int i) -> uint32_t {
        const int page = kv::page_of(c, n, i);
        return page < 0 ? 0u : key_of(c.weights[kv::row_of(c, page, h, i)]);
    };
    constexpr int kAtOnce = 8;   // lookups in flight: pages first, then weights
    for (int b = s; b < min(e, s + kCached); b += kAtOnce * kSelThreads) {
        int page[kAtOnce];
        float w[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int i = b + u * kSelThreads + tid;
            page[u] = i < min(e, s + kCached) ? kv::load(c.table + n * c.W + (i >> c.log_S)) : -1;
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int i = b + u * kSelThreads + tid;
            if (i >= min(e, s + kCached)) break;
            const bool known = page[u] >= 0 && page[u] < c.P;
            if (!known) record_status(c.status, SALA_ERR_BAD_INDEX);
            w[u] = known ? c.weights[kv::row_of(c, page[u], h, i)] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int i = b + u * kSelThreads + tid;
            if (i < min(e, s + kCached)) keys[i - s] = key_of(w[u]);
        }
    }
    __syncthreads();
    auto key = [&](int i) -> uint32_t { return i - s < kCached ? keys[i - s] : load(i); };

    // the K-th largest key, digit by digit; `need` of the keys equal to it stay
    uint32_t threshold = 0xffffffffu, prefix = 0;
    int need = K;
    if (K > 0) {
        const int shifts[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
        uint32_t mask = 0;
#pragma unroll 1
        for (int d = 0; d < 3; ++d) {
            for (int b = tid; b < kBins; b += kSelThreads) hist[b] = 0;
            __syncthreads();
            const uint32_t digits = (1u << bits[d]) - 1u;
            for (int i = s + tid; i < e; i += kSelThreads) {
                const uint32_t k = key(i);
                if ((k & mask) == prefix) atomicAdd(&hist[(k >> shifts[d]) & digits], 1);
            }
            __syncthreads();
            // thread t holds the bins 2 * (1023 - t) + 1 and below it: counted from the top
            const int b1 = 2 * (kSelThreads - 1 - tid) + 1;
            const int c1 = hist[b1], c0 = hist[b1 - 1];
            int run = c1 + c0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += x;
            }
            if (lane == 31) warp_sums[warp].x = run;
            __syncthreads();
            const int before_warp = lane < warp ? warp_sums[lane].x : 0;
            const int before = __reduce_add_sync(0xffffffffu, before_warp) + run - c1 - c0;   // keys in higher bins
            if (before < need && need <= before + c1) found_bin = b1, found_rank = need - before;
            else if (before + c1 < need && need <= before + c1 + c0) found_bin = b1 - 1, found_rank = need - before - c1;
            __syncthreads();
            prefix |= static_cast<uint32_t>(found_bin) << shifts[d];
            mask |= digits << shifts[d];
            need = found_rank;
        }
        threshold = prefix;
    }
    int above = 0, equal = 0;   // stayed so far: forced or heavier, and equal ones that are needed
    const int blocks = (len + kSelThreads - 1) / kSelThreads;
    for (int b = 0; b < blocks; ++b) {
        const int i = b * kSelThreads + tid;
        const bool in = i < len, middle = in && i >= s && i < e;
        const uint32_t k = middle ? key(i) : 0u;
        const bool up = in && (!middle || (K > 0 && k > threshold)), eq = middle && K > 0 && k == threshold;
        int2 total;
        const int2 p = block_prefix(up, eq, warp_sums, &total);
        const int rank = equal + p.y;   // of the equals
        const int at = above + p.x + min(rank, need);   // below the budget, unless a caller's race changes the weights meanwhile
        if ((up || (eq && rank < need)) && at < a.budget) kept[at] = i;
        above += total.x;
        equal += total.y;
    }
}

constexpr int kMoveThreads = 256, kEach = 4;

// Rows kept[i] -> i of one array of one (request, head), `bytes` of a row from `offset` on: 16 bytes a thread and row.
__device__ __forceinline__ void move_rows(const KvArgs &c, int64_t n, int h, const int32_t *kept, int first, int count,
                                          uint8_t *base, int row_bytes, int offset, int bytes) {
    const int per_row = bytes / 16, rows = kMoveThreads / per_row;   // threads of a row, rows at once
    const int row0 = threadIdx.x / per_row;
    base += offset + threadIdx.x % per_row * 16;
    for (int b = first; b < count; b += rows * kEach) {
        uint4 x[kEach];
        int src[kEach], to[kEach];   // pages of row i; -1: it stays as it is
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = b + row0 + e * rows;
            src[e] = i < count ? kv::load(kept + i) : -1;
        }
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = b + row0 + e * rows;
            const bool moves = src[e] >= 0 && src[e] != i;
            const int p = moves ? kv::page_of(c, n, src[e]) : -1;
            to[e] = p >= 0 ? kv::page_of(c, n, i) : -1;
            if (to[e] >= 0) x[e] = *reinterpret_cast<const uint4 *>(base + kv::row_of(c, p, h, src[e]) * row_bytes);
        }
        __syncthreads();   // every source of this block is read
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            if (to[e] >= 0) *reinterpret_cast<uint4 *>(base + kv::row_of(c, to[e], h, b + row0 + e * rows) * row_bytes) = x[e];
    }
}

// The weights of one (request, head), a thread a place.
__device__ __forceinline__ void move_weights(const KvArgs &c, int64_t n, int h, const int32_t *kept, int first, int count) {
    for (int b = first; b < count; b += kMoveThreads * kEach) {
        float x[kEach];
        float *to[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = b + e * kMoveThreads + static_cast<int>(threadIdx.x), src = i < count ? kv::load(kept + i) : -1;
            to[e] = nullptr;
            if (src >= 0 && src != i) {
                const int p = kv::page_of(c, n, src), q = kv::page_of(c, n, i);
                if (p >= 0 && q >= 0) {
                    x[e] = c.weights[kv::row_of(c, p, h, src)];
                    to[e] = c.weights + kv::row_of(c, q, h, i);
                }
            }
        }
        __syncthreads();   // every source of this block is read
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            if (to[e]) *to[e] = x[e];
    }
}

__global__ void __launch_bounds__(kMoveThreads, 6) kv_move_kernel(const KvArgs c, const EvictArgs a, int slices) {
    dependent_start();
    const int64_t n = blockIdx.x / c.H;
    const int h = static_cast<int>(blockIdx.x - n * c.H), part = blockIdx.y;
    const int len = kv::request_len(c, n);
    if (len <= a.budget) return;
    const int32_t *kept = a.kept + static_cast<int64_t>(blockIdx.x) * a.budget;
    if (part == 2 * slices) {
        move_weights(c, n, h, kept, a.sinks, a.budget);
        return;
    }
    const int row = c.e4m3 ? kD : 2 * kD, bytes = row / slices;
    move_rows(c, n, h, kept, a.sinks, a.budget, part < slices ? c.k : c.v, row, part % slices * bytes, bytes);
}

}  // namespace

cudaError_t launch_kv_evict(const KvArgs &c, int64_t budget, int64_t sinks, int64_t recent, int32_t *new_lens,
                            int32_t *kept, int sm_count, cudaStream_t st) {
    const EvictArgs a{static_cast<int>(budget), static_cast<int>(sinks), static_cast<int>(recent), new_lens, kept};
    const unsigned units = static_cast<unsigned>(c.N * c.H);
    {
        LaunchTimer timer(kKKvSelect, st);
        const cudaError_t e = launch_dependent(kv_select_kernel, dim3(units), kSelThreads, st, c, a);
        if (e != cudaSuccess) return e;
    }
    int slices = 1;   // slices of at least 32 bytes until the SMs have work
    while (slices < (c.e4m3 ? 4 : 8) && static_cast<int64_t>(units) * 2 * slices < 4 * sm_count) slices *= 2;
    LaunchTimer timer(kKKvMove, st);
    return launch_dependent(kv_move_kernel, dim3(units, 2 * slices + 1), kMoveThreads, st, c, a, slices);
}

}  // namespace sala

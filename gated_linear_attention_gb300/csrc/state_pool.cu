// The states of a pool as a serving engine manages them: copies between slots and between
// pools, forks into free slots, freeing, and compaction. A slot holds a request's states of all
// layers: pool [L, P, H, 128, 128], slot s of layer l at ((l * P) + s) * H * 128 * 128.
//
// Which slots move is decided on the device (a mask of the used slots, one int32 each), so a
// server needs no host round trip and a captured graph serves every occupancy. The decisions
// are one CTA's prefix counts over the mask; the moving is a plain stream of 16-byte accesses,
// bounded by the memory bandwidth (24 layers x 32 heads: 32 states of 25 MB moved by a compaction in
// 234 us, 6.9 TB/s; 40 forked from 5 parents in 175 us; 16 copied from fp32 to bf16 in 173 us).
#include <algorithm>
#include <type_traits>

#include "launch.h"

namespace sala {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kCopyThreads = 256;
// CTAs of a launch where pairs are many: in a compaction most of them find nothing to move, and with
// 32768 the others are too long (237 us instead of 234)
constexpr int64_t kCopyCtas = 131072;
constexpr int kUnit = kD * kD;   // elements of one head's state

// Exclusive prefix count of `flag` over the CTA (kPlanThreads threads); *total the count.
__device__ int block_rank(bool flag, int *total) {
    __shared__ int warp_count[kPlanWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned m = __ballot_sync(0xffffffffu, flag);
    if (lane == 0) warp_count[warp] = __popc(m);
    __syncthreads();
    int c = warp_count[lane], before = 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, c, off);
        if (lane >= off) c += y;
    }
    *total = __shfl_sync(0xffffffffu, c, 31);
    if (warp) before = __shfl_sync(0xffffffffu, c, warp - 1);
    __syncthreads();
    return before + __popc(m & ((1u << lane) - 1));
}

// children[i] of every request i: the lowest free slots, in order, to the requests whose parent
// is a used slot or -1 (a new state); -1 to the others and once the pool is full.
__global__ void __launch_bounds__(kPlanThreads)
pool_fork_plan_kernel(int32_t *used, int64_t P, const int32_t *parents, int32_t *children, int64_t n,
                      int *status) {
    dependent_start();
    const int tid = threadIdx.x;
    // 1. children[r] = the r-th free slot, for r < n
    int64_t found = 0;
    for (int64_t s0 = 0; s0 < P && found < n; s0 += kPlanThreads) {
        const int64_t s = s0 + tid;
        const bool is_free = s < P && used[s] == 0;
        int total;
        const int64_t r = found + block_rank(is_free, &total);
        if (is_free && r < n) children[r] = static_cast<int32_t>(s);
        found += total;
    }
    if (found > n) found = n;
    // 2. how many requests want a slot
    int64_t wanted = 0;
    auto wants = [&](int64_t i) {
        if (i >= n) return false;
        const int32_t p = parents[i];
        if (p < 0) return p == -1;
        if (p < P && used[p] != 0) return true;
        record_status(status, SALA_ERR_BAD_INDEX);   // past the pool, or of a slot that is free
        return false;
    };
    for (int64_t i0 = 0; i0 < n; i0 += kPlanThreads) {
        int total;
        block_rank(wants(i0 + tid), &total);
        wanted += total;
    }
    // 3. request i takes the slot of its rank among those: ranks do not exceed i, so from the
    // last tile down every entry is read before it is overwritten. Slots are marked at the end:
    // one of them may be the (refused) parent of a request still to be looked at.
    int64_t left = wanted;
    for (int64_t i0 = ((n - 1) / kPlanThreads) * kPlanThreads; i0 >= 0; i0 -= kPlanThreads) {
        const int64_t i = i0 + tid;
        const bool w = wants(i);
        int total;
        const int rank = block_rank(w, &total);
        left -= total;
        const int64_t r = left + rank;
        const int32_t child = w && r < found ? children[r] : -1;
        __syncthreads();
        if (i < n) children[i] = child;
        __syncthreads();
    }
    for (int64_t i = tid; i < n; i += kPlanThreads)
        if (children[i] >= 0) used[children[i]] = 1;
}

// used[s] = 0 for every named slot; a slot that is not in use (or named twice) is reported.
__global__ void pool_free_kernel(int32_t *used, int64_t P, const int32_t *slots, int64_t n, int *status) {
    dependent_start();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const int32_t s = slots[i];
    if (s < 0) return;
    if (s >= P || atomicExch(used + s, 0) == 0) record_status(status, SALA_ERR_BAD_INDEX);
}

// With m used slots: the r-th used slot at or past m moves to the r-th free slot below m.
__global__ void __launch_bounds__(kPlanThreads)
pool_compact_plan_kernel(int32_t *used, int64_t P, int32_t *mapping, int32_t *live) {
    dependent_start();
    const int tid = threadIdx.x;
    auto in_use = [&](int64_t s) { return s < P && used[s] != 0; };
    int64_t m = 0;
    for (int64_t s0 = 0; s0 < P; s0 += kPlanThreads) {
        int total;
        block_rank(in_use(s0 + tid), &total);
        m += total;
    }
    // 1. slots below m; mapping[m + r] = the r-th free one of them (there are as many as used slots
    // past m, so at most P - m)
    int64_t holes = 0;
    for (int64_t s0 = 0; s0 < m; s0 += kPlanThreads) {
        const int64_t s = s0 + tid;
        const bool hole = s < m && !in_use(s);
        int total;
        const int64_t r = holes + block_rank(hole, &total);
        if (hole) mapping[m + r] = static_cast<int32_t>(s);
        if (s < m) mapping[s] = hole ? -1 : static_cast<int32_t>(s);
        holes += total;
    }
    __syncthreads();
    // 2. slots from m: the rank r of used slot s is at most s - m, so from the last tile down every
    // entry of the list is read before it is overwritten
    int64_t left = holes;
    for (int64_t s0 = m + (P - m - 1) / kPlanThreads * kPlanThreads; P > m && s0 >= m; s0 -= kPlanThreads) {
        const int64_t s = s0 + tid;
        const bool mover = in_use(s);
        int total;
        const int rank = block_rank(mover, &total);
        left -= total;
        const int32_t to = mover ? mapping[m + left + rank] : -1;
        __syncthreads();
        if (s < P) mapping[s] = to;
        __syncthreads();
    }
    for (int64_t s = tid; s < P; s += kPlanThreads) used[s] = s < m;
    if (tid == 0) *live = static_cast<int32_t>(m);
}

// What a thread moves at a time: 16 bytes of the wider type (8 bf16 elements, else 4 of both), so
// that each warp access is contiguous on both sides.
template <typename S, typename T>
struct Mover {
    static constexpr bool kSame16 = std::is_same<S, uint16_t>::value && std::is_same<T, uint16_t>::value;
    static constexpr int kN = kSame16 ? 8 : 4;
    using Word = typename std::conditional<kSame16, uint4, float4>::type;

    // (no streaming hint: children of one parent read it from L2, and evict-first loads made a fork
    // of 40 slots from 5 parents 200 us instead of 175)
    static __device__ __forceinline__ Word load(const S *p) {
        if constexpr (std::is_same<S, uint16_t>::value && !kSame16) {
            const uint2 b = __ldg(reinterpret_cast<const uint2 *>(p));
            const float2 f0 = bf16x2_to_float2(b.x), f1 = bf16x2_to_float2(b.y);
            return make_float4(f0.x, f0.y, f1.x, f1.y);
        } else {
            return __ldg(reinterpret_cast<const Word *>(p));
        }
    }
    static __device__ __forceinline__ void store(T *p, Word x) {
        if constexpr (std::is_same<T, uint16_t>::value && !kSame16)
            __stcs(reinterpret_cast<uint2 *>(p), make_uint2(float2_to_bf16x2(x.x, x.y), float2_to_bf16x2(x.z, x.w)));
        else __stcs(reinterpret_cast<Word *>(p), x);
    }
};

struct CopyArgs {
    const void *src_pool;
    void *dst_pool;
    int64_t src_P, dst_P;
    const int32_t *src, *dst;   // src null: pair i reads slot i
    int64_t n;
    int units, H;           // L * H
    bool check;             // pairs come from the caller
    bool same;              // source and destination are one pool
    int *status;
};

// One pair per blockIdx.x, its L * H states dealt over blockIdx.y.
template <typename S, typename T>
__global__ void __launch_bounds__(kCopyThreads) pool_copy_kernel(CopyArgs a) {
    dependent_start();
    const int64_t i = blockIdx.x;
    const int32_t from = a.src ? a.src[i] : static_cast<int32_t>(i), to = a.dst[i];
    if (to < 0) return;
    if (a.check) {
        bool bad = from >= a.src_P || to >= a.dst_P;
        if (!bad)   // a destination belongs to one pair, and no pair reads what another writes
            for (int64_t j = threadIdx.x; j < a.n; j += kCopyThreads)
                bad |= (j < i && a.dst[j] == to) || (a.same && j != i && a.dst[j] >= 0 && a.src[j] == to);
        if (__syncthreads_or(bad)) {
            if (threadIdx.x == 0 && blockIdx.y == 0) record_status(a.status, SALA_ERR_BAD_INDEX);
            return;
        }
    }
    if (a.same && from == to) return;
    for (int unit = blockIdx.y; unit < a.units; unit += gridDim.y) {
        const int l = unit / a.H, h = unit - l * a.H;
        T *d = static_cast<T *>(a.dst_pool) + ((l * a.dst_P + to) * a.H + h) * kUnit;
        const S *s = from < 0 ? nullptr
                              : static_cast<const S *>(a.src_pool) + ((l * a.src_P + from) * a.H + h) * kUnit;
        using M = Mover<S, T>;
        constexpr int kAhead = 8;   // loads in flight
#pragma unroll 1
        for (int e = M::kN * threadIdx.x; e < kUnit; e += kAhead * M::kN * kCopyThreads) {
            typename M::Word x[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) x[i] = s ? M::load(s + e + i * M::kN * kCopyThreads) : typename M::Word{};
#pragma unroll
            for (int i = 0; i < kAhead; ++i) M::store(d + e + i * M::kN * kCopyThreads, x[i]);
        }
    }
}

// CTAs that share a pair: one per head's state, fewer where the pairs are many.
int64_t copy_slices(int64_t pairs, int64_t units) {
    const int64_t most = std::min<int64_t>((kCopyCtas + pairs - 1) / pairs, 65535);   // a grid's y extent
    return std::min(units, most);
}

cudaError_t copy_pairs(const CopyArgs &a, bool src_bf16, bool dst_bf16, int64_t pairs, cudaStream_t st) {
    if (pairs == 0) return cudaSuccess;
    LaunchTimer timer(kKPoolCopy, st);
    const dim3 grid(static_cast<unsigned>(pairs), static_cast<unsigned>(copy_slices(pairs, a.units)));
    void (*kern)(CopyArgs) = src_bf16 ? (dst_bf16 ? pool_copy_kernel<uint16_t, uint16_t>
                                                  : pool_copy_kernel<uint16_t, float>)
                                      : (dst_bf16 ? pool_copy_kernel<float, uint16_t>
                                                  : pool_copy_kernel<float, float>);
    return launch_dependent(kern, grid, kCopyThreads, st, a);
}

}  // namespace

cudaError_t launch_state_pool_copy(const void *src_pool, bool src_bf16, int64_t src_P, void *dst_pool,
                                   bool dst_bf16, int64_t dst_P, const int32_t *src,
                                   const int32_t *dst, int64_t n, int64_t L, int H, int *status,
                                   cudaStream_t st) {
    const CopyArgs a{src_pool, dst_pool, src_P, dst_P, src, dst, n, static_cast<int>(L * H), H,
                     true, src_pool == dst_pool, status};
    return copy_pairs(a, src_bf16, dst_bf16, n, st);
}

cudaError_t launch_state_pool_fork(void *pool, bool bf16, int64_t L, int64_t P, int H, int32_t *used,
                                   const int32_t *parents, int32_t *children, int64_t n, int *status,
                                   cudaStream_t st) {
    {
        LaunchTimer timer(kKPoolPlan, st);
        const cudaError_t e = launch_dependent(pool_fork_plan_kernel, 1, kPlanThreads, st, used, P, parents,
                                               children, n, status);
        if (e != cudaSuccess) return e;
    }
    const CopyArgs a{pool, pool, P, P, parents, children, n, static_cast<int>(L * H), H,
                     false, true, status};
    return copy_pairs(a, bf16, bf16, n, st);
}

cudaError_t launch_state_pool_free(int32_t *used, int64_t P, const int32_t *slots, int64_t n, int *status,
                                   cudaStream_t st) {
    LaunchTimer timer(kKPoolPlan, st);
    return launch_dependent(pool_free_kernel, static_cast<unsigned>((n + 255) / 256), 256, st, used, P, slots,
                            n, status);
}

cudaError_t launch_state_pool_compact(void *pool, bool bf16, int64_t L, int64_t P, int H, int32_t *used,
                                      int32_t *mapping, int32_t *live, cudaStream_t st) {
    {
        LaunchTimer timer(kKPoolPlan, st);
        const cudaError_t e = launch_dependent(pool_compact_plan_kernel, 1, kPlanThreads, st, used, P, mapping,
                                               live);
        if (e != cudaSuccess) return e;
    }
    const CopyArgs a{pool, pool, P, P, nullptr, mapping, P, static_cast<int>(L * H), H, false, true, nullptr};
    return copy_pairs(a, bf16, bf16, P, st);
}

}  // namespace sala

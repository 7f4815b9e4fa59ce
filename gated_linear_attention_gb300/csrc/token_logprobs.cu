// Log probabilities of given tokens, entropy and top alternatives of rows of logits, in one read of the row.
//
// With the row's maximum m:  l = sum exp(x - m),  w = sum exp(x - m) (x - m),  lse = m + log l,
// logp(x) = (x - m) - log l,  entropy = log l - w / l.
// Every thread keeps m, l and w of its own elements; a larger maximum m' moves them to it by
// f = exp(m - m'):  l' = f l,  w' = f (w - (m' - m) l). Pairs join the same way, in a fixed order.
//
// Top alternatives: a thread's m is also the largest of its elements, so the K-th largest of a CTA's 256 maxima
// is a border that the CTA's K largest elements do not lie below. A search by halves finds a border that K to
// 2 K + 8 threads reach; their warps go through those threads' elements again (from L2) and list what reaches the border.
// Ties can make that list long: if it does not fit, the CTA looks for its K largest one by one, each time
// through all of its elements. Places in the order (value, then the lower token) come from counting.
//
// A cluster of up to 8 CTAs shares a row and hands its sums and candidates to the first CTA through distributed
// shared memory.
#include <cfloat>
#include <cooperative_groups.h>

#include "launch.h"
#include "tc.cuh"

namespace sala {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kTop = SALA_LOGPROBS_MAX_TOP;
constexpr int kList = 512;                // candidates of a CTA
constexpr int kAhead = 4;                 // 16-byte loads of a thread in flight
constexpr float kLog2e = 1.4426950408889634f;

struct LogprobArgs {
    const void *x;
    int64_t stride;
    const int32_t *tokens;
    float *logprobs, *entropy;
    int32_t *top_tokens;
    float *top_logprobs;
    int V, M, K;
    int *status;
};

// NaN counts as -inf, +inf as the largest finite number.
__device__ __forceinline__ float clean(float x) { return x == x ? fminf(x, FLT_MAX) : -INFINITY; }

template <typename T>
struct Vec {
    static constexpr int kN = 16 / sizeof(T);
    uint4 r;
    __device__ __forceinline__ void load(const T *p) { r = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ float at(int i) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
};
template <typename T>
__device__ __forceinline__ float logit(const T *p) {
    if constexpr (sizeof(T) == 4) return clean(__ldg(p));
    else return clean(bf16_bits_to_float(__ldg(p)));
}

// Order-preserving whole numbers of floats without NaN; -0 is 0.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = x == 0.f ? 0u : __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Sums {
    float m, l, w;
    __device__ __forceinline__ void move_to(float top) {   // top >= m
        if (m == -INFINITY) {
            m = top;
            return;   // nothing summed yet
        }
        const float d = m - top, f = tc::ex2(d * kLog2e);
        w = f > 0.f ? f * (w + d * l) : 0.f;
        l *= f;
        m = top;
    }
    __device__ __forceinline__ void join(Sums o) {
        const float top = fmaxf(m, o.m);
        if (top == -INFINITY) return;
        move_to(top);
        o.move_to(top);
        l += o.l;
        w += o.w;
    }
    __device__ __forceinline__ void add(float x) {   // x <= m, or NaN
        // what lies 200 below the maximum, NaN and -inf among it, adds nothing
        const float d = fmaxf(x - m, -200.f), e = tc::ex2(d * kLog2e);
        l += e;
        w = fmaf(e, d, w);
    }
};
__device__ __forceinline__ Sums shuffled(Sums s, int o) {
    return {__shfl_xor_sync(0xffffffffu, s.m, o), __shfl_xor_sync(0xffffffffu, s.l, o), __shfl_xor_sync(0xffffffffu, s.w, o)};
}

// The elements of a row that a thread has: 16-byte vectors first, first + kThreads, .. below `end` (in vectors from the
// aligned start of the row), and at most one at the row's ends.
template <typename T>
struct Share {
    const T *row, *body;
    int begin, end;      // vectors of the CTA
    int heads, tails, V, bodies;   // elements before the first vector, behind the last; vectors
    bool ends;           // this CTA has the row's ends

    __device__ __forceinline__ Share(const T *row_, int V_, int rank, int ctas) : row(row_), V(V_) {
        constexpr int kN = Vec<T>::kN;
        heads = min(V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / static_cast<int>(sizeof(T)));
        body = row + heads;
        bodies = (V - heads) / kN;
        tails = V - heads - bodies * kN;
        begin = static_cast<int>(static_cast<int64_t>(bodies) * rank / ctas);
        end = static_cast<int>(static_cast<int64_t>(bodies) * (rank + 1) / ctas);
        ends = rank == 0;
    }
    // the element at the row's ends that thread tid has, or -1
    __device__ __forceinline__ int extra(int tid) const {
        return !ends || tid >= heads + tails ? -1 : tid < heads ? tid : V - tails + (tid - heads);
    }
};

struct Shared {
    Sums sums[kWarps];
    uint32_t keys[kList];
    int index[kList];
    int count;
    // the first CTA's, filled by its cluster
    Sums all[kMaxCluster];
    uint32_t top_keys[kMaxCluster * kTop];
    int top_index[kMaxCluster * kTop];
};

// Writes the K largest of n candidates in order, of equal keys the lower index first, then 0 and -1 (a key of 0 is
// no candidate).
__device__ __forceinline__ void ranked(const uint32_t *keys, const int *index, int n, int K, uint32_t *out_keys, int *out_index) {
    for (int i = threadIdx.x; i < K; i += kThreads) out_keys[i] = 0, out_index[i] = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint32_t k = keys[i];
        const int x = index[i];
        if (k == 0) continue;
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += keys[j] > k || (keys[j] == k && index[j] < x);
        if (rank < K) out_keys[rank] = k, out_index[rank] = x;
    }
}

// The K largest elements of the CTA's share into out (order_of, token), given each thread's maximum.
template <typename T>
__device__ __forceinline__ void cta_top(Shared &sh, const Share<T> &share, float mine, int K, uint32_t *out_keys, int *out_index) {
    constexpr int kN = Vec<T>::kN;
    constexpr uint32_t kNone = 0x007fffffu;   // order_of(-inf)
    const int tid = threadIdx.x, lane = tid & 31;
    const uint32_t key = order_of(mine);
    if (tid == 0) sh.count = 0;
    // a border that at least K threads reach (above -inf: all of them where there are fewer), by halves
    uint32_t lo = kNone + 1, hi = 0xff800000u;   // count(lo) >= K or lo is the least; count(hi) < K
    int reach = __syncthreads_count(key >= lo);
    while (reach > 2 * K + 8 && hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const int n = __syncthreads_count(key >= mid);
        if (n >= K) lo = mid, reach = n;
        else hi = mid;
    }
    // every element that reaches the border, a thread's at a time by its whole warp
    unsigned left = __ballot_sync(0xffffffffu, key >= lo);
    while (left) {
        const int who = (tid & ~31) + __ffs(left) - 1;
        left &= left - 1;
        for (int v = share.begin + who + lane * kThreads; v < share.end; v += 32 * kThreads) {
            Vec<T> x;
            x.load(share.body + static_cast<int64_t>(v) * kN);
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                const uint32_t k = order_of(clean(x.at(e)));
                if (k < lo) continue;
                const int at = atomicAdd(&sh.count, 1);
                if (at < kList) sh.keys[at] = k, sh.index[at] = share.heads + v * kN + e;
            }
        }
        const int extra = share.extra(who);
        if (lane == 0 && extra >= 0) {
            const uint32_t k = order_of(logit(share.row + extra));
            if (k >= lo) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < kList) sh.keys[at] = k, sh.index[at] = extra;
            }
        }
    }
    __syncthreads();
    const int n = sh.count;
    if (n <= kList) {
        ranked(sh.keys, sh.index, n, K, out_keys, out_index);
        return;
    }
    // too many ties: one after the other
    uint32_t last = 0xffffffffu;
    int at = -1;
    for (int r = 0; r < K; ++r) {
        uint32_t best = 0;
        int bi = INT32_MAX;
        auto see = [&](uint32_t k, int i) {
            if (k > kNone && (k < last || (k == last && i > at)) && (k > best || (k == best && i < bi))) best = k, bi = i;
        };
        for (int v = share.begin + tid; v < share.end; v += kThreads) {
            Vec<T> x;
            x.load(share.body + static_cast<int64_t>(v) * kN);
#pragma unroll
            for (int e = 0; e < kN; ++e) see(order_of(clean(x.at(e))), share.heads + v * kN + e);
        }
        const int extra = share.extra(tid);
        if (extra >= 0) see(order_of(logit(share.row + extra)), extra);
        for (int o = 16; o > 0; o /= 2) {
            const uint32_t k = __shfl_xor_sync(0xffffffffu, best, o);
            const int i = __shfl_xor_sync(0xffffffffu, bi, o);
            if (k > best || (k == best && i < bi)) best = k, bi = i;
        }
        __syncthreads();
        if (lane == 0) sh.keys[tid >> 5] = best, sh.index[tid >> 5] = bi;
        __syncthreads();
        best = 0;
        bi = INT32_MAX;
        for (int w = 0; w < kWarps; ++w)
            if (sh.keys[w] > best || (sh.keys[w] == best && sh.index[w] < bi)) best = sh.keys[w], bi = sh.index[w];
        last = best;
        at = bi;
        if (tid == 0) out_keys[r] = best, out_index[r] = best ? bi : -1;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(const LogprobArgs a) {
    constexpr int kN = Vec<T>::kN;
    __shared__ Shared sh;
    dependent_start();
    const cg::cluster_group cluster = cg::this_cluster();
    const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    if (ctas > 1) cluster.barrier_arrive();   // waited for before the first access to another CTA's memory
    const int64_t n = blockIdx.x / ctas;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const T *row = static_cast<const T *>(a.x) + n * a.stride;
    const Share<T> share(row, a.V, rank, ctas);

    Sums s{-INFINITY, 0.f, 0.f};
    for (int v = share.begin + tid; v < share.end; v += kAhead * kThreads) {
        Vec<T> x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (v + u * kThreads < share.end) x[u].load(share.body + static_cast<int64_t>(v + u * kThreads) * kN);
            else x[u].r = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);   // NaN in fp32, -inf in bf16
        }
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int e = 0; e < kN; ++e) top = fmaxf(top, x[u].at(e));   // NaN is passed over
        if (top == INFINITY) {   // counts as the largest finite number
            if (s.m < FLT_MAX) s.move_to(FLT_MAX);
            for (int u = 0; u < kAhead; ++u)
                for (int e = 0; e < kN; ++e) s.add(clean(x[u].at(e)));
            continue;
        }
        if (top > s.m) s.move_to(top);
        if (s.m == -INFINITY) continue;
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int e = 0; e < kN; ++e) s.add(x[u].at(e));
    }
    if (const int extra = share.extra(tid); extra >= 0) {
        const float x = logit(row + extra);
        if (x > s.m) s.move_to(x);
        if (s.m > -INFINITY) s.add(x);
    }
    const float mine = s.m;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) s.join(shuffled(s, o));
    if (lane == 0) sh.sums[warp] = s;

    if (ctas > 1) cluster.barrier_wait();
    Shared *first = ctas > 1 ? cluster.map_shared_rank(&sh, 0) : &sh;
    if (a.K > 0) cta_top(sh, share, mine, a.K, first->top_keys + rank * a.K, first->top_index + rank * a.K);
    __syncthreads();
    if (tid == 0) {
        s = sh.sums[0];
        for (int w = 1; w < kWarps; ++w) s.join(sh.sums[w]);
        first->all[rank] = s;
    }
    if (ctas > 1) cluster.sync();
    else __syncthreads();
    if (rank != 0) return;

    s = sh.all[0];
    for (int c = 1; c < ctas; ++c) s.join(sh.all[c]);
    const bool none = s.m == -INFINITY;
    const float logl = logf(s.l);
    if (tid == 0 && a.entropy) a.entropy[n] = none ? 0.f : fmaxf(0.f, logl - s.w / s.l);
    for (int j = tid; j < a.M; j += kThreads) {
        const int t = __ldg(a.tokens + n * a.M + j);
        if (t >= a.V) record_status(a.status, SALA_ERR_BAD_INDEX);
        a.logprobs[n * a.M + j] = t < 0 || t >= a.V ? 0.f : none ? -INFINITY : (logit(row + t) - s.m) - logl;
    }
    if (a.K == 0) return;
    uint32_t *keys = sh.top_keys;
    int *index = sh.top_index;
    if (ctas > 1) {
        ranked(sh.top_keys, sh.top_index, ctas * a.K, a.K, sh.keys, sh.index);   // the empty places come last
        __syncthreads();
        keys = sh.keys;
        index = sh.index;
    }
    for (int r = tid; r < a.K; r += kThreads) {
        const uint32_t k = keys[r];
        const float x = __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
        a.top_tokens[n * a.K + r] = k ? index[r] : -1;
        a.top_logprobs[n * a.K + r] = k ? (x - s.m) - logl : -INFINITY;
    }
}

// CTAs that share a row.
int cluster_size(int64_t N, int64_t row_bytes, int sm_count) {
    int c = kMaxCluster;
    while (c > 1 && (row_bytes < c * (8 << 10) || (N * c > 8 * sm_count && row_bytes < c * (48 << 10)))) c /= 2;
    return c;
}

}  // namespace

cudaError_t launch_token_logprobs(const void *x, int64_t stride, bool bf16, const int32_t *tokens, float *logprobs,
                                  float *entropy, int32_t *top_tokens, float *top_logprobs, int64_t N, int64_t V,
                                  int M, int K, int sm_count, int *status, cudaStream_t st) {
    LaunchTimer timer(kKTokenLogprobs, st);
    const LogprobArgs a{x, stride, tokens, logprobs, entropy, top_tokens, top_logprobs, static_cast<int>(V), M, K, status};
    const int c = cluster_size(N, V * (bf16 ? 2 : 4), sm_count);
    return launch_dependent_cluster(bf16 ? token_logprobs_kernel<uint16_t> : token_logprobs_kernel<float>,
                                    static_cast<unsigned>(N * c), c, kThreads, 0, st, a);
}

}  // namespace sala

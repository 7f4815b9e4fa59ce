// Log probabilities of given tokens, entropy and top alternatives of rows of logits, in one read of the row.
//
// With the row's maximum m:  l = sum exp(x - m),  w = sum exp(x - m) (x - m),  lse = m + log l,
// logp(x) = (x - m) - log l,  entropy = log l - w / l.
// A larger maximum m' moves sums to it by f = exp(m - m'):  l' = f l,  w' = f (w - (m' - m) l). Pairs join the same
// way, in a fixed order.
//
// Two kernels. The first streams: a row is cut into parts, a warp takes a part, and the loads of its next part are
// in flight while it ends one (a CTA for each row lost a quarter of the time in its first loads and its last sums). It
// leaves the sums of each part and the maximum of each lane. The second joins the parts of a row and finds the top
// alternatives: the K-th largest of the lanes' maxima is a border that the row's K largest elements do not lie below. A
// search by halves finds one that K to 3 K / 2 + 4 of 256 groups of lanes reach, and only the elements of lanes that
// reach it are read again (from L2). What reaches the border is listed; a place in the order (value, then the lower
// token) comes from counting. Where more elements reach it than the list holds, the K largest are looked for one by one, each
// time through the whole row: rows of equal logits, vocabularies that a finite value masks but for fewer than K tokens (256
// rows of 131072 fp32, K = 20: 1.9 ms either way), and bf16 rows of 1025 to 2048 tokens, one part each, with K > 32, as 32
// lanes give no border (256 rows of 2000, K = 64: 99 us; of 2100, which have four parts, 17 us).
//
// The read of the logits bounds the first kernel: 2048 rows of 50021 bf16 41 us with the join, 205 MB at 5 TB/s. With
// 20 alternatives 256 rows of 131072 fp32 (134 MB) take 34 us, 25 of them in the first kernel; in the second the search and the
// second look at the elements wait on each other. One row of 65536 takes 8 us, the latency of the two.
#include <algorithm>
#include <cfloat>

#include "launch.h"
#include "tc.cuh"

namespace sala {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTop = SALA_LOGPROBS_MAX_TOP;
constexpr int kMaxParts = 128;            // parts of a row
constexpr int kList = 1024;               // candidates of a row
constexpr int kAhead = 4;                 // 16-byte loads of a lane for its next step
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLow = -1.7e38f;          // what lies below adds nothing to sums whose maximum is above -1e38
constexpr uint32_t kLowBf16x2 = 0xff00ff00u;   // the same in bf16, -1.7014e38

struct LogprobArgs {
    const void *x;
    int64_t stride, N;
    const int32_t *tokens;
    float *logprobs, *entropy;
    int32_t *top_tokens;
    float *top_logprobs;
    float *sums;         // [N, parts, 4] m, l, w of the parts
    float *maxima;       // [N, parts, 32] of their lanes, null with K = 0
    int V, M, K, parts;
    int *status;
};

// NaN counts as -inf, +inf as the largest finite number.
__device__ __forceinline__ float clean(float x) { return x == x ? fminf(x, FLT_MAX) : -INFINITY; }

template <typename T>
struct Vec {
    static constexpr int kN = 16 / sizeof(T);
    uint4 r;
    __device__ __forceinline__ void load(const T *p) { r = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ float at(int i) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
};
// Larger of each of two bf16 (a NaN loses).
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <typename T>
__device__ __forceinline__ float logit(const T *p) {
    if constexpr (sizeof(T) == 4) return clean(*p);
    else return clean(bf16_bits_to_float(*p));
}

// Order-preserving whole numbers of floats without NaN; -0 is 0.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = x == 0.f ? 0u : __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

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
    // maxima that the packed sums can take: no difference to kLow or above overflows
    __device__ __forceinline__ bool ordinary() const { return fabsf(m) < 1e38f; }
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

constexpr uint32_t kNone = 0x007fffffu;   // order_of(-inf)

// A row's elements: up to a vector's worth before the first 16-byte boundary, vectors, and the rest. Part j of `parts` has the
// vectors [begin(j), begin(j + 1)), lane l of its warp those at l, l + 32, .. from the first; part 0 also has the
// elements at the row's ends, one to a lane.
template <typename T>
struct Row {
    static constexpr int kN = Vec<T>::kN;
    const T *row, *body;
    int heads, tails, V, vectors, parts;
    __device__ __forceinline__ Row(const LogprobArgs &a, int64_t n)
        : row(static_cast<const T *>(a.x) + n * a.stride), V(a.V), parts(a.parts) {
        heads = min(V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / static_cast<int>(sizeof(T)));
        body = row + heads;
        vectors = (V - heads) / kN;
        tails = V - heads - vectors * kN;
    }
    __device__ __forceinline__ int begin(int part) const { return static_cast<int>(static_cast<int64_t>(vectors) * part / parts); }
    __device__ __forceinline__ int end_element(int lane) const {   // -1: none
        return lane >= heads + tails ? -1 : lane < heads ? lane : V - tails + (lane - heads);
    }
    __device__ __forceinline__ int token(int vector, int e) const { return heads + vector * kN + e; }
};

// The sums of a lane's next vectors.
template <typename T>
__device__ __forceinline__ void add_vectors(Sums &s, const Vec<T> (&x)[kAhead]) {
    constexpr int kN = Vec<T>::kN;
    float top = -INFINITY;
    if constexpr (kN == 8) {
        uint32_t t2 = 0xff80ff80u;
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            t2 = max_bf16x2(max_bf16x2(max_bf16x2(t2, x[u].r.x), max_bf16x2(x[u].r.y, x[u].r.z)), x[u].r.w);
        top = fmaxf(__uint_as_float(t2 << 16), __uint_as_float(t2 & 0xffff0000u));
    } else {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int e = 0; e < kN; ++e) top = fmaxf(top, x[u].at(e));   // NaN is passed over
    }
    if (top > s.m) s.move_to(fminf(top, FLT_MAX));   // +inf counts as the largest finite number
    if (s.m == -INFINITY) return;
    if (!s.ordinary()) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int e = 0; e < kN; ++e) s.add(clean(x[u].at(e)));
        return;
    }
    const uint64_t minus_m = tc::pair(-s.m, -s.m), log2e = tc::pair(kLog2e, kLog2e);
    uint64_t l = tc::pair(s.l, 0.f), w = tc::pair(s.w, 0.f);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
        const uint32_t r[4] = {x[u].r.x, x[u].r.y, x[u].r.z, x[u].r.w};
#pragma unroll
        for (int e = 0; e < kN; e += 2) {
            uint64_t y;
            if constexpr (kN == 8) {
                const float2 f = bf16x2_to_float2(max_bf16x2(r[e / 2], kLowBf16x2));
                y = tc::pair(f.x, f.y);
            } else {
                y = tc::pair(fmaxf(__uint_as_float(r[e]), kLow), fmaxf(__uint_as_float(r[e + 1]), kLow));
            }
            const uint64_t d = tc::add2(y, minus_m);
            const float2 p = tc::unpair(tc::mul2(d, log2e));
            const uint64_t ex = tc::pair(tc::ex2(p.x), tc::ex2(p.y));
            l = tc::add2(l, ex);
            w = tc::fma2(ex, d, w);
        }
    }
    s.l = tc::unpair(l).x + tc::unpair(l).y;
    s.w = tc::unpair(w).x + tc::unpair(w).y;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) logprob_parts_kernel(const LogprobArgs a) {
    constexpr int kN = Vec<T>::kN;
    dependent_start();
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps, tasks = a.N * a.parts;
    int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (task >= tasks) return;
    Vec<T> x[kAhead], next[kAhead];
    const T *body = nullptr;     // of the task whose vectors are loaded next
    int at = 0, end = 0;
    float at_end = 0.f;          // the lane's element at the row's ends
    int has_end = 0;
    auto enter = [&](int64_t t) {
        const int64_t n = t / a.parts;
        const int part = static_cast<int>(t - n * a.parts);
        const Row<T> r(a, n);
        body = r.body;
        at = r.begin(part);
        end = r.begin(part + 1);
        const int e = part == 0 ? r.end_element(lane) : -1;
        has_end = e >= 0;
        if (has_end) at_end = logit(r.row + e);
    };
    auto load = [&]() {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int v = at + u * 32 + lane;
            if (v < end) next[u].load(body + static_cast<int64_t>(v) * kN);
            else next[u].r = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);   // NaN in fp32, -inf in bf16
        }
        at += kAhead * 32;
    };
    enter(task);
    load();
    Sums s{-INFINITY, 0.f, 0.f};
    while (true) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) x[u] = next[u];
        const bool last = at >= end;
        const float mine = at_end;
        const int has = has_end;
        if (last && task + warps < tasks) enter(task + warps);
        if (!last || task + warps < tasks) load();
        add_vectors(s, x);
        if (!last) continue;
        if (has) {
            if (mine > s.m) s.move_to(mine);
            if (s.m > -INFINITY) s.add(mine);
        }
        if (a.maxima) a.maxima[task * 32 + lane] = s.m;
#pragma unroll
        for (int o = 16; o > 0; o /= 2) s.join(shuffled(s, o));
        if (lane == 0) *reinterpret_cast<float4 *>(a.sums + task * 4) = make_float4(s.m, s.l, s.w, 0.f);
        task += warps;
        if (task >= tasks) return;
        s = {-INFINITY, 0.f, 0.f};
    }
}

struct Shared {
    uint32_t keys[kList];
    int index[kList];
    int count, lanes;
    uint2 ends[kWarps];
    uint16_t who[kMaxParts * 32];
    uint32_t out_keys[kTop];
    int out_index[kTop];
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

// A border that at least K of the CTA's threads reach with their keys (the least above -inf where there are fewer) and
// not many more, by halves between the least and the largest key.
__device__ __forceinline__ uint32_t border_of(Shared &sh, uint32_t key, int K) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t most = __reduce_max_sync(0xffffffffu, key), least = __reduce_min_sync(0xffffffffu, key);
    __syncthreads();
    if (lane == 0) sh.ends[warp] = make_uint2(least, most);
    __syncthreads();
    uint32_t lo = 0xffffffffu, hi = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) lo = min(lo, sh.ends[w].x), hi = max(hi, sh.ends[w].y);
    ++hi;                          // count(hi) = 0
    lo = max(lo, kNone + 1);       // count(lo) >= K, or lo is the least above -inf
    int reach = kThreads;
    while (reach > K + K / 2 + 4 && hi - lo > 1 && hi > lo) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const int n = __syncthreads_count(key >= mid);
        if (n >= K) lo = mid, reach = n;
        else hi = mid;
    }
    return lo;
}

// The K largest of the n listed candidates, in order.
__device__ __forceinline__ void listed_top(Shared &sh, int n, int K, uint32_t *out_keys, int *out_index) {
    const int tid = threadIdx.x;
    if (n > kThreads / 2) {   // fewer first: counting goes by the square
        uint32_t k[kList / kThreads];
        int x[kList / kThreads];
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < kList / kThreads; ++i) {
            const int at = tid + i * kThreads;
            k[i] = at < n ? sh.keys[at] : 0u;
            x[i] = at < n ? sh.index[at] : -1;
            best = max(best, k[i]);
        }
        const uint32_t lo = border_of(sh, best, K);   // a border of each thread's largest: K candidates reach it
        if (tid == 0) sh.count = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kList / kThreads; ++i)
            if (k[i] >= lo && k[i]) {
                const int at = atomicAdd(&sh.count, 1);
                sh.keys[at] = k[i];
                sh.index[at] = x[i];
            }
        __syncthreads();
        n = sh.count;
    }
    ranked(sh.keys, sh.index, n, K, out_keys, out_index);
}

// The sums of a row, by one warp.
__device__ __forceinline__ Sums row_sums(const LogprobArgs &a, int64_t n, int lane) {
    Sums s{-INFINITY, 0.f, 0.f};
    for (int p = lane; p < a.parts; p += 32) {
        const float4 y = *reinterpret_cast<const float4 *>(a.sums + (n * a.parts + p) * 4);
        s.join({y.x, y.y, y.z});
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) s.join(shuffled(s, o));
    return s;
}

// A thread's first given token of a row and its logit, loaded before the row's sums are there.
struct Asked {
    int token;
    float logit;
};
template <typename T>
__device__ __forceinline__ Asked ask(const LogprobArgs &a, int64_t n, int j) {
    Asked y{-1, 0.f};
    if (j < a.M) y.token = a.tokens[n * a.M + j];
    if (y.token >= 0 && y.token < a.V) y.logit = logit(static_cast<const T *>(a.x) + n * a.stride + y.token);
    return y;
}

// The entropy and the given tokens' log probabilities of a row, by `threads` threads from 0.
template <typename T>
__device__ __forceinline__ void row_results(const LogprobArgs &a, int64_t n, const Sums &s, Asked y, int id, int threads) {
    const bool none = s.m == -INFINITY;
    const float logl = logf(s.l);
    if (id == 0 && a.entropy) a.entropy[n] = none ? 0.f : fmaxf(0.f, logl - s.w / s.l);
    for (int j = id; j < a.M; j += threads) {
        if (j != id) y = ask<T>(a, n, j);
        if (y.token >= a.V) record_status(a.status, SALA_ERR_BAD_INDEX);
        a.logprobs[n * a.M + j] = y.token < 0 || y.token >= a.V ? 0.f : none ? -INFINITY : (y.logit - s.m) - logl;
    }
}

// Without alternatives: a warp a row.
template <typename T>
__global__ void __launch_bounds__(kThreads) logprob_join_kernel(const LogprobArgs a) {
    dependent_start();
    const int lane = threadIdx.x & 31;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (n >= a.N) return;
    const Asked y = ask<T>(a, n, lane);
    row_results<T>(a, n, row_sums(a, n, lane), y, lane, 32);
}

// With alternatives: a CTA a row.
template <typename T>
__global__ void __launch_bounds__(kThreads) logprob_top_kernel(const LogprobArgs a) {
    constexpr int kN = Vec<T>::kN;
    __shared__ Shared sh;
    __shared__ Sums sums;
    dependent_start();
    const int64_t n = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = a.K, lanes = a.parts * 32;
    const Row<T> row(a, n);
    const float *maxima = a.maxima + n * lanes;
    const Asked asked = ask<T>(a, n, tid);
    constexpr int kMine = kMaxParts * 32 / kThreads;   // lanes of a thread, at most
    uint32_t held[kMine], key = kNone;
#pragma unroll
    for (int i = 0; i < kMine; ++i) held[i] = tid + i * kThreads < lanes ? order_of(maxima[tid + i * kThreads]) : 0u;
#pragma unroll
    for (int i = 0; i < kMine; ++i) key = max(key, held[i]);
    if (warp == kWarps - 1) {
        const Sums s = row_sums(a, n, lane);
        if (lane == 0) sums = s;
    }
    if (tid == 0) sh.count = sh.lanes = 0;
    const uint32_t lo = border_of(sh, key, K);
    const Sums s = sums;
#pragma unroll
    for (int i = 0; i < kMine; ++i)
        if (held[i] >= lo) sh.who[atomicAdd(&sh.lanes, 1)] = static_cast<uint16_t>(tid + i * kThreads);
    __syncthreads();
    // every element that reaches the border
    auto list = [&](float y, int i) {
        const uint32_t k = order_of(y);
        if (k < lo) return;
        const int at = atomicAdd(&sh.count, 1);
        if (at < kList) sh.keys[at] = k, sh.index[at] = i;
    };
    const int per = (row.vectors / a.parts + 1 + 31) / 32, items = sh.lanes * per;
    constexpr int kAtOnce = 8;   // loads in flight
    for (int j0 = 0; j0 < items; j0 += kAtOnce * kThreads) {
        Vec<T> x[kAtOnce];
        int at[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int j = j0 + u * kThreads + tid;
            at[u] = -1;
            if (j < items) {
                const int p = j / per, who = sh.who[p], part = who >> 5, v = row.begin(part) + (who & 31) + (j - p * per) * 32;
                if (v < row.begin(part + 1)) at[u] = v;
            }
            if (at[u] >= 0) x[u].load(row.body + static_cast<int64_t>(at[u]) * kN);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            if (at[u] < 0) continue;
#pragma unroll
            for (int e = 0; e < kN; ++e) list(clean(x[u].at(e)), row.token(at[u], e));
        }
    }
    if (tid < 32 && row.end_element(tid) >= 0) list(logit(row.row + row.end_element(tid)), row.end_element(tid));
    row_results<T>(a, n, s, asked, tid, kThreads);
    __syncthreads();
    const int listed = sh.count;
    if (listed <= kList) {
        listed_top(sh, listed, K, sh.out_keys, sh.out_index);
        __syncthreads();
    } else {   // more than the list holds: one after the other
        uint32_t last = 0xffffffffu;
        int at = -1;
        for (int r = 0; r < K; ++r) {
            uint32_t best = 0;
            int bi = INT32_MAX;
            auto see = [&](float y, int i) {
                const uint32_t k = order_of(y);
                if (k > kNone && (k < last || (k == last && i > at)) && (k > best || (k == best && i < bi))) best = k, bi = i;
            };
            for (int v = tid; v < row.vectors; v += kThreads) {
                Vec<T> x;
                x.load(row.body + static_cast<int64_t>(v) * kN);
#pragma unroll
                for (int e = 0; e < kN; ++e) see(clean(x.at(e)), row.token(v, e));
            }
            if (tid < 32 && row.end_element(tid) >= 0) see(logit(row.row + row.end_element(tid)), row.end_element(tid));
            for (int o = 16; o > 0; o /= 2) {
                const uint32_t k = __shfl_xor_sync(0xffffffffu, best, o);
                const int i = __shfl_xor_sync(0xffffffffu, bi, o);
                if (k > best || (k == best && i < bi)) best = k, bi = i;
            }
            __syncthreads();
            if (lane == 0) sh.keys[warp] = best, sh.index[warp] = bi;
            __syncthreads();
            best = 0;
            bi = INT32_MAX;
            for (int w = 0; w < kWarps; ++w)
                if (sh.keys[w] > best || (sh.keys[w] == best && sh.index[w] < bi)) best = sh.keys[w], bi = sh.index[w];
            last = best;
            at = bi;
            if (tid == 0) sh.out_keys[r] = best, sh.out_index[r] = bi;
        }
        __syncthreads();
    }
    const float logl = logf(s.l);
    for (int r = tid; r < K; r += kThreads) {
        const uint32_t k = sh.out_keys[r];
        a.top_tokens[n * K + r] = k ? sh.out_index[r] : -1;
        a.top_logprobs[n * K + r] = k ? (value_of(k) - s.m) - logl : -INFINITY;
    }
}

// Parts of a row: at least 2 KB each, and as many as give every warp the same number of them (as near as it goes) or
// there are warps for. `warps` at once.
int parts_of(int64_t N, int64_t row_bytes, int K, int64_t warps) {
    const int64_t most = std::max<int64_t>(K > 0 && row_bytes > 4096 ? 4 : 1, std::min<int64_t>(kMaxParts, row_bytes / 2048));
    if (N * most <= warps) return static_cast<int>(most);   // one round: the score below grows with p
    int best = 1;
    double score = -1.0;
    for (int64_t p = K > 0 && row_bytes > 4096 ? 4 : 1; p <= most; ++p) {
        const double full = static_cast<double>(row_bytes / p) / static_cast<double>(row_bytes / p + 1024);
        if (full <= score) break;   // no later one is better, whatever its rounds
        const int64_t rounds = (N * p + warps - 1) / warps;
        // the share of the warps at work, less what starting a part costs beside its bytes
        const double busy = static_cast<double>(N * p) / static_cast<double>(rounds * warps);
        const double s = busy * full;
        if (s > score) score = s, best = static_cast<int>(p);
    }
    return best;
}

constexpr int kWarpsPerSm = 32;

}  // namespace

int token_logprobs_parts(int64_t N, int64_t V, bool bf16, int K, int sm_count) {
    return parts_of(N, V * (bf16 ? 2 : 4), K, static_cast<int64_t>(sm_count) * kWarpsPerSm);
}
size_t token_logprobs_scratch(int64_t N, int parts, int K) {
    return static_cast<size_t>(N) * parts * (16 + (K > 0 ? 128 : 0));
}

cudaError_t launch_token_logprobs(const void *x, int64_t stride, bool bf16, const int32_t *tokens, float *logprobs,
                                  float *entropy, int32_t *top_tokens, float *top_logprobs, int64_t N, int64_t V,
                                  int M, int K, void *ws, int parts, int sm_count, int *status, cudaStream_t st) {
    LaunchTimer timer(kKTokenLogprobs, st);
    const int64_t warps = static_cast<int64_t>(sm_count) * kWarpsPerSm;
    float *sums = static_cast<float *>(ws);
    const LogprobArgs a{x, stride, N, tokens, logprobs, entropy, top_tokens, top_logprobs, sums,
                        K > 0 ? sums + N * parts * 4 : nullptr, static_cast<int>(V), M, K, parts, status};
    const int64_t blocks = std::min((N * parts + kWarps - 1) / kWarps, warps / kWarps);
    cudaError_t e = launch_dependent(bf16 ? logprob_parts_kernel<uint16_t> : logprob_parts_kernel<float>,
                                     dim3(static_cast<unsigned>(blocks)), kThreads, st, a);
    if (e != cudaSuccess) return e;
    if (K > 0)
        return launch_dependent(bf16 ? logprob_top_kernel<uint16_t> : logprob_top_kernel<float>,
                                dim3(static_cast<unsigned>(N)), kThreads, st, a);
    return launch_dependent(bf16 ? logprob_join_kernel<uint16_t> : logprob_join_kernel<float>,
                            dim3(static_cast<unsigned>((N + kWarps - 1) / kWarps)), kThreads, st, a);
}

}  // namespace sala

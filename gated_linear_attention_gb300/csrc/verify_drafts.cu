// Verification of drafted tokens against the target's probabilities.
//
// Row n holds K_n <= K drafted tokens x_i drawn from the drafter's distributions q_i, the
// target's distributions p_0 .. p_{K_n} and the random numbers of the row:
//     token i is accepted  <=>  u_i q_i(x_i) < p_i(x_i);   a = the first i that is not, or K_n
//     w(x) = max(p_a(x) - q_a(x), 0)  if token a was rejected, p_a(x) if all were accepted
//     next token = min { x : sum_{y <= x} w(y) > s * sum w }
// which leaves the emitted tokens distributed as the target's own samples.
//
// The sums are taken in whole numbers of 2^-43 (a probability is first rounded to that grid,
// which is exact from 2^-19 up for fp32 and from 2^-35 up for bf16). Whole-number sums do not
// depend on their order, so the token is the same for every split of the vocabulary, and the
// rounding moves a border between two tokens by about 2^-44 times the square root of the
// vocabulary: fp32 sums would move it by up to 2^-24 of the mass before it.
//
// Only the rows p_a and q_a are read in full; the accept test gathers two values per draft.
//
// One CTA per row: warp w sums the w-th of equal parts of the vocabulary, the warp whose part
// holds the drawn number walks through it again.
#include <type_traits>

#include "launch.h"

namespace sala {

namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr float kProbScale = 8796093022208.f;   // 2^43: 2^20 tokens of probability 1 stay below 2^63

// A probability in units of 2^-43 (NaN and negative values as 0, values above 1 as 1).
__device__ __forceinline__ long long prob_units(float p) {
    return p > 0.f ? __float2ll_rn(fminf(p, 1.f) * kProbScale) : 0ll;
}

template <typename T>
__device__ __forceinline__ float prob_load(const T *p) {
    if constexpr (std::is_same<T, float>::value) return __ldg(p);
    else return bf16_bits_to_float(__ldg(p));
}

struct VerifyArgs {
    const void *p, *q;                 // target rows [N * (K + 1)], drafter rows [N * K] or null
    int64_t p_stride, q_stride;        // elements between rows
    const int32_t *x, *num_drafts;     // drafts [N, K]; drafts per row [N] or null
    const float *u, *s;                // [N, K], [N]
    int32_t *tokens, *accepted;        // [N, K + 1], [N]
    int K;
    int64_t V;
    int *status;
};

// The first drafted token of row n that is not accepted, by warp 0 (all lanes return the same).
// *rejected: it was rejected, and not past the row's last draft.
template <typename T>
__device__ int first_rejected(const VerifyArgs &a, int64_t n, bool *rejected) {
    const int lane = threadIdx.x & 31;
    int drafts = a.K;
    if (a.num_drafts) {
        drafts = __ldg(a.num_drafts + n);
        if (drafts < 0 || drafts > a.K) {
            if (lane == 0) record_status(a.status, SALA_ERR_BAD_INDEX);
            drafts = drafts < 0 ? 0 : a.K;
        }
    }
    *rejected = false;
    for (int base = 0; base < drafts; base += 32) {
        const int i = base + lane;
        bool stop = i >= drafts, no = false;
        if (!stop) {
            const int32_t x = __ldg(a.x + n * a.K + i);
            if (x < 0 || x >= a.V) {   // the row's drafts end here
                if (x >= 0) record_status(a.status, SALA_ERR_BAD_INDEX);
                stop = true;
            } else {
                const T *p = static_cast<const T *>(a.p) + (n * (a.K + 1) + i) * a.p_stride;
                const T *q = static_cast<const T *>(a.q) + (n * a.K + i) * a.q_stride;
                // two 24-bit factors: the product is exact in 64 bits
                const double qx = a.q ? static_cast<double>(prob_load(q + x)) : 1.0;
                no = !(static_cast<double>(__ldg(a.u + n * a.K + i)) * qx <
                       static_cast<double>(prob_load(p + x)));
                stop = no;
            }
        }
        const unsigned stops = __ballot_sync(0xffffffffu, stop);
        if (stops) {
            const int first = __ffs(stops) - 1;
            *rejected = __shfl_sync(0xffffffffu, no, first);
            return base + first;
        }
    }
    return drafts;
}

// The weight of token x in the draw, in units of 2^-43.
template <typename T>
__device__ __forceinline__ long long weight(const T *p, const T *q, int64_t one_at, int64_t x) {
    long long w = prob_units(prob_load(p + x));
    if (q) w -= prob_units(prob_load(q + x));
    else if (x == one_at) w -= static_cast<long long>(kProbScale);   // a drafter without probabilities
    return w > 0 ? w : 0;
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) verify_drafts_kernel(VerifyArgs a) {
    dependent_start();
    const int64_t n = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ int first_s;
    __shared__ bool rejected_s;
    __shared__ long long sums[kVerifyWarps];

    if (warp == 0) {
        bool rejected;
        const int first = first_rejected<T>(a, n, &rejected);
        if (lane == 0) {
            first_s = first;
            rejected_s = rejected;
        }
    }
    __syncthreads();
    const int first = first_s;
    const T *p = static_cast<const T *>(a.p) + (n * (a.K + 1) + first) * a.p_stride;
    const T *q = nullptr;
    int64_t one_at = -1;
    if (rejected_s) {
        if (a.q) q = static_cast<const T *>(a.q) + (n * a.K + first) * a.q_stride;
        else one_at = __ldg(a.x + n * a.K + first);
    }
    const int64_t part = (a.V + kVerifyWarps - 1) / kVerifyWarps;
    const int64_t lo = min(a.V, part * warp), hi = min(a.V, lo + part);

    long long total = 0, before = 0;
    for (int pass = 0; pass < 2; ++pass) {
        long long sum = 0;
        for (int64_t x = lo + lane; x < hi; x += 32) sum += weight(p, q, one_at, x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) sums[warp] = sum;
        __syncthreads();
        total = before = 0;
        for (int w = 0; w < kVerifyWarps; ++w) {
            if (w == warp) before = total;
            total += sums[w];
        }
        __syncthreads();
        if (total > 0 || (!q && one_at < 0)) break;
        q = nullptr;   // nothing is left of the target after the drafter's part: draw from the target
        one_at = -1;
    }

    int32_t *out = a.tokens + n * (a.K + 1);
    for (int i = threadIdx.x; i <= a.K; i += kVerifyThreads)
        if (i != first || total == 0) out[i] = i < first ? __ldg(a.x + n * a.K + i) : -1;
    if (threadIdx.x == 0) a.accepted[n] = first;
    if (total == 0) return;

    // the number drawn, in the same units, at most total - 1
    float s = __ldg(a.s + n);
    s = s >= 0.f ? fminf(s, 0.99999994f) : 0.f;
    const long long at = static_cast<long long>(static_cast<double>(s) * static_cast<double>(total));
    if (at < before || at >= before + sums[warp]) return;
    long long run = before;
    for (int64_t x0 = lo; x0 < hi; x0 += 32) {
        const int64_t x = x0 + lane;
        long long c = x < hi ? weight(p, q, one_at, x) : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, c, off);
            if (lane >= off) c += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, run + c > at);
        if (past) {
            if (lane == 0) out[first] = static_cast<int32_t>(x0 + __ffs(past) - 1);
            return;
        }
        run += __shfl_sync(0xffffffffu, c, 31);
    }
}

}  // namespace

cudaError_t launch_verify_drafts(const void *p, int64_t p_stride, const void *q, int64_t q_stride,
                                 bool bf16, const int32_t *x, const int32_t *num_drafts,
                                 const float *u, const float *s, int32_t *tokens,
                                 int32_t *accepted, int64_t N, int K, int64_t V, int *status,
                                 cudaStream_t stream) {
    LaunchTimer timer(kKVerifyDrafts, stream);
    const VerifyArgs a{p, q, p_stride, q_stride, x, num_drafts, u, s, tokens, accepted, K, V, status};
    return bf16 ? launch_dependent(verify_drafts_kernel<uint16_t>, static_cast<unsigned>(N),
                                   kVerifyThreads, stream, a)
                : launch_dependent(verify_drafts_kernel<float>, static_cast<unsigned>(N),
                                   kVerifyThreads, stream, a);
}

}  // namespace sala

// Log probabilities of given tokens, entropy and top alternatives of rows of logits.
//
// With the row's maximum m:  l = sum exp(x - m),  lse = m + log l,  logp(x) = x - lse,
// entropy = log l - (1 / l) sum exp(x - m) (x - m).
#include <cfloat>

#include "launch.h"

namespace sala {
namespace {

constexpr int kThreads = 512;

// NaN counts as -inf, +inf as the largest finite number.
__device__ __forceinline__ float clean(float x) { return x == x ? fminf(x, FLT_MAX) : -INFINITY; }

template <typename T>
__device__ __forceinline__ float logit(const T *p) {
    if constexpr (sizeof(T) == 4) return clean(__ldg(p));
    else return clean(bf16_bits_to_float(__ldg(p)));
}

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

template <typename T>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(const LogprobArgs a) {
    __shared__ float sa[kThreads], sb[kThreads];
    __shared__ int si[kThreads];
    dependent_start();
    const int64_t n = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + n * a.stride;
    const int tid = threadIdx.x;
    float m = -INFINITY;
    for (int i = tid; i < a.V; i += kThreads) m = fmaxf(m, logit(x + i));
    sa[tid] = m;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o /= 2) {
        if (tid < o) sa[tid] = fmaxf(sa[tid], sa[tid + o]);
        __syncthreads();
    }
    m = sa[0];
    __syncthreads();
    const bool none = m == -INFINITY;
    float l = 0.f, w = 0.f;
    for (int i = tid; i < a.V && !none; i += kThreads) {
        const float d = logit(x + i) - m;
        const float e = expf(d);
        l += e;
        w += e > 0.f ? e * d : 0.f;
    }
    sa[tid] = l;
    sb[tid] = w;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o /= 2) {
        if (tid < o) sa[tid] += sa[tid + o], sb[tid] += sb[tid + o];
        __syncthreads();
    }
    l = sa[0];
    w = sb[0];
    __syncthreads();
    const float logl = logf(l);
    if (tid == 0 && a.entropy) a.entropy[n] = none ? 0.f : fmaxf(0.f, logl - w / l);
    for (int j = tid; j < a.M; j += kThreads) {
        const int t = __ldg(a.tokens + n * a.M + j);
        if (t >= a.V) record_status(a.status, SALA_ERR_BAD_INDEX);
        float out = 0.f;
        if (t >= 0 && t < a.V) out = none ? -INFINITY : (logit(x + t) - m) - logl;
        a.logprobs[n * a.M + j] = out;
    }
    float last = INFINITY;
    int at = -1;
    for (int r = 0; r < a.K; ++r) {   // the largest below the one before, lower tokens first
        float best = -INFINITY;
        int bi = INT32_MAX;
        for (int i = tid; i < a.V; i += kThreads) {
            const float y = logit(x + i);
            if ((y < last || (y == last && i > at)) && y > best) best = y, bi = i;
        }
        sa[tid] = best;
        si[tid] = bi;
        __syncthreads();
        for (int o = kThreads / 2; o > 0; o /= 2) {
            if (tid < o && (sa[tid + o] > sa[tid] || (sa[tid + o] == sa[tid] && si[tid + o] < si[tid])))
                sa[tid] = sa[tid + o], si[tid] = si[tid + o];
            __syncthreads();
        }
        last = sa[0];
        at = si[0];
        __syncthreads();
        if (tid == 0) {
            a.top_tokens[n * a.K + r] = last == -INFINITY ? -1 : at;
            a.top_logprobs[n * a.K + r] = last == -INFINITY ? -INFINITY : (last - m) - logl;
        }
    }
}

}  // namespace

cudaError_t launch_token_logprobs(const void *x, int64_t stride, bool bf16, const int32_t *tokens, float *logprobs,
                                  float *entropy, int32_t *top_tokens, float *top_logprobs, int64_t N, int64_t V,
                                  int M, int K, int sm_count, int *status, cudaStream_t st) {
    LaunchTimer timer(kKTokenLogprobs, st);
    const LogprobArgs a{x, stride, tokens, logprobs, entropy, top_tokens, top_logprobs, static_cast<int>(V), M, K, status};
    return launch_dependent(bf16 ? token_logprobs_kernel<uint16_t> : token_logprobs_kernel<float>,
                            dim3(static_cast<unsigned>(N)), kThreads, st, a);
}

}  // namespace sala

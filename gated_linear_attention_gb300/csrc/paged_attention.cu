// Attention of new tokens over a paged cache: a warp for each (token, query head).
#include "kv_cache.cuh"

namespace sala {
namespace {

constexpr int kThreads = 128;

// 4 values of row `row` from dimension d.
__device__ __forceinline__ float4 load4(const uint8_t *pages, bool e4m3, int64_t row, int d) {
    if (e4m3) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(pages + row * kD + d);
        const float2 a = kv::e4m3x2_to_float2(w & 0xffffu), b = kv::e4m3x2_to_float2(w >> 16);
        return make_float4(a.x, a.y, b.x, b.y);
    }
    const uint2 w = *reinterpret_cast<const uint2 *>(pages + (row * kD + d) * 2);
    const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
    return make_float4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ float warp_sum(float x) {
    for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__global__ void __launch_bounds__(kThreads) attend_kernel(const KvArgs c, const uint16_t *__restrict__ q, int64_t q_stride,
                                                          float scale, uint16_t *__restrict__ o, float *__restrict__ lse,
                                                          int G) {
    dependent_start();
    const int64_t item = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31, Hq = G * c.H;
    const int64_t t = item / Hq;
    const int hq = static_cast<int>(item - t * Hq), h = hq / G;
    if (t >= c.T) return;
    const int64_t n = kv::request_of(c, t);
    const kv::Request r = kv::request(c, n);
    const int64_t at = t - r.first;
    if (at < 0 || at >= r.count) return;
    const int64_t place = r.len - r.count + at;
    const uint2 qw = *reinterpret_cast<const uint2 *>(q + t * q_stride + hq * kD + lane * 4);
    const float2 q0 = bf16x2_to_float2(qw.x), q1 = bf16x2_to_float2(qw.y);
    const float ks = c.k_scale ? c.k_scale[h] : 1.f, vs = c.v_scale ? c.v_scale[h] : 1.f;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t j = 0; j <= place; ++j) {
        const int page = kv::page_of(c, n, static_cast<int>(j));
        const int64_t row = kv::row_of(c, page < 0 ? 0 : page, h, static_cast<int>(j));
        const float4 k = load4(c.k, c.e4m3, row, lane * 4), v = load4(c.v, c.e4m3, row, lane * 4);
        const float s = warp_sum(q0.x * k.x + q0.y * k.y + q1.x * k.z + q1.y * k.w) * (scale * ks);
        const float top = fmaxf(m, s), base = top == -INFINITY ? 0.f : top;
        const float f = expf(m - base), p = expf(s - base);
        l = l * f + p;
        acc.x = acc.x * f + p * v.x;
        acc.y = acc.y * f + p * v.y;
        acc.z = acc.z * f + p * v.z;
        acc.w = acc.w * f + p * v.w;
        m = top;
    }
    const float inv = l > 0.f || l != l ? vs / l : 0.f;
    *reinterpret_cast<uint2 *>(o + (t * Hq + hq) * kD + lane * 4) =
        make_uint2(float2_to_bf16x2(acc.x * inv, acc.y * inv), float2_to_bf16x2(acc.z * inv, acc.w * inv));
    if (lse && lane == 0) lse[t * Hq + hq] = m + logf(l);
}

// A warp for each (request, head, place): the weights of its rows, in order.
__global__ void __launch_bounds__(kThreads) weights_kernel(const KvArgs c, const uint16_t *__restrict__ q, int64_t q_stride,
                                                           float scale, const float *__restrict__ lse, int G) {
    dependent_start();
    const int lane = threadIdx.x & 31, h = blockIdx.y, Hq = G * c.H;
    const float ks = c.k_scale ? c.k_scale[h] : 1.f;
    for (int64_t n = blockIdx.z; n < c.N; n += gridDim.z) {
        const kv::Request r = kv::request(c, n);
        for (int64_t j = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); j < r.len; j += gridDim.x * (kThreads / 32)) {
            const int page = kv::page_of(c, n, static_cast<int>(j));
            if (page < 0) continue;
            const int64_t row = kv::row_of(c, page, h, static_cast<int>(j));
            const float4 k = load4(c.k, c.e4m3, row, lane * 4);
            float sum = 0.f;
            const int64_t first = max(int64_t(0), j - (r.len - r.count));
            for (int64_t t = r.first + first; t < r.first + r.count; ++t)
                for (int g = 0; g < G; ++g) {
                    const uint2 qw = *reinterpret_cast<const uint2 *>(q + t * q_stride + (h * G + g) * kD + lane * 4);
                    const float2 q0 = bf16x2_to_float2(qw.x), q1 = bf16x2_to_float2(qw.y);
                    const float s = warp_sum(q0.x * k.x + q0.y * k.y + q1.x * k.z + q1.y * k.w) * (scale * ks);
                    sum += expf(s - lse[t * Hq + h * G + g]);
                }
            if (lane == 0) c.weights[row] += sum;
        }
    }
}

}  // namespace

size_t paged_attention_scratch(const KvArgs &c, int G, bool, bool own_lse, int) {
    return own_lse ? static_cast<size_t>(c.T) * G * c.H * 4 : 0;
}
cudaError_t setup_paged_attention_kernel() { return cudaSuccess; }

cudaError_t launch_paged_attention(const KvArgs &c, const void *q, int64_t q_stride, float scale, void *o, float *lse,
                                   bool accumulate, int G, void *ws, int, cudaStream_t st) {
    if (accumulate && !lse) lse = static_cast<float *>(ws);
    const uint16_t *qp = static_cast<const uint16_t *>(q);
    {
        LaunchTimer timer(kKPagedAttention, st);
        const int64_t blocks = (c.T * G * c.H + kThreads / 32 - 1) / (kThreads / 32);
        if (blocks >= int64_t(1) << 31) return cudaErrorInvalidValue;
        const cudaError_t e = launch_dependent(attend_kernel, dim3(static_cast<unsigned>(blocks)), kThreads, st, c, qp,
                                               q_stride, scale, static_cast<uint16_t *>(o), lse, G);
        if (e != cudaSuccess || !accumulate) return e;
    }
    LaunchTimer timer(kKPagedWeights, st);
    return launch_dependent(weights_kernel, dim3(64, c.H, static_cast<unsigned>(c.N < 65535 ? c.N : 65535)), kThreads, st, c,
                            qp, q_stride, scale, lse, G);
}

}  // namespace sala

// Keys and values of new tokens into the pages of a cache.
//
// A warp takes eight tokens of one head: lanes 0-15 their keys, 16-31 their values, 16 bytes each. The loads of k and v
// need only the tokens' numbers and are issued first; meanwhile eight lanes find a token's request (a binary search
// of the offsets) and page each. (One token a warp, the chain of lookups bounded the kernel: 40 k tokens into e4m3 pages
// took 28 us. Now 10.1 us where the 62 MB stay in L2, and 14.9 us a call on tokens that come from memory, 4.2 TB/s, with
// half of the issue slots and a third of the memory's rate in use: each warp's chain of lookups comes before its stores. One
// token takes 2.1 us, a launch.)
#include "kv_cache.cuh"

namespace sala {
namespace {

constexpr int kThreads = 256, kTokens = 8;

// x / s, correctly rounded where an e4m3 value comes of it (Markstein: with r the correctly rounded 1 / s, one correction
// q - (q s - x) r of q = x r rounds correctly). What lies past 2^10 is clamped anyway; infinities and NaN stay, and so does a zero's
// sign (with x - q s it would not: sums of zeros of both signs are +0).
__device__ __forceinline__ float divided(float x, float s, float r) {
    const float q = x * r;
    return fabsf(q) <= 1024.f ? fmaf(-fmaf(q, s, -x), r, q) : q;
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvArgs c, const uint16_t *k,
                                                             int64_t k_stride, const uint16_t *v,
                                                             int64_t v_stride) {
    dependent_start();
    if (blockIdx.x == 0 && c.cu)   // every pair of offsets is looked at, those without tokens too
        for (int64_t n = threadIdx.x; n < c.N; n += kThreads) kv::request(c, n);
    const int64_t item = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31, part = lane & 15;
    const int64_t t0 = item / c.H * kTokens;
    const int h = static_cast<int>(item % c.H);
    if (t0 >= c.T) return;
    const bool value = lane >= 16;
    const uint16_t *src = (value ? v + t0 * v_stride : k + t0 * k_stride) + h * kD + part * 8;
    const int64_t stride = value ? v_stride : k_stride;
    uint4 x[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i)
        x[i] = t0 + i < c.T ? *reinterpret_cast<const uint4 *>(src + i * stride) : make_uint4(0, 0, 0, 0);
    int64_t row = -1;   // of the token t0 + lane; -1: it has none
    if (lane < kTokens && t0 + lane < c.T) {
        const int64_t n = kv::request_of(c, t0 + lane);
        const kv::Request r = kv::request(c, n);
        const int64_t at = t0 + lane - r.first, place = r.len - r.count + at;
        if (at >= 0 && at < r.count && place >= 0) {   // not behind the last request
            const int page = kv::page_of(c, n, static_cast<int>(place));
            if (page >= 0) row = kv::row_of(c, page, h, static_cast<int>(place));
        }
        if (c.weights && row >= 0) c.weights[row] = 0.f;
    }
    const float *scales = value ? c.v_scale : c.k_scale;
    const float s = E4M3 && scales ? kv::load(scales + h) : 1.f;
    const float inverse = __frcp_rn(s);
    uint8_t *dst = value ? c.v : c.k;
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const int64_t to = __shfl_sync(0xffffffffu, row, i);
        if (to < 0) continue;
        if constexpr (E4M3) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = bf16x2_to_float2(w[j]);
                b[j] = __nv_cvt_float2_to_fp8x2(make_float2(divided(f.x, s, inverse), divided(f.y, s, inverse)), __NV_SATFINITE, __NV_E4M3);
            }
            *reinterpret_cast<uint2 *>(dst + to * kD + part * 8) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
        } else {
            *reinterpret_cast<uint4 *>(dst + (to * kD + part * 8) * 2) = x[i];
        }
    }
}

}  // namespace

cudaError_t launch_kv_append(const KvArgs &c, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                             cudaStream_t st) {
    LaunchTimer timer(kKKvAppend, st);
    const int64_t warps = (c.T + kTokens - 1) / kTokens * c.H, blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks >= int64_t(1) << 31) return cudaErrorInvalidValue;
    return launch_dependent(c.e4m3 ? kv_append_kernel<true> : kv_append_kernel<false>,
                            dim3(static_cast<unsigned>(blocks)), kThreads, st, c, static_cast<const uint16_t *>(k),
                            k_stride, static_cast<const uint16_t *>(v), v_stride);
}

}  // namespace sala

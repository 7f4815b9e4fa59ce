// Keys and values of new tokens into the pages of a cache.
//
// A warp takes one (token, head): lanes 0-15 its key, 16-31 its value, 16 bytes each. The loads of k and v
// need only the token's number and are issued before the token's request (a binary search of the
// offsets) and page are known, so that both chains overlap.
#include "kv_cache.cuh"

namespace sala {
namespace {

constexpr int kThreads = 256;

template <bool E4M3>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvArgs c, const uint16_t *__restrict__ k,
                                                             int64_t k_stride, const uint16_t *__restrict__ v,
                                                             int64_t v_stride) {
    dependent_start();
    if (blockIdx.x == 0 && c.cu)   // every pair of offsets is looked at, those without tokens too
        for (int64_t n = threadIdx.x; n < c.N; n += kThreads) kv::request(c, n);
    const int64_t item = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31, part = lane & 15;
    const int64_t t = item / c.H;
    const int h = static_cast<int>(item - t * c.H);
    if (t >= c.T) return;
    const bool value = lane >= 16;
    const uint16_t *src = (value ? v + t * v_stride : k + t * k_stride) + h * kD + part * 8;
    const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src));
    const int64_t n = kv::request_of(c, t);
    const kv::Request r = kv::request(c, n);
    const int64_t at = t - r.first;
    if (at < 0 || at >= r.count) return;   // behind the last request
    const int64_t place = r.len - r.count + at;
    if (place < 0) return;
    const int page = kv::page_of(c, n, static_cast<int>(place));
    if (page < 0) return;
    const int64_t row = kv::row_of(c, page, h, static_cast<int>(place));
    uint8_t *dst = value ? c.v : c.k;
    if constexpr (E4M3) {
        const float *scales = value ? c.v_scale : c.k_scale;
        const float s = scales ? __ldg(scales + h) : 1.f;
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_to_float2(w[i]);
            b[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f.x, s), __fdiv_rn(f.y, s)), __NV_SATFINITE, __NV_E4M3);
        }
        *reinterpret_cast<uint2 *>(dst + row * kD + part * 8) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
    } else {
        *reinterpret_cast<uint4 *>(dst + (row * kD + part * 8) * 2) = x;
    }
    if (c.weights && lane == 0) c.weights[row] = 0.f;
}

}  // namespace

cudaError_t launch_kv_append(const KvArgs &c, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                             cudaStream_t st) {
    LaunchTimer timer(kKKvAppend, st);
    const int64_t warps = c.T * c.H, blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks >= int64_t(1) << 31) return cudaErrorInvalidValue;
    return launch_dependent(c.e4m3 ? kv_append_kernel<true> : kv_append_kernel<false>,
                            dim3(static_cast<unsigned>(blocks)), kThreads, st, c, static_cast<const uint16_t *>(k),
                            k_stride, static_cast<const uint16_t *>(v), v_stride);
}

}  // namespace sala

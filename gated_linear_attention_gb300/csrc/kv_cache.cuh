// Device helpers over a paged cache (internal): the new tokens and the length of a request, the
// page of a place, and 8-bit floats.
#pragma once

#include <cuda_fp8.h>

#include "launch.h"

namespace sala {
namespace kv {

// A word of an input. A kernel that starts as a programmatic dependent is resident while the work before it may still write
// its inputs, so they are read by plain loads (the read-only path asks for data that stays as it is for the kernel's
// life), which keep their order to the kernel-wide wait and may pass the stores and records of the kernel itself.
__device__ __forceinline__ int32_t load(const int32_t *p) {
    int32_t r;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(r) : "l"(p));
    return r;
}
__device__ __forceinline__ int64_t load(const int64_t *p) {
    int64_t r;
    asm volatile("ld.global.s64 %0, [%1];" : "=l"(r) : "l"(p));
    return r;
}
__device__ __forceinline__ float load(const float *p) {
    float r;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(r) : "l"(p));
    return r;
}

// One request of a call: its new tokens [first, first + count) and its places [0, len). A malformed
// pair of offsets or length is recorded, and the request then has no tokens or no places.
struct Request {
    int64_t first;
    int count, len;
};

__device__ __forceinline__ int request_len(const KvArgs &c, int64_t n) {
    const int len = load(c.lens + n);
    if (len >= 0 && len <= c.W * c.S) return len;
    record_status(c.status, SALA_ERR_BAD_INDEX);
    return 0;
}

__device__ __forceinline__ Request request(const KvArgs &c, int64_t n) {
    Request r;
    r.first = n * c.T_row;
    r.count = static_cast<int>(c.T_row);
    if (c.cu) {
        const int64_t a = load(c.cu + n), b = load(c.cu + n + 1);
        const bool ok = a >= 0 && b >= a && b <= c.T;
        if (!ok) record_status(c.status, SALA_ERR_BAD_SEQLENS);
        r.first = ok ? a : 0;
        r.count = ok ? static_cast<int>(b - a) : 0;
    }
    r.len = request_len(c, n);
    return r;
}

// The request that holds token t of the packed ones: the last whose offset is at most t.
__device__ __forceinline__ int64_t request_of(const KvArgs &c, int64_t t) {
    if (!c.cu) return t / c.T_row;
    int64_t lo = 0, hi = c.N;   // cu[lo] <= t < cu[hi] where the offsets are well formed
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (load(c.cu + mid) <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The page of place i of request n (its length covers i), or -1 where the table holds none.
__device__ __forceinline__ int page_of(const KvArgs &c, int64_t n, int i) {
    const int p = load(c.table + n * c.W + (i >> c.log_S));
    if (p >= 0 && p < c.P) return p;
    record_status(c.status, SALA_ERR_BAD_INDEX);
    return -1;
}

// Row (of 128 values) of a slot in the pages [P, H, S, 128].
__device__ __forceinline__ int64_t row_of(const KvArgs &c, int page, int h, int i) {
    return (static_cast<int64_t>(page) * c.H + h) * c.S + (i & (c.S - 1));
}

// Two e4m3 values in 16 bits -> two floats (exact).
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
    return __half22float2(__half2(h));
}

}  // namespace kv
}  // namespace sala

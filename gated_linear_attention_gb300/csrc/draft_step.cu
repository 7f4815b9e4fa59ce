// Decode step over several drafted tokens on pooled states, with the commit of the step before.
//
// A recurrent state has no history to fall back on: once drafted tokens are in it, the rejected
// ones cannot be taken out. So the states of drafted tokens are never stored. The step that runs
// drafted tokens reads the pool's state and keeps what follows on chip; the step after it, which
// knows how many of them were accepted, adds exactly those to the pool's state and goes on from
// there. Per (sequence, head), with c pending tokens accepted and T new ones:
//     S = exp(pg_1 + .. + pg_c) S + sum_j exp(pg_{j+1} + .. + pg_c) pk_j^T pv_j;  pool = S
//     o_t = scale ( exp(g_1 + .. + g_t) q_t S + sum_{j <= t} exp(g_{j+1} + .. + g_t) (q_t . k_j) v_j )
// One read and one write of the state serve a whole step, whatever its number of tokens: the
// bytes of a one-token decode step. Exponents are sums of gates and never differences, so a gate
// of minus infinity (forget everything) gives exact zeros.
//
// One CTA of 256 threads per (sequence, head); thread (w, l) holds rows [16 w, 16 w + 16) and
// columns [4 l, 4 l + 4) of the state in fp32. Tokens are taken in blocks of 8.
#include <type_traits>

#include "launch.h"

namespace sala {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = kD / kWarps;   // state rows of a warp
constexpr int kBlock = 8;            // tokens in flight

struct DraftArgs {
    const uint16_t *q, *k, *v;
    const float *g;
    const int32_t *num_tokens;   // [N] or null: T each
    const uint16_t *pk, *pv;
    const float *pg;
    const int32_t *accepted;     // [N]: accepted + 1 pending tokens are committed
    float scale;
    void *pool;
    const int32_t *slots;
    int64_t P;
    uint16_t *o;
    int64_t T, T_pend;
    int H;
    int *status;
};

struct Tile {
    float q[kBlock][kD], k[kBlock][kD], v[kBlock][kD];
    float part[kWarps][kBlock][kD];
    float score[kBlock][kBlock];   // exp(g_{j+1} + .. + g_t) (q_t . k_j)
    float gate[kBlock];
    float tail[kBlock];            // exp(g_{j+1} + .. + g_last)
    float head[kBlock];            // exp(g_1 + .. + g_t)
};

// `m` rows of [tokens, H, 128] bf16 into a tile, from token t0 of row n.
__device__ __forceinline__ void load_rows(float (*dst)[kD], const uint16_t *src, int64_t row0, int H, int m) {
    for (int e = threadIdx.x; e < m * (kD / 2); e += kThreads) {
        const int t = e / (kD / 2), c = e % (kD / 2);
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(src + (row0 + static_cast<int64_t>(t) * H) * kD) + c);
        const float2 f = bf16x2_to_float2(w);
        dst[t][2 * c] = f.x;
        dst[t][2 * c + 1] = f.y;
    }
}

// head and tail of the m gates in the tile (thread 0; at most kBlock of them).
__device__ __forceinline__ void gate_sums(Tile &s, int m) {
    if (threadIdx.x == 0) {
        float sum = 0.f;
        for (int t = 0; t < m; ++t) {
            sum += s.gate[t];
            s.head[t] = expf(sum);
        }
        sum = 0.f;
        for (int t = m - 1; t >= 0; --t) {
            s.tail[t] = expf(sum);
            sum += s.gate[t];
        }
    }
}

// S = exp(all gates) S + sum_j tail_j k_j^T v_j over the m tokens of the tile.
__device__ __forceinline__ void advance(float4 *x, const Tile &s, int m, int row0, int lane) {
    const float a = s.head[m - 1];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        x[r].x *= a;
        x[r].y *= a;
        x[r].z *= a;
        x[r].w *= a;
    }
    for (int j = 0; j < m; ++j) {
        float4 v = *reinterpret_cast<const float4 *>(&s.v[j][4 * lane]);
        const float w = s.tail[j];
        v.x *= w;
        v.y *= w;
        v.z *= w;
        v.w *= w;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float k = s.k[j][row0 + r];
            x[r].x = fmaf(k, v.x, x[r].x);
            x[r].y = fmaf(k, v.y, x[r].y);
            x[r].z = fmaf(k, v.z, x[r].z);
            x[r].w = fmaf(k, v.w, x[r].w);
        }
    }
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) draft_step_kernel(DraftArgs a) {
    dependent_start();
    __shared__ Tile s;
    const int unit = blockIdx.x, n = unit / a.H, h = unit - n * a.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = warp * kRows;
    const int32_t slot = __ldg(a.slots + n);
    int64_t commits = a.T_pend ? static_cast<int64_t>(__ldg(a.accepted + n)) + 1 : 0;
    if (commits < 0) commits = 0;
    int64_t tokens = a.num_tokens ? __ldg(a.num_tokens + n) : a.T;
    const bool bad = slot >= a.P || commits > a.T_pend || tokens < 0 || tokens > a.T;
    if (bad && threadIdx.x == 0) record_status(a.status, SALA_ERR_BAD_INDEX);
    const bool skip = bad || slot < 0;
    if (skip) tokens = 0;
    for (int64_t e = tokens * (kD / 8) + threadIdx.x; e < a.T * (kD / 8); e += kThreads) {
        const int64_t t = e / (kD / 8);
        uint16_t *row = a.o + ((n * a.T + t) * a.H + h) * kD;
        reinterpret_cast<uint4 *>(row)[e % (kD / 8)] = make_uint4(0, 0, 0, 0);
    }
    if (skip || (commits == 0 && tokens == 0)) return;

    const int64_t at = (static_cast<int64_t>(slot) * a.H + h) * kD * kD;
    float4 x[kRows];
    if constexpr (kBf16) {
        const uint16_t *S = static_cast<const uint16_t *>(a.pool) + at;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const uint2 w = __ldcs(reinterpret_cast<const uint2 *>(S + (row0 + r) * kD) + lane);
            const float2 f0 = bf16x2_to_float2(w.x), f1 = bf16x2_to_float2(w.y);
            x[r] = make_float4(f0.x, f0.y, f1.x, f1.y);
        }
    } else {
        const float *S = static_cast<const float *>(a.pool) + at;
#pragma unroll
        for (int r = 0; r < kRows; ++r) x[r] = __ldcs(reinterpret_cast<const float4 *>(S + (row0 + r) * kD) + lane);
    }

    // 1. commit the accepted tokens of the step before
    for (int64_t j0 = 0; j0 < commits; j0 += kBlock) {
        const int m = static_cast<int>(min(static_cast<int64_t>(kBlock), commits - j0));
        const int64_t first = (n * a.T_pend + j0) * a.H + h;
        __syncthreads();
        load_rows(s.k, a.pk, first, a.H, m);
        load_rows(s.v, a.pv, first, a.H, m);
        if (threadIdx.x < m) s.gate[threadIdx.x] = __ldg(a.pg + first + static_cast<int64_t>(threadIdx.x) * a.H);
        __syncthreads();
        gate_sums(s, m);
        __syncthreads();
        advance(x, s, m, row0, lane);
    }
    if (commits) {
        if constexpr (kBf16) {
            uint16_t *S = static_cast<uint16_t *>(a.pool) + at;
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                __stcs(reinterpret_cast<uint2 *>(S + (row0 + r) * kD) + lane,
                       make_uint2(float2_to_bf16x2(x[r].x, x[r].y), float2_to_bf16x2(x[r].z, x[r].w)));
        } else {
            float *S = static_cast<float *>(a.pool) + at;
#pragma unroll
            for (int r = 0; r < kRows; ++r) __stcs(reinterpret_cast<float4 *>(S + (row0 + r) * kD) + lane, x[r]);
        }
    }

    // 2. the new tokens
    for (int64_t t0 = 0; t0 < tokens; t0 += kBlock) {
        const int m = static_cast<int>(min(static_cast<int64_t>(kBlock), tokens - t0));
        const int64_t first = (n * a.T + t0) * a.H + h;
        __syncthreads();
        load_rows(s.q, a.q, first, a.H, m);
        load_rows(s.k, a.k, first, a.H, m);
        load_rows(s.v, a.v, first, a.H, m);
        if (threadIdx.x < m) s.gate[threadIdx.x] = __ldg(a.g + first + static_cast<int64_t>(threadIdx.x) * a.H);
        __syncthreads();
        gate_sums(s, m);
        for (int i = warp; i < m * m; i += kWarps) {
            const int t = i / m, j = i - t * m;
            if (j > t) continue;
            float d = 0.f;
#pragma unroll
            for (int c = lane; c < kD; c += 32) d = fmaf(s.q[t][c], s.k[j][c], d);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
            float sum = 0.f;
            for (int i2 = j + 1; i2 <= t; ++i2) sum += s.gate[i2];
            if (lane == 0) s.score[t][j] = expf(sum) * d;
        }
        for (int t = 0; t < m; ++t) {
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float q = s.q[t][row0 + r];
                acc.x = fmaf(q, x[r].x, acc.x);
                acc.y = fmaf(q, x[r].y, acc.y);
                acc.z = fmaf(q, x[r].z, acc.z);
                acc.w = fmaf(q, x[r].w, acc.w);
            }
            *reinterpret_cast<float4 *>(&s.part[warp][t][4 * lane]) = acc;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < m * (kD / 2); e += kThreads) {
            const int t = e / (kD / 2), c = 2 * (e % (kD / 2));
            float a0 = 0.f, a1 = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                a0 += s.part[w][t][c];
                a1 += s.part[w][t][c + 1];
            }
            a0 *= s.head[t];
            a1 *= s.head[t];
            for (int j = 0; j <= t; ++j) {
                a0 = fmaf(s.score[t][j], s.v[j][c], a0);
                a1 = fmaf(s.score[t][j], s.v[j][c + 1], a1);
            }
            reinterpret_cast<uint32_t *>(a.o + (first + static_cast<int64_t>(t) * a.H) * kD)[c / 2] =
                float2_to_bf16x2(a.scale * a0, a.scale * a1);
        }
        if (t0 + kBlock < tokens) advance(x, s, m, row0, lane);
    }
}

}  // namespace

cudaError_t launch_draft_step(const void *q, const void *k, const void *v, const float *g,
                              const int32_t *num_tokens, const void *pend_k, const void *pend_v,
                              const float *pend_g, const int32_t *accepted, float scale, void *pool,
                              bool bf16, const int32_t *slots, int64_t P, void *o, int64_t N,
                              int64_t T, int64_t T_pend, int H, int *status, cudaStream_t stream) {
    LaunchTimer timer(kKDraftStep, stream);
    const DraftArgs a{static_cast<const uint16_t *>(q), static_cast<const uint16_t *>(k),
                      static_cast<const uint16_t *>(v), g, num_tokens,
                      static_cast<const uint16_t *>(pend_k), static_cast<const uint16_t *>(pend_v),
                      pend_g, accepted, scale, pool, slots, P, static_cast<uint16_t *>(o), T, T_pend, H,
                      status};
    const unsigned blocks = static_cast<unsigned>(N * H);
    return bf16 ? launch_dependent(draft_step_kernel<true>, blocks, kThreads, stream, a)
                : launch_dependent(draft_step_kernel<false>, blocks, kThreads, stream, a);
}

}  // namespace sala

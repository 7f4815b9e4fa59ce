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
// A cluster of CTAs reads one row. The vocabulary is cut into one part per warp of the cluster, in
// order; every warp sums its part and hands the sum to the first CTA through distributed shared
// memory, which finds the part that holds the drawn number and goes through it again (from L2).
//
// Bound by the memory for large batches, short of the copy rate by the dependent steps at both ends
// of a row: 256 rows of 131072 fp32 (5 drafts) take 47 us where the bytes of p_a and (for the 76 % of rows with
// a rejection) q_a need 35 us, 1024 rows 148 us (floor 140); one row of 65536 takes 5.8 us, which is latency.
// With bf16 the same bytes take 1.6 times the instructions: 512 rows of 131072 take 56 us (floor 35), with the
// issue slots a half and the memory two fifths busy. Rows of p and q that are not aligned alike are read one
// value at a time: 256 fp32 rows of 50257 take 29.0 us, of 50256 25.1; bf16 23.9 and 19.2.
#include <cooperative_groups.h>

#include <type_traits>

#include "launch.h"
#include "tc.cuh"

namespace sala {

namespace {

namespace cg = cooperative_groups;

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;

template <typename T>
__device__ __forceinline__ float prob_load(const T *p) {
    if constexpr (std::is_same<T, float>::value) return __ldg(p);
    else return bf16_bits_to_float(__ldg(p));
}

// A probability in [0, 1] in units of 2^-43, rounded to nearest even, as hi * 2^21 + lo:
// adding 2 to p rounds it to a multiple of 2^-22, adding
// 3 * 2^-21 to the remainder rounds that to a multiple of 2^-43, and either sum's bits
// hold the multiple in the low mantissa. Both parts carry a constant, which differences lose.
// The second sum is p less (2 + p rounded, less 2 + 3 * 2^-21), a difference that is exact.
// (A conversion to a 64-bit integer gives the same value but goes through the fp64 units, of
// which this GPU has few.)
struct Units {
    int hi, lo;
};
__device__ __forceinline__ Units prob_units(float p) {
    const float a = __fadd_rn(p, 2.f);
    return {__float_as_int(a), __float_as_int(__fsub_rn(p, __fsub_rn(a, 2.000001430511474609375f)))};
}
// The same of two probabilities at a time, in half the instructions (with the packed clamps of bf16 and a
// 64-bit sum per four vectors: 512 rows of 131072 bf16 75 -> 64 us at 8 CTAs a row).
struct Units2 {
    int hi[2], lo[2];
};
__device__ __forceinline__ Units2 prob_units2(float p0, float p1) {
    Units2 u;
    asm("{\n\t.reg .b64 p, a, b;\n\t.reg .b64 two, shift, minus;\n\t"
        "mov.b64 p, {%4, %5};\n\t"
        "mov.b64 two, {%6, %6};\n\t"
        "mov.b64 shift, {%7, %7};\n\t"
        "mov.b64 minus, {%8, %8};\n\t"
        "add.rn.f32x2 a, p, two;\n\t"
        "fma.rn.f32x2 b, a, minus, shift;\n\t"
        "add.rn.f32x2 b, p, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t"
        "mov.b64 {%2, %3}, b;\n\t}"
        : "=r"(u.hi[0]), "=r"(u.hi[1]), "=r"(u.lo[0]), "=r"(u.lo[1])
        : "f"(p0), "f"(p1), "f"(2.f), "f"(2.000001430511474609375f), "f"(-1.f));
    return u;
}
constexpr Units kZeroUnits = {0x40000000, 0x35c00000};   // bits of 2 and of 3 * 2^-21

// Sum of max(p - q, 0) over some tokens, in two 32-bit parts: 256 tokens of probability 1 fit.
struct PartSum {
    int hi = 0, lo = 0;
    __device__ __forceinline__ void add_units(Units p, Units q) {
        hi += p.hi - q.hi;
        lo += p.lo - q.lo;
    }
    // rounding keeps the order, so the larger of p and q has the larger units
    __device__ __forceinline__ void add(float p, float q) {
        q = __saturatef(q);
        add_units(prob_units(fmaxf(__saturatef(p), q)), prob_units(q));
    }
    __device__ __forceinline__ void add(float p) { add_units(prob_units(__saturatef(p)), kZeroUnits); }
    // two tokens whose larger m = max(p, q) and q are in [0, 1]
    __device__ __forceinline__ void add2(float m0, float m1, float q0, float q1) {
        const Units2 m = prob_units2(m0, m1), q = prob_units2(q0, q1);
        add_units({m.hi[0], m.lo[0]}, {q.hi[0], q.lo[0]});
        add_units({m.hi[1], m.lo[1]}, {q.hi[1], q.lo[1]});
    }
    __device__ __forceinline__ void add2(float p0, float p1) {
        const Units2 p = prob_units2(p0, p1);
        add_units({p.hi[0], p.lo[0]}, kZeroUnits);
        add_units({p.hi[1], p.lo[1]}, kZeroUnits);
    }
    __device__ __forceinline__ unsigned long long units() const {
        return static_cast<unsigned long long>(static_cast<long long>(hi) * (1 << 21) + lo);
    }
};
// Sums over a row are unsigned: 2^20 tokens of probability 1 have 2^63 units.
using Sum = unsigned long long;

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
    for (int base = 0; base < a.K; base += 32) {
        const int i = base + lane;
        // all loads that need no other go out together
        const int32_t x = i < a.K ? __ldg(a.x + n * a.K + i) : -1;
        const float u = i < a.K ? __ldg(a.u + n * a.K + i) : 0.f;
        bool stop = true, no = false;   // a negative token ends the row's drafts
        if (x >= 0 && x < a.V) {
            const T *p = static_cast<const T *>(a.p) + (n * (a.K + 1) + i) * a.p_stride;
            const T *q = static_cast<const T *>(a.q) + (n * a.K + i) * a.q_stride;
            // taken into [0, 1] as in the sums (NaN as 0); two 24-bit factors: the product is exact in 64 bits
            const float qx = a.q ? __saturatef(prob_load(q + x)) : 1.f, px = __saturatef(prob_load(p + x));
            no = !(static_cast<double>(u) * qx < static_cast<double>(px));
            stop = no;
        }
        if (i >= drafts) stop = true, no = false;
        const unsigned stops = __ballot_sync(0xffffffffu, stop);
        if (stops) {
            const int first = __ffs(stops) - 1;
            *rejected = __shfl_sync(0xffffffffu, no, first);
            if (lane == first && i < drafts && x >= a.V) record_status(a.status, SALA_ERR_BAD_INDEX);
            return base + first;
        }
    }
    return drafts;
}

// The distribution that a row's next token is drawn from: the target's row p, less the drafter's
// row q or less a certain token (a drafter without probabilities) where a draft was rejected.
template <typename T>
struct Weights {
    const T *p, *q;
    int one_at;

    __device__ __forceinline__ Sum at(int x) const {
        PartSum s;
        if (q) s.add(prob_load(p + x), prob_load(q + x));
        else if (x != one_at) s.add(prob_load(p + x));
        return s.units();
    }
};

__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

// 16 bytes of probabilities
template <typename T>
struct Vec {
    static constexpr int kN = 16 / sizeof(T);
    uint4 w;
    __device__ __forceinline__ void load(const T *p) { w = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ float at(int i) const {
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        if constexpr (sizeof(T) == 4) return __uint_as_float(ws[i]);
        const float2 f = bf16x2_to_float2(ws[i / 2]);
        return i & 1 ? f.y : f.x;
    }
};

// Pairs of bf16, the larger or smaller of each (a NaN yields to the other).
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// s += max(p - q, 0), or p, over 16 bytes of probabilities.
template <typename T, bool kQ>
__device__ __forceinline__ void add_vector(PartSum &s, uint4 p, uint4 q) {
    const uint32_t ps[4] = {p.x, p.y, p.z, p.w}, qs[4] = {q.x, q.y, q.z, q.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const float p0 = __saturatef(__uint_as_float(ps[i])), p1 = __saturatef(__uint_as_float(ps[i + 1]));
            if constexpr (kQ) {
                const float q0 = __saturatef(__uint_as_float(qs[i])), q1 = __saturatef(__uint_as_float(qs[i + 1]));
                s.add2(fmaxf(p0, q0), fmaxf(p1, q1), q0, q1);
            } else {
                s.add2(p0, p1);
            }
        }
    } else {
        constexpr uint32_t kOnes = 0x3f803f80u;   // 1, 1
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 y = bf16x2_to_float2(kQ ? min2(max2(qs[i], 0u), kOnes) : 0u);
            const float2 x = bf16x2_to_float2(min2(max2(ps[i], kQ ? min2(max2(qs[i], 0u), kOnes) : 0u), kOnes));
            if constexpr (kQ) s.add2(x.x, x.y, y.x, y.y);
            else s.add2(x.x, x.y);
        }
    }
}

// Loads run ahead of the sums through shared memory, kAhead vectors of p and of q per lane. Each
// lane copies (cp.async) and reads its own slots, so no barrier is needed.
constexpr int kAhead = 4;
struct Ring {
    uint4 v[2][kAhead][kVerifyThreads];   // p, q
};

// One lane's share of the sum over tokens [lo, hi), `lo` aligned for 16-byte loads of p and, with
// kQ (subtract the drafter's row), of q.
template <typename T, bool kQ>
__device__ __forceinline__ Sum sum_vectors(const Weights<T> &w, int lo, int hi, int lane, Ring &ring) {
    constexpr int kN = Vec<T>::kN;
    Sum sum = 0;
    const T *p = w.p + lo + lane * kN, *q = kQ ? w.q + lo + lane * kN : nullptr;
    const int vectors = (hi - lo) / kN - lane;   // of this lane: 0, 32, 64, ..
    uint4 *mine[2] = {&ring.v[0][0][threadIdx.x], &ring.v[1][0][threadIdx.x]};
    auto load = [&](int v, int slot) {
        const bool ok = v < vectors;   // zeros past the end
        const int at = ok ? v * kN : 0;
        cp_async16(mine[0] + slot * kVerifyThreads, p + at, ok);
        if constexpr (kQ) cp_async16(mine[1] + slot * kVerifyThreads, q + at, ok);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (vectors > 0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load(32 * i, i);
        for (int v = 0; v < vectors; v += 32 * kAhead) {
            PartSum s;
            static_assert(kN * kAhead <= 256, "a part's sum holds them");
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
                const uint4 x = mine[0][i * kVerifyThreads];
                uint4 y{};
                if constexpr (kQ) y = mine[1][i * kVerifyThreads];
                load(v + 32 * (i + kAhead), i);
                add_vector<T, kQ>(s, x, y);
            }
            sum += s.units();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    // fewer than a vector's tokens, where the part ends the row
    const int rest = lo + (hi - lo) / kN * kN + lane;
    if (rest < hi) {
        PartSum s;
        if constexpr (kQ) s.add(prob_load(w.p + rest), prob_load(w.q + rest));
        else s.add(prob_load(w.p + rest));
        sum += s.units();
    }
    return sum;
}

// The sum of the weights of tokens [lo, hi) by one warp; every lane returns it.
template <typename T>
__device__ __forceinline__ Sum sum_part(const Weights<T> &w, int lo, int hi, int lane, Ring &ring) {
    Sum sum = 0;
    const uintptr_t bp = reinterpret_cast<uintptr_t>(w.p), bq = reinterpret_cast<uintptr_t>(w.q);
    if (!w.q || ((bp ^ bq) & 15) == 0) {
        // tokens before the first aligned one (only where the part begins the row)
        const int start = min(hi, lo + static_cast<int>((-(bp + lo * sizeof(T)) & 15) / sizeof(T)));
        PartSum s;
        if (lo + lane < start) {
            if (w.q) s.add(prob_load(w.p + lo + lane), prob_load(w.q + lo + lane));
            else s.add(prob_load(w.p + lo + lane));
        }
        sum = s.units() + (w.q ? sum_vectors<T, true>(w, start, hi, lane, ring)
                               : sum_vectors<T, false>(w, start, hi, lane, ring));
        // the certain token was summed with its whole probability
        if (lane == 0 && w.one_at >= lo && w.one_at < hi) {
            PartSum one;
            one.add(prob_load(w.p + w.one_at));
            sum -= one.units();
        }
    } else {
        // rows whose starts differ modulo 16 bytes: one token at a time, eight in flight
        for (int x = lo + lane; x - lane < hi; x += 8 * 32) {
            float p[8], q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool ok = x + 32 * i < hi;
                p[i] = ok ? prob_load(w.p + x + 32 * i) : 0.f;
                q[i] = ok ? prob_load(w.q + x + 32 * i) : 0.f;
            }
            PartSum s;
#pragma unroll
            for (int i = 0; i < 8; ++i) s.add(p[i], q[i]);
            sum += s.units();
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    return sum;
}

// Inclusive prefix sum over the lanes of a warp.
__device__ __forceinline__ Sum warp_prefix(Sum c, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const Sum y = __shfl_up_sync(0xffffffffu, c, off);
        if (lane >= off) c += y;
    }
    return c;
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) verify_drafts_kernel(VerifyArgs a) {
    dependent_start();
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int64_t n = blockIdx.x / ranks;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ Ring ring;
    __shared__ int first_s, rejected_s;
    __shared__ Sum all[kMaxCluster * kVerifyWarps];   // sums of the parts, in the first CTA
    __shared__ Sum scan[kVerifyWarps];
    cluster.barrier_arrive();   // waited for before the first CTA's memory is written

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
    Weights<T> w{static_cast<const T *>(a.p) + (n * (a.K + 1) + first) * a.p_stride, nullptr, -1};
    if (rejected_s) {
        if (a.q) w.q = static_cast<const T *>(a.q) + (n * a.K + first) * a.q_stride;
        else w.one_at = __ldg(a.x + n * a.K + first);
    }

    // parts: from the second on they begin at 16-byte boundaries of the target's row
    constexpr int kN = Vec<T>::kN;
    const int parts = ranks * kVerifyWarps;
    const int V = static_cast<int>(a.V), head = static_cast<int>((-reinterpret_cast<uintptr_t>(w.p) & 15) / sizeof(T));
    const int len = (V / kN + parts) / parts * kN;
    auto part_begin = [&](int i) { return i == 0 ? 0 : min(V, head + len * i); };

    // every warp hands its sum to the first CTA, which goes on alone: the others make room
    {
        const int i = rank * kVerifyWarps + warp;
        const Sum sum = sum_part(w, part_begin(i), part_begin(i + 1), lane, ring);
        cluster.barrier_wait();
        if (lane == 0) *cluster.map_shared_rank(&all[i], 0) = sum;
        cluster.barrier_arrive();
        if (rank != 0) return;
        cluster.barrier_wait();
    }
    auto sum_all = [&] {
        Sum t = 0;
        for (int j = lane; j < parts; j += 32) t += all[j];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
        return t;
    };
    Sum total = sum_all();
    if (total == 0 && rejected_s) {
        // nothing is left of the target after the drafter's part: draw from the target
        w.q = nullptr;
        w.one_at = -1;
        __syncthreads();
        for (int i = warp; i < parts; i += kVerifyWarps) {
            const Sum sum = sum_part(w, part_begin(i), part_begin(i + 1), lane, ring);
            if (lane == 0) all[i] = sum;
        }
        __syncthreads();
        total = sum_all();
    }

    int32_t *out = a.tokens + n * (a.K + 1);
    for (int i = threadIdx.x; i <= a.K; i += kVerifyThreads)
        if (i != first || total == 0) out[i] = i < first ? __ldg(a.x + n * a.K + i) : -1;
    if (threadIdx.x == 0) a.accepted[n] = first;
    if (total != 0) {
        // the number drawn, in the same units: the whole part of s * total (s is a whole number of
        // 2^-64, or closer to 0 than that)
        float s = __ldg(a.s + n);
        s = s >= 0.f ? fminf(s, 0.99999994f) : 0.f;
        const Sum at = __umul64hi(__float2ull_rz(s * 18446744073709551616.f), total);
        // the part that holds it: every warp finds the same one
        Sum before = 0;
        int part = -1;
        for (int j0 = 0; j0 < parts; j0 += 32) {
            const Sum own = j0 + lane < parts ? all[j0 + lane] : 0;
            const Sum c = before + warp_prefix(own, lane);
            const unsigned past = __ballot_sync(0xffffffffu, c > at);
            if (past) {
                const int l = __ffs(past) - 1;
                part = j0 + l;
                before = __shfl_sync(0xffffffffu, c - own, l);
                break;
            }
            before = __shfl_sync(0xffffffffu, c, 31);
        }
        {
            // each thread sums consecutive vectors of the part (the first thread also what lies before
            // the first whole one), then the one that passes `at` looks for its token
            const int lo = part_begin(part), hi = part_begin(part + 1);
            const int start = part == 0 ? min(hi, head) : lo;
            const int per = ((hi - start + kN - 1) / kN + kVerifyThreads - 1) / kVerifyThreads * kN;
            const int tid = threadIdx.x, x0 = tid == 0 ? lo : min(hi, start + per * tid);
            const int x1 = min(hi, start + per * (tid + 1));
            const bool wide = !w.q || ((reinterpret_cast<uintptr_t>(w.p) ^ reinterpret_cast<uintptr_t>(w.q)) & 15) == 0;
            Sum sum = 0;
            int x = x0;
            if (wide) {
                for (; x < min(start, x1); ++x) sum += w.at(x);
                for (; x + kN <= x1; x += kN) {
                    Vec<T> p, q;
                    p.load(w.p + x);
                    if (w.q) q.load(w.q + x);
                    PartSum s;
#pragma unroll
                    for (int e = 0; e < kN; ++e) {
                        if (w.q) s.add(p.at(e), q.at(e));
                        else s.add(x + e == w.one_at ? 0.f : p.at(e));
                    }
                    sum += s.units();
                }
            }
#pragma unroll 8
            for (; x < x1; ++x) sum += w.at(x);
            const Sum c = warp_prefix(sum, lane);
            if (lane == 31) scan[warp] = c;
            __syncthreads();
            Sum run = before + c - sum;
            for (int i = 0; i < warp; ++i) run += scan[i];
            if (run <= at && at < run + sum) {
                for (x = x0; x < x1; ++x) {
                    run += w.at(x);
                    if (run > at) {
                        out[first] = x;
                        break;
                    }
                }
            }
        }
    }
}

// CTAs that share a row. Each pays some 5 us of dependent steps (the accept test, the hand-over of its
// sums), so it gets at least 12 KB of the row's target probabilities (32 rows of 8000 bf16: 8 CTAs 7.5 us,
// 1 CTA 5.9) and, where the launch fills the SMs anyway, 48 KB (2048 rows of 32000 bf16: 8 CTAs 132 us, 2
// CTAs 61, 1 CTA 54; 1024 rows of 131072 bf16: 8 CTAs 118, 4 CTAs 98, 2 CTAs 101). More CTAs where there is
// more to read: their ends overlap better (1024 rows of 131072 fp32: 8 CTAs 148 us, 4 CTAs 154, 2 CTAs 201).
int cluster_size(int64_t N, int64_t row_bytes, int sm_count) {
    int c = kMaxCluster;
    while (c > 1 && (row_bytes < c * (12 << 10) || (N * c > 8 * sm_count && row_bytes < c * (48 << 10)))) c /= 2;
    return c;
}

// Shared memory asked for beyond a CTA's own so that at most `per_sm` of them share an SM.
constexpr size_t kSmSmem = 227 * 1024, kStaticSmem = sizeof(Ring) + 2048;
size_t room_for(int per_sm) { return kSmSmem / per_sm - kStaticSmem; }
static_assert(kSmSmem / kVerifyFits >= kStaticSmem, "a CTA's own memory fits so often");

// A cluster's CTAs are packed onto as few SMs as hold them, so a small launch would leave most SMs
// idle: it asks for the most memory per CTA with which all its clusters still run at once (32 rows of
// 131072 fp32: 14.3 us packed, 12.2 us spread).
size_t spread(int64_t N, int c, const int *fits) {
    for (int i = 0; c == kMaxCluster && i < kVerifyFits; ++i)
        if (N <= fits[i]) return room_for(i + 1);
    return 0;
}

}  // namespace

cudaError_t setup_verify_drafts_kernel(int *fits) {
    void (*kernels[2])(VerifyArgs) = {verify_drafts_kernel<float>, verify_drafts_kernel<uint16_t>};
    for (auto kern : kernels) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(room_for(1)));
        if (e != cudaSuccess) return e;
    }
    for (int i = 0; i < kVerifyFits; ++i) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kMaxCluster);
        cfg.blockDim = dim3(kVerifyThreads);
        cfg.dynamicSmemBytes = room_for(i + 1);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kMaxCluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&fits[i], verify_drafts_kernel<float>, &cfg) != cudaSuccess) {
            fits[i] = 0;   // no answer: launches are not spread
            cudaGetLastError();
        }
    }
    return cudaSuccess;
}

cudaError_t launch_verify_drafts(const void *p, int64_t p_stride, const void *q, int64_t q_stride,
                                 bool bf16, const int32_t *x, const int32_t *num_drafts,
                                 const float *u, const float *s, int32_t *tokens,
                                 int32_t *accepted, int64_t N, int K, int64_t V, int sm_count,
                                 const int *fits, int *status, cudaStream_t stream) {
    LaunchTimer timer(kKVerifyDrafts, stream);
    const int c = cluster_size(N, V * (bf16 ? 2 : 4), sm_count);
    const size_t room = spread(N, c, fits);
    const VerifyArgs a{p, q, p_stride, q_stride, x, num_drafts, u, s, tokens, accepted, K, V, status};
    return launch_dependent_cluster(bf16 ? verify_drafts_kernel<uint16_t> : verify_drafts_kernel<float>,
                                    static_cast<unsigned>(N * c), c, kVerifyThreads, room, stream, a);
}

}  // namespace sala

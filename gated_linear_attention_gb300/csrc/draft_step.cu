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
// Steps of up to 16 new and 16 pending tokens (draft_step_kernel): one CTA of 4 warps per
// (sequence, head, half of the value columns). The state half goes through shared memory
// (cp.async in, 16-byte stores out); the two products with it run on the tensor cores as
// mma.m16n8k16, 16 being the tokens:
//     commit   D[16 dv x 8 dk] = (w V)^T K     with w_j v_j in fp32 split into bf16 parts
//     read     O[16 t x 8 dv]  = Q S           with S in fp32 split into two bf16 parts
// The accumulator layout of the first is the B operand layout of the second, so the state goes
// from one to the other in registers, 16 key rows at a time, and is never held whole. A token
// that is not there (past the counts) is zero in shared memory; the products among the new
// tokens are taken in fp32 over j <= t only, so nothing of a masked place reaches a result.
// Longer steps (draft_step_long_kernel) run the plain form below.
#include <type_traits>

#include "launch.h"
#include "tc.cuh"

namespace sala {

namespace {

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

// What row n of the batch does: its slot, the commits and the new tokens.
struct Row {
    int32_t slot;
    int64_t commits, tokens;   // 0, 0 for a padding row
};
__device__ __forceinline__ Row read_row(const DraftArgs &a, int n) {
    Row r;
    r.slot = __ldg(a.slots + n);
    r.commits = a.T_pend ? static_cast<int64_t>(__ldg(a.accepted + n)) + 1 : 0;
    r.tokens = a.num_tokens ? __ldg(a.num_tokens + n) : a.T;
    if (r.commits < 0) r.commits = 0;
    const bool bad = r.slot >= a.P || r.commits > a.T_pend || r.tokens < 0 || r.tokens > a.T;
    if (bad && threadIdx.x == 0) record_status(a.status, SALA_ERR_BAD_INDEX);
    if (bad || r.slot < 0) r.commits = r.tokens = 0;
    return r;
}

// ---- steps of up to 16 + 16 tokens ---------------------------------------------------------

constexpr int kTok = 16;             // tokens of an mma operand
constexpr int kHalf = kD / 2;        // value columns of a CTA
constexpr int kStepThreads = 128;    // warp w: columns [16 w, 16 w + 16) of the half

// Shared memory of a CTA (offsets in bytes from a 128-byte aligned base). Rows are cut into
// 16-byte chunks whose places are permuted by the row so that the 8 rows of a matrix fragment (and,
// for fp32 states, the 4 even or odd rows of one) fall into different banks.
template <bool kBf16>
struct StepSmem {
    static constexpr int kStateRow = kHalf * (kBf16 ? 2 : 4);
    static constexpr int kState = 0;
    static constexpr int kPk = kState + kD * kStateRow;      // [16][128] bf16
    static constexpr int kQ = kPk + kTok * kD * 2;
    static constexpr int kK = kQ + kTok * kD * 2;
    static constexpr int kPv = kK + kTok * kD * 2;           // [16][64] bf16
    static constexpr int kV = kPv + kTok * kHalf * 2;
    static constexpr int kScore = kV + kTok * kHalf * 2;     // [16][16] fp32: q_t . k_j
    static constexpr int kDecay = kScore + kTok * kTok * 4;  // [16][16] fp32: exp(g_{j+1} + .. + g_t)
    static constexpr int kBytes = kDecay + kTok * kTok * 4;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// d += a b, m16n8k16, bf16 operands
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float lds_f32(uint32_t addr) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ void sts_f32(uint32_t addr, float x) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}

// Chunk c of row r: rows of 16 chunks (tokens' 128 keys), rows of 8 chunks (64 values in bf16).
__device__ __forceinline__ uint32_t chunk256(int r, int c) { return r * 256 + ((c ^ (r & 7)) << 4); }
__device__ __forceinline__ uint32_t chunk128(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }
// fp32 state half: rows of 16 chunks; 8 columns take two neighbouring ones, which stay together.
__device__ __forceinline__ uint32_t chunk_f32(int r, int c) { return r * 256 + ((c ^ (((r >> 1) & 3) << 1)) << 4); }

// `rows` token rows of [tokens, H, 128] bf16, `chunks` 16-byte chunks each, zeros past `count`.
template <bool kWide>
__device__ __forceinline__ void stage_tokens(uint32_t dst, const uint16_t *src, int64_t row0, int H, int count) {
    constexpr int kChunks = kWide ? 16 : 8;
#pragma unroll
    for (int i = 0; i < kTok * kChunks / kStepThreads; ++i) {
        const int e = threadIdx.x + i * kStepThreads, t = e / kChunks, c = e % kChunks;
        const bool ok = t < count;
        const uint16_t *p = src + (row0 + (ok ? static_cast<int64_t>(t) * H : 0)) * kD + 8 * c;
        cp_async16(dst + (kWide ? chunk256(t, c) : chunk128(t, c)), p, ok);
    }
}

// Lane t holds exp(g_1 + .. + g_t) (head) and exp(g_{t+1} + .. + g_count) (tail) of up to 16 gates, 0 past the count.
struct Gates {
    float g, head, tail;
};
__device__ __forceinline__ Gates gate_scan(const float *g, int64_t row0, int H, int count, int lane) {
    Gates s;
    s.g = lane < count ? __ldg(g + row0 + static_cast<int64_t>(lane) * H) : 0.f;
    float pre = s.g, suf = s.g;
#pragma unroll
    for (int off = 1; off < kTok; off <<= 1) {
        const float a = __shfl_up_sync(0xffffffffu, pre, off), b = __shfl_down_sync(0xffffffffu, suf, off);
        if (lane >= off) pre += a;
        if (lane + off < kTok) suf += b;
    }
    const float next = __shfl_down_sync(0xffffffffu, suf, 1);
    s.head = lane < count ? expf(pre) : 0.f;
    s.tail = lane < count ? expf(lane + 1 < kTok ? next : 0.f) : 0.f;
    return s;
}

// x split into bf16 parts that sum to it: packed pairs (x0 in the low half).
__device__ __forceinline__ uint32_t split_bf16(float &x0, float &x1) {
    const uint32_t w = float2_to_bf16x2(x0, x1);
    const float2 f = bf16x2_to_float2(w);
    x0 -= f.x;
    x1 -= f.y;
    return w;
}

template <bool kBf16>
__global__ void __launch_bounds__(kStepThreads) draft_step_kernel(DraftArgs a) {
    dependent_start();
    using Sm = StepSmem<kBf16>;
    constexpr int kParts = 3;   // of w_j v_j in fp32: what three bf16 parts leave out is below 2^-26 of it
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sm = tc::smem_u32(smem);
    const int unit = blockIdx.x >> 1, half = blockIdx.x & 1, n = unit / a.H, h = unit - n * a.H;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gr = lane >> 2, tq = lane & 3;   // row and column pair of a lane in a fragment
    const Row row = read_row(a, n);
    const int commits = static_cast<int>(row.commits), tokens = static_cast<int>(row.tokens);
    for (int e = tokens * 8 + tid; e < static_cast<int>(a.T) * 8; e += kStepThreads)   // rows past the count
        *reinterpret_cast<uint4 *>(a.o + ((n * a.T + e / 8) * a.H + h) * kD + half * kHalf + 8 * (e % 8)) =
            make_uint4(0, 0, 0, 0);
    if (commits == 0 && tokens == 0) return;

    // 1. everything the CTA reads, in flight at once
    const int64_t at = (static_cast<int64_t>(row.slot) * a.H + h) * kD * kD + half * kHalf;
    constexpr int kChunks = Sm::kStateRow / 16;   // of a state row
#pragma unroll
    for (int i = 0; i < kD * kChunks / kStepThreads; ++i) {
        const int e = tid + i * kStepThreads, r = e / kChunks, c = e % kChunks;
        if constexpr (kBf16)
            cp_async16(sm + Sm::kState + chunk128(r, c), static_cast<const uint16_t *>(a.pool) + at + r * kD + 8 * c, true);
        else
            cp_async16(sm + Sm::kState + chunk_f32(r, c), static_cast<const float *>(a.pool) + at + r * kD + 4 * c, true);
    }
    const int64_t pend0 = n * a.T_pend * a.H + h, new0 = n * a.T * a.H + h;   // token rows of this head
    Gates pg{0.f, 0.f, 0.f}, ng{0.f, 0.f, 0.f};
    if (commits) {
        stage_tokens<true>(sm + Sm::kPk, a.pk, pend0, a.H, commits);
        stage_tokens<false>(sm + Sm::kPv, a.pv + half * kHalf, pend0, a.H, commits);
        pg = gate_scan(a.pg, pend0, a.H, commits, lane);
    }
    if (tokens) {
        stage_tokens<true>(sm + Sm::kQ, a.q, new0, a.H, tokens);
        stage_tokens<true>(sm + Sm::kK, a.k, new0, a.H, tokens);
        stage_tokens<false>(sm + Sm::kV, a.v + half * kHalf, new0, a.H, tokens);
        ng = gate_scan(a.g, new0, a.H, tokens, lane);
    }
    asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    // fragment addresses: matrix `lane / 8` of four, row `lane % 8`
    const int mi = lane >> 3, mr = lane & 7;

    // 2. products among the new tokens: scores by warps 0 and 1, decays by warp 2
    if (tokens && warp < 2 && 8 * warp < tokens) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
            uint32_t qa[4], qb[4], kb[4];
            ldmatrix_x4(qa, sm + Sm::kQ + chunk256(mr + 8 * (mi & 1), 2 * c + (mi >> 1)));
            ldmatrix_x4(qb, sm + Sm::kQ + chunk256(mr + 8 * (mi & 1), 2 * c + 2 + (mi >> 1)));
            ldmatrix_x4(kb, sm + Sm::kK + chunk256(mr + 8 * warp, 2 * c + mi));
            mma(d, qa, kb[0], kb[1]);
            mma(d, qb, kb[2], kb[3]);
        }
        const uint32_t s = sm + Sm::kScore + (gr * kTok + 8 * warp + 2 * tq) * 4;
        sts_f32(s, d[0]);
        sts_f32(s + 4, d[1]);
        sts_f32(s + 8 * kTok * 4, d[2]);
        sts_f32(s + 8 * kTok * 4 + 4, d[3]);
    }
    if (tokens && warp == 2) {
        float sum = 0.f;   // lane j: g_{j+1} + .. + g_t
        for (int t = 0; t < tokens; ++t) {
            const float g = __shfl_sync(0xffffffffu, ng.g, t);
            if (t > lane) sum += g;
            if (lane <= t) sts_f32(sm + Sm::kDecay + (t * kTok + lane) * 4, expf(sum));
        }
    }

    // 3. the state, 16 key rows at a time
    uint32_t wv[kParts][4];
    const float fade = commits ? __shfl_sync(0xffffffffu, pg.head, commits - 1) : 1.f;
    if (commits) {
        uint32_t f[4];   // V^T: (dv, tok), (dv + 8, tok), (dv, tok + 8), (dv + 8, tok + 8)
        ldmatrix_x4_trans(f, sm + Sm::kPv + chunk128(mr + 8 * (mi >> 1), 2 * warp + (mi & 1)));
        const float w0 = __shfl_sync(0xffffffffu, pg.tail, 2 * tq), w1 = __shfl_sync(0xffffffffu, pg.tail, 2 * tq + 1),
                    w2 = __shfl_sync(0xffffffffu, pg.tail, 2 * tq + 8), w3 = __shfl_sync(0xffffffffu, pg.tail, 2 * tq + 9);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 x = bf16x2_to_float2(f[i]);
            x.x *= i < 2 ? w0 : w2;
            x.y *= i < 2 ? w1 : w3;
#pragma unroll
            for (int p = 0; p < kParts; ++p) wv[p][i] = split_bf16(x.x, x.y);
        }
    }
    float o[2][4] = {};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        // x[i][m]: rows 16 c + 8 i + 2 tq, + 1; columns gr, gr + 8 of the warp's 16
        float x[2][4];
        uint32_t sb[4];
        const uint32_t sb_at = sm + Sm::kState + chunk128(16 * c + mr + 8 * (mi >> 1), 2 * warp + (mi & 1));
        const uint32_t sf_at = sm + Sm::kState + chunk_f32(16 * c + 2 * tq, 4 * warp + (gr >> 2)) + (gr & 3) * 4;
        // columns gr + 8 lie two chunks further, in the other pair that the row's permutation joins;
        // the next row has the same permutation
        const uint32_t sf_at8 = sm + Sm::kState + chunk_f32(16 * c + 2 * tq, 4 * warp + 2 + (gr >> 2)) + (gr & 3) * 4;
        if constexpr (kBf16) {
            ldmatrix_x4_trans(sb, sb_at);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 f0 = bf16x2_to_float2(sb[2 * i]), f1 = bf16x2_to_float2(sb[2 * i + 1]);
                x[i][0] = f0.x, x[i][1] = f0.y, x[i][2] = f1.x, x[i][3] = f1.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {   // 8 rows on, the permutation repeats
                x[i][0] = lds_f32(sf_at + i * 8 * 256);
                x[i][1] = lds_f32(sf_at + i * 8 * 256 + 256);
                x[i][2] = lds_f32(sf_at8 + i * 8 * 256);
                x[i][3] = lds_f32(sf_at8 + i * 8 * 256 + 256);
            }
        }
        if (commits) {
            uint32_t kb[4];   // K: (tok, dk), (tok + 8, dk), (tok, dk + 8), (tok + 8, dk + 8)
            ldmatrix_x4_trans(kb, sm + Sm::kPk + chunk256(mr + 8 * (mi & 1), 2 * c + (mi >> 1)));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // summed apart from the state and added to it once: the state is rounded as in fp32
                // arithmetic, whatever the tensor cores' accumulation does
                float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int p = kParts - 1; p >= 0; --p) mma(d, wv[p], kb[2 * i], kb[2 * i + 1]);
#pragma unroll
                for (int m = 0; m < 4; ++m) x[i][m] = fmaf(fade, x[i][m], d[m]);
            }
        }
        // parts of the state for the read; the first is also what a bf16 pool stores
        uint32_t hi[2][2], lo[2][2];   // [rows][columns]
        if (tokens || kBf16) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float x0 = x[i][2 * m], x1 = x[i][2 * m + 1];
                    hi[i][m] = split_bf16(x0, x1);
                    lo[i][m] = float2_to_bf16x2(x0, x1);
                }
            }
        }
        if (commits) {
            if constexpr (kBf16) {
                tc::stmatrix_x4_trans(sb_at, hi[0][0], hi[0][1], hi[1][0], hi[1][1]);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    sts_f32(sf_at + i * 8 * 256, x[i][0]);
                    sts_f32(sf_at + i * 8 * 256 + 256, x[i][1]);
                    sts_f32(sf_at8 + i * 8 * 256, x[i][2]);
                    sts_f32(sf_at8 + i * 8 * 256 + 256, x[i][3]);
                }
            }
        }
        if (tokens) {
            uint32_t qa[4];   // (t, dk), (t + 8, dk), (t, dk + 8), (t + 8, dk + 8)
            ldmatrix_x4(qa, sm + Sm::kQ + chunk256(mr + 8 * (mi & 1), 2 * c + (mi >> 1)));
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                mma(o[m], qa, lo[0][m], lo[1][m]);
                mma(o[m], qa, hi[0][m], hi[1][m]);
            }
        }
    }
    __syncthreads();

    // 4. the state goes back
    if (commits) {
#pragma unroll
        for (int i = 0; i < kD * kChunks / kStepThreads; ++i) {
            const int e = tid + i * kStepThreads, r = e / kChunks, c = e % kChunks;
            const uint8_t *src = smem + Sm::kState + (kBf16 ? chunk128(r, c) : chunk_f32(r, c));
            const uint4 w = *reinterpret_cast<const uint4 *>(src);
            if constexpr (kBf16)
                __stcs(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.pool) + at + r * kD + 8 * c), w);
            else
                __stcs(reinterpret_cast<uint4 *>(static_cast<float *>(a.pool) + at + r * kD + 4 * c), w);
        }
    }

    // 5. o_t = scale ( head_t (Q S)_t + sum_{j <= t} decay_tj score_tj v_j ): rows gr, gr + 8
    if (tokens) {
        const float *score = reinterpret_cast<const float *>(smem + Sm::kScore);
        const float *decay = reinterpret_cast<const float *>(smem + Sm::kDecay);
        const float h0 = __shfl_sync(0xffffffffu, ng.head, gr), h1 = __shfl_sync(0xffffffffu, ng.head, gr + 8);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            o[m][0] *= h0;
            o[m][1] *= h0;
            o[m][2] *= h1;
            o[m][3] *= h1;
        }
        for (int j = 0; j < tokens; ++j) {
            const int c = 2 * warp;   // the warp's two chunks of the value row
            const float2 v0 = bf16x2_to_float2(*reinterpret_cast<const uint32_t *>(smem + Sm::kV + chunk128(j, c) + 4 * tq));
            const float2 v1 = bf16x2_to_float2(*reinterpret_cast<const uint32_t *>(smem + Sm::kV + chunk128(j, c + 1) + 4 * tq));
            if (j <= gr) {
                const float s = score[gr * kTok + j] * decay[gr * kTok + j];
                o[0][0] = fmaf(s, v0.x, o[0][0]);
                o[0][1] = fmaf(s, v0.y, o[0][1]);
                o[1][0] = fmaf(s, v1.x, o[1][0]);
                o[1][1] = fmaf(s, v1.y, o[1][1]);
            }
            if (j <= gr + 8) {
                const float s = score[(gr + 8) * kTok + j] * decay[(gr + 8) * kTok + j];
                o[0][2] = fmaf(s, v0.x, o[0][2]);
                o[0][3] = fmaf(s, v0.y, o[0][3]);
                o[1][2] = fmaf(s, v1.x, o[1][2]);
                o[1][3] = fmaf(s, v1.y, o[1][3]);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = gr + 8 * r;
            if (t >= tokens) continue;
            uint16_t *out = a.o + (new0 + static_cast<int64_t>(t) * a.H) * kD + half * kHalf + 16 * warp + 2 * tq;
#pragma unroll
            for (int m = 0; m < 2; ++m)
                *reinterpret_cast<uint32_t *>(out + 8 * m) = float2_to_bf16x2(a.scale * o[m][2 * r], a.scale * o[m][2 * r + 1]);
        }
    }
}

// ---- longer steps ----------------------------------------------------------------------------
//
// One CTA of 256 threads per (sequence, head); thread (w, l) holds rows [16 w, 16 w + 16) and
// columns [4 l, 4 l + 4) of the state in fp32. Tokens are taken in blocks of 8.

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = kD / kWarps;   // state rows of a warp
constexpr int kBlock = 8;            // tokens in flight

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
__global__ void __launch_bounds__(kThreads) draft_step_long_kernel(DraftArgs a) {
    dependent_start();
    __shared__ Tile s;
    const int unit = blockIdx.x, n = unit / a.H, h = unit - n * a.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = warp * kRows;
    const Row row = read_row(a, n);
    const int64_t commits = row.commits, tokens = row.tokens;
    for (int64_t e = tokens * (kD / 8) + threadIdx.x; e < a.T * (kD / 8); e += kThreads) {
        const int64_t t = e / (kD / 8);
        uint16_t *row = a.o + ((n * a.T + t) * a.H + h) * kD;
        reinterpret_cast<uint4 *>(row)[e % (kD / 8)] = make_uint4(0, 0, 0, 0);
    }
    if (commits == 0 && tokens == 0) return;

    const int64_t at = (static_cast<int64_t>(row.slot) * a.H + h) * kD * kD;
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
    if (T <= kTok && T_pend <= kTok)
        return bf16 ? launch_dependent_cluster(draft_step_kernel<true>, static_cast<unsigned>(2 * N * H), 0,
                                               kStepThreads, StepSmem<true>::kBytes, stream, a)
                    : launch_dependent_cluster(draft_step_kernel<false>, static_cast<unsigned>(2 * N * H), 0,
                                               kStepThreads, StepSmem<false>::kBytes, stream, a);
    return launch_dependent(bf16 ? draft_step_long_kernel<true> : draft_step_long_kernel<false>,
                            static_cast<unsigned>(N * H), kThreads, stream, a);
}

cudaError_t setup_draft_step_kernel() {
    cudaError_t e = cudaFuncSetAttribute(draft_step_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         StepSmem<true>::kBytes);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(draft_step_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                StepSmem<false>::kBytes);
}

}  // namespace sala

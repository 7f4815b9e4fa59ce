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
// Steps of up to 16 new and 16 pending tokens (draft_step_kernel): one persistent CTA per SM. An
// item of work is one (sequence, head, half of the value columns). Two producer warps stage items
// ahead of use in a ring of shared-memory stages (cp.async); each of the groups of 4 consumer warps
// takes every kGroups-th item. The two products with the state run on the tensor cores as
// mma.m16n8k16, 16 (or 8) being the tokens:
//     commit   D[16 dv x 8 dk] = (w V)^T K     with w_j v_j in fp32 split into three bf16 parts
//     read     O[16 t x 8 dv]  = Q S           with S in bf16
// The accumulators of the first are laid out like the B operand of the second, so one pass over the
// state in shared memory, 16 key rows at a time, feeds both. An fp32 state is read after the
// commit, split into two bf16 parts. A bf16 state is read as it was stored, an operand without any
// arithmetic, and what the commit adds to it enters as the pending tokens' own term (Q K^T w) V.
// A token that is not there (past the counts) is zero in shared memory; the products among the new
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
__device__ __forceinline__ Row read_row(const DraftArgs &a, int n, bool report) {
    Row r;
    r.slot = __ldg(a.slots + n);
    r.commits = a.T_pend ? static_cast<int64_t>(__ldg(a.accepted + n)) + 1 : 0;
    r.tokens = a.num_tokens ? __ldg(a.num_tokens + n) : a.T;
    if (r.commits < 0) r.commits = 0;
    const bool bad = r.slot >= a.P || r.commits > a.T_pend || r.tokens < 0 || r.tokens > a.T;
    if (bad && report) record_status(a.status, SALA_ERR_BAD_INDEX);
    if (bad || r.slot < 0) r.commits = r.tokens = 0;
    return r;
}

// ---- steps of up to 16 + 16 tokens ---------------------------------------------------------

constexpr int kHalf = kD / 2;         // value columns of an item
constexpr int kGroupThreads = 128;    // warp w: columns [32 (w % 2), + 32) of the half, key rows [64 (w / 2), + 64)
constexpr int kLoaders = 128;          // threads of the producer warps
constexpr uint64_t kWaitNs = 2000000000ull;   // limit of every wait

// Shared memory (offsets in bytes). Rows are cut into 16-byte chunks whose places are permuted by the
// row so that the 8 rows of a matrix fragment (and the 4 even or odd state rows that a quarter-warp
// reads) fall into different banks. kTok: tokens of an operand, 8 or 16.
struct Item {
    int32_t slot, n, h, half, commits, tokens, pad[2];
};
template <bool kBf16, int kTok>
struct StepSmem {
    // a stage
    static constexpr int kStateRow = kHalf * (kBf16 ? 2 : 4);
    static constexpr int kState = 0;
    static constexpr int kPk = kState + kD * kStateRow;      // [kTok][128] bf16
    static constexpr int kQ = kPk + kTok * kD * 2;
    static constexpr int kK = kQ + kTok * kD * 2;
    static constexpr int kPv = kK + kTok * kD * 2;           // [kTok][64] bf16
    static constexpr int kV = kPv + kTok * kHalf * 2;
    static constexpr int kPg = kV + kTok * kHalf * 2;        // [kTok] fp32
    static constexpr int kG = kPg + kTok * 4;
    static constexpr int kHead = kG + kTok * 4;              // struct Item
    static constexpr int kStage = (kHead + 32 + 255) / 256 * 256;
    // a group's own
    static constexpr int kScore = 0;                         // [kTok][kTok] fp32: q_t . k_j
    static constexpr int kPend = kScore + kTok * kTok * 4;   // [kTok][kTok] fp32: q_t . pk_j
    static constexpr int kDecay = kPend + kTok * kTok * 4;   // [kTok][kTok] fp32: exp(g_{j+1} + .. + g_t)
    static constexpr int kSwap = kDecay + kTok * kTok * 4;   // [4 warps][kTok / 2][32 lanes] fp32: halves of Q S
    static constexpr int kOwn = kSwap + 4 * kTok / 2 * 32 * 4;
    // groups as far as registers go, stages as far as memory goes
    static constexpr int kGroups = kBf16 ? 4 : 3;
    static constexpr int kStages = (232448 - 1024 - kGroups * kOwn) / kStage;
    static constexpr int kBytes = kStages * kStage + kGroups * kOwn;
    static constexpr int kThreads = kGroups * kGroupThreads + kLoaders;
    static_assert(kStages > kGroups, "the loads run ahead");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
// This thread's copies so far count as one arrival on `bar` once they have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void group_sync(int group) {
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(kGroupThreads) : "memory");
}
__device__ __forceinline__ bool group_any(int group, bool p) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"(static_cast<uint32_t>(p)), "r"(group + 1), "n"(kGroupThreads) : "memory");
    return r != 0;
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x2(uint32_t &r0, uint32_t &r1, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x2_trans(uint32_t &r0, uint32_t &r1, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr) : "memory");
}
// d += a b, m16n8k16, bf16 operands
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = c + a b over 16 or 8 tokens (a: 4 or 2 words, b: 2 words or the first)
template <int kTok>
__device__ __forceinline__ void mma_tok(float (&d)[4], const uint32_t *a, uint32_t b0, uint32_t b1, float c0, float c1,
                                        float c2, float c3) {
    if constexpr (kTok == 16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%10, %11, %12, %13};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, "
                     "{%7, %8, %9, %10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(b0), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ float4 lds_f32x4(uint32_t addr) {
    float4 x;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ void sts_f32x4(uint32_t addr, float x0, float x1, float x2, float x3) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(x0), "f"(x1), "f"(x2), "f"(x3) : "memory");
}
__device__ __forceinline__ uint2 lds_u32x2(uint32_t addr) {
    uint2 x;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ void sts_u32x2(uint32_t addr, uint32_t x0, uint32_t x1) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(x0), "r"(x1) : "memory");
}
__device__ __forceinline__ float2 lds_f32x2(uint32_t addr) {
    float2 x;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ void sts_f32x2(uint32_t addr, float x0, float x1) {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x0), "f"(x1) : "memory");
}
__device__ __forceinline__ void sts_f32(uint32_t addr, float x) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}

// Chunk c of row r: rows of 16 chunks (tokens' 128 keys), rows of 8 chunks (64 values in bf16).
__device__ __forceinline__ uint32_t chunk256(int r, int c) { return r * 256 + ((c ^ (r & 7)) << 4); }
__device__ __forceinline__ uint32_t chunk128(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }
// fp32 state half: rows of 16 chunks.
__device__ __forceinline__ uint32_t chunk_f32(int r, int c) { return r * 256 + ((c ^ (((r >> 1) & 3) << 1)) << 4); }

// kTok token rows of [tokens, H, 128] bf16 (kWide: all of a row, else 64 values), zeros past `count`.
template <int kTok, bool kWide>
__device__ __forceinline__ void stage_tokens(uint32_t dst, const uint16_t *src, int64_t row0, int H, int count, int lane) {
    constexpr int kChunks = kWide ? 16 : 8;
#pragma unroll
    for (int i = 0; i < (kTok * kChunks + kLoaders - 1) / kLoaders; ++i) {
        const int e = lane + i * kLoaders, t = e / kChunks, c = e % kChunks;
        if (kTok * kChunks % kLoaders && e >= kTok * kChunks) break;
        const bool ok = t < count;
        const uint16_t *p = src + (row0 + (ok ? static_cast<int64_t>(t) * H : 0)) * kD + 8 * c;
        cp_async16(dst + (kWide ? chunk256(t, c) : chunk128(t, c)), p, ok);
    }
}

// Lane t holds exp(g_1 + .. + g_t) (head) and exp(g_{t+1} + .. + g_count) (tail) of kTok gates, 0 past the count.
struct Gates {
    float g, head, tail;
};
template <int kTok>
__device__ __forceinline__ Gates gate_scan(const uint8_t *at, int count, int lane) {
    Gates s;
    s.g = lane < kTok ? reinterpret_cast<const float *>(at)[lane] : 0.f;   // zeros past the count
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

template <bool kBf16, int kTok>
__device__ __forceinline__ void stage_item(const DraftArgs &a, uint32_t st, const Item &it, int lane) {
    using Sm = StepSmem<kBf16, kTok>;
    const int64_t n = it.n;
    const int h = it.h, half = it.half, commits = it.commits, tokens = it.tokens;
    if (commits == 0 && tokens == 0) return;
    const int64_t at = (static_cast<int64_t>(it.slot) * a.H + h) * kD * kD + half * kHalf;
    constexpr int kChunks = Sm::kStateRow / 16;   // of a state row
#pragma unroll 8
    for (int i = 0; i < kD * kChunks / kLoaders; ++i) {
        const int e = lane + i * kLoaders, r = e / kChunks, c = e % kChunks;
        if constexpr (kBf16)
            cp_async16(st + Sm::kState + chunk128(r, c), static_cast<const uint16_t *>(a.pool) + at + r * kD + 8 * c, true);
        else
            cp_async16(st + Sm::kState + chunk_f32(r, c), static_cast<const float *>(a.pool) + at + r * kD + 4 * c, true);
    }
    const int64_t pend0 = n * a.T_pend * a.H + h, new0 = n * a.T * a.H + h;   // token rows of this head
    if (commits) {
        stage_tokens<kTok, true>(st + Sm::kPk, a.pk, pend0, a.H, commits, lane);
        stage_tokens<kTok, false>(st + Sm::kPv, a.pv + half * kHalf, pend0, a.H, commits, lane);
        if (lane < kTok)
            cp_async4(st + Sm::kPg + 4 * lane, a.pg + pend0 + (lane < commits ? static_cast<int64_t>(lane) * a.H : 0), lane < commits);
    }
    if (tokens) {
        stage_tokens<kTok, true>(st + Sm::kQ, a.q, new0, a.H, tokens, lane);
        stage_tokens<kTok, true>(st + Sm::kK, a.k, new0, a.H, tokens, lane);
        stage_tokens<kTok, false>(st + Sm::kV, a.v + half * kHalf, new0, a.H, tokens, lane);
        if (lane < kTok)
            cp_async4(st + Sm::kG + 4 * lane, a.g + new0 + (lane < tokens ? static_cast<int64_t>(lane) * a.H : 0), lane < tokens);
    }
}

// One item by a group of 4 warps, from its stage `smem` (address `st`); `own`: the group's memory.
template <bool kBf16, int kTok>
__device__ __forceinline__ void run_item(const DraftArgs &a, uint8_t *smem, uint32_t st, uint8_t *own, const Item &it, int group) {
    using Sm = StepSmem<kBf16, kTok>;
    constexpr int kParts = 3;   // of w_j v_j in fp32: what three bf16 parts leave out is below 2^-26 of it
    constexpr int kOct = kTok / 8;
    const int tid = threadIdx.x & (kGroupThreads - 1), warp = tid >> 5, lane = tid & 31;
    const int col = warp & 1, rows = warp >> 1;   // the warp's 32 columns and 64 key rows
    const int gr = lane >> 2, tq = lane & 3;      // row and column pair of a lane in a fragment
    const int mi = lane >> 3, mr = lane & 7;      // matrix and row whose address a lane gives
    const int commits = it.commits, tokens = it.tokens;
    const uint32_t own_at = tc::smem_u32(own);
    Gates pg{0.f, 0.f, 0.f}, ng{0.f, 0.f, 0.f};
    if (commits) pg = gate_scan<kTok>(smem + Sm::kPg, commits, lane);
    if (tokens) ng = gate_scan<kTok>(smem + Sm::kG, tokens, lane);

    // 1. products of the new tokens' queries with 8 keys at a time, one warp each: with the new tokens
    // (first warps), with the pending ones (next warps); decays by warp 3
    const bool pending = warp >= kOct;
    const int oct = pending ? warp - kOct : warp;
    if (tokens && oct < kOct && 8 * oct < (!pending ? tokens : kBf16 ? commits : 0)) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t keys = st + (pending ? Sm::kPk : Sm::kK);
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
            uint32_t qa[4], qb[4], kb[4];
            if constexpr (kTok == 16) {
                ldmatrix_x4(qa, st + Sm::kQ + chunk256(mr + 8 * (mi & 1), 2 * c + (mi >> 1)));
                ldmatrix_x4(qb, st + Sm::kQ + chunk256(mr + 8 * (mi & 1), 2 * c + 2 + (mi >> 1)));
            } else {
                uint32_t q4[4];
                ldmatrix_x4(q4, st + Sm::kQ + chunk256(mr, 2 * c + mi));
                qa[0] = q4[0], qa[2] = q4[1], qb[0] = q4[2], qb[2] = q4[3];
                qa[1] = qa[3] = qb[1] = qb[3] = 0u;
            }
            ldmatrix_x4(kb, keys + chunk256(mr + 8 * oct, 2 * c + mi));
            mma(d, qa, kb[0], kb[1]);
            mma(d, qb, kb[2], kb[3]);
        }
        const uint32_t s = own_at + (pending ? Sm::kPend : Sm::kScore) + (gr * kTok + 8 * oct + 2 * tq) * 4;
        sts_f32x2(s, d[0], d[1]);
        if constexpr (kTok == 16) sts_f32x2(s + 8 * kTok * 4, d[2], d[3]);
    }
    if (tokens && warp == 3) {
        float sum = 0.f;   // lane j: g_{j+1} + .. + g_t
        for (int t = 0; t < tokens; ++t) {
            const float g = __shfl_sync(0xffffffffu, ng.g, t);
            if (t > lane) sum += g;
            if (lane <= t) sts_f32(own_at + Sm::kDecay + (t * kTok + lane) * 4, expf(sum));
        }
    }

    // 2. the state, 16 key rows at a time. The 8 columns of an mma tile are every fourth one, so that
    // a lane's columns 4 gr .. 4 gr + 3 of the four tiles are neighbours: tile j holds column 4 gr + j
    // of lane row gr, and a state row of the lane is one 16-byte (fp32) or 8-byte (bf16) access.
    uint32_t wv[kParts][2][2 * kOct];   // (w V)^T: row gr is column 4 gr + 2 m, row gr + 8 column 4 gr + 2 m + 1
    const float fade = commits ? __shfl_sync(0xffffffffu, pg.head, commits - 1) : 1.f;
    // the lane's columns 4 gr .. + 3 of pending token t's values
    auto pend_values = [&](int t) {
        return lds_u32x2(st + Sm::kPv + chunk128(t, 4 * col + (gr >> 1)) + (gr & 1) * 8);
    };
    if (commits) {
#pragma unroll
        for (int i = 0; i < kOct; ++i) {   // tokens 2 tq + 8 i, + 1
            const int t = 2 * tq + 8 * i;
            const uint2 a0 = pend_values(t), a1 = pend_values(t + 1);
            const float w0 = __shfl_sync(0xffffffffu, pg.tail, t), w1 = __shfl_sync(0xffffffffu, pg.tail, t + 1);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float2 f0 = bf16x2_to_float2(m ? a0.y : a0.x), f1 = bf16x2_to_float2(m ? a1.y : a1.x);
                float x0 = w0 * f0.x, x1 = w1 * f1.x, y0 = w0 * f0.y, y1 = w1 * f1.y;
#pragma unroll
                for (int p = 0; p < kParts; ++p) {
                    wv[p][m][2 * i] = split_bf16(x0, x1);
                    wv[p][m][2 * i + 1] = split_bf16(y0, y1);
                }
            }
        }
    }
    float o[4][4] = {};   // tile j: rows gr, gr + 8; columns 8 tq + j, 8 tq + 4 + j
    // the lane's first state row (even) and the next one, and its rows of the token operands; 16 key
    // rows on, the places of the state repeat and those of the tokens differ by an exclusive or
    const uint32_t st0 = st + Sm::kState + (kBf16 ? chunk128(64 * rows + 2 * tq, 4 * col + (gr >> 1)) + (gr & 1) * 8
                                                  : chunk_f32(64 * rows + 2 * tq, 8 * col + gr));
    const uint32_t st1 = st + Sm::kState + (kBf16 ? chunk128(64 * rows + 2 * tq + 1, 4 * col + (gr >> 1)) + (gr & 1) * 8
                                                  : chunk_f32(64 * rows + 2 * tq + 1, 8 * col + gr));
    const uint32_t frag = kTok == 16 ? (mr + 8 * (mi & 1)) * 256 + (((mi >> 1) ^ mr) << 4)
                                     : mr * 256 + (((mi & 1) ^ mr) << 4);
#pragma unroll
    for (int ci = 0; ci < 4; ++ci) {
        const uint32_t tok_at = frag ^ ((4 * rows + ci) << 5);
        float x[2][2][4];      // rows 8 i + 2 tq + e, column j
        uint32_t hi[2][4];     // the same as B operands: rows 8 i + 2 tq, + 1 of column j
        [[maybe_unused]] uint32_t lo[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t at_row = (16 * ci + 8 * i) * Sm::kStateRow;
            if constexpr (kBf16) {
                const uint2 w0 = lds_u32x2(st0 + at_row), w1 = lds_u32x2(st1 + at_row);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint32_t u0 = m ? w0.y : w0.x, u1 = m ? w1.y : w1.x;
                    const float2 f0 = bf16x2_to_float2(u0), f1 = bf16x2_to_float2(u1);
                    x[i][0][2 * m] = f0.x, x[i][0][2 * m + 1] = f0.y;
                    x[i][1][2 * m] = f1.x, x[i][1][2 * m + 1] = f1.y;
                    hi[i][2 * m] = __byte_perm(u0, u1, 0x5410);
                    hi[i][2 * m + 1] = __byte_perm(u0, u1, 0x7632);
                }
            } else {
                const float4 f0 = lds_f32x4(st0 + at_row), f1 = lds_f32x4(st1 + at_row);
                x[i][0][0] = f0.x, x[i][0][1] = f0.y, x[i][0][2] = f0.z, x[i][0][3] = f0.w;
                x[i][1][0] = f1.x, x[i][1][1] = f1.y, x[i][1][2] = f1.z, x[i][1][3] = f1.w;
            }
        }
        if (commits) {
            uint32_t kb[2][2];   // K: [dk, dk + 8][tok, tok + 8]
            if constexpr (kTok == 16) {
                uint32_t k4[4];
                ldmatrix_x4_trans(k4, st + Sm::kPk + tok_at);
                kb[0][0] = k4[0], kb[0][1] = k4[1], kb[1][0] = k4[2], kb[1][1] = k4[3];
            } else {
                ldmatrix_x2_trans(kb[0][0], kb[1][0], st + Sm::kPk + tok_at);
                kb[0][1] = kb[1][1] = 0u;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    // summed apart from the state and added to it once: the state is rounded as in fp32
                    // arithmetic, whatever the tensor cores' accumulation does
                    float d[4];
                    mma_tok<kTok>(d, wv[kParts - 1][m], kb[i][0], kb[i][1], 0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int p = kParts - 2; p >= 0; --p)
                        mma_tok<kTok>(d, wv[p][m], kb[i][0], kb[i][1], d[0], d[1], d[2], d[3]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float &y = x[i][c & 1][2 * m + (c >> 1)];
                        y = fmaf(fade, y, d[c]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t at_row = (e ? st1 : st0) + (16 * ci + 8 * i) * Sm::kStateRow;
                    const float *y = x[i][e];
                    if constexpr (kBf16) sts_u32x2(at_row, float2_to_bf16x2(y[0], y[1]), float2_to_bf16x2(y[2], y[3]));
                    else sts_f32x4(at_row, y[0], y[1], y[2], y[3]);
                }
            }
        }
        if (tokens) {
            if constexpr (!kBf16) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float x0 = x[i][0][j], x1 = x[i][1][j];
                        hi[i][j] = split_bf16(x0, x1);
                        lo[i][j] = float2_to_bf16x2(x0, x1);
                    }
            }
            uint32_t qa[4];   // (t, dk), (t + 8, dk), (t, dk + 8), (t + 8, dk + 8)
            if constexpr (kTok == 16) {
                ldmatrix_x4(qa, st + Sm::kQ + tok_at);
            } else {
                ldmatrix_x2(qa[0], qa[2], st + Sm::kQ + tok_at);
                qa[1] = qa[3] = 0u;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (!kBf16) mma(o[j], qa, lo[0][j], lo[1][j]);
                mma(o[j], qa, hi[0][j], hi[1][j]);
            }
        }
    }
    // each warp finishes the first (rows = 0) or second four of a lane's 8 columns and hands the sums
    // of the others to the warp with the other key rows
    float *swap = reinterpret_cast<float *>(own + Sm::kSwap);
    if (tokens) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            swap[(warp * kTok / 2 + j) * 32 + lane] = rows ? o[j][0] : o[j][1];
            if constexpr (kTok == 16) swap[(warp * 8 + 4 + j) * 32 + lane] = rows ? o[j][2] : o[j][3];
        }
    }
    group_sync(group);

    // 3. the state goes back
    if (commits) {
        const int64_t at = (static_cast<int64_t>(it.slot) * a.H + it.h) * kD * kD + it.half * kHalf;
        constexpr int kChunks = Sm::kStateRow / 16;
#pragma unroll 8
        for (int i = 0; i < kD * kChunks / kGroupThreads; ++i) {
            const int e = tid + i * kGroupThreads, r = e / kChunks, c = e % kChunks;
            const uint4 w = *reinterpret_cast<const uint4 *>(smem + Sm::kState + (kBf16 ? chunk128(r, c) : chunk_f32(r, c)));
            if constexpr (kBf16)
                __stcs(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.pool) + at + r * kD + 8 * c), w);
            else
                __stcs(reinterpret_cast<uint4 *>(static_cast<float *>(a.pool) + at + r * kD + 4 * c), w);
        }
    }

    // 4. o_t = scale ( head_t (Q S)_t + sum_{j <= t} decay_tj score_tj v_j ), rows gr, gr + 8; bf16: with
    // fade (Q S)_t + sum_j w_j (q_t . pk_j) pv_j in place of (Q S)_t
    if (tokens) {
        const float *score = reinterpret_cast<const float *>(own + Sm::kScore);
        const float *decay = reinterpret_cast<const float *>(own + Sm::kDecay);
        const float h0 = __shfl_sync(0xffffffffu, ng.head, gr), h1 = __shfl_sync(0xffffffffu, ng.head, gr + 8);
        const int first = 32 * col + 8 * tq + 4 * rows;   // the lane's 4 columns
        float y0[4], y1[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y0[j] = (kBf16 ? fade : 1.f) * ((rows ? o[j][1] : o[j][0]) + swap[((warp ^ 2) * kTok / 2 + j) * 32 + lane]);
            if constexpr (kTok == 16) y1[j] = (kBf16 ? fade : 1.f) * ((rows ? o[j][3] : o[j][2]) + swap[((warp ^ 2) * 8 + 4 + j) * 32 + lane]);
        }
        if (kBf16 && commits) {
            const uint32_t pend = own_at + Sm::kPend + (gr * kTok + 2 * tq) * 4;
            uint32_t pa[2][2 * kOct];   // w_j (q_t . pk_j) in two bf16 parts
            uint32_t bv[4][2];          // pv: column 4 gr + j of tokens 2 tq, + 1, + 8, + 9
#pragma unroll
            for (int i = 0; i < kOct; ++i) {
                const int t = 2 * tq + 8 * i;
                const float w0 = __shfl_sync(0xffffffffu, pg.tail, t), w1 = __shfl_sync(0xffffffffu, pg.tail, t + 1);
                float2 s0 = lds_f32x2(pend + 32 * i), s1 = lds_f32x2(pend + 32 * i + (kTok == 16 ? 8 * kTok * 4 : 0));
                if (kTok == 8) s1 = make_float2(0.f, 0.f);
                if (8 * i >= commits) s0 = s1 = make_float2(0.f, 0.f);   // was not computed
                s0.x *= w0, s0.y *= w1, s1.x *= w0, s1.y *= w1;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    pa[p][2 * i] = split_bf16(s0.x, s0.y);
                    pa[p][2 * i + 1] = split_bf16(s1.x, s1.y);
                }
                const uint2 a0 = pend_values(t), a1 = pend_values(t + 1);
                bv[0][i] = __byte_perm(a0.x, a1.x, 0x5410);
                bv[1][i] = __byte_perm(a0.x, a1.x, 0x7632);
                bv[2][i] = __byte_perm(a0.y, a1.y, 0x5410);
                bv[3][i] = __byte_perm(a0.y, a1.y, 0x7632);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float d[4];
                mma_tok<kTok>(d, pa[1], bv[j][0], bv[j][kOct - 1], 0.f, 0.f, 0.f, 0.f);
                mma_tok<kTok>(d, pa[0], bv[j][0], bv[j][kOct - 1], d[0], d[1], d[2], d[3]);
                y0[j] += rows ? d[1] : d[0];
                if constexpr (kTok == 16) y1[j] += rows ? d[3] : d[2];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y0[j] *= h0;
            if constexpr (kTok == 16) y1[j] *= h1;
        }
        for (int j = 0; j < tokens; ++j) {
            const uint2 w = lds_u32x2(st + Sm::kV + chunk128(j, first / 8) + rows * 8);
            const float2 v0 = bf16x2_to_float2(w.x), v1 = bf16x2_to_float2(w.y);
            if (j <= gr) {
                const float s = score[gr * kTok + j] * decay[gr * kTok + j];
                y0[0] = fmaf(s, v0.x, y0[0]);
                y0[1] = fmaf(s, v0.y, y0[1]);
                y0[2] = fmaf(s, v1.x, y0[2]);
                y0[3] = fmaf(s, v1.y, y0[3]);
            }
            if constexpr (kTok == 16) {
                if (j <= gr + 8) {
                    const float s = score[(gr + 8) * kTok + j] * decay[(gr + 8) * kTok + j];
                    y1[0] = fmaf(s, v0.x, y1[0]);
                    y1[1] = fmaf(s, v0.y, y1[1]);
                    y1[2] = fmaf(s, v1.x, y1[2]);
                    y1[3] = fmaf(s, v1.y, y1[3]);
                }
            }
        }
        uint16_t *out = a.o + ((it.n * a.T + gr) * a.H + it.h) * kD + it.half * kHalf + first;
        if (gr < tokens)
            *reinterpret_cast<uint2 *>(out) = make_uint2(float2_to_bf16x2(a.scale * y0[0], a.scale * y0[1]),
                                                         float2_to_bf16x2(a.scale * y0[2], a.scale * y0[3]));
        if constexpr (kTok == 16) {
            if (gr + 8 < tokens)
                *reinterpret_cast<uint2 *>(out + static_cast<int64_t>(8) * a.H * kD) =
                    make_uint2(float2_to_bf16x2(a.scale * y1[0], a.scale * y1[1]),
                               float2_to_bf16x2(a.scale * y1[2], a.scale * y1[3]));
        }
    }
}

template <bool kBf16, int kTok>
__global__ void __launch_bounds__(StepSmem<kBf16, kTok>::kThreads, 1) draft_step_kernel(DraftArgs a, unsigned items) {
    using Sm = StepSmem<kBf16, kTok>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t full[Sm::kStages], empty[Sm::kStages];
    if (threadIdx.x == 0) {
        for (int s = 0; s < Sm::kStages; ++s) {
            tc::mbar_init(&full[s], kLoaders + 1);
            tc::mbar_init(&empty[s], kGroupThreads / 32);
        }
        tc::fence_barrier_init();
    }
    __syncthreads();
    dependent_start();

    // item i: unit i / 2 (n * H + h), column half i % 2; this CTA's k-th goes through stage k % kStages
    const unsigned step = gridDim.x;
    if (threadIdx.x >= Sm::kGroups * kGroupThreads) {
        const int lane = threadIdx.x - Sm::kGroups * kGroupThreads;
        int stage = 0;
        uint32_t parity = 1;   // of the wait for an empty stage: the first round passes at once
        auto read = [&](unsigned item) {
            Item it{};
            if (item < items) {
                const unsigned unit = item >> 1, n = unit / static_cast<unsigned>(a.H);
                const Row row = read_row(a, static_cast<int>(n), lane == 0);
                it = {row.slot, static_cast<int32_t>(n), static_cast<int32_t>(unit - n * a.H), static_cast<int32_t>(item & 1),
                      static_cast<int32_t>(row.commits), static_cast<int32_t>(row.tokens), {0, 0}};
            }
            return it;
        };
        Item next = read(blockIdx.x);
        for (unsigned item = blockIdx.x; item < items; item += step) {
            const Item it = next;
            next = read(item + step);   // its latency hides behind this item's copies
            if (!tc::mbar_wait(&empty[stage], parity, kWaitNs)) {
                record_status(a.status, SALA_ERR_TIMEOUT);
                break;
            }
            uint8_t *at = smem + stage * Sm::kStage;
            stage_item<kBf16, kTok>(a, tc::smem_u32(at), it, lane);
            if (lane == 0) {
                *reinterpret_cast<Item *>(at + Sm::kHead) = it;
                tc::mbar_arrive(&full[stage]);
            }
            cp_async_arrive(&full[stage]);
            if (++stage == Sm::kStages) stage = 0, parity ^= 1;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");   // none of this thread's copies outlives it
        return;
    }

    const int group = threadIdx.x / kGroupThreads, tid = threadIdx.x & (kGroupThreads - 1);
    uint8_t *own = smem + Sm::kStages * Sm::kStage + group * Sm::kOwn;
    int stage = group;
    uint32_t parity = 0;
    for (unsigned item = blockIdx.x + group * step; item < items; item += Sm::kGroups * step) {
        const bool late = !tc::mbar_wait(&full[stage], parity, kWaitNs);
        if (late) record_status(a.status, SALA_ERR_TIMEOUT);
        // also: the group's memory of the item before is free
        if (group_any(group, late)) break;
        uint8_t *at = smem + stage * Sm::kStage;
        const Item it = *reinterpret_cast<const Item *>(at + Sm::kHead);
        for (int e = it.tokens * 8 + tid; e < static_cast<int>(a.T) * 8; e += kGroupThreads)   // rows past the count
            *reinterpret_cast<uint4 *>(a.o + ((it.n * a.T + e / 8) * a.H + it.h) * kD + it.half * kHalf + 8 * (e % 8)) =
                make_uint4(0, 0, 0, 0);
        if (it.commits || it.tokens) run_item<kBf16, kTok>(a, at, tc::smem_u32(at), own, it, group);
        __syncwarp();
        if ((tid & 31) == 0) tc::mbar_arrive(&empty[stage]);
        stage += Sm::kGroups;
        if (stage >= Sm::kStages) stage -= Sm::kStages, parity ^= 1;
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
    const Row row = read_row(a, n, threadIdx.x == 0);
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
                              int64_t T, int64_t T_pend, int H, int sm_count, int *status, cudaStream_t stream) {
    LaunchTimer timer(kKDraftStep, stream);
    const DraftArgs a{static_cast<const uint16_t *>(q), static_cast<const uint16_t *>(k),
                      static_cast<const uint16_t *>(v), g, num_tokens,
                      static_cast<const uint16_t *>(pend_k), static_cast<const uint16_t *>(pend_v),
                      pend_g, accepted, scale, pool, slots, P, static_cast<uint16_t *>(o), T, T_pend, H,
                      status};
    if (T <= 16 && T_pend <= 16) {
        const unsigned items = static_cast<unsigned>(2 * N * H);
        const unsigned grid = items < static_cast<unsigned>(sm_count) ? items : sm_count;
        const bool few = T <= 8 && T_pend <= 8;
        if (bf16)
            return few ? launch_dependent_cluster(draft_step_kernel<true, 8>, grid, 0, StepSmem<true, 8>::kThreads,
                                                  StepSmem<true, 8>::kBytes, stream, a, items)
                       : launch_dependent_cluster(draft_step_kernel<true, 16>, grid, 0, StepSmem<true, 16>::kThreads,
                                                  StepSmem<true, 16>::kBytes, stream, a, items);
        return few ? launch_dependent_cluster(draft_step_kernel<false, 8>, grid, 0, StepSmem<false, 8>::kThreads,
                                              StepSmem<false, 8>::kBytes, stream, a, items)
                   : launch_dependent_cluster(draft_step_kernel<false, 16>, grid, 0, StepSmem<false, 16>::kThreads,
                                              StepSmem<false, 16>::kBytes, stream, a, items);
    }
    return launch_dependent(bf16 ? draft_step_long_kernel<true> : draft_step_long_kernel<false>,
                            static_cast<unsigned>(N * H), kThreads, stream, a);
}

namespace {
template <bool kBf16, int kTok>
cudaError_t allow_smem() {
    return cudaFuncSetAttribute(draft_step_kernel<kBf16, kTok>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                StepSmem<kBf16, kTok>::kBytes);
}
}  // namespace

cudaError_t setup_draft_step_kernel() {
    cudaError_t e = allow_smem<true, 8>();
    if (e == cudaSuccess) e = allow_smem<true, 16>();
    if (e == cudaSuccess) e = allow_smem<false, 8>();
    if (e == cudaSuccess) e = allow_smem<false, 16>();
    return e;
}

}  // namespace sala

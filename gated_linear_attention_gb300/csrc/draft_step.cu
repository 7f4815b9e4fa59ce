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
// ahead of use in a ring of shared-memory stages (TMA); each of the groups of 4 consumer warps takes
// every kGroups-th item and sends the state back from its stage (TMA). The two products with the
// state run on the tensor cores as mma.m16n8k16, 16 (or 8) being the tokens, which are too few for
// the rows of a tcgen05 tile:
//     commit   D[16 dv x 8 dk] = (w V)^T K
//     read     O[16 t x 8 dv]  = Q S
// The accumulators of the first are laid out like the B operand of the second, so one pass over the
// state in shared memory, 16 key rows at a time, feeds both. Operands that are fp32 (w_j v_j, the state, the
// tokens' weights) go in three bf16 parts that sum to them, so every product is exact and the sums are
// fp32 (with two parts of the state and the weights, 17 of 24 bits, o had three times as many elements on
// the wrong side of a bf16 rounding; 256 rows of 5, fp32, took 181 us and not 177, 201 ragged bf16 rows 111 and
// not 113, 256 fp32 rows of 17 328 and not 366). An fp32 state is read after the
// commit. A bf16 state is read as it was stored, an operand without any
// arithmetic, and what the commit adds to it enters as the pending tokens' own term (Q K^T w) V.
// Infinities and NaN: a commit that has them is taken one product at a time (commit_by_one), so that the stored
// state has the recurrence's; o is infinite or NaN where the recurrence's is.
// Places past the counts hold anything: pending tokens there are masked out of every operand, and the
// products among the new tokens go one by one where a value is not finite, so nothing of a masked place
// reaches a result.
// Longer steps (draft_step_long_kernel) take 16 tokens at a time over a state held in shared memory.
//
// Bound by the memory with fp32 states: 256 rows of 5 tokens, 32 heads, 177 us, 6.4 TB/s of what has to
// move; 16 tokens, 192 us (floor 184). With bf16 states the same tokens come with half the bytes and the
// shared-memory accesses and arithmetic of a step show: 5 tokens 112 us (floor 87), 16 tokens 146 us
// (floor 104), 201 ragged rows of up to 16 116 us (floor 76).
#include <type_traits>

#include "chunk_tc.cuh"

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
    if (bad && r.slot >= 0 && report) record_status(a.status, SALA_ERR_BAD_INDEX);   // (a padding row's counts are anything)
    if (bad || r.slot < 0) r.commits = r.tokens = 0;
    return r;
}

// ---- steps of up to 16 + 16 tokens ---------------------------------------------------------

constexpr int kHalf = kD / 2;         // value columns of an item
constexpr int kGroupThreads = 128;    // warp w: columns [32 (w % 2), + 32) of the half, key rows [64 (w / 2), + 64)
constexpr int kOctBytes = 8 * 128;     // 8 tokens x 64 columns: a copy takes 8 tokens, of both halves of the columns or of one

struct Item {
    int32_t slot, n, h, half, commits, tokens, pad[2];
};

// Shared memory (offsets in bytes). Every tile has rows of 128 bytes as TMA lays them out with 128-byte
// swizzle: the 16-byte chunk c of row r is at place c ^ (r % 8), so that the 8 rows of a matrix
// fragment, and the even or odd state rows that a quarter-warp reads, fall into different banks.
// kTok: tokens of an operand, 8 or 16.
template <bool kBf16, int kTok>
struct StepSmem {
    // a stage
    static constexpr int kBoxCols = kBf16 ? 64 : 32;         // state columns of a tile
    static constexpr int kBoxes = kHalf / kBoxCols;
    static constexpr int kStateTile = kD * 128;
    static constexpr int kState = 0;
    static constexpr int kPk = kState + kBoxes * kStateTile; // keys and queries: [kTok / 8][8 tokens][2 halves][64]
    static constexpr int kQ = kPk + kTok / 8 * 2 * kOctBytes;
    static constexpr int kK = kQ + kTok / 8 * 2 * kOctBytes;
    static constexpr int kPv = kK + kTok / 8 * 2 * kOctBytes;   // values of the item's half: [kTok][64]
    static constexpr int kV = kPv + kTok / 8 * kOctBytes;
    static constexpr int kStage = kV + kTok / 8 * kOctBytes;
    static_assert(kStage % 1024 == 0, "tiles begin with their swizzle");
    // beside each stage
    static constexpr int kPg = 0;                            // [kTok] fp32
    static constexpr int kG = kPg + kTok * 4;
    static constexpr int kHead = kG + kTok * 4;              // struct Item
    static constexpr int kSide = kHead + 32;
    // a group's own
    static constexpr int kPitch = kTok + 4;                  // of rows t, so that 8 of them fill the banks
    static constexpr int kRect = kTok * kPitch * 4;          // [t][j] fp32
    static constexpr int kScore = 0;                         // q_t . k_j, over either half of the keys' columns
    static constexpr int kPend = kScore + 2 * kRect;         // q_t . pk_j, the same (bf16 states)
    static constexpr int kDecay = kPend + (kBf16 ? 2 : 0) * kRect;   // exp(g_{j+1} + .. + g_t)
    static constexpr int kOwn = kDecay + kRect;
    // halves of Q S, [4 warps][kTok / 2][32 lanes] fp32, in the place of the queries once they are read
    static constexpr int kSwap = kQ;
    static_assert(4 * kTok / 2 * 32 * 4 <= kK - kQ, "the halves fit");
    // Groups: three keep the memory busy with fp32 states; four with bf16 states and 8 tokens (16 rows of 5
    // tokens 10.0 us, with three 10.2; 64 rows 31.4 and 31.7; 256 rows, all memory, 111.8 and 110.2); with 16
    // tokens the registers of four do not suffice (201 ragged rows: 116 us with three, 120 with four). Stages as
    // far as memory goes.
    static constexpr int kGroups = kBf16 && kTok == 8 ? 4 : 3;
    // (fp32: 4 stages of 33 KB states; with 5 the loads run so far ahead of the stores that the memory
    // serves both more slowly, 256 rows of 5 tokens in 189 us instead of 177)
    static constexpr int kFit = (232448 - 1024 - kGroups * kOwn) / (kStage + kSide);
    static constexpr int kStages = !kBf16 && kFit > 4 ? 4 : kFit;
    // "Full" barriers: a multiple of the groups, so that a barrier's phases are all one group's. Were they
    // as many as the stages, the phases of one would go round the groups, and a group could ask for phase
    // p + 1 before phase p of another group had come, which the parity cannot tell from its end.
    static constexpr int kFulls = (kStages + kGroups - 1) / kGroups * kGroups;
    static constexpr int kSides = kStages * kStage;
    static constexpr int kOwns = kSides + kStages * kSide;
    static constexpr int kBytes = kOwns + kGroups * kOwn;
    static constexpr int kThreads = kGroups * kGroupThreads + 64;   // and two producer warps
    static_assert(kStages > kGroups, "the loads run ahead");
};

// The rings of the four variants, as the tests model them on the host: stages, groups, full barriers.
template <typename Sm>
constexpr bool ring_is(int stages, int groups, int fulls) {
    return Sm::kStages == stages && Sm::kGroups == groups && Sm::kFulls == fulls;
}
static_assert(ring_is<StepSmem<false, 8>>(4, 3, 6));
static_assert(ring_is<StepSmem<false, 16>>(4, 3, 6));
static_assert(ring_is<StepSmem<true, 8>>(9, 4, 12));
static_assert(ring_is<StepSmem<true, 16>>(6, 3, 6));

// pool [P * H, 128, 128]: boxes of one state's 128 rows x 128 bytes; tokens [N, T, H, 2, 64]: boxes of
// 8 tokens of one head (zeros past T), all columns of keys and queries, half of them of values. (A
// copy costs its issuing warp about 90 ns whatever its size: boxes of 4 tokens x 64 columns bounded
// 256 bf16 rows of 5 tokens by their number, at 159 us.)
struct StepMaps {
    CUtensorMap pool, pk, pv, q, k, v;
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// This thread's copies so far count as one arrival on `bar` once they have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, int32_t c0, int32_t c1, int32_t c2,
                                            int32_t c3, int32_t c4, uint64_t *bar) {
    asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1),
                 "r"(c2), "r"(c3), "r"(c4), "r"(tc::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void group_sync(int group) {
    __syncwarp();
    tck::named_sync(group + 9, kGroupThreads);
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

// Chunk c of row r of a tile.
__device__ __forceinline__ uint32_t chunk(int r, int c) { return tck::sw(r, c); }
// Chunk c of column half `half` of token t's keys or queries. (Token rows are two rows apart, so the 8
// rows of a fragment meet in pairs in the banks; that is a tenth of an item's shared-memory reads.)
__device__ __forceinline__ uint32_t wide_chunk(int t, int half, int c) {
    return (t >> 3) * 2 * kOctBytes + tck::sw(2 * (t & 7) + half, c);
}

// Lane t holds exp(g_1 + .. + g_t) (head) and exp(g_{t+1} + .. + g_count) (tail) of kTok gates, 0 past the count.
struct Gates {
    float g, head, tail;
};
template <int kTok>
__device__ __forceinline__ Gates gate_scan(const uint8_t *at, int count, int lane) {
    Gates s;
    s.g = lane < kTok && lane < count ? reinterpret_cast<const float *>(at)[lane] : 0.f;
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

// Products of fp32 values on the tensor cores: a value is the sum of three bf16 parts, 8 of its 24 bits each.
constexpr int kParts = 3;
// The next part of x0 and of x1, a packed pair (x0 in the low half), and what it leaves of them. The bits
// are cut, not rounded, so no part is larger than the value.
__device__ __forceinline__ uint32_t split_bf16(float &x0, float &x1) {
    const uint32_t u0 = __float_as_uint(x0), u1 = __float_as_uint(x1);
    x0 -= __uint_as_float(u0 & 0xffff0000u);
    x1 -= __uint_as_float(u1 & 0xffff0000u);
    return __byte_perm(u0, u1, 0x7632);
}

// Wait for a phase of `bar`, at most tck::kWaitNs, asleep in the barrier between tries.
__device__ __forceinline__ bool ring_wait(uint64_t *bar, uint32_t parity) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = tc::global_timer_ns();
    while (!tc::mbar_try_wait_sleep(bar, parity, 20000))
        if (tc::global_timer_ns() - t0 > tck::kWaitNs) return false;
    return true;
}

// An item's copies into its stage, by two warps: the state and the item itself, and the tokens. The
// barrier takes one arrival from each with the bytes of its tiles, and one from every lane of the
// second for the gates, which are too narrow for the copy engine.
template <bool kBf16, int kTok>
__device__ __forceinline__ void stage_state(const DraftArgs &a, const StepMaps &maps, uint8_t *smem, uint8_t *side, const Item &it,
                                            uint64_t *bar, int lane) {
    using Sm = StepSmem<kBf16, kTok>;
    if (lane != 0) return;
    const int states = it.commits || it.tokens ? Sm::kBoxes : 0;
    *reinterpret_cast<Item *>(side + Sm::kHead) = it;
    tc::mbar_arrive_expect_tx(bar, states * Sm::kStateTile);
    for (int b = 0; b < states; ++b)
        tc::tma_load_3d(smem + Sm::kState + b * Sm::kStateTile, &maps.pool, it.half * kHalf + b * Sm::kBoxCols, 0,
                        static_cast<int32_t>(static_cast<int64_t>(it.slot) * a.H + it.h), bar);
}
template <bool kBf16, int kTok>
__device__ __forceinline__ void stage_tokens(const DraftArgs &a, const StepMaps &maps, uint8_t *smem, uint8_t *side, const Item &it,
                                             uint64_t *bar, int lane) {
    using Sm = StepSmem<kBf16, kTok>;
    const int commits = it.commits, tokens = it.tokens;
    if (lane == 0) {
        const uint32_t at = tc::smem_u32(smem);
        tc::mbar_arrive_expect_tx(bar, (3 * ((commits + 7) / 8) + 5 * ((tokens + 7) / 8)) * kOctBytes);
#pragma unroll
        for (int oct = 0; oct < kTok / 8; ++oct) {
            if (8 * oct < commits) {
                tma_load_5d(at + Sm::kPk + oct * 2 * kOctBytes, &maps.pk, 0, 0, it.h, 8 * oct, it.n, bar);
                tma_load_5d(at + Sm::kPv + oct * kOctBytes, &maps.pv, 0, it.half, it.h, 8 * oct, it.n, bar);
            }
            if (8 * oct < tokens) {
                tma_load_5d(at + Sm::kQ + oct * 2 * kOctBytes, &maps.q, 0, 0, it.h, 8 * oct, it.n, bar);
                tma_load_5d(at + Sm::kK + oct * 2 * kOctBytes, &maps.k, 0, 0, it.h, 8 * oct, it.n, bar);
                tma_load_5d(at + Sm::kV + oct * kOctBytes, &maps.v, 0, it.half, it.h, 8 * oct, it.n, bar);
            }
        }
    }
    __syncwarp();
    const int64_t pend0 = it.n * a.T_pend * a.H + it.h, new0 = it.n * a.T * a.H + it.h;   // token rows of this head
    if (lane < commits) cp_async4(tc::smem_u32(side + Sm::kPg) + 4 * lane, a.pg + pend0 + static_cast<int64_t>(lane) * a.H);
    if (lane < tokens) cp_async4(tc::smem_u32(side + Sm::kG) + 4 * lane, a.g + new0 + static_cast<int64_t>(lane) * a.H);
    cp_async_arrive(bar);
}

// Two neighbouring weights of a row as word i of an A operand in parts.
template <int kWords>
__device__ __forceinline__ void split_row(uint32_t (&pa)[kParts][kWords], int i, float2 w) {
#pragma unroll
    for (int p = 0; p < kParts; ++p) pa[p][i] = split_bf16(w.x, w.y);
}
// Four columns of two neighbouring tokens' values as words i of four B operands.
template <int kWords>
__device__ __forceinline__ void pack_values(uint32_t (&bv)[4][kWords], int i, uint2 a0, uint2 a1, uint32_t mask) {
    bv[0][i] = __byte_perm(a0.x, a1.x, 0x5410) & mask;
    bv[1][i] = __byte_perm(a0.x, a1.x, 0x7632) & mask;
    bv[2][i] = __byte_perm(a0.y, a1.y, 0x5410) & mask;
    bv[3][i] = __byte_perm(a0.y, a1.y, 0x7632) & mask;
}
// Nonzero if either bf16 of the pair is an infinity or NaN: its exponent, all ones, carries.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    return (((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u);
}

// x + 0 w for a pair of bf16: a mark of NaN where one of them is an infinity or NaN.
__device__ __forceinline__ void mark_not_finite(uint32_t &x, uint32_t w) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(x) : "r"(w), "r"(0u));
}

// Columns 4 c .. 4 c + 3 of row r of a state half that begins at element `at` of the pool.
template <bool kBf16>
__device__ __forceinline__ void store_state(void *pool, int64_t at, int r, int c, float4 x) {
    if constexpr (kBf16)
        __stcs(reinterpret_cast<uint2 *>(static_cast<uint16_t *>(pool) + at + r * kD) + c,
               make_uint2(float2_to_bf16x2(x.x, x.y), float2_to_bf16x2(x.z, x.w)));
    else
        __stcs(reinterpret_cast<float4 *>(static_cast<float *>(pool) + at + r * kD) + c, x);
}

// A thread's part of the commit of an item (as they are numbered in the kernels) where infinities or NaN are
// committed, whose parts do not sum to them: the recurrence as it stands, in fp32, from the pool to the pool.
// Every eighth row from `row` to `end` (of whole fours), columns 4 c .. 4 c + 3 of the item's half with
// c = thread % 16. Bound by the latency of a token's loads, which four rows share: one broken row among 256 of 16
// makes an fp32 step 219 us instead of 196 (250 with a row at a time), a bf16 step 167 instead of 150.
template <bool kBf16>
__device__ __forceinline__ void commit_by_one(const DraftArgs &a, unsigned item, int row, int end) {
    const unsigned unit = item >> 1, n = unit / static_cast<unsigned>(a.H), h = unit - n * a.H, half = item & 1;
    const int c = threadIdx.x & 15;
    const Row what = read_row(a, static_cast<int>(n), false);
    const int64_t at = (static_cast<int64_t>(what.slot) * a.H + h) * kD * kD + half * kHalf, pend0 = n * a.T_pend * a.H + h;
    const uint16_t *k = a.pk + pend0 * kD, *v = a.pv + pend0 * kD + half * kHalf;
    const float *g = a.pg + pend0;
    void *pool = a.pool;
    constexpr int kAtOnce = 4;   // rows that share a token's loads
#pragma unroll 1
    for (int r = row; r < end; r += 8 * kAtOnce) {
        float4 x[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            if constexpr (kBf16) {
                const uint2 w = *(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(pool) + at + (r + 8 * i) * kD) + c);
                const float2 f0 = bf16x2_to_float2(w.x), f1 = bf16x2_to_float2(w.y);
                x[i] = make_float4(f0.x, f0.y, f1.x, f1.y);
            } else {
                x[i] = *(reinterpret_cast<const float4 *>(static_cast<const float *>(pool) + at + (r + 8 * i) * kD) + c);
            }
        }
#pragma unroll 1
        for (int64_t t = 0; t < what.commits; ++t) {
            const float fade = expf(__ldg(g + t * a.H));
            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(v + t * a.H * kD) + c);
            const float2 f0 = bf16x2_to_float2(w.x), f1 = bf16x2_to_float2(w.y);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const float key = bf16_bits_to_float(__ldg(k + t * a.H * kD + r + 8 * i));
                x[i] = make_float4(fmaf(fade, x[i].x, key * f0.x), fmaf(fade, x[i].y, key * f0.y), fmaf(fade, x[i].z, key * f1.x),
                                   fmaf(fade, x[i].w, key * f1.y));
            }
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) store_state<kBf16>(pool, at, r + 8 * i, c, x[i]);
    }
}

// One item by a group of 4 warps, from its stage `smem` and what stands beside it; `own`: the group's
// memory. Thread 0 of the group leaves a store of the state in flight that still reads the stage.
// kC, kT: there is something to commit, there are new tokens; kStore: what was committed goes to `pool`
// from here (else it stays in the stage). t0: place of the first new token in its row. Returns, to the whole
// group, whether the commit has infinities or NaN (kStore): it is then not sent, NaN stand for both in it.
template <bool kBf16, int kTok, bool kC, bool kT, bool kStore = kC>
__device__ __forceinline__ bool run_item(const DraftArgs &a, const CUtensorMap *pool, uint8_t *smem, const uint8_t *side,
                                         uint8_t *own, const Item &it, int group, int64_t t0 = 0) {
    using Sm = StepSmem<kBf16, kTok>;
    constexpr int kOct = kTok / 8;
    const int tid = threadIdx.x & (kGroupThreads - 1), warp = tid >> 5, lane = tid & 31;
    const int col = warp & 1, rows = warp >> 1;   // the warp's 32 columns and 64 key rows
    const int gr = lane >> 2, tq = lane & 3;      // row and column pair of a lane in a fragment
    const int mi = lane >> 3, mr = lane & 7;      // matrix and row whose address a lane gives
    const int commits = it.commits, tokens = it.tokens;
    const uint32_t st = tc::smem_u32(smem), own_at = tc::smem_u32(own);
    Gates pg{0.f, 0.f, 0.f}, ng{0.f, 0.f, 0.f};
    if (kC) pg = gate_scan<kTok>(side + Sm::kPg, commits, lane);
    if (kT) ng = gate_scan<kTok>(side + Sm::kG, tokens, lane);

    // 1. decays
    if (kT) {
        // decays of rows t = kOct * 2 * warp + r, lanes j and j + 16 taking turns; sums of g_{j+1} .. g_t
        constexpr int kRows = kTok / 4;
        const int j = lane & 15, turn = lane >> 4;
        float sum = 0.f;
        for (int i = 1; i < kRows * warp; ++i) {
            const float g = __shfl_sync(0xffffffffu, ng.g, i);
            if (i > j) sum += g;
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int t = kRows * warp + r;
            const float g = __shfl_sync(0xffffffffu, ng.g, t);
            if (t > j) sum += g;
            if ((r & 1) == turn && j <= t) sts_f32(own_at + Sm::kDecay + (t * Sm::kPitch + j) * 4, expf(sum));
        }
    }

    // 2. the state, 16 key rows at a time, and on the way the products of queries and keys over those 16
    // columns: with the new keys in the warps of the first 32 values, with the pending ones in the
    // others. The 8 columns of an mma tile are every fourth one, so that
    // a lane's columns 4 gr .. 4 gr + 3 of the four tiles are neighbours: tile j holds column 4 gr + j
    // of lane row gr, and a state row of the lane is one 16-byte (fp32) or 8-byte (bf16) access.
    uint32_t wv[kParts][2][2 * kOct];   // (w V)^T: row gr is column 4 gr + 2 m, row gr + 8 column 4 gr + 2 m + 1
    const float fade = kC ? __shfl_sync(0xffffffffu, pg.head, commits - 1) : 1.f;
    // columns 4 gr .. + 3 of the warp's 32 of token t's values
    auto values = [&](uint32_t tile, int t) { return lds_u32x2(st + tile + chunk(t, 4 * col + (gr >> 1)) + (gr & 1) * 8); };
    uint32_t there[kOct];   // mask of the pending tokens 2 tq + 8 i, + 1 of a packed pair
    // infinities and NaN to commit show in the sums where an fp32 state is read next; else the operands are marked
    constexpr bool kMark = kStore && (kBf16 || !kT);
    [[maybe_unused]] uint32_t mark = 0;
    if (kC) {
#pragma unroll
        for (int i = 0; i < kOct; ++i) {   // tokens 2 tq + 8 i, + 1
            const int t = 2 * tq + 8 * i;
            uint2 a0 = values(Sm::kPv, t), a1 = values(Sm::kPv, t + 1);
            if (t >= commits) a0 = make_uint2(0u, 0u);
            if (t + 1 >= commits) a1 = make_uint2(0u, 0u);
            there[i] = (t < commits ? 0xffffu : 0u) | (t + 1 < commits ? 0xffff0000u : 0u);
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
                if constexpr (kMark) {
                    mark_not_finite(mark, wv[0][m][2 * i]);
                    mark_not_finite(mark, wv[0][m][2 * i + 1]);
                }
            }
        }
    }
    float o[4][4] = {};   // tile j: rows gr, gr + 8; columns 8 tq + j, 8 tq + 4 + j
    // the lane's first state row (even) and the next one, and its rows of the token operands; 16 key
    // rows on, the places of the state repeat and those of the tokens differ by an exclusive or
    const uint32_t tile = st + Sm::kState + (kBf16 ? 0 : col * Sm::kStateTile), odd = kBf16 ? (gr & 1) * 8 : 0;
    const int at_chunk = kBf16 ? 4 * col + (gr >> 1) : gr;
    const uint32_t st0 = tile + chunk(64 * rows + 2 * tq, at_chunk) + odd, st1 = tile + chunk(64 * rows + 2 * tq + 1, at_chunk) + odd;
    const uint32_t frag = kTok == 16 ? wide_chunk(mr + 8 * (mi & 1), rows, mi >> 1) : wide_chunk(mr, rows, mi & 1);
    const uint32_t key_frag = st + (kBf16 && col ? Sm::kPk : Sm::kK) + (kTok == 16 ? wide_chunk(mr + 8 * (mi >> 1), rows, mi & 1) : frag);
    const bool scores = kT && (col == 0 || (kBf16 && kC));
    float sc[kOct][4] = {};   // keys 8 i + 2 tq, + 1; rows gr, gr + 8
    // (16 tokens and fp32 states fill the registers: unrolled four times, 256 rows of 16 spill and take 207 us,
    // twice 192)
#pragma unroll (kBf16 || kTok == 8 || !kStore ? 4 : 2)
    for (int ci = 0; ci < 4; ++ci) {
        const uint32_t tok_at = frag ^ (ci << 5);
        float x[2][2][4];      // rows 8 i + 2 tq + e, column j
        [[maybe_unused]] uint32_t xb[2][4];   // bf16: the same as B operands, rows 8 i + 2 tq, + 1 of column j
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t at_row = (16 * ci + 8 * i) * 128;
            if constexpr (kBf16) {
                const uint2 w0 = lds_u32x2(st0 + at_row), w1 = lds_u32x2(st1 + at_row);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint32_t u0 = m ? w0.y : w0.x, u1 = m ? w1.y : w1.x;
                    const float2 f0 = bf16x2_to_float2(u0), f1 = bf16x2_to_float2(u1);
                    x[i][0][2 * m] = f0.x, x[i][0][2 * m + 1] = f0.y;
                    x[i][1][2 * m] = f1.x, x[i][1][2 * m + 1] = f1.y;
                    xb[i][2 * m] = __byte_perm(u0, u1, 0x5410);
                    xb[i][2 * m + 1] = __byte_perm(u0, u1, 0x7632);
                }
            } else {
                const float4 f0 = lds_f32x4(st0 + at_row), f1 = lds_f32x4(st1 + at_row);
                x[i][0][0] = f0.x, x[i][0][1] = f0.y, x[i][0][2] = f0.z, x[i][0][3] = f0.w;
                x[i][1][0] = f1.x, x[i][1][1] = f1.y, x[i][1][2] = f1.z, x[i][1][3] = f1.w;
            }
        }
        if (kC) {
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
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < kOct; ++e) {
                    kb[i][e] &= there[e];
                    if constexpr (kMark) mark_not_finite(mark, kb[i][e]);
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
                    const uint32_t at_row = (e ? st1 : st0) + (16 * ci + 8 * i) * 128;
                    const float *y = x[i][e];
                    if constexpr (kBf16) sts_u32x2(at_row, float2_to_bf16x2(y[0], y[1]), float2_to_bf16x2(y[2], y[3]));
                    else sts_f32x4(at_row, y[0], y[1], y[2], y[3]);
                }
            }
        }
        if (kT) {
            uint32_t qa[4];   // (t, dk), (t + 8, dk), (t, dk + 8), (t + 8, dk + 8)
            if constexpr (kTok == 16) {
                ldmatrix_x4(qa, st + Sm::kQ + tok_at);
            } else {
                ldmatrix_x2(qa[0], qa[2], st + Sm::kQ + tok_at);
                qa[1] = qa[3] = 0u;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (kBf16) {
                    mma(o[j], qa, xb[0][j], xb[1][j]);
                } else {
                    uint32_t part[kParts][2];
#pragma unroll
                    for (int p = 0; p < kParts; ++p)
#pragma unroll
                        for (int i = 0; i < 2; ++i) part[p][i] = split_bf16(x[i][0][j], x[i][1][j]);
#pragma unroll
                    for (int p = kParts - 1; p >= 0; --p) mma(o[j], qa, part[p][0], part[p][1]);
                }
            }
            if (scores) {
                uint32_t k4[4];
                if constexpr (kTok == 16) ldmatrix_x4(k4, key_frag ^ (ci << 5));
                else ldmatrix_x2(k4[0], k4[1], key_frag ^ (ci << 5));
#pragma unroll
                for (int i = 0; i < kOct; ++i) mma(sc[i], qa, k4[2 * i], k4[2 * i + 1]);
            }
        }
    }
    if (scores) {
        const uint32_t at = own_at + (col ? Sm::kPend : Sm::kScore) + rows * Sm::kRect + (gr * Sm::kPitch + 2 * tq) * 4;
#pragma unroll
        for (int i = 0; i < kOct; ++i) {
            sts_f32x2(at + 32 * i, sc[i][0], sc[i][1]);
            if constexpr (kTok == 16) sts_f32x2(at + 32 * i + 8 * Sm::kPitch * 4, sc[i][2], sc[i][3]);
        }
    }
    if (kStore) tc::fence_proxy_async_smem();
    bool not_finite_commit = false;
    if (kStore) {
        bool odd_sum = mark & 0x7fff7fffu;
        if constexpr (!kMark) {
#pragma unroll
            for (int i = 0; i < 8 * kOct; ++i) odd_sum |= !isfinite(o[i & 3][i >> 2]) && gr + 8 * (i >> 3) < tokens;
        }
        __syncwarp();
        not_finite_commit = tck::named_any(group + 9, kGroupThreads, odd_sum);
    } else {
        group_sync(group);
    }

    // 3. the state goes back
    if (kStore && tid == 0 && !not_finite_commit) {
        for (int b = 0; b < Sm::kBoxes; ++b)
            tc::tma_store_3d(pool, it.half * kHalf + b * Sm::kBoxCols, 0,
                             static_cast<int32_t>(static_cast<int64_t>(it.slot) * a.H + it.h), smem + Sm::kState + b * Sm::kStateTile);
        tc::tma_store_commit();
    }

    // each warp finishes the first (rows = 0) or second four of a lane's 8 columns and hands the sums
    // of the others to the warp with the other key rows
    float *swap = reinterpret_cast<float *>(smem + Sm::kSwap);
    if (kT) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            swap[(warp * kTok / 2 + j) * 32 + lane] = rows ? o[j][0] : o[j][1];
            if constexpr (kTok == 16) swap[(warp * 8 + 4 + j) * 32 + lane] = rows ? o[j][2] : o[j][3];
        }
    }
    if (kT) group_sync(group);

    // 4. o_t = scale ( head_t (Q S)_t + sum_{j <= t} decay_tj score_tj v_j ), rows gr, gr + 8; bf16: with
    // fade (Q S)_t + sum_j w_j (q_t . pk_j) pv_j in place of (Q S)_t
    if (kT) {
        const float h0 = __shfl_sync(0xffffffffu, ng.head, gr), h1 = __shfl_sync(0xffffffffu, ng.head, gr + 8);
        const int first = 32 * col + 8 * tq + 4 * rows;   // the lane's 4 columns
        // products of the lane's rows with tokens t, t + 1, from the two halves of the keys' columns
        auto product = [&](uint32_t rect, int r, int t) {
            const uint32_t at = own_at + rect + (r * Sm::kPitch + t) * 4;
            const float2 x = lds_f32x2(at), y = lds_f32x2(at + Sm::kRect);
            return make_float2(x.x + y.x, x.y + y.y);
        };
        float y0[4], y1[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y0[j] = h0 * (kBf16 ? fade : 1.f) * ((rows ? o[j][1] : o[j][0]) + swap[(warp ^ 2) * kTok / 2 * 32 + j * 32 + lane]);
            if constexpr (kTok == 16)
                y1[j] = h1 * (kBf16 ? fade : 1.f) * ((rows ? o[j][3] : o[j][2]) + swap[((warp ^ 2) * 8 + 4 + j) * 32 + lane]);
        }
        // tokens' weights (A operand, in parts) times their values, 8 or 16 tokens
        auto add_tokens = [&](const uint32_t (&pa)[kParts][2 * kOct], const uint32_t (&bv)[4][kOct]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float d[4];
                mma_tok<kTok>(d, pa[kParts - 1], bv[j][0], bv[j][kOct - 1], 0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int p = kParts - 2; p >= 0; --p) mma_tok<kTok>(d, pa[p], bv[j][0], bv[j][kOct - 1], d[0], d[1], d[2], d[3]);
                y0[j] += rows ? d[1] : d[0];
                if constexpr (kTok == 16) y1[j] += rows ? d[3] : d[2];
            }
        };
        if (kBf16 && kC) {
            uint32_t pa[kParts][2 * kOct], bv[4][kOct];
#pragma unroll
            for (int i = 0; i < kOct; ++i) {
                const int t = 2 * tq + 8 * i;
                const float w0 = __shfl_sync(0xffffffffu, pg.tail, t), w1 = __shfl_sync(0xffffffffu, pg.tail, t + 1);
                float2 s0 = product(Sm::kPend, gr, t), s1 = make_float2(0.f, 0.f);
                if constexpr (kTok == 16) s1 = product(Sm::kPend, gr + 8, t);
                s0.x = t < commits ? s0.x * w0 * h0 : 0.f, s1.x = t < commits ? s1.x * w0 * h1 : 0.f;
                s0.y = t + 1 < commits ? s0.y * w1 * h0 : 0.f, s1.y = t + 1 < commits ? s1.y * w1 * h1 : 0.f;
                split_row(pa, 2 * i, s0);
                split_row(pa, 2 * i + 1, s1);
                pack_values(bv, i, values(Sm::kPv, t), values(Sm::kPv, t + 1), there[i]);
            }
            add_tokens(pa, bv);
        }
        uint32_t bv[4][kOct], odd_values = 0;
#pragma unroll
        for (int i = 0; i < kOct; ++i) {
            const int t = 2 * tq + 8 * i;
            const uint32_t in = (t < tokens ? 0xffffu : 0u) | (t + 1 < tokens ? 0xffff0000u : 0u);
            pack_values(bv, i, values(Sm::kV, t), values(Sm::kV, t + 1), in);
#pragma unroll
            for (int j = 0; j < 4; ++j) odd_values |= not_finite(bv[j][i]);
        }
        if (!__any_sync(0xffffffffu, odd_values != 0)) {
            uint32_t pa[kParts][2 * kOct];
#pragma unroll
            for (int i = 0; i < kOct; ++i) {
                const int t = 2 * tq + 8 * i;
                auto weights = [&](int r) {   // 0 for the tokens after token r
                    const float2 s = product(Sm::kScore, r, t), d = lds_f32x2(own_at + Sm::kDecay + (r * Sm::kPitch + t) * 4);
                    return make_float2(t <= r ? s.x * d.x : 0.f, t + 1 <= r ? s.y * d.y : 0.f);
                };
                split_row(pa, 2 * i, weights(gr));
                split_row(pa, 2 * i + 1, kTok == 16 ? weights(gr + 8) : make_float2(0.f, 0.f));
            }
            add_tokens(pa, bv);
        } else {
            // an infinity or NaN among the values: one product at a time, so that it reaches no token
            // before its own
            for (int j = 0; j < tokens; ++j) {
                const uint2 w = lds_u32x2(st + Sm::kV + chunk(j, first / 8) + rows * 8);
                const float2 v0 = bf16x2_to_float2(w.x), v1 = bf16x2_to_float2(w.y);
                const float v[4] = {v0.x, v0.y, v1.x, v1.y};
#pragma unroll
                for (int r = 0; r < kOct; ++r) {
                    const int t = gr + 8 * r;
                    if (j > t) continue;
                    const float s = product(Sm::kScore, t, j & ~1).x, s1 = product(Sm::kScore, t, j & ~1).y;
                    const float p = (j & 1 ? s1 : s) * reinterpret_cast<const float *>(own + Sm::kDecay)[t * Sm::kPitch + j];
#pragma unroll
                    for (int c = 0; c < 4; ++c) (r ? y1 : y0)[c] = fmaf(p, v[c], (r ? y1 : y0)[c]);
                }
            }
        }
        uint16_t *out = a.o + ((it.n * a.T + t0 + gr) * a.H + it.h) * kD + it.half * kHalf + first;
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
    return not_finite_commit;
}

template <bool kBf16, int kTok>
__global__ void __launch_bounds__(StepSmem<kBf16, kTok>::kThreads, 1) 
draft_step_kernel(DraftArgs a, const __grid_constant__ StepMaps maps, unsigned items) {
    using Sm = StepSmem<kBf16, kTok>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t full[Sm::kFulls], empty[Sm::kStages];
    if (threadIdx.x == 0) {
        for (int s = 0; s < Sm::kFulls; ++s) tc::mbar_init(&full[s], 32 + 2);
        for (int s = 0; s < Sm::kStages; ++s) tc::mbar_init(&empty[s], kGroupThreads / 32);
        tc::fence_barrier_init();
    }
    __syncthreads();
    dependent_start();

    // item i: unit i / 2 (n * H + h), column half i % 2; this CTA's k-th goes through stage k % kStages and
    // is announced on full[k % kFulls]; group k % kGroups takes it. Item k is staged once item k - kStages
    // was taken, so neither kind of barrier is ever two phases ahead of who waits for it.
    const unsigned step = gridDim.x;
    if (threadIdx.x >= Sm::kGroups * kGroupThreads) {
        const int lane = threadIdx.x & 31;
        const bool states = threadIdx.x < Sm::kGroups * kGroupThreads + 32;   // or the tokens
        int stage = 0, next_full = 0;
        uint32_t parity = 1;   // of the wait for an empty stage: the first round passes at once
        auto read = [&](unsigned item) {
            Item it{};
            if (item < items) {
                const unsigned unit = item >> 1, n = unit / static_cast<unsigned>(a.H);
                const Row row = read_row(a, static_cast<int>(n), states && lane == 0);
                it = {row.slot, static_cast<int32_t>(n), static_cast<int32_t>(unit - n * a.H), static_cast<int32_t>(item & 1),
                      static_cast<int32_t>(row.commits), static_cast<int32_t>(row.tokens), {0, 0}};
            }
            return it;
        };
        Item next = read(blockIdx.x);
        unsigned staged = 0;
        for (unsigned item = blockIdx.x; item < items; item += step) {
            const Item it = next;
            next = read(item + step);   // its latency hides behind this item's copies
            if (__any_sync(0xffffffffu, !ring_wait(&empty[stage], parity))) {
                if (lane == 0) record_status(a.status, SALA_ERR_TIMEOUT);
                break;
            }
            uint8_t *at = smem + stage * Sm::kStage, *side = smem + Sm::kSides + stage * Sm::kSide;
            if (states) stage_state<kBf16, kTok>(a, maps, at, side, it, &full[next_full], lane);
            else stage_tokens<kBf16, kTok>(a, maps, at, side, it, &full[next_full], lane);
            ++staged;
            if (++next_full == Sm::kFulls) next_full = 0;
            if (++stage == Sm::kStages) stage = 0, parity ^= 1;
        }
        // no copy outlives the CTA, however it ends: the last ones of every stage have landed
        for (unsigned k = staged > Sm::kStages ? staged - Sm::kStages : 0; k < staged; ++k)
            if (!ring_wait(&full[k % Sm::kFulls], (k / Sm::kFulls) & 1)) break;
        return;
    }

    const int group = threadIdx.x / kGroupThreads, tid = threadIdx.x & (kGroupThreads - 1);
    uint8_t *own = smem + Sm::kOwns + group * Sm::kOwn;
    int stage = group, mine = group;
    uint32_t parity = 0;
    for (unsigned item = blockIdx.x + group * step; item < items; item += Sm::kGroups * step) {
        const bool late = !ring_wait(&full[mine], parity);
        if (late) record_status(a.status, SALA_ERR_TIMEOUT);
        __syncwarp();
        // also: the group's memory of the item before is free
        if (tck::named_any(group + 1, kGroupThreads, late)) break;
        uint8_t *at = smem + stage * Sm::kStage, *side = smem + Sm::kSides + stage * Sm::kSide;
        const Item it = *reinterpret_cast<const Item *>(side + Sm::kHead);
        for (int e = it.tokens * 8 + tid; e < static_cast<int>(a.T) * 8; e += kGroupThreads)   // rows past the count
            *reinterpret_cast<uint4 *>(a.o + ((it.n * a.T + e / 8) * a.H + it.h) * kD + it.half * kHalf + 8 * (e % 8)) =
                make_uint4(0, 0, 0, 0);
        bool odd = false;
        if (it.commits && it.tokens) odd = run_item<kBf16, kTok, true, true>(a, &maps.pool, at, side, own, it, group);
        else if (it.commits) odd = run_item<kBf16, kTok, true, false>(a, &maps.pool, at, side, own, it, group);
        else if (it.tokens) run_item<kBf16, kTok, false, true>(a, &maps.pool, at, side, own, it, group);
        if (odd) commit_by_one<kBf16>(a, item, tid >> 4, kD);
        if (tid == 0) tc::tma_store_wait_read<0>();
        tc::fence_proxy_async_smem();   // the stage was written to, and TMA writes to it next
        __syncwarp();
        if ((tid & 31) == 0) tc::mbar_arrive(&empty[stage]);
        stage = (stage + Sm::kGroups) % Sm::kStages;
        mine += Sm::kGroups;
        if (mine >= Sm::kFulls) mine = group, parity ^= 1;
    }
    if (tid == 0) tc::tma_store_wait_all<0>();
}

// ---- longer steps ----------------------------------------------------------------------------
//
// One CTA of 4 warps per item. The state half stays in shared memory in fp32, whatever the pool's
// type, and blocks of up to 16 tokens go over it: a pass adds one block and reads the state for
// another. The accepted tokens are added first, the last of them in the pass that reads for the first
// new tokens; then the state is stored, and each pass adds the block that the one before read for. All
// copies are asynchronous, a block's at the start of its pass: four CTAs on an SM, which 128 registers a
// thread allow, hide that from each other (with a second buffer for the blocks, which leaves room for
// three, 256 fp32 rows of 17 take a fourteenth longer; with plain loads, nearly twice as long). Bound by the
// passes, a little over 1 us of an SM's time each whatever the block holds: 256 rows of 17, 32 heads, 3 passes,
// 359 us with fp32 states (floor 185), 352 with bf16 (106); 16 rows of 200 after 200, bf16, 175 us (floor 24).

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
// m token rows of [tokens, H, 128]: all of a row (kWide) or the item's half.
template <bool kWide>
__device__ __forceinline__ void put_tokens(uint8_t *dst, const uint16_t *src, int64_t row0, int H, int m) {
    constexpr int kChunks = kWide ? 16 : 8;
    const int c = threadIdx.x % kChunks;
    for (int t = threadIdx.x / kChunks; t < m; t += kGroupThreads / kChunks)
        cp_async16(dst + (kWide ? wide_chunk(t, c >> 3, c & 7) : chunk(t, c)), src + (row0 + static_cast<int64_t>(t) * H) * kD + 8 * c);
}
__device__ __forceinline__ void put_gates(uint8_t *dst, const float *g, int64_t row0, int H, int m) {
    const int t = threadIdx.x;
    if (t < m) cp_async4(tc::smem_u32(dst) + 4 * t, g + row0 + static_cast<int64_t>(t) * H);
}

constexpr size_t kLongBytes = StepSmem<false, 16>::kStage + StepSmem<false, 16>::kSide + StepSmem<false, 16>::kOwn;

template <bool kBf16>
__global__ void __launch_bounds__(kGroupThreads, 4) draft_step_long_kernel(DraftArgs a) {
    dependent_start();
    using Sm = StepSmem<false, 16>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *side = smem + Sm::kStage, *own = side + Sm::kSide;
    const int unit = blockIdx.x >> 1, half = blockIdx.x & 1, n = unit / a.H, h = unit - n * a.H, tid = threadIdx.x;
    const Row row = read_row(a, n, tid == 0);
    for (int64_t e = row.tokens * 8 + tid; e < a.T * 8; e += kGroupThreads)   // rows past the count
        *reinterpret_cast<uint4 *>(a.o + ((n * a.T + e / 8) * a.H + h) * kD + half * kHalf + 8 * (e % 8)) = make_uint4(0, 0, 0, 0);
    if (row.commits == 0 && row.tokens == 0) return;

    // four neighbouring values of the state half: row r, columns 4 c .. 4 c + 3
    const int64_t at = (static_cast<int64_t>(row.slot) * a.H + h) * kD * kD + half * kHalf;
    auto place = [&](int r, int c) {
        return reinterpret_cast<float4 *>(smem + Sm::kState + (c >> 3) * Sm::kStateTile + chunk(r, c & 7));
    };
    const int64_t pend0 = n * a.T_pend * a.H + h, new0 = n * a.T * a.H + h;   // token rows of this head
    const int commits = static_cast<int>(row.commits), tokens = static_cast<int>(row.tokens);   // of one row: fewer than fill the memory
    const int before = (commits + 15) / 16, first_read = before > 1 ? before - 1 : 0;   // passes that add accepted tokens; that do nothing else
    const int passes = max(before, first_read + (tokens + 15) / 16);
    Item it{row.slot, n, h, half, 0, 0, {0, 0}};
    // What pass p adds and reads for: places (negative: nothing) and counts of up to 16 tokens.
    auto plan = [&](int p, int &j0, int &t0) {
        t0 = 16 * (p - first_read), j0 = p < before ? 16 * p : t0 - 16;
        it.tokens = t0 >= 0 ? min(16, tokens - t0) : 0;
        it.commits = j0 >= 0 ? min(16, (p < before ? commits : tokens) - j0) : 0;
    };
    auto load = [&](int p) {
        int j0, t0;
        plan(p, j0, t0);
        if (it.commits) {
            const bool pending = p < before;
            const int64_t first = (pending ? pend0 : new0) + static_cast<int64_t>(j0) * a.H;
            put_tokens<true>(smem + Sm::kPk, pending ? a.pk : a.k, first, a.H, it.commits);
            put_tokens<false>(smem + Sm::kPv, (pending ? a.pv : a.v) + half * kHalf, first, a.H, it.commits);
            put_gates(side + Sm::kPg, pending ? a.pg : a.g, first, a.H, it.commits);
        }
        if (it.tokens) {
            const int64_t first = new0 + static_cast<int64_t>(t0) * a.H;
            put_tokens<true>(smem + Sm::kQ, a.q, first, a.H, it.tokens);
            put_tokens<true>(smem + Sm::kK, a.k, first, a.H, it.tokens);
            put_tokens<false>(smem + Sm::kV, a.v + half * kHalf, first, a.H, it.tokens);
            put_gates(side + Sm::kG, a.g, first, a.H, it.tokens);
        }
    };
    load(0);   // on its way while the state comes
    const int r0 = tid / 16, c0 = tid % 16;   // every eighth row is this thread's
    if constexpr (kBf16) {
        uint2 w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            w[i] = __ldcs(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.pool) + at + (8 * i + r0) * kD) + c0);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 f0 = bf16x2_to_float2(w[i].x), f1 = bf16x2_to_float2(w[i].y);
            *place(8 * i + r0, c0) = make_float4(f0.x, f0.y, f1.x, f1.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            cp_async16(place(8 * i + r0, c0), static_cast<const float *>(a.pool) + at + (8 * i + r0) * kD + 4 * c0);
    }
    for (int p = 0; p < passes; ++p) {
        if (p) {
            __syncthreads();   // all are through with the tokens before
            load(p);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        int j0, t0;
        plan(p, j0, t0);
        if (it.commits && it.tokens) run_item<false, 16, true, true, false>(a, nullptr, smem, side, own, it, 0, t0);
        else if (it.commits) run_item<false, 16, true, false, false>(a, nullptr, smem, side, own, it, 0);
        else run_item<false, 16, false, true, false>(a, nullptr, smem, side, own, it, 0, t0);
        if (p == before - 1) {   // the commit is complete
            __syncthreads();
#pragma unroll 1
            for (int r = r0; r < kD; r += 64) {
                float4 f[8];
                float odd = 0.f;   // NaN: an infinity or NaN among the values
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    f[i] = *place(r + 8 * i, c0);
                    odd = fmaf(f[i].x, 0.f, fmaf(f[i].y, 0.f, fmaf(f[i].z, 0.f, fmaf(f[i].w, 0.f, odd))));
                }
                if (odd != 0.f) {
                    commit_by_one<kBf16>(a, blockIdx.x, r, r + 64);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) store_state<kBf16>(a.pool, at, r + 8 * i, c0, f[i]);
                }
            }
        }
    }
}

cudaError_t pool_map(CUtensorMap *map, const void *pool, bool bf16, int64_t states) {
    const cuuint64_t dims[3] = {kD, kD, static_cast<cuuint64_t>(states)};
    const cuuint64_t row = kD * (bf16 ? 2 : 4), strides[2] = {row, kD * row};
    const cuuint32_t box[3] = {bf16 ? 64u : 32u, kD, 1};
    return tck::encode_tiled(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, pool, dims, strides,
                             box, CU_TENSOR_MAP_SWIZZLE_128B);
}

cudaError_t token_map(CUtensorMap *map, const void *tokens, int64_t N, int64_t T, int H, bool values) {
    const cuuint64_t dims[5] = {64, 2, static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T), static_cast<cuuint64_t>(N)};
    const cuuint64_t strides[4] = {128, 256, dims[2] * 256, dims[3] * dims[2] * 256};
    const cuuint32_t box[5] = {64, values ? 1u : 2u, 1, 8, 1};
    return tck::encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, tokens, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <bool kBf16, int kTok>
cudaError_t launch_step(const DraftArgs &a, const StepMaps &maps, unsigned items, unsigned grid, cudaStream_t stream) {
    using Sm = StepSmem<kBf16, kTok>;
    return launch_dependent_cluster(draft_step_kernel<kBf16, kTok>, grid, 0, Sm::kThreads, Sm::kBytes, stream, a, maps, items);
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
    // the persistent kernel where a step is one pass: 256 rows of 16, bf16, in 146 us, 213 by the kernel
    // for longer ones; fp32 192 and 220; one row of 5, 4.5 and 5.8
    if (T <= 16 && T_pend <= 16) {
        StepMaps maps{};
        cudaError_t e = pool_map(&maps.pool, pool, bf16, P * H);
        if (e == cudaSuccess && T_pend) e = token_map(&maps.pk, pend_k, N, T_pend, H, false);
        if (e == cudaSuccess && T_pend) e = token_map(&maps.pv, pend_v, N, T_pend, H, true);
        if (e == cudaSuccess && T) e = token_map(&maps.q, q, N, T, H, false);
        if (e == cudaSuccess && T) e = token_map(&maps.k, k, N, T, H, false);
        if (e == cudaSuccess && T) e = token_map(&maps.v, v, N, T, H, true);
        if (e != cudaSuccess) return e;
        // operands of 8 tokens where they suffice: 256 bf16 rows of 5 in 112 us, with those of 16 in 144; 256
        // fp32 rows of 5 in 177 and 183, of 8 in 184 and 185, 64 fp32 rows of 5 in 49 and 51, one in 4.5 and 5.1
        const bool few = T <= 8 && T_pend <= 8;
        const unsigned items = static_cast<unsigned>(2 * N * H);
        const unsigned grid = items < static_cast<unsigned>(sm_count) ? items : sm_count;
        return bf16 ? (few ? launch_step<true, 8>(a, maps, items, grid, stream) : launch_step<true, 16>(a, maps, items, grid, stream))
                    : (few ? launch_step<false, 8>(a, maps, items, grid, stream) : launch_step<false, 16>(a, maps, items, grid, stream));
    }
    return launch_dependent_cluster(bf16 ? draft_step_long_kernel<true> : draft_step_long_kernel<false>,
                                    static_cast<unsigned>(2 * N * H), 0, kGroupThreads, kLongBytes, stream, a);
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
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(draft_step_long_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLongBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(draft_step_long_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLongBytes);
    return e;
}

}  // namespace sala

// Causal attention of new tokens over a paged cache.
//
// The G query heads of a key/value head see the same keys, so a row is a (token, head of the group) and a query
// tile holds 128 / G whole tokens: 128 rows at most, contiguous in q for each token. A unit is two such tiles of one
// request and key/value head with all the places that they see, cut into cache tiles of 128 places:
//     S = Q K^T (128 x 128 x 128, tcgen05, fp32 in tensor memory)
//     P = 2^(c S - m), c = scale * k_scale * log2 e, with the row's running maximum m
//     O += P V  (P as bf16 in tensor memory, V from shared memory)
// The running sum takes P before its rounding to bf16; the rounding (2^-9 of each weight on average, to either side)
// averages out in O like the rounding of O itself, and fp32 products would run at a small part of the rate.
// O is rescaled only where the maximum grew by more than 2^8: until then P is at most 2^8 and keeps its relative precision.
//
// One persistent CTA per SM. Every CTA takes an equal share of all cache tiles (a request's number of tiles has a
// closed form, and their running sum over the requests is all that a CTA needs to find its place), so a
// unit may be shared by several CTAs, which leave partial results (O, m, sum) that a last kernel joins. This
// serves one token on a long cache and a full batch alike.
//
// Roles: two groups of eight warps turn scores into weights, one for each query tile (two lanes share a row), one warp
// issues the products, one (two for small pages) loads by TMA, a page (and half of the dimensions) a box. While one group has its
// scores, the tensor core works for the other. A unit with one query tile gives its cache tiles to the groups in
// turn, and the results are joined at its end, by the group that had the first (also in turn: the other one has the next
// unit's scores meanwhile). e4m3 tiles land in a ring of their own and eight more warps
// widen them (exactly) to bf16.
//
// Bounds, at 32 query heads on 2 key/value heads. 256 requests of one token on up to 12288 bf16 places: the cache's 2.15 GB,
// 316 to 321 us = 6.7 TB/s, a copy's rate. A chunk of 4096 tokens on 32768 places: 2.06 TFLOP in 1240 us by itself = 1660 TFLOP/s, the
// products at the clock that the power limit leaves (a library product 1695); calls in a row, with the join of its ends, take 1300 to
// 1360 us, 1510 to 1580 TFLOP/s. A softmax thread has 96 registers and 64 scores: what is not needed between a tile's scores and its
// weights stays out of registers there, which took 120 us off the chunk. 61 requests with 5 tokens on 8192 e4m3 places: 88 us against
// 38 for its bytes, and 256 requests of one token on up to 12288 such places 275 us against 159; the tiles pass shared memory three
// times more (read and stored by the widening, read by the product). fp16 tiles, cheaper to widen, took longer (the queries then
// need a scale for each row to stay in range). One token on 4001 places: 15 us of launch, split, one tile a CTA and join.
//
// What is masked never enters: scores are replaced, not added to, and V is cleared in the rows behind the unit's
// last place (0 times a NaN there would be NaN). Rows of V that some tokens of the unit see and others do not are
// searched for infinities and NaN, which are cleared and put into the results that see them at the end.
#include <type_traits>

#include "paged_tiles.cuh"

namespace sala {
namespace {

using namespace pt;
using tc::mbar_arrive;

constexpr int kRows = 2 * kTile;                 // rows of a unit, at most
constexpr int kMmaWarp = 16, kLoadWarp = 17, kValueWarp = 18;
constexpr uint32_t kS0 = 0, kO0 = 256;           // tensor memory columns: S (and P over it) of the groups, then O
constexpr float kRescale = 8.f;                  // growth of the maximum (log2) that rescales O
// c m beyond which the scores' differences are taken before the factor c. Below it the rounding of c m is 2^-14 at most, no more than
// those of such scores themselves. (As the only way they took a chunk of 4096 tokens on 32768 places from 1316 to 1365 us; as a way of
// their own beside the usual one to 1330, and 256 requests on up to 1000 places with 8 key/value heads from 127 to 134.)
constexpr float kFar = 1024.f;
constexpr uint32_t kIdS = tc::idesc_bf16_f32(128, 128, 0, 0), kIdO = tc::idesc_bf16_f32(128, 128, 0, 1);

// Shared memory of units with Q query tiles: the queries, the ring of cache tiles, the ring of e4m3 tiles. Split: the values
// have a loading warp of their own.
template <bool E4M3, int Q, bool Split>
struct Shape {
    static constexpr int kConvertWarp = Split ? kValueWarp + 1 : kValueWarp;
    static constexpr int kStages = E4M3 ? 4 : 7 - Q, kRaw = E4M3 ? 6 - 2 * Q : 0;
    static constexpr int kThreads = 32 * (E4M3 ? kConvertWarp + kConvertWarps : kConvertWarp);
    static constexpr uint32_t kRawAt = (Q + kStages) * kTileBytes;
    static constexpr uint32_t kAlloc = kRawAt + kRaw * kRawBytes + 1024;   // aligned to the swizzle's 1024 bytes
};

// What the roles of a CTA do next, from the loading warp: cache tiles [t0, t1) of ntok tokens of request n, the first at
// packed token `row` and place `limit` (negative: it sees nothing).
struct alignas(16) Item {
    int64_t row;
    int n, h, ntok, limit, t0, t1;
    int slot;            // where a partial result goes, -1: the item is the whole unit
    int last;
    int pad[2];
    __device__ __forceinline__ int end() const { return max(0, limit + ntok); }   // behind the last place seen
};
constexpr int kItems = 4;

// A unit that this CTA began and others finished: `parts` partial results, from this CTA on (0: none).
struct alignas(16) JoinUnit {
    int64_t row;
    int h, ntok, limit, parts;
};

struct Barriers {
    uint64_t full[6], empty[6];                 // cache tiles
    uint64_t raw_full[6], raw_empty[6];         // e4m3 cache tiles
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t q_full, q_free;
    uint64_t s_full[2], p_full[2], p_rest[2], o_full[2], o_free[2], join;   // P: its first 64 places, the others
    uint64_t drain;
};

// Exponent bits all ones in one of two bf16.
__device__ __forceinline__ uint32_t clear_bad(uint32_t w, bool *bad) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u, *bad = true;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu, *bad = true;
    return w;
}

__device__ __forceinline__ float value_at(const KvArgs &c, int64_t row, int d) {
    if (c.e4m3) return kv::e4m3x2_to_float2(c.v[row * kD + d]).x;
    return bf16_bits_to_float(reinterpret_cast<const uint16_t *>(c.v)[row * kD + d]);
}

// The dimensions in which a value that place `limit` sees, behind place `seen_by_all`, is not finite.
__device__ __noinline__ void bad_dimensions(const KvArgs &c, int64_t n, int h, int seen_by_all, int limit, uint32_t (&dims)[4]) {
    for (int i = 0; i < 4; ++i) dims[i] = 0;
    for (int j = max(0, seen_by_all + 1); j <= limit; ++j) {
        const int page = kv::page_of(c, n, j);
        if (page < 0) continue;
        const int64_t row = kv::row_of(c, page, h, j);
        for (int d = 0; d < kD; ++d)
            if (!isfinite(value_at(c, row, d))) dims[d >> 5] |= 1u << (d & 31);
    }
}

// Factor c of a head's scores: the exponents are c s.
__device__ __forceinline__ float exponent_scale(const AttendArgs &a, int h) {
    return a.scale * (a.c.k_scale ? kv::load(a.c.k_scale + h) : 1.f) * kLog2e;
}

// 2^(c (m - top)): what moves a part of a row with the maximum m to the maximum of all parts. The part's P and sum are
// 2^(c s - [c m]) with the rounded product [c m], so that the difference of the rounded products joins them exactly; where c m
// is far from 0 they are 2^(c (s - m)), and the products' roundings would be more than the difference.
__device__ __forceinline__ float part_factor(float m, float top, float scale) {
    if (m == -INFINITY) return 0.f;
    const float at = __fmul_rn(top, scale);
    return tc::ex2(fabsf(at) > kFar ? (m - top) * scale : __fsub_rn(__fmul_rn(m, scale), at));
}
// c m of a row's maximum, 0 where it has none
__device__ __forceinline__ float exponent_of(float m, float scale) { return m == -INFINITY ? 0.f : m * scale; }
// log sum exp in units of the scores, for the accumulated weights: below c it would lose the score's own bits
__device__ __forceinline__ float score_lse(float m, float l, float scale) { return m + log2f(l) / scale; }

// The 16-lane forms of tensor memory accesses: lanes l and l + 16 of the warp take the same row, 32 columns apart (or
// OFF apart, for a store).
__device__ __forceinline__ void tmem_ld_half_x32(uint32_t taddr, uint32_t (&r)[32]) { tc::tmem_ld_16x32bx2_x32(taddr, r); }
template <int OFF>
__device__ __forceinline__ void tmem_st_16x32bx2_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x32bx2.x16.b32 [%0], %17, "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "n"(OFF)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_half_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8], 32;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_half_x8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x32bx2.x8.b32 [%0], 32, {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

template <bool E4M3, int kQ, bool kSplit>
__global__ void __launch_bounds__(Shape<E4M3, kQ, kSplit>::kThreads, 1)
    paged_attention_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ Maps maps) {
    using Layout = Shape<E4M3, kQ, kSplit>;
    constexpr int kConvertWarp = Layout::kConvertWarp;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Barriers bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, bad_values[2];
    __shared__ Place place;
    __shared__ Item ring[kItems];
    __shared__ float2 other[kTile];   // maxima and sums of the second group, where both have the same rows
    const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *const smem = smem_raw + (base - tc::smem_u32(smem_raw));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
    const KvArgs &c = a.c;
    const AttendWork work{kQ * a.TB};

    if (warp == kMmaWarp) {
        tc::tmem_alloc(&tmem_slot, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < Layout::kStages; ++i) {
            tc::mbar_init(&bar.full[i], E4M3 ? kConvertWarps : 1);
            tc::mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < Layout::kRaw; ++i) {
            tc::mbar_init(&bar.raw_full[i], 1);
            tc::mbar_init(&bar.raw_empty[i], kConvertWarps);
        }
        for (int i = 0; i < kItems; ++i) {
            tc::mbar_init(&bar.item_full[i], 1);
            tc::mbar_init(&bar.item_empty[i], kMmaWarp + 1 + kSplit);
        }
        tc::mbar_init(&bar.q_full, 1);
        tc::mbar_init(&bar.q_free, 1);
        for (int t = 0; t < 2; ++t) {
            tc::mbar_init(&bar.s_full[t], 1);
            tc::mbar_init(&bar.p_full[t], kMmaWarp / 2);
            tc::mbar_init(&bar.p_rest[t], kMmaWarp / 2);
            tc::mbar_init(&bar.o_full[t], 2);
            tc::mbar_init(&bar.o_free[t], kMmaWarp / 2);
        }
        tc::mbar_init(&bar.join, kMmaWarp / 2);
        tc::mbar_init(&bar.drain, 1);
        tc::fence_barrier_init();
        abort_flag = 0;
    }
    wait_for_previous();
    let_dependents_start();   // which so have the lengths, offsets and pages as this kernel has them
    uint32_t *const near = reinterpret_cast<uint32_t *>(smem);   // where the tiles land later
    if (!a.attend_start) scan_requests(c, work, near, near + kInline + 1);
    const Starts starts{a.attend_start ? nullptr : near, a.attend_start};
    const int64_t per_head = starts[c.N], all = per_head * c.H;
    const int64_t begin = range_begin(all, cta, gridDim.x), stop = range_begin(all, cta + 1, gridDim.x);
    const bool idle = begin >= stop;
    if (threadIdx.x == 0 && !idle) place = find(c, work, starts, per_head, begin);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (idle && threadIdx.x == 0) static_cast<JoinUnit *>(a.joins)[cta].parts = 0;
    const uint32_t tmem = tmem_slot;
    volatile int *const aborted = &abort_flag;
    int *const status = c.status;

    // the ring of tiles as they land: keys and values in turn
    constexpr uint32_t kRing = E4M3 ? Layout::kRaw : Layout::kStages;
    uint64_t *const full = E4M3 ? bar.raw_full : bar.full, *const empty = E4M3 ? bar.raw_empty : bar.empty;
    auto tile_at = [](uint32_t st) { return E4M3 ? Layout::kRawAt + st * kRawBytes : (kQ + st) * kTileBytes; };
    // The last copies of a loading warp, those before tile `it`, land before the CTA ends, whoever gave up; `odd`: of the values alone.
    auto drain_tiles = [&](uint32_t it, uint32_t odd) {
        for (uint32_t j = it > kRing ? it - kRing : 0; j < it; ++j)
            if (!kSplit || (j & 1) == odd) tc::mbar_wait(&full[j % kRing], (j / kRing) & 1, tck::kWaitNs);
    };
    if (warp == kLoadWarp && !idle) {
        // ---- loads: Q of each item, then K and V of each cache tile -----------------------------
        uint32_t it = 0, items = 0, q_issued = 0;   // cache tiles and items so far
        bool ok = true;
        JoinUnit join = {0, 0, 0, 0, 0};
        Walk<AttendWork> w;
        w.start_at(c, work, place, begin, stop, cta);
        tc::fence_proxy_async_smem();   // the running sums were there before the tiles
        do {
            const int tok = w.u * work.block, slot = items % kItems;
            Item x;
            x.row = w.r.first + tok;
            x.n = static_cast<int>(w.n);
            x.h = w.h;
            x.ntok = min(work.block, w.r.count - tok);
            x.limit = w.r.len - w.r.count + tok;
            x.t0 = w.t0;
            x.t1 = w.t1;
            x.slot = w.slot;
            x.last = w.pos + (w.t1 - w.t0) >= stop;
            ok = items < kItems || wait_warp(&bar.item_empty[slot], (items / kItems - 1) & 1, aborted, status);
            if (!ok) break;
            if (lane == 0) {
                ring[slot] = x;
                mbar_arrive(&bar.item_full[slot]);
            }
            __syncwarp();
            const int end = x.end(), nt = kQ == 2 && x.ntok > a.TB ? 2 : 1;
            int page = box_page<E4M3>(c, w.n, w.t0, end, lane);   // of the next tile: looked up ahead
            for (int i = w.t0; i < w.t1 && ok; ++i) {
                const int here = page;
                page = i + 1 < w.t1 ? box_page<E4M3>(c, w.n, i + 1, end, lane) : -2;
                for (int kv = 0; kv < 2 && ok; ++kv, ++it) {   // a wait for room for the queries that gave up stands
                    if (kv == 1 && kSplit) continue;
                    const int st = it % kRing;
                    ok = it < kRing || wait_warp(&empty[st], (it / kRing - 1) & 1, aborted, status);
                    if (!ok) break;
                    load_boxes<E4M3>(c, kv ? &maps.v : &maps.k, smem + tile_at(st), i, w.h, here, lane, &full[st]);
                    if (i == w.t0 && kv == 0) {   // behind the first K: its buffer may still be in use
                        ok = items == 0 || wait_warp(&bar.q_free, (items - 1) & 1, aborted, status);
                        if (ok && lane == 0) {
                            tc::mbar_arrive_expect_tx(&bar.q_full, nt * 2 * static_cast<uint32_t>(a.TB * a.G) * 128u);
                            for (int t = 0; t < nt; ++t)
                                load_query_tile(smem + t * kTileBytes, &maps.q, w.h, a.G, x.row + t * a.TB, &bar.q_full);
                        }
                        q_issued += ok;
                        __syncwarp();
                    }
                }
            }
            ++items;
            if (ok && x.last && lane == 0 && x.slot >= 0 && x.t0 == 0)
                join = {x.row, x.h, x.ntok, x.limit, cta_of(all, w.pos + w.tiles - 1, gridDim.x) - cta + 1};
        } while (ok && w.next(c, work, cta));
        if (lane == 0) static_cast<JoinUnit *>(a.joins)[cta] = join;
        if (q_issued) tc::mbar_wait(&bar.q_full, (q_issued - 1) & 1, tck::kWaitNs);
        drain_tiles(it, 0);
    } else if (kSplit && warp == kValueWarp && !idle) {
        // ---- loads of the values where one warp does not keep up ------------------------------------
        uint32_t it = 1, items = 0;
        bool ok = true, last = false;
        do {
            ok = wait_warp(&bar.item_full[items % kItems], (items / kItems) & 1, aborted, status);
            if (!ok) break;
            const Item &x = ring[items % kItems];
            const int n = x.n, h = x.h, end = x.end(), t1 = x.t1;
            last = x.last;
            int page = box_page<E4M3>(c, n, x.t0, end, lane);
            for (int i = x.t0; i < t1; ++i, it += 2) {
                const int here = page, st = it % kRing;
                page = i + 1 < t1 ? box_page<E4M3>(c, n, i + 1, end, lane) : -2;
                ok = it < kRing || wait_warp(&empty[st], (it / kRing - 1) & 1, aborted, status);
                if (!ok) break;
                load_boxes<E4M3>(c, &maps.v, smem + tile_at(st), i, h, here, lane, &full[st]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.item_empty[items % kItems]);
            ++items;
        } while (ok && !last);
        drain_tiles(it, 1);
    } else if (E4M3 && warp >= kConvertWarp && !idle) {
        // ---- e4m3 tiles to bf16 --------------------------------------------------------------------
        constexpr int kRaw = E4M3 ? Layout::kRaw : 1;
        const int id = threadIdx.x - 32 * kConvertWarp;
        const int64_t tiles = 2 * (stop - begin);
        uint4 held[kPieces];   // of the next tile: read while the stores of this one drain
        bool ok = wait_warp(&bar.raw_full[0], 0, aborted, status);
        if (ok) read_pieces(held, smem + Layout::kRawAt, id);
        for (int64_t it = 0; it < tiles && ok; ++it) {
            const int st = it % Layout::kStages, rw = it % kRaw, next = (it + 1) % kRaw;
            ok = it < Layout::kStages || wait_warp(&bar.empty[st], (it / Layout::kStages - 1) & 1, aborted, status);
            if (!ok) break;
            store_pieces(held, smem + (kQ + st) * kTileBytes, id);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.raw_empty[rw]);
            const bool there = it + 1 < tiles && __all_sync(0xffffffffu, tc::mbar_test_wait(&bar.raw_full[next], ((it + 1) / kRaw) & 1));
            if (there) read_pieces(held, smem + Layout::kRawAt + next * kRawBytes, id);
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.full[st]);
            if (it + 1 < tiles && !there) {
                ok = wait_warp(&bar.raw_full[next], ((it + 1) / kRaw) & 1, aborted, status);
                if (ok) read_pieces(held, smem + Layout::kRawAt + next * kRawBytes, id);
            }
        }
    } else if (warp == kMmaWarp && !idle) {
        // ---- products ------------------------------------------------------------------------------
        constexpr int S = Layout::kStages;
        const uint32_t full = tc::smem_u32(bar.full), empty = tc::smem_u32(bar.empty), s_full = tc::smem_u32(bar.s_full);
        const uint32_t p_full = tc::smem_u32(bar.p_full), p_rest = tc::smem_u32(bar.p_rest), o_full = tc::smem_u32(bar.o_full), o_free = tc::smem_u32(bar.o_free);
        const uint32_t q_free = tc::smem_u32(&bar.q_free), q_full = tc::smem_u32(&bar.q_full);
        const uint64_t first_k = desc_k(base), first_mn = desc_mn(base + kQ * kTileBytes);   // of the first tile, the first stage
        uint32_t items = 0, p_parity = 0, o_used = 0, o_parity = 3;   // a bit for each group
        bool ok = true, last = false;
        auto passed = [&](uint32_t b, uint32_t parity) {
            return __all_sync(0xffffffffu, wait_at(b, parity, aborted, status)) != 0;
        };
        auto scores = [&](int t, int q, uint32_t stage) {   // of query tile q, for group t
            if (tc::elect_one()) {
                const uint64_t dq = first_k + q * (kTileBytes >> 4), dk = first_k + (kQ + stage) * (kTileBytes >> 4);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
                    tc::umma_bf16(tmem + kS0 + t * kTile, dq + off, dk + off, kIdS, ks > 0);
                }
                commit_at(s_full + 8 * t);
            }
            __syncwarp();
        };
        auto commit = [&](uint32_t b) {
            if (tc::elect_one()) commit_at(b);
            __syncwarp();
        };
        // O of group t from its P and the values of a stage; `first` of the item, `final` of the item
        auto products = [&](int t, uint32_t stage, bool first, bool final) {
            if (!passed(p_full + 8 * t, p_parity >> t & 1)) return false;
            if (first) {   // the results of the item before are read
                if ((o_used >> t & 1) && !passed(o_free + 8 * t, o_parity >> t & 1)) return false;
                o_used |= 1u << t;
                o_parity ^= 1u << t;
            }
            // the first 64 places' products go while the others' weights are made
            const uint64_t dv = first_mn + stage * (kTileBytes >> 4);
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                if (part == 1 && !passed(p_rest + 8 * t, p_parity >> t & 1)) return false;
                tc::tc_fence_after();
                if (tc::elect_one()) {
#pragma unroll
                    for (int ks = 4 * part; ks < 4 * part + 4; ++ks)
                        tc::umma_bf16_ta(tmem + kO0 + t * kTile, tmem + kS0 + t * kTile + 8 * ks, dv + ks * (2048 >> 4), kIdO,
                                         !first || ks > 0);
                    if (part == 1 && final) commit_at(o_full + 8 * t);
                }
                __syncwarp();
            }
            p_parity ^= 1u << t;
            return true;
        };
        // Clears the rows of V that no token sees, and infinities and NaN in those that not all tokens see: true if any
        auto clean = [&](int shared_from, int end, int i, uint32_t stage) {
            const int p0 = i * kTile;
            uint8_t *v = smem + (kQ + stage) * kTileBytes;
            for (int e = lane + max(0, min(kTile, end - p0)) * 16; e < kTile * 16; e += 32)
                *reinterpret_cast<uint4 *>(v + piece_at(e >> 4, e & 15)) = make_uint4(0, 0, 0, 0);
            bool found = false;
            for (int e = lane + max(0, shared_from - p0) * 16; e < min(kTile, end - p0) * 16; e += 32) {
                uint4 *at = reinterpret_cast<uint4 *>(v + piece_at(e >> 4, e & 15));
                const uint4 y = *at;
                bool here = false;
                const uint4 z = make_uint4(clear_bad(y.x, &here), clear_bad(y.y, &here), clear_bad(y.z, &here),
                                           clear_bad(y.w, &here));
                if (here) *at = z, found = true;
            }
            tc::fence_proxy_async_smem();
            return __any_sync(0xffffffffu, found) != 0;
        };
        Ring<S> k, v;   // the stages of the next keys and values
        v.advance(1);
        do {
            ok = passed(tc::smem_u32(&bar.item_full[items % kItems]), items / kItems & 1);
            if (!ok) break;
            const Item &x = ring[items % kItems];
            auto uniform = [](int y) { return __shfl_sync(0xffffffffu, y, 0); };
            const int t0 = uniform(x.t0), n = uniform(x.t1) - t0, end = uniform(x.end()), shared_from = max(0, uniform(x.limit) + 1);
            const int whole = shared_from / kTile - t0;      // tiles before this one have no row to clear
            const bool two = kQ == 2 && uniform(x.ntok) > a.TB;
            const int lead = two ? 0 : items & 1;   // the group of the first cache tile, which ends the item
            bool bad = false;
            ok = passed(q_full, items & 1) && passed(full + 8 * k.at, k.parity);
            if (!ok) break;
            tc::tc_fence_after();
            if (two) {   // each cache tile for both query tiles
                scores(0, 0, k.at);
                scores(1, 1, k.at);
                commit(empty + 8 * k.at);
                k.advance(2);
                if (n == 1) commit(q_free);
                for (int i = 0; i < n && ok; ++i) {
                    const bool more = i + 1 < n;
                    // The keys are waited for before the products: nothing but issues lies between those and the next
                    // scores. A wait that gave up is noted, and voted on once a tile.
                    bool fine = wait_at(full + 8 * v.at, v.parity, aborted, status);
                    if (i >= whole) bad |= clean(shared_from, end, t0 + i, v.at);
                    if (more) fine &= wait_at(full + 8 * k.at, k.parity, aborted, status);
                    const uint64_t dv = first_mn + v.at * (kTileBytes >> 4), dk = first_k + (kQ + k.at) * (kTileBytes >> 4);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint32_t d = tmem + kO0 + t * kTile, ps = tmem + kS0 + t * kTile, pp = p_parity >> t & 1;
                        if (i == 0 && (o_used >> t & 1)) fine &= wait_at(o_free + 8 * t, o_parity >> t & 1, aborted, status);
                        fine &= wait_at(p_full + 8 * t, pp, aborted, status);
                        tc::tc_fence_after();
                        if (tc::elect_one()) {
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                tc::umma_bf16_ta(d, ps + 8 * ks, dv + ks * (2048 >> 4), kIdO, i > 0 || ks > 0);
                        }
                        fine &= wait_at(p_rest + 8 * t, pp, aborted, status);
                        tc::tc_fence_after();
                        if (tc::elect_one()) {
#pragma unroll
                            for (int ks = 4; ks < 8; ++ks) tc::umma_bf16_ta(d, ps + 8 * ks, dv + ks * (2048 >> 4), kIdO, 1u);
                            if (more) {
                                const uint64_t dq = first_k + t * (kTileBytes >> 4);
#pragma unroll
                                for (int ks = 0; ks < 8; ++ks) {
                                    const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
                                    tc::umma_bf16(ps, dq + off, dk + off, kIdS, ks > 0);
                                }
                                commit_at(s_full + 8 * t);
                            } else {
                                commit_at(o_full + 8 * t);
                            }
                            if (t == 1) {
                                commit_at(empty + 8 * v.at);
                                if (more) commit_at(empty + 8 * k.at);
                                if (i + 2 == n) commit_at(q_free);
                            }
                        }
                    }
                    if (i == 0) o_used = 3, o_parity ^= 3u;
                    p_parity ^= 3u;
                    v.advance(2);
                    if (more) k.advance(2);
                    ok = __all_sync(0xffffffffu, fine) != 0;
                }
            } else {     // one query tile: the groups take the cache tiles in turn
                scores(lead, 0, k.at);
                commit(empty + 8 * k.at);
                k.advance(2);
                if (n > 1) {
                    ok = passed(full + 8 * k.at, k.parity);
                    if (!ok) break;
                    scores(lead ^ 1, 0, k.at);
                    commit(empty + 8 * k.at);
                    k.advance(2);
                }
                if (n <= 2) commit(q_free);
                for (int i = 0; i < n; ++i) {
                    const int t = (i & 1) ^ lead;
                    ok = passed(full + 8 * v.at, v.parity);
                    if (!ok) break;
                    if (i >= whole) bad |= clean(shared_from, end, t0 + i, v.at);
                    ok = products(t, v.at, i < 2, i + 2 >= n);
                    if (!ok) break;
                    commit(empty + 8 * v.at);
                    v.advance(2);
                    if (i + 2 < n) {
                        ok = passed(full + 8 * k.at, k.parity);
                        if (!ok) break;
                        scores(t, 0, k.at);
                        if (tc::elect_one()) {
                            commit_at(empty + 8 * k.at);
                            if (i + 3 == n) commit_at(q_free);
                        }
                        __syncwarp();
                        k.advance(2);
                    }
                }
            }
            if (!ok) break;
            if (tc::elect_one())
                for (int t = 0; t < 2; ++t)
                    if (two || n > 1 || t == lead) {
                        bad_values[t] = bad;
                        mbar_arrive(&bar.o_full[t]);
                    }
            last = uniform(x.last) != 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.item_empty[items % kItems]);
            ++items;
        } while (!last);
        if (tc::elect_one()) {   // products in flight end before the tensor memory is freed, whoever gave up
            tc::umma_commit(&bar.drain);
            tc::mbar_wait(&bar.drain, 0, tck::kWaitNs);
        }
        __syncwarp();
    } else if (warp < kMmaWarp && !idle) {
        // ---- softmax and results: half a row of scores a thread ----------------------------------------
        // Lanes l and l + 16 share a row: columns [0, 32) and [64, 96), or [32, 64) and [96, 128).
        const int t = warp >> 3, half = lane >> 4, r = (warp & 3) * 32 + ((warp >> 2) & 1) * 16 + (lane & 15);
        const int first_row = r & ~15;
        const uint32_t lanes = static_cast<uint32_t>(first_row) << 16;
        const uint32_t ts = tmem + kS0 + t * kTile + lanes;
        constexpr uint32_t kO = kO0 - kS0;   // from a group's S to its O
        // In one register: the parities of score tiles, of items with an O of this group and of joined items, whether an item has
        // a maximum, whether one of the warp's rows has one far from 0, and the items. What an item's rows are is read again after its tiles: registers are short in between.
        uint32_t count = 0;
        constexpr uint32_t kSeen = 1, kMine = 2, kJoined = 4, kBegun = 8, kFarRows = 16, kItem = 32;
        bool ok = true, last = false;
        do {
            ok = wait_warp(&bar.item_full[count / kItem % kItems], (count / (kItem * kItems)) & 1, aborted, status);
            if (!ok) break;
            const Item &x = ring[count / kItem % kItems];
            last = x.last;
            struct Rows {
                bool two, valid, active;   // active: a warp without rows leaves its scores as they are: rows of a product do not mix
                int tile, turn, tok, limit;
            };
            auto rows = [&]() {
                Rows y;
                y.two = kQ == 2 && x.ntok > a.TB;
                y.tile = y.two ? t : 0;
                y.turn = y.two ? 0 : t ^ (count / kItem & 1);   // of the cache tiles: 0, 2, .. (and ends the item) or 1, 3, ..
                y.tok = y.tile * a.TB + r / a.G;
                y.valid = r < a.TB * a.G && y.tok < x.ntok;
                y.active = first_row < a.TB * a.G && y.tile * a.TB + first_row / a.G < x.ntok;
                y.limit = y.valid ? x.limit + y.tok : -1;
                return y;
            };
            const Rows in = rows();
            const bool active = in.active;
            const int step = in.two ? 1 : 2, first = x.t0 + in.turn;
            // the last place seen, from the first score of this thread (a row without a token: as the first token's)
            int keep = (in.valid ? in.limit : x.limit + in.tile * a.TB) - 32 * half - first * kTile;
            const float scale = exponent_scale(a, x.h);
            float m = -INFINITY, l = 0.f;   // the maximum in units of the scores
            count &= ~(kBegun | kFarRows);
            for (int left = (x.t1 - first + step - 1) / step; left > 0; --left, keep -= step * kTile) {
                ok = wait_warp(&bar.s_full[t], count & kSeen ? 1 : 0, aborted, status);
                if (!ok) break;
                count ^= kSeen;
                tc::tc_fence_after();
                if (active) {
                    // bf16: all 64 scores in registers; e4m3, with fewer registers a thread: 32 at a time, twice
                    uint32_t s[E4M3 ? 1 : 2][32];
                    auto load = [&](int q, uint32_t (&x)[32]) {
                        tmem_ld_half_x32(ts + 64 * q, x);
                        tc::tmem_ld_wait();
                        if (keep < 64 + 31)
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (64 * q + j > keep) x[j] = __float_as_uint(-INFINITY);
                    };
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t (&y)[32] = s[E4M3 ? 0 : q];
                        load(q, y);
#pragma unroll
                        for (int j = 0; j < 32; j += 2)
                            top[(j >> 1) & 3] = fmaxf(fmaxf(top[(j >> 1) & 3], __uint_as_float(y[j])), __uint_as_float(y[j + 1]));
                    }
                    float tile_top = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    tile_top = fmaxf(tile_top, __shfl_xor_sync(0xffffffffu, tile_top, 16));
                    if (!(count & kBegun)) {
                        m = tile_top;
                        if (__any_sync(0xffffffffu, fabsf(exponent_of(m, scale)) > kFar)) count |= kFarRows;
                    } else {
                        const bool grow = tile_top > m && !((tile_top - m) * scale <= kRescale);
                        if (__any_sync(0xffffffffu, grow)) {
                            const float f = !grow ? 1.f : m == -INFINITY ? 0.f : tc::ex2((m - tile_top) * scale);
                            if (grow) m = tile_top;
                            if (__any_sync(0xffffffffu, fabsf(exponent_of(m, scale)) > kFar)) count |= kFarRows;
                            l *= f;
#pragma unroll 1
                            for (int q = 0; q < 8; ++q) {   // few at a time: the scores fill the registers
                                uint32_t o[8];
                                const uint32_t at = ts + kO + (q >> 2) * 64 + (q & 3) * 8;
                                tmem_ld_half_x8(at, o);
                                tc::tmem_ld_wait();
#pragma unroll
                                for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tmem_st_half_x8(at, o);
                            }
                        }
                    }
                    // P = 2^(c s - c m) by multiply-adds, whose exponents all have the one rounding of c m. It cancels in P over its sum,
                    // but not where c m is so large that it is a factor out of range: s - m then comes first (exact near the maximum).
                    const float mc = exponent_of(m, scale);
                    uint64_t sum2[2] = {0, 0};   // pairs of zeros
                    const uint64_t scale2 = tc::pair(scale, scale);
                    auto weights = [&](int q, const uint32_t (&z)[32], uint64_t minus) {
                        uint32_t pk[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float2 y = tc::unpair(tc::fma2(
                                tc::pair(__uint_as_float(z[2 * j]), __uint_as_float(z[2 * j + 1])), scale2, minus));
                            const float e0 = tc::ex2(y.x), e1 = tc::ex2(y.y);
                            sum2[j & 1] = tc::add2(sum2[j & 1], tc::pair(e0, e1));
                            pk[j] = float2_to_bf16x2(e0, e1);
                        }
                        tmem_st_16x32bx2_x16<16>(ts + 32 * q, pk);   // P over the left half of S, which both lanes have read
                        if (q == 0) {
                            tc::tmem_st_wait();
                            tc::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bar.p_full[t]);
                        }
                    };
                    if (count & kFarRows) {
                        const bool far = fabsf(mc) > kFar;
                        const float low = far ? 0.f : -mc, shift = far ? m : 0.f;
#pragma unroll 1
                        for (int q = 0; q < 2; ++q) {   // the scores once more: held on from above they would cost the usual way registers
                            uint32_t z[32];
                            load(q, z);
#pragma unroll
                            for (int j = 0; j < 32; ++j) z[j] = __float_as_uint(__uint_as_float(z[j]) - shift);
                            weights(q, z, tc::pair(low, low));
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            if (E4M3) load(q, s[0]);
                            weights(q, s[E4M3 ? 0 : q], tc::pair(-mc, -mc));
                        }
                    }
                    const float2 even = tc::unpair(sum2[0]), odd = tc::unpair(sum2[1]);
                    l += (even.x + even.y) + (odd.x + odd.y);
                    tc::tmem_st_wait();
                }
                count |= kBegun;
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (!active) mbar_arrive(&bar.p_full[t]);
                    mbar_arrive(&bar.p_rest[t]);
                }
            }
            if (!ok) break;
            const auto [two, valid, busy, my_tile, turn, my_tok, limit] = rows();
            const int n = x.t1 - x.t0;
            if (busy) l += __shfl_xor_sync(0xffffffffu, l, 16);
            const bool worked = turn < n;           // this group has an O
            if (worked) {
                ok = wait_warp(&bar.o_full[t], count & kMine ? 1 : 0, aborted, status);
                if (!ok) break;
                count ^= kMine;
                tc::tc_fence_after();
            }
            const bool join = !two && n > 1;        // both groups have an O of the same rows
            float f0 = 1.f, f1 = 0.f;
            if (join && turn == 1) {
                if (lane < 16) other[r] = make_float2(m, l);
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.join);
            } else if (join) {
                ok = wait_warp(&bar.join, count & kJoined ? 1 : 0, aborted, status);
                if (!ok) break;
                tc::tc_fence_after();
                const float2 y = other[r];
                const float top = fmaxf(m, y.x);
                f0 = part_factor(m, top, scale);
                f1 = part_factor(y.x, top, scale);
                l = l * f0 + y.y * f1;
                m = top;
            }
            if (busy && turn == 0) {
                const int slot = x.slot;
                const bool whole = slot < 0, some = limit >= 0;   // some: the row sees a place
                uint32_t dims[4] = {0, 0, 0, 0};
                if (bad_values[t] && valid) bad_dimensions(c, x.n, x.h, x.limit, limit, dims);
                const float vs = c.v_scale ? kv::load(c.v_scale + x.h) : 1.f;
                const float inv = whole ? vs / l : 1.f;
                const int64_t row = (x.row + my_tok) * (a.G * c.H) + x.h * a.G + r % a.G;
                const int64_t prow = static_cast<int64_t>(slot) * kRows + my_tile * kTile + r;
                f0 *= inv;
                f1 *= inv;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int col = (q >> 1) * 64 + (q & 1) * 16, mycol = col + 32 * half;
                    uint32_t o[16];
                    __syncwarp();
                    tc::tmem_ld_16x32bx2_x16(ts + kO + col, o);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f0);
                    if (join) {
                        uint32_t o1[16];
                        tc::tmem_ld_16x32bx2_x16(ts + kO + (t ? -kTile : kTile) + col, o1);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            o[j] = __float_as_uint(fmaf(__uint_as_float(o1[j]), f1, __uint_as_float(o[j])));
                    }
                    const uint32_t bits = (q >> 1 ? (half ? dims[3] : dims[2]) : half ? dims[1] : dims[0]) >> ((q & 1) * 16);
                    if (bits & 0xffffu)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (bits >> j & 1) o[j] = 0x7fc00000u;
                    if (valid && whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.o + row * kD + mycol);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                y[e] = some ? float2_to_bf16x2(__uint_as_float(o[8 * j + 2 * e]), __uint_as_float(o[8 * j + 2 * e + 1]))
                                            : 0u;
                            dst[j] = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    } else if (valid) {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.part_o + prow * kD + mycol);
#pragma unroll
                        for (int j = 0; j < 4; ++j) dst[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    }
                }
                if (valid && half == 0) {
                    if (!whole) {
                        a.part_ml[prow] = make_float2(m, l);
                    } else {
                        if (a.lse) a.lse[row] = some ? (exponent_of(m, scale) + log2f(l)) * kLn2 : -INFINITY;
                        if (a.stats) a.stats[row] = score_lse(m, l, scale);
                    }
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (worked && !(join && turn == 1)) mbar_arrive(&bar.o_free[t]);
                if (join && turn == 0) mbar_arrive(&bar.o_free[t ^ 1]);   // read here
                mbar_arrive(&bar.item_empty[count / kItem % kItems]);
            }
            if (join) count ^= kJoined;
            count += kItem;
        } while (!last);
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// ---- joins the partial results of units that several CTAs share -----------------------------------

// Few rows (one token on a long cache that all CTAs share, in many parts): a block has 8 rows, and four warps a quarter of
// a row's parts each, whose loads would follow one another in one. Otherwise a warp has two rows, mostly in two to four
// parts, whose statistics and values it loads at once. 16 rows of 32 parts take 13 us the second way and 9 the first, units
// of 256 rows the other way round 98 us and 20. Of these the 40 MB of a chunk of 4096 tokens on 32768 places take 16 us
// (26 with a row a warp and one load after the other, 19 with four rows).
constexpr int kJoinWarps = 8, kJoinEach = 2;   // of a block, rows of a warp

template <int kJoinSplit>
__host__ __device__ constexpr int join_rows() { return kJoinSplit > 1 ? kJoinWarps : kJoinEach * kJoinWarps; }   // of a block

// The results of row rr of query tile t: acc / total, its maximum, the factor of its scores.
__device__ __forceinline__ void joined_row(const AttendArgs &a, const JoinUnit &x, int tok, int rr, int lane, float4 acc, float total,
                                           float m, float scale) {
    const bool some = x.limit + tok >= 0;
    const float vs = a.c.v_scale ? kv::load(a.c.v_scale + x.h) : 1.f, inv = vs / total;
    const int64_t out = (x.row + tok) * (a.G * a.c.H) + x.h * a.G + rr % a.G;
    *reinterpret_cast<uint2 *>(a.o + out * kD + lane * 4) =
        some ? make_uint2(float2_to_bf16x2(acc.x * inv, acc.y * inv), float2_to_bf16x2(acc.z * inv, acc.w * inv)) : make_uint2(0, 0);
    if (lane == 0) {
        if (a.lse) a.lse[out] = some ? (exponent_of(m, scale) + log2f(total)) * kLn2 : -INFINITY;
        if (a.stats) a.stats[out] = score_lse(m, total, scale);
    }
}

__device__ __forceinline__ void add_part(float4 &acc, float w, const float4 &v) {
    acc.x += w * v.x;
    acc.y += w * v.y;
    acc.z += w * v.z;
    acc.w += w * v.w;
}

// The sum over parts s, s + split, .. of a row, by a warp; `most`: the maximum over all parts.
__device__ __forceinline__ void join_parts(const AttendArgs &a, int cta, int parts, int row, int s, int split, int lane, float scale,
                                           float4 *acc, float *total, float *most) {
    float top = -INFINITY;
    for (int p = lane; p < parts; p += 32) top = fmaxf(top, a.part_ml[part_slot(cta, p) * kRows + row].x);
    for (int o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    *most = top;
    *total = 0.f;
    *acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = s; p0 < parts; p0 += 32 * split) {   // lane l has the statistics of the l-th of these
        float f = 0.f, l = 0.f;
        const int mine = p0 + lane * split;
        if (mine < parts) {
            const float2 ml = a.part_ml[part_slot(cta, mine) * kRows + row];
            f = part_factor(ml.x, top, scale);
            l = ml.y * f;
        }
        for (int o = 16; o > 0; o /= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
        *total += l;
        const int here = min(32, (parts - p0 + split - 1) / split);
#pragma unroll 8
        for (int i = 0; i < here; ++i)
            add_part(*acc, __shfl_sync(0xffffffffu, f, i),
                     *reinterpret_cast<const float4 *>(a.part_o + (part_slot(cta, p0 + i * split) * kRows + row) * kD + lane * 4));
    }
}

// The token of a unit's row, -1: it has none.
__device__ __forceinline__ int token_of(const AttendArgs &a, const JoinUnit &x, int row) {
    const int rr = row % kTile, tok = row / kTile * a.TB + rr / a.G;
    return rr < a.TB * a.G && tok < x.ntok ? tok : -1;
}

// Rows [row0, row0 + kJoinEach) of a unit in kParts parts, by a warp that has all of their loads in flight.
template <int kParts>
__device__ __forceinline__ void join_rows_at_once(const AttendArgs &a, const JoinUnit &x, int cta, int row0, int lane, float scale) {
    float2 ml[kJoinEach][kParts];
    float4 v[kJoinEach][kParts];
#pragma unroll
    for (int e = 0; e < kJoinEach; ++e)
        if (token_of(a, x, row0 + e) >= 0)
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                const int64_t at = part_slot(cta, p) * kRows + row0 + e;
                ml[e][p] = a.part_ml[at];
                v[e][p] = *reinterpret_cast<const float4 *>(a.part_o + at * kD + lane * 4);
            }
#pragma unroll
    for (int e = 0; e < kJoinEach; ++e) {
        const int tok = token_of(a, x, row0 + e);
        if (tok < 0) continue;
        float top = -INFINITY, total = 0.f;
#pragma unroll
        for (int p = 0; p < kParts; ++p) top = fmaxf(top, ml[e][p].x);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
            const float f = part_factor(ml[e][p].x, top, scale);
            total += ml[e][p].y * f;
            add_part(acc, f, v[e][p]);
        }
        joined_row(a, x, tok, (row0 + e) % kTile, lane, acc, total, top, scale);
    }
}

template <int kJoinSplit>
__global__ void __launch_bounds__(32 * kJoinWarps * kJoinSplit) paged_combine_kernel(const AttendArgs a) {
    dependent_start();
    const int cta = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const JoinUnit x = static_cast<const JoinUnit *>(a.joins)[cta];
    if (x.parts == 0) return;
    const float scale = exponent_scale(a, x.h);
    if constexpr (kJoinSplit > 1) {
        __shared__ float4 sums[kJoinWarps][kJoinSplit][32];
        __shared__ float totals[kJoinWarps][kJoinSplit];
        const int k = warp / kJoinSplit, s = warp % kJoinSplit, row = blockIdx.y * join_rows<kJoinSplit>() + k, tok = token_of(a, x, row);
        float top = -INFINITY;
        if (tok >= 0) {
            float4 acc;
            float total;
            join_parts(a, cta, x.parts, row, s, kJoinSplit, lane, scale, &acc, &total, &top);
            sums[k][s][lane] = acc;
            if (lane == 0) totals[k][s] = total;
        }
        __syncthreads();
        if (tok < 0 || s != 0) return;
        float total = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kJoinSplit; ++i) add_part(acc, 1.f, sums[k][i][lane]), total += totals[k][i];
        joined_row(a, x, tok, row % kTile, lane, acc, total, top, scale);
    } else {
        const int row0 = blockIdx.y * join_rows<1>() + warp * kJoinEach;
        if (x.parts == 2) return join_rows_at_once<2>(a, x, cta, row0, lane, scale);
        if (x.parts == 3) return join_rows_at_once<3>(a, x, cta, row0, lane, scale);
        if (x.parts == 4) return join_rows_at_once<4>(a, x, cta, row0, lane, scale);
        for (int row = row0; row < row0 + kJoinEach; ++row) {
            const int tok = token_of(a, x, row);
            if (tok < 0) continue;
            float4 acc;
            float total, top;
            join_parts(a, cta, x.parts, row, 0, 1, lane, scale, &acc, &total, &top);
            joined_row(a, x, tok, row % kTile, lane, acc, total, top, scale);
        }
    }
}

// ---- running sums of tiles for batches that are too large for each CTA to take them ------------------

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int64_t block_inclusive(int64_t x, int64_t *warp_sums, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    *total = all;
    return before + x;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const KvArgs c, int64_t *attend_start, int64_t *weight_start,
                                                                  int block, int TB) {
    __shared__ int64_t warp_sums[kPlanThreads / 32];
    dependent_start();
    const AttendWork aw{block};
    const WeightWork ww{TB};
    int64_t a_sum = 0, w_sum = 0;
    for (int64_t b = 0; b < c.N; b += kPlanThreads) {
        const int64_t n = b + threadIdx.x;
        int64_t at = 0, wt = 0, total;
        if (n < c.N) {
            const kv::Request r = kv::request(c, n);
            at = tiles_of(aw, r.count, r.len);
            wt = tiles_of(ww, r.count, r.len);
        }
        const int64_t a_end = block_inclusive(at, warp_sums, &total);
        if (n < c.N) attend_start[n + 1] = a_sum + a_end;
        a_sum += total;
        if (weight_start) {
            const int64_t w_end = block_inclusive(wt, warp_sums, &total);
            if (n < c.N) weight_start[n + 1] = w_sum + w_end;
            w_sum += total;
        }
    }
    if (threadIdx.x == 0) {
        attend_start[0] = 0;
        if (weight_start) weight_start[0] = 0;
    }
}

size_t aligned(size_t bytes) { return (bytes + 255) & ~size_t(255); }

// Each CTA takes the running sums itself where there are few requests and 32 bits hold any sum of tiles.
bool near_starts(const KvArgs &c, int G) {
    const int64_t tiles = c.W * c.S / kTile + 1, block = kTile / G;
    return c.N <= kInline && (c.T / block + c.N) < (int64_t(1) << 31) / tiles;
}

size_t lay_out(const KvArgs &c, int G, bool accumulate, int ctas, char *ws, AttendArgs *a) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *r = ws + at;
        at += aligned(bytes);
        return r;
    };
    const bool near = near_starts(c, G);
    const size_t n = (static_cast<size_t>(c.N) + 1) * 8, slots = static_cast<size_t>(ctas) * 2;
    a->attend_start = near ? nullptr : reinterpret_cast<int64_t *>(take(n));
    a->weight_start = near || !accumulate ? nullptr : reinterpret_cast<int64_t *>(take(n));
    a->joins = take(static_cast<size_t>(ctas) * sizeof(JoinUnit));
    a->weight_joins = accumulate ? take(static_cast<size_t>(ctas) * 16) : nullptr;
    a->part_o = reinterpret_cast<float *>(take(slots * kRows * kD * 4));
    a->part_ml = reinterpret_cast<float2 *>(take(slots * kRows * 8));
    a->stats = accumulate ? reinterpret_cast<float *>(take(static_cast<size_t>(c.T) * G * c.H * 4)) : nullptr;
    a->part_w = accumulate ? reinterpret_cast<float *>(take(slots * kTile * 4)) : nullptr;
    return at;
}
}  // namespace

size_t paged_attention_scratch(const KvArgs &c, int G, bool accumulate, int sm_count) {
    AttendArgs a;
    return lay_out(c, G, accumulate, sm_count, nullptr, &a);
}

cudaError_t setup_paged_attention_kernel() {
    cudaError_t e = cudaSuccess;
    auto allow = [&](const void *kernel, size_t bytes) {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    };
    allow(reinterpret_cast<const void *>(paged_attention_kernel<false, 1, false>), Shape<false, 1, false>::kAlloc);
    allow(reinterpret_cast<const void *>(paged_attention_kernel<false, 1, true>), Shape<false, 1, true>::kAlloc);
    allow(reinterpret_cast<const void *>(paged_attention_kernel<false, 2, false>), Shape<false, 2, false>::kAlloc);
    allow(reinterpret_cast<const void *>(paged_attention_kernel<false, 2, true>), Shape<false, 2, true>::kAlloc);
    allow(reinterpret_cast<const void *>(paged_attention_kernel<true, 1, false>), Shape<true, 1, false>::kAlloc);
    allow(reinterpret_cast<const void *>(paged_attention_kernel<true, 1, true>), Shape<true, 1, true>::kAlloc);
    allow(reinterpret_cast<const void *>(paged_attention_kernel<true, 2, false>), Shape<true, 2, false>::kAlloc);
    allow(reinterpret_cast<const void *>(paged_attention_kernel<true, 2, true>), Shape<true, 2, true>::kAlloc);
    return e == cudaSuccess ? setup_paged_weights_kernel() : e;
}

cudaError_t launch_paged_attention(const KvArgs &c, const void *q, int64_t q_stride, float scale, void *o, float *lse,
                                   bool accumulate, int G, void *ws, int sm_count, cudaStream_t st) {
    AttendArgs a;
    lay_out(c, G, accumulate, sm_count, static_cast<char *>(ws), &a);
    a.c = c;
    a.o = static_cast<uint16_t *>(o);
    a.lse = lse;
    a.scale = scale;
    a.G = G;
    a.TB = kTile / G;
    // Units of two query tiles read the cache half as often; units of one leave their room to cache tiles in flight. With
    // more than one tile of tokens a request on average the former count: a chunk of 4096 tokens has each cache tile read
    // by half as many units, where 256 requests of one token, which fill a part of one tile, went from 350 to 340 us when
    // the second query tile's room became a stage.
    const int Q = c.T > c.N * a.TB ? 2 : 1;
    // A warp issues its lanes' boxes one after another, and the 16 of a bf16 tile in pages of 16 places (8 of an e4m3 tile) bound the
    // kernel: a second warp then loads the values. Pages of 16 and the two warps: a chunk of 2048 tokens on 16384 places
    // 456 -> 348 us, 128 requests of one token on up to 12288 places 207 -> 181 (e4m3 195 -> 151), 256 on up to 1000 places and 8
    // key/value heads 161 -> 135, but on up to 120 places 55 -> 62, as the values wait for the item. In pages of 32 the same
    // chunk 352 -> 354 and the requests 172 -> 173 (e4m3 160 -> 150): one warp.
    const bool split = c.S < 32;
    Maps maps;
    cudaError_t e;
    {
        const cuuint64_t dims[3] = {kD, static_cast<cuuint64_t>(G) * c.H, static_cast<cuuint64_t>(c.T)};
        const cuuint64_t strides[2] = {kD * 2, static_cast<cuuint64_t>(q_stride) * 2};
        const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(a.TB)};
        e = tck::encode_tiled(&maps.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
        if (e != cudaSuccess) return e;
    }
    {
        const cuuint64_t dims[3] = {kD, static_cast<cuuint64_t>(c.S), static_cast<cuuint64_t>(c.P) * c.H};
        const cuuint64_t row = c.e4m3 ? kD : 2 * kD, strides[2] = {row, static_cast<cuuint64_t>(c.S) * row};
        const cuuint32_t box[3] = {static_cast<cuuint32_t>(c.e4m3 ? kD : 64), static_cast<cuuint32_t>(c.S < kTile ? c.S : kTile), 1};
        const CUtensorMapDataType type = c.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        const CUtensorMapSwizzle swizzle = c.e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
        e = tck::encode_tiled(&maps.k, type, 3, c.k, dims, strides, box, swizzle);
        if (e == cudaSuccess) e = tck::encode_tiled(&maps.v, type, 3, c.v, dims, strides, box, swizzle);
        if (e != cudaSuccess) return e;
    }
    if (a.attend_start) {
        LaunchTimer timer(kKPagedPlan, st);
        e = launch_dependent(paged_plan_kernel, dim3(1), kPlanThreads, st, c, const_cast<int64_t *>(a.attend_start),
                             const_cast<int64_t *>(a.weight_start), Q * a.TB, a.TB);
        if (e != cudaSuccess) return e;
    }
    {
        LaunchTimer timer(kKPagedAttention, st);
        auto launch = [&](auto kernel, auto shape) {
            using S = decltype(shape);
            return launch_dependent_cluster(kernel, dim3(sm_count), 0, S::kThreads, S::kAlloc, st, a, maps);
        };
        auto launch_split = [&](auto e4m3, auto q) {
            constexpr bool kE = decltype(e4m3)::value;
            constexpr int kQ = decltype(q)::value;
            return split ? launch(paged_attention_kernel<kE, kQ, true>, Shape<kE, kQ, true>{})
                         : launch(paged_attention_kernel<kE, kQ, false>, Shape<kE, kQ, false>{});
        };
        using std::integral_constant;
        const integral_constant<int, 1> one;
        const integral_constant<int, 2> two;
        e = c.e4m3 ? (Q == 2 ? launch_split(std::true_type{}, two) : launch_split(std::true_type{}, one))
                   : (Q == 2 ? launch_split(std::false_type{}, two) : launch_split(std::false_type{}, one));
        if (e != cudaSuccess) return e;
    }
    {
        LaunchTimer timer(kKPagedCombine, st);
        // rows that a unit can have
        const int64_t tokens = c.cu ? c.T : c.T_row;
        const int rows = tokens <= a.TB ? static_cast<int>(tokens) * G : Q * kTile;
        auto launch = [&](auto kernel, int block_rows, int threads) {
            return launch_dependent(kernel, dim3(sm_count, (rows + block_rows - 1) / block_rows), threads, st, a);
        };
        e = rows <= 32 ? launch(paged_combine_kernel<4>, join_rows<4>(), 32 * kJoinWarps * 4)
                       : launch(paged_combine_kernel<1>, join_rows<1>(), 32 * kJoinWarps);
        if (e != cudaSuccess || !accumulate) return e;
    }
    return launch_paged_weights(a, maps, sm_count, st);
}

}  // namespace sala

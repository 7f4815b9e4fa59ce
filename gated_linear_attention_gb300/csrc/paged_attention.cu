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
// One persistent CTA per SM. A plan kernel lists the units with the running sum of their cache tiles; every CTA
// takes an equal share of all tiles, so a unit may be shared by several CTAs, which leave partial results
// (O, m, sum) that a last kernel joins. This serves one token on a long cache and a full batch alike.
//
// Roles: a warpgroup per query tile (a thread holds a row of scores: no shuffles), one warp issues the products,
// the others load. While one tile's scores are in its warpgroup, the tensor core works on the other tile.
// bf16 pages come by TMA, a page (and half of the dimensions) a box; e4m3 pages go through the registers of three
// warps, which widen them (exactly) to bf16.
//
// What is masked never enters: scores are replaced, not added to, and V is cleared in the rows behind the unit's
// last place (0 times a NaN there would be NaN). Rows of V that some tokens of the unit see and others do not are
// searched for infinities and NaN, which are cleared and put into the results that see them at the end.
#include "chunk_tc.cuh"
#include "kv_cache.cuh"

namespace sala {
namespace {

using tc::mbar_arrive;
using tck::wait_or_abort;

constexpr int kTile = 128;                       // rows of a query tile, places of a cache tile
constexpr uint32_t kHalf = kTile * 128;          // bytes of [128 rows x 64 bf16], 128-byte swizzle
constexpr uint32_t kTileBytes = 2 * kHalf;
constexpr int kStages = 5;
constexpr int kRows = 2 * kTile;                 // rows of a unit
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kConvertWarps = 3;                 // loading warps of an e4m3 cache
constexpr uint32_t kSmemBytes = (2 + kStages) * kTileBytes;
constexpr uint32_t kSmemAlloc = kSmemBytes + 1024;   // aligned to the swizzle's 1024 bytes
constexpr uint32_t kS0 = 0, kO0 = 256;           // tensor memory columns: S (and P) of the tiles, then O
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.f;                  // growth of the maximum (log2) that rescales O
constexpr uint32_t kIdS = tc::idesc_bf16_f32(128, 128, 0, 0), kIdO = tc::idesc_bf16_f32(128, 128, 0, 1);

constexpr int threads_of(bool e4m3) { return 32 * (kLoadWarp + (e4m3 ? kConvertWarps : 1)); }

// One unit: tokens [tok, tok + ntok) of request n, the first at packed token `row` and place `limit`
// (negative: it sees nothing), with `tiles` >= 1 cache tiles.
struct alignas(16) Unit {
    int64_t row;
    int32_t n, ntok, limit, tiles, pad[2];
};
static_assert(sizeof(Unit) == 32, "two 16-byte loads");

struct Plan {
    int64_t *total;      // [0] units, [1] cache tiles of a key/value head
    int64_t most;        // units that the arrays hold: malformed offsets may give requests that overlap
    int64_t *start;      // [units + 1] running sum of the tiles
    Unit *units;
    int32_t *first;      // [N] first unit of each request
    float *part_o;       // [2 * CTAs, kRows, 128] partial O
    float2 *part_ml;     // [2 * CTAs, kRows] its maximum (log2) and sum
};

struct AttendArgs {
    KvArgs c;
    Plan p;
    uint16_t *o;
    float *lse;
    float scale;
    int G, TB;           // query heads on a key/value head, tokens of a query tile
};

__host__ __device__ inline int tokens_of_tile(int G) { return kTile / G; }

// ---- plan -------------------------------------------------------------------------------------

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

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const KvArgs c, const Plan p, int tokens) {
    __shared__ int64_t warp_sums[kPlanThreads / 32];
    dependent_start();
    int64_t units = 0;
    for (int64_t b = 0; b < c.N; b += kPlanThreads) {
        const int64_t n = b + threadIdx.x;
        const int64_t mine = n < c.N ? (kv::request(c, n).count + tokens - 1) / tokens : 0;
        int64_t sum;
        const int64_t end = block_inclusive(mine, warp_sums, &sum);
        if (n < c.N) p.first[n] = static_cast<int32_t>(units + end - mine);
        units += sum;
    }
    units = min(units, p.most);
    __syncthreads();
    int64_t tiles = 0;
    for (int64_t b = 0; b < units; b += kPlanThreads) {
        const int64_t u = b + threadIdx.x;
        int64_t mine = 0;
        if (u < units) {
            int64_t lo = 0, hi = c.N;   // the last request whose first unit is at most u
            while (hi - lo > 1) {
                const int64_t mid = (lo + hi) / 2;
                if (p.first[mid] <= u) lo = mid;
                else hi = mid;
            }
            const kv::Request r = kv::request(c, lo);
            Unit x;
            const int64_t tok = (u - p.first[lo]) * tokens;
            x.row = r.first + tok;
            x.n = static_cast<int32_t>(lo);
            x.ntok = static_cast<int32_t>(min(static_cast<int64_t>(tokens), r.count - tok));
            x.limit = static_cast<int32_t>(r.len - r.count + tok);
            x.tiles = max(1, (x.limit + x.ntok + kTile - 1) / kTile);
            x.pad[0] = x.pad[1] = 0;
            p.units[u] = x;
            mine = x.tiles;
        }
        int64_t sum;
        const int64_t end = block_inclusive(mine, warp_sums, &sum);
        if (u < units) p.start[u] = tiles + end - mine;
        tiles += sum;
    }
    if (threadIdx.x == 0) {
        p.start[units] = tiles;
        p.total[0] = units;
        p.total[1] = tiles;
    }
}

// ---- work of a CTA ------------------------------------------------------------------------------

// A CTA's range of the flattened tiles (key/value head outermost). With fewer tiles than CTAs the first
// CTAs get one each, so that no range among those that share a unit is empty.
__device__ __forceinline__ int64_t range_begin(int64_t tiles, int64_t cta, int64_t ctas) {
    if (tiles <= ctas) return min(cta, tiles);
    return tiles / ctas * cta + tiles % ctas * cta / ctas;
}

// The unit that holds tile `at` of a key/value head.
__device__ __forceinline__ int64_t unit_at(const Plan &p, int64_t units, int64_t at) {
    int64_t lo = 0, hi = units;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (p.start[mid] <= at) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Walks the items of a CTA: (key/value head, unit, a range of its tiles).
struct Walk {
    int64_t pos, end, units, u;
    int h, t0, t1;       // tiles [t0, t1) of the unit
    int slot;            // where a partial result goes, -1: the item is the whole unit
    Unit x;

    __device__ __forceinline__ void load(const Plan &p, int64_t per_head, int64_t begin, int cta) {
        x = p.units[u];
        const int64_t at = per_head * h + p.start[u];
        t0 = static_cast<int>(pos - at);
        t1 = static_cast<int>(min(static_cast<int64_t>(x.tiles), end - at));
        slot = t0 == 0 && t1 == x.tiles ? -1 : 2 * cta + (begin <= at ? 1 : 0);
    }
    __device__ __forceinline__ bool next(const Plan &p, int64_t per_head, int64_t begin, int cta) {
        pos += t1 - t0;
        if (pos >= end) return false;
        if (++u == units) u = 0, ++h;
        load(p, per_head, begin, cta);
        return true;
    }
};

struct Barriers {
    uint64_t full[kStages], empty[kStages];     // cache tiles
    uint64_t q_full, q_free;
    uint64_t s_full[2], p_full[2], o_full[2], o_free[2];
    uint64_t drain;
};

// Element offset in bytes of 16-byte piece `piece` (of 16) of a row in a tile.
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
    return (piece >> 3) * kHalf + tck::sw(row, piece & 7);
}

__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
    return tc::smem_desc_sw128(0, 16, 1024) | ((addr >> 4) & 0x3FFFu);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
    return tc::smem_desc_sw128(0, kHalf, 1024) | ((addr >> 4) & 0x3FFFu);
}

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

template <bool E4M3>
__global__ void __launch_bounds__(threads_of(E4M3), 1)
    paged_attention_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Barriers bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, bad_values[2];
    __shared__ int64_t first_unit;
    const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *const smem = smem_raw + (base - tc::smem_u32(smem_raw));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const KvArgs &c = a.c;

    if (warp == kMmaWarp) {
        tc::tmem_alloc(&tmem_slot, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&bar.full[i], E4M3 ? kConvertWarps : 1);
            tc::mbar_init(&bar.empty[i], 1);
        }
        tc::mbar_init(&bar.q_full, 1);
        tc::mbar_init(&bar.q_free, 1);
        for (int t = 0; t < 2; ++t) {
            tc::mbar_init(&bar.s_full[t], 1);
            tc::mbar_init(&bar.p_full[t], 4);
            tc::mbar_init(&bar.o_full[t], 2);
            tc::mbar_init(&bar.o_free[t], 4);
        }
        tc::mbar_init(&bar.drain, 1);
        tc::fence_barrier_init();
        abort_flag = 0;
    }
    dependent_start();
    const int64_t units = a.p.total[0], per_head = a.p.total[1], all = per_head * c.H;
    Walk w;
    w.units = units;
    w.pos = range_begin(all, blockIdx.x, gridDim.x);
    w.end = range_begin(all, blockIdx.x + 1, gridDim.x);
    const int64_t begin = w.pos;
    const bool idle = w.pos >= w.end;
    w.h = idle ? 0 : static_cast<int>(w.pos / per_head);
    if (threadIdx.x == 0 && !idle) first_unit = unit_at(a.p, units, w.pos - per_head * w.h);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    volatile int *const aborted = &abort_flag;
    int *const status = c.status;
    const int cta = blockIdx.x;
    if (!idle) {
        w.u = first_unit;
        w.load(a.p, per_head, begin, cta);
    }

    if (!idle && warp >= kLoadWarp) {
        // ---- loads: Q of each item, then K and V of each cache tile -----------------------------
        const int lw = warp - kLoadWarp;
        uint32_t it = 0, items = 0, q_issued = 0;   // cache tiles and items so far
        const int S = c.S, box = min(S, kTile), boxes = kTile / box;
        bool ok = true;
        do {
            const int end = max(0, w.x.limit + w.x.ntok);
            const int nt = w.x.ntok > a.TB ? 2 : 1;
            auto load_q = [&]() {
                if (lw == 0) {
                    if (items > 0 && !wait_or_abort(&bar.q_free, (items - 1) & 1, aborted, status)) return false;
                    if (lane == 0) {
                        tc::mbar_arrive_expect_tx(&bar.q_full, nt * 2 * static_cast<uint32_t>(a.TB * a.G) * 128u);
                        for (int t = 0; t < nt; ++t)
                            for (int half = 0; half < 2; ++half)
                                tc::tma_load_3d(smem + t * kTileBytes + half * kHalf, &map_q, half * 64, w.h * a.G,
                                                static_cast<int>(w.x.row) + t * a.TB, &bar.q_full);
                    }
                    ++q_issued;
                    __syncwarp();
                }
                return true;
            };
            if constexpr (!E4M3) {
                // lane l: box l / 2 of the tile, half l % 2 of the dimensions; pages of the next tile are looked up ahead
                const int bx = lane >> 1, half = lane & 1;
                auto lookup = [&](int tile) {
                    const int place = tile * kTile + bx * box;
                    return tile < w.t1 && bx < boxes && place < end ? kv::page_of(c, w.x.n, place) : -2;
                };
                int page = lookup(w.t0);
                for (int i = w.t0; i < w.t1 && ok; ++i) {
                    const int here = page;
                    page = lookup(i + 1);
                    const bool mine = here != -2;
                    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine)) * static_cast<uint32_t>(box) * 128u;
                    for (int kv = 0; kv < 2 && ok; ++kv, ++it) {
                        const int st = it % kStages;
                        if (it >= kStages && !wait_or_abort(&bar.empty[st], (it / kStages - 1) & 1, aborted, status)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) {
                            if (bytes) tc::mbar_arrive_expect_tx(&bar.full[st], bytes);
                            else mbar_arrive(&bar.full[st]);
                        }
                        __syncwarp();
                        if (mine)
                            tc::tma_load_3d(smem + (2 + st) * kTileBytes + half * kHalf + bx * box * 128, kv ? &map_v : &map_k,
                                            half * 64, S > kTile ? (i & 1) * kTile : 0, (here < 0 ? 0 : here) * c.H + w.h,
                                            &bar.full[st]);
                        __syncwarp();
                        if (i == w.t0 && kv == 0) ok = load_q();   // behind the first K: its buffer may still be in use
                    }
                }
            } else {
                constexpr int kEach = (1024 + 32 * kConvertWarps - 1) / (32 * kConvertWarps);
                const int id = lw * 32 + lane;
                uint4 next[kEach];
                auto fetch = [&](int tile, bool values) {
#pragma unroll
                    for (int e = 0; e < kEach; ++e) {
                        const int piece = id + e * 32 * kConvertWarps, place = tile * kTile + (piece >> 3);
                        next[e] = make_uint4(0, 0, 0, 0);
                        if (piece < 1024 && tile < w.t1 && place < end) {
                            const int page = kv::page_of(c, w.x.n, place);
                            if (page >= 0)
                                next[e] = __ldg(reinterpret_cast<const uint4 *>((values ? c.v : c.k) +
                                                                                kv::row_of(c, page, w.h, place) * kD) + (piece & 7));
                        }
                    }
                };
                fetch(w.t0, false);
                for (int i = w.t0; i < w.t1 && ok; ++i)
                    for (int kv = 0; kv < 2; ++kv, ++it) {
                        const int st = it % kStages;
                        uint4 cur[kEach];
#pragma unroll
                        for (int e = 0; e < kEach; ++e) cur[e] = next[e];
                        fetch(kv ? i + 1 : i, kv == 0);
                        if (it >= kStages && !wait_or_abort(&bar.empty[st], (it / kStages - 1) & 1, aborted, status)) {
                            ok = false;
                            break;
                        }
                        uint8_t *dst = smem + (2 + st) * kTileBytes;
#pragma unroll
                        for (int e = 0; e < kEach; ++e) {
                            const int piece = id + e * 32 * kConvertWarps;
                            if (piece >= 1024) continue;
                            const uint32_t in[4] = {cur[e].x, cur[e].y, cur[e].z, cur[e].w};
                            uint32_t out[8];
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const float2 lo = kv::e4m3x2_to_float2(in[q] & 0xffffu), hi = kv::e4m3x2_to_float2(in[q] >> 16);
                                out[2 * q] = float2_to_bf16x2(lo.x, lo.y);
                                out[2 * q + 1] = float2_to_bf16x2(hi.x, hi.y);
                            }
                            const int row = piece >> 3, p16 = (piece & 7) * 2;
                            *reinterpret_cast<uint4 *>(dst + piece_at(row, p16)) = make_uint4(out[0], out[1], out[2], out[3]);
                            *reinterpret_cast<uint4 *>(dst + piece_at(row, p16 + 1)) = make_uint4(out[4], out[5], out[6], out[7]);
                        }
                        tc::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.full[st]);
                        if (i == w.t0 && kv == 0 && !load_q()) {
                            ok = false;
                            break;
                        }
                    }
            }
            ++items;
        } while (ok && w.next(a.p, per_head, begin, cta));
        if (!ok) {   // copies in flight land before the CTA ends
            if (q_issued) tc::mbar_wait(&bar.q_full, (q_issued - 1) & 1, tck::kWaitNs);
            if (!E4M3)
                for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
                    tc::mbar_wait(&bar.full[j % kStages], (j / kStages) & 1, tck::kWaitNs);
        }
    } else if (!idle && warp == kMmaWarp) {
        // ---- products ------------------------------------------------------------------------------
        const bool leader = tc::elect_one();
        uint32_t it = 0, items = 0, sp[2] = {0, 0}, used[2] = {0, 0};   // tiles loaded, items, score tiles, items of a query tile
        bool ok = true;
        auto scores = [&](int t, uint32_t stage) {
            if (leader) {
                const uint64_t dq = desc_k(base + t * kTileBytes), dk = desc_k(base + (2 + stage) * kTileBytes);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
                    tc::umma_bf16(tmem + kS0 + t * kTile, dq + off, dk + off, kIdS, ks > 0);
                }
                tc::umma_commit(&bar.s_full[t]);
            }
            __syncwarp();
        };
        do {
            const int nt = w.x.ntok > a.TB ? 2 : 1;
            const int end = max(0, w.x.limit + w.x.ntok), shared_from = max(0, w.x.limit + 1);
            bool bad = false;
            ok = wait_or_abort(&bar.q_full, items & 1, aborted, status) &&
                 wait_or_abort(&bar.full[it % kStages], (it / kStages) & 1, aborted, status);
            if (!ok) break;
            tc::tc_fence_after();
            for (int t = 0; t < nt; ++t) scores(t, it % kStages);
            if (leader) tc::umma_commit(&bar.empty[it % kStages]);
            if (w.t1 - w.t0 == 1 && leader) tc::umma_commit(&bar.q_free);
            for (int i = w.t0; i < w.t1 && ok; ++i) {
                const uint32_t vs = (it + 1) % kStages, ks_next = (it + 2) % kStages;
                const bool more = i + 1 < w.t1;
                ok = wait_or_abort(&bar.full[vs], ((it + 1) / kStages) & 1, aborted, status);
                if (!ok) break;
                const int p0 = i * kTile;
                if (p0 + kTile > shared_from) {   // rows of V that not all tokens see, or none
                    uint8_t *v = smem + (2 + vs) * kTileBytes;
                    for (int e = lane + max(0, min(kTile, end - p0)) * 16; e < kTile * 16; e += 32)
                        *reinterpret_cast<uint4 *>(v + piece_at(e >> 4, e & 15)) = make_uint4(0, 0, 0, 0);
                    bool found = false;
                    for (int e = lane + max(0, shared_from - p0) * 16; e < min(kTile, end - p0) * 16; e += 32) {
                        uint4 *at = reinterpret_cast<uint4 *>(v + piece_at(e >> 4, e & 15));
                        const uint4 x = *at;
                        bool here = false;
                        const uint4 y = make_uint4(clear_bad(x.x, &here), clear_bad(x.y, &here), clear_bad(x.z, &here),
                                                   clear_bad(x.w, &here));
                        if (here) *at = y, found = true;
                    }
                    bad |= __any_sync(0xffffffffu, found) != 0;
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                }
                for (int t = 0; t < nt && ok; ++t) {
                    ok = wait_or_abort(&bar.p_full[t], sp[t] & 1, aborted, status);
                    if (ok && i == w.t0 && used[t] > 0) ok = wait_or_abort(&bar.o_free[t], (used[t] - 1) & 1, aborted, status);
                    if (!ok) break;
                    ++sp[t];
                    tc::tc_fence_after();
                    if (leader) {
                        const uint64_t dv = desc_mn(base + (2 + vs) * kTileBytes);
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            tc::umma_bf16_ta(tmem + kO0 + t * kTile, tmem + kS0 + t * kTile + 8 * ks, dv + ks * (2048 >> 4), kIdO,
                                             i > w.t0 || ks > 0);
                        if (!more) tc::umma_commit(&bar.o_full[t]);
                    }
                    __syncwarp();
                    if (more) {
                        if (t == 0) {
                            ok = wait_or_abort(&bar.full[ks_next], ((it + 2) / kStages) & 1, aborted, status);
                            if (!ok) break;
                            tc::tc_fence_after();
                        }
                        scores(t, ks_next);
                    }
                }
                if (!ok) break;
                if (leader) {
                    tc::umma_commit(&bar.empty[vs]);
                    if (more) tc::umma_commit(&bar.empty[ks_next]);
                    if (i + 2 == w.t1) tc::umma_commit(&bar.q_free);
                }
                __syncwarp();
                it += 2;
            }
            if (!ok) break;
            if (leader)
                for (int t = 0; t < nt; ++t) {
                    bad_values[t] = bad;
                    mbar_arrive(&bar.o_full[t]);
                }
            for (int t = 0; t < nt; ++t) ++used[t];
            ++items;
            __syncwarp();
        } while (w.next(a.p, per_head, begin, cta));
        if (!ok) {   // products in flight end before the tensor memory is freed
            if (leader) {
                tc::umma_commit(&bar.drain);
                tc::mbar_wait(&bar.drain, 0, tck::kWaitNs);
            }
            __syncwarp();
        }
    } else if (!idle) {
        // ---- softmax and results: a row of scores a thread -----------------------------------------
        const int t = warp >> 2, r = threadIdx.x & (kTile - 1);
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + kS0 + t * kTile + lanes, to = tmem + kO0 + t * kTile + lanes;
        const int my_tok = t * a.TB + r / a.G, g = r % a.G;
        const bool in_tile = r < a.TB * a.G;
        const bool warp_in = (warp & 3) * 32 < a.TB * a.G;
        uint32_t seen = 0, items = 0;
        bool ok = true;
        do {
            if (t == 1 && w.x.ntok <= a.TB) continue;
            const bool valid = in_tile && my_tok < w.x.ntok;
            const int limit = valid ? w.x.limit + my_tok : -1;
            const int first_limit = w.x.limit + t * a.TB;
            // a warp without rows leaves its scores as they are: rows of a product do not mix
            const bool active = warp_in && t * a.TB + (warp & 3) * 32 / a.G < w.x.ntok;
            const float scale = a.scale * (c.k_scale ? __ldg(c.k_scale + w.h) : 1.f) * kLog2e;
            float m = -INFINITY, l = 0.f;   // the maximum in units of the scores
            for (int i = w.t0; i < w.t1; ++i) {
                ok = wait_or_abort(&bar.s_full[t], seen & 1, aborted, status);
                if (!ok) break;
                ++seen;
                tc::tc_fence_after();
                if (active) {
                    uint32_t s[4][32];
#pragma unroll
                    for (int q = 0; q < 4; ++q) tc::tmem_ld_32x32b_x32(ts + 32 * q, s[q]);
                    tc::tmem_ld_wait();
                    if (i * kTile + kTile - 1 > first_limit) {
                        const int keep = limit - i * kTile;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (q * 32 + j > keep) s[q][j] = __float_as_uint(-INFINITY);
                    }
                    float top[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        top[q] = __uint_as_float(s[q][0]);
#pragma unroll
                        for (int j = 1; j < 32; ++j) top[q] = fmaxf(top[q], __uint_as_float(s[q][j]));
                    }
                    const float tile_top = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    if (i == w.t0) {
                        m = tile_top;
                    } else {
                        const bool grow = tile_top > m && !((tile_top - m) * scale <= kRescale);
                        if (__any_sync(0xffffffffu, grow)) {
                            const float f = !grow ? 1.f : m == -INFINITY ? 0.f : tc::ex2((m - tile_top) * scale);
                            if (grow) m = tile_top;
                            l *= f;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                uint32_t o[32];
                                tc::tmem_ld_32x32b_x32(to + 32 * q, o);
                                tc::tmem_ld_wait();
#pragma unroll
                                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tc::tmem_st_32x32b_x32(to + 32 * q, o);
                            }
                        }
                    }
                    const float mc = m == -INFINITY ? 0.f : m * scale;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int q = 0; q < 4; q += 2) {
                        uint32_t pk[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const uint32_t *in = s[q + (j >> 4)];
                            const float x = tc::ex2(fmaf(__uint_as_float(in[(2 * j) & 31]), scale, -mc));
                            const float y = tc::ex2(fmaf(__uint_as_float(in[(2 * j + 1) & 31]), scale, -mc));
                            sum[j & 3] += x + y;
                            pk[j] = float2_to_bf16x2(x, y);
                        }
                        tc::tmem_st_32x32b_x32(ts + 16 * q, pk);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tc::tmem_st_wait();
                }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[t]);
            }
            if (!ok) break;
            ok = wait_or_abort(&bar.o_full[t], items & 1, aborted, status);
            if (!ok) break;
            ++items;
            tc::tc_fence_after();
            if (active) {
                const bool whole = w.slot < 0, some = limit >= 0;   // some: the row sees a place
                uint32_t dims[4] = {0, 0, 0, 0};
                if (bad_values[t] && valid) bad_dimensions(c, w.x.n, w.h, w.x.limit, limit, dims);
                const float vs = c.v_scale ? __ldg(c.v_scale + w.h) : 1.f;
                const float inv = whole ? vs / l : 1.f;
                const int64_t row = (w.x.row + my_tok) * (a.G * c.H) + w.h * a.G + g;
                const int64_t prow = static_cast<int64_t>(w.slot) * kRows + t * kTile + r;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t o[32];
                    __syncwarp();
                    tc::tmem_ld_32x32b_x32(to + 32 * q, o);
                    tc::tmem_ld_wait();
                    if (dims[q])
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (dims[q] >> j & 1) o[j] = 0x7fc00000u;
                    if (valid && whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.o + row * kD + 32 * q);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t x[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float lo = __uint_as_float(o[8 * j + 2 * e]), hi = __uint_as_float(o[8 * j + 2 * e + 1]);
                                x[e] = some ? float2_to_bf16x2(lo * inv, hi * inv) : 0u;
                            }
                            dst[j] = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    } else if (valid) {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.p.part_o + prow * kD + 32 * q);
#pragma unroll
                        for (int j = 0; j < 8; ++j) dst[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    }
                }
                if (valid) {
                    const float mc = m == -INFINITY ? 0.f : m * scale;
                    if (!whole) a.p.part_ml[prow] = make_float2(m == -INFINITY ? m : mc, l);
                    else if (a.lse) a.lse[row] = some ? (mc + log2f(l)) * kLn2 : -INFINITY;
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.o_free[t]);
        } while (w.next(a.p, per_head, begin, cta));
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// ---- joins the partial results of units that several CTAs share -----------------------------------

constexpr int kJoinThreads = 256, kJoinRows = 32;

__global__ void __launch_bounds__(kJoinThreads) paged_combine_kernel(const AttendArgs a, int ctas) {
    dependent_start();
    const KvArgs &c = a.c;
    const int64_t units = a.p.total[0], per_head = a.p.total[1], all = per_head * c.H;
    // this CTA's last unit, if it begins here and ends in a later one
    const int cta = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = range_begin(all, cta, ctas), r1 = range_begin(all, cta + 1, ctas);
    if (r0 >= r1 || r1 >= all) return;
    const int h = static_cast<int>((r1 - 1) / per_head);
    const int64_t u = unit_at(a.p, units, r1 - 1 - per_head * h);
    const int64_t from = per_head * h + a.p.start[u], to = per_head * h + a.p.start[u + 1];
    if (from < r0 || to <= r1) return;
    int last = cta + 1;
    while (last + 1 < ctas && range_begin(all, last + 1, ctas) < to) ++last;
    const int parts = last - cta + 1;
    auto slot = [&](int p) { return static_cast<int64_t>(2 * (cta + p) + (p == 0 ? 1 : 0)); };
    const Unit x = a.p.units[u];
    const float vs = c.v_scale ? __ldg(c.v_scale + h) : 1.f;
    for (int k = warp; k < kJoinRows; k += kJoinThreads / 32) {
        const int r = blockIdx.y * kJoinRows + k, t = r / kTile, rr = r - t * kTile;
        const int tok = t * a.TB + rr / a.G;
        if (rr >= a.TB * a.G || tok >= x.ntok) continue;
        float top = -INFINITY;
        for (int p = lane; p < parts; p += 32) top = fmaxf(top, a.p.part_ml[slot(p) * kRows + r].x);
        for (int o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float at = top == -INFINITY ? 0.f : top;
        float total = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p0 = 0; p0 < parts; p0 += 32) {
            float f = 0.f, l = 0.f;
            if (p0 + lane < parts) {
                const float2 ml = a.p.part_ml[slot(p0 + lane) * kRows + r];
                f = ml.x == -INFINITY ? 0.f : tc::ex2(ml.x - at);
                l = ml.y * f;
            }
            for (int o = 16; o > 0; o /= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
            total += l;
            const int here = min(32, parts - p0);
#pragma unroll 4
            for (int p = 0; p < here; ++p) {
                const float w = __shfl_sync(0xffffffffu, f, p);
                const float4 v = *reinterpret_cast<const float4 *>(a.p.part_o + (slot(p0 + p) * kRows + r) * kD + lane * 4);
                acc.x += w * v.x;
                acc.y += w * v.y;
                acc.z += w * v.z;
                acc.w += w * v.w;
            }
        }
        const bool some = x.limit + tok >= 0;
        const float inv = vs / total;
        const int64_t row = (x.row + tok) * (a.G * c.H) + h * a.G + rr % a.G;
        *reinterpret_cast<uint2 *>(a.o + row * kD + lane * 4) =
            some ? make_uint2(float2_to_bf16x2(acc.x * inv, acc.y * inv), float2_to_bf16x2(acc.z * inv, acc.w * inv))
                 : make_uint2(0, 0);
        if (a.lse && lane == 0) a.lse[row] = some ? (at + log2f(total)) * kLn2 : -INFINITY;
    }
}

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

namespace {
size_t aligned(size_t bytes) { return (bytes + 255) & ~size_t(255); }

int64_t most_units(const KvArgs &c, int G) { return c.T / (2 * tokens_of_tile(G)) + c.N; }

size_t lay_out(const KvArgs &c, int G, bool own_lse, int ctas, char *ws, Plan *p, float **lse) {
    const size_t units = static_cast<size_t>(most_units(c, G));
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *r = ws + at;
        at += aligned(bytes);
        return r;
    };
    p->most = static_cast<int64_t>(units);
    p->total = reinterpret_cast<int64_t *>(take(16));
    p->start = reinterpret_cast<int64_t *>(take((units + 1) * 8));
    p->units = reinterpret_cast<Unit *>(take(units * sizeof(Unit)));
    p->first = reinterpret_cast<int32_t *>(take(static_cast<size_t>(c.N) * 4));
    p->part_o = reinterpret_cast<float *>(take(static_cast<size_t>(ctas) * 2 * kRows * kD * 4));
    p->part_ml = reinterpret_cast<float2 *>(take(static_cast<size_t>(ctas) * 2 * kRows * 8));
    *lse = own_lse ? reinterpret_cast<float *>(take(static_cast<size_t>(c.T) * G * c.H * 4)) : nullptr;
    return at;
}
}  // namespace

size_t paged_attention_scratch(const KvArgs &c, int G, bool, bool own_lse, int sm_count) {
    Plan p;
    float *lse;
    return lay_out(c, G, own_lse, sm_count, nullptr, &p, &lse);
}

cudaError_t setup_paged_attention_kernel() {
    for (auto kern : {paged_attention_kernel<false>, paged_attention_kernel<true>}) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_paged_attention(const KvArgs &c, const void *q, int64_t q_stride, float scale, void *o, float *lse,
                                   bool accumulate, int G, void *ws, int sm_count, cudaStream_t st) {
    AttendArgs a;
    float *own;
    lay_out(c, G, accumulate && !lse, sm_count, static_cast<char *>(ws), &a.p, &own);
    a.c = c;
    a.o = static_cast<uint16_t *>(o);
    a.lse = lse ? lse : own;
    a.scale = scale;
    a.G = G;
    a.TB = tokens_of_tile(G);
    CUtensorMap mq, mk, mv;
    cudaError_t e;
    {
        const cuuint64_t dims[3] = {kD, static_cast<cuuint64_t>(G) * c.H, static_cast<cuuint64_t>(c.T)};
        const cuuint64_t strides[2] = {kD * 2, static_cast<cuuint64_t>(q_stride) * 2};
        const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(a.TB)};
        e = tck::encode_tiled(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
        if (e != cudaSuccess) return e;
        mk = mv = mq;   // not read with an e4m3 cache
    }
    if (!c.e4m3) {
        const cuuint64_t dims[3] = {kD, static_cast<cuuint64_t>(c.S), static_cast<cuuint64_t>(c.P) * c.H};
        const cuuint64_t strides[2] = {kD * 2, static_cast<cuuint64_t>(c.S) * kD * 2};
        const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(c.S < kTile ? c.S : kTile), 1};
        e = tck::encode_tiled(&mk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, c.k, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
        if (e == cudaSuccess)
            e = tck::encode_tiled(&mv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, c.v, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
        if (e != cudaSuccess) return e;
    }
    {
        LaunchTimer timer(kKPagedPlan, st);
        e = launch_dependent(paged_plan_kernel, dim3(1), kPlanThreads, st, c, a.p, 2 * a.TB);
        if (e != cudaSuccess) return e;
    }
    {
        LaunchTimer timer(kKPagedAttention, st);
        e = launch_dependent_cluster(c.e4m3 ? paged_attention_kernel<true> : paged_attention_kernel<false>, dim3(sm_count), 0,
                                     threads_of(c.e4m3), kSmemAlloc, st, a, mq, mk, mv);
        if (e != cudaSuccess) return e;
    }
    {
        LaunchTimer timer(kKPagedCombine, st);
        e = launch_dependent(paged_combine_kernel, dim3(sm_count, kRows / kJoinRows), kJoinThreads, st, a, sm_count);
        if (e != cudaSuccess || !accumulate) return e;
    }
    LaunchTimer timer(kKPagedWeights, st);
    return launch_dependent(weights_kernel, dim3(64, c.H, static_cast<unsigned>(c.N < 65535 ? c.N : 65535)), kThreads, st, c,
                            static_cast<const uint16_t *>(q), q_stride, scale, a.lse, G);
}

}  // namespace sala

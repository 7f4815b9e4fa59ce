// The attention weight that each cached token received, added to its running sum.
//
// Runs after the attention, when every row's z = m + log2(sum 2^(c (s - m))) / c is known (c = scale * k_scale * log2 e, m its
// largest score):
//     weights[j] += sum over the rows r that see j of  2^(c (k_j.q_r - z_r))
// z in units of the scores keeps their bits: z >= m also after rounding, so that no weight passes 1, however large the
// scores (with c z held instead, the products' roundings alone are a factor of 2 from |c z| = 2^24 on).
// The scores are made again, transposed: S^T = K Q^T (tcgen05, 128 places x 128 rows). A place is then a lane of
// tensor memory and its sum over the rows a thread's own, without shuffles or atomics, in a fixed order. z is the same
// for all lanes: it enters as one more step of the product, columns of ones beside K and -z as three bf16 terms (24
// bits) beside Q, so that an element costs a multiplication, an exp2 and an addition. (Read from shared memory
// instead, it competed with the operands of the products: 7 query tiles on 6007 places 295 us.)
//
// A unit is a cache tile with the query tiles that see it; CTAs take equal shares of all of them, and units that
// several CTAs share leave partial sums for a last kernel. Four groups of four warps take the score tiles in turn, from
// four buffers in tensor memory. With one query tile for a request (decoding) it stays in shared memory while the
// request's cache tiles pass: the kernel then reads the keys once, which bounds it: 61 requests with 5 tokens on 8192
// e4m3 places, 128 MB of keys, in 48 us (2.7 TB/s; the keys are widened as in the attention). With many tiles the exp2 of
// every score bounds it: 7 prompts of up to 2011 tokens at the end of 6007 places, 201 us for 243 GFLOP. Units of two cache
// tiles, which halve the reads of the queries, took 194 there but 51 for the drafts; reading a score tile's next columns while
// the last are summed changed nothing.
#include "paged_tiles.cuh"

namespace sala {
namespace {

using namespace pt;
using tc::mbar_arrive;

constexpr int kMmaWarp = 16, kLoadWarp = 17, kStatsWarp = 18, kConvertWarp = 19;
constexpr int kGroups = 4;                       // of four warps; score tiles in tensor memory
constexpr uint32_t kAuxBytes = kTile * 32;       // [128 rows x 16 bf16], 32-byte swizzle

template <bool E4M3>
struct Shape {
    static constexpr int kKeys = 3, kQueries = E4M3 ? 2 : 3, kRaw = E4M3 ? 3 : 0;   // tiles in shared memory
    static constexpr int kThreads = 32 * (E4M3 ? kConvertWarp + kConvertWarps : kConvertWarp);
    static constexpr uint32_t kQueriesAt = kKeys * kTileBytes, kRawAt = kQueriesAt + kQueries * kTileBytes;
    static constexpr uint32_t kOnesAt = kRawAt + kRaw * kRawBytes, kAuxAt = kOnesAt + kAuxBytes;
    static constexpr uint32_t kAlloc = kAuxAt + kQueries * kAuxBytes + 1024;
};

// What the roles of a CTA do next, from the loading warp: cache tiles [u0, u0 + nu) of request n with nq query tiles
// from the one whose first token is packed token `row` at place `limit`, `ntok` tokens in all. nu > 1 only with nq = 1.
struct alignas(16) Item {
    int64_t row;
    int n, h, len, u0, nu, nq, ntok, limit;
    int slot;            // where a partial result goes, -1: the item is the whole unit
    int last;
};
constexpr int kItems = 4;

// A cache tile that this CTA began and others finished: `parts` partial sums, from this CTA on (0: none).
struct JoinUnit {
    int n, h, u, parts;
};

struct Barriers {
    uint64_t k_full[3], k_empty[3], q_full[3], q_empty[3], raw_full[5], raw_empty[5];
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t s_full[kGroups], s_free[kGroups];
    // Partial sums, from group b to group a: [a][b]. (With one barrier for a sender a collector an item ahead of it would pass by
    // the parity of the phase before the sender's last.) Sums of a group that are read.
    uint64_t part_full[kGroups][kGroups], part_free[kGroups];
    uint64_t drain;
};

// Byte offset of 16-byte piece `piece` (of 2) of a row in a tile of 16 columns.
__device__ __forceinline__ uint32_t aux_at(int row, int piece) { return row * 32 + ((piece ^ ((row >> 2) & 1)) << 4); }

// Descriptor of such a tile: 32-byte swizzle (layout 6), 256 bytes from 8 rows to the next.
__device__ __forceinline__ uint64_t desc_aux(uint32_t addr) {
    uint64_t d = (addr >> 4) & 0x3FFFu;
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>(256 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(6) << 61;
    return d;
}

template <bool E4M3>
__global__ void __launch_bounds__(Shape<E4M3>::kThreads, 1)
    paged_weights_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ Maps maps) {
    using Layout = Shape<E4M3>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Barriers bar;
    __shared__ float parts[kGroups][kTile];
    __shared__ Item ring[kItems];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ Place place;
    const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *const smem = smem_raw + (base - tc::smem_u32(smem_raw));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
    const KvArgs &c = a.c;
    const WeightWork work{a.TB};

    if (warp == kMmaWarp) {
        tc::tmem_alloc(&tmem_slot, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < Layout::kKeys; ++i) {
            tc::mbar_init(&bar.k_full[i], E4M3 ? kConvertWarps : 1);
            tc::mbar_init(&bar.k_empty[i], 1);
        }
        for (int i = 0; i < Layout::kQueries; ++i) {
            tc::mbar_init(&bar.q_full[i], 2);
            tc::mbar_init(&bar.q_empty[i], 1);
        }
        for (int i = 0; i < Layout::kRaw; ++i) {
            tc::mbar_init(&bar.raw_full[i], 1);
            tc::mbar_init(&bar.raw_empty[i], kConvertWarps);
        }
        for (int i = 0; i < kItems; ++i) {
            tc::mbar_init(&bar.item_full[i], 1);
            tc::mbar_init(&bar.item_empty[i], 18 + (E4M3 ? kConvertWarps : 0));
        }
        for (int i = 0; i < kGroups; ++i) {
            tc::mbar_init(&bar.s_full[i], 1);
            tc::mbar_init(&bar.s_free[i], 4);
            for (int from = 0; from < kGroups; ++from) tc::mbar_init(&bar.part_full[i][from], 4);
            tc::mbar_init(&bar.part_free[i], 4);
        }
        tc::mbar_init(&bar.drain, 1);
        tc::fence_barrier_init();
        abort_flag = 0;
    }
    if (threadIdx.x < kTile) {   // the columns beside K: three ones, then zeros
        *reinterpret_cast<uint4 *>(smem + Layout::kOnesAt + aux_at(threadIdx.x, 0)) = make_uint4(0x3f803f80u, 0x3f80u, 0, 0);
        *reinterpret_cast<uint4 *>(smem + Layout::kOnesAt + aux_at(threadIdx.x, 1)) = make_uint4(0, 0, 0, 0);
        tc::fence_proxy_async_smem();
    }
    // The attention waited for what lay before it and then let the joining of its results, and this kernel, start: the
    // lengths and offsets are there, and only what follows the split of the work waits for the rows' statistics.
    let_dependents_start();
    uint32_t *const near = reinterpret_cast<uint32_t *>(smem);   // where the tiles land later
    if (!a.weight_start) scan_requests(c, work, near, near + kInline + 1);
    const Starts starts{a.weight_start ? nullptr : near, a.weight_start};
    const int64_t per_head = starts[c.N], all = per_head * c.H;
    const int64_t begin = range_begin(all, cta, gridDim.x), stop = range_begin(all, cta + 1, gridDim.x);
    const bool idle = begin >= stop;
    if (threadIdx.x == 0 && !idle) place = find(c, work, starts, per_head, begin);
    wait_for_previous();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (idle && threadIdx.x == 0) static_cast<JoinUnit *>(a.weight_joins)[cta].parts = 0;
    const uint32_t tmem = tmem_slot;
    volatile int *const aborted = &abort_flag;
    int *const status = c.status;
    // the items from the ring, for every role but the loading warp
    uint32_t items = 0;
    auto take = [&](Item &x) {
        if (!wait_warp(&bar.item_full[items % kItems], (items / kItems) & 1, aborted, status)) return false;
        x = ring[items % kItems];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.item_empty[items % kItems]);
        ++items;
        return true;
    };

    if (warp == kLoadWarp && !idle) {
        // ---- loads: a cache tile of keys after another, query tiles ------------------------------------
        constexpr int kRing = E4M3 ? Layout::kRaw : Layout::kKeys;
        uint64_t *const full = E4M3 ? bar.raw_full : bar.k_full, *const empty = E4M3 ? bar.raw_empty : bar.k_empty;
        uint32_t kt = 0, qt = 0;
        bool ok = true;
        JoinUnit join = {0, 0, 0, 0};
        Walk<WeightWork> w;
        w.start_at(c, work, place, begin, stop, cta);
        tc::fence_proxy_async_smem();   // the running sums were there before the tiles
        do {
            const bool single = work.query_tiles(w.r.count) == 1;
            const int q0 = work.first(w.r.count, w.r.len, w.u) + w.t0, slot = items % kItems;
            Item x;
            x.row = w.r.first + q0 * a.TB;
            x.n = static_cast<int>(w.n);
            x.h = w.h;
            x.len = w.r.len;
            x.u0 = w.u;
            x.nu = single ? static_cast<int>(min(static_cast<int64_t>(w.units - w.u), stop - w.pos)) : 1;
            x.nq = w.t1 - w.t0;
            x.ntok = w.r.count - q0 * a.TB;
            x.limit = w.r.len - w.r.count + q0 * a.TB;
            x.slot = w.slot;
            w.u += x.nu - 1;
            w.pos += x.nu - 1;
            x.last = w.pos + (w.t1 - w.t0) >= stop;
            ok = items < kItems || wait_warp(&bar.item_empty[slot], (items / kItems - 1) & 1, aborted, status);
            if (!ok) break;
            if (lane == 0) {
                ring[slot] = x;
                mbar_arrive(&bar.item_full[slot]);
            }
            __syncwarp();
            ++items;
            int page = box_page<E4M3>(c, x.n, x.u0, x.len, lane);   // of the next tile: looked up ahead
            for (int i = 0; i < x.nu && ok; ++i, ++kt) {
                const int here = page, st = kt % kRing;
                page = i + 1 < x.nu ? box_page<E4M3>(c, x.n, x.u0 + i + 1, x.len, lane) : -2;
                ok = kt < kRing || wait_warp(&empty[st], (kt / kRing - 1) & 1, aborted, status);
                if (!ok) break;
                load_boxes<E4M3>(c, &maps.k, smem + (E4M3 ? Layout::kRawAt + st * kRawBytes : st * kTileBytes), x.u0 + i, x.h, here,
                                 lane, &full[st]);
                for (int q = 0; i == 0 && q < x.nq; ++q, ++qt) {
                    const int s = qt % Layout::kQueries;
                    ok = qt < Layout::kQueries || wait_warp(&bar.q_empty[s], (qt / Layout::kQueries - 1) & 1, aborted, status);
                    if (!ok) break;
                    if (lane == 0) {
                        tc::mbar_arrive_expect_tx(&bar.q_full[s], 2 * static_cast<uint32_t>(a.TB * a.G) * 128u);
                        load_query_tile(smem + Layout::kQueriesAt + s * kTileBytes, &maps.q, x.h, a.G, x.row + q * a.TB, &bar.q_full[s]);
                    }
                    __syncwarp();
                }
            }
            if (x.last && x.slot >= 0 && w.t0 == 0)
                join = {x.n, x.h, x.u0, cta_of(all, w.pos + w.tiles - 1, gridDim.x) - cta + 1};
        } while (ok && w.next(c, work, cta));
        if (lane == 0) static_cast<JoinUnit *>(a.weight_joins)[cta] = join;
        // the last copies land before the CTA ends, whoever gave up
        for (uint32_t j = kt > kRing ? kt - kRing : 0; j < kt; ++j)
            tc::mbar_wait(&full[j % kRing], (j / kRing) & 1, tck::kWaitNs);
        for (uint32_t j = qt > Layout::kQueries ? qt - Layout::kQueries : 0; j < qt; ++j)
            tc::mbar_wait(&bar.q_full[j % Layout::kQueries], (j / Layout::kQueries) & 1, tck::kWaitNs);
    } else if (warp == kStatsWarp && !idle) {
        // ---- the columns beside Q: -z of each row ------------------------------------------------------
        uint32_t qt = 0;
        const int Hq = a.G * c.H;
        Item x;
        bool ok = true;
        do {
            ok = take(x);
            if (!ok) break;
            float next[4];
            auto fetch = [&](int q) {   // rows 32 e + lane of query tile q
                const int rows = min(a.TB, x.ntok - q * a.TB) * a.G;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = 32 * e + lane, tok = row / a.G;
                    next[e] = row < rows ? a.stats[(x.row + q * a.TB + tok) * Hq + x.h * a.G + row - tok * a.G] : 0.f;
                }
            };
            fetch(0);
            for (int q = 0; q < x.nq; ++q, ++qt) {
                const int s = qt % Layout::kQueries;
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = next[e];
                if (q + 1 < x.nq) fetch(q + 1);
                ok = qt < Layout::kQueries || wait_warp(&bar.q_empty[s], (qt / Layout::kQueries - 1) & 1, aborted, status);
                if (!ok) break;
                uint8_t *aux = smem + Layout::kAuxAt + s * kAuxBytes;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = -y[e];
                    const float hi = __bfloat162float(__float2bfloat16_rn(v));
                    const float mid = __bfloat162float(__float2bfloat16_rn(v - hi));
                    *reinterpret_cast<uint4 *>(aux + aux_at(32 * e + lane, 0)) =
                        make_uint4(float2_to_bf16x2(hi, mid), float2_to_bf16x2((v - hi) - mid, 0.f), 0, 0);
                    *reinterpret_cast<uint4 *>(aux + aux_at(32 * e + lane, 1)) = make_uint4(0, 0, 0, 0);
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.q_full[s]);
            }
        } while (ok && !x.last);
    } else if (E4M3 && warp >= kConvertWarp && !idle) {
        // ---- e4m3 keys to bf16 ---------------------------------------------------------------------------
        constexpr int kRaw = E4M3 ? Layout::kRaw : 1;
        uint32_t it = 0;
        Item x;
        bool ok = true;
        do {
            ok = take(x);
            for (int i = 0; ok && i < x.nu; ++i, ++it) {
                const int st = it % Layout::kKeys, rw = it % kRaw;
                ok = wait_warp(&bar.raw_full[rw], (it / kRaw) & 1, aborted, status) &&
                     (it < Layout::kKeys || wait_warp(&bar.k_empty[st], (it / Layout::kKeys - 1) & 1, aborted, status));
                if (!ok) break;
                uint4 held[kPieces];
                read_pieces(held, smem + Layout::kRawAt + rw * kRawBytes, threadIdx.x - 32 * kConvertWarp);
                store_pieces(held, smem + st * kTileBytes, threadIdx.x - 32 * kConvertWarp);
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar.k_full[st]);
                    mbar_arrive(&bar.raw_empty[rw]);
                }
            }
        } while (ok && !x.last);
    } else if (warp == kMmaWarp && !idle) {
        // ---- products ------------------------------------------------------------------------------------
        const uint32_t k_full = tc::smem_u32(bar.k_full), k_empty = tc::smem_u32(bar.k_empty), q_full = tc::smem_u32(bar.q_full);
        const uint32_t q_empty = tc::smem_u32(bar.q_empty), s_full = tc::smem_u32(bar.s_full), s_free = tc::smem_u32(bar.s_free);
        const uint64_t first_k = desc_k(base), first_q = desc_k(base + Layout::kQueriesAt);
        const uint64_t ones = desc_aux(base + Layout::kOnesAt), first_aux = desc_aux(base + Layout::kAuxAt);
        Ring<Layout::kKeys> k;
        Ring<Layout::kQueries> q;
        Ring<kGroups> b;
        bool ok = true;
        Item x;
        auto passed = [&](uint32_t at, uint32_t parity) {
            return __all_sync(0xffffffffu, wait_at(at, parity, aborted, status)) != 0;
        };
        // The scores of the next query tile, with `rows` rows, for the next keys, into the next buffer; the tiles' rooms are free
        // after the last of them. As in the attention, a wait that gave up is noted in `fine` and voted on once a tile.
        auto scores = [&](bool fine, int rows, bool query_last, bool keys_last) {
            fine &= wait_at(s_free + 8 * b.at, b.parity ^ 1u, aborted, status);   // passes at once the first time
            tc::tc_fence_after();
            if (tc::elect_one()) {
                const uint32_t id = tc::idesc_bf16_f32(128, (rows + 15) & ~15, 0, 0), d = tmem + b.at * kTile;
                const uint64_t dk = first_k + k.at * (kTileBytes >> 4), dq = first_q + q.at * (kTileBytes >> 4);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t off = ((i >> 2) * kHalf + (i & 3) * 32) >> 4;
                    tc::umma_bf16(d, dk + off, dq + off, id, i > 0);
                }
                // last: what it leaves is small, and the score before it has the attention's own roundings
                tc::umma_bf16(d, ones, first_aux + q.at * (kAuxBytes >> 4), id, 1u);
                commit_at(s_full + 8 * b.at);
                if (query_last) commit_at(q_empty + 8 * q.at);
                if (keys_last) commit_at(k_empty + 8 * k.at);
            }
            b.advance(1);
            return __all_sync(0xffffffffu, fine) != 0;
        };
        do {
            ok = __all_sync(0xffffffffu, take(x)) != 0;
            if (!ok) break;
            const int nu = __shfl_sync(0xffffffffu, x.nu, 0), nq = __shfl_sync(0xffffffffu, x.nq, 0);
            int left = __shfl_sync(0xffffffffu, x.ntok, 0);
            if (nq == 1) {   // a query tile for a run of cache tiles
                const int rows = min(a.TB, left) * a.G;
                ok = passed(q_full + 8 * q.at, q.parity);
                for (int i = 0; i < nu && ok; ++i) {
                    ok = scores(wait_at(k_full + 8 * k.at, k.parity, aborted, status), rows, i + 1 == nu, true);
                    k.advance(1);
                }
                q.advance(1);
            } else {         // a cache tile for a run of query tiles
                ok = passed(k_full + 8 * k.at, k.parity);
                for (int i = 0; i < nq && ok; ++i, left -= a.TB) {
                    ok = scores(wait_at(q_full + 8 * q.at, q.parity, aborted, status), min(a.TB, left) * a.G, true, i + 1 == nq);
                    q.advance(1);
                }
                k.advance(1);
            }
        } while (ok && !__shfl_sync(0xffffffffu, x.last, 0));
        if (tc::elect_one()) {   // products in flight end before the tensor memory is freed, whoever gave up
            tc::umma_commit(&bar.drain);
            tc::mbar_wait(&bar.drain, 0, tck::kWaitNs);
        }
        __syncwarp();
    } else if (warp < kMmaWarp && !idle) {
        // ---- sums: a place a thread ------------------------------------------------------------------------
        const int g = warp >> 2, r = threadIdx.x & (kTile - 1);
        const uint32_t ts = tmem + g * kTile + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        uint32_t tile = 0, done = 0;             // score tiles of the CTA, of this group
        uint32_t sent = 0, flips = 0;             // partial sums handed over; parity of those from each group, a bit each
        bool ok = true;
        Item x{};
        float scale = 0.f;
        // The sum over the rows of query tile q that see place p of the item's cache tile i
        auto sum_tile = [&](int i, int p, int q) {
            ok = wait_warp(&bar.s_full[g], done & 1, aborted, status);
            if (!ok) return 0.f;
            ++done;
            tc::tc_fence_after();
            const int rows = min(a.TB, x.ntok - q * a.TB) * a.G;
            const bool seen = x.limit + q * a.TB >= (x.u0 + i) * kTile + kTile - 1;   // by all rows, every place
            const int ahead = p - x.limit - q * a.TB;
            const int from = ahead <= 0 ? 0 : ahead >= a.TB ? kTile : ahead * a.G;   // rows before it do not see the place
            const uint64_t scale2 = tc::pair(scale, scale);
            uint64_t sum2[2] = {0, 0};   // pairs of zeros
            float rest = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (32 * e >= rows) break;
                uint32_t s[32];
                tc::tmem_ld_32x32b_x32(ts + 32 * e, s);
                tc::tmem_ld_wait();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int n0 = 32 * e + 16 * half;
                    if (seen && n0 + 16 <= rows) {
#pragma unroll
                        for (int j = 16 * half; j < 16 * half + 16; j += 2) {
                            const float2 y = tc::unpair(tc::mul2(tc::pair(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), scale2));
                            sum2[(j >> 1) & 1] = tc::add2(sum2[(j >> 1) & 1], tc::pair(tc::ex2(y.x), tc::ex2(y.y)));
                        }
                    } else if (n0 < rows) {
#pragma unroll
                        for (int j = 16 * half; j < 16 * half + 16; ++j) {
                            const float y = tc::ex2(__uint_as_float(s[j]) * scale);
                            rest += 32 * e + j >= from && 32 * e + j < rows ? y : 0.f;
                        }
                    }
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.s_free[g]);
            const float2 even = tc::unpair(sum2[0]), odd = tc::unpair(sum2[1]);
            return rest + ((even.x + even.y) + (odd.x + odd.y));
        };
        // Where place p's weight lies (null: nowhere, or the item's result is partial), and its value so far
        struct Weight {
            float *at = nullptr, old = 0.f;
        };
        auto look = [&](int p) {
            Weight w;
            if (x.slot < 0 && p < x.len) {
                const int page = kv::page_of(c, x.n, p);
                if (page >= 0) {
                    w.at = c.weights + kv::row_of(c, page, x.h, p);
                    w.old = *w.at;
                }
            }
            return w;
        };
        auto finish = [&](const Weight &w, float total) {
            if (x.slot >= 0) a.part_w[static_cast<int64_t>(x.slot) * kTile + r] = total;
            else if (w.at) *w.at = w.old + total;
        };
        do {
            ok = take(x);
            if (!ok) break;
            scale = a.scale * (c.k_scale ? kv::load(c.k_scale + x.h) : 1.f) * kLog2e;
            const int m = x.nq, p = x.u0 * kTile + r, owner = tile % kGroups;
            const int mine = (g - owner) & (kGroups - 1);   // this group's first tile of the item
            if (m == 1) {        // every fourth cache tile; its weights are looked up a turn ahead
                Weight next;
                if (mine < x.nu) next = look(p + mine * kTile);
                for (int i = mine; i < x.nu && ok; i += kGroups) {
                    const Weight w = next;
                    if (i + kGroups < x.nu) next = look(p + (i + kGroups) * kTile);
                    const float total = sum_tile(i, p + i * kTile, 0);
                    if (ok) finish(w, total);
                }
                tile += x.nu;
                continue;
            }
            tile += m;
            if (mine >= m) continue;
            Weight w;
            if (mine == 0) w = look(p);
            float total = 0.f;
            for (int q = mine; q < m && ok; q += kGroups) total += sum_tile(0, p, q);
            if (!ok) break;
            if (mine > 0) {   // to the group that has the unit's first query tile
                ok = sent == 0 || wait_warp(&bar.part_free[g], (sent - 1) & 1, aborted, status);
                if (!ok) break;
                parts[g][r] = total;
                ++sent;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.part_full[owner][g]);
                continue;
            }
#pragma unroll
            for (int o = 1; o < kGroups; ++o) {
                if (o >= m) break;
                const int from = (g + o) & (kGroups - 1);
                ok = wait_warp(&bar.part_full[g][from], (flips >> from) & 1, aborted, status);
                if (!ok) break;
                flips ^= 1u << from;
                total += parts[from][r];
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.part_free[from]);
            }
            if (ok) finish(w, total);
        } while (ok && !x.last);
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// Adds the partial sums of cache tiles that several CTAs share, in the order of the CTAs.
__global__ void __launch_bounds__(kTile) paged_weights_join_kernel(const AttendArgs a) {
    dependent_start();
    const KvArgs &c = a.c;
    const int cta = blockIdx.x, r = threadIdx.x;
    const JoinUnit x = static_cast<const JoinUnit *>(a.weight_joins)[cta];
    const int64_t p = static_cast<int64_t>(x.u) * kTile + r;
    if (x.parts == 0 || p >= kv::request_len(c, x.n)) return;
    float sum = 0.f;
    for (int i = 0; i < x.parts; ++i) sum += a.part_w[part_slot(cta, i) * kTile + r];
    const int page = kv::page_of(c, x.n, static_cast<int>(p));
    if (page >= 0) c.weights[kv::row_of(c, page, x.h, static_cast<int>(p))] += sum;
}

}  // namespace

namespace pt {

cudaError_t setup_paged_weights_kernel() {
    const cudaError_t e = cudaFuncSetAttribute(paged_weights_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Shape<false>::kAlloc);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(paged_weights_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<true>::kAlloc);
}

cudaError_t launch_paged_weights(const AttendArgs &a, const Maps &maps, int ctas, cudaStream_t st) {
    {
        LaunchTimer timer(kKPagedWeights, st);
        const cudaError_t e =
            a.c.e4m3 ? launch_dependent_cluster(paged_weights_kernel<true>, dim3(ctas), 0, Shape<true>::kThreads,
                                                Shape<true>::kAlloc, st, a, maps)
                     : launch_dependent_cluster(paged_weights_kernel<false>, dim3(ctas), 0, Shape<false>::kThreads,
                                                Shape<false>::kAlloc, st, a, maps);
        if (e != cudaSuccess) return e;
    }
    LaunchTimer timer(kKPagedCombine, st);
    return launch_dependent(paged_weights_join_kernel, dim3(ctas), kTile, st, a);
}

}  // namespace pt
}  // namespace sala

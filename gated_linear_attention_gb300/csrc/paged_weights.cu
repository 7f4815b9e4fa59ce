// The attention weight that each cached token received, added to its running sum.
//
// Runs after the attention, when every row's maximum m and sum l are known:
//     weights[j] += sum over the rows r that see j of  2^(c k_j.q_r - m_r) / l_r
// The scores are made again, transposed: S^T = K Q^T (tcgen05, 128 places x 128 rows). A place is then a lane of
// tensor memory and its sum over the rows a thread's own, without shuffles or atomics, in a fixed order; m and 1 / l
// are the same for all lanes and come from shared memory. Each element costs one multiply-add into exp2 and
// one into the sum.
//
// A unit is a cache tile with the query tiles that see it; CTAs take equal shares of all of them, and units that
// several CTAs share leave partial sums for a last kernel. Two warpgroups take the query tiles in turn, from four
// score buffers in tensor memory. With one query tile for a request (decoding) it stays in shared memory while the
// request's cache tiles pass: the kernel then reads the keys once, which bounds it.
#include "paged_tiles.cuh"

namespace sala {
namespace {

using namespace pt;
using tc::mbar_arrive;
using tck::wait_or_abort;

constexpr int kMmaWarp = 8, kLoadWarp = 9, kConvertWarp = 12;
constexpr int kBuffers = 4;                      // score tiles in tensor memory

template <bool E4M3>
struct Shape {
    static constexpr int kKeys = E4M3 ? 2 : 3, kQueries = E4M3 ? 2 : 3, kRaw = E4M3 ? 5 : 0;   // tiles in shared memory
    static constexpr int kThreads = E4M3 ? 512 : 320;
    static constexpr uint32_t kQueriesAt = kKeys * kTileBytes, kRawAt = kQueriesAt + kQueries * kTileBytes;
    static constexpr uint32_t kAlloc = kRawAt + kRaw * kRawBytes + 1024;
};

struct Barriers {
    uint64_t k_full[3], k_empty[3], q_full[3], q_empty[3], raw_full[5], raw_empty[5];
    uint64_t s_full[kBuffers], s_free[kBuffers];
    uint64_t part_full[2], part_free[2];
    uint64_t drain;
};

// Rows of one query tile of a request: `rows` of them, the first token at place `limit`.
struct Queries {
    int64_t row;         // packed token
    int rows, limit;
    __device__ __forceinline__ Queries(const kv::Request &r, int tile, int TB, int G) {
        const int tok = tile * TB;
        row = r.first + tok;
        rows = min(TB, r.count - tok) * G;
        limit = r.len - r.count + tok;
    }
};

template <bool E4M3>
__global__ void __launch_bounds__(Shape<E4M3>::kThreads, 1)
    paged_weights_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ Maps maps) {
    using Layout = Shape<E4M3>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Barriers bar;
    __shared__ __align__(16) float2 stats[8][kTile];   // a warp's own copy of the rows' maxima and 1 / sums
    __shared__ float parts[2][kTile];
    __shared__ uint32_t near[kInline + 1], sums[kInline / 32];
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
            tc::mbar_init(&bar.q_full[i], 1);
            tc::mbar_init(&bar.q_empty[i], 1);
        }
        for (int i = 0; i < Layout::kRaw; ++i) {
            tc::mbar_init(&bar.raw_full[i], 1);
            tc::mbar_init(&bar.raw_empty[i], kConvertWarps);
        }
        for (int i = 0; i < kBuffers; ++i) {
            tc::mbar_init(&bar.s_full[i], 1);
            tc::mbar_init(&bar.s_free[i], 4);
        }
        for (int t = 0; t < 2; ++t) {
            tc::mbar_init(&bar.part_full[t], 4);
            tc::mbar_init(&bar.part_free[t], 4);
        }
        tc::mbar_init(&bar.drain, 1);
        tc::fence_barrier_init();
        abort_flag = 0;
    }
    dependent_start();
    if (!a.weight_start) scan_requests(c, work, near, sums);
    const Starts starts{a.weight_start ? nullptr : near, a.weight_start};
    const int64_t per_head = starts[c.N], all = per_head * c.H;
    const int64_t begin = range_begin(all, cta, gridDim.x), stop = range_begin(all, cta + 1, gridDim.x);
    const bool idle = begin >= stop;
    if (threadIdx.x == 0 && !idle) place = find(c, work, starts, per_head, begin);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    volatile int *const aborted = &abort_flag;
    int *const status = c.status;
    Walk<WeightWork> w;
    if (!idle) w.start_at(c, work, place, begin, stop, cta);

    if (warp == kLoadWarp && !idle) {
        // ---- loads: a cache tile of keys for each unit, query tiles ------------------------------------
        constexpr int kRing = E4M3 ? Layout::kRaw : Layout::kKeys;
        uint64_t *const full = E4M3 ? bar.raw_full : bar.k_full, *const empty = E4M3 ? bar.raw_empty : bar.k_empty;
        uint32_t kt = 0, qt = 0;
        int64_t held_n = -1;   // the request (and head) whose only query tile is in shared memory
        int held_h = -1;
        int page = box_page<E4M3>(c, w.n, w.u, w.r.len, lane);
        bool ok = true;
        do {
            const int st = kt % kRing;
            ok = kt < kRing || wait_or_abort(&empty[st], (kt / kRing - 1) & 1, aborted, status);
            if (!ok) break;
            load_boxes<E4M3>(c, &maps.k, smem + (E4M3 ? Layout::kRawAt + st * kRawBytes : st * kTileBytes), w.u, w.h, page, lane,
                             &full[st]);
            ++kt;
            const bool single = work.query_tiles(w.r.count) == 1;
            if (!(single && held_n == w.n && held_h == w.h)) {
                const int q0 = work.first(w.r.count, w.r.len, w.u);
                for (int i = w.t0; i < w.t1; ++i, ++qt) {
                    const int s = qt % Layout::kQueries;
                    ok = qt < Layout::kQueries || wait_or_abort(&bar.q_empty[s], (qt / Layout::kQueries - 1) & 1, aborted, status);
                    if (!ok) break;
                    if (lane == 0) {
                        const Queries x(w.r, q0 + i, a.TB, a.G);
                        tc::mbar_arrive_expect_tx(&bar.q_full[s], 2 * static_cast<uint32_t>(a.TB * a.G) * 128u);
                        load_query_tile(smem + Layout::kQueriesAt + s * kTileBytes, &maps.q, w.h, a.G, x.row, &bar.q_full[s]);
                    }
                    __syncwarp();
                }
                held_n = single ? w.n : -1;
                held_h = w.h;
            }
            if (!ok || !w.next(c, work, cta)) break;
            page = box_page<E4M3>(c, w.n, w.u, w.r.len, lane);
        } while (true);
        if (!ok) {   // copies in flight land before the CTA ends
            for (uint32_t j = kt > kRing ? kt - kRing : 0; j < kt; ++j)
                tc::mbar_wait(&full[j % kRing], (j / kRing) & 1, tck::kWaitNs);
            for (uint32_t j = qt > Layout::kQueries ? qt - Layout::kQueries : 0; j < qt; ++j)
                tc::mbar_wait(&bar.q_full[j % Layout::kQueries], (j / Layout::kQueries) & 1, tck::kWaitNs);
        }
    } else if (E4M3 && warp >= kConvertWarp && !idle) {
        // ---- e4m3 keys to bf16 ---------------------------------------------------------------------------
        constexpr int kRaw = E4M3 ? Layout::kRaw : 1;
        uint32_t it = 0;
        do {
            const int st = it % Layout::kKeys, rw = it % kRaw;
            if (!wait_or_abort(&bar.raw_full[rw], (it / kRaw) & 1, aborted, status)) break;
            if (it >= Layout::kKeys && !wait_or_abort(&bar.k_empty[st], (it / Layout::kKeys - 1) & 1, aborted, status)) break;
            convert_tile(smem + Layout::kRawAt + rw * kRawBytes, smem + st * kTileBytes, threadIdx.x - 32 * kConvertWarp);
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar.k_full[st]);
                mbar_arrive(&bar.raw_empty[rw]);
            }
            ++it;
        } while (w.next(c, work, cta));
    } else if (warp == kMmaWarp && !idle) {
        // ---- products ------------------------------------------------------------------------------------
        const bool leader = tc::elect_one();
        uint32_t kt = 0, qt = 0, tile = 0;
        int64_t held_n = -1;
        int held_h = -1, held_slot = 0;
        bool ok = true;
        do {
            const int ks = kt % Layout::kKeys;
            const bool single = work.query_tiles(w.r.count) == 1;
            const bool fresh = !(single && held_n == w.n && held_h == w.h);
            if (fresh && held_n >= 0 && leader) tc::umma_commit(&bar.q_empty[held_slot]);
            ok = wait_or_abort(&bar.k_full[ks], (kt / Layout::kKeys) & 1, aborted, status);
            const int q0 = work.first(w.r.count, w.r.len, w.u);
            for (int i = w.t0; i < w.t1 && ok; ++i, ++tile) {
                const Queries x(w.r, q0 + i, a.TB, a.G);
                const int slot = fresh ? qt % Layout::kQueries : held_slot, b = tile % kBuffers;
                if (fresh) {
                    ok = wait_or_abort(&bar.q_full[slot], (qt / Layout::kQueries) & 1, aborted, status);
                    ++qt;
                }
                ok = ok && (tile < kBuffers || wait_or_abort(&bar.s_free[b], (tile / kBuffers - 1) & 1, aborted, status));
                if (!ok) break;
                tc::tc_fence_after();
                if (leader) {
                    const uint32_t id = tc::idesc_bf16_f32(128, (x.rows + 15) & ~15, 0, 0);
                    const uint64_t dk = desc_k(base + ks * kTileBytes), dq = desc_k(base + Layout::kQueriesAt + slot * kTileBytes);
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        const uint32_t off = ((s >> 2) * kHalf + (s & 3) * 32) >> 4;
                        tc::umma_bf16(tmem + b * kTile, dk + off, dq + off, id, s > 0);
                    }
                    tc::umma_commit(&bar.s_full[b]);
                    if (!single) tc::umma_commit(&bar.q_empty[slot]);
                }
                __syncwarp();
                held_slot = slot;
            }
            if (!ok) break;
            held_n = single ? w.n : -1;
            held_h = w.h;
            if (leader) tc::umma_commit(&bar.k_empty[ks]);
            __syncwarp();
            ++kt;
        } while (w.next(c, work, cta));
        if (!ok) {   // products in flight end before the tensor memory is freed
            if (leader) {
                tc::umma_commit(&bar.drain);
                tc::mbar_wait(&bar.drain, 0, tck::kWaitNs);
            }
            __syncwarp();
        }
    } else if (warp < kMmaWarp && !idle) {
        // ---- sums: a place a thread ------------------------------------------------------------------------
        const int g = warp >> 2, r = threadIdx.x & (kTile - 1), Hq = a.G * c.H;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        float2 *const mine = stats[warp];
        uint32_t tile = 0, sent = 0, got = 0;
        bool ok = true;
        do {
            const int m = w.t1 - w.t0, q0 = work.first(w.r.count, w.r.len, w.u) + w.t0, p = w.u * kTile + r;
            const int owner = tile & 1;
            const float scale = a.scale * (c.k_scale ? __ldg(c.k_scale + w.h) : 1.f) * kLog2e;
            float2 next[4];
            auto fetch = [&](int i) {   // the statistics of the rows 32 e + lane of query tile i of the item
                const Queries x(w.r, q0 + i, a.TB, a.G);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = 32 * e + lane, tok = row / a.G;
                    next[e] = row < x.rows ? a.stats[(x.row + tok) * Hq + w.h * a.G + row - tok * a.G] : make_float2(0.f, 0.f);
                }
            };
            float total = 0.f;
            int i = (tile & 1) == g ? 0 : 1;
            if (i < m) fetch(i);
            for (; i < m; i += 2) {
                const uint32_t k = tile + i, b = k % kBuffers;
                const Queries x(w.r, q0 + i, a.TB, a.G);
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 4; ++e) mine[32 * e + lane] = next[e];
                __syncwarp();
                if (i + 2 < m) fetch(i + 2);
                ok = wait_or_abort(&bar.s_full[b], (k / kBuffers) & 1, aborted, status);
                if (!ok) break;
                tc::tc_fence_after();
                const bool full = x.rows == kTile && x.limit >= w.u * kTile + kTile - 1;
                const int ahead = p - x.limit, from = ahead <= 0 ? 0 : ahead >= a.TB ? kTile : ahead * a.G;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (32 * q >= x.rows) break;
                    uint32_t s[32];
                    tc::tmem_ld_32x32b_x32(tmem + b * kTile + 32 * q + lanes, s);
                    tc::tmem_ld_wait();
                    const float4 *st = reinterpret_cast<const float4 *>(mine + 32 * q);
                    if (full) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float4 y = st[j];
                            const float e0 = tc::ex2(fmaf(__uint_as_float(s[2 * j]), scale, -y.x));
                            const float e1 = tc::ex2(fmaf(__uint_as_float(s[2 * j + 1]), scale, -y.z));
                            sum[(2 * j) & 3] = fmaf(e0, y.y, sum[(2 * j) & 3]);
                            sum[(2 * j + 1) & 3] = fmaf(e1, y.w, sum[(2 * j + 1) & 3]);
                        }
                    } else {   // rows that see the place: not before `from`, not behind the last
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float4 y = st[j];
                            const int n = 32 * q + 2 * j;
                            const float e0 = tc::ex2(fmaf(__uint_as_float(s[2 * j]), scale, -y.x)) * y.y;
                            const float e1 = tc::ex2(fmaf(__uint_as_float(s[2 * j + 1]), scale, -y.z)) * y.w;
                            sum[(2 * j) & 3] += n >= from && n < x.rows ? e0 : 0.f;
                            sum[(2 * j + 1) & 3] += n + 1 >= from && n + 1 < x.rows ? e1 : 0.f;
                        }
                    }
                }
                total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.s_free[b]);
            }
            if (!ok) break;
            if (m > 1 && g != owner) {   // to the warpgroup that has the unit's first query tile
                ok = sent == 0 || wait_or_abort(&bar.part_free[g], (sent - 1) & 1, aborted, status);
                if (!ok) break;
                parts[g][r] = total;
                ++sent;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.part_full[g]);
            } else if (m > 1) {
                ok = wait_or_abort(&bar.part_full[1 - g], got & 1, aborted, status);
                if (!ok) break;
                total += parts[1 - g][r];
                ++got;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.part_free[1 - g]);
            }
            if (g == owner) {
                if (w.slot >= 0) {
                    a.part_w[static_cast<int64_t>(w.slot) * kTile + r] = total;
                } else if (p < w.r.len) {
                    const int page = kv::page_of(c, w.n, p);
                    if (page >= 0) c.weights[kv::row_of(c, page, w.h, p)] += total;
                }
            }
            tile += m;
        } while (w.next(c, work, cta));
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// Adds the partial sums of units that several CTAs share, in the order of the CTAs.
__global__ void __launch_bounds__(kInline) paged_weights_join_kernel(const AttendArgs a, int ctas) {
    __shared__ uint32_t near[kInline + 1], sums[kInline / 32];
    __shared__ Place place;
    dependent_start();
    const KvArgs &c = a.c;
    const WeightWork work{a.TB};
    if (!a.weight_start) scan_requests(c, work, near, sums);
    const Starts starts{a.weight_start ? nullptr : near, a.weight_start};
    const int64_t per_head = starts[c.N], all = per_head * c.H;
    const int cta = blockIdx.x, r = threadIdx.x;
    const int64_t r0 = range_begin(all, cta, ctas), r1 = range_begin(all, cta + 1, ctas);
    if (r0 >= r1 || r1 >= all) return;
    if (r == 0) place = find(c, work, starts, per_head, r1 - 1);
    __syncthreads();
    const kv::Request q = kv::request(c, place.n);
    const int64_t from = place.begin, to = from + work.tiles(q.count, q.len, place.u);
    const int64_t p = static_cast<int64_t>(place.u) * kTile + r;
    if (from < r0 || to <= r1 || r >= kTile || p >= q.len) return;
    const int parts = cta_of(all, to - 1, ctas) - cta + 1;
    float sum = 0.f;
    for (int i = 0; i < parts; ++i) sum += a.part_w[part_slot(cta, i) * kTile + r];
    const int page = kv::page_of(c, place.n, static_cast<int>(p));
    if (page >= 0) c.weights[kv::row_of(c, page, place.h, static_cast<int>(p))] += sum;
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
    return launch_dependent(paged_weights_join_kernel, dim3(ctas), kInline, st, a, ctas);
}

}  // namespace pt
}  // namespace sala

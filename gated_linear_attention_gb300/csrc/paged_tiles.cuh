// What the kernels over a paged cache's tiles share (internal): the split of the work over the CTAs, the shared-
// memory tiles, and how they are filled.
#pragma once

#include "chunk_tc.cuh"
#include "kv_cache.cuh"

namespace sala {
namespace pt {

constexpr int kTile = 128;                       // rows of a query tile, places of a cache tile
constexpr uint32_t kHalf = kTile * 128;          // bytes of [128 rows x 64 bf16], 128-byte swizzle
constexpr uint32_t kTileBytes = 2 * kHalf;
constexpr uint32_t kRawBytes = kTile * kD;       // bytes of a tile of e4m3 values
constexpr int kInline = 256;                     // requests whose prefix every CTA takes for itself
constexpr int kConvertWarps = 8;                 // that widen e4m3 tiles
constexpr int kPieces = 1024 / (32 * kConvertWarps);   // 16-byte pieces of a tile a thread
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// ---- work ----------------------------------------------------------------------------------------

// sum of floor((a i + b) / m) for 0 <= i < n (b >= 0): the remainders' part turns into a sum of the same
// kind with a and m exchanged, as in the Euclidean algorithm.
__host__ __device__ inline int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
    int64_t sum = 0;
    while (true) {
        if (a >= m) sum += n * (n - 1) / 2 * (a / m), a %= m;
        if (b >= m) sum += n * (b / m), b %= m;
        const int64_t y = a * n + b;
        if (y < m) return sum;
        n = y / m;
        b = y % m;
        const int64_t t = m;
        m = a;
        a = t;
    }
}

// x / y for 0 <= x < 2^32 and y > 0: 64-bit divisions are slow.
__host__ __device__ inline int divide(int64_t x, int y) {
    return static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y));
}

// Attention: unit u of a request is its tokens [u * block, (u + 1) * block) with the cache tiles up to the last
// place that they see.
struct AttendWork {
    int block;
    __host__ __device__ int units(int count, int) const { return divide(static_cast<int64_t>(count) + block - 1, block); }
    __host__ __device__ int64_t tiles(int count, int len, int u) const {
        const int64_t base = static_cast<int64_t>(len) - count;
        // more tokens than places: each unit takes all of them, which is more than some see
        const int64_t to = static_cast<int64_t>(u + 1) * block;
        const int64_t end = base < 0 ? len : base + (to < count ? to : count);
        return end > 0 ? (end + kTile - 1) / kTile : 1;
    }
    // tiles of the units before u; u is at most the number of units less 1
    __host__ __device__ int64_t before(int count, int len, int u) const {
        const int64_t base = static_cast<int64_t>(len) - count;
        if (base < 0 || u == 0) return u * tiles(count, len, 0);
        return floor_sum(u, kTile, block, base + block + kTile - 1);
    }
};

// Weights: unit u of a request is its cache tile u with the query tiles (of `block` tokens) that see it.
struct WeightWork {
    int block;
    __host__ __device__ int units(int count, int len) const { return count > 0 ? (len + kTile - 1) / kTile : 0; }
    __host__ __device__ int query_tiles(int count) const { return divide(static_cast<int64_t>(count) + block - 1, block); }
    __host__ __device__ int first(int count, int len, int u) const {
        const int64_t from = static_cast<int64_t>(u) * kTile - (static_cast<int64_t>(len) - count);
        return from > 0 ? divide(from, block) : 0;   // below count
    }
    __host__ __device__ int64_t tiles(int count, int len, int u) const { return query_tiles(count) - first(count, len, u); }
    __host__ __device__ int64_t before(int count, int len, int u) const {
        const int64_t base = static_cast<int64_t>(len) - count;
        const int64_t u0 = base > 0 ? (base + kTile - 1) / kTile : 0;
        const int64_t all = static_cast<int64_t>(u) * query_tiles(count);
        return u > u0 && query_tiles(count) > 1 ? all - floor_sum(u - u0, block, kTile, u0 * kTile - base) : all;
    }
};

template <class Work>
__host__ __device__ inline int64_t tiles_of(const Work &w, int count, int len) {
    const int units = w.units(count, len);
    return units > 0 ? w.before(count, len, units - 1) + w.tiles(count, len, units - 1) : 0;
}

// The requests' running sums of tiles (of one key/value head), N + 1 of them: in shared memory for up to
// kInline requests, else in global memory, from the plan kernel.
struct Starts {
    const uint32_t *near;
    const int64_t *far;
    __device__ __forceinline__ int64_t operator[](int64_t n) const { return near ? near[n] : far[n]; }
};

// A CTA's range of the flattened tiles (key/value head outermost). With fewer tiles than CTAs the first
// CTAs get one each, so that no range among those that share a unit is empty.
__host__ __device__ inline int64_t range_begin(int64_t tiles, int cta, int ctas) {
    if (tiles <= ctas) return cta < tiles ? cta : tiles;
    if (tiles >> 32) return tiles / ctas * cta + tiles % ctas * cta / ctas;
    const uint32_t q = static_cast<uint32_t>(tiles) / ctas, rest = static_cast<uint32_t>(tiles) - q * ctas;   // 64-bit divisions are slow
    return static_cast<int64_t>(q) * cta + rest * cta / ctas;
}
// The CTA that has tile `at`.
__host__ __device__ inline int cta_of(int64_t tiles, int64_t at, int ctas) {
    if (tiles <= ctas) return static_cast<int>(at);
    int cta = static_cast<int>(at / (tiles / ctas + 1));   // at most the one sought
    while (range_begin(tiles, cta + 1, ctas) <= at) ++cta;
    return cta;
}

// Threads 0 .. kInline - 1 of a CTA: running sums of the requests' tiles into `start` [N + 1], N <= kInline.
// `sums` holds kInline / 32 words. Ends with a barrier of the whole CTA.
template <class Work>
__device__ __forceinline__ void scan_requests(const KvArgs &c, const Work &work, uint32_t *start, uint32_t *sums) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t x = 0;
    if (tid < c.N) {
        const kv::Request r = kv::request(c, tid);
        x = static_cast<uint32_t>(tiles_of(work, r.count, r.len));
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31 && warp < kInline / 32) sums[warp] = x;
    __syncthreads();
    if (tid < kInline) {
        for (int w = 0; w < warp; ++w) x += sums[w];
        if (tid < c.N) start[tid + 1] = x;
        if (tid == 0) start[0] = 0;
    }
    __syncthreads();
}

// Where a flattened tile lies: key/value head, request, unit (with its first tile).
struct Place {
    int h, u;
    int64_t n, begin;
};
template <class Work>
__device__ __forceinline__ Place find(const KvArgs &c, const Work &work, const Starts &start, int64_t per_head, int64_t at) {
    Place p;
    p.h = at >> 32 || per_head >> 32 ? static_cast<int>(at / per_head) : divide(at, static_cast<int>(per_head));
    at -= per_head * p.h;
    int64_t lo = 0, hi = c.N;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (start[mid] <= at) lo = mid;
        else hi = mid;
    }
    p.n = lo;
    const kv::Request r = kv::request(c, lo);
    at -= start[lo];
    int a = 0, b = work.units(r.count, r.len);
    while (b - a > 1) {
        const int mid = a + (b - a) / 2;
        if (work.before(r.count, r.len, mid) <= at) a = mid;
        else b = mid;
    }
    p.u = a;
    p.begin = per_head * p.h + start[lo] + work.before(r.count, r.len, a);
    return p;
}

// Walks the items of a CTA: a range [t0, t1) of the tiles of one unit.
template <class Work>
struct Walk {
    int64_t pos, end, n;
    int h, u, units, tiles, t0, t1;
    int slot;            // where a partial result goes, -1: the item is the whole unit
    kv::Request r;

    __device__ __forceinline__ void enter(const Work &work, int cta, int64_t unit_begin) {
        tiles = static_cast<int>(work.tiles(r.count, r.len, u));
        t0 = static_cast<int>(pos - unit_begin);
        const int64_t left = end - unit_begin;
        t1 = left < tiles ? static_cast<int>(left) : tiles;
        slot = t0 == 0 && t1 == tiles ? -1 : 2 * cta + (t0 == 0 ? 1 : 0);
    }
    // the range [from, to), whose first tile lies at p
    __device__ __forceinline__ void start_at(const KvArgs &c, const Work &work, const Place &p, int64_t from, int64_t to, int cta) {
        pos = from;
        end = to;
        h = p.h;
        n = p.n;
        u = p.u;
        r = kv::request(c, n);
        units = work.units(r.count, r.len);
        enter(work, cta, p.begin);
    }
    __device__ __forceinline__ bool next(const KvArgs &c, const Work &work, int cta) {
        pos += t1 - t0;
        if (pos >= end) return false;
        if (++u == units) {
            u = 0;
            do {   // requests without tiles are passed over; one that has some is ahead, as pos < end
                if (++n == c.N) {
                    n = 0;
                    if (++h == c.H) return false;   // the lengths changed under the call
                }
                r = kv::request(c, n);
                units = work.units(r.count, r.len);
            } while (units == 0);
        }
        enter(work, cta, pos);
        return true;
    }
};

// Parts of a unit whose first CTA is `cta`: the slot of part p.
__device__ __forceinline__ int64_t part_slot(int cta, int p) { return 2 * static_cast<int64_t>(cta + p) + (p == 0 ? 1 : 0); }

// ---- tiles ----------------------------------------------------------------------------------------

// Offset in bytes of the 16-byte piece `piece` (of 16) of a row in a bf16 tile.
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
    return (piece >> 3) * kHalf + tck::sw(row, piece & 7);
}
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
    return tc::smem_desc_sw128(0, 16, 1024) | ((addr >> 4) & 0x3FFFu);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
    return tc::smem_desc_sw128(0, kHalf, 1024) | ((addr >> 4) & 0x3FFFu);
}

// A cache tile's boxes, one page (at most 128 places) each, and for bf16 one half of the dimensions: lane l of the
// loading warp has one. Looks up the page of this lane's box: -2: no box, or all of it at or behind `end`.
template <bool E4M3>
__device__ __forceinline__ int box_page(const KvArgs &c, int64_t n, int tile, int end, int lane) {
    const int box = min(c.S, kTile), bx = E4M3 ? lane : lane >> 1;
    const int place = tile * kTile + bx * box;
    return bx < kTile / box && place < end ? kv::page_of(c, n, place) : -2;
}

// Issues the boxes of a tile into `dst` (the whole warp); `bar` gets their bytes.
template <bool E4M3>
__device__ __forceinline__ void load_boxes(const KvArgs &c, const CUtensorMap *map, uint8_t *dst, int tile, int h, int page,
                                           int lane, uint64_t *bar) {
    const int box = min(c.S, kTile);
    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, page != -2)) * static_cast<uint32_t>(box) * 128u;
    if (lane == 0) {
        if (bytes) tc::mbar_arrive_expect_tx(bar, bytes);
        else tc::mbar_arrive(bar);
    }
    __syncwarp();
    if (page != -2) {
        const int y = c.S > kTile ? (tile & 1) * kTile : 0, z = (page < 0 ? 0 : page) * c.H + h;   // an unknown page: any
        if constexpr (E4M3) tc::tma_load_3d(dst + lane * box * kD, map, 0, y, z, bar);
        else tc::tma_load_3d(dst + (lane & 1) * kHalf + (lane >> 1) * box * 128, map, (lane & 1) * 64, y, z, bar);
    }
    __syncwarp();
}

// Thread id's pieces of an e4m3 tile: eight lanes take two rows, the left half of one and the right half of the other, so
// that loads and stores fall on all banks.
__device__ __forceinline__ int piece_row(int id, int e) { return 2 * (((id >> 3) + e * 4 * kConvertWarps) >> 1) + (id >> 2 & 1); }
__device__ __forceinline__ int piece_of_row(int id) { return (id & 3) + 4 * ((id >> 3 & 1) ^ (id >> 2 & 1)); }
__device__ __forceinline__ void read_pieces(uint4 (&x)[kPieces], const uint8_t *raw, int id) {
#pragma unroll
    for (int e = 0; e < kPieces; ++e)
        x[e] = *reinterpret_cast<const uint4 *>(raw + piece_row(id, e) * kD + piece_of_row(id) * 16);
}
// Stores them as bf16 (exact).
__device__ __forceinline__ void store_pieces(const uint4 (&x)[kPieces], uint8_t *dst, int id) {
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
        const int row = piece_row(id, e), p = piece_of_row(id);
        const uint32_t in[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
        uint32_t out[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float2 f = kv::e4m3x2_to_float2(q & 1 ? in[q >> 1] >> 16 : in[q >> 1] & 0xffffu);
            out[q] = float2_to_bf16x2(f.x, f.y);
        }
        *reinterpret_cast<uint4 *>(dst + piece_at(row, 2 * p)) = make_uint4(out[0], out[1], out[2], out[3]);
        *reinterpret_cast<uint4 *>(dst + piece_at(row, 2 * p + 1)) = make_uint4(out[4], out[5], out[6], out[7]);
    }
}

// ---- waits ----------------------------------------------------------------------------------------
// A wait of a whole warp. By itself a lane may run out of time, or see that another role gave up, where its neighbour sees
// the phase complete; what follows may need the whole warp (tensor memory, shuffles, votes), so that the lanes go by a vote.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *status) {
    if (__all_sync(0xffffffffu, tc::mbar_test_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, tck::wait_or_abort_slow(bar, parity, abort_flag, status)) != 0;
}

// ---- barriers by their shared-memory address --------------------------------------------------------
// The warp that issues the products pays for every scalar instruction between two of them (its queue is short), so it
// keeps addresses, stages and parities in registers.

static __device__ __noinline__ bool wait_at_slow(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *status) {
    const uint64_t t0 = tc::global_timer_ns();
    while (true) {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        if (ok) return true;
        if (*abort_flag) return false;
        if (tc::global_timer_ns() - t0 > tck::kWaitNs) {
            *abort_flag = 1;
            record_status(status, SALA_ERR_TIMEOUT);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_at(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *status) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok || wait_at_slow(bar, parity, abort_flag, status);
}
__device__ __forceinline__ void commit_at(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// A place in a ring of N stages and the parity of its phase.
template <int N>
struct Ring {
    uint32_t at = 0, parity = 0;
    __device__ __forceinline__ void advance(uint32_t n) {   // n <= N
        at += n;
        if (at >= N) at -= N, parity ^= 1u;
    }
};

// Query rows: `tokens` tokens of the group's G heads from packed token `row` (rows past the end are zeros).
__device__ __forceinline__ void load_query_tile(uint8_t *dst, const CUtensorMap *map, int h, int G, int64_t row, uint64_t *bar) {
    for (int half = 0; half < 2; ++half)
        tc::tma_load_3d(dst + half * kHalf, map, half * 64, h * G, static_cast<int>(row), bar);
}

struct Maps {
    CUtensorMap q, k, v;
};

// ---- kernels' arguments ----------------------------------------------------------------------------

struct AttendArgs {
    KvArgs c;
    const int64_t *attend_start, *weight_start;   // [N + 1] running sums of tiles, null: each CTA takes them
    void *joins, *weight_joins;   // [CTAs] units that several CTAs share
    float *part_o;       // [2 * CTAs, 256, 128] partial O
    float2 *part_ml;     // [2 * CTAs, 256] its maximum (in units of the scores) and sum
    float *stats;        // [T, Hq] log of each row's sum of exponentials, in units of the scores, or null
    float *part_w;       // [2 * CTAs, 128] partial sums of weights
    uint16_t *o;
    float *lse;
    float scale;
    int G, TB;           // query heads on a key/value head, tokens of a query tile
};

cudaError_t setup_paged_weights_kernel();
cudaError_t launch_paged_weights(const AttendArgs &a, const Maps &maps, int ctas, cudaStream_t st);

}  // namespace pt
}  // namespace sala

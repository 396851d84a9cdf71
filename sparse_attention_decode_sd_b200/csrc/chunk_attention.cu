// chunk_attention.cu -- causal attention of each request's newest positions over its paged cache.
//
//   out[t, h] = sum_i w_i V[b, h/G, i],  w = softmax over 0 <= i <= p of (q[t, h] . K[b, h/G, i]) / sqrt(d)
//
// for row t = row_start[b] + j at position p = N_b - n_b + j.
//
// Rows of a tile.  The G query heads of a KV head read the same K and V, so a tile of 128 rows holds
// floor(128 / G) consecutive tokens times the G heads of one group.  Two tiles make an item (256 rows, one KV
// head of one request); its key/value tiles of 128 positions (and a few more for the item itself) are the units of work,
// and all units of the batch are cut evenly over one CTA per SM (each CTA works out its share from row_start and lens, so there
// is no planning launch).  An item cut by a CTA's border leaves its partial (max, sum, output) in the
// workspace, and merge_chunks_kernel joins the parts in order: the same result every time.
//
// One CTA, warp-specialised around tensor memory (512 columns: scores of the two tiles, outputs of the two
// tiles), with
//   warps 0-3, 4-7   softmax of tile 0 and tile 1, one row per thread
//   warps 8, 10      copies: K and V page by page (one TMA box of 16 rows x 64 values per page and half, in
//                    the 128-byte swizzle, into a ring of 32 KB stages), the two tiles of q
//   warp 9           MMAs (one thread): S = Q K^T from shared memory, O += P V with P in tensor memory
//   warps 12-19      8-bit caches: raw tiles (16 KB + scales) to bf16 stages, exact
// While one tile's warps take the softmax of a unit, the tensor cores work on the other tile: per unit
// P0 V, Q0 K', P1 V, Q1 K' (K' the next unit's keys), so both are busy in turn.  P (bf16) overwrites the first
// half of its scores.
//
// The softmax is what the tensor cores wait for, so it does little per score: one FMA, one exponential, one
// addition, half a conversion.  Weights are exp2(s - m) for a reference m that need not be the running maximum, only
// near it: a row takes its first tile's maximum, and a new one (with its sum and output rescaled, and the tile taken
// again) when a tile's sum passes 2^14, which also catches infinities.  Sums and outputs are fp32 and bf16 has the
// same precision at every magnitude, so nothing is lost.  All exponentials are the special-function unit's: a weight that
// is 0 is exactly 0 and NaN stays NaN.  (A cubic on the FMA pipe for two of eight pairs took 381 us instead of 389 for
// prompts of 1000-4096 tokens, 3.72 ms instead of 3.76 for a long chunk and the same over 8-bit caches, but has to be
// clamped, so that what does not count weighed 2^-112; one more addition to take that off again costs what it gains.)  A
// tile of 128 x 128 takes about 3200 cycles with the wait for its products, where the MMAs of the pair take 2048.
//
// Items of one tile (few tokens: decode, short chunks) split their units between the two warpgroups, even and odd,
// each with a maximum, sum and output of its own, joined at the end: the two sides stay busy in turn all the same.
#include <cuda.h>

#include "cache_format.cuh"
#include "kernels.h"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace sd {

namespace {

constexpr int kTileRows = 128;                 // rows of a query tile, positions of a key/value tile
constexpr int kHalf = 16 * 1024;               // 128 rows of 64 bf16 values
constexpr int kStageBytes = 2 * kHalf;         // a K or V tile in bf16
constexpr int kRawBytes = 16 * 1024;           // the same in 8 bits
constexpr int kScaleTile = 1024;               // scales of K and V of 128 positions
constexpr int kExpandThreads = 256;            // that expand 8-bit tiles (half of them take twice as long: latency)
// What an item costs besides its tiles, in tiles: its first reference, the wait for its last product, its output.  (About
// 10000 cycles, 3300 to a tile.  Counted as 0, CTAs with many short items end last: prompts of 1000-4096 tokens
// took 472 us instead of 400, one of 8192 562 instead of 466; 2: 413 and 481; 4: 402 and 471.)
constexpr int kItemCost = 3;
constexpr float kFarAbove = 16384.f;            // sum of a tile's weights from which its row takes a new reference

template <int kFmt>
struct Layout {
    static constexpr bool k8 = kFmt != kFmtBf16;
    static constexpr int kStages = k8 ? 3 : 5;
    static constexpr int kRaw = k8 ? 3 : 1;
    static constexpr int kScaleSlots = k8 ? 3 : 1;   // (K tile t + 3 is copied only after V tile t is expanded)
    static constexpr int kQ = 0;
    static constexpr int kKv = 2 * kStageBytes;
    static constexpr int kRawOff = kKv + kStages * kStageBytes;
    static constexpr int kScaleOff = kRawOff + (k8 ? kRaw * kRawBytes : 0);
    static constexpr int kCtl = kScaleOff + (k8 ? kScaleSlots * kScaleTile : 0);
    static constexpr int kThreads = k8 ? 640 : 384;
};

struct Request {
    int rs, n, base;   // first row, new rows, positions before them
};

constexpr int kSegments = 4;   // stretches that the copies may run ahead

// One stretch of consecutive units of one item.
struct Segment {
    int b, kvh;
    int rows;     // first row (token) of the item in q and out
    int tokens;   // tokens of the item
    int first;    // position of its first token
    int end;      // positions that its last token sees
    int j0, j1;   // key/value tiles of the stretch (none: the share has ended)
    int tiles;    // key/value tiles of the item
    int last;     // the CTA that has the item's last unit, if the item begins here and goes on there, else -1
    int two;      // the item has a second tile of rows
};

struct Control {
    uint64_t q_full[2], q_empty[2];
    uint64_t kv_full[5], kv_empty[5];
    uint64_t raw_full[3], raw_empty[3];
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t join[2], done;
    uint64_t seg_full[kSegments], seg_empty[kSegments];
    Segment seg[kSegments];
    uint32_t tmem;
    int dead;                // a wait ran out: nothing more is issued
    int b, kvh, pair, unit;  // where this CTA's share starts
    Request start;           // the request of b
    long long scan[20];
    float2 post[2 * kTileRows];   // maximum and sum of the two sides of a one-tile item
};

template <int kFmt>
constexpr int chunk_smem() {
    return Layout<kFmt>::kCtl + (int)sizeof(Control);
}
static_assert(chunk_smem<kFmtBf16>() <= 227 * 1024 && chunk_smem<kFmtFp8>() <= 227 * 1024, "shared memory");

// A bounded wait of a converged warp; false for the whole warp once this or any other wait of the block has run out.
// The caller then leaves its role without another arrival or copy: a barrier that others still use gets no arrival that
// they do not expect.  (The timer and the flag are looked at now and then: reading them in every round costs latency.)
__device__ __forceinline__ bool pipe_wait(uint64_t* bar, uint32_t parity, int* dead, int32_t* status, uint64_t* also = nullptr,
                                          uint32_t also_parity = 0) {
    auto there = [&]() { return mbar_try_wait(bar, parity) && (also == nullptr || mbar_try_wait(also, also_parity)); };
    bool ok = there();
    if (!ok) {
        uint64_t t0 = 0;
        for (uint32_t it = 0; it < kWaitLimitIters && !ok; ++it) {
            ok = there();
            if (!ok && (it & 31) == 31) {
                if (*reinterpret_cast<volatile int*>(dead)) break;
                const uint64_t now = global_timer_ns();
                if (t0 == 0) t0 = now;
                if (now - t0 > kWaitLimitNs) break;
            }
        }
        if (!ok && *reinterpret_cast<volatile int*>(dead) == 0) {
            *reinterpret_cast<volatile int*>(dead) = 1;
            report(status, SD_ERR_TIMEOUT);
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// ---- the batch as units --------------------------------------------------------------------------------
__device__ __forceinline__ Request request(const ChunkArgs& a, int b) {
    Request r;
    r.rs = a.row_start[b];
    r.n = a.row_start[b + 1] - r.rs;
    const int N = a.lens[b];
    r.base = N - r.n;
    if (N < 0 || (long)N > a.n_cap || r.base < 0 || r.n <= a.few) r.n = 0;   // (reported where the shares are worked out)
    return r;
}

// Units of item i of a request: a key/value tile each of the positions that its last token sees, behind kItemCost units
// without a tile for what an item costs besides.  w tokens to an item.
__device__ __forceinline__ int item_units(const Request& r, int i, int w) {
    return kItemCost + (r.base + min(r.n, (i + 1) * w) + kTileRows - 1) / kTileRows;
}
// Units of items 0 .. i - 1.  Over p = 128 / gcd(w, 128) items their number grows by w p / 128 each, so the
// sum over whole periods has a closed form.
__device__ __forceinline__ long long units_before(const Request& r, int i, int items, int w) {
    const int k = min(i, items - 1);
    const int p = kTileRows / min(kTileRows, w & -w), s = w * p / kTileRows;
    const int whole = k / p, rest = k - whole * p;
    long long sum = 0, first = 0;
    if (whole > 0) {
        for (int x = 0; x < p; ++x) first += item_units(r, x, w);
        sum = whole * first + (long long)p * s * whole * (whole - 1) / 2;
    }
    for (int x = 0; x < rest; ++x) sum += item_units(r, x, w) + (long long)whole * s;
    if (i == items) sum += item_units(r, items - 1, w);
    return sum;
}

// CTAs that get units: each of them at least one, so that the parts of a cut item lie in neighbouring CTAs (those that have
// tiles of it: an item's units without a tile come first).
__device__ __forceinline__ long long shares(long long total) { return min(total, (long long)gridDim.x); }

// The first unit of CTA c's share.  (A 64-bit division costs hundreds of cycles, and the start of a short call counts.)
__device__ __forceinline__ long long share_begin(long long total, uint32_t c) {
    const uint32_t parts = (uint32_t)shares(total);
    if (c >= parts) return total;
    if (total < (1ll << 24)) return (uint32_t)total * c / parts;   // (c is below 2^8)
    return total * c / parts;
}

// The CTA that has unit end - 1.
__device__ __forceinline__ int last_share(long long total, long long end) {
    const uint32_t parts = (uint32_t)shares(total);
    if (total < (1ll << 24)) return (int)(((uint32_t)end * parts - 1) / (uint32_t)total);
    return (int)((end * parts - 1) / total);
}

// A CTA's share as stretches, for the copy warp.
struct Walk {
    const ChunkArgs& a;
    int w, b, kvh, i, j, items;
    long long left, u1, total;
    Request r;
    __device__ Walk(const ChunkArgs& args, const Control& c, long long begin, long long end, long long all)
        : a(args), w(2 * args.tpt), b(c.b), kvh(c.kvh), i(c.pair), j(c.unit), left(end - begin), u1(end), total(all) {
        if (left > 0) {
            r = c.start;
            items = (r.n + w - 1) / w;
        }
    }
    __device__ __forceinline__ bool next(Segment& s) {
        if (left <= 0) return false;
        s.b = b;
        s.kvh = kvh;
        s.rows = r.rs + i * w;
        s.tokens = min(w, r.n - i * w);
        s.first = r.base + i * w;
        s.end = s.first + s.tokens;
        s.tiles = (s.end + kTileRows - 1) / kTileRows;
        const int units = kItemCost + s.tiles, to = (int)min((long long)units, j + left);
        s.j0 = max(0, j - kItemCost);
        s.j1 = max(0, to - kItemCost);
        s.two = s.tokens > a.tpt ? 1 : 0;
        left -= to - j;
        if (s.j1 == s.j0) return false;   // (the share ends before the item's first tile: the next one begins it)
        s.last = -1;
        if (left == 0 && s.j0 == 0 && s.j1 < s.tiles)
            s.last = last_share(total, u1 - to + units);
        if (left > 0) {   // the stretch ended with its item
            j = 0;
            if (++i == items) {
                i = 0;
                if (++kvh == a.Hkv) {
                    kvh = 0;
                    do {
                        r = request(a, ++b);
                    } while (r.n == 0);
                    items = (r.n + w - 1) / w;
                }
            }
        }
        return true;
    }
};

// What the merge needs of a CTA whose last item goes on in later CTAs (valid), written by every CTA.
struct TailRecord {
    int valid, rows, tokens, kvh, last, pad[3];
};

// A slot: [32 chunks of four dimensions][256 rows], so that the threads that hold a row each write whole lines.
__device__ __forceinline__ float4* slot_out(const ChunkArgs& a, int slot, int chunk) {
    return reinterpret_cast<float4*>(a.part) + ((long)slot * (kHeadDim / 4) + chunk) * (2 * kTileRows);
}
__device__ __forceinline__ float2* slot_ml(const ChunkArgs& a, int slot) { return a.ml + (long)slot * (2 * kTileRows); }

// The block's share [u0, u1) of the batch's units, its start in `c`, and the checks of row_start and lens.
// False where row_start is not valid (nothing is done then).
__device__ __forceinline__ bool plan(const ChunkArgs& a, Control& c, long long& u0, long long& u1, long long& total) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int per = (a.B + blockDim.x - 1) / blockDim.x, w = 2 * a.tpt;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    bool bad = false;
    long long mine = 0, head = 0;   // (head, last: of the thread's last request, most often its only one)
    Request last = {0, 0, 0};
    for (int b = b0; b < b1; ++b) {
        const int lo = a.row_start[b], hi = a.row_start[b + 1];
        bad = bad || lo < 0 || hi < lo || hi > a.total_rows;
        const int N = a.lens[b];
        if (N < 0 || (long)N > a.n_cap || (hi > lo && hi - lo > N)) {
            if (blockIdx.x == 0) report(a.status, SD_ERR_INVALID_ARG);
            continue;
        }
        if (bad || hi - lo <= a.few) continue;
        last = Request{lo, hi - lo, N - (hi - lo)};
        const int items = (last.n + w - 1) / w;
        head = units_before(last, items, items, w);
        mine += a.Hkv * head;
    }
    if (__syncthreads_or(bad ? 1 : 0)) {
        if (tid == 0 && blockIdx.x == 0) report(a.status, SD_ERR_INVALID_ARG);
        total = u0 = u1 = 0;
        return false;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) c.scan[warp] = incl;
    __syncthreads();
    long long before = incl - mine;
    total = 0;
    for (int x = 0; x < warps; ++x) {
        if (x < warp) before += c.scan[x];
        total += c.scan[x];
    }
    u0 = share_begin(total, blockIdx.x);
    u1 = share_begin(total, blockIdx.x + 1);
    if (u1 > u0 && before <= u0 && u0 < before + mine) {   // the share starts in this thread's requests
        long long at = u0 - before;
        for (int b = b0; b < b1; ++b) {
            const Request r = per == 1 ? last : request(a, b);
            if (r.n == 0) continue;
            const int items = (r.n + w - 1) / w;
            if (per > 1) head = units_before(r, items, items, w);
            if (at >= head * a.Hkv) {
                at -= head * a.Hkv;
                continue;
            }
            c.b = b;
            c.start = r;
            c.kvh = at < (1ll << 31) && head < (1ll << 31) ? (int)((uint32_t)at / (uint32_t)head) : (int)(at / head);
            at -= c.kvh * head;
            int lo = 0, hi = items - 1;   // the last item with units_before <= at
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (units_before(r, mid, items, w) <= at) lo = mid;
                else hi = mid - 1;
            }
            c.pair = lo;
            c.unit = (int)(at - units_before(r, lo, items, w));
            break;
        }
    }
    __syncthreads();
    return true;
}

// The stretches in order, as the copy warp hands them out; one arrival per warp gives a slot back.
struct Stretches {
    Control& c;
    int32_t* status;
    uint32_t n;
    __device__ Stretches(Control& control, int32_t* st) : c(control), status(st), n(0) {}
    __device__ __forceinline__ const Segment* next() {   // null: no more
        const uint32_t slot = n % kSegments;
        const Segment* s = &c.seg[slot];
        return pipe_wait(&c.seg_full[slot], (n / kSegments) & 1, &c.dead, status) && s->j1 > s->j0 ? s : nullptr;
    }
    __device__ __forceinline__ void done() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&c.seg_empty[n % kSegments]);
        ++n;
    }
};

// The order of an item's K and V tiles in the ring, as the MMAs take them: `ahead` (1 or 2) key tiles, then V 0, K ahead,
// V 1, ..., and the last V tiles.  Copy k of 2 count: whether it is V, and its tile t; and the reverse.
__device__ __forceinline__ bool copy_order(int k, int count, int ahead, int& t) {
    if (ahead == 1) {
        t = k >> 1;
        return k & 1;
    }
    const bool v = k == 2 * count - 1 || (k > 0 && (k & 1) == 0);
    t = k == 2 * count - 1 ? count - 1 : v ? k / 2 - 1 : (k + 1) / 2;
    return v;
}
__device__ __forceinline__ int copy_place(bool v, int t, int count, int ahead) {
    if (ahead == 1) return 2 * t + (v ? 1 : 0);
    return v ? min(2 * (t + 1), 2 * count - 1) : max(2 * t - 1, 0);
}

// ---- warp 8: copies -------------------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// Warp 8 hands out the stretches and copies q and K, warp 10 copies V (`v`): the issue of 16 page copies takes about
// half the time that a tile may take, so two warps share it.
template <int kFmt>
__device__ __forceinline__ void copy_warps(const ChunkArgs& a, Control& c, uint8_t* smem, bool v, Walk walk,
                                           const CUtensorMap* qm, const CUtensorMap* m) {
    using L = Layout<kFmt>;
    const int lane = threadIdx.x & 31;
    constexpr int kRing = L::k8 ? L::kRaw : L::kStages;
    uint64_t* full = L::k8 ? c.raw_full : c.kv_full;
    uint64_t* empty = L::k8 ? c.raw_empty : c.kv_empty;
    const uint32_t base = smem_addr(smem);
    const int my = L::k8 ? (lane & 7) : (lane >> 1) & 7;   // the page of the tile that this lane copies
    uint32_t ring = 0, q_count[2] = {0, 0}, unit = 0, segments = 0;
    Stretches stretches(c, a.status);
    bool ok = true;
    while (ok) {
        Segment s;
        if (!v) {
            const bool more = walk.next(s);
            if (!more) s.j0 = s.j1 = 0;
            const uint32_t slot = segments % kSegments;
            ok = pipe_wait(&c.seg_empty[slot], ((segments / kSegments) & 1) ^ 1, &c.dead, a.status);
            if (!ok) break;
            ++segments;
            if (lane == 0) {
                c.seg[slot] = s;
                mbar_arrive(&c.seg_full[slot]);
            }
            __syncwarp();
            if (!more) break;
            for (int t = 0; t < (s.two ? 2 : 1); ++t) {
                ok = ok && pipe_wait(&c.q_empty[t], (q_count[t] & 1) ^ 1, &c.dead, a.status);
                ++q_count[t];
                if (lane == 0 && ok) {
                    mbar_arrive_expect_tx(&c.q_full[t], (uint32_t)(a.tpt * a.G * kRowBytes));
                    for (int h = 0; h < 2; ++h)
                        tma_load_3d(base + L::kQ + t * kStageBytes + h * kHalf, qm, h * 64, s.kvh * a.G,
                                    s.rows + t * a.tpt, &c.q_full[t]);
                }
                __syncwarp();
            }
        } else {
            const Segment* next = stretches.next();
            if (next == nullptr) break;
            s = *next;
            stretches.done();
        }
        const int pages = (s.end + kPageSize - 1) / kPageSize, count = s.j1 - s.j0, ahead = s.two ? 1 : 2;
        auto page_of = [&](int t) {   // -1: none there (behind the last position, or a bad entry)
            const int pi = (s.j0 + t) * (kTileRows / kPageSize) + my;
            if (t >= count || pi >= pages) return -1;
            return a.page_table[(long)s.b * a.max_pages + pi];
        };
        int p0 = page_of(0), p1 = page_of(1), p2 = page_of(2);
        for (int t = 0; t < count && ok; ++t) {
            const int page = p0;
            p0 = p1;
            p1 = p2;
            p2 = page_of(t + 3);
            const bool there = (s.j0 + t) * (kTileRows / kPageSize) + my < pages;
            const bool good = there && page >= 0 && page < a.num_pages;
            if (there && !good) report(a.status, SD_ERR_INDEX_OOB);
            const uint32_t at = ring + copy_place(v, t, count, ahead), st = at % kRing;
            ok = pipe_wait(&empty[st], ((at / kRing) & 1) ^ 1, &c.dead, a.status);
            if (!ok) break;
            uint32_t bytes;
            bool copies;
            if (L::k8) {   // lanes 0-7: elements; lanes 8-15: the scales of both, with K
                copies = good && (lane < 8 || (lane < 16 && !v));
                bytes = __popc(__ballot_sync(0xffffffffu, copies && lane < 8)) * (kPageSize * kHeadDim) +
                        __popc(__ballot_sync(0xffffffffu, copies && lane >= 8)) * (kPageSize * 2 * kScaleBytes);
            } else {
                copies = good && lane < 16;
                bytes = __popc(__ballot_sync(0xffffffffu, copies)) * (kPageSize * kRowBytes / 2);
            }
            if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes);
            __syncwarp();
            if (copies) {
                if (L::k8) {
                    if (lane < 8)
                        tma_load_3d(base + L::kRawOff + st * kRawBytes + my * (kPageSize * kHeadDim), m, 0, s.kvh,
                                    page * kPageSize, &full[st]);
                    else
                        bulk_copy_g2s(smem + L::kScaleOff + ((unit + t) % L::kScaleSlots) * kScaleTile + my * (kPageSize * 2 * kScaleBytes),
                                      a.scales + scale_offset(page, s.kvh, 0, a.Hkv), kPageSize * 2 * kScaleBytes, &full[st]);
                } else {
                    const int h = lane & 1;
                    tma_load_3d(base + L::kKv + st * kStageBytes + h * kHalf + my * (kPageSize * 128), m, h * 64, s.kvh,
                                page * kPageSize, &full[st]);
                }
            }
            __syncwarp();
        }
        ring += 2 * count;
        unit += count;
    }
    // every copy has landed before the block ends; after a wait that ran out, which ones are under way is not known
    for (uint32_t x = ring > (uint32_t)kRing ? ring - kRing : 0; x < ring && ok; ++x)
        ok = pipe_wait(&full[x % kRing], (x / kRing) & 1, &c.dead, a.status);
    if (!ok) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {
        }
    }
}

// ---- warp 9: MMAs -----------------------------------------------------------------------------------------
template <int kFmt>
__device__ __forceinline__ void mma_warp(const ChunkArgs& a, Control& c, uint8_t* smem) {
    using L = Layout<kFmt>;
    const int lane = threadIdx.x & 31;
    const uint32_t base = smem_addr(smem), tm = uniform(c.tmem);
    constexpr uint32_t kQk = mma_idesc(128, 128, false), kPv = mma_idesc(128, 128, true);
    uint32_t ring = 0, q_count[2] = {0, 0}, p_count[2] = {0, 0};
    Stretches stretches(c, a.status);

    bool ok = true;   // else nothing more is issued
    auto wait_stage = [&]() -> uint32_t {   // the next stage of the ring, full
        const uint32_t st = ring % L::kStages;
        ok = ok && pipe_wait(&c.kv_full[st], (ring / L::kStages) & 1, &c.dead, a.status);
        ++ring;
        return st;
    };
    auto qk = [&](int g, int tile, uint32_t st) {
        if (!ok) return;
        const uint32_t qd = smem_desc(base + L::kQ + tile * kStageBytes, 16);
        const uint32_t kd = smem_desc(base + L::kKv + st * kStageBytes, 16);
#pragma unroll
        for (int x = 0; x < 8; ++x) {   // (a descriptor counts its address in 16 bytes)
            const uint32_t off = ((x >> 2) * kHalf + (x & 3) * 32) >> 4;
            mma_ss(tm + g * 128, qd + off, kd + off, kQk, x > 0);
        }
        mma_commit(&c.s_full[g]);
    };
    auto pv = [&](int g, uint32_t st, bool add) {
        const uint32_t vd = smem_desc(base + L::kKv + st * kStageBytes, kHalf);
        ok = ok && pipe_wait(&c.p_full[g], p_count[g] & 1, &c.dead, a.status);
        ++p_count[g];
        if (!ok) return;
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < 8; ++x)
            mma_ts(tm + 256 + g * 128, tm + g * 128 + x * 8, vd + x * (2048 >> 4), kPv, add || x > 0);
    };
    auto commit = [&](uint64_t* bar) {
        if (ok) mma_commit(bar);
    };
    // The value rows behind the item's last position are zeroed: their weights are zero, and 0 * NaN is NaN.
    auto clear_tail = [&](uint32_t st, int from) {
        if (L::k8 || from >= kTileRows || !ok) return;
        uint8_t* v = smem + L::kKv + st * kStageBytes;
        for (int x = from * 8 + lane; x < kTileRows * 8; x += 32) {
            reinterpret_cast<uint4*>(v)[x] = make_uint4(0u, 0u, 0u, 0u);
            reinterpret_cast<uint4*>(v + kHalf)[x] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async();
        __syncwarp();
    };

    while (const Segment* s = stretches.next()) {
        const int count = uniform(s->j1 - s->j0), end = uniform(s->end - s->j0 * kTileRows), two = uniform(s->two);
        ok = pipe_wait(&c.q_full[0], q_count[0] & 1, &c.dead, a.status);
        ++q_count[0];
        if (two) {
            ok = ok && pipe_wait(&c.q_full[1], q_count[1] & 1, &c.dead, a.status);
            ++q_count[1];
            uint32_t k = wait_stage();
            qk(0, 0, k);
            qk(1, 1, k);
            commit(&c.kv_empty[k]);
            auto q_done = [&](int t) {   // the stretch's last scores are under way: the next q may come
                if (t + 1 < count) return;
                commit(&c.q_empty[0]);
                commit(&c.q_empty[1]);
            };
            q_done(0);
            for (int t = 0; t < count && ok; ++t) {
                const uint32_t v = wait_stage();
                const bool more = t + 1 < count;
                clear_tail(v, end - t * kTileRows);
                if (more) k = wait_stage();
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    pv(g, v, t > 0);
                    if (g == 1) commit(&c.kv_empty[v]);
                    if (more) qk(g, g, k);
                    else commit(&c.o_full[g]);
                }
                if (more) {
                    commit(&c.kv_empty[k]);
                    q_done(t + 1);
                }
            }
        } else {
            for (int g = 0; g < 2 && g < count; ++g) {
                const uint32_t k = wait_stage();
                qk(g, 0, k);
                commit(&c.kv_empty[k]);
            }
            if (count <= 2) commit(&c.q_empty[0]);
            for (int t = 0; t < count && ok; ++t) {
                const int g = t & 1;
                const uint32_t v = wait_stage();
                clear_tail(v, end - t * kTileRows);
                pv(g, v, t > 1);
                commit(&c.kv_empty[v]);
                if (t + 2 < count) {
                    const uint32_t k = wait_stage();
                    qk(g, 0, k);
                    commit(&c.kv_empty[k]);
                    if (t + 3 == count) commit(&c.q_empty[0]);
                } else {
                    commit(&c.o_full[g]);
                }
            }
        }
        if (!ok) break;
        stretches.done();
    }
    mma_commit(&c.done);   // everything issued has ended before tensor memory is given back
    __syncwarp();
    mbar_wait(&c.done, 0);
}

// ---- warps 12-19 (8-bit caches): raw tiles to bf16 stages -------------------------------------------------
// The tile at ring position `at`; its rows from `rows` on become zero.  False: a wait ran out.
template <int kFmt>
__device__ __forceinline__ bool expand_tile(const ChunkArgs& a, Control& c, uint8_t* smem, uint32_t at, uint32_t unit, bool v,
                                            int rows) {
    using L = Layout<kFmt>;
    constexpr int kRows = kTileRows / (kExpandThreads / 8);   // rows per thread
    const int tid = threadIdx.x - Layout<kFmt>::kThreads + kExpandThreads;
    const uint32_t raw = at % L::kRaw, st = at % L::kStages;
    if (!pipe_wait(&c.raw_full[raw], (at / L::kRaw) & 1, &c.dead, a.status, &c.kv_empty[st], ((at / L::kStages) & 1) ^ 1))
        return false;
    const uint8_t* src = smem + L::kRawOff + raw * kRawBytes;
    const uint8_t* sc = smem + L::kScaleOff + (unit % L::kScaleSlots) * kScaleTile + (v ? kScaleBytes : 0);
    uint8_t* dst = smem + L::kKv + st * kStageBytes;
    const int c16 = tid & 7, h = c16 >> 2, k0 = 2 * (c16 & 3), r0 = tid >> 3;
    // lanes of the upper half write their second chunk first: eight lanes, eight bank groups
    auto put = [&](int row, const uint4& o0, const uint4& o1) {
        uint8_t* line = dst + h * kHalf + row * 128;
        *reinterpret_cast<uint4*>(line + (((k0 + h) ^ (row & 7)) << 4)) = h ? o1 : o0;
        *reinterpret_cast<uint4*>(line + (((k0 + 1 - h) ^ (row & 7)) << 4)) = h ? o0 : o1;
    };
    uint32_t by[kRows], odd = rows < kTileRows ? 1u : 0u;
#pragma unroll
    for (int x = 0; x < kRows; ++x) by[x] = sc[(x * (kTileRows / kRows) + r0) * (2 * kScaleBytes) + (c16 >> 1)];
#pragma unroll
    for (int x = 0; x < kRows; ++x) odd |= plain_factor<kFmt>(by[x]) ? 0u : 1u;
    if (__all_sync(0xffffffffu, odd == 0u)) {   // the loads of all rows, then their arithmetic side by side
        uint4 e[kRows];
#pragma unroll
        for (int x = 0; x < kRows; ++x)
            e[x] = *reinterpret_cast<const uint4*>(src + (x * (kTileRows / kRows) + r0) * kHeadDim + c16 * 16);
#pragma unroll
        for (int x = 0; x < kRows; ++x) {
            const uint32_t f = factor_plain<kFmt>(by[x]);
            uint4 o0, o1;
            expand4<kFmt>(e[x].x, o0.x, o0.y);
            expand4<kFmt>(e[x].y, o0.z, o0.w);
            expand4<kFmt>(e[x].z, o1.x, o1.y);
            expand4<kFmt>(e[x].w, o1.z, o1.w);
            put(x * (kTileRows / kRows) + r0,
                make_uint4(mul_bf16x2(o0.x, f), mul_bf16x2(o0.y, f), mul_bf16x2(o0.z, f), mul_bf16x2(o0.w, f)),
                make_uint4(mul_bf16x2(o1.x, f), mul_bf16x2(o1.y, f), mul_bf16x2(o1.z, f), mul_bf16x2(o1.w, f)));
        }
    } else {   // the item's last tile, or a scale at the ends of the range
#pragma unroll 1
        for (int x = 0; x < kRows; ++x) {
            const int row = x * (kTileRows / kRows) + r0;
            uint4 o0 = make_uint4(0u, 0u, 0u, 0u), o1 = o0;
            if (row < rows) {
                const uint4 e = *reinterpret_cast<const uint4*>(src + row * kHeadDim + c16 * 16);
                const Factor f = factor_of<kFmt>(sc[row * (2 * kScaleBytes) + (c16 >> 1)]);
                decode4<kFmt>(e.x, f, o0.x, o0.y);
                decode4<kFmt>(e.y, f, o0.z, o0.w);
                decode4<kFmt>(e.z, f, o1.x, o1.y);
                decode4<kFmt>(e.w, f, o1.z, o1.w);
            }
            put(row, o0, o1);
        }
    }
    fence_proxy_async();
    mbar_arrive(&c.raw_empty[raw]);
    mbar_arrive(&c.kv_full[st]);
    return true;
}

template <int kFmt>
__device__ __forceinline__ void expand_warps(const ChunkArgs& a, Control& c, uint8_t* smem) {
    uint32_t ring = 0, unit = 0;
    Stretches stretches(c, a.status);
    while (const Segment* s = stretches.next()) {
        const int count = s->j1 - s->j0, ahead = s->two ? 1 : 2, end = s->end - s->j0 * kTileRows;
        for (int k = 0; k < 2 * count; ++k) {   // (one call: the code of two would crowd the instruction cache)
            int t;
            const bool v = copy_order(k, count, ahead, t);
            if (!expand_tile<kFmt>(a, c, smem, ring + k, unit + t, v, end - t * kTileRows)) return;
        }
        ring += 2 * count;
        unit += count;
        stretches.done();
    }
}

// ---- warps 0-7: softmax and output --------------------------------------------------------------------------
__device__ __forceinline__ void swap_if(uint4& lo, uint4& hi, int mask) {   // the lanes without the bit keep lo, the others hi
    const bool up = threadIdx.x & mask;
    const uint4 t = up ? lo : hi;
    const uint4 r = make_uint4(__shfl_xor_sync(0xffffffffu, t.x, mask), __shfl_xor_sync(0xffffffffu, t.y, mask),
                               __shfl_xor_sync(0xffffffffu, t.z, mask), __shfl_xor_sync(0xffffffffu, t.w, mask));
    if (up) lo = r;
    else hi = r;
}
// Lane i of four gets element i of each of their arrays, in the lanes' order.
__device__ __forceinline__ void transpose4(uint4 (&v)[4]) {
    swap_if(v[0], v[1], 1);
    swap_if(v[2], v[3], 1);
    swap_if(v[0], v[2], 2);
    swap_if(v[1], v[3], 2);
}

// kLook: blocks of 32 scores that are loaded together, and one such step ahead.  Two are faster (4096 tokens over
// 65536 positions in bf16: 3.64 ms against 3.90), one fits the registers that the 8-bit caches' other warps leave.
template <int kLook>
__device__ __forceinline__ void softmax_warps(const ChunkArgs& a, Control& c) {
    const int cta = blockIdx.x;
    const int g = threadIdx.x >> 7, row = threadIdx.x & 127, warp = (threadIdx.x >> 5) & 3;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const uint32_t sc = c.tmem + g * 128 + lanes, oc = c.tmem + 256 + lanes;
    const int tq = row / a.G, gi = row - tq * a.G;
    const float scale = a.scale_log2;
    uint32_t s_count = 0, o_count = 0, joins = 0;
    Stretches stretches(c, a.status);
    if (threadIdx.x == 0) reinterpret_cast<TailRecord*>(a.tail)[cta] = TailRecord{};
    while (const Segment* seg = stretches.next()) {
        const Segment& s = *seg;
        const int tile = s.two ? g : 0, step = s.two ? 1 : 2, count = s.j1 - s.j0;
        const int token = tile * a.tpt + tq;
        const bool valid = tq < a.tpt && token < s.tokens;
        const int lim = valid ? s.first + token : s.end - 1;   // last position that the row sees
        const int lowest = s.first + tile * a.tpt;             // least of these in the tile
        const bool rows_here = __any_sync(0xffffffffu, valid);   // else the warp only keeps the barriers going
        float m = -INFINITY, l = 0.f;
        bool begun = false;
        for (int t = s.two ? 0 : g; t < count; t += step) {
            if (!pipe_wait(&c.s_full[g], s_count & 1, &c.dead, a.status)) return;
            ++s_count;
            if (!rows_here) {
                mbar_arrive(&c.p_full[g]);
                continue;
            }
            tc_fence_after();
            const int col0 = (s.j0 + t) * kTileRows, last = lim - col0;
            const bool border = col0 + kTileRows - 1 > lowest;
            uint32_t r[4][32];
            float add;
            // A row without a reference yet, or (second round) one whose scores have left it far behind, first takes
            // the tile's maximum as its reference; the scores stay in tensor memory until the weights replace them.
            bool look = __any_sync(0xffffffffu, valid && m == -INFINITY);
            for (int round = 0;; ++round) {
                if (look) {
                    float top = -INFINITY;
#pragma unroll 1
                    for (int x = 0; x < 4; ++x) {
                        tmem_ld32(sc + x * 32, r[0]);
                        tmem_wait_ld();
                        tmem_loaded(r[0]);
#pragma unroll
                        for (int y = 0; y < 32; ++y)
                            if (x * 32 + y <= last) top = fmaxf(top, __uint_as_float(r[0][y]));
                    }
                    top = fmaxf(top, m);
                    const float f = m == -INFINITY ? 0.f : ex2((m - top) * scale);
                    m = top;
                    l *= f;
                    if (begun) {
#pragma unroll 1
                        for (int x = 0; x < 4; ++x) {
                            tmem_ld32(oc + g * 128 + x * 32, r[0]);
                            tmem_wait_ld();
                            tmem_loaded(r[0]);
#pragma unroll
                            for (int y = 0; y < 32; ++y) r[0][y] = __float_as_uint(__uint_as_float(r[0][y]) * f);
                            tmem_st32(oc + g * 128 + x * 32, r[0]);
                        }
                    }
                }
                const float shift = m == -INFINITY ? 0.f : -m * scale;
                const uint64_t sc2 = pair_of(scale, scale), sh2 = pair_of(shift, shift);
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                for (int x = 0; x < kLook; ++x) tmem_ld32(sc + x * 32, r[x]);
#pragma unroll
                for (int h = 0; h < 4; h += kLook) {   // the next columns arrive while these are worked on
                    tmem_wait_ld();
#pragma unroll
                    for (int x = h; x < h + kLook; ++x) {
                        tmem_loaded(r[x]);
                        if (x + kLook < 4) tmem_ld32(sc + (x + kLook) * 32, r[x + kLook]);
                    }
                    if (border) {
#pragma unroll
                        for (int x = h; x < h + kLook; ++x)
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                if (x * 32 + y > last) r[x][y] = 0xff800000u;
                    }
#pragma unroll
                    for (int y = 0; y < 16 * kLook; ++y) {   // pair y takes the place of values that were used before
                        const uint32_t(&src)[32] = r[h + (y >> 4)];
                        const int z = (y & 15) * 2;
                        float lo, hi;
                        split_pair(fma2(pair_of(__uint_as_float(src[z]), __uint_as_float(src[z + 1])), sc2, sh2), lo, hi);
                        lo = ex2(lo);
                        hi = ex2(hi);
                        sum[y & 1] = add2(sum[y & 1], pair_of(lo, hi));
                        r[h][y] = pack_bf16x2(lo, hi);
                    }
                }
                float s0, s1;
                split_pair(add2(sum[0], sum[1]), s0, s1);
                add = s0 + s1;
                look = __any_sync(0xffffffffu, valid && !(add <= kFarAbove));
                if (!look || round > 0) break;
            }
            l += add;
            begun = true;
#pragma unroll
            for (int h = 0; h < 4; h += kLook) {
                if (kLook == 1) tmem_st16(sc + h * 16, r[h]);
                else tmem_st32(sc + h * 16, r[h]);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&c.p_full[g]);
        }
        // the stretch's output: final rows, or a part for the merge
        const bool mine = s.two || g < count;
        if (mine) {
            if (!pipe_wait(&c.o_full[g], o_count & 1, &c.dead, a.status)) return;
            ++o_count;
        }
        tc_fence_after();
        const bool whole = s.j0 == 0 && s.j1 == s.tiles;
        const int slot = 2 * cta + (s.j0 > 0 ? 0 : 1);
        float f0 = 1.f, f1 = 0.f;   // weights of the two sides' outputs
        int from = 0, to = 4;       // 32-column blocks that this thread writes
        bool both = false;
        if (!s.two) {
            c.post[g * kTileRows + row] = make_float2(m, l);
            tc_fence_before();
            mbar_arrive(&c.join[0]);
            if (!pipe_wait(&c.join[0], joins & 1, &c.dead, a.status)) return;
            tc_fence_after();
            const float2 p0 = c.post[row], p1 = c.post[kTileRows + row];
            m = fmaxf(p0.x, p1.x);
            const float mm = m == -INFINITY ? 0.f : m;
            f0 = ex2((p0.x - mm) * scale);
            f1 = ex2((p1.x - mm) * scale);
            l = p0.y * f0 + p1.y * f1;
            both = count > 1;
            from = 2 * g;
            to = from + 2;
        }
        const float inv = whole ? 1.f / l : 1.f;
        f0 *= inv;
        f1 *= inv;
        const uint32_t oa = s.two ? oc + g * 128 : oc;
        const int own = valid ? (s.rows + token) * a.Hq + s.kvh * a.G + gi : -1;   // row of out (below 2^31)
        int line[4];                                                                // those of the four lanes
#pragma unroll
        for (int y = 0; y < 4; ++y) line[y] = __shfl_sync(0xffffffffu, own, y, 4);
#pragma unroll 1
        for (int x = rows_here ? from : to; x < to; ++x) {   // (not unrolled: instructions used once per stretch
                                                                 // are fetched anew; 4700 cycles unrolled, 3700 so)
            uint32_t o[32];
            tmem_ld32(oa + x * 32, o);
            tmem_wait_ld();
            tmem_loaded(o);
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f0);
            if (both) {
                uint32_t o1[32];
                tmem_ld32(oa + 128 + x * 32, o1);
                tmem_wait_ld();
                tmem_loaded(o1);
#pragma unroll
                for (int y = 0; y < 32; ++y)
                    o[y] = __float_as_uint(fmaf(__uint_as_float(o1[y]), f1, __uint_as_float(o[y])));
            }
            if (whole) {
                uint4 v[4];
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    v[y] = make_uint4(pack_bf16x2(__uint_as_float(o[y * 8]), __uint_as_float(o[y * 8 + 1])),
                                      pack_bf16x2(__uint_as_float(o[y * 8 + 2]), __uint_as_float(o[y * 8 + 3])),
                                      pack_bf16x2(__uint_as_float(o[y * 8 + 4]), __uint_as_float(o[y * 8 + 5])),
                                      pack_bf16x2(__uint_as_float(o[y * 8 + 6]), __uint_as_float(o[y * 8 + 7])));
                // four lanes write 64 bytes of a row at a time (a lane its own row: 32 lines touched by each store)
                transpose4(v);
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    if (line[y] >= 0)
                        reinterpret_cast<uint4*>(a.out)[(long)line[y] * 16 + x * 4 + (threadIdx.x & 3)] = v[y];
            } else if (valid) {
#pragma unroll
                for (int y = 0; y < 8; ++y)
                    slot_out(a, slot, x * 8 + y)[tile * kTileRows + row] =
                        make_float4(__uint_as_float(o[y * 4]), __uint_as_float(o[y * 4 + 1]), __uint_as_float(o[y * 4 + 2]),
                                    __uint_as_float(o[y * 4 + 3]));
            }
        }
        if (valid && !whole && (s.two || g == 0)) slot_ml(a, slot)[tile * kTileRows + row] = make_float2(m * scale, l);
        tc_fence_before();
        if (!s.two) {   // both sides have read before either goes on
            mbar_arrive(&c.join[1]);
            if (!pipe_wait(&c.join[1], joins & 1, &c.dead, a.status)) return;
            ++joins;
        }
        if (threadIdx.x == 0 && s.last >= 0)
            reinterpret_cast<TailRecord*>(a.tail)[cta] = TailRecord{1, s.rows, s.tokens, s.kvh, s.last, {}};
        stretches.done();
    }
}

template <int kFmt>
__global__ void __launch_bounds__(Layout<kFmt>::kThreads, 1)
    chunk_attention_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ CUtensorMap qm,
                           const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm) {
    using L = Layout<kFmt>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Control& c = *reinterpret_cast<Control*>(smem + L::kCtl);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&c.q_full[x], 1);
            mbar_init(&c.q_empty[x], 1);
            mbar_init(&c.s_full[x], 1);
            mbar_init(&c.p_full[x], 128);
            mbar_init(&c.o_full[x], 1);
            mbar_init(&c.join[x], 256);
        }
        for (int x = 0; x < L::kStages; ++x) {
            mbar_init(&c.kv_full[x], L::k8 ? kExpandThreads : 1);
            mbar_init(&c.kv_empty[x], 1);
        }
        for (int x = 0; x < L::kRaw; ++x) {
            mbar_init(&c.raw_full[x], 1);
            mbar_init(&c.raw_empty[x], kExpandThreads);
        }
        for (int x = 0; x < kSegments; ++x) {
            mbar_init(&c.seg_full[x], 1);
            mbar_init(&c.seg_empty[x], L::k8 ? 18 : 10);   // the warps that read them
        }
        mbar_init(&c.done, 1);
        c.dead = 0;
        mbar_fence_init();
    }
    if (warp == 9) tmem_alloc(smem_addr(&c.tmem), 512);
    pdl_enter();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    long long u0, u1, total;
    const bool any = a.few == 0 || *a.tiles;   // (else every request is cache_decode.cu's)
    if (any) plan(a, c, u0, u1, total);
    if (!any) {
    } else if (warp < 8) {
        regs_up<L::k8 ? 136 : 216>();
        softmax_warps<L::k8 ? 1 : 2>(a, c);
    } else if (warp < 12) {
        regs_down<L::k8 ? 64 : 72>();
        if (warp == 8 || warp == 10) copy_warps<kFmt>(a, c, smem, warp == 10, Walk(a, c, u0, u1, total), &qm, warp == 10 ? &vm : &km);
        if (warp == 9) mma_warp<kFmt>(a, c, smem);
    } else if (L::k8) {
        regs_down<72>();
        expand_warps<kFmt>(a, c, smem);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(c.tmem, 512);
}

// Joins the parts of the items that CTA borders cut.  A warp takes 32 rows (a lane each) and 16 dimensions: its reads of the
// parts are whole lines and its writes whole sectors (with four dimensions, a quarter of a sector, a prompt of 2048 rows
// took 108 us in all instead of 80; two parts at once instead of four: 83).  Every block reads all tail records at once and
// its warps take their work in turn.
constexpr int kMergeThreads = 256, kChunks = 4, kPartsAtOnce = 4;
static_assert(kMergeThreads >= kChunkCtas, "one thread per tail record");
__global__ void __launch_bounds__(kMergeThreads) merge_chunks_kernel(const __grid_constant__ ChunkArgs a, int ctas) {
    __shared__ TailRecord recs[kChunkCtas];
    __shared__ int before[kChunkCtas + 1], scratch[40];
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, rows = a.tpt * a.G;
    if (a.few != 0 && !*a.tiles) return;
    int mine = 0, total;   // blocks of 32 rows
    if (tid < ctas) {
        recs[tid] = reinterpret_cast<const TailRecord*>(a.tail)[tid];
        if (recs[tid].valid) mine = (recs[tid].tokens * a.G + 31) / 32;
    }
    const int at = block_exclusive_scan(mine, scratch, &total);
    if (tid < ctas) before[tid] = at;
    if (tid == 0) before[ctas] = total;
    __syncthreads();
    constexpr int kPer = kHeadDim / 4 / kChunks;   // warps to a block of rows
    total *= kPer;
    for (int w = blockIdx.x + gridDim.x * (tid >> 5); w < total; w += gridDim.x * (kMergeThreads / 32)) {
        const int block = w / kPer, chunk = (w - block * kPer) * kChunks;
        int c = 0, hi = ctas - 1;   // the last CTA with before <= block
        while (c < hi) {
            const int mid = (c + hi + 1) >> 1;
            if (before[mid] <= block) c = mid;
            else hi = mid - 1;
        }
        const TailRecord& rec = recs[c];
        const int k = (block - before[c]) * 32 + lane;
        if (k >= rec.tokens * a.G) continue;
        const int tile = k / rows, r = k - tile * rows, row = tile * kTileRows + r;
        float m = -INFINITY, l = 0.f;
        float4 o[kChunks];
#pragma unroll
        for (int y = 0; y < kChunks; ++y) o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x0 = c; x0 <= rec.last; x0 += kPartsAtOnce) {
            float2 ml[kPartsAtOnce];
            float4 v[kPartsAtOnce][kChunks];
            float top = m;
#pragma unroll
            for (int z = 0; z < kPartsAtOnce; ++z) {
                const int x = x0 + z, slot = 2 * x + (x == c ? 1 : 0);   // this CTA's second, then the first of each later CTA
                ml[z] = make_float2(-INFINITY, 0.f);
                if (x > rec.last) continue;
                ml[z] = slot_ml(a, slot)[row];
#pragma unroll
                for (int y = 0; y < kChunks; ++y) v[z][y] = slot_out(a, slot, chunk + y)[row];
            }
#pragma unroll
            for (int z = 0; z < kPartsAtOnce; ++z) top = fmaxf(top, ml[z].x);
            const float f = m == -INFINITY ? 0.f : ex2(m - top);
            m = top;
            l *= f;
#pragma unroll
            for (int y = 0; y < kChunks; ++y) o[y] = make_float4(o[y].x * f, o[y].y * f, o[y].z * f, o[y].w * f);
#pragma unroll
            for (int z = 0; z < kPartsAtOnce; ++z) {
                if (x0 + z > rec.last) continue;
                const float g = ml[z].x == -INFINITY ? 0.f : ex2(ml[z].x - top);
                l = fmaf(ml[z].y, g, l);
#pragma unroll
                for (int y = 0; y < kChunks; ++y) {
                    o[y].x = fmaf(v[z][y].x, g, o[y].x);
                    o[y].y = fmaf(v[z][y].y, g, o[y].y);
                    o[y].z = fmaf(v[z][y].z, g, o[y].z);
                    o[y].w = fmaf(v[z][y].w, g, o[y].w);
                }
            }
        }
        const float inv = 1.f / l;
        const long dst = (((long)(rec.rows + tile * a.tpt + r / a.G) * a.Hq + rec.kvh * a.G + r % a.G) * 32 + chunk) / 2;
#pragma unroll
        for (int y = 0; y < kChunks; y += 2)
            reinterpret_cast<uint4*>(a.out)[dst + y / 2] =
                make_uint4(pack_bf16x2(o[y].x * inv, o[y].y * inv), pack_bf16x2(o[y].z * inv, o[y].w * inv),
                           pack_bf16x2(o[y + 1].x * inv, o[y + 1].y * inv), pack_bf16x2(o[y + 1].z * inv, o[y + 1].w * inv));
    }
}

template <int kFmt>
cudaError_t launch_format(const ChunkArgs& a, cudaStream_t stream) {
    constexpr bool k8 = Layout<kFmt>::k8;
    CUtensorMap qm, km, vm;
    const long rows = (long)a.num_pages * kPageSize;
    cudaError_t e = encode_rows_map(&qm, a.q, false, a.Hq, a.total_rows, 64, a.G, a.tpt, true);
    if (e == cudaSuccess) e = encode_rows_map(&km, a.K, k8, a.Hkv, rows, k8 ? kHeadDim : 64, 1, kPageSize, !k8);
    if (e == cudaSuccess) e = encode_rows_map(&vm, a.V, k8, a.Hkv, rows, k8 ? kHeadDim : 64, 1, kPageSize, !k8);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(chunk_attention_kernel<kFmt>, cudaFuncAttributeMaxDynamicSharedMemorySize, chunk_smem<kFmt>());
    if (e != cudaSuccess) return e;
    const int ctas = a.sms < kChunkCtas ? a.sms : kChunkCtas;
    e = launch_pdl(chunk_attention_kernel<kFmt>, dim3(ctas), dim3(Layout<kFmt>::kThreads), chunk_smem<kFmt>(), stream, a, qm,
                   km, vm);
    if (e == cudaSuccess && a.few != 0) e = launch_merge_decode(a, stream);
    if (e != cudaSuccess) return e;
    e = launch_pdl(merge_chunks_kernel, dim3(2 * ctas), dim3(kMergeThreads), 0, stream, a, ctas);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

ChunkLayout chunk_layout() {
    ChunkLayout L;
    // two slots per CTA: of 256 rows here, of 8 rows in cache_decode.cu
    const size_t rows = (size_t)2 * kChunkCtas * 2 * kTileRows, few = (size_t)2 * kDecodeShares * 8;
    L.part = 0;
    L.ml = rows * kHeadDim * sizeof(float);
    L.tail = L.ml + rows * sizeof(float2);
    L.few_part = L.tail + kChunkCtas * sizeof(TailRecord);
    L.few_ml = L.few_part + few * kHeadDim * sizeof(float);
    L.few_tail = L.few_ml + few * sizeof(float2);
    L.tiles = L.few_tail + kDecodeShares * sizeof(TailRecord);
    L.total = L.tiles + 256;
    return L;
}

cudaError_t launch_chunk_attention(const ChunkArgs& a, int format, cudaStream_t stream) {
    // Requests over 8-bit caches with at most eight rows (tokens times heads of a group) go to cache_decode.cu: 32 single
    // tokens of four heads to a group over 8K-164K positions of MXFP8 take 1.19 ms there and 1.67 ms here.  How many rows
    // each request has is known on the device only, so both kernels look at the batch and each takes its requests: 31 tokens
    // over 8K-64K positions with a chunk of 2048 rows take 0.79 ms, 1.50 ms with all of them here.  Where there is
    // nothing for this kernel it learns so from one word: 32 tokens over 512 positions 30 us instead of 27, 256 over 4096
    // 495 instead of 502.
    // Calls of so few rows that this weighs more (8 tokens over 512 positions: 23 us instead of 31) go there whole: where no
    // request can have more than eight rows, and up to four times as many where there are no more rows than requests (single
    // tokens, most often).  If one request has them all, four items read its cache in turn: 8 tokens over 32768
    // positions 82 us instead of 52, over 2048 25 instead of 30; with no such limit, 256 over 32768 took 1870 instead of 170.
    ChunkArgs rest = a;
    rest.few = 0;
    if (format != kFmtBf16 && a.G <= 8) {
        const int few = 8 / a.G;
        const bool all = a.total_rows <= few || (a.total_rows <= a.B && a.total_rows <= 4 * few);
        rest.few = all ? 4 * few : few;
        const cudaError_t e = launch_cache_decode(rest, format, stream);
        if (e != cudaSuccess) return e;
        if (all) return launch_merge_decode(rest, stream);
    }
    return format == kFmtBf16 ? launch_format<kFmtBf16>(rest, stream)
           : format == kFmtFp8 ? launch_format<kFmtFp8>(rest, stream) : launch_format<kFmtInt8>(rest, stream);
}

}  // namespace sd

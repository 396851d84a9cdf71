// cache_decode.cu -- chunk attention of few rows per KV head over an 8-bit cache (single tokens, short drafts).
//
// The same result as chunk_attention.cu, for the requests of a batch that have at most eight rows (tokens times the heads
// of a group; in small calls for all of them, eight rows at a time).  There, a 128-row tile would be mostly empty, and
// expanding every 8-bit tile to bf16 in shared memory moves three times the cache's bytes through it (96 KB written and
// read per 33 KB of cache: 3.3 TB/s of cache).
// Here each warp streams pages on its own, one step per page: K, V (one TMA box of 16 rows x 128 bytes each, 128-byte
// swizzle) and the page's 128 scale bytes into a ring of its own, and takes the elements from there straight into
// half-precision fragments, which hold them exactly (mma.sync m16n8k16, the eight rows in the upper half of A):
//   scores   A = q (scaled by a power of two to at most 2 per row), B = K; each block of 32 dimensions has its own
//            accumulator, which takes the block's scale of that position in fp32.
//   outputs  A = the weights, once for each block x: p_i 2^(e_x(i)) c_x with p_i = exp2(s_i - m), B = V, so that block x
//            of V needs no scaling.  m is a running maximum of the scores that may lag by 2^8, and c_x a factor of the
//            row and block that keeps the largest product so far near 2^6: half precision has few exponents, and where
//            the largest scale stands beside a small weight it must not push the others out.  c_x goes from 2^-126 to
//            2^119, so that block scales of 2^-124 still give products of 2^-5.
// Weights enter as half precision (11 bits); their sum is fp32.  All steps of the batch are cut evenly over the warps of
// one wave; items cut by a border leave parts in the workspace, which merge_decode_kernel joins in order.
//
// What bounds it: instructions (about 580 per page of 16 positions; the schedulers issue 60% of the time with 12
// warps per SM, and 16 warps spill registers: 1.51 ms instead of 1.19).  32 single tokens over 8K-164K positions, 32/8
// heads: 1.19 ms in MXFP8 (5.6 GB, 4.7 TB/s), 1.44 ms in MXINT8, whose elements take one more instruction per pair.
#include "cache_half.cuh"
#include "kernels.h"
#include "parts.cuh"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace sd {

namespace {

constexpr int kRows = 8;                     // rows of an item
constexpr int kRing = 4;                     // steps in a warp's ring
constexpr int kCtasPerSm = 12;               // one warp each
// Steps of a share on the average, in small calls (4: the same, 1: 10 us more, for the parts; 16: 5 us more), but no fewer
// shares than items: a warp takes 3 us for each of them, however short (about 170 of one step each: 26 us instead of 53).
constexpr int kLeast = 8;
constexpr float kGrow = 8.f;                 // log2 units that the maximum may lag behind
constexpr int kLift = 6;                     // log2 of what the largest weight is scaled to
constexpr float kTop = 16384.f;              // weights from here on (half precision ends at 65504) rescale their row
constexpr float kMostFactor = 6.6461400e35f; // 2^119: c_x at most (times a weight of up to 2^kGrow it stays finite)

struct Stage {
    uint8_t k[kPageSize][kHeadDim], v[kPageSize][kHeadDim];
};
struct __align__(1024) Smem {
    Stage stage[kRing];
    uint2 scales[kRing][kPageSize];
    uint64_t full[kRing];
};

struct Tail {
    int valid, rows, tokens, kvh, last, pad[3];
};

struct Req {
    int rs, n, base;
};
__device__ __forceinline__ Req req_of(const ChunkArgs& a, int b) {
    Req r;
    r.rs = a.row_start[b];
    r.n = a.row_start[b + 1] - r.rs;
    const int N = a.lens[b];
    r.base = N - r.n;
    if (N < 0 || (long)N > a.n_cap || r.base < 0 || r.n > a.few) r.n = 0;
    return r;
}
// Pages (steps) of item i: all positions that its last token sees.  tw tokens to an item.
__device__ __forceinline__ int item_steps(const Req& r, int i, int tw) {
    return (r.base + min(r.n, (i + 1) * tw) + kPageSize - 1) / kPageSize;
}

__device__ __forceinline__ float* part_of(const ChunkArgs& a, long slot) { return a.few_part + slot * (kRows * kHeadDim); }
__device__ __forceinline__ float2* part_ml(const ChunkArgs& a, long slot) { return a.few_ml + slot * kRows; }

__device__ __forceinline__ void tma_load_rows(uint32_t dst, const void* tmap, int head, int row, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(0), "r"(head), "r"(row), "r"(smem_addr(bar))
        : "memory");
}

template <int kFmt>
__global__ void __launch_bounds__(32, kCtasPerSm)
    cache_decode_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ CUtensorMap km,
                        const __grid_constant__ CUtensorMap vm) {
    extern __shared__ __align__(1024) uint8_t raw[];
    Smem& sm = *reinterpret_cast<Smem*>(raw);
    const int lane = threadIdx.x, n8 = lane >> 2, kq = lane & 3, tw = kRows / a.G;
    if (lane == 0) {
        for (int x = 0; x < kRing; ++x) mbar_init(&sm.full[x], 1);
        mbar_fence_init();
    }
    __syncwarp();
    pdl_enter();

    // ---- the warp's share of all steps ----
    const int per = (a.B + 31) / 32, b0 = min(a.B, lane * per), b1 = min(a.B, b0 + per);
    bool bad = false, more = false;
    long mine = 0, items = 0;
    for (int b = b0; b < b1; ++b) {
        const int lo = a.row_start[b], hi = a.row_start[b + 1], N = a.lens[b];
        bad = bad || lo < 0 || hi < lo || hi > a.total_rows;
        if (N < 0 || (long)N > a.n_cap || (hi > lo && hi - lo > N)) {
            if (blockIdx.x == 0) report(a.status, SD_ERR_INVALID_ARG);
            continue;
        }
        more = more || hi - lo > a.few;
        if (bad || hi == lo || hi - lo > a.few) continue;
        const Req r = {lo, hi - lo, N - (hi - lo)};
        long steps = 0;
        for (int i = 0; i * tw < r.n; ++i) steps += item_steps(r, i, tw);
        mine += steps * a.Hkv;
        items += (long)((r.n + tw - 1) / tw) * a.Hkv;
    }
    Tail* tail = reinterpret_cast<Tail*>(a.few_tail) + blockIdx.x;
    if (lane == 0) *tail = Tail{};
    bad = __any_sync(0xffffffffu, bad);
    more = __any_sync(0xffffffffu, more);
    if (lane == 0 && blockIdx.x == 0) *a.tiles = more && !bad;
    if (bad) {
        if (lane == 0 && blockIdx.x == 0) report(a.status, SD_ERR_INVALID_ARG);
        return;
    }
    long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    const long total = __shfl_sync(0xffffffffu, incl, 31);
#pragma unroll
    for (int o = 16; o; o >>= 1) items += __shfl_xor_sync(0xffffffffu, items, o);
    // (each share has a step: no gaps between parts)
    const long shares = min(max((total + kLeast - 1) / kLeast, items), (long)gridDim.x), w = blockIdx.x;
    if (w >= shares) return;
    const long u0 = total * w / shares, u1 = total * (w + 1) / shares;
    int b = 0, kvh = 0, item = 0, step = 0;
    const bool here = incl - mine <= u0 && u0 < incl;
    if (here) {
        long at = u0 - (incl - mine);
        for (b = b0; b < b1; ++b) {
            const Req r = req_of(a, b);
            long head = 0;
            for (int i = 0; i * tw < r.n; ++i) head += item_steps(r, i, tw);
            if (at < head * a.Hkv) {
                kvh = (int)(at / head);
                at -= kvh * head;
                while (at >= item_steps(r, item, tw)) at -= item_steps(r, item++, tw);
                step = (int)at;
                break;
            }
            at -= head * a.Hkv;
        }
    }
    const int owner = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    b = __shfl_sync(0xffffffffu, b, owner);
    kvh = __shfl_sync(0xffffffffu, kvh, owner);
    item = __shfl_sync(0xffffffffu, item, owner);
    step = __shfl_sync(0xffffffffu, step, owner);

    Req r = req_of(a, b);
    const uint32_t ring = smem_addr(&sm.stage[0]);
    uint32_t issued = 0, taken = 0;   // steps, over all items
    long left = u1 - u0;
    bool ok = true;
    while (left > 0 && ok) {
        const int tokens = min(tw, r.n - item * tw), first = r.base + item * tw, end = first + tokens;
        const int steps = (end + kPageSize - 1) / kPageSize, s0 = step, s1 = (int)min((long)steps, step + left), count = s1 - s0;
        const long row0 = r.rs + (long)item * tw;
        const int tok = n8 / a.G, head = n8 - tok * a.G;
        const bool valid = tok < tokens && tok < tw;
        const int lim = valid ? first + tok : end - 1;
        left -= count;

        // q: row n8, dimensions 32 x + 8 kq .. + 7 of each block x, scaled by a power of two to at most 2
        uint32_t qa[4][4];
        float up;
        {
            uint4 qv[4];
            float big = 0.f;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                qv[x] = make_uint4(0u, 0u, 0u, 0u);
                if (valid)
                    qv[x] = reinterpret_cast<const uint4*>(a.q)[((row0 + tok) * a.Hq + kvh * a.G + head) * 16 + x * 4 + kq];
                const uint32_t t[4] = {qv[x].x, qv[x].y, qv[x].z, qv[x].w};
#pragma unroll
                for (int y = 0; y < 4; ++y) big = fmaxf(big, fmaxf(fabsf(bf16_lo(t[y])), fabsf(bf16_hi(t[y]))));
            }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            float down;
            power_of_two(big, down, up);
            up *= a.scale_log2 * unit_of<kFmt>();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t t[4] = {qv[x].x, qv[x].y, qv[x].z, qv[x].w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const __half2 h = __floats2half2_rn(bf16_lo(t[y]) * down, bf16_hi(t[y]) * down);
                    qa[x][y] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
        }
        float o[4][4][2], m = -INFINITY, l = 0.f;   // [block][tile][column]
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) o[x][y][0] = o[x][y][1] = 0.f;
        float c[4] = {1.f, 1.f, 1.f, 1.f};          // (set when the row sees its first position)

        // page-table entries: 32 steps at a time, a lane each, the next 32 on their way
        const int32_t* table = a.page_table + (long)b * a.max_pages;
        auto entries = [&](int from) { return from + lane < s1 ? __ldg(table + from + lane) : 0; };
        int cur = entries(s0), nxt = entries(s0 + 32);
        auto load = [&](int t, int page) {   // step t of the stretch into the ring
            const uint32_t st = issued % kRing;
            ++issued;
            if (lane == 0) {
                if (page >= 0 && page < a.num_pages) {
                    mbar_arrive_expect_tx(&sm.full[st], kPageSize * (2 * kHeadDim + 2 * kScaleBytes));
                    tma_load_rows(ring + st * sizeof(Stage), &km, kvh, page * kPageSize, &sm.full[st]);
                    tma_load_rows(ring + st * sizeof(Stage) + offsetof(Stage, v), &vm, kvh, page * kPageSize, &sm.full[st]);
                    bulk_copy_g2s(&sm.scales[st][0], a.scales + scale_offset(page, kvh, 0, a.Hkv), kPageSize * 2 * kScaleBytes,
                                  &sm.full[st]);
                } else {
                    report(a.status, SD_ERR_INDEX_OOB);
                    mbar_arrive(&sm.full[st]);
                }
            }
        };
        __syncwarp();   // (the item before has been read)
        for (int t = 0; t < min(count, kRing - 1); ++t) load(t, __shfl_sync(0xffffffffu, cur, t));
        for (int t = 0; t < count; ++t) {
            if ((t & 31) == 0 && t > 0) {
                cur = nxt;
                nxt = entries(s0 + t + 32);
            }
            __syncwarp();   // every lane is done with the stage that is filled now
            const int ahead = t + kRing - 1;
            const int page = __shfl_sync(0xffffffffu, (ahead >> 5) == (t >> 5) ? cur : nxt, ahead & 31);
            if (ahead < count) load(ahead, page);
            const uint32_t st = taken % kRing;
            ok = __all_sync(0xffffffffu, mbar_wait(&sm.full[st], (taken / kRing) & 1));
            ++taken;
            if (!ok) break;
            const Stage& sg = sm.stage[st];

            // scores of positions 2 kq, 2 kq + 1, 2 kq + 8, 2 kq + 9 for row n8
            float s[4] = {0.f, 0.f, 0.f, 0.f};
            uint2 sc[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) sc[y] = sm.scales[st][2 * kq + (y & 1) + 8 * (y >> 1)];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int at = ((2 * x + (kq >> 1)) ^ n8) * 16 + (kq & 1) * 8;   // (rows n8 and n8 + 8 swizzle alike)
                const uint2 w0 = *reinterpret_cast<const uint2*>(&sg.k[n8][at]);
                const uint2 w1 = *reinterpret_cast<const uint2*>(&sg.k[n8 + 8][at]);
                float c0[2] = {0.f, 0.f}, c1[2] = {0.f, 0.f};
                mma_f16_upper(c0, qa[x][0], qa[x][1], half_pair<kFmt, 0>(w0.x), half_pair<kFmt, 1>(w0.x));
                mma_f16_upper(c1, qa[x][0], qa[x][1], half_pair<kFmt, 0>(w1.x), half_pair<kFmt, 1>(w1.x));
                mma_f16_upper(c0, qa[x][2], qa[x][3], half_pair<kFmt, 0>(w0.y), half_pair<kFmt, 1>(w0.y));
                mma_f16_upper(c1, qa[x][2], qa[x][3], half_pair<kFmt, 0>(w1.y), half_pair<kFmt, 1>(w1.y));
                s[0] = fmaf(c0[0], power_of(sc[0].x, x), s[0]);
                s[1] = fmaf(c0[1], power_of(sc[1].x, x), s[1]);
                s[2] = fmaf(c1[0], power_of(sc[2].x, x), s[2]);
                s[3] = fmaf(c1[1], power_of(sc[3].x, x), s[3]);
            }
            const int p0 = (s0 + t) * kPageSize;
            const bool border = p0 + kPageSize > first;   // some row does not see all of the page
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                s[y] *= up;
                if (border && p0 + 2 * kq + (y & 1) + 8 * (y >> 1) > lim) s[y] = -INFINITY;
            }
            const float top = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
            if (border) {
#pragma unroll
                for (int y = 0; y < 4; ++y)   // (what lies behind the last position does not count)
                    if (p0 + 2 * kq + (y & 1) + 8 * (y >> 1) >= end) sc[y].y = 0u;
            }
            bool fresh = false;
            if (__any_sync(0xffffffffu, top - m > kGrow)) {   // (from -infinity: any finite score)
                float mt = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                mt = fmaxf(m, fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2)));
                const float f = mt > m ? ex2(m - mt) : 1.f;
                fresh = m == -INFINITY && mt > m;
                m = mt;
                l *= f;
#pragma unroll
                for (int x = 0; x < 4; ++x) {   // the products' references stay where they are, as far as c reaches
                    // (f is 0 behind a jump of more than 2^7: now * f / c is 0 then, where now / c may be infinite)
                    const float now = fminf(c[x] / f, kMostFactor), g = now * f / c[x];
                    if (mt > -INFINITY && f != 1.f) {
                        c[x] = now;
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            o[x][y][0] *= g;
                            o[x][y][1] *= g;
                        }
                    }
                }
            }
            const float ms = m == -INFINITY ? 0.f : m;
            float p[4], most = 0.f;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                p[y] = ex2(s[y] - ms);
                l += p[y];
            }
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; y += 2)
                    most = max3(most, p[y] * c[x] * power_of(sc[y].y, x), p[y + 1] * c[x] * power_of(sc[y + 1].y, x));
            if (__any_sync(0xffffffffu, fresh || most > kTop)) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float g = 0.f;   // the row's largest product in the page
#pragma unroll
                    for (int y = 0; y < 4; ++y) g = fmaxf(g, p[y] * power_of(sc[y].y, x));
                    g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 1));
                    g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
                    // c to 2^kLift over the power of two at or below it
                    const uint32_t ex = __float_as_uint(g) >> 23;
                    const float now = fminf(__uint_as_float((uint32_t)min(max(254 + kLift - (int)ex, 1), 254) << 23), kMostFactor);
                    if (g < INFINITY && ((fresh && g > 0.f) || g * c[x] > kTop)) {
                        const float h = now / c[x];
                        c[x] = now;
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            o[x][y][0] *= h;
                            o[x][y][1] *= h;
                        }
                    }
                }
            }
            // outputs: positions 2 kq, 2 kq + 1 (and + 8), dimensions 32 x + 4 n8 .. + 3 per lane.  (Weight times factor first:
            // that is finite, and 0 where the weight is; factor times scale may be infinite beside a weight of 0.)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t wa[2], w[4];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const __half2 h = __floats2half2_rn(p[2 * y] * c[x] * power_of(sc[2 * y].y, x),
                                                        p[2 * y + 1] * c[x] * power_of(sc[2 * y + 1].y, x));
                    wa[y] = *reinterpret_cast<const uint32_t*>(&h);
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int row = 2 * kq + (y & 1) + 8 * (y >> 1);
                    w[y] = *reinterpret_cast<const uint32_t*>(&sg.v[row][((2 * x + (n8 >> 2)) ^ (row & 7)) * 16 + (n8 & 3) * 4]);
                    if (border && p0 + row >= end) w[y] = 0u;
                }
                const uint32_t e0 = __byte_perm(w[0], w[1], 0x5140), e1 = __byte_perm(w[0], w[1], 0x7362);
                const uint32_t f0 = __byte_perm(w[2], w[3], 0x5140), f1 = __byte_perm(w[2], w[3], 0x7362);
                mma_f16_upper(o[x][0], wa[0], wa[1], half_pair<kFmt, 0>(e0), half_pair<kFmt, 0>(f0));
                mma_f16_upper(o[x][1], wa[0], wa[1], half_pair<kFmt, 1>(e0), half_pair<kFmt, 1>(f0));
                mma_f16_upper(o[x][2], wa[0], wa[1], half_pair<kFmt, 0>(e1), half_pair<kFmt, 0>(f1));
                mma_f16_upper(o[x][3], wa[0], wa[1], half_pair<kFmt, 1>(e1), half_pair<kFmt, 1>(f1));
            }
        }
        if (!ok) break;
        // row n8: sum over the lanes that share it; block x, dimensions 8 kq + 0 .. 7 of it, in this lane
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const bool whole = s0 == 0 && s1 == steps;
        const long slot = 2 * w + (s0 == 0 ? 1 : 0);
        const float inv = (whole ? 1.f / l : 1.f) * unit_of<kFmt>();
        if (valid) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float f = 1.f / c[x];   // (not times inv first: that may fall below fp32's normal range)
                float v[8];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    v[y] = o[x][y][0] * inv * f;
                    v[4 + y] = o[x][y][1] * inv * f;
                }
                if (whole) {
                    reinterpret_cast<uint4*>(a.out)[((row0 + tok) * a.Hq + kvh * a.G + head) * 16 + x * 4 + kq] =
                        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
                } else {
                    float4* dst = reinterpret_cast<float4*>(part_of(a, slot) + n8 * kHeadDim) + x * 8 + kq * 2;
                    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                    dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                }
            }
            if (!whole && kq == 0) part_ml(a, slot)[n8] = make_float2(m, l);
        }
        if (left == 0 && s0 == 0 && s1 < steps && lane == 0) {   // the item goes on in the next shares
            const long endu = u1 - s1 + steps;
            *tail = Tail{1, (int)row0, tokens, kvh, (int)((endu * shares - 1) / total), {}};
        }
        step = 0;
        if (left > 0 && ++item * tw >= r.n) {
            item = 0;
            if (++kvh == a.Hkv) {
                kvh = 0;
                do {
                    r = req_of(a, ++b);
                } while (r.n == 0);
            }
        }
    }
    if (!ok) {   // a wait ran out: the copies under way get time to land
        if (lane == 0) report(a.status, SD_ERR_TIMEOUT);
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {
        }
    }
}

// Joins the parts of the items that share borders cut: a block takes kCols columns (of four dimensions) of the items that
// begin in its shares, one item at a time, with kGroups groups of threads that take every kGroups-th part, several loads
// at once.
constexpr int kAtOnce = 8;
constexpr int kMine = 32;   // shares of a block at most 
template <int kGroups, int kCols>
__global__ void __launch_bounds__(kGroups * kRows * kCols) merge_decode_kernel(const __grid_constant__ ChunkArgs a, int shares) {
    __shared__ float4 sums[kGroups][kRows][kCols];
    __shared__ float2 mls[kGroups][kRows];
    pdl_enter();
    const int group = threadIdx.x / (kRows * kCols), row = threadIdx.x / kCols % kRows, x8 = threadIdx.x % kCols;
    const int col = blockIdx.y * kCols + x8;
    // the block's tail records all at once
    __shared__ Tail recs[kMine];
    __shared__ int which[kMine], found;
    if (threadIdx.x < 32) {
        const int per = (shares + gridDim.x - 1) / gridDim.x, c = threadIdx.x < per ? blockIdx.x * per + threadIdx.x : shares;
        Tail rec = {};
        if (c < shares) rec = reinterpret_cast<const Tail*>(a.few_tail)[c];
        const uint32_t live = __ballot_sync(0xffffffffu, rec.valid != 0);
        if (rec.valid) {
            const int at = __popc(live & ((1u << threadIdx.x) - 1u));
            recs[at] = rec;
            which[at] = c;
        }
        if (threadIdx.x == 0) found = __popc(live);
    }
    __syncthreads();
    for (int i = 0; i < found; ++i) {
        const Tail rec = recs[i];
        const int c = which[i];
        const bool on = row < rec.tokens * a.G;
        PartSum s = no_parts();
        if (on) {
            for (int x0 = c + group; x0 <= rec.last; x0 += kGroups * kAtOnce) {
                float2 ml[kAtOnce];
                float4 v[kAtOnce];
#pragma unroll
                for (int y = 0; y < kAtOnce; ++y) {
                    const int x = x0 + y * kGroups;
                    const long slot = 2l * x + (x == c ? 1 : 0);   // this share's second, then each later one's first
                    ml[y] = make_float2(-INFINITY, 0.f);
                    v[y] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (x <= rec.last) {
                        ml[y] = part_ml(a, slot)[row];
                        v[y] = reinterpret_cast<const float4*>(part_of(a, slot) + row * kHeadDim)[col];
                    }
                }
                join(s, ml, v);
            }
            if (group > 0) {
                sums[group][row][x8] = s.o;
                if (x8 == 0) mls[group][row] = make_float2(s.m, s.l);
            }
        }
        __syncthreads();
        if (on && group == 0) {
            float2 ml[kGroups];
            float4 v[kGroups];
            ml[0] = make_float2(-INFINITY, 0.f);
            v[0] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 1; x < kGroups; ++x) {
                ml[x] = mls[x][row];
                v[x] = sums[x][row][x8];
            }
            join(s, ml, v);
            const float inv = 1.f / s.l;
            const long dst = ((long)(rec.rows + row / a.G) * a.Hq + rec.kvh * a.G + row % a.G) * 32 + col;
            reinterpret_cast<uint2*>(a.out)[dst] =
                make_uint2(pack_bf16x2(s.o.x * inv, s.o.y * inv), pack_bf16x2(s.o.z * inv, s.o.w * inv));
        }
        __syncthreads();
    }
}

int decode_shares(const ChunkArgs& a) { return min(a.sms * kCtasPerSm, kDecodeShares); }

template <int kFmt>
cudaError_t launch_format(const ChunkArgs& a, cudaStream_t stream) {
    CUtensorMap km, vm;
    const long rows = (long)a.num_pages * kPageSize;
    cudaError_t e = encode_rows_map(&km, a.K, true, a.Hkv, rows, kHeadDim, 1, kPageSize, true);
    if (e == cudaSuccess) e = encode_rows_map(&vm, a.V, true, a.Hkv, rows, kHeadDim, 1, kPageSize, true);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(cache_decode_kernel<kFmt>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
    if (e != cudaSuccess) return e;
    const int ctas = decode_shares(a);
    e = launch_pdl(cache_decode_kernel<kFmt>, dim3(ctas), dim3(32), sizeof(Smem), stream, a, km, vm);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_decode(const ChunkArgs& a, int format, cudaStream_t stream) {
    return format == kFmtFp8 ? launch_format<kFmtFp8>(a, stream) : launch_format<kFmtInt8>(a, stream);
}
cudaError_t launch_merge_decode(const ChunkArgs& a, cudaStream_t stream) {
    // Few items have many parts each (one token over 32768 positions and 8 KV heads: 222): eight groups and a quarter of
    // the columns per block, 34 us for the whole call instead of 64 (eight tokens: 141 instead of 144; over 1024 positions 24
    // instead of 21).  More items have few parts: a block per share (16 tokens over 300 positions: 22 us instead of 29).
    const int shares = decode_shares(a);
    const cudaError_t e =
        (long)a.total_rows * a.Hkv <= 64
            ? launch_pdl(merge_decode_kernel<8, 8>, dim3((shares + kMine / 2 - 1) / (kMine / 2), 4), dim3(8 * kRows * 8), 0,
                         stream, a, shares)
            : launch_pdl(merge_decode_kernel<1, 32>, dim3(shares), dim3(kRows * 32), 0, stream, a, shares);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sd

// cache_sparse.cu -- exact attention over the selected rows of an 8-bit paged cache (the sparse decode of
// sparse_decode.cu, for the formats of cache_format.cuh).
//
//   out[r] = sum_{i in S_r} w_i V_i / sum_{i in S_r} w_i,  w_i = 2^(s_i - m),  s_i = (q_r . K_i) log2(e) / sqrt(d)
//
// per row r = (request, query head).
//
// The slots of idx, padding included, are cut evenly over the warps of one wave: no pass over the rows is needed
// first, full rows (the indexers') balance exactly, and padding costs a read of idx.  A row cut by a share's border
// leaves parts in the workspace; sparse_parts_kernel joins them in order.
//
// One step of a warp takes 16 selected rows, gathered by 16-byte asynchronous copies into a ring of its own in shared
// memory (positions are read about six steps ahead of their use, page entries four, cache rows two).  Both products run
// on the tensor cores (mma.sync m16n8k16) on the 8-bit elements as half-precision values, which hold them exactly;
// one fp32 dot product per row on the CUDA cores took 50 instructions per selected row, this takes about half.
//   scores   A = 16 rows of K, B = q with column n holding only block n of it, so that column n of the result is
//            the dot product over block n, which then takes the block's scale in fp32.  q is scaled by a power of
//            two to at most 2, which half precision holds to 2^-25 of its largest value.
//   outputs  A = the weights: row 2 n + i is part i (high, residual: 22 bits) of w_r 2^(e_n(r)), the weight with
//            the scale of block n folded in, B = V; of the result, block n of the output uses rows 2 n, 2 n + 1.
//            Each block has a reference M_n of its own (near the largest s + e_n), as scales may span more than
//            half precision's range; the sum of the weights has the reference m.
// References lag by up to 2^8 before the accumulators are rescaled.  A step's products are added to the outputs by fp32
// additions, which round to nearest: the tensor cores' own accumulation does not, and its errors, all towards zero, add up
// over a share (root mean square error 1.2e-5 instead of 5.7e-7 over 590 steps, 3.9e-7 instead of 2.9e-7 over 24).  It
// costs nothing at k = N/50 and 6% at k = N/2.
//
// What bounds it: random 128-byte rows.  At 4 x 64 heads x 2621 rows of N = 131072 (168 MB with each row of a group
// read once) the gathers alone take 52 us for K and V, 4 us more for the scales' 32-byte sectors, and 27-40 us when
// the same number of rows is read in order; the whole call takes 64 us.
#include "cache_half.cuh"
#include "kernels.h"
#include "parts.cuh"
#include "tcgen05.cuh"

namespace sd {

namespace {

constexpr int kWarps = 1;          // warps of a CTA (independent of each other: one balances the SMs best)
constexpr int kCtas = 12;          // CTAs per SM (at 13 and more, registers spill and the time grows)
constexpr int kStep = 16;          // selected rows per warp and step
constexpr int kDepth = 2;          // steps whose gathers are in flight: one chunk of 32 slots
constexpr int kRing = kDepth + 1;
constexpr float kGrow = 8.f;       // log2 units that a reference may lag behind
constexpr float kLift = 6.f;       // weights are at most about 2^6, with the lag 2^14: clear of half precision's ends

// Rows of one step.  16-byte chunk c of row r lies at chunk c ^ (2 (r & 3)) of K and c ^ (2 ((r >> 1) & 3)) of V: the rows
// that a fragment load touches at once then fall into different banks.
struct Step {
    uint8_t k[kStep][kHeadDim], v[kStep][kHeadDim];
    uint2 s[kStep];   // scale bytes of K and of V
};
constexpr int kSmem = kWarps * kRing * (int)sizeof(Step);

__device__ __forceinline__ void cp_async_8(uint32_t dst, const void* src, bool valid) {   // (zeros where not valid)
    const int bytes = valid ? 8 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// 2^e of a scale byte.  Byte 255 gives an infinity (NaN with the block's zeros).
template <int kFmt>
__device__ __forceinline__ float scale_of(uint32_t byte) {
    if (kFmt == kFmtFp8) return __uint_as_float(byte << 23);
    const uint32_t bits = byte > 6u ? (byte - 6u) << 23 : 1u << (byte + 16u);
    return __uint_as_float(byte == 255u ? 0x7f800000u : bits);
}
// e itself (byte 255: NaN).
template <int kFmt>
__device__ __forceinline__ float exponent_of(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7fc00000u) : (float)((int)byte - (kFmt == kFmtFp8 ? 127 : 133));
}

__device__ __forceinline__ float* part_out(const CacheSparseArgs& a, long slot) { return a.part + slot * kHeadDim; }

template <int kFmt>
__global__ void __launch_bounds__(kWarps * 32, kCtas) cache_sparse_kernel(const __grid_constant__ CacheSparseArgs a) {
    extern __shared__ __align__(16) Step ring[];
    pdl_enter();
    const int lane = threadIdx.x & 31, grp = lane >> 3, c = lane & 7;   // copies: row within four, 16-byte chunk
    const int n8 = lane >> 2, kq = lane & 3;                              // fragments: row or column, position
    const long w = (long)blockIdx.x * kWarps + (threadIdx.x >> 5), W = a.shares;
    if (w >= W) return;
    const uint32_t ring_at = smem_addr(ring + (threadIdx.x >> 5) * kRing), ring_end = ring_at + kDepth * sizeof(Step);
    // where a lane's chunks of its first row of a step go (of later rows: 4 rows further each time)
    const uint32_t kdst = grp * kHeadDim + (c ^ (2 * grp)) * 16;
    const uint32_t vdst0 = offsetof(Step, v) + grp * kHeadDim + (c ^ (2 * (grp >> 1))) * 16;
    const uint32_t vdst1 = offsetof(Step, v) + grp * kHeadDim + (c ^ (2 * (2 + (grp >> 1)))) * 16;
    const uint8_t* kbase = static_cast<const uint8_t*>(a.K) + c * 16;
    const uint8_t* vbase = static_cast<const uint8_t*>(a.V) + c * 16;
    const long total = (long)a.B * a.Hq * a.k_max;
    const long u1 = total * (w + 1) / W;
    for (long u0 = total * w / W; u0 < u1;) {
        const int r = (int)(u0 / a.k_max), j0 = (int)(u0 - (long)r * a.k_max);
        const int j1 = (int)min((long)a.k_max, j0 + (u1 - u0));
        u0 += j1 - j0;
        const int b = r / a.Hq, h = r - b * a.Hq, kvh = h / a.G;
        const int N = checked_len(a.lens, b, a.n_cap, a.status);
        const int32_t* row = a.idx + (long)r * a.k_max;
        const int32_t* table = a.page_table + (long)b * a.max_pages;

        // q: lane (n, kq) = (lane / 4, lane % 4), n < 4, holds dimensions 32 n + 8 kq .. + 7, the others zero
        uint4 qv = make_uint4(0u, 0u, 0u, 0u);
        if (n8 < 4) qv = reinterpret_cast<const uint4*>(a.q)[(long)r * 16 + n8 * 4 + kq];
        float q[8] = {bf16_lo(qv.x), bf16_hi(qv.x), bf16_lo(qv.y), bf16_hi(qv.y), bf16_lo(qv.z), bf16_hi(qv.z), bf16_lo(qv.w), bf16_hi(qv.w)};
        float big = 0.f;
#pragma unroll
        for (int x = 0; x < 8; ++x) big = fmaxf(big, fabsf(q[x]));
#pragma unroll
        for (int x = 16; x; x >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, x));
        float down, up;
        power_of_two(big, down, up);
        up *= a.scale_log2;
        uint32_t qb[2][2];   // [half of the block][k, k + 8]
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const __half2 v = __floats2half2_rn(q[2 * x] * down, q[2 * x + 1] * down);
            qb[x >> 1][x & 1] = *reinterpret_cast<const uint32_t*>(&v);
        }
        float o[4][4][2], M = -INFINITY, m = -INFINITY, l = 0.f;   // [block][tile][column]; M of block n8 / 2
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) o[x][y][0] = o[x][y][1] = 0.f;

        // Lookups go by chunks of 32 slots, a lane each (two steps): the entry of idx two chunks ahead of the gathers, the
        // page-table entry one ahead.
        auto position = [&](int chunk) {
            const int j = j0 + chunk * 32 + lane;
            return j < j1 ? __ldg(row + j) : -1;
        };
        int before = j0 > 0 ? __ldg(row + j0 - 1) : 0;   // the entry before the chunk (of the row's first: none)
        bool first = j0 == 0;
        auto page_of = [&](int& e) {   // also the checks of the entry; e = -1 where nothing is to be read
            int p = __shfl_up_sync(0xffffffffu, e, 1);
            if (lane == 0) p = before;
            before = __shfl_sync(0xffffffffu, e, 31);
            const bool start = first && lane == 0;
            first = false;
            if (e < 0) return 0;
            if (e >= N || (!start && (p < 0 || p >= e))) {
                report(a.status, e >= N ? SD_ERR_INDEX_OOB : SD_ERR_ORDER);
                e = -1;
                return 0;
            }
            return __ldg(table + e / kPageSize);
        };
        auto resolve = [&](int e, int page) {   // page and slot of the entry, or -1
            if (e < 0) return -1;
            if (page < 0 || page >= a.num_pages) {
                report(a.status, SD_ERR_INDEX_OOB);
                return -1;
            }
            return page * kPageSize + e % kPageSize;
        };
        auto gather = [&](int at, int half, uint32_t stage) {   // 16 rows of a chunk; rows that are not there become zeros
            const int mine = at >= 0 ? at * a.Hkv + kvh : -1;   // cache row (below 2^31)
#pragma unroll
            for (int u = 0; u < kStep / 4; ++u) {
                const int i = __shfl_sync(0xffffffffu, mine, half * kStep + u * 4 + grp);
                const long off = (long)max(i, 0) * kHeadDim;
                cp_async_16(stage + kdst + u * 4 * kHeadDim, kbase + off, i >= 0);
                cp_async_16(stage + (u & 1 ? vdst1 : vdst0) + u * 4 * kHeadDim, vbase + off, i >= 0);
            }
            if ((lane >> 4) == half)
                cp_async_8(stage + offsetof(Step, s) + (lane & 15) * 8,
                           a.scales + (at >= 0 ? scale_offset(at / kPageSize, kvh, at % kPageSize, a.Hkv) : 0), at >= 0);
            cp_async_commit();
        };

        const int steps = (j1 - j0 + kStep - 1) / kStep;
        int e0 = position(0), e1 = position(1), e2 = position(2);
        int p0 = page_of(e0), p1 = page_of(e1);
        int at = resolve(e0, p0);                                     // of the chunk that the gathers are in
        uint32_t live = __ballot_sync(0xffffffffu, at >= 0), ahead = live;   // of the steps computed, and of that chunk
        uint32_t fill = ring_at;
        gather(at, 0, fill);
        gather(at, 1, fill + sizeof(Step));
        fill += kDepth * sizeof(Step);
        uint32_t stage = ring_at;
        for (int t = 0; t < steps; ++t) {
            if ((t & 1) == 0) {   // the gathers reach the next chunk
                live = ahead;
                at = resolve(e1, p1);
                ahead = __ballot_sync(0xffffffffu, at >= 0);
                p1 = page_of(e2);
                e1 = e2;
                e2 = position((t >> 1) + 3);
            } else {
                live >>= kStep;
            }
            __syncwarp();   // every lane is done with the stage that is filled now
            gather(at, t & 1, fill);
            fill = fill == ring_end ? ring_at : fill + (uint32_t)sizeof(Step);
            cp_async_wait<kDepth>();
            __syncwarp();
            const Step& cur = *reinterpret_cast<const Step*>(reinterpret_cast<const uint8_t*>(ring) + (stage - smem_addr(ring)));
            stage = stage == ring_end ? ring_at : stage + (uint32_t)sizeof(Step);

            // scores: rows n8 and n8 + 8, 8 bytes of each block per lane
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int at = ((2 * x + (kq >> 1)) ^ (2 * (n8 & 3))) * 16 + (kq & 1) * 8;
                const uint2 w0 = *reinterpret_cast<const uint2*>(&cur.k[n8][at]);
                const uint2 w1 = *reinterpret_cast<const uint2*>(&cur.k[n8 + 8][at]);
                const bool on = n8 == x;
                mma_f16(d, half_pair<kFmt, 0>(w0.x), half_pair<kFmt, 0>(w1.x), half_pair<kFmt, 1>(w0.x),
                        half_pair<kFmt, 1>(w1.x), on ? qb[0][0] : 0u, on ? qb[0][1] : 0u);
                mma_f16(d, half_pair<kFmt, 0>(w0.y), half_pair<kFmt, 0>(w1.y), half_pair<kFmt, 1>(w0.y),
                        half_pair<kFmt, 1>(w1.y), on ? qb[1][0] : 0u, on ? qb[1][1] : 0u);
            }
            // columns 2 kq, 2 kq + 1 are blocks (kq < 2): scaled and summed
            float s0 = 0.f, s1 = 0.f;
            if (kq < 2) {
                const uint32_t b0 = cur.s[n8].x >> (16 * kq), b1 = cur.s[n8 + 8].x >> (16 * kq);
                s0 = fmaf(d[0], scale_of<kFmt>(b0 & 255u), d[1] * scale_of<kFmt>(b0 >> 8 & 255u)) * up;
                s1 = fmaf(d[2], scale_of<kFmt>(b1 & 255u), d[3] * scale_of<kFmt>(b1 >> 8 & 255u)) * up;
            }
            s0 += __shfl_xor_sync(0xffffffffu, s0, 1);
            s1 += __shfl_xor_sync(0xffffffffu, s1, 1);
            if (!(live >> n8 & 1)) s0 = -INFINITY;
            if (!(live >> (n8 + 8) & 1)) s1 = -INFINITY;
            // rows 2 kq, 2 kq + 1, 2 kq + 8, 2 kq + 9, with the exponents of block n8 / 2
            float s[4], z[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                s[x] = __shfl_sync(0xffffffffu, x < 2 ? s0 : s1, (2 * kq + (x & 1)) * 4);
                const uint32_t byte = cur.s[2 * kq + (x & 1) + 8 * (x >> 1)].y >> (8 * (n8 >> 1)) & 255u;
                z[x] = s[x] + exponent_of<kFmt>(byte);
            }
            const float zt = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])), st = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
            if (__any_sync(0xffffffffu, zt - M > kGrow || st - m > kGrow)) {   // (from -infinity: any finite score)
                float zm = fmaxf(zt, __shfl_xor_sync(0xffffffffu, zt, 1)), sm = fmaxf(st, __shfl_xor_sync(0xffffffffu, st, 1));
                zm = fmaxf(M, fmaxf(zm, __shfl_xor_sync(0xffffffffu, zm, 2)));
                sm = fmaxf(m, fmaxf(sm, __shfl_xor_sync(0xffffffffu, sm, 2)));
                const float fz = zm > M ? ex2(M - zm) : 1.f, fs = sm > m ? ex2(m - sm) : 1.f;
                M = zm;
                m = sm;
                l *= fs;
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        o[x][y][0] *= fz;
                        o[x][y][1] *= fz;
                    }
            }
            const float ms = m == -INFINITY ? 0.f : m, Ms = M == -INFINITY ? 0.f : M - kLift;
            uint32_t wa[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                l += ex2(s[2 * x] - ms) + ex2(s[2 * x + 1] - ms);
                const float w0 = ex2(z[2 * x] - Ms), w1 = ex2(z[2 * x + 1] - Ms);
                const __half2 hi = __floats2half2_rn(w0, w1);
                const float2 back = __half22float2(hi);
                const __half2 lo = __floats2half2_rn(w0 - back.x, w1 - back.y);
                wa[x] = (n8 & 1) ? *reinterpret_cast<const uint32_t*>(&lo) : *reinterpret_cast<const uint32_t*>(&hi);
            }
            // outputs: rows 2 kq, 2 kq + 1 (and + 8), dimensions 32 x + 4 n8 .. + 3 per lane
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t w[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int row = 2 * kq + (y & 1) + 8 * (y >> 1);
                    w[y] = *reinterpret_cast<const uint32_t*>(&cur.v[row][((2 * x + (n8 >> 2)) ^ (2 * kq)) * 16 + (n8 & 3) * 4]);
                }
                const uint32_t e0 = __byte_perm(w[0], w[1], 0x5140), e1 = __byte_perm(w[0], w[1], 0x7362);
                const uint32_t f0 = __byte_perm(w[2], w[3], 0x5140), f1 = __byte_perm(w[2], w[3], 0x7362);
                float t[4][2] = {};
                mma_f16_upper(t[0], wa[0], wa[1], half_pair<kFmt, 0>(e0), half_pair<kFmt, 0>(f0));
                mma_f16_upper(t[1], wa[0], wa[1], half_pair<kFmt, 1>(e0), half_pair<kFmt, 1>(f0));
                mma_f16_upper(t[2], wa[0], wa[1], half_pair<kFmt, 0>(e1), half_pair<kFmt, 0>(f1));
                mma_f16_upper(t[3], wa[0], wa[1], half_pair<kFmt, 1>(e1), half_pair<kFmt, 1>(f1));
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    o[x][y][0] += t[y][0];
                    o[x][y][1] += t[y][1];
                }
            }
        }
        cp_async_wait<0>();
        __syncwarp();
        // the row's sum over the four lanes of a group; outputs: block n8 / 2, high and residual parts added
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const bool whole = j0 == 0 && j1 == a.k_max;
        const float inv = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
        // (in two factors where the block's scales are tiny: 2^(M - m) alone may lie below fp32's range)
        const float d = M - kLift - m, off = d < -64.f ? 64.f : 0.f, back = d < -64.f ? 5.421010862427522e-20f : 1.f;   // 2^-64
        const float f = M == -INFINITY ? 0.f : ex2(d + off) * inv;
        float v[8];   // dimensions 32 (n8 / 2) + 8 kq + 0 .. 7
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                float x = n8 < 2 ? o[0][y][z] : n8 < 4 ? o[1][y][z] : n8 < 6 ? o[2][y][z] : o[3][y][z];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                v[4 * z + y] = x * f * back;   // (M = -infinity: 0, or NaN where every block was one)
            }
        const long slot = 2 * w + (j0 == 0 ? 1 : 0);   // a share's first row may have begun earlier; its last may go on
        float4* dst = reinterpret_cast<float4*>(whole ? a.out + (long)r * kHeadDim : part_out(a, slot)) + (n8 >> 1) * 8 + kq * 2;
        if ((n8 & 1) == 0) {
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
        if (!whole && lane == 0) a.ml[slot] = make_float2(m, l);
    }
}

// Joins the parts of each row that a share's border cut: kSplit warps per row, each with every kSplit-th part, several at
// once, and four dimensions per lane.
constexpr int kFewParts = 16;   // parts of a row up to which one warp joins them (8 heads of 13107 entries, 192 parts: 38 us
                                // for the call with one warp, 14 with 16; 4 parts: 13 us, 15 with 16 warps)
constexpr int kJoinWarps = 4, kAtOnce = 8;
template <int kSplit>
__global__ void __launch_bounds__((kSplit > 1 ? kSplit : kJoinWarps) * 32)
    sparse_parts_kernel(const __grid_constant__ CacheSparseArgs a) {
    __shared__ float4 sums[kSplit][32];
    __shared__ float2 mls[kSplit];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, split = kSplit > 1 ? warp : 0;
    const long r = kSplit > 1 ? blockIdx.x : (long)blockIdx.x * kJoinWarps + warp, rows = (long)a.B * a.Hq, W = a.shares;
    if (r >= rows) return;
    const long total = rows * a.k_max, begin = r * a.k_max, end = begin + a.k_max - 1;
    // the share that holds slot x: the w with total w / W <= x < total (w + 1) / W (rounded down)
    const long w0 = ((begin + 1) * W - 1) / total, w1 = ((end + 1) * W - 1) / total;
    if (w0 == w1) return;
    PartSum s = no_parts();
    for (long x0 = w0 + split; x0 <= w1; x0 += kSplit * kAtOnce) {
        float2 ml[kAtOnce];
        float4 v[kAtOnce];
#pragma unroll
        for (int y = 0; y < kAtOnce; ++y) {
            const long w = x0 + y * kSplit, slot = 2 * w + (w == w0 ? 1 : 0);   // (the row begins in share w0)
            ml[y] = make_float2(-INFINITY, 0.f);
            v[y] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (w <= w1) {
                ml[y] = a.ml[slot];
                v[y] = reinterpret_cast<const float4*>(part_out(a, slot))[lane];
            }
        }
        join(s, ml, v);
    }
    if (kSplit > 1) {
        sums[split][lane] = s.o;
        if (lane == 0) mls[split] = make_float2(s.m, s.l);
        __syncthreads();
        if (split > 0) return;
        float2 ml[kSplit];
        float4 v[kSplit];
#pragma unroll
        for (int y = 0; y < kSplit; ++y) {
            ml[y] = mls[y];
            v[y] = sums[y][lane];
        }
        s = no_parts();
        join(s, ml, v);
    }
    const float inv = s.l > 0.f ? 1.f / s.l : 0.f;
    reinterpret_cast<float4*>(a.out)[r * 32 + lane] = make_float4(s.o.x * inv, s.o.y * inv, s.o.z * inv, s.o.w * inv);
}

template <int kFmt>
cudaError_t launch_format(CacheSparseArgs a, cudaStream_t stream) {
    int per_sm = 0;
    cudaError_t e = cudaFuncSetAttribute(cache_sparse_kernel<kFmt>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, cache_sparse_kernel<kFmt>, kWarps * 32, kSmem);
    if (e != cudaSuccess) return e;
    const long rows = (long)a.B * a.Hq, slots = rows * a.k_max;
    long shares = (long)a.sms * per_sm * kWarps;
    if (shares > kCacheSparseWarps) shares = kCacheSparseWarps;
    if (shares > rows) shares -= shares % rows;   // whole numbers of shares to a row: none starts a second row
    if (shares > slots) shares = slots;           // (a share without a slot would leave a gap between a row's parts)
    a.shares = (int)shares;
    e = launch_pdl(cache_sparse_kernel<kFmt>, dim3((unsigned)((shares + kWarps - 1) / kWarps)), dim3(kWarps * 32), kSmem, stream,
                   a);
    if (e != cudaSuccess) return e;
    e = shares < kFewParts * rows
            ? launch_pdl(sparse_parts_kernel<1>, dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps)), dim3(kJoinWarps * 32), 0,
                         stream, a)
            : launch_pdl(sparse_parts_kernel<16>, dim3((unsigned)rows), dim3(16 * 32), 0, stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_sparse(const CacheSparseArgs& a, int format, cudaStream_t stream) {
    return format == kFmtFp8 ? launch_format<kFmtFp8>(a, stream) : launch_format<kFmtInt8>(a, stream);
}

}  // namespace sd

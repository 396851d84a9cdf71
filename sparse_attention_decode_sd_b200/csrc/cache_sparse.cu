// cache_sparse.cu -- exact attention over the selected rows of an 8-bit paged cache (the sparse decode of
// sparse_decode.cu, for the formats of cache_format.cuh).
//
//   out[r] = sum_{i in S_r} w_i V_i / sum_{i in S_r} w_i,  w_i = 2^((q_r . K_i) log2(e) / sqrt(d) - m)
//
// per row r = (request, query head), m the running maximum (kept within 2^8 of it), everything in fp32.
//
// The slots of idx, padding included, are cut evenly over the warps of one wave: no pass over the rows is needed
// first, full rows (the indexers') balance exactly, and padding costs a read of idx.  Eight lanes take one selected
// row, 16 dimensions each: 16 bytes of K, 16 of V and the row's 8 scale bytes (the factor of a lane's 16
// dimensions is one power of two, applied to its share of the score and, for V, to the weight).  A warp keeps four
// such groups with a maximum, sum and output of their own, joined when the row or the warp's share ends.  Positions
// are read three steps ahead of their use, page entries two, cache rows one, so that only the gathers' throughput
// counts.  A row cut by a share's border leaves parts in the workspace; sparse_parts_kernel joins them in order.
#include "cache_format.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace sd {

namespace {

constexpr int kWarps = 4;          // warps of a CTA (independent of each other)
constexpr int kPer = 2;            // selected rows per group of eight lanes and step
constexpr int kStep = 4 * kPer;    // slots of idx per warp and step
constexpr float kGrow = 8.f;       // log2 units that the maximum may lag behind

// 2^e of a scale byte.  Byte 255 gives an infinity (NaN with the block's zeros).
template <int kFmt>
__device__ __forceinline__ float scale_of(uint32_t byte) {
    if (kFmt == kFmtFp8) return __uint_as_float(byte << 23);
    const uint32_t bits = byte > 6u ? (byte - 6u) << 23 : 1u << (byte + 16u);
    return __uint_as_float(byte == 255u ? 0x7f800000u : bits);
}

// Four elements as fp32, before the scale: e4m3 through the half-precision pair that holds them exactly; int8 as
// 1024 + (x + 128) in half precision, less 1152.
template <int kFmt>
__device__ __forceinline__ void elements4(uint32_t w, float (&x)[4]) {
    uint32_t a, b;
    if (kFmt == kFmtFp8) {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"((uint16_t)w));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(w >> 16)));
    } else {
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t c = 0x64806480u;   // 1152
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(a) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(c));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(b) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(c));
    }
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&b));
    x[0] = lo.x;
    x[1] = lo.y;
    x[2] = hi.x;
    x[3] = hi.y;
}

struct Rows {       // one step's gathers of a lane
    uint4 k[kPer], v[kPer];
    uint2 s[kPer];
    uint32_t live;  // bit u: there is a row
};

__device__ __forceinline__ float* part_out(const CacheSparseArgs& a, long slot) { return a.part + slot * kHeadDim; }

template <int kFmt>
__global__ void __launch_bounds__(kWarps * 32) cache_sparse_kernel(const __grid_constant__ CacheSparseArgs a) {
    pdl_enter();
    const int lane = threadIdx.x & 31, grp = lane >> 3, c = lane & 7;
    const long w = (long)blockIdx.x * kWarps + (threadIdx.x >> 5), W = a.shares;
    if (w >= W) return;
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

        float q[16];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint4 v = reinterpret_cast<const uint4*>(a.q)[(long)r * 16 + c * 2 + x];
            const uint32_t t[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                q[x * 8 + y * 2] = bf16_lo(t[y]) * a.scale_log2;
                q[x * 8 + y * 2 + 1] = bf16_hi(t[y]) * a.scale_log2;
            }
        }
        float o[16], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] = 0.f;

        // lanes 0 .. kStep - 1 look up slot j0 + step * kStep + lane
        auto position = [&](int step) {
            const int j = j0 + step * kStep + lane;
            return lane < kStep && j < j1 ? __ldg(row + j) : -1;
        };
        int before = j0 > 0 ? __ldg(row + j0 - 1) : 0;   // the entry before the step (of the row's first: none)
        bool first = j0 == 0;
        auto page_of = [&](int& e) {   // also the checks of the entry; e = -1 where nothing is to be read
            int p = __shfl_up_sync(0xffffffffu, e, 1);
            if (lane == 0) p = before;
            before = __shfl_sync(0xffffffffu, e, kStep - 1);
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
        auto gather = [&](int e, int page) {
            Rows g;
            int at = -1;   // page and slot
            if (e >= 0) {
                if (page >= 0 && page < a.num_pages) at = page * kPageSize + e % kPageSize;
                else report(a.status, SD_ERR_INDEX_OOB);
            }
            g.live = 0;
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int p = __shfl_sync(0xffffffffu, at, u * 4 + grp);
                g.k[u] = g.v[u] = make_uint4(0u, 0u, 0u, 0u);
                g.s[u] = make_uint2(0u, 0u);
                if (p >= 0) {
                    const long cr = ((long)p * a.Hkv + kvh) * 8 + c;
                    g.k[u] = __ldg(reinterpret_cast<const uint4*>(a.K) + cr);
                    g.v[u] = __ldg(reinterpret_cast<const uint4*>(a.V) + cr);
                    g.s[u] = __ldg(reinterpret_cast<const uint2*>(a.scales + scale_offset(p / kPageSize, kvh, p % kPageSize, a.Hkv)));
                    g.live |= 1u << u;
                }
            }
            return g;
        };

        const int steps = (j1 - j0 + kStep - 1) / kStep;
        int e0 = position(0), e1 = position(1), e2 = position(2);
        int p0 = page_of(e0), p1 = page_of(e1);
        Rows cur = gather(e0, p0);
        for (int t = 0; t < steps; ++t) {
            const int e3 = position(t + 3);
            const int p2 = page_of(e2);
            const Rows nxt = gather(e1, p1);
            float s[kPer], top = -INFINITY;
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const uint32_t kw[4] = {cur.k[u].x, cur.k[u].y, cur.k[u].z, cur.k[u].w};
                float d0 = 0.f, d1 = 0.f;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float k[4];
                    elements4<kFmt>(kw[x], k);
                    d0 = fmaf(k[0], q[x * 4], d0);
                    d1 = fmaf(k[1], q[x * 4 + 1], d1);
                    d0 = fmaf(k[2], q[x * 4 + 2], d0);
                    d1 = fmaf(k[3], q[x * 4 + 3], d1);
                }
                float d = (d0 + d1) * scale_of<kFmt>(cur.s[u].x >> ((c >> 1) * 8) & 255u);
                d += __shfl_xor_sync(0xffffffffu, d, 1);
                d += __shfl_xor_sync(0xffffffffu, d, 2);
                d += __shfl_xor_sync(0xffffffffu, d, 4);
                s[u] = (cur.live >> u & 1) ? d : -INFINITY;
                top = fmaxf(top, s[u]);
            }
            const bool grow = top - m > kGrow;   // (from -infinity: any finite score)
            if (__any_sync(0xffffffffu, grow)) {
                const float f = grow ? ex2(m - top) : 1.f;
                if (grow) m = top;
                l *= f;
#pragma unroll
                for (int x = 0; x < 16; ++x) o[x] *= f;
            }
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const float p = (cur.live >> u & 1) ? ex2(s[u] - m) : 0.f;
                l += p;
                const float pv = p * scale_of<kFmt>(cur.s[u].y >> ((c >> 1) * 8) & 255u);
                const uint32_t vw[4] = {cur.v[u].x, cur.v[u].y, cur.v[u].z, cur.v[u].w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float v[4];
                    elements4<kFmt>(vw[x], v);
#pragma unroll
                    for (int y = 0; y < 4; ++y) o[x * 4 + y] = fmaf(pv, v[y], o[x * 4 + y]);
                }
            }
            cur = nxt;
            e1 = e2;
            e2 = e3;
            p1 = p2;
        }
        // the four groups' parts become one
        float M = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
        const float f = m == -INFINITY ? 0.f : ex2(m - M);
        l *= f;
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const bool whole = j0 == 0 && j1 == a.k_max;
        const float inv = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
#pragma unroll
        for (int x = 0; x < 16; ++x) {
            o[x] *= f;
            o[x] += __shfl_xor_sync(0xffffffffu, o[x], 8);
            o[x] += __shfl_xor_sync(0xffffffffu, o[x], 16);
            o[x] *= inv;
        }
        const long slot = 2 * w + (j0 == 0 ? 1 : 0);   // a share's first row may have begun earlier; its last may go on
        float4* dst = reinterpret_cast<float4*>(whole ? a.out + (long)r * kHeadDim : part_out(a, slot)) + c * 4;
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (grp == x) dst[x] = make_float4(o[x * 4], o[x * 4 + 1], o[x * 4 + 2], o[x * 4 + 3]);
        if (!whole && lane == 0) a.ml[slot] = make_float2(M, l);
    }
}

// Joins the parts of each row that a share's border cut; one warp per row, four dimensions per lane.
constexpr int kJoinWarps = 4;
__global__ void __launch_bounds__(kJoinWarps * 32) sparse_parts_kernel(const __grid_constant__ CacheSparseArgs a) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const long r = (long)blockIdx.x * kJoinWarps + (threadIdx.x >> 5), rows = (long)a.B * a.Hq, W = a.shares;
    if (r >= rows) return;
    const long total = rows * a.k_max, begin = r * a.k_max, end = begin + a.k_max - 1;
    // the share that holds slot x: the w with total w / W <= x < total (w + 1) / W (rounded down)
    const long w0 = ((begin + 1) * W - 1) / total, w1 = ((end + 1) * W - 1) / total;
    if (w0 == w1) return;
    auto slot_of = [&](long w) { return 2 * w + (total * w / W <= begin ? 1 : 0); };
    float m = -INFINITY;
    for (long w = w0 + lane; w <= w1; w += 32) m = fmaxf(m, a.ml[slot_of(w)].x);
#pragma unroll
    for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 8
    for (long w = w0; w <= w1; ++w) {
        const long slot = slot_of(w);
        const float2 ml = a.ml[slot];
        const float4 v = reinterpret_cast<const float4*>(part_out(a, slot))[lane];
        const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
        l = fmaf(ml.y, f, l);
        o.x = fmaf(v.x, f, o.x);
        o.y = fmaf(v.y, f, o.y);
        o.z = fmaf(v.z, f, o.z);
        o.w = fmaf(v.w, f, o.w);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    reinterpret_cast<float4*>(a.out)[r * 32 + lane] = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

template <int kFmt>
cudaError_t launch_format(CacheSparseArgs a, cudaStream_t stream) {
    int per_sm = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, cache_sparse_kernel<kFmt>, kWarps * 32, 0);
    if (e != cudaSuccess) return e;
    const long rows = (long)a.B * a.Hq, slots = rows * a.k_max;
    long shares = (long)a.sms * per_sm * kWarps;
    if (shares > kCacheSparseWarps) shares = kCacheSparseWarps;
    if (shares > slots) shares = slots;   // (a share without a slot would leave a gap between a row's parts)
    a.shares = (int)shares;
    e = launch_pdl(cache_sparse_kernel<kFmt>, dim3((unsigned)((shares + kWarps - 1) / kWarps)), dim3(kWarps * 32), 0, stream, a);
    if (e != cudaSuccess) return e;
    e = launch_pdl(sparse_parts_kernel, dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps)), dim3(kJoinWarps * 32), 0, stream,
                   a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_sparse(const CacheSparseArgs& a, int format, cudaStream_t stream) {
    return format == kFmtFp8 ? launch_format<kFmtFp8>(a, stream) : launch_format<kFmtInt8>(a, stream);
}

}  // namespace sd

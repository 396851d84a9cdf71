// cache_io.cu -- rows of a ragged batch into a paged cache and back out of it, in bf16 or in one of the
// 8-bit microscaling formats (cache_format.cuh).
//
// Both kernels move each byte once and compute little: they are bound by memory (large batches) or by the
// latency of one pass (a decode step).  The unit of work is a run, the rows of one request in one page, for one KV
// head: its page is looked up once, and the page's Quest box comes out of the same pass over the rows.  Each CTA
// counts the runs of every request (a scan over row_start and lens) and takes units in turn.  Sixteen lanes take a
// unit: 8 values of K and 8 of V per lane and row, so that loads and stores are whole 128- or 256-byte rows, and a
// block of 32 values is four neighbouring lanes, whose largest magnitude takes two shuffles.  Several rows are
// loaded before the first one is worked on.
//
// B200: 4 x 16384 rows x 8 heads from bf16 to MXFP8 with boxes 94 us (424 MB: 4.5 TB/s; one row per unit and a walk over the
// page for its box took 383 us, two fp32 factors per value instead of one bf16 product 117 us); 131072 rows x 8 heads
// of MXFP8 to bf16 139 us (814 MB: 5.8 TB/s); a decode step of 32 requests with boxes 10 us
// (8 without the read of each page's earlier rows for its box).
#include "cache_half.cuh"
#include "kernels.h"

namespace sd {

namespace {

constexpr int kIoThreads = 256;
constexpr int kIoCtas = 8;       // CTAs per SM at most (they take units in turn)
constexpr int kIoWave = 32;      // units per SM up to which runs are split
constexpr int kWriteRows = 2;    // rows in flight per unit
constexpr int kReadRows = 8;
constexpr int kEarlierRows = 4;  // rows of a page that were there before, for its box

// The last b with prefix[b] <= run.
__device__ __forceinline__ int request_of(const int* prefix, int B, int run) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= run) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The largest magnitude of eight bf16, as bf16 bits (infinities and NaN are the largest).
__device__ __forceinline__ uint32_t abs_max(const uint4& v) {
    const uint32_t m = max_u16x2(max_u16x2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), max_u16x2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    return max(m & 0xffffu, m >> 16);
}

// Eight values of K and of V of a lane (four lanes are a block): elements and the blocks' scale bytes.
template <int kFmt>
__device__ __forceinline__ void quantise8(const uint4& k, const uint4& v, uint32_t mask, uint2& ke, uint2& ve, uint32_t& kb,
                                          uint32_t& vb) {
    uint32_t m = abs_max(k) | (abs_max(v) << 16);
    m = max_u16x2(m, __shfl_xor_sync(mask, m, 1));
    m = max_u16x2(m, __shfl_xor_sync(mask, m, 2));
    kb = scale_byte<kFmt>(m << 16);
    vb = scale_byte<kFmt>(m & 0xffff0000u);
    ke = make_uint2(encode4<kFmt>(k.x, k.y, kb), encode4<kFmt>(k.z, k.w, kb));
    ve = make_uint2(encode4<kFmt>(v.x, v.y, vb), encode4<kFmt>(v.z, v.w, vb));
    if (kb == 255u) ke = make_uint2(0u, 0u);
    if (vb == 255u) ve = make_uint2(0u, 0u);
}

template <int kFmt>
__device__ __forceinline__ uint4 dequantise8(const uint2& e, uint32_t byte) {
    const Factor f = factor_of<kFmt>(byte);
    uint4 r;
    decode4<kFmt>(e.x, f, r.x, r.y);
    decode4<kFmt>(e.y, f, r.z, r.w);
    return r;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p)); }

__device__ __forceinline__ void box_with(uint4& lo, uint4& hi, const uint4& v) {
    uint32_t* l = reinterpret_cast<uint32_t*>(&lo);
    uint32_t* h = reinterpret_cast<uint32_t*>(&hi);
    const uint32_t* k = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const __nv_bfloat162 kv = *reinterpret_cast<const __nv_bfloat162*>(&k[t]);
        const __nv_bfloat162 mn = __hmin2(*reinterpret_cast<const __nv_bfloat162*>(&l[t]), kv);
        const __nv_bfloat162 mx = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&h[t]), kv);
        l[t] = *reinterpret_cast<const uint32_t*>(&mn);
        h[t] = *reinterpret_cast<const uint32_t*>(&mx);
    }
}

// The runs of the batch: `prefix` (shared memory, [B + 1]) gets the number of runs before each request.  Request b's
// rows are positions begin(b, n, N) .. + n - 1; a bad request is reported and has none.  Returns the number of runs, 0
// where row_start is not valid.
struct Rows {
    int rs, begin, n;   // first row, its position, rows
};
template <bool kRead>
__device__ __forceinline__ Rows rows_of(const CacheIoArgs& a, int b) {
    Rows r;
    r.rs = a.row_start[b];
    r.n = a.row_start[b + 1] - r.rs;
    r.begin = kRead ? a.first[b] : a.lens[b] - r.n;
    return r;
}
template <bool kRead>
__device__ __forceinline__ int plan_runs(const CacheIoArgs& a, int* prefix, int* scratch) {
    const int per = (a.B + kIoThreads - 1) / kIoThreads;
    const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
    bool bad = false;
    int mine = 0;
    for (int b = b0; b < b1; ++b) {
        const int lo = a.row_start[b], hi = a.row_start[b + 1];
        bad = bad || lo < 0 || hi < lo || hi > a.total_rows;
        const int N = a.lens[b], n = hi - lo;
        if (bad || n == 0) continue;
        const int begin = kRead ? a.first[b] : N - n;
        if (N < 0 || (long)N > a.n_cap || begin < 0 || (long)begin + n > N) {
            if (blockIdx.x == 0) report(a.status, SD_ERR_INVALID_ARG);
            continue;
        }
        mine += (begin + n - 1) / kPageSize - begin / kPageSize + 1;
    }
    if (__syncthreads_or(bad ? 1 : 0)) {
        if (threadIdx.x == 0 && blockIdx.x == 0) report(a.status, SD_ERR_INVALID_ARG);
        return 0;
    }
    int total;
    int at = block_exclusive_scan(mine, scratch, &total);
    for (int b = b0; b < b1; ++b) {
        prefix[b] = at;
        const Rows r = rows_of<kRead>(a, b);
        const int N = a.lens[b];
        if (r.n > 0 && N >= 0 && (long)N <= a.n_cap && r.begin >= 0 && (long)r.begin + r.n <= N)
            at += (r.begin + r.n - 1) / kPageSize - r.begin / kPageSize + 1;
    }
    if (threadIdx.x == 0) prefix[a.B] = total;
    __syncthreads();
    return total;
}

// Part `part` of run `run`: the rows whose slots lie in its share of the page.  page -1: a bad entry, reported.
struct Run {
    int page, slot, row, count;
    bool joins;   // the page holds earlier rows of the request
};
template <bool kRead>
__device__ __forceinline__ Run run_of(const CacheIoArgs& a, const int* prefix, int run, int slot0, int slot1) {
    const int b = request_of(prefix, a.B, run);   // (requests without runs share their successor's prefix)
    const Rows r = rows_of<kRead>(a, b);
    const int pi = r.begin / kPageSize + run - prefix[b];
    const int p0 = max(r.begin, pi * kPageSize + slot0), p1 = min(r.begin + r.n, pi * kPageSize + slot1);
    Run u;
    u.page = a.page_table[(long)b * a.max_pages + pi];
    u.slot = p0 - pi * kPageSize;
    u.row = r.rs + p0 - r.begin;
    u.count = p1 - p0;
    u.joins = r.begin > pi * kPageSize;
    if (u.page < 0 || u.page >= a.num_pages) {
        report(a.status, SD_ERR_INDEX_OOB);
        u.count = 0;
    }
    return u;
}

// New rows into the cache, and the Quest box of each run's page: the minimum and maximum of its rows as stored, the new ones
// and those that the request had there before.  (These are read again: the stored box may know rows that a rejected draft
// had in the place of the new ones.  They lie before the new rows' slots, which alone are written here.)  Where runs
// are taken in parts, one more unit per run makes the box alone (from the new rows, rounded again).
template <int kFmt>
__global__ void __launch_bounds__(kIoThreads, 4) cache_write_kernel(const __grid_constant__ CacheIoArgs a) {
    extern __shared__ int prefix[];
    __shared__ int scratch[40];
    pdl_enter();
    const bool apart = a.parts > 1 && a.boxes != nullptr;   // boxes by units of their own
    const int per_run = a.parts + (apart ? 1 : 0), share = kPageSize / a.parts;
    const long units = (long)plan_runs<false>(a, prefix, scratch) * per_run * a.Hkv;
    const int c = threadIdx.x & 15;
    const uint32_t mask = (threadIdx.x & 16) ? 0xffff0000u : 0x0000ffffu;
    for (long it = (long)blockIdx.x * (kIoThreads / 16) + (threadIdx.x >> 4); it < units; it += (long)gridDim.x * (kIoThreads / 16)) {
        const int x = (int)(it / a.Hkv), kvh = (int)(it - (long)x * a.Hkv), run = x / per_run, part = x - run * per_run;
        const bool alone = part == a.parts;
        const Run u = run_of<false>(a, prefix, run, alone ? 0 : part * share, alone ? kPageSize : (part + 1) * share);
        if (u.count <= 0) continue;
        const long src = ((long)u.row * a.Hkv + kvh) * 16 + c;                                    // 16-byte chunks
        const long dst = (((long)u.page * kPageSize + u.slot) * a.Hkv + kvh) * 16 + c;            // 16- or 8-byte chunks
        const long step = (long)a.Hkv * 16;
        uint4* box = a.boxes == nullptr || apart != alone ? nullptr
                                                          : reinterpret_cast<uint4*>(a.boxes) + ((long)u.page * a.Hkv + kvh) * 32 + c;
        uint4 lo = make_uint4(0x7f807f80u, 0x7f807f80u, 0x7f807f80u, 0x7f807f80u);   // +inf, -inf
        uint4 hi = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
        const long page_row = ((long)u.page * kPageSize * a.Hkv + kvh) * 16;   // the page's first row, in chunks
        const bool earlier = box != nullptr && u.joins;
        if (earlier && c < u.slot) {   // a lane each of the request's earlier rows in the page, which are taken below
            const uint8_t* row = static_cast<const uint8_t*>(a.K) + (page_row + c * step) * (kFmt == kFmtBf16 ? 16 : 8);
            prefetch_l2(row);
            if (kFmt == kFmtBf16) prefetch_l2(row + 128);
            else prefetch_l2(a.scales + scale_offset(u.page, kvh, c, a.Hkv));
        }
        for (int j0 = 0; j0 < u.count; j0 += kWriteRows) {
            uint4 k[kWriteRows], v[kWriteRows];
#pragma unroll
            for (int j = 0; j < kWriteRows; ++j)
                if (j0 + j < u.count) {
                    k[j] = __ldg(reinterpret_cast<const uint4*>(a.k_in) + src + (j0 + j) * step);
                    v[j] = __ldg(reinterpret_cast<const uint4*>(a.v_in) + src + (j0 + j) * step);
                }
#pragma unroll
            for (int j = 0; j < kWriteRows; ++j) {
                if (j0 + j >= u.count) continue;
                const long to = dst + (j0 + j) * step;
                if (kFmt == kFmtBf16) {
                    if (!alone) {
                        reinterpret_cast<uint4*>(a.K)[to] = k[j];
                        reinterpret_cast<uint4*>(a.V)[to] = v[j];
                    }
                } else {
                    uint32_t kb, vb;
                    uint2 ke, ve;
                    quantise8<kFmt>(k[j], v[j], mask, ke, ve, kb, vb);
                    if (!alone) {
                        reinterpret_cast<uint2*>(a.K)[to] = ke;
                        reinterpret_cast<uint2*>(a.V)[to] = ve;
                        uint32_t s = kb | vb << 8, t = __shfl_xor_sync(mask, s, 4);   // the row's bytes together
                        s = (c & 4) ? t | s << 16 : s | t << 16;
                        t = __shfl_xor_sync(mask, s, 8);
                        if (c == 0)
                            *reinterpret_cast<uint2*>(a.scales + scale_offset(u.page, kvh, u.slot + j0 + j, a.Hkv)) =
                                make_uint2(__byte_perm(s, t, 0x6420), __byte_perm(s, t, 0x7531));
                    }
                    if (box != nullptr) k[j] = dequantise8<kFmt>(ke, kb);
                }
                if (box != nullptr) box_with(lo, hi, k[j]);
            }
        }
        if (earlier) {
            const uint8_t* sc = kFmt == kFmtBf16 ? nullptr : a.scales + scale_offset(u.page, kvh, 0, a.Hkv) + (c >> 2);
            for (int j0 = 0; j0 < u.slot; j0 += kEarlierRows) {
                uint4 k[kEarlierRows];
                uint2 e[kEarlierRows];
                uint32_t by[kEarlierRows];
#pragma unroll
                for (int j = 0; j < kEarlierRows; ++j) {
                    const int slot = min(j0 + j, u.slot - 1);   // (the last one again: no change to the box)
                    if (kFmt == kFmtBf16) {
                        k[j] = reinterpret_cast<const uint4*>(a.K)[page_row + c + slot * step];
                    } else {
                        e[j] = reinterpret_cast<const uint2*>(a.K)[page_row + c + slot * step];
                        by[j] = sc[slot * 2 * kScaleBytes];
                    }
                }
#pragma unroll
                for (int j = 0; j < kEarlierRows; ++j) box_with(lo, hi, kFmt == kFmtBf16 ? k[j] : dequantise8<kFmt>(e[j], by[j]));
            }
        }
        if (box != nullptr) {
            box[0] = lo;
            box[16] = hi;
        }
    }
}

// Positions first[b] .. first[b] + n_b - 1 of every request back as bf16 rows.
template <int kFmt>
__global__ void __launch_bounds__(kIoThreads, 3) cache_read_kernel(const __grid_constant__ CacheIoArgs a) {
    extern __shared__ int prefix[];
    __shared__ int scratch[40];
    pdl_enter();
    const int share = kPageSize / a.parts;
    const long units = (long)plan_runs<true>(a, prefix, scratch) * a.parts * a.Hkv;
    const int c = threadIdx.x & 15;
    for (long it = (long)blockIdx.x * (kIoThreads / 16) + (threadIdx.x >> 4); it < units; it += (long)gridDim.x * (kIoThreads / 16)) {
        const int x = (int)(it / a.Hkv), kvh = (int)(it - (long)x * a.Hkv), run = x / a.parts, part = x - run * a.parts;
        const Run u = run_of<true>(a, prefix, run, part * share, (part + 1) * share);
        if (u.count <= 0) continue;
        const long src = (((long)u.page * kPageSize + u.slot) * a.Hkv + kvh) * 16 + c;
        const long dst = ((long)u.row * a.Hkv + kvh) * 16 + c;
        const long step = (long)a.Hkv * 16;
        const uint8_t* sc = kFmt == kFmtBf16 ? nullptr : a.scales + scale_offset(u.page, kvh, u.slot, a.Hkv) + (c >> 2);
#pragma unroll
        for (int half = 0; half < 2; ++half) {   // K, V
            const void* from = half ? a.V : a.K;
            uint4* to = reinterpret_cast<uint4*>(half ? a.v_out : a.k_out);
            if (to == nullptr) continue;
            for (int j0 = 0; j0 < u.count; j0 += kReadRows) {
                uint4 r[kReadRows];
                uint2 e[kReadRows];
                uint32_t by[kReadRows];
#pragma unroll
                for (int j = 0; j < kReadRows; ++j)
                    if (j0 + j < u.count) {
                        if (kFmt == kFmtBf16) {
                            r[j] = __ldg(reinterpret_cast<const uint4*>(from) + src + (j0 + j) * step);
                        } else {
                            e[j] = __ldg(reinterpret_cast<const uint2*>(from) + src + (j0 + j) * step);
                            by[j] = __ldg(sc + (j0 + j) * 2 * kScaleBytes + half * kScaleBytes);
                        }
                    }
#pragma unroll
                for (int j = 0; j < kReadRows; ++j)
                    if (j0 + j < u.count) to[dst + (j0 + j) * step] = kFmt == kFmtBf16 ? r[j] : dequantise8<kFmt>(e[j], by[j]);
            }
        }
    }
}

template <typename Kernel>
cudaError_t launch_io(Kernel kernel, CacheIoArgs a, cudaStream_t stream) {
    // at most total_rows / 16 + 2 B runs (and no more than rows)
    const long runs = min((long)a.total_rows, (long)a.total_rows / kPageSize + 2L * a.B);
    // Small batches take runs in parts, so that every SM has work: as many as keep the units within about one wave.
    a.parts = 1;
    while (a.parts < kPageSize && runs * a.Hkv * a.parts * 2 <= (long)a.sms * kIoWave) a.parts *= 2;
    const long units = runs * a.Hkv * (a.parts + (a.parts > 1 && a.boxes != nullptr ? 1 : 0));
    const long want = (units + kIoThreads / 16 - 1) / (kIoThreads / 16), most = (long)a.sms * kIoCtas;
    const unsigned grid = (unsigned)(want < 1 ? 1 : want < most ? want : most);
    cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(kIoThreads), sizeof(int) * (a.B + 1), stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write(const CacheIoArgs& a, int format, cudaStream_t stream) {
    return launch_io(format == kFmtBf16 ? cache_write_kernel<kFmtBf16>
                     : format == kFmtFp8 ? cache_write_kernel<kFmtFp8> : cache_write_kernel<kFmtInt8>, a, stream);
}
cudaError_t launch_cache_read(const CacheIoArgs& a, int format, cudaStream_t stream) {
    return launch_io(format == kFmtBf16 ? cache_read_kernel<kFmtBf16>
                     : format == kFmtFp8 ? cache_read_kernel<kFmtFp8> : cache_read_kernel<kFmtInt8>, a, stream);
}

}  // namespace sd

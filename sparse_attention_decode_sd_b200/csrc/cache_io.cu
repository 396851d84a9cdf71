// cache_io.cu -- rows of a ragged batch into a paged cache and back out of it, in bf16 or in one of the
// 8-bit microscaling formats (cache_format.cuh).
//
// Both kernels move each byte once and compute little: they are bound by memory (large batches) or by the
// latency of one pass (a decode step).  Sixteen lanes take one (row, KV head): 8 values of K and 8 of V per
// lane, so that a warp's loads and stores are whole 128- or 256-byte rows, and a block of 32 values is four
// neighbouring lanes, whose largest magnitude takes two shuffles.
#include "cache_format.cuh"
#include "kernels.h"
#include "ragged.cuh"

namespace sd {

constexpr int kIoThreads = 256;

__device__ __forceinline__ uint32_t abs_max_bits(const uint4& v) {   // of eight bf16, as fp32 bits
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    return m << 16;
}

// Eight values of a lane (four lanes are a block): element bytes and the block's scale byte.
template <int kFmt>
__device__ __forceinline__ uint2 quantise8(const uint4& v, uint32_t mask, uint32_t& byte) {
    uint32_t m = abs_max_bits(v);
    m = max(m, __shfl_xor_sync(mask, m, 1));
    m = max(m, __shfl_xor_sync(mask, m, 2));
    byte = scale_byte<kFmt>(m);
    if (byte == 255u) return make_uint2(0u, 0u);
    float f1, f2;
    inverse_scale<kFmt>(byte, f1, f2);
    return make_uint2(encode4<kFmt>(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y), f1, f2),
                      encode4<kFmt>(bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w), f1, f2));
}

template <int kFmt>
__device__ __forceinline__ uint4 dequantise8(const uint2& e, uint32_t byte) {
    const Factor f = factor_of<kFmt>(byte);
    uint4 r;
    decode4<kFmt>(e.x, f, r.x, r.y);
    decode4<kFmt>(e.y, f, r.z, r.w);
    return r;
}

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

// New rows into the cache.  The first new row of each page also makes the page's Quest box: the minimum and
// maximum, as stored, of the page's new rows and -- when rows were there before -- of the stored box.
template <int kFmt>
__global__ void __launch_bounds__(kIoThreads) cache_write_kernel(CacheIoArgs a) {
    extern __shared__ int rs[];
    pdl_enter();
    if (!load_row_start(a.row_start, a.B, a.total_rows, rs, a.status)) return;
    const int c = threadIdx.x & 15;
    const uint32_t mask = (threadIdx.x & 16) ? 0xffff0000u : 0x0000ffffu;
    const long per_grid = (long)gridDim.x * (kIoThreads / 16);
    const long first = (long)rs[0] * a.Hkv, items = (long)rs[a.B] * a.Hkv;
    for (long it = first + (long)blockIdx.x * (kIoThreads / 16) + (threadIdx.x >> 4); it < items; it += per_grid) {
        const int t = (int)(it / a.Hkv), kvh = (int)(it - (long)t * a.Hkv);
        const long src = it * 16 + c;
        const uint4 kr = reinterpret_cast<const uint4*>(a.k_in)[src];
        const uint4 vr = reinterpret_cast<const uint4*>(a.v_in)[src];
        const int b = request_of(rs, a.B, t);
        const int n = rs[b + 1] - rs[b], N = checked_len(a.lens, b, a.n_cap, a.status);
        if (n > N) {
            report(a.status, SD_ERR_INVALID_ARG);
            continue;
        }
        const int p = N - n + (t - rs[b]);
        const int page = a.page_table[(long)b * a.max_pages + p / kPageSize];
        if (page < 0 || page >= a.num_pages) {
            report(a.status, SD_ERR_INDEX_OOB);
            continue;
        }
        const int slot = p % kPageSize;
        const long row = ((long)page * kPageSize + slot) * a.Hkv + kvh;
        uint4 kept = kr;
        if (kFmt == kFmtBf16) {
            reinterpret_cast<uint4*>(a.K)[row * 16 + c] = kr;
            reinterpret_cast<uint4*>(a.V)[row * 16 + c] = vr;
        } else {
            uint32_t kb, vb;
            const uint2 ke = quantise8<kFmt>(kr, mask, kb), ve = quantise8<kFmt>(vr, mask, vb);
            reinterpret_cast<uint2*>(a.K)[row * 16 + c] = ke;
            reinterpret_cast<uint2*>(a.V)[row * 16 + c] = ve;
            if ((c & 3) == 0) {
                uint8_t* s = a.scales + scale_offset(page, kvh, slot, a.Hkv) + (c >> 2);
                s[0] = (uint8_t)kb;
                s[kScaleBytes] = (uint8_t)vb;
            }
            kept = dequantise8<kFmt>(ke, kb);
        }
        if (a.boxes != nullptr && (slot == 0 || t == rs[b])) {
            uint4* box = reinterpret_cast<uint4*>(a.boxes) + ((long)page * a.Hkv + kvh) * 32 + c;
            uint4 lo = kept, hi = kept;
            if (slot != 0) {
                lo = box[0];
                hi = box[16];
                box_with(lo, hi, kept);
            }
            const int more = min(kPageSize - slot, rs[b + 1] - t);
            for (int j = 1; j < more; ++j) {
                uint4 r = reinterpret_cast<const uint4*>(a.k_in)[src + (long)j * a.Hkv * 16];
                if (kFmt != kFmtBf16) {
                    uint32_t kb;
                    const uint2 ke = quantise8<kFmt>(r, mask, kb);
                    r = dequantise8<kFmt>(ke, kb);
                }
                box_with(lo, hi, r);
            }
            box[0] = lo;
            box[16] = hi;
        }
    }
}

// Positions first[b] .. first[b] + n_b - 1 of every request back as bf16 rows.
template <int kFmt>
__global__ void __launch_bounds__(kIoThreads) cache_read_kernel(CacheIoArgs a) {
    extern __shared__ int rs[];
    pdl_enter();
    if (!load_row_start(a.row_start, a.B, a.total_rows, rs, a.status)) return;
    const int c = threadIdx.x & 15;
    const long per_grid = (long)gridDim.x * (kIoThreads / 16);
    const long first = (long)rs[0] * a.Hkv, items = (long)rs[a.B] * a.Hkv;
    for (long it = first + (long)blockIdx.x * (kIoThreads / 16) + (threadIdx.x >> 4); it < items; it += per_grid) {
        const int t = (int)(it / a.Hkv), kvh = (int)(it - (long)t * a.Hkv);
        const int b = request_of(rs, a.B, t);
        const int n = rs[b + 1] - rs[b], N = checked_len(a.lens, b, a.n_cap, a.status), p0 = a.first[b];
        if (p0 < 0 || (long)p0 + n > N) {
            report(a.status, SD_ERR_INVALID_ARG);
            continue;
        }
        const int p = p0 + (t - rs[b]);
        const int page = a.page_table[(long)b * a.max_pages + p / kPageSize];
        if (page < 0 || page >= a.num_pages) {
            report(a.status, SD_ERR_INDEX_OOB);
            continue;
        }
        const int slot = p % kPageSize;
        const long row = ((long)page * kPageSize + slot) * a.Hkv + kvh;
        const long dst = it * 16 + c;
        const uint8_t* s = kFmt == kFmtBf16 ? nullptr : a.scales + scale_offset(page, kvh, slot, a.Hkv) + (c >> 2);
        if (a.k_out != nullptr) {
            const uint4 r = kFmt == kFmtBf16 ? reinterpret_cast<const uint4*>(a.K)[row * 16 + c]
                                             : dequantise8<kFmt>(reinterpret_cast<const uint2*>(a.K)[row * 16 + c], s[0]);
            reinterpret_cast<uint4*>(a.k_out)[dst] = r;
        }
        if (a.v_out != nullptr) {
            const uint4 r = kFmt == kFmtBf16
                                ? reinterpret_cast<const uint4*>(a.V)[row * 16 + c]
                                : dequantise8<kFmt>(reinterpret_cast<const uint2*>(a.V)[row * 16 + c], s[kScaleBytes]);
            reinterpret_cast<uint4*>(a.v_out)[dst] = r;
        }
    }
}

static cudaError_t launch_io(void (*kernel)(CacheIoArgs), const CacheIoArgs& a, cudaStream_t stream) {
    const long want = ((long)a.total_rows * a.Hkv + kIoThreads / 16 - 1) / (kIoThreads / 16);
    const long most = (long)a.sms * 8;
    const unsigned grid = (unsigned)(want < 1 ? 1 : want < most ? want : most);
    cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(kIoThreads), sizeof(int) * (a.B + 1), stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_cache_write(const CacheIoArgs& a, int format, cudaStream_t stream) {
    return launch_io(format == kFmtBf16 ? cache_write_kernel<kFmtBf16>
                     : format == kFmtFp8 ? cache_write_kernel<kFmtFp8> : cache_write_kernel<kFmtInt8>, a, stream);
}
cudaError_t launch_cache_read(const CacheIoArgs& a, int format, cudaStream_t stream) {
    return launch_io(format == kFmtBf16 ? cache_read_kernel<kFmtBf16>
                     : format == kFmtFp8 ? cache_read_kernel<kFmtFp8> : cache_read_kernel<kFmtInt8>, a, stream);
}

}  // namespace sd

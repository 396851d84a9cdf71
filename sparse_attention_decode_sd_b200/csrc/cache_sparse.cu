// cache_sparse.cu -- exact attention over the selected rows of an 8-bit paged cache (the sparse decode of
// sparse_decode.cu, for the formats of cache_format.cuh).
//
// One warp takes one (request, query head): 32 entries of idx at a time are checked, then visited in
// order; lane l holds dimensions 4 l .. 4 l + 3 of q and of the output, with an fp32 online softmax.
#include "cache_format.cuh"
#include "kernels.h"

namespace sd {

template <int kFmt>
__device__ __forceinline__ void load_row4(const void* base, long row, const uint8_t* scale, int l, float (&x)[4]) {
    uint32_t lo, hi;
    decode4<kFmt>(reinterpret_cast<const uint32_t*>(base)[row * 32 + l], factor_of<kFmt>(scale[l >> 3]), lo, hi);
    x[0] = bf16_lo(lo);
    x[1] = bf16_hi(lo);
    x[2] = bf16_lo(hi);
    x[3] = bf16_hi(hi);
}

template <int kFmt>
__global__ void __launch_bounds__(128) cache_sparse_kernel(CacheSparseArgs a) {
    pdl_enter();
    const int l = threadIdx.x & 31, rows = a.B * a.Hq;
    const int r = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (r >= rows) return;
    const int b = r / a.Hq, h = r - b * a.Hq, kvh = h / a.G;
    const int N = checked_len(a.lens, b, a.n_cap, a.status);
    const uint2 qv = reinterpret_cast<const uint2*>(a.q)[(long)r * 32 + l];
    const float q[4] = {bf16_lo(qv.x), bf16_hi(qv.x), bf16_lo(qv.y), bf16_hi(qv.y)};
    float o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, sum = 0.f;
    int prev = -1;
    bool ended = false;
    for (int j0 = 0; j0 < a.k_max; j0 += 32) {
        const int j = j0 + l;
        const int e = j < a.k_max ? a.idx[(long)r * a.k_max + j] : -1;
        int before = __shfl_up_sync(0xffffffffu, e, 1);
        if (l == 0) before = ended ? -1 : prev;
        const bool first = j == 0;
        // an entry after padding, or not above the one before it
        const bool order = e >= 0 && !first && (before < 0 || e <= before);
        if (order) report(a.status, SD_ERR_ORDER);
        if (e >= N) report(a.status, SD_ERR_INDEX_OOB);
        int page = -1;
        if (e >= 0 && e < N && !order) {
            page = a.page_table[(long)b * a.max_pages + e / kPageSize];
            if (page < 0 || page >= a.num_pages) {
                report(a.status, SD_ERR_INDEX_OOB);
                page = -1;
            }
        }
        prev = __shfl_sync(0xffffffffu, e, 31);
        uint32_t live = __ballot_sync(0xffffffffu, page >= 0);
        const uint32_t gone = __ballot_sync(0xffffffffu, e < 0);
        ended = gone != 0u;
        while (live) {
            const int s0 = __ffs(live) - 1;
            live &= live - 1;
            const int p = __shfl_sync(0xffffffffu, e, s0), pg = __shfl_sync(0xffffffffu, page, s0);
            const int slot = p % kPageSize;
            const long row = ((long)pg * kPageSize + slot) * a.Hkv + kvh;
            const uint8_t* sc = a.scales + scale_offset(pg, kvh, slot, a.Hkv);
            float k[4], v[4];
            load_row4<kFmt>(a.K, row, sc, l, k);
            load_row4<kFmt>(a.V, row, sc + kScaleBytes, l, v);
            float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
            for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
            s *= a.scale_log2;
            const float mn = fmaxf(m, s), c = exp2f(m - mn), w = exp2f(s - mn);
            m = mn;
            sum = sum * c + w;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = o[i] * c + w * v[i];
        }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    reinterpret_cast<float4*>(a.out)[(long)r * 32 + l] = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
}

cudaError_t launch_cache_sparse(const CacheSparseArgs& a, int format, cudaStream_t stream) {
    const dim3 grid((unsigned)((a.B * a.Hq + 3) / 4)), block(128);
    cudaError_t e = format == kFmtFp8 ? launch_pdl(cache_sparse_kernel<kFmtFp8>, grid, block, 0, stream, a)
                                      : launch_pdl(cache_sparse_kernel<kFmtInt8>, grid, block, 0, stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sd

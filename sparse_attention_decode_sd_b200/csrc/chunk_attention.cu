// chunk_attention.cu -- causal attention of each request's newest positions over its paged cache.
//
//   out[t, h] = sum_i w_i V[b, h/G, i],  w = softmax over 0 <= i <= p of (q[t, h] . K[b, h/G, i]) / sqrt(d)
//
// for row t = row_start[b] + j at position p = N_b - n_b + j.  One warp takes one (row, query head): lane l
// holds dimensions 4 l .. 4 l + 3 of q and of the output, walks the positions in order with an fp32
// online softmax and reads each K and V row in its stored form.
#include "cache_format.cuh"
#include "kernels.h"
#include "ragged.cuh"

namespace sd {

// Four consecutive values (dimensions 4 l .. 4 l + 3) of a cache row, as fp32.
template <int kFmt>
__device__ __forceinline__ void load4(const void* base, long row, const uint8_t* scale, int l, float (&x)[4]) {
    uint32_t lo, hi;
    if (kFmt == kFmtBf16) {
        const uint2 v = reinterpret_cast<const uint2*>(base)[row * 32 + l];
        lo = v.x;
        hi = v.y;
    } else {
        decode4<kFmt>(reinterpret_cast<const uint32_t*>(base)[row * 32 + l], factor_of<kFmt>(scale[l >> 3]), lo, hi);
    }
    x[0] = bf16_lo(lo);
    x[1] = bf16_hi(lo);
    x[2] = bf16_lo(hi);
    x[3] = bf16_hi(hi);
}

template <int kFmt>
__global__ void __launch_bounds__(128) chunk_attention_kernel(ChunkArgs a) {
    extern __shared__ int row_starts[];
    pdl_enter();
    if (!load_row_start(a.row_start, a.B, a.total_rows, row_starts, a.status)) return;
    const int l = threadIdx.x & 31;
    const long unit = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int h = (int)(unit % a.Hq);
    const long t = unit / a.Hq;
    if (t >= a.total_rows) return;
    if (t < row_starts[0] || t >= row_starts[a.B]) return;
    const int b = request_of(row_starts, a.B, (int)t), rs = row_starts[b], re = row_starts[b + 1];
    const int N = checked_len(a.lens, b, a.n_cap, a.status);
    if (re - rs > N) {
        report(a.status, SD_ERR_INVALID_ARG);
        return;
    }
    const int seen = N - (re - rs) + (int)(t - rs) + 1, kvh = h / a.G;
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, sum = 0.f;
    load4<kFmtBf16>(a.q, t * a.Hq + h, nullptr, l, q);
    int page = 0;
    for (int p = 0; p < seen; ++p) {
        if (p % kPageSize == 0) {
            page = a.page_table[(long)b * a.max_pages + p / kPageSize];
            if (page < 0 || page >= a.num_pages) {
                report(a.status, SD_ERR_INDEX_OOB);
                return;
            }
        }
        const long row = ((long)page * kPageSize + p % kPageSize) * a.Hkv + kvh;
        const uint8_t* sc = kFmt == kFmtBf16 ? nullptr : a.scales + scale_offset(page, kvh, p % kPageSize, a.Hkv);
        float k[4], v[4];
        load4<kFmt>(a.K, row, sc, l, k);
        load4<kFmt>(a.V, row, kFmt == kFmtBf16 ? nullptr : sc + kScaleBytes, l, v);
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
    const float r = 1.f / sum;
    reinterpret_cast<uint2*>(a.out)[(t * a.Hq + h) * 32 + l] =
        make_uint2(pack_bf16x2(o[0] * r, o[1] * r), pack_bf16x2(o[2] * r, o[3] * r));
}

cudaError_t launch_chunk_attention(const ChunkArgs& a, int format, cudaStream_t stream) {
    const dim3 grid((unsigned)(((long)a.total_rows * a.Hq + 3) / 4)), block(128);
    const size_t smem = sizeof(int) * (a.B + 1);
    cudaError_t e = format == kFmtBf16 ? launch_pdl(chunk_attention_kernel<kFmtBf16>, grid, block, smem, stream, a)
                    : format == kFmtFp8 ? launch_pdl(chunk_attention_kernel<kFmtFp8>, grid, block, smem, stream, a)
                                        : launch_pdl(chunk_attention_kernel<kFmtInt8>, grid, block, smem, stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sd

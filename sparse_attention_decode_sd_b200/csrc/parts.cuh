// parts.cuh -- joining parts of a softmax-weighted sum, each with its own reference m: sum l = sum 2^(s - m) and
// output o = sum 2^(s - m) v of four dimensions.
#pragma once

#include "tcgen05.cuh"

namespace sd {

struct PartSum {
    float m, l;
    float4 o;
};
__device__ __forceinline__ PartSum no_parts() { return {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)}; }

// The reference to m, at least the one so far.
__device__ __forceinline__ void raise(PartSum& s, float m) {
    const float f = m > s.m ? ex2(s.m - m) : 1.f;
    s.m = m;
    s.l *= f;
    s.o = make_float4(s.o.x * f, s.o.y * f, s.o.z * f, s.o.w * f);
}
// n parts at once, (m, l) and output each; parts that are not there have m = -infinity and zeros.
template <int n>
__device__ __forceinline__ void join(PartSum& s, const float2 (&ml)[n], const float4 (&v)[n]) {
    float m = s.m;
#pragma unroll
    for (int y = 0; y < n; ++y) m = fmaxf(m, ml[y].x);
    raise(s, m);
    const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int y = 0; y < n; ++y) {
        const float f = ex2(ml[y].x - ms);
        s.l = fmaf(ml[y].y, f, s.l);
        s.o.x = fmaf(v[y].x, f, s.o.x);
        s.o.y = fmaf(v[y].y, f, s.o.y);
        s.o.z = fmaf(v[y].z, f, s.o.z);
        s.o.w = fmaf(v[y].w, f, s.o.w);
    }
}

}  // namespace sd

// Shared pieces of the layer operators (include/gdn_layer.h): 8-element row
// accesses, the scalar maps, and the fixed-order sum of per-block partials.
#pragma once

#include "../../include/gdn_layer.h"
#include "gdn_internal.cuh"

namespace gdn {

// 8 consecutive elements: one 16-byte access of bf16, two of fp32.
__device__ __forceinline__ void ld8(const float* p, float* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void ld8(const __nv_bfloat16* p, float* v) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void st8(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void st8(__nv_bfloat16* p, const float* v) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// Sum over the L consecutive lanes (L a power of two) that share a row.
template <int L>
__device__ __forceinline__ float lane_sum(float x) {
#pragma unroll
  for (int m = L / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

__device__ __forceinline__ float sigmoidf_(float x) { return 1.f / (1.f + expf(-x)); }
// log(1 + e^x) without overflow for large x and without cancellation for small
__device__ __forceinline__ float softplusf_(float x) {
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}

// out[i] = sum over p of part[p][i], i < n, p < np, in a fixed order; column i
// belongs to array i / C of up to three outputs (NULL: dropped).
cudaError_t col_sum(const float* part, int np, int n, int C, float* o0, float* o1, float* o2,
                    cudaStream_t st);

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t elem_size(int dtype) { return dtype == GDN_DTYPE_BF16 ? 2 : 4; }
inline bool dtype_ok(int d) { return d == GDN_DTYPE_F32 || d == GDN_DTYPE_BF16; }
// A row access of 16 bytes at a time: pointer and stride.
inline bool vec_rows(const void* p, long long ld, int dtype) {
  return aligned(p, 16) && ld >= 0 && (ld * (long long)elem_size(dtype)) % 16 == 0;
}
inline size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace gdn

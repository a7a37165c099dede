// Shared pieces of the layer operators (include/gdn_layer.h): 8-element row
// accesses, the scalar maps, and the fixed-order sum of per-block partials.
#pragma once

#include "../../include/gdn_layer.h"
#include "gdn_internal.cuh"

namespace gdn {

// Two fp32 lanes in one register pair (one instruction for both).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 both2(float a) { return pack2(a, a); }
__device__ __forceinline__ float sum2(f32x2 a) {
  float lo, hi;
  unpack2(a, lo, hi);
  return lo + hi;
}

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
// 8 elements as loaded, converted when used.
template <typename T>
struct Raw8 {
  uint4 u[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> ldraw8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.u[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
__device__ __forceinline__ void cvt8(const Raw8<float>& a, float* v) {
  const uint32_t u[8] = {a.u[0].x, a.u[0].y, a.u[0].z, a.u[0].w,
                         a.u[1].x, a.u[1].y, a.u[1].z, a.u[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
}
__device__ __forceinline__ void cvt8(const Raw8<__nv_bfloat16>& a, float* v) {
  const uint32_t u[4] = {a.u[0].x, a.u[0].y, a.u[0].z, a.u[0].w};
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

// 8 elements as 4 pairs.
__device__ __forceinline__ void cvt8(const Raw8<float>& a, f32x2* v) {
  float f[8];
  cvt8(a, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack2(f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ void cvt8(const Raw8<__nv_bfloat16>& a, f32x2* v) {
  float f[8];
  cvt8(a, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack2(f[2 * i], f[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ void st8(T* p, const f32x2* v) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack2(v[i], f[2 * i], f[2 * i + 1]);
  st8(p, f);
}

// Sum over the L consecutive lanes (L a power of two) that share a row.
template <int L>
__device__ __forceinline__ float lane_sum(float x) {
#pragma unroll
  for (int m = L / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// n / d and n % d for 0 <= n < 2^31 without a division: with l = ceil(log2 d)
// and m = ceil(2^(31+l) / d), m d - 2^(31+l) < d <= 2^l, so n (m d - 2^(31+l)) <
// 2^(31+l) and floor(n m / 2^(31+l)) is the quotient; m < 2^32.
struct FastDiv {
  uint32_t d, m;
  int s;
  explicit FastDiv(int div) : d((uint32_t)div), s(31) {
    while ((1ull << (s - 31)) < d) ++s;
    m = (uint32_t)(((1ull << s) + d - 1) / d);
  }
  __device__ __forceinline__ void operator()(uint32_t n, uint32_t& q, uint32_t& r) const {
    q = (uint32_t)(((unsigned long long)n * m) >> s);
    r = n - q * d;
  }
};

__device__ __forceinline__ float sigmoidf_(float x) { return 1.f / (1.f + expf(-x)); }
// sigmoid of a value that is stored as T: for bf16 results the hardware's
// approximate exponential and reciprocal (below 2e-6 of the value for |x| <= 10, by
// their published bounds, against bf16's 4e-3) instead of the exact library
// sequences, which cost several times the instructions.
template <typename T>
__device__ __forceinline__ float sigmoid_as(float x) {
  return sigmoidf_(x);
}
template <>
__device__ __forceinline__ float sigmoid_as<__nv_bfloat16>(float x) {
  return __fdividef(1.f, 1.f + __expf(-x));
}
// s = sigmoid(x) = 1 / (1 + e) and t = 1 - s = e s, with e = e^-x. The difference 1 - s
// would lose t where s is near 1 (1 % of it at x = 12, all of it past 17). Where e is
// infinite both are 0: s t and s + x s t vanish there too.
template <typename T>
__device__ __forceinline__ void sigmoid_pair(float x, float& s, float& t) {
  const float e = sizeof(T) == 4 ? expf(-x) : __expf(-x);
  s = sizeof(T) == 4 ? 1.f / (1.f + e) : __fdividef(1.f, 1.f + e);
  t = fminf(e, 3e38f) * s;
}
// log(1 + e^x) without overflow for large x and without cancellation for small
__device__ __forceinline__ float softplusf_(float x) {
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}

// Every kernel of these operators is launched while the stream's previous one may
// still run (a launch takes as long as a small call's work) and begins with
// chain(), which waits until that one has ended and its results are visible. What
// a kernel reads may thus be written while it is already resident, so its inputs
// are not __restrict__: their loads stay ordinary ones, behind the wait. Only a
// backward lets its column sums start early; blocks of a next call that did would
// take the slots that the running call leaves, unevenly over the SMs (93 sequences
// of 6 heads, fp32, 64 x 64: 7.5 us a call; started at the end 5.9, unchained 6.4).
__device__ __forceinline__ void chain() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, int smem, cudaStream_t st,
                   int cluster, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// out[i] = sum over p of part[p][i], i < n, p < np, in a fixed order; column i
// belongs to array i / C of up to three outputs (NULL: dropped).
cudaError_t col_sum(const float* part, int np, int n, int C, float* o0, float* o1, float* o2,
                    cudaStream_t st);

// Most rows, sequences or channels where a thread's next ones are int indices: they lie
// less than this margin past its present ones (at most 4 x 4864 rows).
constexpr int MOST_INDEX = 0x7fffffff - (1 << 16);

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t elem_size(int dtype) { return dtype == GDN_DTYPE_BF16 ? 2 : 4; }
inline bool dtype_ok(int d) { return d == GDN_DTYPE_F32 || d == GDN_DTYPE_BF16; }
// A row access of 16 bytes at a time: pointer and stride.
inline bool vec_rows(const void* p, long long ld, int dtype) {
  return aligned(p, 16) && ld >= 0 && (ld * (long long)elem_size(dtype)) % 16 == 0;
}
inline size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace gdn

// Norms of a Gated DeltaNet layer (include/gdn_layer.h): the gated RMS norm of
// each head's output (gdn_gate_norm_*) and the block boundary, i.e. post-norm,
// residual scale, addition and the next block's norm (gdn_res_norm_*).
#include <stdint.h>

#include <algorithm>

#include "gdn_layer.cuh"

namespace gdn {
namespace {

constexpr int GN_NT = 256;     // threads of a block
constexpr int GN_PARTS = 608;  // most partial sums of dw

// act(z) and its derivative
__device__ __forceinline__ void gate(float z, int act, float& a, float& da) {
  const float s = sigmoidf_(z);
  if (act == GDN_GATE_SILU) {
    a = z * s;
    da = s * (1.f + z * (1.f - s));
  } else {
    a = s;
    da = s * (1.f - s);
  }
}

// L lanes (a power of two >= d / 8) per row of d values.
template <typename T, int L>
__global__ void __launch_bounds__(GN_NT)
    k_gate_norm_fwd(long long nrow, int H, int d, int act, long long ldz, float eps,
                    const T* __restrict__ o, const T* __restrict__ z,
                    const float* __restrict__ w, T* __restrict__ y) {
  const int c = (threadIdx.x % L) * 8;
  const long long r = (long long)blockIdx.x * (GN_NT / L) + threadIdx.x / L;
  const bool live = r < nrow && c < d;
  float x[8] = {}, zz[8] = {}, ss = 0.f;
  if (live) {
    const long long t = r / H;
    ld8(o + (size_t)r * d + c, x);
    ld8(z + (size_t)t * ldz + (size_t)(r - t * H) * d + c, zz);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
  ss = lane_sum<L>(ss);
  if (!live) return;
  const float rr = 1.f / sqrtf(ss / (float)d + eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, da;
    gate(zz[i], act, a, da);
    x[i] = x[i] * rr * w[c + i] * a;
  }
  st8(y + (size_t)r * d + c, x);
}

template <typename T, int L>
__global__ void __launch_bounds__(GN_NT)
    k_gate_norm_bwd(long long nrow, int H, int d, int act, long long ldz, float eps,
                    const T* __restrict__ o, const T* __restrict__ z,
                    const float* __restrict__ w, const T* __restrict__ dy, T* __restrict__ dout,
                    T* __restrict__ dz, float* __restrict__ part) {
  __shared__ float red[GN_NT / L][L * 8];
  const int c = (threadIdx.x % L) * 8, gi = threadIdx.x / L;
  const long long step = (long long)gridDim.x * (GN_NT / L);
  float acc[8] = {}, wv[8] = {};
  if (c < d) ld8(w + c, wv);
  for (long long r0 = (long long)blockIdx.x * (GN_NT / L); r0 < nrow; r0 += step) {
    const long long r = r0 + gi;
    const bool live = r < nrow && c < d;
    float x[8] = {}, zz[8] = {}, gy[8] = {}, ss = 0.f, sd = 0.f, a[8], da[8];
    if (live) {
      const long long t = r / H;
      ld8(o + (size_t)r * d + c, x);
      ld8(z + (size_t)t * ldz + (size_t)(r - t * H) * d + c, zz);
      ld8(dy + (size_t)r * d + c, gy);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      gate(zz[i], act, a[i], da[i]);
      ss = fmaf(x[i], x[i], ss);
      sd = fmaf(gy[i] * a[i] * wv[i], x[i], sd);
    }
    ss = lane_sum<L>(ss);
    sd = lane_sum<L>(sd);
    const float rr = 1.f / sqrtf(ss / (float)d + eps), m = sd * rr / (float)d;
    if (!live) continue;
    float go[8], gz[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = x[i] * rr;
      go[i] = rr * (gy[i] * a[i] * wv[i] - n * m);
      gz[i] = gy[i] * n * wv[i] * da[i];
      acc[i] = fmaf(gy[i] * a[i], n, acc[i]);
    }
    st8(dout + (size_t)r * d + c, go);
    st8(dz + (size_t)r * d + c, gz);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) red[gi][c + i] = acc[i];
  __syncthreads();
  for (int i = threadIdx.x; i < d; i += GN_NT) {
    float a = 0.f;
    for (int u = 0; u < GN_NT / L; ++u) a += red[u][i];
    part[(size_t)blockIdx.x * d + i] = a;
  }
}

// ------------------------------------------------------------ block boundary
constexpr int RN_PARTS = 304;  // most partial sums of dw, dw_post, dscale

// Sums of K values over the block (every thread gets them).
template <int K>
__device__ __forceinline__ void block_sum(float* v, float* sm) {
  const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = lane_sum<32>(v[i]);
  __syncthreads();  // sm may still be read from the sum before
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < K; ++i) sm[warp * K + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < K; ++i) {
    v[i] = 0.f;
    for (int u = 0; u < nw; ++u) v[i] += sm[u * K + i];
  }
}

// One block per row, NC 8-element pieces per thread.
template <typename T, typename R, int NC>
__global__ void __launch_bounds__(512)
    k_res_norm_fwd(int C, float eps, const R* h, const T* __restrict__ x,
                   const float* __restrict__ w, const float* __restrict__ w_post,
                   const float* __restrict__ scale, R* h_out, T* __restrict__ y) {
  __shared__ float sm[16];
  const size_t base = (size_t)blockIdx.x * C;
  float hv[NC][8] = {}, xv[NC][8] = {};
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int c = (n * blockDim.x + threadIdx.x) * 8;
    if (c < C) {
      ld8(h + base + c, hv[n]);
      if (x) ld8(x + base + c, xv[n]);
    }
  }
  if (w_post) {
    float s = 0.f;
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(xv[n][i], xv[n][i], s);
    block_sum<1>(&s, sm);
    const float rx = 1.f / sqrtf(s / (float)C + eps);
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int c = (n * blockDim.x + threadIdx.x) * 8;
      if (c < C)
#pragma unroll
        for (int i = 0; i < 8; ++i) xv[n][i] *= rx * w_post[c + i];
    }
  }
  float s = 0.f;
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int c = (n * blockDim.x + threadIdx.x) * 8;
    if (c < C) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        hv[n][i] = scale ? fmaf(scale[c + i], xv[n][i], hv[n][i]) : hv[n][i] + xv[n][i];
        s = fmaf(hv[n][i], hv[n][i], s);
      }
      if (h_out) st8(h_out + base + c, hv[n]);
    }
  }
  block_sum<1>(&s, sm);
  const float r = 1.f / sqrtf(s / (float)C + eps);
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int c = (n * blockDim.x + threadIdx.x) * 8;
    if (c < C) {
#pragma unroll
      for (int i = 0; i < 8; ++i) hv[n][i] *= r * w[c + i];
      st8(y + base + c, hv[n]);
    }
  }
}

// Each block takes every gridDim.x-th row; its sums of dw, dw_post and dscale
// stay in shared memory, every column owned by one thread.
template <typename T, typename R, int NC>
__global__ void __launch_bounds__(512)
    k_res_norm_bwd(int rows, int C, float eps, const R* __restrict__ h, const T* __restrict__ x,
                   const float* __restrict__ w, const float* __restrict__ w_post,
                   const float* __restrict__ scale, const T* __restrict__ dy, const R* dh_out,
                   R* dh, T* __restrict__ dx, int want, float* __restrict__ part) {
  extern __shared__ float acc[];  // [3][C]
  __shared__ float sm[48];
  const int wpost = want & 1, wscale = want & 2;
  for (int i = threadIdx.x; i < 3 * C; i += blockDim.x) acc[i] = 0.f;
  __syncthreads();
  const float inv = 1.f / (float)C;
  for (int row = blockIdx.x; row < rows; row += gridDim.x) {
    const size_t base = (size_t)row * C;
    float hv[NC][8] = {}, gv[NC][8] = {}, xv[NC][8] = {}, dv[NC][8] = {};
    float s[3] = {};
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int c = (n * blockDim.x + threadIdx.x) * 8;
      if (c < C) {
        ld8(h + base + c, hv[n]);
        ld8(dy + base + c, gv[n]);
        if (wpost || wscale) ld8(x + base + c, xv[n]);
        if (dh_out) ld8(dh_out + base + c, dv[n]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[0] = fmaf(hv[n][i], hv[n][i], s[0]);
          s[1] = fmaf(gv[n][i] * w[c + i], hv[n][i], s[1]);
          s[2] = fmaf(xv[n][i], xv[n][i], s[2]);
        }
      }
    }
    block_sum<3>(s, sm);
    const float r = 1.f / sqrtf(s[0] * inv + eps), m = r * s[1] * inv;
    const float rx = wpost ? 1.f / sqrtf(s[2] * inv + eps) : 1.f;
    float e = 0.f;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int c = (n * blockDim.x + threadIdx.x) * 8;
      if (c < C) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float nn = hv[n][i] * r;
          acc[c + i] += gv[n][i] * nn;
          dv[n][i] += r * (gv[n][i] * w[c + i] - nn * m);  // dh'
          xv[n][i] *= rx;
        }
        st8(dh + base + c, dv[n]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float dp = dv[n][i];
          if (wscale) {
            acc[2 * C + c + i] += dp * (wpost ? xv[n][i] * w_post[c + i] : xv[n][i]);
            dp *= scale[c + i];
          }
          if (wpost) {
            acc[C + c + i] += dp * xv[n][i];
            dp *= w_post[c + i];
            e = fmaf(dp, xv[n][i], e);
          }
          dv[n][i] = dp;
        }
      }
    }
    if (wpost) {
      block_sum<1>(&e, sm);
      e *= inv;
    }
    if (dx) {
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const int c = (n * blockDim.x + threadIdx.x) * 8;
        if (c < C) {
          if (wpost)
#pragma unroll
            for (int i = 0; i < 8; ++i) dv[n][i] = rx * (dv[n][i] - xv[n][i] * e);
          st8(dx + base + c, dv[n]);
        }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 3 * C; i += blockDim.x)
    part[(size_t)blockIdx.x * 3 * C + i] = acc[i];
}

// ------------------------------------------------------------------ host side
gdn_status check_gate(const gdn_gate_norm_shape* s) {
  if (!s || s->rows < 0 || s->H < 1 || s->d < 1 || !(s->eps > 0.f)) return GDN_ERR_INVALID_ARG;
  if (s->act != GDN_GATE_SILU && s->act != GDN_GATE_SIGMOID) return GDN_ERR_INVALID_ARG;
  if (!dtype_ok(s->dtype) || s->d % 8 || s->d > 256 || s->H > (1 << 16))
    return GDN_ERR_UNSUPPORTED;
  if ((long long)s->rows * s->H >= (1ll << 32)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}
int lanes_of(int d) {
  int L = 1;
  while (L * 8 < d) L *= 2;
  return L;
}
int gate_parts(const gdn_gate_norm_shape& s) {
  const long long g = GN_NT / lanes_of(s.d), n = (long long)s.rows * s.H;
  return (int)std::min<long long>(GN_PARTS, (n + g - 1) / g);
}

template <typename T, int L>
void launch_gate(const gdn_gate_norm_shape& s, const void* o, const void* z, const float* w,
                 const void* dy, void* out, void* dz, float* part, cudaStream_t st) {
  const long long n = (long long)s.rows * s.H;
  if (!dy)
    k_gate_norm_fwd<T, L><<<(unsigned)((n + GN_NT / L - 1) / (GN_NT / L)), GN_NT, 0, st>>>(
        n, s.H, s.d, s.act, s.ldz, s.eps, (const T*)o, (const T*)z, w, (T*)out);
  else
    k_gate_norm_bwd<T, L><<<gate_parts(s), GN_NT, 0, st>>>(n, s.H, s.d, s.act, s.ldz, s.eps,
                                                           (const T*)o, (const T*)z, w,
                                                           (const T*)dy, (T*)out, (T*)dz, part);
}
template <typename T>
void dispatch_gate(const gdn_gate_norm_shape& s, const void* o, const void* z, const float* w,
                   const void* dy, void* out, void* dz, float* part, cudaStream_t st) {
  switch (lanes_of(s.d)) {
    case 1: return launch_gate<T, 1>(s, o, z, w, dy, out, dz, part, st);
    case 2: return launch_gate<T, 2>(s, o, z, w, dy, out, dz, part, st);
    case 4: return launch_gate<T, 4>(s, o, z, w, dy, out, dz, part, st);
    case 8: return launch_gate<T, 8>(s, o, z, w, dy, out, dz, part, st);
    case 16: return launch_gate<T, 16>(s, o, z, w, dy, out, dz, part, st);
    default: return launch_gate<T, 32>(s, o, z, w, dy, out, dz, part, st);
  }
}

gdn_status check_res(const gdn_res_norm_shape* s) {
  if (!s || s->rows < 0 || s->C < 1 || !(s->eps > 0.f)) return GDN_ERR_INVALID_ARG;
  if (!dtype_ok(s->dtype) || !dtype_ok(s->res_dtype) || s->C % 8 || s->C > 16384)
    return GDN_ERR_UNSUPPORTED;
  if (s->res_dtype != s->dtype && s->res_dtype != GDN_DTYPE_F32) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}
int res_parts(const gdn_res_norm_shape& s) { return std::min(RN_PARTS, s.rows); }
int res_threads(int C, int nc) { return (C / 8 + 32 * nc - 1) / (32 * nc) * 32; }

struct ResArgs {
  const void *h, *x, *dy, *dh_out;
  const float *w, *w_post, *scale;
  void *ho, *y;  // forward: h_out, y; backward: dh, dx
  float* part;
};
template <typename T, typename R, int NC>
cudaError_t launch_res(const gdn_res_norm_shape& s, const ResArgs& a, cudaStream_t st) {
  const int nt = res_threads(s.C, NC);
  if (!a.dy) {
    k_res_norm_fwd<T, R, NC><<<s.rows, nt, 0, st>>>(s.C, s.eps, (const R*)a.h, (const T*)a.x, a.w,
                                                    a.w_post, a.scale, (R*)a.ho, (T*)a.y);
    return cudaGetLastError();
  }
  const int smem = 3 * s.C * (int)sizeof(float);
  const cudaError_t e = cudaFuncSetAttribute(k_res_norm_bwd<T, R, NC>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e) return e;
  k_res_norm_bwd<T, R, NC><<<res_parts(s), nt, smem, st>>>(
      s.rows, s.C, s.eps, (const R*)a.h, (const T*)a.x, a.w, a.w_post, a.scale, (const T*)a.dy,
      (const R*)a.dh_out, (R*)a.ho, (T*)a.y, (a.w_post ? 1 : 0) | (a.scale ? 2 : 0), a.part);
  return cudaGetLastError();
}
template <typename T, typename R>
cudaError_t dispatch_res(const gdn_res_norm_shape& s, const ResArgs& a, cudaStream_t st) {
  if (s.C <= 4096) return launch_res<T, R, 1>(s, a, st);
  if (s.C <= 8192) return launch_res<T, R, 2>(s, a, st);
  return launch_res<T, R, 4>(s, a, st);
}
cudaError_t run_res(const gdn_res_norm_shape& s, const ResArgs& a, cudaStream_t st) {
  if (s.dtype == GDN_DTYPE_F32) return dispatch_res<float, float>(s, a, st);
  if (s.res_dtype == GDN_DTYPE_F32) return dispatch_res<__nv_bfloat16, float>(s, a, st);
  return dispatch_res<__nv_bfloat16, __nv_bfloat16>(s, a, st);
}

}  // namespace
}  // namespace gdn

extern "C" {

gdn_status gdn_gate_norm_fwd(const gdn_gate_norm_shape* shape, const void* o, const void* z,
                             const float* w, void* y, void* stream) {
  using namespace gdn;
  const gdn_status e = check_gate(shape);
  if (e != GDN_OK) return e;
  const gdn_gate_norm_shape& s = *shape;
  if (!w || (s.rows > 0 && (!o || !z || !y))) return GDN_ERR_INVALID_ARG;
  if (!aligned(o, 16) || !vec_rows(z, s.ldz, s.dtype) || !aligned(w, 16) || !aligned(y, 16))
    return GDN_ERR_INVALID_ARG;
  if (s.rows == 0) return GDN_OK;
  cudaStream_t st = (cudaStream_t)stream;
  prof_mark(st, "gate_norm_fwd");
  if (s.dtype == GDN_DTYPE_BF16)
    dispatch_gate<__nv_bfloat16>(s, o, z, w, nullptr, y, nullptr, nullptr, st);
  else
    dispatch_gate<float>(s, o, z, w, nullptr, y, nullptr, nullptr, st);
  prof_mark(st, nullptr);
  return cudaGetLastError() ? GDN_ERR_CUDA : GDN_OK;
}

size_t gdn_gate_norm_workspace_bytes(const gdn_gate_norm_shape* shape) {
  using namespace gdn;
  if (check_gate(shape) != GDN_OK) return 0;
  return round256((size_t)std::max(gate_parts(*shape), 1) * shape->d * sizeof(float));
}

gdn_status gdn_gate_norm_bwd(const gdn_gate_norm_shape* shape, const void* o, const void* z,
                             const float* w, const void* dy, void* dout, void* dz, float* dw,
                             void* workspace, size_t workspace_bytes, void* stream) {
  using namespace gdn;
  const gdn_status e = check_gate(shape);
  if (e != GDN_OK) return e;
  const gdn_gate_norm_shape& s = *shape;
  if (!w || !dw || (s.rows > 0 && (!o || !z || !dy || !dout || !dz))) return GDN_ERR_INVALID_ARG;
  if (!aligned(o, 16) || !vec_rows(z, s.ldz, s.dtype) || !aligned(w, 16) || !aligned(dy, 16) ||
      !aligned(dout, 16) || !aligned(dz, 16) || !aligned(dw, 4))
    return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < gdn_gate_norm_workspace_bytes(shape))
    return GDN_ERR_WORKSPACE;
  cudaStream_t st = (cudaStream_t)stream;
  float* part = (float*)workspace;
  if (s.rows > 0) {
    prof_mark(st, "gate_norm_bwd");
    if (s.dtype == GDN_DTYPE_BF16)
      dispatch_gate<__nv_bfloat16>(s, o, z, w, dy, dout, dz, part, st);
    else
      dispatch_gate<float>(s, o, z, w, dy, dout, dz, part, st);
    if (cudaGetLastError()) return GDN_ERR_CUDA;
  }
  const cudaError_t ce = col_sum(part, gate_parts(s), s.d, s.d, dw, nullptr, nullptr, st);
  prof_mark(st, nullptr);
  return ce ? GDN_ERR_CUDA : GDN_OK;
}

gdn_status gdn_res_norm_fwd(const gdn_res_norm_shape* shape, const void* h, const void* x,
                            const float* w, const float* w_post, const float* scale, void* h_out,
                            void* y, void* stream) {
  using namespace gdn;
  const gdn_status e = check_res(shape);
  if (e != GDN_OK) return e;
  const gdn_res_norm_shape& s = *shape;
  if (!w || (s.rows > 0 && (!h || !y))) return GDN_ERR_INVALID_ARG;
  if (s.rows > 0 && (x == nullptr) != (h_out == nullptr)) return GDN_ERR_INVALID_ARG;
  if (s.rows > 0 && !x && (w_post || scale)) return GDN_ERR_INVALID_ARG;
  if (!aligned(h, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(w_post, 16) ||
      !aligned(scale, 16) || !aligned(h_out, 16) || !aligned(y, 16))
    return GDN_ERR_INVALID_ARG;
  if (s.rows == 0) return GDN_OK;
  cudaStream_t st = (cudaStream_t)stream;
  prof_mark(st, "res_norm_fwd");
  const ResArgs a = {h, x, nullptr, nullptr, w, w_post, scale, h_out, y, nullptr};
  const cudaError_t ce = run_res(s, a, st);
  prof_mark(st, nullptr);
  return ce ? GDN_ERR_CUDA : GDN_OK;
}

size_t gdn_res_norm_workspace_bytes(const gdn_res_norm_shape* shape) {
  using namespace gdn;
  if (check_res(shape) != GDN_OK) return 0;
  return round256((size_t)std::max(res_parts(*shape), 1) * 3 * shape->C * sizeof(float));
}

gdn_status gdn_res_norm_bwd(const gdn_res_norm_shape* shape, const void* h_out, const void* x,
                            const float* w, const float* w_post, const float* scale,
                            const void* dy, const void* dh_out, void* dh, void* dx, float* dw,
                            float* dw_post, float* dscale, void* workspace,
                            size_t workspace_bytes, void* stream) {
  using namespace gdn;
  const gdn_status e = check_res(shape);
  if (e != GDN_OK) return e;
  const gdn_res_norm_shape& s = *shape;
  if (!w || !dw || (w_post == nullptr) != (dw_post == nullptr) ||
      (scale == nullptr) != (dscale == nullptr))
    return GDN_ERR_INVALID_ARG;
  if (s.rows > 0 && (!h_out || !dy || !dh || ((w_post || scale) && (!x || !dx))))
    return GDN_ERR_INVALID_ARG;
  if (!aligned(h_out, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(w_post, 16) ||
      !aligned(scale, 16) || !aligned(dy, 16) || !aligned(dh_out, 16) || !aligned(dh, 16) ||
      !aligned(dx, 16) || !aligned(dw, 4) || !aligned(dw_post, 4) || !aligned(dscale, 4))
    return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < gdn_res_norm_workspace_bytes(shape))
    return GDN_ERR_WORKSPACE;
  cudaStream_t st = (cudaStream_t)stream;
  float* part = (float*)workspace;
  if (s.rows > 0) {
    prof_mark(st, "res_norm_bwd");
    const ResArgs a = {h_out, x, dy, dh_out, w, w_post, scale, dh, dx, part};
    if (run_res(s, a, st)) return GDN_ERR_CUDA;
  }
  const cudaError_t ce = col_sum(part, res_parts(s), 3 * s.C, s.C, dw, dw_post, dscale, st);
  prof_mark(st, nullptr);
  return ce ? GDN_ERR_CUDA : GDN_OK;
}

}  // extern "C"

// The maps before the recurrence (gdn_prep_fwd / gdn_prep_bwd,
// include/gdn_layer.h): unit-norm q and k written for every value head, the
// log-decay and the write strength; and the fixed-order column sum that the
// layer operators' parameter gradients end with.
#include <stdint.h>

#include <algorithm>

#include "gdn_layer.cuh"

namespace gdn {
namespace {

constexpr int PR_NT = 256;     // threads of a block
constexpr int PR_PARTS = 304;  // most partial sums of drate / dbias

// q / k rows: DK / 8 lanes per (token, q or k, key head). Blocks past
// row_blocks: one thread per (token, value head) of the gates.
template <typename T, int DK>
__global__ void __launch_bounds__(PR_NT)
    k_prep_fwd(int rows, int H, int Hk, int row_blocks, long long ldq, long long ldk,
               long long ldg, long long ldb, float q_scale, float eps, const T* __restrict__ q,
               const T* __restrict__ k, const T* __restrict__ xg, const T* __restrict__ xb,
               const float* __restrict__ rate, const float* __restrict__ bias, T* __restrict__ qn,
               T* __restrict__ kn, T* __restrict__ g, T* __restrict__ beta) {
  if ((int)blockIdx.x >= row_blocks) {
    const long long i = (long long)(blockIdx.x - row_blocks) * PR_NT + threadIdx.x;
    if (i >= (long long)rows * H) return;
    const long long t = i / H;
    const int h = (int)(i - t * H);
    stf(g + i, -expf(rate[h]) * softplusf_(ldf(xg + t * ldg + h) + bias[h]));
    stf(beta + i, sigmoidf_(ldf(xb + t * ldb + h)));
    return;
  }
  constexpr int L = DK / 8;
  const int lane = threadIdx.x % L, G = H / Hk;
  const long long r = (long long)blockIdx.x * (PR_NT / L) + threadIdx.x / L;
  const bool live = r < (long long)rows * 2 * Hk;
  const long long t = live ? r / (2 * Hk) : 0;
  const int j = live ? (int)(r - t * 2 * Hk) : 0, is_k = j >= Hk, hk = j - is_k * Hk;
  float x[8];
  ld8((is_k ? k + t * ldk : q + t * ldq) + (size_t)hk * DK + lane * 8, x);
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
  ss = lane_sum<L>(ss);
  const float s = (is_k ? 1.f : q_scale) / sqrtf(ss + eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= s;
  if (!live) return;
  T* out = (is_k ? kn : qn) + ((size_t)t * H + (size_t)hk * G) * DK + lane * 8;
  for (int i = 0; i < G; ++i) st8(out + (size_t)i * DK, x);
}

template <typename T, int DK>
__global__ void __launch_bounds__(PR_NT)
    k_prep_bwd(int rows, int H, int Hk, long long ldq, long long ldk, float q_scale, float eps,
               const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ dqn,
               const T* __restrict__ dkn, T* __restrict__ dq, T* __restrict__ dk) {
  constexpr int L = DK / 8;
  const int lane = threadIdx.x % L, G = H / Hk;
  const long long r = (long long)blockIdx.x * (PR_NT / L) + threadIdx.x / L;
  const bool live = r < (long long)rows * 2 * Hk;
  const long long t = live ? r / (2 * Hk) : 0;
  const int j = live ? (int)(r - t * 2 * Hk) : 0, is_k = j >= Hk, hk = j - is_k * Hk;
  float x[8], d[8] = {};
  ld8((is_k ? k + t * ldk : q + t * ldq) + (size_t)hk * DK + lane * 8, x);
  const T* dp = (is_k ? dkn : dqn) + ((size_t)t * H + (size_t)hk * G) * DK + lane * 8;
  for (int i = 0; i < G; ++i) {
    float e[8];
    ld8(dp + (size_t)i * DK, e);
#pragma unroll
    for (int u = 0; u < 8; ++u) d[u] += e[u];
  }
  float ss = 0.f, xd = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    ss = fmaf(x[i], x[i], ss);
    xd = fmaf(x[i], d[i], xd);
  }
  ss = lane_sum<L>(ss);
  xd = lane_sum<L>(xd);
  const float rr = 1.f / sqrtf(ss + eps), c = (is_k ? 1.f : q_scale) * rr, m = rr * rr * xd;
#pragma unroll
  for (int i = 0; i < 8; ++i) d[i] = c * (d[i] - x[i] * m);
  if (live) st8((is_k ? dk : dq) + ((size_t)t * Hk + hk) * DK + lane * 8, d);
}

// Gates: block = a run of tokens, 32 heads at a time (lane = head, 8 tokens in
// parallel); part[block] = its sums of drate [H] and dbias [H].
template <typename T>
__global__ void __launch_bounds__(PR_NT)
    k_prep_bwd_gates(int rows, int H, int per, long long ldg, long long ldb,
                     const T* __restrict__ xg, const T* __restrict__ xb,
                     const float* __restrict__ rate, const float* __restrict__ bias,
                     const T* __restrict__ dg, const T* __restrict__ dbeta, T* __restrict__ dxg,
                     T* __restrict__ dxb, float* __restrict__ part) {
  __shared__ float red[2][8][32];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const long long t0 = (long long)blockIdx.x * per, t1 = min(t0 + per, (long long)rows);
  for (int h0 = 0; h0 < H; h0 += 32) {
    const int h = h0 + tx;
    float sr = 0.f, sb = 0.f;
    if (h < H) {
      const float er = expf(rate[h]), bi = bias[h];
      for (long long t = t0 + ty; t < t1; t += 8) {
        const float x = ldf(xg + t * ldg + h) + bi, d = ldf(dg + t * H + h);
        const float dx = -d * er * sigmoidf_(x);
        sr = fmaf(d, -er * softplusf_(x), sr);
        sb += dx;
        stf(dxg + t * H + h, dx);
        const float b = sigmoidf_(ldf(xb + t * ldb + h));
        stf(dxb + t * H + h, ldf(dbeta + t * H + h) * b * (1.f - b));
      }
    }
    red[0][ty][tx] = sr;
    red[1][ty][tx] = sb;
    __syncthreads();
    if (ty < 2 && h < H) {
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) a += red[ty][i][tx];
      part[((size_t)blockIdx.x * 2 + ty) * H + h] = a;
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(256)
    k_col_sum(const float* __restrict__ part, int np, int n, int C, float* o0, float* o1,
              float* o2) {
  __shared__ float red[8][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, i = blockIdx.x * 32 + tx;
  float a = 0.f;
  if (i < n)
    for (int p = ty; p < np; p += 8) a += part[(size_t)p * n + i];
  red[ty][tx] = a;
  __syncthreads();
  if (ty || i >= n) return;
  a = 0.f;
#pragma unroll
  for (int u = 0; u < 8; ++u) a += red[u][tx];
  float* o = i < C ? o0 : i < 2 * C ? o1 : o2;
  if (o) o[i % C] = a;
}

int prep_parts(int rows) { return std::min(PR_PARTS, (rows + 31) / 32); }

gdn_status check_prep(const gdn_prep_shape* s) {
  if (!s || s->rows < 0 || s->H < 1 || s->Hk < 1 || s->H % s->Hk || !(s->eps > 0.f) ||
      s->ldg < 0 || s->ldb < 0)
    return GDN_ERR_INVALID_ARG;
  if (!dtype_ok(s->dtype) || (s->dk != 64 && s->dk != 128) || s->H > (1 << 16))
    return GDN_ERR_UNSUPPORTED;
  if ((long long)s->rows * s->H >= (1ll << 33)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

long long row_blocks_of(const gdn_prep_shape& s) {
  const int groups = PR_NT / (s.dk / 8);
  return ((long long)s.rows * 2 * s.Hk + groups - 1) / groups;
}

template <typename T, int DK>
void launch_prep_fwd(const gdn_prep_shape& s, const void* q, const void* k, const void* xg,
                     const void* xb, const float* rate, const float* bias, void* qn, void* kn,
                     void* g, void* beta, cudaStream_t st) {
  const long long rb = row_blocks_of(s);
  const long long gb = ((long long)s.rows * s.H + PR_NT - 1) / PR_NT;
  k_prep_fwd<T, DK><<<(unsigned)(rb + gb), PR_NT, 0, st>>>(
      s.rows, s.H, s.Hk, (int)rb, s.ldq, s.ldk, s.ldg, s.ldb, s.q_scale, s.eps, (const T*)q,
      (const T*)k, (const T*)xg, (const T*)xb, rate, bias, (T*)qn, (T*)kn, (T*)g, (T*)beta);
}

template <typename T, int DK>
void launch_prep_bwd(const gdn_prep_shape& s, const void* q, const void* k, const void* xg,
                     const void* xb, const float* rate, const float* bias, const void* dqn,
                     const void* dkn, const void* dg, const void* dbeta, void* dq, void* dk,
                     void* dxg, void* dxb, float* part, cudaStream_t st) {
  k_prep_bwd<T, DK><<<(unsigned)row_blocks_of(s), PR_NT, 0, st>>>(
      s.rows, s.H, s.Hk, s.ldq, s.ldk, s.q_scale, s.eps, (const T*)q, (const T*)k, (const T*)dqn,
      (const T*)dkn, (T*)dq, (T*)dk);
  const int np = prep_parts(s.rows);
  k_prep_bwd_gates<T><<<np, PR_NT, 0, st>>>(s.rows, s.H, (s.rows + np - 1) / np, s.ldg, s.ldb,
                                            (const T*)xg, (const T*)xb, rate, bias, (const T*)dg,
                                            (const T*)dbeta, (T*)dxg, (T*)dxb, part);
}

}  // namespace

cudaError_t col_sum(const float* part, int np, int n, int C, float* o0, float* o1, float* o2,
                    cudaStream_t st) {
  prof_mark(st, "layer_col_sum");
  k_col_sum<<<(n + 31) / 32, 256, 0, st>>>(part, np, n, C, o0, o1, o2);
  return cudaGetLastError();
}

}  // namespace gdn

extern "C" {

gdn_status gdn_prep_fwd(const gdn_prep_shape* shape, const void* q, const void* k, const void* xg,
                        const void* xb, const float* rate, const float* bias, void* qn, void* kn,
                        void* g, void* beta, void* stream) {
  using namespace gdn;
  const gdn_status e = check_prep(shape);
  if (e != GDN_OK) return e;
  const gdn_prep_shape& s = *shape;
  if (!rate || !bias) return GDN_ERR_INVALID_ARG;
  if (s.rows > 0 && (!q || !k || !xg || !xb || !qn || !kn || !g || !beta))
    return GDN_ERR_INVALID_ARG;
  const size_t es = elem_size(s.dtype);
  if (!vec_rows(q, s.ldq, s.dtype) || !vec_rows(k, s.ldk, s.dtype) || !aligned(xg, es) ||
      !aligned(xb, es) || !aligned(rate, 4) || !aligned(bias, 4) || !aligned(qn, 16) ||
      !aligned(kn, 16) || !aligned(g, 16) || !aligned(beta, 16))
    return GDN_ERR_INVALID_ARG;
  if (s.rows == 0) return GDN_OK;
  cudaStream_t st = (cudaStream_t)stream;
  prof_mark(st, "prep_fwd");
  if (s.dtype == GDN_DTYPE_BF16) {
    if (s.dk == 64)
      launch_prep_fwd<__nv_bfloat16, 64>(s, q, k, xg, xb, rate, bias, qn, kn, g, beta, st);
    else
      launch_prep_fwd<__nv_bfloat16, 128>(s, q, k, xg, xb, rate, bias, qn, kn, g, beta, st);
  } else {
    if (s.dk == 64)
      launch_prep_fwd<float, 64>(s, q, k, xg, xb, rate, bias, qn, kn, g, beta, st);
    else
      launch_prep_fwd<float, 128>(s, q, k, xg, xb, rate, bias, qn, kn, g, beta, st);
  }
  prof_mark(st, nullptr);
  return cudaGetLastError() ? GDN_ERR_CUDA : GDN_OK;
}

size_t gdn_prep_workspace_bytes(const gdn_prep_shape* shape) {
  using namespace gdn;
  if (check_prep(shape) != GDN_OK) return 0;
  return round256((size_t)std::max(prep_parts(shape->rows), 1) * 2 * shape->H * sizeof(float));
}

gdn_status gdn_prep_bwd(const gdn_prep_shape* shape, const void* q, const void* k, const void* xg,
                        const void* xb, const float* rate, const float* bias, const void* dqn,
                        const void* dkn, const void* dg, const void* dbeta, void* dq, void* dk,
                        void* dxg, void* dxb, float* drate, float* dbias, void* workspace,
                        size_t workspace_bytes, void* stream) {
  using namespace gdn;
  const gdn_status e = check_prep(shape);
  if (e != GDN_OK) return e;
  const gdn_prep_shape& s = *shape;
  if (!rate || !bias || !drate || !dbias) return GDN_ERR_INVALID_ARG;
  if (s.rows > 0 && (!q || !k || !xg || !xb || !dqn || !dkn || !dg || !dbeta || !dq || !dk ||
                     !dxg || !dxb))
    return GDN_ERR_INVALID_ARG;
  const size_t es = elem_size(s.dtype);
  if (!vec_rows(q, s.ldq, s.dtype) || !vec_rows(k, s.ldk, s.dtype) || !aligned(xg, es) ||
      !aligned(xb, es) || !aligned(rate, 4) || !aligned(bias, 4) || !aligned(dqn, 16) ||
      !aligned(dkn, 16) || !aligned(dg, 16) || !aligned(dbeta, 16) || !aligned(dq, 16) ||
      !aligned(dk, 16) || !aligned(dxg, 16) || !aligned(dxb, 16) || !aligned(drate, 4) ||
      !aligned(dbias, 4))
    return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < gdn_prep_workspace_bytes(shape))
    return GDN_ERR_WORKSPACE;
  cudaStream_t st = (cudaStream_t)stream;
  float* part = (float*)workspace;
  if (s.rows > 0) {
    prof_mark(st, "prep_bwd");
    if (s.dtype == GDN_DTYPE_BF16) {
      if (s.dk == 64)
        launch_prep_bwd<__nv_bfloat16, 64>(s, q, k, xg, xb, rate, bias, dqn, dkn, dg, dbeta, dq,
                                           dk, dxg, dxb, part, st);
      else
        launch_prep_bwd<__nv_bfloat16, 128>(s, q, k, xg, xb, rate, bias, dqn, dkn, dg, dbeta, dq,
                                            dk, dxg, dxb, part, st);
    } else {
      if (s.dk == 64)
        launch_prep_bwd<float, 64>(s, q, k, xg, xb, rate, bias, dqn, dkn, dg, dbeta, dq, dk, dxg,
                                   dxb, part, st);
      else
        launch_prep_bwd<float, 128>(s, q, k, xg, xb, rate, bias, dqn, dkn, dg, dbeta, dq, dk, dxg,
                                    dxb, part, st);
    }
    if (cudaGetLastError()) return GDN_ERR_CUDA;
  }
  const cudaError_t ce =
      col_sum(part, prep_parts(s.rows), 2 * s.H, s.H, drate, dbias, nullptr, st);
  prof_mark(st, nullptr);
  return ce ? GDN_ERR_CUDA : GDN_OK;
}

}  // extern "C"

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
constexpr int PR_U = 3;        // rows a thread has in flight (forward)
// Rows a thread has in flight (backward): fewer where a row has several gradients.
// (32768 x 16 heads of 128 bf16: 1 row 132 us, 2 rows 117, 4 rows 125.)
constexpr int prep_bwd_rows(bool shared) { return shared ? 1 : 2; }
constexpr int PR_G = 4;        // value heads' gradients loaded together (backward)
constexpr int PR_PARTS = 152;  // most partial sums of drate / dbias

// Row r of the 2 Hk (q heads, then k heads) rows of each token.
struct HeadRow {
  uint32_t t;
  int hk;
  bool is_k;
};
__device__ __forceinline__ HeadRow head_row(uint32_t r, const FastDiv& by2Hk, int Hk) {
  HeadRow h;
  uint32_t j;
  by2Hk(r, h.t, j);
  h.is_k = (int)j >= Hk;
  h.hk = (int)j - (h.is_k ? Hk : 0);
  return h;
}

// q / k rows: x r with r = 1 / sqrt(sum x^2 + eps), DK / 8 lanes per row, PR_U
// rows per thread, all loaded before the first is used. Blocks past row_blocks: one
// thread per (token, value head) of the gates. Bound by the bytes of q, k, qn and
// kn: 32768 tokens of 16 heads of 128 bf16 values 83 us (541 MB, 6.5 TB/s; with 1,
// 2 and 4 rows in flight 98, 90 and 84).
template <typename T, int DK>
__global__ void __launch_bounds__(PR_NT)
    k_prep_fwd(uint32_t nrow, uint32_t ngate, FastDiv by2Hk, FastDiv byH, int G, int row_blocks,
               long long ldq, long long ldk, long long ldg, long long ldb, float q_scale,
               float eps, const T* q, const T* k, const T* xg, const T* xb, const float* rate,
               const float* bias, T* qn, T* kn, T* g, T* beta) {
  chain();
  const int H = (int)byH.d, Hk = (int)by2Hk.d / 2;
  if ((int)blockIdx.x >= row_blocks) {
    const uint32_t i = (blockIdx.x - row_blocks) * PR_NT + threadIdx.x;
    if (i >= ngate) return;
    uint32_t t, h;
    byH(i, t, h);
    stf(g + i, -expf(rate[h]) * softplusf_(ldf(xg + (size_t)t * ldg + h) + bias[h]));
    stf(beta + i, sigmoidf_(ldf(xb + (size_t)t * ldb + h)));
    return;
  }
  constexpr int L = DK / 8, NG = PR_NT / L;
  const int c = threadIdx.x % L * 8;
  const uint32_t r0 = blockIdx.x * (NG * PR_U) + threadIdx.x / L;
  Raw8<T> raw[PR_U];
#pragma unroll
  for (int u = 0; u < PR_U; ++u) {
    const uint32_t r = r0 + u * NG;
    raw[u] = Raw8<T>{};
    if (r < nrow) {
      const HeadRow h = head_row(r, by2Hk, Hk);
      raw[u] = ldraw8((h.is_k ? k + h.t * ldk : q + h.t * ldq) + (size_t)h.hk * DK + c);
    }
  }
#pragma unroll
  for (int u = 0; u < PR_U; ++u) {
    const uint32_t r = r0 + u * NG;
    float x[8], ss = 0.f;
    cvt8(raw[u], x);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    ss = lane_sum<L>(ss);
    if (r >= nrow) continue;
    const HeadRow h = head_row(r, by2Hk, Hk);
    const float s = (h.is_k ? 1.f : q_scale) * rsqrtf(ss + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= s;
    T* out = (h.is_k ? kn : qn) + ((size_t)h.t * H + (size_t)h.hk * G) * DK + c;
    for (int i = 0; i < G; ++i) st8(out + (size_t)i * DK, x);
  }
}

// The gates of a run of tokens, HP heads (a power of two <= 32) at a time, the
// block's other thread dimension over tokens; part[block] = its sums of
// drate [H] and dbias [H].
template <typename T>
__device__ __forceinline__ void prep_bwd_gates(int blk, int rows, int H, int hp_log, int per,
                                               long long ldg, long long ldb, const T* xg,
                                               const T* xb, const float* rate, const float* bias,
                                               const T* dg, const T* dbeta, T* dxg, T* dxb,
                                               float* part) {
  __shared__ float red[2][PR_NT];
  const int hp = 1 << hp_log, tx = threadIdx.x & (hp - 1), ty = threadIdx.x >> hp_log;
  const int ny = PR_NT >> hp_log;
  const int t0 = blk * per, t1 = min(t0 + per, rows);
  for (int h0 = 0; h0 < H; h0 += hp) {
    const int h = h0 + tx;
    float sr = 0.f, sb = 0.f;
    if (h < H) {
      const float er = expf(rate[h]), bi = bias[h];
      for (int t = t0 + ty; t < t1; t += ny) {
        const size_t at = (size_t)t * H + h;
        const float x = ldf(xg + (size_t)t * ldg + h) + bi, d = ldf(dg + at);
        const float db = ldf(dbeta + at);
        float b, nb;  // sigmoid and 1 - sigmoid
        sigmoid_pair<float>(ldf(xb + (size_t)t * ldb + h), b, nb);
        const float dx = -d * er * sigmoidf_(x);
        sr = fmaf(d, -er * softplusf_(x), sr);
        sb += dx;
        stf(dxg + at, dx);
        stf(dxb + at, db * b * nb);
      }
    }
    red[0][threadIdx.x] = sr;
    red[1][threadIdx.x] = sb;
    __syncthreads();
    if (ty < 2 && h < H) {
      float a = 0.f;
      for (int i = 0; i < ny; ++i) a += red[ty][(i << hp_log) + tx];
      part[((size_t)blk * 2 + ty) * H + h] = a;
    }
    __syncthreads();
  }
}

// With d the sum of a key head's G gradients and r as in k_prep_fwd,
//   dx = r (d - r^2 (x . d) x)   (times q_scale for q).
// The first gate_blocks blocks take the gates (their loops over tokens are the
// longest), the others rows as k_prep_fwd. Bound by the bytes of q, k and the
// gradients: 32768 tokens of 16 heads of 128 bf16 values 117 us (812 MB, 6.9 TB/s);
// 8193 of 24 value on 8 key heads, of 128, 31 us (170 MB, 5.5 TB/s: a sixth of it
// is the column sums and the launches).
template <typename T, int DK, bool SHARED>
__global__ void __launch_bounds__(PR_NT)
    k_prep_bwd(uint32_t nrow, FastDiv by2Hk, int G, int gate_blocks, int rows, int H, int hp_log,
               int per, long long ldq, long long ldk, long long ldg, long long ldb, float q_scale,
               float eps, const T* q, const T* k, const T* xg, const T* xb, const float* rate,
               const float* bias, const T* dqn, const T* dkn, const T* dg, const T* dbeta, T* dq,
               T* dk, T* dxg, T* dxb, float* part) {
  chain();
  let_next_start();
  if ((int)blockIdx.x < gate_blocks) {
    prep_bwd_gates<T>(blockIdx.x, rows, H, hp_log, per, ldg, ldb, xg, xb, rate, bias, dg, dbeta,
                      dxg, dxb, part);
    return;
  }
  constexpr int L = DK / 8, NG = PR_NT / L, PR_UB = prep_bwd_rows(SHARED), GL = SHARED ? PR_G : 1;
  const int c = threadIdx.x % L * 8, Hk = (int)by2Hk.d / 2;
  const uint32_t r0 = (blockIdx.x - gate_blocks) * (NG * PR_UB) + threadIdx.x / L;
  float d[PR_UB][8] = {};
  Raw8<T> xr[PR_UB];
  const T* src[PR_UB];
#pragma unroll
  for (int u = 0; u < PR_UB; ++u) {
    const uint32_t r = r0 + u * NG;
    xr[u] = Raw8<T>{};
    src[u] = nullptr;
    if (r < nrow) {
      const HeadRow h = head_row(r, by2Hk, Hk);
      xr[u] = ldraw8((h.is_k ? k + h.t * ldk : q + h.t * ldq) + (size_t)h.hk * DK + c);
      src[u] = (h.is_k ? dkn : dqn) + ((size_t)h.t * H + (size_t)h.hk * G) * DK + c;
    }
  }
  for (int i0 = 0; i0 < (SHARED ? G : 1); i0 += GL) {
    Raw8<T> e[PR_UB][GL];
#pragma unroll
    for (int u = 0; u < PR_UB; ++u)
#pragma unroll
      for (int i = 0; i < GL; ++i) {
        e[u][i] = Raw8<T>{};
        if (src[u] && (!SHARED || i0 + i < G)) e[u][i] = ldraw8(src[u] + (size_t)(i0 + i) * DK);
      }
#pragma unroll
    for (int u = 0; u < PR_UB; ++u)
#pragma unroll
      for (int i = 0; i < GL; ++i) {
        if (SHARED && i0 + i >= G) break;
        float v[8];
        cvt8(e[u][i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[u][j] += v[j];
      }
  }
#pragma unroll
  for (int u = 0; u < PR_UB; ++u) {
    const uint32_t r = r0 + u * NG;
    float x[8], ss = 0.f, xd = 0.f;
    cvt8(xr[u], x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ss = fmaf(x[i], x[i], ss);
      xd = fmaf(x[i], d[u][i], xd);
    }
    ss = lane_sum<L>(ss);
    xd = lane_sum<L>(xd);
    if (r >= nrow) continue;
    const HeadRow h = head_row(r, by2Hk, Hk);
    const float rr = rsqrtf(ss + eps), s = (h.is_k ? 1.f : q_scale) * rr, m = rr * (rr * xd);
#pragma unroll
    for (int i = 0; i < 8; ++i) d[u][i] = s * fmaf(-x[i], m, d[u][i]);
    st8((h.is_k ? dk : dq) + ((size_t)h.t * Hk + h.hk) * DK + c, d[u]);
  }
}

// Block: 32 columns, 32 partials at a time; then warp j adds up column j.
__global__ void __launch_bounds__(1024)
    k_col_sum(const float* part, int np, int n, int C, float* o0, float* o1,
              float* o2) {
  __shared__ float red[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, i0 = blockIdx.x * 32;
  chain();
  float a = 0.f;
  if (i0 + tx < n) {
#pragma unroll 4
    for (int p = ty; p < np; p += 32) a += part[(size_t)p * n + i0 + tx];
  }
  red[ty][tx] = a;
  __syncthreads();
  a = lane_sum<32>(red[tx][ty]);
  const int i = i0 + ty;
  if (tx || i >= n) return;
  float* o = i < C ? o0 : i < 2 * C ? o1 : o2;
  if (o) o[i % C] = a;
}

int prep_parts(int rows) { return std::min(PR_PARTS, (rows + 15) / 16); }

gdn_status check_prep(const gdn_prep_shape* s) {
  if (!s || s->rows < 0 || s->H < 1 || s->Hk < 1 || s->H % s->Hk || !(s->eps > 0.f) ||
      s->ldg < 0 || s->ldb < 0)
    return GDN_ERR_INVALID_ARG;
  if (!dtype_ok(s->dtype) || (s->dk != 64 && s->dk != 128) || s->H > (1 << 16))
    return GDN_ERR_UNSUPPORTED;
  if ((long long)s->rows * 2 * s->H >= (1ll << 31)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

template <typename T, int DK>
void launch_prep_fwd(const gdn_prep_shape& s, const void* q, const void* k, const void* xg,
                     const void* xb, const float* rate, const float* bias, void* qn, void* kn,
                     void* g, void* beta, cudaStream_t st) {
  const uint32_t nrow = (uint32_t)s.rows * 2 * s.Hk, ngate = (uint32_t)s.rows * s.H;
  const uint32_t per = PR_NT / (DK / 8) * PR_U, rb = (nrow + per - 1) / per;
  launch(k_prep_fwd<T, DK>, dim3(rb + (ngate + PR_NT - 1) / PR_NT), dim3(PR_NT), 0, st, 1, nrow,
         ngate, FastDiv(2 * s.Hk), FastDiv(s.H), s.H / s.Hk, (int)rb, s.ldq, s.ldk, s.ldg, s.ldb,
         s.q_scale, s.eps, (const T*)q, (const T*)k, (const T*)xg, (const T*)xb, rate, bias, (T*)qn,
         (T*)kn, (T*)g, (T*)beta);
}

template <typename T, int DK>
void launch_prep_bwd(const gdn_prep_shape& s, const void* q, const void* k, const void* xg,
                     const void* xb, const float* rate, const float* bias, const void* dqn,
                     const void* dkn, const void* dg, const void* dbeta, void* dq, void* dk,
                     void* dxg, void* dxb, float* part, cudaStream_t st) {
  const uint32_t nrow = (uint32_t)s.rows * 2 * s.Hk;
  const bool shared = s.H > s.Hk;
  const uint32_t per = PR_NT / (DK / 8) * prep_bwd_rows(shared), rb = (nrow + per - 1) / per;
  const int np = prep_parts(s.rows);
  int hp_log = 0;
  while ((1 << hp_log) < s.H && hp_log < 5) ++hp_log;
  const auto kernel = shared ? k_prep_bwd<T, DK, true> : k_prep_bwd<T, DK, false>;
  launch(kernel, dim3(np + rb), dim3(PR_NT), 0, st, 1, nrow, FastDiv(2 * s.Hk), s.H / s.Hk, np,
         s.rows, s.H, hp_log, (s.rows + np - 1) / np, s.ldq, s.ldk, s.ldg, s.ldb, s.q_scale, s.eps,
         (const T*)q, (const T*)k, (const T*)xg, (const T*)xb, rate, bias, (const T*)dqn,
         (const T*)dkn, (const T*)dg, (const T*)dbeta, (T*)dq, (T*)dk, (T*)dxg, (T*)dxb, part);
}

}  // namespace

cudaError_t col_sum(const float* part, int np, int n, int C, float* o0, float* o1, float* o2,
                    cudaStream_t st) {
  prof_mark(st, "layer_col_sum");
  return launch(k_col_sum, dim3((n + 31) / 32), dim3(1024), 0, st, 1, part, np, n, C, o0, o1, o2);
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

// Norms of query and key heads with the rotation by the token's position
// (gdn_qk_norm_fwd / gdn_qk_norm_bwd, include/gdn_layer.h).
#include <stdint.h>

#include <algorithm>

#include "gdn_layer.cuh"

namespace gdn {
namespace {

constexpr int QN_NT = 256;     // threads of a block
constexpr int QN_U = 4;        // head rows a thread has in flight (forward)
constexpr int QN_UB = 2;       // and backward (with their gradients)
constexpr int QN_HEADS = 16;   // most heads that share one set of sines and cosines
constexpr int QN_PARTS = 608;  // most blocks of the backward: partial sums of dw

// f / (2 pi) as a fraction of a turn in units of 2^-64, for |f| < 2^40. With f =
// m 2^e (m < 2^53) and C = floor(2^66 / (2 pi)), it is m C 2^(e - 2) up to one unit:
// whole-number products only, so that pos times it, modulo 2^64, is the angle's
// fraction of a turn to 2^-33 for any 32-bit position.
__device__ __forceinline__ unsigned long long turn_step(double f) {
  constexpr unsigned long long C = 0xA2F9836E4E441529ull;  // 2^66 / (2 pi) = 2^65 / pi
  const unsigned long long u = (unsigned long long)__double_as_longlong(f);
  const int ex = (int)(u >> 52) & 0x7ff;
  const unsigned long long m = (u & 0xfffffffffffffull) | (ex ? 1ull << 52 : 0);
  const int s = 2 + 1075 - max(ex, 1);  // right shift of the 128-bit product
  const unsigned long long lo = m * C, hi = __umul64hi(m, C);
  unsigned long long r = 0;
  if (s <= 0)
    r = lo << min(-s, 63);
  else if (s < 64)
    r = (hi << (64 - s)) | (lo >> s);
  else if (s < 128)
    r = hi >> (s - 64);
  return (u >> 63) ? 0ull - r : r;
}

struct QkArgs {
  int Hq, Hk, per, rq, rk;  // heads, heads of an item, repeats of an output head
  int r2;                   // rot / 2
  long long ldq, ldk;
  float q_scale, eps;
};

// The 8 values of a lane and what turns them: y = x cs + (its partner) sn.
struct Turn {
  float cs[8], sn[8];
};

// The steps of this lane's values (pairs: of its 4 pairs, each twice).
template <bool PAIRS>
__device__ __forceinline__ void turn_steps(const double* inv_freq, int r2, int e0,
                                           unsigned long long* st) {
#pragma unroll
  for (int i = 0; i < 8; ++i) st[i] = 0;
  if (e0 >= 2 * r2) return;
  if (PAIRS) {
#pragma unroll
    for (int i = 0; i < 4; ++i) st[i] = turn_step(inv_freq[e0 / 2 + i]);
  } else {
    const int f0 = e0 < r2 ? e0 : e0 - r2;
#pragma unroll
    for (int i = 0; i < 8; ++i) st[i] = turn_step(inv_freq[f0 + i]);
  }
}
// Sines and cosines at a position; `back`: of the opposite angle.
template <bool PAIRS>
__device__ __forceinline__ void turn_at(const unsigned long long* st, int pos, bool first, bool back,
                                        Turn& t) {
  const unsigned long long p = (unsigned long long)(long long)pos;
#pragma unroll
  for (int i = 0; i < (PAIRS ? 4 : 8); ++i) {
    const int ph = (int)((p * st[i]) >> 32);  // [-1/2, 1/2) of a turn
    float s, c;
    sincospif((float)ph * 0x1p-31f, &s, &c);
    if (back) s = -s;
    if (PAIRS) {
      t.cs[2 * i] = t.cs[2 * i + 1] = c;
      t.sn[2 * i] = -s;
      t.sn[2 * i + 1] = s;
    } else {
      t.cs[i] = c;
      t.sn[i] = first ? -s : s;
    }
  }
}
// Every lane of the warp takes part: `partner` is the lane with the other halves
// of this one's pairs (itself where nothing is turned).
template <bool PAIRS>
__device__ __forceinline__ void turn(const Turn& t, int partner, float* x) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = PAIRS ? x[i ^ 1] : __shfl_sync(0xffffffffu, x[i], partner);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], t.cs[i], y[i] * t.sn[i]);
}

// D / 8 lanes hold a head's row, 8 values each, and take `per` heads of one token
// (queries first, then keys), whose sines and cosines they form once; QN_U rows are
// in flight. Items (token, heads) are spread over the grid.
template <typename T, int D, bool PAIRS>
__global__ void __launch_bounds__(QN_NT)
    k_qk_norm_fwd(uint32_t items, FastDiv byParts, FastDiv byT, QkArgs p, const T* q, const T* k,
                  const float* wq, const float* wk, const double* inv_freq, const int* pos, T* qn,
                  T* kn) {
  chain();
  constexpr int L = D / 8, NG = QN_NT / L;
  const int ln = threadIdx.x % L, e0 = 8 * ln, lane = threadIdx.x & 31;
  const bool turned = e0 < 2 * p.r2, first = e0 < p.r2;
  const int partner = PAIRS || !turned ? lane : first ? lane + p.r2 / 8 : lane - p.r2 / 8;
  unsigned long long st[8];
  turn_steps<PAIRS>(inv_freq, p.r2, e0, st);
  float w[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[0][i] = w[1][i] = 1.f;
  if (wq) ld8(wq + e0, w[0]);
  if (wk) ld8(wk + e0, w[1]);
#pragma unroll
  for (int i = 0; i < 8; ++i) w[0][i] *= p.q_scale;
  const int Ht = p.Hq + p.Hk;
  // the same trips for every lane of a warp
  for (uint32_t i0 = blockIdx.x * NG; i0 < items; i0 += gridDim.x * NG) {
    const uint32_t it = i0 + threadIdx.x / L;
    const bool on = it < items;
    uint32_t tok = 0, part = 0;
    if (on) byParts(it, tok, part);
    Turn tn;
    if (p.r2) {
      uint32_t seq, at;
      byT(tok, seq, at);
      turn_at<PAIRS>(st, on && pos ? pos[tok] : (int)at, first, false, tn);
    }
    if (!turned) {
#pragma unroll
      for (int i = 0; i < 8; ++i) tn.cs[i] = 1.f, tn.sn[i] = 0.f;
    }
    const int h1 = on ? min((int)(part + 1) * p.per, Ht) : 0;
    for (int hb = 0; hb < p.per; hb += QN_U) {
      Raw8<T> raw[QN_U];
#pragma unroll
      for (int u = 0; u < QN_U; ++u) {
        const int h = (int)part * p.per + hb + u;
        raw[u] = Raw8<T>{};
        if (hb + u < p.per && h < h1)
          raw[u] = ldraw8((h < p.Hq ? q + (size_t)tok * p.ldq + (size_t)h * D
                                    : k + (size_t)tok * p.ldk + (size_t)(h - p.Hq) * D) +
                          e0);
      }
#pragma unroll
      for (int u = 0; u < QN_U; ++u) {
        const int h = (int)part * p.per + hb + u;
        const bool is_k = h >= p.Hq;
        float x[8], ss = 0.f;
        cvt8(raw[u], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
        const float r = rsqrtf(fmaf(lane_sum<L>(ss), 1.f / D, p.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= r * (is_k ? w[1][i] : w[0][i]);
        if (p.r2) turn<PAIRS>(tn, partner, x);
        if (hb + u >= p.per || h >= h1) continue;
        const int rep = is_k ? p.rk : p.rq, hh = is_k ? h - p.Hq : h;
        const int Ho = is_k ? p.Hk * p.rk : p.Hq * p.rq;
        T* out = (is_k ? kn : qn) + ((size_t)tok * Ho + (size_t)hh * rep) * D + e0;
        for (int i = 0; i < rep; ++i) st8(out + (size_t)i * D, x);
      }
    }
  }
}

// With d the sum of a head's repeated gradients turned back (and times q_scale),
// n = x r, e = d w:   dx = r (e - n mean(e n)),   dw += d n.
// Lanes and items as forward; a thread sums its 8 columns of dwq and dwk over all of
// its rows, the block's lane groups join theirs in order, and part[block] = [dwq, dwk].
template <typename T, int D, bool PAIRS>
__global__ void __launch_bounds__(QN_NT)
    k_qk_norm_bwd(uint32_t items, FastDiv byParts, FastDiv byT, QkArgs p, const T* q, const T* k,
                  const float* wq, const float* wk, const double* inv_freq, const int* pos,
                  const T* dqn, const T* dkn, T* dq, T* dk, float* part_out) {
  chain();
  let_next_start();
  constexpr int L = D / 8, NG = QN_NT / L;
  __shared__ float red[NG][D];
  const int ln = threadIdx.x % L, e0 = 8 * ln, lane = threadIdx.x & 31;
  const bool turned = e0 < 2 * p.r2, first = e0 < p.r2;
  const int partner = PAIRS || !turned ? lane : first ? lane + p.r2 / 8 : lane - p.r2 / 8;
  unsigned long long st[8];
  turn_steps<PAIRS>(inv_freq, p.r2, e0, st);
  float w[2][8], dw[2][8] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[0][i] = w[1][i] = 1.f;
  if (wq) ld8(wq + e0, w[0]);
  if (wk) ld8(wk + e0, w[1]);
  const int Ht = p.Hq + p.Hk;
  for (uint32_t i0 = blockIdx.x * NG; i0 < items; i0 += gridDim.x * NG) {
    const uint32_t it = i0 + threadIdx.x / L;
    const bool on = it < items;
    uint32_t tok = 0, part = 0;
    if (on) byParts(it, tok, part);
    Turn tn;
    if (p.r2) {
      uint32_t seq, at;
      byT(tok, seq, at);
      turn_at<PAIRS>(st, on && pos ? pos[tok] : (int)at, first, true, tn);
    }
    if (!turned) {
#pragma unroll
      for (int i = 0; i < 8; ++i) tn.cs[i] = 1.f, tn.sn[i] = 0.f;
    }
    const int h1 = on ? min((int)(part + 1) * p.per, Ht) : 0;
    for (int hb = 0; hb < p.per; hb += QN_UB) {
      Raw8<T> raw[QN_UB];
      float d[QN_UB][8] = {};
#pragma unroll
      for (int u = 0; u < QN_UB; ++u) {
        const int h = (int)part * p.per + hb + u;
        raw[u] = Raw8<T>{};
        if (hb + u < p.per && h < h1)
          raw[u] = ldraw8((h < p.Hq ? q + (size_t)tok * p.ldq + (size_t)h * D
                                    : k + (size_t)tok * p.ldk + (size_t)(h - p.Hq) * D) +
                          e0);
      }
#pragma unroll
      for (int u = 0; u < QN_UB; ++u) {
        const int h = (int)part * p.per + hb + u;
        if (hb + u >= p.per || h >= h1) continue;
        const bool is_k = h >= p.Hq;
        const int rep = is_k ? p.rk : p.rq, hh = is_k ? h - p.Hq : h;
        const int Ho = is_k ? p.Hk * p.rk : p.Hq * p.rq;
        const T* src = (is_k ? dkn : dqn) + ((size_t)tok * Ho + (size_t)hh * rep) * D + e0;
        for (int i = 0; i < rep; i += 4) {
          Raw8<T> g[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            g[j] = Raw8<T>{};
            if (i + j < rep) g[j] = ldraw8(src + (size_t)(i + j) * D);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (i + j >= rep) break;
            float v[8];
            cvt8(g[j], v);
#pragma unroll
            for (int c = 0; c < 8; ++c) d[u][c] += v[c];
          }
        }
      }
#pragma unroll
      for (int u = 0; u < QN_UB; ++u) {
        const int h = (int)part * p.per + hb + u;
        const bool is_k = h >= p.Hq;
        if (p.r2) turn<PAIRS>(tn, partner, d[u]);
        float x[8], ss = 0.f, ex = 0.f;
        cvt8(raw[u], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!is_k) d[u][i] *= p.q_scale;
          ss = fmaf(x[i], x[i], ss);
          ex = fmaf(d[u][i] * (is_k ? w[1][i] : w[0][i]), x[i], ex);
        }
        ss = lane_sum<L>(ss);
        ex = lane_sum<L>(ex);
        if (hb + u >= p.per || h >= h1) continue;
        // r times the row's sum before r's square: no power of a large r alone
        const float r = rsqrtf(fmaf(ss, 1.f / D, p.eps)), m = r * (r * ex) * (1.f / D);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float wi = is_k ? w[1][i] : w[0][i], g = d[u][i] * (x[i] * r);
          y[i] = r * fmaf(-x[i], m, d[u][i] * wi);
          if (is_k)
            dw[1][i] += g;
          else
            dw[0][i] += g;
        }
        st8(is_k ? dk + ((size_t)tok * p.Hk + (h - p.Hq)) * D + e0
                 : dq + ((size_t)tok * p.Hq + h) * D + e0,
            y);
      }
    }
  }
  if (!part_out) return;
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) red[threadIdx.x / L][e0 + i] = dw[a][i];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += QN_NT) {
      float s = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) s += red[g][c];
      part_out[((size_t)blockIdx.x * 2 + a) * D + c] = s;
    }
  }
}

// ------------------------------------------------------------------ host side
gdn_status check_qk(const gdn_qk_norm_shape* s) {
  if (!s || s->rows < 0 || s->T < 1 || s->Hq < 1 || s->Hk < 1 || s->H < 0 || !(s->eps > 0.f) ||
      (s->style != GDN_ROPE_HALF && s->style != GDN_ROPE_PAIRS))
    return GDN_ERR_INVALID_ARG;
  if (s->H && (s->H % s->Hq || s->H % s->Hk)) return GDN_ERR_INVALID_ARG;
  if (!dtype_ok(s->dtype) || (s->d != 64 && s->d != 128 && s->d != 256) || s->rot < 0 ||
      s->rot > s->d || s->rot % 16)
    return GDN_ERR_UNSUPPORTED;
  const long long heads = (long long)s->Hq + s->Hk;
  if (s->Hq > (1 << 16) || s->Hk > (1 << 16) || s->H > (1 << 16) ||
      s->rows * heads >= (1ll << 31) - (1 << 16))
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// Heads of an item: as many as leave every SM its threads, QN_HEADS at most.
int qk_heads(const gdn_qk_norm_shape& s, int fill) {
  const int Ht = s.Hq + s.Hk, groups = QN_NT / (s.d / 8);
  const long long want = (long long)152 * fill * groups;
  const long long per = (long long)s.rows * Ht / want;
  const int most = std::min(QN_HEADS, Ht);
  int n = (int)std::max(1ll, std::min<long long>(per, most));
  return (Ht + (Ht + n - 1) / n - 1) / ((Ht + n - 1) / n);  // parts of even size
}

struct QkLaunch {
  uint32_t items;
  int parts, per, grid;
};
QkLaunch qk_launch(const gdn_qk_norm_shape& s, bool back) {
  QkLaunch l;
  l.per = qk_heads(s, back ? 4 : 8);
  l.parts = (s.Hq + s.Hk + l.per - 1) / l.per;
  l.items = (uint32_t)s.rows * l.parts;
  const int groups = QN_NT / (s.d / 8);
  l.grid = (int)std::min<long long>(((long long)l.items + groups - 1) / groups,
                                    back ? QN_PARTS : 152 * 8);
  return l;
}
QkArgs qk_args(const gdn_qk_norm_shape& s, int per) {
  return {s.Hq, s.Hk, per, s.H ? s.H / s.Hq : 1, s.H ? s.H / s.Hk : 1, s.rot / 2,
          s.ldq, s.ldk, s.q_scale, s.eps};
}

template <typename T, int D, bool PAIRS>
void launch_fwd(const gdn_qk_norm_shape& s, const void* q, const void* k, const float* wq,
                const float* wk, const double* inv_freq, const int* pos, void* qn, void* kn,
                cudaStream_t st) {
  const QkLaunch l = qk_launch(s, false);
  launch(k_qk_norm_fwd<T, D, PAIRS>, dim3(l.grid), dim3(QN_NT), 0, st, 1, l.items,
         FastDiv(l.parts), FastDiv(s.T), qk_args(s, l.per), (const T*)q, (const T*)k, wq, wk,
         inv_freq, pos, (T*)qn, (T*)kn);
}
template <typename T, int D, bool PAIRS>
void launch_bwd(const gdn_qk_norm_shape& s, const void* q, const void* k, const float* wq,
                const float* wk, const double* inv_freq, const int* pos, const void* dqn,
                const void* dkn, void* dq, void* dk, float* part, cudaStream_t st) {
  const QkLaunch l = qk_launch(s, true);
  launch(k_qk_norm_bwd<T, D, PAIRS>, dim3(l.grid), dim3(QN_NT), 0, st, 1, l.items,
         FastDiv(l.parts), FastDiv(s.T), qk_args(s, l.per), (const T*)q, (const T*)k, wq, wk,
         inv_freq, pos, (const T*)dqn, (const T*)dkn, (T*)dq, (T*)dk, part);
}
template <typename T, int D, typename... A>
void by_style(const gdn_qk_norm_shape& s, A... a) {
  if constexpr (sizeof...(A) == 9) {
    if (s.style == GDN_ROPE_PAIRS) return launch_fwd<T, D, true>(s, a...);
    return launch_fwd<T, D, false>(s, a...);
  } else {
    if (s.style == GDN_ROPE_PAIRS) return launch_bwd<T, D, true>(s, a...);
    return launch_bwd<T, D, false>(s, a...);
  }
}
template <typename T, typename... A>
void by_width(const gdn_qk_norm_shape& s, A... a) {
  switch (s.d) {
    case 64: return by_style<T, 64>(s, a...);
    case 128: return by_style<T, 128>(s, a...);
    default: return by_style<T, 256>(s, a...);
  }
}
template <typename... A>
void dispatch(const gdn_qk_norm_shape& s, A... a) {
  if (s.dtype == GDN_DTYPE_BF16) return by_width<__nv_bfloat16>(s, a...);
  return by_width<float>(s, a...);
}

bool inputs_ok(const gdn_qk_norm_shape& s, const void* q, const void* k, const float* wq,
               const float* wk, const double* inv_freq, const int* pos) {
  return (s.rows == 0 || (q && k)) && (s.rot == 0 || s.rows == 0 || inv_freq) &&
         vec_rows(q, s.ldq, s.dtype) && vec_rows(k, s.ldk, s.dtype) && aligned(wq, 16) &&
         aligned(wk, 16) && aligned(inv_freq, 8) && aligned(pos, 4);
}

}  // namespace
}  // namespace gdn

extern "C" {

gdn_status gdn_qk_norm_fwd(const gdn_qk_norm_shape* shape, const void* q, const void* k,
                           const float* wq, const float* wk, const double* inv_freq,
                           const int* pos, void* qn, void* kn, void* stream) {
  using namespace gdn;
  const gdn_status e = check_qk(shape);
  if (e != GDN_OK) return e;
  const gdn_qk_norm_shape& s = *shape;
  if (!inputs_ok(s, q, k, wq, wk, inv_freq, pos) || (s.rows > 0 && (!qn || !kn)) ||
      !aligned(qn, 16) || !aligned(kn, 16))
    return GDN_ERR_INVALID_ARG;
  if (s.rows == 0) return GDN_OK;
  cudaStream_t st = (cudaStream_t)stream;
  prof_mark(st, "qk_norm_fwd");
  dispatch(s, q, k, wq, wk, inv_freq, pos, qn, kn, st);
  prof_mark(st, nullptr);
  return cudaGetLastError() ? GDN_ERR_CUDA : GDN_OK;
}

size_t gdn_qk_norm_workspace_bytes(const gdn_qk_norm_shape* shape) {
  using namespace gdn;
  if (check_qk(shape) != GDN_OK) return 0;
  const int grid = shape->rows ? qk_launch(*shape, true).grid : 1;
  return round256((size_t)grid * 2 * shape->d * sizeof(float));
}

gdn_status gdn_qk_norm_bwd(const gdn_qk_norm_shape* shape, const void* q, const void* k,
                           const float* wq, const float* wk, const double* inv_freq,
                           const int* pos, const void* dqn, const void* dkn, void* dq, void* dk,
                           float* dwq, float* dwk, void* workspace, size_t workspace_bytes,
                           void* stream) {
  using namespace gdn;
  const gdn_status e = check_qk(shape);
  if (e != GDN_OK) return e;
  const gdn_qk_norm_shape& s = *shape;
  if (!inputs_ok(s, q, k, wq, wk, inv_freq, pos) ||
      (s.rows > 0 && (!dqn || !dkn || !dq || !dk)) || !wq != !dwq || !wk != !dwk ||
      !aligned(dqn, 16) || !aligned(dkn, 16) || !aligned(dq, 16) || !aligned(dk, 16) ||
      !aligned(dwq, 4) || !aligned(dwk, 4))
    return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < gdn_qk_norm_workspace_bytes(shape))
    return GDN_ERR_WORKSPACE;
  cudaStream_t st = (cudaStream_t)stream;
  float* part = (float*)workspace;
  const bool sums = dwq || dwk;
  cudaError_t ce = cudaSuccess;
  if (s.rows > 0) {
    prof_mark(st, "qk_norm_bwd");
    dispatch(s, q, k, wq, wk, inv_freq, pos, dqn, dkn, dq, dk, sums ? part : nullptr, st);
    ce = cudaGetLastError();
    if (ce) return GDN_ERR_CUDA;
  }
  if (sums)
    ce = col_sum(part, s.rows > 0 ? qk_launch(s, true).grid : 0, 2 * s.d, s.d, dwq, dwk, nullptr,
                 st);
  prof_mark(st, nullptr);
  return ce ? GDN_ERR_CUDA : GDN_OK;
}

}  // extern "C"

// The recurrence token by token over a cache of states (gdn_step), and the
// short convolution over a cache of its last inputs (gdn_conv_step):
// include/gdn_layer.h.
#include <stdint.h>

#include "../../include/gdn_conv.h"
#include "gdn_layer.cuh"

namespace gdn {
namespace {

// Where a sequence's tokens and states are.
struct Cache {
  int N, n_tok, n_slots;
  const int *slot_in, *slot_out, *cu, *commit;
};
struct SeqCall {
  int t0, len, commit, in, out;  // in / out: slot or -1
  bool store;                    // the state after `commit` tokens has to be written
};
__device__ __forceinline__ SeqCall seq_call(const Cache& c, int s) {
  SeqCall r;
  r.t0 = s;
  r.len = 1;
  if (c.cu) {
    const int a = c.cu[s], b = c.cu[s + 1];
    const bool ok = a >= 0 && b >= a && b <= c.n_tok;
    r.t0 = ok ? a : 0;
    r.len = ok ? b - a : 0;
  }
  r.commit = c.commit ? min(max(c.commit[s], 0), r.len) : r.len;
  r.in = c.slot_in ? c.slot_in[s] : s;
  r.out = c.slot_out ? c.slot_out[s] : s;
  if ((unsigned)r.in >= (unsigned)c.n_slots) r.in = -1;
  if ((unsigned)r.out >= (unsigned)c.n_slots) r.out = -1;
  r.store = r.out >= 0 && (r.commit > 0 || r.out != r.in);
  return r;
}

constexpr int ST_NT = 128;  // threads of a block
constexpr int ST_COLS = 32; // state columns of a block

// One block: 32 value columns of one head of one sequence, its part of the
// state in registers (thread: 4 columns of every 16th row). With c = S^T k and
// p = S^T q of the old state,
//   u = beta (v - alpha c),   S <- alpha S + k u^T,   o = alpha p + (q.k) u,
// so each token needs one pass over the registers before u and one after it.
template <typename T, int DK>
__global__ void __launch_bounds__(ST_NT)
    k_step(Cache cache, int H, int G, int dv, long long ldq, long long ldk, long long ldv,
           long long ldg, long long ldb, float q_scale, float eps, const T* __restrict__ q,
           const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ g,
           const T* __restrict__ beta, const float* __restrict__ rate,
           const float* __restrict__ bias, float* S, T* __restrict__ o) {
  constexpr int R = DK / 16;
  __shared__ float sq[DK], sk[DK];
  __shared__ float red[4][2][ST_COLS];
  const SeqCall sc = seq_call(cache, blockIdx.y);
  if (sc.len == 0 && !sc.store) return;
  const int slabs = dv / ST_COLS, h = blockIdx.x / slabs, c0 = (blockIdx.x % slabs) * ST_COLS;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tc = tid & 7, tr = tid >> 3;  // columns c0 + 4 tc .., rows tr + 16 r
  float st[R][4];
  if (sc.in >= 0) {
    const float* p = S + ((size_t)sc.in * H + h) * DK * dv + c0 + 4 * tc;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float4 a = *reinterpret_cast<const float4*>(p + (size_t)(tr + 16 * r) * dv);
      st[r][0] = a.x, st[r][1] = a.y, st[r][2] = a.z, st[r][3] = a.w;
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) st[r][0] = st[r][1] = st[r][2] = st[r][3] = 0.f;
  }
  auto store = [&]() {
    float* p = S + ((size_t)sc.out * H + h) * DK * dv + c0 + 4 * tc;
#pragma unroll
    for (int r = 0; r < R; ++r)
      *reinterpret_cast<float4*>(p + (size_t)(tr + 16 * r) * dv) =
          make_float4(st[r][0], st[r][1], st[r][2], st[r][3]);
  };
  if (sc.store && sc.commit == 0) store();
  for (int t = 0; t < sc.len; ++t) {
    const size_t row = (size_t)(sc.t0 + t);
    const T* qp = q + row * ldq + (size_t)(h / G) * DK;
    const T* kp = k + row * ldk + (size_t)(h / G) * DK;
    float qv[DK / 32], kv[DK / 32], qq = 0.f, kk = 0.f, qk = 0.f;
#pragma unroll
    for (int i = 0; i < DK / 32; ++i) {
      qv[i] = ldf(qp + lane + 32 * i);
      kv[i] = ldf(kp + lane + 32 * i);
      qq = fmaf(qv[i], qv[i], qq);
      kk = fmaf(kv[i], kv[i], kk);
      qk = fmaf(qv[i], kv[i], qk);
    }
    qk = lane_sum<32>(qk);
    float qs = 1.f, ks = 1.f, gg = ldf(g + row * ldg + h), bb = ldf(beta + row * ldb + h);
    if (rate) {
      qs = q_scale / sqrtf(lane_sum<32>(qq) + eps);
      ks = 1.f / sqrtf(lane_sum<32>(kk) + eps);
      gg = -expf(rate[h]) * softplusf_(gg + bias[h]);
      bb = sigmoidf_(bb);
    }
    qk *= qs * ks;
    const float alpha = expf(gg);
    __syncthreads();  // the previous token's sq, sk, red are no longer needed
    if (warp == 0) {
#pragma unroll
      for (int i = 0; i < DK / 32; ++i) {
        sq[lane + 32 * i] = qv[i] * qs;
        sk[lane + 32 * i] = kv[i] * ks;
      }
    }
    __syncthreads();
    float c[4] = {}, p[4] = {};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float qi = sq[tr + 16 * r], ki = sk[tr + 16 * r];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[j] = fmaf(ki, st[r][j], c[j]);
        p[j] = fmaf(qi, st[r][j], p[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int m = 8; m < 32; m <<= 1) {
        c[j] += __shfl_xor_sync(0xffffffffu, c[j], m);
        p[j] += __shfl_xor_sync(0xffffffffu, p[j], m);
      }
    }
    if (lane < 8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        red[warp][0][4 * tc + j] = c[j];
        red[warp][1][4 * tc + j] = p[j];
      }
    }
    __syncthreads();
    float u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = 4 * tc + j;
      const float cs = red[0][0][col] + red[1][0][col] + red[2][0][col] + red[3][0][col];
      const float ps = red[0][1][col] + red[1][1][col] + red[2][1][col] + red[3][1][col];
      u[j] = bb * (ldf(v + row * ldv + (size_t)h * dv + c0 + col) - alpha * cs);
      if (tr == 0) stf(o + (row * H + h) * dv + c0 + col, fmaf(alpha, ps, qk * u[j]));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float ki = sk[tr + 16 * r];
#pragma unroll
      for (int j = 0; j < 4; ++j) st[r][j] = fmaf(ki, u[j], alpha * st[r][j]);
    }
    if (sc.store && t + 1 == sc.commit) store();
  }
}

constexpr int CS_NT = 128;  // threads of a block, 4 channels each

// One thread: 4 channels of one sequence; the last W - 1 inputs in registers.
template <typename T, int W>
__global__ void __launch_bounds__(CS_NT)
    k_conv_step(Cache cache, int C, int act, long long ldx, const T* __restrict__ x,
                const float* __restrict__ w, const float* __restrict__ b, T* state,
                T* __restrict__ y) {
  const int c0 = (blockIdx.x * CS_NT + threadIdx.x) * 4;
  if (c0 >= C) return;
  const SeqCall sc = seq_call(cache, blockIdx.y);
  if (sc.len == 0 && !sc.store) return;
  float win[W - 1][4], wr[4][W], br[4];
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      win[j][i] =
          sc.in >= 0 ? ldf(state + ((size_t)sc.in * (W - 1) + j) * C + c0 + i) : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) wr[i][j] = w[(size_t)(c0 + i) * W + j];
    br[i] = b ? b[c0 + i] : 0.f;
  }
  auto store = [&]() {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        stf(state + ((size_t)sc.out * (W - 1) + j) * C + c0 + i, win[j][i]);
  };
  if (sc.store && sc.commit == 0) store();
  for (int t = 0; t < sc.len; ++t) {
    const size_t row = (size_t)(sc.t0 + t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float xc = ldf(x + row * ldx + c0 + i);
      float z = br[i];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) z = fmaf(wr[i][j], win[j][i], z);
      z = fmaf(wr[i][W - 1], xc, z);
      stf(y + row * C + c0 + i, act == GDN_CONV_ACT_SILU ? z * sigmoidf_(z) : z);
#pragma unroll
      for (int j = 0; j < W - 2; ++j) win[j][i] = win[j + 1][i];
      win[W - 2][i] = xc;
    }
    if (sc.store && t + 1 == sc.commit) store();
  }
}

// ------------------------------------------------------------------ host side
gdn_status check_cache(int N, int n_tok, int n_slots, const int* slot_in, const int* slot_out,
                       const int* cu, const int* commit) {
  if (N < 0 || n_tok < 0 || n_slots < 0) return GDN_ERR_INVALID_ARG;
  if (!cu && n_tok != N) return GDN_ERR_INVALID_ARG;
  if ((!slot_in || !slot_out) && n_slots < N) return GDN_ERR_INVALID_ARG;
  if (!aligned(slot_in, 4) || !aligned(slot_out, 4) || !aligned(cu, 4) || !aligned(commit, 4))
    return GDN_ERR_INVALID_ARG;
  if (N > 65535) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

template <typename T, int DK>
void launch_step(const gdn_step_shape& s, const Cache& c, const void* q, const void* k,
                 const void* v, const void* g, const void* beta, const float* rate,
                 const float* bias, float* S, void* o, cudaStream_t st) {
  k_step<T, DK><<<dim3(s.H * (s.dv / ST_COLS), s.N), ST_NT, 0, st>>>(
      c, s.H, s.H / s.Hk, s.dv, s.ldq, s.ldk, s.ldv, s.ldg, s.ldb, s.q_scale, s.eps, (const T*)q,
      (const T*)k, (const T*)v, (const T*)g, (const T*)beta, rate, bias, S, (T*)o);
}

template <typename T, int W>
void launch_conv_step(const gdn_conv_step_shape& s, const Cache& c, const void* x, const float* w,
                      const float* b, void* state, void* y, cudaStream_t st) {
  k_conv_step<T, W><<<dim3((s.C / 4 + CS_NT - 1) / CS_NT, s.N), CS_NT, 0, st>>>(
      c, s.C, s.act, s.ldx, (const T*)x, w, b, (T*)state, (T*)y);
}

template <typename T>
void dispatch_conv_step(const gdn_conv_step_shape& s, const Cache& c, const void* x,
                        const float* w, const float* b, void* state, void* y, cudaStream_t st) {
  switch (s.W) {
    case 2: return launch_conv_step<T, 2>(s, c, x, w, b, state, y, st);
    case 3: return launch_conv_step<T, 3>(s, c, x, w, b, state, y, st);
    case 4: return launch_conv_step<T, 4>(s, c, x, w, b, state, y, st);
    case 5: return launch_conv_step<T, 5>(s, c, x, w, b, state, y, st);
    case 6: return launch_conv_step<T, 6>(s, c, x, w, b, state, y, st);
    case 7: return launch_conv_step<T, 7>(s, c, x, w, b, state, y, st);
    default: return launch_conv_step<T, 8>(s, c, x, w, b, state, y, st);
  }
}

}  // namespace
}  // namespace gdn

extern "C" {

gdn_status gdn_step(const gdn_step_shape* shape, const void* q, const void* k, const void* v,
                    const void* g, const void* beta, const float* rate, const float* bias,
                    float* S, const int* slot_in, const int* slot_out, const int* cu_seqlens,
                    const int* n_commit, void* o, void* stream) {
  using namespace gdn;
  if (!shape) return GDN_ERR_INVALID_ARG;
  const gdn_step_shape& s = *shape;
  const gdn_status e =
      check_cache(s.N, s.n_tok, s.n_slots, slot_in, slot_out, cu_seqlens, n_commit);
  if (e != GDN_OK) return e;
  if (s.H < 1 || s.Hk < 1 || s.H % s.Hk) return GDN_ERR_INVALID_ARG;
  if (!dtype_ok(s.dtype) || (s.dk != 64 && s.dk != 128) ||
      (s.dv != 64 && s.dv != 128 && s.dv != 256) || s.H > (1 << 20))
    return GDN_ERR_UNSUPPORTED;
  if (s.n_tok > 0 && (!q || !k || !v || !g || !beta || !o)) return GDN_ERR_INVALID_ARG;
  if ((s.n_slots > 0 && !S) || (rate == nullptr) != (bias == nullptr)) return GDN_ERR_INVALID_ARG;
  if (rate && !(s.eps > 0.f)) return GDN_ERR_INVALID_ARG;
  const size_t es = elem_size(s.dtype);
  if (!vec_rows(q, s.ldq, s.dtype) || !vec_rows(k, s.ldk, s.dtype) ||
      !vec_rows(v, s.ldv, s.dtype) || s.ldg < 0 || s.ldb < 0 || !aligned(g, es) ||
      !aligned(beta, es) || !aligned(rate, 4) || !aligned(bias, 4) || !aligned(S, 16) ||
      !aligned(o, 16))
    return GDN_ERR_INVALID_ARG;
  if (s.N == 0) return GDN_OK;
  const Cache c = {s.N, s.n_tok, s.n_slots, slot_in, slot_out, cu_seqlens, n_commit};
  cudaStream_t st = (cudaStream_t)stream;
  prof_mark(st, "step");
  if (s.dtype == GDN_DTYPE_BF16) {
    if (s.dk == 64)
      launch_step<__nv_bfloat16, 64>(s, c, q, k, v, g, beta, rate, bias, S, o, st);
    else
      launch_step<__nv_bfloat16, 128>(s, c, q, k, v, g, beta, rate, bias, S, o, st);
  } else {
    if (s.dk == 64)
      launch_step<float, 64>(s, c, q, k, v, g, beta, rate, bias, S, o, st);
    else
      launch_step<float, 128>(s, c, q, k, v, g, beta, rate, bias, S, o, st);
  }
  prof_mark(st, nullptr);
  return cudaGetLastError() ? GDN_ERR_CUDA : GDN_OK;
}

gdn_status gdn_conv_step(const gdn_conv_step_shape* shape, const void* x, const float* w,
                         const float* b, void* state, const int* slot_in, const int* slot_out,
                         const int* cu_seqlens, const int* n_commit, void* y, void* stream) {
  using namespace gdn;
  if (!shape) return GDN_ERR_INVALID_ARG;
  const gdn_conv_step_shape& s = *shape;
  const gdn_status e =
      check_cache(s.N, s.n_tok, s.n_slots, slot_in, slot_out, cu_seqlens, n_commit);
  if (e != GDN_OK) return e;
  if (s.C < 1 || (s.act != GDN_CONV_ACT_NONE && s.act != GDN_CONV_ACT_SILU))
    return GDN_ERR_INVALID_ARG;
  if (!dtype_ok(s.dtype) || s.W < 2 || s.W > 8 || s.C % 4) return GDN_ERR_UNSUPPORTED;
  if ((s.n_tok > 0 && (!x || !y)) || !w || (s.n_slots > 0 && !state)) return GDN_ERR_INVALID_ARG;
  const size_t es = elem_size(s.dtype);
  if (!aligned(x, 4 * es) || s.ldx < 0 || s.ldx % 4 || !aligned(y, 16) || !aligned(state, 16) ||
      !aligned(w, 4) || !aligned(b, 4))
    return GDN_ERR_INVALID_ARG;
  if (s.N == 0) return GDN_OK;
  const Cache c = {s.N, s.n_tok, s.n_slots, slot_in, slot_out, cu_seqlens, n_commit};
  cudaStream_t st = (cudaStream_t)stream;
  prof_mark(st, "conv_step");
  if (s.dtype == GDN_DTYPE_BF16)
    dispatch_conv_step<__nv_bfloat16>(s, c, x, w, b, state, y, st);
  else
    dispatch_conv_step<float>(s, c, x, w, b, state, y, st);
  prof_mark(st, nullptr);
  return cudaGetLastError() ? GDN_ERR_CUDA : GDN_OK;
}

}  // extern "C"

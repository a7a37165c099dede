// The recurrence token by token over a cache of states (gdn_step), and the
// short convolution over a cache of its last inputs (gdn_conv_step):
// include/gdn_layer.h.
#include <stdint.h>

#include <algorithm>

#include "../../include/gdn_conv.h"
#include "gdn_layer.cuh"
#include "gdn_mma.cuh"

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

// 4 consecutive fp32 of shared memory, read again although they have been read
// before: the update of the state must not keep DK registers of k from the dot
// products (the volatile load is what stops the compiler from doing that).
__device__ __forceinline__ ulonglong2 lds4(const float* p) {
  ulonglong2 r;
  asm volatile("ld.volatile.shared.v2.u64 {%0, %1}, [%2];"
               : "=l"(r.x), "=l"(r.y)
               : "r"(smem_u32(p))
               : "memory");
  return r;
}

constexpr int ST_TILE = 8;  // tokens prepared together

// One warp: 32 value columns of one head of one sequence, a whole column of
// the state (DK rows) in each lane's registers. With c = S^T k and p = S^T q of
// the old state,
//   u = beta (v - alpha c),   S <- alpha S + k u^T,   o = alpha p + (q.k) u,
// so a lane needs nothing from other lanes: a token is one pass over its
// registers for c and p and one for the update, with k and q broadcast from
// shared memory. The block's warps share the head; its threads prepare ST_TILE
// tokens' k, q, v, alpha, beta together.
template <typename T, int DK, int dv>
__global__ void __launch_bounds__(dv < 128 ? dv : 128, (DK == 128 ? 3 : 4) * (dv < 128 ? 2 : 1))
    k_step(Cache cache, int H, int G, long long ldq, long long ldk,
           long long ldv, long long ldg, long long ldb, float q_scale, float eps,
           const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
           const T* __restrict__ g, const T* __restrict__ beta, const float* __restrict__ rate,
           const float* __restrict__ bias, float* S, T* __restrict__ o) {
  constexpr int E = DK / 32;  // elements of k and q per lane while preparing
  constexpr int nt = dv < 128 ? dv : 128, parts = dv / nt;  // threads, blocks per head
  __shared__ __align__(16) float sk[ST_TILE][DK], sq[ST_TILE][DK];
  __shared__ float sv[ST_TILE][nt];
  __shared__ float4 sc4[ST_TILE];  // alpha, beta, q.k
  const uint32_t hp = blockIdx.x % (uint32_t)(H * parts), seq = blockIdx.x / (uint32_t)(H * parts);
  const SeqCall sc = seq_call(cache, seq);
  if (sc.len == 0 && !sc.store) return;
  const int h = hp / parts;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c0 = (hp - h * parts) * nt, col = c0 + tid;  // this lane's column
  f32x2 st[DK / 2];
  if (sc.in >= 0) {
    const float* p = S + ((size_t)sc.in * H + h) * DK * dv + col;
#pragma unroll
    for (int r = 0; r < DK / 2; ++r)
      st[r] = pack2(p[(size_t)(2 * r) * dv], p[(size_t)(2 * r + 1) * dv]);
  } else {
#pragma unroll
    for (int r = 0; r < DK / 2; ++r) st[r] = 0;
  }
  auto store = [&]() {
    float* p = S + ((size_t)sc.out * H + h) * DK * dv + col;
#pragma unroll
    for (int r = 0; r < DK / 2; ++r) {
      float lo, hi;
      unpack2(st[r], lo, hi);
      p[(size_t)(2 * r) * dv] = lo;
      p[(size_t)(2 * r + 1) * dv] = hi;
    }
  };
  if (sc.store && sc.commit == 0) store();
  for (int tb = 0; tb < sc.len; tb += ST_TILE) {
    const int nb = min(ST_TILE, sc.len - tb);
    if (tb) __syncthreads();  // the tile before is done with
    for (int i = warp; i < nb; i += nt >> 5) {
      const size_t row = (size_t)(sc.t0 + tb + i);
      const T* qp = q + row * ldq + (size_t)(h / G) * DK + lane * E;
      const T* kp = k + row * ldk + (size_t)(h / G) * DK + lane * E;
      float qv[E], kv[E], qq = 0.f, kk = 0.f, qk = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        qv[e] = ldf(qp + e);
        kv[e] = ldf(kp + e);
      }
      float gg = ldf(g + row * ldg + h), bb = ldf(beta + row * ldb + h);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        qq = fmaf(qv[e], qv[e], qq);
        kk = fmaf(kv[e], kv[e], kk);
        qk = fmaf(qv[e], kv[e], qk);
      }
      qk = lane_sum<32>(qk);
      float qs = 1.f, ks = 1.f;
      if (rate) {
        qs = q_scale / sqrtf(lane_sum<32>(qq) + eps);
        ks = 1.f / sqrtf(lane_sum<32>(kk) + eps);
        gg = -expf(rate[h]) * softplusf_(gg + bias[h]);
        bb = sigmoidf_(bb);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        sq[i][lane * E + e] = qv[e] * qs;
        sk[i][lane * E + e] = kv[e] * ks;
      }
      if (lane == 0) sc4[i] = make_float4(expf(gg), bb, qk * qs * ks, 0.f);
    }
    {
      const T* vp = v + (size_t)(sc.t0 + tb) * ldv + (size_t)h * dv + col;
#pragma unroll
      for (int i = 0; i < ST_TILE; ++i)
        if (i < nb) sv[i][tid] = ldf(vp + (size_t)i * ldv);
    }
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < nb; ++i) {
      const float4 f = sc4[i];
      f32x2 c[2] = {0, 0}, p[2] = {0, 0};
#pragma unroll
      for (int r = 0; r < DK / 4; ++r) {
        const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(&sk[i][4 * r]), q4 = *reinterpret_cast<const ulonglong2*>(&sq[i][4 * r]);
        c[0] = fma2(k4.x, st[2 * r], c[0]);
        p[0] = fma2(q4.x, st[2 * r], p[0]);
        c[1] = fma2(k4.y, st[2 * r + 1], c[1]);
        p[1] = fma2(q4.y, st[2 * r + 1], p[1]);
      }
      const float u = f.y * (sv[i][tid] - f.x * (sum2(c[0]) + sum2(c[1])));
      const float out = fmaf(f.x, sum2(p[0]) + sum2(p[1]), f.z * u);
      stf(o + ((size_t)(sc.t0 + tb + i) * H + h) * dv + col, out);
      const int done = tb + i + 1;
      if (done == sc.len && !(sc.store && sc.commit == done)) break;  // nobody needs this state
      const f32x2 aa = pack2(f.x, f.x), uu = pack2(u, u);
#pragma unroll
      for (int r = 0; r < DK / 4; ++r) {
        const ulonglong2 k4 = lds4(&sk[i][4 * r]);
        st[2 * r] = fma2(aa, st[2 * r], mul2(k4.x, uu));
        st[2 * r + 1] = fma2(aa, st[2 * r + 1], mul2(k4.y, uu));
      }
      if (sc.store && done == sc.commit) store();
    }
  }
}

constexpr int CS_NT = 128;  // threads of a block, 4 channels each
constexpr int CS_LA = 4;    // tokens loaded ahead
constexpr int CS_BLOCKS = 152 * 8;

// 4 channels as loaded, converted when used.
template <typename T>
struct Raw4 {
  uint2 u[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw4<T> ldraw4(const T* p) {
  Raw4<T> r;
  if constexpr (sizeof(T) == 4) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    r.u[0] = make_uint2(a.x, a.y);
    r.u[1] = make_uint2(a.z, a.w);
  } else {
    r.u[0] = *reinterpret_cast<const uint2*>(p);
  }
  return r;
}
__device__ __forceinline__ void cvt4(const Raw4<float>& a, float* v) {
  v[0] = __uint_as_float(a.u[0].x), v[1] = __uint_as_float(a.u[0].y);
  v[2] = __uint_as_float(a.u[1].x), v[3] = __uint_as_float(a.u[1].y);
}
__device__ __forceinline__ void cvt4(const Raw4<__nv_bfloat16>& a, float* v) {
  v[0] = __uint_as_float(a.u[0].x << 16), v[1] = __uint_as_float(a.u[0].x & 0xffff0000u);
  v[2] = __uint_as_float(a.u[0].y << 16), v[3] = __uint_as_float(a.u[0].y & 0xffff0000u);
}
__device__ __forceinline__ void st4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void st4(__nv_bfloat16* p, const float* v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// One thread: 4 channels, whose weights it keeps, of every gridDim.y-th
// sequence; the last W - 1 inputs in registers, the next CS_LA tokens' loads in flight.
template <typename T, int W>
__global__ void __launch_bounds__(CS_NT)
    k_conv_step(Cache cache, int C, int act, long long ldx, const T* __restrict__ x,
                const float* __restrict__ w, const float* __restrict__ b, T* state,
                T* __restrict__ y) {
  const int c0 = (blockIdx.x * CS_NT + threadIdx.x) * 4;
  if (c0 >= C) return;
  float wr[4 * W], br[4] = {};
#pragma unroll
  for (int i = 0; i < W; ++i) cvt4(ldraw4(w + (size_t)c0 * W + 4 * i), wr + 4 * i);
  if (b) cvt4(ldraw4(b + c0), br);
  for (int seq = blockIdx.y; seq < cache.N; seq += gridDim.y) {
    const SeqCall sc = seq_call(cache, seq);
    if (sc.len == 0 && !sc.store) continue;
    const T* xp = x + (size_t)sc.t0 * ldx + c0;
    Raw4<T> xr[CS_LA];
#pragma unroll
    for (int u = 0; u < CS_LA; ++u)
      if (u < sc.len) xr[u] = ldraw4(xp + (size_t)u * ldx);
    float win[W - 1][4] = {};
    if (sc.in >= 0) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        cvt4(ldraw4(state + ((size_t)sc.in * (W - 1) + j) * C + c0), win[j]);
    }
    auto store = [&]() {
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        st4(state + ((size_t)sc.out * (W - 1) + j) * C + c0, win[j]);
    };
    if (sc.store && sc.commit == 0) store();
    T* yp = y + (size_t)sc.t0 * C + c0;
    for (int t0 = 0; t0 < sc.len; t0 += CS_LA) {
#pragma unroll
      for (int u = 0; u < CS_LA; ++u) {
        const int t = t0 + u;
        if (t >= sc.len) break;
        float xc[4], out[4];
        cvt4(xr[u], xc);
        if (t + CS_LA < sc.len) xr[u] = ldraw4(xp + (size_t)(t + CS_LA) * ldx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float z = br[i];
#pragma unroll
          for (int j = 0; j < W - 1; ++j) z = fmaf(wr[i * W + j], win[j][i], z);
          z = fmaf(wr[i * W + W - 1], xc[i], z);
          out[i] = act == GDN_CONV_ACT_SILU ? z * sigmoid_as<T>(z) : z;
#pragma unroll
          for (int j = 0; j < W - 2; ++j) win[j][i] = win[j + 1][i];
          win[W - 2][i] = xc[i];
        }
        st4(yp + (size_t)t * C, out);
        if (sc.store && t + 1 == sc.commit) store();
      }
    }
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
  return GDN_OK;
}

template <typename T, int DK, int DV>
void launch_step(const gdn_step_shape& s, const Cache& c, const void* q, const void* k,
                 const void* v, const void* g, const void* beta, const float* rate,
                 const float* bias, float* S, void* o, cudaStream_t st) {
  constexpr int nt = DV < 128 ? DV : 128;
  k_step<T, DK, DV><<<(unsigned)s.N * s.H * (DV / nt), nt, 0, st>>>(
      c, s.H, s.H / s.Hk, s.ldq, s.ldk, s.ldv, s.ldg, s.ldb, s.q_scale, s.eps, (const T*)q,
      (const T*)k, (const T*)v, (const T*)g, (const T*)beta, rate, bias, S, (T*)o);
}
template <typename T, int DK, typename... A>
void dispatch_step(const gdn_step_shape& s, A... a) {
  switch (s.dv) {
    case 64: return launch_step<T, DK, 64>(s, a...);
    case 128: return launch_step<T, DK, 128>(s, a...);
    default: return launch_step<T, DK, 256>(s, a...);
  }
}

template <typename T, int W>
void launch_conv_step(const gdn_conv_step_shape& s, const Cache& c, const void* x, const float* w,
                      const float* b, void* state, void* y, cudaStream_t st) {
  // as many sequences per thread as leave the GPU CS_BLOCKS blocks
  const int gx = (s.C / 4 + CS_NT - 1) / CS_NT, gy = std::min(s.N, (CS_BLOCKS + gx - 1) / gx);
  k_conv_step<T, W><<<dim3(gx, gy), CS_NT, 0, st>>>(c, s.C, s.act, s.ldx, (const T*)x, w, b,
                                                    (T*)state, (T*)y);
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
      (s.dv != 64 && s.dv != 128 && s.dv != 256) || 2ll * s.N * s.H >= (1ll << 31))
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
      dispatch_step<__nv_bfloat16, 64>(s, c, q, k, v, g, beta, rate, bias, S, o, st);
    else
      dispatch_step<__nv_bfloat16, 128>(s, c, q, k, v, g, beta, rate, bias, S, o, st);
  } else {
    if (s.dk == 64)
      dispatch_step<float, 64>(s, c, q, k, v, g, beta, rate, bias, S, o, st);
    else
      dispatch_step<float, 128>(s, c, q, k, v, g, beta, rate, bias, S, o, st);
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
      !aligned(w, 16) || !aligned(b, 16))
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

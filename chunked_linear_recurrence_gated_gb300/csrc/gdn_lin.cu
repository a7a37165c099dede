// Linear attention with a decay for each head over whole sequences
// (gdn_lin_fwd / gdn_lin_bwd, include/gdn_lin.h): the entry points, and the kernels
// with fp32 products.
//
// Chunks of C = 64 tokens, all at once. With gamma_t the log-decay summed from the
// chunk's start, L_ts = e^{gamma_t - gamma_s} (s <= t, else 0), S the state before
// the chunk and R the gradient of the one behind it:
//   D = (e^{gamma_C - gamma} k)^T v,  S' = e^{gamma_C} S + D      k_lin_sum, k_lin_scan
//   E = scale (e^{gamma} q)^T dO,     R' = e^{gamma_C} R + E
//   o  = scale (P v + e^{gamma} q S),      P = q k^T * L          k_lin_out
//   dq = scale (W k + e^{gamma} dO S^T),   W = dO v^T * L         k_lin_grad
//   dk = scale W^T q + e^{gamma_C - gamma} v R^T
//   dv = scale P^T dO + e^{gamma_C - gamma} k R
// and for the decay every pair (s, t) with s < u <= t counts once in dg_u:
//   dg_u = sum_{s < u <= t} A_ts + sum_{t >= u} a_t + sum_{s < u} b_s + e^{gamma_C} <S, R>,
//   A = scale (q k^T) (dO v^T) L,  a_t = q_t . (far part of dq_t),  b_s = k_s . (that of dk_s):
// sums over the chunk only, of terms that all carry the decay between their tokens. Sums over
// s < u and over t >= u are formed as such, never as a difference of longer ones, so what lies
// behind a token's decay leaves no rounding in its dg.
#include <stdint.h>

#include <algorithm>

#include "gdn_lin.cuh"
#include "gdn_mma.cuh"

namespace gdn {
namespace {

constexpr int LC = 64;    // tokens of a chunk
constexpr int LN_NT = 256;
constexpr int LP = 4;     // floats between rows: both ways to read a fragment (8 rows by 4
                          // columns, 4 by 8) hit every bank at most twice

__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;  // keeps a NaN, which hi does not
}

// C += A B by one warp: 16 rows, NT x 8 columns, K deep; a(m, k) and b(k, n) give the
// operands' elements. Each takes two TF32 parts, the product of the second parts is left out.
// U steps of K are unrolled: for operands in global memory enough that their loads overlap.
template <int NT, int K, int U = 2, class FA, class FB>
__device__ __forceinline__ void mm(float (*c)[4], FA a, FB b) {
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll U
  for (int k0 = 0; k0 < K; k0 += 8) {
    uint32_t ah[4], al[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) split_tf32(a(g + 8 * (i & 1), k0 + t + 4 * (i >> 1)), ah[i], al[i]);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      uint32_t bh[2], bl[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) split_tf32(b(k0 + t + 4 * i, 8 * j + g), bh[i], bl[i]);
      // 8 products at a time in the tensor core, whose sums drop what does not fit; the rest of
      // the sum is rounded (error of a 128-term product 4 times smaller, time the same)
      float d[4] = {};
      mma_tf32(d, al, bh[0], bh[1]);
      mma_tf32(d, ah, bl[0], bl[1]);
      mma_tf32(d, ah, bh[0], bh[1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) c[j][i] += d[i];
    }
  }
}

// gamma of a chunk, in two floats.
struct Gamma {
  float hi[LC], lo[LC];
  __device__ __forceinline__ float to(int t, int s) const {  // gamma_t - gamma_s
    return (hi[t] - hi[s]) + (lo[t] - lo[s]);
  }
};
template <typename T>
__device__ __forceinline__ void chunk_gamma(const LinUnit& u, int h, const T* g, long long ldg,
                                            const float* decay, Gamma& out) {  // one warp
  const int l = threadIdx.x & 31;
  Two c[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = 2 * l + i;
    c[i] = {t < u.len ? lin_decay(decay ? decay[h] : ldf(g + (size_t)(u.row + t) * ldg + h)) : 0.f, 0.f};
  }
  c[1] = add_two(c[0], c[1]);
  const Two before = sum_before(c[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const Two x = add_two(before, c[i]);
    out.hi[2 * l + i] = x.hi;
    out.lo[2 * l + i] = x.lo;
  }
}

// A chunk's rows, all asked for at once (get) and later written as fp32 to shared memory
// (put): zeros behind the chunk's end, row t times f(t).
template <typename T, int D>
struct Rows {
  static constexpr int N = LC * D / 8 / LN_NT;
  Raw8<T> raw[N];
  __device__ __forceinline__ void get(const T* from, long long ld, const LinUnit& u) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = threadIdx.x + n * LN_NT, t = i / (D / 8);
      raw[n] = Raw8<T>{};
      if (t < u.len) raw[n] = ldraw8(from + (size_t)(u.row + t) * ld + i % (D / 8) * 8);
    }
  }
  template <class F>
  __device__ __forceinline__ void put(float* to, const LinUnit& u, F f) const {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = threadIdx.x + n * LN_NT, t = i / (D / 8);
      float x[8];
      cvt8(raw[n], x);
      const float by = t < u.len ? f(t) : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= by;
      st8(to + t * (D + LP) + i % (D / 8) * 8, x);
    }
  }
};

template <typename T>
struct LinIn {
  const T *q, *k, *v, *g, *dout;
  const float* decay;
  long long ldq, ldk, ldv, ldg, ldo;
  float scale;
};

// D (or E) of a chunk, and e^{gamma_C}. Grid (chunk, head, D or E). 15 us for both of 2 x 2049
// tokens x 6 heads, fp32 64 x 64: one chunk's latency, twice (issue 39 %, tensor pipe 31 %).
template <typename T, int DK, int DV, bool BACK>
__global__ void __launch_bounds__(LN_NT)
    k_lin_sum(LinMap m, LinIn<T> in, float* whole, float* D, float* E) {
  chain();
  extern __shared__ __align__(16) float sm[];
  __shared__ Gamma gm;
  LinUnit u;
  if (!lin_unit(m, blockIdx.x, u)) return;
  const int h = blockIdx.y, H = gridDim.y, w = threadIdx.x >> 5;
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  const size_t uh = (size_t)blockIdx.x * H + h;
  const int pass = BACK ? blockIdx.z : 0;
  Rows<T, DK> rx;
  Rows<T, DV> ry;
  rx.get((pass ? in.q : in.k) + (size_t)h * DK, pass ? in.ldq : in.ldk, u);
  ry.get((pass ? in.dout : in.v) + (size_t)h * DV, pass ? in.ldo : in.ldv, u);
  if (w == 0) chunk_gamma(u, h, in.g, in.ldg, in.decay, gm);
  __syncthreads();
  if (threadIdx.x == 0 && pass == 0) whole[uh] = expf(gm.to(LC - 1, 0) + gm.hi[0]);
  float *x = sm, *y = sm + LC * (DK + LP);
  rx.put(x, u, [&](int r) { return pass ? in.scale * expf(gm.hi[r]) : expf(gm.to(LC - 1, r)); });
  ry.put(y, u, [](int) { return 1.f; });
  __syncthreads();
  {
    // 8 warps: 16 rows each of 128, or 4 x 2 halves of the columns
    constexpr int WN = DK == 128 ? 1 : 2, NT = DV / 8 / WN;
    const int m0 = w / WN * 16, n0 = w % WN * (DV / WN);
    float c[NT][4] = {};
    mm<NT, LC>(c, [&](int i, int s) { return x[s * (DK + LP) + m0 + i]; },
               [&](int s, int j) { return y[s * (DV + LP) + n0 + j]; });
    float* out = (pass ? E : D) + uh * DK * DV;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        *reinterpret_cast<float2*>(out + (size_t)(m0 + g + 8 * r) * DV + n0 + 8 * j + 2 * t) =
            make_float2(c[j][2 * r], c[j][2 * r + 1]);
  }
}

// In place over the units of a sequence: D_b becomes the state before unit b
// (z = 0), E_b the gradient of the state behind it (z = 1, from the last unit). `open`:
// the last one to be visited has no sum of its own, and nothing is wanted behind it. D and
// E have the units' layouts (LinLayout), the states of the call their own. Latency: SC_U units'
// elements are asked for at once (33 units of 64 x 64: 7 us; 16 at once 11).
constexpr int SC_NT = 128, SC_U = 8;
__global__ void __launch_bounds__(SC_NT)
    k_lin_scan(LinMap m, int H, int dk, int dv, LinLayout lay, const float* whole_d, float* D,
               const float* S_in, float* S_out, const float* whole_e, float* E, const float* dS_out,
               float* dS_in, bool open, int* status) {
  chain();
  if (m.cu) {
    if (*status != DEV_OK) return;
  } else if (!open && (blockIdx.x | blockIdx.y | blockIdx.z | threadIdx.x) == 0) {
    *status = DEV_OK;
  }
  const int e = blockIdx.x * SC_NT + threadIdx.x, h = blockIdx.y % H, seq = blockIdx.y / H;
  const int n4 = dk * dv / 4;
  const bool back = blockIdx.z;
  if (e >= n4) return;
  int first, n;
  lin_seq(m, seq, first, n);
  if (open && n < 2) return;  // its one unit starts from S_in itself
  float4* at = reinterpret_cast<float4*>(back ? E : D) + e;
  const float* whole = back ? whole_e : whole_d;
  const float* from = back ? dS_out : S_in;
  float* to = back ? dS_in : S_out;
  const size_t sh = (size_t)seq * H + h;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (from) {
    from += sh * n4 * 4;
    if (lay == LIN_ROWS)
      s = reinterpret_cast<const float4*>(from)[e];
    else
      s = *reinterpret_cast<const float4*>(from + (size_t)(e % dk) * dv + e / dk * 4);
  }
  for (int b0 = 0; b0 < n; b0 += SC_U) {
    float4 d[SC_U];
    float a[SC_U];
#pragma unroll
    for (int i = 0; i < SC_U; ++i)
      if (b0 + i < n) {
        const size_t uh = (size_t)(first + (back ? n - 1 - b0 - i : b0 + i)) * H + h;
        const bool has = !open || b0 + i < n - 1;
        d[i] = has ? at[uh * n4] : make_float4(0.f, 0.f, 0.f, 0.f);
        a[i] = has ? whole[uh] : 0.f;
      }
#pragma unroll
    for (int i = 0; i < SC_U; ++i)
      if (b0 + i < n) {
        const size_t uh = (size_t)(first + (back ? n - 1 - b0 - i : b0 + i)) * H + h;
        at[uh * n4] = s;
        s.x = fmaf(a[i], s.x, d[i].x);
        s.y = fmaf(a[i], s.y, d[i].y);
        s.z = fmaf(a[i], s.z, d[i].z);
        s.w = fmaf(a[i], s.w, d[i].w);
      }
  }
  if (to) reinterpret_cast<float4*>(to)[sh * n4 + e] = s;
}

// o of a chunk from the state before it. 8 warps: 4 x 16 rows, 2 halves of the columns.
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(LN_NT)
    k_lin_out(LinMap m, LinIn<T> in, const float* S, T* o) {
  chain();
  extern __shared__ __align__(16) float sm[];
  __shared__ Gamma gm;
  LinUnit u;
  if (!lin_unit(m, blockIdx.x, u)) return;
  constexpr int LK = DK + LP, LV = DV + LP, LL = LC + LP;
  float *q = sm, *k = q + LC * LK, *v = k + LC * LK, *p = v + LC * LV;
  const int h = blockIdx.y, H = gridDim.y, w = threadIdx.x >> 5;
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  S += ((size_t)blockIdx.x * H + h) * DK * DV;
  auto one = [](int) { return 1.f; };
  {
    Rows<T, DK> rq, rk;
    Rows<T, DV> rv;
    rq.get(in.q + (size_t)h * DK, in.ldq, u);
    rk.get(in.k + (size_t)h * DK, in.ldk, u);
    rv.get(in.v + (size_t)h * DV, in.ldv, u);
    rq.put(q, u, one);
    rk.put(k, u, one);
    rv.put(v, u, one);
  }
  if (w == 0) chunk_gamma(u, h, in.g, in.ldg, in.decay, gm);
  __syncthreads();
  const int m0 = w / 2 * 16;
  {
    float c[LC / 16][4] = {};
    const int n0 = w % 2 * (LC / 2);
    mm<LC / 16, DK>(c, [&](int i, int e) { return q[(m0 + i) * LK + e]; },
                    [&](int e, int j) { return k[(n0 + j) * LK + e]; });
#pragma unroll
    for (int j = 0; j < LC / 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = m0 + g + 8 * (i >> 1), s = n0 + 8 * j + 2 * t + (i & 1);
        p[r * LL + s] = s <= r ? c[j][i] * expf(gm.to(r, s)) : 0.f;
      }
  }
  __syncthreads();
  constexpr int NT = DV / 16;
  const int n0 = w % 2 * (DV / 2);
  float c[NT][4] = {};
  mm<NT, DK, 8>(c, [&](int i, int e) { return q[(m0 + i) * LK + e]; },
             [&](int e, int j) { return S[(size_t)e * DV + n0 + j]; });
  const float up[2] = {expf(gm.hi[m0 + g]), expf(gm.hi[m0 + g + 8])};
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[j][i] *= up[i >> 1];
  mm<NT, LC>(c, [&](int i, int s) { return p[(m0 + i) * LL + s]; },
             [&](int s, int j) { return v[s * LV + n0 + j]; });
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = m0 + g + 8 * r;
    if (row >= u.len) continue;
    T* out = o + ((size_t)(u.row + row) * H + h) * DV + n0 + 2 * t;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      stf(out + 8 * j, in.scale * c[j][2 * r]);
      stf(out + 8 * j + 1, in.scale * c[j][2 * r + 1]);
    }
  }
}

// The gradients of a chunk from the state before it and the gradient of the one behind
// it. dgsum [unit, H]: the sum of dg over the chunk (one decay for each head). Its tiles leave
// room for 2 blocks an SM where heads are 64 x 64 (one: 82 us instead of 52 for 2 x 2049 tokens
// x 6 heads); bound by TF32 MMAs and the splitting of their operands in turn (tensor pipe 35 %,
// issue 36 %).
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(LN_NT, DK + DV == 128 ? 2 : 1)
    k_lin_grad(LinMap m, LinIn<T> in, const float* S, const float* R, T* dq, T* dk, T* dv, T* dg,
               float* dgsum) {
  chain();
  extern __shared__ __align__(16) float sm[];
  __shared__ Gamma gm;
  __shared__ float rows[LC], cols[4][LC], far_q[2][LC], far_k[2][LC], cross[LN_NT / 32];
  LinUnit u;
  const int h = blockIdx.y, H = gridDim.y, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t uh = (size_t)blockIdx.x * H + h;
  if (!lin_unit(m, blockIdx.x, u)) {
    if (dgsum && threadIdx.x == 0) dgsum[uh] = 0.f;
    return;
  }
  constexpr int LK = DK + LP, LV = DV + LP, LL = LC + LP;
  float *q = sm, *k = q + LC * LK, *v = k + LC * LK, *d = v + LC * LV, *p = d + LC * LV,
        *wm = p + LC * LL;
  const int g = lane >> 2, t = lane & 3;
  S += uh * DK * DV;
  R += uh * DK * DV;
  auto one = [](int) { return 1.f; };
  {
    Rows<T, DK> rq, rk;
    Rows<T, DV> rv, rd;
    rq.get(in.q + (size_t)h * DK, in.ldq, u);
    rk.get(in.k + (size_t)h * DK, in.ldk, u);
    rv.get(in.v + (size_t)h * DV, in.ldv, u);
    rd.get(in.dout + (size_t)h * DV, in.ldo, u);
    rq.put(q, u, one);
    rk.put(k, u, one);
    rv.put(v, u, one);
    rd.put(d, u, one);
  }
  if (w == 0) chunk_gamma(u, h, in.g, in.ldg, in.decay, gm);
  __syncthreads();
  const int m0 = w / 2 * 16, half = w % 2;
  {
    constexpr int NT = LC / 16;
    const int n0 = half * (LC / 2);
    float a[NT][4] = {}, b[NT][4] = {}, before[2] = {};
    mm<NT, DK>(a, [&](int i, int e) { return q[(m0 + i) * LK + e]; },
               [&](int e, int j) { return k[(n0 + j) * LK + e]; });
    mm<NT, DV>(b, [&](int i, int e) { return d[(m0 + i) * LV + e]; },
               [&](int e, int j) { return v[(n0 + j) * LV + e]; });
    // Pairs s < u <= t with s in this half of the columns: before = a row's sum over s < u, and
    // cols [16 rows][u] its sum over the rows t >= u. rows: the first half's whole sums, which
    // the second half's u are all behind.
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float cs[2] = {};
      const int u = n0 + 8 * j + 2 * t;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int r = m0 + g + 8 * z;
        float x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int s = u + i;
          const float f = s <= r ? in.scale * expf(gm.to(r, s)) : 0.f;
          const float c = a[j][2 * z + i], e = b[j][2 * z + i];
          x[i] = s < r ? c * e * f : 0.f;
          p[r * LL + s] = s <= r ? c * f : 0.f;
          wm[r * LL + s] = s <= r ? e * f : 0.f;
        }
        float up = x[0] + x[1];  // of the lanes up to this one
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          const float y = __shfl_up_sync(0xffffffffu, up, o, 4);
          if (t >= o) up += y;
        }
        float lanes = __shfl_up_sync(0xffffffffu, up, 1, 4);
        if (t == 0) lanes = 0.f;
        if (u <= r) cs[0] += before[z] + lanes;
        if (u < r) cs[1] += before[z] + (lanes + x[0]);
        before[z] += __shfl_sync(0xffffffffu, up, 3, 4);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) cs[i] += __shfl_xor_sync(0xffffffffu, cs[i], o);
        if (g == 0) cols[w / 2][u + i] = cs[i];
      }
    }
    if (half == 0 && t == 0) rows[m0 + g] = before[0], rows[m0 + g + 8] = before[1];
  }
  {
    float x = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x; i < DK * DV / 4; i += LN_NT) {
      const float4 a = reinterpret_cast<const float4*>(S)[i], b = reinterpret_cast<const float4*>(R)[i];
      x = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, x))));
    }
    x = lane_sum<32>(x);
    if (lane == 0) cross[w] = x;
  }
  __syncthreads();
  // rows of c times f, their products with the rows of x summed to far, then more added
  auto finish = [&](auto& c, const float* f, const float* x, int ld, int n0, float* far) {
    constexpr int NT = sizeof(c) / sizeof(c[0]);
    float s[2] = {};
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[j][i] *= f[i >> 1];
        if (far) s[i >> 1] = fmaf(x[(m0 + g + 8 * (i >> 1)) * ld + n0 + 8 * j + 2 * t + (i & 1)],
                                  c[j][i], s[i >> 1]);
      }
    if (!far) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float y = lane_sum<4>(s[i]);
      if (t == 0) far[m0 + g + 8 * i] = y;
    }
  };
  auto store = [&](auto& c, T* to, int D, int n0) {
    constexpr int NT = sizeof(c) / sizeof(c[0]);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = m0 + g + 8 * r;
      if (row >= u.len) continue;
      T* out = to + ((size_t)(u.row + row) * H + h) * D + n0 + 2 * t;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        stf(out + 8 * j, c[j][2 * r]);
        stf(out + 8 * j + 1, c[j][2 * r + 1]);
      }
    }
  };
  const int r0 = m0 + g, r1 = r0 + 8;
  const float up[2] = {in.scale * expf(gm.hi[r0]), in.scale * expf(gm.hi[r1])};
  const float down[2] = {expf(gm.to(LC - 1, r0)), expf(gm.to(LC - 1, r1))};
  {
    const int n0 = half * (DK / 2);
    float c[DK / 16][4] = {};
    mm<DK / 16, DV, 8>(c, [&](int i, int e) { return d[(m0 + i) * LV + e]; },
                    [&](int e, int j) { return S[(size_t)(n0 + j) * DV + e]; });
    finish(c, up, q, LK, n0, far_q[half]);
    mm<DK / 16, LC>(c, [&](int i, int s) { return wm[(m0 + i) * LL + s]; },
                    [&](int s, int j) { return k[s * LK + n0 + j]; });
    store(c, dq, DK, n0);
  }
  {
    const int n0 = half * (DK / 2);
    float c[DK / 16][4] = {};
    mm<DK / 16, DV, 8>(c, [&](int i, int e) { return v[(m0 + i) * LV + e]; },
                    [&](int e, int j) { return R[(size_t)(n0 + j) * DV + e]; });
    finish(c, down, k, LK, n0, far_k[half]);
    mm<DK / 16, LC>(c, [&](int i, int s) { return wm[s * LL + m0 + i]; },
                    [&](int s, int j) { return q[s * LK + n0 + j]; });
    store(c, dk, DK, n0);
  }
  {
    const int n0 = half * (DV / 2);
    float c[DV / 16][4] = {};
    mm<DV / 16, DK, 8>(c, [&](int i, int e) { return k[(m0 + i) * LK + e]; },
                    [&](int e, int j) { return R[(size_t)e * DV + n0 + j]; });
    finish(c, down, k, LK, n0, (float*)nullptr);
    mm<DV / 16, LC>(c, [&](int i, int s) { return p[s * LL + m0 + i]; },
                    [&](int s, int j) { return d[s * LV + n0 + j]; });
    store(c, dv, DV, n0);
  }
  __syncthreads();
  if (w) return;
  float x = 0.f;
#pragma unroll
  for (int i = 0; i < LN_NT / 32; ++i) x += cross[i];
  x *= expf(gm.to(LC - 1, 0) + gm.hi[0]);
  // of this lane's tokens u = 2 l, 2 l + 1: pairs of the chunk; a, and pairs across the
  // halves, over t >= u; b over s < u
  float near[2], a[2], b[2], far[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 2 * lane + i;
    near[i] = (cols[0][r] + cols[1][r]) + (cols[2][r] + cols[3][r]);
    a[i] = far_q[0][r] + far_q[1][r];
    b[i] = far_k[0][r] + far_k[1][r];
    far[i] = rows[r];
  }
  float as = a[0] + a[1], bs = b[0] + b[1], fs = far[0] + far[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_down_sync(0xffffffffu, as, o), z = __shfl_up_sync(0xffffffffu, bs, o),
                f = __shfl_down_sync(0xffffffffu, fs, o);
    if (lane + o < 32) as += y, fs += f;
    if (lane >= o) bs += z;
  }
  // the lanes behind, and before
  as = __shfl_down_sync(0xffffffffu, as, 1), fs = __shfl_down_sync(0xffffffffu, fs, 1);
  bs = __shfl_up_sync(0xffffffffu, bs, 1);
  if (lane == 31) as = fs = 0.f;
  if (lane == 0) bs = 0.f;
  const bool second = 2 * lane >= LC / 2;
  const float d1 = near[1] + (as + a[1]) + (bs + b[0]) + x + (second ? fs + far[1] : 0.f);
  const float d0 = near[0] + (as + a[1] + a[0]) + bs + x + (second ? fs + far[1] + far[0] : 0.f);
  const int t0 = 2 * lane;
  if (dg) {
    if (t0 < u.len) stf(dg + (size_t)(u.row + t0) * H + h, d0);
    if (t0 + 1 < u.len) stf(dg + (size_t)(u.row + t0 + 1) * H + h, d1);
  } else if (dgsum) {  // a call without tokens has neither
    const float sum = lane_sum<32>((t0 < u.len ? d0 : 0.f) + (t0 + 1 < u.len ? d1 : 0.f));
    if (lane == 0) dgsum[uh] = sum;
  }
}

// The units of a packed call, one at least for each sequence. One block: each thread
// counts a run of sequences. The order is a counting sort by the units' chunks; how units of
// the same length stand among each other changes no result.
constexpr int PL_NT = 1024, PL_BINS = 65;
__global__ void __launch_bounds__(PL_NT)
    k_lin_plan(LinMap m, int* first, int* owner, int* order, int chunk, int* status) {
  __shared__ int sums[32], bad, bins[PL_BINS];
  chain();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (tid == 0) bad = m.cu[0] < 0 || m.cu[m.nseq] > m.T;
  if (tid < PL_BINS) bins[tid] = 0;
  auto bin = [&](int len) { return PL_BINS - 1 - min((len + chunk - 1) / chunk, PL_BINS - 1); };
  __syncthreads();
  const int run = (m.nseq + PL_NT - 1) / PL_NT, s0 = min(tid * run, m.nseq),
            s1 = min(s0 + run, m.nseq);
  int n = 0, wrong = 0;
  for (int s = s0; s < s1; ++s) {
    const int len = m.cu[s + 1] - m.cu[s];
    wrong |= m.cu[s + 1] < m.cu[s];
    n += max(1, (int)(((unsigned)max(len, 0) + m.unit - 1) / m.unit));
  }
  if (wrong) bad = 1;
  int up = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, up, d);
    if (lane >= d) up += y;
  }
  if (lane == 31) sums[w] = up;
  __syncthreads();
  int before = up - n;
  for (int i = 0; i < w; ++i) before += sums[i];
  const bool off = bad;
  if (tid == 0) *status = off ? DEV_BAD_CU_SEQLENS : DEV_OK;
  for (int s = s0; s < s1; ++s) {
    first[s] = off ? 0 : before;
    const int k =
        off ? 0 : max(1, (int)(((unsigned)(m.cu[s + 1] - m.cu[s]) + m.unit - 1) / m.unit));
    for (int i = 0; i < k; ++i)
      if (before + i < m.cap) owner[before + i] = s;
    if (order && k) {
      if (k > 1) atomicAdd(bins + bin(m.unit), k - 1);
      atomicAdd(bins + bin(m.cu[s + 1] - m.cu[s] - (k - 1) * m.unit), 1);
    }
    before += k;
  }
  __shared__ int total;
  if (tid == PL_NT - 1) total = off ? 0 : before;
  __syncthreads();
  if (tid == 0) first[m.nseq] = total;
  for (int i = total + tid; i < m.cap; i += PL_NT) {
    owner[i] = -1;
    if (order) order[i] = i;
  }
  if (!order || off) return;
  if (w == 0) {  // bins to first places
    int x[3], at = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      x[i] = 3 * lane + i < PL_BINS ? bins[3 * lane + i] : 0;
      at += x[i];
    }
    int all = at;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, all, d);
      if (lane >= d) all += y;
    }
    at = all - at;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if (3 * lane + i < PL_BINS) bins[3 * lane + i] = at;
      at += x[i];
    }
  }
  __syncthreads();
  for (int s = s0; s < s1; ++s) {
    const int u = first[s], k = max(1, (int)(((unsigned)(m.cu[s + 1] - m.cu[s]) + m.unit - 1) / m.unit));
    if (k > 1) {
      const int at = atomicAdd(bins + bin(m.unit), k - 1);
      for (int i = 0; i < k - 1; ++i)
        if (at + i < m.cap) order[at + i] = u + i;
    }
    const int at = atomicAdd(bins + bin(m.cu[s + 1] - m.cu[s] - (k - 1) * m.unit), 1);
    if (at < m.cap) order[at] = u + k - 1;
  }
}

// ------------------------------------------------------------------ host side
struct SimtPlan {
  LinMap m;
  int *status, *first, *owner;
  float *whole, *dgsum, *D, *E;
  size_t bytes;
};
SimtPlan simt_plan(const gdn_lin_shape& s, const int* cu, bool packed, bool back,
                   unsigned char* ws) {
  SimtPlan p = {};
  const int per = std::max(1, (s.T + LC - 1) / LC);
  p.m = {cu, nullptr, nullptr, s.nseq, s.T, LC, per, packed ? per + s.nseq : per * s.nseq};
  size_t at = 0;
  auto take = [&](size_t n) {
    unsigned char* r = ws + at;
    at += round256(n);
    return r;
  };
  const size_t uh = (size_t)p.m.cap * s.H, state = uh * s.dk * s.dv * sizeof(float);
  p.status = (int*)take(4);
  p.first = (int*)take(packed ? (size_t)(s.nseq + 1) * 4 : 0);
  p.owner = (int*)take(packed ? (size_t)p.m.cap * 4 : 0);
  p.whole = (float*)take(uh * 4);
  p.dgsum = (float*)take(back ? uh * 4 : 0);
  p.D = (float*)take(state);
  p.E = (float*)take(back ? state : 0);
  p.m.first = p.first;
  p.m.owner = p.owner;
  p.bytes = at;
  return p;
}

template <typename T, int DK, int DV>
cudaError_t run_simt(const LinCall& c, bool back) {
  const gdn_lin_shape& s = c.s;
  const SimtPlan p = simt_plan(s, c.cu, c.cu != nullptr, back, c.ws);
  const LinIn<T> in = {(const T*)c.q, (const T*)c.k, (const T*)c.v, (const T*)c.g,
                       (const T*)c.dout, c.decay, s.ldq, s.ldk, s.ldv, s.ldg,
                       (long long)s.H * DV, s.scale};
  cudaError_t e = cudaSuccess;
  if (c.cu && (e = lin_plan(p.m, p.first, p.owner, nullptr, LC, p.status, c.st))) return e;
  dim3 grid(p.m.cap, s.H, back ? 2 : 1);
  constexpr int rows_k = LC * (DK + LP) * 4, rows_v = LC * (DV + LP) * 4, square = LC * (LC + LP) * 4;
  auto go = [&](auto kernel, int smem, auto... a) {
    const cudaError_t f =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return f ? f : launch(kernel, grid, dim3(LN_NT), smem, c.st, 1, p.m, in, a...);
  };
  prof_mark(c.st, "lin_sum");
  e = back ? go(k_lin_sum<T, DK, DV, true>, rows_k + rows_v, p.whole, p.D, p.E)
           : go(k_lin_sum<T, DK, DV, false>, rows_k + rows_v, p.whole, p.D, p.E);
  if (e) return e;
  grid.z = 1;
  prof_mark(c.st, "lin_scan");
  e = launch(k_lin_scan, dim3((DK * DV / 4 + SC_NT - 1) / SC_NT, s.nseq * s.H, back ? 2 : 1),
             dim3(SC_NT), 0, c.st, 1, p.m, s.H, DK, DV, LIN_ROWS, p.whole, p.D, c.S_in, c.S_out,
             p.whole, p.E, c.dS_out, c.dS_in, false, p.status);
  if (e) return e;
  prof_mark(c.st, back ? "lin_grad" : "lin_out");
  e = back ? go(k_lin_grad<T, DK, DV>, 2 * (rows_k + rows_v + square), p.D, p.E, (T*)c.dq, (T*)c.dk,
                (T*)c.dv, (T*)c.dg, c.ddecay ? p.dgsum : nullptr)
           : go(k_lin_out<T, DK, DV>, 2 * rows_k + rows_v + square, p.D, (T*)c.o);
  if (e) return e;
  if (back && c.ddecay) e = col_sum(p.dgsum, p.m.cap, s.H, s.H, c.ddecay, nullptr, nullptr, c.st);
  return e;
}

gdn_status check_lin(const gdn_lin_shape* s) {
  if (!s || s->B < 1 || s->T < 0 || s->H < 1 || s->nseq < 1 || s->ldg < 0)
    return GDN_ERR_INVALID_ARG;
  if (!dtype_ok(s->dtype) || (s->dk != 64 && s->dk != 128) || (s->dv != 64 && s->dv != 128))
    return GDN_ERR_UNSUPPORTED;
  // rows are int; grids have the sequences' heads in y
  if ((long long)s->B * s->T > MOST_INDEX || (long long)s->nseq * s->H > 65535 ||
      (long long)s->nseq + s->T > MOST_INDEX)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// A call of one sequence may be packed or not.
size_t lin_bytes(const gdn_lin_shape& s, bool back) {
  size_t most = 0;
  for (const bool packed : {false, true})
    if (packed ? s.B == 1 : s.nseq == s.B)
      most = std::max(most, lin_tc_takes(s) ? lin_tc_bytes(s, packed, back) : lin_simt_bytes(s, packed, back));
  return most;
}

gdn_status run(const LinCall& c, size_t ws_bytes, bool back) {
  const gdn_lin_shape& s = c.s;
  if (c.cu ? s.B != 1 : s.nseq != s.B) return GDN_ERR_INVALID_ARG;
  const bool rows = s.T > 0;
  if ((rows && (!c.q || !c.k || !c.v || (!c.g && !c.decay))) || (c.g && c.decay))
    return GDN_ERR_INVALID_ARG;
  if (!vec_rows(c.q, s.ldq, s.dtype) || !vec_rows(c.k, s.ldk, s.dtype) ||
      !vec_rows(c.v, s.ldv, s.dtype) || !aligned(c.g, elem_size(s.dtype)) ||
      !aligned(c.decay, 4) || !aligned(c.S_in, 16) || !aligned(c.cu, 4))
    return GDN_ERR_INVALID_ARG;
  if (back) {
    if (rows && (!c.dout || !c.dq || !c.dk || !c.dv)) return GDN_ERR_INVALID_ARG;
    if ((rows && c.g && !c.dg) || !c.g != !c.dg || !c.decay != !c.ddecay) return GDN_ERR_INVALID_ARG;
    if (!aligned(c.dout, 16) || !aligned(c.dS_out, 16) || !aligned(c.dq, 16) ||
        !aligned(c.dk, 16) || !aligned(c.dv, 16) || !aligned(c.dg, elem_size(s.dtype)) ||
        !aligned(c.ddecay, 4) || !aligned(c.dS_in, 16))
      return GDN_ERR_INVALID_ARG;
  } else {
    if (rows && !c.o) return GDN_ERR_INVALID_ARG;
    if (!aligned(c.o, 16) || !aligned(c.S_out, 16)) return GDN_ERR_INVALID_ARG;
  }
  if (!c.ws || !aligned(c.ws, 256) || ws_bytes < lin_bytes(s, back)) return GDN_ERR_WORKSPACE;
  const cudaError_t e = lin_tc_takes(s) ? lin_tc(c, back) : lin_simt(c, back);
  prof_mark(c.st, nullptr);
  return e ? GDN_ERR_CUDA : GDN_OK;
}

}  // namespace

cudaError_t lin_plan(const LinMap& m, int* first, int* owner, int* order, int chunk, int* status,
                     cudaStream_t st) {
  prof_mark(st, "lin_plan");
  return launch(k_lin_plan, dim3(1), dim3(PL_NT), 0, st, 1, m, first, owner, order, chunk, status);
}

cudaError_t lin_scan(const LinMap& m, const gdn_lin_shape& s, const float* whole, float* D,
                     const float* S_in, float* E, const float* whole_e, const float* dS_out,
                     bool back, int* status, cudaStream_t st) {
  prof_mark(st, "lin_scan");
  return launch(k_lin_scan, dim3((s.dk * s.dv / 4 + SC_NT - 1) / SC_NT, s.nseq * s.H, back ? 2 : 1),
                dim3(SC_NT), 0, st, 1, m, s.H, s.dk, s.dv, LIN_KEYS, whole, D, S_in,
                (float*)nullptr, whole_e, E, dS_out, (float*)nullptr, true, status);
}

size_t lin_simt_bytes(const gdn_lin_shape& s, bool packed, bool back) {
  return simt_plan(s, nullptr, packed, back, nullptr).bytes;
}
cudaError_t lin_simt(const LinCall& c, bool back) {
  const bool k64 = c.s.dk == 64, v64 = c.s.dv == 64;
  if (c.s.dtype == GDN_DTYPE_BF16) {
    if (k64) return v64 ? run_simt<__nv_bfloat16, 64, 64>(c, back) : run_simt<__nv_bfloat16, 64, 128>(c, back);
    return v64 ? run_simt<__nv_bfloat16, 128, 64>(c, back) : run_simt<__nv_bfloat16, 128, 128>(c, back);
  }
  if (k64) return v64 ? run_simt<float, 64, 64>(c, back) : run_simt<float, 64, 128>(c, back);
  return v64 ? run_simt<float, 128, 64>(c, back) : run_simt<float, 128, 128>(c, back);
}

}  // namespace gdn

extern "C" {

size_t gdn_lin_workspace_bytes(const gdn_lin_shape* shape, int is_bwd) {
  using namespace gdn;
  if (check_lin(shape) != GDN_OK || (is_bwd != 0 && is_bwd != 1)) return 0;
  return lin_bytes(*shape, is_bwd != 0);
}

gdn_status gdn_lin_fwd(const gdn_lin_shape* shape, const void* q, const void* k, const void* v,
                       const void* g, const float* decay, const float* S_in,
                       const int* cu_seqlens, void* o, float* S_out, void* workspace,
                       size_t workspace_bytes, void* stream) {
  using namespace gdn;
  const gdn_status e = check_lin(shape);
  if (e != GDN_OK) return e;
  LinCall c = {*shape, q, k, v, g, decay, S_in, cu_seqlens, o, S_out};
  c.ws = (unsigned char*)workspace;
  c.st = (cudaStream_t)stream;
  return run(c, workspace_bytes, false);
}

gdn_status gdn_lin_bwd(const gdn_lin_shape* shape, const void* q, const void* k, const void* v,
                       const void* g, const float* decay, const float* S_in,
                       const int* cu_seqlens, const void* dout, const float* dS_out, void* dq,
                       void* dk, void* dv, void* dg, float* ddecay, float* dS_in,
                       void* workspace, size_t workspace_bytes, void* stream) {
  using namespace gdn;
  const gdn_status e = check_lin(shape);
  if (e != GDN_OK) return e;
  LinCall c = {*shape, q, k, v, g, decay, S_in, cu_seqlens, nullptr, nullptr, dout, dS_out,
               dq, dk, dv, dg, ddecay, dS_in, (unsigned char*)workspace, (cudaStream_t)stream};
  return run(c, workspace_bytes, true);
}

}  // extern "C"

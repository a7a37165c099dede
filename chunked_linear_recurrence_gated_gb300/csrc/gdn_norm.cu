// Norms of a Gated DeltaNet layer (include/gdn_layer.h): the gated RMS norm of
// each head's output (gdn_gate_norm_*) and the block boundary, i.e. post-norm,
// residual scale, addition and the next block's norm (gdn_res_norm_*).
#include <stdint.h>

#include <algorithm>

#include "gdn_layer.cuh"
#include "gdn_mma.cuh"

namespace gdn {
namespace {

constexpr int GN_NT = 256;     // threads of a block
constexpr int GN_U = 4;        // rows a thread has in flight (forward)
constexpr int GN_UB = 2;       // rows a thread has in flight (backward)
constexpr int GN_PARTS = 608;  // most partial sums of dw

// act(z) and its derivative
template <typename T>
__device__ __forceinline__ void gate(float z, int act, float& a, float& da) {
  const float s = sigmoid_as<T>(z);
  if (act == GDN_GATE_SILU) {
    a = z * s;
    da = s * (1.f + z * (1.f - s));
  } else {
    a = s;
    da = s * (1.f - s);
  }
}

// z of (token t, head h), row r = t H + h.
__device__ __forceinline__ size_t z_at(uint32_t r, const FastDiv& byH, int d, long long ldz) {
  uint32_t t, h;
  byH(r, t, h);
  return (size_t)t * ldz + (size_t)h * d;
}

// L lanes (a power of two >= d / 8) per row of d values, GN_U rows per thread.
template <typename T, int L>
__global__ void __launch_bounds__(GN_NT)
    k_gate_norm_fwd(uint32_t nrow, FastDiv byH, int d, float inv_d, int act, long long ldz,
                    float eps, const T* __restrict__ o, const T* __restrict__ z,
                    const float* __restrict__ w, T* __restrict__ y) {
  constexpr int NG = GN_NT / L;
  const int c = (threadIdx.x % L) * 8;
  const uint32_t r0 = blockIdx.x * (NG * GN_U) + threadIdx.x / L;
  Raw8<T> xr[GN_U], zr[GN_U];
#pragma unroll
  for (int u = 0; u < GN_U; ++u) {
    const uint32_t r = r0 + u * NG;
    xr[u] = zr[u] = Raw8<T>{};
    if (r < nrow && c < d) {
      xr[u] = ldraw8(o + (size_t)r * d + c);
      zr[u] = ldraw8(z + z_at(r, byH, d, ldz) + c);
    }
  }
  float wv[8] = {};
  if (c < d) ld8(w + c, wv);
#pragma unroll
  for (int u = 0; u < GN_U; ++u) {
    const uint32_t r = r0 + u * NG;
    float x[8], zz[8], ss = 0.f;
    cvt8(xr[u], x);
    cvt8(zr[u], zz);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    ss = lane_sum<L>(ss);
    const float rr = rsqrtf(fmaf(ss, inv_d, eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, da;
      gate<T>(zz[i], act, a, da);
      x[i] = x[i] * rr * (wv[i] * a);
    }
    if (r < nrow && c < d) st8(y + (size_t)r * d + c, x);
  }
}

// Blocks take every gridDim.x-th group of rows; each thread keeps the dw of its
// 8 columns, part[block] = the block's sum.
template <typename T, int L>
__global__ void __launch_bounds__(GN_NT, sizeof(T) == 2 ? GN_PARTS / 152 : 2)
    k_gate_norm_bwd(uint32_t nrow, FastDiv byH, int d, float inv_d, int act, long long ldz,
                    float eps, const T* __restrict__ o, const T* __restrict__ z,
                    const float* __restrict__ w, const T* __restrict__ dy, T* __restrict__ dout,
                    T* __restrict__ dz, float* __restrict__ part) {
  constexpr int NG = GN_NT / L;
  __shared__ float red[NG][L * 8];
  const int c = (threadIdx.x % L) * 8, gi = threadIdx.x / L;
  float acc[8] = {}, wv[8] = {};
  if (c < d) ld8(w + c, wv);
  for (uint32_t b = blockIdx.x * (NG * GN_UB); b < nrow; b += gridDim.x * (NG * GN_UB)) {
    Raw8<T> xr[GN_UB], zr[GN_UB], gr[GN_UB];
#pragma unroll
    for (int u = 0; u < GN_UB; ++u) {
      const uint32_t r = b + u * NG + gi;
      xr[u] = zr[u] = gr[u] = Raw8<T>{};
      if (r < nrow && c < d) {
        xr[u] = ldraw8(o + (size_t)r * d + c);
        zr[u] = ldraw8(z + z_at(r, byH, d, ldz) + c);
        gr[u] = ldraw8(dy + (size_t)r * d + c);
      }
    }
#pragma unroll
    for (int u = 0; u < GN_UB; ++u) {
      const uint32_t r = b + u * NG + gi;
      float x[8], zz[8], gy[8], go[8], ss = 0.f, sd = 0.f;
      cvt8(xr[u], x);
      cvt8(zr[u], zz);
      cvt8(gr[u], gy);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float a, da;
        gate<T>(zz[i], act, a, da);
        zz[i] = gy[i] * (wv[i] * da);
        gy[i] *= a;
        go[i] = gy[i] * wv[i];
        ss = fmaf(x[i], x[i], ss);
        sd = fmaf(go[i], x[i], sd);
      }
      ss = lane_sum<L>(ss);
      sd = lane_sum<L>(sd);
      const float rr = rsqrtf(fmaf(ss, inv_d, eps)), m = sd * rr * inv_d;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = x[i] * rr;
        go[i] = rr * fmaf(-n, m, go[i]);
        zz[i] *= n;
        acc[i] = fmaf(gy[i], n, acc[i]);
      }
      if (r < nrow && c < d) {
        st8(dout + (size_t)r * d + c, go);
        st8(dz + (size_t)r * d + c, zz);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) red[gi][c + i] = acc[i];
  __syncthreads();
  for (int i = threadIdx.x; i < d; i += GN_NT) {
    float a = 0.f;
    for (int u = 0; u < NG; ++u) a += red[u][i];
    part[(size_t)blockIdx.x * d + i] = a;
  }
}

// ------------------------------------------------------------ block boundary
// A team of threads works on one row, 8 columns per thread, so the parameters,
// the row and (backward) the columns' running sums stay in registers. Rows
// wider than RN_COLS are split over the CTAs of a cluster, which exchange their
// sums through distributed shared memory. Each thread prefetches its own 8
// columns of the team's next rows with cp.async into shared-memory slots that
// only it reads: the loads of several rows stay in flight across the two
// reductions of a row, without a barrier of their own.
constexpr int RN_COLS_F = 8192;  // columns of a CTA, forward: 1024 threads of 64 registers
constexpr int RN_COLS_B = 4096;  // backward: 512 threads of 128 registers
constexpr int RN_SLOT = 128;     // floats of a reduction: 8 values of 16 warps, or 1 of 32
constexpr int RN_SMS = 152;

struct Team {
  int C, c;         // row width, this thread's first column
  int rows, first, step;  // this team takes rows first, first + step, ..
  bool on;          // the thread has columns
};

// What a team's reductions go through; buf alternates between calls, so one
// barrier separates a call's reads from the next but one's writes.
template <int CL>
struct TeamRed {
  float* warp;     // [2][RN_SLOT] the warps' sums (unused ones stay 0)
  float4* cta;     // CL > 1: [2][CL][2] the CTAs' sums, written by their owners
  uint64_t* bar;   // CL > 1: [2] completed by CL such writes
  int buf, phase;  // of the next call
  bool dead;       // a wait gave up: every later sum is NaN, so the failure shows
};

// Sum over the warp of each of 8 values in 9 shuffles: each exchange halves the
// values that a lane still carries. Lane l returns value l / 4.
__device__ __forceinline__ float warp_sum8(const float* v) {
  const int lane = threadIdx.x & 31;
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 16;
    a[i] = (up ? v[4 + i] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[4 + i], 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 8;
    b[i] = (up ? a[2 + i] : a[i]) + __shfl_xor_sync(0xffffffffu, up ? a[i] : a[2 + i], 8);
  }
  const bool up = lane & 4;
  float c = (up ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, up ? b[0] : b[1], 4);
  c += __shfl_xor_sync(0xffffffffu, c, 2);
  return c + __shfl_xor_sync(0xffffffffu, c, 1);
}

// The sums of a row split over a cluster: each CTA writes its own (up to 8) into
// every CTA's shared memory with st.async, which also completes the receiver's
// mbarrier. (A cluster barrier instead would have to order the row's global
// stores too: its release waits for them, 6 us per row of 16384 columns against
// DRAM's 2.)
template <int K, int CL>
__device__ __forceinline__ void cluster_sum(float* v, TeamRed<CL>& red) {
  constexpr int N4 = K > 4 ? 2 : 1;  // float4 per CTA
  uint64_t* bar = red.bar + red.buf;
  float4* all = red.cta + red.buf * CL * 2;
  if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, CL * 16 * N4);
  if (threadIdx.x < CL) {
    uint32_t rank, to, tobar;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mapa.shared::cluster.u32 %0, %1, %2;"
        : "=r"(to)
        : "r"(smem_u32(all + 2 * rank)), "r"(threadIdx.x));
    asm("mapa.shared::cluster.u32 %0, %1, %2;"
        : "=r"(tobar)
        : "r"(smem_u32(bar)), "r"(threadIdx.x));
#pragma unroll
    for (int i = 0; i < N4; ++i) {
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = 4 * i + j < K ? v[4 * i + j] : 0.f;
      asm volatile(
          "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], "
          "{%1, %2, %3, %4}, [%5];" ::"r"(to + 16 * i),
          "f"(w[0]), "f"(w[1]), "f"(w[2]), "f"(w[3]), "r"(tobar)
          : "memory");
    }
  }
  const long long t0 = clock64();
  for (uint32_t ok = red.dead; !ok;) {
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"((uint32_t)red.phase)
        : "memory");
    if (!ok && clock64() - t0 > (1ll << 32)) ok = red.dead = true;
  }
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = red.dead ? __int_as_float(0x7fc00000) : 0.f;
#pragma unroll
  for (int r = 0; r < CL; ++r)
#pragma unroll
    for (int i = 0; i < N4; ++i) {
      const float4 a = all[2 * r + i];
      const float w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * i + j < K) v[4 * i + j] += w[j];
    }
  red.phase ^= red.buf;  // both buffers of this phase used: the next phase
}

// Sum over the team and, for rows split over a cluster, over its CTAs.
template <int CL>
__device__ __forceinline__ float team_sum(float v, TeamRed<CL>& red) {
  const int nt = blockDim.x;
  v = lane_sum<32>(v);
  if (CL > 1 || nt > 32) {
    float* slot = red.warp + red.buf * RN_SLOT;
    if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
    named_bar(threadIdx.y + 1, nt);
    v = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (u * 128 >= nt) break;
      const float4 a = reinterpret_cast<const float4*>(slot)[u];
      v += (a.x + a.y) + (a.z + a.w);
    }
  }
  if (CL > 1) cluster_sum<1, CL>(&v, red);
  red.buf ^= 1;
  return v;
}
// The same for 6 values (v has room for 8), teams of up to 16 warps.
template <int CL>
__device__ __forceinline__ void team_sum6(float* v, TeamRed<CL>& red) {
  const int nt = blockDim.x, lane = threadIdx.x & 31;
  v[6] = v[7] = 0.f;
  float mine = warp_sum8(v);
  if (CL > 1 || nt > 32) {
    float* slot = red.warp + red.buf * RN_SLOT;  // [8 values][16 warps]
    if ((lane & 3) == 0) slot[(lane >> 2) * 16 + (threadIdx.x >> 5)] = mine;
    named_bar(threadIdx.y + 1, nt);
    // lane l: value l / 4, warps 4 (l % 4) ..
    const float4 a = reinterpret_cast<const float4*>(slot)[lane];
    mine = (a.x + a.y) + (a.z + a.w);
    mine += __shfl_xor_sync(0xffffffffu, mine, 1);
    mine += __shfl_xor_sync(0xffffffffu, mine, 2);
  }
#pragma unroll
  for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xffffffffu, mine, 4 * i);
  if (CL > 1) cluster_sum<6, CL>(v, red);
  red.buf ^= 1;
}

// A CTA that exits must not be written to any more: every CTA of the cluster
// has received all sums.
template <int CL>
__device__ __forceinline__ void team_end() {
  if (CL > 1) {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}

template <int CL>
__device__ __forceinline__ Team team_of(int rows, int C, TeamRed<CL>& red) {
  __shared__ __align__(16) float warp_sums[8 * 2 * RN_SLOT];  // at most 8 teams
  __shared__ float4 cta_sums[2 * CL * 2];
  __shared__ uint64_t bars[2];
  Team t;
  t.C = C;
  t.rows = rows;
  const int per = (C / 8 + CL - 1) / CL;  // column groups of a CTA
  const int rank = CL == 1 ? 0 : blockIdx.x % CL;
  t.c = (rank * per + threadIdx.x) * 8;
  t.on = (int)threadIdx.x < per && t.c < C;
  t.first = blockIdx.x / CL * blockDim.y + threadIdx.y;
  t.step = gridDim.x / CL * blockDim.y;
  red.warp = warp_sums + threadIdx.y * 2 * RN_SLOT;
  red.cta = cta_sums;
  red.bar = bars;
  red.buf = red.phase = 0;
  red.dead = false;
  for (int i = threadIdx.x; i < 2 * RN_SLOT; i += blockDim.x) red.warp[i] = 0.f;
  if (CL > 1) {
    if (threadIdx.x == 0) {
      mbar_init(bars, 1);
      mbar_init(bars + 1, 1);
      fence_mbar_init();
    }
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    named_bar(threadIdx.y + 1, blockDim.x);
  }
  return t;
}

// Prefetch slots of a thread: slot k of stage s, 16 bytes each, consecutive
// threads consecutive. E elements of 16-byte pieces per tensor.
template <int SLOTS>
struct Ring {
  uint4* base;  // this thread's slot 0 of stage 0
  int nt;
  __device__ __forceinline__ uint4* at(int stage, int k) const {
    return base + (size_t)(stage * SLOTS + k) * nt;
  }
  template <typename T>
  __device__ __forceinline__ void fetch(int stage, int k, const T* p) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      const uint4* src = reinterpret_cast<const uint4*>(p) + i;
      if (sizeof(T) == 2)
        cp16(at(stage, k + i), src, true);
      else  // through L1: the two halves of a sector are fetched by two instructions
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;\n" ::"r"(
                         smem_u32(at(stage, k + i))),
                     "l"(src));
    }
  }
  template <typename T>
  __device__ __forceinline__ void read(int stage, int k, f32x2* v) const {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.u[i] = *at(stage, k + i);
    cvt8(r, v);
  }
};

template <typename T>
constexpr int pieces() { return (int)sizeof(T) / 2; }  // 16-byte pieces of 8 elements
template <typename T, typename R>
constexpr int fwd_slots() { return pieces<R>() + pieces<T>(); }
template <typename T, typename R>
constexpr int fwd_stages() { return fwd_slots<T, R>() == 2 ? 4 : 3; }
template <typename T, typename R>
constexpr int bwd_slots() { return 2 * pieces<R>() + 2 * pieces<T>(); }
template <typename T, typename R>
constexpr int bwd_stages() { return bwd_slots<T, R>() == 4 ? 4 : 3; }

__device__ __forceinline__ void ld8_or(const float* p, bool have, float other, f32x2* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = both2(other);
  if (have) cvt8(ldraw8(p), v);
}

template <typename T, typename R, int CL>
__global__ void __launch_bounds__(1024, 1)
    k_res_norm_fwd(int rows, int C, float inv_C, float eps, const R* h, const T* __restrict__ x,
                   const float* __restrict__ w, const float* __restrict__ w_post,
                   const float* __restrict__ scale, R* h_out, T* __restrict__ y) {
  constexpr int S = fwd_stages<T, R>(), KX = pieces<R>();
  extern __shared__ uint4 smem[];
  const int nt = blockDim.x * blockDim.y;
  Ring<fwd_slots<T, R>()> ring = {smem + threadIdx.y * blockDim.x + threadIdx.x, nt};
  TeamRed<CL> red;
  const Team t = team_of<CL>(rows, C, red);
  auto fetch = [&](int stage, int row) {
    if (t.on && row < t.rows) {
      const size_t at = (size_t)row * C + t.c;
      ring.template fetch<R>(stage, 0, h + at);
      if (x) ring.template fetch<T>(stage, KX, x + at);
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < S; ++s) fetch(s, t.first + s * t.step);
  f32x2 wv[4], pv[4], sv[4];
  ld8_or(w + t.c, t.on, 0.f, wv);
  ld8_or(w_post + t.c, t.on && w_post, 1.f, pv);
  ld8_or(scale + t.c, t.on && scale, 1.f, sv);
  int stage = 0;
  for (int row = t.first; row < t.rows; row += t.step) {
    cp_wait<S - 1>();
    f32x2 hv[4] = {}, xv[4] = {};
    if (t.on) {
      ring.template read<R>(stage, 0, hv);
      if (x) ring.template read<T>(stage, KX, xv);
    }
    const size_t at = (size_t)row * C + t.c;
    if (w_post) {
      f32x2 a = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) a = fma2(xv[i], xv[i], a);
      const f32x2 rx = both2(rsqrtf(fmaf(team_sum(sum2(a), red), inv_C, eps)));
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[i] = mul2(xv[i], mul2(rx, pv[i]));
    }
    f32x2 a = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hv[i] = fma2(sv[i], xv[i], hv[i]);
      a = fma2(hv[i], hv[i], a);
    }
    if (h_out && t.on) st8(h_out + at, hv);
    fetch(stage, row + S * t.step);  // the slot has been read
    if (++stage == S) stage = 0;
    const f32x2 r = both2(rsqrtf(fmaf(team_sum(sum2(a), red), inv_C, eps)));
#pragma unroll
    for (int i = 0; i < 4; ++i) hv[i] = mul2(hv[i], mul2(r, wv[i]));
    if (t.on) st8(y + at, hv);
  }
  cp_wait<0>();
  team_end<CL>();
}

// part [blocks][1 + (w_post) + (scale)][C]: the blocks' sums of dw, dw_post, dscale.
template <typename T, typename R, int CL>
__global__ void __launch_bounds__(512, 1)
    k_res_norm_bwd(int rows, int C, float inv_C, float eps, const R* __restrict__ h,
                   const T* __restrict__ x, const float* __restrict__ w,
                   const float* __restrict__ w_post, const float* __restrict__ scale,
                   const T* __restrict__ dy, const R* dh_out, R* dh, T* __restrict__ dx,
                   float* __restrict__ part) {
  constexpr int S = bwd_stages<T, R>(), KD = pieces<R>(), KG = 2 * pieces<R>(),
                KX = KG + pieces<T>();
  extern __shared__ uint4 smem[];
  const int nt = blockDim.x * blockDim.y;
  Ring<bwd_slots<T, R>()> ring = {smem + threadIdx.y * blockDim.x + threadIdx.x, nt};
  TeamRed<CL> red;
  const Team t = team_of<CL>(rows, C, red);
  const bool with_x = w_post || scale;
  auto fetch = [&](int stage, int row) {
    if (t.on && row < t.rows) {
      const size_t at = (size_t)row * C + t.c;
      ring.template fetch<R>(stage, 0, h + at);
      if (dh_out) ring.template fetch<R>(stage, KD, dh_out + at);
      ring.template fetch<T>(stage, KG, dy + at);
      if (with_x) ring.template fetch<T>(stage, KX, x + at);
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < S; ++s) fetch(s, t.first + s * t.step);
  f32x2 wv[4], sp[4], aw[4] = {}, am[4] = {};  // sp = scale w_post
  ld8_or(w + t.c, t.on, 0.f, wv);
  ld8_or(scale + t.c, t.on && scale, 1.f, sp);
  if (w_post) {
    f32x2 pv[4];
    ld8_or(w_post + t.c, t.on, 0.f, pv);
#pragma unroll
    for (int i = 0; i < 4; ++i) sp[i] = mul2(sp[i], pv[i]);
  }
  int stage = 0;
  for (int row = t.first; row < t.rows; row += t.step) {
    cp_wait<S - 1>();
    f32x2 hv[4] = {}, gw[4] = {}, xv[4] = {}, dv[4] = {}, a[6] = {};
    f32x2 gv[4] = {};
    if (t.on) {
      ring.template read<R>(stage, 0, hv);
      if (dh_out) ring.template read<R>(stage, KD, dv);
      ring.template read<T>(stage, KG, gv);
      if (with_x) ring.template read<T>(stage, KX, xv);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      gw[i] = mul2(gv[i], wv[i]);
      a[0] = fma2(hv[i], hv[i], a[0]);
      a[1] = fma2(gw[i], hv[i], a[1]);
    }
    if (w_post) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2 q = mul2(sp[i], xv[i]);
        a[2] = fma2(xv[i], xv[i], a[2]);
        a[3] = fma2(q, dv[i], a[3]);
        a[4] = fma2(q, gw[i], a[4]);
        a[5] = fma2(q, hv[i], a[5]);
      }
    }
    fetch(stage, row + S * t.step);  // the slot has been read
    if (++stage == S) stage = 0;
    float s[8];
#pragma unroll
    for (int i = 0; i < 6; ++i) s[i] = sum2(a[i]);
    team_sum6(s, red);
    const size_t at = (size_t)row * C + t.c;
    const float r = rsqrtf(fmaf(s[0], inv_C, eps));
    const float rx = w_post ? rsqrtf(fmaf(s[2], inv_C, eps)) : 1.f;
    const float hc = -r * r * r * s[1] * inv_C;  // factor of h in dh
    const f32x2 r2 = both2(r), hc2 = both2(hc), rx2 = both2(rx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      aw[i] = fma2(gv[i], mul2(hv[i], r2), aw[i]);
      dv[i] = fma2(hv[i], hc2, fma2(gw[i], r2, dv[i]));  // dh
      xv[i] = mul2(xv[i], rx2);                          // m
      am[i] = fma2(dv[i], xv[i], am[i]);
    }
    if (t.on) st8(dh + at, dv);
    if (dx) {
      if (w_post) {
        // mean(sp dh m) from the sums of its terms
        const f32x2 e = both2(-rx * inv_C * fmaf(hc, s[5], fmaf(r, s[4], s[3])));
#pragma unroll
        for (int i = 0; i < 4; ++i) dv[i] = mul2(rx2, fma2(xv[i], e, mul2(dv[i], sp[i])));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) dv[i] = mul2(dv[i], sp[i]);
      }
      if (t.on) st8(dx + at, dv);
    }
  }
  cp_wait<0>();
  team_end<CL>();
  // the block's sums, teams joined through shared memory (the ring is drained);
  // sum dh m times scale is dw_post, times w_post dscale
  float* mine = reinterpret_cast<float*>(smem) + (threadIdx.y * blockDim.x + threadIdx.x) * 8;
  const int narr = 1 + (w_post != nullptr) + (scale != nullptr);
  float* out = part + (size_t)(blockIdx.x / CL) * narr * C + t.c;
  auto join = [&](f32x2* v) {
    if (blockDim.y == 1) return;
    __syncthreads();
    st8(mine, v);
    __syncthreads();
    if (threadIdx.y) return;
    for (int u = 1; u < (int)blockDim.y; ++u) {
      f32x2 o[4];
      cvt8(ldraw8(mine + (size_t)u * blockDim.x * 8), o);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = add2(v[i], o[i]);
    }
  };
  join(aw);
  if (with_x) join(am);
  if (threadIdx.y || !t.on) return;
  st8(out, aw);
  if (w_post) {
    f32x2 sv[4];
    ld8_or(scale + t.c, scale, 1.f, sv);
#pragma unroll
    for (int i = 0; i < 4; ++i) sv[i] = mul2(am[i], sv[i]);
    st8(out += C, sv);
  }
  if (scale) {
    f32x2 pv[4];
    ld8_or(w_post + t.c, w_post, 1.f, pv);
#pragma unroll
    for (int i = 0; i < 4; ++i) pv[i] = mul2(am[i], pv[i]);
    st8(out += C, pv);
  }
}

// ------------------------------------------------------------------ host side
gdn_status check_gate(const gdn_gate_norm_shape* s) {
  if (!s || s->rows < 0 || s->H < 1 || s->d < 1 || !(s->eps > 0.f)) return GDN_ERR_INVALID_ARG;
  if (s->act != GDN_GATE_SILU && s->act != GDN_GATE_SIGMOID) return GDN_ERR_INVALID_ARG;
  if (!dtype_ok(s->dtype) || s->d % 8 || s->d > 256 || s->H > (1 << 16))
    return GDN_ERR_UNSUPPORTED;
  if ((long long)s->rows * s->H >= (1ll << 31)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}
int lanes_of(int d) {
  int L = 1;
  while (L * 8 < d) L *= 2;
  return L;
}
int gate_parts(const gdn_gate_norm_shape& s) {
  const long long g = GN_NT / lanes_of(s.d) * GN_UB, n = (long long)s.rows * s.H;
  return (int)std::min<long long>(GN_PARTS, (n + g - 1) / g);
}

template <typename T, int L>
void launch_gate(const gdn_gate_norm_shape& s, const void* o, const void* z, const float* w,
                 const void* dy, void* out, void* dz, float* part, cudaStream_t st) {
  const uint32_t n = (uint32_t)s.rows * (uint32_t)s.H, per = GN_NT / L * GN_U;
  const FastDiv byH(s.H);
  const float inv = 1.f / (float)s.d;
  if (!dy)
    k_gate_norm_fwd<T, L><<<(n + per - 1) / per, GN_NT, 0, st>>>(
        n, byH, s.d, inv, s.act, s.ldz, s.eps, (const T*)o, (const T*)z, w, (T*)out);
  else
    k_gate_norm_bwd<T, L><<<gate_parts(s), GN_NT, 0, st>>>(n, byH, s.d, inv, s.act, s.ldz, s.eps,
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

// How a call's rows are laid out over CTAs; a function of the shape alone, so
// the order of the parameter gradients' sums is too.
struct ResPlan {
  int cl, team, teams;  // CTAs per row, threads of a CTA per row, rows per CTA
  int blocks(int rows, int threads) const {  // CTAs, so that each SM has up to `threads`
    const int all = (rows + teams - 1) / teams;
    return cl * std::min(all, std::max(1, RN_SMS * (threads / (team * teams)) / cl));
  }
};
ResPlan res_plan(int C, int cols) {
  ResPlan p;
  p.cl = C <= cols ? 1 : C <= 2 * cols ? 2 : 4;
  const int groups = (C / 8 + p.cl - 1) / p.cl;
  p.team = (groups + 31) / 32 * 32;
  p.teams = p.team >= 256 || p.cl > 1 ? 1 : 256 / p.team;
  return p;
}
int res_parts(const gdn_res_norm_shape& s) {
  const ResPlan p = res_plan(s.C, RN_COLS_B);
  return p.blocks(s.rows, 512) / p.cl;
}

struct ResArgs {
  const void *h, *x, *dy, *dh_out;
  const float *w, *w_post, *scale;
  void *ho, *y;  // forward: h_out, y; backward: dh, dx
  float* part;
};
template <typename K, typename... A>
cudaError_t launch_rows(K kernel, const ResPlan& p, int blocks, int smem, cudaStream_t st,
                        A... args) {
  if (smem > 32 << 10) {  // with the static part, past what needs no asking
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(p.team, p.teams);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = p.cl;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.cl > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename T, typename R, int CL>
cudaError_t launch_res(const gdn_res_norm_shape& s, const ResArgs& a, const ResPlan& p,
                       cudaStream_t st) {
  const int nt = p.team * p.teams;
  const float inv = 1.f / (float)s.C;
  if (!a.dy)
    return launch_rows(k_res_norm_fwd<T, R, CL>, p, p.blocks(s.rows, 1024),
                       nt * 16 * fwd_slots<T, R>() * fwd_stages<T, R>(), st, s.rows, s.C, inv,
                       s.eps, (const R*)a.h, (const T*)a.x, a.w, a.w_post, a.scale, (R*)a.ho,
                       (T*)a.y);
  return launch_rows(k_res_norm_bwd<T, R, CL>, p, p.blocks(s.rows, 512),
                     nt * 16 * bwd_slots<T, R>() * bwd_stages<T, R>(), st, s.rows, s.C, inv,
                     s.eps, (const R*)a.h, (const T*)a.x, a.w, a.w_post, a.scale,
                     (const T*)a.dy, (const R*)a.dh_out, (R*)a.ho, (T*)a.y, a.part);
}
template <typename T, typename R>
cudaError_t dispatch_res(const gdn_res_norm_shape& s, const ResArgs& a, cudaStream_t st) {
  const ResPlan p = res_plan(s.C, a.dy ? RN_COLS_B : RN_COLS_F);
  switch (p.cl) {
    case 1: return launch_res<T, R, 1>(s, a, p, st);
    case 2: return launch_res<T, R, 2>(s, a, p, st);
    default: return launch_res<T, R, 4>(s, a, p, st);
  }
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
  const int narr = 1 + (w_post != nullptr) + (scale != nullptr);
  const cudaError_t ce = col_sum(part, res_parts(s), narr * s.C, s.C, dw,
                                 w_post ? dw_post : dscale, dscale, st);
  prof_mark(st, nullptr);
  return ce ? GDN_ERR_CUDA : GDN_OK;
}

}  // extern "C"

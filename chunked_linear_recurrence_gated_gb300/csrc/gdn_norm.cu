// Norms of a Gated DeltaNet layer (include/gdn_layer.h): the gated RMS norm of
// each head's output (gdn_gate_norm_*) and the block boundary, i.e. post-norm,
// residual scale, addition and the next block's norm (gdn_res_norm_*).
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "../../include/gdn_profile.h"
#include "gdn_layer.cuh"
#include "gdn_mma.cuh"

namespace gdn {
namespace {

constexpr int GN_NT = 256;     // threads of a block
constexpr int GN_U = 4;        // rows a thread has in flight (forward)
constexpr int GN_UB = 2;       // rows a thread has in flight (backward)
// Blocks of the backward on an SM: bf16 3 of 80 registers, fp32 2; its grid is one
// wave of them (bf16; 4 blocks of 64 registers spill, 110 us against 106) or two.
template <typename T>
constexpr int gate_blocks() { return sizeof(T) == 2 ? 3 : 2; }

template <typename T>
__device__ __forceinline__ float gate(float z, int act) {
  const float s = sigmoid_as<T>(z);
  return act == GDN_GATE_SILU ? z * s : s;
}

// z of (token t, head h), row r = t H + h.
__device__ __forceinline__ size_t z_at(uint32_t r, const FastDiv& byH, int d, long long ldz) {
  uint32_t t, h;
  byH(r, t, h);
  return (size_t)t * ldz + (size_t)h * d;
}

// L lanes (a power of two >= d / 8) per row of d values, GN_U rows per thread, all
// loaded before the first is used. Bound by the bytes of o, z and y: 131072 x 16
// rows of 128 bf16 values 224 us (1.61 GB, 7.2 TB/s).
template <typename T, int L>
__global__ void __launch_bounds__(GN_NT)
    k_gate_norm_fwd(uint32_t nrow, FastDiv byH, int d, float inv_d, int act, long long ldz,
                    float eps, const T* o, const T* z, const float* w, T* y) {
  chain();
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
      x[i] = x[i] * rr * (wv[i] * gate<T>(zz[i], act));
    }
    if (r < nrow && c < d) st8(y + (size_t)r * d + c, x);
  }
}

// Blocks take every gridDim.x-th group of rows; each thread keeps the dw of its 8
// columns, part[block] = the block's sum. The elementwise arithmetic is in pairs:
// the instructions of an element (sigmoid and its derivative among them) come
// close to the memory's time. Bound by the bytes of o, z, dy, do and dz: 16411 x 16
// rows of 256 bf16 values 106 us (672 MB, 6.3 TB/s; 110 with unpaired arithmetic,
// 126 with the next rows in flight through shared memory).
template <typename T, int L>
__global__ void __launch_bounds__(GN_NT, gate_blocks<T>())
    k_gate_norm_bwd(uint32_t nrow, FastDiv byH, int d, float inv_d, int act, long long ldz,
                    float eps, const T* o, const T* z, const float* w, const T* dy, T* dout, T* dz,
                    float* part) {
  constexpr int NG = GN_NT / L;
  __shared__ __align__(16) float red[NG][L * 8];
  chain();
  let_next_start();
  const int c = (threadIdx.x % L) * 8, gi = threadIdx.x / L;
  f32x2 acc[4] = {}, wv[4] = {};
  if (c < d) cvt8(ldraw8(w + c), wv);
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
      f32x2 x[4], ga[4], go[4], gz[4], ss = 0, sd = 0;
      {
        float zz[8];
        f32x2 gy[4];
        cvt8(xr[u], x);
        cvt8(zr[u], zz);
        cvt8(gr[u], gy);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float s0, s1, t0, t1;
          sigmoid_pair<T>(zz[2 * i], s0, t0);
          sigmoid_pair<T>(zz[2 * i + 1], s1, t1);
          const f32x2 s = pack2(s0, s1), t = pack2(t0, t1);
          f32x2 a = s, da = mul2(s, t);
          if (act == GDN_GATE_SILU) {
            a = mul2(s, pack2(zz[2 * i], zz[2 * i + 1]));
            da = fma2(a, t, s);  // s (1 + z (1 - s))
          }
          gz[i] = mul2(mul2(gy[i], wv[i]), da);
          ga[i] = mul2(gy[i], a);
          go[i] = mul2(ga[i], wv[i]);
          ss = fma2(x[i], x[i], ss);
          sd = fma2(go[i], x[i], sd);
        }
      }
      const float s1 = lane_sum<L>(sum2(ss)), s2 = lane_sum<L>(sum2(sd));
      const float rr = rsqrtf(fmaf(s1, inv_d, eps));
      // n = x r; do = r (go - n mean(go n)); dz = gz n; dw += ga n
      const f32x2 r2 = both2(rr), m2 = both2(-s2 * rr * rr * inv_d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2 n = mul2(x[i], r2);
        go[i] = fma2(n, m2, mul2(go[i], r2));
        gz[i] = mul2(gz[i], n);
        acc[i] = fma2(ga[i], n, acc[i]);
      }
      if (r < nrow && c < d) {
        st8(dout + (size_t)r * d + c, go);
        st8(dz + (size_t)r * d + c, gz);
      }
    }
  }
  st8(&red[gi][c], acc);
  __syncthreads();
  for (int i = threadIdx.x; i < d; i += GN_NT) {
    float a = 0.f;
    for (int u = 0; u < NG; ++u) a += red[u][i];
    part[(size_t)blockIdx.x * d + i] = a;
  }
}

// ------------------------------------------------------------ block boundary
// A team of threads works on one row, 8 columns per thread, so the parameters,
// the row and (backward) the columns' running sums stay in registers. Rows wider
// than a CTA are split over the CTAs of a cluster, which exchange their sums
// through distributed shared memory. Each thread prefetches its own columns of
// the team's next rows with cp.async into shared-memory slots that only it
// reads: the loads of several rows stay in flight across a row's reductions,
// without a barrier of their own.
constexpr int RN_COLS_F = 8192;  // columns of a CTA, forward: 1024 threads of 64 registers
constexpr int RN_COLS_B = 4096;  // backward: 512 threads of 128 registers
constexpr int RN_SLOT = 128;     // floats of a reduction: 8 values of 16 warps, or 2 of 32
constexpr int RN_STAGES_B = 3;   // rows a team holds, backward (4 to 6: no faster)
constexpr int RN_SMS = 152;
constexpr long long RN_WAIT = 1ll << 32;  // SM clock cycles (two seconds) that a wait may take
constexpr long long RN_HOLD = 1ll << 26;  // and that a CTA stays after one that ran out

// Set by a wait that ran out, read and cleared by gdn_layer_status.
__device__ int g_exchange_status;

// The rows of a team and the columns of a thread. With an fp32 stream a
// thread's columns are two groups of 4 that lie a team apart, so that a warp's
// 16-byte accesses are whole lines (8 consecutive ones make twice the requests:
// backward, fp32, 4096 columns 176 us instead of 140); otherwise 8 consecutive.
template <bool SPLIT>
struct Team {
  int C, rows, first, step;  // this team takes rows first, first + step, ..
  int c0, c1;                // first columns of the two groups of 4
  bool on0, on1;             // whether they exist
};

template <bool SPLIT, int CL>
__device__ __forceinline__ Team<SPLIT> team_of(int rows, int C) {
  Team<SPLIT> t;
  t.C = C;
  t.rows = rows;
  const int per = (C / 8 + CL - 1) / CL * 8;  // columns of a CTA
  const int base = CL == 1 ? 0 : blockIdx.x % CL * per, end = min(base + per, C);
  t.c0 = base + (SPLIT ? 4 : 8) * threadIdx.x;
  t.c1 = SPLIT ? t.c0 + 4 * blockDim.x : t.c0 + 4;
  t.on0 = t.c0 < end;
  t.on1 = t.c1 < end;
  t.first = blockIdx.x / CL * blockDim.y + threadIdx.y;
  t.step = gridDim.x / CL * blockDim.y;
  return t;
}

// 4 values of an fp32 row, or `other`.
__device__ __forceinline__ void ld4_or(const float* p, bool have, float other, f32x2* v) {
  v[0] = v[1] = both2(other);
  if (have) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = pack2(a.x, a.y);
    v[1] = pack2(a.z, a.w);
  }
}
__device__ __forceinline__ void st4(float* p, const f32x2* v) {
  *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(v[0], v[1]);
}
__device__ __forceinline__ void st4(__nv_bfloat16* p, const f32x2* v) {
  float f[4];
  unpack2(v[0], f[0], f[1]);
  unpack2(v[1], f[2], f[3]);
  const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
// A thread's columns of a parameter row (`other` without one) and of an output row.
template <bool SPLIT>
__device__ __forceinline__ void ld_cols(const float* p, const Team<SPLIT>& t, float other,
                                        f32x2* v) {
  ld4_or(p + t.c0, p && t.on0, other, v);
  ld4_or(p + t.c1, p && t.on1, other, v + 2);
}
template <bool SPLIT, typename T>
__device__ __forceinline__ void st_cols(T* p, const Team<SPLIT>& t, const f32x2* v) {
  if (SPLIT || sizeof(T) == 4) {
    if (t.on0) st4(p + t.c0, v);
    if (t.on1) st4(p + t.c1, v + 2);
  } else if (t.on0) {
    st8(p + t.c0, v);
  }
}

// Prefetch slots of a thread: slot k of stage s, 16 bytes each, consecutive
// threads consecutive. 8 bf16 values take one, 8 fp32 values two.
template <int SLOTS, bool SPLIT>
struct Ring {
  uint4* base;  // this thread's slot 0 of stage 0
  int nt;
  __device__ __forceinline__ uint4* at(int stage, int k) const {
    return base + (size_t)(stage * SLOTS + k) * nt;
  }
  __device__ __forceinline__ void clear(int stages) const {  // what no fetch writes reads as 0
    for (int i = 0; i < stages * SLOTS; ++i) base[(size_t)i * nt] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void fetch(int stage, int k, const float* p,
                                        const Team<SPLIT>& t) const {
    if (t.on0) cp16(at(stage, k), p + t.c0, true);
    if (t.on1) cp16(at(stage, k + 1), p + t.c1, true);
  }
  __device__ __forceinline__ void fetch(int stage, int k, const __nv_bfloat16* p,
                                        const Team<SPLIT>& t) const {
    if (!SPLIT) {
      if (t.on0) cp16(at(stage, k), p + t.c0, true);
      return;
    }
    const uint32_t to = smem_u32(at(stage, k));
    if (t.on0)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(to), "l"(p + t.c0)
                   : "memory");
    if (t.on1)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(to + 8), "l"(p + t.c1)
                   : "memory");
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
constexpr int bwd_slots() { return 2 * pieces<R>() + 2 * pieces<T>(); }
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

// Sums over a team of K values (1, 2 or 6), in two halves: post() gives this
// thread's part, collect() returns the sums of the oldest post not yet collected;
// AHEAD other posts lie between the two. A CTA of a cluster posts p after it has
// collected p - AHEAD - 1, so every other CTA has posted that, so it has collected
// p - 2 AHEAD - 2: what lies in the buffer of post p - BUFS has been read.
// For rows split over a cluster post() also sends the CTA's sums into every
// CTA's shared memory with st.async, which completes the receiver's mbarrier. (A
// cluster barrier instead would have to order the row's global stores too: its
// release waits for them, 6 us per row of 16384 columns against DRAM's 2.)
// A thread whose wait runs out sets g_exchange_status, takes every later sum as NaN
// and sends no more: a send of post p relies on its thread having collected
// p - AHEAD - 1. The other CTAs' waits then run out too, and all reach end().
template <int K, int CL, int AHEAD>
struct TeamSum {
  static constexpr int N4 = K > 4 ? 2 : 1;  // float4 per CTA's sums
  // 2 AHEAD + 2, and a third where two would do (forward, 5000 rows of 16384 bf16
  // columns: 112 us with three, 130 with two)
  static constexpr int BUFS = AHEAD > 0 ? 2 * AHEAD + 2 : 3;
  float* warps;    // [BUFS][RN_SLOT] the warps' sums (unused ones stay 0)
  float4* ctas;    // [BUFS][CL][N4] the CTAs' sums
  uint64_t* bars;  // [BUFS] completed by CL sends
  int in, out;     // buffers of the next post and the next collect
  uint32_t phase;  // parity of the mbarrier of `out`
  bool dead;       // this thread's wait ran out
  long long limit = RN_WAIT;

  __device__ __forceinline__ void init() {
    constexpr int TEAMS = CL > 1 ? 1 : 8;  // at most
    __shared__ __align__(16) float warp_sums[TEAMS * BUFS * RN_SLOT];
    __shared__ float4 cta_sums[BUFS * CL * N4];
    __shared__ uint64_t mbars[BUFS];
    warps = warp_sums + threadIdx.y * BUFS * RN_SLOT;
    ctas = cta_sums;
    bars = mbars;
    in = out = 0;
    phase = 0;
    dead = false;
    for (int i = threadIdx.x; i < BUFS * RN_SLOT; i += blockDim.x) warps[i] = 0.f;
    if (CL > 1) {
      if (threadIdx.x == 0) {
        for (int i = 0; i < BUFS; ++i) mbar_init(mbars + i, 1);
        fence_mbar_init();
      }
      __syncthreads();
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
      named_bar(threadIdx.y + 1, blockDim.x);
    }
  }
  // A CTA that exits must not be written to any more. Past the barrier no CTA of the
  // cluster sends, and whoever has collected all sums has received all sends to its
  // CTA; a thread that gave up does not know that, and stays for far longer than a
  // send can be under way.
  __device__ __forceinline__ void end() {
    if (CL > 1) {
      __syncwarp();
      asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      if (dead) {
        const long long t0 = clock64();
        while (clock64() - t0 < RN_HOLD) {
        }
      }
    }
  }
  __device__ __forceinline__ bool arrived() const {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bars + out)), "r"(phase)
        : "memory");
    return ok != 0;
  }
  // One more try after the time is up: a CTA that was not running meanwhile may find
  // that the sends have long landed.
  __device__ __forceinline__ void wait() {
    if (dead || arrived()) return;
    const long long t0 = clock64();
    for (;;) {
      const bool late = clock64() - t0 > limit;
      if (arrived()) return;
      if (late) break;
    }
    dead = true;
    *(volatile int*)&g_exchange_status = DEV_TIMEOUT;
  }
  // The CTA's sums from the warps'.
  __device__ __forceinline__ void read_warps(int buf, float* v) const {
    const float4* slot = reinterpret_cast<const float4*>(warps + buf * RN_SLOT);
    if (K <= 2) {
#pragma unroll
      for (int i = 0; i < K; ++i) v[i] = 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (u * 128 >= (int)blockDim.x) break;
#pragma unroll
        for (int i = 0; i < K; ++i) {
          const float4 a = slot[8 * i + u];
          v[i] += (a.x + a.y) + (a.z + a.w);
        }
      }
    } else {  // lane l: value l / 4, warps 4 (l % 4) ..
      const float4 a = slot[threadIdx.x & 31];
      float s = (a.x + a.y) + (a.z + a.w);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
#pragma unroll
      for (int i = 0; i < K; ++i) v[i] = __shfl_sync(0xffffffffu, s, 4 * i);
    }
  }
  __device__ __forceinline__ void post(float* v) {
    const int lane = threadIdx.x & 31;
    float* slot = warps + in * RN_SLOT;
    if (K <= 2) {
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const float s = lane_sum<32>(v[i]);
        if (lane == 0) slot[32 * i + (threadIdx.x >> 5)] = s;
      }
    } else {  // [8 values][16 warps]
      v[6] = v[7] = 0.f;
      const float s = warp_sum8(v);
      if ((lane & 3) == 0) slot[(lane >> 2) * 16 + (threadIdx.x >> 5)] = s;
    }
    if (blockDim.x > 32)
      named_bar(threadIdx.y + 1, blockDim.x);
    else
      __syncwarp();
    if (CL > 1 && threadIdx.x < 32) {
      float s[8] = {};
      read_warps(in, s);
      if (lane == 0 && !dead) mbar_arrive_expect_tx(bars + in, CL * 16 * N4);
      if (lane < CL && !dead) {
        uint32_t rank, to, bar;
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        asm("mapa.shared::cluster.u32 %0, %1, %2;"
            : "=r"(to)
            : "r"(smem_u32(ctas + (in * CL + rank) * N4)), "r"(lane));
        asm("mapa.shared::cluster.u32 %0, %1, %2;"
            : "=r"(bar)
            : "r"(smem_u32(bars + in)), "r"(lane));
#pragma unroll
        for (int i = 0; i < N4; ++i)
          asm volatile(
              "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], "
              "{%1, %2, %3, %4}, [%5];" ::"r"(to + 16 * i),
              "f"(s[4 * i]), "f"(s[4 * i + 1]), "f"(s[4 * i + 2]), "f"(s[4 * i + 3]), "r"(bar)
              : "memory");
      }
    }
    if (++in == BUFS) in = 0;
  }
  __device__ __forceinline__ void collect(float* v) {
    if (CL == 1) {
      read_warps(out, v);
    } else {
      wait();
      float s[4 * N4] = {};
#pragma unroll
      for (int r = 0; r < CL; ++r)
#pragma unroll
        for (int i = 0; i < N4; ++i) {
          const float4 a = ctas[(out * CL + r) * N4 + i];
          s[4 * i] += a.x, s[4 * i + 1] += a.y, s[4 * i + 2] += a.z, s[4 * i + 3] += a.w;
        }
#pragma unroll
      for (int i = 0; i < K; ++i) v[i] = dead ? __int_as_float(0x7fc00000) : s[i];
    }
    if (++out == BUFS) {
      out = 0;
      phase ^= 1;
    }
  }
};

// The exchange by itself (gdn_diag_exchange): each of a cluster's CTAs posts
// DIAG_POSTS sums of ones, one ahead of their collection as the backward does; CTA
// `silent` sends nothing, as if its own wait had run out. sums[CTA]: the last sum.
constexpr int DIAG_CL = 4, DIAG_NT = 64, DIAG_POSTS = 9;
__global__ void __launch_bounds__(DIAG_NT) k_exchange(int silent, long long limit, float* sums) {
  chain();
  TeamSum<6, DIAG_CL, 1> sum;
  sum.init();
  sum.limit = limit;
  sum.dead = (int)blockIdx.x == silent;
  float v[8];
  auto post = [&]() {
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = 1.f;
    sum.post(v);
  };
  post();
  for (int p = 0; p < DIAG_POSTS; ++p) {
    if (p + 1 < DIAG_POSTS) post();
    sum.collect(v);
  }
  sum.end();
  if (threadIdx.x == 0) sums[blockIdx.x] = v[5];
}

// With rx = 1 / sqrt(mean x^2 + eps) (1 without w_post) and r the same of h':
//   h' = h + scale w_post rx x,   y = r w h'.
// In a cluster the sum of the next row's x^2 goes with the row's own sum of h'^2,
// one exchange a row instead of two (5000 rows of 16384 bf16 columns 165 -> 115 us,
// 112 as it is now).
// Bound by the bytes of h, x, h_out and y: 20011 rows of 4096 columns, fp32 stream
// and bf16 branch, both norms: 151 us (984 MB, 6.5 TB/s); one row per block with
// plain loads took 305.
template <typename T, typename R, int CL, int S>
__global__ void __launch_bounds__(1024, 1)
    k_res_norm_fwd(int rows, int C, float inv_C, float eps, const R* h, const T* x, const float* w,
                   const float* w_post, const float* scale, R* h_out, T* y) {
  constexpr int KX = pieces<R>();
  constexpr bool SPLIT = sizeof(R) == 4;
  extern __shared__ uint4 smem[];
  const Ring<fwd_slots<T, R>(), SPLIT> ring = {
      smem + threadIdx.y * blockDim.x + threadIdx.x, (int)(blockDim.x * blockDim.y)};
  const Team<SPLIT> t = team_of<SPLIT, CL>(rows, C);
  chain();
  if (!t.on0 || !t.on1 || !x) ring.clear(S);
  auto fetch = [&](int stage, int row) {
    if (row < t.rows) {
      ring.fetch(stage, 0, h + (size_t)row * C, t);
      if (x) ring.fetch(stage, KX, x + (size_t)row * C, t);
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < S; ++s) fetch(s, t.first + s * t.step);
  TeamSum<CL == 1 ? 1 : 2, CL, 0> sum;
  sum.init();
  f32x2 wv[4], pv[4], sv[4];
  ld_cols(w, t, 0.f, wv);
  ld_cols(w_post, t, 1.f, pv);
  ld_cols(scale, t, 1.f, sv);
  float s[2] = {};  // sums over a row of h_out^2 and of the branch's x^2
  auto square = [&](int stage) {
    f32x2 xv[4], a = 0;
    ring.template read<T>(stage, KX, xv);
#pragma unroll
    for (int i = 0; i < 4; ++i) a = fma2(xv[i], xv[i], a);
    return sum2(a);
  };
  int stage = 0;
  if (CL > 1 && w_post && t.first < t.rows) {
    cp_wait<S - 1>();
    s[1] = square(0);
    sum.post(s);
    sum.collect(s);
  }
  for (int row = t.first; row < t.rows; row += t.step) {
    const int next = stage + 1 == S ? 0 : stage + 1;
    cp_wait<CL == 1 ? S - 1 : S - 2>();
    f32x2 hv[4], xv[4], a = 0;
    ring.template read<R>(stage, 0, hv);
    ring.template read<T>(stage, KX, xv);
    if (w_post) {
      float x2 = s[1];
      if (CL == 1) {
        x2 = square(stage);
        sum.post(&x2);
        sum.collect(&x2);
      }
      const f32x2 rx = both2(rsqrtf(fmaf(x2, inv_C, eps)));
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[i] = mul2(xv[i], mul2(rx, pv[i]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hv[i] = fma2(sv[i], xv[i], hv[i]);
      a = fma2(hv[i], hv[i], a);
    }
    if (h_out) st_cols(h_out + (size_t)row * C, t, hv);
    fetch(stage, row + S * t.step);  // the slot has been read
    stage = next;
    s[0] = sum2(a);
    if (CL > 1 && w_post) s[1] = row + t.step < t.rows ? square(next) : 0.f;
    sum.post(s);
    sum.collect(s);
    const f32x2 r = both2(rsqrtf(fmaf(s[0], inv_C, eps)));
#pragma unroll
    for (int i = 0; i < 4; ++i) hv[i] = mul2(hv[i], mul2(r, wv[i]));
    st_cols(y + (size_t)row * C, t, hv);
  }
  cp_wait<0>();
  sum.end();
}

// part [blocks][1 + (w_post) + (scale)][C]: the blocks' sums of dw, dw_post, dscale.
// With n = h r, m = x rx (x without w_post), sp = scale w_post:
//   dh = dh_out + r dy w - r^3 mean(dy w h) h
//   dx = rx (sp dh - m mean(sp dh m)),   dw_post = scale sum dh m,   dscale = w_post sum dh m
// and mean(sp dh m) is a combination of sums that do not need dh, so a row takes
// one reduction, of 6 sums. In a cluster the next row's sums are formed and posted
// before this row's are collected, so that the exchange's latency passes behind a
// row's work (4000 rows of 16384 bf16 columns 369 -> 320 us, 177 with as many clusters
// as fit and then 191 two rows ahead; 169 as it is now); within a CTA reading the row twice for
// that costs more than it hides (32768 rows of 2048: 135 us against 127). Bound by
// the bytes of h, dh_out, dy, x, dh and dx: 32768 rows of 2048 bf16 columns, both
// norms, 124 us (805 MB, 6.5 TB/s). bf16 rows in clusters are bound by no one counter:
// the 16 warps that the registers leave an SM issue in 62 % of the cycles at 5120 and
// 16384 columns, DRAM at 60 % of its peak, the warps waiting in turn on fixed latencies,
// shared memory, the barrier and the exchange (as many fp32 values take 92 % of the
// bytes' time: theirs is twice as long).
template <typename T, typename R, int CL>
__global__ void __launch_bounds__(512, 1)
    k_res_norm_bwd(int rows, int C, float inv_C, float eps, const R* h, const T* x, const float* w,
                   const float* w_post, const float* scale, const T* dy, const R* dh_out, R* dh,
                   T* dx, float* part) {
  constexpr int S = RN_STAGES_B, AHEAD = CL == 1 ? 0 : 1;
  constexpr int KD = pieces<R>(), KG = 2 * pieces<R>(), KX = KG + pieces<T>();
  constexpr bool SPLIT = sizeof(R) == 4;
  extern __shared__ uint4 smem[];
  const Ring<bwd_slots<T, R>(), SPLIT> ring = {
      smem + threadIdx.y * blockDim.x + threadIdx.x, (int)(blockDim.x * blockDim.y)};
  const Team<SPLIT> t = team_of<SPLIT, CL>(rows, C);
  const bool with_x = w_post || scale;
  chain();
  let_next_start();
  if (!t.on0 || !t.on1 || !dh_out || !with_x) ring.clear(S);
  auto fetch = [&](int stage, int row) {
    if (row < t.rows) {
      const size_t at = (size_t)row * C;
      ring.fetch(stage, 0, h + at, t);
      if (dh_out) ring.fetch(stage, KD, dh_out + at, t);
      ring.fetch(stage, KG, dy + at, t);
      if (with_x) ring.fetch(stage, KX, x + at, t);
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < S; ++s) fetch(s, t.first + s * t.step);
  TeamSum<6, CL, AHEAD> sum;
  sum.init();
  f32x2 wv[4], sp[4], aw[4] = {}, am[4] = {};
  ld_cols(w, t, 0.f, wv);
  {
    f32x2 pv[4];
    ld_cols(scale, t, 1.f, sp);
    ld_cols(w_post, t, 1.f, pv);
#pragma unroll
    for (int i = 0; i < 4; ++i) sp[i] = mul2(sp[i], pv[i]);
  }
  struct Row {
    f32x2 h[4], g[4], x[4], d[4];
  };
  auto read = [&](int stage, Row& v) {
    ring.template read<R>(stage, 0, v.h);
    ring.template read<R>(stage, KD, v.d);
    ring.template read<T>(stage, KG, v.g);
    ring.template read<T>(stage, KX, v.x);
  };
  auto post = [&](const Row& v) {
    f32x2 a[6] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 gw = mul2(v.g[i], wv[i]);
      a[0] = fma2(v.h[i], v.h[i], a[0]);
      a[1] = fma2(gw, v.h[i], a[1]);
      if (w_post) {
        const f32x2 q = mul2(sp[i], v.x[i]);
        a[2] = fma2(v.x[i], v.x[i], a[2]);
        a[3] = fma2(q, v.d[i], a[3]);
        a[4] = fma2(q, gw, a[4]);
        a[5] = fma2(q, v.h[i], a[5]);
      }
    }
    float s[8];
#pragma unroll
    for (int i = 0; i < 6; ++i) s[i] = sum2(a[i]);
    sum.post(s);
  };
  if (AHEAD > 0 && t.first < t.rows) {
    Row v;
    cp_wait<S - 1>();
    read(0, v);
    post(v);
  }
  int stage = 0;
  for (int row = t.first; row < t.rows; row += t.step) {
    Row v;
    if (row + AHEAD * t.step < t.rows) {
      cp_wait<S - 1 - AHEAD>();
      read(stage + AHEAD < S ? stage + AHEAD : stage + AHEAD - S, v);
      post(v);
    }
    float s[8];
    sum.collect(s);
    if (AHEAD > 0) read(stage, v);
    f32x2 *hv = v.h, *gv = v.g, *xv = v.x, *dv = v.d;
    const size_t at = (size_t)row * C;
    fetch(stage, row + S * t.step);  // the slot has been read
    if (++stage == S) stage = 0;
    const float r = rsqrtf(fmaf(s[0], inv_C, eps));
    const float rx = w_post ? rsqrtf(fmaf(s[2], inv_C, eps)) : 1.f;
    // factor of h in dh; r^3 by itself may overflow where eps is small and s[1] 0
    const float hc = -r * (r * (r * s[1])) * inv_C;
    const f32x2 r2 = both2(r), hc2 = both2(hc), rx2 = both2(rx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 gr = mul2(gv[i], r2);
      aw[i] = fma2(gr, hv[i], aw[i]);
      dv[i] = fma2(hv[i], hc2, fma2(gr, wv[i], dv[i]));  // dh
      xv[i] = mul2(xv[i], rx2);                          // m
      am[i] = fma2(dv[i], xv[i], am[i]);
    }
    st_cols(dh + at, t, dv);
    if (dx) {
      // mean(sp dh m) from the sums of its terms
      const f32x2 e = both2(w_post ? -rx * inv_C * fmaf(hc, s[5], fmaf(r, s[4], s[3])) : 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dv[i] = mul2(dv[i], sp[i]);
        if (w_post) dv[i] = mul2(rx2, fma2(xv[i], e, dv[i]));
      }
      st_cols(dx + at, t, dv);
    }
  }
  cp_wait<0>();
  sum.end();
  // the block's sums, teams joined through shared memory (the ring is drained)
  float* mine = reinterpret_cast<float*>(smem) + (threadIdx.y * blockDim.x + threadIdx.x) * 8;
  const int narr = 1 + (w_post != nullptr) + (scale != nullptr);
  float* out = part + (size_t)(blockIdx.x / CL) * narr * C;
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
  if (threadIdx.y) return;
  st_cols(out, t, aw);
  auto times = [&](const float* p) {
    f32x2 v[4];
    ld_cols(p, t, 1.f, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(am[i], v[i]);
    st_cols(out += C, t, v);
  };
  if (w_post) times(scale);
  if (scale) times(w_post);
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
  const int most = s.dtype == GDN_DTYPE_BF16 ? 152 * gate_blocks<__nv_bfloat16>()
                                             : 152 * 2 * gate_blocks<float>();
  return (int)std::min<long long>(most, (n + g - 1) / g);
}

template <typename T, int L>
cudaError_t launch_gate(const gdn_gate_norm_shape& s, const void* o, const void* z,
                        const float* w, const void* dy, void* out, void* dz, float* part,
                        cudaStream_t st) {
  const uint32_t n = (uint32_t)s.rows * (uint32_t)s.H, per = GN_NT / L * GN_U;
  const FastDiv byH(s.H);
  const float inv = 1.f / (float)s.d;
  if (!dy) {
    return launch(k_gate_norm_fwd<T, L>, dim3((n + per - 1) / per), dim3(GN_NT), 0, st, 1, n, byH,
                  s.d, inv, s.act, (long long)s.ldz, s.eps, (const T*)o, (const T*)z, w, (T*)out);
  }
  return launch(k_gate_norm_bwd<T, L>, dim3(gate_parts(s)), dim3(GN_NT), 0, st, 1, n, byH, s.d,
                inv, s.act, (long long)s.ldz, s.eps, (const T*)o, (const T*)z, w, (const T*)dy,
                (T*)out, (T*)dz, part);
}
template <typename T>
cudaError_t dispatch_gate(const gdn_gate_norm_shape& s, const void* o, const void* z,
                          const float* w, const void* dy, void* out, void* dz, float* part,
                          cudaStream_t st) {
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
  if (!dtype_ok(s->dtype) || !dtype_ok(s->res_dtype) || s->C % 8 || s->C > 16384 ||
      s->rows > MOST_INDEX)
    return GDN_ERR_UNSUPPORTED;
  if (s->res_dtype != s->dtype && s->res_dtype != GDN_DTYPE_F32) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// SMs that clusters can fill: of 4 CTAs of an SM each 36 fit, not 38, and two more
// than fit would run after the others (4000 rows of 16384 bf16 columns 169 us, with 38
// 305; of 8, three CTAs to an SM, 51, not 54: 5000 rows of 10240 columns 144, with 54 213).
int cluster_sms(int cl) { return cl == 8 ? 136 : cl == 4 ? 144 : RN_SMS; }

// How a call's rows are laid out over CTAs; a function of the shape alone, so
// the order of the parameter gradients' sums is too.
struct ResPlan {
  int cl, team, teams;  // CTAs per row, threads of a CTA per row, rows per CTA
  int blocks(int rows, int threads) const {  // CTAs, so that each SM has up to `threads`
    const int all = (rows + teams - 1) / teams;
    return cl * std::min(all, std::max(1, cluster_sms(cl) * (threads / (team * teams)) / cl));
  }
};
ResPlan res_plan(int C, bool bwd) {
  const int cols = bwd ? RN_COLS_B : RN_COLS_F, most = cols / 8;  // threads of an SM
  const auto team = [&](int cl) { return ((C / 8 + cl - 1) / cl + 31) / 32 * 32; };
  const auto filled = [&](int cl) { return most / team(cl) * team(cl) * cluster_sms(cl); };
  ResPlan p;
  p.cl = 1;
  while (C > p.cl * cols) p.cl *= 2;
  // smaller CTAs where they fill the SMs better (backward, 16000 rows of 5120 bf16
  // columns: 234 us in clusters of 2, 196 in 4; 5000 of 10240: 164 in 4, 144 in 8);
  // not where one CTA holds a row (20000 of 2560: 120 either way, mixed 124 and 127)
  if (bwd && p.cl > 1 && 10 * filled(2 * p.cl) > 11 * filled(p.cl)) p.cl *= 2;
  p.team = team(p.cl);
  p.teams = p.team >= 256 || p.cl > 1 ? 1 : 256 / p.team;
  return p;
}
int res_parts(const gdn_res_norm_shape& s) {
  const ResPlan p = res_plan(s.C, true);
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
  return launch(kernel, dim3(blocks), dim3(p.team, p.teams), smem, st, p.cl, args...);
}
template <typename T, typename R, int CL>
cudaError_t launch_res(const gdn_res_norm_shape& s, const ResArgs& a, const ResPlan& p,
                       cudaStream_t st) {
  const int nt = p.team * p.teams;
  const float inv = 1.f / (float)s.C;
  if constexpr (CL <= 2) {  // forward rows take two CTAs at most
    if (!a.dy) {
      // rows in flight: 4, where that is what an SM's shared memory holds for 1024
      // threads; 3 for fp32 streams, and for mixed types in CTAs of 1024 threads
      // (mixed, 4096 columns: 152 us with 4, 171 with 3; 8192: 135 with 4, 123 with 3)
      constexpr int slots = fwd_slots<T, R>();
      auto go = [&](auto stages) {
        constexpr int S = decltype(stages)::value;
        return launch_rows(k_res_norm_fwd<T, R, CL, S>, p, p.blocks(s.rows, 1024),
                           nt * 16 * slots * S, st, s.rows, s.C, inv, s.eps, (const R*)a.h,
                           (const T*)a.x, a.w, a.w_post, a.scale, (R*)a.ho, (T*)a.y);
      };
      if constexpr (slots == 3 && CL == 1) {
        if (p.team > 512) return go(std::integral_constant<int, 3>());
      }
      constexpr int usual = slots == 4 || (slots == 3 && CL != 1) ? 3 : 4;
      return go(std::integral_constant<int, usual>());
    }
  }
  return launch_rows(k_res_norm_bwd<T, R, CL>, p, p.blocks(s.rows, 512),
                     nt * 16 * bwd_slots<T, R>() * RN_STAGES_B, st, s.rows, s.C, inv, s.eps,
                     (const R*)a.h, (const T*)a.x, a.w, a.w_post, a.scale, (const T*)a.dy,
                     (const R*)a.dh_out, (R*)a.ho, (T*)a.y, a.part);
}
template <typename T, typename R>
cudaError_t dispatch_res(const gdn_res_norm_shape& s, const ResArgs& a, cudaStream_t st) {
  const ResPlan p = res_plan(s.C, a.dy != nullptr);
  switch (p.cl) {
    case 1: return launch_res<T, R, 1>(s, a, p, st);
    case 2: return launch_res<T, R, 2>(s, a, p, st);
    case 4: return launch_res<T, R, 4>(s, a, p, st);
    default: return launch_res<T, R, 8>(s, a, p, st);
  }
}
cudaError_t run_res(const gdn_res_norm_shape& s, const ResArgs& a, cudaStream_t st) {
  if (s.dtype == GDN_DTYPE_F32) return dispatch_res<float, float>(s, a, st);
  if (s.res_dtype == GDN_DTYPE_F32) return dispatch_res<__nv_bfloat16, float>(s, a, st);
  return dispatch_res<__nv_bfloat16, __nv_bfloat16>(s, a, st);
}

cudaError_t run_exchange(int silent, long long limit, float* sums, cudaStream_t st) {
  return launch(k_exchange, dim3(DIAG_CL), dim3(DIAG_NT), 0, st, DIAG_CL, silent, limit, sums);
}
gdn_status take_status(cudaStream_t st) {
  if (cudaStreamSynchronize(st) != cudaSuccess) return GDN_ERR_CUDA;
  int word = 0;
  const int zero = 0;
  if (cudaMemcpyFromSymbol(&word, g_exchange_status, sizeof(int)) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (word == DEV_OK) return GDN_OK;
  if (cudaMemcpyToSymbol(g_exchange_status, &zero, sizeof(int)) != cudaSuccess)
    return GDN_ERR_CUDA;
  return GDN_ERR_TIMEOUT;
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
  const cudaError_t ce =
      s.dtype == GDN_DTYPE_BF16
          ? dispatch_gate<__nv_bfloat16>(s, o, z, w, nullptr, y, nullptr, nullptr, st)
          : dispatch_gate<float>(s, o, z, w, nullptr, y, nullptr, nullptr, st);
  prof_mark(st, nullptr);
  return ce ? GDN_ERR_CUDA : GDN_OK;
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
    if (s.dtype == GDN_DTYPE_BF16
            ? dispatch_gate<__nv_bfloat16>(s, o, z, w, dy, dout, dz, part, st)
            : dispatch_gate<float>(s, o, z, w, dy, dout, dz, part, st))
      return GDN_ERR_CUDA;
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

gdn_status gdn_layer_status(void* stream) { return gdn::take_status((cudaStream_t)stream); }

int gdn_diag_exchange(float* sums, int silent, int limit_log2, void* stream) {
  using namespace gdn;
  if (!sums || !aligned(sums, 4) || silent < -1 || silent >= DIAG_CL) return GDN_ERR_INVALID_ARG;
  const int lg = std::min(std::max(limit_log2, 10), 32);
  return run_exchange(silent, 1ll << lg, sums, (cudaStream_t)stream) ? GDN_ERR_CUDA : GDN_OK;
}

}  // extern "C"

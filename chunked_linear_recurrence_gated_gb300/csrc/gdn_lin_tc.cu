// Linear attention with a decay for each head over whole sequences, bf16
// (gdn_lin_fwd / gdn_lin_bwd, include/gdn_lin.h) on the 5th-generation tensor cores.
//
// One pass over a sequence carries a state through chunks of C = 128 tokens. With x, y,
// z the rows of three tensors and gamma, L, S, R as in gdn_lin.cu,
//   out_t = sum_{s <= t} L_ts (x_t . y_s) z_s + e^{gamma_t} x_t S
//   S <- e^{gamma_C} S + sum_s e^{gamma_C - gamma_s} y_s z_s^T
// is the forward (x, y, z = q, k, v) and dq (dO, v, k with the state's transpose). dk, dv
// and dg come from one pass from the end, which carries R.
//
// A sequence is cut into units of chunks, so that there is a CTA for every SM where
// there are few sequences and heads: k_lin_tc_state sums each unit's own contribution to
// the state (it reads y and z only), k_lin_scan joins them along the sequence, and the
// passes then start every unit from its state.
//
// Rounding. Products of inputs are exact in the tensor core's fp32 sums. A state, and a
// weighted operand of a state's update, is taken as two bf16 parts (2^-17 of itself),
// because states leave the call in fp32 and because dg is a running difference of sums
// over whole units. The masked products P = L x y^T are rounded to bf16 once before they
// meet z, as their result is when it is stored.
#include <cuda.h>
#include <stdint.h>

#include <algorithm>

#include "gdn_internal.cuh"
#include "gdn_lin.cuh"
#include "gdn_mma.cuh"
#include "gdn_umma.cuh"

namespace gdn {
namespace {

typedef __nv_bfloat16 bf;

constexpr int TC = 128;          // tokens of a chunk
constexpr int NEPI = 512;        // 16 warps on the accumulators: 4 lane quarters x 4 column groups
constexpr int NTHR = NEPI + 32;  // and one that copies, issues the MMAs and forms the decay factors
constexpr uint32_t HALF_TILE = TC * 128;  // 64 columns of a chunk's rows

// ------------------------------------------------------------------ TMEM access
// D (+)= A B with A in tensor memory (row i in lane i, two values of the reduced
// dimension in each column).
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                        bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// 16 columns of this thread's lane from registers; wait before telling others.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}
template <int N>  // 16 or 32 columns
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float* v) {
#pragma unroll
  for (int i = 0; i < N; i += 16) tmem_ld16(taddr + i, v + i);
}
template <int N>
__device__ __forceinline__ void tmem_st_f(uint32_t taddr, const float* v) {
#pragma unroll
  for (int i = 0; i < N; i += 16) {
    uint32_t r[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(v[i + j]);
    tmem_st16(taddr + i, r);
  }
}

// ------------------------------------------------------------------ shared memory
// K-major operand: rows of 64 reduced values, 64-wide halves `half` bytes apart; step kk
// of 16. MN-major operand: rows of the reduced dimension.
__device__ __forceinline__ uint64_t kmaj(uint32_t base, uint32_t half, int kk) {
  return umma_desc(base + (kk >> 2) * half + 32 * (kk & 3), 16, 1024);
}
__device__ __forceinline__ uint64_t mnmaj(uint32_t base, uint32_t half, int kk) {
  return umma_desc(base + 2048 * kk, half, 1024);
}
__device__ __forceinline__ float bf_at(const unsigned char* p) {
  return __uint_as_float((uint32_t)*reinterpret_cast<const unsigned short*>(p) << 16);
}
// Columns [c, c + 8) of row r of a tile of 64-wide halves.
__device__ __forceinline__ unsigned char* at8(unsigned char* tile, uint32_t half, int r, int c) {
  return tile + (c >> 6) * half + r * 128 + ((((c & 63) >> 3) ^ (r & 7)) << 4);
}
__device__ __forceinline__ uint32_t pack2bf(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Two values as packed first parts and packed rests.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack2bf(a, b);
  lo = pack2bf(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}
// N values of row r from column c into the tiles of the first parts and of the rests.
template <int N>
__device__ __forceinline__ void put_split(unsigned char* hi, unsigned char* lo, uint32_t half, int r,
                                          int c, const float* v) {
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) split2(v[i + 2 * j], v[i + 2 * j + 1], h[j], l[j]);
    *reinterpret_cast<uint4*>(at8(hi, half, r, c + i)) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(at8(lo, half, r, c + i)) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

// Decay factors of a chunk.
struct Vec {
  float hi[TC], lo[TC];  // gamma, as the sum of two floats
  float row[TC];         // e^{gamma_t - gamma_{b-1}}, b the first token of t's block of 32
  float up[TC];          // e^{gamma_t}
  float down[TC];        // e^{gamma_C - gamma_t}
  float tab[3][TC];      // [b - 1][s]: e^{gamma_{32 b - 1} - gamma_s} for s < 32 b
  float whole, pad[3];   // e^{gamma_C}
};

// The log-decays of a chunk, 4 tokens for each lane of a warp, loaded ahead of their use.
struct Raw {
  float x[4];
};
__device__ __forceinline__ Raw raw_decay(int row, int len, int h, const bf* g, long long ldg,
                                         const float* decay) {
  const int l = threadIdx.x & 31;
  Raw r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 4 * l + i;
    r.x[i] = t < len ? lin_decay(decay ? decay[h] : ldf(g + (size_t)(row + t) * ldg + h)) : 0.f;
  }
  return r;
}
// gamma summed in 64 bits (differences of neighbours keep 24 bits however large it is).
__device__ __forceinline__ void sum_decay(const Raw& r, float* hi, float* lo) {
  const int l = threadIdx.x & 31;
  double c[4], sum = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = (sum += (double)r.x[i]);
  double all = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, all, d);
    if (l >= d) all += y;
  }
  const double before = all - sum;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double x = before + c[i];
    hi[i] = (float)x;
    lo[i] = (float)(x - (double)hi[i]);
  }
}
__device__ __forceinline__ float exp_diff(float h1, float l1, float h0, float l0) {
  return expf((h1 - h0) + (l1 - l0));
}
__device__ __forceinline__ void fill_vec(const Raw& r, Vec& v) {  // one warp
  const int l = threadIdx.x & 31;
  float hi[4], lo[4], eh[4], el[4];
  sum_decay(r, hi, lo);
#pragma unroll
  for (int b = 0; b < 4; ++b) {  // the ends of the blocks
    eh[b] = __shfl_sync(0xffffffffu, hi[3], 8 * b + 7);
    el[b] = __shfl_sync(0xffffffffu, lo[3], 8 * b + 7);
  }
  const int blk = l >> 3;  // of 32 tokens
  const float ah = blk == 0 ? 0.f : blk == 1 ? eh[0] : blk == 2 ? eh[1] : eh[2];
  const float al = blk == 0 ? 0.f : blk == 1 ? el[0] : blk == 2 ? el[1] : el[2];
  float o[4] = {};
  auto put = [&](float* to) {
    reinterpret_cast<float4*>(to)[l] = make_float4(o[0], o[1], o[2], o[3]);
  };
  reinterpret_cast<float4*>(v.hi)[l] = make_float4(hi[0], hi[1], hi[2], hi[3]);
  reinterpret_cast<float4*>(v.lo)[l] = make_float4(lo[0], lo[1], lo[2], lo[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = exp_diff(hi[i], lo[i], ah, al);
  put(v.row);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = exp_diff(hi[i], lo[i], 0.f, 0.f);
  put(v.up);
  if (l == 31) v.whole = o[3];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = exp_diff(eh[3], el[3], hi[i], lo[i]);
  put(v.down);
#pragma unroll
  for (int b = 0; b < 3; ++b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = blk <= b ? exp_diff(eh[b], el[b], hi[i], lo[i]) : 0.f;
    put(v.tab[b]);
  }
}

// ------------------------------------------------------------------ shared pieces
struct Who {  // a thread's part of an accumulator
  int tid, w, l, q4, cq, lane;
  bool epi, ctl;  // works on accumulators; is the thread that copies and issues
};
__device__ __forceinline__ Who who() {
  Who t;
  t.tid = threadIdx.x;
  t.w = t.tid >> 5;
  t.l = t.tid & 31;
  t.q4 = t.w & 3;
  t.cq = (t.w >> 2) & 3;
  t.lane = 32 * t.q4 + t.l;
  t.epi = t.tid < NEPI;
  t.ctl = t.tid == NEPI;
  return t;
}

// What the kernels of a call share.
struct Args {
  LinMap m;
  int H, chunks;  // heads; chunks of a unit
  float scale;
  const bf* g;
  const float* decay;
  long long ldg;
  int* status;
};

// One 128-token tile of D columns.
template <int D>
__device__ __forceinline__ void load_tile(unsigned char* to, const CUtensorMap* map, int h, int tok,
                                          int seq, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, D * TC * 2);
#pragma unroll
  for (int c = 0; c < D; c += 64) tma_load_4d(to + (c >> 6) * HALF_TILE, map, c, h, tok, seq, bar);
}
// Rows [len, TC) of a tile of D columns as zeros (a packed call's next sequence is there).
template <int D>
__device__ __forceinline__ void zero_rows(unsigned char* tile, int len, int tid) {
  constexpr int P = D / 8;
  for (int i = tid; i < (TC - len) * P; i += NEPI)
    *reinterpret_cast<uint4*>(at8(tile, HALF_TILE, len + i / P, i % P * 8)) = make_uint4(0, 0, 0, 0);
}
// The weighted transpose of a tile's column `lane` (tokens [32 cq, 32 cq + 32)) as packed
// first parts and rests: an operand in tensor memory with the tokens as reduced dimension.
__device__ __forceinline__ void weigh(const unsigned char* tile, const Who& t, const float* wt,
                                      float by, int len, uint32_t* hi, uint32_t* lo) {
  const unsigned char* col = tile + (t.lane >> 6) * HALF_TILE + (t.lane & 7) * 2;
  const int piece = (t.lane & 63) >> 3, s0 = 32 * t.cq;
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 w4 = *reinterpret_cast<const float4*>(wt + s0 + i);
    const float w[4] = {w4.x, w4.y, w4.z, w4.w};
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int s = s0 + i + j;
      const float y = bf_at(col + s * 128 + ((piece ^ (s & 7)) << 4));
      x[j] = s < len ? y * (by * w[j]) : 0.f;
    }
    split2(x[0], x[1], hi[i / 2], lo[i / 2]);
    split2(x[2], x[3], hi[i / 2 + 1], lo[i / 2 + 1]);
  }
}
// This thread's N elements (row lane, columns c0..) of a state [DY][DZ], or of one that is
// kept transposed in memory (TR).
template <int DY, int DZ, bool TR, int N>
__device__ __forceinline__ void load_state(const float* from, int lane, int c0, float* s) {
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = 0.f;
  if (!from || lane >= DY) return;
  if (TR) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = from[(size_t)(c0 + i) * DY + lane];
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(from + (size_t)lane * DZ + c0 + i);
      s[i] = x.x, s[i + 1] = x.y, s[i + 2] = x.z, s[i + 3] = x.w;
    }
  }
}
template <int DY, int DZ, bool TR, int N>
__device__ __forceinline__ void store_state(float* to, int lane, int c0, const float* s) {
  if (!to || lane >= DY) return;
  if (TR) {
#pragma unroll
    for (int i = 0; i < N; ++i) to[(size_t)(c0 + i) * DY + lane] = s[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(to + (size_t)lane * DZ + c0 + i) =
          make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
  }
}
// N values times `by` as bf16 to consecutive addresses (16-byte aligned).
template <int N>
__device__ __forceinline__ void store_row(bf* to, const float* v, float by) {
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = pack2bf(by * v[i + 2 * j], by * v[i + 2 * j + 1]);
    *reinterpret_cast<uint4*>(to + i) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}
// After a wait that ran out: this CTA's copies still under way are waited for, with a
// limit, before its shared memory is given up.
__device__ __forceinline__ void drain(uint64_t* bars, int n, uint32_t phases) {
  for (int i = 0; i < n; ++i) {
    int off = 0;
    mbar_wait(bars + i, (phases >> i) & 1, &off, 1ll << 24);
  }
}

constexpr uint32_t slot_bytes(int a, int b) { return (a > b ? a : b) * TC * 2; }

// ------------------------------------------------------------------ a unit's own sum
// E = sum over the unit of (its decay to the unit's end, or REV: from the unit's start,
// times scale) y z^T, and the unit's whole decay. Not for a sequence's last unit (REV: its
// first), whose state nobody starts from. The MMAs of a chunk run under the weighing of
// the next one and the update from the one before; three chunks' tiles are in flight.
struct StateVec {
  float w[TC];
  float whole, pad[3];
};
template <int DY, int DZ>
struct StateSm {
  static constexpr uint32_t SLOT = slot_bytes(DY, DZ), STAGES = 3;
  static constexpr uint32_t VEC = 2 * STAGES * SLOT, BAR = VEC + 4 * sizeof(StateVec);
  static constexpr uint32_t BYTES = BAR + 128 + 1024;
};
template <int DY, int DZ, bool REV, bool TR>
__global__ void __launch_bounds__(NTHR, 1)
    k_lin_tc_state(Args a, float* whole, float* out, bool clear, const __grid_constant__ CUtensorMap my,
                   const __grid_constant__ CUtensorMap mz) {
  using L = StateSm<DY, DZ>;
  constexpr int N = DZ / 4;
  constexpr uint32_t D0 = 0, Y0 = 256;  // two accumulators, two operands of two parts
  chain();
  if (clear && blockIdx.x == 0 && threadIdx.x == 0) *a.status = DEV_OK;
  const int unit = blockIdx.x / a.H, h = blockIdx.x - unit * a.H;
  LinUnit u;
  if (!lin_unit(a.m, unit, u)) return;
  if (u.at == (REV ? 0 : u.n - 1)) return;
  const Who t = who();
  extern __shared__ __align__(1024) unsigned char smraw[];
  unsigned char* sb = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
  StateVec* vec = reinterpret_cast<StateVec*>(sb + L::VEC);
  uint64_t* full = reinterpret_cast<uint64_t*>(sb + L::BAR);  // [STAGES]
  uint64_t* done = full + L::STAGES;                          // [2] MMAs of a chunk
  uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 2);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  const int nch = (u.len + TC - 1) / TC;
  if (t.ctl) {
    for (int i = 0; i < (int)L::STAGES + 2; ++i) mbar_init(full + i, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (t.w == NEPI / 32) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *tslot, tl = tm + ((uint32_t)(32 * t.q4) << 16);
  auto chunk = [&](int i) { return REV ? nch - 1 - i : i; };
  auto load = [&](int i) {  // the control thread
    const int c = chunk(i), st = i % L::STAGES;
    const int tok = a.m.cu ? u.row + c * TC : u.at * a.m.unit + c * TC, seq = a.m.cu ? 0 : u.seq;
    unsigned char* to = sb + 2 * st * L::SLOT;
    mbar_arrive_expect_tx(full + st, (DY + DZ) * TC * 2);
#pragma unroll
    for (int e = 0; e < DY; e += 64) tma_load_4d(to + (e >> 6) * HALF_TILE, &my, e, h, tok, seq, full + st);
#pragma unroll
    for (int e = 0; e < DZ; e += 64)
      tma_load_4d(to + L::SLOT + (e >> 6) * HALF_TILE, &mz, e, h, tok, seq, full + st);
  };
  auto raw = [&](int i) {
    const int c = chunk(i);
    return raw_decay(u.row + c * TC, min(TC, u.len - c * TC), h, a.g, a.ldg, a.decay);
  };
  auto fill = [&](const Raw& r, StateVec& v) {
    float hi[4], lo[4];
    sum_decay(r, hi, lo);
    const float eh = __shfl_sync(0xffffffffu, hi[3], 31), el = __shfl_sync(0xffffffffu, lo[3], 31);
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = REV ? a.scale * exp_diff(hi[i], lo[i], 0.f, 0.f) : exp_diff(eh, el, hi[i], lo[i]);
    reinterpret_cast<float4*>(v.w)[t.l] = make_float4(o[0], o[1], o[2], o[3]);
    if (t.l == 0) v.whole = exp_diff(eh, el, 0.f, 0.f);
  };
  if (t.ctl)
    for (int i = 0; i < min(nch, (int)L::STAGES); ++i) load(i);
  if (!t.epi) {
    fill(raw(0), vec[0]);
    if (nch > 1) fill(raw(1), vec[1]);
  }
  float s[N], all = 1.f;
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = 0.f;
  auto update = [&](int i) {  // from chunk i's accumulator
    mbar_wait(done + (i & 1), (i >> 1) & 1, abort);
    tc_fence_after();
    if (t.lane < DY) {
      float d[N];
      tmem_ld<N>(tl + D0 + 128 * (i & 1) + N * t.cq, d);
      const float wh = vec[i & 3].whole;
#pragma unroll
      for (int j = 0; j < N; ++j) s[j] = fmaf(wh, s[j], d[j]);
    }
    all *= vec[i & 3].whole;
    tc_fence_before();
  };
  __syncthreads();
  for (int i = 0; i < nch; ++i) {
    const int st = i % L::STAGES, len = min(TC, u.len - chunk(i) * TC);
    unsigned char* y = sb + 2 * st * L::SLOT;
    if (t.epi) {
      mbar_wait(full + st, (i / L::STAGES) & 1, abort);
      if (t.lane < DY) {
        uint32_t hi[16], lo[16];
        weigh(y, t, vec[i & 3].w, 1.f, len, hi, lo);
        tmem_st16(tl + Y0 + 128 * (i & 1) + 16 * t.cq, hi);
        tmem_st16(tl + Y0 + 128 * (i & 1) + 64 + 16 * t.cq, lo);
        tmem_st_wait();
      }
      if (len < TC && a.m.cu) {
        zero_rows<DZ>(y + L::SLOT, len, t.tid);
        fence_proxy_async_smem();
      }
      tc_fence_before();
    }
    if (__syncthreads_or(*abort != 0)) break;
    if (t.epi) {
      if (i) update(i - 1);
    } else {
      if (t.l == 0) {
        tc_fence_after();
        mbar_wait(full + st, (i / L::STAGES) & 1, abort);
        const uint32_t z = smem_u32(y + L::SLOT);
        constexpr uint32_t id = umma_idesc(128, DZ, 0, 1);
#pragma unroll 1
        for (int p = 0; p < 2; ++p)
#pragma unroll 1
          for (int kk = 0; kk < TC / 16; ++kk)
            umma_ts(tm + D0 + 128 * (i & 1), tm + Y0 + 128 * (i & 1) + 64 * p + 8 * kk,
                    mnmaj(z, HALF_TILE, kk), id, p || kk);
        umma_commit(done + (i & 1));
      }
      __syncwarp();
      // two ahead: visible behind the next chunk's barrier; four kept, for the chunk before
      // this one is still to be added
      if (i + 2 < nch) fill(raw(i + 2), vec[(i + 2) & 3]);
      if (t.l == 0 && i) {  // the chunk before is done with its tiles
        mbar_wait(done + ((i - 1) & 1), ((i - 1) >> 1) & 1, abort);
        if (i - 1 + (int)L::STAGES < nch && !*abort) load(i - 1 + L::STAGES);
      }
    }
  }
  if (t.epi && nch) update(nch - 1);
  const size_t uh = (size_t)unit * a.H + h;
  if (t.epi) store_state<DY, DZ, TR, N>(out + uh * DY * DZ, t.lane, N * t.cq, s);
  if (t.tid == 0) whole[uh] = all;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (t.ctl && *abort) {
    *a.status = DEV_TIMEOUT;
    drain(full, L::STAGES, 0);
    drain(full, L::STAGES, ~0u);
  }
  __syncthreads();
  if (t.w == NEPI / 32) tmem_dealloc(tm, 512);
}

// ------------------------------------------------------------------ forward and dq
// Per chunk: P = x y^T and x S (MMAs) under the weighing of y; P masked into tensor memory
// and x S scaled in place; P z onto it and the state's sum (MMAs); result and state. The
// tiles x, y, z take the four slots in turn: y and z of the next chunk are copied as soon
// as x and y are done with, x of the one after behind z.
template <int DY, int DZ>
struct PassSm {
  static constexpr uint32_t SLOT = slot_bytes(DY, DZ), STATE = DY * DZ * 2, HALF_S = DY * 128;
  static constexpr uint32_t S_HI = 4 * SLOT, S_LO = S_HI + STATE, VEC = S_LO + STATE;
  static constexpr uint32_t PART = VEC + 2 * sizeof(Vec), BAR = PART + 4 * TC * 4;
  static constexpr uint32_t BYTES = BAR + 128 + 1024;
};
template <int DY, int DZ, bool DQ>
__global__ void __launch_bounds__(NTHR, 1)
    k_lin_tc_pass(Args a, const float* S_in, const float* S_unit, float* S_out, bf* out, const bf* q,
                  long long ldq, float* far, bool clear, const __grid_constant__ CUtensorMap mx,
                  const __grid_constant__ CUtensorMap my, const __grid_constant__ CUtensorMap mz) {
  using L = PassSm<DY, DZ>;
  constexpr int N = DZ / 4;
  constexpr uint32_t P0 = 0, O0 = 128, Y0 = 256, D0 = 384;
  chain();
  if (clear && blockIdx.x == 0 && threadIdx.x == 0) *a.status = DEV_OK;
  const int unit = blockIdx.x / a.H, h = blockIdx.x - unit * a.H;
  LinUnit u;
  if (!lin_unit(a.m, unit, u)) return;
  const Who t = who();
  extern __shared__ __align__(1024) unsigned char smraw[];
  unsigned char* sb = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
  unsigned char *s_hi = sb + L::S_HI, *s_lo = sb + L::S_LO;
  Vec* vec = reinterpret_cast<Vec*>(sb + L::VEC);
  float* part = reinterpret_cast<float*>(sb + L::PART);
  uint64_t* full = reinterpret_cast<uint64_t*>(sb + L::BAR);  // [4]
  uint64_t *bar_a = full + 4, *bar_c = full + 5;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(full + 6);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  const int nch = (u.len + TC - 1) / TC;
  if (t.ctl) {
    for (int i = 0; i < 6; ++i) mbar_init(full + i, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (t.w == NEPI / 32) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *tslot, tl = tm + ((uint32_t)(32 * t.q4) << 16);
  auto load = [&](int n) {  // tile n: x, y or z of chunk n / 3 (the control thread)
    const int c = n / 3, kind = n - 3 * c;
    if (c >= nch) return;
    const int tok = a.m.cu ? u.row + c * TC : u.at * a.m.unit + c * TC, seq = a.m.cu ? 0 : u.seq;
    unsigned char* to = sb + (n & 3) * L::SLOT;
    if (kind == 0)
      load_tile<DY>(to, &mx, h, tok, seq, full + (n & 3));
    else if (kind == 1)
      load_tile<DY>(to, &my, h, tok, seq, full + (n & 3));
    else
      load_tile<DZ>(to, &mz, h, tok, seq, full + (n & 3));
  };
  auto tile = [&](int n) { return sb + (n & 3) * L::SLOT; };
  auto wait_tile = [&](int n) { return mbar_wait(full + (n & 3), (n >> 2) & 1, abort); };
  auto raw = [&](int c) {
    return raw_decay(u.row + c * TC, min(TC, u.len - c * TC), h, a.g, a.ldg, a.decay);
  };
  if (t.ctl)
    for (int n = 0; n < 4; ++n) load(n);
  const size_t sh = ((size_t)u.seq * a.H + h) * DY * DZ, uh = ((size_t)unit * a.H + h) * DY * DZ;
  float s[N];
  if (t.epi) {
    load_state<DY, DZ, DQ, N>(u.at ? S_unit + uh : S_in ? S_in + sh : nullptr, t.lane, N * t.cq, s);
    if (t.lane < DY) put_split<N>(s_hi, s_lo, L::HALF_S, t.lane, N * t.cq, s);
    fence_proxy_async_smem();
  } else if (nch) {
    fill_vec(raw(0), vec[0]);
  }
  __syncthreads();
  for (int c = 0; c < nch; ++c) {
    const int len = min(TC, u.len - c * TC), n0 = 3 * c;
    const Vec& v = vec[c & 1];
    const int row = u.row + c * TC + t.lane;  // of this thread's result
    const bool on = t.lane < len;
    if (t.ctl) {
      wait_tile(n0);
      wait_tile(n0 + 1);
      tc_fence_after();
      const uint32_t x = smem_u32(tile(n0)), y = smem_u32(tile(n0 + 1));
#pragma unroll 1
      for (int kk = 0; kk < DY / 16; ++kk)
        umma_bf16(tm + P0, kmaj(x, HALF_TILE, kk), kmaj(y, HALF_TILE, kk),
                  umma_idesc(128, 128, 0, 0), kk > 0);
#pragma unroll 1
      for (int p = 0; p < 2; ++p)
#pragma unroll 1
        for (int kk = 0; kk < DY / 16; ++kk)
          umma_bf16(tm + O0, kmaj(x, HALF_TILE, kk), mnmaj(smem_u32(p ? s_lo : s_hi), L::HALF_S, kk),
                    umma_idesc(128, DZ, 0, 1), p || kk);
      umma_commit(bar_a);
    }
    if (t.epi) {
      uint4 qr[DQ ? N / 8 : 1];
      if (DQ) {
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
          qr[i] = make_uint4(0, 0, 0, 0);
          if (on)
            qr[i] = *reinterpret_cast<const uint4*>(q + (size_t)row * ldq + (size_t)h * DZ +
                                                    N * t.cq + 8 * i);
        }
      }
      wait_tile(n0 + 1);
      if (t.lane < DY) {
        uint32_t hi[16], lo[16];
        weigh(tile(n0 + 1), t, v.down, 1.f, len, hi, lo);
        tmem_st16(tl + Y0 + 16 * t.cq, hi);
        tmem_st16(tl + Y0 + 64 + 16 * t.cq, lo);
      }
      mbar_wait(bar_a, c & 1, abort);
      tc_fence_after();
      // P: this thread's row t, columns [32 cq, 32 cq + 32)
      uint32_t p[16];
      if (t.cq > t.q4) {
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = 0;
      } else {
        float x[32];
        tmem_ld<32>(tl + P0 + 32 * t.cq, x);
        if (t.cq == t.q4) {
          const float gh = v.hi[t.lane], gl = v.lo[t.lane];
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 h4 = *reinterpret_cast<const float4*>(v.hi + 32 * t.cq + i);
            const float4 l4 = *reinterpret_cast<const float4*>(v.lo + 32 * t.cq + i);
            const float hh[4] = {h4.x, h4.y, h4.z, h4.w}, ll[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              x[i + j] = i + j <= t.l ? x[i + j] * __expf((gh - hh[j]) + (gl - ll[j])) : 0.f;
          }
        } else {
          const float r = v.row[t.lane];
          const float* tb = v.tab[t.q4 - 1] + 32 * t.cq;
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(tb + i);
            x[i] *= r * f.x;
            x[i + 1] *= r * f.y;
            x[i + 2] *= r * f.z;
            x[i + 3] *= r * f.w;
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = pack2bf(x[2 * i], x[2 * i + 1]);
      }
      tc_fence_before();
      named_bar(1 + t.q4, 128);  // the lane quarter's columns of x y^T have been read
      tc_fence_after();
      tmem_st16(tl + P0 + 16 * t.cq, p);
      float o[N], up = v.up[t.lane];
      tmem_ld<N>(tl + O0 + N * t.cq, o);
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] *= up;
      tmem_st_f<N>(tl + O0 + N * t.cq, o);
      if (DQ) {  // q_t . (far part of dq_t)
        float f = 0.f;
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
          const uint32_t w4[4] = {qr[i].x, qr[i].y, qr[i].z, qr[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f = fmaf(__uint_as_float(w4[j] << 16), o[8 * i + 2 * j], f);
            f = fmaf(__uint_as_float(w4[j] & 0xffff0000u), o[8 * i + 2 * j + 1], f);
          }
        }
        part[t.cq * TC + t.lane] = a.scale * f;
      }
      tmem_st_wait();
      if (len < TC && a.m.cu) {
        wait_tile(n0 + 2);
        zero_rows<DZ>(tile(n0 + 2), len, t.tid);
        fence_proxy_async_smem();
      }
      tc_fence_before();
    }
    __syncthreads();
    if (!t.epi) {
      if (t.l == 0) {
        tc_fence_after();
        if (!*abort) {
          load(n0 + 4);
          load(n0 + 5);
        }
        wait_tile(n0 + 2);
        const uint32_t z = smem_u32(tile(n0 + 2));
        constexpr uint32_t id = umma_idesc(128, DZ, 0, 1);
#pragma unroll 1
        for (int kk = 0; kk < TC / 16; ++kk)
          umma_ts(tm + O0, tm + P0 + 8 * kk, mnmaj(z, HALF_TILE, kk), id, true);
#pragma unroll 1
        for (int p = 0; p < 2; ++p)
#pragma unroll 1
          for (int kk = 0; kk < TC / 16; ++kk)
            umma_ts(tm + D0, tm + Y0 + 64 * p + 8 * kk, mnmaj(z, HALF_TILE, kk), id, p || kk);
        umma_commit(bar_c);
      }
      __syncwarp();
      if (c + 1 < nch) fill_vec(raw(c + 1), vec[(c + 1) & 1]);
      if (t.l == 0) {
        mbar_wait(bar_c, c & 1, abort);
        if (!*abort) load(n0 + 6);
      }
    } else {
      if (DQ && t.tid < len)
        far[(size_t)row * a.H + h] = (part[t.tid] + part[TC + t.tid]) +
                                     (part[2 * TC + t.tid] + part[3 * TC + t.tid]);
      mbar_wait(bar_c, c & 1, abort);
      tc_fence_after();
      float o[N];
      if (t.lane < DY) {
        tmem_ld<N>(tl + D0 + N * t.cq, o);
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = fmaf(v.whole, s[i], o[i]);
        put_split<N>(s_hi, s_lo, L::HALF_S, t.lane, N * t.cq, s);
        fence_proxy_async_smem();
      }
      tmem_ld<N>(tl + O0 + N * t.cq, o);
      if (on) store_row<N>(out + ((size_t)row * a.H + h) * DZ + N * t.cq, o, a.scale);
      tc_fence_before();
    }
    if (__syncthreads_or(*abort != 0)) break;
  }
  if (t.epi && u.at == u.n - 1 && S_out) store_state<DY, DZ, DQ, N>(S_out + sh, t.lane, N * t.cq, s);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (t.ctl && *abort) {
    *a.status = DEV_TIMEOUT;
    drain(full, 4, 0);
    drain(full, 4, ~0u);
  }
  __syncthreads();
  if (t.w == NEPI / 32) tmem_dealloc(tm, 512);
}

// ------------------------------------------------------------------ dk, dv and dg
// From a unit's last chunk to its first, with R in registers (row: key, as in memory).
// Rows of the accumulators are the tokens s, columns the tokens t they act on:
//   k q^T, v dO^T (masked, L_ts), v R^T and k R (scaled by e^{gamma_C - gamma_s});
//   dk = P2 q onto the one, dv = P1 dO onto the other; then R's sum scale (e^gamma q)^T dO.
// dg runs along: with rows and cols the sums of A (gdn_lin.cu) over s and over t,
//   dg_u = X + sum_{t >= u} (rows_t + a_t - cols_t - b_t),  X' = X + sum_t (a_t - b_t),
// X = <S, R> behind the chunk, taken from the states themselves at the unit's end.
template <int DK, int DV>
struct BackSm {
  static constexpr uint32_t SLOT = slot_bytes(DK, DV), STATE = DK * DV * 2, HALF_R = DK * 128;
  static constexpr uint32_t V = 0, K = SLOT, Q = 2 * SLOT, DO = 3 * SLOT;
  static constexpr uint32_t R_HI = 4 * SLOT, R_LO = R_HI + STATE, VEC = R_LO + STATE;
  static constexpr uint32_t ROWS = VEC + 2 * sizeof(Vec), COLS = ROWS + 4 * TC * 4,
                            FAR = COLS + 4 * TC * 4, RED = FAR + 4 * TC * 4, BAR = RED + 64;
  static constexpr uint32_t BYTES = BAR + 128 + 1024;
};
// x[0..31] summed over the warp's lanes; lane j returns the sum of x[j].
__device__ __forceinline__ float lane_columns(float* x) {
  const int l = threadIdx.x & 31;
#pragma unroll
  for (int o = 16, n = 16; o >= 1; o >>= 1, n >>= 1) {
    const bool up = (l & o) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? x[i] : x[n + i], keep = up ? x[n + i] : x[i];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return x[0];
}

template <int DK, int DV>
__global__ void __launch_bounds__(NTHR, 1)
    k_lin_tc_back(Args a, const float* dS_out, const float* R_unit, const float* S_unit,
                  const float* S_end, float* dS_in, const float* far, bf* dk, bf* dv, bf* dg,
                  float* dgsum, const __grid_constant__ CUtensorMap mq,
                  const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                  const __grid_constant__ CUtensorMap mo) {
  using L = BackSm<DK, DV>;
  constexpr int NK = DK / 4, NV = DV / 4;
  constexpr uint32_t A1 = 0, A2 = 128, G1 = 256, G2 = 384;  // G1: dk, then R's sum; G2: dv
  chain();
  const int unit = blockIdx.x / a.H, h = blockIdx.x - unit * a.H;
  const size_t uh = (size_t)unit * a.H + h;
  LinUnit u;
  if (!lin_unit(a.m, unit, u)) {
    if (dgsum && threadIdx.x == 0) dgsum[uh] = 0.f;
    return;
  }
  const Who t = who();
  extern __shared__ __align__(1024) unsigned char smraw[];
  unsigned char* sb = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
  unsigned char *r_hi = sb + L::R_HI, *r_lo = sb + L::R_LO;
  Vec* vec = reinterpret_cast<Vec*>(sb + L::VEC);
  float* rows = reinterpret_cast<float*>(sb + L::ROWS);  // [lane quarter][t]
  float* cols = reinterpret_cast<float*>(sb + L::COLS);  // [column group][s]
  float* farb = reinterpret_cast<float*>(sb + L::FAR);   // [column group][s]
  float* red = reinterpret_cast<float*>(sb + L::RED);
  uint64_t* full = reinterpret_cast<uint64_t*>(sb + L::BAR);  // [4] v, k, q, dO
  uint64_t *bar_a = full + 4, *bar_f = full + 5, *bar_c = full + 6, *bar_e = full + 7;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(full + 8);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  const int nch = (u.len + TC - 1) / TC;
  if (t.ctl) {
    for (int i = 0; i < 8; ++i) mbar_init(full + i, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (t.w == NEPI / 32) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *tslot, tl = tm + ((uint32_t)(32 * t.q4) << 16);
  auto load = [&](int kind, int i) {  // a tile of the i-th chunk from the end (control thread)
    if (i >= nch) return;
    const int c = nch - 1 - i;
    const int tok = a.m.cu ? u.row + c * TC : u.at * a.m.unit + c * TC, seq = a.m.cu ? 0 : u.seq;
    unsigned char* to = sb + kind * L::SLOT;
    if (kind == 0)
      load_tile<DV>(to, &mv, h, tok, seq, full);
    else if (kind == 1)
      load_tile<DK>(to, &mk, h, tok, seq, full + 1);
    else if (kind == 2)
      load_tile<DK>(to, &mq, h, tok, seq, full + 2);
    else
      load_tile<DV>(to, &mo, h, tok, seq, full + 3);
  };
  auto raw = [&](int i) {
    const int c = nch - 1 - i;
    return raw_decay(u.row + c * TC, min(TC, u.len - c * TC), h, a.g, a.ldg, a.decay);
  };
  if (t.ctl)
    for (int k = 0; k < 4; ++k) load(k, 0);
  const size_t sh = ((size_t)u.seq * a.H + h) * DK * DV;
  const bool last = u.at == u.n - 1;
  float r[NV];
  if (t.epi) {
    const float* from = last ? (dS_out ? dS_out + sh : nullptr) : R_unit + uh * DK * DV;
    load_state<DK, DV, false, NV>(from, t.lane, NV * t.cq, r);
    if (t.lane < DK) put_split<NV>(r_hi, r_lo, L::HALF_R, t.lane, NV * t.cq, r);
    fence_proxy_async_smem();
    const float* S = !from ? nullptr : last ? S_end + sh : S_unit + (uh + a.H) * DK * DV;
    float x = 0.f;
    if (S && t.lane < DK) {
#pragma unroll
      for (int i = 0; i < NV; i += 4) {
        const float4 y = *reinterpret_cast<const float4*>(S + (size_t)t.lane * DV + NV * t.cq + i);
        x = fmaf(r[i], y.x, x);
        x = fmaf(r[i + 1], y.y, x);
        x = fmaf(r[i + 2], y.z, x);
        x = fmaf(r[i + 3], y.w, x);
      }
    }
    x = lane_sum<32>(x);
    if (t.l == 0) red[t.w] = x;
  } else if (nch) {
    fill_vec(raw(0), vec[0]);
  }
  __syncthreads();
  float X = 0.f, sum = 0.f;  // of warp 0
  if (t.w == 0)
    for (int i = 0; i < NEPI / 32; ++i) X += red[i];
  for (int i = 0; i < nch; ++i) {
    const int c = nch - 1 - i, len = min(TC, u.len - c * TC), ph = i & 1;
    const Vec& v = vec[ph];
    const int row0 = u.row + c * TC, row = row0 + t.lane;
    const bool on = t.lane < len;
    if (len < TC && a.m.cu) {
      if (t.epi) {
        mbar_wait(full + 2, ph, abort);
        mbar_wait(full + 3, ph, abort);
        zero_rows<DK>(sb + L::Q, len, t.tid);
        zero_rows<DV>(sb + L::DO, len, t.tid);
        fence_proxy_async_smem();
      }
      __syncthreads();
    }
    if (t.ctl) {
      const uint32_t sv = smem_u32(sb + L::V), sk = smem_u32(sb + L::K), sq = smem_u32(sb + L::Q),
                     so = smem_u32(sb + L::DO);
      tc_fence_after();
      mbar_wait(full + 1, ph, abort);
      mbar_wait(full + 2, ph, abort);
#pragma unroll 1
      for (int kk = 0; kk < DK / 16; ++kk)
        umma_bf16(tm + A1, kmaj(sk, HALF_TILE, kk), kmaj(sq, HALF_TILE, kk),
                  umma_idesc(128, 128, 0, 0), kk > 0);
      mbar_wait(full + 0, ph, abort);
      mbar_wait(full + 3, ph, abort);
#pragma unroll 1
      for (int kk = 0; kk < DV / 16; ++kk)
        umma_bf16(tm + A2, kmaj(sv, HALF_TILE, kk), kmaj(so, HALF_TILE, kk),
                  umma_idesc(128, 128, 0, 0), kk > 0);
      umma_commit(bar_a);
#pragma unroll 1
      for (int p = 0; p < 2; ++p)
#pragma unroll 1
        for (int kk = 0; kk < DV / 16; ++kk)
          umma_bf16(tm + G1, kmaj(sv, HALF_TILE, kk), kmaj(smem_u32(p ? r_lo : r_hi), L::HALF_R, kk),
                    umma_idesc(128, DK, 0, 0), p || kk);
#pragma unroll 1
      for (int p = 0; p < 2; ++p)
#pragma unroll 1
        for (int kk = 0; kk < DK / 16; ++kk)
          umma_bf16(tm + G2, kmaj(sk, HALF_TILE, kk), mnmaj(smem_u32(p ? r_lo : r_hi), L::HALF_R, kk),
                    umma_idesc(128, DV, 0, 1), p || kk);
      umma_commit(bar_f);
    }
    if (t.epi) {
      uint32_t qh[16], ql[16], p1[16], p2[16];
      mbar_wait(full + 2, ph, abort);
      if (t.lane < DK) weigh(sb + L::Q, t, v.up, a.scale, len, qh, ql);
      mbar_wait(bar_a, ph, abort);
      tc_fence_after();
      // this thread's row s, columns t in [32 cq, 32 cq + 32)
      if (t.cq < t.q4) {
#pragma unroll
        for (int j = 0; j < 16; ++j) p1[j] = p2[j] = 0;
        cols[t.cq * TC + t.lane] = 0.f;
        rows[t.q4 * TC + 32 * t.cq + t.l] = 0.f;
      } else {
        float x[32], y[32], f[4], cs = 0.f;
        tmem_ld<32>(tl + A1 + 32 * t.cq, x);
        tmem_ld<32>(tl + A2 + 32 * t.cq, y);
        const bool diag = t.cq == t.q4;
        const float gh = v.hi[t.lane], gl = v.lo[t.lane];
        const float tb = diag ? 0.f : a.scale * v.tab[t.cq - 1][t.lane];
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          if (diag) {
            const float4 h4 = *reinterpret_cast<const float4*>(v.hi + 32 * t.cq + j);
            const float4 l4 = *reinterpret_cast<const float4*>(v.lo + 32 * t.cq + j);
            const float hh[4] = {h4.x, h4.y, h4.z, h4.w}, ll[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              f[e] = a.scale * __expf((hh[e] - gh) + (ll[e] - gl));
          } else {
            const float4 f4 = *reinterpret_cast<const float4*>(v.row + 32 * t.cq + j);
            f[0] = tb * f4.x, f[1] = tb * f4.y, f[2] = tb * f4.z, f[3] = tb * f4.w;
          }
          float z[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool in = !diag || j + e >= t.l;
            const float px = in ? x[j + e] * f[e] : 0.f, py = in ? y[j + e] * f[e] : 0.f;
            z[e] = !diag || j + e > t.l ? x[j + e] * py : 0.f;
            cs += z[e];
            x[j + e] = px;
            y[j + e] = py;
          }
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            p1[(j + e) / 2] = pack2bf(x[j + e], x[j + e + 1]);
            p2[(j + e) / 2] = pack2bf(y[j + e], y[j + e + 1]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) x[j + e] = z[e];
        }
        cols[t.cq * TC + t.lane] = cs;
        const float rs = lane_columns(x);
        rows[t.q4 * TC + 32 * t.cq + t.l] = rs;
      }
      tc_fence_before();
      named_bar(1 + t.q4, 128);  // the lane quarter's products have been read
      tc_fence_after();
      tmem_st16(tl + A1 + 16 * t.cq, p1);
      tmem_st16(tl + A2 + 16 * t.cq, p2);
      if (t.lane < DK) {
        tmem_st16(tl + A1 + 64 + 16 * t.cq, qh);
        tmem_st16(tl + A2 + 64 + 16 * t.cq, ql);
      }
      mbar_wait(bar_f, ph, abort);
      tc_fence_after();
      const float down = v.down[t.lane];
      {
        float x[NK], b = 0.f;
        tmem_ld<NK>(tl + G1 + NK * t.cq, x);
#pragma unroll
        for (int j = 0; j < NK; j += 8) {
          const uint4 k4 = *reinterpret_cast<const uint4*>(
              at8(sb + L::K, HALF_TILE, t.lane, NK * t.cq + j));
          const uint32_t kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[j + 2 * e] *= down;
            x[j + 2 * e + 1] *= down;
            b = fmaf(__uint_as_float(kk[e] << 16), x[j + 2 * e], b);
            b = fmaf(__uint_as_float(kk[e] & 0xffff0000u), x[j + 2 * e + 1], b);
          }
        }
        farb[t.cq * TC + t.lane] = b;
        tmem_st_f<NK>(tl + G1 + NK * t.cq, x);
      }
      {
        float x[NV];
        tmem_ld<NV>(tl + G2 + NV * t.cq, x);
#pragma unroll
        for (int j = 0; j < NV; ++j) x[j] *= down;
        tmem_st_f<NV>(tl + G2 + NV * t.cq, x);
      }
      tmem_st_wait();
      tc_fence_before();
    }
    __syncthreads();
    if (!t.epi) {
      if (t.l == 0) {
        tc_fence_after();
        const uint32_t sq = smem_u32(sb + L::Q), so = smem_u32(sb + L::DO);
        if (!*abort) {
          load(0, i + 1);
          load(1, i + 1);
        }
#pragma unroll 1
        for (int kk = 0; kk < TC / 16; ++kk)
          umma_ts(tm + G1, tm + A2 + 8 * kk, mnmaj(sq, HALF_TILE, kk), umma_idesc(128, DK, 0, 1), true);
#pragma unroll 1
        for (int kk = 0; kk < TC / 16; ++kk)
          umma_ts(tm + G2, tm + A1 + 8 * kk, mnmaj(so, HALF_TILE, kk), umma_idesc(128, DV, 0, 1), true);
        umma_commit(bar_c);
      }
      __syncwarp();
      if (i + 1 < nch) fill_vec(raw(i + 1), vec[ph ^ 1]);
    } else {
      if (t.w == 0) {  // dg: 4 tokens for each lane
        float x[4], ab = 0.f, suf = 0.f;
#pragma unroll
        for (int j = 3; j >= 0; --j) {
          const int e = 4 * t.l + j;
          float rw = 0.f, cl = 0.f, b = 0.f, f = 0.f;
          if (e < len) {
            f = far[(size_t)(row0 + e) * a.H + h];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              rw += rows[p * TC + e];
              cl += cols[p * TC + e];
              b += farb[p * TC + e];
            }
          }
          ab += f - b;
          x[j] = (suf += (rw - cl) + (f - b));
        }
        float all = suf;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float y = __shfl_down_sync(0xffffffffu, all, o);
          if (t.l + o < 32) all += y;
        }
        const float behind = all - suf + X;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 4 * t.l + j;
          if (e >= len) break;
          if (dg)
            dg[(size_t)(row0 + e) * a.H + h] = __float2bfloat16_rn(x[j] + behind);
          else
            sum += x[j] + behind;
        }
        X += lane_sum<32>(ab);
      }
      mbar_wait(bar_c, ph, abort);
      tc_fence_after();
      float x[NK > NV ? NK : NV];
      tmem_ld<NK>(tl + G1 + NK * t.cq, x);
      if (on) store_row<NK>(dk + ((size_t)row * a.H + h) * DK + NK * t.cq, x, 1.f);
      tmem_ld<NV>(tl + G2 + NV * t.cq, x);
      if (on) store_row<NV>(dv + ((size_t)row * a.H + h) * DV + NV * t.cq, x, 1.f);
      tc_fence_before();
    }
    __syncthreads();
    if (!t.epi) {
      if (t.l == 0) {
        tc_fence_after();
        if (!*abort) load(2, i + 1);
        const uint32_t so = smem_u32(sb + L::DO);
#pragma unroll 1
        for (int p = 0; p < 2; ++p)
#pragma unroll 1
          for (int kk = 0; kk < TC / 16; ++kk)
            umma_ts(tm + G1, tm + (p ? A2 : A1) + 64 + 8 * kk, mnmaj(so, HALF_TILE, kk),
                    umma_idesc(128, DV, 0, 1), p || kk);
        umma_commit(bar_e);
        mbar_wait(bar_e, ph, abort);
        if (!*abort) load(3, i + 1);
      }
      __syncwarp();
    } else {
      mbar_wait(bar_e, ph, abort);
      tc_fence_after();
      if (t.lane < DK) {
        float x[NV];
        tmem_ld<NV>(tl + G1 + NV * t.cq, x);
#pragma unroll
        for (int j = 0; j < NV; ++j) r[j] = fmaf(v.whole, r[j], x[j]);
        put_split<NV>(r_hi, r_lo, L::HALF_R, t.lane, NV * t.cq, r);
        fence_proxy_async_smem();
      }
      tc_fence_before();
    }
    if (__syncthreads_or(*abort != 0)) break;
  }
  if (t.epi && u.at == 0 && dS_in) store_state<DK, DV, false, NV>(dS_in + sh, t.lane, NV * t.cq, r);
  if (t.w == 0 && dgsum) {
    sum = lane_sum<32>(sum);
    if (t.l == 0) dgsum[uh] = sum;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (t.ctl && *abort) {
    *a.status = DEV_TIMEOUT;
    drain(full, 4, 0);
    drain(full, 4, ~0u);
  }
  __syncthreads();
  if (t.w == NEPI / 32) tmem_dealloc(tm, 512);
}

// ------------------------------------------------------------------ host side
// Chunks of a unit. A pass takes as many waves of CTAs as there are units of all heads
// for the GPU's SMs, each as long as a unit (plus about a chunk to start); more than one
// unit of a sequence also needs the units' own sums (y and z only: half a chunk's time)
// and the scan.
constexpr int SMS = 152;
int unit_chunks(const gdn_lin_shape& s, bool packed) {
  const long long nc = std::max(1, (s.T + TC - 1) / TC);
  if (packed) {  // the lengths are known on the device only: some waves of equal units
    const long long all = (nc + s.nseq / 2) * s.H;
    return (int)std::min(64ll, std::max(4ll, (all + SMS * 4 - 1) / (SMS * 4)));
  }
  const long long chains = (long long)s.nseq * s.H;
  double best = 1e300;
  int per = (int)nc;
  for (long long n = 1; n <= nc && n <= 256; ++n) {
    const long long len = (nc + n - 1) / n, units = (nc + len - 1) / len;
    const double waves = (double)((chains * units + SMS - 1) / SMS);
    double cost = waves * (len + 1.0);
    if (units > 1) {
      const double first = (double)((chains * (units - 1) + SMS - 1) / SMS);
      cost += first * (0.5 * len + 1.0) + 2.0 + 0.0135 * chains * units;
    }
    if (cost < best) best = cost, per = (int)len;
  }
  return per;
}

struct TcPlan {
  LinMap m;
  int chunks;
  bool many;  // a sequence may have several units
  int *status, *first, *owner;
  float *whole[2], *dgsum, *D, *E, *S_end, *far;
  size_t bytes;
};
TcPlan tc_plan(const gdn_lin_shape& s, const int* cu, bool packed, bool back, unsigned char* ws) {
  TcPlan p = {};
  p.chunks = unit_chunks(s, packed);
  const int unit = p.chunks * TC, per = std::max(1, (s.T + unit - 1) / unit);
  p.m = {cu, nullptr, nullptr, s.nseq, s.T, unit, per, packed ? per + s.nseq : per * s.nseq};
  p.many = per > 1;
  size_t at = 0;
  auto take = [&](size_t n) {
    unsigned char* r = ws + at;
    at += round256(n);
    return r;
  };
  const size_t uh = (size_t)p.m.cap * s.H, one = (size_t)s.dk * s.dv * sizeof(float);
  p.status = (int*)take(4);
  p.first = (int*)take(packed ? (size_t)(s.nseq + 1) * 4 : 0);
  p.owner = (int*)take(packed ? (size_t)p.m.cap * 4 : 0);
  p.whole[0] = (float*)take(uh * 4);
  p.D = (float*)take(p.many ? uh * one : 0);
  if (back) {
    p.whole[1] = (float*)take(uh * 4);
    p.E = (float*)take(p.many ? uh * one : 0);
    p.dgsum = (float*)take(uh * 4);
    p.S_end = (float*)take((size_t)s.nseq * s.H * one);
    p.far = (float*)take((size_t)s.B * s.T * s.H * 4);
  }
  p.m.first = p.first;
  p.m.owner = p.owner;
  p.bytes = at;
  return p;
}

// [B][T][H][d] bf16 rows `ld` apart as boxes of 64 columns of 128 tokens of one head.
cudaError_t tile_map(CUtensorMap* map, const void* base, const gdn_lin_shape& s, int d, long long ld) {
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)s.H, (cuuint64_t)s.T, (cuuint64_t)s.B};
  const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * s.T};
  return make_tile_map(map, base, dims, strides, TC);
}

template <class K>
cudaError_t allow(K kernel, uint32_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int DK, int DV>
cudaError_t run_tc(const LinCall& c, bool back) {
  const gdn_lin_shape& s = c.s;
  const TcPlan p = tc_plan(s, c.cu, c.cu != nullptr, back, c.ws);
  const Args a = {p.m, s.H, p.chunks, s.scale, (const bf*)c.g, c.decay, s.ldg, p.status};
  CUtensorMap mq, mk, mv, mo;
  cudaError_t e;
  if ((e = tile_map(&mq, c.q, s, DK, s.ldq)) || (e = tile_map(&mk, c.k, s, DK, s.ldk)) ||
      (e = tile_map(&mv, c.v, s, DV, s.ldv)))
    return e;
  if (back && (e = tile_map(&mo, c.dout, s, DV, (long long)s.H * DV))) return e;
  if (c.cu && (e = lin_plan(p.m, p.first, p.owner, p.status, c.st))) return e;
  bool clear = !c.cu;  // the first kernel of an unpacked call resets the status word
  const dim3 grid(p.m.cap * s.H), block(NTHR);
  auto go = [&](auto kernel, uint32_t smem, auto... rest) {
    const cudaError_t f = allow(kernel, smem);
    return f ? f : launch(kernel, grid, block, (int)smem, c.st, 1, a, rest...);
  };
  if (p.many) {
    prof_mark(c.st, "lin_tc_state");
    e = back ? go(k_lin_tc_state<DV, DK, false, true>, StateSm<DV, DK>::BYTES, p.whole[0], p.D, clear, mv, mk)
             : go(k_lin_tc_state<DK, DV, false, false>, StateSm<DK, DV>::BYTES, p.whole[0], p.D, clear, mk, mv);
    if (e) return e;
    clear = false;
    if (back) {
      prof_mark(c.st, "lin_tc_state");
      e = go(k_lin_tc_state<DK, DV, true, false>, StateSm<DK, DV>::BYTES, p.whole[1], p.E, false, mq, mo);
      if (e) return e;
    }
    e = lin_scan(p.m, s, p.whole[0], p.D, c.S_in, p.E, p.whole[1], c.dS_out, back, p.status, c.st);
    if (e) return e;
  }
  prof_mark(c.st, back ? "lin_tc_dq" : "lin_tc_fwd");
  if (!back)
    return go(k_lin_tc_pass<DK, DV, false>, PassSm<DK, DV>::BYTES, c.S_in, p.D, c.S_out, (bf*)c.o,
              (const bf*)nullptr, 0ll, (float*)nullptr, clear, mq, mk, mv);
  e = go(k_lin_tc_pass<DV, DK, true>, PassSm<DV, DK>::BYTES, c.S_in, p.D,
         c.dS_out ? p.S_end : (float*)nullptr, (bf*)c.dq, (const bf*)c.q, s.ldq, p.far, clear, mo, mv, mk);
  if (e) return e;
  prof_mark(c.st, "lin_tc_back");
  e = go(k_lin_tc_back<DK, DV>, BackSm<DK, DV>::BYTES, c.dS_out, p.E, p.D, p.S_end, c.dS_in, p.far,
         (bf*)c.dk, (bf*)c.dv, (bf*)c.dg, c.ddecay ? p.dgsum : nullptr, mq, mk, mv, mo);
  if (e) return e;
  if (c.ddecay) e = col_sum(p.dgsum, p.m.cap, s.H, s.H, c.ddecay, nullptr, nullptr, c.st);
  return e;
}

}  // namespace

// bf16 calls whose rows TMA can take: token rows apart (tensor maps have no zero
// strides), strides below 2^40 bytes. Others take the fp32 kernels.
bool lin_tc_takes(const gdn_lin_shape& s) {
  if (s.dtype != GDN_DTYPE_BF16 || s.T < 1) return false;
  const long long k = (long long)s.H * s.dk, v = (long long)s.H * s.dv;
  const long long most = (1ll << 39) / s.T;
  return s.ldq >= k && s.ldk >= k && s.ldv >= v && s.ldq < most && s.ldk < most && s.ldv < most &&
         (long long)s.nseq * s.H + ((long long)s.T * s.H) / TC < (1ll << 30);
}
size_t lin_tc_bytes(const gdn_lin_shape& s, bool packed, bool back) {
  return tc_plan(s, nullptr, packed, back, nullptr).bytes;
}
cudaError_t lin_tc(const LinCall& c, bool back) {
  if (c.s.dk == 64) return c.s.dv == 64 ? run_tc<64, 64>(c, back) : run_tc<64, 128>(c, back);
  return c.s.dv == 64 ? run_tc<128, 64>(c, back) : run_tc<128, 128>(c, back);
}

}  // namespace gdn

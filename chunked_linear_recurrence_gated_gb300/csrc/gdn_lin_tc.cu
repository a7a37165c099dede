// Linear attention with a decay for each head over whole sequences, bf16
// (gdn_lin_fwd / gdn_lin_bwd, include/gdn_lin.h) on the 5th-generation tensor cores.
//
// One pass over a sequence carries a state through chunks of C = 128 tokens. With x, y,
// z the rows of three tensors and gamma, L, S, R as in gdn_lin.cu,
//   out_t = sum_{s <= t} L_ts (x_t . y_s) z_s + e^{gamma_t} x_t S
//   S <- e^{gamma_C} S + sum_s e^{gamma_C - gamma_s} k_s v_s^T
// is the forward (x, y, z = q, k, v) and dq (dO, v, k with S^T for S). dk, dv and dg come from
// one pass from the end, which carries R.
//
// A sequence is cut into units of chunks, so that there is a CTA for every SM where
// there are few sequences and heads: k_lin_tc_state sums each unit's own contribution to
// the state (it reads y and z only), k_lin_scan joins them along the sequence, and the
// passes then start every unit from its state.
//
// Rounding. Products of inputs are exact in the tensor core's fp32 sums. A state, and a
// weighted operand of a state's update, is taken as two bf16 parts (2^-17 of itself),
// because states leave the call in fp32 and because ddecay, which does too, sums products with
// them; o and dv, which are rounded to bf16 themselves, take a state's first part alone. The
// masked products P = L x y^T are rounded to bf16 once before they meet z, as their result is
// when it is stored.
#include <cuda.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "gdn_internal.cuh"
#include "gdn_lin.cuh"
#include "gdn_mma.cuh"
#include "gdn_umma.cuh"

namespace gdn {
namespace {

typedef __nv_bfloat16 bf;

constexpr int TC = 128;          // tokens of a chunk
constexpr int NEPI = 256;        // 8 warps on the accumulators: 4 lane quarters x 2 column groups
// The kernel of the units' own sums: these, a warp that copies and issues the MMAs, one for
// the weights.
constexpr int CTL = 8, DEC = 9, NTHR = 320;
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
// Columns of this thread's lane from registers; tmem_st_wait before telling others.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// 16 lanes x 16 columns as ldmatrix leaves them: in register 2 k + j thread i has lane
// 8 j + i / 4, column 4 k + i % 4.
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]),
        "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* v) {
#pragma unroll
  for (int i = 0; i < 32; i += 16) {
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
// N values of row r from column c into the tiles of the first parts and (REST) of the rests.
template <int N, bool REST>
__device__ __forceinline__ void put_split(unsigned char* hi, unsigned char* lo, uint32_t half, int r,
                                          int c, const float* v) {
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) split2(v[i + 2 * j], v[i + 2 * j + 1], h[j], l[j]);
    *reinterpret_cast<uint4*>(at8(hi, half, r, c + i)) = make_uint4(h[0], h[1], h[2], h[3]);
    if (REST) *reinterpret_cast<uint4*>(at8(lo, half, r, c + i)) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

// ------------------------------------------------------------------ decay factors
// Weights of a state's update as pairs of bf16, first parts and rests.
struct Weights {
  uint32_t hi[TC / 2], lo[TC / 2];
  float whole, pad[3];  // e^{gamma_C}
};
// Of a chunk: L_ts = row[t] tab[b - 1][s] for t in the block b of 32 behind that of s. Within
// a block it is row[t] own[s] where the block's decay leaves both factors within fp32's range
// (`mild`, a block's), else the exponential of the difference.
struct Vec {
  Weights w;
  float hi[TC], lo[TC];  // gamma, as the sum of two floats
  float row[TC];         // e^{gamma_t - gamma_a}, a the last token before t's block
  float far[TC];         // forward: e^{gamma_t}; back: e^{gamma_C - gamma_t}
  float own[TC];         // e^{gamma_a - gamma_s}
  float tab[3][TC];      // [b - 1][s]: e^{gamma_{32 b - 1} - gamma_s} for s < 32 b
  int mild[4];
};

// The log-decays of a chunk, 4 tokens for each lane of a warp: loaded a chunk ahead of their
// use and not touched before it, so that nothing waits for them.
struct Raw {
  uint32_t x[4];
};
__device__ __forceinline__ Raw raw_decay(int row, int len, int h, const bf* g, long long ldg,
                                         const float* decay) {
  const int l = threadIdx.x & 31;
  Raw r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 4 * l + i;
    r.x[i] = 0;
    if (t < len)
      r.x[i] = decay ? __float_as_uint(decay[h])
                     : *reinterpret_cast<const unsigned short*>(g + (size_t)(row + t) * ldg + h);
  }
  return r;
}
__device__ __forceinline__ float decay_value(uint32_t x, bool wide) {
  return lin_decay(__uint_as_float(wide ? x : x << 16));
}
__device__ __forceinline__ void sum_decay(const Raw& r, bool wide, float* hi, float* lo) {
  Two c[4];
  c[0] = {decay_value(r.x[0], wide), 0.f};
#pragma unroll
  for (int i = 1; i < 4; ++i) c[i] = add_two(c[i - 1], {decay_value(r.x[i], wide), 0.f});
  const Two before = sum_before(c[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const Two x = add_two(before, c[i]);
    hi[i] = x.hi;
    lo[i] = x.lo;
  }
}
// e^{a - b}. The hardware's exponential: off by 2^-21 and by 2^-24 of the exponent, far
// below what bf16 products and 2^-16 of a weight keep of it.
__device__ __forceinline__ float exp_diff(float h1, float l1, float h0, float l0) {
  return __expf((h1 - h0) + (l1 - l0));
}
// e^{gamma_C}: it is multiplied up over all chunks that a state passes, so it is good to the
// last bits (2^-23 of itself).
__device__ __forceinline__ float exp_whole(float h, float l) {
  const float e = expf(h);
  return fmaf(e, l, e);
}
// Weights of the state's update: to the chunk's end, or (BACK) scale times from its start.
template <bool BACK>
__device__ __forceinline__ void fill_weights(const float* hi, const float* lo, float scale, Weights& w) {
  const int l = threadIdx.x & 31;
  const float eh = __shfl_sync(0xffffffffu, hi[3], 31), el = __shfl_sync(0xffffffffu, lo[3], 31);
  float o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = BACK ? scale * exp_diff(hi[i], lo[i], 0.f, 0.f) : exp_diff(eh, el, hi[i], lo[i]);
#pragma unroll
  for (int i = 0; i < 2; ++i) split2(o[2 * i], o[2 * i + 1], w.hi[2 * l + i], w.lo[2 * l + i]);
  if (l == 0) w.whole = exp_whole(eh, el);
}
// One of two warps' part of a chunk's factors (each sums gamma for itself: one warp took
// 9 thousand cycles for all of them, twice what the rest of a chunk needs).
constexpr int DEC_WARPS = 2;
template <bool BACK>
__device__ __forceinline__ void fill_vec(int part, const Raw& r, bool wide, float scale, Vec& v) {
  const int l = threadIdx.x & 31, blk = l >> 3;  // this lane's block of 32 tokens
  float hi[4], lo[4], o[4] = {};
  sum_decay(r, wide, hi, lo);
  auto put = [&](float* to) {
    reinterpret_cast<float4*>(to)[l] = make_float4(o[0], o[1], o[2], o[3]);
  };
  auto put_tab = [&](int b) {
    const float eh = __shfl_sync(0xffffffffu, hi[3], 8 * b + 7);
    const float el = __shfl_sync(0xffffffffu, lo[3], 8 * b + 7);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = blk <= b ? exp_diff(eh, el, hi[i], lo[i]) : 0.f;
    put(v.tab[b]);
  };
  if (part == 0) {
    put_tab(0);
    fill_weights<BACK>(hi, lo, scale, v.w);
    const float eh = __shfl_sync(0xffffffffu, hi[3], 31), el = __shfl_sync(0xffffffffu, lo[3], 31);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = BACK ? exp_diff(eh, el, hi[i], lo[i]) : exp_diff(hi[i], lo[i], 0.f, 0.f);
    put(v.far);
  } else {
    put_tab(1);
    put_tab(2);
    reinterpret_cast<float4*>(v.hi)[l] = make_float4(hi[0], hi[1], hi[2], hi[3]);
    reinterpret_cast<float4*>(v.lo)[l] = make_float4(lo[0], lo[1], lo[2], lo[3]);
    const int from = max(8 * blk - 1, 0);  // the lane with the end of the block before
    float ah = __shfl_sync(0xffffffffu, hi[3], from), al = __shfl_sync(0xffffffffu, lo[3], from);
    if (blk == 0) ah = al = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = exp_diff(hi[i], lo[i], ah, al);
    put(v.row);
    bool small = true;  // every factor between e^-80 and e^80
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      small = small && o[i] > 1.9e-35f && o[i] < 5.5e34f;
      o[i] = exp_diff(ah, al, hi[i], lo[i]);
    }
    put(v.own);
    const uint32_t all = __ballot_sync(0xffffffffu, small);
    if (l < 4) v.mild[l] = (all >> (8 * l) & 0xffu) == 0xffu;
  }
}

// ------------------------------------------------------------------ shared pieces
struct Who {  // a thread's part of an accumulator: row `lane`, column group cg
  int tid, w, l, q4, cg, lane;
};
__device__ __forceinline__ Who who() {
  Who t;
  t.tid = threadIdx.x;
  t.w = t.tid >> 5;
  t.l = t.tid & 31;
  t.q4 = t.w & 3;
  t.cg = (t.w >> 2) & 1;
  t.lane = 32 * t.q4 + t.l;
  return t;
}
// A warp's part of an event is done: its threads' tensor-memory accesses and, with SMEM,
// their writes of operand tiles.
template <bool SMEM>
__device__ __forceinline__ void warp_done(uint64_t* bar) {
  if (SMEM) fence_proxy_async_smem();
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// The warps of the own sums' kernel meet; true if any has seen a wait run out.
__device__ __forceinline__ bool meet(volatile int* abort) { return __syncthreads_or(*abort) != 0; }

// What the kernels of a call share.
struct Args {
  LinMap m;
  int H;
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
// dg needs e^{gamma_C} <S, R>, S the state before a chunk and R the gradient of the one behind
// it, and they are never together: dq leaves S of every chunk where both are more than zeros
// in the workspace, as units' states.
__device__ __forceinline__ bool crossed(const LinUnit& u, int c, int nch, bool in, bool out) {
  return (c > 0 || u.at > 0 || in) && (c < nch - 1 || u.at < u.n - 1 || out);
}
// Its index: one more for each chunk, as later sequences start on later rows.
__device__ __forceinline__ size_t crossing(const LinUnit& u, int c) {
  return (size_t)((u.row + c * TC) / TC + u.seq);
}
__device__ __forceinline__ uint32_t bf2(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ __nv_bfloat162 bf2(uint32_t x) {
  return *reinterpret_cast<__nv_bfloat162*>(&x);
}
// The weighted transpose of a warp's 32 columns of a tile (64 tokens) into tensor memory,
// an operand with the tokens as reduced dimension, 32 of them STEP columns apart: first parts
// at `to`, rests at `rest`. With y a value and w = wh + wl its weight, hi = y wh rounded, and y wh - hi + y wl is
// the rest: fused multiply-adds of pairs, the first difference exact.
template <int STEP = 16>
__device__ __forceinline__ void weigh(const unsigned char* tile, const Who& t, const Weights& w,
                                      int len, uint32_t to, uint32_t rest) {
  const uint32_t base = smem_u32(tile) + (t.q4 >> 1) * HALF_TILE;
  const int piece = (t.q4 & 1) * 4 + (t.l >> 3), r7 = t.l & 7;
  const uint32_t at = base + (64 * t.cg + r7) * 128 + ((piece ^ r7) << 4);
  const int p0 = 32 * t.cg + (t.l & 3);
#pragma unroll 1
  for (int g = 0; g < 2; ++g) {  // 32 tokens
    uint32_t hi[2][8], lo[2][8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t y[4];
      ldsm_x4_t(at + (32 * g + 8 * k) * 128, y[0], y[1], y[2], y[3]);
      const int p = p0 + 16 * g + 4 * k;
      if (len < TC) {
        const uint32_t keep = (2 * p < len ? 0xffffu : 0u) | (2 * p + 1 < len ? 0xffff0000u : 0u);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] &= keep;
      }
      const __nv_bfloat162 wh = bf2(w.hi[p]), wl = bf2(w.lo[p]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 v = bf2(y[j]), a = __hmul2_rn(v, wh);
        hi[j >> 1][2 * k + (j & 1)] = bf2(a);
        lo[j >> 1][2 * k + (j & 1)] = bf2(__hfma2(v, wl, __hfma2(v, wh, __hneg2(a))));
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // 16 lanes
      tmem_st_frag(to + (16u * j << 16) + STEP * (2 * t.cg + g), hi[j]);
      tmem_st_frag(rest + (16u * j << 16) + STEP * (2 * t.cg + g), lo[j]);
    }
  }
}
// This thread's N elements (row lane, columns c0..) of a state [DK][DV].
template <int DK, int DV, int N>
__device__ __forceinline__ void load_state(const float* from, int lane, int c0, float* s) {
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = 0.f;
  if (!from || lane >= DK) return;
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 x = *reinterpret_cast<const float4*>(from + (size_t)lane * DV + c0 + i);
    s[i] = x.x, s[i + 1] = x.y, s[i + 2] = x.z, s[i + 3] = x.w;
  }
}
template <int DK, int DV, int N>
__device__ __forceinline__ void store_state(float* to, int lane, int c0, const float* s) {
  if (!to || lane >= DK) return;
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *reinterpret_cast<float4*>(to + (size_t)lane * DV + c0 + i) =
        make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
}
// The same of a unit's state in the workspace, [DZ / 4][DY][4]: whole lines for a warp, where
// rows of DZ would take 32 pieces of 16 bytes (8 thousand cycles for 64 KB).
template <int DY, int N>
__device__ __forceinline__ void load_unit(const float* from, int lane, int c0, float* s) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (lane < DY) x = *reinterpret_cast<const float4*>(from + ((size_t)(c0 + i) / 4 * DY + lane) * 4);
    s[i] = x.x, s[i + 1] = x.y, s[i + 2] = x.z, s[i + 3] = x.w;
  }
}
template <int DY, int N>
__device__ __forceinline__ void store_unit(float* to, int lane, int c0, const float* s) {
  if (lane >= DY) return;
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *reinterpret_cast<float4*>(to + ((size_t)(c0 + i) / 4 * DY + lane) * 4) =
        make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
}
// s <- by s + an accumulator's N columns (an even number of 32s).
template <int N>
__device__ __forceinline__ void add_state(uint32_t taddr, float by, float* s) {
#pragma unroll
  for (int i = 0; i < N; i += 32) {
    float d[32];
    tmem_ld32(taddr + i, d);
#pragma unroll
    for (int j = 0; j < 32; ++j) s[i + j] = fmaf(by, s[i + j], d[j]);
  }
}
// An accumulator's N columns times `by` as packed bf16.
template <int N>
__device__ __forceinline__ void take_row(uint32_t taddr, float by, uint32_t* p) {
#pragma unroll
  for (int i = 0; i < N; i += 32) {
    float v[32];
    tmem_ld32(taddr + i, v);
#pragma unroll
    for (int j = 0; j < 16; ++j) p[i / 2 + j] = pack2bf(by * v[2 * j], by * v[2 * j + 1]);
  }
}
// These rows into memory through 2 KB of shared memory of the warp's own (32 rows of 32
// columns, 64-byte swizzle) that the copy engine stores: it writes while the warp goes on,
// which would wait for its own stores (an SM sends about 25 bytes a cycle). direct: a tile
// whose last rows are another sequence's, stored row by row.
template <int N>
__device__ __forceinline__ void leave_rows(const uint32_t* p, unsigned char* stage, const CUtensorMap* map,
                                           int col, int h, int tok, int seq, bf* out, bool direct,
                                           int rows) {
  const int l = threadIdx.x & 31;
  if (direct) {
    if (l < rows)
#pragma unroll
      for (int i = 0; i < N / 2; i += 4)
        *reinterpret_cast<uint4*>(out + 2 * i) = make_uint4(p[i], p[i + 1], p[i + 2], p[i + 3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < N; i += 32) {
    if (l == 0) bulk_wait_read();  // the rows before have left
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t* u = p + i / 2 + 4 * k;
      *reinterpret_cast<uint4*>(stage + l * 64 + ((k ^ (l >> 1 & 3)) << 4)) =
          make_uint4(u[0], u[1], u[2], u[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (l == 0) {
      if (rows > 0)
        asm volatile(
            "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];\n" ::"l"(
                reinterpret_cast<uint64_t>(map)),
            "r"(col + i), "r"(h), "r"(tok), "r"(seq), "r"(smem_u32(stage))
            : "memory");
      bulk_commit();
    }
  }
}
constexpr uint32_t STAGE = 2048;  // bytes of a warp
// After a wait that ran out: this CTA's copies still under way are waited for, with a
// limit, before its shared memory is given up.
__device__ __forceinline__ void drain(uint64_t* bars, int n, uint32_t phases) {
  for (int i = 0; i < n; ++i) {
    int off = 0;
    mbar_wait(bars + i, (phases >> i) & 1, &off, 1ll << 24);
  }
}
// Barriers, the abort flag and tensor memory; returns its address.
__device__ __forceinline__ uint32_t set_up(const Who& t, int ctl, uint64_t* bars, int n, int decs,
                                           int teams, int both, uint32_t* tslot, volatile int* abort) {
  // n barriers (the last `decs` events of the decay warps), then events of the 8 warps of a
  // team, then of two teams
  if (t.tid == ctl * 32) {
    for (int i = 0; i < n + teams + both; ++i)
      mbar_init(bars + i, i < n - decs ? 1 : i < n ? DEC_WARPS : i < n + teams ? 8 : 16);
    *abort = 0;
    fence_mbar_init();
  }
  if (t.tid < 8) reinterpret_cast<volatile int*>(tslot + 2)[t.tid] = 0;  // counters behind the flag
  if (t.w == ctl) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return *tslot;
}
__device__ __forceinline__ void tear_down(const Who& t, int ctl, uint64_t* full, int n, uint32_t tm,
                                          volatile int* abort, int* status) {
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (t.tid == ctl * 32 && *abort) {
    *status = DEV_TIMEOUT;
    drain(full, n, 0);
    drain(full, n, ~0u);
  }
  __syncthreads();
  if (t.w == ctl) {
    __syncwarp();
    tmem_dealloc(tm, 512);
  }
}

constexpr uint32_t slot_bytes(int a, int b) { return (a > b ? a : b) * TC * 2; }

// ------------------------------------------------------------------ a unit's own sum
// E = sum over the unit of (its decay to the unit's end, or REV: from the unit's start,
// times scale) y z^T, and the unit's whole decay. Not for a sequence's last unit (REV: its
// first), whose state nobody starts from. The MMAs of a chunk run under the weighing of
// the next one and the update from the one before; three chunks' tiles are in flight. Bound by
// the loads and the weighing side by side: 53 us for k and v of 32768 tokens x 16 heads (5.1
// TB/s; issue 28 %, tensor pipe 29 %).
template <int DY, int DZ>
struct StateSm {
  static constexpr int THREADS = NTHR;
  static constexpr uint32_t SLOT = slot_bytes(DY, DZ), STAGES = 3;
  static constexpr uint32_t VEC = 2 * STAGES * SLOT, BAR = VEC + 4 * sizeof(Weights);
  static constexpr uint32_t BYTES = BAR + 128 + 1024;
};
template <int DY, int DZ, bool REV>
__global__ void __launch_bounds__(NTHR, 1)
    k_lin_tc_state(Args a, float* whole, float* out, bool clear, const __grid_constant__ CUtensorMap my,
                   const __grid_constant__ CUtensorMap mz) {
  using L = StateSm<DY, DZ>;
  constexpr int N = DZ / 2, ST = L::STAGES;
  constexpr uint32_t D0 = 0, Y0 = 256;  // two accumulators, two operands of two parts
  chain();
  if (clear && blockIdx.x == 0 && threadIdx.x == 0) *a.status = DEV_OK;
  const int nth = blockIdx.x / a.H, h = blockIdx.x - nth * a.H, unit = lin_nth(a.m, nth);
  LinUnit u;
  if (!lin_unit(a.m, unit, u)) return;
  if (u.at == (REV ? 0 : u.n - 1)) return;
  const Who t = who();
  extern __shared__ __align__(1024) unsigned char smraw[];
  unsigned char* sb = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
  Weights* vec = reinterpret_cast<Weights*>(sb + L::VEC);
  uint64_t* full = reinterpret_cast<uint64_t*>(sb + L::BAR);  // [ST]
  uint64_t* done = full + ST;                                 // [2] MMAs of a chunk
  uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 2);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  const int nch = (u.len + TC - 1) / TC;
  auto chunk = [&](int i) { return REV ? nch - 1 - i : i; };
  auto raw = [&](int i) {
    const int c = chunk(i);
    return raw_decay(u.row + c * TC, min(TC, u.len - c * TC), h, a.g, a.ldg, a.decay);
  };
  Raw ahead = {};  // of the first chunk, on its way while barriers and tensor memory are set up
  if (t.w == DEC && nch) ahead = raw(0);
  const uint32_t tm = set_up(t, CTL, full, ST + 2, 0, 0, 0, tslot, abort);
  auto tile = [&](int i) { return sb + 2 * (i % ST) * L::SLOT; };  // y, and z a slot behind it
  if (t.w < CTL) {
    const uint32_t tl = tm + ((uint32_t)(32 * t.q4) << 16);
    float s[N], all = 1.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = 0.f;
    auto update = [&](int i) {  // from chunk i's accumulator
      mbar_wait(done + (i & 1), (i >> 1) & 1, abort);
      tc_fence_after();
      const float wh = vec[i & 3].whole;
      if (t.lane < DY) add_state<N>(tl + D0 + 128 * (i & 1) + N * t.cg, wh, s);
      all *= wh;
      tc_fence_before();
    };
    meet(abort);
    for (int i = 0; i < nch; ++i) {
      const int len = min(TC, u.len - chunk(i) * TC);
      mbar_wait(full + i % ST, (i / ST) & 1, abort);
      if (t.lane < DY) {
        weigh(tile(i), t, vec[i & 3], len, tl + Y0 + 128 * (i & 1), tl + Y0 + 128 * (i & 1) + 64);
        tmem_st_wait();
      }
      if (len < TC && a.m.cu) {
        zero_rows<DZ>(tile(i) + L::SLOT, len, t.tid);
        fence_proxy_async_smem();
      }
      tc_fence_before();
      if (meet(abort)) break;
      if (i) update(i - 1);
    }
    if (nch) update(nch - 1);
    const size_t uh = (size_t)unit * a.H + h;
    store_unit<DY, N>(out + uh * DY * DZ, t.lane, N * t.cg, s);
    if (t.tid == 0) whole[uh] = all;
  } else if (t.w == CTL) {
    auto load = [&](int i) {
      const int c = chunk(i);
      const int tok = a.m.cu ? u.row + c * TC : u.at * a.m.unit + c * TC, seq = a.m.cu ? 0 : u.seq;
      uint64_t* bar = full + i % ST;
      mbar_arrive_expect_tx(bar, (DY + DZ) * TC * 2);
#pragma unroll
      for (int e = 0; e < DY; e += 64)
        tma_load_4d(tile(i) + (e >> 6) * HALF_TILE, &my, e, h, tok, seq, bar);
#pragma unroll
      for (int e = 0; e < DZ; e += 64)
        tma_load_4d(tile(i) + L::SLOT + (e >> 6) * HALF_TILE, &mz, e, h, tok, seq, bar);
    };
    if (t.l == 0)
      for (int i = 0; i < min(nch, ST); ++i) load(i);
    __syncwarp();
    meet(abort);
    for (int i = 0; i < nch; ++i) {
      if (meet(abort)) break;
      if (t.l == 0) {
        tc_fence_after();
        mbar_wait(full + i % ST, (i / ST) & 1, abort);
        const uint32_t z = smem_u32(tile(i) + L::SLOT);
#pragma unroll 1
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int kk = 0; kk < TC / 16; ++kk)
            umma_ts(tm + D0 + 128 * (i & 1), tm + Y0 + 128 * (i & 1) + 64 * p + 8 * kk,
                    mnmaj(z, HALF_TILE, kk), umma_idesc(128, DZ, 0, 1), p || kk);
        umma_commit(done + (i & 1));
        if (i) {  // the chunk before is done with its tiles
          mbar_wait(done + ((i - 1) & 1), ((i - 1) >> 1) & 1, abort);
          if (i - 1 + ST < nch && !*abort) load(i - 1 + ST);
        }
      }
      __syncwarp();
    }
  } else {
    auto fill = [&](const Raw& r, int i) {
      float hi[4], lo[4];
      sum_decay(r, a.decay != nullptr, hi, lo);
      fill_weights<REV>(hi, lo, a.scale, vec[i & 3]);
    };
    if (nch) {
      const Raw second = nch > 1 ? raw(1) : Raw{};
      fill(ahead, 0);
      if (nch > 1) fill(second, 1);
      if (nch > 2) ahead = raw(2);
    }
    meet(abort);
    for (int i = 0; i < nch; ++i) {
      if (meet(abort)) break;
      // two ahead: visible behind the next chunk's meeting; four kept, for the chunk before
      // this one is still to be added
      if (i + 2 < nch) fill(ahead, i + 2);
      if (i + 3 < nch) ahead = raw(i + 3);
    }
  }
  tear_down(t, CTL, full, ST, tm, abort, a.status);
}

// ------------------------------------------------------------------ forward and dq
// Two teams of 8 warps work on a chunk's accumulators at the same time, each 128 rows x 2
// groups of columns, and tell the warp that issues the MMAs by events. One takes P = x y^T
// (masked, in place), scales x S and, once P z is on it, the result; the other weighs k and
// adds up the state. In one team of either size the two strings of loads, arithmetic and
// waits stood one behind the other (7 to 10 thousand cycles a chunk).
//   MMAs: x S (state ready, result read) | P z, the state's sum (P, x S and k ready) | x y^T
//   of the next chunk (P z done)
// The tiles x, y, z take the slots in turn, each as soon as the one before is done with it.
// Bound by the chain products -> mask -> P z -> result of a chunk, 7.5 thousand cycles: 115 us
// for the forward of 32768 tokens x 16 heads of 128 (4.6 TB/s; issue 41 %, tensor pipe 36 %),
// 175 us for dq, whose state's product has two parts and which leaves 64 KB of states a chunk
// for dg (153 without).
// The warp that issues the MMAs keeps asking the barriers: beside the warps of lane quarter 3,
// which have the least to do with P (on the scheduler of quarter 0 the backward took 588 us
// instead of 578 for 32768 tokens x 16 heads).
constexpr int P_LOAD = 16, P_DEC = 17, P_CTL = 19, P_NTHR = 640;
// Registers of the two teams' warpgroups and of the last one: together within what is launched.
constexpr int P_REGS = 96, TEAM_REGS = 104, LAST_REGS = 64;
static_assert((P_NTHR - 128) * TEAM_REGS + 128 * LAST_REGS <= P_NTHR * P_REGS, "the pool of the launch");
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(TEAM_REGS));
}
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(LAST_REGS));
}
constexpr long long WAIT_LIMIT = 1ll << 32;  // cycles without progress (mbar_wait's own limit)
static_assert(P_DEC + DEC_WARPS == P_CTL && (P_CTL + 1) * 32 == P_NTHR, "the last warpgroup");
template <int DY, int DZ, bool DQ>
struct PassSm {
  static constexpr int THREADS = P_NTHR;
  // the forward, without second parts of the state, has room for the next chunk's y ahead of
  // the slot of this one's x
  static constexpr int SLOTS = DQ ? 4 : 5;
  static constexpr int DK = DQ ? DZ : DY, DV = DQ ? DY : DZ;
  static constexpr uint32_t SLOT = slot_bytes(DY, DZ), STATE = DY * DZ * 2, HALF_S = DK * 128;
  static constexpr uint32_t S_HI = SLOTS * SLOT, S_LO = S_HI + STATE, VEC = S_LO + (DQ ? STATE : 0);
  static constexpr uint32_t PART = VEC + 2 * sizeof(Vec), OUT = (PART + 4 * TC * 4 + 511) / 512 * 512;
  static constexpr uint32_t BAR = OUT + 8 * STAGE, BYTES = BAR + 192 + 1024;
};
template <int DY, int DZ, bool DQ>
__global__ void __launch_bounds__(P_NTHR, 1)
    k_lin_tc_pass(Args a, const float* S_in, const float* S_unit, float* S_out, bf* out, const bf* q,
                  long long ldq, float* far, float* S_chunk, bool end, bool clear,
                  const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my,
                  const __grid_constant__ CUtensorMap mz, const __grid_constant__ CUtensorMap mo) {
  using L = PassSm<DY, DZ, DQ>;
  constexpr int SL = L::SLOTS, DK = L::DK, DV = L::DV;
  constexpr int N = DZ / 2, NS = DV / 2;  // columns of a thread: of the result, of the state
  constexpr int KEYS = DQ ? 2 : 1, VALUES = 3 - KEYS;  // which of a chunk's tiles are k's and v's
  constexpr uint32_t P0 = 0, O0 = 128, Y0 = 256, D0 = 384;
  chain();
  if (clear && blockIdx.x == 0 && threadIdx.x == 0) *a.status = DEV_OK;
  const int nth = blockIdx.x / a.H, h = blockIdx.x - nth * a.H, unit = lin_nth(a.m, nth);
  LinUnit u;
  if (!lin_unit(a.m, unit, u)) return;
  const Who t = who();
  extern __shared__ __align__(1024) unsigned char smraw[];
  unsigned char* sb = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
  unsigned char *s_hi = sb + L::S_HI, *s_lo = sb + L::S_LO;
  Vec* vec = reinterpret_cast<Vec*>(sb + L::VEC);
  float* part = reinterpret_cast<float*>(sb + L::PART);
  uint64_t* full = reinterpret_cast<uint64_t*>(sb + L::BAR);  // [SL]
  // MMAs: x y^T, x S, P z, the state's sum; decay factors are there [2 buffers]
  uint64_t *bar_p = full + SL, *bar_s = bar_p + 1, *bar_o = bar_p + 2, *bar_d = bar_p + 3, *ev_v = bar_p + 4;
  // events of a team: P and x S ready; result read; k weighed; state ready; of both: decay
  // factors used [2]. A barrier's next phase but one always depends on all who wait for it,
  // so nobody can miss a phase.
  uint64_t *ev_p = ev_v + 2, *ev_o = ev_p + 1, *ev_y = ev_p + 2, *ev_s = ev_p + 3, *ev_u = ev_p + 4;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(ev_u + 2);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  // what the issuing thread has seen done: P z, the state's sum, x S, x y^T, k weighed
  volatile int* seen = reinterpret_cast<volatile int*>(tslot + 2);
  const int nch = (u.len + TC - 1) / TC;
  auto raw = [&](int c) {
    return raw_decay(u.row + c * TC, min(TC, u.len - c * TC), h, a.g, a.ldg, a.decay);
  };
  const bool decs = t.w >= P_DEC && t.w < P_DEC + DEC_WARPS;
  Raw ahead = {};  // of the first chunk, on its way while barriers and tensor memory are set up
  if (decs && nch) ahead = raw(0);
  const uint32_t tm = set_up(t, P_CTL, full, SL + 6, 2, 4, 2, tslot, abort);
  const uint32_t tl = tm + ((uint32_t)(32 * t.q4) << 16);
  auto tile = [&](int n) { return sb + n % SL * L::SLOT; };  // tile n: x, y or z of chunk n / 3
  auto wait_tile = [&](int n) { return mbar_wait(full + n % SL, n / SL & 1, abort); };
  // After a wait that ran out every role goes through its chunks without waiting.
  if (t.w < 8) {  // ---- P and the result
    more_registers();
    for (int c = 0; c < nch; ++c) {
      const int len = min(TC, u.len - c * TC), ph = c & 1;
      const Vec& v = vec[ph];
      const int row = u.row + c * TC + t.lane;  // of this thread's result
      const bool on = t.lane < len;
      mbar_wait(ev_v + ph, (c >> 1) & 1, abort);
      // This thread's row t, columns [64 cg, 64 cg + 64) of x y^T, 32 at a time; as bf16 pairs
      // into the first half of the same columns. So the second group, whose pairs go where the
      // first one's products are, waits until those have been read. The factors are loaded
      // together: under the MMAs a load of shared memory takes hundreds of cycles.
      const float r = v.row[t.lane];
      const bool mild = v.mild[t.q4];
#pragma unroll 1
      for (int j = 0; j < 2; ++j) {
        const int blk = 2 * t.cg + j;
        float f[32], x[32];
        if (blk <= t.q4) {
          const float* tb = (blk == t.q4 ? v.own : v.tab[t.q4 - 1]) + 32 * blk;
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 y = *reinterpret_cast<const float4*>(tb + i);
            f[i] = y.x, f[i + 1] = y.y, f[i + 2] = y.z, f[i + 3] = y.w;
          }
        }
        if (j == 0) {
          mbar_wait(bar_p, ph, abort);
          tc_fence_after();
        }
        uint32_t p[16];
        if (blk > t.q4) {
#pragma unroll
          for (int i = 0; i < 16; ++i) p[i] = 0;
        } else {
          tmem_ld32(tl + P0 + 32 * blk, x);
          if (blk < t.q4) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) p[i / 2] = pack2bf(x[i] * (r * f[i]), x[i + 1] * (r * f[i + 1]));
          } else if (mild) {
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              p[i / 2] = pack2bf(i <= t.l ? x[i] * (r * f[i]) : 0.f,
                                 i < t.l ? x[i + 1] * (r * f[i + 1]) : 0.f);
          } else {
            const float gh = v.hi[t.lane], gl = v.lo[t.lane];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 h2 = *reinterpret_cast<const float2*>(v.hi + 32 * blk + i);
              const float2 l2 = *reinterpret_cast<const float2*>(v.lo + 32 * blk + i);
              p[i / 2] = pack2bf(i <= t.l ? x[i] * __expf((gh - h2.x) + (gl - l2.x)) : 0.f,
                                 i < t.l ? x[i + 1] * __expf((gh - h2.y) + (gl - l2.y)) : 0.f);
            }
          }
        }
        if (j != t.cg) {  // the first group behind its second read, the second before it writes
          tc_fence_before();
          named_bar(2 + t.q4, 64);
          tc_fence_after();
        }
        tmem_st16(tl + P0 + 32 * t.cg + 16 * j, p);
      }
      // this thread's part of q's row, and of the next chunk's into the L2
      uint4 qr[DQ ? N / 8 : 1];
      if (DQ) {
        const bf* from = q + (size_t)row * ldq + (size_t)h * DZ + N * t.cg;
#pragma unroll
        for (int j = 0; j < N / 8; ++j) {
          qr[j] = make_uint4(0, 0, 0, 0);
          if (on) qr[j] = reinterpret_cast<const uint4*>(from)[j];
        }
        if ((c + 1) * TC + t.lane < u.len)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(from + (size_t)TC * ldq));
      }
      mbar_wait(bar_s, ph, abort);
      tc_fence_after();
      const float up = v.far[t.lane];
      float f = 0.f;  // q_t . (far part of dq_t)
#pragma unroll(DQ ? 2 : 1)
      for (int i = 0; i < N; i += 32) {
        float o[32];
        tmem_ld32(tl + O0 + N * t.cg + i, o);
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] *= up;
        tmem_st32(tl + O0 + N * t.cg + i, o);
        if (DQ) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 y = qr[i / 8 + j];
            const uint32_t w4[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f = fmaf(__uint_as_float(w4[e] << 16), o[8 * j + 2 * e], f);
              f = fmaf(__uint_as_float(w4[e] & 0xffff0000u), o[8 * j + 2 * e + 1], f);
            }
          }
        }
      }
      tmem_st_wait();
      warp_done<false>(ev_p);
      if (t.l == 0) mbar_arrive(ev_u + ph);
      if (DQ) {
        float* sums = part + 2 * TC * ph;
        sums[t.cg * TC + t.lane] = a.scale * f;
        named_bar(6, 256);
        if (t.tid < len) far[(size_t)row * a.H + h] = sums[t.tid] + sums[TC + t.tid];
      }
      mbar_wait(bar_o, ph, abort);
      tc_fence_after();
      const int tok = (a.m.cu ? u.row : u.at * a.m.unit) + c * TC + 32 * t.q4;
      uint32_t res[N / 2];
      take_row<N>(tl + O0 + N * t.cg, a.scale, res);
      warp_done<false>(ev_o);
      leave_rows<N>(res, sb + L::OUT + t.w * STAGE, &mo, N * t.cg, h, tok, a.m.cu ? 0 : u.seq,
                    out + ((size_t)row * a.H + h) * DZ + N * t.cg, len < TC && a.m.cu, len - 32 * t.q4);
    }
    if (t.l == 0) bulk_wait_all();
  } else if (t.w < 16) {  // ---- the state
    more_registers();
    const size_t sh = ((size_t)u.seq * a.H + h) * DY * DZ, uh = ((size_t)unit * a.H + h) * DY * DZ;
    float s[NS];
    // S_out may be S_in: a sequence's last unit writes it at any time, so the first of many
    // starts from the scan's copy
    if (u.n > 1)
      load_unit<DK, NS>(S_unit + uh, t.lane, NS * t.cg, s);
    else
      load_state<DK, DV, NS>(S_in ? S_in + sh : nullptr, t.lane, NS * t.cg, s);
    if (t.lane < DK) put_split<NS, DQ>(s_hi, s_lo, L::HALF_S, t.lane, NS * t.cg, s);
    warp_done<true>(ev_s);
    for (int c = 0; c < nch; ++c) {
      const int len = min(TC, u.len - c * TC), n0 = 3 * c, ph = c & 1;
      const Vec& v = vec[ph];
      // ahead of the weighing (behind it dq takes 185 us instead of 175 for 32768 x 16 heads)
      if (DQ && crossed(u, c, nch, S_in, end))
        store_unit<DK, NS>(S_chunk + (crossing(u, c) * a.H + h) * DK * DV, t.lane, NS * t.cg, s);
      mbar_wait(ev_v + ph, (c >> 1) & 1, abort);
      wait_tile(n0 + KEYS);
      if (len < TC && a.m.cu) {  // rows of the next sequence would meet zeros, which NaN survives
        wait_tile(n0 + VALUES);
        zero_rows<DV>(tile(n0 + VALUES), len, t.tid - 256);
        if (DQ) {
          zero_rows<DK>(tile(n0 + KEYS), len, t.tid - 256);
          named_bar(7, 256);
        }
      }
      if (t.lane < DK) {
        weigh(tile(n0 + KEYS), t, v.w, len, tl + Y0, tl + Y0 + 64);
        tmem_st_wait();
      }
      warp_done<true>(ev_y);
      mbar_wait(bar_d, ph, abort);
      tc_fence_after();
      if (t.lane < DK) {
        add_state<NS>(tl + D0 + NS * t.cg, v.w.whole, s);
        mbar_wait(bar_s, ph, abort);  // x S has read the tiles
        put_split<NS, DQ>(s_hi, s_lo, L::HALF_S, t.lane, NS * t.cg, s);
      }
      warp_done<true>(ev_s);
      if (t.l == 0) mbar_arrive(ev_u + ph);
    }
    if (!DQ && u.at == u.n - 1 && S_out) store_state<DK, DV, NS>(S_out + sh, t.lane, NS * t.cg, s);
  } else {
    fewer_registers();
    if (t.w == P_LOAD && t.l == 0) {  // ---- copies
      auto load = [&](int n) {
        const int c = n / 3, kind = n - 3 * c;
        if (c >= nch || *abort) return;
        const int tok = a.m.cu ? u.row + c * TC : u.at * a.m.unit + c * TC, seq = a.m.cu ? 0 : u.seq;
        uint64_t* bar = full + n % SL;
        if (kind == 0)
          load_tile<DY>(tile(n), &mx, h, tok, seq, bar);
        else if (kind == 1)
          load_tile<DY>(tile(n), &my, h, tok, seq, bar);
        else
          load_tile<DZ>(tile(n), &mz, h, tok, seq, bar);
      };
      for (int n = 0; n < SL; ++n) load(n);
      const long long t0 = clock64();
      for (int n = SL; n < 3 * nch; ++n) {  // tile n - SL, whose slot it takes, is done with
        const int c = (n - SL) / 3, kind = n - SL - 3 * c;
        while (!*abort && !(kind == 0      ? seen[2] > c && seen[3] > c
                            : kind == KEYS ? seen[4] > c && seen[DQ ? 0 : 3] > c
                                           : seen[1] > c && seen[DQ ? 3 : 0] > c)) {
          __nanosleep(40);  // its scheduler is others' too
          if (clock64() - t0 > 64 * WAIT_LIMIT) *abort = 1;  // the issuing thread gives up before
        }
        __threadfence_block();
        load(n);
      }
    } else if (t.w == P_CTL && t.l == 0) {  // ---- MMAs
      // Each kind of work goes out as soon as what it needs is there, the products that a team
      // waits for first. Issued so far: P z, the state's sum, x S, x y^T (chunks), tiles; seen
      // done of each, and of the teams' events. Nothing is issued before its forerunner has
      // been seen done, and nothing that lets an event happen again before that event has been
      // seen: so no barrier is ever two phases ahead of what is asked about it.
      int cz = 0, cd = 0, cs = 0, cp = 0;
      int bz = 0, bd = 0, bs = 0, bp = 0, wp = 0, wy = 0, ws = 0, wo = 0;
      auto see = [&](uint64_t* bar, int& i, int most, int tell) {
        if (i < most && mbar_test(bar, i & 1)) {
          ++i;
          if (tell == 4) __threadfence_block();  // the teams' reads of the tile are seen with it
          if (tell >= 0) seen[tell] = i;
        }
      };
      auto have = [&](int n) { return mbar_test(full + n % SL, n / SL & 1); };
      long long t0 = clock64();
      while ((bz < nch || bd < nch) && !*abort) {
        see(bar_o, bz, cz, 0);
        see(bar_d, bd, cd, 1);
        see(bar_s, bs, cs, 2);
        see(bar_p, bp, cp, 3);
        see(ev_y, wy, nch, 4);
        see(ev_p, wp, nch, -1);
        see(ev_s, ws, nch, -1);
        see(ev_o, wo, nch, -1);
        bool idle = true;
        if (cz < cs && cz == bz && wp > cz && have(3 * cz + 2) &&
            (!a.m.cu || u.len - cz * TC >= TC || wy > cz)) {  // a tail's z has been zeroed
          tc_fence_after();
          const uint32_t z = smem_u32(tile(3 * cz + 2));
#pragma unroll
          for (int kk = 0; kk < TC / 16; ++kk)
            umma_ts(tm + O0, tm + P0 + 8 * kk, mnmaj(z, HALF_TILE, kk), umma_idesc(128, DZ, 0, 1), true);
          umma_commit(bar_o);
          ++cz;
          idle = false;
        }
        if (cd < cp && cd <= cz && cd == bd && wy > cd && ws > cd && have(3 * cd + VALUES)) {
          tc_fence_after();
          const uint32_t z = smem_u32(tile(3 * cd + VALUES));
#pragma unroll 1
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int kk = 0; kk < TC / 16; ++kk)
              umma_ts(tm + D0, tm + Y0 + 64 * p + 8 * kk, mnmaj(z, HALF_TILE, kk),
                      umma_idesc(128, DV, 0, 1), p || kk);
          umma_commit(bar_d);
          ++cd;
          idle = false;
        }
        // the state and x are ready, the result before has been read
        if (cs < cp && cs <= cz && cs == bs && ws > cs && wo >= cs) {
          tc_fence_after();
          const uint32_t x = smem_u32(tile(3 * cs));
          // the forward's result takes the first part alone, which is as good as its own bits;
          // 4 steps unrolled: instruction fetch (all of them 182 us, 4 of them 174)
#pragma unroll 1
          for (int p = 0; p < (DQ ? 2 : 1); ++p)
#pragma unroll 4
            for (int kk = 0; kk < DY / 16; ++kk) {
              const uint32_t st = smem_u32(p ? s_lo : s_hi);
              umma_bf16(tm + O0, kmaj(x, HALF_TILE, kk),
                        DQ ? kmaj(st, L::HALF_S, kk) : mnmaj(st, L::HALF_S, kk),
                        umma_idesc(128, DZ, 0, DQ ? 0 : 1), p || kk);
            }
          umma_commit(bar_s);
          ++cs;
          idle = false;
        }
        // P of the chunk before has been read (dq: and a tail's y has been zeroed)
        if (cp < nch && cp == bp && bz >= cp && have(3 * cp) && have(3 * cp + 1) &&
            (!DQ || !a.m.cu || u.len - cp * TC >= TC || wy > cp)) {
          tc_fence_after();
          const uint32_t x = smem_u32(tile(3 * cp)), y = smem_u32(tile(3 * cp + 1));
#pragma unroll 4
          for (int kk = 0; kk < DY / 16; ++kk)
            umma_bf16(tm + P0, kmaj(x, HALF_TILE, kk), kmaj(y, HALF_TILE, kk),
                      umma_idesc(128, 128, 0, 0), kk > 0);
          umma_commit(bar_p);
          ++cp;
          idle = false;
        }
        if (!idle)
          t0 = clock64();
        else if (clock64() - t0 > WAIT_LIMIT)
          *abort = 1;
      }
    } else if (decs) {
      const bool wide = a.decay != nullptr;
      for (int c = 0; c < nch; ++c) {
        if (c > 1) mbar_wait(ev_u + (c & 1), ((c >> 1) + 1) & 1, abort);  // those of chunk c - 2
        fill_vec<false>(t.w - P_DEC, ahead, wide, 1.f, vec[c & 1]);
        if (c + 1 < nch) ahead = raw(c + 1);
        __syncwarp();
        if (t.l == 0) mbar_arrive(ev_v + (c & 1));
      }
    }
  }
  tear_down(t, P_CTL, full, SL, tm, abort, a.status);
}

// ------------------------------------------------------------------ dk, dv and dg
// From a unit's last chunk to its first, with R in registers (row: key, as in memory). The
// rows of a chunk's accumulators are its tokens s, the columns the tokens t they act on:
//   k q^T, v dO^T (masked by L_ts, t >= s, as P1 and P2), v R^T and k R (scaled by
//   e^{gamma_C - gamma_s}); dk = P2 q onto the one, dv = P1 dO onto the other;
//   R <- e^{gamma_C} R + (weighed q)^T dO.
// Two teams as above: one takes the masked products and the results, the other weighs q,
// adds up R, scales the products with R and writes R's next tiles. dg is summed in the warp
// that issues the copies, of every pair s < u <= t of tokens (or states) for itself and never
// as a difference of longer sums, in which what lies behind a forgotten state would leave its
// roundings: with b, k the blocks of 32 tokens of t and u,
//   dg_u = sum_{t >= u} a_t + sum_{s < u} b_s + e^{gamma_C} <S, R>            (gdn_lin.cu)
//        + pairs in u's block + (s in it, t in later ones) + (s in earlier ones, t in it)
//        + (s in earlier blocks, t in later ones).
// <S, R> takes S as dq left it and R from the second team's registers, while R's sum is on its
// way (by the first team from R's tiles, with warp-level MMAs, the kernel took 280 us instead of
// 243 for 32768 x 16 heads; by the decay warps 352).
// Bound by the chain P -> results -> R's sum -> products of the next chunk, 14 thousand cycles
// of which the MMAs are 7: 243 us for 32768 tokens x 16 heads of 128 (issue 41 %, tensor pipe
// 31 %; without <S, R> 224 us; P by one team of the two 280).
template <int DK, int DV>
struct BackSm {
  static constexpr int THREADS = P_NTHR;
  static constexpr uint32_t SLOT = slot_bytes(DK, DV), STATE = DK * DV * 2, HALF_R = DK * 128;
  static constexpr uint32_t R_HI = 4 * SLOT, R_LO = R_HI + STATE, VEC = R_LO + STATE;
  static constexpr uint32_t ROWS = VEC + 2 * sizeof(Vec), COLS = ROWS + 4 * TC * 4,
                            FAR = COLS + 3 * TC * 4, RED = FAR + 2 * TC * 4;
  static constexpr uint32_t OUT = (RED + 64 + 511) / 512 * 512, BAR = OUT + 8 * STAGE;
  static constexpr uint32_t BYTES = BAR + 256 + 1024;
};
// x[0..W-1] summed over the warp's lanes; lane j < W returns the sum of x[j].
template <int W>
__device__ __forceinline__ float lane_columns(float* x) {
  const int l = threadIdx.x & 31;
#pragma unroll
  for (int o = W / 2, n = W / 2; o >= 1; o >>= 1, n >>= 1) {
    const bool up = (l & o) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? x[i] : x[n + i], keep = up ? x[n + i] : x[i];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
#pragma unroll
  for (int o = 16; o >= W; o >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
  return x[0];
}
// This thread's row s of k q^T and v dO^T at the 32 columns t of block blk: as masked P1 and
// P2 in bf16 pairs over the second half of the same columns. Of the sums of A it leaves, in
// rows[0..31] by columns, those over the warp; in s's own block those of the pairs s < u <= t
// by u. Returns the row's sum over a later block. 8 columns at a time from the last, so that
// sums over t >= u run along, in a loop that stays rolled for the instruction cache (16 columns
// twice unrolled: the kernel takes 24 us more for 32768 tokens x 16 heads).
__device__ __forceinline__ float mask_block(uint32_t a1, uint32_t a2, const Vec& v, int blk, const Who& t,
                                            float scale, float* rows) {
  const bool diag = blk == t.q4, direct = diag && !v.mild[blk];
  const float tb = scale * (diag ? v.own[t.lane] : v.tab[blk - 1][t.lane]);
  float gh = 0.f, gl = 0.f, cs = 0.f;
  if (direct) gh = v.hi[t.lane], gl = v.lo[t.lane];
  constexpr int W = 8;
  a1 += 32 * blk;
  a2 += 32 * blk;
#pragma unroll 1
  for (int g = 32 - W; g >= 0; g -= W) {
    float x[W], y[W];
    uint32_t p1[W / 2], p2[W / 2];
    tmem_ld8(a1 + g, x);
    tmem_ld8(a2 + g, y);
#pragma unroll
    for (int e = W - 2; e >= 0; e -= 2) {
      const int col = 32 * blk + g + e;
      const float2 f2 = *reinterpret_cast<const float2*>(v.row + col);
      float f[2] = {tb * f2.x, tb * f2.y};
      if (direct) {
        const float2 h2 = *reinterpret_cast<const float2*>(v.hi + col);
        const float2 l2 = *reinterpret_cast<const float2*>(v.lo + col);
        f[0] = scale * __expf((h2.x - gh) + (l2.x - gl));
        f[1] = scale * __expf((h2.y - gh) + (l2.y - gl));
      }
      float px[2], py[2];
#pragma unroll
      for (int z = 1; z >= 0; --z) {
        const bool in = !diag || g + e + z >= t.l, behind = !diag || g + e + z > t.l;
        px[z] = in ? x[e + z] * f[z] : 0.f;
        py[z] = in ? y[e + z] * f[z] : 0.f;
        const float pair = behind ? x[e + z] * py[z] : 0.f;
        cs += pair;
        x[e + z] = !diag ? pair : behind ? cs : 0.f;
      }
      p1[e / 2] = pack2bf(px[0], px[1]);
      p2[e / 2] = pack2bf(py[0], py[1]);
    }
    tmem_st4(a1 + 16 + g / 2, p1);
    tmem_st4(a2 + 16 + g / 2, p2);
    const float sum = lane_columns<W>(x);
    if (t.l < W) rows[g + t.l] = sum;
  }
  return cs;
}

template <int DK, int DV>
__global__ void __launch_bounds__(P_NTHR, 1)
    k_lin_tc_back(Args a, const float* dS_out, const float* R_unit, const float* S_chunk, bool start,
                  float* dS_in, const float* far, bf* dk, bf* dv, bf* dg, float* dgsum,
                  const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
                  const __grid_constant__ CUtensorMap mdk, const __grid_constant__ CUtensorMap mdv) {
  using L = BackSm<DK, DV>;
  constexpr int NK = DK / 2, NV = DV / 2;
  // A1: k q^T, then P1 in the second half of every 32 columns; A2: v dO^T, then P2; the first
  // halves: the weighed q of the next chunk; G1: products with R for dk; G2: R's sum, then products with R for dv
  constexpr uint32_t A1 = 0, A2 = 128, G1 = 256, G2 = 384;
  chain();
  const int nth = blockIdx.x / a.H, h = blockIdx.x - nth * a.H, unit = lin_nth(a.m, nth);
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
  float* cols = reinterpret_cast<float*>(sb + L::COLS);  // [the block's distance - 1][s]
  float* farb = reinterpret_cast<float*>(sb + L::FAR);   // [column group][s]
  float* red = reinterpret_cast<float*>(sb + L::RED);    // [2][warp] parts of e^{gamma_C} <S, R>
  uint64_t* full = reinterpret_cast<uint64_t*>(sb + L::BAR);  // [4] v, k, q, dO
  // MMAs: R's sum, k q^T and v dO^T, products with R, results; decay factors are there [2]
  uint64_t *bar_e = full + 4, *bar_a = full + 5, *bar_f = full + 6, *bar_c = full + 7, *ev_v = full + 8;
  // events of a team: q weighed; R's sum added; products with R scaled; R's tiles written;
  // results read; of both: P1 and P2 written; decay factors used [2]
  uint64_t *ev_q = full + 10, *ev_g = full + 11, *ev_x = full + 12, *ev_r = full + 13, *ev_o = full + 14,
           *ev_p = full + 15, *ev_u = full + 16;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(full + 18);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  // what the issuing thread has seen done: A, products with R, results; events ev_x, ev_p
  volatile int* seen = reinterpret_cast<volatile int*>(tslot + 2);
  // q and dO of a chunk take the slots of v and k of the one before, which are done with
  // early, v and k those of q and dO
  auto slot = [&](int kind, int i) { return sb + (kind ^ (i & 1 ? 2 : 0)) * L::SLOT; };
  const int nch = (u.len + TC - 1) / TC;
  auto raw = [&](int i) {
    const int c = nch - 1 - i;
    return raw_decay(u.row + c * TC, min(TC, u.len - c * TC), h, a.g, a.ldg, a.decay);
  };
  const bool decs = t.w >= P_DEC && t.w < P_DEC + DEC_WARPS;
  Raw ahead = {};  // of the first chunk to be taken, as above
  if (decs && nch) ahead = raw(0);
  const uint32_t tm = set_up(t, P_CTL, full, 10, 2, 5, 3, tslot, abort);
  const uint32_t tl = tm + ((uint32_t)(32 * t.q4) << 16);
  const size_t sh = ((size_t)u.seq * a.H + h) * DK * DV;
  if (t.w < 8) {  // ---- masked products and results
    more_registers();
    for (int i = 0; i < nch; ++i) {
      const int c = nch - 1 - i, len = min(TC, u.len - c * TC), ph = i & 1;
      const Vec& v = vec[ph];
      mbar_wait(ev_v + ph, (i >> 1) & 1, abort);
      mbar_wait(bar_a, ph, abort);
      tc_fence_after();
      float cs = 0.f;
      if (t.q4 + t.cg < 4)
        cs = mask_block(tl + A1, tl + A2, v, t.q4 + t.cg, t, a.scale, rows + t.q4 * TC + 32 * (t.q4 + t.cg));
      if (t.cg == 1 || t.q4 == 3)  // nothing in the blocks before the diagonal
        for (int b = t.cg == 1 ? 0 : 2; b < (t.cg == 1 && t.q4 == 3 ? 2 : t.q4); ++b) {
          const uint32_t none[16] = {};
          tmem_st16(tl + A1 + 32 * b + 16, none);
          tmem_st16(tl + A2 + 32 * b + 16, none);
        }
      if (t.cg) cols[t.lane] = cs;
      tmem_st_wait();
      warp_done<false>(ev_p);
      if (t.l == 0) mbar_arrive(ev_u + ph);
      mbar_wait(bar_c, ph, abort);
      tc_fence_after();
      uint32_t rk[NK / 2], rv[NV / 2];
      take_row<NK>(tl + G1 + NK * t.cg, 1.f, rk);
      take_row<NV>(tl + G2 + NV * t.cg, 1.f, rv);
      warp_done<false>(ev_o);
      unsigned char* stage = sb + L::OUT + t.w * STAGE;
      const size_t mine = (size_t)(u.row + c * TC + t.lane) * a.H + h;
      const int tok = (a.m.cu ? u.row : u.at * a.m.unit) + c * TC + 32 * t.q4, seq = a.m.cu ? 0 : u.seq;
      const bool direct = len < TC && a.m.cu;
      leave_rows<NK>(rk, stage, &mdk, NK * t.cg, h, tok, seq, dk + mine * DK + NK * t.cg, direct,
                     len - 32 * t.q4);
      leave_rows<NV>(rv, stage, &mdv, NV * t.cg, h, tok, seq, dv + mine * DV + NV * t.cg, direct,
                     len - 32 * t.q4);
    }
    if (t.l == 0) bulk_wait_all();
  } else if (t.w < 16) {  // ---- R and the products with it
    more_registers();
    float r[NV];
    // dS_in may be dS_out: of many units none reads it
    if (u.n > 1)
      load_unit<DK, NV>(R_unit + uh * DK * DV, t.lane, NV * t.cg, r);
    else
      load_state<DK, DV, NV>(dS_out ? dS_out + sh : nullptr, t.lane, NV * t.cg, r);
    if (t.lane < DK) put_split<NV, true>(r_hi, r_lo, L::HALF_R, t.lane, NV * t.cg, r);
    warp_done<true>(ev_r);
    for (int i = 0; i < nch; ++i) {
      const int c = nch - 1 - i, len = min(TC, u.len - c * TC), ph = i & 1;
      const Vec& v = vec[ph];
      mbar_wait(ev_v + ph, (i >> 1) & 1, abort);
      mbar_wait(full + 2, ph, abort);
      if (len < TC && a.m.cu) {
        mbar_wait(full + 3, ph, abort);
        zero_rows<DK>(slot(2, i), len, t.tid - 256);
        zero_rows<DV>(slot(3, i), len, t.tid - 256);
        named_bar(6, 256);
      }
      if (i) mbar_wait(ev_p, ph ^ 1, abort);  // the products have been read
      tc_fence_after();
      if (t.lane < DK) {
        weigh<32>(slot(2, i), t, v.w, len, tl + A1, tl + A2);
        tmem_st_wait();
      }
      warp_done<true>(ev_q);
      // this thread's part of <S, R>, while R's sum is on its way; infinities behind a forgotten
      // state do not count
      const float whole = v.w.whole;
      float dot = 0.f;
      if (whole != 0.f && crossed(u, c, nch, start, dS_out)) {
        const float* S = S_chunk + (crossing(u, c) * a.H + h) * DK * DV;
        if (t.lane < DK) {
#pragma unroll
          for (int e = 0; e < NV; e += 4) {
            const float4 y = *reinterpret_cast<const float4*>(S + ((size_t)(NV * t.cg + e) / 4 * DK + t.lane) * 4);
            dot = fmaf(r[e], y.x, dot);
            dot = fmaf(r[e + 1], y.y, dot);
            dot = fmaf(r[e + 2], y.z, dot);
            dot = fmaf(r[e + 3], y.w, dot);
          }
        }
      }
      dot = lane_sum<32>(dot);
      if (t.l == 0) red[8 * ph + t.w - 8] = whole == 0.f ? 0.f : whole * dot;
      mbar_wait(bar_e, ph, abort);
      tc_fence_after();
      if (t.lane < DK) add_state<NV>(tl + G2 + NV * t.cg, v.w.whole, r);
      warp_done<false>(ev_g);
      // the third and fourth block behind the diagonal: the first lane quarters have most of P
      mbar_wait(bar_a, ph, abort);
      tc_fence_after();
      float cs = 0.f;
      if (t.q4 + t.cg < 2) {
        const int blk = t.q4 + t.cg + 2;
        cs = mask_block(tl + A1, tl + A2, v, blk, t, a.scale, rows + t.q4 * TC + 32 * blk);
        tmem_st_wait();
      }
      cols[(1 + t.cg) * TC + t.lane] = cs;
      warp_done<false>(ev_p);
      const float down = v.far[t.lane];
      mbar_wait(bar_f, ph, abort);
      tc_fence_after();
      float b = 0.f;
#pragma unroll 1
      for (int e = 0; e < NK; e += 16) {
        float x[16];
        uint32_t y[16];
        tmem_ld16(tl + G1 + NK * t.cg + e, x);
#pragma unroll
        for (int j = 0; j < 16; j += 8) {
          const uint4 k4 = *reinterpret_cast<const uint4*>(
              at8(slot(1, i), HALF_TILE, t.lane, NK * t.cg + e + j));
          const uint32_t kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            x[j + 2 * z] *= down;
            x[j + 2 * z + 1] *= down;
            b = fmaf(__uint_as_float(kk[z] << 16), x[j + 2 * z], b);
            b = fmaf(__uint_as_float(kk[z] & 0xffff0000u), x[j + 2 * z + 1], b);
          }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(x[j]);
        tmem_st16(tl + G1 + NK * t.cg + e, y);
      }
      farb[t.cg * TC + t.lane] = b;
#pragma unroll 1
      for (int e = 0; e < NV; e += 16) {
        float x[16];
        uint32_t y[16];
        tmem_ld16(tl + G2 + NV * t.cg + e, x);
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(x[j] * down);
        tmem_st16(tl + G2 + NV * t.cg + e, y);
      }
      tmem_st_wait();
      warp_done<false>(ev_x);
      if (t.l == 0) mbar_arrive(ev_u + ph);
      if (t.lane < DK) put_split<NV, true>(r_hi, r_lo, L::HALF_R, t.lane, NV * t.cg, r);
      warp_done<true>(ev_r);
    }
    if (u.at == 0 && dS_in) store_state<DK, DV, NV>(dS_in + sh, t.lane, NV * t.cg, r);
  } else {
    fewer_registers();
    if (t.w == P_LOAD) {  // ---- copies, and dg
      auto load = [&](int kind, int i) {  // a tile of the i-th chunk from the end
        if (i >= nch || *abort || t.l) return;
        const int c = nch - 1 - i;
        const int tok = a.m.cu ? u.row + c * TC : u.at * a.m.unit + c * TC, seq = a.m.cu ? 0 : u.seq;
        if (kind == 0)
          load_tile<DV>(slot(kind, i), &mv, h, tok, seq, full);
        else if (kind == 1)
          load_tile<DK>(slot(kind, i), &mk, h, tok, seq, full + 1);
        else if (kind == 2)
          load_tile<DK>(slot(kind, i), &mq, h, tok, seq, full + 2);
        else
          load_tile<DV>(slot(kind, i), &mo, h, tok, seq, full + 3);
      };
      const long long t0 = clock64();
      auto until = [&](int which, int n) {  // the issuing thread has seen `which` n times
        while (!*abort && seen[which] < n) {
          __nanosleep(40);
          if (clock64() - t0 > 64 * WAIT_LIMIT) *abort = 1;  // it gives up long before
        }
        __threadfence_block();
        __syncwarp();
      };
      for (int k = 3; k >= 0; --k) load(k, 0);
      float sum = 0.f;
      for (int i = 0; i < nch; ++i) {
        const int c = nch - 1 - i, len = min(TC, u.len - c * TC), row0 = u.row + c * TC;
        // the next chunk's S into the L2
        if (t.l == 0 && c > 0 && crossed(u, c - 1, nch, start, dS_out))
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(
                           S_chunk + (crossing(u, c - 1) * a.H + h) * DK * DV),
                       "r"(DK * DV * 4)
                       : "memory");
        float fa[4] = {};  // a of the tokens 4 l ..
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (4 * t.l + j < len) fa[j] = far[(size_t)(row0 + 4 * t.l + j) * a.H + h];
        until(0, i + 1);
        until(1, i + 1);
        load(2, i + 1);  // where v was
        until(3, i + 1);
        load(3, i + 1);  // where k was
        until(4, i + 1);
        // of this lane's tokens e in the block k: pairs in it; ones with s in an earlier block
        // and t = e; with s = e and t in a later block; b; and the sums over the lane's t of
        // the pairs with s in the first and in the second block
        const int k = t.l >> 3;
        float own[4], with_t[4], with_s[4], fb[4], first = 0.f, second = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 4 * t.l + j;
          own[j] = with_t[j] = with_s[j] = fb[j] = 0.f;
          if (e >= len) continue;
          const float r0 = rows[e], r1 = rows[TC + e], r2 = rows[2 * TC + e], r3 = rows[3 * TC + e];
          own[j] = k == 0 ? r0 : k == 1 ? r1 : k == 2 ? r2 : r3;
          with_t[j] = k == 0 ? 0.f : k == 1 ? r0 : k == 2 ? r0 + r1 : r0 + r1 + r2;
          with_s[j] = cols[e] + (cols[TC + e] + cols[2 * TC + e]);
          fb[j] = farb[e] + farb[TC + e];
          first += r0;
          second += r1;
        }
        float X = 0.f;
        for (int j = 0; j < 8; ++j) X += red[8 * (i & 1) + j];
        // k before the sums are stored: the next chunk's sums are written behind its products
        until(2, i + 1);
        load(1, i + 1);
        load(0, i + 1);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          first += __shfl_xor_sync(0xffffffffu, first, o);
          second += __shfl_xor_sync(0xffffffffu, second, o);
        }
        const float p02 = __shfl_sync(0xffffffffu, first, 16), p03 = __shfl_sync(0xffffffffu, first, 24),
                    p13 = __shfl_sync(0xffffffffu, second, 24);
        const float across = k == 1 ? p02 + p03 : k == 2 ? p03 + p13 : 0.f;
        // a and with_t over the lanes behind (the latter in the block), b and with_s over those before
        float sa = (fa[0] + fa[1]) + (fa[2] + fa[3]), st = (with_t[0] + with_t[1]) + (with_t[2] + with_t[3]);
        float sb = (fb[0] + fb[1]) + (fb[2] + fb[3]), ss = (with_s[0] + with_s[1]) + (with_s[2] + with_s[3]);
        const int l8 = t.l & 7;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float y = __shfl_down_sync(0xffffffffu, sa, o), z = __shfl_up_sync(0xffffffffu, sb, o);
          if (t.l + o < 32) sa += y;
          if (t.l >= o) sb += z;
          if (o < 8) {
            const float yt = __shfl_down_sync(0xffffffffu, st, o, 8), zs = __shfl_up_sync(0xffffffffu, ss, o, 8);
            if (l8 + o < 8) st += yt;
            if (l8 >= o) ss += zs;
          }
        }
        sa = __shfl_down_sync(0xffffffffu, sa, 1), st = __shfl_down_sync(0xffffffffu, st, 1, 8);
        sb = __shfl_up_sync(0xffffffffu, sb, 1), ss = __shfl_up_sync(0xffffffffu, ss, 1, 8);
        if (t.l == 31) sa = 0.f;
        if (l8 == 7) st = 0.f;
        if (t.l == 0) sb = 0.f;
        if (l8 == 0) ss = 0.f;
        float x[4];
#pragma unroll
        for (int j = 3; j >= 0; --j) x[j] = (sa += fa[j]) + (st += with_t[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] += own[j] + ((sb + ss) + (across + X));
          sb += fb[j], ss += with_s[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 4 * t.l + j;
          if (e >= len) break;
          if (dg)
            dg[(size_t)(row0 + e) * a.H + h] = __float2bfloat16_rn(x[j]);
          else
            sum += x[j];
        }
        __syncwarp();
      }
      if (dgsum) {
        sum = lane_sum<32>(sum);
        if (t.l == 0) dgsum[uh] = sum;
      }
    } else if (t.w == P_CTL && t.l == 0) {  // ---- MMAs, as in the forward
      int ce = 0, ca = 0, cf = 0, cc = 0, be = 0, ba = 0, bfr = 0, bc = 0;
      int wq = 0, wg = 0, wx = 0, wr = 0, wp = 0, wo = 0;
      auto see = [&](uint64_t* bar, int& i, int most, int tell) {
        if (i < most && mbar_test(bar, i & 1)) {
          ++i;
          // an event of the teams: what they wrote for dg is seen with it
          if (tell >= 3) __threadfence_block();
          if (tell >= 0) seen[tell] = i;
        }
      };
      auto have = [&](int kind, int i) { return mbar_test(full + kind, i & 1); };
      auto at16 = [](int kk) { return 32 * (kk >> 1) + 8 * (kk & 1); };  // columns of a step of P
      long long t0 = clock64();
      while (bc < nch && !*abort) {
        see(bar_c, bc, cc, 2);
        see(ev_x, wx, nch, 3);
        see(ev_p, wp, nch, 4);
        see(bar_f, bfr, cf, 1);
        see(bar_e, be, ce, -1);
        see(bar_a, ba, ca, 0);
        see(ev_g, wg, nch, -1);
        see(ev_q, wq, nch, -1);
        see(ev_o, wo, nch, -1);
        see(ev_r, wr, nch, -1);
        bool idle = true;
        if (cc < nch && cc == bc && wp > cc && wx > cc) {  // results
          tc_fence_after();
          const uint32_t sq = smem_u32(slot(2, cc)), so = smem_u32(slot(3, cc));
#pragma unroll
          for (int kk = 0; kk < TC / 16; ++kk)
            umma_ts(tm + G1, tm + A2 + 16 + at16(kk), mnmaj(sq, HALF_TILE, kk), umma_idesc(128, DK, 0, 1), true);
#pragma unroll
          for (int kk = 0; kk < TC / 16; ++kk)
            umma_ts(tm + G2, tm + A1 + 16 + at16(kk), mnmaj(so, HALF_TILE, kk), umma_idesc(128, DV, 0, 1), true);
          umma_commit(bar_c);
          ++cc;
          idle = false;
        }
        // R's sum: q weighed, the results before read
        if (ce < nch && ce == be && wq > ce && wo >= ce && have(3, ce)) {
          tc_fence_after();
          const uint32_t so = smem_u32(slot(3, ce));
#pragma unroll 1
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int kk = 0; kk < TC / 16; ++kk)
              umma_ts(tm + G2, tm + (p ? A2 : A1) + at16(kk), mnmaj(so, HALF_TILE, kk),
                      umma_idesc(128, DV, 0, 1), p || kk);
          umma_commit(bar_e);
          ++ce;
          idle = false;
        }
        // products: the weighed q has been used
        if (ca < be && ca == ba && have(2, ca) && have(1, ca) && have(0, ca)) {
          tc_fence_after();
          const uint32_t sv = smem_u32(slot(0, ca)), sk = smem_u32(slot(1, ca)),
                         sq = smem_u32(slot(2, ca)), so = smem_u32(slot(3, ca));
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk)
            umma_bf16(tm + A1, kmaj(sk, HALF_TILE, kk), kmaj(sq, HALF_TILE, kk),
                      umma_idesc(128, 128, 0, 0), kk > 0);
#pragma unroll
          for (int kk = 0; kk < DV / 16; ++kk)
            umma_bf16(tm + A2, kmaj(sv, HALF_TILE, kk), kmaj(so, HALF_TILE, kk),
                      umma_idesc(128, 128, 0, 0), kk > 0);
          umma_commit(bar_a);
          ++ca;
          idle = false;
        }
        // products with R: its tiles written, its sum added from where they go
        if (cf < ca && cf == bfr && wg > cf && wr > cf) {
          tc_fence_after();
          const uint32_t sv = smem_u32(slot(0, cf)), sk = smem_u32(slot(1, cf));
#pragma unroll 1
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int kk = 0; kk < DV / 16; ++kk)
              umma_bf16(tm + G1, kmaj(sv, HALF_TILE, kk), kmaj(smem_u32(p ? r_lo : r_hi), L::HALF_R, kk),
                        umma_idesc(128, DK, 0, 0), p || kk);
          // dv takes the first part alone: it is rounded to as many bits when it is stored
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk)
            umma_bf16(tm + G2, kmaj(sk, HALF_TILE, kk), mnmaj(smem_u32(r_hi), L::HALF_R, kk),
                      umma_idesc(128, DV, 0, 1), kk > 0);
          umma_commit(bar_f);
          ++cf;
          idle = false;
        }
        if (!idle)
          t0 = clock64();
        else if (clock64() - t0 > WAIT_LIMIT)
          *abort = 1;
      }
    } else if (decs) {
      const bool wide = a.decay != nullptr;
      for (int i = 0; i < nch; ++i) {
        if (i > 1) mbar_wait(ev_u + (i & 1), ((i >> 1) + 1) & 1, abort);  // those of chunk i - 2
        fill_vec<true>(t.w - P_DEC, ahead, wide, a.scale, vec[i & 1]);
        if (i + 1 < nch) ahead = raw(i + 1);
        __syncwarp();
        if (t.l == 0) mbar_arrive(ev_v + (i & 1));
      }
    }
  }
  tear_down(t, P_CTL, full, 4, tm, abort, a.status);
}

// ------------------------------------------------------------------ host side
// Chunks of a unit. A pass takes as many waves of CTAs as there are units of all heads
// for the GPU's SMs, each as long as a unit (plus about a chunk to start); more than one
// unit of a sequence also needs the units' own sums (y and z only: half a chunk's time)
// and the scan.
constexpr int SMS = 152, MOST_CHUNKS = 64;
int unit_chunks(const gdn_lin_shape& s, bool packed) {
  const long long nc = std::max(1, (s.T + TC - 1) / TC);
  if (packed) {  // the lengths are known on the device only: no unit longer than an SM's share
    const long long all = (nc + s.nseq / 2) * s.H;
    return (int)std::min((long long)MOST_CHUNKS, std::max(4ll, (all + SMS - 1) / SMS));
  }
  const long long chains = (long long)s.nseq * s.H;
  double best = 1e300;
  int per = (int)nc;
  for (long long n = 1, len = nc; n <= nc && n <= 256; n = (nc - 1) / (len - 1) + 1) {
    len = (nc + n - 1) / n;  // the next n is the first with a smaller one
    const long long units = (nc + len - 1) / len;
    const double waves = (double)((chains * units + SMS - 1) / SMS);
    double cost = waves * (len + 1.0);
    if (units > 1) {
      const double first = (double)((chains * (units - 1) + SMS - 1) / SMS);
      cost += first * (0.5 * len + 1.0) + 2.0 + 0.0135 * chains * units;
    }
    if (cost < best) best = cost, per = (int)len;
    if (len == 1) break;
  }
  return per;
}

struct TcPlan {
  LinMap m;
  int chunks;
  bool many;  // a sequence may have several units
  int *status, *first, *owner, *order;
  float *whole[2], *dgsum, *D, *E, *S_chunk, *far;
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
  p.order = (int*)take(packed ? (size_t)p.m.cap * 4 : 0);
  p.whole[0] = (float*)take(uh * 4);
  p.D = (float*)take(p.many ? uh * one : 0);
  if (back) {
    p.whole[1] = (float*)take(uh * 4);
    p.E = (float*)take(p.many ? uh * one : 0);
    p.dgsum = (float*)take(uh * 4);
    p.S_chunk = (float*)take(((size_t)s.B * s.T / TC + s.nseq) * s.H * one);
    p.far = (float*)take((size_t)s.B * s.T * s.H * 4);
  }
  p.m.first = p.first;
  p.m.owner = p.owner;
  p.m.order = packed ? p.order : nullptr;
  p.bytes = at;
  return p;
}

// [B][T][H][d] bf16 rows `ld` apart as boxes of 64 columns of 128 tokens of one head.
cudaError_t tile_map(CUtensorMap* map, const void* base, const gdn_lin_shape& s, int d, long long ld) {
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)s.H, (cuuint64_t)s.T, (cuuint64_t)s.B};
  const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * s.T};
  return make_tile_map(map, base, dims, strides, 64, TC);
}
// A result [B][T][H][d], contiguous, as boxes of 32 columns of 32 tokens.
cudaError_t out_map(CUtensorMap* map, const void* base, const gdn_lin_shape& s, int d) {
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)s.H, (cuuint64_t)s.T, (cuuint64_t)s.B};
  const cuuint64_t ld = (cuuint64_t)s.H * d * 2, strides[3] = {(cuuint64_t)d * 2, ld, ld * s.T};
  return make_tile_map(map, base, dims, strides, 32, 32);
}

// Shared memory of a kernel, and whether its launch holds the registers that its warpgroups
// share out (a smaller pool would leave them waiting).
template <auto KERNEL>
cudaError_t allow(uint32_t bytes, int registers) {
  static std::atomic<int> has{0};  // asked again after a failure
  if (!has.load(std::memory_order_relaxed)) {
    cudaFuncAttributes f;
    const cudaError_t e = cudaFuncGetAttributes(&f, KERNEL);
    if (e) return e;
    has.store(f.numRegs, std::memory_order_relaxed);
  }
  if (has.load(std::memory_order_relaxed) < registers) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int DK, int DV>
cudaError_t run_tc(const LinCall& c, bool back) {
  const gdn_lin_shape& s = c.s;
  const TcPlan p = tc_plan(s, c.cu, c.cu != nullptr, back, c.ws);
  const Args a = {p.m, s.H, s.scale, (const bf*)c.g, c.decay, s.ldg, p.status};
  CUtensorMap mq, mk, mv, mo, mdq, mdk, mdv;
  cudaError_t e;
  if ((e = tile_map(&mq, c.q, s, DK, s.ldq)) || (e = tile_map(&mk, c.k, s, DK, s.ldk)) ||
      (e = tile_map(&mv, c.v, s, DV, s.ldv)))
    return e;
  if (back) {
    if ((e = tile_map(&mo, c.dout, s, DV, (long long)s.H * DV)) || (e = out_map(&mdq, c.dq, s, DK)) ||
        (e = out_map(&mdk, c.dk, s, DK)) || (e = out_map(&mdv, c.dv, s, DV)))
      return e;
  } else if ((e = out_map(&mo, c.o, s, DV))) {
    return e;
  }
  if (c.cu && (e = lin_plan(p.m, p.first, p.owner, p.order, TC, p.status, c.st))) return e;
  bool clear = !c.cu;  // the first kernel of an unpacked call resets the status word
  const dim3 grid(p.m.cap * s.H);
  auto go = [&](auto kernel, cudaError_t ready, uint32_t smem, int threads, auto... rest) {
    return ready ? ready : launch(kernel, grid, dim3(threads), (int)smem, c.st, 1, a, rest...);
  };
#define GO(kernel, Sm, regs, ...) \
  go(kernel, allow<kernel>(Sm::BYTES, regs), Sm::BYTES, Sm::THREADS, __VA_ARGS__)
  using State = StateSm<DK, DV>;
  if (p.many) {
    prof_mark(c.st, "lin_tc_state");
    e = GO((k_lin_tc_state<DK, DV, false>), State, 0, p.whole[0], p.D, clear, mk, mv);
    if (e) return e;
    clear = false;
    if (back) {
      prof_mark(c.st, "lin_tc_state");
      e = GO((k_lin_tc_state<DK, DV, true>), State, 0, p.whole[1], p.E, false, mq, mo);
      if (e) return e;
    }
    e = lin_scan(p.m, s, p.whole[0], p.D, c.S_in, p.E, p.whole[1], c.dS_out, back, p.status, c.st);
    if (e) return e;
  }
  using PassKV = PassSm<DK, DV, false>;
  using PassVK = PassSm<DV, DK, true>;
  using Back = BackSm<DK, DV>;
  prof_mark(c.st, back ? "lin_tc_dq" : "lin_tc_fwd");
  if (!back)
    return GO((k_lin_tc_pass<DK, DV, false>), PassKV, P_REGS, c.S_in, p.D, c.S_out, (bf*)c.o,
              (const bf*)nullptr, 0ll, (float*)nullptr, (float*)nullptr, false, clear, mq, mk, mv, mo);
  e = GO((k_lin_tc_pass<DV, DK, true>), PassVK, P_REGS, c.S_in, p.D, (float*)nullptr, (bf*)c.dq,
         (const bf*)c.q, s.ldq, p.far, p.S_chunk, c.dS_out != nullptr, clear, mo, mv, mk, mdq);
  if (e) return e;
  prof_mark(c.st, "lin_tc_back");
  e = GO((k_lin_tc_back<DK, DV>), Back, P_REGS, c.dS_out, p.E, p.S_chunk, c.S_in != nullptr, c.dS_in,
         p.far, (bf*)c.dk, (bf*)c.dv, (bf*)c.dg, c.ddecay ? p.dgsum : nullptr, mq, mk, mv, mo, mdk, mdv);
#undef GO
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

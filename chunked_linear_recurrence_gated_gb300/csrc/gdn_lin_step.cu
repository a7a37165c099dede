// Linear attention with a decay for each head, token by token over a cache of
// states (gdn_lin_step, include/gdn_lin.h).
#include <stdint.h>

#include <algorithm>

#include "../../include/gdn_lin.h"
#include "gdn_cache.cuh"
#include "gdn_layer.cuh"

namespace gdn {
namespace {

// Columns of a block and blocks of an SM. The states' bytes bound it: 256 sequences x 32 heads
// of 128 x 128 take 152 us, the measured copy rate (64 columns by 5 blocks 151, but one
// sequence 2.9 us instead of 2.5); 45 sequences x 24 heads with 1 to 8 tokens 25 us (63 %, 64
// columns 28), where the arithmetic of the longer ones stands beside the loads.
constexpr int LS_COLS = 32, LS_BLOCKS = 8;
constexpr int LS_NT = 128;   // threads of a block
constexpr int LS_TILE = 8;   // tokens whose q, k and v are in shared memory together

// One block: COLS columns of one head's state of one sequence, in registers: a
// thread has 4 columns of R consecutive rows. Per token S <- a S + k v^T and the
// thread's part of q S (3 fp32 multiply-adds per element, two at a time), whose
// sums over the block's row groups are joined once per tile of tokens. ONE: every sequence
// has one token, which is asked for together with the state (167 -> 151 us of the batch).
template <typename T, int DK, int COLS>
struct LinStep {
  static constexpr int CG = COLS / 4;        // threads of a row
  static constexpr int RG = LS_NT / CG;      // row groups
  static constexpr int R = DK / RG;          // rows of a thread
  static_assert(R % 4 == 0 && CG <= 32, "whole 16-byte pieces of k and q, rows inside a warp");
};

template <typename T, int DK, int DV, int COLS, bool ONE>
__global__ void __launch_bounds__(LS_NT, LS_BLOCKS)
    k_lin_step(Cache cache, FastDiv byHP, int G, long long ldq, long long ldk, long long ldv,
               long long ldg, float scale, const T* q, const T* k, const T* v, const T* g,
               const float* decay, float* S, T* o) {
  using L = LinStep<T, DK, COLS>;
  constexpr int PARTS = DV / COLS, NW = LS_NT / 32, TILE = ONE ? 1 : LS_TILE;
  __shared__ __align__(16) float sk[TILE][DK], sq[TILE][DK], sv[TILE][COLS];
  __shared__ __align__(16) float red[TILE][NW][COLS];
  __shared__ float sa[TILE];
  chain();
  uint32_t seq, hp;
  byHP(blockIdx.x, seq, hp);
  const SeqCall sc = seq_call(cache, seq);
  if (sc.len == 0 && !sc.store) return;
  const int H = (int)byHP.d / PARTS, h = hp / PARTS, c0 = (hp - h * PARTS) * COLS;
  const int tid = threadIdx.x, cg = tid % L::CG, rg = tid / L::CG, warp = tid >> 5;
  const size_t base = ((size_t)h * DK + rg * L::R) * DV + c0 + cg * 4;
  f32x2 s[L::R][2];
  float4 x[L::R];
#pragma unroll
  for (int i = 0; i < L::R; ++i) x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (sc.in >= 0) {
    const float* p = S + (size_t)sc.in * H * DK * DV + base;
#pragma unroll
    for (int i = 0; i < L::R; ++i) x[i] = *reinterpret_cast<const float4*>(p + (size_t)i * DV);
  }
  auto take = [&]() {
#pragma unroll
    for (int i = 0; i < L::R; ++i) s[i][0] = pack2(x[i].x, x[i].y), s[i][1] = pack2(x[i].z, x[i].w);
  };
  if (!ONE) take();
  auto store = [&]() {
    float* p = S + (size_t)sc.out * H * DK * DV + base;
#pragma unroll
    for (int i = 0; i < L::R; ++i) {
      float4 x;
      unpack2(s[i][0], x.x, x.y);
      unpack2(s[i][1], x.z, x.w);
      *reinterpret_cast<float4*>(p + (size_t)i * DV) = x;
    }
  };
  auto load_tile = [&](int tb, int nb) {
    for (int i = tid; i < nb * (DK / 8) * 2; i += LS_NT) {
      const int t = i / (DK / 4), e = i % (DK / 8) * 8;
      const bool is_q = i / (DK / 8) & 1;
      const size_t row = (size_t)(sc.t0 + tb + t);
      float y[8];
      ld8((is_q ? q + row * ldq : k + row * ldk) + (size_t)(h / G) * DK + e, y);
      st8((is_q ? sq[t] : sk[t]) + e, y);
    }
    for (int i = tid; i < nb * (COLS / 8); i += LS_NT) {
      const int t = i / (COLS / 8), e = i % (COLS / 8) * 8;
      float y[8];
      ld8(v + (size_t)(sc.t0 + tb + t) * ldv + (size_t)h * DV + c0 + e, y);
      st8(sv[t] + e, y);
    }
    if (tid < nb)
      sa[tid] = expf(decay ? decay[h] : ldf(g + (size_t)(sc.t0 + tb + tid) * ldg + h));
  };
  if (ONE) {
    load_tile(0, 1);
    take();
  }
  if (sc.store && sc.commit == 0) store();
  for (int tb = 0; tb < (ONE ? 1 : sc.len); tb += TILE) {
    const int nb = ONE ? 1 : min(TILE, sc.len - tb);
    if (tb) __syncthreads();  // the tile before is done with
    if (!ONE) load_tile(tb, nb);
    __syncthreads();
    for (int t = 0; t < nb; ++t) {
      const f32x2 a = both2(sa[t]);
      const float4 vv = *reinterpret_cast<const float4*>(sv[t] + cg * 4);
      const f32x2 v0 = pack2(vv.x, vv.y), v1 = pack2(vv.z, vv.w);
      f32x2 o0 = pack2(0.f, 0.f), o1 = o0;
#pragma unroll
      for (int i = 0; i < L::R; i += 4) {
        const float4 kk = *reinterpret_cast<const float4*>(sk[t] + rg * L::R + i);
        const float4 qq = *reinterpret_cast<const float4*>(sq[t] + rg * L::R + i);
        const float kr[4] = {kk.x, kk.y, kk.z, kk.w}, qr[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x2 k2 = both2(kr[j]), q2 = both2(qr[j]);
          s[i + j][0] = fma2(k2, v0, mul2(a, s[i + j][0]));
          s[i + j][1] = fma2(k2, v1, mul2(a, s[i + j][1]));
          o0 = fma2(q2, s[i + j][0], o0);
          o1 = fma2(q2, s[i + j][1], o1);
        }
      }
      float p[4];
      unpack2(o0, p[0], p[1]);
      unpack2(o1, p[2], p[3]);
#pragma unroll
      for (int m = 16; m >= L::CG; m >>= 1)
#pragma unroll
        for (int c = 0; c < 4; ++c) p[c] += __shfl_xor_sync(0xffffffffu, p[c], m);
      if ((tid & 31) < L::CG)
        *reinterpret_cast<float4*>(red[t][warp] + cg * 4) = make_float4(p[0], p[1], p[2], p[3]);
      if (sc.store && tb + t + 1 == sc.commit) store();
    }
    __syncthreads();
    for (int i = tid; i < nb * COLS; i += LS_NT) {
      const int t = i / COLS, c = i % COLS;
      float x = red[t][0][c];
#pragma unroll
      for (int w = 1; w < NW; ++w) x += red[t][w][c];
      stf(o + ((size_t)(sc.t0 + tb + t) * H + h) * DV + c0 + c, scale * x);
    }
  }
}

template <typename T, int DK, int DV, int COLS>
void launch_cols(const gdn_lin_step_shape& s, const Cache& c, const void* q, const void* k,
                 const void* v, const void* g, const float* decay, float* S, void* o,
                 cudaStream_t st) {
  constexpr int parts = DV / COLS;
  auto go = [&](auto kernel) {
    launch(kernel, dim3((unsigned)s.N * s.H * parts), dim3(LS_NT), 0, st, 1, c, FastDiv(s.H * parts),
           s.H / s.Hk, s.ldq, s.ldk, s.ldv, s.ldg, s.scale, (const T*)q, (const T*)k, (const T*)v,
           (const T*)g, decay, S, (T*)o);
  };
  if (c.cu)
    go(k_lin_step<T, DK, DV, COLS, false>);
  else
    go(k_lin_step<T, DK, DV, COLS, true>);
}
template <typename T, int DK, int DV, typename... A>
void launch_lin_step(const gdn_lin_step_shape& s, A... a) {
  launch_cols<T, DK, DV, LS_COLS>(s, a...);
}
template <typename T, typename... A>
void dispatch_lin_step(const gdn_lin_step_shape& s, A... a) {
  if (s.dk == 64) {
    if (s.dv == 64) return launch_lin_step<T, 64, 64>(s, a...);
    return launch_lin_step<T, 64, 128>(s, a...);
  }
  if (s.dv == 64) return launch_lin_step<T, 128, 64>(s, a...);
  return launch_lin_step<T, 128, 128>(s, a...);
}

}  // namespace
}  // namespace gdn

extern "C" gdn_status gdn_lin_step(const gdn_lin_step_shape* shape, const void* q, const void* k,
                                   const void* v, const void* g, const float* decay, float* S,
                                   const int* slot_in, const int* slot_out, const int* cu_seqlens,
                                   const int* n_commit, void* o, void* stream) {
  using namespace gdn;
  if (!shape) return GDN_ERR_INVALID_ARG;
  const gdn_lin_step_shape& s = *shape;
  const gdn_status e =
      check_cache(s.N, s.n_tok, s.n_slots, slot_in, slot_out, cu_seqlens, n_commit);
  if (e != GDN_OK) return e;
  if (s.H < 1 || s.Hk < 1 || s.H % s.Hk) return GDN_ERR_INVALID_ARG;
  if (!dtype_ok(s.dtype) || (s.dk != 64 && s.dk != 128) || (s.dv != 64 && s.dv != 128) ||
      8ll * s.N * s.H >= (1ll << 31))
    return GDN_ERR_UNSUPPORTED;
  if (s.n_tok > 0 && (!q || !k || !v || !o || (!g && !decay))) return GDN_ERR_INVALID_ARG;
  if ((g && decay) || (s.n_slots > 0 && !S)) return GDN_ERR_INVALID_ARG;
  if (!vec_rows(q, s.ldq, s.dtype) || !vec_rows(k, s.ldk, s.dtype) ||
      !vec_rows(v, s.ldv, s.dtype) || (g && s.ldg < 0) || !aligned(g, elem_size(s.dtype)) ||
      !aligned(decay, 4) || !aligned(S, 16) || !aligned(o, 16))
    return GDN_ERR_INVALID_ARG;
  if (s.N == 0) return GDN_OK;
  const Cache c = {s.N, s.n_tok, s.n_slots, slot_in, slot_out, cu_seqlens, n_commit};
  cudaStream_t st = (cudaStream_t)stream;
  prof_mark(st, "lin_step");
  if (s.dtype == GDN_DTYPE_BF16)
    dispatch_lin_step<__nv_bfloat16>(s, c, q, k, v, g, decay, S, o, st);
  else
    dispatch_lin_step<float>(s, c, q, k, v, g, decay, S, o, st);
  prof_mark(st, nullptr);
  return cudaGetLastError() ? GDN_ERR_CUDA : GDN_OK;
}

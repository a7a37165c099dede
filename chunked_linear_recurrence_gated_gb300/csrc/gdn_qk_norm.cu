// Norms of query and key heads with the rotation by the token's position
// (gdn_qk_norm_fwd / gdn_qk_norm_bwd, include/gdn_layer.h).
#include <stdint.h>

#include <algorithm>

#include "gdn_layer.cuh"

namespace gdn {
namespace {

constexpr int QN_NT = 256;     // threads of a block
constexpr int QN_SMS = 152;
// Head rows that a thread has in flight (backward: with their gradients), and blocks of an SM.
// What has to come from memory bounds both: 32768 tokens x 32 heads x 128 in bf16 take 91 us
// (87 % of the measured copy rate); 4 rows by 3 blocks 92, 2 by 3 99, 1 by 4 104. The backward
// of 8193 tokens x (24 + 8 heads of 24) 51 us (68 %, its registers leave room for no more than
// 2 blocks): 1 row by 4 blocks 75, 4 rows by one block 60; 608 blocks' partial sums 54.
constexpr int QN_U = 2, QN_BLOCKS = 4;
constexpr int QN_UB = 2, QN_BLOCKS_B = 2;
constexpr int QN_HEADS = 16;   // most heads that share one set of sines and cosines
constexpr int QN_PARTS = QN_SMS * QN_BLOCKS_B;  // most blocks of the backward: partial sums of dw

// f / (2 pi) as a fraction of a turn in units of 2^-64, for |f| < 2^40, less than a unit below
// the exact one. With f = m 2^e (m < 2^53) and C = floor(2^130 / (2 pi)), it is m C 2^(e - 66) in
// whole numbers (64 bits of C alone would be off by f / 4 units), so that pos times it, modulo
// 2^64, is the angle's fraction of a turn to 2^-33 for any 32-bit position.
__device__ __forceinline__ unsigned long long turn_step(double f) {
  constexpr unsigned long long C = 0xA2F9836E4E441529ull, REST = 0xFC2757D1F534DDC0ull;  // 2 / pi
  const unsigned long long u = (unsigned long long)__double_as_longlong(f);
  const int ex = (int)(u >> 52) & 0x7ff;
  const unsigned long long m = (u & 0xfffffffffffffull) | (ex ? 1ull << 52 : 0);
  const int s = 2 + 1075 - max(ex, 1);  // right shift of the upper 128 bits of the product
  const unsigned long long low = __umul64hi(m, REST), lo = m * C + low;
  const unsigned long long hi = __umul64hi(m, C) + (lo < low);
  unsigned long long r = 0;
  if (s <= 0)
    r = lo << min(-s, 63);
  else if (s < 64)
    r = (hi << (64 - s)) | (lo >> s);
  else if (s < 128)
    r = hi >> (s - 64);
  return (u >> 63) ? 0ull - r : r;
}

// The queries or the keys of a call. A block has one of the two, so weight, repeats and
// strides are the same for all of its rows; the first `blocks` blocks have the queries.
template <typename T>
struct QkSide {
  const T* x;       // [rows][heads][D], rows ld apart
  const T* dy;      // backward: [rows][heads * rep][D]
  T* out;           // forward: like dy; backward: [rows][heads][D]
  const float* w;
  long long ld;
  FastDiv byParts;  // items (token, heads) of a token
  uint32_t items;
  int heads, per, rep, blocks;  // heads of an item, repeats of an output head
  float scale;
};
template <typename T>
struct QkArgs {
  QkSide<T> side[2];
  FastDiv byT;
  int r2;  // rot / 2
  float eps;
  const double* inv_freq;
  const int* pos;
};

// A thread's part of a head's row: 8 values from e0, as 4 pairs, by one of D / 8 lanes.
// What turns them: y = x cs + (its partner) sn.
struct Turn {
  f32x2 cs[4], sn[4];
};
template <int D, bool PAIRS>
struct Lane {
  int e0, partner, f0;  // partner: the lane with the other halves of this one's pairs
  bool turned, first;
  __device__ __forceinline__ Lane(int r2) {
    const int l = threadIdx.x & 31;
    e0 = 8 * (threadIdx.x % (D / 8));
    turned = e0 < 2 * r2;
    first = e0 < r2;
    partner = PAIRS || !turned ? l : first ? l + r2 / 8 : l - r2 / 8;
    f0 = PAIRS ? e0 / 2 : first ? e0 : e0 - r2;
  }
};

// The steps of all pairs, for the block.
__device__ __forceinline__ void fill_steps(const double* inv_freq, int r2, unsigned long long* steps) {
  for (int i = threadIdx.x; i < r2; i += QN_NT) steps[i] = turn_step(inv_freq[i]);
}
// Sines and cosines at a position; BACK: of the opposite angle. For bf16 rows they are the
// hardware's, off by 2^-20 where a value is rounded by 2^-9 of itself (sincospif of 8 angles
// costs as much as the rest of 4 rows).
template <typename T, bool PAIRS, bool BACK>
__device__ __forceinline__ void turn_at(const unsigned long long* steps, int pos, bool turned, bool first,
                                        Turn& t) {
  const unsigned long long p = (unsigned long long)(long long)pos;
#pragma unroll
  for (int i = 0; i < 4; ++i) t.cs[i] = both2(1.f), t.sn[i] = both2(0.f);
  if (!turned) return;
  float sn[8], cs[8];
#pragma unroll
  for (int i = 0; i < (PAIRS ? 4 : 8); ++i) {
    const float ph = (float)(int)((p * steps[i]) >> 32) * 0x1p-31f;  // [-1, 1) half turns
    if (sizeof(T) == 2) {
      const float a = ph * 3.14159265f;
      sn[i] = __sinf(a);
      cs[i] = __cosf(a);
    } else {
      sincospif(ph, &sn[i], &cs[i]);
    }
    if (BACK) sn[i] = -sn[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (PAIRS) {
      t.cs[i] = both2(cs[i]);
      t.sn[i] = pack2(-sn[i], sn[i]);
    } else {
      t.cs[i] = pack2(cs[2 * i], cs[2 * i + 1]);
      t.sn[i] = first ? pack2(-sn[2 * i], -sn[2 * i + 1]) : pack2(sn[2 * i], sn[2 * i + 1]);
    }
  }
}
// Every lane of the warp takes part.
template <bool PAIRS>
__device__ __forceinline__ void turn(const Turn& t, int partner, f32x2* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack2(x[i], a, b);
    f32x2 y;
    if (PAIRS) {
      y = pack2(b, a);
    } else {
      a = __shfl_sync(0xffffffffu, a, partner);
      b = __shfl_sync(0xffffffffu, b, partner);
      y = pack2(a, b);
    }
    x[i] = fma2(x[i], t.cs[i], mul2(y, t.sn[i]));
  }
}

// A thread's place in the walk over a side's items: U heads at a time of one token.
template <typename T, int U>
struct Walk {
  uint32_t it, tok;
  int h, end;   // heads [h, end) of the item are left
  bool on;
  __device__ __forceinline__ void start(const QkSide<T>& s, uint32_t item) {
    it = item;
    on = it < s.items;
    uint32_t part = 0;
    tok = 0;
    if (on) s.byParts(it, tok, part);
    h = (int)part * s.per;
    end = on ? min(h + s.per, s.heads) : h;
  }
  __device__ __forceinline__ bool has(int u) const { return h + u < end; }
};

template <typename T, int U>
__device__ __forceinline__ void load_rows(const QkSide<T>& s, const Walk<T, U>& at, int e0, int D,
                                          Raw8<T>* raw) {
  const T* x = s.x + (size_t)at.tok * s.ld + (size_t)at.h * D + e0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    raw[u] = Raw8<T>{};
    if (at.has(u)) raw[u] = ldraw8(x + (size_t)u * D);
  }
}

// D / 8 lanes hold a head's row, 8 values each, and take `per` heads of one token, whose
// sines and cosines they form once. The next QN_U rows are on their way while these are
// worked on. Items are spread over the grid.
template <typename T, int D, bool PAIRS>
__global__ void __launch_bounds__(QN_NT, QN_BLOCKS)
    k_qk_norm_fwd(const __grid_constant__ QkArgs<T> a) {
  chain();
  constexpr int L = D / 8, NG = QN_NT / L;
  __shared__ __align__(16) unsigned long long steps[D / 2];
  const bool is_k = blockIdx.x >= a.side[0].blocks;
  const QkSide<T>& s = a.side[is_k];
  const Lane<D, PAIRS> me(a.r2);
  const uint32_t stride = (uint32_t)s.blocks * NG;
  const uint32_t i0 = (blockIdx.x - (is_k ? a.side[0].blocks : 0)) * NG;
  Walk<T, QN_U> at;
  at.start(s, i0 + threadIdx.x / L);
  Raw8<T> raw[QN_U];
  load_rows<T, QN_U>(s, at, me.e0, D, raw);
  fill_steps(a.inv_freq, a.r2, steps);
  f32x2 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = both2(s.scale);
  if (s.w) {
    float v[8];
    ld8(s.w + me.e0, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2(v[2 * i] * s.scale, v[2 * i + 1] * s.scale);
  }
  __syncthreads();
  // the same trips for every lane of a warp
  for (uint32_t base = i0; base < s.items; base += stride) {
    Turn tn;
    if (a.r2) {
      uint32_t seq, in_seq;
      a.byT(at.tok, seq, in_seq);
      turn_at<T, PAIRS, false>(steps + me.f0, a.pos && at.on ? a.pos[at.tok] : (int)in_seq, me.turned,
                               me.first, tn);
    }
    for (int hb = 0; hb < s.per; hb += QN_U) {
      Walk<T, QN_U> next = at;
      next.h += QN_U;
      if (hb + QN_U >= s.per) next.start(s, at.it + stride);
      Raw8<T> ahead[QN_U];
      load_rows<T, QN_U>(s, next, me.e0, D, ahead);
      T* out = s.out + ((size_t)at.tok * s.heads + at.h) * s.rep * D + me.e0;
#pragma unroll
      for (int u = 0; u < QN_U; ++u) {
        f32x2 x[4], ss = both2(0.f);
        cvt8(raw[u], x);
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fma2(x[i], x[i], ss);
        const f32x2 r = both2(rsqrtf(fmaf(lane_sum<L>(sum2(ss)), 1.f / D, a.eps)));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], mul2(r, w[i]));
        if (a.r2) turn<PAIRS>(tn, me.partner, x);
        if (at.has(u))
          for (int i = 0; i < s.rep; ++i) st8(out + (size_t)(u * s.rep + i) * D, x);
      }
      at = next;
#pragma unroll
      for (int u = 0; u < QN_U; ++u) raw[u] = ahead[u];
    }
  }
}

// With d the sum of a head's repeated gradients turned back (and times scale),
// n = x r, e = d w:   dx = r (e - n mean(e n)),   dw += d n.
// Lanes and items as forward; a thread sums its 8 columns of dw over all of its rows, the
// block's lane groups join theirs in order, and part[block] = [dwq, dwk].
template <typename T, int D, bool PAIRS>
__global__ void __launch_bounds__(QN_NT, QN_BLOCKS_B)
    k_qk_norm_bwd(const __grid_constant__ QkArgs<T> a, float* part_out) {
  chain();
  let_next_start();
  constexpr int L = D / 8, NG = QN_NT / L, U = QN_UB;
  __shared__ __align__(16) unsigned long long steps[D / 2];
  __shared__ float red[NG][D];
  const bool is_k = blockIdx.x >= a.side[0].blocks;
  const QkSide<T>& s = a.side[is_k];
  const Lane<D, PAIRS> me(a.r2);
  const uint32_t stride = (uint32_t)s.blocks * NG;
  const uint32_t i0 = (blockIdx.x - (is_k ? a.side[0].blocks : 0)) * NG;
  auto load_dy = [&](const Walk<T, U>& at, int i, Raw8<T>* g) {
    const T* dy = s.dy + (((size_t)at.tok * s.heads + at.h) * s.rep + i) * D + me.e0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      g[u] = Raw8<T>{};
      if (at.has(u)) g[u] = ldraw8(dy + (size_t)u * s.rep * D);
    }
  };
  Walk<T, U> at;
  at.start(s, i0 + threadIdx.x / L);
  Raw8<T> raw[U], g[U];
  load_rows<T, U>(s, at, me.e0, D, raw);
  load_dy(at, 0, g);
  fill_steps(a.inv_freq, a.r2, steps);
  f32x2 w[4], dw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = both2(s.scale), dw[i] = both2(0.f);
  if (s.w) {
    float v[8];
    ld8(s.w + me.e0, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2(v[2 * i] * s.scale, v[2 * i + 1] * s.scale);
  }
  __syncthreads();
  for (uint32_t base = i0; base < s.items; base += stride) {
    Turn tn;
    if (a.r2) {
      uint32_t seq, in_seq;
      a.byT(at.tok, seq, in_seq);
      turn_at<T, PAIRS, true>(steps + me.f0, a.pos && at.on ? a.pos[at.tok] : (int)in_seq, me.turned,
                              me.first, tn);
    }
    for (int hb = 0; hb < s.per; hb += U) {
      Walk<T, U> next = at;
      next.h += U;
      if (hb + U >= s.per) next.start(s, at.it + stride);
      Raw8<T> ahead[U], gnext[U];
      load_rows<T, U>(s, next, me.e0, D, ahead);
      f32x2 d[U][4];
#pragma unroll
      for (int u = 0; u < U; ++u) cvt8(g[u], d[u]);
      for (int i = 1; i < s.rep; ++i) {
        load_dy(at, i, g);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          f32x2 v[4];
          cvt8(g[u], v);
#pragma unroll
          for (int c = 0; c < 4; ++c) d[u][c] = add2(d[u][c], v[c]);
        }
      }
      load_dy(next, 0, gnext);
      T* out = s.out + ((size_t)at.tok * s.heads + at.h) * D + me.e0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (a.r2) turn<PAIRS>(tn, me.partner, d[u]);
        f32x2 x[4], ss = both2(0.f), ex = ss;
        cvt8(raw[u], x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ss = fma2(x[i], x[i], ss);
          ex = fma2(mul2(d[u][i], w[i]), x[i], ex);
        }
        // r times the row's sum before r's square: no power of a large r alone
        const float r = rsqrtf(fmaf(lane_sum<L>(sum2(ss)), 1.f / D, a.eps));
        const f32x2 r2 = both2(r), m = both2(-(r * (r * lane_sum<L>(sum2(ex))) * (1.f / D)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dw[i] = fma2(d[u][i], mul2(x[i], r2), dw[i]);  // rows past the item's are zeros
          x[i] = mul2(r2, fma2(x[i], m, mul2(d[u][i], w[i])));
        }
        if (at.has(u)) st8(out + (size_t)u * D, x);
      }
      at = next;
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = ahead[u], g[u] = gnext[u];
    }
  }
  if (!part_out) return;
  float* mine = red[threadIdx.x / L] + me.e0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unpack2(dw[i], mine[2 * i], mine[2 * i + 1]);
    mine[2 * i] *= s.scale;
    mine[2 * i + 1] *= s.scale;
  }
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += QN_NT) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NG; ++i) sum += red[i][c];
    part_out[((size_t)blockIdx.x * 2 + is_k) * D + c] = sum;
    part_out[((size_t)blockIdx.x * 2 + !is_k) * D + c] = 0.f;
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

// Heads of an item: as many as leave every SM its threads, QN_HEADS at most; blocks in
// proportion to what the sides move.
struct QkLaunch {
  int per[2], parts[2], blocks[2];
  uint32_t items[2];
};
QkLaunch qk_launch(const gdn_qk_norm_shape& s, bool back) {
  QkLaunch l;
  const int heads[2] = {s.Hq, s.Hk}, Ht = s.Hq + s.Hk, groups = QN_NT / (s.d / 8);
  const int most = back ? QN_PARTS : QN_SMS * 2 * QN_BLOCKS;
  const long long per = (long long)s.rows * Ht / ((long long)QN_SMS * 4 * groups);
  double bytes[2];
  for (int i = 0; i < 2; ++i) {
    const int n = (int)std::max(1ll, std::min<long long>(per, std::min(QN_HEADS, heads[i])));
    l.parts[i] = (heads[i] + n - 1) / n;
    l.per[i] = (heads[i] + l.parts[i] - 1) / l.parts[i];  // parts of even size
    l.items[i] = (uint32_t)s.rows * l.parts[i];
    bytes[i] = heads[i] * ((back ? 2.0 : 1.0) + (s.H ? s.H / heads[i] : 1));
  }
  for (int i = 0; i < 2; ++i) {
    const int share = std::max(1, (int)(most * bytes[i] / (bytes[0] + bytes[1])));
    l.blocks[i] = (int)std::min<long long>(((long long)l.items[i] + groups - 1) / groups, share);
  }
  return l;
}
template <typename T>
QkArgs<T> qk_args(const gdn_qk_norm_shape& s, const QkLaunch& l, const void* q, const void* k,
                  const float* wq, const float* wk, const double* inv_freq, const int* pos,
                  const void* dqn, const void* dkn, void* oq, void* ok) {
  auto side = [&](int i, const void* x, const void* dy, void* out, const float* w, long long ld, int heads,
                  float scale) {
    return QkSide<T>{(const T*)x, (const T*)dy, (T*)out,   w,     ld,
                     FastDiv(l.parts[i]), l.items[i], heads, l.per[i], s.H ? s.H / heads : 1,
                     l.blocks[i], scale};
  };
  return {{side(0, q, dqn, oq, wq, s.ldq, s.Hq, s.q_scale), side(1, k, dkn, ok, wk, s.ldk, s.Hk, 1.f)},
          FastDiv(s.T), s.rot / 2, s.eps, inv_freq, pos};
}

template <typename T, int D, bool PAIRS>
void launch_fwd(const gdn_qk_norm_shape& s, const void* q, const void* k, const float* wq,
                const float* wk, const double* inv_freq, const int* pos, void* qn, void* kn,
                cudaStream_t st) {
  const QkLaunch l = qk_launch(s, false);
  launch(k_qk_norm_fwd<T, D, PAIRS>, dim3(l.blocks[0] + l.blocks[1]), dim3(QN_NT), 0, st, 1,
         qk_args<T>(s, l, q, k, wq, wk, inv_freq, pos, nullptr, nullptr, qn, kn));
}
template <typename T, int D, bool PAIRS>
void launch_bwd(const gdn_qk_norm_shape& s, const void* q, const void* k, const float* wq,
                const float* wk, const double* inv_freq, const int* pos, const void* dqn,
                const void* dkn, void* dq, void* dk, float* part, cudaStream_t st) {
  const QkLaunch l = qk_launch(s, true);
  launch(k_qk_norm_bwd<T, D, PAIRS>, dim3(l.blocks[0] + l.blocks[1]), dim3(QN_NT), 0, st, 1,
         qk_args<T>(s, l, q, k, wq, wk, inv_freq, pos, dqn, dkn, dq, dk), part);
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
  const QkLaunch l = qk_launch(*shape, true);
  const int grid = std::max(1, l.blocks[0] + l.blocks[1]);
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
  const QkLaunch l = qk_launch(s, true);
  if (sums)
    ce = col_sum(part, s.rows > 0 ? l.blocks[0] + l.blocks[1] : 0, 2 * s.d, s.d, dwq, dwk, nullptr,
                 st);
  prof_mark(st, nullptr);
  return ce ? GDN_ERR_CUDA : GDN_OK;
}

}  // extern "C"

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

constexpr int ST_TILE = 8;  // tokens evaluated together: the N extent of the MMAs
// Blocks of 2 warps take 32 columns of a state, a whole line of its rows. Calls of
// more than 8 waves take blocks of 4, which fetch k and q half as often, where the
// coarser last wave costs less than that: 128 sequences of 32 heads of 128 x 128,
// fp32, up to 16 tokens, 149 us in blocks of 4, 169 of 2; 45 of 16 heads of
// 128 x 256, bf16, up to 8 tokens, 32.2 against 31.8.
constexpr int ST_WIDE_COLS = 8 * 152 * 6 * 64;  // columns of a call for blocks of 4
// Blocks that an SM has to have registers for: with dk 128 what its shared memory
// holds (for 12 of 2 warps, 80 registers instead of 96: 16 tokens of one sequence
// 7.6 us instead of 7.2). Half the state leaves room for more: 512 sequences of 32
// heads of 64 x 64, one token, 84 us with 8 blocks of 4 warps, 90 with 6 (at 64
// registers these kernels spill 64 to 84 bytes; calls of several tokens have not been
// timed with 6); small fp32 calls lose by it (93 sequences of 6 heads of 64 x 64:
// 5.6 us with 10, 5.9 with 12).
constexpr int step_blocks(int warps, int dk, bool bf16) {
  return warps == 4 ? (dk == 64 ? 8 : 6) : dk == 64 && bf16 ? 12 : 10;
}

// Two consecutive elements.
__device__ __forceinline__ void ld2(const float* p, float* v) {
  const float2 a = *reinterpret_cast<const float2*>(p);
  v[0] = a.x;
  v[1] = a.y;
}
__device__ __forceinline__ void ld2(const __nv_bfloat16* p, float* v) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
  v[0] = __uint_as_float(u << 16);
  v[1] = __uint_as_float(u & 0xffff0000u);
}

__device__ __forceinline__ void st2(float* p, float a, float b) {
  *reinterpret_cast<float2*>(p) = make_float2(a, b);
}
__device__ __forceinline__ void st2(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}

// Shared memory read again: an ordinary load would be merged with the one for
// the dot products, and the whole state kept in registers between the two.
__device__ __forceinline__ float2 ld2_again(const float* p) {
  float2 r;
  asm volatile("ld.volatile.shared.v2.f32 {%0, %1}, [%2];"
               : "=f"(r.x), "=f"(r.y)
               : "r"(smem_u32(p)));
  return r;
}

// fp32 as two TF32 values (11 significant bits each): the first rounded to
// nearest, so the second holds the rest to 2^-24 of x (truncating the first would
// leave 2^-22, and errors of one sign). A NaN that the addition carries out of the
// first stays in the second.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}
// Two values of k or q as TF32 operands: bf16 values are exact in the first
// part, fp32 ones take both.
__device__ __forceinline__ void operand2(const __nv_bfloat16* p, uint32_t* hi, uint32_t*) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
  hi[0] = u << 16;
  hi[1] = u & 0xffff0000u;
}
__device__ __forceinline__ void operand2(const float* p, uint32_t* hi, uint32_t* lo) {
  const float2 u = *reinterpret_cast<const float2*>(p);
  split_tf32(u.x, hi[0], lo[0]);
  split_tf32(u.y, hi[1], lo[1]);
}
__device__ __forceinline__ void operand1(const __nv_bfloat16* p, uint32_t& hi, uint32_t&) {
  hi = (uint32_t)*reinterpret_cast<const unsigned short*>(p) << 16;
}
__device__ __forceinline__ void operand1(const float* p, uint32_t& hi, uint32_t& lo) {
  split_tf32(*p, hi, lo);
}
// D = A B
__device__ __forceinline__ void mma_tf32z(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// One block: 16 NW value columns of one head of one sequence, 16 per warp; the
// state's columns stay in shared memory. ST_TILE tokens at a time, with S the
// state before them, Gamma_t = alpha_0 .. alpha_t and D_tj = alpha_{j+1} .. alpha_t
// (running products, no quotients of decays):
//   c_t = S^T k_t, p_t = S^T q_t
//   u_t = beta_t (v_t - Gamma_t c_t - sum_{j<t} D_tj (k_t.k_j) u_j)
//   o_t = Gamma_t p_t + sum_{j<=t} D_tj (q_t.k_j) u_j
//   S  <- Gamma_n S + sum_j (D_nj k_j) u_j^T
// which is the token-by-token rule with the state's updates inside the tile
// written out, so the state is read and written once per tile. c, p, the dot
// products and the sum over tokens in the last line are m16n8k8 TF32 MMAs; fp32
// operands (the state, u, fp32 k and q) are taken as two TF32 parts each, to 2^-23 of
// themselves, without the product of the second parts: products are good to 2^-21.6
// (fp32 state off by 1.9e-7 of its 2-norm against 64 bits, about twice what plain fp32
// is; token by token in fp32 the call below takes 330 us, not 186). k and q are used
// as they are in memory; their norms scale the results. S^T (16 columns x 8 rows) is read as A fragments with
// the reduced rows in the order 0 2 4 6 1 3 5 7, in which the fragment is also the
// accumulator's of the update. The state itself is only ever updated by an fp32
// multiply-add (the tensor core's own accumulation would truncate). The sums over
// j are done with selects, never by multiplying with zero: a token that is NaN
// leaves the tokens before it alone. A tile of one token (generation) takes fp32
// multiply-adds in the same layout: the MMAs would use an eighth of their N.
// Lane (g, t) = (lane / 4, lane % 4): columns 2g, 2g + 1, tokens 2t, 2t + 1.
//
// Bound by the state's bytes; with drafted tokens also by the phases of a block
// (load, compute, store), which the few waves of a call pass together. What decided
// (256 x 32 heads of 128 x 128, 8 tokens): 20 to 24 warps per SM (states in
// registers left room for 12 to 16, and the phases did not overlap: 330 us token by
// token, 234 in tiles; in shared memory 186), the swizzle (without it one block less
// per SM, 208 us), and loads of whole lines (see below). One token: 153 us (1.03 GB,
// 6.8 TB/s). 45 sequences of 16 heads of 128 x 256 with up to 8 tokens: 31.8 us
// (142 MB, 4.5 TB/s).
template <typename T, int DK, int NW>
struct StepTile {
  static constexpr int COLS = 16 * NW;
  static constexpr int LD = DK + 8;  // the rows of a fragment start in different banks
  // the block's columns of the state; column c of row r is at c ^ (8 (r / 2 mod 4)),
  // which puts the rows of a fragment into different banks too
  float s[DK * COLS];
  T k[ST_TILE * LD], q[ST_TILE * LD];
};

template <typename T, int DK, int DV, int NW>
__global__ void __launch_bounds__(NW * 32, step_blocks(NW, DK, sizeof(T) == 2))
    k_step(Cache cache, FastDiv byHP, int G, long long ldq, long long ldk, long long ldv,
           long long ldg, long long ldb, float q_scale, float eps, const T* q, const T* k,
           const T* v, const T* g, const T* beta, const float* rate, const float* bias, float* S,
           T* o) {
  using Tile = StepTile<T, DK, NW>;
  constexpr int COLS = Tile::COLS, PARTS = DV / COLS, KS = DK / 8, NT = NW * 32;
  constexpr int LD = Tile::LD;
  constexpr int EP = 16 / (int)sizeof(T);      // elements of 16 bytes
  constexpr int KP = DK / EP;                  // 16-byte pieces of a row
  constexpr int RP = COLS / 4;                 // of a state row
  constexpr int SB = 4;                        // 8-row steps whose loads go ahead of their stores
  constexpr bool TWO = sizeof(T) == 4;         // k and q take two parts
  chain();
  extern __shared__ __align__(16) unsigned char smem[];
  Tile& sm = *reinterpret_cast<Tile*>(smem);
  uint32_t seq, hp;
  byHP(blockIdx.x, seq, hp);
  const SeqCall sc = seq_call(cache, seq);
  if (sc.len == 0 && !sc.store) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, lg = lane >> 2, lt = lane & 3;
  const int H = (int)byHP.d / PARTS, h = hp / PARTS, c0 = (hp - h * PARTS) * COLS;
  const int lcol = warp * 16 + 2 * lg;  // this lane's first column of the block's
  auto tile = [&](int tb) {
    const int n = min(ST_TILE, sc.len - tb), c = sc.commit - tb;
    // a tile that is not the last one ends at the commit
    return sc.store && c > 0 && c < n && tb + n < sc.len ? c : n;
  };
  // A tile's rows of k and q into shared memory (rows past nb: zeros), its gates
  // (lane i: token i mod 8) and v (this lane's columns and tokens) into registers.
  float al, be, a[2][2];
  auto fetch = [&](int tb, int nb) {
    for (int i = tid; i < ST_TILE * 2 * KP; i += NT) {
      const int t = i / (2 * KP), e = i % KP * EP;
      const bool is_q = i / KP & 1;
      const size_t row = (size_t)(sc.t0 + tb + (t < nb ? t : 0));
      cp16((is_q ? sm.q : sm.k) + t * LD + e,
           (is_q ? q + row * ldq : k + row * ldk) + (size_t)(h / G) * DK + e, t < nb);
    }
    al = be = 0.f;
    if ((lane & 7) < nb) {
      const size_t row = (size_t)(sc.t0 + tb + (lane & 7));
      al = ldf(g + row * ldg + h);
      be = ldf(beta + row * ldb + h);
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      a[0][y] = a[1][y] = 0.f;
      if (2 * lt + y < nb) {
        float x[2];
        ld2(v + (size_t)(sc.t0 + tb + 2 * lt + y) * ldv + (size_t)h * DV + c0 + lcol, x);
        a[0][y] = x[0];
        a[1][y] = x[1];
      }
    }
  };
  int nb = tile(0);
  if (nb > 0) fetch(0, nb);
  // The block's part of the state, whole 128-byte lines at a time: an SM gets
  // about one line request in 5 cycles to L2, so the 64 bytes that a warp's
  // fragments take of a row would halve the rate.
  const size_t base = ((size_t)h * DK + tid / RP) * DV + c0 + tid % RP * 4;
  float* mine = sm.s + tid / RP * COLS + (tid % RP * 4 ^ 8 * (tid / RP >> 1 & 3));
  static_assert(NT / RP == 8, "a thread's rows have the same swizzle");
  if (sc.in >= 0) {
    const float* p = S + (size_t)sc.in * H * DK * DV + base;
#pragma unroll
    for (int i = 0; i < DK * RP / NT; ++i)
      cp16(mine + i * (NT / RP) * COLS, p + i * (NT / RP) * DV, true);
  } else {
#pragma unroll
    for (int i = 0; i < DK * RP / NT; ++i)
      *reinterpret_cast<float4*>(mine + i * (NT / RP) * COLS) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  cp_commit();
  auto store = [&]() {  // between barriers
    float* p = S + (size_t)sc.out * H * DK * DV + base;
#pragma unroll
    for (int i = 0; i < DK * RP / NT; ++i)
      *reinterpret_cast<float4*>(p + i * (NT / RP) * DV) =
          *reinterpret_cast<const float4*>(mine + i * (NT / RP) * COLS);
  };
  const float er = rate ? -expf(rate[h]) : 0.f, bi = rate ? bias[h] : 0.f;
  // This lane's state elements of 8 rows: (column 2g, row 8s+2t), (2g+1, ..), and row 8s+2t+1
  float* frag = sm.s + 2 * lt * COLS + (lcol ^ 8 * lt);
  if (sc.store && sc.commit == 0) {
    cp_wait<0>();  // a thread's own pieces
    store();
  }
  for (int tb = 0; tb < sc.len; tb += nb) {
    if (tb) {
      nb = tile(tb);
      __syncthreads();  // the tile before is done with
      fetch(tb, nb);
      cp_commit();
    }
    const int done = tb + nb;
    // whether the state after the tile's first nu tokens is needed
    const bool keep = sc.store && tb < sc.commit && sc.commit <= done;
    const int nu = keep ? sc.commit - tb : nb;
    if (rate) {
      al = er * softplusf_(al + bi);
      be = sigmoidf_(be);
    }
    al = (lane & 7) < nb ? expf(al) : 1.f;
    cp_wait<0>();
    __syncthreads();
    if (nb == 1) {
      // this lane's rows' parts of c and p of its columns, |k|^2, |q|^2, q.k
      float c[2] = {}, p[2] = {}, n[3] = {};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        float kr[2], qr[2];
        ld2(sm.k + 8 * s + 2 * lt, kr);
        ld2(sm.q + 8 * s + 2 * lt, qr);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 x = *reinterpret_cast<const float2*>(frag + (8 * s + r) * COLS);
          c[0] = fmaf(kr[r], x.x, c[0]);
          c[1] = fmaf(kr[r], x.y, c[1]);
          p[0] = fmaf(qr[r], x.x, p[0]);
          p[1] = fmaf(qr[r], x.y, p[1]);
          n[0] = fmaf(kr[r], kr[r], n[0]);
          n[1] = fmaf(qr[r], qr[r], n[1]);
          n[2] = fmaf(qr[r], kr[r], n[2]);
        }
      }
      const float ks = rate ? rsqrtf(lane_sum<4>(n[0]) + eps) : 1.f;
      const float qs = rate ? q_scale * rsqrtf(lane_sum<4>(n[1]) + eps) : 1.f;
      const float alpha = __shfl_sync(0xffffffffu, al, 0), bk = ks * __shfl_sync(0xffffffffu, be, 0);
      const float qk = qs * lane_sum<4>(n[2]);
      float u[2], w[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float vx = __shfl_sync(0xffffffffu, a[x][0], lane & ~3);
        u[x] = bk * fmaf(-alpha * ks, lane_sum<4>(c[x]), vx);  // with the factor of k
        w[x] = fmaf(alpha * qs, lane_sum<4>(p[x]), qk * u[x]);
      }
      if (lt == 0) {
        T* op = o + ((size_t)(sc.t0 + tb) * H + h) * DV + c0 + lcol;
        st2(op, w[0], w[1]);
      }
      if (done == sc.len && !keep) break;
#pragma unroll
      for (int s0 = 0; s0 < KS; s0 += SB) {
        float kr[SB][2];
        float2 old[SB][2];
#pragma unroll
        for (int s = 0; s < SB; ++s) {
          ld2(sm.k + 8 * (s0 + s) + 2 * lt, kr[s]);
#pragma unroll
          for (int r = 0; r < 2; ++r) old[s][r] = ld2_again(frag + (8 * (s0 + s) + r) * COLS);
        }
#pragma unroll
        for (int s = 0; s < SB; ++s)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            *reinterpret_cast<float2*>(frag + (8 * (s0 + s) + r) * COLS) =
                make_float2(fmaf(alpha, old[s][r].x, kr[s][r] * u[0]),
                            fmaf(alpha, old[s][r].y, kr[s][r] * u[1]));
      }
      if (keep) {
        __syncthreads();
        store();
      }
      continue;
    }
    // c, p [column][token] and dot products [k token, q token][k token]; the
    // second parts of the split products are summed apart
    float c[2][4] = {}, p[2][4] = {}, d[2][4] = {}, k2 = 0.f, q2 = 0.f;
    const T *kp = sm.k + lg * LD + 2 * lt, *qp = sm.q + lg * LD + 2 * lt;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      uint32_t kh[2], kl[2], qh[2], ql[2], sh[4], sl[4];
      operand2(kp + 8 * s, kh, kl);
      operand2(qp + 8 * s, qh, ql);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 x = *reinterpret_cast<const float2*>(frag + (8 * s + r) * COLS);
        split_tf32(x.x, sh[2 * r], sl[2 * r]);
        split_tf32(x.y, sh[2 * r + 1], sl[2 * r + 1]);
      }
      mma_tf32(c[0], sh, kh[0], kh[1]);
      mma_tf32(p[0], sh, qh[0], qh[1]);
      const uint32_t ah[4] = {kh[0], qh[0], kh[1], qh[1]};
      mma_tf32(d[0], ah, kh[0], kh[1]);
      mma_tf32(c[1], sl, kh[0], kh[1]);
      mma_tf32(p[1], sl, qh[0], qh[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = __uint_as_float(kh[i]), y = __uint_as_float(qh[i]);
        if (TWO) x += __uint_as_float(kl[i]), y += __uint_as_float(ql[i]);
        k2 = fmaf(x, x, k2);
        q2 = fmaf(y, y, q2);
      }
      if (TWO) {
        const uint32_t al4[4] = {kl[0], ql[0], kl[1], ql[1]};
        mma_tf32(d[1], ah, kl[0], kl[1]);
        mma_tf32(c[1], sh, kl[0], kl[1]);
        mma_tf32(p[1], sh, ql[0], ql[1]);
        mma_tf32(d[1], al4, kh[0], kh[1]);
      }
    }
    float ks = 1.f, qs = 1.f;  // factors of k and q of token g
    if (rate) {
      ks = rsqrtf(lane_sum<4>(k2) + eps);
      qs = q_scale * rsqrtf(lane_sum<4>(q2) + eps);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[0][i] += c[1][i];
      p[0][i] += p[1][i];
      d[0][i] = (d[0][i] + d[1][i]) * (i < 2 ? ks : qs);  // rows: k token g, q token g
    }
    // Of this lane's tokens t = 2 lt + y: f[y] = Gamma_t, last[y] = D_nt (n = nu) and, for
    // j <= t, the factors of u_j: ek[y][j] = -D_tj k_t.k_j, eq[y][j] = D_tj q_t.k_j.
    float ek[2][ST_TILE], eq[2][ST_TILE], f[2] = {1.f, 1.f}, last[2] = {1.f, 1.f}, gamma = 1.f;
#pragma unroll
    for (int j = ST_TILE - 1; j >= 0; --j) {
      const float aj = __shfl_sync(0xffffffffu, al, j);
      if (j < nu) gamma *= aj;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int from = 8 * lt + 4 * y + (j >> 1);  // row t of d
        ek[y][j] = -f[y] * __shfl_sync(0xffffffffu, d[0][j & 1], from);
        eq[y][j] = f[y] * __shfl_sync(0xffffffffu, d[0][2 + (j & 1)], from);
        if (j <= 2 * lt + y)
          f[y] *= aj;
        else if (j < nu)
          last[y] *= aj;
      }
    }
    float w[2][2], bt[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int t = 2 * lt + y;
      const float kt = __shfl_sync(0xffffffffu, ks, 4 * t);
      const float qt = __shfl_sync(0xffffffffu, qs, 4 * t);
      bt[y] = kt * __shfl_sync(0xffffffffu, be, t);  // u_j = beta_j a_j, with the factor of k_j
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        a[x][y] = fmaf(-f[y] * kt, c[0][2 * x + y], a[x][y]);
        w[x][y] = f[y] * qt * p[0][2 * x + y];
      }
    }
#pragma unroll
    for (int j = 0; j < ST_TILE; ++j) {
      if (j >= nb) break;
      const int src = (lane & ~3) | (j >> 1);
      const float u0 = __shfl_sync(0xffffffffu, bt[j & 1] * a[0][j & 1], src);
      const float u1 = __shfl_sync(0xffffffffu, bt[j & 1] * a[1][j & 1], src);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int t = 2 * lt + y;
        if (t > j) {
          a[0][y] = fmaf(ek[y][j], u0, a[0][y]);
          a[1][y] = fmaf(ek[y][j], u1, a[1][y]);
        }
        if (t >= j) {
          w[0][y] = fmaf(eq[y][j], u0, w[0][y]);
          w[1][y] = fmaf(eq[y][j], u1, w[1][y]);
        }
      }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y)
      if (2 * lt + y < nb) {
        T* op = o + ((size_t)(sc.t0 + tb + 2 * lt + y) * H + h) * DV + c0 + lcol;
        st2(op, w[0][y], w[1][y]);
      }
    if (done == sc.len && !keep) break;
    uint32_t uh[4], ul[4];  // A fragment of D_nj u_j: columns x tokens
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        split_tf32(2 * lt + y < nu ? last[y] * (bt[y] * a[x][y]) : 0.f, uh[2 * y + x],
                   ul[2 * y + x]);
#pragma unroll
    for (int s0 = 0; s0 < KS; s0 += SB) {
      float e[SB][4];
      float2 old[SB][2];
#pragma unroll
      for (int s = 0; s < SB; ++s) {
        uint32_t kh[2], kl[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          operand1(sm.k + (2 * lt + y) * LD + 8 * (s0 + s) + lg, kh[y], kl[y]);
          if (2 * lt + y >= nu) kh[y] = kl[y] = 0;  // 0 times a NaN would reach the state
          old[s][y] = *reinterpret_cast<const float2*>(frag + (8 * (s0 + s) + y) * COLS);
        }
        mma_tf32z(e[s], ul, kh[0], kh[1]);
        if (TWO) mma_tf32(e[s], uh, kl[0], kl[1]);
        mma_tf32(e[s], uh, kh[0], kh[1]);
      }
#pragma unroll
      for (int s = 0; s < SB; ++s)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          *reinterpret_cast<float2*>(frag + (8 * (s0 + s) + r) * COLS) =
              make_float2(fmaf(gamma, old[s][r].x, e[s][r]), fmaf(gamma, old[s][r].y, e[s][2 + r]));
    }
    if (keep) {
      __syncthreads();
      store();
    }
  }
}

constexpr int CS_NT = 128;  // threads of a block, 4 channels each
// Tokens of a sequence loaded ahead (fp32, 1024 sequences of up to 7 tokens: 66 us
// with 4, 61 with 6; bf16, 301 of up to 6: 13.1 with 4, 13.4 with 6). The widest fp32
// rows of two sequences would pass 48 KB with 6.
template <typename T, int W>
constexpr int CS_LA = sizeof(T) == 4 && W < 8 ? 6 : 4;
constexpr int CS_BLOCKS = 152 * 16;  // twice what is resident, so that blocks overlap

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

// 4 channels into shared memory without a register in between.
__device__ __forceinline__ void cp4(Raw4<float>* to, const float* p) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(to)), "l"(p)
               : "memory");
}
__device__ __forceinline__ void cp4(Raw4<__nv_bfloat16>* to, const __nv_bfloat16* p) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(smem_u32(to)), "l"(p)
               : "memory");
}

// Sequences whose inputs a thread has in flight: 3, or what 48 KB hold.
template <typename T, int W>
constexpr int conv_stages() {
  constexpr int one = (W - 1 + CS_LA<T, W>) * CS_NT * (int)sizeof(Raw4<T>);
  static_assert(2 * one <= 48 << 10, "what a kernel may use without asking");
  return 3 * one <= 48 << 10 ? 3 : 2;
}

// One thread: 4 channels, whose weights it keeps, of every gridDim.y-th
// sequence; the last W - 1 inputs in registers. Bound by the bytes of the cache
// and of x and y, behind the latency of the index entries and then of the inputs:
// the cached rows and the first CS_LA new ones of the next sequences are in
// flight into shared-memory slots that only this thread reads. 1024 sequences of
// 6144 bf16 channels, one token: 24.6 us (97 MB, 4.0 TB/s); with plain loads 29, two
// sequences ahead in registers 38.
template <typename T, int W>
__global__ void __launch_bounds__(CS_NT, W <= 4 && sizeof(T) == 2 ? 8 : 4)
    k_conv_step(Cache cache, int C, int act, long long ldx, const T* x, const float* w,
                const float* b, T* state, T* y) {
  constexpr int ST = conv_stages<T, W>(), SLOTS = W - 1 + CS_LA<T, W>;
  __shared__ __align__(16) Raw4<T> ring[ST * SLOTS * CS_NT];
  chain();
  const int c0 = (blockIdx.x * CS_NT + threadIdx.x) * 4;
  if (c0 >= C) return;
  x += c0, y += c0, state += c0;
  Raw4<T>* mine = ring + threadIdx.x;  // slot i of stage s: mine[(s SLOTS + i) CS_NT]
  auto fetch = [&](int stage, int seq) {
    if (seq < cache.N) {
      const SeqCall sc = seq_call(cache, seq);
      Raw4<T>* to = mine + stage * SLOTS * CS_NT;
      if (sc.in >= 0 && (sc.len > 0 || sc.store)) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
          cp4(to + j * CS_NT, state + ((size_t)sc.in * (W - 1) + j) * C);
      }
#pragma unroll
      for (int u = 0; u < CS_LA<T, W>; ++u)
        if (u < sc.len) cp4(to + (W - 1 + u) * CS_NT, x + (size_t)(sc.t0 + u) * ldx);
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < ST; ++s) fetch(s, blockIdx.y + s * gridDim.y);
  float wr[4 * W], br[4] = {};
#pragma unroll
  for (int i = 0; i < W; ++i) cvt4(ldraw4(w + (size_t)c0 * W + 4 * i), wr + 4 * i);
  if (b) cvt4(ldraw4(b + c0), br);
  int stage = 0;
  for (int seq = blockIdx.y; seq < cache.N; seq += gridDim.y) {
    const SeqCall sc = seq_call(cache, seq);
    cp_wait<ST - 1>();
    const Raw4<T>* from = mine + stage * SLOTS * CS_NT;
    float win[W - 1][4] = {};
    if (sc.in >= 0) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) cvt4(from[j * CS_NT], win[j]);
    }
    auto store = [&]() {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) st4(state + ((size_t)sc.out * (W - 1) + j) * C, win[j]);
    };
    if (sc.store && sc.commit == 0) store();
    Raw4<T> past;  // the next token's input past the first CS_LA
    if (sc.len > CS_LA<T, W>) past = ldraw4(x + (size_t)(sc.t0 + CS_LA<T, W>) * ldx);
    for (int t = 0; t < sc.len; ++t) {
      float xc[4], out[4];
      cvt4(t < CS_LA<T, W> ? from[(W - 1 + t) * CS_NT] : past, xc);
      if (t >= CS_LA<T, W> && t + 1 < sc.len) past = ldraw4(x + (size_t)(sc.t0 + t + 1) * ldx);
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
      st4(y + (size_t)(sc.t0 + t) * C, out);
      if (sc.store && t + 1 == sc.commit) store();
    }
    fetch(stage, seq + ST * gridDim.y);  // the stage has been read
    if (++stage == ST) stage = 0;
  }
  cp_wait<0>();
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

template <typename T, int DK, int DV, int NW>
void launch_step_warps(const gdn_step_shape& s, const Cache& c, const void* q, const void* k,
                       const void* v, const void* g, const void* beta, const float* rate,
                       const float* bias, float* S, void* o, cudaStream_t st) {
  constexpr int smem = sizeof(StepTile<T, DK, NW>), parts = DV / (16 * NW);
  static_assert(smem <= 48 << 10, "what a kernel may use without asking");
  launch(k_step<T, DK, DV, NW>, dim3((unsigned)s.N * s.H * parts), dim3(NW * 32), smem, st, 1, c,
         FastDiv(s.H * parts), s.H / s.Hk, s.ldq, s.ldk, s.ldv, s.ldg, s.ldb, s.q_scale, s.eps,
         (const T*)q, (const T*)k, (const T*)v, (const T*)g, (const T*)beta, rate, bias, S, (T*)o);
}
template <typename T, int DK, int DV, typename... A>
void launch_step(const gdn_step_shape& s, A... a) {
  if ((long long)s.N * s.H * DV < ST_WIDE_COLS)
    return launch_step_warps<T, DK, DV, 2>(s, a...);
  return launch_step_warps<T, DK, DV, 4>(s, a...);
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
  launch(k_conv_step<T, W>, dim3(gx, gy), dim3(CS_NT), 0, st, 1, c, s.C, s.act,
         (long long)s.ldx, (const T*)x, w, b, (T*)state, (T*)y);
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
      (s.dv != 64 && s.dv != 128 && s.dv != 256) || 8ll * s.N * s.H >= (1ll << 31))
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
  if (!dtype_ok(s.dtype) || s.W < 2 || s.W > 8 || s.C % 4 || s.C > MOST_INDEX ||
      s.N > MOST_INDEX)
    return GDN_ERR_UNSUPPORTED;
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

// Shared pieces of linear attention over whole sequences (include/gdn_lin.h): the
// units of tokens that the kernels work on, and the workspace.
#pragma once

#include "../../include/gdn_lin.h"
#include "gdn_layer.cuh"

namespace gdn {

// Units of `unit` tokens, anchored at the start of every sequence. Fixed-length
// calls: `per` units for each of the nseq sequences of T rows; packed ones: the
// tables that k_lin_plan wrote.
struct LinMap {
  const int* cu;     // packed: DEVICE cu_seqlens; fixed: nullptr
  const int* first;  // packed: first unit of each sequence [nseq + 1]
  const int* owner;  // packed: sequence of each unit [cap] (-1: none)
  int nseq, T, unit, per, cap;
  const int* order;  // packed, or nullptr: the units, longest first [cap]
};
// Unit that the i-th group of blocks takes. Blocks start in order, so the long units do not
// stand behind the short ones.
__device__ __forceinline__ int lin_nth(const LinMap& m, int i) { return m.order ? m.order[i] : i; }

struct LinUnit {
  int seq, row, len;  // its sequence, first row and tokens
  int at, n;          // its index in the sequence and the sequence's units
};
__device__ __forceinline__ bool lin_unit(const LinMap& m, int i, LinUnit& u) {
  int t0, t1;
  if (!m.cu) {
    u.seq = i / m.per;
    u.at = i - u.seq * m.per;
    u.n = m.per;
    t0 = u.seq * m.T;
    t1 = t0 + m.T;
  } else {
    u.seq = m.owner[i];
    if (u.seq < 0) return false;
    const int f = m.first[u.seq];
    u.at = i - f;
    u.n = m.first[u.seq + 1] - f;
    t0 = m.cu[u.seq];
    t1 = m.cu[u.seq + 1];
  }
  u.row = t0 + u.at * m.unit;
  u.len = min(m.unit, t1 - u.row);
  return true;
}
// First unit and number of units of a sequence.
__device__ __forceinline__ void lin_seq(const LinMap& m, int s, int& first, int& n) {
  first = m.cu ? m.first[s] : s * m.per;
  n = m.cu ? m.first[s + 1] - first : m.per;
}

// A log-decay of a token. Below -1e4 every factor is 0 all the same, and sums of
// the clamped values stay finite where those of -inf would give NaN differences.
__device__ __forceinline__ float lin_decay(float g) { return g < -1e4f ? -1e4f : g; }

// gamma summed as pairs of floats (2^-47 of itself: differences of neighbours keep their
// 24 bits where gamma itself is in the thousands; FP64 has 1/64 of the rate, and all wait for it).
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two add_two(Two a, Two b) {
  const float s = a.hi + b.hi, v = s - a.hi;
  const float e = (a.hi - (s - v)) + (b.hi - v) + (a.lo + b.lo);
  Two r;
  r.hi = s + e;
  r.lo = e - (r.hi - s);
  return r;
}
// The sum of the lanes before this one.
__device__ __forceinline__ Two sum_before(Two x) {
  const int l = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Two y = {__shfl_up_sync(0xffffffffu, x.hi, d), __shfl_up_sync(0xffffffffu, x.lo, d)};
    if (l >= d) x = add_two(y, x);
  }
  const Two r = {__shfl_up_sync(0xffffffffu, x.hi, 1), __shfl_up_sync(0xffffffffu, x.lo, 1)};
  return l ? r : Two{0.f, 0.f};
}

// Layouts of a unit's state [dk][dv] in the workspace: as it is, or so that a warp whose
// threads have a key's row each moves 4 elements of 32 rows in one piece: [dv / 4][dk][4].
enum LinLayout { LIN_ROWS, LIN_KEYS };

// What a whole call takes.
struct LinCall {
  gdn_lin_shape s;
  const void *q, *k, *v, *g;
  const float* decay;
  const float* S_in;
  const int* cu;
  void* o;
  float* S_out;
  // backward
  const void* dout;
  const float* dS_out;
  void *dq, *dk, *dv, *dg;
  float *ddecay, *dS_in;
  unsigned char* ws;
  cudaStream_t st;
};

// Writes the tables of a packed call (order: units of at most 64 times `chunk` tokens, or
// nullptr); the status word: DEV_OK or DEV_BAD_CU_SEQLENS.
cudaError_t lin_plan(const LinMap& m, int* first, int* owner, int* order, int chunk, int* status,
                     cudaStream_t st);

// In place over the units of a sequence, D[unit, H, dk, dv] with the units' decays
// whole[unit, H]: D becomes the state before each unit; with `back` also E the gradient
// of the state behind it. The last unit's own D (the first one's E) is not read.
cudaError_t lin_scan(const LinMap& m, const gdn_lin_shape& s, const float* whole, float* D,
                     const float* S_in, float* E, const float* whole_e, const float* dS_out,
                     bool back, int* status, cudaStream_t st);

// bf16 kernels on tcgen05 (gdn_lin_tc.cu).
bool lin_tc_takes(const gdn_lin_shape& s);
size_t lin_tc_bytes(const gdn_lin_shape& s, bool packed, bool back);
cudaError_t lin_tc(const LinCall& c, bool back);

// fp32 kernels (gdn_lin.cu).
size_t lin_simt_bytes(const gdn_lin_shape& s, bool packed, bool back);
cudaError_t lin_simt(const LinCall& c, bool back);

}  // namespace gdn

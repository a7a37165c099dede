// Sequences with a few new tokens each over a cache of states (gdn_step,
// gdn_conv_step, gdn_lin_step): what each of them has to do.
#pragma once

#include "gdn_layer.cuh"

namespace gdn {

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

inline gdn_status check_cache(int N, int n_tok, int n_slots, const int* slot_in,
                              const int* slot_out, const int* cu, const int* commit) {
  if (N < 0 || n_tok < 0 || n_slots < 0) return GDN_ERR_INVALID_ARG;
  if (!cu && n_tok != N) return GDN_ERR_INVALID_ARG;
  if ((!slot_in || !slot_out) && n_slots < N) return GDN_ERR_INVALID_ARG;
  if (!aligned(slot_in, 4) || !aligned(slot_out, 4) || !aligned(cu, 4) || !aligned(commit, 4))
    return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

}  // namespace gdn

// paged_rows.h -- the slots of a paged cache that a query token keeps, and the
// steps they take. Plain C++ besides the markers, so that its arithmetic is
// checked on the host at the ends of its range as well.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define DSA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define DSA_HOST_DEVICE inline
#endif

namespace dsa {

// What a query token attends to: its sequence, last slot and recent slots.
struct PaRow {
  int seq, last;               // last = -1: nothing
  int lo;                      // first recent slot kept (dense: first slot kept)
  int wbase;                   // lo rounded down to 16 or (steps of 32 and more) 32 slots
  int steps;                   // of `step` slots, at least one
};

// Token at position `at` of sequence `seq`: sequences of `cap` slots (below
// 2^31), `list_steps` steps of listed blocks where there is a list.
DSA_HOST_DEVICE PaRow pa_row_at(int64_t cap, int num_seqs, int window, bool list, int list_steps,
                                int step, int seq, int at) {
  PaRow r{0, -1, 0, 0, 1};
  const int64_t pos = at;
  if (seq < 0 || seq >= num_seqs || pos < 0) return r;
  // window counts back from the token, which may stand past the table
  int64_t lo = list || window > 0 ? pos + 1 - window : 0;
  if (lo < 0) lo = 0;
  r.seq = seq;
  r.last = static_cast<int>(pos < cap ? pos : cap - 1);
  if (lo > static_cast<int64_t>(r.last) + 1) lo = static_cast<int64_t>(r.last) + 1;
  r.lo = static_cast<int>(lo);
  r.wbase = r.lo & ~(step < 32 ? step - 1 : 31);
  // (the difference first: last + step can pass 2^31)
  r.steps = r.lo <= r.last ? (r.last - r.wbase) / step + 1 : 0;
  if (list) r.steps += list_steps;
  if (r.steps < 1) r.steps = 1;
  return r;
}

}  // namespace dsa

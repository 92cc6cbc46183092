// Device helpers of the paged caches, shared by pages.cu and paged_attn.cu.
#pragma once

#include "common.cuh"

namespace jssa {

// A bit of the device status word beside those of common.cuh.
constexpr int DEVFLAG_NO_PAGES = 16;  // too few free pages or table entries (nothing changed)

// The packed rows of one sequence's newest tokens: rows [q0, q0 + nq) at positions
// [len - nq, len).
struct NewTokens {
  int64_t q0;
  int nq, len;
};

// The newest tokens of sequence b.  A sequence whose length is outside [0, cap], or whose rows
// are out of order, past n_tokens, or more than its length or than max_q, is left out (nq = 0)
// and flagged.
__device__ __forceinline__ NewTokens new_tokens(const int32_t* q_begin, const int32_t* seq_lens, int b, int64_t cap,
                                                int64_t n_tokens, int64_t max_q, int* status) {
  const int64_t q0 = q_begin[b], q1 = q_begin[b + 1], len = seq_lens[b];
  if (len < 0 || len > cap || q0 < 0 || q1 < q0 || q1 > n_tokens || q1 - q0 > len || q1 - q0 > max_q) {
    flag_error(status, DEVFLAG_BAD_SEQ_LEN);
    return {0, 0, 0};
  }
  return {q0, static_cast<int>(q1 - q0), static_cast<int>(len)};
}

// The sequence that packed row i belongs to: the last whose first row is at or before i.
__device__ __forceinline__ int sequence_of(const int32_t* q_begin, int B, int64_t i) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (q_begin[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace jssa

// paged_common.cuh — what the kernels over a paged K/V cache share: where a call's rows stand and
// which keys they see.
#pragma once

#include "ec_common.cuh"
#include "ec_internal.h"

namespace ec {
namespace paged {

// Position of row r of sequence b; -1 when it lies outside [0, L).
EC_DEV int position(const RowPlaces& at, int b, int r, int L) {
  int64_t p = r;
  if (at.idx != nullptr) p = __ldg(at.idx + b * at.stride + r);
  else if (at.start != nullptr) p += __ldg(at.start + b);
  return p >= 0 && p < L ? static_cast<int>(p) : -1;
}

// Keys of sequence b: kv_len, cut at the scope's end; -1 for a length outside [0, L].
EC_DEV int key_count(const int32_t* kv_len, int b, int L, int scope_hi) {
  if (kv_len == nullptr) return scope_hi;
  const int n = __ldg(kv_len + b);
  return n < 0 || n > L ? -1 : min(n, scope_hi);
}

}  // namespace paged
}  // namespace ec

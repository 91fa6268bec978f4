// fa_checks.h -- argument checks shared by the C-ABI translation units. Host code only.
#pragma once

#include <algorithm>

#include "../../include/fa.h"
#include "fa_internal.h"

namespace fa {

// Checks a paged cache; on FA_OK *out describes it (fa_paged_api.cu).
fa_status check_paged_pool(const fa_paged_kv* c, fa_dtype dt, PagedPool* out);

// Weights [B, Hkv, w_keys] whose rows do not overlap; strides in elements, of an
// axis of one entry ignored. Rows (b, h) and (b', h') overlap where their
// distance, (b - b') batch + (h - h') head, is less than a row.
inline bool weight_strides_ok(long long batch, long long head, int w_keys, int B, int Hkv) {
  constexpr long long kMost = 1ll << 40;  // elements: what follows stays far inside 64 bits
  if (w_keys < 1 || (Hkv > 1 && (head < w_keys || head > kMost)) || (B > 1 && (batch < w_keys || batch > kMost)))
    return false;
  if (B == 1 || Hkv == 1) return true;
  // one axis inside the other, as nearly always
  const long long small = std::min(batch, head), large = std::max(batch, head), inner = batch < head ? B : Hkv;
  if ((large - w_keys) / (inner - 1) >= small) return true;
  // else, for each distance along the axis of fewer entries, the nearest two along the other
  const long long few = B < Hkv ? batch : head, many = B < Hkv ? head : batch;
  const int n_few = std::min(B, Hkv), n_many = std::max(B, Hkv);
  for (int i = 1; i < n_few; ++i) {
    const long long at = i * few, k = std::min(at / many, n_many - 1ll);
    if (at - k * many < w_keys) return false;
    if (k + 1 < n_many && (k + 1) * many - at < w_keys) return false;
  }
  return true;
}

}  // namespace fa

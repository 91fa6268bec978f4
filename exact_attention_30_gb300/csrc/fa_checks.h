// fa_checks.h -- argument checks shared by the C-ABI translation units. Host code only.
#pragma once

#include "../../include/fa.h"
#include "fa_internal.h"

namespace fa {

// Checks a paged cache; on FA_OK *out describes it (fa_paged_api.cu).
fa_status check_paged_pool(const fa_paged_kv* c, fa_dtype dt, PagedPool* out);

// Weights [B, Hkv, w_keys] whose rows do not overlap; strides in elements, of an
// axis of one entry ignored.
inline bool weight_strides_ok(long long batch, long long head, int w_keys, int B, int Hkv) {
  return w_keys >= 1 && (Hkv == 1 || head >= w_keys) && (B == 1 || batch >= w_keys);
}

}  // namespace fa

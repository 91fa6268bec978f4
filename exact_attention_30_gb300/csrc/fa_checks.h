// fa_checks.h -- argument checks shared by the C-ABI translation units. Host code only.
#pragma once

#include "../../include/fa.h"
#include "fa_internal.h"

namespace fa {

// Checks a paged cache; on FA_OK *out describes it (fa_paged_api.cu).
fa_status check_paged_pool(const fa_paged_kv* c, fa_dtype dt, PagedPool* out);

}  // namespace fa

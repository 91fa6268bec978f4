// prompt.cuh -- device-side view of a packed batch of prompts, and the order in
// which CTAs take its blocks (of queries, or of keys).
#pragma once

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

struct PromptView {
  int q0, n;  // first packed token and tokens (queries) of the sequence
  int k0, m;  // first packed key (0 in a paged cache) and keys; query i sees the keys j <= m - n + i
};

// Sequence b. What the device arrays hold is checked (offsets in order and
// within the tensors, lengths within the limits of the call): a sequence that
// fails is empty, n = m = 0, and `bad` is set.
__device__ __forceinline__ PromptView prompt_view(const PromptSeqs& s, int b, bool& bad) {
  PromptView v;
  const int c0 = __ldg(s.cu_q + b), c1 = __ldg(s.cu_q + b + 1);
  int d0 = 0, d1;
  if (s.cu_k != nullptr) {
    d0 = __ldg(s.cu_k + b);
    d1 = __ldg(s.cu_k + b + 1);
  } else {
    d1 = __ldg(s.seq_lens + b);
  }
  const bool ok = 0 <= c0 && c0 <= c1 && c1 <= s.total_q && c1 - c0 <= s.max_q && 0 <= d0 && d0 <= d1 &&
                  d1 <= s.total_k && d1 - d0 <= s.max_k;
  bad = bad || !ok;
  v.q0 = ok ? c0 : 0;
  v.n = ok ? c1 - c0 : 0;
  v.k0 = ok ? d0 : 0;
  v.m = ok ? d1 - d0 : 0;
  return v;
}

// The backward's workspace: first slot (128 rows) of sequence b whose first
// packed token is q0. Slots of different sequences do not overlap: between two
// of them ceil(n / tile_tokens) <= floor((q0 + n) / tile_tokens) + 1 - floor(q0 / tile_tokens).
__device__ __forceinline__ int prompt_slot(int q0, int b, int tile_tokens) { return q0 / tile_tokens + b; }

// The blocks of a batch by levels: sequence b has `count` blocks, on the levels
// base .. base + count - 1, and a higher level is more work. Blocks are listed
// from the highest level down (the longest first, so that the short ones fill
// the last wave), sequences in order within a level.
struct PromptSpan {
  int base, count;
};

// Blocks of `per` tokens each: their level is how many blocks' worth of keys
// their last query sees.
__device__ __forceinline__ PromptSpan query_span(const PromptView& v, int per) {
  const int past = v.m - v.n;
  return PromptSpan{past > 0 ? past / per : 0, (v.n + per - 1) / per};
}

__device__ __forceinline__ int warp_sum(int x) { return __reduce_add_sync(0xffffffffu, x); }

// Whole warp: blocks of all sequences, and the highest level plus one. span(b)
// is the span of sequence b; the lanes keep those of the first 32 sequences.
template <class F>
__device__ __forceinline__ int count_blocks(int B, int lane, const F& span, PromptSpan& first, int& top) {
  first = lane < B ? span(lane) : PromptSpan{0, 0};
  int n = first.count, hi = first.count ? first.base + first.count : 0;
  for (int b = lane + 32; b < B; b += 32) {
    const PromptSpan s = span(b);
    n += s.count;
    if (s.count) hi = max(hi, s.base + s.count);
  }
  top = __reduce_max_sync(0xffffffffu, hi);
  return warp_sum(n);
}

// Whole warp: block `idx` (< count_blocks) of the list: its sequence, and its
// index within the sequence. The level by bisection: blocks on levels >= L are
// sum_b min(max(base + count - L, 0), count).
template <class F>
__device__ __forceinline__ void find_block(int B, int lane, const F& span, const PromptSpan& first, int top, int idx,
                                           int& seq, int& block) {
  auto at_least = [&](int L) {
    int n = min(max(first.base + first.count - L, 0), first.count);
    for (int b = lane + 32; b < B; b += 32) {
      const PromptSpan s = span(b);
      n += min(max(s.base + s.count - L, 0), s.count);
    }
    return warp_sum(n);
  };
  int lo = 0, hi = top, above = 0;  // at_least(lo) > idx >= above = at_least(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1, n = at_least(mid);
    if (n > idx) {
      lo = mid;
    } else {
      hi = mid;
      above = n;
    }
  }
  int r = idx - above;  // index among the sequences with a block on level lo
  seq = 0;
  block = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const PromptSpan s = b0 == 0 ? first : (b0 + lane < B ? span(b0 + lane) : PromptSpan{0, 0});
    const unsigned here = __ballot_sync(0xffffffffu, s.base <= lo && lo < s.base + s.count);
    const int n = __popc(here);
    if (r < n) {
      const bool mine = ((here >> lane) & 1u) && __popc(here & ((1u << lane) - 1u)) == r;
      const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
      seq = b0 + src;
      block = lo - __shfl_sync(0xffffffffu, s.base, src);
      return;
    }
    r -= n;
  }
}

}  // namespace fa

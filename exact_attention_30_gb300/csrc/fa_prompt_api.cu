// fa_prompt_api.cu -- the C ABI of the prompt operators (fa_prompt_fwd,
// fa_prompt_paged, fa_prompt_bwd, fa_prompt_key_weights and its paged form):
// argument validation, tensor maps, plans and launch. Host code only.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/fa.h"
#include "fa_checks.h"
#include "fa_internal.h"

using namespace fa;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Elements between the tokens of a packed [total, heads, d] tensor.
bool token_stride_ok(long long s, int total, int heads, int d) {
  return total == 1 || (s >= (long long)heads * d && s % 8 == 0 && s <= (1ll << 38));
}
long long token_stride(long long s, int total, int heads, int d) { return total == 1 ? (long long)heads * d : s; }

fa_status check_heads(int B, int Hq, int Hkv, int d, fa_dtype dt) {
  if (B < 1 || Hq < 1 || Hkv < 1 || d < 1 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (dt != FA_F32 && dt != FA_BF16) return FA_ERR_INVALID_ARG;
  if (dt != FA_BF16 || (d != 64 && d != 128)) return FA_ERR_UNSUPPORTED;
  if (Hq / Hkv > kPromptMaxGroup || (long long)B * Hkv > (1 << 24)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

fa_status check_sizes(int B, int Hq, int Hkv, int total_q, int total_k, int max_q, int max_k, int d, float scale,
                      fa_dtype dt) {
  const fa_status s = check_heads(B, Hq, Hkv, d, dt);
  if (s != FA_OK) return s;
  if (total_q < 1 || total_k < 1 || max_q < 1 || max_k < 1 || max_q > total_q || max_k > total_k)
    return FA_ERR_INVALID_ARG;
  if (total_q > kPromptMaxTokens || total_k > kPromptMaxTokens) return FA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// Blocks of `per` tokens that B sequences of at most max_len tokens, `total`
// in all, can have.
long long most_blocks(int B, int total, int max_len, int per) {
  const long long by_total = total / per + (long long)B;
  const long long by_len = (long long)B * ((max_len + per - 1) / per);
  return std::min(by_total, by_len);
}

// The longest that a warp may wait for another one. Some wait for a whole block:
// the scheduler for its end, the output warps for a query tile's last P V. Its
// `tiles` steps take 0.7 to 1.4 us each, and finding it among B sequences some
// 0.2 us for each 32 of them and level of the list (24 at most).
unsigned long long wait_limit(long long tiles, int B) {
  return std::max(kDefaultWaitLimitNs, 16000ull * (unsigned long long)tiles + 1000ull * (unsigned long long)B);
}

// Packed queries (or O, dO, dQ): (d, head of the group, token, K/V head).
bool encode_grouped(CUtensorMap* m, const void* p, long long stride, int G, int Hkv, int total, int tile_tokens, int d) {
  const long long dims[4] = {d, G, total, Hkv}, strides[3] = {d, stride, (long long)G * d};
  const int box[4] = {64, G, tile_tokens, 1};
  return encode_bf16(m, p, 4, dims, strides, box);
}
// Packed keys or values: (d, token, head).
bool encode_keys(CUtensorMap* m, const void* p, long long stride, int Hkv, int total, int box_rows, int d) {
  const long long dims[3] = {d, total, Hkv}, strides[2] = {stride, d};
  const int box[3] = {64, box_rows, 1};
  return encode_bf16(m, p, 3, dims, strides, box);
}

// Scratch of the backward: fp32 dQ accumulator, two statistics per row, split
// units' partial dV and dK, and the main kernel's schedule (item counter, total,
// sequence order, B + 1 prefix sums).
struct BwdLayout {
  long long slots, rows;  // workspace slots per K/V head, rows of 128 of all heads
  long long units;        // at least as many (K/V head, key tile) units as there are
  int splits;
  size_t lse2, drow, part, sched, total;
};
BwdLayout bwd_layout(int B, int G, int Hkv, int total_q, int total_k, int max_q, int max_k, int d) {
  BwdLayout L{};
  L.slots = (long long)total_q / prompt_tile_tokens(G) + B + 1;
  L.rows = L.slots * Hkv * 128;
  L.units = most_blocks(B, total_k, max_k, 128) * Hkv;
  L.splits = plan_prompt_bwd_splits(L.units, (max_q + prompt_tile_tokens(G) - 1) / prompt_tile_tokens(G), fwd_slots());
  L.lse2 = align_up((size_t)L.rows * d * sizeof(float), 256);
  L.drow = L.lse2 + align_up((size_t)L.rows * sizeof(float), 256);
  L.part = L.drow + align_up((size_t)L.rows * sizeof(float), 256);
  L.sched = L.part + (L.splits > 1 ? (size_t)L.units * L.splits * 2 * 128 * d * sizeof(float) : 0);
  L.total = L.sched + align_up(sizeof(int) * (3 + 2 * (size_t)B), 256);
  return L;
}

struct FwdPlan {
  long long max_blocks;
  int splits;
  size_t lpart, blocks, total;  // scratch: partial rows, their log-sum-exps, the blocks
};
FwdPlan fwd_plan(int B, int G, int Hkv, int total_q, int max_q, int max_k, int d) {
  FwdPlan p{};
  p.max_blocks = most_blocks(B, total_q, max_q, 2 * prompt_tile_tokens(G));
  p.splits = plan_prompt_splits(p.max_blocks * Hkv, (max_k + 127) / 128, fwd_slots());
  if (p.splits > 1) {
    const size_t rows = (size_t)p.max_blocks * Hkv * p.splits * 256;
    p.lpart = align_up(rows * d * sizeof(float), 256);
    p.blocks = p.lpart + align_up(rows * sizeof(float), 256);
    p.total = p.blocks + align_up((size_t)p.max_blocks * Hkv * sizeof(int4), 256);
  }
  return p;
}

// What fa_prompt_fwd and fa_prompt_paged check alike.
fa_status check_fwd(const void* Q, long long q_stride, const void* O, long long o_stride, const float* LSE,
                    const int* cu_q, int B, int Hq, int Hkv, int total_q, int max_q, int d, const void* workspace) {
  if (!Q || !O || !LSE || !cu_q) return FA_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(O, 16) || !aligned(LSE, 4) || !aligned(cu_q, 4) || !aligned(workspace, 256))
    return FA_ERR_INVALID_ARG;
  if (!token_stride_ok(q_stride, total_q, Hq, d) || !token_stride_ok(o_stride, total_q, Hq, d)) return FA_ERR_INVALID_ARG;
  // rows of all blocks (key ranges are planned only where there are few)
  if (most_blocks(B, total_q, max_q, 2 * prompt_tile_tokens(Hq / Hkv)) * Hkv > 0x7fffffff / 256) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// What they do alike, once everything is checked and the keys' part of `a` stands.
fa_status fwd_launch(PromptFwdArgs& a, const void* Q, long long q_stride, void* O, long long o_stride, float* LSE,
                     const int* cu_q, int B, int Hq, int total_q, int max_q, long long key_bytes, void* workspace,
                     size_t workspace_bytes, int d, float scale, void* stream) {
  const int G = Hq / a.Hkv;
  a.seqs.cu_q = cu_q;
  a.seqs.B = B;
  a.seqs.total_q = total_q;
  a.seqs.max_q = max_q;
  a.O = O;
  a.o_stride = token_stride(o_stride, total_q, Hq, d);
  a.LSE = LSE;
  a.G = G;
  a.tile_tokens = prompt_tile_tokens(G);
  a.g_div = fast_div((unsigned)G);
  a.heads_per_group = causal_heads_per_group(a.Hkv, key_bytes, 96ll << 20);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.wait_limit_ns = wait_limit((a.seqs.max_k + 127) / 128, B);
  a.status = device_status_ptr();
  if (!a.status) return FA_ERR_CUDA;
  const FwdPlan p = fwd_plan(B, G, a.Hkv, total_q, max_q, a.seqs.max_k, d);
  a.max_blocks = p.max_blocks;
  a.splits = workspace ? p.splits : 1;
  a.slots = fwd_slots();
  if (a.splits > 1) {
    if (workspace_bytes < p.total) return FA_ERR_INVALID_ARG;
    a.Opart = static_cast<float*>(workspace);
    a.Lpart = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.lpart);
    a.blocks = reinterpret_cast<int4*>(static_cast<char*>(workspace) + p.blocks);
  }
  if (!encode_grouped(&a.tmQ, Q, token_stride(q_stride, total_q, Hq, d), G, a.Hkv, total_q, a.tile_tokens, d) ||
      !encode_grouped(&a.tmO, O, a.o_stride, G, a.Hkv, total_q, a.tile_tokens, d))
    return FA_ERR_CUDA;
  return launch_prompt_fwd(a, d, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// What the two entry points of the keys' weights check alike, and do alike.
fa_status check_weights(const void* Q, long long q_stride, const float* LSE, const float* W, long long w_batch,
                        long long w_head, int w_keys, const int* cu_q, int B, int Hq, int Hkv, int total_q, int window,
                        int d, int flags) {
  if (!Q || !LSE || !W || !cu_q || window < 0 || (flags & ~FA_ACCUMULATE)) return FA_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(LSE, 4) || !aligned(W, 4) || !aligned(cu_q, 4)) return FA_ERR_INVALID_ARG;
  if (!token_stride_ok(q_stride, total_q, Hq, d) || !weight_strides_ok(w_batch, w_head, w_keys, B, Hkv))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}
fa_status weights_launch(PromptWeightArgs& a, const void* Q, long long q_stride, const float* LSE, float* W,
                         long long w_batch, long long w_head, int w_keys, const int* cu_q, int B, int Hq, int total_q,
                         int max_q, int window, int d, float scale, int flags, void* stream) {
  a.G = Hq / a.Hkv;
  a.tile_tokens = prompt_tile_tokens(a.G);
  a.g_div = fast_div((unsigned)a.G);
  a.seqs.cu_q = cu_q;
  a.seqs.B = B;
  a.seqs.total_q = total_q;
  a.seqs.max_q = max_q;
  a.LSE = LSE;
  a.W = W;
  a.w_batch = w_batch;
  a.w_head = w_head;
  a.w_keys = w_keys;
  a.window = window;
  a.accumulate = flags & FA_ACCUMULATE ? 1 : 0;
  a.heads_per_group = causal_heads_per_group(a.Hkv, 2ll * total_q * a.G * d, 96ll << 20);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.wait_limit_ns = wait_limit((max_q + a.tile_tokens - 1) / a.tile_tokens, B);
  a.status = device_status_ptr();
  if (!a.status) return FA_ERR_CUDA;
  if (a.max_units * a.Hkv > 0x7fffffffll) return FA_ERR_UNSUPPORTED;
  if (!encode_grouped(&a.tmQ, Q, token_stride(q_stride, total_q, Hq, d), a.G, a.Hkv, total_q, a.tile_tokens, d))
    return FA_ERR_CUDA;
  return launch_prompt_weights(a, d, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

namespace fa {

int plan_prompt_splits(long long units, int key_tiles, int slots) {
  if (units < 1 || key_tiles < 1 || slots < 1) return 1;
  float best = 0.f;
  int splits = 1;
  for (int s = 1; s <= key_tiles && s <= kPrefixMaxSplits; ++s) {
    const float cost = prompt_split_cost((float)units, key_tiles, slots, s);
    if (s == 1 || cost < best) {
      best = cost;
      splits = s;
    }
  }
  return splits;
}

}  // namespace fa

extern "C" {

fa_status fa_prompt_fwd(const void* Q, const void* K, const void* V, long long q_stride, long long k_stride,
                        long long v_stride, void* O, long long o_stride, float* LSE, const int* cu_seqlens_q,
                        const int* cu_seqlens_k, int B, int Hq, int Hkv, int total_q, int total_k, int max_seqlen_q,
                        int max_seqlen_k, void* workspace, size_t workspace_bytes, int d, float scale, fa_dtype dt,
                        void* stream) {
  fa_status s = check_sizes(B, Hq, Hkv, total_q, total_k, max_seqlen_q, max_seqlen_k, d, scale, dt);
  if (s != FA_OK) return s;
  s = check_fwd(Q, q_stride, O, o_stride, LSE, cu_seqlens_q, B, Hq, Hkv, total_q, max_seqlen_q, d, workspace);
  if (s != FA_OK) return s;
  if (!K || !V || !cu_seqlens_k) return FA_ERR_INVALID_ARG;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(cu_seqlens_k, 4)) return FA_ERR_INVALID_ARG;
  if (!token_stride_ok(k_stride, total_k, Hkv, d) || !token_stride_ok(v_stride, total_k, Hkv, d))
    return FA_ERR_INVALID_ARG;
  PromptFwdArgs a;
  std::memset(&a, 0, sizeof(a));
  a.Hkv = Hkv;
  a.seqs.cu_k = cu_seqlens_k;
  a.seqs.total_k = total_k;
  a.seqs.max_k = max_seqlen_k;
  if (!encode_keys(&a.tmK, K, token_stride(k_stride, total_k, Hkv, d), Hkv, total_k, 128, d) ||
      !encode_keys(&a.tmV, V, token_stride(v_stride, total_k, Hkv, d), Hkv, total_k, 128, d))
    return FA_ERR_CUDA;
  return fwd_launch(a, Q, q_stride, O, o_stride, LSE, cu_seqlens_q, B, Hq, total_q, max_seqlen_q, 4ll * total_k * d,
                    workspace, workspace_bytes, d, scale, stream);
}

size_t fa_prompt_fwd_workspace_bytes(int B, int Hq, int Hkv, int total_q, int max_seqlen_q, int max_seqlen_k, int d,
                                     fa_dtype dt) {
  if (check_heads(B, Hq, Hkv, d, dt) != FA_OK || total_q < 1 || max_seqlen_q < 1 || max_seqlen_q > total_q ||
      max_seqlen_k < 1)
    return 0;
  // a table can hold more keys than a sequence may have
  return fwd_plan(B, Hq / Hkv, Hkv, total_q, max_seqlen_q, std::min(max_seqlen_k, kPagedMaxKeys), d).total;
}

fa_status fa_prompt_paged(const void* Q, long long q_stride, const fa_paged_kv* cache, const int* block_tables,
                          int max_pages, const int* seq_lens, void* O, long long o_stride, float* LSE,
                          const int* cu_seqlens_q, int B, int Hq, int total_q, int max_seqlen_q, void* workspace,
                          size_t workspace_bytes, float scale, fa_dtype dt, void* stream) {
  PromptFwdArgs a;
  std::memset(&a, 0, sizeof(a));
  fa_status s = check_paged_pool(cache, dt, &a.pool);
  if (s != FA_OK) return s;
  if (max_pages < 1) return FA_ERR_INVALID_ARG;
  const long long most = std::min<long long>((long long)max_pages * cache->page_size, kPagedMaxKeys);
  s = check_sizes(B, Hq, cache->kv_heads, total_q, (int)most, max_seqlen_q, (int)most, cache->d, scale, dt);
  if (s != FA_OK) return s;
  s = check_fwd(Q, q_stride, O, o_stride, LSE, cu_seqlens_q, B, Hq, cache->kv_heads, total_q, max_seqlen_q, cache->d,
                workspace);
  if (s != FA_OK) return s;
  if (!block_tables || !seq_lens || !aligned(block_tables, 4) || !aligned(seq_lens, 4)) return FA_ERR_INVALID_ARG;
  a.Hkv = cache->kv_heads;
  a.seqs.seq_lens = seq_lens;
  a.seqs.total_k = (int)most;
  a.seqs.max_k = (int)most;
  a.block_tables = block_tables;
  a.max_pages = max_pages;
  a.page_div = fast_div((unsigned)cache->page_size);
  a.box_rows = pool_box_rows(cache->page_size, 128);
  if (!encode_pool_bf16(&a.tmK, a.pool, false, cache->d, a.box_rows) ||
      !encode_pool_bf16(&a.tmV, a.pool, true, cache->d, a.box_rows))
    return FA_ERR_CUDA;
  const long long keys = std::min<long long>((long long)cache->num_pages * cache->page_size, B * most);
  return fwd_launch(a, Q, q_stride, O, o_stride, LSE, cu_seqlens_q, B, Hq, total_q, max_seqlen_q, 4 * keys * cache->d,
                    workspace, workspace_bytes, cache->d, scale, stream);
}

size_t fa_prompt_bwd_workspace_bytes(int B, int Hq, int Hkv, int total_q, int total_k, int max_seqlen_q,
                                     int max_seqlen_k, int d, fa_dtype dt) {
  if (check_sizes(B, Hq, Hkv, total_q, total_k, max_seqlen_q, max_seqlen_k, d, 1.f, dt) != FA_OK) return 0;
  const BwdLayout L = bwd_layout(B, Hq / Hkv, Hkv, total_q, total_k, max_seqlen_q, max_seqlen_k, d);
  return L.rows > 0x7fffffffll ? 0 : L.total;
}

fa_status fa_prompt_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO, long long q_stride,
                        long long k_stride, long long v_stride, long long o_stride, long long do_stride,
                        const float* LSE, void* dQ, void* dK, void* dV, long long dq_stride, long long dk_stride,
                        long long dv_stride, const int* cu_seqlens_q, const int* cu_seqlens_k, void* workspace,
                        size_t workspace_bytes, int B, int Hq, int Hkv, int total_q, int total_k, int max_seqlen_q,
                        int max_seqlen_k, int d, float scale, fa_dtype dt, void* stream) {
  const fa_status s = check_sizes(B, Hq, Hkv, total_q, total_k, max_seqlen_q, max_seqlen_k, d, scale, dt);
  if (s != FA_OK) return s;
  if (!Q || !K || !V || !O || !dO || !LSE || !dQ || !dK || !dV || !cu_seqlens_q || !cu_seqlens_k || !workspace)
    return FA_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(O, 16) || !aligned(dO, 16) || !aligned(dQ, 16) ||
      !aligned(dK, 16) || !aligned(dV, 16) || !aligned(LSE, 4) || !aligned(cu_seqlens_q, 4) ||
      !aligned(cu_seqlens_k, 4) || !aligned(workspace, 256))
    return FA_ERR_INVALID_ARG;
  if (!token_stride_ok(q_stride, total_q, Hq, d) || !token_stride_ok(o_stride, total_q, Hq, d) ||
      !token_stride_ok(do_stride, total_q, Hq, d) || !token_stride_ok(dq_stride, total_q, Hq, d) ||
      !token_stride_ok(k_stride, total_k, Hkv, d) || !token_stride_ok(v_stride, total_k, Hkv, d) ||
      !token_stride_ok(dk_stride, total_k, Hkv, d) || !token_stride_ok(dv_stride, total_k, Hkv, d))
    return FA_ERR_INVALID_ARG;
  const int G = Hq / Hkv;
  const BwdLayout L = bwd_layout(B, G, Hkv, total_q, total_k, max_seqlen_q, max_seqlen_k, d);
  if (Hkv > 65535 || L.rows > 0x7fffffffll) return FA_ERR_UNSUPPORTED;
  if (workspace_bytes < L.total) return FA_ERR_INVALID_ARG;
  PromptBwdArgs a;
  std::memset(&a, 0, sizeof(a));
  a.seqs.cu_q = cu_seqlens_q;
  a.seqs.cu_k = cu_seqlens_k;
  a.seqs.B = B;
  a.seqs.total_q = total_q;
  a.seqs.total_k = total_k;
  a.seqs.max_q = max_seqlen_q;
  a.seqs.max_k = max_seqlen_k;
  a.Hkv = Hkv;
  a.G = G;
  a.tile_tokens = prompt_tile_tokens(G);
  a.g_div = fast_div((unsigned)G);
  a.slots = (int)L.slots;
  a.o_stride = token_stride(o_stride, total_q, Hq, d);
  a.do_stride = token_stride(do_stride, total_q, Hq, d);
  a.dq_stride = token_stride(dq_stride, total_q, Hq, d);
  a.dk_stride = token_stride(dk_stride, total_k, Hkv, d);
  a.dv_stride = token_stride(dv_stride, total_k, Hkv, d);
  a.O = O;
  a.dO = dO;
  a.LSE = LSE;
  a.dQ = dQ;
  a.dK = dK;
  a.dV = dV;
  char* ws = static_cast<char*>(workspace);
  a.dQacc = reinterpret_cast<float*>(ws);
  a.lse2 = reinterpret_cast<float*>(ws + L.lse2);
  a.Drow = reinterpret_cast<float*>(ws + L.drow);
  a.item_counter = reinterpret_cast<int*>(ws + L.sched);
  a.nseq = B;
  if (L.units > (1 << 28)) return FA_ERR_UNSUPPORTED;
  a.items = (int)L.units * L.splits;
  a.splits = L.splits;
  a.dKVpart = L.splits > 1 ? reinterpret_cast<float*>(ws + L.part) : nullptr;
  a.seq.causal = 1;
  a.seq.H = Hkv;
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.wait_limit_ns = kDefaultWaitLimitNs;
  a.debug_skip_q = -1;
  a.status = device_status_ptr();
  if (!a.status) return FA_ERR_CUDA;
  if (!encode_grouped(&a.tmQ, Q, token_stride(q_stride, total_q, Hq, d), G, Hkv, total_q, a.tile_tokens, d) ||
      !encode_grouped(&a.tmdO, dO, a.do_stride, G, Hkv, total_q, a.tile_tokens, d) ||
      !encode_keys(&a.tmK, K, token_stride(k_stride, total_k, Hkv, d), Hkv, total_k, 128, d) ||
      !encode_keys(&a.tmV, V, token_stride(v_stride, total_k, Hkv, d), Hkv, total_k, 128, d) ||
      !encode_acc_f32(&a.tmDQacc, a.dQacc, L.rows, d))
    return FA_ERR_CUDA;
  return launch_prompt_bwd(a, d, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_prompt_key_weights(const void* Q, const void* K, long long q_stride, long long k_stride, const float* LSE,
                                float* W, long long w_batch_stride, long long w_head_stride, int w_keys,
                                const int* cu_seqlens_q, const int* cu_seqlens_k, int B, int Hq, int Hkv, int total_q,
                                int total_k, int max_seqlen_q, int max_seqlen_k, int window, int d, float scale,
                                int flags, fa_dtype dt, void* stream) {
  fa_status s = check_sizes(B, Hq, Hkv, total_q, total_k, max_seqlen_q, max_seqlen_k, d, scale, dt);
  if (s != FA_OK) return s;
  s = check_weights(Q, q_stride, LSE, W, w_batch_stride, w_head_stride, w_keys, cu_seqlens_q, B, Hq, Hkv, total_q, window,
                    d, flags);
  if (s != FA_OK) return s;
  if (!K || !cu_seqlens_k || !aligned(K, 16) || !aligned(cu_seqlens_k, 4) || !token_stride_ok(k_stride, total_k, Hkv, d))
    return FA_ERR_INVALID_ARG;
  PromptWeightArgs a;
  std::memset(&a, 0, sizeof(a));
  a.Hkv = Hkv;
  a.seqs.cu_k = cu_seqlens_k;
  a.seqs.total_k = total_k;
  a.seqs.max_k = max_seqlen_k;
  if (!encode_keys(&a.tmK, K, token_stride(k_stride, total_k, Hkv, d), Hkv, total_k, 128, d)) return FA_ERR_CUDA;
  a.max_units = most_blocks(B, total_k, max_seqlen_k, 256);
  return weights_launch(a, Q, q_stride, LSE, W, w_batch_stride, w_head_stride, w_keys, cu_seqlens_q, B, Hq, total_q,
                        max_seqlen_q, window, d, scale, flags, stream);
}

fa_status fa_prompt_key_weights_paged(const void* Q, long long q_stride, const fa_paged_kv* cache,
                                      const int* block_tables, int max_pages, const int* seq_lens, const float* LSE,
                                      float* W, long long w_batch_stride, long long w_head_stride, int w_keys,
                                      const int* cu_seqlens_q, int B, int Hq, int total_q, int max_seqlen_q, int window,
                                      float scale, int flags, fa_dtype dt, void* stream) {
  PromptWeightArgs a;
  std::memset(&a, 0, sizeof(a));
  fa_status s = check_paged_pool(cache, dt, &a.pool);
  if (s != FA_OK) return s;
  if (max_pages < 1) return FA_ERR_INVALID_ARG;
  const long long most = std::min<long long>((long long)max_pages * cache->page_size, kPagedMaxKeys);
  s = check_sizes(B, Hq, cache->kv_heads, total_q, (int)most, max_seqlen_q, (int)most, cache->d, scale, dt);
  if (s != FA_OK) return s;
  s = check_weights(Q, q_stride, LSE, W, w_batch_stride, w_head_stride, w_keys, cu_seqlens_q, B, Hq, cache->kv_heads,
                    total_q, window, cache->d, flags);
  if (s != FA_OK) return s;
  if (!block_tables || !seq_lens || !aligned(block_tables, 4) || !aligned(seq_lens, 4)) return FA_ERR_INVALID_ARG;
  a.Hkv = cache->kv_heads;
  a.seqs.seq_lens = seq_lens;
  a.seqs.total_k = (int)most;
  a.seqs.max_k = (int)most;
  a.block_tables = block_tables;
  a.max_pages = max_pages;
  a.box_rows = pool_box_rows(cache->page_size, 128);
  if (!encode_pool_bf16(&a.tmK, a.pool, false, cache->d, a.box_rows)) return FA_ERR_CUDA;
  a.max_units = (long long)B * ((std::min<long long>(most, w_keys) + 255) / 256);
  return weights_launch(a, Q, q_stride, LSE, W, w_batch_stride, w_head_stride, w_keys, cu_seqlens_q, B, Hq, total_q,
                        max_seqlen_q, window, cache->d, scale, flags, stream);
}

}  // extern "C"

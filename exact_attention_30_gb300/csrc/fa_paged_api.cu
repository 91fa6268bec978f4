// fa_paged_api.cu -- the C ABI of the paged key/value cache operators
// (fa_kv_append, fa_decode_paged, fa_decode_shared): argument validation and
// launch. Host code only.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/fa.h"
#include "fa_internal.h"

using namespace fa;

namespace {

constexpr int kMaxPageSize = 65536;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A stride of an axis of `extent` entries: a multiple of 8 elements (16-byte
// vectors) of at least `min` elements. An axis of one entry has no stride.
bool stride_ok(long long stride, int extent, long long min) {
  return extent == 1 || (stride >= min && stride % 8 == 0 && stride <= (1ll << 38));
}

fa_status check_pool(const fa_paged_kv* c, fa_dtype dt, PagedPool* out) {
  if (!c || !c->k || !c->v) return FA_ERR_INVALID_ARG;
  if (dt != FA_F32 && dt != FA_BF16) return FA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->kv_heads < 1 || c->page_size < 1 || c->d < 1) return FA_ERR_INVALID_ARG;
  if (dt != FA_BF16 || (c->d != 64 && c->d != 128)) return FA_ERR_UNSUPPORTED;
  if (c->page_size % 8 != 0 || c->page_size > kMaxPageSize) return FA_ERR_UNSUPPORTED;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return FA_ERR_INVALID_ARG;
  if (!stride_ok(c->k_page_stride, c->num_pages, c->d) || !stride_ok(c->k_head_stride, c->kv_heads, c->d) ||
      !stride_ok(c->k_row_stride, c->page_size, c->d) || !stride_ok(c->v_page_stride, c->num_pages, c->d) ||
      !stride_ok(c->v_head_stride, c->kv_heads, c->d) || !stride_ok(c->v_row_stride, c->page_size, c->d))
    return FA_ERR_INVALID_ARG;
  // an axis of one entry gets a stride that a tensor map accepts
  auto st = [&](long long s, int extent) { return extent == 1 ? (long long)c->d : s; };
  PagedPool p{};
  p.k = c->k;
  p.v = c->v;
  p.k_page = st(c->k_page_stride, c->num_pages);
  p.k_head = st(c->k_head_stride, c->kv_heads);
  p.k_row = c->k_row_stride;
  p.v_page = st(c->v_page_stride, c->num_pages);
  p.v_head = st(c->v_head_stride, c->kv_heads);
  p.v_row = c->v_row_stride;
  p.num_pages = c->num_pages;
  p.kv_heads = c->kv_heads;
  p.page_size = c->page_size;
  *out = p;
  return FA_OK;
}

fa_status check_decode(int B, int Hq, int Hkv, int Nq, int d, fa_dtype dt) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Nq < 1 || d < 1 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (dt != FA_F32 && dt != FA_BF16) return FA_ERR_INVALID_ARG;
  if (dt != FA_BF16 || (d != 64 && d != 128)) return FA_ERR_UNSUPPORTED;
  if ((long long)(Hq / Hkv) * Nq > kPagedMaxRows) return FA_ERR_UNSUPPORTED;
  if ((long long)B * Hkv > (1 << 24)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Strides of a [B, H, N, d] view (NULL: dense).
bool view_strides(const long long* s, int B, int H, int N, int d, long long* sb, long long* sh, long long* sr) {
  if (!s) {
    *sr = d;
    *sh = (long long)N * d;
    *sb = (long long)H * N * d;
    return true;
  }
  if (!stride_ok(s[0], B, d) || !stride_ok(s[1], H, d) || !stride_ok(s[2], N, d)) return false;
  *sb = B == 1 ? 0 : s[0];
  *sh = H == 1 ? 0 : s[1];
  *sr = N == 1 ? 0 : s[2];
  return true;
}

// Keys that a table of max_pages pages can hold.
int most_keys(int max_pages, int page_size) {
  const long long n = (long long)max_pages * page_size;
  return n < kPagedMaxKeys ? (int)n : kPagedMaxKeys;
}

// Layout and plan of a decode, functions of its sizes and the device alone. A
// decoding loop asks for the same ones again and again, and trying all numbers
// of key ranges costs the host 2 us: each thread keeps its last.
struct Schedule {
  int dev, B, Hkv, rows, prefix_len, d, most;
  bool narrow;
  PagedLayout layout;
  PrefixPlan plan;
};
const Schedule* schedule(int B, int Hkv, int rows, int prefix_len, int d, int most, bool narrow) {
  thread_local Schedule last = {-1, 0, 0, 0, 0, 0, 0, false, {}, {}};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  if (last.dev == dev && last.B == B && last.Hkv == Hkv && last.rows == rows && last.prefix_len == prefix_len &&
      last.d == d && last.most == most && last.narrow == narrow)
    return &last;
  last.dev = -1;
  last.layout = paged_layout(B, Hkv, rows, prefix_len, d);
  if (last.layout.ctas < 1) return nullptr;
  if (last.layout.pre_splits > 0)
    last.plan = plan_prefix_beside(B, rows, Hkv, prefix_len, d, last.layout.pre_splits, last.layout.ctas, fwd_slots(), most,
                                   narrow);
  last.B = B;
  last.Hkv = Hkv;
  last.rows = rows;
  last.prefix_len = prefix_len;
  last.d = d;
  last.most = most;
  last.narrow = narrow;
  last.dev = dev;
  return &last;
}

fa_status decode_impl(const void* Q, const long long* q_strides, const fa_paged_kv* cache,
                      const int* prefix_pages, int prefix_len, const int* block_tables, int max_pages,
                      const int* seq_lens, void* O, const long long* o_strides, float* LSE,
                      void* workspace, size_t workspace_bytes, int B, int Hq, int Nq, float scale,
                      fa_dtype dt, void* stream, int debug_skip = -1,
                      unsigned long long limit_ns = kDefaultWaitLimitNs) {
  PagedDecodeArgs a;
  std::memset(&a, 0, sizeof(a));
  fa_status s = check_pool(cache, dt, &a.pool);
  if (s != FA_OK) return s;
  s = check_decode(B, Hq, cache->kv_heads, Nq, cache->d, dt);
  if (s != FA_OK) return s;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (!Q || !O || !LSE || !block_tables || !seq_lens || !workspace || max_pages < 1) return FA_ERR_INVALID_ARG;
  if (prefix_len < 0 || prefix_len > kPagedMaxKeys || (prefix_len > 0 && !prefix_pages)) return FA_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(O, 16) || !aligned(LSE, 4) || !aligned(block_tables, 4) ||
      !aligned(seq_lens, 4) || !aligned(prefix_pages, 4) || !aligned(workspace, 256))
    return FA_ERR_INVALID_ARG;
  if (!view_strides(q_strides, B, Hq, Nq, cache->d, &a.q_b, &a.q_h, &a.q_r) ||
      !view_strides(o_strides, B, Hq, Nq, cache->d, &a.o_b, &a.o_h, &a.o_r))
    return FA_ERR_INVALID_ARG;
  const int most = most_keys(max_pages, cache->page_size);
  const Schedule* sched = schedule(B, cache->kv_heads, Hq / cache->kv_heads * Nq, prefix_len, cache->d, most,
                                   cache->page_size % 16 != 0);
  if (!sched) return FA_ERR_CUDA;
  const PagedLayout& L = sched->layout;
  if (workspace_bytes < L.total) return FA_ERR_INVALID_ARG;
  a.status = device_status_ptr();
  if (!a.status) return FA_ERR_CUDA;
  // boxes never cross a page's end, and a sequence's last one is loaded whole:
  // sequences that their table keeps short (up to 512 keys) get boxes of up to 16
  // rows (4 to 7% faster), others, which may be long, of up to 64 (3% faster than 16)
  const int most_shift = most <= 512 ? 4 : 6;
  while (a.box_shift < most_shift && cache->page_size % (2 << a.box_shift) == 0) ++a.box_shift;
  if (!encode_pool_bf16(&a.tmK, a.pool, false, cache->d, 1 << a.box_shift) ||
      !encode_pool_bf16(&a.tmV, a.pool, true, cache->d, 1 << a.box_shift))
    return FA_ERR_CUDA;
  char* ws = static_cast<char*>(workspace);
  a.ctas = L.ctas;
  a.page_div = fast_div((unsigned)cache->page_size);
  a.nq_div = fast_div((unsigned)Nq);
  a.rows_div = fast_div((unsigned)(Hq / cache->kv_heads * Nq));
  a.ctas_div = fast_div((unsigned)L.ctas);
  a.n_seq = L.n_seq;
  a.slot_rows = L.slot_rows;
  a.group_shift = L.group_shift;
  a.Opart = reinterpret_cast<float*>(ws);
  a.Lpart = reinterpret_cast<float*>(ws + L.lpart);
  a.unit_ctas = reinterpret_cast<int2*>(ws + L.unit_ctas);
  a.begun = reinterpret_cast<int2*>(ws + L.begun);
  a.Q = Q;
  a.O = O;
  a.LSE = LSE;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.prefix_pages = prefix_pages;
  a.prefix_len = prefix_len;
  a.B = B;
  a.G = Hq / cache->kv_heads;
  a.Nq = Nq;
  a.max_pages = max_pages;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.wait_limit_ns = limit_ns;
  a.debug_skip_tile = debug_skip;
  if (L.pre_splits > 0) {
    PrefixArgs p;
    std::memset(static_cast<void*>(&p), 0, sizeof(p));
    p.pool = a.pool;
    p.box_rows = cache->page_size & -cache->page_size;
    if (p.box_rows > 128) p.box_rows = 128;
    p.rows = B * a.G * Nq;
    const PrefixPlan& plan = sched->plan;
    const long long units = ((long long)p.rows + 255) / 256 * cache->kv_heads;
    p.Opart = reinterpret_cast<float*>(ws + L.pre_opart);
    p.Lpart = reinterpret_cast<float*>(ws + L.pre_lpart);
    if (!encode_pool_bf16(&p.tmK, a.pool, false, cache->d, p.box_rows) ||
        !encode_pool_bf16(&p.tmV, a.pool, true, cache->d, p.box_rows) ||
        !encode_part_f32(&p.tmOpart, p.Opart, units * plan.splits * 256, cache->d))
      return FA_ERR_CUDA;
    p.seq.H = cache->kv_heads;
    p.seq.N = prefix_len;
    p.seq.total = prefix_len;
    p.BH = cache->kv_heads;
    p.scale_log2 = a.scale_log2;
    p.status = a.status;
    p.wait_limit_ns = a.wait_limit_ns;
    p.n_tail = (int)units;
    p.splits = plan.splits;
    p.debug_skip_kv = debug_skip;
    p.Qrows = Q;
    p.q_b = a.q_b;
    p.q_h = a.q_h;
    p.q_r = a.q_r;
    p.prefix_pages = prefix_pages;
    p.G = a.G;
    p.Nq = Nq;
    if (launch_prefix_bf16(p, cache->d, static_cast<cudaStream_t>(stream)) != cudaSuccess) return FA_ERR_CUDA;
    a.pre_splits = plan.splits;
    a.early_ctas = plan.early_ctas;
    a.early_steps = plan.early_steps;
    a.early_div = fast_div((unsigned)(plan.early_ctas > 0 ? plan.early_ctas : 1));
    a.pre_Opart = p.Opart;
    a.pre_Lpart = p.Lpart;
  }
  return launch_decode_paged_bf16(a, cache->d, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                                  : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

fa_status fa_kv_append(const void* K, const void* V, long long k_stride, long long v_stride, const void* Q,
                       void* Qout, long long q_stride, long long qout_stride, int Hq,
                       const fa_paged_kv* cache, const int* block_tables, int max_pages,
                       const int* seq_lens, const int* cu_seqlens, int B, int total, const float* cos,
                       const float* sin, int rot_dim, int max_positions, const int* positions, int flags,
                       fa_dtype dt, void* stream) {
  AppendArgs a;
  std::memset(&a, 0, sizeof(a));
  const fa_status s = check_pool(cache, dt, &a.pool);
  if (s != FA_OK) return s;
  const int d = cache->d;
  if (flags & ~FA_ROPE_INTERLEAVED) return FA_ERR_INVALID_ARG;
  if (B < 1 || total < 1 || max_pages < 1 || Hq < 0 || (Q == nullptr) != (Hq == 0) ||
      (Qout == nullptr) != (Hq == 0))
    return FA_ERR_INVALID_ARG;
  if (!K || !V || !block_tables || !seq_lens || (!cu_seqlens && total % B != 0)) return FA_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > d) return FA_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (rot_dim > 0 && (!cos || !sin || max_positions < 1)) return FA_ERR_INVALID_ARG;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(Q, 16) || !aligned(Qout, 16) ||
      !aligned(cos, 16) || !aligned(sin, 16) || !aligned(block_tables, 4) || !aligned(seq_lens, 4) ||
      !aligned(cu_seqlens, 4) || !aligned(positions, 4))
    return FA_ERR_INVALID_ARG;
  const long long kv_row = (long long)cache->kv_heads * d, q_row = (long long)Hq * d;
  if (!stride_ok(k_stride, total, kv_row) || !stride_ok(v_stride, total, kv_row)) return FA_ERR_INVALID_ARG;
  if (Hq > 0 && (!stride_ok(q_stride, total, q_row) || !stride_ok(qout_stride, total, q_row)))
    return FA_ERR_INVALID_ARG;
  if (Q != nullptr && Q == Qout && total > 1 && q_stride != qout_stride) return FA_ERR_INVALID_ARG;
  a.status = device_status_ptr();
  if (!a.status) return FA_ERR_CUDA;
  a.K = K;
  a.V = V;
  a.Q = Q;
  a.Qout = Qout;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_stride = q_stride;
  a.qout_stride = qout_stride;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.cu_seqlens = cu_seqlens;
  a.cos = cos;
  a.sin = sin;
  a.positions = positions;
  a.B = B;
  a.Hq = Hq;
  a.total = total;
  a.max_pages = max_pages;
  a.rot_dim = rot_dim;
  a.max_positions = max_positions;
  a.interleaved = (flags & FA_ROPE_INTERLEAVED) != 0;
  return launch_append_bf16(a, d, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_decode_shared_workspace_bytes(int B, int Hq, int Hkv, int Nq, int prefix_len, int d, fa_dtype dt) {
  if (check_decode(B, Hq, Hkv, Nq, d, dt) != FA_OK || prefix_len < 0 || prefix_len > kPagedMaxKeys) return 0;
  return paged_layout(B, Hkv, Hq / Hkv * Nq, prefix_len, d).total;
}

size_t fa_decode_paged_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d, fa_dtype dt) {
  return fa_decode_shared_workspace_bytes(B, Hq, Hkv, Nq, 0, d, dt);
}

fa_status fa_decode_shared_plan(int B, int Hq, int Hkv, int Nq, int prefix_len, int d, int page_size, int max_pages,
                                int sms, int* key_ranges, int* prefix_ctas) {
  if (!key_ranges || !prefix_ctas || sms < 0 || sms > 65536 || page_size < 1 || max_pages < 1) return FA_ERR_INVALID_ARG;
  const fa_status s = check_decode(B, Hq, Hkv, Nq, d, FA_BF16);
  if (s != FA_OK) return s;
  if (prefix_len < 0 || prefix_len > kPagedMaxKeys) return FA_ERR_INVALID_ARG;
  if (page_size % 8 != 0 || page_size > kMaxPageSize) return FA_ERR_UNSUPPORTED;
  const PrefixPlan p = plan_shared(B, Hq / Hkv * Nq, Hkv, prefix_len, d, sms, most_keys(max_pages, page_size),
                                   page_size % 16 != 0);
  if (p.splits < 0) return FA_ERR_CUDA;
  *key_ranges = p.splits;
  *prefix_ctas = (int)(((long long)B * (Hq / Hkv) * Nq + 255) / 256 * Hkv * p.splits);
  return FA_OK;
}

fa_status fa_decode_paged(const void* Q, const long long* q_strides, const fa_paged_kv* cache,
                          const int* block_tables, int max_pages, const int* seq_lens, void* O,
                          const long long* o_strides, float* LSE, void* workspace, size_t workspace_bytes,
                          int B, int Hq, int Nq, float scale, fa_dtype dt, void* stream) {
  return decode_impl(Q, q_strides, cache, nullptr, 0, block_tables, max_pages, seq_lens, O, o_strides, LSE,
                     workspace, workspace_bytes, B, Hq, Nq, scale, dt, stream);
}

fa_status fa_decode_shared(const void* Q, const long long* q_strides, const fa_paged_kv* cache,
                           const int* prefix_pages, int prefix_len, const int* block_tables, int max_pages,
                           const int* seq_lens, void* O, const long long* o_strides, float* LSE,
                           void* workspace, size_t workspace_bytes, int B, int Hq, int Nq, float scale,
                           fa_dtype dt, void* stream) {
  return decode_impl(Q, q_strides, cache, prefix_pages, prefix_len, block_tables, max_pages, seq_lens, O,
                     o_strides, LSE, workspace, workspace_bytes, B, Hq, Nq, scale, dt, stream);
}

fa_status fa_debug_decode_skip_load(const void* Q, const long long* q_strides, const fa_paged_kv* cache,
                                    const int* prefix_pages, int prefix_len, const int* block_tables,
                                    int max_pages, const int* seq_lens, void* O, const long long* o_strides,
                                    float* LSE, void* workspace, size_t workspace_bytes, int B, int Hq, int Nq,
                                    float scale, int skip_tile, long long limit_ns, void* stream) {
  if (skip_tile < 1) return FA_ERR_INVALID_ARG;
  return decode_impl(Q, q_strides, cache, prefix_pages, prefix_len, block_tables, max_pages, seq_lens, O,
                     o_strides, LSE, workspace, workspace_bytes, B, Hq, Nq, scale, FA_BF16, stream, skip_tile,
                     clamp_limit(limit_ns));
}

}  // extern "C"

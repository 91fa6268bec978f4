// paged_append.cu -- new keys and values into a paged cache, the keys and the
// queries rotated by their position on the way.
//
// For each rotated pair (a, b) of a head at position p, with the angle of
// pair i given by its cosine and sine c, s:
//   a' = a c - b s,   b' = a s + b c            (fp32, rounded once to bf16)
// Everything else is a copy, so the operator is bound by memory: every q, k
// and v element is read once and written once, and a token's row of cosines
// and sines once.
//
// A warp works on one token, on a chunk of its heads (q, then k, then v heads)
// at a time. A lane owns two 16-byte vectors of a head: the two halves of eight
// rotated pairs, so that both partners of a pair meet in one lane's registers
// and the same cosines serve every head. The loads of the first chunk are
// issued before the chain of dependent look-ups (sequence and length, page)
// starts. Three shapes of the same work, in us for 256 / 1024 / 4096 / 32768
// tokens of 32 + 16 heads of 128 (a plain copy of the bytes takes 0.9 / 3.8 /
// 15.2 / 121):
//   a warp per pass over 4 heads              3.27 / 6.42 / 20.7 / 152
//   a warp per four passes                    3.30 / 5.08 / 18.4 / 128
//   a warp per token, two passes at a time    5.54 / 7.79 / 16.6 / 123
// The first spreads the few tokens of a decode step over the SMs (one token:
// 2.4 against 5.4 us), the last looks a token's place up once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;
constexpr int kFewWarps = 512;
constexpr int kManyTokens = 2048;
constexpr unsigned kFull = 0xffffffffu;

// Where packed token t belongs: the largest b with cu[b] <= t, the first packed
// token after its new ones and its length. A 32-way search; its final round,
// over at most 32 sequences, brings all three at once (one round trip to memory
// for up to 32 sequences, two for up to 1024). Where a sequence's offsets do not
// lie within the tokens, none of these is its own (kNone): a wrong end would
// move them over keys that are in the cache already.
struct Place {
  int b, last, len;  // b = -1: cu[0] > t
};
constexpr int kNone = -1;  // as `last`: before every token
__device__ __forceinline__ Place find_place(const AppendArgs& a, int t, int lane) {
  int lo = 0, hi = a.B;
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) >> 5;
    const int i = lo + step * lane;
    const unsigned m = __ballot_sync(kFull, i < hi && __ldg(a.cu_seqlens + i) <= t);
    if (m == 0) return Place{-1, 0, 0};
    lo += step * (31 - __clz(m));
    hi = min(lo + step, hi);
  }
  const int i = min(lo + lane, hi - 1);
  const int begin = __ldg(a.cu_seqlens + i), end = __ldg(a.cu_seqlens + i + 1), len = __ldg(a.seq_lens + i);
  const unsigned m = __ballot_sync(kFull, lo + lane < hi && begin <= t);
  if (m == 0) return Place{-1, 0, 0};
  const int src = 31 - __clz(m);
  const int last = begin >= 0 && end <= a.total ? end : kNone;
  return Place{lo + src, __shfl_sync(kFull, last, src), __shfl_sync(kFull, len, src)};
}

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Eight pairs (x element e, y element e); c, s: their cosines and sines.
__device__ __forceinline__ void rotate_halves(uint4& x, uint4& y, const float (&c)[8], const float (&s)[8]) {
  uint32_t* xw = &x.x;
  uint32_t* yw = &y.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a0 = bf_lo(xw[i]), a1 = bf_hi(xw[i]), b0 = bf_lo(yw[i]), b1 = bf_hi(yw[i]);
    xw[i] = pack_bf16x2(a0 * c[2 * i] - b0 * s[2 * i], a1 * c[2 * i + 1] - b1 * s[2 * i + 1]);
    yw[i] = pack_bf16x2(a0 * s[2 * i] + b0 * c[2 * i], a1 * s[2 * i + 1] + b1 * c[2 * i + 1]);
  }
}
// Eight neighbouring pairs: four in x, four in y.
__device__ __forceinline__ void rotate_neighbours(uint4& x, uint4& y, const float (&c)[8], const float (&s)[8]) {
  uint32_t* xw = &x.x;
  uint32_t* yw = &y.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a0 = bf_lo(xw[i]), b0 = bf_hi(xw[i]), a1 = bf_lo(yw[i]), b1 = bf_hi(yw[i]);
    xw[i] = pack_bf16x2(a0 * c[i] - b0 * s[i], a0 * s[i] + b0 * c[i]);
    yw[i] = pack_bf16x2(a1 * c[4 + i] - b1 * s[4 + i], a1 * s[4 + i] + b1 * c[4 + i]);
  }
}

template <int D, int PASSES, bool LOOP>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a, int chunks, int per_token) {
  constexpr int U = D / 16;    // lanes of a head
  constexpr int HPP = 32 / U;  // heads of a pass
  // a decode behind this kernel may be set up meanwhile; it waits for the end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long gw = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const long long warps = (long long)gridDim.x * (kThreads / 32);
  // every pair of offsets is looked at by some warp, whatever the tokens meet
  if (a.cu_seqlens != nullptr) {
    for (long long b = gw * 32 + lane; b < a.B; b += warps * 32) {
      const int c0 = __ldg(a.cu_seqlens + b), c1 = __ldg(a.cu_seqlens + b + 1);
      if (c0 < 0 || c1 < c0 || c1 > a.total) report_status(a.status, kStatusBadSeqlens);
    }
  }
  // per_token warps share a token's chunks of heads
  if (gw >= (long long)a.total * per_token) return;
  const int t = (int)(gw / per_token);
  int chunk = (int)(gw - (long long)t * per_token);
  const int u = lane % U, hl = lane / U;
  const int Hkv = a.pool.kv_heads, heads = a.Hq + 2 * Hkv;
  const int rot = a.rot_dim;
  const bool rotated = 16 * u < rot;
  // this lane's two vectors: element offsets within a head
  int e0, e1;
  if (a.interleaved || !rotated) {
    e0 = 16 * u;
    e1 = e0 + 8;
  } else {
    e0 = 8 * u;
    e1 = (rot >> 1) + 8 * u;
  }
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.Q);
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.K);
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.V);
  uint4 x[PASSES], y[PASSES];
  auto load = [&]() {
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int h = (chunk * PASSES + p) * HPP + hl;
      x[p] = y[p] = make_uint4(0u, 0u, 0u, 0u);
      if (h < heads) {
        const __nv_bfloat16* src = h < a.Hq         ? q + t * a.q_stride + (long long)h * D
                                   : h < a.Hq + Hkv ? k + t * a.k_stride + (long long)(h - a.Hq) * D
                                                    : v + t * a.v_stride + (long long)(h - a.Hq - Hkv) * D;
        x[p] = *reinterpret_cast<const uint4*>(src + e0);
        y[p] = *reinterpret_cast<const uint4*>(src + e1);
      }
    }
  };
  load();
  // where the token goes
  int b, last, len;  // its sequence, the first packed token after that, the length
  if (a.cu_seqlens == nullptr) {
    const int n = a.total / a.B;
    b = t / n;
    last = (b + 1) * n;
    len = __ldg(a.seq_lens + b);
  } else {
    const Place p = find_place(a, t, lane);
    b = p.b;
    last = p.last;
    len = p.len;
    if (b < 0) return;      // before the first sequence: padding
    if (t >= last) return;  // behind the last sequence: padding; or its offsets are wrong, as reported above
  }
  if (len == 0) return;  // a padding sequence
  const long long pos = (long long)len - last + t;
  const int ps = a.pool.page_size;
  bool ok = pos >= 0 && pos < (long long)a.max_pages * ps;
  long long p_rot = pos;
  if (ok && rot > 0) {
    if (a.positions != nullptr) p_rot = __ldg(a.positions + t);
    ok = p_rot >= 0 && p_rot < a.max_positions;
  }
  int page = -1, row = 0;
  if (ok) {
    const int pi = (int)(pos / ps);
    row = (int)(pos - (long long)pi * ps);
    page = __ldg(a.block_tables + (long long)b * a.max_pages + pi);
    ok = page >= 0 && page < a.pool.num_pages;
  }
  if (!ok) {
    if (lane == 0) report_status(a.status, kStatusBadSeqlens);
    return;
  }
  float c[8], s[8];
  if (rotated) {
    const float4* cp = reinterpret_cast<const float4*>(a.cos + p_rot * (rot >> 1) + 8 * u);
    const float4* sp = reinterpret_cast<const float4*>(a.sin + p_rot * (rot >> 1) + 8 * u);
    const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
    c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w;
    c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
    s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w;
    s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
  }
  __nv_bfloat16* kd = static_cast<__nv_bfloat16*>(a.pool.k) + (long long)page * a.pool.k_page + (long long)row * a.pool.k_row;
  __nv_bfloat16* vd = static_cast<__nv_bfloat16*>(a.pool.v) + (long long)page * a.pool.v_page + (long long)row * a.pool.v_row;
  __nv_bfloat16* qd = static_cast<__nv_bfloat16*>(a.Qout) + t * a.qout_stride;
  do {
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int h = (chunk * PASSES + p) * HPP + hl;
      if (h >= heads) continue;
      if (rotated && h < a.Hq + Hkv) {
        if (a.interleaved) rotate_neighbours(x[p], y[p], c, s);
        else rotate_halves(x[p], y[p], c, s);
      }
      __nv_bfloat16* dst = h < a.Hq         ? qd + (long long)h * D
                           : h < a.Hq + Hkv ? kd + (h - a.Hq) * a.pool.k_head
                                            : vd + (h - a.Hq - Hkv) * a.pool.v_head;
      *reinterpret_cast<uint4*>(dst + e0) = x[p];
      *reinterpret_cast<uint4*>(dst + e1) = y[p];
    }
    chunk += per_token;
    if (LOOP && chunk < chunks) load();
  } while (LOOP && chunk < chunks);
}

template <int D, int PASSES, bool LOOP>
cudaError_t launch_passes(const AppendArgs& a, cudaStream_t st) {
  constexpr int HPP = 32 / (D / 16);
  const int heads = a.Hq + 2 * a.pool.kv_heads;
  const int chunks = (heads + HPP * PASSES - 1) / (HPP * PASSES), per_token = LOOP ? 1 : chunks;
  const long long warps = (long long)a.total * per_token;
  const long long blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  append_kernel<D, PASSES, LOOP><<<(unsigned)blocks, kThreads, 0, st>>>(a, chunks, per_token);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const AppendArgs& a, cudaStream_t st) {
  constexpr int HPP = 32 / (D / 16);
  const int heads = a.Hq + 2 * a.pool.kv_heads;
  const long long warps4 = (long long)a.total * ((heads + 4 * HPP - 1) / (4 * HPP));
  if (a.total >= kManyTokens) return launch_passes<D, 2, true>(a, st);
  return warps4 < kFewWarps ? launch_passes<D, 1, false>(a, st) : launch_passes<D, 4, false>(a, st);
}

}  // namespace

cudaError_t launch_append_bf16(const AppendArgs& a, int d, cudaStream_t st) {
  if (d == 128) return launch_d<128>(a, st);
  if (d == 64) return launch_d<64>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace fa

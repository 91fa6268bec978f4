// paged_weights.cu -- the attention weight that each cached key got from the
// newest tokens of its sequence (a decoding step).
//
//   w_bhj (+)= sum over the query heads of K/V head h and the new tokens i that
//              see key j of exp(scale * q_i . k_j - LSE_i),
// after the step's attention, whose log-sum-exp it takes.
//
// Bound by the keys, which are read once (the values are not): 4 bytes of
// weights go with 256 bytes of a key. A warp takes 32 keys at a time: 16-byte
// loads straight into the fragments of 16 x 8 x 16 warp-level products, keys on
// the rows and query rows on the columns, 8 KB in flight per warp and 16 warps
// to an SM. The order of the elements in a product's depth is free, so a
// thread's two fragments of two depth steps are 16 neighbouring bytes of a key
// row, in the queries' fragments alike. No shared memory, no barrier.
//
// The tiles of 32 keys of all sequences and heads are laid end to end and cut
// into equal shares, one per CTA, on the device; a share's tiles go round its
// warps. Each weight is one thread's sum over the columns and two shuffles, in a
// fixed order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 8;
constexpr int kTile = 32;  // keys of a warp's tile

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Tiles per K/V head of a sequence of `len` keys; 0 for one that is out of range.
__device__ __forceinline__ int seq_tiles(const PagedWeightArgs& a, int b, int& len) {
  len = __ldg(a.seq_lens + b);
  return len > 0 && len <= a.most_keys && len <= a.w_keys ? (len + kTile - 1) / kTile : 0;
}

// NT: 8-column tiles of query rows (G * Nq <= 8 NT).
template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT <= 2 ? 2 : 1) paged_weights_kernel(const __grid_constant__ PagedWeightArgs a) {
  constexpr int S = D / 32;  // 16-byte pieces per thread and key row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r8 = lane >> 2, q4 = lane & 3;
  // Tiles of all sequences, by all lanes; then the sequence in which this CTA's
  // share begins.
  long long total = 0;
  bool bad = false;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    int len = 0, t = 0;
    if (b0 + lane < a.B) {
      t = seq_tiles(a, b0 + lane, len);
      bad = bad || (t == 0 && len != 0);
    }
    total += __reduce_add_sync(0xffffffffu, t);
  }
  if (blockIdx.x == 0 && warp == 0 && bad) report_status(a.status, kStatusBadSeqlens);
  total *= a.Hkv;
  const long long end = total * (blockIdx.x + 1) / gridDim.x;
  long long at = total * blockIdx.x / gridDim.x + warp;  // this warp's tile
  if (at >= end) return;
  int b = 0, len = 0, tiles = 0;
  long long first = 0;  // first tile of sequence b
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    int l = 0;
    const int t = b0 + lane < a.B ? seq_tiles(a, b0 + lane, l) : 0;
    const int n = __reduce_add_sync(0xffffffffu, t);
    if (first + (long long)n * a.Hkv > at) {
      int sum = t;  // inclusive scan of the 32 sequences' tiles
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      const unsigned over = __ballot_sync(0xffffffffu, first + (long long)sum * a.Hkv > at);
      const int src = __ffs(over) - 1;
      b = b0 + src;
      len = __shfl_sync(0xffffffffu, l, src);
      tiles = __shfl_sync(0xffffffffu, t, src);
      first += (long long)(__shfl_sync(0xffffffffu, sum, src) - tiles) * a.Hkv;
      break;
    }
    first += (long long)n * a.Hkv;
  }

  int head = -1, old_b = -1;
  const int R = a.G * a.Nq;
  uint4 qf[NT <= 2 ? NT : 1][S];  // the queries' fragments (more tiles: loaded as they are used)
  float nl[2 * NT];               // -LSE * log2(e) of this thread's columns
  int limit[2 * NT];              // keys that they see; 0 past the last row
  const __nv_bfloat16* qp[NT];
  for (; at < end; at += kWarps) {
    while (at >= first + (long long)tiles * a.Hkv) {
      first += (long long)tiles * a.Hkv;
      do {
        ++b;
        tiles = seq_tiles(a, b, len);
      } while (tiles == 0);  // a sequence with tiles follows: at < end <= total
    }
    const int local = (int)(at - first), h = local / tiles, key0 = (local - h * tiles) * kTile;
    if (h != head || b != old_b) {
      head = h;
      old_b = b;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // row of the queries on this thread's column of the fragments
        const int r = 8 * n + r8, rr = r < R ? r : R - 1, g = a.nq_div(rr);
        qp[n] = static_cast<const __nv_bfloat16*>(a.Q) + b * a.q_b + (long long)(h * a.G + g) * a.q_h + (long long)(rr - g * a.Nq) * a.q_r + 8 * q4;
        if constexpr (NT <= 2) {
#pragma unroll
          for (int s = 0; s < S; ++s) qf[n][s] = __ldg(reinterpret_cast<const uint4*>(qp[n] + 32 * s));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = 8 * n + 2 * q4 + e;
          nl[2 * n + e] = -INFINITY;
          limit[2 * n + e] = 0;
          if (c < R) {
            const int gc = a.nq_div(c), i = c - gc * a.Nq;
            const float x = __ldg(a.LSE + ((long long)b * a.Hkv * a.G + h * a.G + gc) * a.Nq + i);
            nl[2 * n + e] = x == -INFINITY ? x : -x * 1.4426950408889634f;
            limit[2 * n + e] = len - a.Nq + 1 + i;
          }
        }
      }
    }
    // 32 keys: rows r8 + 8 i of the tile, 16 bytes at 8 q4 + 32 s of each
    uint4 kf[4][S];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = key0 + 8 * i;  // 8 keys lie in one page
      int page = 0, row = 0;
      bool there = key < len;
      if (there) {
        const int pi = a.page_div(key);
        row = key - pi * a.pool.page_size;
        page = __ldg(a.block_tables + (long long)b * a.max_pages + pi);
        if (page < 0 || page >= a.pool.num_pages) {
          if (lane == 0) report_status(a.status, kStatusBadSeqlens);
          there = false;
        }
      }
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.pool.k) + page * a.pool.k_page + h * a.pool.k_head +
                               (long long)(row + r8) * a.pool.k_row + 8 * q4;
#pragma unroll
      for (int s = 0; s < S; ++s)
        kf[i][s] = there ? __ldg(reinterpret_cast<const uint4*>(p + 32 * s)) : make_uint4(0u, 0u, 0u, 0u);
    }
    // weights of keys r8 and r8 + 8 of each half, over this thread's columns
    float lo[2] = {0.f, 0.f}, hi[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (NT > 2 && 8 * n >= R) break;
      float c[2][4] = {};
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const uint4 q = NT <= 2 ? qf[NT <= 2 ? n : 0][s] : __ldg(reinterpret_cast<const uint4*>(qp[n] + 32 * s));
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint4 x = kf[2 * m][s], y = kf[2 * m + 1][s];
          mma_16816(c[m], x.x, y.x, x.y, y.y, q.x, q.y);
          mma_16816(c[m], x.z, y.z, x.w, y.w, q.z, q.w);
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int j = key0 + 16 * m + r8;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int lim = limit[2 * n + e];
          const float p0 = ex2_approx(fmaf(c[m][e], a.scale_log2, nl[2 * n + e]));
          const float p1 = ex2_approx(fmaf(c[m][2 + e], a.scale_log2, nl[2 * n + e]));
          lo[m] += j < lim ? p0 : 0.f;
          hi[m] += j + 8 < lim ? p1 : 0.f;
        }
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        lo[m] += __shfl_xor_sync(0xffffffffu, lo[m], o);
        hi[m] += __shfl_xor_sync(0xffffffffu, hi[m], o);
      }
      const int j = key0 + 16 * m + r8 + 8 * q4;  // lanes q4 = 0 and 1 store
      if (q4 < 2 && j < len) {
        float* w = a.W + (long long)b * a.w_batch + (long long)h * a.w_head + j;
        const float x = q4 == 0 ? lo[m] : hi[m];
        *w = a.accumulate && j < len - a.Nq ? *w + x : x;  // new keys have no weight yet
      }
    }
  }
}

template <int D>
cudaError_t launch_d(const PagedWeightArgs& a, cudaStream_t st) {
  const int rows = a.G * a.Nq;
  if (a.ctas < 1) return cudaErrorInvalidValue;
  if (rows <= 8) paged_weights_kernel<D, 1><<<a.ctas, kWarps * 32, 0, st>>>(a);
  else if (rows <= 16) paged_weights_kernel<D, 2><<<a.ctas, kWarps * 32, 0, st>>>(a);
  else if (rows <= 64) paged_weights_kernel<D, 8><<<a.ctas, kWarps * 32, 0, st>>>(a);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_weights(const PagedWeightArgs& a, int d, cudaStream_t st) {
  if (d == 128) return launch_d<128>(a, st);
  if (d == 64) return launch_d<64>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace fa

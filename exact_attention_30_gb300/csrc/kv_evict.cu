// kv_evict.cu -- eviction from a paged cache by weight: of each sequence and K/V
// head the `recent` newest keys stay, and of the others those with the largest
// weights (ties: the older key), `budget` in all. What stays keeps its order and
// moves together: key i of those that stay to row i mod page_size of page
// new_tables[b][i / page_size].
//
// 1. evict_select_kernel, one CTA per (sequence, head): the weight of the last
//    key that stays by a radix selection over 11, 11 and 10 bits of the weights'
//    order (a histogram in shared memory, its suffix sums, the digit that holds
//    the rank), then one pass over the weights in order that counts and lists.
//    Bound by its passes over the weights (4 bytes a key and pass, from L2) and
//    by latency: a few barriers per pass.
// 2. evict_move_kernel copies the rows. Bound by memory: each row that stays is
//    read and written once; in place, rows that do not move are left alone. In
//    place a row may only be written when the row it held has been read: since
//    those that stay keep their order, row i's new content comes from a row >= i,
//    so a CTA that goes through the rows in order, reading a batch before it
//    writes it, never loses one. Rows of one head cannot be shared out among
//    CTAs, therefore, but their columns can: keys and values, and pieces of 32 to
//    128 bytes of a row, are CTAs of their own.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kBins = 2048;
constexpr int kPerThread = 4;  // neighbouring weights of a thread in the listing pass

// Weights as unsigned numbers in the same order: NaN above all, -0 equal to 0.
__device__ __forceinline__ unsigned order_of(float w) {
  if (w != w) return 0xffffffffu;
  const unsigned x = __float_as_uint(w + 0.f);
  return x & 0x80000000u ? ~x : x | 0x80000000u;
}

// Exclusive sum over the block's threads of `x`, and the total. `part`: 32 ints.
__device__ __forceinline__ int block_scan(int x, int* part, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int sum = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  if (lane == 31) part[warp] = sum;
  __syncthreads();
  int p = part[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, p, o);
    if (lane >= o) p += y;
  }
  total = __shfl_sync(0xffffffffu, p, 31);
  const int before = warp > 0 ? __shfl_sync(0xffffffffu, p, warp - 1) : 0;
  __syncthreads();
  return before + sum - x;
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int hist[kBins];
  __shared__ int part[32];
  __shared__ int found_bin, found_above;
  const int h = blockIdx.x, b = blockIdx.y, t = threadIdx.x;
  int len = a.seq_lens[b];
  if (len < 0 || len > a.most_keys || len > a.w_keys) {
    if (h == 0 && t == 0) report_status(a.status, kStatusBadSeqlens);
    len = 0;  // nothing stays and nothing moves
  }
  const float* w = a.W + (long long)b * a.w_batch + (long long)h * a.w_head;
  float* out_w = a.Wout + (long long)b * a.wout_batch + (long long)h * a.wout_head;
  int* kept = a.kept + ((long long)b * a.Hkv + h) * a.budget;
  const int count = min(len, a.budget), recent = min(a.recent, len);
  const int old = len - recent;   // keys that the weights decide on
  const int need = count - recent;  // how many of them stay
  for (int i = count + t; i < a.budget; i += kSelectThreads) kept[i] = -1;

  unsigned least = 0;   // order of the last weight that stays
  int ties = 0;         // how many of that order stay
  if (need < old && need > 0) {
    unsigned prefix = 0, mask = 0;
    int rank = need;  // rank, from the top, of the last one that stays among those that match the prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const unsigned digits = pass == 2 ? 1023u : 2047u;
      for (int i = t; i < kBins; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int j = t; j < old; j += kSelectThreads) {
        const unsigned x = order_of(w[j]);
        if ((x & mask) == prefix) atomicAdd(&hist[(x >> shift) & digits], 1);
      }
      __syncthreads();
      // bins from the top: thread t has bins 2047 - 2 t and 2046 - 2 t
      const int x0 = hist[kBins - 1 - 2 * t], x1 = hist[kBins - 2 - 2 * t];
      int total;
      const int above = block_scan(x0 + x1, part, total);
      if (above < rank && rank <= above + x0) {
        found_bin = kBins - 1 - 2 * t;
        found_above = above;
      } else if (above + x0 < rank && rank <= above + x0 + x1) {
        found_bin = kBins - 2 - 2 * t;
        found_above = above + x0;
      }
      __syncthreads();
      prefix |= (unsigned)found_bin << shift;
      mask |= digits << shift;
      rank -= found_above;
      __syncthreads();
    }
    least = prefix;
    ties = rank;
  }
  // The list, in order. Before key j stay the larger weights before it and at
  // most `ties` of those equal to the last.
  const bool all = need >= old;
  int larger = 0, equal = 0;  // before this chunk
  if (need > 0) {
#pragma unroll 1
    for (int j0 = 0; j0 < old; j0 += kSelectThreads * kPerThread) {
      const int j = j0 + t * kPerThread;
      float x[kPerThread];
      int mine = 0;  // larger ones in the low half, equal ones in the high half
      unsigned gt = 0, eq = 0;
#pragma unroll
      for (int e = 0; e < kPerThread; ++e) {
        x[e] = 0.f;
        if (j + e < old) {
          x[e] = w[j + e];
          const unsigned u = order_of(x[e]);
          if (all || u > least) gt |= 1u << e;
          else if (u == least) eq |= 1u << e;
        }
      }
      mine = __popc(gt) | __popc(eq) << 16;
      int total;
      const int before = block_scan(mine, part, total);  // also: the chunk is read before it is written
      int ng = larger + (before & 0xffff), ne = equal + (before >> 16);
#pragma unroll
      for (int e = 0; e < kPerThread; ++e) {
        const bool is_eq = eq >> e & 1u;
        if ((gt >> e & 1u) || (is_eq && ne < ties)) {
          const int pos = ng + min(ne, ties);
          kept[pos] = j + e;
          out_w[pos] = x[e];
        }
        ng += gt >> e & 1u;
        ne += is_eq;
      }
      larger += total & 0xffff;
      equal += total >> 16;
      __syncthreads();
    }
  }
  // the newest ones
#pragma unroll 1
  for (int j0 = 0; j0 < recent; j0 += kSelectThreads) {
    const int j = j0 + t;
    const float x = j < recent ? w[old + j] : 0.f;
    __syncthreads();
    if (j < recent) {
      kept[need + j] = old + j;
      out_w[need + j] = x;
    }
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveLoads = 8;  // 16-byte loads of a thread in flight

// CTA (piece, head, sequence); pieces: keys, then values, a.pieces columns each.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  const int h = blockIdx.y, b = blockIdx.z, t = threadIdx.x;
  const bool values = (int)blockIdx.x >= a.pieces;
  const int piece = (int)blockIdx.x - (values ? a.pieces : 0);
  if (blockIdx.x == 0 && h == 0 && t == 0) {
    const int len = a.seq_lens[b];
    a.new_lens[b] = len < 0 || len > a.most_keys || len > a.w_keys ? len : min(len, a.budget);
  }
  const int* kept = a.kept + ((long long)b * a.Hkv + h) * a.budget;
  const int* from = a.block_tables + (long long)b * a.max_pages;
  const int* to = a.new_tables + (long long)b * a.new_pages;
  __nv_bfloat16* pool = static_cast<__nv_bfloat16*>(values ? a.pool.v : a.pool.k);
  const long long s_page = values ? a.pool.v_page : a.pool.k_page, s_head = values ? a.pool.v_head : a.pool.k_head,
                  s_row = values ? a.pool.v_row : a.pool.k_row;
  pool += h * s_head + piece * (a.d / a.pieces);
  const int units = a.d / a.pieces / 8;       // 16-byte units of a row here (a power of two)
  const int rows = kMoveThreads / units;      // rows of one load of the block
  const int u = t & (units - 1), r = t / units;
  for (int i0 = 0; i0 < a.budget; i0 += rows * kMoveLoads) {
    uint4 x[kMoveLoads];
    __nv_bfloat16* dst[kMoveLoads];
    int src[kMoveLoads];
    bool more = false;
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e) {
      const int i = i0 + e * rows + r;
      src[e] = i < a.budget ? __ldg(kept + i) : -1;
      more = more || src[e] >= 0;
    }
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e) {
      dst[e] = nullptr;
      if (src[e] < 0) continue;
      const int i = i0 + e * rows + r;
      const int pf = a.page_div(src[e]), pt = a.page_div(i);
      const int page_f = __ldg(from + pf), page_t = __ldg(to + pt);
      if (page_f < 0 || page_f >= a.pool.num_pages || page_t < 0 || page_t >= a.pool.num_pages) {
        report_status(a.status, kStatusBadSeqlens);
        continue;
      }
      const int row_f = src[e] - pf * a.pool.page_size, row_t = i - pt * a.pool.page_size;
      if (page_f == page_t && row_f == row_t) continue;  // it stays where it is
      dst[e] = pool + page_t * s_page + row_t * s_row + 8 * u;
      x[e] = *reinterpret_cast<const uint4*>(pool + page_f * s_page + row_f * s_row + 8 * u);
    }
    // the batch has been read before any of it is written (and all threads
    // leave together, behind the last key that stays)
    if (!__syncthreads_or(more)) break;
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e)
      if (dst[e] != nullptr) *reinterpret_cast<uint4*>(dst[e]) = x[e];
  }
}

}  // namespace

int evict_pieces(int B, int Hkv, int d, int sms) {
  // pieces of at least 32 bytes (a sector) of a row, as many as give every SM
  // eight blocks to run at once
  int pieces = 1;
  while (pieces * 32 < d * 2 && (long long)B * Hkv * 2 * pieces < 8ll * sms) pieces *= 2;
  return pieces;
}

cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t st) {
  evict_select_kernel<<<dim3((unsigned)a.Hkv, (unsigned)a.B), kSelectThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  evict_move_kernel<<<dim3((unsigned)(2 * a.pieces), (unsigned)a.Hkv, (unsigned)a.B), kMoveThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace fa

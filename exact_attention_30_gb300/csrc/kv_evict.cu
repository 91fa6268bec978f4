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
//    What fits is held in shared memory, weights and list, and read and written
//    once. Bound by latency (some 20 barriers) and the histogram's atomics.
// 2. evict_move_kernel copies the rows. Bound by memory: each row that stays is
//    read and written once; in place, rows that do not move are left alone. In
//    place a row may only be written when the row it held has been read: since
//    those that stay keep their order, row i's new content comes from a row >= i,
//    so a CTA that goes through the rows in order, reading a batch before it
//    writes it, never loses one. Rows of one head cannot be shared out among
//    CTAs, therefore, but their columns can: keys and values, and pieces of 64 or
//    128 bytes of a row, are CTAs of their own. Into other pages, rows are shared
//    out instead, and whole (a warp's load of 32-byte pieces touches 16 lines:
//    8 x 8 x 2048 rows of 256 bytes took 41 us so). The next batch's indices and
//    pages are looked up while this one's rows are on their way.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kBins = 2048;
constexpr size_t kSelectMostBytes = 208 * 1024;  // of weights and list (counts in 16 bits: at most 53248 keys)
constexpr int kPerThread = 4;  // neighbouring weights of a thread in the listing pass

// Weights as unsigned numbers in the same order (NaN above all, -0 equal to 0),
// and back.
__device__ __forceinline__ unsigned order_of(float w) {
  if (w != w) return 0xffffffffu;
  const unsigned x = __float_as_uint(w + 0.f);
  return x & 0x80000000u ? ~x : x | 0x80000000u;
}

__device__ __forceinline__ float weight_of(unsigned u) { return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u); }

// Exclusive sum over the block's threads of `x`, and the total. `part`: 32 ints.
template <int THREADS>
__device__ __forceinline__ int block_scan(int value, int* part, int& total) {
  constexpr int WARPS = THREADS / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned x = (unsigned)value;  // two counts in one word may pass 31 bits in the total
  unsigned sum = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  if (lane == 31) part[warp] = (int)sum;
  __syncthreads();
  unsigned p = lane < WARPS ? (unsigned)part[lane] : 0u;
#pragma unroll
  for (int o = 1; o < WARPS; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, p, o);
    if (lane >= o) p += y;
  }
  total = (int)__shfl_sync(0xffffffffu, p, WARPS - 1);
  const unsigned before = warp > 0 ? __shfl_sync(0xffffffffu, p, warp - 1) : 0u;
  __syncthreads();
  return (int)(before + sum - x);
}

// Bin i of the histogram, one word in 33 left out: a thread's eight neighbouring
// bins then fall on banks of their own.
__device__ __forceinline__ int bin_at(int i) { return i + (i >> 5); }

// HELD: the weights' orders are put into (dynamic) shared memory first and read
// there; else they are found from memory in each pass.
template <int THREADS, bool HELD>
__global__ void __launch_bounds__(THREADS) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int BPT = kBins / THREADS;  // bins of a thread
  extern __shared__ __align__(16) unsigned held[];
  __shared__ int hist[kBins + kBins / 32];
  __shared__ int part[32];
  __shared__ int found_bin, found_above;
  const int h = blockIdx.x, b = blockIdx.y, t = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the move's CTAs may come; they wait for this grid
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
  for (int i = count + t; i < a.budget; i += THREADS) kept[i] = -1;
  for (int i = t; i < kBins + kBins / 32; i += THREADS) hist[i] = 0;
  if constexpr (HELD) {
    const int whole = (reinterpret_cast<uintptr_t>(w) & 15) == 0 ? len / 4 : 0;
#pragma unroll 4
    for (int j = t; j < whole; j += THREADS) {
      const float4 y = reinterpret_cast<const float4*>(w)[j];
      reinterpret_cast<uint4*>(held)[j] = make_uint4(order_of(y.x), order_of(y.y), order_of(y.z), order_of(y.w));
    }
    // (rows that do not begin on 16 bytes, every second or third of an odd width)
#pragma unroll 8
    for (int j = 4 * whole + t; j < len; j += THREADS) held[j] = order_of(w[j]);
  }
  __syncthreads();

  unsigned least = 0;   // order of the last weight that stays
  int ties = 0;         // how many of that order stay
  if (need < old && need > 0) {
    unsigned prefix = 0, mask = 0;
    int rank = need;  // rank, from the top, of the last one that stays among those that match the prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const unsigned digits = pass == 2 ? 1023u : 2047u;
      auto count_one = [&](unsigned u) {
        if ((u & mask) == prefix) atomicAdd(&hist[bin_at((u >> shift) & digits)], 1);
      };
      if constexpr (HELD) {
#pragma unroll 2
        for (int j = 4 * t; j < old; j += 4 * THREADS) {
          const uint4 u = *reinterpret_cast<const uint4*>(held + j);
          count_one(u.x);
          if (j + 1 < old) count_one(u.y);
          if (j + 2 < old) count_one(u.z);
          if (j + 3 < old) count_one(u.w);
        }
      } else {
#pragma unroll 4
        for (int j = t; j < old; j += THREADS) count_one(order_of(w[j]));
      }
      __syncthreads();
      // bins from the top: thread t has the BPT bins below kBins - t BPT, and
      // clears them for the next pass
      int n[BPT], mine = 0, total;
#pragma unroll
      for (int e = 0; e < BPT; ++e) {
        int* bin = &hist[bin_at(kBins - 1 - t * BPT - e)];
        mine += n[e] = *bin;
        *bin = 0;
      }
      int above = block_scan<THREADS>(mine, part, total);
      if (above < rank && rank <= above + mine) {
#pragma unroll
        for (int e = 0; e < BPT; ++e) {
          if (above < rank && rank <= above + n[e]) {
            found_bin = kBins - 1 - t * BPT - e;
            found_above = above;
          }
          above += n[e];
        }
      }
      __syncthreads();
      prefix |= (unsigned)found_bin << shift;
      mask |= digits << shift;
      rank -= found_above;
    }
    least = prefix;
    ties = rank;
  }
  // The list, in order. Before key j stay the larger weights before it and at
  // most `ties` of those equal to the last.
  const bool all = need >= old;
  if constexpr (HELD) {
    // A run of keys to each warp: counted, then listed 32 at a time behind what
    // the warps before it list. Larger ones are counted in the low half of a word,
    // equal ones in the high half. (Four neighbouring keys to a lane, counts summed
    // over the lanes: 12800 cycles for the list of 32499 weights, 8900 by ballots.)
    __shared__ unsigned counts[32];
    constexpr int WARPS = THREADS / 32;
    const int warp = t >> 5, lane = t & 31;
    int* list = reinterpret_cast<int*>(held + a.held_words);
    const int run = ((old + WARPS - 1) / WARPS + 31) & ~31;
    const int first = warp * run, last = need > 0 ? min(old, first + run) : 0;
    unsigned n = 0;
#pragma unroll 4
    for (int j = first + lane; j < last; j += 32) {
      const unsigned u = held[j];
      n += (all || u > least ? 1u : 0u) + (u == least ? 0x10000u : 0u);  // (none equal where all stay: least is 0, no weight's)
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) counts[warp] = n;
    __syncthreads();
    n = __reduce_add_sync(0xffffffffu, lane < warp ? counts[lane] : 0u);
    int ng = (int)(n & 0xffffu), ne = (int)(n >> 16);
    const unsigned before = (1u << lane) - 1u;
#pragma unroll 4
    for (int j0 = first; j0 < last; j0 += 32) {
      const int j = j0 + lane;
      const unsigned u = j < last ? held[j] : 0u;
      const bool gt = j < last && (all || u > least), eq = j < last && u == least;
      const unsigned mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
      if (me == 0u) {  // nearly always; counting a mask's bits takes a warp eight cycles
        if (gt) list[ng + __popc(mg & before) + min(ne, ties)] = j;
      } else {
        const int e = ne + __popc(me & before);
        if (gt || (eq && e < ties)) list[ng + __popc(mg & before) + min(e, ties)] = j;
        ne += __popc(me);
      }
      ng += __popc(mg);
    }
    // and out in order, the newest ones behind (stored as they were found, a few
    // lanes of a warp at a time, the lists of 2048 out of 30000 took 6 us)
    __syncthreads();
    for (int i = t; i < count; i += THREADS) {
      const int j = i < need ? list[i] : old + i - need;
      kept[i] = j;
      out_w[i] = weight_of(held[j]);
    }
  } else {
    int larger = 0, equal = 0;  // before this chunk
    if (need > 0) {
#pragma unroll 1
      for (int j0 = 0; j0 < old; j0 += THREADS * kPerThread) {
        const int j = j0 + t * kPerThread;
        float y[kPerThread];
        unsigned gt = 0, eq = 0;
#pragma unroll
        for (int e = 0; e < kPerThread; ++e) {
          y[e] = 0.f;
          if (j + e < old) {
            y[e] = w[j + e];
            const unsigned u = order_of(y[e]);
            if (all || u > least) gt |= 1u << e;
            else if (u == least) eq |= 1u << e;
          }
        }
        // larger ones in the low half, equal ones in the high half
        int total;
        const int before = block_scan<THREADS>(__popc(gt) | __popc(eq) << 16, part, total);  // also: the chunk is read before it is written
        int ng = larger + (before & 0xffff), ne = equal + (before >> 16);
#pragma unroll
        for (int e = 0; e < kPerThread; ++e) {
          const bool is_eq = eq >> e & 1u;
          if ((gt >> e & 1u) || (is_eq && ne < ties)) {
            const int pos = ng + min(ne, ties);
            kept[pos] = j + e;
            out_w[pos] = y[e];
          }
          ng += gt >> e & 1u;
          ne += is_eq;
        }
        larger += total & 0xffff;
        equal += total >> 16;
      }
    }
    // the newest ones
#pragma unroll 1
    for (int j0 = 0; j0 < recent; j0 += THREADS) {
      const int j = j0 + t;
      __syncthreads();  // what the batch before wrote lies before what this one reads
      const float y = j < recent ? w[old + j] : 0.f;
      __syncthreads();
      if (j < recent) {
        kept[need + j] = old + j;
        out_w[need + j] = y;
      }
    }
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveLoads = 4;  // 16-byte loads of a thread in flight

// CTA (part, head, sequence): parts are pieces of a row's columns (in place) or
// shares of the rows, of the keys first, then of the values.
__global__ void __launch_bounds__(kMoveThreads, 4) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the lists are there
  const int h = blockIdx.y, b = blockIdx.z, t = threadIdx.x;
  const int parts = a.pieces * a.shares;
  const bool values = (int)blockIdx.x >= parts;
  const int part = (int)blockIdx.x - (values ? parts : 0);
  const int piece = part % a.pieces, share = part / a.pieces;
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
  const int units = a.d / a.pieces / 8;       // 16-byte units of a row here (a power of two)
  const int rows = kMoveThreads / units;      // rows of one load of the block
  pool += h * s_head + piece * (a.d / a.pieces) + 8 * (t & (units - 1));
  const int r = t / units;
  const int batch = rows * kMoveLoads;
  // offsets of source and destination of this thread's row e of the batch at
  // i0, source -1: nothing to copy; whether any key of the batch stays
  long long src[kMoveLoads], dst[kMoveLoads];
  auto look_up = [&](int i0) {
    int j[kMoveLoads];
    bool more = false;
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e) {
      const int i = i0 + e * rows + r;
      j[e] = i < a.budget ? __ldcg(kept + i) : -1;
      more = more || j[e] >= 0;
    }
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e) {
      src[e] = -1;
      if (j[e] < 0) continue;
      const int i = i0 + e * rows + r;
      const int pf = a.page_div(j[e]), pt = a.page_div(i);
      const int page_f = __ldg(from + pf), page_t = __ldg(to + pt);
      if (page_f < 0 || page_f >= a.pool.num_pages || page_t < 0 || page_t >= a.pool.num_pages) {
        report_status(a.status, kStatusBadSeqlens);
        continue;
      }
      const long long x = page_f * s_page + (j[e] - pf * a.pool.page_size) * s_row;
      dst[e] = page_t * s_page + (i - pt * a.pool.page_size) * s_row;
      if (x != dst[e]) src[e] = x;  // else it stays where it is
    }
    return more;
  };
  const int stride = a.shares * batch;
  int i0 = share * batch;
  if (i0 >= a.budget) return;
  bool more = look_up(i0);
  while (true) {
    // the block leaves together, behind the last key that stays
    if (!__syncthreads_or(more)) break;
    uint4 x[kMoveLoads];
    __nv_bfloat16* out[kMoveLoads];
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e) {
      out[e] = src[e] >= 0 ? pool + dst[e] : nullptr;
      if (src[e] >= 0) x[e] = *reinterpret_cast<const uint4*>(pool + src[e]);
    }
    i0 += stride;
    more = i0 < a.budget && look_up(i0);
    __syncthreads();  // the batch has been read before any of it is written
#pragma unroll
    for (int e = 0; e < kMoveLoads; ++e)
      if (out[e] != nullptr) *reinterpret_cast<uint4*>(out[e]) = x[e];
  }
}

template <int THREADS, bool HELD>
cudaError_t launch_select(const EvictArgs& a, size_t bytes, cudaStream_t st) {
  // for the most that any call needs: two calls at once ask for the same
  static std::atomic<unsigned char> asked[kMaxSharedMemoryDevices];
  const cudaError_t e = HELD ? ask_shared_memory(reinterpret_cast<const void*>(evict_select_kernel<THREADS, HELD>),
                                                 (int)kSelectMostBytes, asked)
                             : cudaSuccess;
  if (e != cudaSuccess) return e;
  evict_select_kernel<THREADS, HELD><<<dim3((unsigned)a.Hkv, (unsigned)a.B), THREADS, bytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

void evict_split(int B, int Hkv, int d, int budget, bool in_place, int sms, int* pieces, int* shares) {
  // eight blocks for each SM, of whole rows; fewer where a share would be less than a batch of rows
  *pieces = *shares = 1;
  const long long ctas = 2ll * B * Hkv, want = 8ll * sms;
  if (in_place) {
    while (*pieces * 64 < d * 2 && ctas * *pieces < want) *pieces *= 2;
    return;
  }
  const int batch = kMoveThreads / (d / 8) * kMoveLoads;
  const long long most = ((long long)budget + batch - 1) / batch;
  long long s = (want + ctas - 1) / ctas;
  if (s > most) s = most;
  *shares = s < 1 ? 1 : (int)s;
}

cudaError_t launch_kv_evict(const EvictArgs& args, cudaStream_t st) {
  // threads by the longest sequence that the rows can hold: up to 16 weights each
  // with 256, up to 52 with 1024; past shared memory a form that holds none
  EvictArgs a = args;
  const int most = a.most_keys < a.w_keys ? a.most_keys : a.w_keys;
  a.held_words = (most + 3) / 4 * 4;
  const size_t bytes = ((size_t)a.held_words + (most < a.budget ? most : a.budget)) * 4;
  cudaError_t e;
  if (bytes > kSelectMostBytes) e = launch_select<1024, false>(a, 0, st);
  else if (most <= 4096) e = launch_select<256, true>(a, bytes, st);
  else e = launch_select<1024, true>(a, bytes, st);
  if (e != cudaSuccess) return e;
  // the move's CTAs come while the selection ends, and wait for it
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * a.pieces * a.shares), (unsigned)a.Hkv, (unsigned)a.B);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, a);
}

}  // namespace fa

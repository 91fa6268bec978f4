// prompt_weights.cu -- the attention weight that each key of a prompt got.
//
//   w_hj = sum over the query heads of K/V head h and the counted tokens i
//          (the last `window` of a sequence, or all) that see key j of
//          exp(scale * q_i . k_j - LSE_i),
// from the forward's log-sum-exp, so one product and one exponential per score
// and nothing else: P is summed where it is computed.
//
// Keys are the rows of the products (S^T = K Q^T, a TMEM lane per key), so that
// a thread adds up its own key's weights over the query tiles and no thread
// needs another's. A unit is 256 keys (two tiles) of a sequence and K/V head,
// which stay in shared memory while the query tiles (128 rows: all heads of the
// group, prompt_fwd.cu) that see them stream through a ring; the next unit's
// keys load meanwhile. Two tiles of keys per query tile, because one product of
// 512 cycles per 32 KB of queries would ask the L2 for 18 TB/s. S is double
// buffered in tensor memory for each key tile (four buffers of 128 columns).
//
// Products and exponentials need 1024 cycles a unit and query tile each (8192
// FLOP and 32 exponentials per cycle and SM). Measured: 1900 by the tensor pipe's
// share (8 prompts of 361 to 6925 tokens, 32 heads on 8: 452 us; the last 64 tokens
// of six of 5627 to 18982: 44 us, of which most is the beginning and end of units of
// two query tiles). The products alone took 1530, an SM's warps issue 470
// instructions for 32 keys and 128 query rows where 280 do the sum, each wait takes
// a hundred cycles even when it is over. So a warp takes whole query tiles in turn
// with its twin (halves of each: 493 us), and statistics and scores are awaited at
// once (503 us one after the other). Other ways that were slower: keys as first
// operands in tensor memory, which leaves three S buffers for both tiles (2400);
// four keys to a thread, by loads of 16 lanes, which need a quarter of the
// statistics (2150); loads of 16 columns (2040).
//
// Sums: 64 weights, 16 of each of four query tiles, in each of eight fp32
// accumulators, and their sums with a compensation term (Kahan's), in an order that
// a unit's own tiles decide.
//
// Warps 0: producer, 1: MMA issuer, 2: scheduler, 3: statistics, 4-19: weights,
// four warps to the even and to the odd query tiles of each key tile (with
// eight warps, two to a scheduler, waits and latencies were not covered: 8192
// tokens, 32 heads 398 us). Units are listed longest first and taken over
// from CTAs that have not begun, as in prompt_fwd.cu. Every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "prompt.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

template <int D>
struct WCfg {
  static constexpr int CH = D / 64;
  static constexpr int CHUNK = 128 * 128;
  static constexpr int TILE = CH * CHUNK;  // 128 rows x D bf16
  static constexpr int QS = 3;             // query tiles in flight
  static constexpr int OFF_K = 0;          // [2 units][2 tiles]
  static constexpr int OFF_Q = OFF_K + 4 * TILE;
  static constexpr int OFF_STAT = OFF_Q + QS * TILE;  // [QS][128] -LSE * log2(e)
  static constexpr int IRING = 3, ITEM_INTS = 12;  // units published ahead (short ones: many)
  static constexpr int OFF_PART = OFF_STAT + QS * 512;  // [2 tiles][128] sums over the odd query tiles
  static constexpr int OFF_BARS = OFF_PART + 2 * 512;
  // k_full[2], k_empty[2], q_full[QS], q_empty[QS], st_full[QS], st_empty[QS], s_full[2][2], s_free[2][2],
  // part_full[2], part_free[2], item_full, item_empty [IRING each], cancel, near, drain
  static constexpr int NBARS = 4 + 4 * QS + 12 + 2 * IRING + 3;
  static constexpr int OFF_ITEMS = (OFF_BARS + NBARS * 8 + 15) / 16 * 16;
  static constexpr int OFF_CANCEL = OFF_ITEMS + IRING * ITEM_INTS * 4;
  static constexpr int OFF_MISC = OFF_CANCEL + 16;
  static constexpr int BYTES = OFF_MISC + 8;
  static constexpr int MOST = 227 * 1024;
  // 1 KB of alignment slack where it fits; the kernel checks the alignment
  static constexpr int ALLOC = BYTES + 1024 <= MOST ? BYTES + 1024 : MOST;
  static constexpr int THREADS = 640;
  static constexpr uint32_t S_COL(int t, int b) { return 256u * t + 128u * b; }
};

// A unit in the ring: K/V head, first packed key and its index in the sequence,
// keys of the sequence from there on, query tiles, how many of them key tile 1
// does not meet, first packed token of the first query tile, tokens of the
// sequence from there on, the token (from there on) whose diagonal is the unit's
// first key, sequence, index of its first new key. All -1: no more units.
enum : int { kWHead, kWKey, kWKey0, kWLeft, kWTiles, kWSkip1, kWTok, kWTokens, kWDiag, kWSeq, kWNew, kWInts };

struct WUnit {
  int f[kWInts];
};

// Whole warp: the units of grid index `u` are `per` neighbours in the list (one,
// unless the grid is smaller than the list, as over pages): unit `sub` of them;
// false past the last one of all.
template <bool PAGED>
__device__ __forceinline__ bool weight_unit(const PromptWeightArgs& a, long long u, int sub, int lane, bool report, int& per,
                                            WUnit& k) {
  bool bad = false;
  auto span = [&](int b) {
    const PromptView v = prompt_view(a.seqs, b, bad);
    bad = bad || (v.n > 0 && v.m > a.w_keys);
    const bool there = v.n > 0 && v.m <= a.w_keys;
    return PromptSpan{0, there ? (v.m + 255) / 256 : 0};
  };
  PromptSpan first;
  int top;
  const int total = count_blocks(a.seqs.B, lane, span, first, top);
  if (report && bad) report_status(a.status, kStatusBadSeqlens);
  const long long units = (long long)total * a.Hkv;
  if constexpr (PAGED) {
    per = units > gridDim.x ? (int)((units + gridDim.x - 1) / gridDim.x) : 1;
    u = u * per + sub;
  }
  if (u >= units) return false;
  const int hpg = a.heads_per_group;
  const int group = (int)(u / ((long long)total * hpg));
  const int local = (int)(u - (long long)group * total * hpg);
  const int heads = min(hpg, a.Hkv - group * hpg);
  const int idx = local / heads;
  int seq, block;
  find_block(a.seqs.B, lane, span, first, top, idx, seq, block);
  const PromptView v = prompt_view(a.seqs, seq, bad);
  const int TP = a.tile_tokens, past = v.m - v.n;
  const int kb = (v.m + 255) / 256 - 1 - block;  // the first keys are seen by the most tokens
  const int key0 = kb * 256;
  const int from = a.window > 0 && a.window < v.n ? v.n - a.window : 0;  // the first token that counts
  // query tiles begin at multiples of TP from the first token that counts
  auto first_tile = [&](int key) { return max(key - past - from, 0) / TP; };
  const int tiles = (v.n - from + TP - 1) / TP, i0 = first_tile(key0);
  const int tok = from + i0 * TP;
  k.f[kWHead] = group * hpg + local - idx * heads;
  k.f[kWKey] = v.k0 + key0;
  k.f[kWKey0] = key0;
  k.f[kWLeft] = v.m - key0;
  k.f[kWTiles] = tiles - i0;
  k.f[kWSkip1] = v.m > key0 + 128 ? first_tile(key0 + 128) - i0 : tiles - i0;
  k.f[kWTok] = v.q0 + tok;
  k.f[kWTokens] = v.n - tok;
  k.f[kWDiag] = key0 - past - tok;
  k.f[kWSeq] = seq;
  k.f[kWNew] = past;
  return true;
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(640, 1) prompt_weights_kernel(const __grid_constant__ PromptWeightArgs a) {
  using C = WCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t pad = ((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw);
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = smem_u32(smem);
  if (pad + C::BYTES > (uint32_t)C::ALLOC) {
    // cannot place the swizzled tiles: report and leave before touching anything
    if (threadIdx.x == 0) report_status(a.status, kStatusTimeout);
    return;
  }
  const uint32_t bar0 = sbase + C::OFF_BARS;
  auto BAR = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  const int B_KFULL = 0, B_KEMPTY = 2, B_QFULL = 4, B_QEMPTY = B_QFULL + C::QS, B_STFULL = B_QEMPTY + C::QS,
            B_STEMPTY = B_STFULL + C::QS, B_SFULL = B_STEMPTY + C::QS, B_SFREE = B_SFULL + 4, B_PART = B_SFREE + 4, B_ITF = B_PART + 4,
            B_ITE = B_ITF + C::IRING, B_CANCEL = B_ITE + C::IRING, B_NEAR = B_CANCEL + 1, B_DRAIN = B_NEAR + 1;
  volatile int* items = reinterpret_cast<volatile int*>(smem + C::OFF_ITEMS);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int TP = a.tile_tokens, RT = TP * a.G;

  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(BAR(B_KFULL + b), 1);
      mbar_init(BAR(B_KEMPTY + b), 1);
    }
    for (int s = 0; s < C::QS; ++s) {
      mbar_init(BAR(B_QFULL + s), 1);
      mbar_init(BAR(B_QEMPTY + s), 1);
      mbar_init(BAR(B_STFULL + s), 1);
      mbar_init(BAR(B_STEMPTY + s), 8);  // one arrival per weights warp of the tile
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(BAR(B_SFULL + i), 1);
      mbar_init(BAR(B_SFREE + i), 4);
      mbar_init(BAR(B_PART + i), 4);  // part_full[2], part_free[2]
    }
    for (int s = 0; s < C::IRING; ++s) {
      mbar_init(BAR(B_ITF + s), 1);
      mbar_init(BAR(B_ITE + s), 19);  // producer, MMA, statistics, 16 weights warps
    }
    mbar_init(BAR(B_CANCEL), 1);
    mbar_init(BAR(B_NEAR), 1);
    mbar_init(BAR(B_DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_u32((const void*)tmem_slot), 512);
  {
    // rows RT .. 127 of the query slots (G does not divide 128) stay zero
    const int per_slot = (128 - RT) * C::CH * 8;
    for (int e = threadIdx.x; e < C::QS * per_slot; e += C::THREADS) {
      const int slot = e / per_slot, u = e - slot * per_slot, r = RT + u / (C::CH * 8), x = u % (C::CH * 8);
      *reinterpret_cast<uint4*>(smem + C::OFF_Q + slot * C::TILE + (x >> 3) * C::CHUNK + r * 128 + (x & 7) * 16) =
          make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto wait = [&](int b, uint32_t parity) { return wait_warp(BAR(b), parity, a.status, a.wait_limit_ns); };
  auto get_item = [&](int i) { return wait(B_ITF + i % C::IRING, (i / C::IRING) & 1); };
  auto item = [&](int i, int what) {
    return __shfl_sync(0xffffffffu, (int)items[(i % C::IRING) * C::ITEM_INTS + what], 0);
  };
  auto release_item = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(BAR(B_ITE + i % C::IRING));
  };
  bool ok = true;

  if (warp == 2) {
    // ---------------------------------------------------------- scheduler
    long long u = blockIdx.x;  // grid index in work, -1 past the last unit
    int sub = 0, per = 1;      // its unit in work, and units
    int asked = 0;             // questions for a CTA that has not begun
    auto take_over = [&](int& next) {
      if (lane == 0) {
        mbar_arrive_expect_tx(BAR(B_CANCEL), 16);
        clc_try_cancel(sbase + C::OFF_CANCEL, BAR(B_CANCEL));
      }
      if (!wait(B_CANCEL, asked & 1)) return false;
      ++asked;
      next = clc_next_cta(sbase + C::OFF_CANCEL);
      fence_proxy_async_smem();
      __syncwarp();
      return true;
    };
    int next = 0;
    for (int i = 0; ok && u >= 0; ++i) {
      const int s = i % C::IRING;
      if (i >= C::IRING) ok = wait(B_ITE + s, ((i / C::IRING) - 1) & 1);
      // not before the unit in work is near its end: a CTA with a long one would
      // hold the next back from those that run dry
      if (ok && i > 0) ok = wait(B_NEAR, (i - 1) & 1);
      if (ok && i > 0 && (!PAGED || ++sub == per)) {
        sub = 0;
        ok = take_over(next);
        u = next;
      }
      if (!ok) break;
      WUnit k;
      if (u >= 0 && !weight_unit<PAGED>(a, u, sub, lane, u == 0 && sub == 0, per, k)) u = -1;
      if (lane == 0) {
        volatile int* d = items + s * C::ITEM_INTS;
#pragma unroll
        for (int e = 0; e < kWInts; ++e) d[e] = u >= 0 ? k.f[e] : -1;
        mbar_arrive(BAR(B_ITF + s));
      }
      __syncwarp();
    }
    // What has not begun finds nothing either: taken over here, where that takes
    // a question, rather than begun, which takes 1.3 us on an SM of its own.
    if constexpr (PAGED)
      while (ok && next >= 0) ok = take_over(next);
  } else if (warp == 0) {
    // ---------------------------------------------------------- producer
    const int nbox = PAGED ? 128 / a.box_rows : 1;
    const bool mine = PAGED ? lane < nbox * C::CH : lane == 0;
    const int box = PAGED ? lane % nbox : 0, chunk = PAGED ? lane / nbox : 0;
    if (lane == 0) {
      tma_prefetch_desc(&a.tmQ);
      tma_prefetch_desc(&a.tmK);
    }
    int g0 = 0, units = 0, last_q = -1;
    for (int i = 0; ok; ++i) {
      if (!get_item(i)) { ok = false; break; }
      const int left = item(i, kWLeft);
      if (left < 0) break;
      const int head = item(i, kWHead), tiles = item(i, kWTiles), tok = item(i, kWTok);
      const int kbuf = i & 1;
      if (i >= 2 && !wait(B_KEMPTY + kbuf, ((i >> 1) - 1) & 1)) { ok = false; break; }
      units = i + 1;
      if constexpr (PAGED) {
        const int keys = min(left, 256);
        const int boxes = (keys + a.box_rows - 1) / a.box_rows;
        if (lane == 0) mbar_arrive_expect_tx(BAR(B_KFULL + kbuf), (uint32_t)(boxes * a.box_rows * 128 * C::CH));
        __syncwarp();
        const int* table = a.block_tables + (size_t)item(i, kWSeq) * a.max_pages;
        const int key0 = item(i, kWKey0);
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          const int at = t * 128 + box * a.box_rows;
          if (mine && at < keys) {
            const int pi = (key0 + at) / a.pool.page_size;
            int page = __ldg(table + pi);
            if (page < 0 || page >= a.pool.num_pages) {
              report_status(a.status, kStatusBadSeqlens);
              page = a.pool.num_pages;  // outside the tensor: reads as zeros
            }
            tma_load_4d(sbase + C::OFF_K + (2 * kbuf + t) * C::TILE + chunk * C::CHUNK + box * a.box_rows * 128, &a.tmK,
                        BAR(B_KFULL + kbuf), chunk * 64, key0 + at - pi * a.pool.page_size, head, page);
          }
        }
      } else if (lane == 0) {
        const int n_t = left > 128 ? 2 : 1, key = items[(i % C::IRING) * C::ITEM_INTS + kWKey];
        mbar_arrive_expect_tx(BAR(B_KFULL + kbuf), (uint32_t)(n_t * C::TILE));
        for (int t = 0; t < n_t; ++t)
          for (int c = 0; c < C::CH; ++c)
            tma_load_3d(sbase + C::OFF_K + (2 * kbuf + t) * C::TILE + c * C::CHUNK, &a.tmK, BAR(B_KFULL + kbuf), c * 64,
                        key + 128 * t, head);
      }
      __syncwarp();
      for (int j = 0; j < tiles; ++j) {
        if (__any_sync(0xffffffffu, *abort_flag != 0)) { ok = false; break; }
        const int g = g0 + j, s = g % C::QS;
        if (g >= C::QS && !wait(B_QEMPTY + s, ((g / C::QS) - 1) & 1)) { ok = false; break; }
        if (lane == 0) {
          mbar_arrive_expect_tx(BAR(B_QFULL + s), (uint32_t)(RT * 128 * C::CH));
          for (int c = 0; c < C::CH; ++c)
            tma_load_4d(sbase + C::OFF_Q + s * C::TILE + c * C::CHUNK, &a.tmQ, BAR(B_QFULL + s), c * 64, 0, tok + j * TP,
                        head);
        }
        __syncwarp();
        last_q = g;
        if (j == max(0, tiles - 4) && lane == 0) mbar_arrive(BAR(B_NEAR));
      }
      if (!ok) break;
      g0 += tiles;
      release_item(i);
    }
    if (!ok) *abort_flag = 1;
    // drain: what was asked for last must have landed before exit
    for (int i = max(0, units - 2); i < units; ++i) wait(B_KFULL + (i & 1), (i >> 1) & 1);
    for (int g = max(0, last_q - C::QS + 1); g <= last_q; ++g)
      wait(B_QFULL + g % C::QS, (g / C::QS) & 1);
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    const uint32_t leader = elect_one();
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
    const uint64_t dK0 = sdesc_sw128(sbase + C::OFF_K, 16, 1024), dQ0 = sdesc_sw128(sbase + C::OFF_Q, 16, 1024);
    // query tile g has S buffer g % 2 of each key tile
    int g0 = 0;              // query tiles before this unit
    int used0 = 0, used1 = 0;  // S tiles of key tile 1 so far, by buffer (key tile 0 has one for each query tile)
    for (int i = 0; ok; ++i) {
      if (!get_item(i)) { ok = false; break; }
      const int tiles = item(i, kWTiles), skip1 = item(i, kWSkip1);
      if (tiles < 0) break;
      if (!wait(B_KFULL + (i & 1), (i >> 1) & 1)) { ok = false; break; }
#pragma unroll 1
      for (int j = 0; j < tiles; ++j) {
        const int gone = *abort_flag;
        const int g = g0 + j, s = g % C::QS;
        // (S of the first two query tiles: a phase before the barrier's first, which is over)
        ok = wait_warp2(BAR(B_QFULL + s), (g / C::QS) & 1, BAR(B_SFREE + (g & 1)), ((g >> 1) - 1) & 1, a.status,
                        a.wait_limit_ns) && !__any_sync(0xffffffffu, gone != 0);
        if (!ok) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t == 1 && j < skip1) continue;
          const int b = g & 1;
          if (t == 1) {
            const int n = b ? used1 : used0;  // the buffer's S tiles before this one
            if (!wait(B_SFREE + 2 + b, (n - 1) & 1)) { ok = false; break; }
            if (b) ++used1;
            else ++used0;
          }
          tc_fence_after();
          const uint64_t ka = dK0 + (uint64_t)(((2 * (i & 1) + t) * C::TILE) >> 4);
          const uint64_t qb = dQ0 + (uint64_t)((s * C::TILE) >> 4);
          const uint32_t dcol = tmem + C::S_COL(t, 0) + 128u * (uint32_t)b;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = (uint64_t)(((kk >> 2) * C::CHUNK + (kk & 3) * 32) >> 4);
            mma_ss(dcol, ka + off, qb + off, idesc, kk > 0 ? 1u : 0u, leader);
          }
          mma_commit(BAR(B_SFULL + 2 * t + b), leader);
        }
        if (!ok) break;
        mma_commit(BAR(B_QEMPTY + s), leader);
      }
      if (!ok) break;
      mma_commit(BAR(B_KEMPTY + (i & 1)), leader);
      g0 += tiles;
      release_item(i);
    }
    if (!ok) *abort_flag = 1;
    mma_commit(BAR(B_DRAIN), leader);  // every product issued has finished before TMEM is released
    wait(B_DRAIN, 0);
  } else if (warp == 3) {
    // ---------------------------------------------------------- statistics
    // -LSE * log2(e) of a query tile's rows, lane l: rows 4 l .. 4 l + 3; -inf
    // (weight zero) for rows past the sequence, and where the row saw no key
    // One warp does this for all: few instructions a tile (a division for each
    // row and tile made it the kernel's bound), loads three tiles ahead.
    int tk[4];             // token of the row within its tile; past every tile: no such row
    long long at[4];       // offset of its statistic from that of the group's first head and the tile's first token
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 4 * lane + e, x = a.g_div(r);
      tk[e] = r < RT ? x : 0x7fffffff;
      at[e] = (long long)(r - x * a.G) * a.seqs.total_q + x;
    }
    uint32_t slot = 0, slot_phase = 1;
    for (int i = 0; ok; ++i) {
      if (!get_item(i)) { ok = false; break; }
      const int tiles = item(i, kWTiles);
      if (tiles < 0) break;
      const int tokens = item(i, kWTokens);
      const float* base = a.LSE + (long long)item(i, kWHead) * a.G * a.seqs.total_q + item(i, kWTok);
      float ahead[3][4];
      auto fetch = [&](int j, float (&x)[4]) {
        const int left = tokens - j * TP;  // not positive past the last tile: nothing is read
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = tk[e] < left ? __ldg(base + (long long)j * TP + at[e]) : -INFINITY;
      };
      fetch(0, ahead[0]);
      fetch(1, ahead[1]);
      fetch(2, ahead[2]);
#pragma unroll 1
      for (int j = 0; j < tiles; ++j) {
        float4 x;
        x.x = ahead[0][0] == -INFINITY ? -INFINITY : -ahead[0][0] * 1.4426950408889634f;
        x.y = ahead[0][1] == -INFINITY ? -INFINITY : -ahead[0][1] * 1.4426950408889634f;
        x.z = ahead[0][2] == -INFINITY ? -INFINITY : -ahead[0][2] * 1.4426950408889634f;
        x.w = ahead[0][3] == -INFINITY ? -INFINITY : -ahead[0][3] * 1.4426950408889634f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ahead[0][e] = ahead[1][e];
          ahead[1][e] = ahead[2][e];
        }
        fetch(j + 3, ahead[2]);
        if (!wait(B_STEMPTY + slot, slot_phase)) { ok = false; break; }
        reinterpret_cast<float4*>(smem + C::OFF_STAT + slot * 512)[lane] = x;
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_STFULL) + 8 * slot);
        if (++slot == C::QS) {
          slot = 0;
          slot_phase ^= 1u;
        }
      }
      if (!ok) break;
      release_item(i);
    }
  } else {
    // ---------------------------------------------------------- weights
    const int t = (warp >> 2 & 1) ^ 1, odd = warp >= 12, wq = warp & 3;  // key tile, query tiles
    const int row = wq * 32 + lane;                                       // key of the tile
    const uint32_t s_addr = tmem + ((uint32_t)(wq * 32) << 16) + C::S_COL(t, odd);
    const uint64_t c22 = f2_pack(a.scale_log2, a.scale_log2);
    // The loop over query tiles is bound by the instructions it issues: 280 for
    // the sum over 128 columns of 32 keys, and what comes on top. So ring positions are
    // counted, not divided out, masks are rare, and sums are joined only every fourth tile.
    uint32_t slot = odd, slot_phase = 0;  // ring position of this warp's next query tile
    int g0 = 0;                           // query tiles before the unit
    int c = 0;                            // S tiles of this warp so far
    const uint32_t bar_stat = BAR(B_STFULL), bar_s = BAR(B_SFULL + 2 * t + odd);
    for (int i = 0; ok; ++i) {
      if (!get_item(i)) { ok = false; break; }
      const int tiles = item(i, kWTiles);
      if (tiles < 0) break;
      const int skip = t == 0 ? 0 : item(i, kWSkip1);
      // the token (from the unit's first tile's on) whose diagonal is the key tile's first key
      const int j0 = (g0 & 1) ^ odd;  // this warp's first query tile of the unit
      int first = item(i, kWDiag) + 128 * t - j0 * TP;
      int tokens = item(i, kWTokens) - j0 * TP;  // from the next query tile on
      g0 += tiles;
      uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
      float total = 0.f, lost = 0.f;
      auto join = [&]() {
        const float2 sa = f2_unpack(fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3])));
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = 0ull;
        const float y = __fsub_rn(__fadd_rn(sa.x, sa.y), lost), z = __fadd_rn(total, y);
        lost = __fsub_rn(__fsub_rn(z, total), y);
        if (!(fabsf(lost) < INFINITY)) lost = 0.f;  // an infinite weight stays infinite (inf - inf is NaN)
        total = z;
      };
#pragma unroll 1
      for (int j = j0; j < tiles; j += 2) {
        if (j < skip) {
          if (!wait_warp(bar_stat + 8 * slot, slot_phase, a.status, a.wait_limit_ns)) { ok = false; break; }
        } else {
          if (!wait_warp2(bar_stat + 8 * slot, slot_phase, bar_s, c & 1, a.status, a.wait_limit_ns)) { ok = false; break; }
          tc_fence_after();
          const float* nl = reinterpret_cast<const float*>(smem + C::OFF_STAT + slot * 512);
          if (first + 127 > 0 || tokens * a.G < 128) {
            // Columns that a key's weight has no part in (before its diagonal,
            // behind the sequence's end: they may hold anything) become -inf
            // where they stand: a few tiles to a unit, and no mask below.
            const int lo = a.G * max(first + row, 0), hi = a.G * min(tokens, 128);
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t r[32];
              tmem_ld32(s_addr + 32 * q, r);
              tmem_ld_wait();
#pragma unroll
              for (int u = 0; u < 32; ++u)
                r[u] = 32 * q + u < lo || 32 * q + u >= hi ? __float_as_uint(-INFINITY) : r[u];
              tmem_st32(s_addr + 32 * q, r);
            }
            tmem_st_wait();
          }
          auto add = [&](const uint32_t (&r)[32], int q) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float4 n4 = *reinterpret_cast<const float4*>(nl + 32 * q + 4 * k);
              const float2 x = f2_unpack(ffma2(f2_pack(__uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1])), c22, f2_pack(n4.x, n4.y)));
              const float2 y = f2_unpack(ffma2(f2_pack(__uint_as_float(r[4 * k + 2]), __uint_as_float(r[4 * k + 3])), c22, f2_pack(n4.z, n4.w)));
              sum[2 * (k & 1)] = fadd2(sum[2 * (k & 1)], f2_pack(ex2_approx(x.x), ex2_approx(x.y)));
              sum[2 * (k & 1) + 1] = fadd2(sum[2 * (k & 1) + 1], f2_pack(ex2_approx(y.x), ex2_approx(y.y)));
            }
          };
          // each load is under way while the one before is exponentiated (both
          // awaited first: 611 us instead of 521 for 8 prompts of 361 to 6925 tokens)
          uint32_t ra[32], rb[32];
          tmem_ld32(s_addr, ra);
          tmem_ld_wait_dep(ra);
          tmem_ld32(s_addr + 32, rb);
          add(ra, 0);
          tmem_ld_wait_dep(rb);
          tmem_ld32(s_addr + 64, ra);
          add(rb, 1);
          tmem_ld_wait_dep(ra);
          tmem_ld32(s_addr + 96, rb);
          add(ra, 2);
          tmem_ld_wait_dep(rb);
          // all of S is in registers: its buffer takes the tile after next
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(B_SFREE + 2 * t + odd));
          add(rb, 3);
          ++c;
          // every fourth of the unit's own tiles: which weights are added up together
          // must not depend on the units that this CTA had before
          if ((j & 6) == 6) join();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_STEMPTY) + 8 * slot);
        first -= 2 * TP;
        tokens -= 2 * TP;
        slot += 2;
        if (slot >= C::QS) {
          slot -= C::QS;
          slot_phase ^= 1u;
        }
      }
      if (!ok) break;
      join();
      // the odd query tiles' sums go to the even ones' warps
      volatile float* part = reinterpret_cast<float*>(smem + C::OFF_PART + t * 512) + row;
      if (odd) {
        if (i > 0 && !wait(B_PART + 2 + t, (i - 1) & 1)) { ok = false; break; }
        *part = total;
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_PART + t));
        release_item(i);
        continue;
      }
      if (!wait(B_PART + t, i & 1)) { ok = false; break; }
      total += *part;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_PART + 2 + t));
      const int left = item(i, kWLeft), key = item(i, kWKey0) + 128 * t + row, fresh = item(i, kWNew);
      float* w = a.W + (long long)item(i, kWSeq) * a.w_batch + (long long)item(i, kWHead) * a.w_head + key;
      // keys that are new with these tokens have no weight yet
      if (128 * t + row < left) *w = a.accumulate && key < fresh ? *w + total : total;
      release_item(i);
    }
  }
  if (!ok) *abort_flag = 1;

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool PAGED>
cudaError_t launch_d(const PromptWeightArgs& a, cudaStream_t st) {
  using C = WCfg<D>;
  static_assert(C::BYTES <= C::MOST, "shared memory budget");
  const long long ctas = a.max_units * a.Hkv;
  if (a.max_units < 1 || ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  static std::atomic<unsigned char> asked[kMaxSharedMemoryDevices];
  cudaError_t e = ask_shared_memory(reinterpret_cast<const void*>(prompt_weights_kernel<D, PAGED>), C::ALLOC, asked);
  if (e != cudaSuccess) return e;
  // A CTA per unit that there can be, most of them taken over. Where a cache's
  // tables are far wider than its sequences nearly all would find nothing: 24 to an
  // SM then, which share the list out among them in runs of neighbours. 8 sequences
  // of 1500 keys in tables of 131072, 64 tokens: 24 us, 410 with a CTA for each unit
  // that there could be. With fewer CTAs the runs of long lists leave a tail: 16
  // whole prompts of 1000 to 20000 tokens in full tables 2530 us, 2940 with 16 to an
  // SM, or with one that goes through the list in strides.
  const int sms = fwd_slots();
  const long long most = PAGED && sms > 0 ? 24ll * sms : ctas;
  prompt_weights_kernel<D, PAGED><<<(unsigned)(ctas < most ? ctas : most), C::THREADS, C::ALLOC, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_weights(const PromptWeightArgs& a, int d, cudaStream_t st) {
  const bool paged = a.seqs.cu_k == nullptr;
  if (d == 128) return paged ? launch_d<128, true>(a, st) : launch_d<128, false>(a, st);
  if (d == 64) return paged ? launch_d<64, true>(a, st) : launch_d<64, false>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace fa

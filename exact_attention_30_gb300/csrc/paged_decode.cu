// paged_decode.cu -- attention of a few new queries per sequence against a
// paged key/value cache, with or without a prefix that all sequences share.
//
// For query row r of a sequence, over the shared prefix's keys and then the
// own keys it sees:
//   O_r = sum_j exp(s_rj - m_r) V_j / l_r,   LSE_r = m_r + ln l_r,
//   s = scale * q.k,
// with the online softmax of "Lesson 1: FlashAttention core idea" §3; partial
// results over disjoint keys merge by the same rule.
//
// Schedule. A unit is one K/V head of one sequence: R = G * Nq query rows
// against its keys, in tiles of 64. All units' tiles are laid end to end and
// cut into equal shares, one per resident CTA, so a batch of very different
// lengths fills the GPU evenly and one long sequence is spread over all of it.
// The lengths live on the device, so each CTA finds its share itself (a block
// scan over the lengths). A share may end inside a unit; such a unit's pieces
// leave normalised fp32 partial results and base-2 log-sum-exps in the
// workspace, at most two per CTA, and decode_merge_kernel combines them in a
// fixed order (results do not depend on timing). A unit that lies in one share
// is written out directly.
//
// A shared prefix with no more rows than fit a unit (those of every sequence,
// B * R <= 64 per K/V head) is one more sequence of the same grid. With more
// rows it is a matrix product of its own (launch_prefix_bf16), and only its
// partial results meet the own keys' here.
//
// CTA: one producer warp and 4 consumer warps per 16 query rows. The producer
// reads page numbers a tile ahead and lets each lane issue one TMA box (64
// columns of up to 64 rows of one page) into a ring of tiles. Consumer warp
// kw owns keys 16 kw .. 16 kw + 15 of every tile and keeps its own running
// maximum, sum and output in registers: no exchange between warps until the
// piece ends. Bytes bound this kernel (4 d bytes per key against 4 d R flops);
// with keys split over warps the warp-level mma.sync needs no barrier, no
// tensor-memory round trip and no transposed copy of P per tile, which is what
// a short cache's latency consists of, and its rate is far from the limit up
// to 32 rows.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
// tolerated growth of a row's maximum (log2 units) before its output is rescaled
constexpr float kRescaleLog2 = 8.0f;
constexpr float kLn2 = 0.69314718055994531f;

template <int D, int MT>
struct Cfg {
  static constexpr int BK = 64;              // keys per tile
  static constexpr int CH = D / 64;          // 128-byte column chunks of a row
  static constexpr int CHUNK = BK * 128;     // 64 rows x 128 bytes, swizzled
  static constexpr int KV = CH * CHUNK;      // the keys or the values of a tile
  static constexpr int STAGE = 2 * KV;
  static constexpr int CONSUMERS = 4 * MT;   // warps
  static constexpr int THREADS = 32 * (1 + CONSUMERS);
  // fp32 [4 key quarters][16 rows][DW columns] per 16 rows, where a piece's
  // warps meet, DW columns at a time
  static constexpr int DW = MT == 1 ? D : D / 2;
  static constexpr int MERGE = 4 * 16 * DW * 4;
  // One 16-row group: its merge fits the piece's last stage, and two CTAs
  // share an SM, one loading while the other one merges. More rows: one CTA.
  static constexpr bool MERGE_IN_STAGE = MT == 1;
  static constexpr int CTAS = MT == 1 ? 2 : 1;
  static constexpr int STAGES = (MT == 1 ? 3 : MT == 2 ? 5 : 4) * (D == 128 ? 1 : 2);
  static constexpr int OFF_MERGE = STAGES * STAGE;
  static constexpr int OFF_ML = OFF_MERGE + (MERGE_IN_STAGE ? 0 : MT * MERGE);  // fp32 m, l [MT][4][16]
  static constexpr int OFF_SCAN = OFF_ML + MT * 4 * 16 * 8;  // int64 [32] warp sums, share start
  static constexpr int OFF_BAR = OFF_SCAN + 48 * 8;
  static constexpr int SMEM = OFF_BAR + 2 * STAGES * 8;
  static constexpr int SMEM_ALLOC = SMEM + 1024;  // base rounded up to 1024 (swizzle atom)
  static_assert(!MERGE_IN_STAGE || MERGE <= STAGE, "merge space");
  static_assert(CTAS * (SMEM_ALLOC + 1024) <= 228 * 1024, "shared memory budget");
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c[16 rows x 8] += a[16 x 16] b[16 x 8], bf16 in, fp32 out. Lane 4g + q holds
// c rows g (0, 1) and g + 8 (2, 3), columns 2q, 2q + 1.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void named_bar(int id, int count) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// Keys of sequence s (s = B: the shared prefix); a bad length is reported and
// counts as zero.
__device__ __forceinline__ int seq_keys(const PagedDecodeArgs& a, int s) {
  if (s >= a.B) return a.prefix_len;
  const int n = __ldg(a.seq_lens + s);
  if (n < 0 || n > kPagedMaxKeys || n > (long long)a.max_pages * a.pool.page_size) {
    report_status(a.status, kStatusBadSeqlens);
    return 0;
  }
  return n;
}

// The share of CTA w: tiles [t0, t1) of all units' tiles laid end to end,
// and where t0 lies.
struct Share {
  long long left;  // tiles
  int seq;         // sequence of the first tile
  int head, tile;  // K/V head and tile within the unit
};

template <class C>
__device__ __forceinline__ Share find_share(const PagedDecodeArgs& a, uint8_t* smem) {
  long long* warp_sum = reinterpret_cast<long long*>(smem + C::OFF_SCAN);  // [32]
  int* start = reinterpret_cast<int*>(smem + C::OFF_SCAN + 32 * 8);        // seq, head, tile
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int WARPS = C::THREADS / 32;
  const int chunk = (a.n_seq + C::THREADS - 1) / C::THREADS;
  const int s0 = min(tid * chunk, a.n_seq), s1 = min(s0 + chunk, a.n_seq);
  long long sum = 0;
  for (int s = s0; s < s1; ++s) sum += (seq_keys(a, s) + C::BK - 1) / C::BK;
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const long long v = warp_sum[w];
    before += w < warp ? v : 0;
    total += v;
  }
  const int Hkv = a.pool.kv_heads;
  const long long T = total * Hkv;
  const long long W = T < (long long)gridDim.x ? T : (long long)gridDim.x;  // CTAs with work
  const long long w = blockIdx.x;
  Share sh{0, 0, 0, 0};
  if (w < W) {
    const long long t0 = T * w / W;
    sh.left = T * (w + 1) / W - t0;
    const long long hi = (before + incl) * Hkv, lo = hi - sum * Hkv;
    if (lo <= t0 && t0 < hi) {  // t0 lies in this thread's chunk of sequences
      long long at = t0 - lo;
      for (int s = s0; s < s1; ++s) {
        const long long n = (seq_keys(a, s) + C::BK - 1) / C::BK;
        if (at < n * Hkv) {
          start[0] = s;
          start[1] = (int)(at / n);
          start[2] = (int)(at - at / n * n);
          break;
        }
        at -= n * Hkv;
      }
    }
  }
  __syncthreads();
  sh.seq = start[0];
  sh.head = start[1];
  sh.tile = start[2];
  return sh;
}

// Walks a share piece by piece (a piece: a unit's tiles within the share);
// producer and consumers walk the same way.
struct Walk {
  Share sh;
  int len, tiles, next_len;

  __device__ __forceinline__ void load(const PagedDecodeArgs& a, int bk) {
    tiles = (len + bk - 1) / bk;
    next_len = sh.seq + 1 < a.n_seq ? seq_keys(a, sh.seq + 1) : 0;  // on its way while this one is worked on
  }
  __device__ __forceinline__ void begin(const PagedDecodeArgs& a, const Share& s, int bk) {
    sh = s;
    len = s.left > 0 ? seq_keys(a, s.seq) : 0;
    load(a, bk);
  }
  __device__ __forceinline__ int piece() const {
    const int n = tiles - sh.tile;
    return sh.left < n ? (int)sh.left : n;
  }
  __device__ __forceinline__ void advance(const PagedDecodeArgs& a, int n, int bk) {
    sh.left -= n;
    sh.tile = 0;
    if (sh.left <= 0 || ++sh.head < a.pool.kv_heads) return;
    sh.head = 0;
    do {
      ++sh.seq;
      len = next_len;
      load(a, bk);
    } while (len == 0 && sh.seq + 1 < a.n_seq);
  }
};

// Partial result of unit u's piece in CTA w. A piece that begins its unit and
// does not end it: the CTA's second slot; one that continues a unit: the
// first. Units of one piece that still need a merge (with a prefix's part)
// have slots of their own behind those.
__device__ __forceinline__ long long part_slot(const PagedDecodeArgs& a, int w, bool begins, bool ends, long long unit) {
  if (begins && ends) return 2ll * a.ctas + unit;
  return 2ll * w + (begins ? 1 : 0);
}

// All rows of sequence s: no key, so O = 0 and LSE = -inf.
template <int D>
__device__ void empty_rows(const PagedDecodeArgs& a, int s) {
  const int Hq = a.pool.kv_heads * a.G, rows = Hq * a.Nq;
  for (long long e = threadIdx.x; e < (long long)rows * (D / 8); e += blockDim.x) {
    const int row = (int)(e / (D / 8)), c = (int)(e - (long long)row * (D / 8)) * 8;
    const int hq = row / a.Nq, i = row - hq * a.Nq;
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.O) + s * a.o_b + hq * a.o_h + i * a.o_r + c) = make_uint4(0u, 0u, 0u, 0u);
    if (c == 0) a.LSE[(long long)s * rows + row] = -INFINITY;
  }
}

template <int D, int MT>
__global__ void __launch_bounds__(Cfg<D, MT>::THREADS, Cfg<D, MT>::CTAS)
    decode_paged_kernel(const __grid_constant__ PagedDecodeArgs a) {
  using C = Cfg<D, MT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto FULL = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto EMPTY = [&](int s) { return bar0 + 8u * (uint32_t)(C::STAGES + s); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(FULL(s), 1);
      mbar_init(EMPTY(s), C::CONSUMERS);
    }
    fence_mbar_init();
  }
  // the merge kernel may be set up meanwhile; it waits for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Share share = find_share<C>(a, smem);
  if (a.prefix_len == 0) {
    if (threadIdx.x == 0) a.begun[blockIdx.x] = -1;
    // rows of sequences without keys
    for (int s = blockIdx.x; s < a.B; s += gridDim.x)
      if (seq_keys(a, s) == 0) empty_rows<D>(a, s);
    __syncthreads();  // begun[] may be written again below, by another thread
  }
  if (share.left <= 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // as at the end
    return;
  }
  Walk wk;
  wk.begin(a, share, C::BK);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const int nbox = C::BK / a.box_rows;      // boxes of a chunk's 64 rows
    const bool mine = lane < nbox * 2 * C::CH;
    const int box = lane % nbox, col = lane / nbox;  // this lane's box; keys' chunks, then values'
    const bool is_v = col >= C::CH;
    const int chunk = is_v ? col - C::CH : col;
    const CUtensorMap* map = is_v ? &a.tmV : &a.tmK;
    const uint32_t dst0 = sbase + (is_v ? C::KV : 0) + chunk * C::CHUNK + box * a.box_rows * 128;
    if (lane == 0) {
      tma_prefetch_desc(&a.tmK);
      tma_prefetch_desc(&a.tmV);
    }
    const int ps = a.pool.page_size;
    int it = 0;
    bool ok = true;
    while (ok && wk.sh.left > 0 && wk.piece() > 0) {
      const int n = wk.piece(), len = wk.len, head = wk.sh.head, first = wk.sh.tile;
      const int* table = wk.sh.seq < a.B ? a.block_tables + (long long)wk.sh.seq * a.max_pages : a.prefix_pages;
      // page and row of this lane's box, a tile ahead
      auto look_up = [&](int tile, int& page, int& row) {
        const int key = tile * C::BK + box * a.box_rows;
        page = -1;
        row = 0;
        if (mine && key < len) {
          const int pi = key / ps;
          row = key - pi * ps;
          page = __ldg(table + pi);
        }
      };
      int page, row;
      look_up(first, page, row);
      for (int j = 0; j < n; ++j, ++it) {
        const int s = it % C::STAGES;
        const int left = len - (first + j) * C::BK;  // keys from this tile on
        const int boxes = left >= C::BK ? nbox : (left + a.box_rows - 1) / a.box_rows;
        int next_page = -1, next_row = 0;
        if (j + 1 < n) look_up(first + j + 1, next_page, next_row);
        if (!mbar_wait_warp(EMPTY(s), ((it / C::STAGES) & 1) ^ 1, a.status, a.wait_limit_ns)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(FULL(s), (uint32_t)(boxes * a.box_rows * 128 * 2 * C::CH));
        __syncwarp();
        if (mine && box < boxes) {
          if (page < 0 || page >= a.pool.num_pages) {
            report_status(a.status, kStatusBadSeqlens);
            page = a.pool.num_pages;  // outside the tensor: reads as zeros
          }
          tma_load_4d(dst0 + s * C::STAGE, map, FULL(s), chunk * 64, row, head, page);
        }
        page = next_page;
        row = next_row;
      }
      wk.advance(a, n, C::BK);
    }
    // copies in flight land before the CTA ends, also when a wait ran out
    for (int t = it - C::STAGES < 0 ? 0 : it - C::STAGES; t < it; ++t)
      mbar_wait_warp(FULL(t % C::STAGES), (t / C::STAGES) & 1, a.status, a.wait_limit_ns);
    return;
  }

  // -------------------------------------------------------------- consumers
  // After a wait ran out a warp goes on without waiting or computing, so that
  // it still reaches every barrier; the status word tells.
  const int cw = warp - 1, mt = cw >> 2, kw = cw & 3;
  const int g = lane >> 2, q = lane & 3;
  const int Hkv = a.pool.kv_heads, Hq = Hkv * a.G, R = a.G * a.Nq;
  const float c2 = a.scale_log2;
  const int ra = mt * 16 + g, rb = ra + 8;  // this lane's query rows
  float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML) + mt * 64;  // [4][16]
  const uint32_t k_off = (uint32_t)((kw * 16 + (lane >> 4) * 8 + (lane & 7)) * 128);
  const uint32_t v_off = (uint32_t)(C::KV + (kw * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * 128);
  const uint32_t k_u = (lane >> 3) & 1, v_u = lane >> 4, sw = lane & 7;
  bool ok = true;
  int it = 0;
  while (wk.sh.left > 0 && wk.piece() > 0) {
    const int n = wk.piece(), first = wk.sh.tile, seq = wk.sh.seq, head = wk.sh.head, len = wk.len;
    const bool pre = seq >= a.B;
    const int rows = pre ? a.B * R : R;
    // row r of this unit: batch entry, query head, new token
    auto row_at = [&](int r, int& b, int& hq, int& i) {
      b = seq;
      if (pre) {
        b = r / R;
        r -= b * R;
      }
      i = r % a.Nq;
      hq = head * a.G + r / a.Nq;
    };
    uint32_t qf[D / 16][4];
    int lim_a = len, lim_b = len;  // keys that rows ra and rb see
    {
      int b, hq, i;
      const uint32_t* qa = nullptr;
      const uint32_t* qb = nullptr;
      const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(a.Q);
      if (ra < rows) {
        row_at(ra, b, hq, i);
        qa = reinterpret_cast<const uint32_t*>(Q + b * a.q_b + hq * a.q_h + i * a.q_r) + q;
        if (!pre) lim_a = len - a.Nq + 1 + i;
      }
      if (rb < rows) {
        row_at(rb, b, hq, i);
        qb = reinterpret_cast<const uint32_t*>(Q + b * a.q_b + hq * a.q_h + i * a.q_r) + q;
        if (!pre) lim_b = len - a.Nq + 1 + i;
      }
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        qf[ks][0] = qa ? __ldg(qa + ks * 8) : 0u;
        qf[ks][1] = qb ? __ldg(qb + ks * 8) : 0u;
        qf[ks][2] = qa ? __ldg(qa + ks * 8 + 4) : 0u;
        qf[ks][3] = qb ? __ldg(qb + ks * 8 + 4) : 0u;
      }
    }
    const int seen = pre ? len : max(0, len - a.Nq + 1);  // keys that every row sees
    const bool active = mt * 16 < rows;                   // else these warps only keep step
    float acc[D / 8][4];
#pragma unroll
    for (int nn = 0; nn < D / 8; ++nn) acc[nn][0] = acc[nn][1] = acc[nn][2] = acc[nn][3] = 0.f;
    float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;
    for (int j = 0; j < n; ++j, ++it) {
      const int s = it % C::STAGES;
      if (ok) ok = mbar_wait_warp(FULL(s), (it / C::STAGES) & 1, a.status, a.wait_limit_ns);
      const int k0 = (first + j) * C::BK + kw * 16;  // this warp's keys
      if (ok && active && k0 < len) {
        const uint32_t st = sbase + s * C::STAGE;
        float x[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t kf[4];
          ldmatrix4(kf, st + k_off + (ks >> 2) * C::CHUNK + ((((2 * ks + k_u) & 7) ^ sw) << 4));
          mma16816(x[0], qf[ks], kf[0], kf[1]);
          mma16816(x[1], qf[ks], kf[2], kf[3]);
        }
        const bool edge = k0 + 16 > seen;  // some key of this warp is hidden from some row
        if (edge) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (k0 + 8 * t + 2 * q + (c & 1) >= (c < 2 ? lim_a : lim_b)) x[t][c] = -INFINITY;
        }
        float t_a = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
        float t_b = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
        t_a = fmaxf(t_a, __shfl_xor_sync(kFull, t_a, 1));
        t_b = fmaxf(t_b, __shfl_xor_sync(kFull, t_b, 1));
        t_a = fmaxf(t_a, __shfl_xor_sync(kFull, t_a, 2)) * c2;
        t_b = fmaxf(t_b, __shfl_xor_sync(kFull, t_b, 2)) * c2;
        const bool up_a = t_a > m_a + kRescaleLog2, up_b = t_b > m_b + kRescaleLog2;
        if (__any_sync(kFull, up_a || up_b)) {  // always at a row's first key
          const float f_a = up_a ? ex2_approx(m_a - t_a) : 1.f, f_b = up_b ? ex2_approx(m_b - t_b) : 1.f;
          m_a = up_a ? t_a : m_a;
          m_b = up_b ? t_b : m_b;
          l_a *= f_a;
          l_b *= f_b;
#pragma unroll
          for (int nn = 0; nn < D / 8; ++nn) {
            acc[nn][0] *= f_a;
            acc[nn][1] *= f_a;
            acc[nn][2] *= f_b;
            acc[nn][3] *= f_b;
          }
        }
        const float n_a = m_a == -INFINITY ? 0.f : -m_a, n_b = m_b == -INFINITY ? 0.f : -m_b;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          x[t][0] = ex2_approx(fmaf(x[t][0], c2, n_a));
          x[t][1] = ex2_approx(fmaf(x[t][1], c2, n_a));
          x[t][2] = ex2_approx(fmaf(x[t][2], c2, n_b));
          x[t][3] = ex2_approx(fmaf(x[t][3], c2, n_b));
          l_a += x[t][0] + x[t][1];
          l_b += x[t][2] + x[t][3];
        }
        // P is rounded to bf16 for the product (half a step of each weight);
        // the sums l keep the unrounded weights
        const uint32_t pf[4] = {pack_bf16x2(x[0][0], x[0][1]), pack_bf16x2(x[0][2], x[0][3]),
                                pack_bf16x2(x[1][0], x[1][1]), pack_bf16x2(x[1][2], x[1][3])};
        // values of keys that some row does not see stay out of the product
        // (0 times NaN); keys 2q, 2q + 1 and 8 + 2q, 8 + 2q + 1 are this lane's
        uint32_t keep0 = kFull, keep1 = kFull;
        if (edge) {
          auto keep = [&](int k) { return (k < seen ? 0xffffu : 0u) | (k + 1 < seen ? 0xffff0000u : 0u); };
          keep0 = keep(k0 + 2 * q);
          keep1 = keep(k0 + 8 + 2 * q);
        }
#pragma unroll
        for (int np = 0; np < D / 16; ++np) {
          uint32_t vf[4];
          ldmatrix4_t(vf, st + v_off + (np >> 2) * C::CHUNK + ((((2 * np + v_u) & 7) ^ sw) << 4));
          if (edge) {
            vf[0] &= keep0;
            vf[1] &= keep1;
            vf[2] &= keep0;
            vf[3] &= keep1;
          }
          mma16816(acc[2 * np], pf, vf[0], vf[1]);
          mma16816(acc[2 * np + 1], pf, vf[2], vf[3]);
        }
        if (edge && len > seen) {
          // the newest keys, seen by some rows only: added row by row
          for (int k = max(k0, seen); k < min(k0 + 16, len); ++k) {
            const int c = k - k0, src = (lane & 28) | ((c & 7) >> 1);
            const float pa = (c & 8) ? ((c & 1) ? x[1][1] : x[1][0]) : ((c & 1) ? x[0][1] : x[0][0]);
            const float pb = (c & 8) ? ((c & 1) ? x[1][3] : x[1][2]) : ((c & 1) ? x[0][3] : x[0][2]);
            const float p_a = __shfl_sync(kFull, pa, src), p_b = __shfl_sync(kFull, pb, src);
            const int r = kw * 16 + c;
            const uint8_t* vr = smem + s * C::STAGE + C::KV + r * 128 + q * 4;
#pragma unroll
            for (int nn = 0; nn < D / 8; ++nn) {
              const uint32_t v2 = *reinterpret_cast<const uint32_t*>(vr + (nn >> 3) * C::CHUNK + (((nn & 7) ^ (r & 7)) << 4));
              const float v0 = __uint_as_float(v2 << 16), v1 = __uint_as_float(v2 & 0xffff0000u);
              if (k < lim_a) {
                acc[nn][0] = fmaf(p_a, v0, acc[nn][0]);
                acc[nn][1] = fmaf(p_a, v1, acc[nn][1]);
              }
              if (k < lim_b) {
                acc[nn][2] = fmaf(p_b, v0, acc[nn][2]);
                acc[nn][3] = fmaf(p_b, v1, acc[nn][3]);
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0 && !(C::MERGE_IN_STAGE && j + 1 == n)) mbar_arrive(EMPTY(s));
    }

    if (!active) {
      wk.advance(a, n, C::BK);
      continue;
    }
    // the four warps of each 16 rows meet: common maximum, then the sum of
    // their outputs, each already scaled by its share of the total
    l_a += __shfl_xor_sync(kFull, l_a, 1);
    l_b += __shfl_xor_sync(kFull, l_b, 1);
    l_a += __shfl_xor_sync(kFull, l_a, 2);
    l_b += __shfl_xor_sync(kFull, l_b, 2);
    if (q == 0) {
      ml[kw * 16 + g] = make_float2(m_a, l_a);
      ml[kw * 16 + g + 8] = make_float2(m_b, l_b);
    }
    named_bar(1 + mt, 128);  // also: every warp has read its keys of the last stage
    float f_a, f_b, lse_a, lse_b;
    auto combine = [&](int r, float m_own, float& f, float& lse) {
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) mm = fmaxf(mm, ml[w * 16 + r].x);
      const float mu = mm == -INFINITY ? 0.f : mm;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 t = ml[w * 16 + r];
        ll = fmaf(t.y, ex2_approx(t.x - mu), ll);
      }
      f = ll == 0.f ? 0.f : ex2_approx(m_own - mu) / ll;
      lse = ll == 0.f ? -INFINITY : mm + __log2f(ll);
    };
    combine(g, m_a, f_a, lse_a);
    combine(g + 8, m_b, f_b, lse_b);
    const int last_stage = (it - 1) % C::STAGES;
    float* om = reinterpret_cast<float*>(smem + (C::MERGE_IN_STAGE ? last_stage * C::STAGE : C::OFF_MERGE + mt * C::MERGE));
    const bool begins = first == 0, ends = first + n == wk.tiles;
    const long long unit = (long long)seq * Hkv + head;
    const bool direct = begins && ends && a.prefix_len == 0;
    const long long slot = part_slot(a, blockIdx.x, begins, ends, unit);
    const int ct = kw * 32 + lane;  // thread of the 16 rows' 128
    if (mt == 0 && ct == 0) {
      if (begins) a.unit_ctas[unit].x = blockIdx.x;
      if (ends) a.unit_ctas[unit].y = blockIdx.x;
      if (begins && !ends) a.begun[blockIdx.x] = unit;
    }
    // row r's column c lies at c ^ 8 (r & 7): the eight rows of a store differ in banks
    constexpr int DW = C::DW;
    const int sg = (8 * g) & (DW - 1);
#pragma unroll
    for (int d0 = 0; d0 < D; d0 += DW) {
      if (d0 > 0) named_bar(1 + mt, 128);  // the columns before these have been read
#pragma unroll
      for (int nn = 0; nn < DW / 8; ++nn) {
        const float* x = acc[d0 / 8 + nn];
        const int c = (8 * nn + 2 * q) ^ sg;
        *reinterpret_cast<float2*>(om + (kw * 16 + g) * DW + c) = make_float2(x[0] * f_a, x[1] * f_a);
        *reinterpret_cast<float2*>(om + (kw * 16 + g + 8) * DW + c) = make_float2(x[2] * f_b, x[3] * f_b);
      }
      named_bar(1 + mt, 128);
#pragma unroll
      for (int e = ct; e < 16 * (DW / 4); e += 128) {
        const int r = e / (DW / 4), c = (e - r * (DW / 4)) * 4;
        const int rr = mt * 16 + r;
        if (rr >= rows) continue;
        const float* p = om + r * DW + (c ^ ((8 * r) & 56 & (DW - 1)));
        float4 y = *reinterpret_cast<const float4*>(p);
#pragma unroll
        for (int w = 1; w < 4; ++w) {
          const float4 z = *reinterpret_cast<const float4*>(p + w * 16 * DW);
          y.x += z.x;
          y.y += z.y;
          y.z += z.z;
          y.w += z.w;
        }
        if (direct) {
          int b, hq, i;
          row_at(rr, b, hq, i);
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.O) + b * a.o_b + hq * a.o_h + i * a.o_r + d0 + c;
          *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
        } else {
          *reinterpret_cast<float4*>(a.Opart + (slot * a.slot_rows + rr) * D + d0 + c) = y;
        }
      }
    }
    if (kw == 0 && q == 0) {
      auto put = [&](int r, float lse) {
        if (r >= rows) return;
        if (direct) {
          int b, hq, i;
          row_at(r, b, hq, i);
          a.LSE[((long long)b * Hq + hq) * a.Nq + i] = lse * kLn2;
        } else {
          a.Lpart[slot * a.slot_rows + r] = lse;
        }
      };
      put(ra, lse_a);
      put(rb, lse_b);
    }
    if (C::MERGE_IN_STAGE) {
      fence_proxy_async_smem();  // the stage's next writer is the TMA
      __syncwarp();
      if (lane == 0) mbar_arrive(EMPTY(last_stage));
    }
    wk.advance(a, n, C::BK);
  }
  // a prefix's kernel ends before this one does, so the merge sees both
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Rows of units that were not written out directly: partial results of the
// own keys (and of the prefix) merged by maximum and sum, in order of the
// CTAs. One block per query row, one warp per partial result at a time.
constexpr int kMergeWarps = 4;
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) decode_merge_kernel(const __grid_constant__ PagedDecodeArgs a) {
  constexpr int E = D / 32;
  __shared__ float sm[kMergeWarps], sl[kMergeWarps], so[kMergeWarps][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hkv = a.pool.kv_heads, R = a.G * a.Nq;
  const int r = (int)(blockIdx.x % R);
  // without a prefix only the units that a share's end cuts have parts
  const long long unit = a.prefix_len == 0 ? a.begun[blockIdx.x / R] : blockIdx.x / R;
  if (unit < 0) return;
  const int b = (int)(unit / Hkv), head = (int)(unit - (long long)b * Hkv);
  int own_first = 0, own_n = 0;
  if (seq_keys(a, b) > 0) {
    const int2 c = a.unit_ctas[unit];
    own_first = c.x;
    own_n = c.y - c.x + 1;
  }
  int pre_first = 0, pre_n = 0;
  const long long pre_unit = (long long)a.B * Hkv + head;
  long long pre_row = 0;  // kernel of its own: row of the first part, parts 256 rows apart
  if (a.pre_splits > 0) {
    const int rr = b * R + r, qblocks = (a.B * R + 255) / 256;
    pre_n = a.pre_splits;
    pre_row = ((long long)head * qblocks + rr / 256) * a.pre_splits * 256 + rr % 256;
  } else if (a.prefix_len > 0) {
    const int2 c = a.unit_ctas[pre_unit];
    pre_first = c.x;
    pre_n = c.y - c.x + 1;
  }
  float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int p = warp; p < own_n + pre_n; p += kMergeWarps) {
    const bool own = p < own_n;
    const int i = own ? p : p - own_n;
    const float* O = a.Opart;
    const float* Ls = a.Lpart;
    long long row;
    if (own || a.pre_splits == 0) {
      const long long slot = part_slot(a, (own ? own_first : pre_first) + i, i == 0, i + 1 == (own ? own_n : pre_n), own ? unit : pre_unit);
      row = slot * a.slot_rows + (own ? r : b * R + r);
    } else {
      O = a.pre_Opart;
      Ls = a.pre_Lpart;
      row = pre_row + 256ll * i;
    }
    const float L = Ls[row];
    float x[E];
    const float* src = O + row * D + lane * E;
    if constexpr (E == 4) {
      const float4 v = *reinterpret_cast<const float4*>(src);
      x[0] = v.x; x[1] = v.y; x[2 % E] = v.z; x[3 % E] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(src);
      x[0] = v.x; x[1] = v.y;
    }
    const float mn = fmaxf(m, L), mu = mn == -INFINITY ? 0.f : mn;
    const float f = ex2_approx(m - mu), w = ex2_approx(L - mu);
    m = mn;
    l = fmaf(l, f, w);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], f, w * x[e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  if (warp != 0) return;
  float mm = -INFINITY;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) mm = fmaxf(mm, sm[w]);
  const float mu = mm == -INFINITY ? 0.f : mm;
  float ll = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    const float f = ex2_approx(sm[w] - mu);
    ll = fmaf(sl[w], f, ll);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(so[w][lane * E + e], f, acc[e]);
  }
  const float inv = ll == 0.f ? 0.f : 1.f / ll;
  const int i = r % a.Nq, hq = head * a.G + r / a.Nq;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.O) + b * a.o_b + hq * a.o_h + i * a.o_r + lane * E;
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2 % E] * inv, acc[3 % E] * inv));
  else
    *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (lane == 0)
    a.LSE[((long long)b * Hkv * a.G + hq) * a.Nq + i] = ll == 0.f ? -INFINITY : (mm + __log2f(ll)) * kLn2;
}

template <int D, int MT>
cudaError_t launch(const PagedDecodeArgs& a, unsigned merge_blocks, cudaStream_t st) {
  using C = Cfg<D, MT>;
  // programmatic dependent launches: the own keys' kernel takes the SMs that a
  // prefix's kernel leaves idle (and waits for that kernel's end before its
  // own), the merge is set up while the main kernel runs
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = a.pre_splits > 0 ? 1 : 0;
  cfg.gridDim = dim3((unsigned)a.ctas);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM_ALLOC;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_paged_kernel<D, MT>, a);
  if (e != cudaSuccess) return e;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(merge_blocks);
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, decode_merge_kernel<D>, a);
}

// Also allows the kernel its shared memory on the current device; every launch
// follows a paged_layout() on the same device.
template <int D, int MT>
int ctas_per_sm() {
  using C = Cfg<D, MT>;
  if (cudaFuncSetAttribute(decode_paged_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC) !=
      cudaSuccess)
    return 0;
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, decode_paged_kernel<D, MT>, C::THREADS, C::SMEM_ALLOC) !=
      cudaSuccess)
    return 0;
  return n;
}

constexpr int kMaxDevices = 64;
std::mutex g_slots_mu;
int g_slots[kMaxDevices][2][3] = {};  // [device][d == 128][16, 32, 64 rows] -> resident CTAs

int resident_ctas(int d, int mt) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> lk(g_slots_mu);
  int& slot = g_slots[dev][d == 128][mt >> 1];
  if (slot == 0) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    const int n = d == 128 ? (mt == 1 ? ctas_per_sm<128, 1>() : mt == 2 ? ctas_per_sm<128, 2>() : ctas_per_sm<128, 4>())
                           : (mt == 1 ? ctas_per_sm<64, 1>() : mt == 2 ? ctas_per_sm<64, 2>() : ctas_per_sm<64, 4>());
    slot = sms * n;
  }
  return slot;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

PagedLayout paged_layout(int B, int Hkv, int rows, int prefix_len, int d) {
  PagedLayout L{};
  const long long pre_rows = prefix_len > 0 ? (long long)B * rows : 0;
  const bool own_kernel = pre_rows > kPagedMaxRows;
  const long long most = pre_rows > rows && !own_kernel ? pre_rows : rows;
  const int mt = most <= 16 ? 1 : most <= 32 ? 2 : 4;
  L.ctas = resident_ctas(d, mt);
  if (L.ctas <= 0) return L;
  L.slot_rows = 16 * mt;
  L.n_seq = B + (pre_rows > 0 && !own_kernel ? 1 : 0);
  const size_t units = (size_t)L.n_seq * Hkv;
  const size_t slots = 2 * (size_t)L.ctas + (prefix_len > 0 ? units : 0);
  L.lpart = up256(slots * L.slot_rows * d * sizeof(float));
  L.unit_ctas = L.lpart + up256(slots * L.slot_rows * sizeof(float));
  L.begun = L.unit_ctas + up256(units * sizeof(int2));
  L.total = L.pre_opart = L.begun + up256((size_t)L.ctas * sizeof(long long));
  if (own_kernel) {
    const long long pre_units = (pre_rows + 255) / 256 * Hkv;
    L.pre_splits = plan_prefix_splits(pre_units, (int)(((long long)prefix_len + 127) / 128), fwd_slots());
    if (L.pre_splits < 1) {
      L.ctas = 0;
      return L;
    }
    const size_t parts = (size_t)pre_units * L.pre_splits * 256;
    L.pre_lpart = L.pre_opart + up256(parts * d * sizeof(float));
    L.total = L.pre_lpart + up256(parts * sizeof(float));
  }
  return L;
}

cudaError_t launch_decode_paged_bf16(const PagedDecodeArgs& a, int d, cudaStream_t st) {
  const long long rows = a.prefix_len > 0 ? (long long)a.B * a.pool.kv_heads * a.G * a.Nq : (long long)a.ctas * a.G * a.Nq;
  if (rows > 0x7fffffffll || a.ctas < 1) return cudaErrorInvalidValue;
  const unsigned blocks = (unsigned)rows;
  if (d == 128) {
    if (a.slot_rows == 16) return launch<128, 1>(a, blocks, st);
    if (a.slot_rows == 32) return launch<128, 2>(a, blocks, st);
    return launch<128, 4>(a, blocks, st);
  }
  if (d == 64) {
    if (a.slot_rows == 16) return launch<64, 1>(a, blocks, st);
    if (a.slot_rows == 32) return launch<64, 2>(a, blocks, st);
    return launch<64, 4>(a, blocks, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa

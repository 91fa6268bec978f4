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
// The lengths live on the device, so each CTA finds its share itself (a warp's
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
// What beginning and ending a unit costs, in tiles, when the keys are shared out
constexpr int kUnitSteps = 2;
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
  // One 16-row group: each warp's output fits the place of its keys and values
  // in the piece's last stage, and two CTAs share an SM, one loading while the
  // other one merges. More rows: space of its own, one CTA.
  static constexpr bool MERGE_IN_STAGE = MT == 1;
  static constexpr int CTAS = MT == 1 ? 2 : 1;
  static constexpr int STAGES = (MT == 2 ? 4 : 3) * (D == 128 ? 1 : 2);
  // Queries as fragments in registers, or read from shared memory per tile
  // (one group: 1% faster than in registers, which then spill; four groups
  // leave 96 registers). FB: K or V fragments loaded at a time.
  static constexpr bool Q_IN_SMEM = MT != 2;
  static constexpr int FB = MT == 4 ? 1 : 4;
  static constexpr int QBUF = 16 * MT * D * 2;  // a unit's queries; two, one being filled for the next unit
  static constexpr int OFF_MERGE = STAGES * STAGE;
  static constexpr int OFF_Q = OFF_MERGE + (MERGE_IN_STAGE ? 0 : MT * MERGE);
  static constexpr int OFF_ML = OFF_Q + 2 * QBUF;               // fp32 m, l [MT][4][16]
  static constexpr int OFF_ROWS = OFF_ML + MT * 4 * 16 * 8;     // RowInfo [2][16 MT]: own keys, prefix
  static constexpr int OFF_SHARE = OFF_ROWS + 2 * 16 * MT * 24;  // the CTA's Share
  static constexpr int OFF_BAR = OFF_SHARE + 48;
  static constexpr int SMEM = OFF_BAR + 2 * STAGES * 8;
  static constexpr int SMEM_ALLOC = SMEM + 1024;  // base rounded up to 1024 (swizzle atom)
  static_assert(!MERGE_IN_STAGE || MERGE == STAGE, "merge space");
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
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes global -> shared by this thread's copy groups; zeros unless `valid`.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
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

// Where row r of a unit lies: offsets of its query and output from those of
// the unit's first batch entry and head, and how many of the newest keys it
// does not see. Row r is new token r mod Nq of the unit's query head r / Nq; a
// prefix's rows are those of sequence 0, 1, ...
struct RowInfo {
  long long q, o;
  int hidden;
};

// Steps that an early CTA rather takes on top than leaves to CTAs that start
// after the prefix's kernel (about their start-up time)
constexpr int kEarlySlack = 6;

// CTA w of W takes steps [begin(w), begin(w + 1)) of T. The first `early` CTAs
// run beside a prefix's kernel and take `more` steps each in that time; the
// rest is shared equally by all (the first `extra` CTAs take one more). Few
// more steps than that: the early ones share them all.
struct Cut {
  long long per, extra, more;
  int early, ctas;
  __device__ __forceinline__ Cut(const PagedDecodeArgs& a, long long T) : more(a.early_steps), early(a.early_ctas), ctas(a.ctas) {
    long long rest = T - early * more;
    FastDiv div = a.ctas_div;
    if (early > 0 && rest < (long long)early * kEarlySlack) {
      rest = T;
      more = 0;
      ctas = early;
      div = a.early_div;
    }
    if (rest < (1ll << 31)) per = div((int)rest);  // always, but for caches of terabytes
    else per = rest / ctas;
    extra = rest - per * ctas;
  }
  __device__ __forceinline__ long long begin(int w) const {
    const int c = min(w, ctas);
    return c * per + min((long long)c, extra) + min(w, early) * more;
  }
  // the CTA from w on that has step t
  __device__ __forceinline__ int owner(int w, long long t) const {
    int lo = w, hi = ctas;  // begin(lo) <= t < begin(hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (begin(mid) <= t) lo = mid;
      else hi = mid;
    }
    return lo;
  }
};

// A unit's steps: one per tile and kUnitSteps for what it costs to begin and
// end one (queries, merge, output); its tiles are its last steps.
__device__ __forceinline__ int unit_steps(int keys, int bk) { return keys > 0 ? (keys + bk - 1) / bk + kUnitSteps : 0; }

// The share of a CTA, and where its first step lies.
struct Share {
  long long left;  // steps
  long long at;    // first step among all
  long long T;     // all steps
  int seq;         // sequence of the first step
  int head, step;  // K/V head and step within the unit
};

// Found by one warp: each lane adds up the steps of a run of sequences.
template <class C>
__device__ __forceinline__ Share find_share(const PagedDecodeArgs& a, int lane) {
  const int chunk = (a.n_seq + 31) >> 5;
  const int s0 = min(lane * chunk, a.n_seq), s1 = min(s0 + chunk, a.n_seq);
  long long sum = 0;
  for (int s = s0; s < s1; ++s) sum += unit_steps(seq_keys(a, s), C::BK);
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  const int Hkv = a.pool.kv_heads;
  Share sh;
  sh.T = __shfl_sync(kFull, incl, 31) * Hkv;
  const Cut cut(a, sh.T);
  sh.at = cut.begin(blockIdx.x);
  sh.left = cut.begin(blockIdx.x + 1) - sh.at;
  const long long hi = incl * Hkv, lo = hi - sum * Hkv;
  const bool here = lo <= sh.at && sh.at < hi;  // the first step lies in this lane's sequences
  int seq = 0, head = 0, step = 0;
  if (here) {
    long long at = sh.at - lo;
    for (int s = s0; s < s1; ++s) {
      const int n = unit_steps(seq_keys(a, s), C::BK);
      const long long all = (long long)n * Hkv;
      if (at < all) {
        head = all < (1ll << 31) ? (int)at / n : (int)(at / n);
        step = (int)(at - (long long)head * n);
        seq = s;
        break;
      }
      at -= all;
    }
  }
  const unsigned who = __ballot_sync(kFull, here);
  const int src = who ? __ffs(who) - 1 : 0;
  sh.seq = __shfl_sync(kFull, seq, src);
  sh.head = __shfl_sync(kFull, head, src);
  sh.step = __shfl_sync(kFull, step, src);
  return sh;
}

// Walks a share unit by unit; the producer and the consumers walk alike. A
// piece may hold no tile (a share that ends before a unit's first one).
struct Walk {
  Share sh;
  int len, tiles, next_len;

  __device__ __forceinline__ void load(const PagedDecodeArgs& a, int bk) {
    tiles = (len + bk - 1) / bk;
    next_len = sh.seq + 1 < a.n_seq ? seq_keys(a, sh.seq + 1) : 0;  // on its way while this one is worked on
  }
  // false: nothing to do
  __device__ __forceinline__ bool begin(const PagedDecodeArgs& a, const Share& s, int bk) {
    sh = s;
    if (sh.left <= 0) return false;
    len = seq_keys(a, s.seq);
    load(a, bk);
    return tile_count() > 0 || advance(a, bk);
  }
  __device__ __forceinline__ int first_tile() const { return max(0, sh.step - kUnitSteps); }
  __device__ __forceinline__ int tile_count() const {
    const long long end = sh.left < tiles + kUnitSteps - sh.step ? sh.step + sh.left : tiles + kUnitSteps;
    return max(0, (int)end - kUnitSteps) - first_tile();
  }
  // first step of this unit among all
  __device__ __forceinline__ long long unit_at() const { return sh.at - sh.step; }
  // to the next piece with a tile; false at the share's end
  __device__ __forceinline__ bool advance(const PagedDecodeArgs& a, int bk) {
    do {
      const int n = tiles + kUnitSteps - sh.step;
      sh.left -= n;
      sh.at += n;
      sh.step = 0;
      if (sh.left <= 0) return false;
      if (++sh.head >= a.pool.kv_heads) {
        sh.head = 0;
        do {
          if (++sh.seq >= a.n_seq) return false;
          len = next_len;
          load(a, bk);
        } while (len == 0);
      }
    } while (tile_count() <= 0);
    return true;
  }
};

// Slot of the partial result of a unit's piece in CTA w. A piece that begins its unit and
// does not end it: the CTA's second slot; one that continues a unit: the
// first. Units of one piece that still need a merge (with a prefix's part)
// have slots of their own behind those.
__device__ __forceinline__ long long part_slot(const PagedDecodeArgs& a, int w, bool begins, bool ends, long long unit) {
  if (begins && ends) return 2ll * a.ctas + unit;
  return 2ll * w + (begins ? 1 : 0);
}

// All rows of sequence s: no key, so O = 0 and LSE = -inf.
template <int D>
__device__ __noinline__ void empty_rows(const PagedDecodeArgs& a, int s, int thread, int threads) {
  const int Hq = a.pool.kv_heads * a.G, rows = Hq * a.Nq;
  for (long long e = thread; e < (long long)rows * (D / 8); e += threads) {
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
  // Launched while the kernel before it may still run: nothing of global
  // memory is read or written before that one's end (a prefix's kernel of its
  // own has waited for it), but the tables may come into L2: length, page and
  // keys are three dependent look-ups. The merge kernel is set up in the same
  // way meanwhile.
  {
    const long long line = (long long)blockIdx.x * C::THREADS + threadIdx.x;
    const char* const lens = reinterpret_cast<const char*>(a.seq_lens);
    const char* const tables = reinterpret_cast<const char*>(a.block_tables);
    if (line * 128 < (long long)a.B * a.max_pages * 4) prefetch_l2(tables + line * 128);
    if (line * 128 < (long long)a.B * 4) prefetch_l2(lens + line * 128);
  }
  if (a.pre_splits == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int Hkv = a.pool.kv_heads, R = a.G * a.Nq;
  RowInfo* row_info = reinterpret_cast<RowInfo*>(smem + C::OFF_ROWS);
  Share* shared_share = reinterpret_cast<Share*>(smem + C::OFF_SHARE);
  if (warp == 0) {
    const Share found = find_share<C>(a, lane);
    if (lane == 0) *shared_share = found;
  } else {
    for (int e = threadIdx.x - 32; e < (a.prefix_len > 0 ? 2 : 1) * 16 * MT; e += C::THREADS - 32) {
      const int p = e & (16 * MT - 1);
      const int b = e < 16 * MT ? 0 : a.rows_div(p), r = p - b * R, g = a.nq_div(r), i = r - g * a.Nq;
      row_info[e] = RowInfo{b * a.q_b + g * a.q_h + i * a.q_r, b * a.o_b + g * a.o_h + i * a.o_r,
                            e < 16 * MT ? a.Nq - 1 - i : 0};
    }
  }
  __syncthreads();
  Walk wk;
  const bool any = wk.begin(a, *shared_share, C::BK);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0 && a.prefix_len == 0) a.begun[blockIdx.x] = make_int2(-1, 0);
    if (!any) return;
    const int nbox = C::BK >> a.box_shift;    // boxes of a chunk's 64 rows
    const bool mine = lane < nbox * 2 * C::CH;
    const int box = lane & (nbox - 1), col = lane >> (6 - a.box_shift);  // this lane's box; keys' chunks, then values'
    const bool is_v = col >= C::CH;
    const int chunk = is_v ? col - C::CH : col;
    const CUtensorMap* map = is_v ? &a.tmV : &a.tmK;
    const uint32_t dst0 = sbase + (is_v ? C::KV : 0) + chunk * C::CHUNK + ((box * 128) << a.box_shift);
    if (lane == 0) {
      tma_prefetch_desc(&a.tmK);
      tma_prefetch_desc(&a.tmV);
    }
    const Cut cut(a, wk.sh.T);
    // a tile's boxes, and page, row and head of this lane's; looked up one
    // tile ahead, across units too
    struct Tile {
      int boxes, page, row, head;
    };
    auto look_up = [&](int tile) {
      Tile t;
      const int key0 = tile * C::BK, left = wk.len - key0;
      t.boxes = left >= C::BK ? nbox : (left + (1 << a.box_shift) - 1) >> a.box_shift;
      t.page = -1;
      t.row = 0;
      t.head = wk.sh.head;
      if (mine && box < t.boxes) {
        const int* table = wk.sh.seq < a.B ? a.block_tables + (long long)wk.sh.seq * a.max_pages : a.prefix_pages;
        const int key = key0 + (box << a.box_shift), pi = a.page_div(key);
        t.row = key - pi * a.pool.page_size;
        t.page = __ldg(table + pi);
      }
      return t;
    };
    int tile = wk.first_tile(), tile_end = tile + wk.tile_count(), it = 0;
    Tile t = look_up(tile);
    for (bool more = true; more; ++it) {
      if (tile == 0 && lane == 0) {
        // this CTA begins the unit; the one that has its last step ends it
        const long long end = wk.unit_at() + kUnitSteps + wk.tiles;
        const bool whole = end <= wk.sh.at + wk.sh.left;
        if (a.prefix_len > 0 || !whole) {
          const int unit = wk.sh.seq * Hkv + wk.sh.head, last = whole ? (int)blockIdx.x : cut.owner(blockIdx.x, end - 1);
          if (a.prefix_len > 0) a.unit_ctas[unit] = make_int2(blockIdx.x, last);
          else a.begun[blockIdx.x] = make_int2(unit, last);
        }
      }
      if (++tile == tile_end) {
        more = wk.advance(a, C::BK);
        tile = wk.first_tile();
        tile_end = tile + wk.tile_count();
      }
      const Tile next = more ? look_up(tile) : t;
      const int s = it % C::STAGES;
      if (!mbar_wait_warp(EMPTY(s), ((it / C::STAGES) & 1) ^ 1, a.status, a.wait_limit_ns)) break;
      if (lane == 0) mbar_arrive_expect_tx(FULL(s), (uint32_t)((t.boxes * 128 * 2 * C::CH) << a.box_shift));
      __syncwarp();
      if (mine && box < t.boxes) {
        if (t.page < 0 || t.page >= a.pool.num_pages) {
          report_status(a.status, kStatusBadSeqlens);
          t.page = a.pool.num_pages;  // outside the tensor: reads as zeros
        }
        tma_load_4d(dst0 + s * C::STAGE, map, FULL(s), chunk * 64, t.row, t.head, t.page);
      }
      t = next;
    }
    // copies in flight land before the CTA ends, also when a wait ran out
    for (int u = it - C::STAGES < 0 ? 0 : it - C::STAGES; u < it; ++u)
      mbar_wait_warp(FULL(u % C::STAGES), (u / C::STAGES) & 1, a.status, a.wait_limit_ns);
    return;
  }

  // -------------------------------------------------------------- consumers
  // After a wait ran out a warp goes on without waiting or computing, so that
  // it still reaches every barrier; the status word tells.
  const int cw = warp - 1, mt = cw >> 2, kw = cw & 3;
  const int g = lane >> 2, q = lane & 3;
  const int ct = kw * 32 + lane;  // thread of the 16 rows' 128
  const float c2 = a.scale_log2;
  const int ra = mt * 16 + g, rb = ra + 8;  // this lane's query rows
  float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML) + mt * 64;  // [4][16]
  const uint32_t k_off = (uint32_t)((kw * 16 + (lane >> 4) * 8 + (lane & 7)) * 128);
  const uint32_t v_off = (uint32_t)(C::KV + (kw * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * 128);
  const uint32_t k_u = (lane >> 3) & 1, v_u = lane >> 4, sw = lane & 7;
  // A unit's 16 query rows, D / 8 vectors each, vector u of row r at u ^ (r & 7)
  const uint32_t q_buf = sbase + C::OFF_Q + mt * 16 * D * 2;
  const uint32_t q_off = (uint32_t)((((lane >> 3) & 1) * 8 + (lane & 7)) * D * 2), q_u = lane >> 4;
  auto fetch_q = [&](int seq, int head, int buf) {
    const bool pre = seq >= a.B;
    const int rows = pre ? a.B * R : R;
    const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(a.Q) + (pre ? 0 : seq * a.q_b) + (long long)head * a.G * a.q_h;
#pragma unroll
    for (int e = ct; e < 16 * (D / 8); e += 128) {
      const int r = e / (D / 8), u = e - r * (D / 8);
      const bool valid = mt * 16 + r < rows;
      const __nv_bfloat16* src = base + (valid ? row_info[(pre ? 16 * MT : 0) + mt * 16 + r].q + u * 8 : 0);
      copy16(q_buf + buf * C::QBUF + r * (D * 2) + ((u ^ (r & 7)) << 4), src, valid);
    }
  };
  if (any) fetch_q(wk.sh.seq, wk.sh.head, 0);
  if (a.prefix_len == 0) {
    // rows of sequences without keys
    for (int s = blockIdx.x; s < a.B; s += gridDim.x)
      if (seq_keys(a, s) == 0) empty_rows<D>(a, s, threadIdx.x - 32, C::THREADS - 32);
  }
  bool ok = true;
  int it = 0, qb = 0;
  for (bool more = any; more; qb ^= 1) {
    const int n = wk.tile_count(), first = wk.first_tile(), seq = wk.sh.seq, head = wk.sh.head, len = wk.len;
    const bool begins = first == 0, ends = first + n == wk.tiles;
    const bool pre = seq >= a.B;
    const int rows = pre ? a.B * R : R;
    const RowInfo* info = row_info + (pre ? 16 * MT : 0);
    const int seen = pre ? len : max(0, len - a.Nq + 1);  // keys that every row sees
    const bool active = mt * 16 < rows;                   // else these warps only keep step
    copies_done();
    named_bar(1 + mt, 128);  // this unit's queries are there; the other buffer has been read
    uint32_t qf[C::Q_IN_SMEM ? C::FB : D / 16][4];
    if constexpr (!C::Q_IN_SMEM) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) ldmatrix4(qf[ks], q_buf + qb * C::QBUF + q_off + (((2 * ks + q_u) ^ sw) << 4));
    }
    more = wk.advance(a, C::BK);
    if (more) fetch_q(wk.sh.seq, wk.sh.head, qb ^ 1);
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
        // scores in two chains of products, each half of the head
        float x[2][4], y[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) x[t][c] = y[t][c] = 0.f;
        auto k_at = [&](int ks) { return st + k_off + (ks >> 2) * C::CHUNK + ((((2 * ks + k_u) & 7) ^ sw) << 4); };
        auto v_at = [&](int np) { return st + v_off + (np >> 2) * C::CHUNK + ((((2 * np + v_u) & 7) ^ sw) << 4); };
        constexpr int FB = C::FB;  // fragments loaded at a time
        uint32_t f[FB][4];         // of K, then of V
#pragma unroll
        for (int k1 = 0; k1 < D / 16; k1 += FB) {
#pragma unroll
          for (int i = 0; i < FB; ++i) ldmatrix4(f[i], k_at(k1 + i));
          if constexpr (C::Q_IN_SMEM) {
#pragma unroll
            for (int i = 0; i < FB; ++i) ldmatrix4(qf[i], q_buf + qb * C::QBUF + q_off + (((2 * (k1 + i) + q_u) ^ sw) << 4));
          }
#pragma unroll
          for (int i = 0; i < FB; ++i) {
            const uint32_t(&qk)[4] = qf[C::Q_IN_SMEM ? i : k1 + i];
            mma16816((k1 + i) & 1 ? y[0] : x[0], qk, f[i][0], f[i][1]);
            mma16816((k1 + i) & 1 ? y[1] : x[1], qk, f[i][2], f[i][3]);
          }
        }
        // the first values are on their way while the weights are computed
#pragma unroll
        for (int i = 0; i < FB; ++i) ldmatrix4_t(f[i], v_at(i));
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) x[t][c] += y[t][c];
        const bool edge = k0 + 16 > seen;  // some key of this warp is hidden from some row
        int lim_a = len, lim_b = len;      // keys that rows ra and rb see
        if (edge) {
          lim_a -= ra < rows ? info[ra].hidden : 0;
          lim_b -= rb < rows ? info[rb].hidden : 0;
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
        for (int n1 = 0; n1 < D / 16; n1 += FB) {
          if (n1 > 0) {
#pragma unroll
            for (int i = 0; i < FB; ++i) ldmatrix4_t(f[i], v_at(n1 + i));
          }
#pragma unroll
          for (int i = 0; i < FB; ++i) {
            if (edge) {
              f[i][0] &= keep0;
              f[i][1] &= keep1;
              f[i][2] &= keep0;
              f[i][3] &= keep1;
            }
            mma16816(acc[2 * (n1 + i)], pf, f[i][0], f[i][1]);
            mma16816(acc[2 * (n1 + i) + 1], pf, f[i][2], f[i][3]);
          }
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

    if (!active) continue;
    // the four warps of each 16 rows meet in shared memory: maxima, sums and
    // outputs as they are, weighted and added by whoever writes them out
    l_a += __shfl_xor_sync(kFull, l_a, 1);
    l_b += __shfl_xor_sync(kFull, l_b, 1);
    l_a += __shfl_xor_sync(kFull, l_a, 2);
    l_b += __shfl_xor_sync(kFull, l_b, 2);
    if (q == 0) {
      ml[kw * 16 + g] = make_float2(m_a, l_a);
      ml[kw * 16 + g + 8] = make_float2(m_b, l_b);
    }
    const int last_stage = (it - 1) % C::STAGES;
    uint8_t* om = smem + (C::MERGE_IN_STAGE ? last_stage * C::STAGE : C::OFF_MERGE + mt * C::MERGE);
    // Column c of row r of warp w. In the stage a warp takes the place of its
    // own 16 keys and values (nobody else reads those): 32 columns per chunk.
    // 16-byte (32-byte) units permuted by the row, so that the eight rows of a
    // store differ in banks.
    auto om_at = [&](int w, int r, int c) {
      if (C::MERGE_IN_STAGE) return om + (c >> 5) * C::CHUNK + w * 2048 + r * 128 + (((c & 31) * 4) ^ ((r & 7) << 4));
      return om + ((w * 16 + r) * C::DW + (c ^ ((8 * r) & 56 & (C::DW - 1)))) * 4;
    };
    const long long unit = (long long)seq * Hkv + head;
    const bool direct = begins && ends && a.prefix_len == 0;
    const long long part_row = part_slot(a, blockIdx.x, begins, ends, unit) * a.slot_rows;
    const long long o_unit = (pre ? 0 : seq * a.o_b) + (long long)head * a.G * a.o_h;
    constexpr int DW = C::DW;
    const int group_rows = min(16, rows - mt * 16);
#pragma unroll
    for (int d0 = 0; d0 < D; d0 += DW) {
      if (d0 > 0) named_bar(1 + mt, 128);  // the columns before these have been read
      if (g < group_rows) {
#pragma unroll
        for (int nn = 0; nn < DW / 8; ++nn) {
          const float* x = acc[d0 / 8 + nn];
          *reinterpret_cast<float2*>(om_at(kw, g, 8 * nn + 2 * q)) = make_float2(x[0], x[1]);
        }
      }
      if (g + 8 < group_rows) {
#pragma unroll
        for (int nn = 0; nn < DW / 8; ++nn) {
          const float* x = acc[d0 / 8 + nn];
          *reinterpret_cast<float2*>(om_at(kw, g + 8, 8 * nn + 2 * q)) = make_float2(x[2], x[3]);
        }
      }
      named_bar(1 + mt, 128);
      for (int e = ct; e < group_rows * (DW / 4); e += 128) {
        const int r = e / (DW / 4), c = (e - r * (DW / 4)) * 4;
        const int rr = mt * 16 + r;
        float2 t[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) t[w] = ml[w * 16 + r];
        const float mm = fmaxf(fmaxf(t[0].x, t[1].x), fmaxf(t[2].x, t[3].x));
        const float mu = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float f = ex2_approx(t[w].x - mu);
          const float4 z = *reinterpret_cast<const float4*>(om_at(w, r, c));
          ll = fmaf(t[w].y, f, ll);
          y.x = fmaf(z.x, f, y.x);
          y.y = fmaf(z.y, f, y.y);
          y.z = fmaf(z.z, f, y.z);
          y.w = fmaf(z.w, f, y.w);
        }
        const float inv = ll == 0.f ? 0.f : __fdividef(1.f, ll);
        y.x *= inv;
        y.y *= inv;
        y.z *= inv;
        y.w *= inv;
        const float lse = ll == 0.f ? -INFINITY : mm + __log2f(ll);
        if (direct) {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.O) + o_unit + info[rr].o + d0 + c;
          *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
          if (d0 + c == 0) a.LSE[unit * R + rr] = lse * kLn2;
        } else {
          *reinterpret_cast<float4*>(a.Opart + (part_row + rr) * D + d0 + c) = y;
          if (d0 + c == 0) a.Lpart[part_row + rr] = lse;
        }
      }
    }
    if (C::MERGE_IN_STAGE) {
      fence_proxy_async_smem();  // the stage's next writer is the TMA
      __syncwarp();
      if (lane == 0) mbar_arrive(EMPTY(last_stage));
    }
  }
  // a prefix's kernel ends before this one does, so the merge sees both; one
  // CTA waits for that, the others make room
  if (blockIdx.x + 1 == gridDim.x) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Rows of units that were not written out directly: partial results of the
// own keys (and of the prefix) merged by maximum and sum, in order of the
// CTAs. WPR warps share a row, each taking every WPR-th partial result, and
// meet in shared memory: without a prefix few rows have parts, but a long
// sequence has one from each of many CTAs (WPR = 8); with one every row has
// parts, as many as the prefix has key ranges (WPR = 1 up to 16, else 8).
constexpr int kMergeWarps = 8;
template <int D, int WPR, bool PREFIX>
__global__ void __launch_bounds__(32 * kMergeWarps) decode_merge_kernel(const __grid_constant__ PagedDecodeArgs a) {
  constexpr int E = D / 32;
  constexpr int AHEAD = 4;  // partial results in flight per warp
  __shared__ float sm[kMergeWarps], sl[kMergeWarps], so[kMergeWarps][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!PREFIX) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % WPR;
  const int Hkv = a.pool.kv_heads, R = a.G * a.Nq;
  const unsigned item = blockIdx.x * (kMergeWarps / WPR) + warp / WPR;
  const unsigned group = item / (unsigned)R;
  const int r = (int)(item - group * (unsigned)R);
  int unit, own_first, own_n, pre_first = 0, pre_n = 0;
  long long pre_row = 0;  // a prefix's kernel of its own: row of the first part, parts 256 rows apart
  int b, head;
  if (!PREFIX) {
    // without a prefix only the units that a share's end cuts have parts
    const int2 c = a.begun[group];
    if (c.x < 0) return;  // the whole block
    unit = c.x;
    own_first = (int)group;
    own_n = c.y - own_first + 1;
    b = unit / Hkv;
    head = unit - b * Hkv;
  } else {
    if (item >= (unsigned)(a.B * Hkv) * (unsigned)R) return;  // the whole block, if its warps share a row
    unit = (int)group;
    b = unit / Hkv;
    head = unit - b * Hkv;
    const int2 c = a.unit_ctas[unit];  // not written for a sequence without keys
    own_first = c.x;
    own_n = seq_keys(a, b) > 0 ? c.y - c.x + 1 : 0;
    if (a.pre_splits > 0) {
      const int rr = b * R + r, qblocks = (a.B * R + 255) / 256;
      pre_n = a.pre_splits;
      pre_row = ((long long)head * qblocks + rr / 256) * a.pre_splits * 256 + rr % 256;
    } else {
      const int2 cp = a.unit_ctas[a.B * Hkv + head];
      pre_first = cp.x;
      pre_n = cp.y - cp.x + 1;
    }
  }
  float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  const int n = own_n + pre_n;
  for (int p0 = part; p0 < n; p0 += AHEAD * WPR) {
    float L[AHEAD], x[AHEAD][E];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int p = p0 + k * WPR;
      L[k] = -INFINITY;
#pragma unroll
      for (int e = 0; e < E; ++e) x[k][e] = 0.f;
      if (p >= n) continue;
      const bool own = p < own_n;
      const int i = own ? p : p - own_n;
      const float* O = a.Opart;
      const float* Ls = a.Lpart;
      long long row;
      if (own || a.pre_splits == 0) {
        const int u = own ? unit : a.B * Hkv + head;
        const long long slot = part_slot(a, (own ? own_first : pre_first) + i, i == 0, i + 1 == (own ? own_n : pre_n), u);
        row = slot * a.slot_rows + (own ? r : b * R + r);
      } else {
        O = a.pre_Opart;
        Ls = a.pre_Lpart;
        row = pre_row + 256ll * i;
      }
      L[k] = Ls[row];
      const float* src = O + row * D + lane * E;
      if constexpr (E == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        x[k][0] = v.x; x[k][1] = v.y; x[k][2 % E] = v.z; x[k][3 % E] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        x[k][0] = v.x; x[k][1] = v.y;
      }
    }
    float mn = m;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) mn = fmaxf(mn, L[k]);
    const float mu = mn == -INFINITY ? 0.f : mn;
    const float f = ex2_approx(m - mu);
    m = mn;
    l *= f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= f;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const float w = ex2_approx(L[k] - mu);
      l += w;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w, x[k][e], acc[e]);
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
    __syncthreads();
    if (warp != 0) return;
    m = -INFINITY;
#pragma unroll
    for (int w = 0; w < WPR; ++w) m = fmaxf(m, sm[w]);
    const float mu = m == -INFINITY ? 0.f : m;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      const float f = ex2_approx(sm[w] - mu);
      l = fmaf(sl[w], f, l);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(so[w][lane * E + e], f, acc[e]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int g = r / a.Nq, i = r - g * a.Nq, hq = head * a.G + g;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.O) + b * a.o_b + hq * a.o_h + i * a.o_r + lane * E;
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2 % E] * inv, acc[3 % E] * inv));
  else
    *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (lane == 0) a.LSE[(long long)unit * R + r] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
}

template <int D, int MT>
cudaError_t launch(const PagedDecodeArgs& a, cudaStream_t st) {
  using C = Cfg<D, MT>;
  // programmatic dependent launches: each kernel is set up while the one
  // before it runs; the own keys' kernel takes the SMs that a prefix's kernel
  // leaves idle (and waits for that kernel's end before its own). The first
  // kernel of a call with a prefix is launched plainly: 1 to 7 us better when
  // calls follow one another.
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = a.prefix_len == 0 || a.pre_splits > 0 ? 1 : 0;
  cfg.gridDim = dim3((unsigned)a.ctas);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM_ALLOC;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_paged_kernel<D, MT>, a);
  if (e != cudaSuccess) return e;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.dynamicSmemBytes = 0;
  const unsigned rows = (unsigned)(a.G * a.Nq);
  if (a.prefix_len == 0) {
    cfg.gridDim = dim3((unsigned)a.ctas * rows);
    return cudaLaunchKernelEx(&cfg, decode_merge_kernel<D, kMergeWarps, false>, a);
  }
  const unsigned all = (unsigned)(a.B * a.pool.kv_heads) * rows;
  // parts of a prefix that is part of the grid: about one per CTA and head
  const int parts = a.pre_splits > 0 ? a.pre_splits : a.ctas / a.pool.kv_heads;
  if (parts > 16) {
    cfg.gridDim = dim3(all);
    return cudaLaunchKernelEx(&cfg, decode_merge_kernel<D, kMergeWarps, true>, a);
  }
  cfg.gridDim = dim3((all + kMergeWarps - 1) / kMergeWarps);
  return cudaLaunchKernelEx(&cfg, decode_merge_kernel<D, 1, true>, a);
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
  L.total = L.pre_opart = L.begun + up256((size_t)L.ctas * sizeof(int2));
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

PrefixPlan plan_prefix_beside(int B, int rows, int Hkv, int prefix_len, int d, int max_splits, int ctas, int sms,
                              int own_keys) {
  // Times in us, measured on a GB300: a prefix's CTA takes kStart and, per tile
  // of 128 keys, 1.76 (two tiles of query rows) or 1.05 (one), two thirds of
  // that at d = 64. An own keys' CTA beside it takes kOwnStart and 0.75 per
  // step of 32 KB, or what all such CTAs' bytes take at 6 GB/ms; one that finds
  // its SM only after the prefix's costs kLate before the rest goes on.
  constexpr double kStart = 11.0, kOwnStart = 2.0, kStep = 0.75, kLate = 4.0, kStepAll = 32768.0 / 6e6;
  const int n_kv = (int)(((long long)prefix_len + 127) / 128);
  const long long units = ((long long)B * rows + 255) / 256 * Hkv;
  const double tile = ((long long)B * rows > 128 ? 1.76 : 1.05) * (d == 128 ? 1.0 : 0.67);
  const double steps = (double)B * Hkv * (own_keys * (double)d / 8192.0 + kUnitSteps + 0.5);
  PrefixPlan best{max_splits, 0, 0};
  double best_us = -1;
  for (int s = 1; s <= max_splits; ++s) {
    const long long waves = (units * s + sms - 1) / sms;
    const double pre_us = kStart + (double)waves * ((n_kv + s - 1) / s) * tile;
    const int early = waves == 1 ? (sms - (int)(units * s)) * (ctas / sms) : 0;
    const double step = early * kStepAll > kStep ? early * kStepAll : kStep;
    const int more = early > 0 && pre_us > kOwnStart ? (int)((pre_us - kOwnStart) / step) : 0;
    double us = pre_us;
    if (early > 0 && steps <= early * (double)(more + kEarlySlack)) {
      const double own_us = kOwnStart + steps / early * step;
      us = own_us > us ? own_us : us;
    } else {
      us += kLate + (steps - early * (double)more) * kStepAll;
    }
    if (best_us < 0 || us < best_us) {
      best_us = us;
      best = PrefixPlan{s, early, more};
    }
  }
  return best;
}

cudaError_t launch_decode_paged_bf16(const PagedDecodeArgs& a, int d, cudaStream_t st) {
  if (a.ctas < 1) return cudaErrorInvalidValue;
  if (d == 128) {
    if (a.slot_rows == 16) return launch<128, 1>(a, st);
    if (a.slot_rows == 32) return launch<128, 2>(a, st);
    return launch<128, 4>(a, st);
  }
  if (d == 64) {
    if (a.slot_rows == 16) return launch<64, 1>(a, st);
    if (a.slot_rows == 32) return launch<64, 2>(a, st);
    return launch<64, 4>(a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa

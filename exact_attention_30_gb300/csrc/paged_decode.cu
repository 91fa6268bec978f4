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
// workspace, at most two per CTA, and a second kernel combines them in a
// fixed order (results do not depend on timing). A unit that lies in one share
// is written out directly.
//
// A shared prefix with no more rows than fit a unit (those of every sequence,
// B * R <= 32 per K/V head) is one more sequence of the same grid. With more
// rows it is a matrix product of its own (launch_prefix_bf16), and only its
// partial results meet the own keys' here.
//
// CTA: one producer warp and four consumer warps per 16 (or 8) query rows. The
// producer reads page numbers a tile ahead and lets each lane issue one TMA box
// (64 columns of up to 64 rows of one page) into a ring of tiles. Consumer warp
// kw owns keys 16 kw .. 16 kw + 15 of every tile and keeps its own running
// maximum, sum and output in registers: no exchange between warps until the
// piece ends. Bytes bound this kernel (4 d bytes per key against 4 d R flops):
// with keys split over warps the warp-level mma.sync needs no barrier and no
// tensor-memory round trip per tile, which is what a short cache's latency
// consists of. Up to 16 rows its rate is far from the limit, and two CTAs share an
// SM, one loading while the other one merges; with 17 to 32 a tile's products take
// 1.0 us against 0.73 for its bytes, and they bound the kernel.
//
// Measured on a GB300, GPU time of a call: 8 sequences of 32768 keys (8 heads,
// 8 queries each, d = 128) 163 us, 6.6 TB/s, 97% of a copy's rate; 48 of 100
// to 9000 keys (8 heads, 4 queries each) 77 us, 6.1 TB/s. The same kernel
// that loads and does not compute takes 162 and 77: loads, not products, bound
// long caches. 20 sequences of 333 to 4097 keys (16 heads, 4 new tokens,
// d = 64) 26 us against 18 for the bytes; without arithmetic as well, so it is the
// loading that is slow there (4.7 TB/s). One sequence of 701 keys 7.4 us: about
// 4 us of the chain length - page - keys and 2 us of merge.
//
// More than 32 rows are two units, the second of which finds the keys in L2: 32
// units of 16384 keys 95 us with 64 rows, 54 with 32, 51 with 16, 47 with 4.
//
// Tried and slower: 64 rows in one unit (16 consumer warps of 112 registers, 211
// us for those); tiles of 128 keys at d = 64 (27 -> 32 us); the merge done
// by the last CTA of a unit, by a ticket (one sequence 7.7 -> 13 us); 32 keys
// per warp, pairs of warps on alternate tiles (long 164 -> 178 us); a ring and
// a share for every warp (long 165 -> 192 us: the TMA takes over 100 cycles per
// box, and consumers that issue wait for it).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

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

// ROWS: query rows of a unit, 8, 16 or 32 (fewer are padded). BESIDE: on
// the few SMs that a prefix's kernel leaves, where the latency of units bounds
// the own keys rather than memory: three CTAs per SM with two stages each
// (8 rows, whose registers allow it; 128 samples 57.5 -> 54 us): 1 for one new
// token, 2 for several (keys that only some rows see cost registers, which
// spill: 56.8 us). 0, elsewhere: two with three stages, fewer parts to merge (48
// ragged sequences 78.5 against 79.6, 299 of 165 keys 18.3 against 20.2 us).
template <int D_, int ROWS_, int BESIDE>
struct Cfg {
  static constexpr int D = D_, ROWS = ROWS_;
  static constexpr bool MANY_NEW = BESIDE != 1;  // more than one new token: keys that only some rows see
  static constexpr int MT = ROWS < 16 ? 1 : ROWS / 16;  // groups of rows, four consumer warps each
  static constexpr int OWN_ROWS = ROWS == 32 ? kPagedMaxRows : 16;  // query rows of a K/V head
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
  // One group of rows: each warp's output fits the place of its keys and
  // values in the piece's last stage, and several CTAs share an SM, one loading
  // while another one merges. More rows: space of its own, one CTA.
  static constexpr bool MERGE_IN_STAGE = MT == 1;
  static constexpr int CTAS = MT > 1 ? 1 : BESIDE ? 3 : 2;
  static constexpr int STAGES = (MT == 2 ? 4 : BESIDE ? 2 : 3) * (D == 128 ? 1 : 2);
  static_assert(!BESIDE || ROWS == 8, "registers");
  // Queries as fragments in registers, or read from shared memory per tile (16
  // rows, 32 at d = 128: 1 to 4% faster than in registers, which then spill).
  // FB: K or V fragments loaded at a time.
  static constexpr bool Q_IN_SMEM = ROWS == 16 || (ROWS == 32 && D == 128);
  static constexpr int FB = 4;
  static constexpr int QBUF = 16 * MT * D * 2;  // a unit's queries; two, one being filled for the next unit
  static constexpr int OFF_MERGE = STAGES * STAGE;
  static constexpr int OFF_Q = OFF_MERGE + (MERGE_IN_STAGE ? 0 : MT * MERGE);
  static constexpr int OFF_ML = OFF_Q + 2 * QBUF;               // fp32 m, l [MT][4][16]
  static constexpr int OFF_ROWS = OFF_ML + MT * 4 * 16 * 8;     // RowInfo [OWN_ROWS], prefix's [16 MT]
  static constexpr int OFF_SHARE = OFF_ROWS + (OWN_ROWS + 16 * MT) * 24;  // the CTA's Share
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
// An 8 x 8 matrix of 16-bit elements, one pair per lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
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
  const int n = a.seq_lens[s];
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

// Which of a pair of values, of keys k and k + 1, are of the first n keys.
__device__ __forceinline__ uint32_t keep_pair(int k, int n) { return (k < n ? 0xffffu : 0u) | (k + 1 < n ? 0xffff0000u : 0u); }

// Top bits of those halves of a pair of bf16 that are infinite or NaN.
__device__ __forceinline__ uint32_t non_finite(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// The newest keys (seen .. len - 1) are hidden from some rows, whose weights
// there are zero. Their values go through the product like all others, but
// what is not finite (0 times it is NaN) is taken out of the fragments f, of
// which first and second say what belongs to such keys (each register is a pair
// of keys: of the first eight at even places, or in the first half of four).
// True if there was any in the warp.
template <int FB, bool ODD_IS_SECOND>
__device__ __forceinline__ bool take_out(uint32_t (&f)[FB][4], uint32_t first, uint32_t second) {
  uint32_t hit = 0;
#pragma unroll
  for (int i = 0; i < FB; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) hit |= non_finite(f[i][e]) & ((ODD_IS_SECOND ? e & 1 : e >> 1) ? second : first);
  if (!__any_sync(kFull, hit != 0)) return false;
#pragma unroll
  for (int i = 0; i < FB; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      f[i][e] &= ~(((non_finite(f[i][e]) >> 15) * 0xffffu) & ((ODD_IS_SECOND ? e & 1 : e >> 1) ? second : first));
  return true;
}

// Steps that an early CTA rather takes on top than leaves to CTAs that start
// after the prefix's kernel (about their start-up time)
constexpr int kEarlySlack = 4;

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

// Units of a sequence. More than 32 rows of a K/V head are several groups, which
// follow one another, so that the second one finds the head's keys in L2.
template <class C>
__device__ __forceinline__ int group_shift(const PagedDecodeArgs& a) {
  return C::ROWS == 32 ? a.group_shift : 0;
}
template <class C>
__device__ __forceinline__ int unit_heads(const PagedDecodeArgs& a) {
  return a.pool.kv_heads << group_shift<C>(a);
}

// A unit's steps: one per tile and kUnitSteps for what it costs to begin and
// end one (queries, merge, output); its tiles are its last steps.
__device__ __forceinline__ int unit_steps(int keys, int bk) { return keys > 0 ? (keys + bk - 1) / bk + kUnitSteps : 0; }

// The share of a CTA, and where its first step lies.
struct Share {
  long long left;  // steps
  long long at;    // first step among all
  long long T;     // all steps
  int seq;         // sequence of the first step
  int head, step;  // unit of the sequence, and step within it
  int empty;       // whether some sequence has no keys
};

// Found by one warp: each lane adds up the steps of a run of sequences.
template <class C>
__device__ __forceinline__ Share find_share(const PagedDecodeArgs& a, int lane) {
  const int chunk = (a.n_seq + 31) >> 5;
  const int s0 = min(lane * chunk, a.n_seq), s1 = min(s0 + chunk, a.n_seq);
  long long sum = 0;
  bool empty = false;
  for (int s = s0; s < s1; ++s) {
    const int n = unit_steps(seq_keys(a, s), C::BK);
    sum += n;
    empty |= n == 0;
  }
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  const int heads = unit_heads<C>(a);
  Share sh;
  sh.T = __shfl_sync(kFull, incl, 31) * heads;
  const Cut cut(a, sh.T);
  sh.at = cut.begin(blockIdx.x);
  sh.left = cut.begin(blockIdx.x + 1) - sh.at;
  const long long hi = incl * heads, lo = hi - sum * heads;
  const bool here = lo <= sh.at && sh.at < hi;  // the first step lies in this lane's sequences
  int seq = 0, head = 0, step = 0;
  if (here) {
    long long at = sh.at - lo;
    for (int s = s0; s < s1; ++s) {
      const int n = unit_steps(seq_keys(a, s), C::BK);
      const long long all = (long long)n * heads;
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
  sh.empty = __any_sync(kFull, empty);
  return sh;
}

// Walks a share unit by unit; the producer and the consumers walk alike. A
// piece may hold no tile (a share that ends before a unit's first one).
template <class C>
struct Walk {
  Share sh;
  int len, tiles, next_len;

  __device__ __forceinline__ void load(const PagedDecodeArgs& a) {
    tiles = (len + C::BK - 1) / C::BK;
    next_len = sh.seq + 1 < a.n_seq ? seq_keys(a, sh.seq + 1) : 0;  // on its way while this one is worked on
  }
  // false: nothing to do
  __device__ __forceinline__ bool begin(const PagedDecodeArgs& a, const Share& s) {
    sh = s;
    if (sh.left <= 0) return false;
    len = seq_keys(a, s.seq);
    load(a);
    return tile_count() > 0 || advance(a);
  }
  __device__ __forceinline__ int first_tile() const { return max(0, sh.step - kUnitSteps); }
  __device__ __forceinline__ int tile_count() const {
    const long long end = sh.left < tiles + kUnitSteps - sh.step ? sh.step + sh.left : tiles + kUnitSteps;
    return max(0, (int)end - kUnitSteps) - first_tile();
  }
  // first step of this unit among all
  __device__ __forceinline__ long long unit_at() const { return sh.at - sh.step; }
  // to the next piece with a tile; false at the share's end
  __device__ __forceinline__ bool advance(const PagedDecodeArgs& a) {
    do {
      const int n = tiles + kUnitSteps - sh.step;
      sh.left -= n;
      sh.at += n;
      sh.step = 0;
      if (sh.left <= 0) return false;
      if (++sh.head >= unit_heads<C>(a)) {
        sh.head = 0;
        do {
          if (++sh.seq >= a.n_seq) return false;
          len = next_len;
          load(a);
        } while (len == 0);
      }
    } while (tile_count() <= 0);
    return true;
  }
};

// Slot of the partial result of a unit's piece in CTA w. A piece that begins its
// unit and does not end it: the CTA's second slot; one that continues a unit:
// the first. Units of one piece that still need a merge (with a prefix's part)
// have slots of their own behind those.
__device__ __forceinline__ long long part_slot(const PagedDecodeArgs& a, int w, bool begins, bool ends, long long unit) {
  if (begins && ends) return 2ll * a.ctas + unit;
  return 2ll * w + (begins ? 1 : 0);
}

// Rows of sequences without keys: O = 0, LSE = -inf. Warp w of n writes those
// of every n-th (sequence, K/V head).
template <int D>
__device__ __noinline__ void empty_rows(const PagedDecodeArgs& a, int w, int n) {
  const int Hkv = a.pool.kv_heads, R = a.G * a.Nq, lane = threadIdx.x & 31;
  constexpr int U = D / 8;  // lanes of a row
  for (int unit = w; unit < a.B * Hkv; unit += n) {
    const int b = unit / Hkv, head = unit - b * Hkv;
    if (seq_keys(a, b) != 0) continue;
    for (int r = lane / U; r < R; r += 32 / U) {
      const int g = a.nq_div(r), i = r - g * a.Nq;
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.O) + b * a.o_b + (long long)(head * a.G + g) * a.o_h + i * a.o_r +
                                (lane & (U - 1)) * 8) = make_uint4(0u, 0u, 0u, 0u);
      if ((lane & (U - 1)) == 0) a.LSE[(long long)unit * R + r] = -INFINITY;
    }
  }
}

// What a consumer warp holds of a unit while it works on its 16 keys of every
// tile: running maximum, sum and unnormalised output of the unit's rows.
// lane = 4 g + q throughout.
//
// Up to 16 rows: S = Q K^T and O = P V with the query rows on the products'
// 16 rows; the scores leave the first product in the layout in which the
// second one takes them.
template <class C>
struct WarpRows16 {
  static constexpr int D = C::D, FB = C::FB;
  static constexpr int ROWS = 16;
  int g, q, kw, ra, rb;                    // ra, rb: this lane's rows of the unit
  uint32_t k_off, v_off, k_u, v_u, sw, q_off, q_u, q_at;
  uint32_t qf[C::Q_IN_SMEM ? FB : D / 16][4];
  float acc[D / 8][4];
  float m_a, m_b, l_a, l_b;

  __device__ __forceinline__ void init(int lane, int kw_, int mt) {
    g = lane >> 2;
    q = lane & 3;
    kw = kw_;
    ra = mt * 16 + g;
    rb = ra + 8;
    k_off = (uint32_t)((kw * 16 + (lane >> 4) * 8 + (lane & 7)) * 128);
    v_off = (uint32_t)(C::KV + (kw * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * 128);
    k_u = (lane >> 3) & 1;
    v_u = lane >> 4;
    sw = lane & 7;
    q_off = (uint32_t)((((lane >> 3) & 1) * 8 + (lane & 7)) * D * 2);
    q_u = lane >> 4;
  }
  __device__ __forceinline__ void load_q(uint32_t (&f)[4], int ks) { ldmatrix4(f, q_at + q_off + (((2 * ks + q_u) ^ sw) << 4)); }
  __device__ __forceinline__ void begin(uint32_t q_smem) {
    q_at = q_smem;
    if constexpr (!C::Q_IN_SMEM) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) load_q(qf[ks], ks);
    }
#pragma unroll
    for (int nn = 0; nn < D / 8; ++nn) acc[nn][0] = acc[nn][1] = acc[nn][2] = acc[nn][3] = 0.f;
    m_a = m_b = -INFINITY;
    l_a = l_b = 0.f;
  }
  // Keys k0 .. k0 + 15 of a unit of `len`, of which every row sees `seen`.
  __device__ __forceinline__ void tile(uint32_t st, const uint8_t* stage, int k0, int len, int seen, const RowInfo* info, int rows,
                                       float c2) {
    // scores in two chains of products, each half of the head
    float x[2][4], y[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) x[t][c] = y[t][c] = 0.f;
    auto k_at = [&](int ks) { return st + k_off + (ks >> 2) * C::CHUNK + ((((2 * ks + k_u) & 7) ^ sw) << 4); };
    auto v_at = [&](int np) { return st + v_off + (np >> 2) * C::CHUNK + ((((2 * np + v_u) & 7) ^ sw) << 4); };
    uint32_t f[FB][4];  // of K, then of V
#pragma unroll
    for (int k1 = 0; k1 < D / 16; k1 += FB) {
#pragma unroll
      for (int i = 0; i < FB; ++i) ldmatrix4(f[i], k_at(k1 + i));
      if constexpr (C::Q_IN_SMEM) {
#pragma unroll
        for (int i = 0; i < FB; ++i) load_q(qf[i], k1 + i);
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
    // values behind the last key stay out of the product (0 times NaN); keys
    // 2q, 2q + 1 and 8 + 2q, 8 + 2q + 1 are this lane's
    const uint32_t keep0 = edge ? keep_pair(k0 + 2 * q, len) : kFull, keep1 = edge ? keep_pair(k0 + 8 + 2 * q, len) : kFull;
    if (C::MANY_NEW && edge && len > seen) {
      newest(stage, k0, len, seen, lim_a, lim_b, keep0, keep1, x, pf, v_at);
      return;
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
  }
  // P V for keys of which some are hidden from some row (more than one new
  // token): apart from the rest, which must not hold its registers.
  template <class At>
  __device__ __forceinline__ void newest(const uint8_t* stage, int k0, int len, int seen, int lim_a, int lim_b, uint32_t keep0, uint32_t keep1,
                                         const float (&x)[2][4], const uint32_t (&pf)[4], const At& v_at) {
    const uint32_t some0 = ~keep_pair(k0 + 2 * q, seen), some1 = ~keep_pair(k0 + 8 + 2 * q, seen);
    bool taken = false;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      uint32_t f[1][4];
      ldmatrix4_t(f[0], v_at(n));
      f[0][0] &= keep0;
      f[0][1] &= keep1;
      f[0][2] &= keep0;
      f[0][3] &= keep1;
      taken |= take_out<1, true>(f, some0, some1);
      mma16816(acc[2 * n], pf, f[0][0], f[0][1]);
      mma16816(acc[2 * n + 1], pf, f[0][2], f[0][3]);
    }
    if (taken) {
      // what was taken out goes to the rows that see it
      for (int k = max(k0, seen); k < min(k0 + 16, len); ++k) {
        const int c = k - k0, src = (g << 2) | ((c & 7) >> 1);
        const float pa = (c & 8) ? ((c & 1) ? x[1][1] : x[1][0]) : ((c & 1) ? x[0][1] : x[0][0]);
        const float pb = (c & 8) ? ((c & 1) ? x[1][3] : x[1][2]) : ((c & 1) ? x[0][3] : x[0][2]);
        const float p_a = __shfl_sync(kFull, pa, src), p_b = __shfl_sync(kFull, pb, src);
        const int r = kw * 16 + c;
        const uint8_t* vr = stage + C::KV + r * 128 + q * 4;
#pragma unroll
        for (int nn = 0; nn < D / 8; ++nn) {
          const uint32_t v2 = *reinterpret_cast<const uint32_t*>(vr + (nn >> 3) * C::CHUNK + (((nn & 7) ^ (r & 7)) << 4));
          const float v0 = __uint_as_float(v2 << 16), v1 = __uint_as_float(v2 & 0xffff0000u);
          if (!isfinite(v0)) {
            if (k < lim_a) acc[nn][0] = fmaf(p_a, v0, acc[nn][0]);
            if (k < lim_b) acc[nn][2] = fmaf(p_b, v0, acc[nn][2]);
          }
          if (!isfinite(v1)) {
            if (k < lim_a) acc[nn][1] = fmaf(p_a, v1, acc[nn][1]);
            if (k < lim_b) acc[nn][3] = fmaf(p_b, v1, acc[nn][3]);
          }
        }
      }
    }
  }
  // Maxima and sums of the rows, [4 warps][16].
  __device__ __forceinline__ void put_sums(float2* ml) {
    l_a += __shfl_xor_sync(kFull, l_a, 1);
    l_b += __shfl_xor_sync(kFull, l_b, 1);
    l_a += __shfl_xor_sync(kFull, l_a, 2);
    l_b += __shfl_xor_sync(kFull, l_b, 2);
    if (q == 0) {
      ml[kw * 16 + g] = make_float2(m_a, l_a);
      ml[kw * 16 + g + 8] = make_float2(m_b, l_b);
    }
  }
  // Column c of row r of warp w's output. In the stage a warp takes the place
  // of its own 16 keys and values (nobody else reads those): 32 columns per
  // chunk. 16-byte (32-byte) units permuted by the row, so that the eight rows
  // of a store differ in banks.
  static __device__ __forceinline__ uint8_t* om_at(uint8_t* om, int w, int r, int c) {
    if (C::MERGE_IN_STAGE) return om + (c >> 5) * C::CHUNK + w * 2048 + r * 128 + (((c & 31) * 4) ^ ((r & 7) << 4));
    return om + ((w * 16 + r) * C::DW + (c ^ ((8 * r) & 56 & (C::DW - 1)))) * 4;
  }
  // Columns d0 .. d0 + DW - 1 of the group's first n rows.
  __device__ __forceinline__ void put_out(uint8_t* om, int d0, int n) {
#pragma unroll
    for (int nn = 0; nn < C::DW / 8; ++nn) {
      // (d0 is a constant in the unrolled caller)
      const float* x = acc[d0 / 8 + nn];
      if (g < n) *reinterpret_cast<float2*>(om_at(om, kw, g, 8 * nn + 2 * q)) = make_float2(x[0], x[1]);
      if (g + 8 < n) *reinterpret_cast<float2*>(om_at(om, kw, g + 8, 8 * nn + 2 * q)) = make_float2(x[2], x[3]);
    }
  }
};

// Up to 8 rows (one new token of up to 8 query heads): S^T = K Q^T and
// O^T = V^T P^T, keys and columns on the products' 16 rows and the query rows
// on their 8 columns, half the products, exponentials and registers of the
// form above. P^T changes layout by a transposition of its 8 x 8 halves.
template <class C>
struct WarpRows8 {
  static constexpr int D = C::D, FB = C::FB;
  static constexpr int ROWS = 8;
  int g, q, kw;                  // this lane's rows: 2q, 2q + 1; its keys of the warp's 16: g, g + 8
  uint32_t k_off, v_off, u_k, u_v, sw, q_off;
  uint32_t qf[D / 32][4];
  float acc[D / 16][4];          // columns 16 i + g (+ 8) of rows 2q, 2q + 1
  float m0, m1, l0, l1;

  __device__ __forceinline__ void init(int lane, int kw_, int) {
    g = lane >> 2;
    q = lane & 3;
    kw = kw_;
    k_off = (uint32_t)((kw * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * 128);
    u_k = lane >> 4;
    v_off = (uint32_t)(C::KV + (kw * 16 + (lane >> 4) * 8 + (lane & 7)) * 128);
    u_v = (lane >> 3) & 1;
    sw = lane & 7;
    q_off = (uint32_t)((lane & 7) * D * 2);
  }
  __device__ __forceinline__ void begin(uint32_t q_smem) {
    const uint32_t u = (uint32_t)((threadIdx.x & 31) >> 3);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) ldmatrix4(qf[i], q_smem + q_off + (((4 * i + u) ^ sw) << 4));
#pragma unroll
    for (int i = 0; i < D / 16; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
  }
  __device__ __forceinline__ void tile(uint32_t st, const uint8_t* stage, int k0, int len, int seen, const RowInfo* info, int rows,
                                       float c2) {
    float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};  // two chains of products
    auto k_at = [&](int ks) { return st + k_off + (ks >> 2) * C::CHUNK + ((((2 * ks + u_k) & 7) ^ sw) << 4); };
    auto v_at = [&](int np) { return st + v_off + (np >> 2) * C::CHUNK + ((((2 * np + u_v) & 7) ^ sw) << 4); };
    uint32_t f[FB][4];  // of K, then of V
#pragma unroll
    for (int k1 = 0; k1 < D / 16; k1 += FB) {
#pragma unroll
      for (int i = 0; i < FB; ++i) ldmatrix4(f[i], k_at(k1 + i));
#pragma unroll
      for (int i = 0; i < FB; ++i) {
        const int ks = k1 + i;
        mma16816(ks & 1 ? y : x, f[i], qf[ks >> 1][2 * (ks & 1)], qf[ks >> 1][2 * (ks & 1) + 1]);
      }
    }
    // the first values are on their way while the weights are computed
#pragma unroll
    for (int i = 0; i < FB; ++i) ldmatrix4_t(f[i], v_at(i));
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] += y[c];
    const bool edge = k0 + 16 > seen;  // some key of this warp is hidden from some row
    int lim0 = len, lim1 = len;        // keys that rows 2q and 2q + 1 see
    if (edge) {
      if (C::MANY_NEW) {
        lim0 -= 2 * q < rows ? info[2 * q].hidden : 0;
        lim1 -= 2 * q + 1 < rows ? info[2 * q + 1].hidden : 0;
      }
      if (k0 + g >= lim0) x[0] = -INFINITY;
      if (k0 + g >= lim1) x[1] = -INFINITY;
      if (k0 + g + 8 >= lim0) x[2] = -INFINITY;
      if (k0 + g + 8 >= lim1) x[3] = -INFINITY;
    }
    float t0 = fmaxf(x[0], x[2]), t1 = fmaxf(x[1], x[3]);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      t0 = fmaxf(t0, __shfl_xor_sync(kFull, t0, o));
      t1 = fmaxf(t1, __shfl_xor_sync(kFull, t1, o));
    }
    t0 *= c2;
    t1 *= c2;
    const bool up0 = t0 > m0 + kRescaleLog2, up1 = t1 > m1 + kRescaleLog2;
    if (__any_sync(kFull, up0 || up1)) {  // always at a row's first key
      const float f0 = up0 ? ex2_approx(m0 - t0) : 1.f, f1 = up1 ? ex2_approx(m1 - t1) : 1.f;
      m0 = up0 ? t0 : m0;
      m1 = up1 ? t1 : m1;
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        acc[i][0] *= f0;
        acc[i][1] *= f1;
        acc[i][2] *= f0;
        acc[i][3] *= f1;
      }
    }
    const float n0 = m0 == -INFINITY ? 0.f : -m0, n1 = m1 == -INFINITY ? 0.f : -m1;
    x[0] = ex2_approx(fmaf(x[0], c2, n0));
    x[1] = ex2_approx(fmaf(x[1], c2, n1));
    x[2] = ex2_approx(fmaf(x[2], c2, n0));
    x[3] = ex2_approx(fmaf(x[3], c2, n1));
    l0 += x[0] + x[2];
    l1 += x[1] + x[3];
    // P is rounded to bf16 for the product (half a step of each weight);
    // the sums l keep the unrounded weights
    const uint32_t b0 = transpose8(pack_bf16x2(x[0], x[1])), b1 = transpose8(pack_bf16x2(x[2], x[3]));
    // values behind the last key stay out of the product (0 times NaN); keys
    // 2q, 2q + 1 and 8 + 2q, 8 + 2q + 1 are this lane's
    const uint32_t keep0 = edge ? keep_pair(k0 + 2 * q, len) : kFull, keep1 = edge ? keep_pair(k0 + 8 + 2 * q, len) : kFull;
    if (C::MANY_NEW && edge && len > seen) {
      newest(stage, k0, len, seen, lim0, lim1, keep0, keep1, x, b0, b1, v_at);
      return;
    }
#pragma unroll
    for (int i1 = 0; i1 < D / 16; i1 += FB) {
      if (i1 > 0) {
#pragma unroll
        for (int i = 0; i < FB; ++i) ldmatrix4_t(f[i], v_at(i1 + i));
      }
#pragma unroll
      for (int i = 0; i < FB; ++i) {
        if (edge) {
          f[i][0] &= keep0;
          f[i][1] &= keep0;
          f[i][2] &= keep1;
          f[i][3] &= keep1;
        }
        mma16816(acc[i1 + i], f[i], b0, b1);
      }
    }
  }
  // P V for keys of which some are hidden from some row (more than one new
  // token): apart from the rest, which must not hold its registers.
  template <class At>
  __device__ __forceinline__ void newest(const uint8_t* stage, int k0, int len, int seen, int lim0, int lim1, uint32_t keep0, uint32_t keep1,
                                         const float (&x)[4], uint32_t b0, uint32_t b1, const At& v_at) {
    const uint32_t some0 = ~keep_pair(k0 + 2 * q, seen), some1 = ~keep_pair(k0 + 8 + 2 * q, seen);
    bool taken = false;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t f[1][4];
      ldmatrix4_t(f[0], v_at(i));
      f[0][0] &= keep0;
      f[0][1] &= keep0;
      f[0][2] &= keep1;
      f[0][3] &= keep1;
      taken |= take_out<1, false>(f, some0, some1);
      mma16816(acc[i], f[0], b0, b1);
    }
    if (taken) {
      // what was taken out goes to the rows that see it
      for (int k = max(k0, seen); k < min(k0 + 16, len); ++k) {
        const int c = k - k0, src = ((c & 7) << 2) | q;
        const float p0 = __shfl_sync(kFull, (c & 8) ? x[2] : x[0], src), p1 = __shfl_sync(kFull, (c & 8) ? x[3] : x[1], src);
        const int r = kw * 16 + c;
        const uint8_t* vr = stage + C::KV + r * 128 + g * 2;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint8_t* p = vr + (i >> 2) * C::CHUNK;
          const float v0 = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p + (((2 * i & 7) ^ (r & 7)) << 4)) << 16);
          const float v1 = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p + ((((2 * i + 1) & 7) ^ (r & 7)) << 4)) << 16);
          if (!isfinite(v0)) {
            if (k < lim0) acc[i][0] = fmaf(p0, v0, acc[i][0]);
            if (k < lim1) acc[i][1] = fmaf(p1, v0, acc[i][1]);
          }
          if (!isfinite(v1)) {
            if (k < lim0) acc[i][2] = fmaf(p0, v1, acc[i][2]);
            if (k < lim1) acc[i][3] = fmaf(p1, v1, acc[i][3]);
          }
        }
      }
    }
  }
  __device__ __forceinline__ void put_sums(float2* ml) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(kFull, l0, o);
      l1 += __shfl_xor_sync(kFull, l1, o);
    }
    if (g == 0) {
      ml[kw * 16 + 2 * q] = make_float2(m0, l0);
      ml[kw * 16 + 2 * q + 1] = make_float2(m1, l1);
    }
  }
  // In the stage, the place of the warp's own 16 keys: 64 columns of 8 rows
  // per chunk, 32-byte units permuted by the pair of rows (a store's four).
  static __device__ __forceinline__ uint8_t* om_at(uint8_t* om, int w, int r, int c) {
    return om + (c >> 6) * C::CHUNK + w * 2048 + r * 256 + ((c & 63) ^ ((r >> 1) << 3)) * 4;
  }
  __device__ __forceinline__ void put_out(uint8_t* om, int, int n) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      if (2 * q < n) {
        *reinterpret_cast<float*>(om_at(om, kw, 2 * q, 16 * i + g)) = acc[i][0];
        *reinterpret_cast<float*>(om_at(om, kw, 2 * q, 16 * i + g + 8)) = acc[i][2];
      }
      if (2 * q + 1 < n) {
        *reinterpret_cast<float*>(om_at(om, kw, 2 * q + 1, 16 * i + g)) = acc[i][1];
        *reinterpret_cast<float*>(om_at(om, kw, 2 * q + 1, 16 * i + g + 8)) = acc[i][3];
      }
    }
  }
};

template <int D, int ROWS, int BESIDE>
__global__ void __launch_bounds__(Cfg<D, ROWS, BESIDE>::THREADS, Cfg<D, ROWS, BESIDE>::CTAS)
    decode_paged_kernel(const __grid_constant__ PagedDecodeArgs a) {
  using C = Cfg<D, ROWS, BESIDE>;
  constexpr int MT = C::MT;
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
  // keys are three dependent look-ups. (They are then read by plain loads: a
  // read-only load might be moved above the wait.) The merge kernel is set up
  // in the same way meanwhile.
  {
    const long long line = (long long)blockIdx.x * C::THREADS + threadIdx.x;
    const char* const lens = reinterpret_cast<const char*>(a.seq_lens);
    const char* const tables = reinterpret_cast<const char*>(a.block_tables);
    if (line * 128 < (long long)a.B * a.max_pages * 4) prefetch_l2(tables + line * 128);
    if (line * 128 < (long long)a.B * 4) prefetch_l2(lens + line * 128);
  }
  if (a.pre_splits == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int R = a.G * a.Nq, shift = group_shift<C>(a);
  RowInfo* row_info = reinterpret_cast<RowInfo*>(smem + C::OFF_ROWS);
  Share* shared_share = reinterpret_cast<Share*>(smem + C::OFF_SHARE);
  if (warp == 0) {
    const Share found = find_share<C>(a, lane);
    if (lane == 0) *shared_share = found;
  } else {
    for (int e = threadIdx.x - 32; e < C::OWN_ROWS + (a.prefix_len > 0 ? 16 * MT : 0); e += C::THREADS - 32) {
      const bool own = e < C::OWN_ROWS;
      const int p = own ? e : e - C::OWN_ROWS;
      const int b = own ? 0 : a.rows_div(p), r = p - b * R, g = a.nq_div(r), i = r - g * a.Nq;
      row_info[e] = RowInfo{b * a.q_b + g * a.q_h + i * a.q_r, b * a.o_b + g * a.o_h + i * a.o_r, own ? a.Nq - 1 - i : 0};
    }
  }
  __syncthreads();
  Walk<C> wk;
  const bool any = wk.begin(a, *shared_share);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0 && a.prefix_len == 0) a.begun[blockIdx.x] = make_int2(-1, 0);
    if (!any) return;
    const int nbox = C::BK >> a.box_shift;    // boxes of a chunk's 64 rows
    const bool mine = lane < nbox * 2 * C::CH;
    const int box = lane & (nbox - 1), col = lane >> (6 - a.box_shift);  // this lane's box; the keys' chunks, then the values'
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
      t.head = wk.sh.head >> shift;
      if (mine && box < t.boxes) {
        const int* table = wk.sh.seq < a.B ? a.block_tables + (long long)wk.sh.seq * a.max_pages : a.prefix_pages;
        const int key = key0 + (box << a.box_shift), pi = a.page_div(key);
        t.row = key - pi * a.pool.page_size;
        t.page = table[pi];
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
          const int unit = wk.sh.seq * unit_heads<C>(a) + wk.sh.head, last = whole ? (int)blockIdx.x : cut.owner(blockIdx.x, end - 1);
          if (a.prefix_len > 0) a.unit_ctas[unit] = make_int2(blockIdx.x, last);
          else a.begun[blockIdx.x] = make_int2(unit, last);
        }
      }
      if (++tile == tile_end) {
        more = wk.advance(a);
        tile = wk.first_tile();
        tile_end = tile + wk.tile_count();
      }
      const Tile next = more ? look_up(tile) : t;
      const int s = it % C::STAGES;
      if (!mbar_wait_warp(EMPTY(s), ((it / C::STAGES) & 1) ^ 1, a.status, a.wait_limit_ns)) break;
      const bool load = it != a.debug_skip_tile;
      if (load && lane == 0) mbar_arrive_expect_tx(FULL(s), (uint32_t)((t.boxes * 128 * 2 * C::CH) << a.box_shift));
      __syncwarp();
      if (load && mine && box < t.boxes) {
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
  // it still reaches every barrier, and frees no stage any more: the producer
  // then stops by a wait of its own, before a stage's barrier is used again
  // whose copies are still in flight. The status word tells.
  const int cw = warp - 1, mt = cw >> 2, kw = cw & 3;
  const int ct = kw * 32 + lane;  // thread of the group's 128
  const float c2 = a.scale_log2;
  float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML) + mt * 64;  // [4][16]
  // A unit's 16 query rows, D / 8 vectors each, vector u of row r at u ^ (r & 7)
  const uint32_t q_buf = sbase + C::OFF_Q + mt * 16 * D * 2;
  using Warp = std::conditional_t<ROWS == 8, WarpRows8<C>, WarpRows16<C>>;
  Warp st;
  st.init(lane, kw, mt);
  auto fetch_q = [&](int seq, int unit_head, int buf) {
    const bool pre = seq >= a.B;
    const int head = unit_head >> shift, r0 = (unit_head - (head << shift)) * ROWS;
    const int rows = pre ? a.B * R : R - r0;
    const RowInfo* info = row_info + (pre ? C::OWN_ROWS : r0) + mt * 16;
    const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(a.Q) + (pre ? 0 : seq * a.q_b) + (long long)head * a.G * a.q_h;
#pragma unroll
    for (int e = ct; e < Warp::ROWS * (D / 8); e += 128) {
      const int r = e / (D / 8), u = e - r * (D / 8);
      const bool valid = mt * 16 + r < rows;
      const __nv_bfloat16* src = base + (valid ? info[r].q + u * 8 : 0);
      copy16(q_buf + buf * C::QBUF + r * (D * 2) + ((u ^ (r & 7)) << 4), src, valid);
    }
  };
  if (any) fetch_q(wk.sh.seq, wk.sh.head, 0);
  if (a.prefix_len == 0 && shared_share->empty) empty_rows<D>(a, blockIdx.x * C::CONSUMERS + cw, gridDim.x * C::CONSUMERS);
  bool ok = true;
  int it = 0, qb = 0;
  for (bool more = any; more; qb ^= 1) {
    const int n = wk.tile_count(), first = wk.first_tile(), seq = wk.sh.seq, unit_head = wk.sh.head, len = wk.len;
    const int head = unit_head >> shift, r0 = (unit_head - (head << shift)) * ROWS;
    const bool begins = first == 0, ends = first + n == wk.tiles;
    const bool pre = seq >= a.B;
    const int rows = pre ? a.B * R : min(ROWS, R - r0);
    const RowInfo* info = row_info + (pre ? C::OWN_ROWS : r0);
    const int seen = pre ? len : max(0, len - a.Nq + 1);  // keys that every row sees
    const bool active = mt * 16 < rows;                   // else these warps only keep step
    copies_done();
    named_bar(1 + mt, 128);  // this unit's queries are there; the other buffer has been read
    st.begin(q_buf + qb * C::QBUF);
    more = wk.advance(a);
    if (more) fetch_q(wk.sh.seq, wk.sh.head, qb ^ 1);
    for (int j = 0; j < n; ++j, ++it) {
      const int s = it % C::STAGES;
      if (ok) ok = mbar_wait_warp(FULL(s), (it / C::STAGES) & 1, a.status, a.wait_limit_ns);
      const int k0 = (first + j) * C::BK + kw * 16;  // this warp's keys
      if (ok && active && k0 < len) st.tile(sbase + s * C::STAGE, smem + s * C::STAGE, k0, len, seen, info, rows, c2);
      __syncwarp();
      if (ok && lane == 0 && !(C::MERGE_IN_STAGE && j + 1 == n)) mbar_arrive(EMPTY(s));
    }

    if (!active) continue;
    // the four warps of a group of rows meet in shared memory: maxima, sums
    // and outputs as they are, weighted and added by whoever writes them out
    st.put_sums(ml);
    const int last_stage = (it - 1) % C::STAGES;
    uint8_t* om = smem + (C::MERGE_IN_STAGE ? last_stage * C::STAGE : C::OFF_MERGE + mt * C::MERGE);
    const long long unit = (long long)seq * unit_heads<C>(a) + unit_head;
    const bool direct = begins && ends && a.prefix_len == 0;
    const long long part_row = part_slot(a, blockIdx.x, begins, ends, unit) * a.slot_rows;
    const long long o_unit = (pre ? 0 : seq * a.o_b) + (long long)head * a.G * a.o_h;
    constexpr int DW = C::DW;
    const int group_rows = min(16, rows - mt * 16);
#pragma unroll
    for (int d0 = 0; d0 < D; d0 += DW) {
      if (d0 > 0) named_bar(1 + mt, 128);  // the columns before these have been read
      st.put_out(om, d0, group_rows);
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
          const float4 z = *reinterpret_cast<const float4*>(Warp::om_at(om, w, r, c));
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
          if (d0 + c == 0) a.LSE[(unit >> shift) * R + r0 + rr] = lse * kLn2;
        } else {
          *reinterpret_cast<float4*>(a.Opart + (part_row + rr) * D + d0 + c) = y;
          if (d0 + c == 0) a.Lpart[part_row + rr] = lse;
        }
      }
    }
    if (C::MERGE_IN_STAGE) {
      fence_proxy_async_smem();  // the stage's next writer is the TMA
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(EMPTY(last_stage));
    }
  }
  // a prefix's kernel ends before this one does, so the merge sees both; one
  // CTA waits for that, the others make room
  if (blockIdx.x + 1 == gridDim.x) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Rows of units that were not written out directly: partial results of the
// own keys (and of the prefix) merged by maximum and sum, in order of the CTAs.
constexpr int kMergeWarps = 8;

// The parts of a row: those of the CTAs that share its unit, then the prefix's.
struct Parts {
  int unit, slot_row;     // unit, and the row in its slots
  int own_first, own_n;   // CTAs
  int pre_unit, pre_slot_row, pre_first, pre_n;  // the same of a prefix that is part of the grid
  long long pre_row;      // a prefix's kernel of its own: row of the first part, parts 256 rows apart
};

// A warp's share of a row: every step-th part from `part` on; a lane has D / 32 columns.
template <int D, bool PREFIX>
struct RowSum {
  static constexpr int E = D / 32;
  static constexpr int AHEAD = 4;  // partial results in flight per warp
  float m = -INFINITY, l = 0.f, acc[E];

  __device__ __forceinline__ void add(const PagedDecodeArgs& a, const Parts& P, int part, int step, int lane) {
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    const int n = P.own_n + P.pre_n;
    for (int p0 = part; p0 < n; p0 += AHEAD * step) {
      float L[AHEAD], x[AHEAD][E];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int p = p0 + k * step;
        L[k] = -INFINITY;
#pragma unroll
        for (int e = 0; e < E; ++e) x[k][e] = 0.f;
        if (p >= n) continue;
        const bool own = !PREFIX || p < P.own_n;
        const int i = own ? p : p - P.own_n;
        const float* O = a.Opart;
        const float* Ls = a.Lpart;
        long long row;
        if (own) {
          row = part_slot(a, P.own_first + i, i == 0, i + 1 == P.own_n, P.unit) * a.slot_rows + P.slot_row;
        } else if (a.pre_splits == 0) {
          row = part_slot(a, P.pre_first + i, i == 0, i + 1 == P.pre_n, P.pre_unit) * a.slot_rows + P.pre_slot_row;
        } else {
          O = a.pre_Opart;
          Ls = a.pre_Lpart;
          row = P.pre_row + 256ll * i;
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
  }
  // Groups of STEP warps meet; the first of each has the row's sum afterwards.
  template <int STEP>
  __device__ __forceinline__ void meet(int warp, int lane) {
    __shared__ float sm[kMergeWarps], sl[kMergeWarps], so[kMergeWarps][D];
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
    named_bar(1 + warp / STEP, 32 * STEP);
    if (warp % STEP == 0) {
      m = -INFINITY;
#pragma unroll
      for (int w = 0; w < STEP; ++w) m = fmaxf(m, sm[warp + w]);
      const float mu = m == -INFINITY ? 0.f : m;
      l = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
      for (int w = 0; w < STEP; ++w) {
        const float f = ex2_approx(sm[warp + w] - mu);
        l = fmaf(sl[warp + w], f, l);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(so[warp + w][lane * E + e], f, acc[e]);
      }
    }
  }
  // Row r of sequence b and K/V head `head`
  __device__ __forceinline__ void store(const PagedDecodeArgs& a, int b, int head, int r, int lane) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int g = a.nq_div(r), i = r - g * a.Nq, hq = head * a.G + g;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.O) + b * a.o_b + hq * a.o_h + i * a.o_r + lane * E;
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2 % E] * inv, acc[3 % E] * inv));
    else
      *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    if (lane == 0)
      a.LSE[((long long)b * a.pool.kv_heads + head) * a.G * a.Nq + r] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
  }
};

// Without a prefix only the units that a share's end cuts have parts. Items are
// (CTA that begins such a unit, row of the unit); a block looks at every
// gridDim.x-th of them at once, one per lane, as many are none, and shares its
// warps out among those that are: eight to a single row (a long sequence has
// parts of many CTAs), one to each of many.
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_cut_kernel(const __grid_constant__ PagedDecodeArgs a, int rows) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned mine = blockIdx.x + lane * gridDim.x;  // at most 32 per block
  const bool there = mine < (unsigned)(a.ctas * rows);
  const int cta = there ? (rows < a.slot_rows ? a.rows_div((int)mine) : (int)(mine / (unsigned)rows)) : 0;
  const int row = (int)mine - cta * rows;
  const int2 c = there ? a.begun[cta] : make_int2(-1, 0);
  const int n = c.y - cta + 1;
  unsigned rest = __ballot_sync(kFull, c.x >= 0);
  // the next kMergeWarps / STEP of the items, STEP warps each
  auto merge = [&](auto STEP) {
    unsigned from = rest;
#pragma unroll
    for (int k = 0; k < kMergeWarps / STEP; ++k) {
      if (k < warp / STEP) from &= from - 1;
      rest &= rest - 1;
    }
    const int at = __ffs(from) - 1;  // this warp's item, or -1
    Parts P{};
    P.unit = __shfl_sync(kFull, c.x, at & 31);
    P.slot_row = __shfl_sync(kFull, row, at & 31);
    P.own_first = __shfl_sync(kFull, cta, at & 31);
    P.own_n = at < 0 ? 0 : __shfl_sync(kFull, n, at & 31);
    RowSum<D, false> sum;
    sum.add(a, P, warp % STEP, STEP, lane);
    if constexpr (decltype(STEP)::value > 1) sum.template meet<decltype(STEP)::value>(warp, lane);
    if (at >= 0 && warp % STEP == 0) {
      const int heads = a.pool.kv_heads << a.group_shift, b = P.unit / heads, h = P.unit - b * heads, head = h >> a.group_shift;
      const int r = (h - (head << a.group_shift)) * a.slot_rows + P.slot_row;
      if (r < a.G * a.Nq) sum.store(a, b, head, r, lane);  // the unit may have fewer rows than others
    }
  };
  while (rest != 0) {
    const int items = __popc(rest);
    if (items == 1) merge(std::integral_constant<int, 8>{});
    else if (items <= 4) merge(std::integral_constant<int, 2>{});
    else merge(std::integral_constant<int, 1>{});
    if (rest != 0) __syncthreads();
  }
}

// With a prefix every row has parts, as many as the prefix has key ranges. WPR
// warps share a row.
template <int D, int WPR>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_prefix_kernel(const __grid_constant__ PagedDecodeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hkv = a.pool.kv_heads, R = a.G * a.Nq;
  const unsigned item = blockIdx.x * (kMergeWarps / WPR) + warp / WPR;
  if (item >= (unsigned)(a.B * Hkv) * (unsigned)R) return;  // all warps of a row alike, here and below
  const int group = (int)(item / (unsigned)R), r = (int)(item - group * (unsigned)R);
  const int b = group / Hkv, head = group - b * Hkv, rg = a.group_shift == 0 ? 0 : r / 32;
  // a unit whose CTA gave up on a wait may have no entry, and then no result
  auto in_grid = [&](int2 c) { return (unsigned)c.x <= (unsigned)c.y && (unsigned)c.y < (unsigned)a.ctas; };
  Parts P{};
  P.unit = (group << a.group_shift) + rg;
  P.slot_row = r - rg * 32;
  const int2 c = a.unit_ctas[P.unit];  // not written for a sequence without keys
  P.own_first = c.x;
  P.own_n = seq_keys(a, b) > 0 ? c.y - c.x + 1 : 0;
  if (a.pre_splits > 0) {
    const int rr = b * R + r, qblocks = (a.B * R + 255) / 256;
    P.pre_n = a.pre_splits;
    P.pre_row = ((long long)head * qblocks + rr / 256) * a.pre_splits * 256 + rr % 256;
  } else {
    P.pre_unit = a.B * Hkv + head;
    P.pre_slot_row = b * R + r;
    const int2 cp = a.unit_ctas[P.pre_unit];
    P.pre_first = cp.x;
    P.pre_n = cp.y - cp.x + 1;
    if (!in_grid(cp)) return;
  }
  if (P.own_n != 0 && !in_grid(c)) return;
  RowSum<D, true> sum;
  sum.add(a, P, warp % WPR, WPR, lane);
  if constexpr (WPR > 1) sum.template meet<WPR>(warp, lane);
  if (warp % WPR == 0) sum.store(a, b, head, r, lane);
}

// Warps per row of merge_prefix_kernel. Up to four parts of a row are one round
// of loads, more take several: more warps for a row while all rows find room at
// once, and beyond 16 parts anyway (768 rows of 12 parts: 16.3 -> 14.2 us of the
// call).
int merge_warps(long long rows, int parts) {
  int n = 1;
  while (n < kMergeWarps && (parts > 16 * n || (parts > 4 * n && rows * n <= 3000))) n *= 2;
  return n;
}

template <int D, int ROWS, int BESIDE>
cudaError_t launch(const PagedDecodeArgs& a, cudaStream_t st) {
  using C = Cfg<D, ROWS, BESIDE>;
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_paged_kernel<D, ROWS, BESIDE>, a);
  if (e != cudaSuccess) return e;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.dynamicSmemBytes = 0;
  const int rows = a.G * a.Nq;
  if (a.prefix_len == 0) {
    // as many blocks as find room at once, each for several (CTA, row) items
    const int unit_rows = rows < a.slot_rows ? rows : a.slot_rows, most = a.slot_rows == 32 ? 4 : 2;
    cfg.gridDim = dim3((unsigned)(a.ctas * (unit_rows < most ? unit_rows : most)));
    return cudaLaunchKernelEx(&cfg, merge_cut_kernel<D>, a, unit_rows);
  }
  const unsigned all = (unsigned)(a.B * a.pool.kv_heads) * (unsigned)rows;
  // parts of a prefix that is part of the grid: about one per CTA and head
  const int parts = a.pre_splits > 0 ? a.pre_splits : a.ctas / a.pool.kv_heads;
  const int wpr = merge_warps(all, parts);
  cfg.gridDim = dim3((all * wpr + kMergeWarps - 1) / kMergeWarps);
  return cudaLaunchKernelEx(&cfg, wpr == 8   ? merge_prefix_kernel<D, 8>
                                  : wpr == 4 ? merge_prefix_kernel<D, 4>
                                  : wpr == 2 ? merge_prefix_kernel<D, 2>
                                             : merge_prefix_kernel<D, 1>, a);
}

// Also allows the kernel its shared memory on the current device; every launch
// follows a paged_layout() on the same device.
template <int D, int ROWS, int BESIDE>
int ctas_per_sm() {
  using C = Cfg<D, ROWS, BESIDE>;
  if (cudaFuncSetAttribute(decode_paged_kernel<D, ROWS, BESIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC) !=
      cudaSuccess)
    return 0;
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, decode_paged_kernel<D, ROWS, BESIDE>, C::THREADS, C::SMEM_ALLOC) !=
      cudaSuccess)
    return 0;
  return n;
}

// Rows of a K/V head up to which a prefix is one more sequence of the grid
constexpr int kGridPrefixRows = 32;

constexpr int kMaxDevices = 64;
std::mutex g_slots_mu;
int g_slots[kMaxDevices][2][4] = {};  // [device][d == 128][8, 16, 32 rows, 8 beside a prefix] -> resident CTAs

template <int D>
int ctas_per_sm(int rows, bool beside) {
  return rows == 8    ? (beside ? std::min(ctas_per_sm<D, 8, 1>(), ctas_per_sm<D, 8, 2>()) : ctas_per_sm<D, 8, 0>())
         : rows == 16 ? ctas_per_sm<D, 16, 0>()
                      : ctas_per_sm<D, 32, 0>();
}

int resident_ctas(int d, int rows, bool beside) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> lk(g_slots_mu);
  int& slot = g_slots[dev][d == 128][rows == 8 ? (beside ? 3 : 0) : rows == 16 ? 1 : 2];
  if (slot == 0) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    slot = sms * (d == 128 ? ctas_per_sm<128>(rows, beside) : ctas_per_sm<64>(rows, beside));
  }
  return slot;
}

template <int D>
cudaError_t launch_d(const PagedDecodeArgs& a, cudaStream_t st) {
  switch (a.slot_rows) {
    case 8: return a.pre_splits == 0 ? launch<D, 8, 0>(a, st) : a.Nq == 1 ? launch<D, 8, 1>(a, st) : launch<D, 8, 2>(a, st);
    case 16: return launch<D, 16, 0>(a, st);
    default: return launch<D, 32, 0>(a, st);
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

PagedLayout paged_layout(int B, int Hkv, int rows, int prefix_len, int d) {
  PagedLayout L{};
  const long long pre_rows = prefix_len > 0 ? (long long)B * rows : 0;
  const bool own_kernel = pre_rows > kGridPrefixRows;
  const long long most = pre_rows > rows && !own_kernel ? pre_rows : rows;
  L.slot_rows = most <= 8 ? 8 : most <= 16 ? 16 : 32;
  while ((L.slot_rows << L.group_shift) < rows) ++L.group_shift;
  L.ctas = resident_ctas(d, L.slot_rows, own_kernel);
  if (L.ctas <= 0) return L;
  L.n_seq = B + (pre_rows > 0 && !own_kernel ? 1 : 0);
  const size_t units = (size_t)L.n_seq * Hkv << L.group_shift;
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
                              int most_keys, bool narrow) {
  // Times in us, measured on a GB300. A prefix's CTA takes kStart and, per tile
  // of 128 keys, 1.76 (two tiles of query rows) or 1.05 (one), two thirds of
  // that at d = 64. An own keys' CTA beside it takes kOwnStart and per step (64
  // keys) 0.75, 0.6 at d = 64, 1.1 and 1.5 steps more per unit with more than 16
  // rows at d = 128, or what all such CTAs' bytes take at 6 GB/ms; one that finds
  // its SM only after the prefix's costs kLate, in which the others go on. Boxes
  // of 8 rows: a third more per tile, twice as much per step. Each
  // key range is a partial result per row, written once and read once, four of
  // them in a round of the merge.
  //
  // How many own keys the sequences have is not known here, and the width of
  // their table says little: it is the longest context a server allows, and a
  // captured graph keeps its plan while they grow. So the plan is the one that
  // loses least against each length's own best plan, over lengths from 32 to 2048
  // keys as far as the table can hold them. (A quarter of the table's width taken
  // for the length: 64 questions, 100 to 700 own keys, 75 us in a table of 768
  // keys and 477 in one of 131072; now 75 in both. By the times above the loss
  // is 2 to 4% in the mean over shapes, whatever the length.)
  constexpr int kLengths[] = {32, 128, 512, 2048}, kMost = 4;
  constexpr double kStart = 11.0, kOwnStart = 2.0, kLate = 3.0, kPartBytes = 4e6, kRound = 1.0;
  const bool wide = rows > 16 && d == 128;
  const double kStep = (wide ? 1.1 : d == 128 ? 0.75 : 0.6) * (narrow ? 2 : 1), kStepAll = 256.0 * d / 6e6;
  const int n_kv = (int)(((long long)prefix_len + 127) / 128);
  const long long all_rows = (long long)B * rows, units = (all_rows + 255) / 256 * Hkv;
  const double tile = (all_rows > 128 ? 1.76 : 1.05) * (d == 128 ? 1.0 : 0.67) * (narrow ? 1.33 : 1.0);
  const double own_units = (double)B * Hkv * (rows > 32 ? 2 : 1);
  const double part_us = (double)all_rows * Hkv * d * 8.0 / kPartBytes;
  int lengths[kMost], n_lengths = 0;
  while (n_lengths < kMost && (n_lengths == 0 || kLengths[n_lengths] <= most_keys)) {
    lengths[n_lengths] = std::min(kLengths[n_lengths], most_keys);
    ++n_lengths;
  }
  PrefixPlan plans[kPrefixMaxSplits];
  double us[kPrefixMaxSplits][kMost], least[kMost];
  for (int s = 1; s <= max_splits; ++s) {
    const long long waves = (units * s + sms - 1) / sms;
    const double pre_us = kStart + (double)waves * ((n_kv + s - 1) / s) * tile;
    const int early = waves == 1 ? (sms - (int)(units * s)) * (ctas / sms) : 0;
    const double step = early * kStepAll > kStep ? early * kStepAll : kStep;
    const int more = early > 0 ? (int)((pre_us + kLate - kOwnStart) / step) : 0;
    const int per_round = 4 * merge_warps(all_rows * Hkv, s);
    plans[s - 1] = PrefixPlan{s, early, more};
    for (int i = 0; i < n_lengths; ++i) {
      const double steps = own_units * (lengths[i] / 64.0 + kUnitSteps + (wide ? 2.0 : 0.5));
      double& t = us[s - 1][i];
      t = s * part_us + (s + per_round) / per_round * kRound;
      if (early > 0 && steps <= early * (double)more)
        t += std::max(pre_us, kOwnStart + steps / early * step);
      else
        t += pre_us + kLate + (steps - early * (double)more) * kStepAll;
      least[i] = s == 1 ? t : std::min(least[i], t);
    }
  }
  int best = 0;
  double best_loss = -1;
  for (int s = 0; s < max_splits; ++s) {
    double loss = 0;
    for (int i = 0; i < n_lengths; ++i) loss += us[s][i] / least[i];
    if (best_loss < 0 || loss < best_loss) {
      best_loss = loss;
      best = s;
    }
  }
  return plans[best];
}

PrefixPlan plan_shared(int B, int rows, int Hkv, int prefix_len, int d, int sms, int most_keys, bool narrow) {
  int max_splits, ctas;
  if (sms == 0) {
    const PagedLayout L = paged_layout(B, Hkv, rows, prefix_len, d);
    if (L.ctas < 1) return PrefixPlan{-1, 0, 0};
    max_splits = L.pre_splits;
    ctas = L.ctas;
    sms = fwd_slots();
  } else {
    const long long all_rows = (long long)B * rows;
    max_splits = prefix_len > 0 && all_rows > kGridPrefixRows
                     ? plan_prefix_splits((all_rows + 255) / 256 * Hkv, (int)(((long long)prefix_len + 127) / 128), sms)
                     : 0;
    ctas = sms * (rows <= 8 ? Cfg<128, 8, 1>::CTAS : rows <= 16 ? Cfg<128, 16, 0>::CTAS : Cfg<128, 32, 0>::CTAS);
  }
  if (max_splits < 1) return PrefixPlan{0, 0, 0};
  return plan_prefix_beside(B, rows, Hkv, prefix_len, d, max_splits, ctas, sms, most_keys, narrow);
}

cudaError_t launch_decode_paged_bf16(const PagedDecodeArgs& a, int d, cudaStream_t st) {
  if (a.ctas < 1) return cudaErrorInvalidValue;
  return d == 128 ? launch_d<128>(a, st) : d == 64 ? launch_d<64>(a, st) : cudaErrorInvalidValue;
}

}  // namespace fa

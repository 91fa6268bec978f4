// prompt_fwd.cu -- causal attention of packed prompts with grouped heads.
//
// What it computes, for each sequence of n query tokens and m >= 0 keys and
// each query head hq on K/V head h = hq / G:
//   O_i = sum_{j <= m - n + i} exp(s_ij - m_i) V_j / l_i,  s_ij = scale * q_i . k_j,
//   LSE_i = m_i + ln(l_i);  a query that sees no key: O_i = 0, LSE_i = -inf.
//
// The G query heads of a K/V head are rows of one problem: a query tile holds
// TP = floor(128 / G) tokens of all G heads (row r: head r mod G of token
// r / G), which a 4-D TMA box (64 columns, G heads, TP tokens) lays out at
// once. So a prompt of 37 tokens with four heads fills 148 rows of two tiles
// instead of 37 of four, and a CTA's keys and values serve 2 TP tokens of every
// head.
//
// A block is two query tiles of one sequence and K/V head, whose key tiles are
// those of the second one's last query. Products and online softmax are those of
// the forward in attn_fwd_bf16.cu (described there). What differs: each tile
// visits its own number of key tiles, the diagonal of a tile can cross two key
// tiles (masked scores are replaced where they stand, in tensor memory, in a pass
// of its own: a few tiles to a block, and no mask in the loop), rows may see no
// key at all, and keys come either packed (one TMA box per 128 keys) or from the
// pages of a cache (one box per page or part of one, issued by the lanes of a
// producer warp). What stands behind a sequence's last key (another sequence's
// rows, old rows of a page, NaN included) has no influence: its scores are
// replaced, the products over keys end at the last one, and the up to 15 rows of
// V that their last step still reads are set to zero. P is rounded to bf16 for its
// product, its sum is not.
//
// Blocks are listed longest first (prompt.cuh), found from the offsets on the
// device, so a captured graph follows them. CTAs are persistent: near the end of
// its block a CTA's scheduler warp takes over the index of one that has not begun
// (cluster launch control), so that the next block's loads and first products run
// under the last one's softmax, while four warps of their own take the last one's
// output away (16384 tokens, 32 heads: one block per CTA 1442 TFLOP/s, blocks taken
// over 1728, with output warps 1839; taken over earlier, a long block would hold
// the next one back). Few blocks with many keys are split into key ranges, whose
// partial results prompt_merge_kernel combines by their maxima and sums.
//
// Bound, per pair of query tiles and 128 keys and SM, in cycles: products 2048
// (d = 128) or 1024 (d = 64), exponentials 1024. Measured on long prompts: 2640
// (1860 TFLOP/s) and 1950 (1260). What is between is the chain from scores to
// weights to the next product. Products are issued hardly ahead of their execution
// (three at most), an answer from a barrier takes a hundred cycles even when it is
// over, and beside two softmax warps an instruction takes ten. With d = 128 tensor
// memory is full with two tiles' S and O, so a tile's next S can only follow its
// P V; with d = 64 three S buffers in turn take that out of the chain (1000 TFLOP/s
// without, 1190 with), and S and P V are issued by a warp each (1200, 1260 with
// loops of few instructions). Times in a batch: 16 prompts of 128 to 7821 tokens (32
// heads on 8, d = 128) 960 to 1020 us by the box, one of 32768 tokens 4.95 to 5.2 ms, the next turns of six
// chats (d = 64, pages of 32 keys) 83 us, one of 37 tokens 12.5 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "fa_internal.h"
#include "fwd_tile.cuh"
#include "prompt.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

struct PromptBlock {
  PromptView v;
  int seq, head;
  int tok0;        // first token of tile 0; tile 1 begins TP tokens later
  int kt0;         // first key tile of this part
  int n0, n1;      // key tiles of the query tiles 0 and 1, from kt0 on
  int unit;        // index of the block in the list
  int parts;       // key ranges of each block
};

// Whole warp: the block and key range of CTA `u`; false past the last one.
__device__ __forceinline__ bool prompt_block(const PromptFwdArgs& a, long long u, int lane, bool report,
                                             PromptBlock& k, int& part) {
  const int per = 2 * a.tile_tokens;
  bool bad = false;
  auto span = [&](int b) { return query_span(prompt_view(a.seqs, b, bad), per); };
  PromptSpan first;
  int top;
  const int total = count_blocks(a.seqs.B, lane, span, first, top);
  if (report && bad) report_status(a.status, kStatusBadSeqlens);
  // The host's plan may come from a table far wider than its sequences, of fewer
  // blocks than there can be: the same cost decides here again, for those that
  // there are, lane by lane (60 tokens after 840 in a table of 131072 keys: 37 us
  // by the host's plan, 23 so).
  k.parts = 1;
  if (a.splits > 1) {
    const int tiles = (int)min(((long long)(top + 1) * per + 127) / 128, 1ll << 24);
    const int most_parts = min(a.splits, max(tiles, 1));
    unsigned best = 0xffffffffu;  // costs are positive: their bits are in their order
    for (int s = lane + 1; s <= most_parts; s += 32) {
      const unsigned cost = __float_as_uint(prompt_split_cost((float)total * (float)a.Hkv, tiles, a.slots, s));
      if (cost < best) {
        best = cost;
        k.parts = s;
      }
    }
    const unsigned least = __reduce_min_sync(0xffffffffu, best);
    k.parts = (int)__reduce_min_sync(0xffffffffu, best == least ? (unsigned)k.parts : 0xffffffffu);
  }
  part = (int)(u % k.parts);
  const long long w = u / k.parts;
  // Offsets that run back and forth can give more blocks than there is room for
  // among the partial results; with fewer ranges than the host planned, CTAs
  // enough to reach them. (A sequence whose offsets run back is reported above.)
  if (w >= min((long long)total, a.max_blocks) * a.Hkv) return false;
  const int hpg = a.heads_per_group;
  const int group = (int)(w / ((long long)total * hpg));
  const int local = (int)(w - (long long)group * total * hpg);
  const int heads = min(hpg, a.Hkv - group * hpg);
  const int idx = local / heads;
  int block;
  find_block(a.seqs.B, lane, span, first, top, idx, k.seq, block);
  k.head = group * hpg + local - idx * heads;
  k.unit = (int)w;
  k.v = prompt_view(a.seqs, k.seq, bad);
  k.tok0 = block * per;
  auto key_tiles = [&](int t0) {  // of the query tile that begins with token t0
    const int seen = k.v.m - k.v.n + min(k.v.n, t0 + a.tile_tokens);  // keys of its last query
    return t0 < k.v.n && seen > 0 ? (seen + 127) / 128 : 0;
  };
  const int n0 = key_tiles(k.tok0), n1 = key_tiles(k.tok0 + a.tile_tokens), most = max(n0, n1);
  k.kt0 = (int)((long long)part * most / k.parts);
  const int end = (int)((long long)(part + 1) * most / k.parts);
  k.n0 = max(0, min(n0, end) - k.kt0);
  k.n1 = max(0, min(n1, end) - k.kt0);
  return true;
}

// Warps 0: producer (of pages: Q and K), 1: MMA issuer (d = 64: the S products),
// 2: scheduler (and of pages the producer of V), 3: d = 64: the P V products; 4-7
// and 8-11: softmax of query tiles 0 and 1; 12-15: output. Shared memory: that of
// the two-tile forward, a tile of O on its way out, the rows' sums on their way to
// the output warps and a ring of published blocks.
template <int D>
struct PromptCfg : FwdCfg<D> {
  using F = FwdCfg<D>;
  static constexpr int NTHREADS = 512;
  // Scores: with d = 128 a buffer for each query tile, over which its weights P
  // go. With d = 64 three of them in turn: while one tile's P V and the other's
  // softmax are at work, the next S is there already.
  static constexpr bool TURNS = D == 64;
  static constexpr int SBUF = TURNS ? 3 : 2;
  // Barriers that tell a query tile's softmax of its next S, in turn: as many as
  // S can be ahead of it, so that none is a phase ahead of its waiter.
  static constexpr int SFULLS = TURNS ? 3 : 1;
  static constexpr uint32_t S_COL(int b) { return 128u * b; }
  static constexpr uint32_t O_COL(int t) { return 128u * SBUF + (uint32_t)D * t; }
  static constexpr int OFF_STAGE = F::OFF_BAR;  // behind the K/V ring: 128 rows of O, as the query tiles are laid out
  static constexpr int OFF_STAT = OFF_STAGE + F::TILE_BYTES;  // float [2 blocks][2 tiles][128 rows]: sums of weights
  static constexpr int IRING = 2;  // blocks published: the one in work and the next
  static constexpr int ITEM_INTS = 12;
  static constexpr int OFF_BARS = OFF_STAT + 2 * 2 * 128 * 4;
  // q_full[2], q_empty[2], k_full, v_full, k_empty, v_empty [STAGES each], s_full[2][SFULLS], p_full, s_done
  // [SBUF each], o_done[2], o_free[2], l_full[2 tiles][2 blocks], stage_full, stage_free, item_full, item_empty [IRING each],
  // cancel, near, drain
  static constexpr int NBARS = 4 + 4 * F::STAGES + 2 * SFULLS + 2 * SBUF + 10 + 2 * IRING + 3;
  static constexpr int OFF_ITEMS = (OFF_BARS + NBARS * 8 + 15) / 16 * 16;
  static constexpr int OFF_CANCEL = OFF_ITEMS + IRING * ITEM_INTS * 4;  // 16 bytes: the next CTA index
  static constexpr int OFF_MISC = OFF_CANCEL + 16;                      // TMEM base, abort flag
  static constexpr int BYTES = OFF_MISC + 8;
  static constexpr int MOST = 227 * 1024;
  // 1 KB of alignment slack where it fits; the kernel checks the alignment
  static constexpr int ALLOC = BYTES + 1024 <= MOST ? BYTES + 1024 : MOST;
  // Registers per thread of the control, softmax and output warps, out of the
  // launch's 128 each: control + 2 softmax + out = 512.
  static constexpr int R_CONTROL = D == 128 ? 64 : 88, R_SOFTMAX = D == 128 ? 176 : 160, R_OUT = D == 128 ? 96 : 104;
  static_assert(128 * (R_CONTROL + 2 * R_SOFTMAX + R_OUT) <= NTHREADS * 128, "register split");
};

// What the ring holds of a block: its sequence's first packed token and tokens,
// the K/V head, tile 0's first token, the first key tile, the key tiles of query
// tiles 0 and 1 (-1: no more blocks), its rows among the partial results, the
// sequence's first packed key and index, and of the keys from the first tile on,
// those that tile 0's first row sees and those that there are.
enum : int { kItQ0, kItN, kItHead, kItTok0, kItKt0, kItN0, kItN1, kItPart, kItK0, kItSeq, kItFirst, kItLeft };

template <int D, bool PAGED>
__global__ void __launch_bounds__(512, 1) prompt_fwd_kernel(const __grid_constant__ PromptFwdArgs a) {
  using C = PromptCfg<D>;
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
  const int B_QFULL = 0, B_QEMPTY = 2, B_KFULL = 4, B_VFULL = B_KFULL + C::STAGES, B_KEMPTY = B_VFULL + C::STAGES,
            B_VEMPTY = B_KEMPTY + C::STAGES, B_SFULL = B_VEMPTY + C::STAGES, B_PFULL = B_SFULL + 2 * C::SFULLS,
            B_SDONE = B_PFULL + C::SBUF, B_ODONE = B_SDONE + C::SBUF, B_OFREE = B_ODONE + 2, B_LFULL = B_OFREE + 2,
            B_STAGE = B_LFULL + 4, B_ITF = B_STAGE + 2, B_ITE = B_ITF + C::IRING, B_CANCEL = B_ITE + C::IRING, B_NEAR = B_CANCEL + 1,
            B_DRAIN = B_NEAR + 1;
  volatile int* items = reinterpret_cast<volatile int*>(smem + C::OFF_ITEMS);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int TP = a.tile_tokens, RT = TP * a.G;  // tokens and rows of a query tile

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(BAR(B_QFULL + t), 1);
      mbar_init(BAR(B_QEMPTY + t), 1);
      mbar_init(BAR(B_ODONE + t), 1);
      for (int k = 0; k < C::SFULLS; ++k) mbar_init(BAR(B_SFULL + t * C::SFULLS + k), 1);
      mbar_init(BAR(B_OFREE + t), 4);  // one arrival per output warp
      mbar_init(BAR(B_LFULL + 2 * t), 4);  // a barrier for every other block: a tile without rows
      mbar_init(BAR(B_LFULL + 2 * t + 1), 4);  // is done at once, and its waiter may be a block behind
    }
    for (int b = 0; b < C::SBUF; ++b) {
      mbar_init(BAR(B_PFULL + b), 4);  // one arrival per softmax warp
      mbar_init(BAR(B_SDONE + b), 1);
    }
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(BAR(B_KFULL + s), 1);
      mbar_init(BAR(B_VFULL + s), 1);
      mbar_init(BAR(B_KEMPTY + s), 1);
      mbar_init(BAR(B_VEMPTY + s), 1);
    }
    for (int s = 0; s < C::IRING; ++s) {
      mbar_init(BAR(B_ITF + s), 1);   // the scheduler
      mbar_init(BAR(B_ITE + s), 14 + (PAGED ? 1 : 0) + (C::TURNS ? 1 : 0));  // the warps that read it: producers, MMA, softmax, output
    }
    mbar_init(BAR(B_STAGE), 4);      // stage_full: one arrival per output warp
    mbar_init(BAR(B_STAGE + 1), 1);  // stage_free
    mbar_init(BAR(B_CANCEL), 1);
    mbar_init(BAR(B_NEAR), 1);
    mbar_init(BAR(B_DRAIN), C::TURNS ? 2 : 1);  // the issuing warps
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_u32((const void*)tmem_slot), C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The rows RT .. 127 of a query tile (G does not divide 128) hold whatever
  // shared memory held: rows are independent, and these are not written out.

  auto wait = [&](int b, uint32_t parity) { return wait_warp(BAR(b), parity, a.status, a.wait_limit_ns); };
  // Both at once (an answer takes a hundred cycles, and the products issued last
  // some hundreds), and whether any warp has given up.
  auto wait2 = [&](int b, uint32_t parity, int b2, uint32_t parity2) {
    const int gone = *abort_flag;
    const bool here = mbar_try_wait2(BAR(b), parity, BAR(b2), parity2);
    if (__all_sync(0xffffffffu, here && gone == 0)) return true;
    return !__any_sync(0xffffffffu, gone != 0) && wait(b, parity) && wait(b2, parity2);
  };
  // Waits for the i-th block of this CTA (a consuming warp; false if the wait
  // ran out), and reads of it, until release_item(i).
  auto get_item = [&](int i) { return wait(B_ITF + i % C::IRING, (i / C::IRING) & 1); };
  // (broadcast: the compiler keeps what is the same in all lanes, and what
  // follows from it, in uniform registers, where the products' operands go)
  auto item = [&](int i, int what) {
    return __shfl_sync(0xffffffffu, (int)items[(i % C::IRING) * C::ITEM_INTS + what], 0);
  };
  auto release_item = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(BAR(B_ITE + i % C::IRING));
  };

  if (warp < 4) {
    set_max_registers_dec<C::R_CONTROL>();
    // The i-th block of this CTA, found and published (warp 2): its own, then what
    // CTAs that have not begun leave to it. u: its index, -1 behind the last one.
    long long u = blockIdx.x;
    auto publish = [&](int i) {
      const int s = i % C::IRING;
      if (i >= C::IRING && !wait(B_ITE + s, ((i / C::IRING) - 1) & 1)) return false;
      if (i > 0) {
        // the CTA that would begin next gives its index to this one, if any is left
        if (lane == 0) {
          mbar_arrive_expect_tx(BAR(B_CANCEL), 16);
          clc_try_cancel(sbase + C::OFF_CANCEL, BAR(B_CANCEL));
        }
        if (!wait(B_CANCEL, (i - 1) & 1)) return false;
        u = clc_next_cta(sbase + C::OFF_CANCEL);
        fence_proxy_async_smem();  // read before the next answer is written there
        __syncwarp();
      }
      PromptBlock b;
      int part = 0;
      const long long asked = u;
      if (u >= 0 && !prompt_block(a, u, lane, u == 0, b, part)) u = -1;
      // for the merge: where the block's rows go and their ranges (no tokens:
      // there is no such block; the CTAs are at least as many as the blocks there can be)
      if (a.splits > 1 && asked >= 0 && part == 0 && lane == 0 && asked / b.parts < a.max_blocks * a.Hkv)
        a.blocks[asked / b.parts] = u >= 0 ? make_int4(b.v.q0 + b.tok0, b.v.n - b.tok0, b.head, b.parts) : make_int4(0, 0, 0, 0);
      if (lane == 0) {
        volatile int* d = items + s * C::ITEM_INTS;
        d[kItQ0] = b.v.q0;
        d[kItN] = b.v.n;
        d[kItHead] = b.head;
        d[kItTok0] = b.tok0;
        d[kItKt0] = b.kt0;
        d[kItN0] = u >= 0 ? b.n0 : -1;
        d[kItN1] = b.n1;
        d[kItPart] = b.unit * a.splits + part;
        d[kItK0] = b.v.k0;
        d[kItSeq] = b.seq;
        d[kItFirst] = b.v.m - b.v.n + b.tok0 + 1 - b.kt0 * C::BN;
        d[kItLeft] = b.v.m - b.kt0 * C::BN;
        mbar_arrive(BAR(B_ITF + s));
      }
      __syncwarp();
      return true;
    };
    if (!PAGED && warp == 2) {
      // ---------------------------------------------------------- scheduler
      bool ok = true;
      for (int i = 0; ok && u >= 0; ++i) {
        // Not before the block in work is near its end: a CTA with a long one would
        // hold the next back from those that run dry.
        if (i > 0) ok = wait(B_NEAR, (i - 1) & 1);
        ok = ok && publish(i);
      }
      if (!ok) *abort_flag = 1;
    } else if (warp == 0 || warp == 2) {
      // ---------------------------------------------------------- producers
      // Of packed tensors warp 0 loads all. Of pages warp 2 loads V, and publishes
      // the next block behind a block's last load: with pages of 32 keys a tile
      // takes four boxes of each, whose issue by one warp is longer than the tile's
      // softmax (six chats' next turns, d = 64: 106 us, 97 with two warps; of packed
      // tensors two warps are slower, 1160 TFLOP/s to 1197).
      // One lane issues the packed tensors' boxes; a paged cache's boxes have a
      // lane each (box `box` of the 64-column chunk `chunk` of a tile).
      const int nbox = PAGED ? C::BN / a.box_rows : 1;
      const bool mine = PAGED ? lane < nbox * C::CH : lane == 0;
      const int box = PAGED ? lane % nbox : 0, chunk = PAGED ? lane / nbox : 0;
      const bool of_k = warp == 0;
      const CUtensorMap* map = of_k ? &a.tmK : &a.tmV;
      const int ring = of_k ? C::OFF_K : C::OFF_V, full = of_k ? B_KFULL : B_VFULL, empty = of_k ? B_KEMPTY : B_VEMPTY;
      if (lane == 0) {
        if (of_k) tma_prefetch_desc(&a.tmQ);
        tma_prefetch_desc(map);
        if (!PAGED) tma_prefetch_desc(&a.tmV);
      }
      bool ok = of_k || publish(0);
      int g0 = 0, q0_used = 0, q1_used = 0;  // key tiles, and loads of each Q slot, before this block
      int last = -1, last_v = -1;            // last tiles whose loads were issued, by ring position
      for (int i = 0; ok; ++i) {
        if (!get_item(i)) { ok = false; break; }
        const int n0 = item(i, kItN0), n1 = item(i, kItN1), n_max = max(n0, n1);
        if (n0 < 0) break;
        const int kt0 = item(i, kItKt0), left = item(i, kItLeft), head = item(i, kItHead);
        const int key0 = item(i, kItK0) + kt0 * C::BN, tok = item(i, kItQ0) + item(i, kItTok0);
        const int* table = PAGED ? a.block_tables + (size_t)item(i, kItSeq) * a.max_pages : nullptr;
        // a lane's page and first row of key tile j; row = -1: it has no box there
        auto look_up = [&](int j, int& page, int& row) {
          page = 0;
          row = -1;
          if constexpr (PAGED) {
            const int key = j * C::BN + box * a.box_rows;  // from kt0 on
            if (mine && key < left) {
              const int at = kt0 * C::BN + key, pi = a.page_div(at);
              row = at - pi * a.pool.page_size;
              page = __ldg(table + pi);  // first used a tile later
            }
          }
        };
        // bytes of a tile's boxes that hold keys of the sequence
        auto tile_bytes = [&](int j) {
          if constexpr (!PAGED) return (uint32_t)C::TILE_BYTES;
          const int keys = left - j * C::BN;
          const int boxes = keys >= C::BN ? nbox : (keys + a.box_rows - 1) / a.box_rows;
          return (uint32_t)(boxes * a.box_rows * 128 * C::CH);
        };
        // tile j of K or V into its ring's slot, once that is free
        auto load = [&](const CUtensorMap* map, int ring, int full, int empty, int j, int page, int row, int& at) {
          const int g = g0 + j, s = g % C::STAGES;
          if (!wait(empty + s, ((g / C::STAGES) & 1) ^ 1)) return false;
          if (lane == 0) mbar_arrive_expect_tx(BAR(full + s), tile_bytes(j));
          __syncwarp();
          const uint32_t dst = sbase + ring + s * C::TILE_BYTES;
          if constexpr (PAGED) {
            if ((unsigned)page >= (unsigned)a.pool.num_pages) {
              report_status(a.status, kStatusBadSeqlens);
              page = a.pool.num_pages;  // outside the tensor: reads as zeros
            }
            if (row >= 0)
              tma_load_4d(dst + chunk * C::CHUNK_BYTES + box * a.box_rows * 128, map, BAR(full + s), chunk * 64, row, head, page);
          } else if (lane == 0) {
            for (int c = 0; c < C::CH; ++c)
              tma_load_3d(dst + c * C::CHUNK_BYTES, map, BAR(full + s), c * 64, key0 + j * C::BN, head);
          }
          at = g;
          return true;
        };
        auto load_q = [&](int t, int& used) {  // once the block before has read the slot
          if ((t == 0 ? n0 : n1) == 0) return true;
          if (used > 0 && !wait(B_QEMPTY + t, (used - 1) & 1)) return false;
          ++used;
          if (lane == 0) {
            mbar_arrive_expect_tx(BAR(B_QFULL + t), (uint32_t)(RT * 128 * C::CH));
            for (int c = 0; c < C::CH; ++c)
              tma_load_4d(sbase + C::OFF_Q + (t * C::CH + c) * C::CHUNK_BYTES, &a.tmQ, BAR(B_QFULL + t), c * 64, 0,
                          tok + t * TP, head);
          }
          __syncwarp();
          return true;
        };
        int page, row;
        look_up(0, page, row);
        for (int j = 0; j < n_max; ++j) {
          if (__any_sync(0xffffffffu, *abort_flag != 0)) { ok = false; break; }
          int next_page = 0, next_row = -1;
          if (j + 1 < n_max) look_up(j + 1, next_page, next_row);
          ok = load(map, ring, full, empty, j, page, row, last);
          if (of_k && j == 0) ok = ok && load_q(0, q0_used) && load_q(1, q1_used);
          if constexpr (!PAGED) ok = ok && load(&a.tmV, C::OFF_V, B_VFULL, B_VEMPTY, j, page, row, last_v);
          if (!ok) break;
          page = next_page;
          row = next_row;
          if (!PAGED && j == max(0, n_max - 3) && lane == 0) mbar_arrive(BAR(B_NEAR));
        }
        if (!ok) break;
        if (!PAGED && n_max == 0 && lane == 0) mbar_arrive(BAR(B_NEAR));
        if (!of_k && !publish(i + 1)) { ok = false; break; }
        g0 += n_max;
        release_item(i);
      }
      if (!ok) *abort_flag = 1;
      // drain: what was asked for last must have landed before exit
      if (q0_used > 0) wait(B_QFULL + 0, (q0_used - 1) & 1);
      if (q1_used > 0) wait(B_QFULL + 1, (q1_used - 1) & 1);
      for (int g = max(0, last - C::STAGES + 1); g <= last; ++g) wait(full + g % C::STAGES, (g / C::STAGES) & 1);
      for (int g = max(0, last_v - C::STAGES + 1); g <= last_v; ++g) wait(B_VFULL + g % C::STAGES, (g / C::STAGES) & 1);
    } else if (warp == 1 || (C::TURNS && warp == 3)) {
      // ---------------------------------------------------------- MMA issuer
      // A product is issued as the one three before it ends, so the issuing warp
      // has some hundred cycles between two waits, each of which takes as long.
      // With S in turns, warp 1 issues the S products and warp 3 the P V.
      const uint32_t leader = elect_one();
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, D, false, true);
      const uint64_t dQ0 = sdesc_sw128(sbase + C::OFF_Q, 16, 1024);
      const uint64_t dK0 = sdesc_sw128(sbase + C::OFF_K, 16, 1024);
      const uint64_t dV0 = sdesc_sw128(sbase + C::OFF_V, C::CHUNK_BYTES, 1024);
      // S of tile t against the keys in slot s, into buffer b, told by the tile's
      // barrier f; `last`: the block's last for this tile
      auto issue_s = [&](int t, int s, int b, int f, bool last) {
        const uint64_t qa = dQ0 + (uint64_t)((t * C::TILE_BYTES) >> 4);
        const uint64_t kb = dK0 + (uint64_t)((s * C::TILE_BYTES) >> 4);
        const uint32_t dcol = tmem + C::S_COL(b);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk >> 2) * C::CHUNK_BYTES + (kk & 3) * 32) >> 4);
          mma_ss(dcol, qa + off, kb + off, idesc_s, kk > 0 ? 1u : 0u, leader);
        }
        mma_commit(BAR(B_SFULL + t * C::SFULLS + f), leader);
        if (last) mma_commit(BAR(B_QEMPTY + t), leader);
      };
      // P V over a whole tile, and over the first `keys` keys (those that the
      // tile's last query sees) in steps of 16
      auto issue_pv = [&](int t, int s, int b, bool acc) {
        const uint64_t vb = dV0 + (uint64_t)((s * C::TILE_BYTES) >> 4);
        const uint32_t dcol = tmem + C::O_COL(t), acol = tmem + C::S_COL(b);
#pragma unroll
        for (int kk = 0; kk < C::BN / 16; ++kk)
          mma_ts(dcol, acol + kk * 8, vb + (uint64_t)((kk * 2048) >> 4), idesc_o, (acc || kk > 0) ? 1u : 0u, leader);
        if constexpr (C::TURNS) mma_commit(BAR(B_SDONE + b), leader);
      };
      auto issue_pv_keys = [&](int t, int s, int b, bool acc, int keys) {
        const uint64_t vb = dV0 + (uint64_t)((s * C::TILE_BYTES) >> 4);
        const uint32_t dcol = tmem + C::O_COL(t), acol = tmem + C::S_COL(b);
#pragma unroll 1
        for (int kk = 0; kk < C::BN / 16 && 16 * kk < keys; ++kk)
          mma_ts(dcol, acol + kk * 8, vb + (uint64_t)((kk * 2048) >> 4), idesc_o, (acc || kk > 0) ? 1u : 0u, leader);
        if constexpr (C::TURNS) mma_commit(BAR(B_SDONE + b), leader);
      };
      // V has landed in slot s with `keys` keys of the sequence: rows behind them
      // that the last step would read become zero.
      auto clean_v = [&](int s, int keys) {
        if (keys < C::BN && (keys & 15) != 0) {
          const int n_rows = 16 - (keys & 15);
          for (int e = lane; e < n_rows * C::CH * 8; e += 32) {
            const int r = keys + e / (C::CH * 8), u = e % (C::CH * 8);
            *reinterpret_cast<uint4*>(smem + C::OFF_V + s * C::TILE_BYTES + (u >> 3) * C::CHUNK_BYTES + r * 128 +
                                      (u & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
      };
      bool ok = true;
      if constexpr (C::TURNS) {
        // The (key tile, query tile) pairs in order, tile 0 before tile 1, block
        // after block: pair x has S buffer x % 3.
        int g0 = 0;                      // key tiles before the block
        int used0 = 0, used1 = 0;        // blocks with such a tile before it
        int buf = 0;                     // the next pair's buffer,
        uint32_t turn = warp == 1 ? 1u : 0u;  // and the parity that it waits for (S of the first round: for nothing)
        int f0 = 0, f1 = 0;              // the next S's barrier, by query tile
        auto next_buffer = [&]() {
          turn ^= buf == C::SBUF - 1;
          buf = buf == C::SBUF - 1 ? 0 : buf + 1;
        };
#pragma unroll 1
        for (int i = 0; ok; ++i) {
          ok = get_item(i);
          if (!ok) break;
          const int n0 = item(i, kItN0), n1 = item(i, kItN1), n_max = max(n0, n1);
          if (n0 < 0) break;
          if (warp == 1) {
            if (n0 > 0) ok = wait(B_QFULL, used0 & 1);
            if (n1 > 0) ok = ok && wait(B_QFULL + 1, used1 & 1);
            int j = 0;
            // whole tiles of both, in as few instructions as can be: with the
            // softmax warps beside it each takes this warp ten cycles
#pragma unroll 1
            for (const int n = min(n0, n1) - 1; ok && j < n; ++j) {
              const int g = g0 + j, s = g % C::STAGES;
              ok = wait2(B_KFULL + s, (g / C::STAGES) & 1, B_SDONE + buf, turn);
              if (!ok) break;
              tc_fence_after();
              issue_s(0, s, buf, f0, false);
              f0 = f0 == C::SFULLS - 1 ? 0 : f0 + 1;
              next_buffer();
              ok = wait(B_SDONE + buf, turn);
              if (!ok) break;
              tc_fence_after();
              issue_s(1, s, buf, f1, false);
              mma_commit(BAR(B_KEMPTY + s), leader);
              f1 = f1 == C::SFULLS - 1 ? 0 : f1 + 1;
              next_buffer();
            }
#pragma unroll 1
            for (; ok && j < n_max; ++j) {
              const int g = g0 + j, s = g % C::STAGES;
              const uint32_t pk = (g / C::STAGES) & 1;
              if (j < n0) {
                ok = wait2(B_KFULL + s, pk, B_SDONE + buf, turn);
                if (!ok) break;
                tc_fence_after();
                issue_s(0, s, buf, f0, j + 1 == n0);
                f0 = f0 == C::SFULLS - 1 ? 0 : f0 + 1;
                next_buffer();
              }
              if (j < n1) {
                ok = wait2(B_KFULL + s, pk, B_SDONE + buf, turn);
                if (!ok) break;
                tc_fence_after();
                issue_s(1, s, buf, f1, j + 1 == n1);
                f1 = f1 == C::SFULLS - 1 ? 0 : f1 + 1;
                next_buffer();
              }
              mma_commit(BAR(B_KEMPTY + s), leader);
            }
          } else {
            const int first = item(i, kItFirst) - 1, left = item(i, kItLeft);
            // the accumulators have left tensor memory
            if (n0 > 0 && used0 > 0) ok = wait(B_OFREE, (used0 - 1) & 1);
            if (n1 > 0 && used1 > 0) ok = ok && wait(B_OFREE + 1, (used1 - 1) & 1);
            int j = 0;
#pragma unroll 1
            while (ok && j < n_max) {
              const int g = g0 + j, s = g % C::STAGES;
              const uint32_t pv = (g / C::STAGES) & 1;
              if (j > 0 && j + 1 < min(n0, n1)) {  // as above
                ok = wait2(B_VFULL + s, pv, B_PFULL + buf, turn);
                if (!ok) break;
                tc_fence_after();
                issue_pv(0, s, buf, true);
                next_buffer();
                ok = wait(B_PFULL + buf, turn);
                if (!ok) break;
                tc_fence_after();
                issue_pv(1, s, buf, true);
                mma_commit(BAR(B_VEMPTY + s), leader);
                next_buffer();
                ++j;
                continue;
              }
              bool clean = false;
#pragma unroll 1
              for (int t = 0; t < C::QT; ++t) {
                const int nt = t == 0 ? n0 : n1;
                if (j >= nt) continue;
                ok = wait2(B_VFULL + s, pv, B_PFULL + buf, turn);
                if (!ok) break;
                if (!clean) clean_v(s, left - j * C::BN);
                clean = true;
                tc_fence_after();
                const int keys = min(first + (t + 1) * TP, left) - j * C::BN;
                if (keys >= C::BN) issue_pv(t, s, buf, j > 0);
                else issue_pv_keys(t, s, buf, j > 0, keys);
                if (j + 1 == nt) mma_commit(BAR(B_ODONE + t), leader);
                next_buffer();
              }
              mma_commit(BAR(B_VEMPTY + s), leader);
              ++j;
            }
          }
          if (!ok) break;
          used0 += n0 > 0;
          used1 += n1 > 0;
          g0 += n_max;
          release_item(i);
        }
      } else {
        ok = get_item(0);
        int n0 = item(0, kItN0), n1 = item(0, kItN1);  // key tiles of the block's query tiles
        int g0 = 0;              // key tiles before this block
        int c0 = 0, c1 = 0;      // key tiles of query tiles 0 and 1 before it
        int q0_used = 0, q1_used = 0;  // blocks with such a tile before it
        int s_done = 0;  // bit t: the block's first S of tile t has been issued
        // The first S of tile t (of nt key tiles) of a block whose keys begin at ring position g
        // (`now`: only if its operands are there).
        auto first_s = [&](int t, int nt, int g, bool now) {
          if (nt == 0 || (s_done >> t & 1)) return true;
          const int s = g % C::STAGES;
          const uint32_t pk = (g / C::STAGES) & 1, pq = (t == 0 ? q0_used : q1_used) & 1;
          if (now && !__all_sync(0xffffffffu, mbar_test(BAR(B_KFULL + s), pk) && mbar_test(BAR(B_QFULL + t), pq)))
            return true;
          if (!now && !(wait(B_KFULL + s, pk) && wait(B_QFULL + t, pq))) return false;
          tc_fence_after();
          issue_s(t, s, t, 0, nt == 1);
          if (t == 0) ++q0_used;
          else ++q1_used;
          s_done |= 1 << t;
          return true;
        };
        for (int i = 0; ok && n0 >= 0; ++i) {
          const int n_max = max(n0, n1);
          int next0 = -1, next1 = 0;
          bool fetched = false;
          auto fetch = [&]() {
            if (!fetched && !get_item(i + 1)) return false;
            next0 = item(i + 1, kItN0);
            next1 = item(i + 1, kItN1);
            return fetched = true;
          };
#pragma unroll 1
          for (int t = 0; ok && t < C::QT; ++t) ok = first_s(t, t == 0 ? n0 : n1, g0, false);
          if (!ok) break;
          s_done = 0;
          // before the block's first P V: the accumulator has left tensor memory
          auto o_free = [&](int t, int j) {
            const int used = t == 0 ? q0_used : q1_used;
            return j > 0 || used <= 1 || wait(B_OFREE + t, used & 1);
          };
          if (n_max > 0) mma_commit(BAR(B_KEMPTY + g0 % C::STAGES), leader);
          // The tiles that neither query tile ends near: whole keys, a next S for
          // both. The loop is kept short (a wait and sixteen products per tile):
          // what its warp does between two waits, and what it does to the
          // instruction cache, is on the path from one softmax to the next
          // (16384 tokens, 32 heads, d = 128: 1385 TFLOP/s with the last tiles'
          // cases in it).
          const int n_lean = min(n0, n1) - 2;
          int j = 0;
#pragma unroll 1
          for (; j < n_lean; ++j) {
            const int g = g0 + j, s = g % C::STAGES, s1 = (g + 1) % C::STAGES;
            const uint32_t ph1 = ((g + 1) / C::STAGES) & 1;
            ok = wait2(B_VFULL + s, (g / C::STAGES) & 1, B_PFULL, (uint32_t)(c0 + j) & 1u);
#pragma unroll
            for (int t = 0; t < C::QT; ++t) {
              ok = ok && (t == 0 || wait(B_PFULL + 1, (uint32_t)(c1 + j) & 1u)) && o_free(t, j);
              if (!ok) break;
              tc_fence_after();
              issue_pv(t, s, t, j > 0);
              if (t == 0) {
                ok = wait(B_KFULL + s1, ph1);
                if (!ok) break;
                tc_fence_after();
              }
              issue_s(t, s1, t, 0, false);
            }
            if (!ok) break;
            mma_commit(BAR(B_VEMPTY + s), leader);
            mma_commit(BAR(B_KEMPTY + s1), leader);
          }
          if (!ok) break;
#pragma unroll 1
          for (; j < n_max; ++j) {
            if (__any_sync(0xffffffffu, *abort_flag != 0)) { ok = false; break; }
            const int g = g0 + j, s = g % C::STAGES, s1 = (g + 1) % C::STAGES;
            const uint32_t ph = (g / C::STAGES) & 1, ph1 = ((g + 1) / C::STAGES) & 1;
            bool k_next = false, v_here = false;  // K_{j+1}, V_j have landed
            auto need_v = [&]() {
              if (!v_here) {
                if (!wait(B_VFULL + s, ph)) return false;
                clean_v(s, item(i, kItLeft) - j * C::BN);
              }
              return v_here = true;
            };
            auto next_s = [&](int t) {
              if (!k_next && !wait(B_KFULL + s1, ph1)) return false;
              k_next = true;
              tc_fence_after();
              issue_s(t, s1, t, 0, j + 2 == (t == 0 ? n0 : n1));
              return true;
            };
#pragma unroll 1
            for (int t = 0; t < C::QT; ++t) {
              const uint32_t pt = (uint32_t)((t == 0 ? c0 : c1) + j) & 1u;
              const int nt = t == 0 ? n0 : n1;
              if (j < nt) {
                const bool more = j + 1 < nt;
                // keys of this tile that the query tile's last query sees
                const int keys = min(item(i, kItFirst) - 1 + (t + 1) * TP, item(i, kItLeft)) - j * C::BN;
                // P overwrites S: P_j V_j must be issued before S_{j+1}
                if (!need_v() || !wait(B_PFULL + t, pt) || !o_free(t, j)) { ok = false; break; }
                tc_fence_after();
                issue_pv_keys(t, s, t, j > 0, keys);
                if (!more) mma_commit(BAR(B_ODONE + t), leader);
                if (more && !next_s(t)) { ok = false; break; }
              }
              if (j + 1 == n_max) {
                // this tile is done with the block: the next block's first S, if
                // its operands are there already
                if (!fetch()) { ok = false; break; }
                if (next0 >= 0 && !first_s(t, t == 0 ? next0 : next1, g0 + n_max, true)) {
                  ok = false;
                  break;
                }
              }
            }
            if (!ok) break;
            mma_commit(BAR(B_VEMPTY + s), leader);
            if (j + 1 < n_max) mma_commit(BAR(B_KEMPTY + s1), leader);
          }
          if (!ok || !fetch()) { ok = false; break; }
          release_item(i);
          g0 += n_max;
          c0 += n0;
          c1 += n1;
          n0 = next0;
          n1 = next1;
        }
      }
      if (!ok && lane == 0) *abort_flag = 1;
      // drain every MMA issued before TMEM can be released
      mma_commit(BAR(B_DRAIN), leader);
      wait(B_DRAIN, 0);
    }
  } else if (warp < 12) {
    set_max_registers_inc<C::R_SOFTMAX>();
    // -------------------------------------------------------------- softmax
    const int t = (warp - 4) >> 2;  // query tile of this warpgroup
    const int wq = warp & 3;             // TMEM lane quarter
    const int row = wq * 32 + lane;      // row of the tile
    const uint32_t lane_addr = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t o_addr = lane_addr + C::O_COL(t);
    const float c2 = a.scale_log2;
    const uint64_t c22 = f2_pack(c2, c2);
    bool ok = true;
    int c = 0, pairs = 0;  // key tiles of this query tile, and of both, before the block
    for (int i = 0; ok; ++i) {
      int n_own, sees, first;  // keys from kt0 on that this row and the tile's first row see
      if (!get_item(i)) { ok = false; break; }
      const int n0 = item(i, kItN0), n1 = item(i, kItN1), both = min(n0, n1);
      if (n0 < 0) break;
      n_own = t == 0 ? n0 : n1;
      // TURNS: the place of key tile j among the pairs of key and query tiles
      auto pair = [&](int j) { return pairs + j + (j < both ? j + t : both); };
      first = item(i, kItFirst) + t * TP;
      sees = min(first + a.g_div(row), item(i, kItLeft));
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < n_own; ++j) {
        if (__any_sync(0xffffffffu, *abort_flag != 0)) { ok = false; break; }
        const int buf = C::TURNS ? pair(j) % C::SBUF : t;
        const uint32_t s_addr = lane_addr + C::S_COL(buf);
        const bool w = wait_phase(BAR(B_SFULL + t * C::SFULLS + (c + j) % C::SFULLS), ((c + j) / C::SFULLS) & 1, a.status,
                                  a.wait_limit_ns);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        tc_fence_after();
        // the diagonal of the tile's first query decides whether any row has
        // masked columns here
        const bool mask_tile = first - j * C::BN < C::BN;
        const int valid = sees - j * C::BN;
        if (mask_tile || j == 0) {
          // A few tiles to a block: masked scores are replaced where they stand
          // (no mask in the pass below), and the first tile's maximum is the
          // row's first reference.
          float top = -INFINITY;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t r[32];
            tmem_ld32(s_addr + 32 * q, r);
            tmem_ld_wait();
            if (mask_tile) {
              mask_cols32(r, 32 * q, valid);
              tmem_st32(s_addr + 32 * q, r);
            }
#pragma unroll
            for (int u = 0; u < 16; ++u) top = fmax3(top, __uint_as_float(r[2 * u]), __uint_as_float(r[2 * u + 1]));
          }
          if (j == 0) m_ref = top * c2;
          if (mask_tile) tmem_st_wait();
        }
        // The speculative pass against the reference max of the tiles before, the
        // tile's own max alongside; a tile whose max exceeds it by more than
        // kRescaleLog2 is done again. A row that has met no key yet has m_ref =
        // -inf: what is added to its scores, -inf, is 0.
        float mx[4];
        uint64_t sm2[4];
        float alpha = 1.f;
        bool moved = false;
        uint32_t pk[64];
#pragma unroll 1
        while (true) {
#pragma unroll
          for (int u = 0; u < 4; ++u) { mx[u] = -INFINITY; sm2[u] = 0ull; }
          const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
          const uint64_t nm2 = f2_pack(neg, neg);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r[64];  // 64 columns of S at a time
            tmem_ld32(s_addr + 64 * h, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
            tmem_ld32(s_addr + 64 * h + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < 32; ++u) {
              const float x0 = __uint_as_float(r[2 * u]), x1 = __uint_as_float(r[2 * u + 1]);
              mx[u & 3] = fmax3(mx[u & 3], x0, x1);
              const float2 x = f2_unpack(ffma2(f2_pack(x0, x1), c22, nm2));
              const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
              sm2[u & 3] = fadd2(sm2[u & 3], f2_pack(p0, p1));
              pk[32 * h + u] = pack_bf16x2(p0, p1);
            }
          }
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
          const bool need = mt > m_ref + kRescaleLog2;
          if (!__any_sync(0xffffffffu, need)) break;
          if (need) {
            alpha = ex2_approx(m_ref - mt);
            m_ref = mt;
          }
          moved = true;
        }
        tmem_st32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
        tmem_st32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
        const float2 sa = f2_unpack(fadd2(fadd2(sm2[0], sm2[1]), fadd2(sm2[2], sm2[3])));
        l = l * alpha + (sa.x + sa.y);
        // O can be rescaled once P V of the tile before is complete: with a buffer
        // for each query tile it is, since S has come behind it in the same buffer
        if (j > 0 && moved) {
          if constexpr (C::TURNS) {
            const bool d = wait_phase(BAR(B_SDONE + pair(j - 1) % C::SBUF), (pair(j - 1) / C::SBUF) & 1, a.status,
                                      a.wait_limit_ns);
            if (!__all_sync(0xffffffffu, d)) { ok = false; break; }
            tc_fence_after();
          }
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(o_addr + 32 * q, o);
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
            tmem_st32(o_addr + 32 * q, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_PFULL + buf));
      }
      tmem_st_wait();  // no TMEM store may be in flight when the loop is left early
      if (!ok) break;
      c += n_own;
      pairs += n0 + n1;
      // the row's sum goes to the output warps, its log-sum-exp out from here
      reinterpret_cast<float*>(smem + C::OFF_STAT)[((i & 1) * 2 + t) * 128 + row] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_LFULL + 2 * t + (i & 1)));
      const float lse2 = m_ref + __log2f(l);  // -inf for a row without keys
      const int n = item(i, kItN), tok0 = item(i, kItTok0) + t * TP, tok_in = a.g_div(row);
      if (a.splits > 1) {
        if (tok0 < n) a.Lpart[((long long)item(i, kItPart) * 2 + t) * C::BM + row] = lse2;
      } else {
        const int q0 = item(i, kItQ0), hq0 = item(i, kItHead) * a.G;
        if (row < RT && tok0 + tok_in < n)
          a.LSE[(size_t)(hq0 + row - tok_in * a.G) * a.seqs.total_q + q0 + tok0 + tok_in] = lse2 * 0.69314718055994531f;
      }
      release_item(i);
    }
    if (!ok) *abort_flag = 1;
  } else {
    set_max_registers_dec<C::R_OUT>();
    // -------------------------------------------------------------- output
    // O of both tiles leaves tensor memory here, so that the softmax warps go on
    // to the next block at once, whose first P V follows two microseconds later:
    // by then the accumulators have to be free. So a tile is staged as fast as
    // it can be read, and a TMA store takes it out of the staging buffer.
    const int wq = warp & 3;
    const uint32_t lane_addr = tmem + ((uint32_t)(wq * 32) << 16);
    const int row = wq * 32 + lane;
    const int rsub = lane >> 3, unit = lane & 7;
    bool ok = true;
    int o0_used = 0, o1_used = 0;  // blocks with such a tile before
    int staged = 0;      // tiles staged so far
    if (lane == 0 && wq == 0) tma_prefetch_desc(&a.tmO);
    for (int i = 0; ok; ++i) {
      if (!get_item(i)) { ok = false; break; }
      const int n0 = item(i, kItN0), n1 = item(i, kItN1);
      if (n0 < 0) break;
      const int n = item(i, kItN);
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        const int n_own = t == 0 ? n0 : n1, tok0 = item(i, kItTok0) + t * TP;
        // the row's sum, then its last P V
        if (!wait(B_LFULL + 2 * t + (i & 1), (i >> 1) & 1)) { ok = false; break; }
        const float l = reinterpret_cast<const float*>(smem + C::OFF_STAT)[((i & 1) * 2 + t) * 128 + row];
        if (tok0 >= n) continue;  // no such tile
        const bool any = n_own > 0, some = any && l != 0.f;
        const float inv_l = some ? 1.f / l : 0.f;
        const uint32_t o_addr = lane_addr + C::O_COL(t);
        // 32 columns of the row, normalised (zeros for a row without keys)
        auto read_o = [&](int q, uint32_t (&r)[32]) {
          if (any) {
            tmem_ld32(o_addr + 32 * q, r);
            tmem_ld_wait();
          }
#pragma unroll
          for (int u = 0; u < 32; ++u) r[u] = some ? __float_as_uint(__uint_as_float(r[u]) * inv_l) : 0u;
        };
        auto free_o = [&]() {  // the tensor memory has been read
          tc_fence_before();
          __syncwarp();
          if (any && lane == 0) mbar_arrive(BAR(B_OFREE + t));
        };
        if (any) {
          int& used = t == 0 ? o0_used : o1_used;
          if (!wait(B_ODONE + t, used & 1)) { ok = false; break; }
          ++used;
        }
        tc_fence_after();
        if (a.splits > 1) {
          // fp32 rows of this key range (one without keys leaves only its
          // log-sum-exp), 128 bytes of each row of the warp at a time
          const long long prow0 = ((long long)item(i, kItPart) * 2 + t) * C::BM + wq * 32;
          uint8_t* stage = smem + C::OFF_STAGE + wq * (32 * 128);
          if (any) {
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              uint32_t r[32];
              read_o(q, r);
#pragma unroll
              for (int u = 0; u < 8; ++u)
                *reinterpret_cast<uint4*>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) =
                    make_uint4(r[4 * u], r[4 * u + 1], r[4 * u + 2], r[4 * u + 3]);
              __syncwarp();
#pragma unroll
              for (int u = 0; u < 8; ++u) {
                const int rr = 4 * u + rsub;
                const float4 y = *reinterpret_cast<const float4*>(stage + rr * 128 + ((unit ^ (rr & 7)) << 4));
                *reinterpret_cast<float4*>(a.Opart + (prow0 + rr) * D + 32 * q + 4 * unit) = y;
              }
              __syncwarp();
            }
          }
          free_o();
          continue;
        }
        // the tile before has left the staging buffer
        if (staged > 0 && !wait(B_STAGE + 1, (staged - 1) & 1)) { ok = false; break; }
        uint8_t* stage = smem + C::OFF_STAGE;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t r[32];
          read_o(q, r);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            *reinterpret_cast<uint4*>(stage + (q >> 1) * C::CHUNK_BYTES + row * 128 + (((4 * (q & 1) + u) ^ (row & 7)) << 4)) =
                make_uint4(pack_bf16x2(__uint_as_float(r[8 * u]), __uint_as_float(r[8 * u + 1])),
                           pack_bf16x2(__uint_as_float(r[8 * u + 2]), __uint_as_float(r[8 * u + 3])),
                           pack_bf16x2(__uint_as_float(r[8 * u + 4]), __uint_as_float(r[8 * u + 5])),
                           pack_bf16x2(__uint_as_float(r[8 * u + 6]), __uint_as_float(r[8 * u + 7])));
        }
        free_o();
        const long long tok_q = item(i, kItQ0) + tok0;
        const int head = item(i, kItHead);
        const bool whole = tok0 + TP <= n;
        if (whole) {
          fence_proxy_async_smem();
        } else {
          // a sequence's last, partial tile: the warp's rows, 16 lanes to one
          constexpr int LPR = D / 8;
          const int x = lane % LPR;
#pragma unroll 1
          for (int k = 0; k < 32; k += 32 / LPR) {
            const int tr = wq * 32 + k + lane / LPR, tk = a.g_div(tr);
            const uint4 y = *reinterpret_cast<const uint4*>(stage + (x >> 3) * C::CHUNK_BYTES + tr * 128 +
                                                            (((x & 7) ^ (tr & 7)) << 4));
            if (tr < RT && tok0 + tk < n)
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.O) + (tok_q + tk) * a.o_stride +
                                        (long long)(head * a.G + tr - tk * a.G) * D + 8 * x) = y;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_STAGE));
        if (wq == 0) {
          if (!wait(B_STAGE, staged & 1)) { ok = false; break; }
          if (lane == 0) {
            if (whole) {
#pragma unroll
              for (int c = 0; c < C::CH; ++c)
                tma_store_4d(&a.tmO, sbase + C::OFF_STAGE + c * C::CHUNK_BYTES, c * 64, 0, (int)tok_q, head);
              bulk_commit_group();
              bulk_wait_group_read<0>();
            }
            mbar_arrive(BAR(B_STAGE + 1));
          }
          __syncwarp();
        }
        ++staged;
      }
      if (ok) release_item(i);
    }
    if (!ok) *abort_flag = 1;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Combines the key ranges of a block: row r gets O = sum_p w_p O_p / sum_p w_p
// with w_p = 2^(L_p - max L), LSE = (max L + log2 sum_p w_p) ln 2. One CTA per
// 64 rows of a block, eight rows to a warp (lanes along d, their loads in flight
// together), ranges without keys (L = -inf) not read.
template <int D>
__global__ void __launch_bounds__(256) prompt_merge_kernel(const __grid_constant__ PromptFwdArgs a) {
  constexpr int ROWS = 8, LPR = D / 4, RPW = 32 / LPR, STEPS = ROWS / RPW;  // rows of a warp, lanes to a row, rows at once
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  const int unit = (int)(blockIdx.x >> 2);
  const int4 k = a.blocks[unit];  // first packed token, tokens of the sequence from there on, K/V head, key ranges
  const int br0 = (int)(blockIdx.x & 3) * 64 + warp * ROWS;  // rows of the block, of one query tile
  const int t = br0 >> 7, row0 = br0 & 127;
  // what a launch that gave up left unwritten is not followed
  if (k.x < 0 || k.y > a.seqs.total_q - k.x || (unsigned)k.z >= (unsigned)a.Hkv || k.w > a.splits) return;
  // the rows that there are begin the eight: rows of a sequence's end lack the last ones
  const int live = min(ROWS, min(a.tile_tokens, k.y - t * a.tile_tokens) * a.G - row0);
  if (live <= 0) return;
  const long long p0 = (long long)unit * a.splits * 256 + br0 + sub;
  const float* lpart = a.Lpart + p0;
  const float4* opart = reinterpret_cast<const float4*>(a.Opart + p0 * D) + l;
  float top[STEPS], sum[STEPS];
  float4 acc[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    top[i] = -INFINITY;
    sum[i] = 0.f;
    acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int p = 0; p < k.w; ++p) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) top[i] = fmaxf(top[i], lpart[p * 256 + i * RPW]);  // rows past `live`: any value
  }
  for (int p = 0; p < k.w; ++p) {
    float lp[STEPS];
    float4 x[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      lp[i] = i * RPW + sub < live ? lpart[i * RPW] : -INFINITY;
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (lp[i] != -INFINITY) x[i] = opart[i * RPW * LPR];
    }
    lpart += 256;
    opart += 256 * LPR;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      if (lp[i] == -INFINITY) continue;
      const float w = ex2_approx(lp[i] - top[i]);
      sum[i] += w;
      if (!(w > 0.f)) continue;  // nothing of what is too small, an infinity included
      acc[i].x = fmaf(w, x[i].x, acc[i].x);
      acc[i].y = fmaf(w, x[i].y, acc[i].y);
      acc[i].z = fmaf(w, x[i].z, acc[i].z);
      acc[i].w = fmaf(w, x[i].w, acc[i].w);
    }
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int r = i * RPW + sub;
    if (r >= live) break;
    const int row = row0 + r, tk = a.g_div(row), hq = k.z * a.G + row - tk * a.G;
    const long long tok = k.x + t * a.tile_tokens + tk;
    const float inv = sum[i] == 0.f ? 0.f : 1.f / sum[i];
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.O) + tok * a.o_stride + (long long)hq * D + 4 * l) =
        make_uint2(pack_bf16x2(acc[i].x * inv, acc[i].y * inv), pack_bf16x2(acc[i].z * inv, acc[i].w * inv));
    if (l == 0) a.LSE[(size_t)hq * a.seqs.total_q + tok] = (top[i] + __log2f(sum[i])) * 0.69314718055994531f;
  }
}

template <int D, bool PAGED>
cudaError_t launch_d(const PromptFwdArgs& a, cudaStream_t st) {
  using C = PromptCfg<D>;
  static_assert(C::BYTES <= C::MOST, "shared memory budget");
  const long long ctas = a.max_blocks * a.Hkv * a.splits;
  if (a.splits < 1 || a.max_blocks < 1 || ctas > 0x7fffffffll || (a.splits > 1 && (!a.Opart || !a.Lpart)))
    return cudaErrorInvalidValue;
  static std::atomic<unsigned char> asked[kMaxSharedMemoryDevices];
  cudaError_t e = ask_shared_memory(reinterpret_cast<const void*>(prompt_fwd_kernel<D, PAGED>), C::ALLOC, asked);
  if (e != cudaSuccess) return e;
  prompt_fwd_kernel<D, PAGED><<<(unsigned)ctas, C::NTHREADS, C::ALLOC, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.splits == 1) return e;
  prompt_merge_kernel<D><<<(unsigned)(a.max_blocks * a.Hkv * 4), 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_fwd(const PromptFwdArgs& a, int d, cudaStream_t st) {
  const bool paged = a.seqs.cu_k == nullptr;
  if (d == 128) return paged ? launch_d<128, true>(a, st) : launch_d<128, false>(a, st);
  if (d == 64) return paged ? launch_d<64, true>(a, st) : launch_d<64, false>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace fa

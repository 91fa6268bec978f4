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
// CTA = one block: two query tiles of one sequence and K/V head. Warp roles,
// products, tensor-memory columns and the online softmax are those of the
// forward in attn_fwd_bf16.cu (described there). What differs: each tile visits
// its own number of key tiles (its last query's diagonal), the diagonal of a
// tile can cross two key tiles, rows may see no key at all, and keys come either
// packed (one TMA box per 128 keys) or from the pages of a cache (one box per
// page or part of one, issued by the lanes of the producer warp). What stands
// behind a sequence's last key (another sequence's rows, old rows of a page, NaN
// included) has no influence: its scores are replaced, the products over keys
// end at the last one, and the up to 15 rows of V that their last step still
// reads are set to zero.
//
// Blocks are listed longest first (prompt.cuh); each CTA finds its own from the
// offsets on the device, so a captured graph follows them. Few blocks with many
// keys are split into key ranges, whose partial results prompt_merge_kernel
// combines by their maxima and sums.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

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
  part = (int)(u % a.splits);
  const long long w = u / a.splits;
  if (w >= (long long)total * a.Hkv) return false;
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
  k.kt0 = (int)((long long)part * most / a.splits);
  const int end = (int)((long long)(part + 1) * most / a.splits);
  k.n0 = max(0, min(n0, end) - k.kt0);
  k.n1 = max(0, min(n1, end) - k.kt0);
  return true;
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(FwdCfg<D>::THREADS, 1) prompt_fwd_kernel(const __grid_constant__ PromptFwdArgs a) {
  using C = FwdCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto BAR = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  const int B_QFULL = 0;
  const int B_KFULL = C::QT, B_VFULL = C::QT + C::STAGES, B_KEMPTY = C::QT + 2 * C::STAGES,
            B_VEMPTY = C::QT + 3 * C::STAGES;
  const int B_SFULL = C::QT + 4 * C::STAGES, B_PFULL = B_SFULL + C::QT, B_ODONE = B_PFULL + C::QT;
  const int B_SFREE = B_ODONE + C::QT;  // S read by the softmax (own-P layout only)
  const int B_DRAIN = B_SFREE + C::QT;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_BAR + C::NBAR * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + C::NBAR * 8 + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  PromptBlock k;
  int part;
  if (!prompt_block(a, blockIdx.x, lane, blockIdx.x == 0 && warp == 0, k, part)) return;  // the whole CTA
  const int n = k.v.n, m = k.v.m, past = m - n;
  const int n_max = max(k.n0, k.n1);
  const int kt0 = k.kt0;
  auto n_of = [&](int t) { return t == 0 ? k.n0 : k.n1; };
  const int TP = a.tile_tokens, RT = TP * a.G;  // tokens and rows of a query tile

  if (threadIdx.x == 0) {
    for (int t = 0; t < C::QT; ++t) mbar_init(BAR(B_QFULL + t), 1);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(BAR(B_KFULL + s), 1);
      mbar_init(BAR(B_VFULL + s), 1);
      mbar_init(BAR(B_KEMPTY + s), 1);
      mbar_init(BAR(B_VEMPTY + s), 1);
    }
    for (int t = 0; t < C::QT; ++t) {
      mbar_init(BAR(B_SFULL + t), 1);
      mbar_init(BAR(B_PFULL + t), 4);  // one arrival per softmax warp
      mbar_init(BAR(B_ODONE + t), 1);
      mbar_init(BAR(B_SFREE + t), 4);
    }
    mbar_init(BAR(B_DRAIN), 1);
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

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // One lane issues the packed tensors' boxes; a paged cache's boxes have a
    // lane each (box `box` of the 64-column chunk `chunk` of a tile).
    const int nbox = PAGED ? C::BN / a.box_rows : 1;
    const bool mine = PAGED ? lane < nbox * C::CH : lane == 0;
    const int box = PAGED ? lane % nbox : 0, chunk = PAGED ? lane / nbox : 0;
    auto look_up = [&](int tile, int& page, int& row) {
      page = -1;
      row = 0;
      if constexpr (PAGED) {
        const int key = tile * C::BN + box * a.box_rows;
        if (mine && key < m) {
          const int pi = key / a.pool.page_size;
          row = key - pi * a.pool.page_size;
          page = __ldg(a.block_tables + (size_t)k.seq * a.max_pages + pi);
          if (page < 0 || page >= a.pool.num_pages) {
            report_status(a.status, kStatusBadSeqlens);
            page = a.pool.num_pages;  // outside the tensor: reads as zeros
          }
        }
      }
    };
    // bytes of a tile's boxes that hold keys of the sequence
    auto tile_bytes = [&](int j) {
      if constexpr (!PAGED) return (uint32_t)C::TILE_BYTES;
      const int left = m - (kt0 + j) * C::BN;
      const int boxes = left >= C::BN ? nbox : (left + a.box_rows - 1) / a.box_rows;
      return (uint32_t)(boxes * a.box_rows * 128 * C::CH);
    };
    auto load = [&](const CUtensorMap* map, int off, int bar, int s, int j, int page, int row) {
      const uint32_t dst = sbase + off + s * C::TILE_BYTES;
      if constexpr (PAGED) {
        if (page >= 0)
          tma_load_4d(dst + chunk * C::CHUNK_BYTES + box * a.box_rows * 128, map, BAR(bar + s), chunk * 64, row, k.head, page);
      } else if (lane == 0) {
        for (int c = 0; c < C::CH; ++c)
          tma_load_3d(dst + c * C::CHUNK_BYTES, map, BAR(bar + s), c * 64, k.v.k0 + (kt0 + j) * C::BN, k.head);
      }
    };
    auto load_q = [&](int t) {
      if (lane == 0 && n_of(t) > 0) {
        mbar_arrive_expect_tx(BAR(B_QFULL + t), (uint32_t)(RT * 128 * C::CH));
        for (int c = 0; c < C::CH; ++c)
          tma_load_4d(sbase + C::OFF_Q + (t * C::CH + c) * C::CHUNK_BYTES, &a.tmQ, BAR(B_QFULL + t), c * 64, 0,
                      k.v.q0 + k.tok0 + t * TP, k.head);
      }
    };
    if (lane == 0) {
      tma_prefetch_desc(&a.tmQ);
      tma_prefetch_desc(&a.tmK);
      tma_prefetch_desc(&a.tmV);
    }
    load_q(0);
    bool q1 = false;  // tile 1's queries are asked for after the first keys
    int last_k = -1, last_v = -1;  // last tile whose load was issued
    int skipped = -1;
    int page, row;
    look_up(kt0, page, row);
    for (int j = 0; j < n_max; ++j) {
      if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
      const int s = j % C::STAGES;
      const uint32_t ph = (j / C::STAGES) & 1;
      int next_page = -1, next_row = 0;
      if (j + 1 < n_max) look_up(kt0 + j + 1, next_page, next_row);
      if (!mbar_wait_warp(BAR(B_KEMPTY + s), ph ^ 1, a.status, a.wait_limit_ns)) { *abort_flag = 1; break; }
      if (j != a.debug_skip_kv) {
        if (lane == 0) mbar_arrive_expect_tx(BAR(B_KFULL + s), tile_bytes(j));
        __syncwarp();
        load(&a.tmK, C::OFF_K, B_KFULL, s, j, page, row);
      } else {
        skipped = j;
      }
      last_k = j;
      if (j == 0) {
        load_q(1);
        q1 = true;
      }
      if (!mbar_wait_warp(BAR(B_VEMPTY + s), ph ^ 1, a.status, a.wait_limit_ns)) { *abort_flag = 1; break; }
      if (lane == 0) mbar_arrive_expect_tx(BAR(B_VFULL + s), tile_bytes(j));
      __syncwarp();
      load(&a.tmV, C::OFF_V, B_VFULL, s, j, page, row);
      last_v = j;
      page = next_page;
      row = next_row;
    }
    // drain: the last load issued into each buffer must have landed before exit
    if (k.n0 > 0) mbar_wait_warp(BAR(B_QFULL + 0), 0, a.status, a.wait_limit_ns);
    if (q1 && k.n1 > 0) mbar_wait_warp(BAR(B_QFULL + 1), 0, a.status, a.wait_limit_ns);
    for (int j = max(0, last_k - C::STAGES + 1); j <= last_k; ++j)
      if (j != skipped) mbar_wait_warp(BAR(B_KFULL + j % C::STAGES), (j / C::STAGES) & 1, a.status, a.wait_limit_ns);
    for (int j = max(0, last_v - C::STAGES + 1); j <= last_v; ++j)
      mbar_wait_warp(BAR(B_VFULL + j % C::STAGES), (j / C::STAGES) & 1, a.status, a.wait_limit_ns);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t leader = elect_one();
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t idesc_o = idesc_bf16_f32(128, D, false, true);
    const uint64_t dQ0 = sdesc_sw128(sbase + C::OFF_Q, 16, 1024);
    const uint64_t dK0 = sdesc_sw128(sbase + C::OFF_K, 16, 1024);
    const uint64_t dV0 = sdesc_sw128(sbase + C::OFF_V, C::CHUNK_BYTES, 1024);
    auto issue_s = [&](int t, int s) {
      const uint64_t qa = dQ0 + (uint64_t)((t * C::TILE_BYTES) >> 4);
      const uint64_t kb = dK0 + (uint64_t)((s * C::TILE_BYTES) >> 4);
      const uint32_t dcol = tmem + C::S_COL(t);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = (uint64_t)(((kk >> 2) * C::CHUNK_BYTES + (kk & 3) * 32) >> 4);
        mma_ss(dcol, qa + off, kb + off, idesc_s, kk > 0 ? 1u : 0u, leader);
      }
      mma_commit(BAR(B_SFULL + t), leader);
    };
    // P V over the keys that the tile's last query sees, in steps of 16
    auto issue_pv = [&](int t, int s, int j) {
      const uint64_t vb = dV0 + (uint64_t)((s * C::TILE_BYTES) >> 4);
      const uint32_t dcol = tmem + C::O_COL(t), acol = tmem + C::P_COL(t);
      const int keys = past + min(n, k.tok0 + (t + 1) * TP) - (kt0 + j) * C::BN;
#pragma unroll
      for (int kk = 0; kk < C::BN / 16; ++kk)
        mma_ts(dcol, acol + kk * 8, vb + (uint64_t)((kk * 2048) >> 4), idesc_o, (j > 0 || kk > 0) ? 1u : 0u,
               16 * kk >= keys ? 0u : leader);
      mma_commit(BAR(B_ODONE + t), leader);
    };
    // V_j has landed in slot s: rows behind the last key that the last step
    // would read become zero.
    auto clean_v = [&](int j, int s) {
      const int keys = m - (kt0 + j) * C::BN;
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
    auto wait = [&](int b, uint32_t parity) { return mbar_wait_warp(BAR(b), parity, a.status, a.wait_limit_ns); };
    bool ok = true;
    if (n_max > 0) {
      ok = wait(B_KFULL + 0, 0);
      for (int t = 0; ok && t < C::QT; ++t) {
        if (n_of(t) == 0) continue;
        if (!wait(B_QFULL + t, 0)) { ok = false; break; }
        tc_fence_after();
        issue_s(t, 0);
      }
      if (ok) mma_commit(BAR(B_KEMPTY + 0), leader);
    }
    for (int j = 0; ok && j < n_max; ++j) {
      if (__any_sync(0xffffffffu, *abort_flag != 0)) { ok = false; break; }
      const int s = j % C::STAGES;
      const uint32_t ph = (j / C::STAGES) & 1;
      const int s1 = (j + 1) % C::STAGES;
      const uint32_t ph1 = ((j + 1) / C::STAGES) & 1;
      bool k_next = false, v_here = false;  // K_{j+1}, V_j have landed
      auto need_v = [&]() {
        if (!v_here) {
          if (!wait(B_VFULL + s, ph)) return false;
          clean_v(j, s);
        }
        return v_here = true;
      };
      auto next_s = [&](int t) {
        if (!k_next && !wait(B_KFULL + s1, ph1)) return false;
        k_next = true;
        tc_fence_after();
        issue_s(t, s1);
        return true;
      };
      for (int t = 0; ok && t < C::QT; ++t) {
        if (j >= n_of(t)) continue;
        const bool more = j + 1 < n_of(t);
        if constexpr (C::P_OWN) {
          // P has its own columns: S_{j+1} goes first, P_j V_j follows
          if (more && !(wait(B_SFREE + t, j & 1) && next_s(t))) { ok = false; break; }
          if (!wait(B_PFULL + t, j & 1) || !need_v()) { ok = false; break; }
          tc_fence_after();
          issue_pv(t, s, j);
        } else {
          // P overwrites S: P_j V_j must be issued before S_{j+1}
          if (!need_v() || !wait(B_PFULL + t, j & 1)) { ok = false; break; }
          tc_fence_after();
          issue_pv(t, s, j);
          if (more && !next_s(t)) { ok = false; break; }
        }
      }
      if (!ok) break;
      mma_commit(BAR(B_VEMPTY + s), leader);
      if (j + 1 < n_max) mma_commit(BAR(B_KEMPTY + s1), leader);
    }
    if (!ok && lane == 0) *abort_flag = 1;
    // drain every MMA issued before TMEM can be released
    mma_commit(BAR(B_DRAIN), leader);
    wait(B_DRAIN, 0);
  } else {
    // ------------------------------------------------------------ softmax
    const int t = (warp - C::SW0) >> 2;  // query tile of this warpgroup
    const int wq = warp & 3;             // TMEM lane quarter
    const int row = wq * 32 + lane;      // row of the tile
    const int tok_in = a.g_div(row), g = row - tok_in * a.G;
    const int tok0 = k.tok0 + t * TP;    // first token of the tile
    const int tok = tok0 + tok_in;
    const bool live = row < RT && tok < n;
    const int n_own = n_of(t);
    const uint32_t lane_addr = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t s_addr = lane_addr + C::S_COL(t);
    const uint32_t o_addr = lane_addr + C::O_COL(t);
    const float c2 = a.scale_log2;
    const uint64_t c22 = f2_pack(c2, c2);
    float m_ref = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n_own; ++j) {
      if (__any_sync(0xffffffffu, *abort_flag != 0)) { ok = false; break; }
      const bool w = mbar_wait(BAR(B_SFULL + t), j & 1, a.status, a.wait_limit_ns);
      if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
      tc_fence_after();
      // keys of this tile that the row sees: the tile's first query's diagonal
      // decides whether any row has masked columns here
      const int key0 = (kt0 + j) * C::BN;
      const bool mask_tile = past + tok0 + 1 - key0 < C::BN;
      const int valid = min(past + tok + 1, m) - key0;
      float mx[4];
      uint64_t sm2[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) { mx[u] = -INFINITY; sm2[u] = 0ull; }
      bool need;
      float alpha = 1.f;
      // a row that has met no key yet: what is added to its scores (-inf) is 0
      const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
      if constexpr (C::P_OWN) {
        const uint32_t p_addr = lane_addr + C::P_COL(t);
        if (!softmax_pass_own_p<true>(s_addr, p_addr, mask_tile, valid, c22, f2_pack(neg_m, neg_m), mx, sm2, j > 0,
                                      BAR(B_ODONE + t), (uint32_t)(j - 1) & 1u, a.status, a.wait_limit_ns)) {
          ok = false;
          break;
        }
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
        need = mt > m_ref + kRescaleLog2;
        if (__any_sync(0xffffffffu, need)) {
          const float m_new = need ? mt : m_ref;
          alpha = need ? ex2_approx(m_ref - m_new) : 1.f;
#pragma unroll
          for (int u = 0; u < 4; ++u) sm2[u] = 0ull;
          tmem_st_wait();  // the speculative P is overwritten below
          const float neg_new = m_new == -INFINITY ? 0.f : -m_new;
          softmax_pass_own_p<false>(s_addr, p_addr, mask_tile, valid, c22, f2_pack(neg_new, neg_new), mx, sm2, false, 0u,
                                    0u, a.status, a.wait_limit_ns);
          m_ref = m_new;
        }
        // S_j has been read: S_{j+1} may be written over it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_SFREE + t));
      } else {
        // The speculative pass against the reference max of the tiles before,
        // the tile's own max alongside; a tile whose max exceeds it by more than
        // kRescaleLog2 is done again. 64 columns of S are in registers at a time.
        uint32_t pk[64];
        auto pass = [&](auto with_max, float neg) {
          const uint64_t nm2 = f2_pack(neg, neg);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r[64];
            tmem_ld32(s_addr + 64 * h, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
            tmem_ld32(s_addr + 64 * h + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
            tmem_ld_wait();
            if (mask_tile) {
#pragma unroll
              for (int i = 0; i < 64; ++i) r[i] = 64 * h + i >= valid ? __float_as_uint(-INFINITY) : r[i];
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float s0 = __uint_as_float(r[2 * i]), s1 = __uint_as_float(r[2 * i + 1]);
              if constexpr (with_max) mx[i & 3] = fmax3(mx[i & 3], s0, s1);
              const float2 x = f2_unpack(ffma2(f2_pack(s0, s1), c22, nm2));
              const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
              sm2[i & 3] = fadd2(sm2[i & 3], f2_pack(p0, p1));
              pk[32 * h + i] = pack_bf16x2(p0, p1);
            }
          }
        };
        pass(std::true_type{}, neg_m);
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
        need = mt > m_ref + kRescaleLog2;
        if (__any_sync(0xffffffffu, need)) {
          const float m_new = need ? mt : m_ref;
          alpha = need ? ex2_approx(m_ref - m_new) : 1.f;
#pragma unroll
          for (int u = 0; u < 4; ++u) sm2[u] = 0ull;
          pass(std::false_type{}, m_new == -INFINITY ? 0.f : -m_new);
          m_ref = m_new;
        }
        tmem_st32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
        tmem_st32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
      }
      const float2 sa = f2_unpack(fadd2(fadd2(sm2[0], sm2[1]), fadd2(sm2[2], sm2[3])));
      l = l * alpha + (sa.x + sa.y);
      // P V of the tile before is complete here (attn_fwd_bf16.cu): O can be rescaled
      if (j > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tmem_ld32(o_addr + 32 * q, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st32(o_addr + 32 * q, o);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_PFULL + t));
    }
    tmem_st_wait();  // no TMEM store may be in flight when the loop is left early
    if (ok && n_own > 0) {
      const bool w = mbar_wait(BAR(B_ODONE + t), (n_own - 1) & 1, a.status, a.wait_limit_ns);
      ok = __all_sync(0xffffffffu, w);
    }
    const bool parts = a.splits > 1;
    // every warp that shares an epilogue barrier takes the same decision (both
    // tiles' warps where they stage over the other tile's buffers)
    if (parts) ok = named_bar_and<1>(256, ok);
    else if (t == 0) ok = named_bar_and<2>(128, ok);
    else ok = named_bar_and<3>(128, ok);
    if (!ok) *abort_flag = 1;
    const float inv_l = l == 0.f ? 0.f : 1.f / l;
    if (ok && tok0 < n) {
      tc_fence_after();
      // 32 columns of this row of O, normalised; zeros where the tile has no key
      auto read_o = [&](int q, float (&x)[32]) {
        uint32_t r[32];
        if (n_own > 0) {
          tmem_ld32(o_addr + 32 * q, r);
          tmem_ld_wait();
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = n_own > 0 && l != 0.f ? __uint_as_float(r[i]) * inv_l : 0.f;
      };
      const float lse2 = m_ref + __log2f(l);  // -inf for a row without keys
      if (parts) {
        // fp32 rows of this key range; a range without keys leaves only its log-sum-exp
        const long long prow0 = ((long long)k.unit * a.splits + part) * (2 * C::BM) + t * C::BM;
        a.Lpart[prow0 + row] = lse2;
        if (n_own > 0) {
          uint8_t* stage = smem + C::OFF_Q + t * (D * 512);
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            float x[32];
            read_o(q, x);
            uint8_t* b = stage + q * 16384 + row * 128;
#pragma unroll
            for (int u = 0; u < 8; ++u)
              *reinterpret_cast<float4*>(b + ((u ^ (row & 7)) << 4)) =
                  make_float4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
          }
          fence_proxy_async_smem();
          if (t == 0) named_bar_sync<2>(128);
          else named_bar_sync<3>(128);
          if (warp == C::SW0 + 4 * t && lane == 0) {
#pragma unroll
            for (int q = 0; q < D / 32; ++q)
              tma_store_2d(&a.tmOpart, smem_u32(stage + q * 16384), q * 32, (int)prow0);
            bulk_commit_group();
            bulk_wait_group_read<0>();
          }
        }
      } else {
        // A tile whose tokens are all of its sequence leaves through the tile's
        // Q slot by TMA; a sequence's last, partial tile row by row from there
        // (16 lanes a 256-byte row).
        uint8_t* stage = smem + C::OFF_Q + t * C::TILE_BYTES;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          float x[32];
          read_o(q, x);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int c0 = 32 * q + 8 * v, u = (c0 & 63) >> 3;
            *reinterpret_cast<uint4*>(stage + (c0 >> 6) * C::CHUNK_BYTES + row * 128 + ((u ^ (row & 7)) << 4)) =
                make_uint4(pack_bf16x2(x[8 * v], x[8 * v + 1]), pack_bf16x2(x[8 * v + 2], x[8 * v + 3]),
                           pack_bf16x2(x[8 * v + 4], x[8 * v + 5]), pack_bf16x2(x[8 * v + 6], x[8 * v + 7]));
          }
        }
        if (tok0 + TP <= n) {
          fence_proxy_async_smem();
          if (t == 0) named_bar_sync<2>(128);
          else named_bar_sync<3>(128);
          if (warp == C::SW0 + 4 * t && lane == 0) {
#pragma unroll
            for (int c = 0; c < C::CH; ++c)
              tma_store_4d(&a.tmO, smem_u32(stage + c * C::CHUNK_BYTES), c * 64, 0, k.v.q0 + tok0, k.head);
            bulk_commit_group();
            bulk_wait_group_read<0>();  // the slot read before the CTA exits
          }
        } else {
          __syncwarp();
          constexpr int LPR = D / 8;  // lanes to a row
#pragma unroll 4
          for (int i = 0; i < 32; i += 32 / LPR) {
            const int r = wq * 32 + i + lane / LPR, u = lane % LPR;
            const int tk = a.g_div(r);
            const uint4 x = *reinterpret_cast<const uint4*>(stage + (u >> 3) * C::CHUNK_BYTES + r * 128 +
                                                            (((u & 7) ^ (r & 7)) << 4));
            if (r < RT && tok0 + tk < n)
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.O) + (long long)(k.v.q0 + tok0 + tk) * a.o_stride +
                                        (long long)(k.head * a.G + r - tk * a.G) * D + 8 * u) = x;
          }
        }
        if (live)
          a.LSE[(size_t)(k.head * a.G + g) * a.seqs.total_q + k.v.q0 + tok] = lse2 * 0.69314718055994531f;
      }
    }
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
// 32 rows of a block, a warp per row (lanes along d), ranges without keys (L =
// -inf) not read.
template <int D>
__global__ void __launch_bounds__(256) prompt_merge_kernel(const __grid_constant__ PromptFwdArgs a) {
  constexpr int PER = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  PromptBlock k;
  int part;
  if (!prompt_block(a, (long long)blockIdx.x / 8 * a.splits, lane, false, k, part)) return;
  const int RT = a.tile_tokens * a.G;
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const int br = (int)(blockIdx.x & 7) * 32 + warp * 4 + i;  // row of the block
    const int t = br >> 7, row = br & 127;
    const int tk = a.g_div(row), tok = k.tok0 + t * a.tile_tokens + tk;
    if (row >= RT || tok >= k.v.n) continue;
    const long long p0 = (long long)k.unit * a.splits * 256 + br;
    float L = -INFINITY;
    for (int p = lane; p < a.splits; p += 32) L = fmaxf(L, a.Lpart[p0 + 256ll * p]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L = fmaxf(L, __shfl_xor_sync(0xffffffffu, L, o));
    float acc[PER], sum = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    for (int p = 0; p < a.splits; ++p) {
      const float lp = a.Lpart[p0 + 256ll * p];
      if (lp == -INFINITY) continue;
      const float w = exp2f(lp - L);
      sum += w;
      const float* src = a.Opart + (p0 + 256ll * p) * D + lane * PER;
      if constexpr (PER == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        acc[0] = fmaf(w, x.x, acc[0]);
        acc[1] = fmaf(w, x.y, acc[1]);
        acc[2] = fmaf(w, x.z, acc[2]);
        acc[3] = fmaf(w, x.w, acc[3]);
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        acc[0] = fmaf(w, x.x, acc[0]);
        acc[1] = fmaf(w, x.y, acc[1]);
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int hq = k.head * a.G + row - tk * a.G;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.O) + (long long)(k.v.q0 + tok) * a.o_stride + (long long)hq * D + lane * PER;
    if constexpr (PER == 4)
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
    else
      *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    if (lane == 0)
      a.LSE[(size_t)hq * a.seqs.total_q + k.v.q0 + tok] = (L + __log2f(sum)) * 0.69314718055994531f;
  }
}

template <int D, bool PAGED>
cudaError_t launch_d(const PromptFwdArgs& a, cudaStream_t st) {
  using C = FwdCfg<D>;
  static_assert(C::SMEM_ALLOC <= 227 * 1024, "shared memory budget");
  static_assert(C::QT * D * 512 <= C::OFF_BAR - C::OFF_Q, "partial rows fit the tile buffers");
  const long long ctas = a.max_blocks * a.Hkv * a.splits;
  if (a.splits < 1 || a.max_blocks < 1 || ctas > 0x7fffffffll || (a.splits > 1 && (!a.Opart || !a.Lpart)))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(prompt_fwd_kernel<D, PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::SMEM_ALLOC);
  if (e != cudaSuccess) return e;
  prompt_fwd_kernel<D, PAGED><<<(unsigned)ctas, C::THREADS, C::SMEM_ALLOC, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.splits == 1) return e;
  prompt_merge_kernel<D><<<(unsigned)(a.max_blocks * a.Hkv * 8), 256, 0, st>>>(a);
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

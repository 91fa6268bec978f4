// fwd_tile.cuh -- what the two-tile forward kernels share: the layout of a CTA
// (two 128-row query tiles against 128-key tiles) in shared and tensor memory,
// and the softmax over a row of scores in tensor memory.
#pragma once

#include "ptx.cuh"

namespace fa {
namespace {

constexpr float kRescaleLog2 = 8.0f;  // tolerated growth of the running max before O is rescaled

template <int D>
struct FwdCfg {
  static constexpr int BM = 128;  // query rows per tile (TMEM lanes)
  static constexpr int QT = 2;    // query tiles per CTA
  static constexpr int BN = 128;  // keys per KV tile
  static constexpr int CH = D / 64;  // 128-byte column chunks per row
  static constexpr int STAGES = (D == 128) ? 2 : 4;
  static constexpr int CHUNK_BYTES = 128 * 128;  // one 128-row x 128-byte swizzled chunk
  static constexpr int TILE_BYTES = CH * CHUNK_BYTES;  // 128 rows x D bf16
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + QT * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + STAGES * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_V + STAGES * TILE_BYTES;
  static constexpr int NBAR = QT + 4 * STAGES + 4 * QT + 1;
  static constexpr int SMEM_BYTES = OFF_BAR + NBAR * 8 + 16;
  static constexpr int SMEM_ALLOC = SMEM_BYTES + 1024;  // slack for 1024-byte alignment
  // warps: 0 producer, 1 MMA, 2-5 and 6-9 the softmax warpgroups of query
  // tiles 0 and 1 (any four consecutive warps cover the four TMEM lane
  // quarters); 320 threads leave 200 registers per thread
  static constexpr int SW0 = 2;
  static constexpr int THREADS = 32 * (SW0 + 4 * QT);
  static constexpr uint32_t TMEM_COLS = 512;
  // TMEM columns: S_t at 128*t, O_t at 256 + D*t. With d = 64 the last 128
  // columns are free and hold P_t (64 columns of bf16 pairs each), so P can
  // be written while S is still being read; with d = 128 P goes over S.
  static constexpr bool P_OWN = (D == 64);
  static constexpr uint32_t S_COL(int t) { return 128u * t; }
  static constexpr uint32_t O_COL(int t) { return 256u + (uint32_t)D * t; }
  static constexpr uint32_t P_COL(int t) { return P_OWN ? 256u + 2u * D + 64u * t : S_COL(t); }
};

// Scores past `valid` (ragged tail, causal diagonal) become -inf.
__device__ __forceinline__ void mask_cols32(uint32_t (&r)[32], int c0, int valid) {
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = c0 + i >= valid ? __float_as_uint(-INFINITY) : r[i];
}

// One 32-column chunk of a row of S: p = 2^(s*c2 - m) for column pairs
// (packed fp32 arithmetic), the row sums in four packed accumulators, the row
// max alongside when asked, and the chunk's P as bf16 pairs.
template <bool WITH_MAX>
__device__ __forceinline__ void softmax_chunk32(const uint32_t (&r)[32], uint32_t (&pk)[16],
                                                uint64_t c22, uint64_t nm2, float (&mx)[4],
                                                uint64_t (&sm2)[4]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float s0 = __uint_as_float(r[2 * i]), s1 = __uint_as_float(r[2 * i + 1]);
    if (WITH_MAX) mx[i & 3] = fmax3(mx[i & 3], s0, s1);
    const float2 x = f2_unpack(ffma2(f2_pack(s0, s1), c22, nm2));
    const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
    sm2[i & 3] = fadd2(sm2[i & 3], f2_pack(p0, p1));
    pk[i] = pack_bf16x2(p0, p1);
  }
}

// A 128-column row of S read in four 32-column chunks, each load in flight
// while the chunk before it is exponentiated; each chunk's P goes to TMEM
// columns of its own. Before the first P store the thread waits for the
// previous P V product to finish reading those columns (o_wait, on the
// o_done barrier); false if that bounded wait expired (nothing stored then).
template <bool WITH_MAX>
__device__ __forceinline__ bool softmax_pass_own_p(uint32_t s_addr, uint32_t p_addr,
                                                   bool mask_tile, int valid, uint64_t c22,
                                                   uint64_t nm2, float (&mx)[4],
                                                   uint64_t (&sm2)[4], bool o_wait,
                                                   uint32_t o_done, uint32_t o_parity,
                                                   int* status, unsigned long long limit_ns) {
  uint32_t ra[32], rb[32], pk[16];
  tmem_ld32(s_addr, ra);
  tmem_ld_wait_dep(ra);
  // not unrolled: fully unrolled, ptxas batches the exponentials of all the
  // chunks and runs out of registers
#pragma unroll 1
  for (int c = 0; c < 4; c += 2) {
    tmem_ld32(s_addr + 32 * (c + 1), rb);
    if (mask_tile) mask_cols32(ra, 32 * c, valid);
    softmax_chunk32<WITH_MAX>(ra, pk, c22, nm2, mx, sm2);
    if (c == 0 && o_wait &&
        !__all_sync(0xffffffffu, mbar_wait(o_done, o_parity, status, limit_ns))) {
      tmem_ld_wait();  // the load in flight lands before its registers go away
      return false;
    }
    tmem_st16(p_addr + 16 * c, pk);
    tmem_ld_wait_dep(rb);
    if (c + 2 < 4) tmem_ld32(s_addr + 32 * (c + 2), ra);
    if (mask_tile) mask_cols32(rb, 32 * (c + 1), valid);
    softmax_chunk32<WITH_MAX>(rb, pk, c22, nm2, mx, sm2);
    tmem_st16(p_addr + 16 * (c + 1), pk);
    if (c + 2 < 4) tmem_ld_wait_dep(ra);
  }
  return true;
}

// -m, what is added to the scaled scores of a row of maximum m. A prefix's rows
// may have met nothing but scores of -inf yet (infinite keys): those have weight
// zero, where -inf + inf would be NaN.
template <bool PREFIX>
__device__ __forceinline__ float minus_max(float m) {
  return PREFIX && m == -INFINITY ? 0.f : -m;
}

}  // namespace
}  // namespace fa

// paged_decode.cu -- attention of a few new queries per sequence against a
// paged key/value cache, with or without a prefix that all sequences share.
//
// For query row r of a sequence, over the shared prefix's keys and then the
// own keys it sees:
//   O_r = sum_j exp(s_rj - m_r) V_j / l_r,   LSE_r = m_r + ln l_r,
//   s = scale * q.k,
// with the online softmax of "Lesson 1: FlashAttention core idea" §3.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;

// One block per query row; 128 keys at a time, one per thread for the scores,
// one output column per thread for P V.
template <int D>
__global__ void __launch_bounds__(kThreads) decode_rows_kernel(const __grid_constant__ PagedDecodeArgs a) {
  __shared__ float qs[D];
  __shared__ float ps[kThreads];
  __shared__ long long voff[kThreads];
  __shared__ float red[4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hq = a.pool.kv_heads * a.G;
  const long long row = blockIdx.x;
  const int i = (int)(row % a.Nq);
  const int hq = (int)(row / a.Nq % Hq);
  const int b = (int)(row / a.Nq / Hq);
  const int h = hq / a.G;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.Q) + b * a.q_b + hq * a.q_h + i * a.q_r;
  if (tid < D) qs[tid] = __bfloat162float(q[tid]);
  __syncthreads();
  int len = __ldg(a.seq_lens + b);
  if (len < 0 || len > (long long)a.max_pages * a.pool.page_size) {
    if (tid == 0) report_status(a.status, kStatusBadSeqlens);
    len = 0;
  }
  const int own = max(0, len - a.Nq + 1 + i);
  const long long n = (long long)a.prefix_len + own;
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (long long j0 = 0; j0 < n; j0 += kThreads) {
    const long long j = j0 + tid;
    float x = -INFINITY;
    if (j < n) {
      const bool pre = j < a.prefix_len;
      const int jj = (int)(pre ? j : j - a.prefix_len);
      const int pi = jj / a.pool.page_size, r = jj - pi * a.pool.page_size;
      const int page = __ldg(pre ? a.prefix_pages + pi : a.block_tables + (long long)b * a.max_pages + pi);
      voff[tid] = -1;
      if (page >= 0 && page < a.pool.num_pages) {
        const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.pool.k) + page * a.pool.k_page + h * a.pool.k_head + r * a.pool.k_row;
        float dot = 0.f;
        for (int e = 0; e < D; ++e) dot = fmaf(qs[e], __bfloat162float(k[e]), dot);
        x = dot * a.scale_log2;
        voff[tid] = page * a.pool.v_page + h * a.pool.v_head + r * a.pool.v_row;
      } else {
        report_status(a.status, kStatusBadSeqlens);
      }
    }
    float mt = x;
    for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    if (lane == 0) red[warp] = mt;
    __syncthreads();
    const float m_new = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = exp2f(m - m_use);
    ps[tid] = exp2f(x - m_use);
    m = m_new;
    l *= alpha;
    acc *= alpha;
    __syncthreads();
    const int cnt = (int)min((long long)kThreads, n - j0);
    for (int jj = 0; jj < cnt; ++jj) {
      l += ps[jj];
      if (tid < D && voff[jj] >= 0)
        acc = fmaf(ps[jj], __bfloat162float(static_cast<const __nv_bfloat16*>(a.pool.v)[voff[jj] + tid]), acc);
    }
    __syncthreads();
  }
  if (tid < D)
    (static_cast<__nv_bfloat16*>(a.O) + b * a.o_b + hq * a.o_h + i * a.o_r)[tid] =
        __float2bfloat16_rn(l != 0.f ? acc / l : 0.f);
  if (tid == 0) a.LSE[row] = l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

cudaError_t launch_decode_paged_bf16(const PagedDecodeArgs& a, int d, cudaStream_t st) {
  const long long rows = (long long)a.B * a.pool.kv_heads * a.G * a.Nq;
  if (rows > 0x7fffffffll) return cudaErrorInvalidValue;
  if (d == 128) decode_rows_kernel<128><<<(unsigned)rows, kThreads, 0, st>>>(a);
  else if (d == 64) decode_rows_kernel<64><<<(unsigned)rows, kThreads, 0, st>>>(a);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

}  // namespace fa

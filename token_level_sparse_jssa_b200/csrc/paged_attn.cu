// Attention of each sequence's newest tokens over a paged cache: causal, with an optional
// sliding window and sinks.
//
// One block per (token row, query head); each of its 4 warps takes every fourth visible
// position, with a lane's share of the head dims in registers and an online softmax in fp32;
// the warps' states are merged in shared memory.
#include "common.cuh"
#include "launch.h"
#include "paged.cuh"

namespace jssa {
namespace {

template <int D>
__global__ void __launch_bounds__(128) paged_attn_simple_kernel(PagedAttnArgs a) {
  constexpr int PL = D / 32;
  __shared__ float m_s[4], l_s[4], o_s[4][D];
  const int64_t i = blockIdx.x;
  const int hq = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = sequence_of(a.q_begin, a.B, i);
  const NewTokens r = new_tokens(a.q_begin, a.seq_lens, b, static_cast<int64_t>(a.max_pages) * a.pool.page_size,
                                 a.n_tokens, a.max_q_len, a.status);
  if (i < r.q0 || i >= r.q0 + r.nq) return;
  const int64_t pos = r.len - r.nq + (i - r.q0);
  const int64_t win = a.window > 0 ? max64(0, pos + 1 - a.window) : 0;
  const int64_t sinks = min64(win, a.n_sinks);  // visible: [0, sinks) and [win, pos]
  const int64_t n = sinks + pos + 1 - win;
  const int h = hq / (a.Hq / a.pool.Hkv);
  const __nv_bfloat16* K = static_cast<const __nv_bfloat16*>(a.pool.K) + h * a.pool.ks[1];
  const __nv_bfloat16* V = static_cast<const __nv_bfloat16*>(a.pool.V) + h * a.pool.vs[1];
  const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(a.Q) + i * a.q_stride + static_cast<int64_t>(hq) * D;
  float q[PL], o[PL], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < PL; ++e) {
    q[e] = __bfloat162float(Q[lane + 32 * e]);
    o[e] = 0.f;
  }
  for (int64_t j = warp; j < n; j += 4) {
    const int64_t t = j < sinks ? j : win + j - sinks;
    const int p = a.table[static_cast<int64_t>(b) * a.max_pages + t / a.pool.page_size];
    if (p < 0 || p >= a.pool.n_pages) {
      if (lane == 0) flag_error(a.status, DEVFLAG_BAD_INDEX);
      continue;
    }
    const __nv_bfloat16* kr = K + p * a.pool.ks[0] + (t % a.pool.page_size) * a.pool.ks[2];
    const __nv_bfloat16* vr = V + p * a.pool.vs[0] + (t % a.pool.page_size) * a.pool.vs[2];
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < PL; ++e) s = fmaf(q[e], __bfloat162float(kr[lane + 32 * e]), s);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    s *= a.sm_scale;
    const float mn = fmaxf(m, s), alpha = expf(m - mn), w = expf(s - mn);
    l = l * alpha + w;
    m = mn;
#pragma unroll
    for (int e = 0; e < PL; ++e) o[e] = fmaf(w, __bfloat162float(vr[lane + 32 * e]), o[e] * alpha);
  }
  if (lane == 0) m_s[warp] = m, l_s[warp] = l;
#pragma unroll
  for (int e = 0; e < PL; ++e) o_s[warp][lane + 32 * e] = o[e];
  __syncthreads();
  const float M = fmaxf(fmaxf(m_s[0], m_s[1]), fmaxf(m_s[2], m_s[3]));
  float L = 0.f, w[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    w[u] = M == -INFINITY ? 0.f : expf(m_s[u] - M);
    L += w[u] * l_s[u];
  }
  const int64_t row = i * a.Hq + hq;
  for (int e = threadIdx.x; e < D; e += 128) {
    float v = 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u) v = fmaf(w[u], o_s[u][e], v);
    v = L > 0.f ? v / L : 0.f;
    if (a.out_bf16) static_cast<__nv_bfloat16*>(a.O)[row * D + e] = __float2bfloat16_rn(v);
    else static_cast<float*>(a.O)[row * D + e] = v;
  }
  if (a.lse && threadIdx.x == 0) a.lse[row] = L > 0.f ? M + logf(L) : -INFINITY;
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttnArgs& a, int num_sms, cudaStream_t s) {
  (void)num_sms;
  const dim3 grid(static_cast<unsigned>(a.n_tokens), a.Hq);
  switch (a.pool.d) {
    case 64: return launch_ex(paged_attn_simple_kernel<64>, grid, dim3(128), 0, s, 0, a);
    case 128: return launch_ex(paged_attn_simple_kernel<128>, grid, dim3(128), 0, s, 0, a);
    case 256: return launch_ex(paged_attn_simple_kernel<256>, grid, dim3(128), 0, s, 0, a);
  }
  return cudaErrorNotSupported;
}

}  // namespace jssa

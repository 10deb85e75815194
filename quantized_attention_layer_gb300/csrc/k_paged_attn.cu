// k_paged_attn.cu -- attention of a ragged batch over the paged 8-bit key/value cache.
//
//   s_p = scale ks[page(p)] sum_d q_d kc[p][d]   (softcap: cap tanh(s / cap)),
//   o = sum_p softmax(s)_p vs[page(p)] vc[p]
// over the positions row i of a sequence's n rows sees: p <= P = len - n + i (all p < len
// when bidirectional), p > P - window with a window.  One pass with a running maximum.
//
// One warp per (row, query head); a lane holds hd / 32 adjacent dims of q and of the output.
#include "hfa_common.cuh"
#include "hfa_internal.h"
#include "hfa_paged.h"

namespace hfa {
namespace {

template <int HD>
__global__ void __launch_bounds__(128) paged_attn_kernel(const PagedAttnArgs a) {
  constexpr int D = HD / 32;
  const PagedView& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * 4 + warp;
  const int row = (int)(item / p.nh), h = (int)(item % p.nh);
  if (row >= a.total) return;
  const int b = find_seq(p.batch, row, [&](int i) { return a.cu[i]; });
  const int n = a.cu[b + 1] - a.cu[b], len = a.len[b];
  if (n * (p.nh / p.nkv) <= kPagedStepRows) return;  // the step kernel's
  const bool bad = len < 0 || len > p.max_pages * p.ps;
  if (bad && lane == 0) atomicOr(p.err, kErrBadPosition);
  const int P = len - n + row - a.cu[b];
  int hi = a.bidir ? len : P + 1;
  int lo = a.window ? P - a.window + 1 : 0;
  if (lo < 0) lo = 0;
  if (bad) hi = 0;
  float q[D], o[D];
  const size_t at = (size_t)row * a.q_stride + h * HD + lane * D;
#pragma unroll
  for (int i = 0; i < D; ++i) {
    q[i] = a.f32 ? ((const float*)a.q)[at + i] : __bfloat162float(((const __nv_bfloat16*)a.q)[at + i]);
    o[i] = 0.f;
  }
  const int kv = h / (p.nh / p.nkv);
  float m = -INFINITY, l = 0.f;
  for (int k = lo; k < hi; ++k) {
    const int page = p.table[(size_t)b * p.max_pages + (k >> p.ps_log2)];
    if ((unsigned)page >= (unsigned)p.num_pages) {
      if (lane == 0) atomicOr(p.err, kErrBadPosition);
      continue;
    }
    const size_t pg = (size_t)page * p.nkv + kv;
    const size_t off = (pg * p.ps + (k & (p.ps - 1))) * HD + lane * D;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < D; ++i) s += q[i] * (float)p.k_codes[off + i];
    s = warp_sum(s) * p.k_scales[pg] * a.qscale;
    if (a.cap_log2 != 0.f) s = a.cap_log2 * tanhf(s);
    const float mn = fmaxf(m, s);
    const float corr = exp2f(m - mn), w = exp2f(s - mn);
    const float wv = w * p.v_scales[pg];
    l = l * corr + w;
    m = mn;
#pragma unroll
    for (int i = 0; i < D; ++i) o[i] = o[i] * corr + wv * (float)p.v_codes[off + i];
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const size_t ot = ((size_t)row * p.nh + h) * HD + lane * D;
#pragma unroll
  for (int i = 0; i < D; ++i) {
    if (a.f32)
      ((float*)a.o)[ot + i] = o[i] * inv;
    else
      ((__nv_bfloat16*)a.o)[ot + i] = __float2bfloat16_rn(o[i] * inv);
  }
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t s) {
  const unsigned grid = (unsigned)(((long long)a.total * a.p.nh + 3) / 4);
  if (a.p.hd == 64) paged_attn_kernel<64><<<grid, 128, 0, s>>>(a);
  else if (a.p.hd == 128) paged_attn_kernel<128><<<grid, 128, 0, s>>>(a);
  else paged_attn_kernel<256><<<grid, 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace hfa

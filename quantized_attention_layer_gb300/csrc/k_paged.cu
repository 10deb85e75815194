// k_paged.cu -- the paged 8-bit key/value cache: rows going in (per-head norms, NeoX RoPE,
// codes with one scale for each page and head) and decoded rows coming out.
//
// Append.  For head row x at position P: y = x w rsqrt(mean x^2 + eps) (when the handle has
// the norm), the pairs (y_i, y_{i+hd/2}) rotated by P theta^(-2i/hd) / f_i, and
//   a  = max |y| over the rows the call writes into the page (one head),
//   s' = max(s, a / 127), s the page's scale or 0 for a page begun by this call,
//   codes before the first written slot: rint(c (s / s')), written ones: rint(y / s').
// One CTA owns a (sequence, page) and walks over some KV heads, so the maximum of a page
// meets in one block and nothing is atomic: results do not depend on timing.  A thread holds
// 16 values of a row, 8 of each half, so both members of its pairs are its own and the
// cosines and sines of its position, computed once, serve every q and k head of the walk.
// Memory-bound: rows are read once with 16-byte loads and codes written once.
#include "hfa_common.cuh"
#include "hfa_finish.cuh"
#include "hfa_internal.h"
#include "hfa_paged.h"

namespace hfa {
namespace {

constexpr int kAppendThreads = 512;  // most threads of an append CTA

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = pack_bf2(__float2bfloat16_rn(v[2 * i]), __float2bfloat16_rn(v[2 * i + 1]));
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// A row unit as it lies in memory (8 values of each half), and as values.
template <class T>
struct RawUnit {
  static constexpr int W = sizeof(T) * 8 / 16;  // 16-byte words of 8 values
  uint4 lo[W], hi[W];
};
template <class T>
__device__ __forceinline__ void load_raw(const T* p, int half, bool on, RawUnit<T>& u) {
#pragma unroll
  for (int i = 0; i < RawUnit<T>::W; ++i) {
    u.lo[i] = u.hi[i] = make_uint4(0u, 0u, 0u, 0u);
    if (on) {
      // plain loads: the queries may be overwritten in place
      u.lo[i] = reinterpret_cast<const uint4*>(p)[i];
      u.hi[i] = reinterpret_cast<const uint4*>(p + half)[i];
    }
  }
}
__device__ __forceinline__ void values8(const uint4 (&r)[1], float (&v)[8]) {
  const uint32_t w[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void values8(const uint4 (&r)[2], float (&v)[8]) {
  v[0] = __uint_as_float(r[0].x), v[1] = __uint_as_float(r[0].y);
  v[2] = __uint_as_float(r[0].z), v[3] = __uint_as_float(r[0].w);
  v[4] = __uint_as_float(r[1].x), v[5] = __uint_as_float(r[1].y);
  v[6] = __uint_as_float(r[1].z), v[7] = __uint_as_float(r[1].w);
}

// |x| for finite x, 0 for NaN and infinities
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}
// code of y under 1 / scale: ties to even, infinities to +-127, NaN to 0
__device__ __forceinline__ uint32_t code_of(float y, float inv) {
  float t = y * inv;
  t = t == t ? fminf(fmaxf(t, -127.f), 127.f) : 0.f;
  return (uint32_t)__float2int_rn(t) & 0xffu;
}
__device__ __forceinline__ uint2 codes8(const float (&y)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    w[h] = code_of(y[4 * h], inv) | code_of(y[4 * h + 1], inv) << 8 |
           code_of(y[4 * h + 2], inv) << 16 | code_of(y[4 * h + 3], inv) << 24;
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ uint32_t recode4(uint32_t w, float r) {
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = (int)(int8_t)(w >> (8 * i));
    o |= ((uint32_t)__float2int_rn((float)c * r) & 0xffu) << (8 * i);
  }
  return o;
}

// One row unit (16 values: lo the 8 at 8 c, hi the 8 at hd/2 + 8 c): RMS norm over the row,
// whose HD / 16 units sit in adjacent lanes, times the weight (NULL: 1).
template <int HD>
__device__ __forceinline__ void unit_norm(float (&lo)[8], float (&hi)[8], const float* w, int c,
                                          float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss += lo[i] * lo[i] + hi[i] * hi[i];
#pragma unroll
  for (int o = 1; o < HD / 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float inv = rsqrtf(ss / HD + eps);
  float wl[8], wh[8];
  if (w) {
    load8(w + 8 * c, wl);
    load8(w + HD / 2 + 8 * c, wh);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] *= w ? inv * wl[i] : inv;
    hi[i] *= w ? inv * wh[i] : inv;
  }
}
__device__ __forceinline__ void rotate(float (&lo)[8], float (&hi)[8], const float (&cs)[8],
                                       const float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x0 = lo[i], x1 = hi[i];
    lo[i] = x0 * cs[i] - x1 * sn[i];
    hi[i] = x0 * sn[i] + x1 * cs[i];
  }
}

// The cosines and sines of a CTA's page when its rows do not fit one unit a thread: float4
// (cos, sin, cos, sin) of pairs 8 c + 2 i, 8 c + 2 i + 1 of slot s at index (4 s + i) U + c,
// so that the lanes of a row read adjacent 16-byte words.
template <int HD>
__device__ __forceinline__ void load_turn(const float4* tab, int slot, int c, float (&cs)[8],
                                          float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 t = tab[(4 * slot + i) * (HD / 16) + c];
    cs[2 * i] = t.x, sn[2 * i] = t.y, cs[2 * i + 1] = t.z, sn[2 * i + 1] = t.w;
  }
}

// BIG: the page's ps * HD / 16 row units exceed 512 threads (pages of 128 at hd 128, of 64 or
// 128 at hd 256): the threads loop over them, the turns live in shared memory, and K and V
// rows are read twice (the second time from L2), once for the maximum and once for the codes.
template <int HD, bool BIG, class T>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const PagedAppendArgs a) {
  constexpr int U = HD / 16;  // units of a row
  extern __shared__ float4 s_turn[];
  __shared__ int s_seq;
  __shared__ float s_max[2][2][kAppendThreads / 32];  // [head parity][K, V][warp]
  const PagedView& p = a.p;
  const int ps = p.ps;
  const int item = blockIdx.x;
  // sequence b owns items cu[b] / ps + 2 b .. : n rows touch at most n / ps + 2 pages
  int b;
  if (a.single) {
    b = item;
  } else {
    if (threadIdx.x < 32) {
      const int f = find_seq(p.batch, item, [&](int i) { return (a.cu[i] >> p.ps_log2) + 2 * i; });
      if (threadIdx.x == 0) s_seq = f;
    }
    __syncthreads();
    b = s_seq;
  }
  const int row0 = a.cu[b], n = a.cu[b + 1] - row0, start = a.start[b];
  if (n <= 0) return;
  if (row0 < 0 || row0 > a.total - n || start < 0 || start > p.max_pages * ps - n) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrBadPosition);
    return;
  }
  const int j = (start >> p.ps_log2) + (a.single ? 0 : item - ((row0 >> p.ps_log2) + 2 * b));
  const int page0 = j << p.ps_log2;  // position of the page's slot 0
  if (page0 >= start + n) return;
  const int page = __ldg(p.table + (size_t)b * p.max_pages + j);  // checked below: the rows load meanwhile
  const int first = max(start - page0, 0), last = min(start + n - page0, ps);
  const int c = threadIdx.x % U, slot0 = threadIdx.x / U;
  const int rstep = blockDim.x / U;
  const int G = p.nh / p.nkv;
  const int kv0 = blockIdx.y * a.kv_per_cta;
  const int kv1 = min(kv0 + a.kv_per_cta, p.nkv);
  const long long tok0 = (long long)row0 + page0 - start;  // row of slot 0
  const int warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  auto written = [&](int slot) { return slot >= first && slot < last; };
  auto load_kv = [&](int kv, int slot, RawUnit<T>& k, RawUnit<T>& v) {
    const bool on = written(slot) && kv < kv1;
    load_raw((const T*)a.k + (tok0 + slot) * a.k_stride + kv * HD + 8 * c, HD / 2, on, k);
    load_raw((const T*)a.v + (tok0 + slot) * a.v_stride + kv * HD + 8 * c, HD / 2, on, v);
  };
  // QC query heads at a time: their loads are in flight together
  constexpr int QC = sizeof(T) == 2 ? 4 : 2;
  const int q0 = kv0 * G, q1 = kv1 * G;
  auto load_q = [&](int h, int slot, RawUnit<T> (&q)[QC]) {
#pragma unroll
    for (int i = 0; i < QC; ++i)
      load_raw((const T*)a.q + (tok0 + slot) * a.q_stride + (h + i) * HD + 8 * c, HD / 2,
               a.q && written(slot) && h + i < q1, q[i]);
  };
  RawUnit<T> rk, rv;
  if (!BIG) load_kv(kv0, slot0, rk, rv);

  float cs[8], sn[8];
  for (int slot = slot0; slot < ps; slot += rstep) {
    if (!written(slot)) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) rope_cs(page0 + slot, a.rope_g[8 * c + i], cs[i], sn[i]);
    if (BIG) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s_turn[(4 * slot + i) * U + c] = make_float4(cs[2 * i], sn[2 * i], cs[2 * i + 1], sn[2 * i + 1]);
    }
  }  // a thread reads back only what it wrote itself: no barrier
  if ((unsigned)page >= (unsigned)p.num_pages) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrBadPosition);
    return;
  }

  // the K and V values of a unit, normed and rotated.  Every lane of a warp calls it together
  // (the norm's sum goes over the lanes of a row).
  auto kv_values = [&](int slot, const RawUnit<T>& k, const RawUnit<T>& v, float (&kl)[8],
                       float (&kh)[8], float (&vl)[8], float (&vh)[8]) {
    values8(k.lo, kl);
    values8(k.hi, kh);
    values8(v.lo, vl);
    values8(v.hi, vh);
    if (a.w_k) unit_norm<HD>(kl, kh, a.w_k, c, a.eps);
    if (a.v_unit_norm) unit_norm<HD>(vl, vh, nullptr, c, a.eps);
    if (written(slot)) {
      if (BIG) load_turn<HD>(s_turn, slot, c, cs, sn);
      rotate(kl, kh, cs, sn);
    }
  };
  auto top_of = [&](const float (&lo)[8], const float (&hi)[8], float m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(finite_abs(lo[i]), finite_abs(hi[i])));
    return m;
  };

  for (int kv = kv0; kv < kv1; ++kv) {
    const size_t pg = (size_t)page * p.nkv + kv;
    const size_t base = pg * ps * HD;
    float kl[8], kh[8], vl[8], vh[8];
    uint2 old[4];
    float s_old[2] = {0.f, 0.f};
    float m[2] = {0.f, 0.f};
    if (first > 0) {
      s_old[0] = p.k_scales[pg];
      s_old[1] = p.v_scales[pg];
      if (!BIG && slot0 < first) {  // early: needed only if the scale grows
        const size_t at = base + (size_t)slot0 * HD + 8 * c;
        old[0] = *reinterpret_cast<const uint2*>(p.k_codes + at);
        old[1] = *reinterpret_cast<const uint2*>(p.k_codes + at + HD / 2);
        old[2] = *reinterpret_cast<const uint2*>(p.v_codes + at);
        old[3] = *reinterpret_cast<const uint2*>(p.v_codes + at + HD / 2);
      }
    }
    for (int slot = slot0; slot < ps; slot += rstep) {
      if (BIG) load_kv(kv, slot, rk, rv);
      kv_values(slot, rk, rv, kl, kh, vl, vh);
      if (written(slot)) {
        m[0] = top_of(kl, kh, m[0]);
        m[1] = top_of(vl, vh, m[1]);
      }
      if (!BIG) break;
    }
    if (!BIG) load_kv(kv + 1, slot0, rk, rv);  // the next head's, while this one is coded
    float* sm = &s_max[kv & 1][0][0];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m[t] = fmaxf(m[t], __shfl_xor_sync(0xffffffffu, m[t], o));
      if ((threadIdx.x & 31) == 0) sm[t * (kAppendThreads / 32) + warp] = m[t];
    }
    __syncthreads();  // also: every thread has read the old scales
    float inv[2], ratio[2];
    bool grown[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float top = 0.f;
      for (int w = 0; w < nwarps; ++w) top = fmaxf(top, sm[t * (kAppendThreads / 32) + w]);
      const float so = s_old[t] > 0.f ? finite_abs(s_old[t]) : 0.f;
      float sc = fmaxf(so, top / 127.f);
      if (sc < 1.17549435e-38f) sc = 0.f;
      inv[t] = sc > 0.f ? 1.f / sc : 0.f;
      ratio[t] = sc > 0.f ? so / sc : 0.f;
      grown[t] = sc != s_old[t];
      if (threadIdx.x == 0) (t == 0 ? p.k_scales : p.v_scales)[pg] = sc;
    }
    for (int slot = slot0; slot < ps; slot += rstep) {
      if (BIG) {
        load_kv(kv, slot, rk, rv);
        kv_values(slot, rk, rv, kl, kh, vl, vh);
      }
      const size_t at = base + (size_t)slot * HD + 8 * c;
      if (written(slot)) {
        *reinterpret_cast<uint2*>(p.k_codes + at) = codes8(kl, inv[0]);
        *reinterpret_cast<uint2*>(p.k_codes + at + HD / 2) = codes8(kh, inv[0]);
        *reinterpret_cast<uint2*>(p.v_codes + at) = codes8(vl, inv[1]);
        *reinterpret_cast<uint2*>(p.v_codes + at + HD / 2) = codes8(vh, inv[1]);
      } else if (slot < first) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!grown[t]) continue;
          int8_t* dst = (t == 0 ? p.k_codes : p.v_codes) + at;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint2* at8 = reinterpret_cast<uint2*>(dst + h * (HD / 2));
            const uint2 w = BIG ? *at8 : old[2 * t + h];
            *at8 = make_uint2(recode4(w.x, ratio[t]), recode4(w.y, ratio[t]));
          }
        }
      }
      if (!BIG) break;
    }
  }
  if (!a.q) return;
  for (int slot = slot0; slot < ps; slot += rstep) {
    const bool on = written(slot);
    if (BIG && on) load_turn<HD>(s_turn, slot, c, cs, sn);
    for (int h = q0; h < q1; h += QC) {
      RawUnit<T> rq[QC];
      load_q(h, slot, rq);
#pragma unroll
      for (int i = 0; i < QC; ++i) {
        if (h + i >= q1) break;
        float ql[8], qh[8];
        values8(rq[i].lo, ql);
        values8(rq[i].hi, qh);
        if (a.w_q) unit_norm<HD>(ql, qh, a.w_q, c, a.eps);
        if (on) {
          rotate(ql, qh, cs, sn);
          T* op = (T*)a.q_out + ((tok0 + slot) * p.nh + h + i) * HD + 8 * c;
          store8(op, ql);
          store8(op + HD / 2, qh);
        }
      }
    }
    if (!BIG) break;
  }
}

template <int HD, bool BIG, class T>
cudaError_t launch_append(const PagedAppendArgs& a, dim3 grid, int threads, cudaStream_t s) {
  const size_t smem = BIG ? (size_t)a.p.ps * HD * 4 : 0;  // ps * (HD / 16) * 4 float4
  if (BIG) {
    const cudaError_t e = cudaFuncSetAttribute(paged_append_kernel<HD, BIG, T>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  paged_append_kernel<HD, BIG, T><<<grid, threads, smem, s>>>(a);
  return cudaGetLastError();
}
template <class T>
cudaError_t launch_append_t(const PagedAppendArgs& a, dim3 grid, int threads, bool big,
                            cudaStream_t s) {
  if (a.p.hd == 64) return launch_append<64, false, T>(a, grid, threads, s);
  if (a.p.hd == 128)
    return big ? launch_append<128, true, T>(a, grid, threads, s)
               : launch_append<128, false, T>(a, grid, threads, s);
  return big ? launch_append<256, true, T>(a, grid, threads, s)
             : launch_append<256, false, T>(a, grid, threads, s);
}

// Read: one CTA decodes one page's rows of some KV heads, 16 codes (one 16-byte load, two
// 16-byte stores) a thread and step; memory-bound.
__global__ void __launch_bounds__(256) paged_read_kernel(const PagedReadArgs a) {
  const PagedView& p = a.p;
  const int b = blockIdx.y;
  const int start = a.start[b], n = a.count[b];
  if (n <= 0) return;
  if (start < 0 || start + (long long)n > (long long)p.max_pages * p.ps ||
      start + (long long)n > a.capacity) {
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(p.err, kErrBadPosition);
    return;
  }
  const int U = p.hd / 16;
  const int kv0 = blockIdx.z * a.heads_per_cta;
  const int heads = min(a.heads_per_cta, p.nkv - kv0);
  const int jend = (start + n - 1) >> p.ps_log2;
  for (int j = (start >> p.ps_log2) + blockIdx.x; j <= jend; j += gridDim.x) {
    const int page = p.table[(size_t)b * p.max_pages + j];
    if ((unsigned)page >= (unsigned)p.num_pages) {
      if (threadIdx.x == 0) atomicOr(p.err, kErrBadPosition);
      continue;
    }
    const int page0 = j << p.ps_log2;
    const int first = max(start - page0, 0), last = min(start + n - page0, p.ps);
    const int per = (last - first) * U;  // units of one head's rows
#pragma unroll 4
    for (int i = threadIdx.x; i < 2 * heads * per; i += blockDim.x) {
      const int hu = i / per, u = i - hu * per;
      const int t = hu >= heads, kv = kv0 + hu - t * heads;
      const int slot = first + u / U, c = u % U;
      const size_t pg = (size_t)page * p.nkv + kv;
      const int8_t* codes = t ? p.v_codes : p.k_codes;
      const float sc = __ldg((t ? p.v_scales : p.k_scales) + pg);
      const uint4 w4 = __ldg(reinterpret_cast<const uint4*>(codes + (pg * p.ps + slot) * p.hd) + c);
      const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
      uint32_t o[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int s0 = 16 * (q & 1);
        o[q] = pack_bf2(__float2bfloat16_rn((float)(int8_t)(w[q >> 1] >> s0) * sc),
                        __float2bfloat16_rn((float)(int8_t)(w[q >> 1] >> (s0 + 8)) * sc));
      }
      __nv_bfloat16* dst = (t ? a.v_cache : a.k_cache) +
                           (((size_t)b * p.nkv + kv) * a.capacity + page0 + slot) * p.hd + 16 * c;
      reinterpret_cast<uint4*>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
      reinterpret_cast<uint4*>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a0, bool f32, int items, int sms,
                                cudaStream_t s) {
  PagedAppendArgs a = a0;
  const int units = a.p.ps * (a.p.hd / 16);
  const int threads = units < kAppendThreads ? units : kAppendThreads;
  // KV heads per CTA: as many as leave every SM eight CTAs (the position's cosines and sines
  // are computed once per CTA)
  int per = 1;
  while (per < a.p.nkv && (long long)items * ((a.p.nkv + 2 * per - 1) / (2 * per)) >= 8LL * sms) per *= 2;
  a.kv_per_cta = per;
  const dim3 grid(items, (a.p.nkv + per - 1) / per);
  const bool big = units > threads;
  return f32 ? launch_append_t<float>(a, grid, threads, big, s)
             : launch_append_t<__nv_bfloat16>(a, grid, threads, big, s);
}

cudaError_t launch_paged_read(const PagedReadArgs& a0, int max_count, int sms, cudaStream_t s) {
  PagedReadArgs a = a0;
  const int pages = (max_count + a.p.ps - 2) / a.p.ps + 1;
  // heads per CTA: up to 32 KB of codes while every SM keeps eight CTAs
  int per = 1;
  while (per < a.p.nkv && 2 * per * 2 * a.p.ps * a.p.hd <= 32768 &&
         (long long)pages * a.p.batch * ((a.p.nkv + 2 * per - 1) / (2 * per)) >= 8LL * sms)
    per *= 2;
  a.heads_per_cta = per;
  const dim3 grid(pages, a.p.batch, (a.p.nkv + per - 1) / per);
  paged_read_kernel<<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace hfa

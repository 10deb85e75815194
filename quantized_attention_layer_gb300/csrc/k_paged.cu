// k_paged.cu -- the paged 8-bit key/value cache: rows going in (per-head norms, NeoX RoPE,
// codes with one scale for each page and head) and decoded rows coming out.
//
// Append.  For head row x at position P: y = x w rsqrt(mean x^2 + eps) (when the handle has
// the norm), the pairs (y_i, y_{i+hd/2}) rotated by P theta^(-2i/hd) / f_i, and
//   a  = max |y| over the rows the call writes into the page (one head),
//   s' = max(s, a / 127), s the page's scale or 0 for a page begun by this call,
//   codes before the first written slot: rint(c (s / s')), written ones: rint(y / s').
// One CTA owns a (sequence, page) and walks over some KV heads, so the maximum of a page
// meets in one block and nothing is atomic: results do not depend on timing.  Other CTAs of
// the page rotate the queries, four heads' loads in flight together.  A thread holds 8 values
// of a row, 4 of each half, so both members of its pairs are its own, and few registers: four
// CTAs of 256 threads share an SM, one loading while another computes (with 16 values a thread
// and 16 warps an SM an 8K prompt took 53 us for 47, 3.9 TB/s).  Memory-bound by design; the
// issue slots come next (about 20 instructions a value).
#include "hfa_common.cuh"
#include "hfa_finish.cuh"
#include "hfa_internal.h"
#include "hfa_paged.h"

namespace hfa {
namespace {

constexpr int kAppendThreads = 256;  // most threads of an append CTA

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 a = ld_global(reinterpret_cast<const float4*>(p));
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// A row unit: 4 values of each half as they lie in memory.  Plain loads: the queries may be
// overwritten in place.
template <class T>
struct RawUnit;
template <>
struct RawUnit<__nv_bfloat16> {
  using Word = uint2;
  Word lo, hi;
};
template <>
struct RawUnit<float> {
  using Word = float4;
  Word lo, hi;
};
template <class T>
__device__ __forceinline__ void load_raw(const T* p, int half, bool on, RawUnit<T>& u) {
  using Word = typename RawUnit<T>::Word;
  u.lo = u.hi = Word{};
  if (on) {
    u.lo = *reinterpret_cast<const Word*>(p);
    u.hi = *reinterpret_cast<const Word*>(p + half);
  }
}
__device__ __forceinline__ void values4(uint2 r, float (&v)[4]) {
  v[0] = __uint_as_float(r.x << 16), v[1] = __uint_as_float(r.x & 0xffff0000u);
  v[2] = __uint_as_float(r.y << 16), v[3] = __uint_as_float(r.y & 0xffff0000u);
}
__device__ __forceinline__ void values4(float4 r, float (&v)[4]) {
  v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
}

// |x| for finite x, 0 for NaN and infinities
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}
// the larger magnitude, NaN if there is one
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// code of y under 1 / scale: ties to even, infinities to +-127, NaN to 0
__device__ __forceinline__ uint32_t code_of(float y, float inv) {
  float t = y * inv;
  t = t == t ? fminf(fmaxf(t, -127.f), 127.f) : 0.f;
  return (uint32_t)__float2int_rn(t) & 0xffu;
}
// Codes of 4 values.  Finite ones are at most 127 (1 + 3 * 2^-24) scales: adding 1.5 * 2^23
// rounds them to the nearest integer, ties to even, whose low byte is the code.
__device__ __forceinline__ uint32_t codes4(const float (&y)[4], float inv, bool finite) {
  if (finite) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(fmaf(y[i], inv, 12582912.f));
    return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
  }
  return code_of(y[0], inv) | code_of(y[1], inv) << 8 | code_of(y[2], inv) << 16 | code_of(y[3], inv) << 24;
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

// 1 / rms of a row, whose HD / 8 units (8 values: lo the 4 at 4 c, hi the 4 at hd/2 + 4 c)
// sit in adjacent lanes.
template <int HD>
__device__ __forceinline__ float row_rms(const float (&lo)[4], const float (&hi)[4], float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) ss += lo[i] * lo[i] + hi[i] * hi[i];
#pragma unroll
  for (int o = 1; o < HD / 8; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  return rsqrtf(ss / HD + eps);
}
// The rotation of a unit's pairs with the norm's weights folded in:
// (lo, hi) -> (lo w_lo cos - hi w_hi sin, lo w_lo sin + hi w_hi cos).
struct Turn {
  float a[4], b[4], c[4], d[4];
};
__device__ __forceinline__ void make_turn(Turn& t, const float (&cs)[4], const float (&sn)[4],
                                          const float* w, int c, int half) {
  float wl[4], wh[4];
  if (w) {
    load4(w + 4 * c, wl);
    load4(w + half + 4 * c, wh);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t.a[i] = w ? wl[i] * cs[i] : cs[i];
    t.b[i] = w ? wh[i] * sn[i] : sn[i];
    t.c[i] = w ? wl[i] * sn[i] : sn[i];
    t.d[i] = w ? wh[i] * cs[i] : cs[i];
  }
}
__device__ __forceinline__ void rotate(float (&lo)[4], float (&hi)[4], const Turn& t, bool norm,
                                       float inv) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = lo[i], x1 = hi[i];
    lo[i] = x0 * t.a[i] - x1 * t.b[i];
    hi[i] = x0 * t.c[i] + x1 * t.d[i];
  }
  if (norm) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] *= inv;
      hi[i] *= inv;
    }
  }
}

// The cosine and sine of slot s of a page are those of the page's first position, formed once
// per CTA, turned by s: (c0 cs - s0 ss, s0 cs + c0 ss) with a table of the slots' (cs, ss).
// BIG: the page's ps * HD / 8 row units exceed 256 threads: the threads loop over them, and K
// and V rows are read twice (the second time from L2), for the maximum and for the codes.
template <int HD, bool BIG, class T>
__global__ void __launch_bounds__(kAppendThreads, 4) paged_append_kernel(const PagedAppendArgs a) {
  constexpr int U = HD / 8;  // units of a row
  // (cos, sin) of pairs 4 c + 2 i, 4 c + 2 i + 1 at the page's first position: index i U + c
  __shared__ float4 s_base[HD / 4];
  __shared__ int s_seq;
  // [round of heads, modulo 3][K, V][warp]: a slot is written again only behind a barrier that
  // follows its last read
  __shared__ float s_max[3][2][kAppendThreads / 32];
  const PagedView& p = a.p;
  const int ps = p.ps;
  const int item = blockIdx.x;
  pdl_wait();
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
  const int page = ld_global(p.table + (size_t)b * p.max_pages + j);  // checked below: the rows load meanwhile
  const int first = max(start - page0, 0), last = min(start + n - page0, ps);
  const int c = threadIdx.x % U, slot0 = threadIdx.x / U;
  const int rstep = blockDim.x / U;
  // the CTAs of a page: the first kv_groups take its K and V heads, the others query heads
  const bool queries = (int)blockIdx.y >= a.kv_groups;
  const int kv0 = blockIdx.y * a.kv_per_cta;
  const int kv1 = queries ? 0 : min(kv0 + a.kv_per_cta, p.nkv);
  const int q0 = queries ? ((int)blockIdx.y - a.kv_groups) * a.q_per_cta : 0;
  const int q1 = queries ? min(q0 + a.q_per_cta, p.nh) : 0;
  const long long tok0 = (long long)row0 + page0 - start;  // row of slot 0
  const int warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  auto written = [&](int slot) { return slot >= first && slot < last; };
  auto load_kv = [&](int kv, int slot, RawUnit<T>& k, RawUnit<T>& v) {
    const bool on = written(slot) && kv < kv1;
    load_raw((const T*)a.k + (tok0 + slot) * a.k_stride + kv * HD + 4 * c, HD / 2, on, k);
    load_raw((const T*)a.v + (tok0 + slot) * a.v_stride + kv * HD + 4 * c, HD / 2, on, v);
  };
  // QC query heads at a time: their loads are in flight together
  constexpr int QC = sizeof(T) == 2 ? 4 : 2;
  auto load_q = [&](int h, int slot, RawUnit<T> (&q)[QC]) {
#pragma unroll
    for (int i = 0; i < QC; ++i)
      load_raw((const T*)a.q + (tok0 + slot) * a.q_stride + (h + i) * HD + 4 * c, HD / 2,
               written(slot) && h + i < q1, q[i]);
  };
  RawUnit<T> rk, rv;
  if (!BIG && !queries) load_kv(kv0, slot0, rk, rv);

  float cs[4], sn[4];
  for (int i = threadIdx.x; i < HD / 2; i += blockDim.x) {
    float2 v;
    rope_cs(page0, a.rope_g[i], v.x, v.y);
    reinterpret_cast<float2*>(s_base)[2 * ((i % 4 / 2) * U + i / 4) + i % 2] = v;
  }
  __syncthreads();
  auto turn_of = [&](int slot) {
    const float4* tab = a.slot_turn + ((size_t)slot * U + c) * 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 t = ld_global(tab + i), o = s_base[i * U + c];
      cs[2 * i] = o.x * t.x - o.y * t.y;
      sn[2 * i] = o.y * t.x + o.x * t.y;
      cs[2 * i + 1] = o.z * t.z - o.w * t.w;
      sn[2 * i + 1] = o.w * t.z + o.z * t.w;
    }
  };
  Turn turn;
  if (queries) {
    for (int slot = slot0; slot < ps; slot += rstep) {
      const bool on = written(slot);
      RawUnit<T> rq[QC];
      load_q(q0, slot, rq);
      if (on) turn_of(slot);
      make_turn(turn, cs, sn, a.w_q, c, HD / 2);
      for (int h = q0; h < q1; h += QC) {
        if (h > q0) load_q(h, slot, rq);
#pragma unroll
        for (int i = 0; i < QC; ++i) {
          if (h + i >= q1) break;
          float ql[4], qh[4];
          values4(rq[i].lo, ql);
          values4(rq[i].hi, qh);
          const float inv = a.w_q ? row_rms<HD>(ql, qh, a.eps) : 1.f;
          if (on) {
            rotate(ql, qh, turn, a.w_q != nullptr, inv);
            T* op = (T*)a.q_out + ((tok0 + slot) * p.nh + h + i) * HD + 4 * c;
            store4(op, ql);
            store4(op + HD / 2, qh);
          }
        }
      }
      if (!BIG) break;
    }
    return;
  }
  if (!BIG && written(slot0)) turn_of(slot0);
  if ((unsigned)page >= (unsigned)p.num_pages) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrBadPosition);
    return;
  }

  // the K and V values of a unit, normed and rotated.  Every lane of a warp calls it together
  // (the norm's sum goes over the lanes of a row).
  if (!BIG) make_turn(turn, cs, sn, a.w_k, c, HD / 2);
  auto kv_values = [&](int slot, const RawUnit<T>& k, const RawUnit<T>& v, float (&kl)[4],
                       float (&kh)[4], float (&vl)[4], float (&vh)[4]) {
    values4(k.lo, kl);
    values4(k.hi, kh);
    values4(v.lo, vl);
    values4(v.hi, vh);
    const float inv = a.w_k ? row_rms<HD>(kl, kh, a.eps) : 1.f;
    if (a.v_unit_norm) {
      const float iv = row_rms<HD>(vl, vh, a.eps);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        vl[i] *= iv;
        vh[i] *= iv;
      }
    }
    if (written(slot)) {
      if (BIG) {
        turn_of(slot);
        make_turn(turn, cs, sn, a.w_k, c, HD / 2);
      }
      rotate(kl, kh, turn, a.w_k != nullptr, inv);
    }
  };
  // the largest magnitude so far: NaN or infinite once a value is not finite, or over the
  // finite ones alone
  auto top_of = [&](const float (&lo)[4], const float (&hi)[4], float m, bool all) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = all ? max_nan(m, max_nan(fabsf(lo[i]), fabsf(hi[i])))
              : fmaxf(m, fmaxf(finite_abs(lo[i]), finite_abs(hi[i])));
    return m;
  };

  for (int kv = kv0; kv < kv1; ++kv) {
    const size_t pg = (size_t)page * p.nkv + kv;
    const size_t base = pg * ps * HD;
    float kl[4], kh[4], vl[4], vh[4];
    uint32_t old[4];
    float s_old[2] = {0.f, 0.f};
    if (first > 0) {
      s_old[0] = p.k_scales[pg];
      s_old[1] = p.v_scales[pg];
      if (!BIG && slot0 < first) {  // early: needed only if the scale grows
        const size_t at = base + (size_t)slot0 * HD + 4 * c;
        old[0] = *reinterpret_cast<const uint32_t*>(p.k_codes + at);
        old[1] = *reinterpret_cast<const uint32_t*>(p.k_codes + at + HD / 2);
        old[2] = *reinterpret_cast<const uint32_t*>(p.v_codes + at);
        old[3] = *reinterpret_cast<const uint32_t*>(p.v_codes + at + HD / 2);
      }
    }
    // the page's maxima; a block that holds something not finite looks again at the rest
    float tops[2];
    bool finite = true;
    for (int round = 0; round < 2; ++round) {
      float m[2] = {0.f, 0.f};
      for (int slot = slot0; slot < ps; slot += rstep) {
        if (BIG) load_kv(kv, slot, rk, rv);
        if (BIG || round == 0) kv_values(slot, rk, rv, kl, kh, vl, vh);
        if (written(slot)) {
          m[0] = top_of(kl, kh, m[0], round == 0);
          m[1] = top_of(vl, vh, m[1], round == 0);
        }
        if (!BIG) break;
      }
      if (!BIG && round == 0) load_kv(kv + 1, slot0, rk, rv);  // the next head's, while this one is coded
      float* sm = &s_max[(2 * kv + round) % 3][0][0];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m[t] = max_nan(m[t], __shfl_xor_sync(0xffffffffu, m[t], o));
        if ((threadIdx.x & 31) == 0) sm[t * (kAppendThreads / 32) + warp] = m[t];
      }
      __syncthreads();  // also: every thread has read the old scales
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        tops[t] = 0.f;
        for (int w = 0; w < nwarps; ++w) tops[t] = max_nan(tops[t], sm[t * (kAppendThreads / 32) + w]);
      }
      if (round == 0 && tops[0] <= 3.402823466e38f && tops[1] <= 3.402823466e38f) break;
      finite = false;
    }
    float inv[2], ratio[2];
    bool grown[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float so = s_old[t] > 0.f ? finite_abs(s_old[t]) : 0.f;
      float sc = fmaxf(so, tops[t] / 127.f);
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
      const size_t at = base + (size_t)slot * HD + 4 * c;
      if (written(slot)) {
        *reinterpret_cast<uint32_t*>(p.k_codes + at) = codes4(kl, inv[0], finite);
        *reinterpret_cast<uint32_t*>(p.k_codes + at + HD / 2) = codes4(kh, inv[0], finite);
        *reinterpret_cast<uint32_t*>(p.v_codes + at) = codes4(vl, inv[1], finite);
        *reinterpret_cast<uint32_t*>(p.v_codes + at + HD / 2) = codes4(vh, inv[1], finite);
      } else if (slot < first) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!grown[t]) continue;
          int8_t* dst = (t == 0 ? p.k_codes : p.v_codes) + at;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t* at4 = reinterpret_cast<uint32_t*>(dst + h * (HD / 2));
            *at4 = recode4(BIG ? *at4 : old[2 * t + h], ratio[t]);
          }
        }
      }
      if (!BIG) break;
    }
  }
}

template <int HD, bool BIG, class T>
cudaError_t launch_append(const PagedAppendArgs& a, dim3 grid, int threads, cudaStream_t s) {
  return paged_launch(paged_append_kernel<HD, BIG, T>, grid, threads, 0, s, a);
}
template <class T>
cudaError_t launch_append_t(const PagedAppendArgs& a, dim3 grid, int threads, bool big,
                            cudaStream_t s) {
  if (a.p.hd == 64)
    return big ? launch_append<64, true, T>(a, grid, threads, s)
               : launch_append<64, false, T>(a, grid, threads, s);
  if (a.p.hd == 128)
    return big ? launch_append<128, true, T>(a, grid, threads, s)
               : launch_append<128, false, T>(a, grid, threads, s);
  return big ? launch_append<256, true, T>(a, grid, threads, s)
             : launch_append<256, false, T>(a, grid, threads, s);
}

// Read: one CTA decodes one page's rows of some KV heads; a thread takes the 8 codes of chunk
// c of rows r, r + 256 / U, ...: one 8-byte load and one 16-byte store each, so that a warp's
// store is 512 whole bytes, four rows' loads in flight.  Memory-bound: 32K tokens (8 heads, hd
// 128, 201 MB) 38 us, 5.2 TB/s.
template <int HD>
__global__ void __launch_bounds__(256) paged_read_kernel(const PagedReadArgs a) {
  constexpr int U = HD / 8, RP = 256 / U, NB = 4;
  const PagedView& p = a.p;
  const int b = blockIdx.y;
  pdl_wait();
  const int start = a.start[b], n = a.count[b];
  if (n <= 0) return;
  if (start < 0 || start > p.max_pages * p.ps - n || start > a.capacity - n) {
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(p.err, kErrBadPosition);
    return;
  }
  const int c = threadIdx.x % U, r0 = threadIdx.x / U;
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
    const int blocks = (last - first + RP - 1) / RP;  // row blocks of one head
    const int steps = 2 * heads * blocks;
    for (int s0 = 0; s0 < steps; s0 += NB) {
      uint2 w[NB];
      float sc[NB];
      size_t at[NB];
#pragma unroll
      for (int x = 0; x < NB; ++x) {
        const int hu = (s0 + x) / blocks, slot = first + (s0 + x - hu * blocks) * RP + r0;
        const int t = hu >= heads, kv = kv0 + hu - t * heads;
        const bool on = s0 + x < steps && slot < last;
        at[x] = (size_t)-1;
        if (on) {
          const size_t pg = (size_t)page * p.nkv + kv;
          sc[x] = ld_global((t ? p.v_scales : p.k_scales) + pg);
          w[x] = ld_global(reinterpret_cast<const uint2*>((t ? p.v_codes : p.k_codes) + (pg * p.ps + slot) * HD) + c);
          at[x] = (((size_t)b * p.nkv + kv) * a.capacity + page0 + slot) * HD + 8 * c;
        }
      }
#pragma unroll
      for (int x = 0; x < NB; ++x) {
        if (at[x] == (size_t)-1) continue;
        const uint32_t u[2] = {w[x].x, w[x].y};
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int sh = 16 * (q & 1);
          const float lo = (float)(int8_t)(u[q >> 1] >> sh) * sc[x];
          const float hi = (float)(int8_t)(u[q >> 1] >> (sh + 8)) * sc[x];
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[q]) : "f"(hi), "f"(lo));
        }
        *reinterpret_cast<uint4*>(((s0 + x) / blocks >= heads ? a.v_cache : a.k_cache) + at[x]) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a0, bool f32, int items, int sms,
                                cudaStream_t s) {
  PagedAppendArgs a = a0;
  const int units = a.p.ps * (a.p.hd / 8);
  const int threads = units < kAppendThreads ? units : kAppendThreads;
  // Heads per CTA: as many as leave every SM eight CTAs (the turns of its rows are formed once
  // per CTA), the query heads in steps of the four whose loads are in flight together
  auto groups = [&](int heads, int per) { return (heads + per - 1) / per; };
  int per = 1, qper = 4;
  while (per < a.p.nkv && (long long)items * groups(a.p.nkv, 2 * per) >= 8LL * sms) per *= 2;
  while (qper < a.p.nh && (long long)items * groups(a.p.nh, 2 * qper) >= 4LL * sms) qper *= 2;
  a.kv_per_cta = per;
  a.q_per_cta = qper;
  a.kv_groups = groups(a.p.nkv, per);
  const dim3 grid(items, a.kv_groups + (a.q ? groups(a.p.nh, qper) : 0));
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
  auto kern = a.p.hd == 64 ? paged_read_kernel<64> : a.p.hd == 128 ? paged_read_kernel<128> : paged_read_kernel<256>;
  return paged_launch(kern, grid, 256, 0, s, a);
}

}  // namespace hfa

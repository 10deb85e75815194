// k_paged_step.cu -- attention of few rows (rows x query heads of a KV head <= 8: single
// tokens, or a few at small groups) over the paged 8-bit cache.
//
//   s_p = scale ks[page(p)] sum_d q_d kc[p][d]   (softcap: cap tanh(s / cap)),
//   o   = sum_p softmax(s)_p vs[page(p)] vc[p],   codes kc, vc, scales ks, vs per page and head.
//
// Memory-bound: every code is read once.  The keys of all (sequence, KV head) units are one
// list of 16-key blocks (a block never straddles a page, so it has one K and one V scale),
// dealt out in equal contiguous ranges over the CTAs whatever the lengths of the sequences
// (a unit counts for a few blocks more than it has).
// Inside a CTA the warps take blocks in turn; each warp streams its own blocks through its
// own ring of shared-memory slots by TMA (swizzled boxes of 16 rows), so no warp waits for
// another until the range leaves a unit.  Table entries and scales are fetched 32 blocks at
// a time, one block a lane, half a batch ahead of their use.
//
// Both products run on mma.sync m16n8k16 in fp16, which holds the codes exactly: a code
// byte becomes fp16 by one byte permute and one subtract for two.  Query rows take MMA rows
// 0..7 as hi(q 2^-e) and rows 8..15 as the remainder lo (22 bits together, 2^e restored in
// the f32 score), the softmax weights likewise.  A K word read by ldmatrix holds four
// adjacent dims of one key; the MMA's k index walks the dims in that order and the query
// fragments follow it.  A V word read by ldmatrix.trans holds two adjacent dims of two keys:
// the permute that widens it also splits even from odd dims, two n8 tiles.
//
// The running maximum is kept lazily: it moves (and the accumulators are rescaled) only when
// a score exceeds it by 2^8, which a warp vote finds without any shuffle.  The V scale enters
// in the exponent: weights are w = 2^(s + log2 vs - mw) with a maximum mw of their own, the
// denominator l = sum 2^(s - m): fp16 weights then keep their bits whatever the pages' scales.
//
// 4 sequences of 128K keys (40/8 heads, hd 128, 1.07 GB): 195 us, 5.5 TB/s; 64 ragged ones of up
// to 8K (473 MB) 99.7 us, 4.7 TB/s: what a unit costs beside its blocks (below) is the rest.
#include "hfa_common.cuh"
#include "hfa_internal.h"
#include "hfa_paged.h"

namespace hfa {
namespace {

template <int HD>
struct StepCfg {
  static constexpr int NC = 8;                           // warps of a CTA
  static constexpr int CPS = HD == 256 ? 1 : 2;          // CTAs per SM
  static constexpr int BOXW = HD < 128 ? HD : 128;       // bytes of a TMA box row
  static constexpr int NBOX = HD / BOXW;
  static constexpr int SWM = BOXW == 128 ? 7 : 3;        // swizzled row bits
  static constexpr int TILE = 16 * HD;                   // codes of one block, K or V
  static constexpr int SLOT = 2 * TILE;
  static constexpr int KS = HD / 16;
  static constexpr int RS = kPagedRecord(HD);            // record: O[HD], mw, m, l, pad
  static constexpr int QF = KS * 32 * 16;                // query fragments
  // the merge area: NC / 2 warps' records of R rows, or the merge weights (R x CTAs)
  static constexpr int red_floats(int rows) {
    return rows * (NC / 2 * RS > kPagedMaxParts ? NC / 2 * RS : kPagedMaxParts);
  }
  static constexpr int MAXNS = HD == 64 ? 6 : 4;
};

constexpr float kNoMax = -1e30f;  // "no score yet"; finite, so differences are never NaN
// What a unit costs beside its blocks (queries, barriers, merge), in blocks: the ranges are
// dealt out over blocks + this.  Fitted to the cycles of CTAs with 3 and with 9 pieces of 64
// ragged sequences: 11200 a piece, 303 a block.  So a short range also never holds the end of
// one unit and the beginning of the next (1 token, 1K keys 15.2 -> 10 us, 8 such sequences 20
// -> 14.7; 24 and 52 differ by 0 to 2 %).
constexpr int kUnitCost = 36;
constexpr float kLazy = 8.f;      // how far (log2) a score may exceed the running maximum

// shared address of byte `byte` of row `row` of a block's tile
template <class Cfg>
__device__ __forceinline__ uint32_t tile_addr(uint32_t tile, int row, int byte) {
  const int box = byte / Cfg::BOXW, bb = byte - box * Cfg::BOXW;
  const uint32_t lin = (uint32_t)(row * Cfg::BOXW + bb);
  return tile + (uint32_t)(box * 16 * Cfg::BOXW) + (lin ^ (((lin >> 7) & Cfg::SWM) << 4));
}

// blocks of sequence b (per KV head): those that any of its rows sees, one (empty) block when
// there is none, 0 when this kernel does not serve the sequence
struct SeqPlan {
  int row0, n, len, lo, blocks;  // first row, rows, keys, first block
};
__device__ __forceinline__ SeqPlan plan_seq(const PagedAttnArgs& a, int b, int G) {
  SeqPlan s;
  s.row0 = ld_global(a.cu + b);
  s.n = ld_global(a.cu + b + 1) - s.row0;
  s.len = ld_global(a.len + b);
  s.lo = 0;
  s.blocks = 0;
  if (s.n <= 0 || s.n * G > kPagedStepRows || s.row0 < 0 || s.row0 > a.total - s.n) return s;
  if (s.len < 0 || s.len > a.p.max_pages * a.p.ps) {
    atomicOr(a.p.err, kErrBadPosition);
    s.len = 0;
  }
  // the first row's first key .. the last key
  const int lo = a.window ? s.len - s.n - a.window + 1 : 0;
  s.lo = lo > 0 ? lo >> 4 : 0;
  s.blocks = ((s.len + 15) >> 4) - s.lo;
  if (s.blocks < 1) s.blocks = 1;
  return s;
}

// Adds 1 by one thread between two barriers: covers the accesses of the whole CTA before the
// first and after the second, cheaper than a fence by every thread.
__device__ __forceinline__ int ticket_add(int* at) {
  int before;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(at) : "memory");
  return before;
}

template <int HD>
__global__ void __launch_bounds__(StepCfg<HD>::NC * 32, StepCfg<HD>::CPS)
    paged_step_kernel(const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv, const PagedAttnArgs a, int ns,
                      int max_rows) {
  using Cfg = StepCfg<HD>;
  constexpr int NC = Cfg::NC, RS = Cfg::RS, KS = Cfg::KS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align1024(smem_raw);
  const PagedView& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = p.nh / p.nkv;
  // layout: rings [NC][ns], query fragments, merge area, barriers, prefix
  uint8_t* ring = smem + warp * ns * Cfg::SLOT;
  uint4* qf = reinterpret_cast<uint4*>(smem + NC * ns * Cfg::SLOT);
  float* red = reinterpret_cast<float*>(qf + KS * 32);
  uint64_t* bars = reinterpret_cast<uint64_t*>(red + Cfg::red_floats(max_rows)) + warp * Cfg::MAXNS;
  int* s_misc = reinterpret_cast<int*>(bars + (NC - warp) * Cfg::MAXNS);            // [8]
  float* s_rowf = reinterpret_cast<float*>(s_misc + 8);                              // [8]
  int* s_warp = reinterpret_cast<int*>(s_rowf + 8);                                  // [NC]
  unsigned* pre = reinterpret_cast<unsigned*>(s_warp + NC);  // [batch + 1]: blocks (times KV heads) before each sequence

  if (lane == 0) {
    for (int i = 0; i < ns; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
  }
  pdl_wait();  // the launch overlaps the end of the kernel before it, nothing else does
  // ------------------------------------------------------------------ prefix over the batch
  {
    const int per = (p.batch + NC * 32 - 1) / (NC * 32);
    const int b0 = threadIdx.x * per;
    unsigned sum = 0, one = 0;
    for (int i = 0; i < per; ++i)
      if (b0 + i < p.batch) sum += one = plan_seq(a, b0 + i, G).blocks;
    unsigned inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) s_warp[warp] = (int)inc;
    __syncthreads();
    unsigned before = inc - sum;
    for (int w = 0; w < warp; ++w) before += (unsigned)s_warp[w];
    for (int i = 0; i < per; ++i)
      if (b0 + i < p.batch) {
        pre[b0 + i] = before;
        before += per == 1 ? one : (unsigned)plan_seq(a, b0 + i, G).blocks;
      }
    if (threadIdx.x == NC * 32 - 1) pre[p.batch] = before;
    __syncthreads();
  }
  const long long W = (long long)pre[p.batch] * p.nkv;  // all blocks
  constexpr int cost = kUnitCost;
  const long long V = W + (long long)cost * p.batch * p.nkv;  // blocks and the units' costs
  // CTAs at work: two blocks a warp before another CTA joins (one: 4K keys 13.0 -> 14.1 us)
  long long A = (V + 2 * NC - 1) / (2 * NC);
  if (A > gridDim.x) A = gridDim.x;
  if (blockIdx.x >= A) return;
  // the last sequence b with (pre[b] + cost b) nkv <= x
  auto seq_of = [&](long long x, int cost) {
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (((long long)pre[mid] + (long long)cost * mid) * p.nkv <= x) lo = mid; else hi = mid;
    }
    return lo;
  };
  // blocks before place v of the costed list (a unit: its cost, then its blocks)
  auto blocks_before = [&](long long v) {
    const int b = seq_of(v, cost);
    const int nb = (int)(pre[b + 1] - pre[b]);
    if (v >= V) return W;
    if (nb == 0) return (long long)pre[b] * p.nkv;
    const uint32_t rem = (uint32_t)(v - ((long long)pre[b] + (long long)cost * b) * p.nkv);
    const uint32_t kv = rem / (uint32_t)(nb + cost);
    const int off = (int)(rem - kv * (uint32_t)(nb + cost)) - cost;
    return (long long)pre[b] * p.nkv + (long long)kv * nb + (off > 0 ? off : 0);
  };
  const long long t0 = blocks_before(V * blockIdx.x / A), t1 = blocks_before(V * (blockIdx.x + 1) / A);

  // ------------------------------------------------------------------ this warp's blocks
  const int count = (int)(t1 - t0 > warp ? (t1 - t0 - warp + NC - 1) / NC : 0);
  // batches of 32 blocks, one a lane: the next one (fetched half a batch ahead), the one being
  // copied, the one being consumed (the ring is shorter than a batch, so these two at most).
  // TMA row and K scale are -1 for a block without a visible key or on a refused page.
  int pg_next = 0, row_next = -1, key_next = -1, kvh_next = 0;
  float ks_next = -1.f, vs_next = 0.f;
  int row_cur = -1;
  float ks_cur = -1.f, lvs_cur = 0.f, ks_use = -1.f, lvs_use = 0.f;
  auto fetch_pages = [&](int k) {  // blocks k .. k + 31: table entries
    key_next = -1;
    if (k + lane < count) {
      const long long tt = t0 + warp + (long long)(k + lane) * NC;
      const int b = seq_of(tt, 0);
      const SeqPlan s = plan_seq(a, b, G);
      const uint32_t u = (uint32_t)(tt - (long long)pre[b] * p.nkv);
      kvh_next = (int)(u / (uint32_t)s.blocks);
      const int key0 = (s.lo + (int)(u - (uint32_t)kvh_next * (uint32_t)s.blocks)) << 4;
      if (key0 < s.len) {
        key_next = key0;
        pg_next = ld_global(p.table + (size_t)b * p.max_pages + (key0 >> p.ps_log2));
      }
    }
  };
  auto fetch_scales = [&]() {
    ks_next = -1.f;
    vs_next = 0.f;
    row_next = -1;
    if (key_next >= 0) {
      if ((unsigned)pg_next < (unsigned)p.num_pages) {
        const size_t u = (size_t)pg_next * p.nkv + kvh_next;
        ks_next = ld_global(p.k_scales + u);
        vs_next = ld_global(p.v_scales + u);
        row_next = (int)u * p.ps + (key_next & (p.ps - 1));
      } else {
        atomicOr(p.err, kErrBadPosition);
      }
    }
  };
  const uint32_t ring0 = smem_u32(ring), bar0 = smem_u32(bars);
  // the next block into the slot at `dst`, `bar`
  int issued = 0;
  auto advance = [&](uint32_t dst, uint32_t bar) {
    if (issued >= count) return;
    const int x = issued & 31;
    if (x == 0) {
      row_cur = row_next;
      ks_cur = ks_next;
      lvs_cur = vs_next > 0.f ? log2f(vs_next) : -INFINITY;
      fetch_pages(issued + 32);
    } else if (x == 16) {
      fetch_scales();
    }
    const int row = __shfl_sync(0xffffffffu, row_cur, x);
    if (lane == 0) {
      if (row >= 0) {
        bar_expect(bar, Cfg::SLOT);
#pragma unroll
        for (int j = 0; j < Cfg::NBOX; ++j) {
          box_load(dst + j * 16 * Cfg::BOXW, &tmk, bar, j * Cfg::BOXW, row);
          box_load(dst + Cfg::TILE + j * 16 * Cfg::BOXW, &tmv, bar, j * Cfg::BOXW, row);
        }
      } else {
        bar_arrive(bar);
      }
    }
    ++issued;
  };
  // one row of a unit's queries (row = token * G + head) is one warp's to fetch, a piece ahead,
  // and to turn into fragments; a lane holds quads lane, lane + 32, ... of it, zeros past its end
  static_assert(NC == kPagedStepRows, "a warp per row");
  constexpr int Q = (HD + 127) / 128;
  uint2 raw[Q][2];  // four bf16 (the first two words) or f32 values each
  auto fetch_row = [&](long long x) {
    const int b = seq_of(x, 0);
    const SeqPlan s = plan_seq(a, b, G);
    const int kvh = (int)((uint32_t)(x - (long long)pre[b] * p.nkv) / (uint32_t)s.blocks);
    const int tok = warp / G;
    const size_t qo = (size_t)(s.row0 + tok) * a.q_stride + (size_t)(kvh * G + warp - tok * G) * HD;
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const int d = 4 * (lane + 32 * j);
      raw[j][0] = raw[j][1] = make_uint2(0u, 0u);
      if (warp < s.n * G && d < HD) {
        if (a.f32) {
          const uint4 v = ld_global(reinterpret_cast<const uint4*>((const float*)a.q + qo + d));
          raw[j][0] = make_uint2(v.x, v.y);
          raw[j][1] = make_uint2(v.z, v.w);
        } else {
          raw[j][0] = ld_global(reinterpret_cast<const uint2*>((const __nv_bfloat16*)a.q + qo + d));
        }
      }
    }
  };
  fetch_pages(0);
  if (t0 < t1) fetch_row(t0);
  fetch_scales();
  for (int i = 0; i < ns; ++i) advance(ring0 + i * Cfg::SLOT, bar0 + 8 * i);
  // shared offsets of this lane's ldmatrix rows: rows 0..15 of a tile, 16-byte chunk c + (lane / 16)
  uint32_t off[KS / 2];
#pragma unroll
  for (int c = 0; c < KS; c += 2)
    off[c / 2] = tile_addr<Cfg>(0, ((lane >> 3) & 1) * 8 + (lane & 7), 16 * (c + (lane >> 4)));

  // ------------------------------------------------------------------ pieces of units
  bool dead = false;  // a wait gave up: no more reads, the barriers still match
  int pos = warp, use = 0;  // the next block: its place in the CTA's range, its lane in the batch
  uint32_t slot = ring0, bar = bar0, phase = 0;
  const uint32_t ring_end = ring0 + ns * Cfg::SLOT;
  long long at = t0;   // first block of the piece
  while (at < t1) {
    const int b = seq_of(at, 0);
    const SeqPlan sq = plan_seq(a, b, G);
    const long long ub = (long long)pre[b] * p.nkv;
    const int kvh = (int)((uint32_t)(at - ub) / (uint32_t)sq.blocks);
    const long long u0 = ub + (long long)kvh * sq.blocks, u1 = u0 + sq.blocks;
    const long long end = u1 < t1 ? u1 : t1;
    const int rows = sq.n * G;
    {
      const int r = warp;
      float x[Q][4];
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        if (a.f32) {
          x[j][0] = __uint_as_float(raw[j][0].x), x[j][1] = __uint_as_float(raw[j][0].y);
          x[j][2] = __uint_as_float(raw[j][1].x), x[j][3] = __uint_as_float(raw[j][1].y);
        } else {
          x[j][0] = __uint_as_float(raw[j][0].x << 16), x[j][1] = __uint_as_float(raw[j][0].x & 0xffff0000u);
          x[j][2] = __uint_as_float(raw[j][0].y << 16), x[j][3] = __uint_as_float(raw[j][0].y & 0xffff0000u);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(x[j][i]));
      }
#pragma unroll
      for (int of = 16; of > 0; of >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, of));
    // 2^-e by its exponent bits: the row's largest component lands in [1, 8)
      const uint32_t E = min(max((__float_as_uint(top) >> 23) & 255u, 1u), 252u);
      const float down = __uint_as_float((254u - E) << 23);
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        const int quad = lane + 32 * j;
        __half xh[4], xl[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_f16(x[j][i] * down, xh[i], xl[i]);
        if (4 * quad < HD)
          qf[(quad >> 2) * 32 + r * 4 + (quad & 3)] = make_uint4(
              pack_h2(xh[0], xh[1]), pack_h2(xl[0], xl[1]), pack_h2(xh[2], xh[3]), pack_h2(xl[2], xl[3]));
      }
      if (lane == 0) s_rowf[r] = __uint_as_float(E << 23) * a.qscale;
    }
    if (end < t1) fetch_row(end);
    __syncthreads();
    // row g: its keys [lo, hi)
    const float rowf = s_rowf[g];
    const int P = sq.len - sq.n + g / G;
    const int hi = g < rows ? (a.bidir ? sq.len : P + 1) : 0;
    const int lo = a.window ? P - a.window + 1 : 0;
    // keys that every row sees
    const int all_hi = a.bidir ? sq.len : sq.len - sq.n + 1;
    const int all_lo = a.window ? sq.len - a.window : 0;
    float m = kNoMax, mw = kNoMax, l = 0.f;
    float o[KS][2][4];
#pragma unroll
    for (int c = 0; c < KS; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][0][e] = o[c][1][e] = 0.f;

    const int mine_end = (int)(end - t0);
    // the block at place x starts at key key_base + 16 x
    const int key_base = (sq.lo + (int)(t0 - u0)) * 16;
    for (; pos < mine_end; pos += NC) {
      if (use == 0) {  // turned for the copies ns blocks ago at the latest
        ks_use = ks_cur;
        lvs_use = lvs_cur;
      }
      if (!dead && !__all_sync(0xffffffffu, bar_wait(bar, phase, p.err))) dead = true;
      const float ks = __shfl_sync(0xffffffffu, ks_use, use);
      const float lvs = __shfl_sync(0xffffffffu, lvs_use, use);
      if (!dead && ks >= 0.f) {
        const int key0 = key_base + 16 * pos;
        const uint32_t kt = slot, vt = slot + Cfg::TILE;
        // S = Q K^T over 16 keys: tiles of keys 0..7 and 8..15
        float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < KS; c += 2) {
          uint32_t w[4];
          ldmatrix_x4(kt + off[c / 2], w[0], w[1], w[2], w[3]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 qa = qf[(c + i) * 32 + lane];
            const uint32_t A4[4] = {qa.x, qa.y, qa.z, qa.w};
            const uint32_t x0 = w[2 * i] ^ 0x80808080u, x1 = w[2 * i + 1] ^ 0x80808080u;
            mma_f16(s0, A4, u8x2_to_h2(x0, kSelLo), u8x2_to_h2(x0, kSelHi));
            mma_f16(s1, A4, u8x2_to_h2(x1, kSelLo), u8x2_to_h2(x1, kSelHi));
          }
        }
        const float f = rowf * ks;
        float s[4] = {(s0[0] + s0[2]) * f, (s0[1] + s0[3]) * f, (s1[0] + s1[2]) * f,
                      (s1[1] + s1[3]) * f};
        if (a.cap_log2 != 0.f) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[e] = a.cap_log2 * tanhf(s[e]);
        }
        if (key0 < all_lo || key0 + 16 > all_hi) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + 2 * t + (e & 1) + 8 * (e >> 1);
            if (key >= hi || key < lo) s[e] = -INFINITY;
          }
        }
        const float top = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
        if (__any_sync(0xffffffffu, top > fminf(m, mw - lvs) + kLazy)) {
          float r = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 2));
          const float mn = fmaxf(m, r), wn = fmaxf(mw, r + lvs);
          l *= exp2f(m - mn);
          const float corr = exp2f(mw - wn);
          m = mn;
          mw = wn;
#pragma unroll
          for (int c = 0; c < KS; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[c][0][e] *= corr;
              o[c][1][e] *= corr;
            }
        }
        uint32_t PA[4];
        {
          const float shift = lvs - mw;
          l += (ex2_approx(s[0] - m) + ex2_approx(s[1] - m)) + (ex2_approx(s[2] - m) + ex2_approx(s[3] - m));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float w0 = ex2_approx(s[2 * h] + shift), w1 = ex2_approx(s[2 * h + 1] + shift);
            const __half2 hi2 = __floats2half2_rn(w0, w1);
            const float2 back = __half22float2(hi2);
            const __half2 lo2 = __floats2half2_rn(w0 - back.x, w1 - back.y);
            PA[2 * h] = *reinterpret_cast<const uint32_t*>(&hi2);
            PA[2 * h + 1] = *reinterpret_cast<const uint32_t*>(&lo2);
          }
        }
#pragma unroll
        for (int c = 0; c < KS; c += 2) {
          uint32_t w[4];
          ldmatrix_x4_trans(vt + off[c / 2], w[0], w[1], w[2], w[3]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t x0 = w[2 * i] ^ 0x80808080u, x1 = w[2 * i + 1] ^ 0x80808080u;
            mma_f16(o[c + i][0], PA, u8x2_to_h2(x0, 0x4240u), u8x2_to_h2(x1, 0x4240u));
            mma_f16(o[c + i][1], PA, u8x2_to_h2(x0, 0x4341u), u8x2_to_h2(x1, 0x4341u));
          }
        }
      }
      // every lane's reads of the slot have fed the MMAs above: the slot may be refilled
      __syncwarp();
      if (!dead) advance(slot, bar);
      use = (use + 1) & 31;
      slot += Cfg::SLOT;
      bar += 8;
      if (slot == ring_end) slot = ring0, bar = bar0, phase ^= 1;
    }

    // ---------------------------------------------------------------- the CTA's record
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    // dims 16 c + 4 t .. + 3 of row g
    auto o4 = [&](int c) {
      return make_float4(o[c][0][0] + o[c][0][2], o[c][1][0] + o[c][1][2], o[c][0][1] + o[c][0][3],
                         o[c][1][1] + o[c][1][3]);
    };
    float* mine = red + (size_t)(warp % (NC / 2)) * rows * RS + g * RS;
    if (warp >= NC / 2 && g < rows) {
#pragma unroll
      for (int c = 0; c < KS; ++c) *reinterpret_cast<float4*>(mine + 16 * c + 4 * t) = o4(c);
      if (t == 0) *reinterpret_cast<float4*>(mine + HD) = make_float4(mw, m, l, 0.f);
    }
    __syncthreads();
    if (warp < NC / 2) {
      const float4 y = g < rows ? *reinterpret_cast<const float4*>(mine + HD)
                                : make_float4(kNoMax, kNoMax, 0.f, 0.f);
      __syncwarp();  // the four lanes of a row have read what one of them overwrites
      const float wn = fmaxf(mw, y.x), mn = fmaxf(m, y.y);
      const float fa = exp2f(mw - wn), fb = exp2f(y.x - wn);
      if (g < rows) {
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        float4* q4 = reinterpret_cast<float4*>(mine + 16 * c + 4 * t);
        const float4 u = o4(c), v = *q4;
        *q4 = make_float4(u.x * fa + v.x * fb, u.y * fa + v.y * fb, u.z * fa + v.z * fb,
                          u.w * fa + v.w * fb);
      }
      if (t == 0)
        *reinterpret_cast<float4*>(mine + HD) =
            make_float4(wn, mn, l * exp2f(m - mn) + y.z * exp2f(y.y - mn), 0.f);
      }
    }
    __syncthreads();
    const bool whole = at == u0 && end == u1;
    float* part = a.records + ((size_t)blockIdx.x * 2 + (at == u0)) * kPagedStepRows * RS;
    constexpr int Q4 = HD / 4;
    for (int i = threadIdx.x; i < rows * Q4; i += NC * 32) {
      const int r = i / Q4, d4 = i - r * Q4;
      float wm[NC / 2], mm = kNoMax, wx = kNoMax, ll = 0.f;
#pragma unroll
      for (int w = 0; w < NC / 2; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(red + ((size_t)w * rows + r) * RS + HD);
        wm[w] = y.x;
        wx = fmaxf(wx, y.x);
        const float mn = fmaxf(mm, y.y);
        ll = ll * exp2f(mm - mn) + y.z * exp2f(y.y - mn);
        mm = mn;
      }
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < NC / 2; ++w) {
        const float f = exp2f(wm[w] - wx);
        const float4 v = reinterpret_cast<const float4*>(red + ((size_t)w * rows + r) * RS)[d4];
        acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
      }
      if (whole) {
        const float f = ll > 0.f ? exp2f(wx - mm) / ll : 0.f;
        paged_store_o4(a, sq.row0 + r / G, kvh * G + r % G, 4 * d4,
                       make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f));
      } else {
        reinterpret_cast<float4*>(part + r * RS)[d4] = acc;
        if (d4 == 0) *reinterpret_cast<float4*>(part + r * RS + HD) = make_float4(wx, mm, ll, 0.f);
      }
    }
    if (!whole) {
      // CTAs first .. last hold parts of this unit; the last to finish combines them
      const long long v0 = u0 + (long long)cost * ((long long)b * p.nkv + kvh + 1);  // first block's place
      const int first = (int)(((v0 + 1) * A - 1) / V), last = (int)(((v0 + sq.blocks) * A - 1) / V);
      const int parts = last - first + 1;
      __syncthreads();
      if (threadIdx.x == 0) s_misc[0] = ticket_add(a.tickets + first) == parts - 1;
      __syncthreads();
      if (s_misc[0]) {
        if (threadIdx.x == 0) a.tickets[first] = 0;
        // record i of the unit: CTA first + i, its tail piece (slot 1) for i = 0
        auto rec = [&](int i, int r) {
          return a.records + (((size_t)(first + i) * 2 + (i == 0)) * kPagedStepRows + r) * RS;
        };
        if (parts <= 16) {
          // few parts: four at a time, every load of four in one round, under a running maximum
          for (int i = threadIdx.x; i < rows * Q4; i += NC * 32) {
            const int r = i / Q4, d4 = i - r * Q4;
            float wx = kNoMax, mm = kNoMax, ll = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int j0 = 0; j0 < parts; j0 += 4) {
              float4 y[4], v[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float* p4 = rec(j0 + j < parts ? j0 + j : 0, r);
                y[j] = __ldcg(reinterpret_cast<const float4*>(p4 + HD));
                v[j] = __ldcg(reinterpret_cast<const float4*>(p4) + d4);
                if (j0 + j >= parts) y[j] = make_float4(kNoMax, kNoMax, 0.f, 0.f);
              }
              const float wn = fmaxf(fmaxf(fmaxf(y[0].x, y[1].x), fmaxf(y[2].x, y[3].x)), wx);
              const float mn = fmaxf(fmaxf(fmaxf(y[0].y, y[1].y), fmaxf(y[2].y, y[3].y)), mm);
              const float f0 = exp2f(wx - wn);
              ll *= exp2f(mm - mn);
              acc.x *= f0, acc.y *= f0, acc.z *= f0, acc.w *= f0;
              wx = wn;
              mm = mn;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (j0 + j >= parts) break;
                ll += y[j].z * exp2f(y[j].y - mm);
                const float f = exp2f(y[j].x - wx);
                acc.x += f * v[j].x, acc.y += f * v[j].y, acc.z += f * v[j].z, acc.w += f * v[j].w;
              }
            }
            const float f = ll > 0.f ? exp2f(wx - mm) / ll : 0.f;
            paged_store_o4(a, sq.row0 + r / G, kvh * G + r % G, 4 * d4,
                           make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f));
          }
          at = end;
          continue;
        }
        float* wsm = red;  // [rows][parts]
        for (int r = warp; r < rows; r += NC) {
          float wx = kNoMax, mm = kNoMax;
          for (int i = lane; i < parts; i += 32) {
            const float4 y = __ldcg(reinterpret_cast<const float4*>(rec(i, r) + HD));
            wx = fmaxf(wx, y.x);
            mm = fmaxf(mm, y.y);
          }
#pragma unroll
          for (int of = 16; of > 0; of >>= 1) {
            wx = fmaxf(wx, __shfl_xor_sync(0xffffffffu, wx, of));
            mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, of));
          }
          float ll = 0.f;
          for (int i = lane; i < parts; i += 32) {
            const float4 y = __ldcg(reinterpret_cast<const float4*>(rec(i, r) + HD));
            ll += y.z * exp2f(y.y - mm);
            wsm[r * parts + i] = exp2f(y.x - wx);
          }
          ll = warp_sum(ll);
          const float f = ll > 0.f ? exp2f(wx - mm) / ll : 0.f;
          __syncwarp();
          for (int i = lane; i < parts; i += 32) wsm[r * parts + i] *= f;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < rows * Q4; i += NC * 32) {
          const int r = i / Q4, d4 = i - r * Q4;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int j = 0; j < parts; ++j) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(rec(j, r)) + d4);
            const float f = wsm[r * parts + j];
            acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
          }
          paged_store_o4(a, sq.row0 + r / G, kvh * G + r % G, 4 * d4, acc);
        }
      }
    }
    at = end;
    // red and s_misc are next written behind the barrier that follows the next piece's
    // query fragments, and qf only holds what every warp has finished with
  }
  // a warp that gave up: its copies still in flight land before the CTA may exit
  if (dead) {
    for (int i = issued > ns ? issued - ns : 0; i < issued; ++i) paged_wait(&bars[i % ns], (i / ns) & 1, p.err);
  }
}

template <int HD>
cudaError_t launch_step_hd(const PagedAttnArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                           long long blocks, int max_rows, int sms, cudaStream_t s) {
  using Cfg = StepCfg<HD>;
  const size_t fixed = 1024 + Cfg::QF + (size_t)Cfg::red_floats(max_rows) * 4 +
                       Cfg::NC * Cfg::MAXNS * 8 + (16 + Cfg::NC + a.p.batch + 1) * 4;
  const size_t budget = (Cfg::CPS == 2 ? 113 : 226) * 1024;
  int ns = (int)((budget - fixed) / (Cfg::NC * Cfg::SLOT));
  if (ns > Cfg::MAXNS) ns = Cfg::MAXNS;
  const size_t smem = fixed + (size_t)ns * Cfg::NC * Cfg::SLOT;
  cudaError_t e = cudaFuncSetAttribute(paged_step_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  long long grid = (blocks + (long long)kUnitCost * a.p.batch * a.p.nkv + 2 * Cfg::NC - 1) / (2 * Cfg::NC);
  if (grid > (long long)sms * Cfg::CPS) grid = (long long)sms * Cfg::CPS;
  if (grid > kPagedMaxParts) grid = kPagedMaxParts;
  if (grid < 1) grid = 1;
  return paged_launch(paged_step_kernel<HD>, dim3((unsigned)grid), Cfg::NC * 32, smem, s, tk, tv, a, ns, max_rows);
}

}  // namespace

cudaError_t launch_paged_step(const PagedAttnArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                              long long blocks, int max_rows, int sms, cudaStream_t s) {
  if (a.p.hd == 64) return launch_step_hd<64>(a, tk, tv, blocks, max_rows, sms, s);
  if (a.p.hd == 128) return launch_step_hd<128>(a, tk, tv, blocks, max_rows, sms, s);
  return launch_step_hd<256>(a, tk, tv, blocks, max_rows, sms, s);
}

}  // namespace hfa

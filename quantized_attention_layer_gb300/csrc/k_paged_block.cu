// k_paged_block.cu -- attention of blocks of rows (verification blocks, prompt chunks, whole
// prompts) over the paged 8-bit cache, on the 5th-generation tensor cores.
//
//   s_p = scale ks[page(p)] sum_d q_d kc[p][d]   (softcap: cap tanh(s / cap)),
//   o   = sum_p softmax(s)_p vs[page(p)] vc[p],   codes kc, vc, scales ks, vs per page and head,
// over the positions row i of a sequence's n rows sees: p <= P = len - n + i (all p < len when
// bidirectional), p > P - window with a window.
//
// The rows of a KV head are its query heads of each token in turn (row = token G + head), so a
// tile of 128 rows reads each key once for all of them.  One CTA takes QT tiles of 128 rows
// (two at hd 64 and 128, one at hd 256, where O fills half of TMEM) and walks over tiles of
// KT keys:
//   S = Q Kc^T  (M = 128 rows, N = KT keys, K = hd)   fp16 in, f32 in TMEM
//   O += P Vc   (M = 128 rows, N = hd, K = KT keys)   P fp16 in TMEM over S's own columns
// The codes are exact in fp16.  Q is the bf16 row scaled by a power of two (exact but for parts
// 2^-25 below the row's largest); the page's K scale multiplies the f32 scores 16 keys at a
// time, its V scale enters the weights' exponent:
//   w = 2^(s + log2 vs - mw), mw the running maximum of s + log2 vs, l = sum w / vs,
// so that rounding P to fp16 costs 2^-11 of a weight whatever the scales, below the bf16
// rounding of the output.  mw moves lazily: a step forms its weights under the old mw, and only
// when 16 of them add up to more than 2^12 does the row's thread find the maximum, rescale its
// O in TMEM and form them again.  So most steps need no maximum at all.
//
// Roles: a warpgroup per S buffer does the softmax (a thread owns a row: no shuffles), the
// converter warps turn int8 codes into the fp16 operand tiles (global to registers a tile
// ahead, widened by one permute and one subtract for two codes, stored in the 128-byte swizzled
// order of the MMA; V is read in place as an MN-major operand), and one warp issues the
// MMAs: while one S buffer is in its softmax the tensor cores work for the other.
// Bound: per 128 x 128 scores at hd 128 the tensor cores need 1024 cycles and the shared memory
// that feeds them about 1150.  Measured 1600: the softmax of a row tile (2000 cycles for 128
// keys) and its own two products follow one another, and two row tiles leave gaps.  An 8K prompt
// (32/8 heads, hd 128, 550 GFLOP) takes 411 us, 1340 TFLOP/s.  Before its first tile a CTA spends
// 9000 cycles (item, queries), behind its last one about 4300.
//
// When there are fewer (sequence, KV head, row tile) items than SMs, S CTAs share an item, each
// a contiguous part of its key tiles; a second kernel adds their records.
#include "hfa_common.cuh"
#include "hfa_internal.h"
#include "hfa_paged.h"

namespace hfa {
namespace {

// ONE: no CTA of the call has more than one row tile
template <int HD, bool ONE = HD == 256>
struct BlockCfg {
  static constexpr int QT = ONE ? 1 : 2;          // row tiles of a CTA
  static constexpr int ROWS = HD == 256 ? 128 : 256;  // rows that the CTAs are dealt out by
  static constexpr int KT = HD == 256 ? 64 : 128; // keys of a tile
  static constexpr int NG = KT / 16;              // 16-key groups: one scale each
  static constexpr int UK = 64, UPT = KT / UK;    // keys of a softmax step, steps of a tile
  static constexpr int SMW = QT * 4;              // softmax warps
  static constexpr int NCW = 15 - SMW;            // converter warps; warp 15 issues the MMAs
  static constexpr int THREADS = 512;
  static constexpr int BOXES = HD / 64;
  static constexpr int QBOX = 128 * 128;          // bytes of a 64-dim box of a row tile
  static constexpr int QTILE = BOXES * QBOX;
  static constexpr int KBOX = KT * 128;
  static constexpr int KTILE = BOXES * KBOX;
  static constexpr int NST = 2;                   // operand stages of K and of V
  static constexpr int NSC = 4;                   // scale slots (see sc_full)
  static constexpr int SMEM_OPS = QT * QTILE + 2 * NST * KTILE;
  static constexpr size_t SMEM = 1024 + SMEM_OPS + ROWS * 4 + NSC * (NG * 16 + 16) + 256;
  static constexpr int O_COL = QT * 2 * UK;       // TMEM: two steps' S a row tile, then O
  static constexpr int CPR = HD / 16;             // 16-byte chunks of a row of codes
  static constexpr int RPU = 32 / CPR;            // rows of a converter's unit: 32 chunks
  static constexpr int NU = KT / RPU;             // units of a tile
  static constexpr int PER = (NU + NCW - 1) / NCW;  // units of one warp
  // tiles of codes in a converter's registers: with one row tile (and more converter warps) the
  // loads' latency shows (two tiles: 31.8 us, one: 32.4)
  static constexpr int DEPTH = ONE ? 2 : 1;
  static_assert(O_COL + QT * HD <= 512, "TMEM");
  static_assert(16 % RPU == 0, "a unit lies in one group");
  static_assert(SMEM <= 232448, "shared memory");
};

constexpr float kNoMax = -1e30f;
constexpr float kMostWeight = 4096.f;  // the sum of 16 weights above which the maximum moves
constexpr float kZeroLvs = -100.f;  // log2 vs of a page whose scale is 0 (its codes count as 0)

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24) | (b_mn ? 1u << 16 : 0u);
}
// The MMAs and commits, executed by a whole warp of which one lane issues: operands that the
// warp shares stay in uniform registers, where a single thread would move each one there.
// D[tmem] (+)= A[smem desc] * B[smem desc]^T
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem desc]^T
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 w, {%6, %7};\n\tfma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ uint32_t cvt_h2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// tanh to about 1e-7 absolute from one exponential and one reciprocal
__device__ __forceinline__ float tanh_ex2(float x) {
  const float e = ex2_approx(fminf(x, 20.f) * 2.885390082f);  // e^(2x); 20: tanh is 1
  return 1.f - 2.f * rcp_approx(1.f + e);
}

// The keys the tile sees, and its rows' place: everything a role needs of its item.
struct BlockItem {
  int b, kvh, row0, n, len;   // sequence, KV head, first row of the packed arrays, rows, keys
  int r0, rows;               // first (token, head) row of the CTA's tiles, rows in them
  int lo, hi;                 // keys that some row sees
  int t0, t1;                 // key tiles of this CTA
};
// x / G for 0 <= x < 2^29 and G <= 8: x ceil(2^32 / G) >> 32 is exact there
struct DivG {
  uint32_t magic;
  __device__ __forceinline__ explicit DivG(int G) : magic(G > 1 ? 0xffffffffu / (uint32_t)G + 1u : 0u) {}
  __device__ __forceinline__ int operator()(int x) const { return magic ? (int)__umulhi((uint32_t)x, magic) : x; }
};
// lower and upper limit of the keys row r (token r / G) sees
__device__ __forceinline__ int2 row_keys(const PagedAttnArgs& a, const BlockItem& it, int tok) {
  const int P = it.len - it.n + tok;
  const int hi = a.bidir ? it.len : P + 1;
  const int lo = a.window ? P - a.window + 1 : 0;
  return make_int2(lo > 0 ? lo : 0, hi > 0 ? hi : 0);
}
// false: the slot has no rows.  One warp calls it together.
template <int HD>
__device__ __forceinline__ bool block_item(const PagedAttnArgs& a, int splits, int bid, BlockItem* out) {
  using Cfg = BlockCfg<HD>;
  const PagedView& p = a.p;
  const int G = p.nh / p.nkv;
  BlockItem it;
  const int split = bid % splits;
  const int u = bid / splits;
  it.kvh = u % p.nkv;
  const int slot = u / p.nkv;
  // sequence b owns slots cu[b] G / ROWS + b ..: n G rows need at most n G / ROWS + 1
  auto base = [&](int i) { return (int)((long long)a.cu[i] * G / Cfg::ROWS) + i; };
  it.b = find_seq(p.batch, slot, base);
  it.row0 = a.cu[it.b];
  it.n = a.cu[it.b + 1] - it.row0;
  it.len = a.len[it.b];
  if (it.n <= 0 || (long long)it.n * G <= kPagedStepRows || it.row0 < 0 || it.row0 > a.total - it.n) return false;
  const int R = it.n * G;
  const int tiles = (R + Cfg::ROWS - 1) / Cfg::ROWS;
  const int i = slot - base(it.b);
  if (i >= tiles) return false;
  if (it.len < 0 || it.len > p.max_pages * p.ps) {
    if ((threadIdx.x & 31) == 0) atomicOr(p.err, kErrBadPosition);
    it.len = 0;
  }
  it.r0 = (tiles - 1 - i) * Cfg::ROWS;  // the longest rows first
  it.rows = min(Cfg::ROWS, R - it.r0);
  const int tok0 = it.r0 / G, tok1 = (it.r0 + it.rows - 1) / G;
  const int2 k0 = row_keys(a, it, tok0), k1 = row_keys(a, it, tok1);
  it.lo = k0.x;
  it.hi = k1.y;
  if (it.hi > it.len) it.hi = it.len;
  const int ta = it.lo / Cfg::KT, tb = (it.hi + Cfg::KT - 1) / Cfg::KT;
  const int nt = tb > ta ? tb - ta : 0;
  const int per = (nt + splits - 1) / splits;
  it.t0 = ta + min(split * per, nt);
  it.t1 = ta + min((split + 1) * per, nt);
  *out = it;
  return true;
}

// ONE: no CTA of the call has more than one row tile.  Its scores then come by steps, in the
// other of two buffers, and run while a step is in its softmax; with two row tiles the other
// tile's work does, and scores come by whole tiles (by steps they read Q twice).  16 rows of 4
// sequences over 8K keys took 32.5 us by steps and 37.5 by tiles, an 8K prompt 458 and 412.
template <int HD, bool CAP, bool ONE>
__global__ void __launch_bounds__(BlockCfg<HD, ONE>::THREADS, 1)
    paged_block_kernel(const PagedAttnArgs a, int splits) {
  using Cfg = BlockCfg<HD, ONE>;
  constexpr int QT = Cfg::QT, KT = Cfg::KT, NG = Cfg::NG, UK = Cfg::UK, UPT = Cfg::UPT, HG = UK / 16, NST = Cfg::NST, NSC = Cfg::NSC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align1024(smem_raw);
  uint8_t* q_s = smem;
  uint8_t* k_s = smem + QT * Cfg::QTILE;
  uint8_t* v_s = k_s + NST * Cfg::KTILE;
  float* s_rowf = reinterpret_cast<float*>(smem + Cfg::SMEM_OPS);  // [ROWS] qscale 2^e
  // [NSC][NG] K scale (-1: the group is not visible), log2 of the V scale, 1 / the V scale
  float4* s_sc = reinterpret_cast<float4*>(s_rowf + Cfg::ROWS);
  int* s_flag = reinterpret_cast<int*>(s_sc + NSC * NG);  // [NSC] some group is refused
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_flag + NSC);
  uint64_t* q_full = bars;            // 1
  uint64_t* k_full = bars + 1;        // [NST] converted K tiles
  uint64_t* v_full = k_full + NST;
  uint64_t* k_free = v_full + NST;    // [NST] the MMAs have read them
  uint64_t* v_free = k_free + NST;
  uint64_t* sc_full = v_free + NST;   // [NSC] scales.  Slot i of tile t + NSC is written once
                                      // tile t + NSC - NST's S is done, hence after every
                                      // softmax of tile t
  uint64_t* s_full = sc_full + NSC;   // [2] the scores of a row tile's keys are there; ONE: of a step
  uint64_t* p_full = s_full + 4;      // [QT][2] its weights are written
  uint64_t* pv_done = p_full + 4;     // [QT] each step's O += P V is complete
  uint64_t* o_full = pv_done + 2;     // [QT] the last one is
  uint64_t* drain = o_full + 2;      // after an abort: what was issued is complete
  volatile int* s_abort = reinterpret_cast<volatile int*>(drain + 1);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1) + 1;
  BlockItem* s_item = reinterpret_cast<BlockItem*>(s_tmem + 1);

  const PagedView& p = a.p;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int G = p.nh / p.nkv;
  pdl_wait();
  if (warp == 0) {
    BlockItem it;
    const bool on = block_item<HD>(a, splits, blockIdx.x, &it);
    if (lane == 0) {
      if (!on) it.rows = 0;
      *s_item = it;
    }
  } else if (warp == 1) {
    if (lane == 0) {
      mbar_init(q_full, Cfg::SMW);
      for (int i = 0; i < NST; ++i) {
        mbar_init(&k_full[i], Cfg::NCW);
        mbar_init(&v_full[i], Cfg::NCW);
        mbar_init(&k_free[i], 1);
        mbar_init(&v_free[i], 1);
      }
      for (int i = 0; i < NSC; ++i) mbar_init(&sc_full[i], 1);
      for (int i = 0; i < 2; ++i) mbar_init(&s_full[i], 1);
      for (int i = 0; i < 2 * QT; ++i) mbar_init(&p_full[i], 4);
      for (int i = 0; i < QT; ++i) {
        mbar_init(&pv_done[i], 1);
        mbar_init(&o_full[i], 1);
      }
      mbar_init(drain, 1);
      *s_abort = 0;
      fence_barrier_init();
    }
  }
  __syncthreads();
  const BlockItem it = *s_item;
  if (it.rows == 0) return;
  if (warp == 2) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int tiles = !ONE && it.rows > 128 ? QT : 1;  // row tiles with rows
  const int nt = it.t1 - it.t0;

  if (warp < Cfg::SMW) {
    // ================================================================== softmax warps
    const int j = warp >> 2;  // row tile
    const int quad = warp & 3;
    const DivG divg(G);
    // ---- queries: a warp's 32 rows, L lanes a row with 8 dims each; every load of a round in
    // flight at once
    {
      constexpr int L = HD / 8 < 32 ? HD / 8 : 32;  // lanes of a row
      constexpr int RPI = 32 / L;                   // rows of an instruction
      constexpr int NI = 32 / RPI, NB = NI < 16 ? NI : 16;
      const int c = lane % L;
#pragma unroll 1
      for (int i0 = 0; i0 < NI; i0 += NB) {
        uint4 w[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int r = quad * 32 + (i0 + i) * RPI + lane / L;  // row of the tile
          const int R = it.r0 + j * 128 + r, tok = divg(R);
          w[i] = make_uint4(0u, 0u, 0u, 0u);
          if (j * 128 + r < it.rows)
            w[i] = ld_global(reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.q +
                                                        (size_t)(it.row0 + tok) * a.q_stride +
                                                        (size_t)(it.kvh * G + R - tok * G) * HD + 8 * c));
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int r = quad * 32 + (i0 + i) * RPI + lane / L;
          // largest exponent of the row (the bf16 exponent bits of either half)
          uint32_t e = 0;
          const uint32_t ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) e = max(e, max((ww[x] >> 7) & 255u, (ww[x] >> 23) & 255u));
#pragma unroll
          for (int o = 1; o < L; o <<= 1) e = max(e, __shfl_xor_sync(0xffffffffu, e, o));
          e = min(max(e, 1u), 252u);
          const float down = __uint_as_float((254u - e) << 23);
          uint32_t hw[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            hw[x] = cvt_h2(__uint_as_float(ww[x] << 16) * down, __uint_as_float(ww[x] & 0xffff0000u) * down);
          const int box = c >> 3, ch = c & 7;
          *reinterpret_cast<uint4*>(q_s + j * Cfg::QTILE + box * Cfg::QBOX + r * 128 +
                                    ((ch ^ (r & 7)) << 4)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
          if (c == 0) s_rowf[j * 128 + r] = __uint_as_float(e << 23) * a.qscale;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    // ---- this thread's row
    const int r = quad * 32 + lane;
    const bool on = j * 128 + r < it.rows;
    const int tok = divg(it.r0 + j * 128 + r);
    int2 lim = on ? row_keys(a, it, tok) : make_int2(0, 0);
    if (lim.y > it.len) lim.y = it.len;
    // keys that every row of the warp sees: [wlo, whi)
    int wlo = lim.x, whi = on ? lim.y : 0x7fffffff;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      wlo = max(wlo, __shfl_xor_sync(0xffffffffu, wlo, o));
      whi = min(whi, __shfl_xor_sync(0xffffffffu, whi, o));
    }
    const float rowf = s_rowf[j * 128 + r];  // written by this warp
    const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
    float mw = kNoMax, l = 0.f;
    bool ok = true;
    const uint32_t t_o = t_lane + Cfg::O_COL + j * HD;
    const int steps = j < tiles ? nt * UPT : 0;
#pragma unroll 1
    for (int u = 0; u < steps; ++u) {
      const int sb = 2 * j + (u & 1);
      const int i = u / UPT, sc = i % NSC;
      const int kh = it.t0 * KT + u * UK;  // first key
      const uint32_t t_h = t_lane + sb * UK;
      if (u % UPT == 0) {
        ok = paged_wait(&sc_full[sc], (i / NSC) & 1, p.err, (const volatile int*)s_abort) &&
             (!ONE ? paged_wait(&s_full[j], i & 1, p.err, (const volatile int*)s_abort)
                   : paged_wait(&s_full[u & 1], (u >> 1) & 1, p.err, (const volatile int*)s_abort));
      } else if (ONE) {
        ok = paged_wait(&s_full[u & 1], (u >> 1) & 1, p.err, (const volatile int*)s_abort);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const float4* f4 = s_sc + sc * NG + (u % UPT) * HG;
      const bool masked = kh < wlo || kh + UK > whi || s_flag[sc];
      // the columns of group c that hold keys this row sees
      auto from = [&](int c) { return lim.x - (kh + 16 * c); };
      auto to = [&](int c) { return f4[c].x >= 0.f ? lim.y - (kh + 16 * c) : 0; };
      uint32_t w[HG / 2][16];
      float sums;
      bool raise = u == 0;  // there is no maximum yet
      for (int round = 0; round < 2; ++round) {
        uint32_t x[HG][16];
        if (raise) {
          // ---- rare: the maximum moves, O and l follow
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < HG; ++c) {
            tmem_ld16_nowait(t_h + 16 * c, x[0]);
            tmem_wait_ld();
            float gm = -INFINITY;
            const int e0 = masked ? from(c) : 0, e1 = masked ? to(c) : 16;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e >= e0 && e < e1) gm = fmaxf(gm, __uint_as_float(x[0][e]));
            if (gm != -INFINITY) {
              const float4 f = f4[c];
              float s = gm * (f.x * rowf);
              if (CAP) s = a.cap_log2 * tanh_ex2(s);
              top = fmaxf(top, s + f.y);
            }
          }
          const float mn = fmaxf(mw, top);
          const float corr = exp2f(mw - mn);
          l *= corr;
          mw = mn;
          if (u > 0) {
            ok = __all_sync(0xffffffffu,
                            paged_wait(&pv_done[j], (u - 1) & 1, p.err, (const volatile int*)s_abort));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < HD / 16; ++c) {
              uint32_t y[16];
              tmem_ld16_nowait(t_o + 16 * c, y);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * corr);
              tmem_st16(t_o + 16 * c, y);
            }
          }
        }
        // ---- weights under the present maximum: 16 scores become 8 words
#pragma unroll
        for (int c = 0; c < HG; ++c) tmem_ld16_nowait(t_h + 16 * c, x[c]);
        tmem_wait_ld();
        float most = 0.f;
        sums = 0.f;
        auto weights = [&](int c, int from, int to) {
          const float4 f = f4[c];
          const float kq = f.x * rowf, sh = f.y - mw;
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float2 s = make_float2(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
            if (!CAP) {
              s = fma2(s, make_float2(kq, kq), make_float2(sh, sh));
            } else {
              s = mul2(s, make_float2(kq, kq));
              s.x = a.cap_log2 * tanh_ex2(s.x) + sh;
              s.y = a.cap_log2 * tanh_ex2(s.y) + sh;
            }
            s.x = ex2_approx(s.x);
            s.y = ex2_approx(s.y);
            if (e < from || e >= to) s.x = 0.f;
            if (e + 1 < from || e + 1 >= to) s.y = 0.f;
            sum = add2(sum, s);
            w[c >> 1][8 * (c & 1) + (e >> 1)] = cvt_h2(s.x, s.y);
          }
          most = fmaxf(most, sum.x + sum.y);
          sums += (sum.x + sum.y) * f.z;
        };
        if (!masked) {
#pragma unroll
          for (int c = 0; c < HG; ++c) weights(c, 0, 16);
        } else {
#pragma unroll
          for (int c = 0; c < HG; ++c) weights(c, from(c), to(c));
        }
        // formed again when they are too large: they are then at most 1 (up to the rounding of
        // scores past 2^24, hence the limit on the rounds)
        raise = __any_sync(0xffffffffu, most > kMostWeight);
        if (!raise) break;
      }
      if (!ok) break;
      l += sums;
#pragma unroll
      for (int c = 0; c < HG / 2; ++c) tmem_st16(t_h + 16 * c, w[c]);  // over the scores
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[sb]);
    }
    if (!ok) *s_abort = 1;
    // ---- the rows' output
    if (ok && steps > 0) {
      ok = __all_sync(0xffffffffu, paged_wait(&o_full[j], 0, p.err, (const volatile int*)s_abort));
      if (!ok) *s_abort = 1;
    }
    tc_fence_after();
    if (ok) {
      if (splits == 1) {
        // rows to bf16, through the query tile's place (its MMAs are done) so that a warp stores
        // whole rows: 16-byte chunk c of row r at (c XOR (r % 8))
        const float f = l > 0.f ? 1.f / l : 0.f;
        uint8_t* stage = q_s + j * Cfg::QTILE + quad * 32 * (HD * 2);
#pragma unroll 1
        for (int c = 0; c < HD / 16; c += 4) {
          uint32_t x[4][16];
#pragma unroll
          for (int h = 0; h < 4; ++h)
            if (steps > 0) tmem_ld16_nowait(t_o + 16 * (c + h), x[h]);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              w[e] = steps > 0 ? pack_bf2(__float2bfloat16_rn(__uint_as_float(x[h][2 * e]) * f),
                                          __float2bfloat16_rn(__uint_as_float(x[h][2 * e + 1]) * f))
                               : 0u;
#pragma unroll
            for (int y = 0; y < 2; ++y)
              *reinterpret_cast<uint4*>(stage + lane * (HD * 2) + (((2 * (c + h) + y) ^ (lane & 7)) << 4)) =
                  make_uint4(w[4 * y], w[4 * y + 1], w[4 * y + 2], w[4 * y + 3]);
          }
        }
        __syncwarp();
        constexpr int L = HD / 8;  // chunks of a row
#pragma unroll 4
        for (int i = lane; i < 32 * L; i += 32) {
          const int row = i / L, c = i % L;
          const int rr = j * 128 + quad * 32 + row;
          if (rr >= it.rows) break;
          const int R = it.r0 + rr, tk = divg(R);
          *reinterpret_cast<uint4*>((__nv_bfloat16*)a.o +
                                    ((size_t)(it.row0 + tk) * p.nh + it.kvh * G + (R - tk * G)) * HD + 8 * c) =
              *reinterpret_cast<const uint4*>(stage + row * (HD * 2) + ((c ^ (row & 7)) << 4));
        }
      } else {
        float* rec = a.block_records + ((size_t)blockIdx.x * Cfg::ROWS + j * 128 + r) * kPagedRecord(HD);
        if (steps > 0) {
#pragma unroll 4
          for (int c = 0; c < HD / 16; ++c) {
            uint32_t x[16];
            tmem_ld16_nowait(t_o + 16 * c, x);
            tmem_wait_ld();
            if (on) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                reinterpret_cast<uint4*>(rec + 16 * c)[e] =
                    make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
            }
          }
        }
        if (on) *reinterpret_cast<float4*>(rec + HD) = make_float4(mw, l, 0.f, 0.f);
      }
    }
  } else if (warp < Cfg::SMW + Cfg::NCW) {
    // ================================================================== converter warps
    const int cw = warp - Cfg::SMW;
    // a unit's lanes: four chunks of each row, then the next four: the eight lanes of a store's
    // phase come from two rows and hit eight different 16-byte columns
    constexpr int PER = Cfg::PER, RPU = Cfg::RPU;
    const int rr = (lane >> 2) % RPU, chunk = (lane & 3) + 4 * (lane / (4 * RPU));
    // unit x of this warp: rows RPU (cw + NCW x) ..
    auto unit_row = [&](int x) { return (cw + Cfg::NCW * x) * RPU + rr; };
    // where a unit's codes go: 32 bytes of the swizzled fp16 tile, columns 2 (chunk % 4) and
    // + 1 of box chunk / 4 (the second is the first with bit 4 turned)
    uint32_t place[PER];
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      const int row = unit_row(x);
      place[x] = (chunk >> 2) * Cfg::KBOX + row * 128 + ((2 * (chunk & 3)) ^ (row & 7)) * 16;
    }
    // table entries and scales come TB tiles at a time, lane l's for group l % NG of the batch's
    // tile l / NG: a warp that uses a load's result may wait for every later load too (they share
    // scoreboards), so that happens twice a batch and not twice a tile
    constexpr int TB = 32 / NG;
    static_assert(TB >= 4 && TB - Cfg::DEPTH >= 2, "entries, rows and scales are two tiles apart");
    auto key_of = [&](int batch) { return (it.t0 + batch * TB + lane / NG) * KT + 16 * (lane % NG); };
    auto wanted = [&](int batch) {
      return batch * TB + lane / NG < nt && key_of(batch) < it.hi && key_of(batch) + 16 > it.lo;
    };
    const int* table = p.table + (size_t)it.b * p.max_pages;
    auto fetch_page = [&](int batch) {
      return wanted(batch) ? ld_global(table + (key_of(batch) >> p.ps_log2)) : 0;
    };
    // the group's first row in the pools, -1 when nothing of it is read (outside the visible
    // keys), -2 for a refused page
    auto group_row = [&](int batch, int pg) {
      if (!wanted(batch)) return -1;
      if ((unsigned)pg >= (unsigned)p.num_pages) return -2;
      return (pg * p.nkv + it.kvh) * p.ps + (key_of(batch) & (p.ps - 1));
    };
    // rows that nobody sees come from the pool's first row: finite codes of weight 0
    auto load = [&](const int8_t* codes, int rows, int i, uint4 (&w)[PER]) {  // tile i's
      const int8_t* at = codes + 16 * chunk;
      const int rows0 = max(rows, 0), from = i % TB * NG;
#pragma unroll
      for (int x = 0; x < PER; ++x) {
        const int row = unit_row(x);
        const int base = __shfl_sync(0xffffffffu, rows0, from + (row >> 4));
        if ((x + 1) * Cfg::NCW <= Cfg::NU || row < KT)
          w[x] = ld_global(reinterpret_cast<const uint4*>(at + (size_t)(base + (row & 15)) * HD));
      }
    };
    auto store = [&](uint8_t* tile, const uint4 (&w)[PER]) {
#pragma unroll
      for (int x = 0; x < PER; ++x) {
        if ((x + 1) * Cfg::NCW > Cfg::NU && unit_row(x) >= KT) break;
        const uint32_t u[4] = {w[x].x ^ 0x80808080u, w[x].y ^ 0x80808080u, w[x].z ^ 0x80808080u,
                               w[x].w ^ 0x80808080u};
        *reinterpret_cast<uint4*>(tile + place[x]) =
            make_uint4(u8x2_to_h2(u[0], kSelLo), u8x2_to_h2(u[0], kSelHi), u8x2_to_h2(u[1], kSelLo),
                       u8x2_to_h2(u[1], kSelHi));
        *reinterpret_cast<uint4*>(tile + (place[x] ^ 16)) =
            make_uint4(u8x2_to_h2(u[2], kSelLo), u8x2_to_h2(u[2], kSelHi), u8x2_to_h2(u[3], kSelLo),
                       u8x2_to_h2(u[3], kSelHi));
      }
    };
    auto scales = [&](int gr, float& k, float& v) {
      k = v = 0.f;
      if (gr >= 0) {
        k = ld_global(p.k_scales + (gr >> p.ps_log2));
        v = ld_global(p.v_scales + (gr >> p.ps_log2));
      }
    };
    // in flight: the codes of DEPTH tiles, the rows and scales of the next batch
    constexpr int DEPTH = Cfg::DEPTH;
    uint4 kws[DEPTH][PER], vws[DEPTH][PER];
    float ks, vs, ks1 = 0.f, vs1 = 0.f;
    int pg1 = 0;
    int grow = group_row(0, fetch_page(0)), grow1 = -1;
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      load(p.k_codes, grow, d, kws[d]);
      load(p.v_codes, grow, d, vws[d]);
    }
    scales(grow, ks, vs);
    const bool lead = cw == 0;
    // tile i: false when a wait gave up
    auto convert = [&](int i, uint4 (&kw)[PER], uint4 (&vw)[PER]) {
      const int st = i % NST, sc = i % NSC, bt = i % TB;
      const uint32_t ph = ((i / NST) & 1) ^ 1;
      if (bt == 0) {
        if (i > 0) grow = grow1, ks = ks1, vs = vs1;
        pg1 = fetch_page(i / TB + 1);
      } else if (bt == 2) {
        grow1 = group_row(i / TB + 1, pg1);
        scales(grow1, ks1, vs1);
      }
      const int grow_ahead = bt >= TB - DEPTH ? grow1 : grow;  // of the batch of tile i + DEPTH
      bool ok = i < NST || paged_wait(&k_free[st], ph, p.err, (const volatile int*)s_abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return false;
      const bool mine = lane / NG == bt;  // this lane's group is of tile i
      if (lead) {
        const bool any_bad = __any_sync(0xffffffffu, mine && grow == -2);
        if (mine) {
          const bool live = vs > 0.f;
          s_sc[sc * NG + lane % NG] = make_float4(grow >= 0 ? ks : -1.f, live ? log2f(vs) : kZeroLvs,
                                                  live ? 1.f / vs : 1.2676506e30f /* 2^100 */, 0.f);
        }
        if (lane == 0) {
          s_flag[sc] = any_bad;
          if (any_bad) atomicOr(p.err, kErrBadPosition);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_full[sc]);
      }
      store(k_s + st * Cfg::KTILE, kw);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[st]);
      load(p.k_codes, grow_ahead, i + DEPTH, kw);
      ok = i < NST || paged_wait(&v_free[st], ph, p.err, (const volatile int*)s_abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return false;
      // pages with V scale 0 count as zeros, whatever their codes
      const uint32_t zero = __ballot_sync(0xffffffffu, mine && grow >= 0 && !(vs > 0.f)) >> (bt * NG);
      if (zero) {
#pragma unroll
        for (int x = 0; x < PER; ++x)
          if (zero >> (unit_row(x) >> 4) & 1u) vw[x] = make_uint4(0u, 0u, 0u, 0u);
      }
      store(v_s + st * Cfg::KTILE, vw);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[st]);
      load(p.v_codes, grow_ahead, i + DEPTH, vw);
      return true;
    };
    for (int i = 0; i < nt; i += DEPTH) {
      bool ok = true;
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) ok = ok && (i + d >= nt || convert(i + d, kws[d], vws[d]));
      if (!ok) {
        *s_abort = 1;
        break;
      }
    }
  } else {
    // ================================================================== MMA issuer
    // a wait whose outcome the warp shares: the elections below need every lane
    auto wait = [&](uint64_t* bar, uint32_t ph) {
      return (bool)__all_sync(0xffffffffu, paged_wait(bar, ph, p.err, (const volatile int*)s_abort));
    };
    constexpr uint32_t idS = idesc_f16_f32(128, ONE ? UK : KT, false);
    constexpr uint32_t idO = idesc_f16_f32(128, HD, true);
    const uint32_t qa = smem_u32(q_s), ka = smem_u32(k_s), va = smem_u32(v_s);
    // S = Q K^T for row tile j: of tile x, or (ONE) of step x
    auto issue_s = [&](int x, int j) {
      const int tile = ONE ? x / UPT : x;
      const uint32_t d = tmem + (ONE ? x & 1 : 2 * j) * UK;
      // descriptors count addresses in 16 bytes: steps are added to the first one
      const uint64_t qd = smem_desc_sw128(qa + j * Cfg::QTILE),
                     kd = smem_desc_sw128(ka + tile % NST * Cfg::KTILE + (ONE ? x % UPT * (UK * 128) : 0));
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk)
        mma_ss(d, qd + (((kk >> 2) * Cfg::QBOX + (kk & 3) * 32) >> 4),
               kd + (((kk >> 2) * Cfg::KBOX + (kk & 3) * 32) >> 4), idS, kk != 0);
      mma_commit(&s_full[ONE ? x & 1 : j]);
    };
    // O += P V of step u, once its weights are there
    auto issue_pv = [&](int u, int j) {
      const int sb = 2 * j + (u & 1);
      const uint64_t vd = smem_desc_sw128_mn(va + (u / UPT % NST) * Cfg::KTILE + (u % UPT) * (UK * 128), Cfg::KBOX);
      if (!wait(&p_full[sb], (u >> 1) & 1)) return false;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < UK / 16; ++kk)
        mma_ts(tmem + Cfg::O_COL + j * HD, tmem + sb * UK + kk * 8, vd + ((kk * 2048) >> 4), idO,
               (u | kk) != 0);
      mma_commit(&pv_done[j]);
      return true;
    };
    bool ok = wait(q_full, 0);
    if (!ONE) {
      // tile i: P V of tile i - 1, then S of tile i over it, for one row tile while the other is
      // in its softmax
      for (int i = 0; ok && i <= nt; ++i) {
        if (i > 0) ok = wait(&v_full[(i - 1) % NST], ((i - 1) / NST) & 1);
        for (int j = 0; ok && j < tiles; ++j) {
          if (i > 0) {
            ok = issue_pv(UPT * (i - 1), j) && issue_pv(UPT * (i - 1) + 1, j);
            if (ok && i == nt) mma_commit(&o_full[j]);
          }
          if (i < nt) {
            if (ok && j == 0) ok = wait(&k_full[i % NST], (i / NST) & 1);
            if (!ok) break;
            tc_fence_after();
            issue_s(i, j);
          }
        }
        if (!ok) break;
        if (i > 0) mma_commit(&v_free[(i - 1) % NST]);
        if (i < nt) mma_commit(&k_free[i % NST]);
      }
    } else {
      // S of step u + 1 runs while step u is in its softmax, over step u - 1
      const int steps = nt * UPT;
      for (int u = -1; ok && u < steps; ++u) {
        if (u + 1 < steps) {
          const int x = (u + 1) / UPT;
          if ((u + 1) % UPT == 0) ok = wait(&k_full[x % NST], (x / NST) & 1);
          if (!ok) break;
          tc_fence_after();
          issue_s(u + 1, 0);
          if ((u + 2) % UPT == 0) mma_commit(&k_free[x % NST]);
        }
        if (u >= 0) {
          const int x = u / UPT;
          if (u % UPT == 0) ok = wait(&v_full[x % NST], (x / NST) & 1);
          ok = ok && issue_pv(u, 0);
          if (!ok) break;
          if (u == steps - 1) mma_commit(&o_full[0]);
          if ((u + 1) % UPT == 0) mma_commit(&v_free[x % NST]);
        }
      }
    }
    if (!ok) {
      // what was issued finishes before the tensor memory goes
      *s_abort = 1;
      mma_commit(drain);
      paged_wait(drain, 0, p.err);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, 512);
}

// Adds the parts of items shared by several CTAs: a warp per row.
template <int HD>
__global__ void __launch_bounds__(256) paged_block_merge_kernel(const PagedAttnArgs a, int splits) {
  using Cfg = BlockCfg<HD>;
  constexpr int RS = kPagedRecord(HD);
  const PagedView& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.nh / p.nkv;
  pdl_wait();
  BlockItem it;
  const int u = blockIdx.x / (Cfg::ROWS / 8);
  if (!block_item<HD>(a, splits, u * splits, &it)) return;
  const int r = (blockIdx.x % (Cfg::ROWS / 8)) * 8 + warp;
  if (r >= it.rows) return;
  const float* rec = a.block_records + ((size_t)u * splits * Cfg::ROWS + r) * RS;
  const size_t step = (size_t)Cfg::ROWS * RS;
  float M = kNoMax, my_m = kNoMax, my_l = 0.f;
  if (lane < splits) {
    const float2 y = __ldcg(reinterpret_cast<const float2*>(rec + lane * step + HD));
    my_m = y.x;
    my_l = y.y;
  }
  M = my_m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float f = my_l > 0.f ? exp2f(my_m - M) : 0.f;
  const float l = warp_sum(f * my_l);
  f = l > 0.f ? f / l : 0.f;
  const int R = it.r0 + r, tok = R / G;
  constexpr int Q = (HD + 127) / 128;
  float4 acc[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < splits; ++s) {
    const float w = __shfl_sync(0xffffffffu, f, s);
    if (w == 0.f) continue;  // a part without visible keys wrote no O
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int d = 4 * (lane + 32 * q);
      if (d < HD) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(rec + s * step + d));
        acc[q].x += w * v.x, acc[q].y += w * v.y, acc[q].z += w * v.z, acc[q].w += w * v.w;
      }
    }
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int d = 4 * (lane + 32 * q);
    if (d < HD) paged_store_o4(a, it.row0 + tok, it.kvh * G + R - tok * G, d, acc[q]);
  }
}

template <int HD>
cudaError_t launch_block_hd(const PagedAttnArgs& a, int slots, int splits, bool one, cudaStream_t s) {
  using Cfg = BlockCfg<HD>;
  const bool cap = a.cap_log2 != 0.f;
  auto kern = cap ? paged_block_kernel<HD, true, true> : paged_block_kernel<HD, false, true>;
  size_t smem = BlockCfg<HD, true>::SMEM;
  if constexpr (Cfg::QT == 2)
    if (!one) {
      kern = cap ? paged_block_kernel<HD, true, false> : paged_block_kernel<HD, false, false>;
      smem = Cfg::SMEM;
    }
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int units = slots * a.p.nkv;
  e = paged_launch(kern, dim3((unsigned)(units * splits)), Cfg::THREADS, smem, s, a, splits);
  if (e != cudaSuccess || splits == 1) return e;
  return paged_launch(paged_block_merge_kernel<HD>, dim3((unsigned)(units * (Cfg::ROWS / 8))), 256, 0, s, a, splits);
}

}  // namespace

int paged_block_rows(int hd) { return hd == 256 ? BlockCfg<256>::ROWS : BlockCfg<128>::ROWS; }
int paged_block_keys(int hd) { return hd == 256 ? BlockCfg<256>::KT : BlockCfg<128>::KT; }

cudaError_t launch_paged_block(const PagedAttnArgs& a, int slots, int splits, int max_rows, cudaStream_t s) {
  const bool one = max_rows <= 128;
  if (a.p.hd == 64) return launch_block_hd<64>(a, slots, splits, one, s);
  if (a.p.hd == 128) return launch_block_hd<128>(a, slots, splits, one, s);
  return launch_block_hd<256>(a, slots, splits, one, s);
}

}  // namespace hfa

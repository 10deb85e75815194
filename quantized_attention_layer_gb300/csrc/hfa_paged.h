// hfa_paged.h -- the paged 8-bit key/value cache: launch arguments shared by its kernels
// (k_paged.cu: append and read; k_paged_step.cu, k_paged_block.cu: attention) and its C entries
// (hfa_paged_api.cu).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace hfa {

// The pool and the batch, as every kernel sees them.
struct PagedView {
  int8_t* k_codes;      // [num_pages, nkv, ps, hd]
  int8_t* v_codes;
  float* k_scales;      // [num_pages, nkv]
  float* v_scales;
  const int* table;     // [batch, max_pages]
  int num_pages, max_pages;
  int ps, ps_log2;      // page size
  int nh, nkv, hd;
  int batch;
  unsigned* err;        // the handle's error word
};

struct PagedAppendArgs {
  PagedView p;
  const int* cu;        // [batch + 1]
  const int* start;     // [batch]
  int total;            // rows of the packed arrays (bounds the rows cu may name)
  int single;           // every sequence has at most one row
  // a page's CTAs: kv_groups of kv_per_cta K and V heads, then groups of q_per_cta query heads
  int kv_groups, kv_per_cta, q_per_cta;
  const void *q, *k, *v;  // q nullable
  long long q_stride, k_stride, v_stride;  // elements
  void* q_out;
  const float2* rope_g;  // [hd/2] (hi, lo) of theta^(-2i/hd) / (2 pi) / f_i
  const float4* slot_turn;  // [ps][hd/4] (cos, sin) of pairs 2i and 2i + 1 at positions 0 .. ps - 1
  const float* w_q;     // nullable [hd]
  const float* w_k;
  int v_unit_norm;
  float eps;
};

struct PagedReadArgs {
  PagedView p;
  const int* start;     // [batch]
  const int* count;
  int heads_per_cta;
  int capacity;
  __nv_bfloat16* k_cache;  // [batch, nkv, capacity, hd]
  __nv_bfloat16* v_cache;
};

struct PagedAttnArgs {
  PagedView p;
  const int* cu;        // [batch + 1]
  const int* len;       // [batch]
  int total;            // rows
  const void* q;
  long long q_stride;   // elements
  void* o;              // dense [total, nh, hd]
  int f32;              // q and o are f32, else bf16
  int window, bidir;
  float qscale;         // scale * log2 e, or scale / softcap
  float cap_log2;       // softcap * log2 e, 0 = none
  int* tickets;         // [kPagedMaxParts], zero between calls: parts of a unit that are done, at the
                        // number of the unit's first CTA (a CTA is the first of one shared unit at most)
  float* records;       // [2 * kPagedMaxParts][kPagedStepRows][kPagedRecord(hd)]
  float* block_records;  // [CTAs][rows of a CTA][kPagedRecord(hd)], with splits > 1
};

// The step kernel (k_paged_step.cu) serves the sequences whose rows x heads of a KV head are
// at most kPagedStepRows, on at most kPagedMaxParts CTAs.  A record holds one row's part of
// the attention: O[hd], the maximum of s + log2 vs its weights refer to, the maximum of s,
// the denominator, a pad.
constexpr int kPagedStepRows = 8;
constexpr int kPagedMaxParts = 320;
constexpr int kPagedMaxSplits = 32;
__host__ __device__ constexpr int kPagedRecord(int hd) { return hd + 4; }

cudaError_t launch_paged_append(const PagedAppendArgs& a, bool f32, int items, int sms, cudaStream_t s);
cudaError_t launch_paged_read(const PagedReadArgs& a, int max_count, int sms, cudaStream_t s);
// The block kernel (k_paged_block.cu) serves the others, paged_block_rows(hd) rows x heads and
// paged_block_keys(hd) keys at a time.  slots: total * G / rows + batch; splits (at most
// kPagedMaxSplits): CTAs that share the keys of an item; max_rows: most rows x heads of a KV head
// of a sequence.
int paged_block_rows(int hd);
int paged_block_keys(int hd);
cudaError_t launch_paged_block(const PagedAttnArgs& a, int slots, int splits, int max_rows, cudaStream_t s);
// blocks: the 16-key blocks of the sequences it serves, times nkv; max_rows: their most rows x
// heads of a KV head; tk, tv: byte views of the pools in boxes of 16 rows
cudaError_t launch_paged_step(const PagedAttnArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                              long long blocks, int max_rows, int sms, cudaStream_t s);

// Launches a kernel that may start while the one before it ends: it waits for that one
// (pdl_wait) before its first access to global memory and to tensor memory.  2 us a call at the
// head of a kernel (1 token, 1K keys: 18.5 -> 16 us).  None of these kernels lets the one behind
// it start before its own end: that one may be of another file and read before it waits.
template <class... P, class... T>
cudaError_t paged_launch(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s,
                         T... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ------------------------------------------------------------------ device helpers
#ifdef __CUDACC__
// Loads of data that the kernel before may have written.  They stay behind pdl_wait, where a
// load declared read-only (__ldg) could be moved before it, or find a line that this SM's L1
// took in before.
__device__ __forceinline__ int ld_global(const int* p) {
  int x;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ float ld_global(const float* p) {
  float x;
  asm volatile("ld.global.b32 %0, [%1];" : "=f"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ uint2 ld_global(const uint2* p) {
  uint2 x;
  asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "l"(p));
  return x;
}
__device__ __forceinline__ uint4 ld_global(const uint4* p) {
  uint4 x;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
  return x;
}
__device__ __forceinline__ float4 ld_global(const float4* p) {
  const uint4 x = ld_global(reinterpret_cast<const uint4*>(p));
  return make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w));
}
// The same by shared-window address (no generic pointer to convert in a loop).
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// mbar_wait with its limit in SM cycles (about 2 s): between two tries it reads the cycle
// counter, a few cycles, where the nanosecond timer takes long enough to delay every hand-over
// of a pipeline that waits on each tile
constexpr long long kPagedWaitCycles = 4000000000ll;
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, unsigned* err,
                                         const volatile int* abort = nullptr) {
  if (bar_try(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (bar_try(bar, parity)) return true;
    if (abort && *abort) return false;
    if (clock64() - t0 > kPagedWaitCycles) break;
  }
  atomicOr(err, kErrWaitTimeout);
  return false;
}
__device__ __forceinline__ bool paged_wait(uint64_t* bar, uint32_t parity, unsigned* err,
                                           const volatile int* abort = nullptr) {
  return bar_wait(smem_u32(bar), parity, err, abort);
}
// a 2-D TMA box by shared-window addresses
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// four adjacent dims of an output row
__device__ __forceinline__ void paged_store_o4(const PagedAttnArgs& a, int row, int h, int d, float4 v) {
  const size_t at = ((size_t)row * a.p.nh + h) * a.p.hd + d;
  if (a.f32) {
    *reinterpret_cast<float4*>((float*)a.o + at) = v;
  } else {
    *reinterpret_cast<uint2*>((__nv_bfloat16*)a.o + at) =
        make_uint2(pack_bf2(__float2bfloat16_rn(v.x), __float2bfloat16_rn(v.y)),
                   pack_bf2(__float2bfloat16_rn(v.z), __float2bfloat16_rn(v.w)));
  }
}
// The sequence that owns slot i of a ragged index space: sequence b owns slots
// base(b) .. base(b + 1) - 1 with base not decreasing and base(0) = 0.  One warp narrows the
// range 32-fold a round (one load round trip up to 32 sequences, two up to 1024).
template <class Base>
__device__ __forceinline__ int find_seq(int batch, int i, const Base& base) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int off = lane * step;
    const bool le = off < n && base(lo + off) <= i;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    const int sel = (c > 0 ? c - 1 : 0) * step;
    lo += sel;
    n = min(step, n - sel);
  }
  return lo;
}
#endif

}  // namespace hfa

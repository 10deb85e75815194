// hfa_paged_api.cu -- C entries of the paged 8-bit key/value cache: argument checks, launch
// sizes and workspace layout (include/hfa.h).  Kernels: k_paged.cu,
// k_paged_step.cu, k_paged_block.cu.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <new>
#include <vector>

#include "hfa_common.cuh"
#include "hfa_internal.h"
#include "hfa_paged.h"

struct hfa_paged {
  hfa_paged_desc d;
  int device = 0, num_sms = 0;
  int ps_log2 = 0;
  void* block = nullptr;  // error word, RoPE table, norm weights, the slots' turns
  unsigned* err = nullptr;
  float2* rope_g = nullptr;
  float4* slot_turn = nullptr;
  float* w_q = nullptr;
  float* w_k = nullptr;
  char msg[512] = {0};
};

namespace {

thread_local char g_paged_error[512];

hfa_status fail(hfa_paged* p, hfa_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(p ? p->msg : g_paged_error, 512, fmt, ap);
  va_end(ap);
  return st;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

hfa_status validate(const hfa_paged_desc* d) {
  if (!d) return fail(nullptr, HFA_EINVAL, "desc is NULL");
  if (d->num_heads <= 0 || d->num_kv_heads <= 0 || d->num_heads % d->num_kv_heads)
    return fail(nullptr, HFA_EINVAL, "num_heads=%d must be a positive multiple of num_kv_heads=%d",
                d->num_heads, d->num_kv_heads);
  if (d->num_heads / d->num_kv_heads > 8)
    return fail(nullptr, HFA_EUNSUPPORTED, "GQA group %d > 8", d->num_heads / d->num_kv_heads);
  if (d->num_kv_heads > 4096)
    return fail(nullptr, HFA_EUNSUPPORTED, "num_kv_heads=%d > 4096", d->num_kv_heads);
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
    return fail(nullptr, HFA_EUNSUPPORTED, "head_dim=%d (supported: 64, 128, 256)", d->head_dim);
  if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128)
    return fail(nullptr, HFA_EUNSUPPORTED, "page_size=%d (supported: 16, 32, 64, 128)", d->page_size);
  if (d->num_pages <= 0 || d->max_pages <= 0)
    return fail(nullptr, HFA_EINVAL, "num_pages=%d, max_pages=%d", d->num_pages, d->max_pages);
  if ((long long)d->num_pages * d->num_kv_heads * d->page_size >= (1ll << 31))
    return fail(nullptr, HFA_EUNSUPPORTED, "a pool of 2^31 rows or more");
  if ((long long)d->max_pages * d->page_size >= (1 << 24))
    return fail(nullptr, HFA_EINVAL, "max_pages * page_size = %lld, not below 2^24",
                (long long)d->max_pages * d->page_size);
  if (d->flags & ~(HFA_F_V_UNIT_NORM | HFA_F_BLOCK_BIDIR))
    return fail(nullptr, HFA_EINVAL, "flags 0x%x", d->flags);
  if (d->window < 0) return fail(nullptr, HFA_EINVAL, "window=%d", d->window);
  if (d->window > 0 && (d->flags & HFA_F_BLOCK_BIDIR))
    return fail(nullptr, HFA_EINVAL, "HFA_F_BLOCK_BIDIR with a window");
  if (!(d->eps >= 0.f) || !(d->rope_theta > 0.f) || !isfinite(d->eps) || !isfinite(d->rope_theta))
    return fail(nullptr, HFA_EINVAL, "eps, rope_theta out of range");
  if (!(d->attn_scale > 0.f) || !(d->softcap >= 0.f) || !isfinite(d->attn_scale) ||
      !isfinite(d->softcap))
    return fail(nullptr, HFA_EINVAL, "attn_scale, softcap out of range");
  return HFA_OK;
}

// the current device is the handle's
hfa_status check_device(hfa_paged* p) {
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(p, HFA_EDEVICE, "no CUDA device: %s", cudaGetErrorString(e));
  if (dev != p->device)
    return fail(p, HFA_EDEVICE, "the current device is %d, the cache's %d", dev, p->device);
  return HFA_OK;
}

hfa_status check_pages(hfa_paged* p, const hfa_pages* pg) {
  if (!pg) return fail(p, HFA_EINVAL, "pages is NULL");
  if (!pg->k_codes || !pg->k_scales || !pg->v_codes || !pg->v_scales || !pg->table_dev)
    return fail(p, HFA_EINVAL, "a pool pointer or the table is NULL");
  if (!aligned16(pg->k_codes) || !aligned16(pg->v_codes))
    return fail(p, HFA_EINVAL, "the codes must be 16-byte aligned");
  return HFA_OK;
}

// cu: 0 = cu[0] <= cu[1] ...; *total = cu[batch], *longest = the most rows of a sequence
hfa_status check_cu(hfa_paged* p, int batch, const int32_t* cu, int* total, int* longest) {
  if (cu[0] != 0) return fail(p, HFA_EINVAL, "cu[0]=%d, not 0", cu[0]);
  int most = 0;
  for (int b = 0; b < batch; ++b) {
    const long long n = (long long)cu[b + 1] - cu[b];
    if (n < 0 || n > (1 << 24)) return fail(p, HFA_EINVAL, "cu[%d]=%d after cu[%d]=%d", b + 1, cu[b + 1], b, cu[b]);
    if (n > most) most = (int)n;
  }
  *total = cu[batch];
  *longest = most;
  return HFA_OK;
}

hfa::PagedView view(const hfa_paged* p, const hfa_pages* pg, int batch) {
  hfa::PagedView v{};
  v.k_codes = pg->k_codes;
  v.v_codes = pg->v_codes;
  v.k_scales = pg->k_scales;
  v.v_scales = pg->v_scales;
  v.table = pg->table_dev;
  v.num_pages = p->d.num_pages;
  v.max_pages = p->d.max_pages;
  v.ps = p->d.page_size;
  v.ps_log2 = p->ps_log2;
  v.nh = p->d.num_heads;
  v.nkv = p->d.num_kv_heads;
  v.hd = p->d.head_dim;
  v.batch = batch;
  v.err = p->err;
  return v;
}

// the pages a call writes: inside the pool, none twice
hfa_status check_written(hfa_paged* p, int batch, const int32_t* cu, const int32_t* start,
                         const int32_t* table) {
  static thread_local std::vector<uint64_t> seen;  // a bit per page, all clear between calls
  const int ps = p->d.page_size, np = p->d.num_pages;
  const size_t words = ((size_t)np + 63) / 64;
  try {
    if (seen.size() < words) seen.resize(words, 0);
  } catch (const std::bad_alloc&) {
    return fail(p, HFA_ENOMEM, "host memory for the page check");
  }
  hfa_status st = HFA_OK;
  int b = 0, bad_j = -1;
  for (; b < batch && st == HFA_OK; ++b) {
    const int n = cu[b + 1] - cu[b];
    if (n == 0) continue;
    const int32_t* row = table + (size_t)b * p->d.max_pages;
    for (int j = start[b] / ps; j <= (start[b] + n - 1) / ps; ++j) {
      const int pg = row[j];
      if (pg < 0 || pg >= np) {
        st = fail(p, HFA_EINVAL, "table[%d][%d]=%d outside the pool of %d pages", b, j, pg, np);
        bad_j = j;
        break;
      }
      const uint64_t bit = 1ull << (pg & 63);
      if (seen[pg >> 6] & bit) {
        st = fail(p, HFA_EINVAL, "page %d (table[%d][%d]) would be written twice", pg, b, j);
        bad_j = j;
        break;
      }
      seen[pg >> 6] |= bit;
    }
  }
  for (int c = 0; c < b; ++c) {  // clear what was set
    const int n = cu[c + 1] - cu[c];
    if (n == 0) continue;
    const int32_t* row = table + (size_t)c * p->d.max_pages;
    const int end = (c == b - 1 && st != HFA_OK) ? bad_j - 1 : (start[c] + n - 1) / ps;
    for (int j = start[c] / ps; j <= end; ++j) seen[row[j] >> 6] &= ~(1ull << (row[j] & 63));
  }
  return st;
}

// workspace: [tickets][records of the step kernel][records of the block kernel, when its (row
// tile, KV head) slots are few enough to be shared by several CTAs].  The tickets, which have to
// be zero when a call begins, lie at the same place for every batch and handle.
long long block_slots(const hfa_paged_desc& d, int batch, int total) {
  return (long long)total * (d.num_heads / d.num_kv_heads) / hfa::paged_block_rows(d.head_dim) + batch;
}
long long block_units(const hfa_paged_desc& d, int batch, int total) {
  return block_slots(d, batch, total) * d.num_kv_heads;
}
constexpr size_t kTicketBytes = (hfa::kPagedMaxParts * sizeof(int) + 255) / 256 * 256;
size_t record_bytes(int hd) {
  return (size_t)2 * hfa::kPagedMaxParts * hfa::kPagedStepRows * hfa::kPagedRecord(hd) * sizeof(float);
}

}  // namespace

extern "C" hfa_status hfa_paged_create(const hfa_paged_desc* desc, const float* w_q,
                                       const float* w_k, const float* factors, void* stream,
                                       hfa_paged** out) {
  if (!out) return fail(nullptr, HFA_EINVAL, "out is NULL");
  *out = nullptr;
  const hfa_status st = validate(desc);
  if (st != HFA_OK) return st;
  const int hd = desc->head_dim;
  if (factors)
    for (int i = 0; i < hd / 2; ++i)
      if (!(factors[i] > 0.f) || !isfinite(factors[i]))
        return fail(nullptr, HFA_EINVAL, "factors[%d] must be finite and > 0", i);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(nullptr, HFA_EDEVICE, "no CUDA device: %s", cudaGetErrorString(e));
  int major = 0, minor = 0, sms = 0;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (major != 10 || minor != 3 || sms <= 0)
    return fail(nullptr, HFA_EDEVICE, "the device is sm_%d%d; libhfa is built for sm_103a only", major, minor);
  hfa_paged* p = new (std::nothrow) hfa_paged();
  if (!p) return fail(nullptr, HFA_ENOMEM, "host memory");
  p->d = *desc;
  p->device = dev;
  p->num_sms = sms;
  while ((1 << p->ps_log2) < desc->page_size) ++p->ps_log2;
  // one allocation: 256 bytes of error word, the frequencies and the weights (256 floats each),
  // then the cosines and sines of positions 0 .. page_size - 1
  const int half = hd / 2;
  std::vector<float> host;
  try {
    host.resize(256 + (size_t)desc->page_size * hd);
  } catch (const std::bad_alloc&) {
    delete p;
    return fail(nullptr, HFA_ENOMEM, "host memory");
  }
  for (int i = 0; i < half; ++i) {
    double v = pow((double)desc->rope_theta, -2.0 * i / hd) / (2.0 * M_PI);
    if (factors) v /= (double)factors[i];
    host[2 * i] = (float)v;
    host[2 * i + 1] = (float)(v - (double)host[2 * i]);
    for (int s = 0; s < desc->page_size; ++s) {
      const double turns = s * v, part = 2.0 * M_PI * (turns - floor(turns));
      host[256 + ((size_t)s * half + i) * 2] = (float)cos(part);
      host[256 + ((size_t)s * half + i) * 2 + 1] = (float)sin(part);
    }
  }
  const size_t bytes = 256 + (3 * 256 + (size_t)desc->page_size * hd) * sizeof(float);
  e = cudaMalloc(&p->block, bytes);
  if (e != cudaSuccess) {
    delete p;
    return fail(nullptr, HFA_ENOMEM, "cudaMalloc: %s", cudaGetErrorString(e));
  }
  float* f = (float*)((char*)p->block + 256);
  p->err = (unsigned*)p->block;
  p->rope_g = (float2*)f;
  p->w_q = w_q ? f + 256 : nullptr;
  p->w_k = w_k ? f + 512 : nullptr;
  p->slot_turn = (float4*)(f + 768);
  cudaStream_t s = (cudaStream_t)stream;
  e = cudaMemsetAsync(p->block, 0, bytes, s);
  if (e == cudaSuccess) e = cudaMemcpyAsync(f, host.data(), hd * sizeof(float), cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(p->slot_turn, host.data() + 256, (size_t)desc->page_size * hd * sizeof(float),
                        cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess && w_q) e = cudaMemcpyAsync(p->w_q, w_q, hd * sizeof(float), cudaMemcpyDeviceToDevice, s);
  if (e == cudaSuccess && w_k) e = cudaMemcpyAsync(p->w_k, w_k, hd * sizeof(float), cudaMemcpyDeviceToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) {
    cudaFree(p->block);
    delete p;
    return fail(nullptr, HFA_ECUDA, "the handle's tables: %s", cudaGetErrorString(e));
  }
  *out = p;
  return HFA_OK;
}

extern "C" hfa_status hfa_paged_destroy(hfa_paged* p) {
  if (!p) return HFA_EINVAL;
  cudaDeviceSynchronize();
  cudaFree(p->block);
  delete p;
  return HFA_OK;
}

extern "C" const char* hfa_paged_last_error(const hfa_paged* p) { return p ? p->msg : g_paged_error; }

extern "C" hfa_status hfa_paged_check_status(hfa_paged* p, void* stream) {
  if (!p) return fail(nullptr, HFA_EINVAL, "the handle is NULL");
  const hfa_status st = check_device(p);
  if (st != HFA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  unsigned w = 0;
  cudaError_t e = cudaMemcpyAsync(&w, p->err, sizeof w, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && w) e = cudaMemsetAsync(p->err, 0, sizeof w, s);
  if (e != cudaSuccess) return fail(p, HFA_ECUDA, "reading the error word: %s", cudaGetErrorString(e));
  if (w & hfa::kErrWaitTimeout) return fail(p, HFA_EDEVICE, "a bounded wait gave up");
  if (w) return fail(p, HFA_EDEVICE, "a position or page outside its range was skipped");
  return HFA_OK;
}

extern "C" hfa_status hfa_paged_append(hfa_paged* p, void* stream, int batch, const int32_t* cu_dev,
                                       const int32_t* cu_host, const int32_t* start_dev,
                                       const int32_t* start_host, const void* q, long long q_stride,
                                       const void* k, long long k_stride, const void* v,
                                       long long v_stride, int dtype, const hfa_pages* pages,
                                       void* q_out) {
  if (!p) return fail(nullptr, HFA_EINVAL, "the handle is NULL");
  hfa_status st = check_pages(p, pages);
  if (st != HFA_OK) return st;
  if (batch < 1 || batch > 4096) return fail(p, HFA_EINVAL, "batch=%d", batch);
  if (!cu_dev || !cu_host || !start_dev || !start_host || !pages->table_host)
    return fail(p, HFA_EINVAL, "cu, start or the host table is NULL");
  if (dtype != HFA_BF16 && dtype != HFA_F32) return fail(p, HFA_EINVAL, "dtype=%d", dtype);
  int total = 0, longest = 0;
  st = check_cu(p, batch, cu_host, &total, &longest);
  if (st != HFA_OK) return st;
  const hfa_paged_desc& d = p->d;
  const int cap = d.max_pages * d.page_size;
  for (int b = 0; b < batch; ++b)
    if (start_host[b] < 0 || start_host[b] > cap - (cu_host[b + 1] - cu_host[b]))
      return fail(p, HFA_ERANGE, "sequence %d: positions from %d, %d of them, outside a table of %d tokens",
                  b, start_host[b], cu_host[b + 1] - cu_host[b], cap);
  if (total == 0) return HFA_OK;
  if (!k || !v || (q && !q_out)) return fail(p, HFA_EINVAL, "a row pointer is NULL");
  const int per16 = dtype == HFA_F32 ? 4 : 8;
  const long long qrow = (long long)d.num_heads * d.head_dim, kvrow = (long long)d.num_kv_heads * d.head_dim;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q ? q_out : nullptr) ||
      (q && q_stride % per16) || k_stride % per16 || v_stride % per16)
    return fail(p, HFA_EINVAL, "rows and strides must be multiples of 16 bytes");
  if ((q && q_stride < qrow) || k_stride < kvrow || v_stride < kvrow)
    return fail(p, HFA_EINVAL, "a row stride is shorter than the row");
  if (q && q == q_out && q_stride != qrow)
    return fail(p, HFA_EINVAL, "q_out may be q only when q is dense");
  st = check_written(p, batch, cu_host, start_host, pages->table_host);
  if (st != HFA_OK) return st;
  st = check_device(p);
  if (st != HFA_OK) return st;
  hfa::PagedAppendArgs a{};
  a.p = view(p, pages, batch);
  a.cu = cu_dev;
  a.start = start_dev;
  a.total = total;
  a.single = longest == 1;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = q_out;
  a.rope_g = p->rope_g;
  a.slot_turn = p->slot_turn;
  a.w_q = p->w_q;
  a.w_k = p->w_k;
  a.v_unit_norm = (d.flags & HFA_F_V_UNIT_NORM) != 0;
  a.eps = d.eps;
  const int items = a.single ? batch : total / d.page_size + 2 * batch;
  const cudaError_t e = hfa::launch_paged_append(a, dtype == HFA_F32, items, p->num_sms, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail(p, HFA_ECUDA, "append launch: %s", cudaGetErrorString(e));
  return HFA_OK;
}

extern "C" size_t hfa_paged_workspace_bytes(const hfa_paged* p, int batch, int total_rows) {
  if (!p || batch < 1 || batch > 4096 || total_rows < 0) return 0;
  const int G = p->d.num_heads / p->d.num_kv_heads;
  size_t blocks = 0;
  if ((long long)total_rows * G > hfa::kPagedStepRows &&
      block_units(p->d, batch, total_rows) * 2 <= hfa::kPagedMaxParts)
    blocks = (size_t)hfa::kPagedMaxParts * hfa::paged_block_rows(p->d.head_dim) *
             hfa::kPagedRecord(p->d.head_dim) * sizeof(float);
  return kTicketBytes + record_bytes(p->d.head_dim) + blocks;
}

extern "C" hfa_status hfa_paged_attention(hfa_paged* p, void* stream, int batch,
                                          const int32_t* cu_dev, const int32_t* cu_host,
                                          const int32_t* len_dev, const int32_t* len_host,
                                          const void* q, long long q_stride, int dtype,
                                          const hfa_pages* pages, void* ws, size_t ws_bytes,
                                          void* o) {
  if (!p) return fail(nullptr, HFA_EINVAL, "the handle is NULL");
  hfa_status st = check_pages(p, pages);
  if (st != HFA_OK) return st;
  if (batch < 1 || batch > 4096) return fail(p, HFA_EINVAL, "batch=%d", batch);
  if (!cu_dev || !cu_host || !len_dev || !len_host) return fail(p, HFA_EINVAL, "cu or len is NULL");
  if (dtype != HFA_BF16 && dtype != HFA_F32) return fail(p, HFA_EINVAL, "dtype=%d", dtype);
  int total = 0, longest = 0;
  st = check_cu(p, batch, cu_host, &total, &longest);
  if (st != HFA_OK) return st;
  const hfa_paged_desc& d = p->d;
  const int cap = d.max_pages * d.page_size;
  for (int b = 0; b < batch; ++b)
    if (len_host[b] < 0 || len_host[b] > cap)
      return fail(p, HFA_ERANGE, "len[%d]=%d outside a table of %d tokens", b, len_host[b], cap);
  if (dtype == HFA_F32 && longest * (d.num_heads / d.num_kv_heads) > 8)
    return fail(p, HFA_EUNSUPPORTED, "f32 queries: %d rows of a GQA group of %d (at most 8 together)",
                longest, d.num_heads / d.num_kv_heads);
  if (total == 0) return HFA_OK;
  if (!q || !o || !ws) return fail(p, HFA_EINVAL, "q, o or the workspace is NULL");
  if (!aligned16(q) || !aligned16(o) || !aligned16(ws) || q_stride % (dtype == HFA_F32 ? 4 : 8))
    return fail(p, HFA_EINVAL, "q, o, the workspace and the row stride must be multiples of 16 bytes");
  if (q_stride < (long long)d.num_heads * d.head_dim)
    return fail(p, HFA_EINVAL, "the row stride is shorter than the row");
  const size_t need = hfa_paged_workspace_bytes(p, batch, total);
  if (ws_bytes < need) return fail(p, HFA_EINVAL, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  st = check_device(p);
  if (st != HFA_OK) return st;
  hfa::PagedAttnArgs a{};
  a.p = view(p, pages, batch);
  a.cu = cu_dev;
  a.len = len_dev;
  a.total = total;
  a.q = q;
  a.q_stride = q_stride;
  a.o = o;
  a.f32 = dtype == HFA_F32;
  a.window = d.window;
  a.bidir = (d.flags & HFA_F_BLOCK_BIDIR) != 0;
  const float log2e = 1.4426950408889634f;
  a.qscale = d.softcap > 0.f ? d.attn_scale / d.softcap : d.attn_scale * log2e;
  a.cap_log2 = d.softcap * log2e;
  a.tickets = (int*)ws;
  a.records = (float*)((char*)ws + kTicketBytes);
  // the sequences of few rows, and the others
  const int G = d.num_heads / d.num_kv_heads;
  long long blocks = 0;
  int few = 0;
  long long items = 0, most_tiles = 0;  // of the block kernel
  const int rows_per = hfa::paged_block_rows(d.head_dim), keys_per = hfa::paged_block_keys(d.head_dim);
  for (int b = 0; b < batch; ++b) {
    const int n = cu_host[b + 1] - cu_host[b];
    if (n == 0) continue;
    if ((long long)n * G > hfa::kPagedStepRows) {
      items += ((long long)n * G + rows_per - 1) / rows_per * d.num_kv_heads;
      long long seen = len_host[b];
      if (d.window && seen > (long long)d.window + rows_per / G) seen = (long long)d.window + rows_per / G;
      if (seen / keys_per + 1 > most_tiles) most_tiles = seen / keys_per + 1;
      continue;
    }
    if (n * G > few) few = n * G;
    const int lo = d.window ? len_host[b] - n - d.window + 1 : 0;
    const int nb = (len_host[b] + 15) / 16 - (lo > 0 ? lo / 16 : 0);
    blocks += (long long)(nb < 1 ? 1 : nb) * d.num_kv_heads;
  }
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (few) {
    CUtensorMap tk, tv;
    const long long rows = (long long)d.num_pages * d.num_kv_heads * d.page_size;
    const int box = d.head_dim < 128 ? d.head_dim : 128;
    if (hfa_encode_u8_map(&tk, pages->k_codes, rows, d.head_dim, box, 16) != HFA_OK ||
        hfa_encode_u8_map(&tv, pages->v_codes, rows, d.head_dim, box, 16) != HFA_OK)
      return fail(p, HFA_EINVAL, "cannot describe the pool to the TMA unit");
    e = hfa::launch_paged_step(a, tk, tv, blocks, few, p->num_sms, s);
  }
  if (e == cudaSuccess && items) {
    const long long units = block_units(d, batch, total);
    if (units * hfa::kPagedMaxSplits >= (1ll << 31)) return fail(p, HFA_EUNSUPPORTED, "too many row tiles");
    a.block_records = (float*)((char*)a.records + record_bytes(d.head_dim));
    // with fewer items than SMs, as many CTAs an item as fill the SMs and have a key tile each
    long long splits = p->num_sms / items;
    if (splits > hfa::kPagedMaxSplits) splits = hfa::kPagedMaxSplits;
    if (splits > most_tiles) splits = most_tiles;
    if (splits > hfa::kPagedMaxParts / units) splits = hfa::kPagedMaxParts / units;
    if (splits < 1) splits = 1;
    e = hfa::launch_paged_block(a, (int)block_slots(d, batch, total), (int)splits, longest * G, s);
  }
  if (e != cudaSuccess) return fail(p, HFA_ECUDA, "attention launch: %s", cudaGetErrorString(e));
  return HFA_OK;
}

extern "C" hfa_status hfa_paged_read(hfa_paged* p, void* stream, int batch, const int32_t* start_dev,
                                     const int32_t* start_host, const int32_t* count_dev,
                                     const int32_t* count_host, const hfa_pages* pages, int capacity,
                                     void* k_cache, void* v_cache) {
  if (!p) return fail(nullptr, HFA_EINVAL, "the handle is NULL");
  hfa_status st = check_pages(p, pages);
  if (st != HFA_OK) return st;
  if (batch < 1 || batch > 4096) return fail(p, HFA_EINVAL, "batch=%d", batch);
  if (!start_dev || !start_host || !count_dev || !count_host || !k_cache || !v_cache)
    return fail(p, HFA_EINVAL, "a pointer argument is NULL");
  if (!aligned16(k_cache) || !aligned16(v_cache))
    return fail(p, HFA_EINVAL, "the caches must be 16-byte aligned");
  if (capacity < 1) return fail(p, HFA_EINVAL, "capacity=%d", capacity);
  const hfa_paged_desc& d = p->d;
  const int cap = d.max_pages * d.page_size;
  const int most = cap < capacity ? cap : capacity;
  int longest = 0;
  for (int b = 0; b < batch; ++b) {
    if (count_host[b] < 0 || start_host[b] < 0 || count_host[b] > most || start_host[b] > most - count_host[b])
      return fail(p, HFA_ERANGE, "sequence %d: positions from %d, %d of them, outside %d tokens", b,
                  start_host[b], count_host[b], most);
    if (count_host[b] > longest) longest = count_host[b];
  }
  if (longest == 0) return HFA_OK;
  st = check_device(p);
  if (st != HFA_OK) return st;
  hfa::PagedReadArgs a{};
  a.p = view(p, pages, batch);
  a.start = start_dev;
  a.count = count_dev;
  a.capacity = capacity;
  a.k_cache = (__nv_bfloat16*)k_cache;
  a.v_cache = (__nv_bfloat16*)v_cache;
  const cudaError_t e = hfa::launch_paged_read(a, longest, p->num_sms, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail(p, HFA_ECUDA, "read launch: %s", cudaGetErrorString(e));
  return HFA_OK;
}

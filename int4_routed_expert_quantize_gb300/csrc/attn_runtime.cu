// Host side of the paged-cache attention (coli_attn.h): argument checks, the workspace, the tensor maps
// of a bound cache and the launch sequences.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <new>

#include "attn_internal.h"

using namespace coli;

struct coli_attn {
  coli_attn_config cfg{};
  int device = 0, num_sms = 0, page_shift = 0, prefix_tokens = 0;
  char* arena = nullptr;  // the workspace: one allocation
  float* part_o = nullptr;
  float2* part_ml = nullptr;
  AttnRec* rec = nullptr;
  uint32_t* seq_pos = nullptr;
  // the tensor-memory kernel's (beside the split kernel's: one call may run both)
  float* part_o2 = nullptr;
  float2* part_ml2 = nullptr;
  AttnRec* rec2 = nullptr;
  float *dense_o = nullptr, *dense_o2 = nullptr;
  float2 *dense_ml = nullptr, *dense_ml2 = nullptr;
  uint8_t* redo = nullptr;
  int* redo_any = nullptr;
  uint64_t* turn = nullptr;
  int32_t* status = nullptr;
};

struct coli_attn_kv {
  coli_attn_cache c{};
  int n_kv = 0, head_dim = 0, page = 0, dtype = 0, device = 0;
  int code = 0;  // COLI_ATTN_CODE_*: an 8-bit cache (and dtype is the handle's); 0: of the handle's type
  float *k_scale = nullptr, *v_scale = nullptr;
  int64_t ks_page = 0, ks_head = 0, vs_page = 0, vs_head = 0;
  AttnKvMaps maps;
};

namespace {

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                CUtensorMapFloatOOBfill);

// the driver's tensor-map encoder, looked up through the runtime (no link against libcuda)
EncodeTiled encoder() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// cache memory as [page][head][slot][value], boxes of 64 values (8-bit codes: of a whole head) x `slots` slots
bool cache_map(CUtensorMap* map, const void* base, const coli_attn_kv& kv, int64_t ps, int64_t hs,
               int64_t ss, int slots) {
  EncodeTiled fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)kv.head_dim, (cuuint64_t)kv.page, (cuuint64_t)kv.n_kv,
                              (cuuint64_t)kv.c.n_pages};
  const cuuint64_t size = kv.code ? 1 : 2;
  const cuuint64_t strides[3] = {(cuuint64_t)ss * size, (cuuint64_t)hs * size, (cuuint64_t)ps * size};
  const cuuint32_t box[4] = {kv.code ? (cuuint32_t)kv.head_dim : 64, (cuuint32_t)(kv.page < slots ? kv.page : slots), 1, 1};
  const cuuint32_t unit[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type = kv.code                       ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : kv.dtype == COLI_ATTN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return fn(map, type, 4, const_cast<void*>(base), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box[0] * size == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// carves `count` elements off the arena at byte `at`, 256-byte aligned
template <class T>
void carve(T** p, char* arena, size_t* at, size_t count) {
  *p = reinterpret_cast<T*>(arena + *at);
  *at += (count * sizeof(T) + 255) / 256 * 256;
}

// the workspace in the arena (nullptr: its size alone); what has to be zero comes first, *zero bytes of it
size_t lay_out(coli_attn* h, char* arena, size_t* zero) {
  const coli_attn_config& c = h->cfg;
  // partials: two per CTA of the split kernels (2 CTAs an SM) and of the tensor-memory kernels
  const size_t D = c.head_dim, ctas = split_grid(h->num_sms), rows = 2 * ctas * kSplitMaxRows,
               rows2 = 2 * (size_t)h->num_sms * kTileRows;
  // the prefix call keeps every row twice
  const size_t dense = (size_t)h->prefix_tokens * c.n_q;
  size_t at = 0;
  carve(&h->status, arena, &at, 4);
  carve(&h->redo_any, arena, &at, 2);
  carve(&h->redo, arena, &at, (size_t)c.max_tokens * c.n_kv);
  *zero = at;
  carve(&h->turn, arena, &at, kAttnMaxPairs);
  carve(&h->rec, arena, &at, ctas);
  carve(&h->rec2, arena, &at, (size_t)h->num_sms);
  carve(&h->seq_pos, arena, &at, (size_t)c.max_seqs + 3);
  carve(&h->part_ml, arena, &at, rows);
  carve(&h->part_ml2, arena, &at, rows2);
  carve(&h->dense_ml, arena, &at, dense);
  carve(&h->dense_ml2, arena, &at, dense);
  carve(&h->part_o, arena, &at, rows * D);
  carve(&h->part_o2, arena, &at, rows2 * D);
  carve(&h->dense_o, arena, &at, dense * D);
  carve(&h->dense_o2, arena, &at, dense * D);
  return at;
}

constexpr int kMaxDevices = 64;
bool g_configured[kMaxDevices] = {};
std::mutex g_mutex;

// shared-memory attributes, once per device
cudaError_t configure_device(int dev) {
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (g_configured[dev]) return cudaSuccess;
  cudaError_t e = configure_attn_split();
  if (e == cudaSuccess) e = configure_attn_tile();
  if (e == cudaSuccess) e = configure_attn_qsplit();
  if (e == cudaSuccess) e = configure_attn_qtile();
  if (e == cudaSuccess) g_configured[dev] = true;
  return e;
}

bool misaligned(const void* p, int64_t stride) { return ((uintptr_t)p & 15u) || (stride & 7); }

// Whether heads' tokens of `width` elements share memory: dimensions of `extent` entries every `stride`, in any order.
// Each has to step over all that the smaller strides cover.
bool overlap(const int64_t (&stride)[3], const int64_t (&extent)[3], int64_t width) {
  int by[3] = {0, 1, 2};
  std::sort(by, by + 3, [&](int a, int b) { return stride[a] < stride[b]; });
  __int128 span = width;
  for (int i : by) {
    if (extent[i] < 2) continue;  // never stepped
    if (stride[i] < span) return true;
    span += (__int128)(extent[i] - 1) * stride[i];
  }
  return false;
}

int check_device(int device) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return COLI_ECUDA;
  return dev == device ? COLI_OK : COLI_ESTATE;
}

int check_call(const coli_attn* h, const coli_attn_kv* kv, const coli_attn_batch* b) {
  if (!h || !kv || !b) return COLI_EINVAL;
  const coli_attn_config& c = h->cfg;
  if (kv->n_kv != c.n_kv || kv->head_dim != c.head_dim || kv->page != c.page || kv->dtype != c.dtype ||
      kv->device != h->device)
    return COLI_EINVAL;
  if (b->n_tokens < 0 || b->n_tokens > c.max_tokens || b->n_seqs < 0 || b->n_seqs > c.max_seqs) return COLI_EINVAL;
  if (b->n_tokens == 0) return COLI_OK;
  if (b->n_seqs == 0 || !b->q_start || !b->kv_len || b->max_pages < 0 ||
      (b->table_stride < b->max_pages && b->table_stride != 0) || b->max_q < 1 || (b->max_pages > 0 && !b->table) ||
      ((int64_t)b->max_pages << h->page_shift) > kAttnNoWindow)
    return COLI_EINVAL;
  return check_device(h->device);
}

constexpr float kLog2E = 1.44269504088896340736f;

AttnParams params(const coli_attn* h, const coli_attn_kv* kv, const coli_attn_batch* b, const void* q,
                  int64_t q_stride, void* out, int64_t out_stride, float* lse, float scale) {
  AttnParams p = {};
  p.q = q, p.q_stride = q_stride, p.out = out, p.out_stride = out_stride, p.lse = lse;
  p.out_sectors = (((uintptr_t)out | (uintptr_t)out_stride * 2) & 31u) == 0;
  p.q_start = b->q_start, p.kv_len = b->kv_len, p.table = b->table, p.table_stride = b->table_stride;
  p.n_seqs = b->n_seqs, p.n_tokens = b->n_tokens, p.max_pages = b->max_pages, p.max_q = b->max_q;
  p.n_q = h->cfg.n_q, p.n_kv = h->cfg.n_kv, p.group = h->cfg.n_q / h->cfg.n_kv, p.head_dim = h->cfg.head_dim;
  p.page_shift = h->page_shift, p.n_pages = (int)kv->c.n_pages;
  p.window = kAttnNoWindow, p.sinks = 0;
  p.scale_log2 = scale * kLog2E;
  p.part_o = h->part_o, p.part_ml = h->part_ml, p.rec = h->rec, p.seq_pos = h->seq_pos;
  p.k_page = kv->c.k_page_stride, p.k_head = kv->c.k_head_stride, p.k_slot = kv->c.k_slot_stride;
  p.v_page = kv->c.v_page_stride, p.v_head = kv->c.v_head_stride, p.v_slot = kv->c.v_slot_stride;
  p.kc = kv->c.k, p.vc = kv->c.v;
  p.k_scale = kv->k_scale, p.v_scale = kv->v_scale;
  p.ks_page = kv->ks_page, p.ks_head = kv->ks_head, p.vs_page = kv->vs_page, p.vs_head = kv->vs_head;
  p.redo = h->redo, p.redo_any = h->redo_any, p.unit_cost = kSplitUnitCost;
  p.status = h->status;
  return p;
}

// queries as [token][head][value], boxes of 64 values x the heads of a key head x half a block's tokens
bool query_map(CUtensorMap* map, const coli_attn* h, const void* q, int64_t q_stride, int n_tokens) {
  EncodeTiled fn = encoder();
  if (!fn) return false;
  const int G = h->cfg.n_q / h->cfg.n_kv;
  const cuuint64_t dims[3] = {(cuuint64_t)h->cfg.head_dim, (cuuint64_t)h->cfg.n_q, (cuuint64_t)n_tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)h->cfg.head_dim * 2, (cuuint64_t)q_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(tile_block_tokens(G) / 2)};
  const cuuint32_t unit[3] = {1, 1, 1};
  return fn(map, h->cfg.dtype == COLI_ATTN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            3, const_cast<void*>(q), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// switches a launch's parameters to the tensor-memory kernel's workspace and blocks
void use_tile(const coli_attn* h, AttnParams* p) {
  p->part_o = h->part_o2, p->part_ml = h->part_ml2, p->rec = h->rec2;
  p->unit_cost = kTileUnitCost;
  p->block_tokens = tile_block_tokens(p->group);
}

// Whether rows of `wa` elements every `sa` from a and of `wb` every `sb` from b (n of either) share memory.  Rows of the
// same stride may lie between one another (slices of one wider row).
bool collide(const void* a, int64_t sa, int64_t wa, const void* b, int64_t sb, int64_t wb, int64_t n) {
  const int64_t x = (int64_t)((uintptr_t)a / 2), y = (int64_t)((uintptr_t)b / 2);
  if (x + (n - 1) * sa + wa <= y || y + (n - 1) * sb + wb <= x) return false;
  if (sa != sb) return true;
  const int64_t gap = (((y - x) % sa) + sa) % sa;  // b's row starts so far behind one of a's
  return gap < wa || gap + wb > sa;
}

int query_args(const coli_attn* h, int64_t n_tokens, const void* q, int64_t q_stride, const void* out,
               int64_t out_stride, float scale) {
  const int64_t width = (int64_t)h->cfg.n_q * h->cfg.head_dim;
  if (!q || !out || misaligned(q, q_stride) || misaligned(out, out_stride) || q_stride < width ||
      out_stride < width || !(scale > 0.f) || !std::isfinite(scale * kLog2E))
    return COLI_EINVAL;
  return collide(q, q_stride, width, out, out_stride, width, n_tokens) ? COLI_EINVAL : COLI_OK;
}

// Whether a prefix call of more than kSplitMaxRows rows a key head takes the sequences' own keys and the prefix in one launch
// of the tensor-memory kernel.  A unit of own keys costs that kernel about 2 us more than the split kernel, a second launch
// about 5 us, so: up to two such units an SM.  us, one launch / two, by sequences and tokens of prefix + own keys, 8 key
// heads: 16, 8000 + 40 22.3 / 28.0; 32, 2000 + 1000 39.8 / 41.4, 32000 + 40 51.2 / 56.0; 64, 2000 + 40 40.6 / 32.8,
// 32000 + 1000 101 / 94.  (The split kernel's blocks cannot hold one token of more than kSplitMaxRows heads a key head.)
bool one_prefix_launch(const coli_attn* h, int n_seqs) {
  return h->cfg.n_q / h->cfg.n_kv > kSplitMaxRows || (int64_t)n_seqs * h->cfg.n_kv <= 2 * h->num_sms;
}

// the work list's positions are 32-bit: its length is bounded by the page tables' widths (or the window)
int list_fits(const AttnParams& p, int keys) {
  const int64_t len = (int64_t)(p.pre_pages > p.max_pages ? p.pre_pages : p.max_pages) << p.page_shift;
  int64_t span = len;
  if (p.window < kAttnNoWindow && p.window + (int64_t)p.block_tokens + p.sinks + 2 * keys < len)
    span = p.window + (int64_t)p.block_tokens + p.sinks + 2 * keys;
  const int64_t blocks = p.n_tokens / p.block_tokens;  // whole ones: each sequence, and the prefix, may have one more
  const int64_t units = (blocks + p.n_seqs + (p.pre_len ? blocks + 1 : 0)) * p.n_kv;
  return units <= 0x7FFFFFFF / (span / keys + 2 + p.unit_cost) ? COLI_OK : COLI_EUNSUPPORTED;
}

// a cache's memory: codes of one byte in units of 16, values of the 16-bit types in units of 8
int check_cache(const coli_attn* h, const coli_attn_cache& c, int unit) {
  if (!c.k || !c.v || c.n_pages < 1 || c.n_pages > 0x7FFFFFFE) return COLI_EINVAL;
  const int64_t D = h->cfg.head_dim;
  const int64_t strides[6] = {c.k_page_stride, c.k_head_stride, c.k_slot_stride,
                              c.v_page_stride, c.v_head_stride, c.v_slot_stride};
  for (int64_t s : strides)
    if (s < D || (s & (unit - 1)) || s >= (1LL << 38)) return COLI_EINVAL;
  const int64_t extent[3] = {c.n_pages, h->cfg.n_kv, h->cfg.page};
  if (overlap({c.k_page_stride, c.k_head_stride, c.k_slot_stride}, extent, D) ||
      overlap({c.v_page_stride, c.v_head_stride, c.v_slot_stride}, extent, D))
    return COLI_EINVAL;
  if (((uintptr_t)c.k & 15u) || ((uintptr_t)c.v & 15u)) return COLI_EINVAL;
  return COLI_OK;
}

bool bad_scales(const coli_attn* h, const float* base, int64_t n_pages, int64_t page_stride, int64_t head_stride) {
  const int64_t width = h->cfg.page, extent[3] = {n_pages, h->cfg.n_kv, 1};
  for (int64_t s : {page_stride, head_stride})
    if (s < width || (s & 3) || s >= (1LL << 36)) return true;
  return !base || ((uintptr_t)base & 15u) || overlap({page_stride, head_stride, width}, extent, width);
}

int bind(const coli_attn* h, coli_attn_kv* kv, const coli_attn_cache& c) {
  kv->c = c;
  kv->n_kv = h->cfg.n_kv, kv->head_dim = h->cfg.head_dim, kv->page = h->cfg.page;
  kv->dtype = h->cfg.dtype, kv->device = h->device;
  return cache_map(&kv->maps.k64, c.k, *kv, c.k_page_stride, c.k_head_stride, c.k_slot_stride, kSplitKeys) &&
                 cache_map(&kv->maps.v64, c.v, *kv, c.v_page_stride, c.v_head_stride, c.v_slot_stride, kSplitKeys) &&
                 cache_map(&kv->maps.k128, c.k, *kv, c.k_page_stride, c.k_head_stride, c.k_slot_stride, kTileKeys) &&
                 cache_map(&kv->maps.v128, c.v, *kv, c.v_page_stride, c.v_head_stride, c.v_slot_stride, kTileKeys)
             ? COLI_OK
             : COLI_ECUDA;
}

}  // namespace

bool coli::rows_map(CUtensorMap* map, const void* x, int dtype, int cols, int tokens, int64_t stride, int box) {
  EncodeTiled fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)tokens}, strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t boxes[2] = {64, (cuuint32_t)box}, unit[2] = {1, 1};
  return fn(map, dtype == COLI_ATTN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
            const_cast<void*>(x), dims, strides, boxes, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

extern "C" int coli_attn_create(const coli_attn_config* cfg, coli_attn** out) {
  if (out) *out = nullptr;
  if (!cfg || !out) return COLI_EINVAL;
  const coli_attn_config& c = *cfg;
  if (c.n_kv < 1 || c.n_kv > 256 || c.n_q < 1 || c.n_q % c.n_kv || c.max_tokens < 1 || c.max_tokens > 4194304 ||
      c.max_seqs < 1 || c.max_seqs > kAttnMaxSeqs || c.rot_dim < 0 || c.page < 1 || c.head_dim < 1)
    return COLI_EINVAL;
  if (c.rot_interleaved != 0 && c.rot_interleaved != 1) return COLI_EINVAL;
  if (c.rot_dim > 0 && !c.inv_freq && !(c.rope_base > 0.0 && std::isfinite(c.rope_base))) return COLI_EINVAL;
  if ((c.head_dim != 64 && c.head_dim != 128) || (c.dtype != COLI_ATTN_BF16 && c.dtype != COLI_ATTN_FP16) ||
      c.n_q / c.n_kv > kAttnMaxGroup || c.rot_dim > c.head_dim || c.rot_dim % 16)
    return COLI_EUNSUPPORTED;
  if (c.page < 16 || c.page > 256 || (c.page & (c.page - 1))) return COLI_EUNSUPPORTED;
  int shift = 4;
  while ((1 << shift) < c.page) ++shift;
  uint64_t turn[kAttnMaxPairs] = {};
  for (int i = 0; i < c.rot_dim / 2; ++i) {
    const long double f = c.inv_freq ? (long double)c.inv_freq[i]
                                     : powl((long double)c.rope_base, -2.0L * i / c.rot_dim);
    if (!std::isfinite((double)f)) return COLI_EINVAL;
    long double t = f / 6.283185307179586476925286766559005768L;
    t -= floorl(t);  // whole turns do not count
    long double v = floorl(t * 18446744073709551616.0L + 0.5L);
    turn[i] = v >= 18446744073709551616.0L ? 0 : (uint64_t)v;
  }

  coli_attn* h = new (std::nothrow) coli_attn();
  if (!h) return COLI_ENOMEM;
  h->cfg = c;
  h->cfg.inv_freq = nullptr;  // read above; not kept
  h->page_shift = shift;
  int rc = COLI_OK;
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
      configure_device(h->device) != cudaSuccess)
    rc = COLI_ECUDA;
  if (!rc) {
    const int64_t pt = (int64_t)kAttnPrefixRows * c.max_seqs;
    h->prefix_tokens = (int)(pt < c.max_tokens ? pt : c.max_tokens);
    size_t zero;
    void* p = nullptr;
    if (cudaMalloc(&p, lay_out(h, nullptr, &zero)) != cudaSuccess) {
      rc = COLI_ENOMEM;
    } else {
      h->arena = static_cast<char*>(p);
      lay_out(h, h->arena, &zero);
      if (cudaMemset(h->arena, 0, zero) != cudaSuccess ||
          cudaMemcpy(h->turn, turn, sizeof(turn), cudaMemcpyHostToDevice) != cudaSuccess ||
          cudaStreamSynchronize(cudaStreamLegacy) != cudaSuccess)
        rc = COLI_ECUDA;
    }
  }
  if (rc) {
    cudaGetLastError();
    if (h->arena) cudaFree(h->arena);
    delete h;
    return rc;
  }
  *out = h;
  return COLI_OK;
}

extern "C" void coli_attn_destroy(coli_attn* h) {
  if (!h) return;
  cudaDeviceSynchronize();
  cudaFree(h->arena);
  delete h;
}

extern "C" int coli_attn_cache_bind(coli_attn* h, const coli_attn_cache* cache, coli_attn_kv** out) {
  if (out) *out = nullptr;
  if (!h || !cache || !out) return COLI_EINVAL;
  int rc = check_cache(h, *cache, 8);
  if (!rc) rc = check_device(h->device);
  if (rc) return rc;
  coli_attn_kv* kv = new (std::nothrow) coli_attn_kv();
  if (!kv) return COLI_ENOMEM;
  rc = bind(h, kv, *cache);
  if (rc) {
    delete kv;
    return rc;
  }
  *out = kv;
  return COLI_OK;
}

extern "C" int coli_attn_qcache_bind(coli_attn* h, const coli_attn_qcache* cache, coli_attn_kv** out) {
  if (out) *out = nullptr;
  if (!h || !cache || !out) return COLI_EINVAL;
  const coli_attn_qcache& q = *cache;
  if (q.type != COLI_ATTN_CODE_INT8 && q.type != COLI_ATTN_CODE_E4M3) return COLI_EINVAL;
  int rc = check_cache(h, q.codes, 16);
  if (!rc && (bad_scales(h, q.k_scale, q.codes.n_pages, q.k_scale_page_stride, q.k_scale_head_stride) ||
              bad_scales(h, q.v_scale, q.codes.n_pages, q.v_scale_page_stride, q.v_scale_head_stride)))
    rc = COLI_EINVAL;
  if (!rc) rc = check_device(h->device);
  if (rc) return rc;
  coli_attn_kv* kv = new (std::nothrow) coli_attn_kv();
  if (!kv) return COLI_ENOMEM;
  kv->code = q.type;
  kv->k_scale = q.k_scale, kv->v_scale = q.v_scale;
  kv->ks_page = q.k_scale_page_stride, kv->ks_head = q.k_scale_head_stride;
  kv->vs_page = q.v_scale_page_stride, kv->vs_head = q.v_scale_head_stride;
  rc = bind(h, kv, q.codes);
  if (rc) {
    delete kv;
    return rc;
  }
  *out = kv;
  return COLI_OK;
}

extern "C" void coli_attn_cache_release(coli_attn_kv* kv) { delete kv; }

extern "C" int coli_attn_append(coli_attn* h, const coli_attn_kv* kv, const coli_attn_batch* b,
                                const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                const void* v, int64_t v_stride, void* q_out, int64_t q_out_stride,
                                const int32_t* pos_base, void* stream) {
  const int rc = check_call(h, kv, b);
  if (rc) return rc;
  if (b->n_tokens == 0) return COLI_OK;
  const int64_t kvw = (int64_t)h->cfg.n_kv * h->cfg.head_dim, qw = (int64_t)h->cfg.n_q * h->cfg.head_dim;
  if (!k || !v || misaligned(k, k_stride) || misaligned(v, v_stride) || k_stride < kvw || v_stride < kvw)
    return COLI_EINVAL;
  if ((q == nullptr) != (q_out == nullptr)) return COLI_EINVAL;
  if (q && (misaligned(q, q_stride) || misaligned(q_out, q_out_stride) || q_stride < qw || q_out_stride < qw ||
            ((q != q_out || q_stride != q_out_stride) && collide(q, q_stride, qw, q_out, q_out_stride, qw, b->n_tokens)) ||
            collide(k, k_stride, kvw, q_out, q_out_stride, qw, b->n_tokens) ||
            collide(v, v_stride, kvw, q_out, q_out_stride, qw, b->n_tokens)))
    return COLI_EINVAL;
  AttnAppend a = {};
  a.q = q, a.k = k, a.v = v, a.q_out = q_out, a.kc = kv->c.k, a.vc = kv->c.v;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride, a.q_out_stride = q_out_stride;
  a.kp = kv->c.k_page_stride, a.kh = kv->c.k_head_stride, a.ks = kv->c.k_slot_stride;
  a.vp = kv->c.v_page_stride, a.vh = kv->c.v_head_stride, a.vs = kv->c.v_slot_stride;
  a.q_start = b->q_start, a.kv_len = b->kv_len, a.table = b->table, a.table_stride = b->table_stride;
  a.n_seqs = b->n_seqs, a.n_tokens = b->n_tokens, a.max_pages = b->max_pages;
  a.n_pages = (int)kv->c.n_pages, a.page_shift = h->page_shift;
  a.n_q = h->cfg.n_q, a.n_kv = h->cfg.n_kv, a.head_dim = h->cfg.head_dim;
  a.rot = h->cfg.rot_dim, a.interleaved = h->cfg.rot_interleaved;
  a.pos_base = pos_base, a.turn = h->turn, a.status = h->status;
  a.code = kv->code, a.k_scale = kv->k_scale, a.v_scale = kv->v_scale;
  a.ksp = kv->ks_page, a.ksh = kv->ks_head, a.vsp = kv->vs_page, a.vsh = kv->vs_head;
  return launch_attn_append(a, h->cfg.dtype, h->num_sms, (cudaStream_t)stream) == cudaSuccess ? COLI_OK
                                                                                               : COLI_ECUDA;
}

extern "C" int coli_attn_window(coli_attn* h, const coli_attn_kv* kv, const coli_attn_batch* b, const void* q,
                                int64_t q_stride, int window, int sinks, float scale, void* out,
                                int64_t out_stride, float* lse, void* stream) {
  int rc = check_call(h, kv, b);
  if (rc) return rc;
  if (sinks < 0) return COLI_EINVAL;
  if (b->n_tokens == 0) return COLI_OK;
  rc = query_args(h, b->n_tokens, q, q_stride, out, out_stride, scale);
  if (rc) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  AttnParams p = params(h, kv, b, q, q_stride, out, out_stride, lse, scale);
  if (window >= 0 && window < kAttnNoWindow) p.window = window, p.sinks = sinks;
  // One kernel takes the whole batch: the split kernel where no sequence has more than kSplitMaxRows rows a key head, else
  // the tensor-memory kernel, its single tokens too.  us, split / tensor memory, 8 key heads of 128, every sequence of so many
  // rows: 30 rows, one sequence of 8000 tokens 17.2 / 20.0, 8 of them 37.9 / 37.3, 32 of 1000 26.5 / 29.3; 60 rows
  // 26.8 / 20.6, 52.4 / 38.4, 40.0 / 30.1 (split kernel in blocks of 64 rows).  A launch of either kernel for the sequences that
  // suit it: 8 of up to 96 rows 26.5 / one launch 16.7, 40 mixed ones of 4000 tokens 146 / 125.
  const int64_t seq_rows = (int64_t)b->max_q * p.group;
  cudaError_t e;
  if (seq_rows <= kSplitMaxRows) {
    const int rows = split_rows(seq_rows), ctas = split_grid(h->num_sms);
    p.block_tokens = rows / p.group;
    rc = list_fits(p, kSplitKeys);
    if (rc) return rc;
    e = kv->code ? launch_attn_qsplit(p, kv->maps.k64, kv->maps.v64, rows, h->cfg.dtype, kv->code, h->num_sms, st)
                 : launch_attn_split(p, kv->maps.k64, kv->maps.v64, rows, h->cfg.dtype, h->num_sms, st);
    if (e == cudaSuccess) e = launch_attn_combine(p, rows, (int)seq_rows, ctas, h->cfg.dtype, st);
  } else {
    use_tile(h, &p);
    CUtensorMap qm;
    rc = list_fits(p, kTileKeys);
    if (rc) return rc;
    if (!query_map(&qm, h, q, q_stride, b->n_tokens)) return COLI_ECUDA;
    e = kv->code ? launch_attn_qtile(p, qm, kv->maps.k128, kv->maps.v128, h->cfg.dtype, kv->code, h->num_sms, st)
                 : launch_attn_tile(p, qm, kv->maps.k128, kv->maps.v128, h->cfg.dtype, h->num_sms, st);
    if (e == cudaSuccess) e = launch_attn_combine(p, kTileRows, (int)(seq_rows < kTileRows ? seq_rows : kTileRows), h->num_sms, h->cfg.dtype, st);
  }
  return e == cudaSuccess ? COLI_OK : COLI_ECUDA;
}

extern "C" int coli_attn_prefix(coli_attn* h, const coli_attn_kv* kv, const coli_attn_batch* b,
                                const int32_t* prefix_table, int prefix_pages, const int32_t* prefix_len,
                                const void* q, int64_t q_stride, float scale, void* out, int64_t out_stride,
                                float* lse, void* stream) {
  int rc = check_call(h, kv, b);
  if (rc) return rc;
  if (kv->code) return COLI_EUNSUPPORTED;
  if (prefix_pages < 0 || (prefix_pages > 0 && !prefix_table) || !prefix_len ||
      ((int64_t)prefix_pages << h->page_shift) > kAttnNoWindow || b->n_tokens > h->prefix_tokens)
    return COLI_EINVAL;
  if (b->n_tokens == 0) return COLI_OK;
  rc = query_args(h, b->n_tokens, q, q_stride, out, out_stride, scale);
  if (rc) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  AttnParams own = params(h, kv, b, q, q_stride, out, out_stride, lse, scale);
  own.dense_o[0] = h->dense_o, own.dense_ml[0] = h->dense_ml;
  own.dense_o[1] = h->dense_o2, own.dense_ml[1] = h->dense_ml2;
  AttnParams pre = own;
  pre.pre_len = prefix_len, pre.pre_table = prefix_table, pre.pre_pages = prefix_pages;
  const int64_t all_rows = (int64_t)b->n_tokens * own.group;
  CUtensorMap qm;
  cudaError_t e;
  if (all_rows <= kSplitMaxRows) {  // one launch, the prefix as one more sequence of all tokens
    const int rows = split_rows(all_rows);
    pre.block_tokens = rows / own.group;
    rc = list_fits(pre, kSplitKeys);
    if (rc) return rc;
    e = launch_attn_split(pre, kv->maps.k64, kv->maps.v64, rows, h->cfg.dtype, h->num_sms, st);
    if (e == cudaSuccess) e = launch_attn_join(pre, rows, pre, true, 0, h->cfg.dtype, st);
  } else if (one_prefix_launch(h, b->n_seqs)) {  // as above
    use_tile(h, &pre);
    rc = list_fits(pre, kTileKeys);
    if (rc) return rc;
    if (!query_map(&qm, h, q, q_stride, b->n_tokens)) return COLI_ECUDA;
    e = launch_attn_tile(pre, qm, kv->maps.k128, kv->maps.v128, h->cfg.dtype, h->num_sms, st);
    if (e == cudaSuccess) e = launch_attn_join(pre, kTileRows, pre, true, 0, h->cfg.dtype, st);
  } else {
    const int rows = split_rows((int64_t)b->max_q * own.group);
    own.block_tokens = rows / own.group;
    use_tile(h, &pre);
    pre.n_seqs = 0;
    pre.seq_pos = nullptr;  // the split kernel's, at the same time
    pre.late_wait = 1;
    rc = list_fits(own, kSplitKeys);
    if (!rc) rc = list_fits(pre, kTileKeys);
    if (rc) return rc;
    if (!query_map(&qm, h, q, q_stride, b->n_tokens)) return COLI_ECUDA;
    e = launch_attn_split(own, kv->maps.k64, kv->maps.v64, rows, h->cfg.dtype, h->num_sms, st);
    if (e == cudaSuccess)
      e = launch_attn_tile(pre, qm, kv->maps.k128, kv->maps.v128, h->cfg.dtype, h->num_sms, st);
    if (e == cudaSuccess) e = launch_attn_join(own, rows, pre, false, h->num_sms, h->cfg.dtype, st);
  }
  return e == cudaSuccess ? COLI_OK : COLI_ECUDA;
}

extern "C" int coli_attn_status(coli_attn* h, void* stream) {
  if (!h) return COLI_EINVAL;
  const int rc = check_device(h->device);
  if (rc) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  int32_t v = 0;
  if (cudaMemcpyAsync(&v, h->status, sizeof(v), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaMemsetAsync(h->status, 0, sizeof(v), st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
    return COLI_ECUDA;
  return v;
}

extern "C" int coli_attn_launches(const coli_attn* h, int op, int n_seqs) {
  if (!h || op < 0 || op > 2 || n_seqs < 1) return COLI_EINVAL;
  return op == 0 ? 1 : op == 1 ? 2 : one_prefix_launch(h, n_seqs) ? 2 : 3;
}

// A KV cache in pages of the caller's device memory: address lookups shared by the speculative-decoding
// kernels, and the host checks their entry points have in common.
#pragma once

#include "hs_internal.cuh"

// positions of a request, and entries of a list, at most: the kernels count entries, rounded up to
// whole tiles, in 32 bits
constexpr int32_t kMaxPositions = INT32_MAX - 65535;

constexpr int kSmsHint = 152;  // to size grids by

// i / d by a multiplication with ceil(2^32 / d): exact while i * d < 2^32
struct Div {
  uint32_t d, m;
  __device__ __forceinline__ uint32_t operator()(uint32_t i) const { return d == 1u ? i : __umulhi(i, m); }
};
inline Div div_by(int d) { return Div{(uint32_t)(d > 0 ? d : 1), d > 1 ? (uint32_t)((0x100000000ull + d - 1) / d) : 0u}; }

struct PagedRows {
  uint8_t* base;         // [num_pages][page_tokens][rec]
  const int32_t* table;  // [R][max_pages] or null: the identity
  int64_t num_pages, rec;
  int32_t page_tokens, max_pages;
  uint32_t* err;         // or null
};

// Row number of position p of request r, or -1 with *err_bits raised: `outside` for a position the
// request's table does not reach, HS_DEVERR_PAGE for a table entry that is no page.
__device__ __forceinline__ int64_t paged_row(const PagedRows& c, int r, int64_t p, uint32_t outside,
                                             uint32_t* err_bits) {
  if (p < 0 || p >= (int64_t)c.max_pages * c.page_tokens) {
    *err_bits |= outside;
    return -1;
  }
  // a 32-bit division wherever the position allows it
  const int64_t pg = (p >> 31) == 0 ? (int64_t)((uint32_t)p / (uint32_t)c.page_tokens) : p / c.page_tokens;
  const int64_t page = c.table != nullptr ? (int64_t)c.table[(int64_t)r * c.max_pages + pg] : (int64_t)r * c.max_pages + pg;
  if (page < 0 || page >= c.num_pages) {
    *err_bits |= (uint32_t)HS_DEVERR_PAGE;
    return -1;
  }
  return page * c.page_tokens + (p - pg * c.page_tokens);
}

__device__ __forceinline__ void report(uint32_t* err, uint32_t bits) {
  if (bits != 0u && err != nullptr) atomicOr(err, bits);
}

// Makes `dev` current for a call and puts the caller's device back.
struct HsOnDevice {
  int prev = -1, dev;
  bool ok;
  explicit HsOnDevice(int d) : dev(d) {
    ok = cudaGetDevice(&prev) == cudaSuccess && (prev == d || cudaSetDevice(d) == cudaSuccess);
    if (!ok) cudaGetLastError();
  }
  ~HsOnDevice() {
    if (prev >= 0 && prev != dev) cudaSetDevice(prev);
  }
};

// the fields of hs_config that the paged calls read
inline int hs_check_shape(const hs_config* c) {
  if (c == nullptr) return HS_ERR_ARG;
  if (c->num_requests < 1 || c->num_requests > 65535) return HS_ERR_CONFIG;
  if (c->layout != HS_LAYOUT_MLA && c->layout != HS_LAYOUT_GQA) return HS_ERR_CONFIG;
  if (c->num_q_heads < 1 || c->num_kv_heads < 1 || c->num_q_heads % c->num_kv_heads != 0) return HS_ERR_CONFIG;
  if (c->num_q_heads > 1024) return HS_ERR_CONFIG;
  if (c->head_dim_qk < 8 || c->head_dim_qk > 576 || c->head_dim_qk % 8 != 0) return HS_ERR_CONFIG;
  if (c->head_dim_v < 8 || c->head_dim_v > 576 || c->head_dim_v % 8 != 0) return HS_ERR_CONFIG;
  if (c->layout == HS_LAYOUT_MLA && (c->num_kv_heads != 1 || c->head_dim_v > c->head_dim_qk)) return HS_ERR_CONFIG;
  return HS_OK;
}

inline int hs_check_paged(const hs_config* c, const hs_paged_kv* kv) {
  if (kv == nullptr || kv->d_pages == nullptr || !hs_aligned(kv->d_pages, 16)) return HS_ERR_ARG;
  if (!hs_aligned(kv->d_table, 4) || !hs_aligned(kv->d_err, 4)) return HS_ERR_ARG;
  if (kv->num_pages < 1 || kv->page_tokens < 1 || kv->max_pages < 1 || kv->cuda_device < 0) return HS_ERR_ARG;
  if (kv->num_pages > (int64_t)INT32_MAX / kv->page_tokens) return HS_ERR_ARG;
  if (kv->max_pages > kMaxPositions / kv->page_tokens) return HS_ERR_ARG;
  if (kv->d_table == nullptr && (int64_t)c->num_requests * kv->max_pages > kv->num_pages) return HS_ERR_ARG;
  return HS_OK;
}

inline PagedRows hs_paged_rows(const hs_config* c, const hs_paged_kv* kv) {
  PagedRows p;
  p.base = (uint8_t*)kv->d_pages;
  p.table = kv->d_table;
  p.num_pages = kv->num_pages;
  p.rec = hs_record_bytes(c);
  p.page_tokens = kv->page_tokens;
  p.max_pages = kv->max_pages;
  p.err = kv->d_err;
  return p;
}

// Wait for the stream's preceding kernel.  Unlike hs_pdl_enter this does not let the successor start
// early: a pool's attention that follows the resolve of its layer waits for that resolve alone, so a
// kernel enqueued between the two (rotating its queries, say) has to be complete before it starts.
__device__ __forceinline__ void hs_pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch with programmatic dependent launch: may start while the stream's preceding kernel drains.
template <typename K, typename... Args>
inline cudaError_t hs_launch_pdl(K kern, dim3 grid, dim3 block, size_t smem, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Eviction from a paged cache by accumulated attention weight.
//
// Of the n entries of a request, `keep` stay: its first f, its last c, and of the others the keep - f - c with the largest
// weights, the earlier of equal ones.  They keep their order and move to the front.  Two kernels: the choice, a CTA for
// each list of weights (a request's, or one of its KV heads'), and the moves, which device memory bounds: a record's
// share that moves is read once and written once.  16 requests from 8192 to 4096 entries, 8 KV heads of 128 each by itself: 63 us, the
// choice 16 and the moves 45, 6.4 TB/s; one request from 2049 to 2048: 9.7 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "hs_paged.cuh"

namespace {

struct EvictArgs {
  PagedRows kv;
  const int64_t* len;
  const float* w;
  float* w_out;
  int64_t* len_out;
  const int64_t* first_of;  // [R] or null: first
  int64_t cap;              // entries of a list of weights
  int R, lists, keep, first, recent;
  int page_shift;           // log2 of the tokens of a page, -1: no power of two
  int2* move;               // [R][lists][keep]: source and destination row of entry i, where they differ
  float* w_tmp;             // [R][lists][keep]
  int2* meta;               // [R][lists]: entries that stay, first of them that moves
};

// ---- the choice ----------------------------------------------------------------------------------
//
// The m-th largest weight by radix selection, 11 bits at a time until a bin stays whole, over keys that order as the weights do, less
// the smallest of them (weights crowd into a few exponents: without that most of a warp's counts meet in the same bins); then one ordered pass that
// gives every entry that stays its place.  A warp takes a contiguous run of entries in that pass, so two barriers are enough; the
// weights and the request's pages wait in shared memory where they fit.

constexpr int kPickThreads = 1024, kBins = 2048;
constexpr int kCached = 44 * 1024;  // weights kept in shared memory at most
constexpr int kPages = 4 * 1024;    // entries of the page table, likewise

// orders as the weights: NaN above everything, -0 as 0
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// paged_row of a position within the pages, whose first table entries are at hand
__device__ __forceinline__ int row_of(const PagedRows& c, int shift, const int32_t* first, int count, int r, int p, uint32_t* bad) {
  const int pg = shift >= 0 ? p >> shift : (int)((unsigned)p / (unsigned)c.page_tokens);
  int page;
  if (pg < count) page = first[pg];
  else page = c.table != nullptr ? c.table[(int64_t)r * c.max_pages + pg] : r * c.max_pages + pg;
  if ((unsigned)page >= (unsigned)c.num_pages) {
    *bad |= (uint32_t)HS_DEVERR_PAGE;
    return -1;
  }
  return page * c.page_tokens + (p - pg * c.page_tokens);  // below 2^31, as all rows are
}

__global__ void __launch_bounds__(kPickThreads) k_evict_pick(const EvictArgs a, int cached, int pages) {
  extern __shared__ float s_w[];  // weights, then the page table
  __shared__ int s_hist[kBins], s_warp[32], s_eq[32], s_bin, s_want, s_all, s_hole;
  __shared__ uint32_t s_min, s_max;
  hs_pdl_wait();
  // the only kernel that may start early is this call's own second one, which waits for this one
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int list = blockIdx.x, r = blockIdx.y;
  const int64_t n64 = a.len[r], f64 = a.first_of != nullptr ? a.first_of[r] : a.first;
  const int64_t at = (int64_t)r * a.lists + list;
  const float* w = a.w + at * a.cap;
  float* w_out = a.w_out + at * a.cap;
  const bool bad = n64 < 0 || n64 > a.cap || n64 > (int64_t)a.kv.max_pages * a.kv.page_tokens || f64 < 0 ||
                   f64 > (int64_t)a.keep - a.recent;
  if (bad || n64 <= a.keep) {  // stays as it is
    if (bad && tid == 0 && list == 0) report(a.kv.err, (uint32_t)HS_DEVERR_LOC);
    if (tid == 0) a.meta[at] = make_int2(bad ? -1 : (int)n64, bad ? -1 : (int)n64);
    if (!bad && w_out != w)
      for (int64_t i = tid; i < n64; i += kPickThreads) w_out[i] = w[i];
    return;
  }
  const int n = (int)n64, f = (int)f64, to = n - a.recent;  // the weights decide in [f, to)
  const bool in_smem = n <= cached;
  int32_t* s_pages = (int32_t*)(s_w + cached);
  if (tid == 0) {
    s_hole = n;
    s_min = 0xffffffffu;
    s_max = 0u;
  }
  __syncthreads();
  for (int i = tid; i < pages; i += kPickThreads) s_pages[i] = a.kv.table[(int64_t)r * a.kv.max_pages + i];
  uint32_t least = 0xffffffffu, most = 0u;
  for (int i = tid; i < n; i += kPickThreads) {
    const float x = w[i];
    if (in_smem) s_w[i] = x;
    if (i >= f && i < to) {
      least = min(least, key_of(x));
      most = max(most, key_of(x));
    }
  }
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) {
    atomicMin(&s_min, least);
    atomicMax(&s_max, most);
  }
  const float* src = in_smem ? s_w : w;
  uint32_t limit = 0xffffffffu;      // the key of the last one chosen
  int want = a.keep - f - a.recent;  // of those at it, how many stay
  if (want > 0) {
    __syncthreads();
    limit = s_min;  // the least key of those that are counted; `shift`: log2 of the keys of a bin
    uint32_t span = s_max - limit;
    int shift = max(0, 21 - __clz(span));
#pragma unroll 1
    for (;;) {
      s_hist[tid] = 0;
      s_hist[tid + kPickThreads] = 0;
      __syncthreads();
      for (int i = f + tid; i < to; i += kPickThreads) {
        const uint32_t k = key_of(src[i]) - limit;
        if (k <= span) atomicAdd(&s_hist[k >> shift], 1);
      }
      __syncthreads();
      // entries in the bins above a thread's two
      const int h0 = s_hist[2 * tid], h1 = s_hist[2 * tid + 1];
      int incl = h0 + h1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_down_sync(0xffffffffu, incl, o);
        if (lane + o < 32) incl += y;
      }
      if (lane == 0) s_warp[warp] = incl;
      __syncthreads();
      int above = __reduce_add_sync(0xffffffffu, lane > warp ? s_warp[lane] : 0);
      above += incl - h0 - h1;
      if (above < want && want <= above + h1) {
        s_bin = 2 * tid + 1;
        s_want = want - above;
        s_all = want == above + h1;
      } else if (above + h1 < want && want <= above + h1 + h0) {
        s_bin = 2 * tid;
        s_want = want - above - h1;
        s_all = want == above + h1 + h0;
      }
      __syncthreads();
      limit += (uint32_t)s_bin << shift;
      want = s_want;
      if (s_all != 0) want = n;  // all of the bin stay: those above its first key, and those at it
      if (shift == 0 || s_all != 0) break;
      span = (1u << shift) - 1u;
      shift = max(0, shift - 11);
    }
  }
  // places: those that stay for sure (more weight, or first or recent), and the first `want` of those at the limit
  const int run = ((n + 31) / 32 + 31) / 32 * 32, p0 = warp * run, p1 = min(n, p0 + run);
  int sure = 0, eq = 0, hole = n;
  uint32_t bits = 0u;
  __syncthreads();
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 1) {
      if (lane == 0) {
        s_warp[warp] = sure;
        s_eq[warp] = eq;
      }
      __syncthreads();
      sure = lane < warp ? s_warp[lane] : 0;
      eq = lane < warp ? s_eq[lane] : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        sure += __shfl_xor_sync(0xffffffffu, sure, o);
        eq += __shfl_xor_sync(0xffffffffu, eq, o);
      }
    }
    for (int base = p0; base < p1; base += 32) {
      const int p = base + lane;
      const bool on = p < p1, mid = on && p >= f && p < to;
      const float x = on ? src[p] : 0.f;
      const uint32_t k = mid ? key_of(x) : 0u;
      const bool is_sure = on && (!mid || k > limit), is_eq = mid && k == limit;
      const uint32_t bs = __ballot_sync(0xffffffffu, is_sure), be = __ballot_sync(0xffffffffu, is_eq);
      if (pass == 1 && on) {
        const uint32_t below = (1u << lane) - 1u;
        const int e = eq + __popc(be & below);
        const int rank = sure + __popc(bs & below) + min(e, want);
        if (is_sure || (is_eq && e < want)) {
          if (in_smem) w_out[rank] = x;
          else a.w_tmp[at * a.keep + rank] = x;
          if (rank != p) {
            const int from = row_of(a.kv, a.page_shift, s_pages, pages, r, p, &bits);
            a.move[at * a.keep + rank] = make_int2(from, row_of(a.kv, a.page_shift, s_pages, pages, r, rank, &bits));
          }
        } else {
          hole = min(hole, p);
        }
      }
      sure += __popc(bs);
      eq += __popc(be);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) hole = min(hole, __shfl_xor_sync(0xffffffffu, hole, o));
  if (lane == 0) atomicMin(&s_hole, hole);
  report(a.kv.err, bits);
  __syncthreads();
  if (!in_smem)
    for (int i = tid; i < a.keep; i += kPickThreads) w_out[i] = a.w_tmp[at * a.keep + i];
  for (int i = a.keep + tid; i < n; i += kPickThreads) w_out[i] = 0.f;
  if (tid == 0) a.meta[at] = make_int2(a.keep, s_hole);
}

// ---- the moves -----------------------------------------------------------------------------------
//
// Entry i comes from a place p_i > i, and p_i >= i + 1 ascends.  A CTA owns a slice of bytes of a request's records and moves it
// for all entries in order, a batch at a time.  A store goes to place i, whose old record is the source of an entry <= i,
// in this batch or an earlier one: so the stores of a batch wait for all threads' loads of it, and the loads of
// the next batch, whose sources lie behind all of these places, need not wait for the stores.

constexpr int kMoveThreads = 256, kFlight = 8;  // records of a thread in a batch

__global__ void __launch_bounds__(kMoveThreads) k_evict_move(const EvictArgs a, int slices, int slice) {
  hs_pdl_wait();
  const int r = blockIdx.y, s = blockIdx.x, tid = threadIdx.x;
  const int list = s / slices;
  const int64_t at = (int64_t)r * a.lists + list;
  const int2 meta = a.meta[at];
  if (s == 0 && tid == 0) a.len_out[r] = meta.x >= 0 ? meta.x : a.len[r];
  const int cols = slice >> 4, rows = kMoveThreads / cols;  // 16-byte columns; records at once
  const int64_t share = a.kv.rec / a.lists, in = (int64_t)(s - list * slices) * slice + 16 * (tid % cols);
  const bool on = in < share;
  const int64_t col = list * share + in;
  const int2* move = a.move + at * a.keep;
  const int step = rows * kFlight, mine = tid / cols;
  int2 m[kFlight];
  uint4 v[kFlight];
  auto look = [&](int i0) {
#pragma unroll
    for (int x = 0; x < kFlight; ++x) {
      const int i = i0 + x * rows + mine;
      m[x] = on && i < meta.x ? move[i] : make_int2(-1, -1);
    }
  };
  if (meta.y >= meta.x) return;
  look(meta.y);
#pragma unroll 1
  for (int i0 = meta.y; i0 < meta.x; i0 += step) {
    int dst[kFlight];
#pragma unroll
    for (int x = 0; x < kFlight; ++x) {
      dst[x] = m[x].x >= 0 ? m[x].y : -1;
      if (dst[x] >= 0) v[x] = *(const uint4*)(a.kv.base + (int64_t)m[x].x * a.kv.rec + col);
    }
    look(i0 + step);
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kFlight; ++x)
      if (dst[x] >= 0) *(uint4*)(a.kv.base + (int64_t)dst[x] * a.kv.rec + col) = v[x];
  }
}

int64_t meta_bytes(const hs_config* c, int lists) { return ((int64_t)c->num_requests * lists * (int64_t)sizeof(int2) + 15) / 16 * 16; }

}  // namespace

extern "C" int64_t hs_evict_workspace(const hs_config* cfg, int lists, int keep) {
  const int rc = hs_check_shape(cfg);
  if (rc != HS_OK) return rc;
  if ((lists != 1 && lists != cfg->num_kv_heads) || keep < 1 || keep > kMaxPositions) return HS_ERR_ARG;
  return meta_bytes(cfg, lists) + (int64_t)cfg->num_requests * lists * keep * (int64_t)(sizeof(int2) + sizeof(float));
}

extern "C" int hs_evict(const hs_config* cfg, const hs_paged_kv* kv, const hs_evict_args* args, void* stream) {
  int rc = hs_check_shape(cfg);
  if (rc == HS_OK) rc = hs_check_paged(cfg, kv);
  if (rc != HS_OK) return rc;
  if (args == nullptr) return HS_ERR_ARG;
  const hs_evict_args& g = *args;
  if (g.d_len == nullptr || g.d_len_out == nullptr || g.d_weights == nullptr || g.d_weights_out == nullptr) return HS_ERR_ARG;
  if (!hs_aligned(g.d_len, 8) || !hs_aligned(g.d_len_out, 8) || !hs_aligned(g.d_weights, 4) || !hs_aligned(g.d_weights_out, 4) ||
      !hs_aligned(g.d_first, 8) || !hs_aligned(g.d_workspace, 16))
    return HS_ERR_ARG;
  if ((g.lists != 1 && g.lists != cfg->num_kv_heads) || g.capacity < 1 || g.capacity > kMaxPositions) return HS_ERR_ARG;
  if (g.keep < 1 || g.keep > kMaxPositions || g.recent < 0 || g.recent > g.keep) return HS_ERR_ARG;
  if (g.d_first == nullptr && (g.first < 0 || g.first > g.keep - g.recent)) return HS_ERR_ARG;
  if ((int64_t)cfg->num_requests * g.lists * g.capacity > INT64_MAX / 8) return HS_ERR_ARG;
  // in place, or apart
  const uintptr_t w = (uintptr_t)g.d_weights, o = (uintptr_t)g.d_weights_out,
                  bytes = (uintptr_t)cfg->num_requests * g.lists * g.capacity * sizeof(float);
  if (w != o && w < o + bytes && o < w + bytes) return HS_ERR_ARG;
  const uintptr_t l = (uintptr_t)g.d_len, lo = (uintptr_t)g.d_len_out, lb = (uintptr_t)cfg->num_requests * sizeof(int64_t);
  if (l != lo && l < lo + lb && lo < l + lb) return HS_ERR_ARG;
  if (g.d_workspace == nullptr || g.workspace_bytes < hs_evict_workspace(cfg, g.lists, g.keep)) return HS_ERR_SCRATCH;
  HsOnDevice on(kv->cuda_device);
  if (!on.ok) return HS_ERR_CUDA;
  EvictArgs a{};
  a.kv = hs_paged_rows(cfg, kv);
  a.len = g.d_len;
  a.w = g.d_weights;
  a.w_out = g.d_weights_out;
  a.len_out = g.d_len_out;
  a.first_of = g.d_first;
  a.cap = g.capacity;
  a.R = cfg->num_requests;
  a.lists = g.lists;
  a.keep = g.keep;
  a.first = g.first;
  a.recent = g.recent;
  a.page_shift = -1;
  for (int x = 0; x < 31; ++x)
    if (kv->page_tokens == 1 << x) a.page_shift = x;
  a.meta = (int2*)g.d_workspace;
  a.move = (int2*)((uint8_t*)g.d_workspace + meta_bytes(cfg, g.lists));
  a.w_tmp = (float*)(a.move + (int64_t)a.R * a.lists * a.keep);
  const int cached = (int)(g.capacity < kCached ? g.capacity : kCached);
  const int pages = kv->d_table == nullptr ? 0 : kv->max_pages < kPages ? kv->max_pages : kPages;
  static bool done[64];
  if (kv->cuda_device >= 64 || !done[kv->cuda_device]) {
    if (hs_raise_smem_limit(k_evict_pick, (kCached + kPages) * 4) != cudaSuccess) return HS_ERR_CUDA;
    if (kv->cuda_device < 64) done[kv->cuda_device] = true;
  }
  cudaError_t e = hs_launch_pdl(k_evict_pick, dim3(a.lists, a.R), dim3(kPickThreads), (cached + pages) * 4, (cudaStream_t)stream, a, cached, pages);
  if (e != cudaSuccess) return HS_ERR_CUDA;
  // as wide a slice as still gives every SM two CTAs
  const int64_t share = a.kv.rec / a.lists;
  int slice = 512;
  while (slice > 32 && (int64_t)a.R * a.lists * ((share + slice - 1) / slice) < 2 * kSmsHint) slice /= 2;
  const int slices = (int)((share + slice - 1) / slice);
  e = hs_launch_pdl(k_evict_move, dim3(slices * a.lists, a.R), dim3(kMoveThreads), 0, (cudaStream_t)stream, a, slices, slice);
  return e == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

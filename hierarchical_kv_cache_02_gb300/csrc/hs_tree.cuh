// Tree attention: arguments, record lookups and the division of the work, shared by its kernels.
#pragma once

#include <cuda_bf16.h>

#include <string.h>

#include "hs_paged.cuh"
#include "hs_tc.cuh"

namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct TreeArgs {
  PagedRows kv;             // paged form; err is the pool's error word in the pool's form
  const uint64_t* slot_pt;  // pool form: [R][slot_pages] device address of each buffer page, else null
  const int32_t* slot_cap;  // [R] slots a buffer holds
  int slot_pages, slot_shift;
  const uint8_t* draft;     // pool form: [R][T][rec]
  const uint16_t* q;        // [R][T][Hq][dqk]
  const int64_t* len;       // [R], paged form
  const int32_t* locs;      // [R][k] or null
  const uint64_t* mask;     // [R][T][words]
  const int32_t* nodes;     // [R] or null
  uint16_t* out;            // [R][T][Hq][dv]
  int R, T, k, words, Hq, Hkv, dqk, dv;
  int kstride, voff;        // values: KV head g's key at g * kstride, its value voff further on
  float qscale;             // scale * log2(e)
  int stall;                // test hook (hs_debug_stall_next): one arrival of a CTA's first tile is left out
};

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *(const uint32_t*)&v;
}

// context length (paged form); a negative one becomes one behind which no node has a position either
__device__ __forceinline__ int64_t context_of(const TreeArgs& a, int r, uint32_t* bad) {
  if (a.len == nullptr) return 0;
  const int64_t n = a.len[r];
  if (n < 0) *bad |= (uint32_t)HS_DEVERR_LOC;
  return n < 0 ? -(1ll << 40) : n;
}
// the nodes in use
__device__ __forceinline__ int nodes_of(const TreeArgs& a, int r, uint32_t* bad) {
  if (a.nodes == nullptr) return a.T;
  const int n = a.nodes[r];
  if (n < 0 || n > a.T) *bad |= (uint32_t)HS_DEVERR_LOC;
  return min(max(n, 0), a.T);
}
// entries of the context of request r: its positions or its list
__device__ __forceinline__ int64_t entries_of(const TreeArgs& a, int r, int64_t len, uint32_t* bad) {
  if (a.locs != nullptr) return a.k;
  const int64_t cap = (int64_t)a.kv.max_pages * a.kv.page_tokens;
  if (len > cap) *bad |= (uint32_t)HS_DEVERR_LOC;
  return max((int64_t)0, min(len, cap));
}

// record of context entry e, or null (padding, or bad with a bit raised)
__device__ __forceinline__ const uint8_t* entry_record(const TreeArgs& a, int r, int64_t e, uint32_t* bad) {
  int64_t p = e;
  if (a.locs != nullptr) {
    p = a.locs[(int64_t)r * a.k + e];
    if (p == -1) return nullptr;
  }
  if (a.slot_pt != nullptr) {
    if (p < 0 || p >= a.slot_cap[r]) {
      *bad |= (uint32_t)HS_DEVERR_LOC;
      return nullptr;
    }
    return hs_slot_addr(a.slot_pt + (int64_t)r * a.slot_pages, a.slot_shift, a.kv.rec, (int)p);
  }
  const int64_t row = paged_row(a.kv, r, p, (uint32_t)HS_DEVERR_LOC, bad);
  return row < 0 ? nullptr : a.kv.base + row * a.kv.rec;
}
__device__ __forceinline__ const uint8_t* node_record(const TreeArgs& a, int r, int64_t len, int j, uint32_t* bad) {
  if (a.draft != nullptr) return a.draft + ((int64_t)r * a.T + j) * a.kv.rec;
  const int64_t row = paged_row(a.kv, r, len + j, (uint32_t)HS_DEVERR_LOC, bad);
  return row < 0 ? nullptr : a.kv.base + row * a.kv.rec;
}

// ---- division of the work among the CTAs of the tensor-core kernels ---------------------------------
//
// A request's entries are its context, padded to a multiple of 4, then its nodes; they are cut into tiles
// of TT.  An item is the work of one accumulator over all tiles of a request (a KV head and one or two
// groups of nodes, or a slice of the value dims); the tiles of all items of all requests form one
// sequence, request by request and item by item, of which every worker takes an equal, contiguous
// share.  (Each item begins with `begin` units of no tile, which stand for what a portion costs beside its tiles:
// loading its queries, storing its result.)  Lengths live on the device alone, so each CTA finds its share
// itself.  A worker's portion of an item that does not hold all its tiles becomes a partial: slot 0 of the worker when the portion
// starts inside the item, else slot 1 (a worker has at most one of each); k_tree_combine joins them.

constexpr int kPortions = 10;  // portions a round of a CTA holds per worker
constexpr int kWindow = 16;    // requests a round looks at per worker

struct Portion {
  int r, t0, t1;        // tiles [t0, t1) of an item of request r
  int head, pair;       // the item: head * np + pair
  int n, len, nn;       // context entries, position of node 0 (negative: the nodes have none), nodes in use
};

struct PlanState {  // shared memory
  Portion port[2][kPortions];
  long long off[2], left[2];  // units into request cur, units still to take
  int cur[2], nport[2];
  int wn[2][kWindow], wlen[2][kWindow];
  short wnn[2][kWindow];
  long long scan[16];
};

struct WorkSplit {
  int items, np;         // per request; of them per KV head
  int begin;             // units of an item before its tiles
  int groups;            // workers of a CTA: worker w = group * gridDim.x + CTA; or
  int pairs;             // 1: two neighbouring CTAs are one worker
  long long* prefix;     // [R + 1] units (of one item) before each request, written by CTA 0
  float *part, *ml;      // [workers][2 slots][dims / 8][rows][8], [workers][2][rows][2]: maximum (base 2) and sum
  int rows;              // accumulator rows of a portion
};

template <int TT>
__device__ __forceinline__ long long tiles_of(int n, int nn) {
  return nn == 0 ? 0 : (((long long)n + 3) / 4 * 4 + nn + TT - 1) / TT;
}
__device__ __forceinline__ void request_of(const TreeArgs& a, int r, int* n, int* len, int* nn, uint32_t* bad) {
  const int64_t l = context_of(a, r, bad);
  *nn = nodes_of(a, r, bad);
  *n = (int)entries_of(a, r, l, bad);
  *len = l > INT32_MAX ? -1 - HS_MAX_TREE_NODES : (int)max(l, (int64_t)(-1 - HS_MAX_TREE_NODES));
}
// Shares of `total` tiles: the first total % workers workers take one more than the others.
struct Shares {
  long long per, more;  // more: workers with per + 1
  __device__ __forceinline__ Shares(long long total, int workers) {
    per = div_small(total, workers);
    more = total - per * workers;
  }
  __device__ __forceinline__ static long long div_small(long long x, long long y) {  // x >= 0, y > 0
    return ((unsigned long long)x | (unsigned long long)y) >> 32 == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
  }
  __device__ __forceinline__ long long start(int w) const { return w * per + min((long long)w, more); }
  __device__ __forceinline__ int worker(long long x) const {  // the one that holds tile x
    const long long big = more * (per + 1);
    return (int)(x < big ? div_small(x, per + 1) : more + div_small(x - big, per));
  }
};

template <int TT>
__device__ __forceinline__ long long units_of(const WorkSplit& ws, int n, int nn) {
  return nn == 0 ? 0 : tiles_of<TT>(n, nn) + ws.begin;
}

// Worker g's next portions, by one thread; window[i] is request first + i.
template <int TT>
__device__ __forceinline__ void plan_walk(const TreeArgs& a, const WorkSplit& ws, PlanState* s, int g, int first, int i,
                                          long long off, long long left) {
  int np = 0;
#pragma unroll 1
  while (left > 0 && np < kPortions && i < kWindow && first + i < a.R) {
    const int n = s->wn[g][i], nn = s->wnn[g][i];
    const long long U = units_of<TT>(ws, n, nn);
    if (off >= U * ws.items) {
      off -= U * ws.items;
      ++i;
      continue;
    }
    const int item = (int)Shares::div_small(off, U);
    const long long u0 = off - item * U, u1 = min(U, u0 + left);
    left -= u1 - u0;
    off += u1 - u0;
    if (u1 <= ws.begin) continue;  // nothing but the item's first units
    Portion p;
    p.r = first + i;
    p.head = item / ws.np;
    p.pair = item - p.head * ws.np;
    p.t0 = (int)max(0ll, u0 - ws.begin);
    p.t1 = (int)(u1 - ws.begin);
    p.n = n;
    p.len = s->wlen[g][i];
    p.nn = nn;
    s->port[g][np++] = p;
  }
  s->nport[g] = np;
  s->left[g] = first + i < a.R ? left : 0;  // lengths that change under the call must not keep it going
  s->off[g] = off;
  s->cur[g] = first + i;
}

// The next portions of each worker; false when no worker has any left.  Every thread calls it.
template <int TT>
__device__ __forceinline__ bool plan_round(const TreeArgs& a, const WorkSplit& ws, PlanState* s) {
  if (s->left[0] <= 0 && s->left[1] <= 0) return false;  // the same in every thread: written before a barrier
  const int tid = threadIdx.x;
  const bool all = a.R <= kWindow;  // then the window starts at request 0 and is there already
  if (!all && tid < 2 * kWindow) {
    const int g = tid / kWindow, i = tid - g * kWindow;
    if (s->left[g] > 0 && s->cur[g] + i < a.R) {
      uint32_t bad = 0u;
      int n, len, nn;
      request_of(a, s->cur[g] + i, &n, &len, &nn, &bad);
      s->wn[g][i] = n;
      s->wlen[g][i] = len;
      s->wnn[g][i] = (short)nn;
    }
  }
  __syncthreads();
  if (tid == 0 || tid == 32) {
    const int g = tid >> 5, cur = s->cur[g];
    if (s->left[g] > 0) plan_walk<TT>(a, ws, s, g, all ? 0 : cur, all ? cur : 0, s->off[g], s->left[g]);
    else s->nport[g] = 0;
  }
  __syncthreads();
  return true;
}

// Where each worker of this CTA starts, and its first portions; false when there is nothing to do.  Every
// thread of the CTA calls it.  (Here and in the kernels code size counts: a CTA fetches every instruction
// anew, and lives for some tens of microseconds.)
template <int TT>
__device__ __forceinline__ bool plan_start(const TreeArgs& a, const WorkSplit& ws, PlanState* s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x;
  if (a.R <= kWindow) {  // a lane a request: warp g finds worker g's place by itself
    if (warp < 2) {
      const int g = warp;
      uint32_t bad = 0u;
      int n = 0, len = 0, nn = 0;
      if (lane < a.R) {
        request_of(a, lane, &n, &len, &nn, &bad);
        s->wn[g][lane] = n;
        s->wlen[g][lane] = len;
        s->wnn[g][lane] = (short)nn;
      }
      const int U = (int)units_of<TT>(ws, n, nn);  // 16 requests of 2^31 entries: below 2^30
      int incl = U;
#pragma unroll
      for (int o = 1; o < kWindow; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const int total = __shfl_sync(0xffffffffu, incl, kWindow - 1);
      const Shares sh((long long)total * ws.items, (int)(gridDim.x >> ws.pairs) * ws.groups);
      const int w = g * (int)gridDim.x + (int)(blockIdx.x >> ws.pairs);
      const long long s0 = sh.start(w), left = g < ws.groups ? sh.start(w + 1) - s0 : 0;
      const long long off = s0 - (long long)(incl - U) * ws.items;
      const uint32_t here = __ballot_sync(0xffffffffu, off >= 0 && off < (long long)U * ws.items);
      if (g == 0 && blockIdx.x == 0) {
        if (lane < a.R) ws.prefix[lane] = incl - U;
        if (lane == 0) ws.prefix[a.R] = total;
        report(a.kv.err, bad);
      }
      const int r = here != 0u ? __ffs(here) - 1 : 0;
      const long long at = __shfl_sync(0xffffffffu, off, r);
      __syncwarp();
      if (lane == 0) plan_walk<TT>(a, ws, s, g, 0, r, at, left);
    }
    __syncthreads();
    return s->nport[0] + s->nport[1] > 0 || s->left[0] + s->left[1] > 0;
  }
  const int each = (a.R + nthr - 1) / nthr, r0 = min(tid * each, a.R), r1 = min(r0 + each, a.R);
  uint32_t bad = 0u;
  long long mine = 0, run = 0, s0[2] = {-1, -1};
  // the first pass counts each thread's units, the second finds the places among them
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    int n = 0, len = 0, nn = 0;
    long long U = mine;  // one request a thread: known from the first pass
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
      if (pass == 0 || each > 1) {
        request_of(a, r, &n, &len, &nn, &bad);
        U = units_of<TT>(ws, n, nn);
      }
      if (pass == 0) {
        mine += U;
      } else {
        if (blockIdx.x == 0) ws.prefix[r] = run;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const long long off = s0[g] - run * ws.items;
          if (s0[g] >= 0 && off >= 0 && off < U * ws.items) {
            s->cur[g] = r;
            s->off[g] = off;
          }
        }
        run += U;
      }
    }
    if (pass == 0) {
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) s->scan[warp] = incl;
      __syncthreads();
      long long total = 0;
      for (int w = 0; w < (nthr >> 5); ++w) {
        if (w == warp) run = total;
        total += s->scan[w];
      }
      run += incl - mine;
      const Shares sh(total * ws.items, (int)(gridDim.x >> ws.pairs) * ws.groups);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int w = g * (int)gridDim.x + (int)(blockIdx.x >> ws.pairs);
        const long long x = sh.start(w), left = g < ws.groups ? sh.start(w + 1) - x : 0;
        if (left > 0) s0[g] = x;
        if (tid == 0) s->left[g] = left;
      }
      if (blockIdx.x == 0 && tid == 0) ws.prefix[a.R] = total;
    }
  }
  if (blockIdx.x == 0) report(a.kv.err, bad);
  __syncthreads();
  return plan_round<TT>(a, ws, s);
}

// A producer lane's lookups of its entry of each tile of a portion list, in three steps, each a tile ahead of
// the next, so that the latencies of the list and of the page table stay out of the way: A the position (a
// list entry), B the page, C the record.
struct Lookahead {
  // what an entry is: 0 nothing, 1 context, 2 a node in the cache, 3 a node among the drafts
  struct Look {
    int kind, r, p, head;
    uint64_t page;
  } la, lb;
  int ap, at, row;  // place of step A; the record's row, for copies in boxes (rows_end: none)
  uint64_t now;     // the record's address, 0: none
  bool begun;

  // One tile further; after the first three calls `now` and `row` are those of the first tile.  `mine`: the
  // lane's entry in a tile; `lines`: 128-byte lines of the record (from the portion's KV head on) to bring
  // into L2 now, a tile before they are copied.
  __device__ __forceinline__ void step(const TreeArgs& a, const Portion* list, int count, int tile, int mine, int rows_end,
                                       int lines, uint32_t* bad) {
    {  // C
      const Look& l = lb;
      now = 0ull;
      row = rows_end;
      if (l.kind == 3) {
        now = (uint64_t)(uintptr_t)a.draft + (uint64_t)((int64_t)l.r * a.T + l.p) * (uint64_t)a.kv.rec;
      } else if (l.kind != 0 && a.slot_pt != nullptr) {
        now = l.page + (uint64_t)l.p * (uint64_t)a.kv.rec;
      } else if (l.kind != 0 && l.page < (uint64_t)a.kv.num_pages) {
        row = (int)l.page * a.kv.page_tokens + l.p;
        now = (uint64_t)(uintptr_t)a.kv.base + (uint64_t)row * (uint64_t)a.kv.rec;
      } else if (l.kind != 0) {
        *bad |= (uint32_t)HS_DEVERR_PAGE;
      }
      if (now != 0ull) {
#pragma unroll 1
        for (int x = 0; x < lines; ++x)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(now + (uint64_t)(2 * l.head + 128 * x)));
      }
    }
    {  // B; p becomes the place in the page
      Look& l = lb;
      l = la;
      const int most = a.slot_pt != nullptr ? (l.kind == 1 ? a.slot_cap[l.r] : 0) : a.kv.max_pages * a.kv.page_tokens;
      if (l.kind == 1 && a.locs != nullptr && l.p == -1) l.kind = 0;
      if ((l.kind == 1 || l.kind == 2) && (unsigned)l.p >= (unsigned)most) {
        *bad |= (uint32_t)HS_DEVERR_LOC;
        l.kind = 0;
      }
      if (l.kind == 1 || l.kind == 2) {
        if (a.slot_pt != nullptr) {
          l.page = a.slot_pt[(int64_t)l.r * a.slot_pages + (l.p >> a.slot_shift)];
          l.p &= (1 << a.slot_shift) - 1;
        } else {
          const unsigned pg = (unsigned)l.p / (unsigned)a.kv.page_tokens;
          l.p -= (int)(pg * (unsigned)a.kv.page_tokens);
          l.page = a.kv.table != nullptr ? (uint64_t)(int64_t)a.kv.table[(int64_t)l.r * a.kv.max_pages + pg]
                                         : (uint64_t)((int64_t)l.r * a.kv.max_pages + pg);
        }
      }
    }
    {  // A
      Look& l = la;
      l.kind = 0;
      l.r = 0;
      if (ap < count) {
        const Portion& P = list[ap];
        const int n4 = (int)(((unsigned)P.n + 3u) & ~3u), e = at * tile + mine;
        l.r = P.r;
        l.head = P.head * a.kstride;
        if (e < P.n) {
          l.kind = 1;
          l.p = a.locs != nullptr ? a.locs[(int64_t)P.r * a.k + e] : e;
        } else if (e >= n4 && e - n4 < P.nn) {
          l.kind = a.draft != nullptr ? 3 : 2;
          l.p = a.draft != nullptr ? e - n4 : P.len + (e - n4);
        }
        if (++at == P.t1) {
          ++ap;
          if (ap < count) at = list[ap].t0;
        }
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ void swap_both(T& x, T& y) {
  const T z = x;
  x = y;
  y = z;
}
__device__ __forceinline__ bool warp_wait_small(uint64_t* bar, uint32_t parity, volatile uint32_t* abort) {
  bool w = true;
  if ((threadIdx.x & 31) == 0) w = mbar_wait_small(bar, parity, abort);
  return __shfl_sync(0xffffffffu, w ? 1 : 0, 0) != 0;
}

// one OR over the threads of a named barrier
__device__ __forceinline__ bool bar_or(int id, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)x)
      : "memory");
  return r != 0u;
}

__device__ __forceinline__ bool bad_pair(uint32_t w) {  // an infinity or NaN among two bf16
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t good_pair(uint32_t w) {
  return ((w & 0x7f80u) == 0x7f80u ? 0u : w & 0xffffu) | ((w & 0x7f800000u) == 0x7f800000u ? 0u : w & 0xffff0000u);
}

// bits j0 .. j0 + 31 of a node's visibility among the nn nodes in use (bits before 0 are clear); first: the
// first word of m, at hand
__device__ __forceinline__ uint32_t mask_bits(const uint64_t* m, uint64_t first, int words, int nn, int j0) {
  if (j0 <= -32 || j0 >= nn) return 0u;
  const int s = max(j0, 0), w = s >> 6, b = s & 63;
  uint64_t x = (w == 0 ? first : m[w]) >> b;
  if (b > 32 && w + 1 < words) x |= m[w + 1] << (64 - b);
  uint32_t v = (uint32_t)x;
  if (nn - s < 32) v &= (1u << (nn - s)) - 1u;
  return v << (s - j0);
}

// What a row does not see, in its scores in tensor memory: -infinity.  (Apart from the loops over the scores, which
// so have one form: code that a CTA meets for the first time costs about half a microsecond a kilobyte.)
template <int WORDS>
__device__ __forceinline__ void mask_scores(uint32_t ts, const uint32_t (&w)[WORDS]) {
#pragma unroll 1
  for (int x = 0; x < WORDS; ++x) {
    float v[32];
    tmem_ld32(ts + 32u * x, v);
    uint32_t b = w[0];
#pragma unroll
    for (int i = 1; i < WORDS; ++i) b = x == i ? w[i] : b;
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = (b >> j) & 1u ? v[j] : -INFINITY;
    tmem_st32(ts + 32u * x, v);
  }
}

// Takes infinite and NaN values out of the rows [y0, y1) of a tile of `blocks` 128-byte column blocks, `block`
// bytes apart, with `group` bytes from 8 rows to the next (the swizzle moves bytes within a row's 128 only).
// Thread `id` of `threads`; true: it found some.
__device__ __forceinline__ bool clean_rows(uint8_t* tile, int block, int group, int blocks, int y0, int y1, int id, int threads) {
  bool found = false;
#pragma unroll 1
  for (int i = id; i < (y1 - y0) * blocks * 8; i += threads) {
    const int x = i & 7, z = i >> 3, b = z % blocks, y = y0 + z / blocks;
    uint4* at = (uint4*)(tile + b * block + (y >> 3) * group + (y & 7) * 128 + 16 * x);
    const uint4 u = *at;
    if (bad_pair(u.x) || bad_pair(u.y) || bad_pair(u.z) || bad_pair(u.w)) {
      found = true;
      *at = make_uint4(good_pair(u.x), good_pair(u.y), good_pair(u.z), good_pair(u.w));
    }
  }
  if (found) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  return found;
}

// ---- joining the partials of an item -------------------------------------------------------------

constexpr int kJoinThreads = 128;  // 89.4 us instead of 90.7 with 256 on 8 ragged requests x 64 nodes: more of them fit an SM

struct CombineArgs {
  const int32_t* nodes;
  uint16_t* out;
  WorkSplit ws;
  int R, T, Hq, workers;
  int G, MT, per;  // rows of a node, nodes of a 128-row tile, row tiles of an item
  int np;          // items: KV head * np + group of row tiles
  int flat;        // a shared latent: item i holds the rows [flat i, flat (i + 1)) of all node x head rows
};

// A thread holds W dims of a row, neighbouring threads neighbouring rows, with F partials on their way to it; items
// that one worker held whole are written by it.  What it costs is round trips to what other SMs have just written,
// about 1 us each, where there is little to join, and else the SMs' room for threads and loads: see launch_combine.
template <int DV, int W, int F>
__global__ void __launch_bounds__(kJoinThreads, W == 8 ? 7 : 1) k_tree_combine(CombineArgs c) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int item = blockIdx.x, r = blockIdx.y, idx = blockIdx.z * kJoinThreads + threadIdx.x;
  const long long p0 = c.ws.prefix[r], U = c.ws.prefix[r + 1] - p0, total = c.ws.prefix[c.R];
  int nn = c.T;
  if (c.nodes != nullptr) nn = min(max(c.nodes[r], 0), c.T);
  if (U == 0) return;
  // the 8 / W threads of 8 dims of a row are neighbours
  const int rows = c.ws.rows, part = idx % (8 / W), at = idx / (8 / W), blk = at / rows, row = at - blk * rows, x = row & 127;
  const int mt = c.flat ? 0 : (item % c.np) * c.per + (row >> 7);
  const int t = c.flat ? (item * c.flat + row) / c.Hq : mt * c.MT + x / c.G;
  const int h = c.flat ? (item * c.flat + row) % c.Hq : item / c.np * c.G + x % c.G;
  if (blk >= DV / 8 || (!c.flat && x >= c.G * c.MT) || t >= nn) return;
  const Shares sh(total * c.ws.items, c.workers);
  const long long a = p0 * c.ws.items + item * U;
  const int wf = sh.worker(a + c.ws.begin), wl = sh.worker(a + U - 1);
  if (wf == wl) return;
  float M = -INFINITY, L = 0.f, acc[W];
#pragma unroll
  for (int i = 0; i < W; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int w0 = wf; w0 <= wl; w0 += F) {
    float2 ml[F];
    float4 v[F][W / 4];
#pragma unroll
    for (int j = 0; j < F; ++j) {
      const int w = w0 + j;
      ml[j] = make_float2(-INFINITY, 0.f);
      if (w > wl) continue;
      const long long slot = ((long long)w * 2 + (w == wf ? 1 : 0)) * rows;
      const float4* p = (const float4*)(c.ws.part + slot * DV + ((long long)blk * rows + row) * 8 + W * part);
      ml[j] = *(const float2*)(c.ws.ml + (slot + row) * 2);
#pragma unroll
      for (int i = 0; i < W / 4; ++i) v[j][i] = p[i];
    }
    float mn = M;
#pragma unroll
    for (int j = 0; j < F; ++j) mn = fmaxf(mn, ml[j].x);
    const float al = M == mn ? 1.f : exp2f(M - mn);
    M = mn;
    L *= al;
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] *= al;
#pragma unroll
    for (int j = 0; j < F; ++j) {
      if (w0 + j > wl) continue;
      // -infinity: nothing seen (sum 0), or NaN scores alone (NaN).  A weight of 0 counts all the same: what the row saw
      // may be infinite or NaN, and what it saw nothing of holds zeros
      const float wt = ml[j].x == -INFINITY ? ml[j].y : exp2f(ml[j].x - M);
      L = fmaf(wt, ml[j].y, L);
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        acc[4 * i] = fmaf(wt, v[j][i].x, acc[4 * i]);
        acc[4 * i + 1] = fmaf(wt, v[j][i].y, acc[4 * i + 1]);
        acc[4 * i + 2] = fmaf(wt, v[j][i].z, acc[4 * i + 2]);
        acc[4 * i + 3] = fmaf(wt, v[j][i].w, acc[4 * i + 3]);
      }
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  uint2* dst = (uint2*)(c.out + (((int64_t)r * c.T + t) * c.Hq + h) * DV + 8 * blk + W * part);
  if (W == 8) {
    *(uint4*)dst = make_uint4(pack(acc[0] * inv, acc[1] * inv), pack(acc[2] * inv, acc[3] * inv), pack(acc[W - 4] * inv, acc[W - 3] * inv),
                              pack(acc[W - 2] * inv, acc[W - 1] * inv));
  } else {
    *dst = make_uint2(pack(acc[0] * inv, acc[1] * inv), pack(acc[2] * inv, acc[3] * inv));
  }
}
template <int DV>
cudaError_t launch_combine(const CombineArgs& c, cudaStream_t st) {
  auto ctas = [&](int w) { return (c.ws.rows * (DV / w) + kJoinThreads - 1) / kJoinThreads; };
  // Up to two CTAs an SM it is latency: 12.6 us (the call) instead of 13.7 on 1 request x 4 nodes x 1000 positions.  More
  // threads with fewer loads each else: 72.5 us instead of 74.3 on 4 requests x 5 nodes over shared latents.
  if ((int64_t)c.ws.items * c.R * ctas(8) <= 2 * kSmsHint)
    return hs_launch_pdl(k_tree_combine<DV, 4, 8>, dim3(c.ws.items, c.R, ctas(4)), dim3(kJoinThreads), 0, st, c);
  return hs_launch_pdl(k_tree_combine<DV, 8, 4>, dim3(c.ws.items, c.R, ctas(8)), dim3(kJoinThreads), 0, st, c);
}

bool encode(CUtensorMap* m, const void* base, int dims, const cuuint64_t* size, const cuuint64_t* stride,
            const cuuint32_t* box) {
  const EncodeFn fn = tensor_map_encoder();
  const cuuint32_t one[4] = {1, 1, 1, 1};
  memset(m, 0, sizeof(*m));
  return fn != nullptr && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)dims, const_cast<void*>(base), size, stride, box,
                             one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The shared-memory limit of a kernel, raised once per device.
template <typename K>
cudaError_t allow_smem(K kern, size_t bytes, bool* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done[dev])) return e;
  e = hs_raise_smem_limit(kern, (int)bytes);
  if (e == cudaSuccess && dev < 64) done[dev] = true;
  return e;
}

}  // namespace

// ---- host ------------------------------------------------------------------------------------------

// The workspace: the tiles before each request, then (32-byte aligned, whatever the workspace's alignment)
// the partials and their statistics.
inline int64_t hs_tree_workspace_bytes(const hs_config* c, int64_t workers, int64_t rows, int64_t dims) {
  return (int64_t)(c->num_requests + 1) * (int64_t)sizeof(int64_t) + 64 + workers * 2 * rows * (dims + 2) * (int64_t)sizeof(float);
}
inline void hs_tree_workspace(void* w, const hs_config* c, int64_t workers, int64_t rows, int64_t dims, long long** prefix,
                              float** part, float** ml) {
  *prefix = (long long*)w;
  *part = (float*)(((uintptr_t)(*prefix + c->num_requests + 1) + 31u) & ~(uintptr_t)31u);
  *ml = *part + workers * 2 * rows * dims;
}

// Launch plans of the tensor-core kernels.  `usable`: the shape is theirs.
struct hs_tree_plan {
  bool usable;
  int64_t workspace;
};
hs_tree_plan hs_tree_gqa_plan(const hs_config* c, int nodes, int num_sms);
hs_tree_plan hs_tree_mla_plan(const hs_config* c, int nodes, int num_sms);
int hs_tree_mla_launch(const hs_config* c, const hs_tree_args* g, const void* tree_args, int num_sms, cudaStream_t st);
int hs_tree_gqa_launch(const hs_config* c, const hs_tree_args* g, const void* tree_args, int num_sms, cudaStream_t st);

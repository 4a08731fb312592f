// Attention of one new token a request over a paged cache whose requests share prefixes: segments, the division of the
// work, the joining of its pieces; shared by the kernels.
#pragma once

#include "hs_tree.cuh"

namespace {

struct PrefixArgs {
  PagedRows kv;
  const uint16_t* q;      // [R][Hq][dqk]
  const int64_t* len;     // [R]
  const int32_t* groups;  // [ngroups + 1]
  const int64_t* prefix;  // [ngroups]
  uint16_t* out;          // [R][Hq][dv]
  float* weights;         // [R][lists][cap] or null
  int64_t cap;
  float* scores;          // [R][Hq][score_cols], in units of log2, with weights
  int64_t score_cols;
  float2* stats;          // [R][Hq] maximum and 1 / sum of each row, with weights
  int R, ngroups, Hq, Hkv, dqk, dv, lists;
  int kstride, voff;      // values: KV head g's key at g * kstride, its value voff further on
  float qscale;           // scale * log2(e)
  float decay;
  int stall;              // test hook (hs_debug_stall_prefix): arrivals that a barrier of a worker's first tile waits for in vain
};

// ---- segments ------------------------------------------------------------------------------------
//
// Segment g < ngroups is group g's prefix, whose rows are all its requests'; segment ngroups + r what request r has for
// itself.  A request's result joins its own segment's and its group's.

struct Segment {
  int lead, r0, nr;  // request whose table is read; the requests
  int p0, p1;        // positions
};

__device__ __forceinline__ int64_t positions_of(const PrefixArgs& a) { return (int64_t)a.kv.max_pages * a.kv.page_tokens; }

// Whether the bounds of groups g, g + step, ... are sound.
__device__ __forceinline__ bool bounds_ok(const PrefixArgs& a, int g, int step) {
  bool ok = true;
  for (; g < a.ngroups; g += step) ok = ok && a.groups[g] >= 0 && a.groups[g] <= a.groups[g + 1] && a.groups[g + 1] <= a.R;
  return ok;
}
// Requests and prefix of group g, with sound bounds.
__device__ __forceinline__ Segment group_segment(const PrefixArgs& a, int g, uint32_t* bad) {
  const int64_t p = a.prefix[g];
  const bool out = p < 0 || p > positions_of(a);
  if (out) *bad |= (uint32_t)HS_DEVERR_LOC;
  Segment s;
  s.r0 = s.lead = a.groups[g];
  s.nr = a.groups[g + 1] - s.r0;
  s.p0 = 0;
  s.p1 = s.nr >= 1 && !out ? (int)p : 0;
  return s;
}
// The group of request r, -1: none.
__device__ __forceinline__ int group_of(const PrefixArgs& a, int r) {
  int x = 0, n = a.ngroups;
  while (n > 1) {  // the last that begins at or before r
    const int half = n >> 1;
    if (a.groups[x + half] <= r) x += half;
    n -= half;
  }
  return a.ngroups > 0 && a.groups[x] <= r && r < a.groups[x + 1] ? x : -1;
}
// What request r shares: its group's segment, empty without one.
__device__ __forceinline__ Segment shared_segment(const PrefixArgs& a, int r, bool ok, int* g) {
  uint32_t quiet = 0u;  // the segment itself reports its errors
  *g = ok ? group_of(a, r) : -1;
  if (*g < 0) return Segment{r, r, 1, 0, 0};
  return group_segment(a, *g, &quiet);
}
// What it has for itself behind `shared` positions; shorter than them, or of a bad length, it has nothing to see: p1 = 0.
__device__ __forceinline__ Segment own_segment(const PrefixArgs& a, int r, int shared, uint32_t* bad) {
  const int64_t n = a.len[r];
  Segment s{r, r, 1, shared, (int)n};
  if (n < shared || n > positions_of(a)) {
    if (n != 0) *bad |= (uint32_t)HS_DEVERR_LOC;
    s.p0 = s.p1 = 0;
  }
  return s;
}
// Segment v, and its group (-1: none) with that one's segment.
__device__ __forceinline__ Segment segment_of(const PrefixArgs& a, int v, bool ok, uint32_t* bad, int* g, Segment* shared) {
  const int r = v - a.ngroups;
  *g = !ok ? -1 : r < 0 ? v : group_of(a, r);
  *shared = Segment{0, 0, 0, 0, 0};
  uint32_t quiet = 0u;  // a group's errors are reported with its own segment
  if (*g >= 0) *shared = group_segment(a, *g, &quiet);
  if (r < 0) {
    *bad |= quiet;
    return *shared;
  }
  return own_segment(a, r, shared->p1, bad);
}

// ---- division of the work ------------------------------------------------------------------------
//
// A segment's rows are cut into row tiles, an item is one KV head with one or two of them over all the segment's tiles of
// entries; the tiles of all items of all segments form one sequence in units of time, of which every worker (a CTA, or a pair)
// takes an equal share.  A worker's portion of an item leaves its partial sums in rows of its own: the rows of all items before
// it, and `most` for each worker before it, which no two portions share.

struct PrefixSplit {
  int heads;             // KV heads
  int flat;              // row tiles of 128 (request, query head) rows, whatever the request; else
  int G, MT;             // a row tile is MT requests of G rows each
  Div mt;                // by MT
  int pairs;             // 1: an item has two row tiles where there are two left, 0: one
  int tile_shift;        // log2 of the entries of a tile
  Div cost, cost2;       // units of a tile with one and with two row tiles
  int begin;             // units of an item's beginning
  int copies;            // partials of a row in a portion: 2 where two groups share the tiles of one row tile
  int most;              // rows of a portion at most
  int group_rows;        // rows that a group's segment takes for each of its requests at most; a request's own takes 2 Hq
  int workers;
  long long* units;      // [ngroups + 1] before each group's segment and in all, written by the first CTA
  struct PrefixRequest* of; // [R], likewise
  int together;          // rows that a CTA of the join takes: they are neighbours in all their partials
  float *part, *ml;      // of each copy of a portion [dv / 8][rows][8], so that neighbouring rows are stored side by side; and
                         // [rows][4]: maximum (base 2), sum of rounded weights, of exact ones
};

// What the join has to know of a request.
struct __align__(16) PrefixRequest {
  long long units;        // before its own segment
  int p0, p1;             // its own positions; p1 = 0: it sees nothing
  int g, r0, nr, pad;     // its group (-1: none) and that one's requests
};

struct Shape1 {  // a segment's division
  int base, tiles, nmt, np, rows;  // first entry of tile 0; row tiles, items of a head, rows of a portion
  int item;                        // units of a full item
  long long head;                  // of a KV head
};
__device__ __forceinline__ Shape1 shape_of(const PrefixArgs& a, const PrefixSplit& w, const Segment& s) {
  Shape1 x;
  x.base = s.p0 & ~31;
  x.tiles = s.p1 > s.p0 ? (int)(((unsigned)(s.p1 - x.base) + (1u << w.tile_shift) - 1u) >> w.tile_shift) : 0;
  x.nmt = w.flat ? (s.nr * a.Hq + 127) >> 7 : (int)w.mt((uint32_t)(s.nr + w.MT - 1));
  x.np = (x.nmt + w.pairs) >> w.pairs;
  x.rows = w.flat ? min(128, s.nr * a.Hq) : w.G * min(s.nr, w.MT) * w.copies;
  x.item = x.tiles * (int)(w.pairs ? w.cost2.d : w.cost.d) + w.begin;
  x.head = (long long)(x.nmt >> w.pairs) * x.item;
  if (w.pairs && (x.nmt & 1)) x.head += x.tiles * (int)w.cost.d + w.begin;
  if (x.tiles == 0) x.head = 0;
  return x;
}
// The first row of partials of a segment of the requests from r0 on.  Segments' rows are in the order of their units, so that a
// portion's, most * worker further on, are its own (see PPortion).
__device__ __forceinline__ long long rows_before(const PrefixArgs& a, const PrefixSplit& w, bool group, int r0) {
  return group ? (long long)w.group_rows * r0 : (long long)w.group_rows * a.R + 2ll * a.Hq * r0;
}
// Tile t of an item belongs to the worker that holds its first unit: tiles from unit u on.
__device__ __forceinline__ int tile_at(long long u, int begin, const Div& cost, int tiles) {
  const long long x = min(u - begin, (long long)tiles * (int)cost.d);
  return x <= 0 ? 0 : (int)cost((uint32_t)x + cost.d - 1u);
}

struct PPortion {
  int lead, r0, cnt;    // request whose table is read, first request of the row tiles (flat: first row), requests (rows) in them
  int p0, p1, base;     // positions [p0, p1), tile t begins at base + t * tile
  int t0, t1;           // equal: no portion, the list's end
  short head, both;     // both: two row tiles
  short first, own;     // first: group of tile t0 when not both; own: a request's own segment
  int stride;           // rows of a copy of the partials
  long long row;        // first row of the partials
};

// A worker's portions go through a ring, from the warp that finds them to the others.
constexpr int kPrefixRing = 8;

struct PrefixPlan {  // shared memory
  union {
    PPortion port[kPrefixRing];
    long long scan[32];  // of each warp of the CTA, before the first portion
  };
  uint64_t full[kPrefixRing], empty[kPrefixRing];
  long long off, left;  // units into segment cur, units to take
  int cur, ok;          // ok: the groups' bounds are sound
  Segment seg;          // segment cur
};
__device__ __forceinline__ void prefix_plan_init(PrefixPlan* s, int readers) {
  for (int i = 0; i < kPrefixRing; ++i) {
    mbar_init(&s->full[i], 1u);
    mbar_init(&s->empty[i], (uint32_t)readers);
  }
}

__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// Where this worker starts: every thread of the CTA calls it.  (What small calls cost is the way to the first tile: round trips,
// one for lengths and groups together, and instructions met for the first time, about half a microsecond a kilobyte.)
__device__ __forceinline__ void prefix_start(const PrefixArgs& a, const PrefixSplit& w, PrefixPlan* s, int worker) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, G = a.ngroups, V = G + a.R;
  const int each = (V + nthr - 1) / nthr, v0 = min(tid * each, V), v1 = min(v0 + each, V);
  if (v0 < V) prefetch_l1(v0 < G ? a.prefix + v0 : a.len + (v0 - G));
  const bool ok = __syncthreads_and(bounds_ok(a, tid, nthr)) != 0;
  uint32_t bad = ok ? 0u : (uint32_t)HS_DEVERR_LOC;
  if (tid == 0) {
    s->left = 0;
    s->ok = ok;
  }
  long long before = 0, mine = 0, total = 0, start = 0;  // units: before this thread's segments, theirs, in all
  Shares sh(0, 1);
  int g = -1;
  Segment sg{0, 0, 0, 0, 0}, shared{0, 0, 0, 0, 0};
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int v = v0; v < v1; ++v) {
      long long u = mine;
      if (pass == 0 || each > 1) {  // one segment a thread: known in the second pass
        sg = segment_of(a, v, ok, &bad, &g, &shared);
        u = shape_of(a, w, sg).head * w.heads;
      }
      if (pass == 0) {
        mine += u;
        continue;
      }
      if (blockIdx.x == 0) {
        if (v < G) w.units[v] = before;
        else w.of[v - G] = PrefixRequest{before, sg.p0, sg.p1, g, shared.r0, shared.nr, 0};
      }
      if (start >= before && start < before + u) {
        s->cur = v;
        s->seg = sg;
        s->off = start - before;
        s->left = sh.start(worker + 1) - start;
      }
      before += u;
    }
    if (pass != 0) break;
    if (blockIdx.x == 0) report(a.kv.err, bad);
    long long incl = 0;
#pragma unroll 1
    for (int level = 0; level < 2; ++level) {  // within the warp, then over the warps
      long long y = level == 0 ? mine : lane < (nthr >> 5) ? s->scan[lane] : 0;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const long long z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
      }
      if (level == 0) {
        incl = y;
        if (lane == 31) s->scan[warp] = y;
        __syncthreads();
      } else {
        total = __shfl_sync(0xffffffffu, y, 31);
        before = incl - mine + (warp > 0 ? __shfl_sync(0xffffffffu, y, warp - 1) : 0);
      }
    }
    sh = Shares(total, w.workers);
    start = sh.start(worker);
    if (blockIdx.x == 0 && tid == 0) w.units[G] = total;
    if (blockIdx.x != 0 && !(start >= before && start < before + mine)) break;
  }
  __syncthreads();
}

// The portions of this worker, by one warp: a lane an item.
__device__ __forceinline__ void prefix_walk(const PrefixArgs& a, const PrefixSplit& w, PrefixPlan* s, int worker, volatile uint32_t* abort) {
  const int lane = threadIdx.x & 31, V = a.ngroups + a.R;
  long long off = s->off, left = s->left;
  int cur = s->cur, from = cur, turn = 0, made = 0;
  Segment sg = s->seg, ahead = sg;  // ahead: segment from + lane (at first: each lane the first one)
#pragma unroll 1
  while (left > 0) {
    const Shape1 x = shape_of(a, w, sg);
    const long long U = x.head * w.heads;
    if (off < U) {
      const int head0 = (int)Shares::div_small(off, x.head);
      const int pair0 = x.np == 1 ? 0 : (int)min((long long)(x.np - 1), Shares::div_small(off - head0 * x.head, x.item));
      const int k0 = head0 * x.np + pair0, k = k0 + lane, head = x.np == 1 ? k : (int)((unsigned)k / (unsigned)x.np), pair = k - head * x.np;
      const bool both = w.pairs && 2 * pair + 1 < x.nmt;
      const Div& cost = both ? w.cost2 : w.cost;
      const long long at = head * x.head + (long long)pair * x.item;  // the item's first unit
      const long long u0 = off - at, u1 = off + left - at;
      PPortion p;
      p.t0 = p.t1 = 0;
      if (head < w.heads && u1 > 0) {
        p.t0 = tile_at(u0, w.begin, cost, x.tiles);
        p.t1 = tile_at(u1, w.begin, cost, x.tiles);
      }
      const bool has = p.t0 < p.t1;  // else no tile begins here
      const uint32_t who = __ballot_sync(0xffffffffu, has), odd = __ballot_sync(0xffffffffu, has && !both && ((p.t1 - p.t0) & 1) != 0);
      const uint32_t below = (1u << lane) - 1u;
      const int mine = __popc(who & below), n = __popc(who);
      p.lead = sg.lead;
      p.r0 = w.flat ? sg.r0 * a.Hq + 128 * pair : sg.r0 + (pair << w.pairs) * w.MT;
      p.cnt = w.flat ? min(128, sg.nr * a.Hq - 128 * pair) : min(w.MT << w.pairs, sg.nr - (pair << w.pairs) * w.MT);
      p.p0 = sg.p0;
      p.p1 = sg.p1;
      p.base = x.base;
      p.head = (short)head;
      p.both = both;
      p.own = cur >= a.ngroups;
      p.first = (short)((turn + __popc(odd & below)) & 1);
      p.stride = w.copies == 2 ? x.rows >> 1 : x.rows;
      p.row = rows_before(a, w, cur < a.ngroups, sg.r0) + (long long)k * x.rows + (long long)worker * w.most;
      turn = (turn + __popc(odd)) & 1;
      // one after the other: a reader may need a portion before it can release an earlier one
#pragma unroll 1
      for (int b = 0; b < n; ++b) {
        bool fine = true;
        if (has && mine == b) {
          const int i = made + b, slot = i % kPrefixRing;
          fine = mbar_wait_small(&s->empty[slot], (uint32_t)((i / kPrefixRing) & 1) ^ 1u, abort);
          if (fine) {
            s->port[slot] = p;
            mbar_arrive(&s->full[slot]);
          }
        }
        if (!__all_sync(0xffffffffu, fine)) {
          *abort = 1u;
          return;
        }
      }
      made += n;
      // on to what follows these 32 items
      const int last = k0 + 32, lh = x.np == 1 ? last : (int)((unsigned)last / (unsigned)x.np);
      const long long next = lh >= w.heads ? U : lh * x.head + (long long)(last - lh * x.np) * x.item;
      const long long step = min(left, next - off);
      off += step;
      left -= step;
      if (off < U) continue;
    }
    off -= U;
    if (left == 0 || ++cur >= V) break;
    if (cur == from + 1 || cur >= from + 33) {  // 32 segments at a time, a lane each
      from = cur - 1;
      uint32_t quiet = 0u;
      int g;
      Segment shared;
      if (cur + lane < V) ahead = segment_of(a, cur + lane, s->ok != 0, &quiet, &g, &shared);
    }
    const int src = cur - from - 1;
    sg.lead = sg.r0 = __shfl_sync(0xffffffffu, ahead.r0, src);
    sg.nr = __shfl_sync(0xffffffffu, ahead.nr, src);
    sg.p0 = __shfl_sync(0xffffffffu, ahead.p0, src);
    sg.p1 = __shfl_sync(0xffffffffu, ahead.p1, src);
  }
  if (lane == 0) {
    const int slot = made % kPrefixRing;
    if (mbar_wait_small(&s->empty[slot], (uint32_t)((made / kPrefixRing) & 1) ^ 1u, abort)) {
      s->port[slot].t0 = s->port[slot].t1 = 0;
      mbar_arrive(&s->full[slot]);
    } else {
      *abort = 1u;
    }
  }
}

// Portion i of the list, by whoever reads it; false: a wait that gave up.  It stays in place until it is released by every reader.
__device__ __forceinline__ bool portion_wait(PrefixPlan* s, int i, volatile uint32_t* abort) {
  return mbar_wait_small(&s->full[i % kPrefixRing], (uint32_t)((i / kPrefixRing) & 1), abort);
}
__device__ __forceinline__ const PPortion& portion_at(const PrefixPlan* s, int i) { return s->port[i % kPrefixRing]; }
// The same for a whole warp: a copy (t0 = t1: no more, or the wait gave up), and its release when `done`.
__device__ __forceinline__ PPortion portion_take(PrefixPlan* s, int i, bool done, bool* ok, volatile uint32_t* abort) {
  PPortion p;
  p.t0 = p.t1 = 0;
  if (*ok) *ok = __all_sync(0xffffffffu, portion_wait(s, i, abort));
  if (*ok) p = portion_at(s, i);
  __syncwarp();
  if (*ok && done && (threadIdx.x & 31) == 0) mbar_arrive(&s->empty[i % kPrefixRing]);
  return p;
}

// ---- joining ---------------------------------------------------------------------------------------

// The running sum of a row's partials: 8 of its dims, maximum, sums of rounded and of exact weights.
struct Joined {
  float m = -INFINITY, l = 0.f, le = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(const float4& s, const float4& x, const float4& y) {
    const float mn = fmaxf(m, s.x);
    // -infinity: nothing seen (sum 0), or NaN scores alone (NaN).  A weight of 0 counts all the same: what the row saw may
    // be infinite or NaN, and what it saw nothing of holds zeros
    const float al = m == mn ? 1.f : exp2f(m - mn), wt = s.x == -INFINITY ? s.y : exp2f(s.x - mn);
    m = mn;
    l = l * al + wt * s.y;
    le = le * al + wt * s.z;
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(wt, v[i], acc[i] * al);
  }
  __device__ __forceinline__ void add(const float* part, const float* ml, long long row, int dv, int d) {
    const float* p = part + row * dv + d;
    add(*(const float4*)(ml + 4 * row), *(const float4*)p, *(const float4*)(p + 4));
  }
  __device__ __forceinline__ void store(const PrefixArgs& a, int r, int h, int d) const {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *(uint4*)(a.out + ((int64_t)r * a.Hq + h) * a.dv + d) =
        make_uint4(pack(acc[0] * inv, acc[1] * inv), pack(acc[2] * inv, acc[3] * inv), pack(acc[4] * inv, acc[5] * inv),
                   pack(acc[6] * inv, acc[7] * inv));
    if (a.stats != nullptr && d == 0) a.stats[(int64_t)r * a.Hq + h] = make_float2(m == -INFINITY ? 0.f : m, le == 0.f ? 0.f : 1.f / le);
  }
};

// The partials of an item, or of one row of it: where each worker's are.
struct Pieces {
  long long item, base;    // units before the item; its first row of partials
  Div cost;
  int begin, tiles, first, copies, stride, row, n;  // first worker, partials a worker, rows of each, the row's place in them, partials in all
  // of row (r, h), h the first of a KV head's where rows are not flat
  __device__ __forceinline__ void of(const PrefixArgs& a, const PrefixSplit& w, const Shares& sh, const Segment& sg, bool group, long long units,
                                     int r, int h) {
    n = 0;
    const Shape1 sp = shape_of(a, w, sg);
    if (sp.tiles == 0) return;
    const int j = r - sg.r0, flat = j * a.Hq + h, mt = w.flat ? flat >> 7 : (int)w.mt((uint32_t)j);
    row = w.flat ? flat & 127 : (j - mt * w.MT) * w.G;
    const int head = w.flat ? 0 : h / w.G, pair = mt >> w.pairs;
    const bool both = w.pairs && 2 * pair + 1 < sp.nmt;
    begin = w.begin;
    cost = both ? w.cost2 : w.cost;
    tiles = sp.tiles;
    stride = w.copies == 2 ? sp.rows >> 1 : sp.rows;
    copies = both ? 1 : w.copies;
    item = units + head * sp.head + (long long)pair * sp.item;
    base = rows_before(a, w, group, sg.r0) + (long long)(head * sp.np + pair) * sp.rows + (both ? (mt & 1) * stride : 0);
    first = sh.worker(item + begin);
    n = copies * (sh.worker(item + begin + (long long)(sp.tiles - 1) * (int)cost.d) - first + 1);
  }
  // the first row of partial i, -1: its worker has no tile (or too few for a second copy)
  __device__ __forceinline__ int at(const PrefixSplit& w, const Shares& sh, int i) const {
    const int wk = first + (copies == 2 ? i >> 1 : i), copy = copies == 2 ? i & 1 : 0;
    const int t0 = tile_at(sh.start(wk) - item, begin, cost, tiles), t1 = tile_at(sh.start(wk + 1) - item, begin, cost, tiles);
    return t1 - t0 > copy ? (int)(base + (long long)wk * w.most + copy * stride) : -1;
  }
};

// A CTA joins rows of a request that are together in all partials: the G of a KV head, or (flat) up to four.  Its first threads find
// the partials' places, kPrefixList at a time; then a thread takes 8 dims of a row from every `slices`-th partial, kPrefixAhead of
// them on their way at a time, and the slices are summed in order.
// What it costs is a chain of round trips, and instructions met for the first time: it starts while the attention still runs, and
// goes through the first of them once on made-up numbers.  16 requests over 32768 shared positions: 50.1 us; without that 50.7, with one
// slice 54.3, with one partial on its way 51.6 (8 requests of 64 heads over latents 64.0 instead of 58.8).
constexpr int kPrefixAhead = 3, kPrefixList = 64;

template <int DV, int THREADS>
__global__ void __launch_bounds__(THREADS, 768 / THREADS) k_prefix_join(const PrefixArgs a, const PrefixSplit w, int slices) {
  constexpr int vecs = DV >> 3;
  __shared__ Pieces s_piece[2];  // of its own segment, of its group's
  __shared__ long long s_share[2];
  __shared__ int s_row[kPrefixList];
  __shared__ float s_acc[THREADS][8];
  __shared__ float4 s_ml[THREADS];
  const int tid = threadIdx.x, r = blockIdx.x, rows = w.together, h0 = blockIdx.y * rows, units = rows * vecs;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    if (pass != 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      // only this call's own last kernel may start early, which waits for this one
      if (a.weights != nullptr) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    if (tid < 2) {  // a thread a segment
      PrefixRequest q{0, 0, 64, -1, r, 1, 0};
      long long total = 4 * w.workers;
      if (pass != 0) {
        q = w.of[r];
        total = w.units[a.ngroups];
      }
      const Shares sh(total, w.workers);
      const bool group = tid == 1;
      const Segment sg = !group ? Segment{r, r, 1, q.p0, q.p1} : Segment{q.r0, q.r0, q.nr, 0, q.g >= 0 ? q.p0 : 0};
      s_piece[tid].n = s_piece[tid].row = s_piece[tid].stride = 0;
      if (q.p1 > 0) s_piece[tid].of(a, w, sh, sg, group, !group ? q.units : q.g > 0 ? w.units[q.g] : 0, r, h0);
      if (!group) {
        s_share[0] = sh.per;
        s_share[1] = sh.more;
      }
    }
  }
  const int u0 = units * slices <= THREADS ? tid % units : tid, slice = units * slices <= THREADS ? tid / units : 0;
#pragma unroll 1
  for (int ub = 0; ub < units; ub += THREADS) {  // more than one turn: more rows than threads, one slice
    const int u = ub + u0, vec = u / rows, x = u - vec * rows;  // neighbouring threads: neighbouring rows
    const bool on = u < units && slice < slices;
    Joined sum;
#pragma unroll 1
    for (int c0 = 0;; c0 += kPrefixList) {
      __syncthreads();
      const int own = s_piece[0].n, m = min(own + s_piece[1].n - c0, kPrefixList);
      if (m <= 0) break;
      if (tid < m) {
        const int i = c0 + tid, x = i < own ? 0 : 1;
        Shares sh(0, 1);
        sh.per = s_share[0];
        sh.more = s_share[1];
        s_row[tid] = s_piece[x].at(w, sh, i - x * own);
      }
      __syncthreads();
      if (!on) continue;
      const int row0 = s_piece[0].row + x, row1 = s_piece[1].row + x;
      const int at0 = (vec * s_piece[0].stride + row0) * 8, at1 = (vec * s_piece[1].stride + row1) * 8;
#pragma unroll 1
      for (int i0 = slice; i0 < m; i0 += kPrefixAhead * slices) {
        float4 l[kPrefixAhead], y[kPrefixAhead][2];
        int row[kPrefixAhead];
#pragma unroll
        for (int k = 0; k < kPrefixAhead; ++k) {
          const int i = i0 + k * slices;
          row[k] = i < m ? s_row[i] : -1;
          if (row[k] >= 0) {
            const bool mine = c0 + i < own;
            const float* p = w.part + (long long)row[k] * DV + (mine ? at0 : at1);
            l[k] = *(const float4*)(w.ml + 4ll * (row[k] + (mine ? row0 : row1)));
            y[k][0] = *(const float4*)p;
            y[k][1] = *(const float4*)(p + 4);
          }
        }
#pragma unroll
        for (int k = 0; k < kPrefixAhead; ++k)
          if (row[k] >= 0) sum.add(l[k], y[k][0], y[k][1]);
      }
    }
    if (slices > 1) {
      s_ml[tid] = make_float4(sum.m, sum.l, sum.le, 0.f);
      *(float4*)&s_acc[tid][0] = make_float4(sum.acc[0], sum.acc[1], sum.acc[2], sum.acc[3]);
      *(float4*)&s_acc[tid][4] = make_float4(sum.acc[4], sum.acc[5], sum.acc[6], sum.acc[7]);
      __syncthreads();
      if (slice == 0)
        for (int k = 1; k < slices; ++k)
          sum.add(s_ml[tid + k * units], *(const float4*)&s_acc[tid + k * units][0], *(const float4*)&s_acc[tid + k * units][4]);
    }
    if (on && slice == 0) sum.store(a, r, h0 + x, 8 * vec);
  }
}

template <int DV, int THREADS>
cudaError_t launch_join_by(const PrefixArgs& a, const PrefixSplit& w, cudaStream_t st) {
  const int rows = w.together, units = rows * (DV / 8);
  int slices = 1;
  while (2 * slices * units <= THREADS) slices *= 2;
  return hs_launch_pdl(k_prefix_join<DV, THREADS>, dim3(a.R, a.Hq / rows), dim3(THREADS), 0, st, a, w, slices);
}
template <int DV>
cudaError_t launch_join(const PrefixArgs& a, const PrefixSplit& w, cudaStream_t st) {
  // as many threads as the SMs hold at once: few CTAs have twice as many, for twice as many slices
  const bool few = (int64_t)a.R * (a.Hq / w.together) <= kSmsHint;
  return few ? launch_join_by<DV, 512>(a, w, st) : launch_join_by<DV, 256>(a, w, st);
}

}  // namespace

// ---- host ------------------------------------------------------------------------------------------

// Launch plans of the tensor-core kernels: `rows` of partials, 0: the shape is not theirs.
struct hs_prefix_plan {
  int64_t rows;
};
// The start of the workspace: units of the groups, the requests.
inline int64_t hs_prefix_head_bytes(int64_t groups, int64_t requests) {
  return ((groups + 1) * (int64_t)sizeof(long long) + 15) / 16 * 16 + requests * (int64_t)sizeof(PrefixRequest);
}
inline void hs_prefix_head(void* ws, int groups, PrefixSplit* w) {
  w->units = (long long*)ws;
  w->of = (PrefixRequest*)((uint8_t*)ws + hs_prefix_head_bytes(groups, 0));
}
hs_prefix_plan hs_prefix_gqa_plan(const hs_config* c, int num_sms);
hs_prefix_plan hs_prefix_mla_plan(const hs_config* c, int num_sms);
int hs_prefix_gqa_launch(const hs_config* c, const void* prefix_args, void* head, void* partials, int num_sms, cudaStream_t st);
int hs_prefix_mla_launch(const hs_config* c, const void* prefix_args, void* head, void* partials, int num_sms, cudaStream_t st);

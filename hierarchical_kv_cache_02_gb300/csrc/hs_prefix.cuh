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
  int* ok;                // whether the groups' bounds ascend within [0, R], written by the first kernel
  int R, ngroups, Hq, Hkv, dqk, dv, lists;
  int kstride, voff;      // values: KV head g's key at g * kstride, its value voff further on
  float qscale;           // scale * log2(e)
  float decay;
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
// Requests and prefix of group g, with sound bounds.  A group of one shares nothing: its prefix counts as the request's own.
__device__ __forceinline__ Segment group_segment(const PrefixArgs& a, int g, uint32_t* bad) {
  const int64_t p = a.prefix[g];
  const bool out = p < 0 || p > positions_of(a);
  if (out) *bad |= (uint32_t)HS_DEVERR_LOC;
  Segment s;
  s.r0 = s.lead = a.groups[g];
  s.nr = a.groups[g + 1] - s.r0;
  s.p0 = 0;
  s.p1 = s.nr >= 2 && !out ? (int)p : 0;
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
__device__ __forceinline__ Segment segment_of(const PrefixArgs& a, int v, bool ok, uint32_t* bad) {
  if (v < a.ngroups) return ok ? group_segment(a, v, bad) : Segment{0, 0, 0, 0, 0};
  int g;
  return own_segment(a, v - a.ngroups, shared_segment(a, v - a.ngroups, ok, &g).p1, bad);
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
  int per;               // row tiles of an item at most
  int tile;              // entries of a tile
  int cost, cost2, begin;  // units of a tile with one and with two row tiles, and of an item's beginning
  int copies;            // partials of a row in a portion: 2 where two groups share the tiles of one row tile
  int most;              // rows of a portion at most
  int workers;
  long long *units, *rows;  // [ngroups + R + 1] before each segment, written by the first CTA
  float *part, *ml;      // [rows][dv], [rows][4]: maximum (base 2), sum of rounded weights, of exact ones
};

struct Shape1 {  // a segment's division
  int base, tiles, nmt, np, rows;  // first entry of tile 0; row tiles, items of a head, rows of a portion
  long long item, head;            // units of a full item, of a KV head
};
__device__ __forceinline__ Shape1 shape_of(const PrefixArgs& a, const PrefixSplit& w, const Segment& s) {
  Shape1 x;
  x.base = s.p0 & ~31;
  x.tiles = s.p1 > s.p0 ? (int)(((unsigned)(s.p1 - x.base) + (unsigned)w.tile - 1u) / (unsigned)w.tile) : 0;
  x.nmt = w.flat ? (s.nr * a.Hq + 127) >> 7 : (s.nr + w.MT - 1) / w.MT;
  x.np = (x.nmt + w.per - 1) / w.per;
  x.rows = w.flat ? min(128, s.nr * a.Hq) : w.G * min(s.nr, w.MT) * w.copies;
  x.item = (long long)x.tiles * (w.per == 2 ? w.cost2 : w.cost) + w.begin;
  x.head = w.per == 2 ? (x.nmt >> 1) * x.item + (x.nmt & 1) * ((long long)x.tiles * w.cost + w.begin) : x.np * x.item;
  if (x.tiles == 0) x.head = 0;
  return x;
}
__device__ __forceinline__ long long units_of(const PrefixSplit& w, const Shape1& x) { return x.head * w.heads; }
__device__ __forceinline__ long long rows_of(const PrefixSplit& w, const Shape1& x) {
  return x.tiles == 0 ? 0 : (long long)w.heads * x.np * x.rows;
}
// Tile t of an item belongs to the worker that holds its first unit: tiles from unit u on.
__device__ __forceinline__ int tile_at(long long u, int begin, int cost, int tiles) {
  const long long x = u - begin;
  return x <= 0 ? 0 : (int)min((long long)tiles, Shares::div_small(x + cost - 1, cost));
}

constexpr int kPrefixPortions = 12, kPrefixWindow = 24;

struct PPortion {
  int lead, r0, cnt;    // request whose table is read, first request of the row tiles (flat: first row), requests (rows) in them
  int p0, p1, base;     // positions [p0, p1), tile t begins at base + t * tile
  int t0, t1;
  short head, both;     // both: two row tiles
  short first, own;     // first: group of tile t0 when not both; own: a request's own segment
  int stride;           // rows of a copy of the partials
  long long row;        // first row of the partials
};

struct PrefixPlan {  // shared memory
  PPortion port[kPrefixPortions];
  Segment win[kPrefixWindow];
  long long off, left, rows;  // units into segment cur, units still to take, rows before segment cur
  int cur, nport, turn;       // turn: the group that takes the next single tile
  int ok;                     // the groups' bounds are sound
  long long scan[2][16];
};

// The next portions, by one thread; the window holds the segments from cur on.
__device__ __forceinline__ void prefix_walk(const PrefixArgs& a, const PrefixSplit& w, PrefixPlan* s, int worker) {
  int np = 0, i = 0;
  const int V = a.ngroups + a.R, cur = s->cur;
  long long off = s->off, left = s->left, rows = s->rows;
#pragma unroll 1
  while (left > 0 && np < kPrefixPortions && i < kPrefixWindow && cur + i < V) {
    const Segment sg = s->win[i];
    const Shape1 x = shape_of(a, w, sg);
    if (off >= units_of(w, x)) {
      off -= units_of(w, x);
      rows += rows_of(w, x);
      ++i;
      continue;
    }
    const int head = (int)Shares::div_small(off, x.head);
    const long long in = off - head * x.head;
    const int pair = (int)min((long long)(x.np - 1), Shares::div_small(in, x.item));
    const bool both = w.per == 2 && 2 * pair + 1 < x.nmt;
    const int cost = both ? w.cost2 : w.cost;
    const long long u0 = in - pair * x.item, end = (long long)x.tiles * cost + w.begin, u1 = min(end, u0 + left);
    left -= u1 - u0;
    off += u1 - u0;
    PPortion p;
    p.t0 = tile_at(u0, w.begin, cost, x.tiles);
    p.t1 = tile_at(u1, w.begin, cost, x.tiles);
    if (u1 == end) p.t1 = x.tiles;
    if (p.t0 >= p.t1) continue;  // no tile begins here
    p.lead = sg.lead;
    p.r0 = w.flat ? sg.r0 * a.Hq + 128 * pair : sg.r0 + w.per * pair * w.MT;
    p.cnt = w.flat ? min(128, sg.nr * a.Hq - 128 * pair) : min(w.per * w.MT, sg.nr - w.per * pair * w.MT);
    p.p0 = sg.p0;
    p.p1 = sg.p1;
    p.base = x.base;
    p.head = (short)head;
    p.both = both;
    p.own = cur + i >= a.ngroups;
    p.first = (short)s->turn;
    if (!both) s->turn = (s->turn + p.t1 - p.t0) & 1;
    p.stride = x.rows / w.copies;
    p.row = rows + (long long)(head * x.np + pair) * x.rows + (long long)worker * w.most;
    s->port[np++] = p;
  }
  s->nport = np;
  s->left = cur + i < V ? left : 0;  // lengths that change under the call must not keep it going
  s->off = off;
  s->rows = rows;
  s->cur = cur + i;
}

// The next portions of this worker; false when none are left.  Every thread of the CTA calls it.
__device__ __forceinline__ bool prefix_round(const PrefixArgs& a, const PrefixSplit& w, PrefixPlan* s, int worker) {
  __syncthreads();  // the portions in hand are done with
  if (s->left <= 0) return false;  // the same in every thread: written before a barrier
  const int tid = threadIdx.x;
  if (tid < kPrefixWindow && s->cur + tid < a.ngroups + a.R) {
    uint32_t quiet = 0u;
    s->win[tid] = segment_of(a, s->cur + tid, s->ok != 0, &quiet);
  }
  __syncthreads();
  if (tid == 0) prefix_walk(a, w, s, worker);
  __syncthreads();
  return true;
}

// Where this worker starts, and its first portions; false when there is nothing to do.  Every thread calls it.
__device__ __forceinline__ bool prefix_start(const PrefixArgs& a, const PrefixSplit& w, PrefixPlan* s, int worker) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, V = a.ngroups + a.R;
  const int each = (V + nthr - 1) / nthr, v0 = min(tid * each, V), v1 = min(v0 + each, V);
  const bool ok = __syncthreads_and(bounds_ok(a, tid, nthr)) != 0;
  uint32_t bad = ok ? 0u : (uint32_t)HS_DEVERR_LOC;
  long long mu = 0, mr = 0;  // this thread's units and rows
  for (int v = v0; v < v1; ++v) {
    const Shape1 x = shape_of(a, w, segment_of(a, v, ok, &bad));
    mu += units_of(w, x);
    mr += rows_of(w, x);
  }
  long long iu = mu, ir = mr;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, iu, o), z = __shfl_up_sync(0xffffffffu, ir, o);
    if (lane >= o) {
      iu += y;
      ir += z;
    }
  }
  if (lane == 31) {
    s->scan[0][warp] = iu;
    s->scan[1][warp] = ir;
  }
  __syncthreads();
  long long total = 0, trows = 0, bu = 0, br = 0;
  for (int x = 0; x < (nthr >> 5); ++x) {
    if (x == warp) {
      bu = total;
      br = trows;
    }
    total += s->scan[0][x];
    trows += s->scan[1][x];
  }
  bu += iu - mu;
  br += ir - mr;
  const Shares sh(total, w.workers);
  const long long start = sh.start(worker), left = sh.start(worker + 1) - start;
  if (blockIdx.x == 0) {
    report(a.kv.err, bad);
    if (tid == 0) {
      w.units[V] = total;
      w.rows[V] = trows;
      *a.ok = ok;
    }
  }
  if (tid == 0) {
    s->ok = ok;
    s->left = left;
    s->turn = 0;
  }
  if (blockIdx.x == 0 || (left > 0 && start >= bu && start < bu + mu)) {
    uint32_t quiet = 0u;
    for (int v = v0; v < v1; ++v) {
      long long u = mu, rw = mr;  // one segment a thread: known
      if (each > 1) {
        const Shape1 x = shape_of(a, w, segment_of(a, v, ok, &quiet));
        u = units_of(w, x);
        rw = rows_of(w, x);
      }
      if (blockIdx.x == 0) {
        w.units[v] = bu;
        w.rows[v] = br;
      }
      if (start >= bu && start < bu + u) {
        s->cur = v;
        s->off = start - bu;
        s->rows = br;
      }
      bu += u;
      br += rw;
    }
  }
  return prefix_round(a, w, s, worker);
}

// ---- joining ---------------------------------------------------------------------------------------

constexpr int kPrefixJoinThreads = 128;

// The running sum of a row's partials: 8 of its dims, maximum, sums of rounded and of exact weights.
struct Joined {
  float m = -INFINITY, l = 0.f, le = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(const float* part, const float* ml, long long row, int dv, int d) {
    const float4 s = *(const float4*)(ml + 4 * row);
    const float4 x = *(const float4*)(part + row * dv + d), y = *(const float4*)(part + row * dv + d + 4);
    const float mn = fmaxf(m, s.x);
    // -infinity: nothing seen (sum 0), or NaN scores alone (NaN).  A weight of 0 counts all the same: what the row saw may
    // be infinite or NaN, and what it saw nothing of holds zeros
    const float al = m == mn ? 1.f : exp2f(m - mn), wt = s.x == -INFINITY ? (s.y == 0.f ? 0.f : s.y) : exp2f(s.x - mn);
    m = mn;
    l = l * al + wt * s.y;
    le = le * al + wt * s.z;
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(wt, v[i], acc[i] * al);
  }
  __device__ __forceinline__ void store(const PrefixArgs& a, int r, int h, int d) const {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *(uint4*)(a.out + ((int64_t)r * a.Hq + h) * a.dv + d) =
        make_uint4(pack(acc[0] * inv, acc[1] * inv), pack(acc[2] * inv, acc[3] * inv), pack(acc[4] * inv, acc[5] * inv),
                   pack(acc[6] * inv, acc[7] * inv));
    if (a.stats != nullptr && d == 0) a.stats[(int64_t)r * a.Hq + h] = make_float2(m == -INFINITY ? 0.f : m, le == 0.f ? 0.f : 1.f / le);
  }
};

// A thread holds 8 dims of a (request, query head) row; its partials are those of its own segment and of its group's.
template <int DV>
__global__ void __launch_bounds__(kPrefixJoinThreads) k_prefix_join(const PrefixArgs a, const PrefixSplit w) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int vecs = DV >> 3;
  const int rows = a.Hq * vecs;
  const int at = blockIdx.x * kPrefixJoinThreads + threadIdx.x, r = blockIdx.y;
  if (at >= rows) return;
  const int h = at / vecs, d = 8 * (at - h * vecs), V = a.ngroups + a.R;
  const Shares sh(w.units[V], w.workers);
  int g;
  uint32_t quiet = 0u;
  const Segment shared = shared_segment(a, r, *a.ok != 0, &g), own = own_segment(a, r, shared.p1, &quiet);
  Joined sum;
  const bool live = own.p1 > 0;
#pragma unroll 1
  for (int x = 0; x < 2 && live; ++x) {
    const Segment sg = x == 0 ? own : shared;
    const int v = x == 0 ? a.ngroups + r : g;
    const Shape1 sp = shape_of(a, w, sg);
    if (sp.tiles == 0) continue;
    const int j = r - sg.r0;
    const int flat = j * a.Hq + h, mt = w.flat ? flat >> 7 : j / w.MT;
    const int row = w.flat ? flat & 127 : (j - mt * w.MT) * w.G + h % w.G;
    const int head = w.flat ? 0 : h / w.G, pair = mt / w.per;
    const bool both = w.per == 2 && 2 * pair + 1 < sp.nmt;
    const int cost = both ? w.cost2 : w.cost, stride = sp.rows / w.copies;
    const long long item = w.units[v] + head * sp.head + pair * sp.item, end = (long long)sp.tiles * cost + w.begin;
    const long long base = w.rows[v] + (long long)(head * sp.np + pair) * sp.rows + row;
    const int wf = sh.worker(item + w.begin), wl = sh.worker(item + w.begin + (long long)(sp.tiles - 1) * cost);
#pragma unroll 1
    for (int wk = wf; wk <= wl; ++wk) {
      const long long u0 = sh.start(wk) - item, u1 = sh.start(wk + 1) - item;
      const int t0 = tile_at(u0, w.begin, cost, sp.tiles), t1 = u1 >= end ? sp.tiles : tile_at(u1, w.begin, cost, sp.tiles);
      if (t0 >= t1) continue;
      const long long at_row = base + (long long)wk * w.most;
      if (both) {
        sum.add(w.part, w.ml, at_row + (mt & 1) * stride, DV, d);
      } else {
        sum.add(w.part, w.ml, at_row, DV, d);
        if (w.copies == 2 && t1 - t0 > 1) sum.add(w.part, w.ml, at_row + stride, DV, d);
      }
    }
  }
  sum.store(a, r, h, d);
}

}  // namespace

// ---- host ------------------------------------------------------------------------------------------

// Launch plans of the tensor-core kernels: `rows` of partials, 0: the shape is not theirs.
struct hs_prefix_plan {
  int64_t rows;
};
hs_prefix_plan hs_prefix_gqa_plan(const hs_config* c, int num_sms);
hs_prefix_plan hs_prefix_mla_plan(const hs_config* c, int num_sms);
int hs_prefix_gqa_launch(const hs_config* c, const void* prefix_args, void* units, void* partials, int num_sms, cudaStream_t st);
int hs_prefix_mla_launch(const hs_config* c, const void* prefix_args, void* units, void* partials, int num_sms, cudaStream_t st);

// Tree attention over GQA records on the 5th-generation tensor cores.
//
// Rows of an accumulator are (node, query head of one KV head) pairs: MT = 128 / G nodes of G heads.  Per
// tile of 128 entries S = Q K^T (128 x 128 x D) and O += P V (128 x D x 128), both tcgen05.mma with the
// accumulators in tensor memory; the weights P go back to tensor memory over their scores and enter the
// second product from there, rounded to bf16, as the tensor cores take both operands of a product in one type and V is
// bf16 (2^-8 of a weight at most; the sum that divides is of the rounded ones, so that weights still add up to 1).  Two softmax warpgroups, a thread per row, each with its own S and O:
//   one tile of rows (T <= MT): each group is a worker of its own with its own share of the entries, so
//     that one group's softmax runs beside the other's products;
//   more rows: the groups take two tiles of rows over the same entries, which are loaded once for both.
// Four producer warps fill a ring of K and V tiles (128-byte swizzled): a dense context in boxes of 16 or 32 rows
// by TMA where its pages allow, everything else row by row in 16-byte copies (TMA's gather of four rows measured
// slower: its instructions leave a warp one lane at a time, 75 ns each).
// Device memory bounds it while MT-tiles are few: 64 KB a tile and SM at 6.8 TB/s are 1.46 us, the products
// of one tile of rows 0.54 us at the tensor cores' rate.  Measured: 4 requests x 131072 positions x 16 nodes x 32
// heads 360 us (6.0 TB/s); 16 x 8 nodes over 2048 listed positions 40.8 us (136 MB read, 3.4 TB/s: half of it the
// rows' latency, start and joining of the partials); 8 ragged requests of up to 16384 x 64 nodes 89.9 us (860 TFLOP/s,
// tensor cores active 43%).  There a turn of a group is its products (two times 520 cycles) and what their hand-overs
// take (500 from the value product's end to the scores, 450 from the scores to the other group's turn), 2050 of the 4100
// cycles of a tile, in which its softmax takes 1870.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "hs_tc.cuh"
#include "hs_tree.cuh"

namespace {

constexpr int kTile = 128;
constexpr int kProducers = 4;
// Warps 0-7 are the softmax groups; the others stand where they share a quarter of the SM's issue slots with the
// least: the products' warp (every cycle of it counts) beside warps 3 and 7, which have no rows when there are
// few; the producers in the second and third quarter.  Warps 8 and 12 have nothing to do.
constexpr int kWarpMma = 11, kThreads = 15 * 32;
__device__ __forceinline__ int producer_of(int warp) { return warp == 9 || warp == 10 ? warp - 9 : warp == 13 || warp == 14 ? warp - 11 : -1; }
constexpr int kMaskRing = 8;   // tiles of validity bits per group: more than the ring can run ahead
constexpr float kLazy = 8.f;   // log2 headroom before the running maximum is raised
constexpr size_t kSmemCap = 227 * 1024;

template <int D, bool SHARED>
struct Shape {
  static constexpr int kCh = D / 64;                 // 64-value (128-byte) column blocks
  static constexpr int kBlk = kTile * 128;           // bytes of one block of a tile
  static constexpr int kSlot = kCh * kBlk;           // a K or V tile; also a Q tile
  // How K and V lie: bytes from 8 records to the next 8, and from a 64-value block to the next.  Shared, a group's
  // blocks one after the other, so that one copy brings all blocks of 16 or 32 records: their number is what copies
  // cost there (94 us instead of 100 on 8 ragged requests x 64 nodes in pages of 16).  Unshared, block by block: memory
  // bounds these, and copies of 128-byte rows use it better (357 us instead of 397 on 4 x 131072 positions).
  static constexpr int kGroup = SHARED ? kCh * 1024 : 1024, kBlock = SHARED ? 1024 : kTile * 128;
  static constexpr int kRing = D == 128 ? 5 : 11;
  static constexpr size_t kDyn = (size_t)(2 + kRing) * kSlot + 1024;
};

struct TcArgs {
  TreeArgs a;
  WorkSplit ws;
  int G, MT, np, shared;   // np: row tiles (shared: pairs of them) of a KV head
  int nmt;                 // row tiles of a KV head
  int seg;                 // dense contexts whose pages hold multiples of it: rows per box (32 or 16), else 0
  int negate;              // the scale is negative: qscale is its magnitude, the scores' products are negated
  int ctx_rows;            // rows of the cache: a box that starts there reads zeros
};

struct Control {
  PlanState plan;
  __align__(8) uint64_t full[11], empty[11];
  uint64_t qfull[2], s[2], p[2], pv[2], mask[2][kMaskRing];
  uint64_t fin;
  uint32_t valid[2][kMaskRing][4];
  uint32_t vplace[2][kMaskRing];  // where a tile's values are: ring slot * 2 + phase
  uint32_t tmem, abort;
};

// A number known when compiled, where another call passes an int.
template <int N>
struct Const {
  __device__ __forceinline__ operator int() const { return N; }
};

template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// A place in a portion list, with what is needed of the portion.
struct Cursor {
  const Portion* list;
  int count, p, t, t0, t1;
  bool pairs;                           // shared: both groups take part (the last pair of row tiles may be single)
  __device__ __forceinline__ void fetch(const TcArgs& c) {
    if (p >= count) return;
    const Portion& P = list[p];
    t = t0 = uniform(P.t0);
    t1 = uniform(P.t1);
    pairs = !c.shared || 2 * uniform(P.pair) + 1 < c.nmt;
  }
  __device__ __forceinline__ void open(const Portion* l, int n, const TcArgs& c) {
    list = l;
    count = uniform(n);
    p = 0;
    fetch(c);
  }
  __device__ __forceinline__ bool left() const { return p < count; }
  __device__ __forceinline__ void next(const TcArgs& c) {
    if (++t == t1) {
      ++p;
      fetch(c);
    }
  }
};

template <int D, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1)
    k_tree_gqa(const TcArgs c, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap segmap) {
  using C = Shape<D, SHARED>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Control ct;
  const TreeArgs& a = c.a;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t q_u = smem_u32(smem), ring_u = q_u + 2 * C::kSlot;
  volatile uint32_t* abort = &ct.abort;
  if (tid == 0) {
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(&ct.full[i], kProducers * 32);
      mbar_init(&ct.empty[i], 1u);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&ct.qfull[g], 1u);
      mbar_init(&ct.s[g], 1u);
      mbar_init(&ct.p[g], 128u);
      mbar_init(&ct.pv[g], 1u);
      for (int i = 0; i < kMaskRing; ++i) mbar_init(&ct.mask[g][i], kProducers);
    }
    mbar_init(&ct.fin, 1u);
    ct.abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ct.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 9 && lane == 0) {
    prefetch_map(&qmap);
    if (c.seg != 0) prefetch_map(&segmap);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the only kernel that may start early is this call's own combine, which waits for this one
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  bool go = plan_start<kTile>(a, c.ws, &ct.plan);
  tc_fence_after();
  const uint32_t tb = ct.tmem;
  // tensor memory: 128 columns of scores a group (their first 64 become the weights), then D of O a group

  // state that runs on through the rounds, each used by one role
  Ring<C::kRing> ring;             // producers and products
  int tiles0 = 0, tiles1 = 0;      // producers: tiles of each group loaded; products: finished
  int portions0 = 0, portions1 = 0;  // products: portions of each group begun
  int nt = 0, nm = 0;              // softmax: tiles, tiles of the mask ring
  int sent = 0;                    // producers: ring loads issued; first softmax thread: query loads
  bool ok = true;
  uint32_t bad = 0u;

  for (; go; go = plan_round<kTile>(a, c.ws, &ct.plan)) {
    const int ng = SHARED ? 1 : 2;  // portion lists
    // whether group g takes part in an item: the last pair of row tiles may be a single one
    auto present = [&](int g, const Portion& p) { return !SHARED || 2 * p.pair + g < c.nmt; };
    auto count_of = [&](int g) { return ct.plan.nport[g < ng ? g : 0]; };
    auto list_of = [&](int g) -> const Portion* { return ct.plan.port[g < ng ? g : 0]; };
    // The groups take turns: the products O_g(i) then S_g(i + 1), in the first turn S_g(0) alone; the ring's loads
    // K_g(i), V_g(i).  (Values loaded right behind their keys: the lookups and addresses serve both, and a
    // head's key and value are neighbours in memory.)

    const int pw = producer_of(warp);
    if (pw >= 0) {
      // ---------------- producers: 32 entries of every tile each ----------------
      // lane y looks up entry y of the warp's 32
      const int crow = lane >> 3, cch = lane & 7;
      Lookahead ahead0 = {}, ahead1 = {};  // two variables, never exchanged: a move would wait for a load on its way
      Cursor k0, k1;
      k0.open(list_of(0), count_of(0), c);
      k1.open(list_of(1), ng > 1 ? count_of(1) : 0, c);
      ahead0.at = k0.t;
      ahead1.at = k1.t;
      auto look = [&](Lookahead& l) {
        l.step(a, k0.list, k0.count, kTile, 32 * pw + lane, c.ctx_rows, c.seg == 0 ? 2 * C::kCh : 0, &bad);
      };
      // one tile a turn, the groups by turns: k0 is the group at hand, exchanged with the other after its turn
      int g = 0;
      for (int idle = 0; idle < ng;) {
        ++idle;
        if (k0.left()) {
          idle = 0;
          const Portion& P = k0.list[k0.p];
          // the lookups of the group's next tile follow the copies of this one
#pragma unroll 1
          for (int behind = 0; behind < 2; ++behind) {
            if (g == 0) {
#pragma unroll 1
              for (int x = behind ? 1 : ahead0.begun ? 0 : 3; x > 0; --x) look(ahead0);
              ahead0.begun = true;
            } else {
#pragma unroll 1
              for (int x = behind ? 1 : ahead1.begun ? 0 : 3; x > 0; --x) look(ahead1);
              ahead1.begun = true;
            }
            if (behind) break;
            const uint64_t now = g == 0 ? ahead0.now : ahead1.now;
            const int now_row = g == 0 ? ahead0.row : ahead1.row;
            const bool boxed = c.seg != 0 && k0.t * kTile + 32 * pw + 32 <= P.n;
            const int x0 = P.head * a.kstride;
            uint32_t vplace = 0u;
#pragma unroll 1
            for (int val = 0; val < 2; ++val) {
              vplace = (uint32_t)ring.slot * 2u + ring.phase;
              if (ok) ok = warp_wait_small(&ct.empty[ring.slot], ring.phase ^ 1u, abort);
              if (ok) {
                const uint32_t dst = ring_u + (uint32_t)(ring.slot * C::kSlot + 4 * pw * C::kGroup);
                uint64_t* full = &ct.full[ring.slot];
                if (boxed) {
                  if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(32 * D * 2));
                  else mbar_arrive(full);
                  if (SHARED) {
                    __syncwarp();
                    if (lane % c.seg == 0)
                      tma_load_4d(dst + (uint32_t)((lane >> 3) * C::kGroup), &segmap, 0, 0, (x0 + val * D) >> 6, now_row >> 3, full);
                    __syncwarp();
                  } else {
                    const int box = lane >> 2, row = __shfl_sync(0xffffffffu, now_row, (box * c.seg) & 31);
                    if (box * c.seg < 32 && (lane & 3) < C::kCh)
                      tma_load_2d(dst + (uint32_t)((lane & 3) * C::kBlock + box * c.seg * 128), &segmap, x0 + val * D + 64 * (lane & 3),
                                  row, full);
                  }
                } else {
                  // 16 bytes a lane: rows 4 i .. 4 i + 3, swizzled as the boxes are
                  const int off = 2 * (x0 + val * D) + 16 * cch;
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    const int row = 4 * i + crow;
                    const uint64_t src = __shfl_sync(0xffffffffu, now, row);
                    const uint32_t to = dst + (uint32_t)((row >> 3) * C::kGroup + (row & 7) * 128 + ((cch ^ (row & 7)) << 4)), n = src != 0ull ? 16u : 0u;
                    const uint8_t* from = src != 0ull ? (const uint8_t*)(uintptr_t)src + off : (const uint8_t*)a.q;
#pragma unroll
                    for (int b = 0; b < C::kCh; ++b) cp_async16_zfill(to + b * C::kBlock, src != 0ull ? from + 128 * b : from, n);
                  }
                  cp_async_arrive_noinc(full);
                }
                ++sent;
              }
              ring.next();
            }
            const uint32_t word = __ballot_sync(0xffffffffu, now != 0ull);
            int& n = g == 0 ? tiles0 : tiles1;
            if (ok && lane == 0) {
              ct.valid[g][n % kMaskRing][pw] = word;
              if (pw == 0) ct.vplace[g][n % kMaskRing] = vplace;
              if (!(a.stall != 0 && n == 0 && pw == 1 && blockIdx.x == 0)) mbar_arrive(&ct.mask[g][n % kMaskRing]);
            }
            ++n;
          }
          k0.next(c);
        }
        if (ng > 1) {
          swap_both(k0, k1);
          g ^= 1;
        }
      }
    } else if (warp == kWarpMma) {
      // ---------------- products ----------------
      const uint32_t tu = (uint32_t)uniform((int)tb);
      const uint32_t id_s = umma_idesc_bf16(128, 128, 0, 0) | (c.negate ? kNegateA : 0u), id_o = umma_idesc_bf16(128, D, 0, 1);
      const uint32_t dq0 = (uint32_t)uniform((int)umma_sdesc_lo(q_u, 16)), dk0 = (uint32_t)uniform((int)umma_sdesc_lo(ring_u, 16));
      // V as it lies: blocks of 64 values, 8 entries a group, the value dims contiguous
      const uint32_t dv0 = (uint32_t)uniform((int)umma_sdesc_lo(ring_u, C::kBlock));
      constexpr uint32_t kSlotStep = C::kSlot >> 4, kBlkStep = C::kBlk >> 4;
      // O_g(i): the weights, and the values (shared: the first group's wait for these serves both)
      auto values = [&](auto gc, const Cursor& p, const Ring<C::kRing>& v, int done) {
        const int g = gc;  // a constant or not
        const bool last_user = !SHARED || g == 1 || !p.pairs;
        if (!SHARED || g == 0) {
          if (ok) ok = uniform_wait2(&ct.p[g], (uint32_t)(done & 1), &ct.full[v.slot], v.phase, abort);
          // copies of 16 bytes are generic-proxy writes; the tensor cores read through the async proxy
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        } else if (ok) {
          ok = uniform_wait(&ct.p[g], (uint32_t)(done & 1), abort);
        }
        tc_fence_after();
        if (ok && elect_one()) {
          const uint32_t ts = tu + 128u * g, to = tu + 256u + (uint32_t)(D * g), dv = dv0 + (uint32_t)v.slot * kSlotStep;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            umma_bf16_ta<C::kGroup>(to, ts + 8u * ks, dv + ks * (2 * C::kGroup >> 4), id_o, (p.t != p.t0 || ks != 0) ? 1u : 0u);
          umma_commit(&ct.pv[g]);
          if (last_user) umma_commit(&ct.empty[v.slot]);
        }
        __syncwarp();
      };
      // S_g(i): the keys; and the weights of the tile before share its columns: their product has to be complete
      auto scores = [&](auto gc, const Cursor& k, const Ring<C::kRing>& at, int done, int portions) {
        const int g = gc;  // a constant or not
        const bool last_user = !SHARED || g == 1 || !k.pairs;
        if (ok && k.t == k.t0) ok = uniform_wait(&ct.qfull[g], (uint32_t)(portions & 1), abort);  // this portion's queries
        if (!SHARED || g == 0) {
          if (ok && done > 0)
            ok = uniform_wait2(&ct.full[at.slot], at.phase, &ct.pv[g], (uint32_t)((done - 1) & 1), abort);
          else if (ok)
            ok = uniform_wait(&ct.full[at.slot], at.phase, abort);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // as above
        } else if (ok && done > 0) {
          ok = uniform_wait(&ct.pv[g], (uint32_t)((done - 1) & 1), abort);
        }
        tc_fence_after();
        if (ok && elect_one()) {
          const uint32_t ts = tu + 128u * g, dq = dq0 + (uint32_t)g * kSlotStep, dk = dk0 + (uint32_t)at.slot * kSlotStep;
#pragma unroll
          for (int b = 0; b < C::kCh; ++b)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_bf16_lo<C::kGroup>(ts, dq + b * kBlkStep + 2 * ks, dk + b * (C::kBlock >> 4) + 2 * ks, id_s, (b | ks) != 0 ? 1u : 0u);
          umma_commit(&ct.s[g]);
          if (last_user) umma_commit(&ct.empty[at.slot]);
        }
        __syncwarp();
      };
      // Shared, each group's turn is code of its own (91 us instead of 94 on 8 ragged requests x 64 nodes: exchanging the
      // groups' state took a tenth of a turn); unshared, where memory bounds it, the code is common, as the start counts
      // (40.5 us instead of 41.3 on 16 requests x 8 nodes over 2048 listed rows).
      const Const<0> g0;
      const Const<1> g1;
      Ring<C::kRing> v0, v1;  // where the values of the tile in hand are
      Cursor k0, p0;              // next scores and next values
      k0.open(list_of(0), count_of(0), c);
      p0 = k0;
      bool due0 = false, due1 = false;  // scores done whose values are not
      if (SHARED) {
        while (due0 || k0.left()) {
          const bool more = k0.left();
          const Ring<C::kRing> at = ring;  // where the keys are
          if (more) {
            ring.next();
            v1 = ring;
            ring.next();
          }
          due1 = due0 && p0.pairs;
          if (due0) values(g0, p0, v0, tiles0++);
          const bool first = more && k0.t == k0.t0;
          if (more) scores(g0, k0, at, tiles0, portions0);
          if (due1) values(g1, p0, v0, tiles1++);
          if (more && k0.pairs) scores(g1, k0, at, tiles1, portions1);
          portions0 += first;
          portions1 += first && k0.pairs;
          if (due0) p0.next(c);
          if (more) k0.next(c);
          due0 = more;
          v0 = v1;
        }
      } else {
        // k0, p0, due0 and v0 are those of the group at hand, exchanged with the other's after its turn
        Cursor k1, p1;
        k1.open(list_of(1), count_of(1), c);
        p1 = k1;
        int g = 0;
        for (int idle = 0; idle < 2;) {
          ++idle;
          int done = g == 0 ? tiles0 : tiles1;
          if (due0) {
            idle = 0;
            values(g, p0, v0, done++);
            p0.next(c);
          }
          due0 = k0.left();
          if (due0) {
            idle = 0;
            const Ring<C::kRing> at = ring;
            ring.next();
            v0 = ring;
            ring.next();
            const bool first = k0.t == k0.t0;
            scores(g, k0, at, done, g == 0 ? portions0 : portions1);
            if (g == 0) portions0 += first;
            else portions1 += first;
            k0.next(c);
          }
          if (g == 0) tiles0 = done;
          else tiles1 = done;
          swap_both(k0, k1);
          swap_both(p0, p1);
          swap_both(due0, due1);
          swap_both(v0, v1);
          g ^= 1;
        }
      }
    } else if (warp < 8) {
      // ---------------- softmax: group g, thread = row = TMEM lane ----------------
      // (A warp comes together, by a vote or __syncwarp, behind each branch that its lanes may take apart: accesses to tensor memory
      // are the whole warp's, and nothing else promises that it is whole there.)
      const int g = warp >> 2, row = tid & 127;
      const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t ts = tb + 128u * g + lane_base, to = tb + 256u + (uint32_t)(D * g) + lane_base;
      const int lt = row / c.G, hq = row - lt * c.G;
      auto load_q = [&](const Portion& P) {  // by the group's first thread
        ++sent;
        mbar_arrive_expect_tx(&ct.qfull[g], (uint32_t)(C::kCh * c.G * c.MT * 128));
        const int h = P.head, mt = SHARED ? 2 * P.pair + g : 0;
        for (int b = 0; b < C::kCh; ++b)
          tma_load_4d(q_u + (uint32_t)(g * C::kSlot + b * C::kBlk), &qmap, 64 * b, h * c.G, mt * c.MT, P.r, &ct.qfull[g]);
      };
      const Portion* list = list_of(g);
      const int count = count_of(g);
      auto next_q = [&](int i) {  // the queries of the next portion this group takes part in
        while (i < count && !present(g, list[i])) ++i;
        if (i < count) load_q(list[i]);
      };
      for (int pi = 0; pi < count; ++pi) {
        const Portion P = list[pi];
        if (pi == 0 && row == 0 && ok) next_q(0);
        if (!present(g, P)) {
          nm += P.t1 - P.t0;
          continue;
        }
        const bool both = SHARED && present(1, P);
        const int h = P.head, mt = SHARED ? 2 * P.pair + g : 0, t = mt * c.MT + lt;
        const int n4 = (int)(((unsigned)P.n + 3u) & ~3u);
        const bool row_ok = row < c.G * c.MT && t < P.nn;
        const bool warp_ok = __any_sync(0xffffffffu, row_ok);
        const uint64_t* mw = a.mask + ((int64_t)P.r * a.T + (row_ok ? t : 0)) * a.words;
        const uint64_t mfirst = mw[0];
        float m = -INFINITY, l = 0.f;
        bool dirty = false;  // a node's value is infinite or NaN
        for (int tile = P.t0; tile < P.t1; ++tile) {
          const int j0 = (int)((long long)tile * kTile - n4);  // node of the tile's first entry
          const bool nodes = j0 + kTile > 0;
          if (ok) ok = mbar_wait_small(&ct.s[g], (uint32_t)(nt & 1), abort);
          tc_fence_after();
          if (row == 0 && tile == P.t1 - 1) {  // the last scores of the portion are done: the next one's queries
            if (ok) next_q(pi + 1);
          }
          const int mg = SHARED ? 0 : g;
          if (ok) ok = mbar_wait_small(&ct.mask[mg][nm % kMaskRing], (uint32_t)((nm / kMaskRing) & 1), abort);
          ok = __all_sync(0xffffffffu, ok);
          uint32_t w[4];
          bool full = !nodes;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            w[x] = ct.valid[mg][nm % kMaskRing][x];
            full = full && w[x] == 0xffffffffu;
          }
          if (nodes) {
            // entries that are nodes: valid ones that this row sees
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int jw = j0 + 32 * x;
              const uint32_t ctx = jw >= 0 ? 0u : (jw <= -32 ? 0xffffffffu : (1u << -jw) - 1u);
              w[x] &= ctx | (row_ok ? mask_bits(mw, mfirst, a.words, P.nn, jw) : 0u);
            }
            const uint32_t vp = ct.vplace[mg][nm % kMaskRing];
            if (ok) ok = mbar_wait_small(&ct.full[vp >> 1], vp & 1u, abort);
            ok = __all_sync(0xffffffffu, ok);
            const bool d = ok && clean_rows(smem + (2 + (vp >> 1)) * C::kSlot, C::kBlock, C::kGroup, C::kCh, max(0, -j0),
                                            min(kTile, P.nn - j0), both ? tid : row, both ? 256 : 128);
            if (bar_or(both ? 3 : 1 + g, both ? 256 : 128, d)) dirty = true;
          }
          ++nm;
          ++nt;
          __syncwarp();
          if (ok && warp_ok) {
            // Scores 64 at a time: what a load from tensor memory costs is its wait.
            float mx = -INFINITY, my = -INFINITY;
            float v[64];
            if (!full) mask_scores(ts, w);
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
              tmem_ld64(ts + 64u * x, v);
#pragma unroll
              for (int j = 0; j < 64; j += 4) {
                mx = fmaxf(fmaxf(mx, v[j]), v[j + 1]);
                my = fmaxf(fmaxf(my, v[j + 2]), v[j + 3]);
              }
            }
            mx = fmaxf(mx, my);
            mx *= a.qscale;  // positive: a negative scale is in the products' sign, zero is the smallest number
            const bool raise = mx > m + kLazy;
            if (__any_sync(0xffffffffu, raise)) {
              const float mn = raise ? mx : m;
              const float al = (mn == m || m == -INFINITY) ? 1.f : fast_exp2(m - mn);
              m = mn;
              l *= al;
              __syncwarp();
              if (tile != P.t0) {
#pragma unroll 1
                for (int x = 0; x < D / 32; ++x) {
                  float o[32];
                  tmem_ld32(to + 32u * x, o);
#pragma unroll
                  for (int j = 0; j < 32; ++j) o[j] *= al;
                  tmem_st32(to + 32u * x, o);
                }
              }
            }
            const float base = m == -INFINITY ? 0.f : m;  // nothing seen so far: every weight is 0
            float sum0 = 0.f, sum1 = 0.f;
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
              tmem_ld64(ts + 64u * x, v);
              uint32_t pk[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                float p0, p1;
                fma2(p0, p1, v[2 * j], v[2 * j + 1], a.qscale, -base);
                pk[j] = pack_bf16(fast_exp2(p0), fast_exp2(p1));
                add2(sum0, sum1, lo(pk[j]), hi(pk[j]));  // the rounded weights, as the product takes them
              }
              tmem_st32u(ts + 32u * x, pk);
            }
            l += sum0 + sum1;
            tmem_st_wait();
          }
          tc_fence_before();
          mbar_arrive(&ct.p[g]);
        }
        // the portion's result: complete, or a partial
        if (ok) ok = mbar_wait_small(&ct.pv[g], (uint32_t)((nt - 1) & 1), abort);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        if (ok && warp_ok) {
          const bool whole = P.t0 == 0 && P.t1 == (int)tiles_of<kTile>(P.n, P.nn);
          const int wk = (SHARED ? 0 : g) * (int)gridDim.x + (int)blockIdx.x;
          const long long slot = ((long long)wk * 2 + (P.t0 > 0 ? 0 : 1)) * c.ws.rows;
          const int srow = (SHARED ? 128 * g : 0) + row;
          const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
#pragma unroll 1
          for (int x = 0; x < D / 32; ++x) {
            float o[32];
            __syncwarp();
            tmem_ld32(to + 32u * x, o);
            if (dirty && row_ok) {
              // values left out of the product (they would have reached every row): into the rows that see them
              for (int j = max(0, P.t0 * kTile - n4); j < min((long long)P.nn, (long long)P.t1 * kTile - n4); ++j) {
                if (((mw[j >> 6] >> (j & 63)) & 1ull) == 0ull) continue;
                const uint8_t* rec = node_record(a, P.r, P.len, j, &bad);
                if (rec == nullptr) continue;
                const uint32_t* vr = (const uint32_t*)rec + ((int64_t)h * a.kstride + a.voff + 32 * x) / 2;
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                  const uint32_t u = vr[y];
                  if ((u & 0x7f80u) == 0x7f80u) o[2 * y] += lo(u);
                  if ((u & 0x7f800000u) == 0x7f800000u) o[2 * y + 1] += hi(u);
                }
              }
            }
            if (row_ok) {
              if (whole) {
                uint4* dst = (uint4*)(a.out + (((int64_t)P.r * a.T + t) * a.Hq + (int64_t)h * c.G + hq) * D + 32 * x);
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  dst[y] = make_uint4(pack_bf16(o[8 * y] * inv, o[8 * y + 1] * inv), pack_bf16(o[8 * y + 2] * inv, o[8 * y + 3] * inv),
                                      pack_bf16(o[8 * y + 4] * inv, o[8 * y + 5] * inv), pack_bf16(o[8 * y + 6] * inv, o[8 * y + 7] * inv));
              } else {
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  st_global_v8(c.ws.part + slot * D + ((long long)(4 * x + y) * c.ws.rows + srow) * 8, o + 8 * y);
              }
            }
          }
          if (row_ok && !whole) *(float2*)(c.ws.ml + (slot + srow) * 2) = make_float2(m, l);
        }
        tc_fence_before();
        __syncwarp();
      }
    }
    if (!ok) *abort = 1u;
    __syncwarp();
  }
  if (!ok) {
    *abort = 1u;
    if (lane == 0) report(a.kv.err, (uint32_t)HS_DEVERR_TIMEOUT);
  }
  report(a.kv.err, bad);
  // after a wait that gave up, copies and products may still be in flight: they end before the CTA does
  volatile uint32_t never = 0u;
  if (warp == kWarpMma) {
    if (elect_one()) umma_commit(&ct.fin);  // by the thread whose products they are
    __syncwarp();
    warp_wait(&ct.fin, 0u, &never);
  }
  __syncthreads();
  if (producer_of(warp) >= 0) asm volatile("cp.async.wait_all;" ::: "memory");
  if (*abort != 0u && lane == 0) {
    const uint64_t t0 = global_ns();
    if (producer_of(warp) >= 0) {
#pragma unroll 1
      for (int i = max(0, sent - C::kRing); i < sent; ++i)
        while (!mbar_try_wait(&ct.full[i % C::kRing], (uint32_t)((i / C::kRing) & 1)) && global_ns() - t0 < 1000000000ull) {
        }
    } else if ((warp & 3) == 0 && warp < 8 && sent > 0) {
      while (!mbar_try_wait(&ct.qfull[warp >> 2], (uint32_t)((sent - 1) & 1)) && global_ns() - t0 < 1000000000ull) {
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  tc_fence_after();
  if (warp == kWarpMma) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tb) : "memory");
}

// ---- host ------------------------------------------------------------------------------------------

struct Plan {
  int D, G, MT, nmt, shared, np, items, rows, workers;
};

bool plan_of(const hs_config* c, int T, int sms, Plan* p) {
  if (c->layout != HS_LAYOUT_GQA || c->head_dim_qk != c->head_dim_v) return false;
  if (c->head_dim_qk != 64 && c->head_dim_qk != 128) return false;
  p->D = c->head_dim_qk;
  p->G = c->num_q_heads / c->num_kv_heads;
  if (p->G > 128) return false;
  p->MT = 128 / p->G < T ? 128 / p->G : T;
  p->nmt = (T + p->MT - 1) / p->MT;
  p->shared = p->nmt > 1;
  p->np = p->shared ? (p->nmt + 1) / 2 : 1;
  p->items = c->num_kv_heads * p->np;
  p->rows = p->shared ? 256 : p->G * p->MT;
  p->workers = p->shared ? sms : 2 * sms;
  return true;
}

template <int D, bool SHARED>
cudaError_t launch(const TcArgs& c, const Plan& p, int sms, const CUtensorMap& q, const CUtensorMap& seg, const CombineArgs& cb,
                   cudaStream_t st) {
  static_assert(Shape<D, SHARED>::kDyn + sizeof(Control) <= kSmemCap, "shared memory of a CTA");
  static bool done[64];
  cudaError_t e = allow_smem(k_tree_gqa<D, SHARED>, Shape<D, SHARED>::kDyn, done);
  if (e != cudaSuccess) return e;
  e = hs_launch_pdl(k_tree_gqa<D, SHARED>, dim3(sms), dim3(kThreads), Shape<D, SHARED>::kDyn, st, c, q, seg);
  if (e != cudaSuccess) return e;
  return launch_combine<D>(cb, st);
}

}  // namespace

hs_tree_plan hs_tree_gqa_plan(const hs_config* c, int nodes, int num_sms) {
  Plan p;
  hs_tree_plan r = {plan_of(c, nodes, num_sms, &p), 0};
  if (r.usable) r.workspace = hs_tree_workspace_bytes(c, p.workers, p.rows, p.D);
  return r;
}

int hs_tree_gqa_launch(const hs_config* cfg, const hs_tree_args* g, const void* tree_args, int num_sms, cudaStream_t st) {
  Plan p;
  if (!plan_of(cfg, g->nodes, num_sms, &p)) return HS_ERR_CONFIG;
  TcArgs c{};
  c.a = *(const TreeArgs*)tree_args;
  c.G = p.G;
  c.MT = p.MT;
  c.np = p.np;
  c.shared = p.shared;
  c.nmt = p.nmt;
  c.ws.items = p.items;
  c.ws.np = p.np;
  c.ws.groups = p.shared ? 1 : 2;
  // unshared, the other group works while one changes its portion: 40.2, 41.7 and 43.3 us with 0 to 2 on 16 requests
  // x 8 nodes over 2048 listed rows; shared, 98.6, 96.3, 94.3 and 95.8 us with 0 to 3 on 8 ragged requests x 64 nodes
  c.ws.begin = p.shared ? 2 : 0;
  c.ws.rows = p.rows;
  hs_tree_workspace(g->d_workspace, cfg, p.workers, p.rows, p.D, &c.ws.prefix, &c.ws.part, &c.ws.ml);
  if (c.a.qscale < 0.f) {
    c.negate = 1;
    c.a.qscale = -c.a.qscale;
  }
  c.a.qscale = fmaxf(c.a.qscale, 1.17549435e-38f);  // times -infinity has to stay -infinity
  CUtensorMap qm, seg;
  memset(&seg, 0, sizeof(seg));
  if (c.a.slot_pt == nullptr && c.a.locs == nullptr) {
    const int pt = c.a.kv.page_tokens;
    c.seg = pt % 32 == 0 ? 32 : pt % 16 == 0 ? 16 : 0;
    c.ctx_rows = (int)(c.a.kv.num_pages * pt);
    // unshared: value, record; shared: value, record of a group, block, group
    const cuuint64_t rec = (cuuint64_t)c.a.kv.rec, size[2] = {rec / 2, (cuuint64_t)c.ctx_rows}, stride[1] = {rec};
    const cuuint64_t size4[4] = {64, 8, rec / 128, (cuuint64_t)c.ctx_rows / 8}, stride4[3] = {rec, 128, 8 * rec};
    const cuuint32_t box[2] = {64, (cuuint32_t)c.seg}, box4[4] = {64, 8, (cuuint32_t)p.D / 64, (cuuint32_t)c.seg / 8};
    if (c.seg != 0 && !(p.shared ? encode(&seg, c.a.kv.base, 4, size4, stride4, box4) : encode(&seg, c.a.kv.base, 2, size, stride, box)))
      c.seg = 0;
  }
  const cuuint64_t row = (cuuint64_t)p.D * 2;
  const cuuint64_t qsize[4] = {(cuuint64_t)p.D, (cuuint64_t)cfg->num_q_heads, (cuuint64_t)g->nodes, (cuuint64_t)cfg->num_requests};
  const cuuint64_t qstride[3] = {row, row * cfg->num_q_heads, row * cfg->num_q_heads * g->nodes};
  const cuuint32_t qbox[4] = {64, (cuuint32_t)p.G, (cuuint32_t)p.MT, 1};
  if (!encode(&qm, c.a.q, 4, qsize, qstride, qbox)) return HS_ERR_CUDA;
  CombineArgs cb{};
  cb.nodes = c.a.nodes;
  cb.out = c.a.out;
  cb.ws = c.ws;
  cb.R = c.a.R;
  cb.T = c.a.T;
  cb.Hq = c.a.Hq;
  cb.workers = p.workers;
  cb.G = p.G;
  cb.MT = p.MT;
  cb.per = p.shared ? 2 : 1;
  cb.np = p.np;
  const auto run = p.D == 128 ? (p.shared ? launch<128, true> : launch<128, false>) : (p.shared ? launch<64, true> : launch<64, false>);
  const cudaError_t e = run(c, p, num_sms, qm, seg, cb, st);
  return e == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

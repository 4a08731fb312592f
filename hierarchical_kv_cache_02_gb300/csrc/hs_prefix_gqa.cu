// Attention of one new token a request over GQA records, shared prefixes read once for 2 MT requests, on the 5th-generation tensor cores.
//
// Rows of an accumulator are (request, query head of one KV head) pairs: MT = 128 / G requests of G heads for a prefix, one
// request's G heads for what it has for itself.  Per tile of 128 entries S = Q K^T (128 x 128 x D) and O += P V (128 x D x 128),
// both tcgen05.mma with the accumulators in tensor memory; the weights P go back to tensor memory over their scores and enter the
// second product from there, rounded to bf16, as both operands of a product have one type and V is bf16 (2^-8 of a weight at
// most; the sum that divides is of the rounded ones, so that weights still add up to 1).  Two softmax warpgroups, a thread per
// row, each with its own S and O:
//   two row tiles: the groups take one each over the same entries, which are loaded once for both;
//   one row tile: the groups take its tiles of entries by turns, so that one's softmax runs beside the other's products.
// Four producer warps fill a ring of K and V tiles (128-byte swizzled): in boxes of 16 or 32 records by TMA where the pages
// allow, at a segment's ends and everywhere else record by record in 16-byte copies.
// Device memory bounds it while row tiles are few: 64 KB a tile and SM at 6.8 TB/s are 1.46 us, the products of one row tile
// 0.56 us at the tensor cores' rate.  With two row tiles it is each group's chain: softmax 1770 cycles, of which the powers are 1030 (8
// a number), then 1690 until the next scores are there (P's arrival to the value product's issue 250, the products 530 each).
// 16 requests over 32768 shared positions (32 / 8 heads of 128): 50 us, 4.2 TB/s; 64 over 131072: 149 us, 4.6 TB/s and 0.9 PFLOP/s.
// What was slower: two threads a row (54 and 177 us: 16 warps, the halves' maxima exchanged); a part of the powers as polynomials; the
// weights handed over in two parts (no gain); scores 64 entries at a time (200).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "hs_prefix.cuh"

namespace {

constexpr int kTile = 128;
constexpr int kProducers = 4;
// Warps 0-7 are the softmax groups; the products' warp stands beside warps 3 and 7, which have no rows when there are few, the
// producers and the warp that finds the portions in the first three quarters of the SM.  Warp 12 has nothing to do.
constexpr int kWarpMma = 11, kWarpPlan = 8, kThreads = 15 * 32;
__device__ __forceinline__ int producer_of(int warp) { return warp == 9 || warp == 10 ? warp - 9 : warp == 13 || warp == 14 ? warp - 11 : -1; }
constexpr int kMaskRing = 8;   // tiles of validity bits: more than the ring can run ahead
constexpr float kLazy = 8.f;   // log2 headroom before the running maximum is raised
constexpr size_t kSmemCap = 227 * 1024;

template <int D>
struct Shape {
  static constexpr int kCh = D / 64;                 // 64-value (128-byte) column blocks
  static constexpr int kBlk = kTile * 128;           // bytes of one block of a tile
  static constexpr int kSlot = kCh * kBlk;           // a K or V tile; also a Q tile
  static constexpr int kRing = D == 128 ? 5 : 11;
  static constexpr size_t kDyn = (size_t)(2 + kRing) * kSlot + 1024;
};

struct GqaArgs {
  PrefixArgs a;
  PrefixSplit w;
  int seg;       // pages that hold multiples of it: records per box (32 or 16), else 0
  int negate;    // the scale is negative: qscale is its magnitude, the scores' products are negated
  int ctx_rows;  // rows of the cache: a box that starts there reads zeros
};

struct Control {
  PrefixPlan plan;
  __align__(8) uint64_t full[11], empty[11];
  uint64_t qfull[2], s[2], p[2], pv[2], mask[kMaskRing];
  uint64_t fin;
  uint32_t valid[kMaskRing][4];
  uint32_t tmem, abort;
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

// W: the scores of requests' own positions are kept, and the exact sums of weights.
template <int D, bool W>
__global__ void __launch_bounds__(kThreads, 1)
    k_prefix_gqa(const __grid_constant__ GqaArgs c, const __grid_constant__ CUtensorMap qmany, const __grid_constant__ CUtensorMap qone,
                 const __grid_constant__ CUtensorMap segmap) {
  using C = Shape<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Control ct;
  const PrefixArgs& a = c.a;
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
    }
    for (int i = 0; i < kMaskRing; ++i) mbar_init(&ct.mask[i], kProducers + (i == 0 ? a.stall : 0));
    mbar_init(&ct.fin, 1u);
    prefix_plan_init(&ct.plan, kProducers + 1 + 8);
    ct.abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ct.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 9 && lane == 0) {
    prefetch_map(&qmany);
    prefetch_map(&qone);
    if (c.seg != 0) prefetch_map(&segmap);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the only kernel that may start early is this call's own join, which waits for this one
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  prefix_start(a, c.w, &ct.plan, (int)blockIdx.x);
  tc_fence_after();
  const uint32_t tb = ct.tmem;
  // tensor memory: 128 columns of scores a group (their first 64 become the weights), then D of O a group

  int sent = 0;  // producers: ring loads issued; first softmax thread: query loads
  bool ok = true;
  uint32_t bad = 0u;
  PrefixPlan* plan = &ct.plan;

  {
    const int pw = producer_of(warp);
    if (pw >= 0) {
      // ---------------- producers: 32 entries of every tile each, a lane's lookup of one ----------------
      const int crow = lane >> 3, cch = lane & 7;
      Ring<C::kRing> ring;
      int tiles = 0;               // loaded
      int page = 0, at = -1;       // the next tile's entry: its page, looked at only when it is used, and place in it (-1: nothing seen)
      PPortion L = portion_take(plan, 0, false, &ok, abort);  // the lookups' portion, a tile ahead of the copies
      int nl = 0, lt = L.t0;
      auto look = [&]() {
        at = -1;
        if (L.t0 == L.t1) return;
        const int p = L.base + lt * kTile + 32 * pw + lane;
        if (p >= L.p0 && p < L.p1) {
          const unsigned pg = (unsigned)p / (unsigned)a.kv.page_tokens;
          at = p - (int)(pg * (unsigned)a.kv.page_tokens);
          page = a.kv.table != nullptr ? a.kv.table[(int64_t)L.lead * a.kv.max_pages + pg] : L.lead * a.kv.max_pages + (int)pg;
        }
        if (++lt == L.t1) {
          L = portion_take(plan, ++nl, false, &ok, abort);
          lt = L.t0;
        }
      };
      PPortion P = L;
      look();
#pragma unroll 1
      for (int pi = 0; P.t0 < P.t1; ++pi) {
        if (lane == 0) mbar_arrive(&plan->empty[pi % kPrefixRing]);  // the lookups took it before
        const int x0 = P.head * a.kstride;
#pragma unroll 1
        for (int t = P.t0; t < P.t1; ++t, ++tiles) {
          const bool seen = at >= 0 && (unsigned)page < (unsigned)a.kv.num_pages;
          if (at >= 0 && !seen) bad |= (uint32_t)HS_DEVERR_PAGE;
          const int row = seen ? page * a.kv.page_tokens + at : c.ctx_rows;
          const int e0 = P.base + t * kTile + 32 * pw;
          const bool boxed = c.seg != 0 && e0 >= P.p0 && e0 + 32 <= P.p1;
          look();
#pragma unroll 1
          for (int val = 0; val < 2; ++val) {
            if (ok) ok = warp_wait_small(&ct.empty[ring.slot], ring.phase ^ 1u, abort);
            if (ok) {
              const uint32_t dst = ring_u + (uint32_t)(ring.slot * C::kSlot + 4 * pw * 1024);
              uint64_t* full = &ct.full[ring.slot];
              if (boxed) {
                if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(32 * D * 2));
                else mbar_arrive(full);
                __syncwarp();
                const int box = lane >> 2, brow = __shfl_sync(0xffffffffu, row, (box * c.seg) & 31);
                if (box * c.seg < 32 && (lane & 3) < C::kCh)
                  tma_load_2d(dst + (uint32_t)((lane & 3) * C::kBlk + box * c.seg * 128), &segmap, x0 + val * D + 64 * (lane & 3), brow, full);
                __syncwarp();
              } else {
                // 16 bytes a lane: rows 4 i .. 4 i + 3, swizzled as the boxes are
                const int off = 2 * (x0 + val * D) + 16 * cch;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const int y = 4 * i + crow, src = __shfl_sync(0xffffffffu, seen ? row : -1, y);
                  const uint32_t to = dst + (uint32_t)(y * 128 + ((cch ^ (y & 7)) << 4)), n = src >= 0 ? 16u : 0u;
                  const uint8_t* from = src >= 0 ? a.kv.base + (int64_t)src * a.kv.rec + off : (const uint8_t*)a.q;
#pragma unroll
                  for (int b = 0; b < C::kCh; ++b) cp_async16_zfill(to + b * C::kBlk, src >= 0 ? from + 128 * b : from, n);
                }
                cp_async_arrive_noinc(full);
              }
              ++sent;
            }
            ring.next();
          }
          const uint32_t word = __ballot_sync(0xffffffffu, seen);
          if (ok && lane == 0) {
            ct.valid[tiles % kMaskRing][pw] = word;
            mbar_arrive(&ct.mask[tiles % kMaskRing]);
          }
        }
        P = portion_take(plan, pi + 1, false, &ok, abort);
      }
    } else if (warp == kWarpMma) {
      // ---------------- products ----------------
      const uint32_t tu = (uint32_t)uniform((int)tb);
      const uint32_t id_s = umma_idesc_bf16(128, 128, 0, 0) | (c.negate ? kNegateA : 0u), id_o = umma_idesc_bf16(128, D, 0, 1);
      const uint32_t dq0 = (uint32_t)uniform((int)umma_sdesc_lo(q_u, 16)), dk0 = (uint32_t)uniform((int)umma_sdesc_lo(ring_u, 16));
      // V as it lies: blocks of 64 values, 8 entries a group, the value dims contiguous
      const uint32_t dv0 = (uint32_t)uniform((int)umma_sdesc_lo(ring_u, C::kBlk));
      constexpr uint32_t kSlotStep = C::kSlot >> 4, kBlkStep = C::kBlk >> 4;
      // O_g of its last task: the weights, and the values
      auto values = [&](int g, int slot, uint32_t phase, bool first, bool last, int done) {
        if (ok) ok = uniform_wait2(&ct.p[g], (uint32_t)(done & 1), &ct.full[slot], phase, abort);
        // copies of 16 bytes are generic-proxy writes; the tensor cores read through the async proxy
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_after();
        if (ok && elect_one()) {
          const uint32_t ts = tu + 128u * g, to = tu + 256u + (uint32_t)(D * g), dv = dv0 + (uint32_t)slot * kSlotStep;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) umma_bf16_ta(to, ts + 8u * ks, dv + ks * (2048 >> 4), id_o, (!first || ks != 0) ? 1u : 0u);
          umma_commit(&ct.pv[g]);
          if (last) umma_commit(&ct.empty[slot]);
        }
        __syncwarp();
      };
      // S_g of its next task: the keys; and the weights of the task before share its columns: their product has to be complete
      auto scores = [&](int g, const Ring<C::kRing>& at, bool first, bool last, int done, int portions) {
        if (ok && first) ok = uniform_wait(&ct.qfull[g], (uint32_t)(portions & 1), abort);  // this portion's queries
        if (ok && done > 0)
          ok = uniform_wait2(&ct.full[at.slot], at.phase, &ct.pv[g], (uint32_t)((done - 1) & 1), abort);
        else if (ok)
          ok = uniform_wait(&ct.full[at.slot], at.phase, abort);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // as above
        tc_fence_after();
        if (ok && elect_one()) {
          const uint32_t ts = tu + 128u * g, dq = dq0 + (uint32_t)g * kSlotStep, dk = dk0 + (uint32_t)at.slot * kSlotStep;
#pragma unroll
          for (int b = 0; b < C::kCh; ++b)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_bf16_lo(ts, dq + b * kBlkStep + 2 * ks, dk + b * kBlkStep + 2 * ks, id_s, (b | ks) != 0 ? 1u : 0u);
          umma_commit(&ct.s[g]);
          if (last) umma_commit(&ct.empty[at.slot]);
        }
        __syncwarp();
      };
      Ring<C::kRing> ring;
      int done0 = 0, done1 = 0;    // tasks of each group whose values were issued
      int begun0 = 0, begun1 = 0;  // portions of each group begun
      // a group's task whose values are due, and where they are; two that are at one place share them
      bool due0 = false, due1 = false;
      int vslot0 = 0, vslot1 = 0;
      uint32_t vphase0 = 0u, vphase1 = 0u;
      bool vfirst0 = false, vfirst1 = false;
#pragma unroll 1
      for (int pi = 0;; ++pi) {
        const PPortion P = portion_take(plan, pi, true, &ok, abort);
        const int t0 = uniform(P.t0), t1 = uniform(P.t1), both = uniform(P.both), first = uniform(P.first);
        if (t0 == t1) break;
#pragma unroll 1
        for (int t = t0; t < t1; ++t) {
          const Ring<C::kRing> k = ring;  // where the keys are
          ring.next();
          const Ring<C::kRing> v = ring;
          ring.next();
          const int turn = (first + t - t0) & 1;
          if (both || turn == 0) {
            const bool one = both ? t == t0 : t - t0 < 2;  // the group's first task of the portion
            if (due0) values(0, vslot0, vphase0, vfirst0, !(due1 && vslot1 == vslot0), done0++);
            scores(0, k, one, !both, done0, begun0);
            begun0 += one;
            due0 = true;
            vslot0 = v.slot;
            vphase0 = v.phase;
            vfirst0 = one;
          }
          if (both || turn == 1) {
            const bool one = both ? t == t0 : t - t0 < 2;
            if (due1) values(1, vslot1, vphase1, vfirst1, !(due0 && vslot0 == vslot1), done1++);
            scores(1, k, one, true, done1, begun1);
            begun1 += one;
            due1 = true;
            vslot1 = v.slot;
            vphase1 = v.phase;
            vfirst1 = one;
          }
        }
      }
      if (due0) values(0, vslot0, vphase0, vfirst0, !(due1 && vslot1 == vslot0), done0++);
      if (due1) values(1, vslot1, vphase1, vfirst1, true, done1++);
    } else if (warp < 8) {
      // ---------------- softmax: group g, thread = row = TMEM lane ----------------
      // (A warp comes together, by a vote or __syncwarp, behind each branch that its lanes may take apart: accesses to tensor memory
      // are the whole warp's, and nothing else promises that it is whole there.)
      const int g = warp >> 2, row = tid & 127;
      const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t ts = tb + 128u * g + lane_base, to = tb + 256u + (uint32_t)(D * g) + lane_base;
      const int lr = row / c.w.G, hq = row - lr * c.w.G;
      auto takes = [&](const PPortion& P) { return P.both || P.first == g || P.t1 - P.t0 > 1; };
      int tiles = 0, done = 0;  // tiles so far, tasks of this group
      auto next_q = [&](int i) {  // the queries of the next portion this group takes part in, by the group's first thread
        for (;; ++i) {
          if (!portion_wait(plan, i, abort)) return;
          const PPortion& P = portion_at(plan, i);
          if (P.t0 == P.t1) return;
          if (!takes(P)) continue;
          ++sent;
          mbar_arrive_expect_tx(&ct.qfull[g], (uint32_t)(C::kCh * c.w.G * (P.own ? 1 : c.w.MT) * 128));
          const int r0 = P.r0 + (P.both && g == 1 ? c.w.MT : 0);
          for (int b = 0; b < C::kCh; ++b)
            tma_load_4d(q_u + (uint32_t)(g * C::kSlot + b * C::kBlk), P.own ? &qone : &qmany, 64 * b, P.head * c.w.G, r0, 0, &ct.qfull[g]);
          return;
        }
      };
      if (row == 0) next_q(0);
      __syncwarp();
#pragma unroll 1
      for (int pi = 0;; ++pi) {
        const PPortion P = portion_take(plan, pi, true, &ok, abort);
        if (P.t0 == P.t1) break;
        if (!takes(P)) {
          tiles += P.t1 - P.t0;
          continue;
        }
        const int off = P.both ? 0 : (g - P.first) & 1, step = P.both ? 1 : 2;  // this group's tiles: t0 + off, then every step-th
        const int cnt = P.both && g == 1 ? P.cnt - c.w.MT : min(P.cnt, c.w.MT);
        const bool row_ok = row < c.w.G * cnt;
        const bool warp_ok = __any_sync(0xffffffffu, row_ok);
        float m = -INFINITY, l = 0.f, le = 0.f;
        for (int tile = P.t0 + off; tile < P.t1; tile += step) {
          const int nm = tiles + tile - P.t0;
          if (ok) ok = mbar_wait2(&ct.s[g], (uint32_t)(done & 1), &ct.mask[nm % kMaskRing], (uint32_t)((nm / kMaskRing) & 1), abort);
          tc_fence_after();
          if (row == 0 && tile + step >= P.t1) {  // the last scores of the portion are done: the next one's queries
            if (ok) next_q(pi + 1);
          }
          ok = __all_sync(0xffffffffu, ok);
          ++done;
          __syncwarp();
          if (ok && warp_ok) {
            uint32_t w[4];
            bool full = true;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              w[x] = ct.valid[nm % kMaskRing][x];
              full = full && w[x] == 0xffffffffu;
            }
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
              le *= al;
              __syncwarp();
              if (tile != P.t0 + off) {
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
            float sum0 = 0.f, sum1 = 0.f, exact0 = 0.f, exact1 = 0.f;
            float* keep = nullptr;
            if (W && P.own && row_ok)
              keep = a.scores + ((int64_t)P.r0 * a.Hq + P.head * c.w.G + hq) * a.score_cols + P.base + tile * kTile;
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
              tmem_ld64(ts + 64u * x, v);
              uint32_t pk[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                float p0, p1;
                fma2(p0, p1, v[2 * j], v[2 * j + 1], a.qscale, -base);
                p0 = fast_exp2(p0);
                p1 = fast_exp2(p1);
                pk[j] = pack_bf16(p0, p1);
                add2(sum0, sum1, lo(pk[j]), hi(pk[j]));  // the rounded weights, as the product takes them
                if (W) add2(exact0, exact1, p0, p1);
              }
              tmem_st32u(ts + 32u * x, pk);
              if (W && keep != nullptr) {
#pragma unroll
                for (int j = 0; j < 64; ++j) v[j] *= a.qscale;
#pragma unroll
                for (int j = 0; j < 64; j += 8) st_global_v8(keep + 64 * x + j, v + j);
              }
              if (W) __syncwarp();
            }
            l += sum0 + sum1;
            le += exact0 + exact1;
            tmem_st_wait();
          }
          tc_fence_before();
          mbar_arrive(&ct.p[g]);
        }
        // the portion's partial sums
        if (ok) ok = mbar_wait_small(&ct.pv[g], (uint32_t)((done - 1) & 1), abort);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        if (ok && warp_ok) {
          const long long first = P.row + (long long)(P.both ? g : off) * P.stride;  // of this copy
#pragma unroll 1
          for (int x = 0; x < D / 32; ++x) {
            float o[32];
            __syncwarp();
            tmem_ld32(to + 32u * x, o);
            if (row_ok) {
#pragma unroll
              for (int y = 0; y < 4; ++y) st_global_v8(c.w.part + first * D + ((4 * x + y) * P.stride + row) * 8, o + 8 * y);
            }
          }
          if (row_ok) *(float4*)(c.w.ml + 4 * (first + row)) = make_float4(m, l, le, 0.f);
        }
        tiles += P.t1 - P.t0;
        tc_fence_before();
        __syncwarp();
      }
    } else if (warp == kWarpPlan) {
      prefix_walk(a, c.w, plan, (int)blockIdx.x, abort);
    }
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

bool split_of(const hs_config* c, int sms, PrefixSplit* w) {
  if (c->layout != HS_LAYOUT_GQA || c->head_dim_qk != c->head_dim_v) return false;
  if (c->head_dim_qk != 64 && c->head_dim_qk != 128) return false;
  const int G = c->num_q_heads / c->num_kv_heads;
  if (G > 128) return false;
  w->heads = c->num_kv_heads;
  w->flat = 0;
  w->G = G;
  w->MT = 128 / G < c->num_requests ? 128 / G : c->num_requests;
  w->mt = div_by(w->MT);
  w->pairs = 1;
  w->tile_shift = 7;
  w->cost = div_by(4);
  w->cost2 = div_by(6);
  w->begin = 5;  // measured on heads of 128 alone: 151.7 us for 64 requests over 131072 with 3, 148.3 with 5, 152.3 with 8
  w->copies = 2;
  w->most = 256;
  w->group_rows = 3 * c->num_q_heads;
  w->together = G;
  w->workers = sms;
  return true;
}

template <int D, bool W>
cudaError_t launch(const GqaArgs& c, const CUtensorMap& qm, const CUtensorMap& q1, const CUtensorMap& seg, cudaStream_t st) {
  static_assert(Shape<D>::kDyn + sizeof(Control) <= kSmemCap, "shared memory of a CTA");
  static bool done[64];
  cudaError_t e = allow_smem(k_prefix_gqa<D, W>, Shape<D>::kDyn, done);
  if (e != cudaSuccess) return e;
  e = hs_launch_pdl(k_prefix_gqa<D, W>, dim3(c.w.workers), dim3(kThreads), Shape<D>::kDyn, st, c, qm, q1, seg);
  if (e != cudaSuccess) return e;
  return launch_join<D>(c.a, c.w, st);
}

}  // namespace

// Rows of partials: a request's own segment takes 2 Hq of them; a group of n requests 2 Hq min(n, MT) for every two row tiles, of
// which there are at most n / (2 MT) + 1, so at most 3 Hq n; and what keeps the workers' apart.
hs_prefix_plan hs_prefix_gqa_plan(const hs_config* c, int num_sms) {
  PrefixSplit w;
  if (!split_of(c, num_sms, &w)) return {0};
  return {(w.group_rows + 2ll * c->num_q_heads) * c->num_requests + (int64_t)w.workers * w.most};
}

int hs_prefix_gqa_launch(const hs_config* cfg, const void* prefix_args, void* head, void* partials, int num_sms, cudaStream_t st) {
  GqaArgs c{};
  c.a = *(const PrefixArgs*)prefix_args;
  if (!split_of(cfg, num_sms, &c.w)) return HS_ERR_CONFIG;
  const int D = c.a.dqk;
  hs_prefix_head(head, c.a.ngroups, &c.w);
  c.w.part = (float*)partials;
  c.w.ml = c.w.part + hs_prefix_gqa_plan(cfg, num_sms).rows * D;
  if (c.a.qscale < 0.f) {
    c.negate = 1;
    c.a.qscale = -c.a.qscale;
  }
  c.a.qscale = fmaxf(c.a.qscale, 1.17549435e-38f);  // times -infinity has to stay -infinity
  CUtensorMap qm, q1, seg;
  memset(&seg, 0, sizeof(seg));
  const int pt = c.a.kv.page_tokens;
  c.seg = pt % 32 == 0 ? 32 : pt % 16 == 0 ? 16 : 0;
  c.ctx_rows = (int)(c.a.kv.num_pages * pt);
  const cuuint64_t rec = (cuuint64_t)c.a.kv.rec, size[2] = {rec / 2, (cuuint64_t)c.ctx_rows}, stride[1] = {rec};
  const cuuint32_t box[2] = {64, (cuuint32_t)c.seg};
  if (c.seg != 0 && !encode(&seg, c.a.kv.base, 2, size, stride, box)) c.seg = 0;
  const cuuint64_t row = (cuuint64_t)D * 2;
  const cuuint64_t qsize[4] = {(cuuint64_t)D, (cuuint64_t)c.a.Hq, (cuuint64_t)c.a.R, 1};
  const cuuint64_t qstride[3] = {row, row * c.a.Hq, row * c.a.Hq * c.a.R};
  const cuuint32_t box_many[4] = {64, (cuuint32_t)c.w.G, (cuuint32_t)c.w.MT, 1}, box_one[4] = {64, (cuuint32_t)c.w.G, 1, 1};
  if (!encode(&qm, c.a.q, 4, qsize, qstride, box_many) || !encode(&q1, c.a.q, 4, qsize, qstride, box_one)) return HS_ERR_CUDA;
  const auto run = D == 128 ? (c.a.scores != nullptr ? launch<128, true> : launch<128, false>)
                            : (c.a.scores != nullptr ? launch<64, true> : launch<64, false>);
  return run(c, qm, q1, seg, st) == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

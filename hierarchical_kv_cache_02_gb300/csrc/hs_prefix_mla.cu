// Attention of one new token a request over shared-latent records (576 values, the first 512 of them V), shared prefixes read
// once for 128 rows, on the 5th-generation tensor cores.
//
// The rows of a segment are its requests' query heads one after the other; an item is 128 of them, whatever the head count, and
// the work of two CTAs, a cluster on neighbouring SMs: each holds 64 rows' queries (72 KB), and the products are the pair's
// (cta_group::2).  Per tile of 64 records
//   S = Q K^T (128 x 64 x 576): a CTA holds the keys of 32 records, whole;
//   O += P V (128 x 512 x 64): a CTA holds 256 of the values of all 64 records.  The weights P are rounded to bf16, as both
//   operands of a product have one type and V is bf16 (2^-8 of a weight at most; the sum that divides is of the rounded).
// Rows 0-63 of an accumulator are the even CTA's, in both: its first half of columns in lanes 0-63 of tensor memory, the second
// in 64-127.  So two threads share a row, half of a tile's entries and half of the dims each.  The even CTA's warp issues for
// both; what has landed in the odd one, and its weights, are passed on by warps of their own, by arrivals with release at the
// cluster's scope on the even one's barriers.
// The products bound it from below: 18 MFLOP a tile and pair are 0.72 us at the tensor cores' rate.  A tile takes 1.28 us, the chain
// of its softmax: scores read and their maximum 530 cycles, the two threads' exchange 280, powers 390, the weights' place and the
// rescaling's votes 460, weights stored and handed over 500.  (With half the products, or half the values loaded, it takes 2 and 0 us
// less.)  8 requests of 64 heads over 32768 shared positions: 59 us, 0.62 PFLOP/s.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "hs_tc.cuh"
#include "hs_prefix.cuh"

namespace {

constexpr int kTile = 64, kRows = 128, kDim = 576, kValue = 512;
constexpr int kChunks = kDim / 64;                // 128-byte column blocks of a record
constexpr int kBlk = 64 * 128;                    // bytes of one block of 64 rows of the queries or weights
constexpr int kQ = kChunks * kBlk;                // a CTA's queries
// Tiles lie in groups of 8 records, a group's blocks one after the other: one copy brings 16 records' blocks.
constexpr int kKGroup = kChunks * 1024, kVGroup = 4 * 1024;
constexpr int kKBuf = 4 * kKGroup, kVBuf = 8 * kVGroup;  // 32 whole records; 256 values of 64 records
// Warps 0-3 are the softmax; the products' warp shares a quarter of the SM's issue slots with one of them alone.
constexpr int kWarpMma = 7, kPassKeys = 8, kPassValues = 10, kWarpPlan = 11, kThreads = 12 * 32;
__device__ __forceinline__ int key_producer(int warp) { return warp == 4 || warp == 5 ? warp - 4 : -1; }
__device__ __forceinline__ int value_producer(int warp) { return warp == 6 ? 0 : warp == 9 ? 1 : -1; }
constexpr int kMaskRing = 4;
constexpr int kAhead = 4;                         // accumulators of scores
constexpr float kLazy = 8.f;                      // log2 headroom before the running maximum is raised
constexpr size_t kDyn = (size_t)kQ + 2 * kBlk + 2 * (kKBuf + kVBuf);  // from a 1 KB boundary on
constexpr uint32_t kScores = 256;                 // first column of the scores, behind O's 256

struct MlaArgs {
  PrefixArgs a;
  PrefixSplit w;
  int seg;       // dense contexts whose pages hold multiples of 16: rows per box (16), else 0
  int ctx_rows;  // rows of the cache: a box that starts there reads zeros
  int negate;    // the scale is negative: qscale is its magnitude, the scores' products are negated
};

struct MlaControl {
  PrefixPlan plan;
  __align__(8) uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
  uint64_t kready[2], vready[2], qready;  // even CTA: full in both
  uint64_t qfull, s[kAhead], p[2], podd[2], pv[2], pair[2], mask[kMaskRing], fin;  // p: even CTA; podd: odd CTA, its own warps'
  uint32_t valid[kMaskRing][2];
  // Of the same shape, [..][half][row], so that a row's bytes are the same in both: pair_sync joins the two warps of 32 rows alone,
  // and the other two may be a portion's end ahead.
  union {
    float most[2][2][64];  // of a tile, by turns
    float sums[2][2][64];  // at a portion's end: of the rounded weights, of the exact ones
  };
  uint32_t tmem, abort;
};
static_assert(kTile == 64, "the split's tiles");
static_assert(kDyn + sizeof(MlaControl) <= 227 * 1024, "shared memory of a CTA");

// A box into this CTA's memory whose bytes are counted by a barrier of either CTA of the pair (bar: a cluster's address)
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
// Whether a tile comes in whole boxes, in both CTAs: then they are counted by the even one's barriers, and nothing has to be
// passed on.
__device__ __forceinline__ bool direct(const MlaArgs& c, const PPortion& P, int tile) {
  const int e0 = P.base + tile * kTile;
  return c.seg != 0 && e0 >= P.p0 && e0 + kTile <= P.p1;
}

// A producer lane's lookup of its entry of each tile, a tile ahead of the copies.  What the table says is looked at only when it is
// used: until then nothing waits for it.
struct Lookup {
  PPortion L;               // the next lookup's portion
  int nl = 0, lt;           // its number, the tile
  int page = 0, at = -1;    // what was found: the page, and the place in it (-1: nothing seen there)
  __device__ __forceinline__ void next(const PrefixArgs& a, PrefixPlan* plan, int mine, bool* ok, volatile uint32_t* abort) {
    at = -1;
    if (L.t0 == L.t1) return;
    const int p = L.base + lt * kTile + mine;
    if (p >= L.p0 && p < L.p1) {
      const unsigned pg = (unsigned)p / (unsigned)a.kv.page_tokens;
      at = p - (int)(pg * (unsigned)a.kv.page_tokens);
      page = a.kv.table != nullptr ? a.kv.table[(int64_t)L.lead * a.kv.max_pages + pg] : L.lead * a.kv.max_pages + (int)pg;
    }
    if (++lt == L.t1) {
      L = portion_take(plan, ++nl, false, ok, abort);
      lt = L.t0;
    }
  }
  __device__ __forceinline__ int row(const PrefixArgs& a) const {  // -1: nothing seen, -2: a bad page
    return at < 0 ? -1 : (unsigned)page < (unsigned)a.kv.num_pages ? page * a.kv.page_tokens + at : -2;
  }
};

// W: the scores of requests' own positions are kept, and the exact sums of weights.
template <bool W>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_prefix_mla(const __grid_constant__ MlaArgs c, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ MlaControl ct;
  const PrefixArgs& a = c.a;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int rank = uniform((int)cluster_rank());
  uint8_t* smem = smem_raw;
  const uint32_t q_u = smem_u32(smem), p_u = q_u + kQ, k_u = p_u + 2 * kBlk, v_u = k_u + 2 * kKBuf;
  if ((q_u & 1023u) != 0u) {  // all of a CTA's memory is used: there is no room to round up, and none is needed
    if (tid == 0) report(a.kv.err, (uint32_t)HS_DEVERR_TIMEOUT);
    return;
  }
  volatile uint32_t* abort = &ct.abort;
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ct.kfull[b], 64u);
      mbar_init(&ct.vfull[b], 64u);
      mbar_init(&ct.kempty[b], 1u);
      mbar_init(&ct.vempty[b], 1u);
      mbar_init(&ct.kready[b], 2u);
      mbar_init(&ct.vready[b], 2u);
    }
    for (int i = 0; i < kAhead; ++i) mbar_init(&ct.s[i], 1u);
    mbar_init(&ct.qready, 2u);
    mbar_init(&ct.qfull, 1u);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ct.p[i], 5u + (i == 0 ? (uint32_t)a.stall : 0u));
      mbar_init(&ct.podd[i], 4u);
      mbar_init(&ct.pv[i], 1u);
      mbar_init(&ct.pair[i], 2u);
    }
    for (int i = 0; i < kMaskRing; ++i) mbar_init(&ct.mask[i], 2u);
    mbar_init(&ct.fin, 1u);
    prefix_plan_init(&ct.plan, 11);  // the warps that read it
    ct.abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ct.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == 4 && lane == 0) {
    prefetch_map(&qmap);
    if (c.seg != 0) {
      prefetch_map(&kmap);
      prefetch_map(&vmap);
    }
  }
  __syncwarp();
  cluster_sync();  // both CTAs' barriers are there
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the only kernel that may start early is this call's own join, which waits for this one
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  const int worker = (int)blockIdx.x >> 1;
  prefix_start(a, c.w, &ct.plan, worker);
  tc_fence_after();
  const uint32_t tb = ct.tmem;

  int nt = 0;    // tiles so far, of each role
  int nq = 0;    // portions so far (products); query loads (first softmax thread)
  int sent = 0;  // producers: tiles whose copies were issued
  bool ok = true;
  uint32_t bad = 0u;
  PrefixPlan* plan = &ct.plan;

  {
    if (key_producer(warp) >= 0) {
      // ---------------- keys: 16 whole records of this CTA's 32 of a tile, looked up by lanes 0-15 ----------------
      const int first = 16 * key_producer(warp), crow = lane >> 3, cch = lane & 7;
      const uint32_t kready = in_cta(smem_u32(ct.kready), 0);
      Lookup ahead;
      ahead.L = portion_take(plan, 0, false, &ok, abort);
      ahead.lt = ahead.L.t0;
      PPortion P = ahead.L;
      ahead.next(a, plan, 32 * rank + first + (lane & 15), &ok, abort);
      int kt = P.t0;
#pragma unroll 1
      for (int pi = 0; P.t0 < P.t1;) {
        if (kt == P.t0 && lane == 0) mbar_arrive(&plan->empty[pi % kPrefixRing]);  // the lookups took it before
        const int found = ahead.row(a);
        if (found == -2) bad |= (uint32_t)HS_DEVERR_PAGE;
        const bool seen = found >= 0;
        const int row = seen ? found : c.ctx_rows;
        const int e0 = P.base + kt * kTile + 32 * rank + first;
        ahead.next(a, plan, 32 * rank + first + (lane & 15), &ok, abort);
        const int b = nt & 1;
        const uint32_t dst = k_u + (uint32_t)(b * kKBuf + (first >> 3) * kKGroup);
        uint64_t* full = &ct.kfull[b];
        if (ok) ok = warp_wait_small(&ct.kempty[b], (uint32_t)(((nt >> 1) & 1) ^ 1), abort);
        if (ok) {
          if (direct(c, P, kt)) {
            if (lane == 0) {
              if (rank == 0) mbar_arrive_expect_tx(&ct.kready[b], 4u * kKGroup);  // of both CTAs
              tma_load_pair(dst, &kmap, 0, 0, 0, row >> 3, kready + 8u * b);
            }
            __syncwarp();
            mbar_arrive(full);
          } else if (c.seg != 0 && e0 >= P.p0 && e0 + 16 <= P.p1) {
            if (lane == 0) mbar_arrive_expect_tx(full, 2u * kKGroup);
            else mbar_arrive(full);
            __syncwarp();
            if (lane == 0) tma_load_4d(dst, &kmap, 0, 0, 0, row >> 3, full);
            __syncwarp();
          } else {
            // 16 bytes a lane: rows 4 i .. 4 i + 3, swizzled as the boxes are
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int y = 4 * i + crow;
              const int src = __shfl_sync(0xffffffffu, seen ? row : -1, y);
              const uint32_t to = dst + (uint32_t)((y >> 3) * kKGroup + (y & 7) * 128 + ((cch ^ (y & 7)) << 4)), n = src >= 0 ? 16u : 0u;
              const uint8_t* from = src >= 0 ? a.kv.base + (int64_t)src * a.kv.rec + 16 * cch : (const uint8_t*)a.q;
#pragma unroll
              for (int h = 0; h < kChunks; ++h) cp_async16_zfill(to + h * 1024, src >= 0 ? from + 128 * h : from, n);
            }
            cp_async_arrive_noinc(full);
          }
          sent = nt + 1;
        }
        ++nt;
        if (++kt == P.t1) {
          P = portion_take(plan, ++pi, false, &ok, abort);
          kt = P.t0;
        }
      }
    } else if (value_producer(warp) >= 0) {
      // ---------------- values: this CTA's 256 of 32 records of every tile, a lane's lookup each ----------------
      const int half = value_producer(warp), crow = lane >> 3, cch = lane & 7;
      const uint32_t vready = in_cta(smem_u32(ct.vready), 0);
      Lookup ahead;
      ahead.L = portion_take(plan, 0, false, &ok, abort);
      ahead.lt = ahead.L.t0;
      PPortion P = ahead.L;
      ahead.next(a, plan, 32 * half + lane, &ok, abort);
      int kt = P.t0;
#pragma unroll 1
      for (int pi = 0; P.t0 < P.t1;) {
        if (kt == P.t0 && lane == 0) mbar_arrive(&plan->empty[pi % kPrefixRing]);  // the lookups took it before
        const int found = ahead.row(a);
        const bool seen = found >= 0;
        const int row = seen ? found : c.ctx_rows;
        const int e0 = P.base + kt * kTile + 32 * half;
        ahead.next(a, plan, 32 * half + lane, &ok, abort);
        const int b = nt & 1;
        const uint32_t dst = v_u + (uint32_t)(b * kVBuf + 4 * half * kVGroup);
        uint64_t* full = &ct.vfull[b];
        const uint32_t word = __ballot_sync(0xffffffffu, seen);
        // ahead of the wait: the softmax begins with the scores, before the values' place is free.  (What is overwritten is
        // of four tiles before, whose product was complete before the last tile's place was.)
        if (ok && lane == 0) {
          ct.valid[nt % kMaskRing][half] = word;
          mbar_arrive(&ct.mask[nt % kMaskRing]);
        }
        if (ok) ok = warp_wait_small(&ct.vempty[b], (uint32_t)(((nt >> 1) & 1) ^ 1), abort);
        if (ok) {
          if (direct(c, P, kt)) {
            if (lane == 0 && rank == 0) mbar_arrive_expect_tx(&ct.vready[b], 8u * kVGroup);  // of both CTAs
            __syncwarp();
            if ((lane & 15) == 0) tma_load_pair(dst + (uint32_t)((lane >> 3) * kVGroup), &vmap, 0, 0, 4 * rank, row >> 3, vready + 8u * b);
            __syncwarp();
            mbar_arrive(full);
          } else if (c.seg != 0 && e0 >= P.p0 && e0 + 32 <= P.p1) {
            if (lane == 0) mbar_arrive_expect_tx(full, 4u * kVGroup);
            else mbar_arrive(full);
            __syncwarp();
            if ((lane & 15) == 0) tma_load_4d(dst + (uint32_t)((lane >> 3) * kVGroup), &vmap, 0, 0, 4 * rank, row >> 3, full);
            __syncwarp();
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int y = 4 * i + crow;
              const int src = __shfl_sync(0xffffffffu, seen ? row : -1, y);
              const uint32_t to = dst + (uint32_t)((y >> 3) * kVGroup + (y & 7) * 128 + ((cch ^ (y & 7)) << 4)), n = src >= 0 ? 16u : 0u;
              const uint8_t* from = src >= 0 ? a.kv.base + (int64_t)src * a.kv.rec + 512 * rank + 16 * cch : (const uint8_t*)a.q;
#pragma unroll
              for (int h = 0; h < 4; ++h) cp_async16_zfill(to + h * 1024, src >= 0 ? from + 128 * h : from, n);
            }
            cp_async_arrive_noinc(full);
          }
          sent = nt + 1;
        }
        ++nt;
        if (++kt == P.t1) {
          P = portion_take(plan, ++pi, false, &ok, abort);
          kt = P.t0;
        }
      }
    } else if (warp == kWarpMma && rank == 0) {
      // ---------------- products ----------------
      // S(i) waits for tile i's keys, O(i) for its weights and values; whichever is ready is issued.
      const uint32_t tu = (uint32_t)uniform((int)tb);
      const uint32_t id_s = umma_idesc_bf16(kRows, kTile, 0, 0) | (c.negate ? kNegateA : 0u);
      const uint32_t id_o = umma_idesc_bf16(kRows, 256, 0, 1);
      const uint32_t dq = (uint32_t)uniform((int)umma_sdesc_lo(q_u, 16)), dk = (uint32_t)uniform((int)umma_sdesc_lo(k_u, 16));
      const uint32_t dp = (uint32_t)uniform((int)umma_sdesc_lo(p_u, 16));
      // V as it lies: blocks of 64 values 1 KB apart, 8 entries a group, the value dims contiguous
      const uint32_t dv = (uint32_t)uniform((int)umma_sdesc_lo(v_u, 1024));
      // the next scores' and the next values' place: portion, tiles left in it (0: no more), whether it is its first tile;
      // ahead: tiles whose scores were issued and whose values were not
      int kp = 0, vp = 0, ahead = 0;
      auto tiles_of = [&](int i) {
        const PPortion P = portion_take(plan, i, false, &ok, abort);
        return uniform(P.t1 - P.t0);
      };
      int kl = tiles_of(0), vl = kl;
      bool kfirst = true, vfirst = true;
      while (vl > 0) {
        const int i = nt + ahead, bs = i & 1, b = nt & 1;
        const bool more = kl > 0 && ahead < kAhead;
        bool scores = ahead == 0;
        if (ok) {
          ok = false;
          const uint32_t kq = (uint32_t)((i >> 1) & 1), vq = (uint32_t)((nt >> 1) & 1);
          WaitLimit limit;
#pragma unroll 1
          for (;;) {
            const bool y0 = cluster_test(&ct.p[b], vq), y1 = cluster_test(&ct.vready[b], vq),
                       y2 = cluster_test(&ct.kready[bs], kq), y3 = !kfirst || cluster_test(&ct.qready, (uint32_t)(nq & 1));
            ok = __all_sync(0xffffffffu, ahead != 0 && y0 && y1);
            if (ok) break;
            ok = scores = __all_sync(0xffffffffu, more && y2 && y3);
            if (ok) break;
            if (__any_sync(0xffffffffu, *abort != 0u || limit.over())) break;
          }
          if (!ok) scores = ahead == 0;
        }
        tc_fence_after();
        if (scores) {
          if (kfirst) ++nq;
          const uint32_t to = tu + kScores + 32u * (i % kAhead), y = dk + (uint32_t)(bs * (kKBuf >> 4));
          if (ok && elect_one()) {
#pragma unroll
            for (int h = 0; h < kChunks; ++h)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                umma2_bf16_lo<kKGroup>(to, dq + h * (kBlk >> 4) + 2 * ks, y + h * 64 + 2 * ks, id_s, (h | ks) != 0 ? 1u : 0u);
            umma2_commit(&ct.s[i % kAhead]);
            umma2_commit(&ct.kempty[bs]);
          }
          __syncwarp();
          ++ahead;
          kfirst = --kl == 0;
          if (kfirst) kl = tiles_of(++kp);
          continue;
        }
        if (ok && elect_one()) {
          const uint32_t y = dv + (uint32_t)(b * (kVBuf >> 4));
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma2_bf16_lo<kVGroup>(tu + 128u * h, dp + (uint32_t)(b * (kBlk >> 4)) + 2 * ks, y + 2 * h * 64 + ks * (2 * kVGroup >> 4), id_o,
                                     (!vfirst || ks != 0) ? 1u : 0u);
          umma2_commit(&ct.vempty[b]);
          umma2_commit(&ct.pv[b]);
        }
        __syncwarp();
        ++nt;
        --ahead;
        vfirst = --vl == 0;
        if (vfirst) {
          if (lane == 0) mbar_arrive(&plan->empty[vp % kPrefixRing]);
          vl = tiles_of(++vp);  // the scores' place is there already
        }
      }
    } else if (warp == kWarpMma) {
      // ---------------- the odd CTA's weights, passed on to the even one ----------------
      // (Its softmax does not wait for that: an arrival with release at the cluster's scope takes 0.8 us, half of a tile's time.)
      const uint32_t p_bar = in_cta(smem_u32(ct.p), 0);
#pragma unroll 1
      for (int pi = 0;; ++pi) {
        const PPortion P = portion_take(plan, pi, true, &ok, abort);
        if (P.t0 == P.t1) break;
#pragma unroll 1
        for (int tile = P.t0; tile < P.t1; ++tile, ++nt) {
          if (ok) ok = warp_wait_small(&ct.podd[nt & 1], (uint32_t)((nt >> 1) & 1), abort);
          tc_fence_after();
          tc_fence_before();
          if (ok && lane == 0) cluster_arrive(p_bar + 8u * (nt & 1));
        }
      }
    } else if (warp == kPassKeys || warp == kPassValues) {
      // ---------------- what the products take is there, passed on to the even CTA ----------------
      // (Copies of 16 bytes are generic-proxy writes; the tensor cores read through the async proxy.)
      const bool keys = warp == kPassKeys;
      uint64_t* full = keys ? ct.kfull : ct.vfull;
      const uint32_t ready = in_cta(smem_u32(keys ? ct.kready : ct.vready), 0), qr = in_cta(smem_u32(&ct.qready), 0);
#pragma unroll 1
      for (int pi = 0;; ++pi) {
        const PPortion P = portion_take(plan, pi, true, &ok, abort);
        if (P.t0 == P.t1) break;
        if (keys) {
          if (ok) ok = warp_wait_small(&ct.qfull, (uint32_t)(nq & 1), abort);
          ++nq;
          if (ok && lane == 0) cluster_arrive(qr);
        }
        for (int tile = P.t0; tile < P.t1; ++tile, ++nt) {
          if (ok) ok = warp_wait_small(&full[nt & 1], (uint32_t)((nt >> 1) & 1), abort);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          if (ok && lane == 0 && !direct(c, P, tile)) {
            if (rank == 0) mbar_arrive(&(keys ? ct.kready : ct.vready)[nt & 1]);
            else cluster_arrive(ready + 8u * (nt & 1));
          }
        }
      }
    } else if (warp < 4) {
      // ---------------- softmax: two threads a row, half of a tile's entries and half of the dims each ----------------
      // (A warp comes together, by a vote or __syncwarp, behind each branch that its lanes may take apart: accesses to tensor memory
      // are the whole warp's, and nothing else promises that it is whole there.)
      const int row = tid & 63, half = tid >> 6;
      const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
      uint64_t* pair = &ct.pair[warp & 1];
      uint32_t met = 0u;
      auto pair_sync = [&]() {  // the two warps of 32 rows; like every wait it gives up
        __syncwarp();
        if (lane == 0) mbar_arrive(pair);
        if (ok) ok = mbar_wait_small(pair, met, abort);
        met ^= 1u;
        ok = __all_sync(0xffffffffu, ok);
      };
      auto load_q = [&](int i) {  // of portion i, by the first thread
        if (!portion_wait(plan, i, abort)) return;
        const PPortion& P = portion_at(plan, i);
        if (P.t0 == P.t1) return;
        mbar_arrive_expect_tx(&ct.qfull, (uint32_t)kQ);
        for (int b = 0; b < kChunks; ++b) tma_load_2d(q_u + (uint32_t)(b * kBlk), &qmap, 64 * b, P.r0 + 64 * rank, &ct.qfull);
        ++nq;
      };
      if (tid == 0) load_q(0);
      __syncwarp();
#pragma unroll 1
      for (int pi = 0;; ++pi) {
        const PPortion P = portion_take(plan, pi, true, &ok, abort);
        if (P.t0 == P.t1) break;
        const bool row_ok = 64 * rank + row < P.cnt;
        const bool warp_ok = __any_sync(0xffffffffu, row_ok);
        float m = -INFINITY, l = 0.f, le = 0.f;  // the sums: of this thread's entries
        for (int tile = P.t0; tile < P.t1; ++tile, ++nt) {
          const int b = nt & 1;
          if (ok) ok = mbar_wait2(&ct.s[nt % kAhead], (uint32_t)((nt / kAhead) & 1), &ct.mask[nt % kMaskRing],
                                  (uint32_t)((nt / kMaskRing) & 1), abort);
          if (tid == 0 && tile == P.t1 - 1 && ok) load_q(pi + 1);  // the last scores are done
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
          const uint32_t w = ct.valid[nt % kMaskRing][half];
          const bool live = ok && warp_ok;
          float v[32], mx = -INFINITY;
          if (live) {
            tmem_ld32(tb + lane_base + kScores + 32u * (nt % kAhead), v);
            if (w != 0xffffffffu) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = (w >> j) & 1u ? v[j] : -INFINITY;
            }
            float my = -INFINITY;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              mx = fmaxf(fmaxf(mx, v[j]), v[j + 1]);
              my = fmaxf(fmaxf(my, v[j + 2]), v[j + 3]);
            }
            mx = fmaxf(mx, my) * a.qscale;
          }
          ct.most[b][half][row] = mx;
          pair_sync();
          if (live) {
            mx = fmaxf(mx, ct.most[b][half ^ 1][row]);
            const bool raise = mx > m + kLazy;
            const bool any = __any_sync(0xffffffffu, raise);
            const float mo = m;
            if (raise) m = mx;
            const float base = m == -INFINITY ? 0.f : m;  // nothing seen so far: every weight is 0
            uint32_t pk[16];
            float sum = 0.f, s1 = 0.f, exact = 0.f, e1 = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float p0, p1;
              fma2(p0, p1, v[2 * j], v[2 * j + 1], a.qscale, -base);
              p0 = fast_exp2(p0);
              p1 = fast_exp2(p1);
              pk[j] = pack_bf16(p0, p1);
              add2(sum, s1, lo(pk[j]), hi(pk[j]));  // the rounded weights, as the product takes them
              if (W) add2(exact, e1, p0, p1);
            }
            if (W && P.own && row_ok) {
              float* keep = a.scores + ((int64_t)P.r0 + 64 * rank + row) * a.score_cols + P.base + tile * kTile + 32 * half;
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] *= a.qscale;
#pragma unroll
              for (int j = 0; j < 32; j += 8) st_global_v8(keep + j, v + j);
            }
            if (W) __syncwarp();
            // P's place is free once the product two tiles before is complete; O may be rescaled once the last one is
            if (nt > 1) ok = mbar_wait_small(&ct.pv[b], (uint32_t)(((nt >> 1) - 1) & 1), abort);
            if (any && tile != P.t0 && ok) ok = mbar_wait_small(&ct.pv[b ^ 1], (uint32_t)(((nt - 1) >> 1) & 1), abort);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            if (any) {
              const float al = (m == mo || mo == -INFINITY) ? 1.f : fast_exp2(mo - m);
              l *= al;
              le *= al;
              __syncwarp();
              if (tile != P.t0 && ok) {
#pragma unroll 1
                for (int x = 0; x < 8; ++x) {
                  float o[32];
                  tmem_ld32(tb + lane_base + 32u * x, o);
#pragma unroll
                  for (int j = 0; j < 32; ++j) o[j] *= al;
                  tmem_st32(tb + lane_base + 32u * x, o);
                }
              }
            }
            l += sum + s1;
            le += exact + e1;
            // P, K-major and swizzled like the queries: 64 entries are one 128-byte row
#pragma unroll
            for (int x = 0; x < 4; ++x)
              *(uint4*)(smem + kQ + b * kBlk + row * 128 + (((4 * half + x) ^ (row & 7)) << 4)) =
                  make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          } else if (ok && nt > 1) {
            ok = mbar_wait_small(&ct.pv[b], (uint32_t)(((nt >> 1) - 1) & 1), abort);  // no phase of it may pass unseen
            ok = __all_sync(0xffffffffu, ok);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(rank == 0 ? &ct.p[b] : &ct.podd[b]);
        }
        // the portion's partial sums
        if (ok) ok = mbar_wait_small(&ct.pv[(nt - 1) & 1], (uint32_t)(((nt - 1) >> 1) & 1), abort);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        ct.sums[0][half][row] = l;
        ct.sums[1][half][row] = le;
        pair_sync();
        l += ct.sums[0][half ^ 1][row];
        le += ct.sums[1][half ^ 1][row];
        pair_sync();  // the next tile's maxima take their place
        if (ok && warp_ok) {
          const int mine = 64 * rank + row;
#pragma unroll 1
          for (int x = 0; x < 8; ++x) {
            float o[32];
            __syncwarp();
            tmem_ld32(tb + lane_base + 32u * x, o);
            if (row_ok) {
#pragma unroll
              for (int y = 0; y < 4; ++y) st_global_v8(c.w.part + P.row * kValue + ((32 * half + 4 * x + y) * P.stride + mine) * 8, o + 8 * y);
            }
          }
          if (row_ok && half == 0) *(float4*)(c.w.ml + 4 * (P.row + mine)) = make_float4(m, l, le, 0.f);
        }
        tc_fence_before();
        __syncwarp();
      }
    } else if (warp == kWarpPlan) {
      prefix_walk(a, c.w, plan, worker, abort);
      if (*abort != 0u) ok = false;
    }
    if (!ok) {  // the other CTA gives up, too
      *abort = 1u;
      asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(in_cta(smem_u32(&ct.abort), (uint32_t)(rank ^ 1))) : "memory");
    }
    __syncwarp();
  }
  if (!ok && lane == 0) report(a.kv.err, (uint32_t)HS_DEVERR_TIMEOUT);
  report(a.kv.err, bad);
  // after a wait that gave up, copies and products may still be in flight: they end before the CTAs do
  volatile uint32_t never = 0u;
  if (warp == kWarpMma) {
    if (rank == 0 && elect_one()) umma2_commit(&ct.fin);  // by the thread whose products they are
    __syncwarp();
    warp_wait(&ct.fin, 0u, &never);
  }
  __syncthreads();
  const int kpw = key_producer(warp), vpw = value_producer(warp);
  if (kpw >= 0 || vpw >= 0) asm volatile("cp.async.wait_all;" ::: "memory");
  if (*abort != 0u && lane == 0) {
    const uint64_t t0 = global_ns();
    if (kpw >= 0 || vpw >= 0) {
      uint64_t* full = kpw >= 0 ? ct.kfull : ct.vfull;
#pragma unroll 1
      for (int i = max(0, sent - 2); i < sent; ++i)
        while (!mbar_try_wait(&full[i & 1], (uint32_t)((i >> 1) & 1)) && global_ns() - t0 < 1000000000ull) {
        }
      // The boxes that the even CTA's barriers count, into both CTAs: the odd one waits for it below.  A tile's place is free when
      // both CTAs' copies two tiles before were used, so the odd one's may be of two tiles that this one made none for; then their
      // barriers never complete, and the limit is the time that they have.
      uint64_t* ready = kpw >= 0 ? ct.kready : ct.vready;
      if (rank == 0 && c.seg != 0) {
#pragma unroll 1
        for (int i = max(0, sent - 2); i < sent + 2; ++i)
          while (!mbar_try_wait(&ready[i & 1], (uint32_t)((i >> 1) & 1)) && global_ns() - t0 < 1000000000ull) {
          }
      }
    } else if (warp == 0 && nq > 0) {
      while (!mbar_try_wait(&ct.qfull, (uint32_t)((nq - 1) & 1)) && global_ns() - t0 < 1000000000ull) {
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync();  // neither CTA's memory is used by the other any more
  tc_fence_after();
  if (warp == kWarpMma) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tb) : "memory");
}

// ---- host ------------------------------------------------------------------------------------------

void split_of(const hs_config* c, int num_sms, PrefixSplit* w) {
  w->heads = 1;
  w->flat = 1;
  w->G = w->MT = 1;
  w->mt = div_by(1);
  w->pairs = 0;
  w->tile_shift = 6;
  w->cost = w->cost2 = div_by(1);
  w->begin = 3;
  w->copies = 1;
  w->most = kRows;
  w->group_rows = 2 * c->num_q_heads;
  w->together = c->num_q_heads % 4 == 0 ? 4 : 1;  // items begin at multiples of 128 rows
  w->workers = num_sms / 2;
}

template <bool W>
cudaError_t launch(const MlaArgs& c, const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  static bool done[64];
  cudaError_t e = allow_smem(k_prefix_mla<W>, kDyn, done);
  if (e == cudaSuccess) e = hs_launch_pdl(k_prefix_mla<W>, dim3(2 * c.w.workers), dim3(kThreads), kDyn, st, c, qm, km, vm);
  if (e != cudaSuccess) return e;
  return launch_join<kValue>(c.a, c.w, st);
}

}  // namespace

// Rows of partials: an item's are its rows in use, and what is left of a last one: at most 2 Hq for a request alone, and 2 Hq n
// for a group of n; and what keeps the workers' apart.
hs_prefix_plan hs_prefix_mla_plan(const hs_config* c, int num_sms) {
  if (c->layout != HS_LAYOUT_MLA || c->head_dim_qk != kDim || c->head_dim_v != kValue || num_sms < 2) return {0};
  return {4ll * c->num_requests * c->num_q_heads + (int64_t)(num_sms / 2) * kRows};
}

int hs_prefix_mla_launch(const hs_config* cfg, const void* prefix_args, void* head, void* partials, int num_sms, cudaStream_t st) {
  MlaArgs c{};
  c.a = *(const PrefixArgs*)prefix_args;
  split_of(cfg, num_sms, &c.w);
  hs_prefix_head(head, c.a.ngroups, &c.w);
  c.w.part = (float*)partials;
  c.w.ml = c.w.part + hs_prefix_mla_plan(cfg, num_sms).rows * kValue;
  if (c.a.qscale < 0.f) {
    c.negate = 1;
    c.a.qscale = -c.a.qscale;
  }
  c.a.qscale = fmaxf(c.a.qscale, 1.17549435e-38f);  // times -infinity has to stay -infinity
  CUtensorMap qm, km, vm;
  memset(&km, 0, sizeof(km));
  memset(&vm, 0, sizeof(vm));
  const cuuint64_t rec = kDim * 2;
  c.ctx_rows = (int)(c.a.kv.num_pages * c.a.kv.page_tokens);
  if (c.a.kv.page_tokens % 16 == 0) {
    c.seg = 16;
    const cuuint64_t size[4] = {64, 8, kChunks, (cuuint64_t)c.ctx_rows / 8}, stride[3] = {rec, 128, 8 * rec};
    const cuuint32_t kbox[4] = {64, 8, kChunks, 2}, vbox[4] = {64, 8, 4, 2};
    if (!encode(&km, c.a.kv.base, 4, size, stride, kbox) || !encode(&vm, c.a.kv.base, 4, size, stride, vbox)) c.seg = 0;
  }
  const cuuint64_t qsize[2] = {kDim, (cuuint64_t)c.a.R * c.a.Hq}, qstride[1] = {rec};
  const cuuint32_t qbox[2] = {64, 64};
  if (!encode(&qm, c.a.q, 2, qsize, qstride, qbox)) return HS_ERR_CUDA;
  const cudaError_t e = c.a.scores != nullptr ? launch<true>(c, qm, km, vm, st) : launch<false>(c, qm, km, vm, st);
  return e == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

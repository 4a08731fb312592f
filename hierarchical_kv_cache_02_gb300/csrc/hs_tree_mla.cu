// Tree attention over shared-latent records (576 values, the first 512 of them V) on the 5th-generation tensor
// cores.
//
// The rows of a request are its (node, query head) pairs one after the other; an item is 128 of them, whatever the
// head count, and the work of two CTAs, a cluster on neighbouring SMs: each holds 64 rows' queries (72 KB), and the
// products are the pair's (cta_group::2).  Per tile of 64 records
//   S = Q K^T (128 x 64 x 576): a CTA holds the keys of 32 records, whole;
//   O += P V (128 x 512 x 64): a CTA holds 256 of the values of all 64 records.  The weights P are rounded to bf16, as both
//   operands of a product have one type and V is bf16 (2^-8 of a weight at most; the sum that divides is of the rounded).
// So a CTA loads 68 KB a tile, the keys free their memory as soon as the scores are done, and two tiles of each fit
// beside the queries.  (One CTA for itself, 64 rows: a tile is key and value at once, 72 KB that stay from the
// scores to the value product, and an accumulator of 64 rows runs the tensor cores at half their rate; two such tiles
// fit: 97 and 55 us on the two cases below.  128 rows of a CTA: their queries leave room for one tile.)
// Rows 0-63 of an accumulator are the even CTA's, in both: its first half of columns in lanes 0-63 of tensor memory,
// the second in 64-127.  So two threads share a row, half of a tile's entries and half of the dims each.
// The even CTA's warp issues for both; what has landed in the odd one is passed on by an arrival on its barriers.
// What bounds it: the chain from one value product to the next.  Its weights may be stored once the product before is
// complete, and are handed to the even CTA by an arrival with release at the cluster's scope, which takes about 1000
// cycles; a tile takes about 3000, its products 1800.  Measured: 4 ragged requests of up to 32768 x 5 nodes x 64 heads
// 96.0 us (534 TFLOP/s, tensor cores active 30%), 8 x 8 nodes over 2048 listed positions 50.7 us.  (Arrivals with the default scope, the CTA's,
// took 72.5 and 43.7 us, but order nothing for the other CTA.  The hand-over by a warp of its own: 105 and 52 us;
// polls without ordering and a fence behind them: 122 and 59 us.)
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "hs_tc.cuh"
#include "hs_tree.cuh"

namespace {

constexpr int kTile = 64, kRows = 128, kDim = 576, kValue = 512;
constexpr int kChunks = kDim / 64;                // 128-byte column blocks of a record
constexpr int kBlk = 64 * 128;                    // bytes of one block of 64 rows of the queries or weights
constexpr int kQ = kChunks * kBlk;                // a CTA's queries
// Tiles lie in groups of 8 records, a group's blocks one after the other: one copy brings 16 records' blocks.
constexpr int kKGroup = kChunks * 1024, kVGroup = 4 * 1024;
constexpr int kKBuf = 4 * kKGroup, kVBuf = 8 * kVGroup;  // 32 whole records; 256 values of 64 records
// Warps 0-3 are the softmax; the products' warp shares a quarter of the SM's issue slots with one of them alone.
constexpr int kWarpMma = 7, kPassKeys = 8, kPassValues = 10, kThreads = 11 * 32;
__device__ __forceinline__ int key_producer(int warp) { return warp == 4 || warp == 5 ? warp - 4 : -1; }
__device__ __forceinline__ int value_producer(int warp) { return warp == 6 ? 0 : warp == 9 ? 1 : -1; }
constexpr int kMaskRing = 4;
constexpr int kAhead = 4;                         // accumulators of scores
constexpr float kLazy = 8.f;                      // log2 headroom before the running maximum is raised
constexpr size_t kDyn = (size_t)kQ + kBlk + 2 * (kKBuf + kVBuf) + 1024;
constexpr uint32_t kScores = 256;                 // first column of the scores, behind O's 256

struct MlaArgs {
  TreeArgs a;
  WorkSplit ws;
  int seg;       // dense contexts whose pages hold multiples of 16: rows per box (16), else 0
  int ctx_rows;  // rows of the cache: a box that starts there reads zeros
  int negate;    // the scale is negative: qscale is its magnitude, the scores' products are negated
};

struct MlaControl {
  PlanState plan;
  __align__(8) uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
  uint64_t kready[2], vready[2], qready;  // even CTA: full in both
  uint64_t qfull, s[kAhead], p, pv, mask[kMaskRing], fin;
  uint64_t told[2];  // the other CTA's softmax is through with a portion's nodes (two: it can be one portion ahead)
  uint32_t valid[kMaskRing][2];
  float most[2][2][64], sums[2][64];
  uint32_t tmem, abort, dirty;
};
static_assert(kDyn + sizeof(MlaControl) <= 227 * 1024, "shared memory of a CTA");

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_tree_mla(const MlaArgs c, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ MlaControl ct;
  const TreeArgs& a = c.a;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int rank = uniform((int)cluster_rank());
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t q_u = smem_u32(smem), p_u = q_u + kQ, k_u = p_u + kBlk, v_u = k_u + 2 * kKBuf;
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
    mbar_init(&ct.p, 8u);
    mbar_init(&ct.pv, 1u);
    for (int i = 0; i < kMaskRing; ++i) mbar_init(&ct.mask[i], 2u);
    mbar_init(&ct.fin, 1u);
    for (int i = 0; i < 2; ++i) mbar_init(&ct.told[i], 4u);
    ct.abort = ct.dirty = 0u;
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
  // the only kernel that may start early is this call's own combine, which waits for this one
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  bool go = plan_start<kTile>(a, c.ws, &ct.plan);
  tc_fence_after();
  const uint32_t tb = ct.tmem;

  // state that runs on through the rounds
  int nt = 0;                      // tiles so far, of each role
  int nq = 0;                      // portions so far (products); query loads (first softmax thread)
  int sent = 0;                    // producers: tiles whose copies were issued
  int nd = 0;                      // softmax: portions with nodes
  bool ok = true;
  uint32_t bad = 0u;

  for (; go; go = plan_round<kTile>(a, c.ws, &ct.plan)) {
    const Portion* list = ct.plan.port[0];
    const int count = ct.plan.nport[0];
    if (key_producer(warp) >= 0) {
      // ---------------- keys: 16 whole records of this CTA's 32 of a tile, looked up by lanes 0-15 ----------------
      const int first = 16 * key_producer(warp), crow = lane >> 3, cch = lane & 7;
      Lookahead ahead = {};
      ahead.at = count > 0 ? list[0].t0 : 0;
      int kp = 0, kt = ahead.at;
#pragma unroll 1
      for (int x = -2; kp < count; ++x) {
        ahead.step(a, list, count, kTile, 32 * rank + first + (lane & 15), c.ctx_rows, lane < 16 ? kChunks : 0, &bad);
        if (x < 0) continue;  // the steps' head start
        const Portion& P = list[kp];
        const int b = nt & 1;
        const uint32_t dst = k_u + (uint32_t)(b * kKBuf + (first >> 3) * kKGroup);
        uint64_t* full = &ct.kfull[b];
        if (ok) ok = warp_wait_small(&ct.kempty[b], (uint32_t)(((nt >> 1) & 1) ^ 1), abort);
        if (ok) {
          if (c.seg != 0 && kt * kTile + 32 * rank + first + 16 <= P.n) {
            if (lane == 0) mbar_arrive_expect_tx(full, 2u * kKGroup);
            else mbar_arrive(full);
            __syncwarp();
            if (lane == 0) tma_load_4d(dst, &kmap, 0, 0, 0, ahead.row >> 3, full);
          } else {
            // 16 bytes a lane: rows 4 i .. 4 i + 3, swizzled as the boxes are
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int y = 4 * i + crow;
              const uint64_t src = __shfl_sync(0xffffffffu, ahead.now, y);
              const uint32_t to = dst + (uint32_t)((y >> 3) * kKGroup + (y & 7) * 128 + ((cch ^ (y & 7)) << 4)), n = src != 0ull ? 16u : 0u;
              const uint8_t* from = src != 0ull ? (const uint8_t*)(uintptr_t)src + 16 * cch : (const uint8_t*)a.q;
#pragma unroll
              for (int h = 0; h < kChunks; ++h) cp_async16_zfill(to + h * 1024, src != 0ull ? from + 128 * h : from, n);
            }
            cp_async_arrive_noinc(full);
          }
          sent = nt + 1;
        }
        ++nt;
        if (++kt == P.t1) {
          ++kp;
          if (kp < count) kt = list[kp].t0;
        }
      }
    } else if (value_producer(warp) >= 0) {
      // ---------------- values: this CTA's 256 of 32 records of every tile, a lane's lookup each ----------------
      const int half = value_producer(warp), crow = lane >> 3, cch = lane & 7;
      Lookahead ahead = {};
      ahead.at = count > 0 ? list[0].t0 : 0;
      int kp = 0, kt = ahead.at;
#pragma unroll 1
      for (int x = -2; kp < count; ++x) {
        ahead.step(a, list, count, kTile, 32 * half + lane, c.ctx_rows, 0, &bad);
        if (x < 0) continue;
        const Portion& P = list[kp];
        const int b = nt & 1;
        const uint32_t dst = v_u + (uint32_t)(b * kVBuf + 4 * half * kVGroup);
        uint64_t* full = &ct.vfull[b];
        if (ok) ok = warp_wait_small(&ct.vempty[b], (uint32_t)(((nt >> 1) & 1) ^ 1), abort);
        const uint32_t word = __ballot_sync(0xffffffffu, ahead.now != 0ull);
        if (ok) {
          if (lane == 0) {
            ct.valid[nt % kMaskRing][half] = word;
            mbar_arrive(&ct.mask[nt % kMaskRing]);
          }
          if (c.seg != 0 && kt * kTile + 32 * half + 32 <= P.n) {
            if (lane == 0) mbar_arrive_expect_tx(full, 4u * kVGroup);
            else mbar_arrive(full);
            __syncwarp();
            if ((lane & 15) == 0) tma_load_4d(dst + (uint32_t)((lane >> 3) * kVGroup), &vmap, 0, 0, 4 * rank, ahead.row >> 3, full);
            __syncwarp();
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int y = 4 * i + crow;
              const uint64_t src = __shfl_sync(0xffffffffu, ahead.now, y);
              const uint32_t to = dst + (uint32_t)((y >> 3) * kVGroup + (y & 7) * 128 + ((cch ^ (y & 7)) << 4)), n = src != 0ull ? 16u : 0u;
              const uint8_t* from = src != 0ull ? (const uint8_t*)(uintptr_t)src + 512 * rank + 16 * cch : (const uint8_t*)a.q;
#pragma unroll
              for (int h = 0; h < 4; ++h) cp_async16_zfill(to + h * 1024, src != 0ull ? from + 128 * h : from, n);
            }
            cp_async_arrive_noinc(full);
          }
          sent = nt + 1;
        }
        ++nt;
        if (++kt == P.t1) {
          ++kp;
          if (kp < count) kt = list[kp].t0;
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
      const int n = uniform(count);
      // the next scores' and the next values' place: portion, tiles left in it, whether it is its first tile;
      // ahead: tiles whose scores were issued and whose values were not
      int kp = 0, kl = 0, vp = 0, vl = 0, ahead = 0;
      bool kfirst = true, vfirst = true;
      if (n > 0) kl = vl = uniform(list[0].t1 - list[0].t0);
      while (vp < n) {
        const int i = nt + ahead, bs = i & 1, b = nt & 1;
        const bool more = kp < n && ahead < kAhead;
        bool scores = ahead == 0;
        if (ok) {
          ok = false;
          const uint32_t kq = (uint32_t)((i >> 1) & 1), vq = (uint32_t)((nt >> 1) & 1);
          WaitLimit limit;
#pragma unroll 1
          for (;;) {
            const bool y0 = cluster_test(&ct.p, (uint32_t)(nt & 1)), y1 = cluster_test(&ct.vready[b], vq),
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
          if (kfirst && ++kp < n) kl = uniform(list[kp].t1 - list[kp].t0);
          continue;
        }
        if (ok && elect_one()) {
          const uint32_t y = dv + (uint32_t)(b * (kVBuf >> 4));
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma2_bf16_lo<kVGroup>(tu + 128u * h, dp + 2 * ks, y + 2 * h * 64 + ks * (2 * kVGroup >> 4), id_o,
                                     (!vfirst || ks != 0) ? 1u : 0u);
          umma2_commit(&ct.vempty[b]);
          umma2_commit(&ct.pv);
        }
        __syncwarp();
        ++nt;
        --ahead;
        vfirst = --vl == 0;
        if (vfirst && ++vp < n) vl = uniform(list[vp].t1 - list[vp].t0);
      }
    } else if (warp == kPassKeys || warp == kPassValues) {
      // ---------------- what the products take is there, passed on to the even CTA ----------------
      // (Copies of 16 bytes are generic-proxy writes; the tensor cores read through the async proxy.)
      const bool keys = warp == kPassKeys;
      uint64_t* full = keys ? ct.kfull : ct.vfull;
      const uint32_t ready = in_cta(smem_u32(keys ? ct.kready : ct.vready), 0), qr = in_cta(smem_u32(&ct.qready), 0);
      for (int pi = 0; pi < count; ++pi) {
        if (keys) {
          if (ok) ok = warp_wait_small(&ct.qfull, (uint32_t)(nq & 1), abort);
          ++nq;
          if (ok && lane == 0) cluster_arrive(qr);
        }
        for (int tile = list[pi].t0; tile < list[pi].t1; ++tile, ++nt) {
          if (ok) ok = warp_wait_small(&full[nt & 1], (uint32_t)((nt >> 1) & 1), abort);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          if (ok && lane == 0) cluster_arrive(ready + 8u * (nt & 1));
        }
      }
    } else if (warp < 4) {
      // ---------------- softmax: two threads a row, half of a tile's entries and half of the dims each ----------------
      // (A warp comes together, by a vote or __syncwarp, behind each branch that its lanes may take apart: accesses to tensor memory
      // are the whole warp's, and nothing else promises that it is whole there.)
      const int row = tid & 63, half = tid >> 6;
      const uint32_t lane_base = (uint32_t)(warp * 32) << 16, p_bar = in_cta(smem_u32(&ct.p), 0);
      auto pair_sync = [&]() { asm volatile("barrier.cta.sync %0, 64;" ::"r"(2 + (warp & 1)) : "memory"); };
      auto load_q = [&](const Portion& P) {  // by the first thread
        mbar_arrive_expect_tx(&ct.qfull, (uint32_t)kQ);
        const int r0 = (int)((int64_t)P.r * a.T * a.Hq + (int64_t)kRows * P.head) + 64 * rank;
        for (int b = 0; b < kChunks; ++b) tma_load_2d(q_u + (uint32_t)(b * kBlk), &qmap, 64 * b, r0, &ct.qfull);
        ++nq;
      };
      if (tid == 0 && count > 0 && ok) load_q(list[0]);
      for (int pi = 0; pi < count; ++pi) {
        const Portion P = list[pi];
        const int flat = kRows * P.head + 64 * rank + row, t = flat / a.Hq;
        const int n4 = (int)(((unsigned)P.n + 3u) & ~3u);
        const bool row_ok = t < P.nn;
        const bool warp_ok = __any_sync(0xffffffffu, row_ok);
        const uint64_t* mw = a.mask + ((int64_t)P.r * a.T + (row_ok ? t : 0)) * a.words;
        const uint64_t mfirst = mw[0];
        float m = -INFINITY, l = 0.f;  // l: of this thread's entries
        bool dirty = false;  // a node's value is infinite or NaN
        for (int tile = P.t0; tile < P.t1; ++tile, ++nt) {
          const int b = nt & 1;
          const int j0 = (int)((long long)tile * kTile - n4);  // node of the tile's first entry
          const bool nodes = j0 + kTile > 0;
          if (ok) ok = mbar_wait2(&ct.s[nt % kAhead], (uint32_t)((nt / kAhead) & 1), &ct.mask[nt % kMaskRing],
                                  (uint32_t)((nt / kMaskRing) & 1), abort);
          if (tid == 0 && tile == P.t1 - 1 && pi + 1 < count && ok) load_q(list[pi + 1]);  // the last scores are done
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
          uint32_t w = ct.valid[nt % kMaskRing][half];
          if (nodes) {
            // entries that are nodes: valid ones that this row sees
            const int jw = j0 + 32 * half;
            const uint32_t ctx = jw >= 0 ? 0u : (jw <= -32 ? 0xffffffffu : (1u << -jw) - 1u);
            w &= ctx | (row_ok ? mask_bits(mw, mfirst, a.words, P.nn, jw) : 0u);
            // infinite and NaN values would reach every row of the product: they are taken out here and
            // added to the rows that see them at the end
            if (ok) ok = mbar_wait_small(&ct.vfull[b], (uint32_t)((nt >> 1) & 1), abort);
            const bool d = ok && clean_rows(smem + kQ + kBlk + 2 * kKBuf + b * kVBuf, 1024, kVGroup, 4, max(0, -j0),
                                            min(kTile, P.nn - j0), tid, 128);
            if (bar_or(1, 128, d)) {
              dirty = true;
              if (lane == 0)  // the other CTA's rows take their values from here, too; read there behind ct.told
                asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(in_cta(smem_u32(&ct.dirty), (uint32_t)(rank ^ 1))) : "memory");
            }
            ok = __all_sync(0xffffffffu, ok);
          }
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
            // the value product before this tile's: O may be rescaled, and P rewritten, once it is complete
            const bool done = nt == 0 || mbar_test(&ct.pv, (uint32_t)((nt - 1) & 1));
            const bool raise = mx > m + kLazy;
            const bool any = __any_sync(0xffffffffu, raise);
            const float mo = m;
            if (raise) m = mx;
            const float base = m == -INFINITY ? 0.f : m;  // nothing seen so far: every weight is 0
            uint32_t pk[16];
            float sum = 0.f, s1 = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float p0, p1;
              fma2(p0, p1, v[2 * j], v[2 * j + 1], a.qscale, -base);
              pk[j] = pack_bf16(fast_exp2(p0), fast_exp2(p1));
              add2(sum, s1, lo(pk[j]), hi(pk[j]));  // the rounded weights, as the product takes them
            }
            if (!done) ok = mbar_wait_small(&ct.pv, (uint32_t)((nt - 1) & 1), abort);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            if (any) {
              const float al = (m == mo || mo == -INFINITY) ? 1.f : fast_exp2(mo - m);
              l *= al;
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
            // P, K-major and swizzled like the queries: 64 entries are one 128-byte row
#pragma unroll
            for (int x = 0; x < 4; ++x)
              *(uint4*)(smem + kQ + row * 128 + (((4 * half + x) ^ (row & 7)) << 4)) =
                  make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          } else if (ok && nt > 0) {
            ok = mbar_wait_small(&ct.pv, (uint32_t)((nt - 1) & 1), abort);  // no phase of it may pass unseen
            ok = __all_sync(0xffffffffu, ok);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0 && !(a.stall != 0 && nt == 0 && tid == 64 && blockIdx.x == 1)) cluster_arrive(p_bar);
          if (nodes && tile == P.t1 - 1 && lane == 0) cluster_arrive(in_cta(smem_u32(&ct.told[nd & 1]), (uint32_t)(rank ^ 1)));
        }
        // the portion's result: complete, or a partial
        if (ok) ok = mbar_wait_small(&ct.pv, (uint32_t)((nt - 1) & 1), abort);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        if ((long long)P.t1 * kTile > n4) {  // it holds nodes: the other CTA has looked at its half of their values
          if (ok) ok = cluster_wait(&ct.told[nd & 1], (uint32_t)((nd >> 1) & 1), abort);
          ok = __all_sync(0xffffffffu, ok);
          ++nd;
        }
        ct.sums[half][row] = l;
        pair_sync();
        l += ct.sums[half ^ 1][row];
        if (ok && warp_ok) {
          const bool whole = P.t0 == 0 && P.t1 == (int)tiles_of<kTile>(P.n, P.nn);
          const long long slot = ((long long)(blockIdx.x >> 1) * 2 + (P.t0 > 0 ? 0 : 1)) * kRows;
          const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
          dirty = dirty || *(volatile uint32_t*)&ct.dirty != 0u;
#pragma unroll 1
          for (int x = 0; x < 8; ++x) {
            float o[32];
            __syncwarp();
            tmem_ld32(tb + lane_base + 32u * x, o);
            const int dim = 256 * half + 32 * x;
            if (dirty && row_ok) {
              for (int j = max(0, P.t0 * kTile - n4); j < min((long long)P.nn, (long long)P.t1 * kTile - n4); ++j) {
                if (((mw[j >> 6] >> (j & 63)) & 1ull) == 0ull) continue;
                const uint8_t* rec = node_record(a, P.r, P.len, j, &bad);
                if (rec == nullptr) continue;
                const uint32_t* vr = (const uint32_t*)rec + dim / 2;
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
                uint4* dst = (uint4*)(a.out + ((int64_t)P.r * a.T * a.Hq + flat) * kValue + dim);
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  dst[y] = make_uint4(pack_bf16(o[8 * y] * inv, o[8 * y + 1] * inv), pack_bf16(o[8 * y + 2] * inv, o[8 * y + 3] * inv),
                                      pack_bf16(o[8 * y + 4] * inv, o[8 * y + 5] * inv), pack_bf16(o[8 * y + 6] * inv, o[8 * y + 7] * inv));
              } else {
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  st_global_v8(c.ws.part + slot * kValue + ((dim / 8 + y) * kRows + 64 * rank + row) * 8, o + 8 * y);
              }
            }
          }
          if (row_ok && !whole && half == 0) *(float2*)(c.ws.ml + (slot + 64 * rank + row) * 2) = make_float2(m, l);
        }
        tc_fence_before();
        __syncwarp();
      }
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

bool usable(const hs_config* c) {
  return c->layout == HS_LAYOUT_MLA && c->head_dim_qk == kDim && c->head_dim_v == kValue &&
         (int64_t)c->num_requests * HS_MAX_TREE_NODES * c->num_q_heads <= (int64_t)INT32_MAX;
}
int items_of(const hs_config* c, int T) { return (T * c->num_q_heads + kRows - 1) / kRows; }

}  // namespace

hs_tree_plan hs_tree_mla_plan(const hs_config* c, int nodes, int num_sms) {
  hs_tree_plan r = {usable(c) && num_sms >= 2, 0};
  if (r.usable) r.workspace = hs_tree_workspace_bytes(c, num_sms / 2, kRows, kValue);
  return r;
}

int hs_tree_mla_launch(const hs_config* cfg, const hs_tree_args* g, const void* tree_args, int num_sms, cudaStream_t st) {
  const int pairs = num_sms / 2;
  MlaArgs c{};
  c.a = *(const TreeArgs*)tree_args;
  c.ws.items = items_of(cfg, g->nodes);
  c.ws.np = 1;
  c.ws.groups = 1;
  c.ws.pairs = 1;
  c.ws.begin = 2;  // 76.0, 74.2, 72.9 and 73.0 us with 0 to 3 on 4 ragged requests of up to 32768 (before hand-overs
                   // between the CTAs had the cluster's scope)
  c.ws.rows = kRows;
  hs_tree_workspace(g->d_workspace, cfg, pairs, kRows, kValue, &c.ws.prefix, &c.ws.part, &c.ws.ml);
  if (c.a.qscale < 0.f) {
    c.negate = 1;
    c.a.qscale = -c.a.qscale;
  }
  c.a.qscale = fmaxf(c.a.qscale, 1.17549435e-38f);  // times -infinity has to stay -infinity
  CUtensorMap qm, km, vm;
  memset(&km, 0, sizeof(km));
  memset(&vm, 0, sizeof(vm));
  const cuuint64_t rec = kDim * 2;
  if (c.a.slot_pt == nullptr && c.a.locs == nullptr && c.a.kv.page_tokens % 16 == 0) {
    c.seg = 16;
    c.ctx_rows = (int)(c.a.kv.num_pages * c.a.kv.page_tokens);
    const cuuint64_t size[4] = {64, 8, kChunks, (cuuint64_t)c.ctx_rows / 8}, stride[3] = {rec, 128, 8 * rec};
    const cuuint32_t kbox[4] = {64, 8, kChunks, 2}, vbox[4] = {64, 8, 4, 2};
    if (!encode(&km, c.a.kv.base, 4, size, stride, kbox) || !encode(&vm, c.a.kv.base, 4, size, stride, vbox)) c.seg = 0;
  }
  const cuuint64_t qsize[2] = {kDim, (cuuint64_t)cfg->num_requests * g->nodes * cfg->num_q_heads}, qstride[1] = {rec};
  const cuuint32_t qbox[2] = {64, 64};
  if (!encode(&qm, c.a.q, 2, qsize, qstride, qbox)) return HS_ERR_CUDA;
  CombineArgs cb{};
  cb.nodes = c.a.nodes;
  cb.out = c.a.out;
  cb.ws = c.ws;
  cb.R = c.a.R;
  cb.T = c.a.T;
  cb.Hq = c.a.Hq;
  cb.workers = pairs;
  cb.flat = kRows;
  static bool done[64];
  cudaError_t e = allow_smem(k_tree_mla, kDyn, done);
  if (e == cudaSuccess) e = hs_launch_pdl(k_tree_mla, dim3(2 * pairs), dim3(kThreads), kDyn, st, c, qm, km, vm);
  if (e == cudaSuccess) e = launch_combine<kValue>(cb, st);
  return e == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

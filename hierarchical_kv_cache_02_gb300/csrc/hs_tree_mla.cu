// Tree attention over shared-latent records (576 values, the first 512 of them V) on the 5th-generation tensor
// cores.
//
// The rows of a request are its (node, query head) pairs one after the other; an item is 64 of them, whatever the
// head count.  A CTA holds their queries in shared memory (72 KB) and two tiles of 64 records (72 KB each): a
// latent is key and value at once, so a tile is loaded once and stays from the scores to the value product.
// Per tile S = Q K^T (64 x 64 x 576) and O += P V (64 x 512 x 64).  An accumulator of 64 rows takes 16 of every 32
// lanes of tensor memory, so O's two halves of 256 dims share columns (lanes 0-15 and 16-31 of each
// quarter), and so do the scores of even and odd tiles.  The scores of the next tile are issued before the
// value product of the one at hand, so the softmax (one warpgroup, a thread per row) runs beside them.
// 128 rows with half of the dims in an accumulator would use the tensor cores better, but their queries leave
// 80 KB for records: not enough to load one tile while the values of another wait for its weights.
// What bounds it: at full rate the products of a tile take 2176 cycles of a 64-row accumulator.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "hs_tc.cuh"
#include "hs_tree.cuh"

namespace {

constexpr int kTile = 64, kRows = 64, kDim = 576, kValue = 512;
constexpr int kChunks = kDim / 64;                // 128-byte column blocks of a tile
// A tile's blocks come and go in two parts: 0-3, the values' first half, and 4-8.
constexpr int kParts = 2;
__host__ __device__ constexpr int part_from(int part) { return 4 * part; }
__host__ __device__ constexpr int part_blocks(int part) { return 4 + part; }
constexpr int kBlk = 64 * 128;                    // bytes of one block of 64 rows of the queries or weights
constexpr int kBuf = kChunks * kBlk;              // the queries; also a tile
// A tile lies in groups of 8 records, a group's blocks one after the other: one copy brings 4 or 5 blocks of 16
// records.  (Block by block, 9 copies a warp and tile, their issue alone took a third of the tile's time.)
constexpr int kGroup = kChunks * 1024;
// Warps 0-3 are the softmax; the products' warp shares a quarter of the SM's issue slots with one of them alone.
constexpr int kProducers = 4, kWarpMma = 7, kThreads = 10 * 32;
__device__ __forceinline__ int producer_of(int warp) { return warp >= 4 && warp <= 6 ? warp - 4 : warp == 9 ? 3 : -1; }
constexpr int kMaskRing = 4;
constexpr float kLazy = 8.f;                      // log2 headroom before the running maximum is raised
constexpr size_t kDyn = 3 * (size_t)kBuf + kBlk + 1024;
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
  __align__(8) uint64_t full[2][kParts], empty[2][kParts];
  uint64_t qfull, s[2], p, pv, mask[kMaskRing], fin;
  uint32_t valid[kMaskRing][kProducers];
  uint32_t tmem, abort;
};
static_assert(kDyn + sizeof(MlaControl) <= 227 * 1024, "shared memory of a CTA");

__global__ void __launch_bounds__(kThreads, 1)
    k_tree_mla(const MlaArgs c, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap segmap0,
               const __grid_constant__ CUtensorMap segmap1) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ MlaControl ct;
  const TreeArgs& a = c.a;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t q_u = smem_u32(smem), p_u = q_u + kBuf, buf_u = p_u + kBlk;
  volatile uint32_t* abort = &ct.abort;
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      for (int i = 0; i < kParts; ++i) {
        mbar_init(&ct.full[b][i], kProducers * 32);
        mbar_init(&ct.empty[b][i], 1u);
      }
      mbar_init(&ct.s[b], 1u);
    }
    mbar_init(&ct.qfull, 1u);
    mbar_init(&ct.p, 128u);
    mbar_init(&ct.pv, 1u);
    for (int i = 0; i < kMaskRing; ++i) mbar_init(&ct.mask[i], kProducers);
    mbar_init(&ct.fin, 1u);
    ct.abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ct.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 4 && lane == 0) {
    prefetch_map(&qmap);
    if (c.seg != 0) {
      prefetch_map(&segmap0);
      prefetch_map(&segmap1);
    }
  }
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
  int sent = 0;                    // producers: tile parts whose copies were issued
  bool ok = true;
  uint32_t bad = 0u;

  for (; go; go = plan_round<kTile>(a, c.ws, &ct.plan)) {
    const Portion* list = ct.plan.port[0];
    const int count = ct.plan.nport[0];
    const int pw = producer_of(warp);
    if (pw >= 0) {
      // ---------------- producers: 16 entries of every tile each, looked up by lanes 0-15 ----------------
      const int crow = lane >> 3, cch = lane & 7;
      Lookahead ahead = {};
      ahead.at = count > 0 ? list[0].t0 : 0;
      int kp = 0, kt = ahead.at;
#pragma unroll 1
      for (int x = -2; kp < count; ++x) {
        ahead.step(a, list, count, kTile, 16 * pw + (lane & 15), c.ctx_rows, lane < 16 ? kChunks : 0, &bad);
        if (x < 0) continue;  // the steps' head start
        const Portion& P = list[kp];
        const bool boxed = c.seg != 0 && kt * kTile + 16 * pw + 16 <= P.n;
        const int b = nt & 1;
        const uint32_t dst = buf_u + (uint32_t)(b * kBuf + 2 * pw * kGroup);
        const int row = __shfl_sync(0xffffffffu, ahead.row, 0);
#pragma unroll 1
        for (int part = 0; part < kParts; ++part) {
          if (ok) ok = warp_wait_small(&ct.empty[b][part], (uint32_t)(((nt >> 1) & 1) ^ 1), abort);
          if (!ok) continue;
          uint64_t* full = &ct.full[b][part];
          const int ch0 = part_from(part), nch = part_blocks(part);
          if (boxed) {
            if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(nch * 16 * 128));
            else mbar_arrive(full);
            __syncwarp();
            if (lane == 0) {
#pragma unroll
              for (int g = 0; g < 2; ++g)
                tma_load_4d(dst + (uint32_t)(g * kGroup + ch0 * 1024), part == 0 ? &segmap0 : &segmap1, 0, 0, ch0, (row >> 3) + g, full);
            }
          } else {
            // 16 bytes a lane: rows 4 i .. 4 i + 3, swizzled as the boxes are
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int y = 4 * i + crow;
              const uint64_t src = __shfl_sync(0xffffffffu, ahead.now, y);
              const uint32_t to = dst + (uint32_t)((y >> 3) * kGroup + ch0 * 1024 + (y & 7) * 128 + ((cch ^ (y & 7)) << 4)), n = src != 0ull ? 16u : 0u;
              const uint8_t* from = src != 0ull ? (const uint8_t*)(uintptr_t)src + 128 * ch0 + 16 * cch : (const uint8_t*)a.q;
#pragma unroll
              for (int h = 0; h < 5; ++h)
                if (h < nch) cp_async16_zfill(to + h * 1024, src != 0ull ? from + 128 * h : from, n);
            }
            cp_async_arrive_noinc(full);
          }
          sent = 2 * nt + part + 1;
        }
        const uint32_t word = __ballot_sync(0xffffffffu, ahead.now != 0ull) & 0xffffu;
        if (ok && lane == 0) {
          ct.valid[nt % kMaskRing][pw] = word;
          mbar_arrive(&ct.mask[nt % kMaskRing]);
        }
        ++nt;
        if (++kt == P.t1) {
          ++kp;
          if (kp < count) kt = list[kp].t0;
        }
      }
    } else if (warp == kWarpMma) {
      // ---------------- products ----------------
      // S(i) waits for tile i's records, O(i) for its weights, and S(i + 2) takes the buffer that O(i) leaves.
      // Whichever is ready is issued, values first: they set a buffer free.
      const uint32_t tu = (uint32_t)uniform((int)tb);
      const uint32_t id_s = umma_idesc_bf16(kRows, kTile, 0, 0) | (c.negate ? kNegateA : 0u);
      const uint32_t id_o = umma_idesc_bf16(kRows, 256, 0, 1);
      const uint32_t dq = (uint32_t)uniform((int)umma_sdesc_lo(q_u, 16)), dk = (uint32_t)uniform((int)umma_sdesc_lo(buf_u, 16));
      const uint32_t dp = (uint32_t)uniform((int)umma_sdesc_lo(p_u, 16));
      // V as it lies: blocks of 64 values 1 KB apart, 8 entries a group, the value dims contiguous
      const uint32_t dv = (uint32_t)uniform((int)umma_sdesc_lo(buf_u, 1024));
      const int n = uniform(count);
      // the next scores' and the next values' place: portion, tiles left in it, whether it is its first tile;
      // ahead: tiles whose scores were issued and whose values were not; part: of the scores to come
      int kp = 0, kl = 0, vp = 0, vl = 0, ahead = 0, part = 0;
      bool kfirst = true, vfirst = true;
      if (n > 0) kl = vl = uniform(list[0].t1 - list[0].t0);
      while (vp < n) {
        const int i = nt + ahead, bs = i & 1;
        const bool more = kp < n && ahead < 2;
        bool scores = ahead == 0;
        if (ahead != 0 && ok) {
          ok = false;
#pragma unroll 1
          for (uint32_t x = 0; x < (1u << 22); ++x) {
            ok = uniform_test(&ct.p, (uint32_t)(nt & 1));
            if (ok) break;
            if (more) {
              ok = scores = uniform_test(&ct.full[bs][part], (uint32_t)((i >> 1) & 1)) &&
                            (!kfirst || part != 0 || uniform_test(&ct.qfull, (uint32_t)(nq & 1)));
              if (ok) break;
            }
            if (__any_sync(0xffffffffu, *abort != 0u)) break;
          }
        }
        if (scores) {
          if (kfirst && part == 0) {  // this portion's queries
            if (ok) ok = uniform_wait(&ct.qfull, (uint32_t)(nq & 1), abort);
            ++nq;
          }
          if (ok) ok = uniform_wait(&ct.full[bs][part], (uint32_t)((i >> 1) & 1), abort);
          // copies of 16 bytes are generic-proxy writes; the tensor cores read through the async proxy
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          tc_fence_after();
          const uint32_t to = tu + kScores + ((uint32_t)(16 * bs) << 16);
          const uint32_t x = dq + part_from(part) * (kBlk >> 4), y = dk + (uint32_t)(bs * (kBuf >> 4)) + part_from(part) * 64;
          if (ok && elect_one()) {
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                umma_bf16_lo<kGroup>(to, x + h * (kBlk >> 4) + 2 * ks, y + h * 64 + 2 * ks, id_s, (part | h | ks) != 0 ? 1u : 0u);
            if (part == kParts - 1) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) umma_bf16_lo<kGroup>(to, x + 4 * (kBlk >> 4) + 2 * ks, y + 4 * 64 + 2 * ks, id_s, 1u);
              umma_commit(&ct.s[bs]);
            }
          }
          __syncwarp();
          if (++part < kParts) continue;
          part = 0;
          ++ahead;
          kfirst = --kl == 0;
          if (kfirst && ++kp < n) kl = uniform(list[kp].t1 - list[kp].t0);
          continue;
        }
        const int b = nt & 1;
        tc_fence_after();
        if (ok && elect_one()) {
          const uint32_t y = dv + (uint32_t)(b * (kBuf >> 4));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_bf16_lo<kGroup>(tu + ((uint32_t)(16 * h) << 16), dp + 2 * ks, y + 4 * h * 64 + ks * (2 * kGroup >> 4), id_o,
                                   (!vfirst || ks != 0) ? 1u : 0u);
            umma_commit(&ct.empty[b][h]);
          }
          umma_commit(&ct.pv);
        }
        __syncwarp();
        ++nt;
        --ahead;
        vfirst = --vl == 0;
        if (vfirst && ++vp < n) vl = uniform(list[vp].t1 - list[vp].t0);
      }
    } else if (warp < 4) {
      // ---------------- softmax: 16 rows a warp ----------------
      // Scores (of even tiles in lanes 0-15 of tensor memory, of odd ones in 16-31) are read as four threads a row
      // hold them, lane / 4 and lane / 4 + 8, so that all threads work on a tile; O a thread per row, lane & 15,
      // dims 0-255 or 256-511.
      const int row = 16 * warp + (lane & 15), side = lane >> 4;
      const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
      auto load_q = [&](const Portion& P) {  // by the first thread
        mbar_arrive_expect_tx(&ct.qfull, (uint32_t)kBuf);
        const int r0 = (int)((int64_t)P.r * a.T * a.Hq + (int64_t)kRows * P.head);
        for (int b = 0; b < kChunks; ++b) tma_load_2d(q_u + (uint32_t)(b * kBlk), &qmap, 64 * b, r0, &ct.qfull);
        ++nq;
      };
      if (tid == 0 && count > 0 && ok) load_q(list[0]);
      for (int pi = 0; pi < count; ++pi) {
        const Portion P = list[pi];
        const int flat = kRows * P.head + row, t = flat / a.Hq;
        const int n4 = (int)(((unsigned)P.n + 3u) & ~3u);
        const bool row_ok = t < P.nn;
        const bool warp_ok = __any_sync(0xffffffffu, row_ok);
        const uint64_t* mw = a.mask + ((int64_t)P.r * a.T + (row_ok ? t : 0)) * a.words;
        const uint64_t mfirst = mw[0];
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // of rows lane / 4 and + 8; l: this thread's columns
        bool dirty = false;  // a node's value is infinite or NaN
        for (int tile = P.t0; tile < P.t1; ++tile, ++nt) {
          const int b = nt & 1;
          const int j0 = (int)((long long)tile * kTile - n4);  // node of the tile's first entry
          const bool nodes = j0 + kTile > 0;
          if (ok) ok = mbar_wait_small(&ct.s[b], (uint32_t)((nt >> 1) & 1), abort);
          tc_fence_after();
          if (tid == 0 && tile == P.t1 - 1 && pi + 1 < count && ok) load_q(list[pi + 1]);  // the last scores are done
          if (ok) ok = mbar_wait_small(&ct.mask[nt % kMaskRing], (uint32_t)((nt / kMaskRing) & 1), abort);
          ok = __all_sync(0xffffffffu, ok);
          uint32_t w[2];  // of row lane & 15
#pragma unroll
          for (int x = 0; x < 2; ++x) w[x] = ct.valid[nt % kMaskRing][2 * x] | (ct.valid[nt % kMaskRing][2 * x + 1] << 16);
          const bool full = !nodes && (w[0] & w[1]) == 0xffffffffu;
          if (nodes) {
            // entries that are nodes: valid ones that this row sees
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int jw = j0 + 32 * x;
              const uint32_t ctx = jw >= 0 ? 0u : (jw <= -32 ? 0xffffffffu : (1u << -jw) - 1u);
              w[x] &= ctx | (row_ok ? mask_bits(mw, mfirst, a.words, P.nn, jw) : 0u);
            }
            // infinite and NaN values would reach every row of the product: they are taken out here and
            // added to the rows that see them at the end.  Their scores are done.
            for (int i = 0; i < kParts; ++i)
              if (ok) ok = mbar_wait_small(&ct.full[b][i], (uint32_t)((nt >> 1) & 1), abort);
            const bool d = ok && clean_rows(smem + kBuf + kBlk + b * kBuf, 1024, kGroup, kValue / 64, max(0, -j0),
                                             min(kTile, P.nn - j0), tid, 128);
            if (bar_or(1, 128, d)) dirty = true;
            ok = __all_sync(0xffffffffu, ok);
          }
          if (ok && warp_ok) {
            float v[32];
            tmem_ld_16x64(tb + lane_base + kScores + ((uint32_t)(16 * b) << 16), v);
            if (!full) {
#pragma unroll
              for (int h = 0; h < 4; ++h) {  // row (lane / 4) + 8 (h & 1), 32 columns
                const uint32_t bits = __shfl_sync(0xffffffffu, w[h >> 1], (lane >> 2) + 8 * (h & 1)) >> (2 * (lane & 3));
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                  const int j = 16 * (h >> 1) + 4 * (x >> 1) + 2 * (h & 1) + (x & 1);
                  v[j] = (bits >> (8 * (x >> 1) + (x & 1))) & 1u ? v[j] : -INFINITY;
                }
              }
            }
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              mx[0] = fmaxf(fmaxf(mx[0], v[j]), v[j + 1]);
              mx[1] = fmaxf(fmaxf(mx[1], v[j + 2]), v[j + 3]);
            }
            bool any = false;
            float al[2], base[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
              mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2)) * a.qscale;
              const float mo = m[h];
              if (mx[h] > mo + kLazy) {
                m[h] = mx[h];
                any = true;
              }
              al[h] = (m[h] == mo || mo == -INFINITY) ? 1.f : fast_exp2(mo - m[h]);
              base[h] = m[h] == -INFINITY ? 0.f : m[h];  // nothing seen so far: every weight is 0
            }
            any = __any_sync(0xffffffffu, any);
            uint32_t pk[16];
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float p0, p1;
              fma2(p0, p1, v[2 * j], v[2 * j + 1], a.qscale, -base[j & 1]);
              pk[j] = pack_bf16(fast_exp2(p0), fast_exp2(p1));
              add2(sum[2 * (j & 1)], sum[2 * (j & 1) + 1], lo(pk[j]), hi(pk[j]));  // the rounded weights, as the product takes them
            }
            // the value product before this tile's: O may be rescaled, and P rewritten, once it is complete
            if (nt > 0) ok = mbar_wait_small(&ct.pv, (uint32_t)((nt - 1) & 1), abort);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            if (any && tile != P.t0 && ok) {
              const float x0 = __shfl_sync(0xffffffffu, al[0], 4 * (lane & 7)), x1 = __shfl_sync(0xffffffffu, al[1], 4 * (lane & 7));
              const float f = (lane & 8) != 0 ? x1 : x0;
#pragma unroll 1
              for (int x = 0; x < 8; ++x) {
                float o[32];
                tmem_ld32(tb + lane_base + 32u * x, o);
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] *= f;
                tmem_st32(tb + lane_base + 32u * x, o);
              }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) l[h] = fmaf(l[h], al[h], sum[2 * h] + sum[2 * h + 1]);
            // P, K-major and swizzled like the queries: 64 entries are one 128-byte row
#pragma unroll
            for (int x = 0; x < 4; ++x)
              stmatrix_x4(p_u + (uint32_t)(row * 128 + (((2 * x + side) ^ (row & 7)) << 4)), pk[4 * x], pk[4 * x + 1], pk[4 * x + 2],
                          pk[4 * x + 3]);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          } else if (ok && nt > 0) {
            ok = mbar_wait_small(&ct.pv, (uint32_t)((nt - 1) & 1), abort);  // no phase of it may pass unseen
            ok = __all_sync(0xffffffffu, ok);
          }
          tc_fence_before();
          mbar_arrive(&ct.p);
        }
        // the portion's result: complete, or a partial
        if (ok) ok = mbar_wait_small(&ct.pv, (uint32_t)((nt - 1) & 1), abort);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        if (ok && warp_ok) {
          const bool whole = P.t0 == 0 && P.t1 == (int)tiles_of<kTile>(P.n, P.nn);
          const long long slot = ((long long)blockIdx.x * 2 + (P.t0 > 0 ? 0 : 1)) * kRows;
          float mr = 0.f, lr = 0.f;  // of row lane & 15
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            const float x = __shfl_sync(0xffffffffu, m[h], 4 * (lane & 7)), y = __shfl_sync(0xffffffffu, l[h], 4 * (lane & 7));
            if (h == ((lane >> 3) & 1)) mr = x, lr = y;
          }
          const float inv = whole ? (lr == 0.f ? 0.f : 1.f / lr) : 1.f;
#pragma unroll 1
          for (int x = 0; x < 8; ++x) {
            float o[32];
            tmem_ld32(tb + lane_base + 32u * x, o);
            const int dim = 256 * side + 32 * x;
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
                  st_global_v8(c.ws.part + slot * kValue + ((dim / 8 + y) * kRows + row) * 8, o + 8 * y);
              }
            }
          }
          if (row_ok && !whole && side == 0) *(float2*)(c.ws.ml + (slot + row) * 2) = make_float2(mr, lr);
        }
        tc_fence_before();
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
      for (int i = max(0, sent - 4); i < sent; ++i)
        while (!mbar_try_wait(&ct.full[(i >> 1) & 1][i & 1], (uint32_t)((i >> 2) & 1)) && global_ns() - t0 < 1000000000ull) {
        }
    } else if (warp == 0 && nq > 0) {
      while (!mbar_try_wait(&ct.qfull, (uint32_t)((nq - 1) & 1)) && global_ns() - t0 < 1000000000ull) {
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tb) : "memory");
}

// ---- host ------------------------------------------------------------------------------------------

bool usable(const hs_config* c) {
  return c->layout == HS_LAYOUT_MLA && c->head_dim_qk == kDim && c->head_dim_v == kValue &&
         (int64_t)c->num_requests * HS_MAX_TREE_NODES * c->num_q_heads <= (int64_t)INT32_MAX;
}
int items_of(const hs_config* c, int T) { return (T * c->num_q_heads + kRows - 1) / kRows; }

}  // namespace

hs_tree_plan hs_tree_mla_plan(const hs_config* c, int nodes, int num_sms) {
  hs_tree_plan r = {usable(c), 0};
  if (r.usable) r.workspace = hs_tree_workspace_bytes(c, num_sms, kRows, kValue);
  return r;
}

int hs_tree_mla_launch(const hs_config* cfg, const hs_tree_args* g, const void* tree_args, int num_sms, cudaStream_t st) {
  MlaArgs c{};
  c.a = *(const TreeArgs*)tree_args;
  c.ws.items = items_of(cfg, g->nodes);
  c.ws.np = 1;
  c.ws.groups = 1;
  c.ws.begin = 1;
  c.ws.rows = kRows;
  hs_tree_workspace(g->d_workspace, cfg, num_sms, kRows, kValue, &c.ws.prefix, &c.ws.part, &c.ws.ml);
  if (c.a.qscale < 0.f) {
    c.negate = 1;
    c.a.qscale = -c.a.qscale;
  }
  c.a.qscale = fmaxf(c.a.qscale, 1.17549435e-38f);  // times -infinity has to stay -infinity
  CUtensorMap qm, seg[2];
  memset(seg, 0, sizeof(seg));
  const cuuint64_t rec = kDim * 2;
  if (c.a.slot_pt == nullptr && c.a.locs == nullptr && c.a.kv.page_tokens % 16 == 0) {
    c.seg = 16;
    c.ctx_rows = (int)(c.a.kv.num_pages * c.a.kv.page_tokens);
    const cuuint64_t size[4] = {64, 8, kChunks, (cuuint64_t)c.ctx_rows / 8}, stride[3] = {rec, 128, 8 * rec};
    for (int i = 0; i < kParts; ++i) {
      const cuuint32_t box[4] = {64, 8, (cuuint32_t)part_blocks(i), 1};
      if (!encode(&seg[i], c.a.kv.base, 4, size, stride, box)) c.seg = 0;
    }
  }
  const cuuint64_t qsize[2] = {kDim, (cuuint64_t)cfg->num_requests * g->nodes * cfg->num_q_heads}, qstride[1] = {rec};
  const cuuint32_t qbox[2] = {64, kRows};
  if (!encode(&qm, c.a.q, 2, qsize, qstride, qbox)) return HS_ERR_CUDA;
  CombineArgs cb{};
  cb.nodes = c.a.nodes;
  cb.out = c.a.out;
  cb.ws = c.ws;
  cb.R = c.a.R;
  cb.T = c.a.T;
  cb.Hq = c.a.Hq;
  cb.workers = num_sms;
  cb.flat = kRows;
  static bool done[64];
  cudaError_t e = allow_smem(k_tree_mla, kDyn, done);
  if (e == cudaSuccess) e = hs_launch_pdl(k_tree_mla, dim3(num_sms), dim3(kThreads), kDyn, st, c, qm, seg[0], seg[1]);
  if (e == cudaSuccess)
    e = hs_launch_pdl(k_tree_combine<kValue>, combine_grid(c.ws.items, cfg->num_requests, kRows, kValue), dim3(256), 0, st, cb);
  return e == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

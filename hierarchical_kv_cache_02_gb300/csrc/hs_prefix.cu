// Attention of one new token a request over a paged cache, the prefixes that requests share read for many of them at a time, and the
// weights it gives to what they do not share.
//
// For request r, query head h, over the positions p below its length:
//   s_p = scale <q, K(p)>,  o = sum_p 2^(s_p log2(e) - m) V(p) / sum_p 2^(s_p log2(e) - m),
// and, for a list of weights (a KV head's, or the request's), w_p = decay w_p + sum_h 2^(s_p log2(e) - m_h) / l_h.
// The sums l_h are complete only at the end, so the scores of a request's own positions, 32 bits each, are kept for a last kernel:
// 8 bytes a query head and position beside a record of 4 KB (8 KV heads of 128) or of 1152 bytes.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "hs_prefix.cuh"

namespace {

// ---- any shape, on CUDA cores --------------------------------------------------------------------
//
// A CTA per (query head, request, part of its positions), its four warps take the positions in turn.  A lane holds every 32nd
// group of 8 values of a head (head dims up to 576 = 72 groups: at most three).  It reads a record once for every query head, and
// a shared one for every request.

constexpr int kAnyJoinThreads = 256;
constexpr int kAnyWarps = 4, kAnyGroups = 3, kAnyParts = 64;

// What the tensor cores' kernels find out on their way: whether the groups are sound, and the requests.
__global__ void __launch_bounds__(1024) k_prefix_check(const PrefixArgs a, PrefixRequest* of) {
  hs_pdl_wait();
  const int tid = threadIdx.x;
  const bool ok = __syncthreads_and(bounds_ok(a, tid, 1024)) != 0;
  uint32_t bad = ok ? 0u : (uint32_t)HS_DEVERR_LOC;
  if (ok)
    for (int g = tid; g < a.ngroups; g += 1024) group_segment(a, g, &bad);
  for (int r = tid; r < a.R; r += 1024) {
    int g;
    const Segment shared = shared_segment(a, r, ok, &g), own = own_segment(a, r, shared.p1, &bad);
    of[r] = PrefixRequest{0, own.p0, own.p1, g, shared.r0, shared.nr, 0};
  }
  report(a.kv.err, bad);
}

__global__ void __launch_bounds__(kAnyWarps * 32) k_prefix_any(const PrefixArgs a, const PrefixRequest* of, float* part, float* ml, int parts) {
  __shared__ float s_acc[kAnyWarps][kAnyGroups * 32 * 8];
  __shared__ float s_m[kAnyWarps], s_l[kAnyWarps];
  hs_pdl_wait();
  const int h = blockIdx.x, r = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t bad = 0u;
  const PrefixRequest own = of[r];
  // parts of whole groups of 32 positions
  const int chunks = (int)(((unsigned)own.p1 + 31u) >> 5), each = (chunks + parts - 1) / parts;
  const int64_t e0 = 32 * (int64_t)each * blockIdx.z;
  const int e1 = (int)min((int64_t)own.p1, e0 + 32 * (int64_t)each);
  const int kg = a.dqk / 8, vg = a.dv / 8;
  const int64_t koff = (int64_t)(h / (a.Hq / a.Hkv)) * a.kstride, row = (int64_t)r * a.Hq + h;
  float q[kAnyGroups][8], acc[kAnyGroups][8];
#pragma unroll
  for (int x = 0; x < kAnyGroups; ++x) {
    const int gi = lane + 32 * x;
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (gi < kg) u = *(const uint4*)(a.q + row * a.dqk + 8 * gi);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[x][2 * i] = lo(w[i]);
      q[x][2 * i + 1] = hi(w[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[x][i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t p = e0 + warp; p < e1; p += kAnyWarps) {
    const int64_t at = paged_row(a.kv, p < own.p0 ? own.r0 : r, p, (uint32_t)HS_DEVERR_LOC, &bad);
    float s = -INFINITY;
    const uint16_t* kp = (const uint16_t*)(a.kv.base + at * a.kv.rec) + koff;
    if (at >= 0) {
      s = 0.f;
#pragma unroll
      for (int x = 0; x < kAnyGroups; ++x) {
        const int gi = lane + 32 * x;
        if (gi < kg) {
          const uint4 u = *(const uint4*)(kp + 8 * gi);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s = fmaf(q[x][2 * i], lo(w[i]), s);
            s = fmaf(q[x][2 * i + 1], hi(w[i]), s);
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      s *= a.qscale;
    }
    if (a.scores != nullptr && lane == 0 && p >= own.p0) a.scores[row * a.score_cols + p] = s;
    if (at < 0) continue;
    // -infinity: weight 0 whatever the maximum, but a value that is infinite or NaN counts.  NaN: fmaxf keeps the
    // maximum, the weight is NaN
    const float mn = fmaxf(m, s);
    const float al = m == mn ? 1.f : exp2f(m - mn), w8 = s == -INFINITY ? 0.f : exp2f(s - mn);
    m = mn;
    l = l * al + w8;
#pragma unroll
    for (int x = 0; x < kAnyGroups; ++x) {
      const int gi = lane + 32 * x;
      if (gi < vg) {
        const uint4 u = *(const uint4*)(kp + a.voff + 8 * gi);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[x][2 * i] = fmaf(w8, lo(w[i]), acc[x][2 * i] * al);
          acc[x][2 * i + 1] = fmaf(w8, hi(w[i]), acc[x][2 * i + 1] * al);
        }
      }
    }
  }
  report(a.kv.err, bad);
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int x = 0; x < kAnyGroups; ++x)
#pragma unroll
    for (int i = 0; i < 8; ++i) s_acc[warp][(lane + 32 * x) * 8 + i] = acc[x][i];
  __syncthreads();
  float M = -INFINITY, L = 0.f, wt[kAnyWarps];
#pragma unroll
  for (int w = 0; w < kAnyWarps; ++w) M = fmaxf(M, s_m[w]);
#pragma unroll
  for (int w = 0; w < kAnyWarps; ++w) {
    wt[w] = s_m[w] == -INFINITY ? (s_l[w] == 0.f ? 0.f : NAN) : exp2f(s_m[w] - M);  // NaN scores alone: NaN
    L += wt[w] * s_l[w];
  }
  const int64_t to = row * parts + blockIdx.z;
  for (int d = threadIdx.x; d < a.dv; d += kAnyWarps * 32) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kAnyWarps; ++w) x = fmaf(wt[w], s_acc[w][d], x);
    part[to * a.dv + d] = x;
  }
  if (threadIdx.x == 0) *(float4*)(ml + 4 * to) = make_float4(M, L, L, 0.f);
}

__global__ void __launch_bounds__(kAnyJoinThreads) k_prefix_any_join(const PrefixArgs a, const float* part, const float* ml, int parts) {
  hs_pdl_wait();
  const int vecs = a.dv >> 3, at = blockIdx.x * kAnyJoinThreads + threadIdx.x, r = blockIdx.y;
  if (at >= a.Hq * vecs) return;
  const int h = at / vecs, d = 8 * (at - h * vecs);
  const long long row = ((long long)r * a.Hq + h) * parts;
  Joined sum;
  for (int x = 0; x < parts; ++x) sum.add(part, ml, row + x, a.dv, d);
  sum.store(a, r, h, d);
}

// ---- weights -------------------------------------------------------------------------------------

constexpr int kWeighThreads = 256, kWeighEach = 4;

// CTAs share a request's list; a thread takes kWeighEach positions at a time and sums over the list's query heads.  A round trip
// for the request's place, one for the statistics, one for the scores (one position at a time: 73.6 us instead of 70.5 for 16 requests of up
// to 8192 positions, 32 query heads, attention included).
__global__ void __launch_bounds__(kWeighThreads) k_prefix_weigh(const PrefixArgs a, const PrefixRequest* of) {
  __shared__ float2 s_stats[1024];
  hs_pdl_wait();
  const int list = blockIdx.y, r = blockIdx.z, heads = a.Hq / a.lists;
  const PrefixRequest q = of[r];
  if (q.p1 > a.cap && threadIdx.x == 0 && blockIdx.x == 0 && list == 0) report(a.kv.err, (uint32_t)HS_DEVERR_LOC);
  const int64_t end = min((int64_t)q.p1, a.cap), each = (int64_t)gridDim.x * kWeighThreads * kWeighEach;
  int64_t p = q.p0 + (int64_t)blockIdx.x * kWeighThreads * kWeighEach + threadIdx.x;
  if (p - threadIdx.x >= end) return;  // the whole CTA
  const int64_t h0 = (int64_t)r * a.Hq + list * heads;
  for (int h = threadIdx.x; h < heads; h += kWeighThreads) s_stats[h] = a.stats[h0 + h];
  __syncthreads();
  float* w = a.weights + ((int64_t)r * a.lists + list) * a.cap;
  for (; p < end; p += each) {
    float sum[kWeighEach], old[kWeighEach];
#pragma unroll
    for (int x = 0; x < kWeighEach; ++x) {
      sum[x] = 0.f;
      old[x] = p + x * kWeighThreads < end ? w[p + x * kWeighThreads] : 0.f;
    }
    const float* s = a.scores + h0 * a.score_cols + p;
#pragma unroll 4
    for (int h = 0; h < heads; ++h, s += a.score_cols) {
      const float2 st = s_stats[h];
#pragma unroll
      for (int x = 0; x < kWeighEach; ++x)
        if (p + x * kWeighThreads < end) sum[x] = fmaf(exp2f(s[x * kWeighThreads] - st.x), st.y, sum[x]);
    }
#pragma unroll
    for (int x = 0; x < kWeighEach; ++x)
      if (p + x * kWeighThreads < end) w[p + x * kWeighThreads] = fmaf(a.decay, old[x], sum[x]);
  }
}

// ---- host ----------------------------------------------------------------------------------------

int num_sms_of(int device) {
  static int sms[64];  // the same value whoever writes it
  if (device < 0) return 0;
  if (device < 64 && sms[device] > 0) return sms[device];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (device < 64) sms[device] = n;
  return n;
}

// Parts of a request's positions in the kernel for any shape: enough for a few CTAs an SM.
int any_parts(const hs_config* c, int sms) {
  const int64_t rows = (int64_t)c->num_requests * c->num_q_heads;
  const int64_t p = (8ll * sms + rows - 1) / rows;
  return (int)(p < 1 ? 1 : p > kAnyParts ? kAnyParts : p);
}

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

struct Layout {  // of the workspace
  hs_prefix_plan tc;
  int parts;
  int64_t partials, stats, scores, cols, end;
};
int64_t score_cols(const hs_paged_kv* kv) {
  return up((int64_t)kv->max_pages * kv->page_tokens, 32) + 128;  // a last tile may reach beyond the positions
}
bool layout_of(const hs_config* c, const hs_paged_kv* kv, int groups, bool weigh, int sms, Layout* l) {
  l->tc = c->layout == HS_LAYOUT_GQA ? hs_prefix_gqa_plan(c, sms) : hs_prefix_mla_plan(c, sms);
  l->parts = any_parts(c, sms);
  const int64_t rows = l->tc.rows > 0 ? l->tc.rows : (int64_t)c->num_requests * c->num_q_heads * l->parts;
  const int64_t heads = (int64_t)c->num_requests * c->num_q_heads;
  l->cols = score_cols(kv);
  l->partials = up(hs_prefix_head_bytes(groups, c->num_requests), 32);
  l->stats = l->partials + up(rows * (c->head_dim_v + 4) * (int64_t)sizeof(float), 32);
  l->scores = l->stats + (weigh ? up(heads * (int64_t)sizeof(float2), 32) : 0);
  if (weigh && l->cols > (INT64_MAX / 8) / heads) return false;
  l->end = l->scores + (weigh ? heads * l->cols * (int64_t)sizeof(float) : 0) + 32;
  return true;
}

thread_local int stall_next;  // test hook, of the calling thread

int check_prefix(const hs_config* c, const hs_prefix_args* g) {
  if (g == nullptr || g->d_q == nullptr || g->d_len == nullptr || g->d_out == nullptr) return HS_ERR_ARG;
  if (!hs_aligned(g->d_q, 16) || !hs_aligned(g->d_len, 8) || !hs_aligned(g->d_out, 16) || !hs_aligned(g->d_groups, 4) ||
      !hs_aligned(g->d_prefix, 8) || !hs_aligned(g->d_weights, 4) || !hs_aligned(g->d_workspace, 16))
    return HS_ERR_ARG;
  if (g->groups < 0 || g->groups > c->num_requests) return HS_ERR_ARG;
  if (g->groups > 0 && (g->d_groups == nullptr || g->d_prefix == nullptr)) return HS_ERR_ARG;
  if (!isfinite(g->scale * kLog2e)) return HS_ERR_ARG;  // what the kernels multiply by
  if (g->d_weights != nullptr) {
    if ((g->lists != 1 && g->lists != c->num_kv_heads) || g->capacity < 1 || g->capacity > kMaxPositions || !isfinite(g->decay))
      return HS_ERR_ARG;
  }
  // outputs are written while other rows' queries are still read
  const uintptr_t rows = (uintptr_t)c->num_requests * c->num_q_heads, q = (uintptr_t)g->d_q, o = (uintptr_t)g->d_out;
  if (q < o + 2 * rows * c->head_dim_v && o < q + 2 * rows * c->head_dim_qk) return HS_ERR_ARG;
  return HS_OK;
}

}  // namespace

extern "C" int64_t hs_prefix_attn_workspace(const hs_config* cfg, const hs_paged_kv* kv, int groups, int weights) {
  int rc = hs_check_shape(cfg);
  if (rc == HS_OK) rc = hs_check_paged(cfg, kv);
  if (rc != HS_OK) return rc;
  if (groups < 0 || groups > cfg->num_requests) return HS_ERR_ARG;
  const int sms = num_sms_of(kv->cuda_device);
  if (sms < 1) return HS_ERR_CUDA;
  Layout l;
  return layout_of(cfg, kv, groups, weights != 0, sms, &l) ? l.end : (int64_t)HS_ERR_ARG;
}

extern "C" int hs_debug_stall_prefix(void) {
  stall_next = 1;
  return HS_OK;
}

extern "C" int hs_prefix_attn(const hs_config* cfg, const hs_paged_kv* kv, const hs_prefix_args* args, void* stream) {
  int rc = hs_check_shape(cfg);
  if (rc == HS_OK) rc = hs_check_paged(cfg, kv);
  if (rc == HS_OK) rc = check_prefix(cfg, args);
  if (rc != HS_OK) return rc;
  const hs_prefix_args& g = *args;
  HsOnDevice on(kv->cuda_device);
  if (!on.ok) return HS_ERR_CUDA;
  const int sms = num_sms_of(kv->cuda_device);
  if (sms < 1) return HS_ERR_CUDA;
  Layout l;
  const bool weigh = g.d_weights != nullptr;
  if (!layout_of(cfg, kv, g.groups, weigh, sms, &l)) return HS_ERR_ARG;
  if (g.d_workspace == nullptr || g.workspace_bytes < l.end) return HS_ERR_SCRATCH;
  uint8_t* ws = (uint8_t*)(((uintptr_t)g.d_workspace + 31u) & ~(uintptr_t)31u);
  PrefixArgs a{};
  a.kv = hs_paged_rows(cfg, kv);
  a.q = (const uint16_t*)g.d_q;
  a.len = g.d_len;
  a.groups = g.d_groups;
  a.prefix = g.d_prefix;
  a.out = (uint16_t*)g.d_out;
  a.R = cfg->num_requests;
  a.ngroups = g.groups;
  a.Hq = cfg->num_q_heads;
  a.Hkv = cfg->num_kv_heads;
  a.dqk = cfg->head_dim_qk;
  a.dv = cfg->head_dim_v;
  if (cfg->layout == HS_LAYOUT_GQA) {
    a.kstride = cfg->head_dim_qk + cfg->head_dim_v;
    a.voff = cfg->head_dim_qk;
  }
  a.qscale = g.scale * kLog2e;
  PrefixSplit head;
  hs_prefix_head(ws, g.groups, &head);
  if (weigh) {
    a.weights = g.d_weights;
    a.cap = g.capacity;
    a.lists = g.lists;
    a.decay = g.decay;
    a.stats = (float2*)(ws + l.stats);
    a.scores = (float*)(ws + l.scores);
    a.score_cols = l.cols;
  }
  cudaStream_t st = (cudaStream_t)stream;
  if (l.tc.rows > 0) {
    a.stall = stall_next;  // consumed by this launch
    stall_next = 0;
    rc = (cfg->layout == HS_LAYOUT_GQA ? hs_prefix_gqa_launch : hs_prefix_mla_launch)(cfg, &a, ws, ws + l.partials, sms, st);
    if (rc != HS_OK) return rc;
  } else {
    float* part = (float*)(ws + l.partials);
    float* ml = part + (int64_t)a.R * a.Hq * l.parts * a.dv;
    cudaError_t e = hs_launch_pdl(k_prefix_check, dim3(1), dim3(1024), 0, st, a, head.of);
    if (e == cudaSuccess)
      e = hs_launch_pdl(k_prefix_any, dim3(a.Hq, a.R, l.parts), dim3(kAnyWarps * 32), 0, st, a, (const PrefixRequest*)head.of, part, ml, l.parts);
    if (e == cudaSuccess)
      e = hs_launch_pdl(k_prefix_any_join, dim3((a.Hq * (a.dv / 8) + kAnyJoinThreads - 1) / kAnyJoinThreads, a.R),
                        dim3(kAnyJoinThreads), 0, st, a, (const float*)part, (const float*)ml, l.parts);
    if (e != cudaSuccess) return HS_ERR_CUDA;
  }
  if (weigh) {
    // a few CTAs an SM in all; the positions that there are is known on the device alone
    const int64_t lists = (int64_t)a.R * a.lists, most = (a.cap + kWeighThreads * kWeighEach - 1) / (kWeighThreads * kWeighEach);
    int64_t ctas = (8ll * sms + lists - 1) / lists;
    ctas = ctas < 1 ? 1 : ctas > most ? most : ctas;
    if (hs_launch_pdl(k_prefix_weigh, dim3((unsigned)ctas, a.lists, a.R), dim3(kWeighThreads), 0, st, a, (const PrefixRequest*)head.of) !=
        cudaSuccess)
      return HS_ERR_CUDA;
  }
  return HS_OK;
}

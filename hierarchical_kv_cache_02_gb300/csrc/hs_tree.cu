// Attention for a tree of drafted tokens over a cache.
//
// For node i of request r and query head h, over the context's entries and the nodes that i sees:
//   s_e = scale <q, K(e)>,  o = sum_e 2^(s_e log2(e) - m) V(e) / sum_e 2^(s_e log2(e) - m).
// On the tensor cores a context record serves many (node, query head) rows at once: at few rows device memory bounds
// it, at many the products.  The kernel below, for every other shape, reads a record anew for each of them.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "hs_tree.cuh"

namespace {

// Any shape: a CTA per (node, query head, request), its four warps take the entries in turn and merge
// their running maxima, sums and accumulators at the end.  A lane holds every 32nd group of 8 values of
// a head (head dims up to 576 = 72 groups: at most three).  Latency of its loads bounds it, each warp's one record after
// the other: 16 requests x 8 nodes x 32 heads of 80 over 2048 listed positions 4.1 ms (plain torch products 0.70 ms, the
// tensor cores' kernel with heads of 128 0.041 ms); 1 request x 4 nodes x 1000 positions 321 us (plain 638 us).
constexpr int kAnyWarps = 4, kAnyGroups = 3;

__global__ void __launch_bounds__(kAnyWarps * 32) k_tree_any(TreeArgs a) {
  __shared__ float s_acc[kAnyWarps][kAnyGroups * 32 * 8];
  __shared__ float s_m[kAnyWarps], s_l[kAnyWarps];
  hs_pdl_wait();
  const int t = blockIdx.x / a.Hq, h = blockIdx.x - t * a.Hq, r = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t bad = 0u;
  const int64_t len = context_of(a, r, &bad);
  const int nn = nodes_of(a, r, &bad);
  const int64_t n = entries_of(a, r, len, &bad);
  if (t >= nn) {
    if (threadIdx.x == 0) report(a.kv.err, bad);
    return;
  }
  const int kg = a.dqk / 8, vg = a.dv / 8;
  const int64_t koff = (int64_t)(h / (a.Hq / a.Hkv)) * a.kstride;
  const int64_t row = ((int64_t)r * a.T + t) * a.Hq + h;
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
  const uint64_t* mask = a.mask + ((int64_t)r * a.T + t) * a.words;
  float m = -INFINITY, l = 0.f;
  for (int64_t e = warp; e < n + nn; e += kAnyWarps) {
    const uint8_t* rec;
    if (e < n) {
      rec = entry_record(a, r, e, &bad);
    } else {
      const int j = (int)(e - n);
      if (((mask[j >> 6] >> (j & 63)) & 1ull) == 0ull) continue;
      rec = node_record(a, r, len, j, &bad);
    }
    if (rec == nullptr) continue;
    const uint16_t* kp = (const uint16_t*)rec + koff;
    float s = 0.f;
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
    // -infinity: weight 0 whatever the maximum, but a value that is infinite or NaN counts.  NaN: fmaxf keeps the
    // maximum, the weight is NaN
    const float mn = fmaxf(m, s);
    const float al = m == mn ? 1.f : exp2f(m - mn), p = s == -INFINITY ? 0.f : exp2f(s - mn);
    m = mn;
    l = l * al + p;
#pragma unroll
    for (int x = 0; x < kAnyGroups; ++x) {
      const int gi = lane + 32 * x;
      if (gi < vg) {
        const uint4 u = *(const uint4*)(kp + a.voff + 8 * gi);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[x][2 * i] = fmaf(p, lo(w[i]), acc[x][2 * i] * al);
          acc[x][2 * i + 1] = fmaf(p, hi(w[i]), acc[x][2 * i + 1] * al);
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
  const float inv = L == 0.f ? 0.f : 1.f / L;
  for (int d = 2 * threadIdx.x; d < a.dv; d += 2 * kAnyWarps * 32) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kAnyWarps; ++w) {
      x = fmaf(wt[w], s_acc[w][d], x);
      y = fmaf(wt[w], s_acc[w][d + 1], y);
    }
    *(uint32_t*)(a.out + row * a.dv + d) = pack(x * inv, y * inv);
  }
}

int check_tree(const hs_config* c, const hs_tree_args* g) {
  if (g == nullptr) return HS_ERR_ARG;
  if (g->d_q == nullptr || g->d_mask == nullptr || g->d_out == nullptr) return HS_ERR_ARG;
  if (!hs_aligned(g->d_q, 16) || !hs_aligned(g->d_out, 16) || !hs_aligned(g->d_mask, 8) || !hs_aligned(g->d_locs, 4) ||
      !hs_aligned(g->d_nodes, 4) || !hs_aligned(g->d_len, 8) || !hs_aligned(g->d_workspace, 16))
    return HS_ERR_ARG;
  if (g->nodes < 1 || g->nodes > HS_MAX_TREE_NODES) return HS_ERR_ARG;
  if (!isfinite(g->scale * kLog2e)) return HS_ERR_ARG;  // what the kernels multiply by
  // outputs are written while other rows' queries are still read
  const uintptr_t rows = (uintptr_t)c->num_requests * g->nodes * c->num_q_heads, q = (uintptr_t)g->d_q, o = (uintptr_t)g->d_out;
  if (q < o + 2 * rows * c->head_dim_v && o < q + 2 * rows * c->head_dim_qk) return HS_ERR_ARG;
  return HS_OK;
}

TreeArgs tree_args(const hs_config* c, const hs_tree_args* g) {
  TreeArgs a{};
  a.q = (const uint16_t*)g->d_q;
  a.locs = g->d_locs;
  a.mask = g->d_mask;
  a.nodes = g->d_nodes;
  a.out = (uint16_t*)g->d_out;
  a.R = c->num_requests;
  a.T = g->nodes;
  a.words = (g->nodes + 63) / 64;
  a.Hq = c->num_q_heads;
  a.Hkv = c->num_kv_heads;
  a.dqk = c->head_dim_qk;
  a.dv = c->head_dim_v;
  if (c->layout == HS_LAYOUT_GQA) {
    a.kstride = c->head_dim_qk + c->head_dim_v;
    a.voff = c->head_dim_qk;
  }
  a.qscale = g->scale * kLog2e;
  return a;
}

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

// The tensor-core kernel for the shapes it takes, else the one for any shape.
int launch_tree(const hs_config* c, const hs_tree_args* g, const TreeArgs& a, int device, cudaStream_t st) {
  const int sms = num_sms_of(device);
  if (sms < 1) return HS_ERR_CUDA;
  const bool mla = c->layout == HS_LAYOUT_MLA;
  const hs_tree_plan p = mla ? hs_tree_mla_plan(c, g->nodes, sms) : hs_tree_gqa_plan(c, g->nodes, sms);
  if (p.usable) {
    if (g->d_workspace == nullptr || g->workspace_bytes < p.workspace) return HS_ERR_SCRATCH;
    return mla ? hs_tree_mla_launch(c, g, &a, sms, st) : hs_tree_gqa_launch(c, g, &a, sms, st);
  }
  const cudaError_t e = hs_launch_pdl(k_tree_any, dim3(a.T * a.Hq, a.R), dim3(kAnyWarps * 32), 0, st, a);
  return e == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

}  // namespace

extern "C" int64_t hs_tree_attn_workspace(const hs_config* cfg, int nodes, int cuda_device) {
  const int rc = hs_check_shape(cfg);
  if (rc != HS_OK) return rc;
  if (nodes < 1 || nodes > HS_MAX_TREE_NODES || cuda_device < 0) return HS_ERR_ARG;
  const int sms = num_sms_of(cuda_device);
  if (sms < 1) return HS_ERR_CUDA;
  return (cfg->layout == HS_LAYOUT_MLA ? hs_tree_mla_plan(cfg, nodes, sms) : hs_tree_gqa_plan(cfg, nodes, sms)).workspace;
}

extern "C" int hs_tree_attn(const hs_config* cfg, const hs_paged_kv* kv, const hs_tree_args* args, void* stream) {
  int rc = hs_check_shape(cfg);
  if (rc == HS_OK) rc = hs_check_paged(cfg, kv);
  if (rc == HS_OK) rc = check_tree(cfg, args);
  if (rc != HS_OK) return rc;
  if (args->d_len == nullptr || (args->d_locs != nullptr && (args->top_k < 1 || args->top_k > kMaxPositions)))
    return HS_ERR_ARG;
  HsOnDevice on(kv->cuda_device);
  if (!on.ok) return HS_ERR_CUDA;
  TreeArgs a = tree_args(cfg, args);
  a.kv = hs_paged_rows(cfg, kv);
  a.len = args->d_len;
  a.k = args->d_locs != nullptr ? args->top_k : 0;
  return launch_tree(cfg, args, a, kv->cuda_device, (cudaStream_t)stream);
}

extern "C" int hs_pool_tree_attn(hs_pool* pool, int layer, const hs_tree_args* args, const void* d_draft,
                                 void* stream) {
  if (pool == nullptr) return HS_ERR_ARG;
  const hs_config& c = pool->cfg;
  int rc = hs_check_shape(&c);
  if (rc == HS_OK) rc = check_tree(&c, args);
  if (rc != HS_OK) return rc;
  if (layer < 0 || layer >= c.num_layers || args->d_locs == nullptr || d_draft == nullptr || !hs_aligned(d_draft, 16))
    return HS_ERR_ARG;
  if (c.fetch_in_attention != 0) return HS_ERR_CONFIG;
  HsOnDevice on(pool->device);
  if (!on.ok) return HS_ERR_CUDA;
  TreeArgs a = tree_args(&c, args);
  a.kv.rec = pool->rec;
  a.kv.err = pool->err_global;
  a.slot_pt = pool->slot_table + (int64_t)layer * c.num_requests * pool->slot_pages;
  a.slot_cap = pool->slot_cap + (int64_t)layer * c.num_requests;
  a.slot_pages = pool->slot_pages;
  a.slot_shift = pool->slot_shift;
  a.draft = (const uint8_t*)d_draft;
  a.k = c.top_k;
  a.stall = (pool->debug_stall & HS_STALL_TREE) != 0;  // test hook, consumed by this launch
  pool->debug_stall &= ~HS_STALL_TREE;
  pool->last_res_layer = -1;  // an attention after this one waits for the whole stream
  return launch_tree(&c, args, a, pool->device, (cudaStream_t)stream);
}

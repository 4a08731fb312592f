// Rotate-and-append to a paged cache, and keeping the accepted path of a tree of drafts.
//
// Both move records and compute next to nothing, so device memory bounds the large calls and latency
// the small ones.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "hs_paged.cuh"

namespace {

// ---- append ------------------------------------------------------------------------------------
//
// Rotation of a pair (x, y) by the angle phi = a * inv_freq_j of position a:
//   x' = x cos phi - y sin phi,  y' = y cos phi + x sin phi.
// The angle is reduced in integers: a * turns_j mod 2^64 is the fraction of a turn exactly, so far
// positions lose nothing; its top 32 bits, as a signed number of half turns, go through sincospif.

constexpr int kAppThreads = 256;
constexpr int kAppTokens = 4;  // tokens of a CTA

struct AppendArgs {
  PagedRows kv;
  const int32_t* cu;
  const int64_t* start;
  const int64_t* rope_pos;
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  const uint64_t* turns;
  int64_t kts, khs, vts, vhs, qts, qhs, ots, ohs;  // strides in values
  int R, N, Hkv, Hq, dqk, dv;                      // dv = 0: the record is the key alone (shared latent)
  int half, k_off, q_off, q_dim, interleaved;      // half = rotary_dim / 2
};

struct Vec8 {
  uint32_t w[4];
};
__device__ __forceinline__ Vec8 ld8(const uint16_t* p) {
  const uint4 u = *(const uint4*)p;
  return Vec8{{u.x, u.y, u.z, u.w}};
}
__device__ __forceinline__ void st8(uint16_t* p, const Vec8& v) {
  *(uint4*)p = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}
__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *(const uint32_t*)&v;
}

// Units of one head: each moves 8 or 16 values.  A half-form unit u < half / 8 turns values 8u.. with
// their partners half further on; an interleaved unit u < half / 4 turns the four pairs of values 8u..;
// the remaining units copy 8 values each.
__device__ __forceinline__ int head_units(int dim, int half, int interleaved) {
  return interleaved ? dim / 8 : dim / 8 - half / 8;
}

__device__ __forceinline__ void turn_unit(const uint16_t* src, uint16_t* dst, int u, int off, int half, int interleaved,
                                          const float2* cs) {
  if (interleaved) {
    const int d = 8 * u;  // values in record order; the rotated ones are [off, off + 2 half)
    Vec8 x = ld8(src + d);
    const int j = (d - off) >> 1;
    if (d >= off && j < half) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 c = cs[j + i];
        const float a = lo(x.w[i]), b = hi(x.w[i]);
        x.w[i] = pack(a * c.x - b * c.y, b * c.x + a * c.y);
      }
    }
    st8(dst + d, x);
    return;
  }
  if (u < half / 8) {
    const int j = 8 * u;
    Vec8 x = ld8(src + off + j), y = ld8(src + off + half + j);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 c0 = cs[j + 2 * i], c1 = cs[j + 2 * i + 1];
      const float a0 = lo(x.w[i]), a1 = hi(x.w[i]), b0 = lo(y.w[i]), b1 = hi(y.w[i]);
      x.w[i] = pack(a0 * c0.x - b0 * c0.y, a1 * c1.x - b1 * c1.y);
      y.w[i] = pack(b0 * c0.x + a0 * c0.y, b1 * c1.x + a1 * c1.y);
    }
    st8(dst + off + j, x);
    st8(dst + off + half + j, y);
    return;
  }
  int d = 8 * (u - half / 8);  // the values that are only copied: before and behind the rotated ones
  if (d >= off) d += 2 * half;
  st8(dst + d, ld8(src + d));
}

__global__ void __launch_bounds__(kAppThreads) k_append_rotated(AppendArgs a) {
  extern __shared__ float2 s_cs[];                 // [kAppTokens][half] cosine and sine of each pair
  __shared__ int64_t s_row[kAppTokens], s_pos[kAppTokens];  // record row (-1: not stored), angle position
  __shared__ int s_live[kAppTokens];
  hs_pdl_wait();
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * kAppTokens, nt = min(kAppTokens, a.N - t0);
  if (tid < nt) {
    const int t = t0 + tid;
    // the last request whose first token is not behind t
    int x = 0, y = a.R;
    while (y - x > 1) {
      const int m = (x + y) >> 1;
      if (a.cu[m] <= t) x = m;
      else y = m;
    }
    const int c0 = a.cu[x], c1 = a.cu[x + 1];
    const bool live = c0 <= t && t < c1;
    int64_t row = -1, pos = 0;
    if (live) {
      uint32_t bad = 0u;
      pos = a.start[x] + (t - c0);
      row = paged_row(a.kv, x, pos, (uint32_t)HS_DEVERR_APPEND, &bad);
      report(a.kv.err, bad);
      if (a.rope_pos != nullptr) pos = a.rope_pos[t];
    }
    s_live[tid] = live;
    s_row[tid] = row;
    s_pos[tid] = pos;
  }
  __syncthreads();
  for (int i = tid; i < nt * a.half; i += kAppThreads) {
    const int t = i / a.half, j = i - t * a.half;
    const uint64_t turn = (uint64_t)s_pos[t] * a.turns[j];
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    s_cs[i] = make_float2(c, s);
  }
  __syncthreads();
  const int head_rec = a.dqk + a.dv;
  // keys
  const int ku = head_units(a.dqk, a.half, a.interleaved), kn = a.Hkv * ku;
  for (int i = tid; i < nt * kn; i += kAppThreads) {
    const int t = i / kn, w = i - t * kn, h = w / ku, u = w - h * ku;
    if (s_row[t] < 0) continue;
    turn_unit(a.k + (int64_t)(t0 + t) * a.kts + (int64_t)h * a.khs,
              (uint16_t*)(a.kv.base + s_row[t] * a.kv.rec) + h * head_rec, u, a.k_off, a.half, a.interleaved,
              s_cs + t * a.half);
  }
  // values
  if (a.dv > 0) {
    const int vu = a.dv / 8, vn = a.Hkv * vu;
    for (int i = tid; i < nt * vn; i += kAppThreads) {
      const int t = i / vn, w = i - t * vn, h = w / vu, u = w - h * vu;
      if (s_row[t] < 0) continue;
      st8((uint16_t*)(a.kv.base + s_row[t] * a.kv.rec) + h * head_rec + a.dqk + 8 * u,
          ld8(a.v + (int64_t)(t0 + t) * a.vts + (int64_t)h * a.vhs + 8 * u));
    }
  }
  // queries
  if (a.q != nullptr) {
    const int qu = head_units(a.q_dim, a.half, a.interleaved), qn = a.Hq * qu;
    for (int i = tid; i < nt * qn; i += kAppThreads) {
      const int t = i / qn, w = i - t * qn, h = w / qu, u = w - h * qu;
      if (!s_live[t]) continue;
      turn_unit(a.q + (int64_t)(t0 + t) * a.qts + (int64_t)h * a.qhs,
                a.q_out + (int64_t)(t0 + t) * a.ots + (int64_t)h * a.ohs, u, a.q_off, a.half, a.interleaved,
                s_cs + t * a.half);
    }
  }
}

// ---- keep path ---------------------------------------------------------------------------------
//
// Node i of the path moves from row path[i] >= i to row i behind the context.  A thread owns a 16-byte
// column of a request's records and moves it for all nodes in order, so no thread reads what another
// writes; in a batch of loads before its stores, a store goes to row i and every later load reads a row
// path[j] >= j > i, so nothing is overwritten before it is read.

constexpr int kKeepThreads = 128;
constexpr int kKeepBatch = 8;  // records in flight per thread

__global__ void __launch_bounds__(kKeepThreads) k_keep_path(PagedRows kv, const int64_t* len, const int32_t* path,
                                                            int path_len, const int32_t* count) {
  hs_pdl_wait();
  const int r = blockIdx.y;
  const int col = blockIdx.x * kKeepThreads + threadIdx.x;
  const int cols = (int)(kv.rec / 16);
  uint32_t bad = 0u;
  const int given = count[r];
  const int n = min(max(given, 0), path_len);
  if (n != given) bad |= (uint32_t)HS_DEVERR_LOC;
  const int64_t base = len[r];
  for (int i0 = 0; i0 < n; i0 += kKeepBatch) {
    uint4 v[kKeepBatch];
    int64_t to[kKeepBatch];
#pragma unroll
    for (int x = 0; x < kKeepBatch; ++x) {
      to[x] = -1;
      if (i0 + x < n) {
        const int p = path[(int64_t)r * path_len + i0 + x];
        if (p < i0 + x) {
          bad |= (uint32_t)HS_DEVERR_LOC;
        } else {
          const int64_t src = paged_row(kv, r, base + p, (uint32_t)HS_DEVERR_LOC, &bad);
          to[x] = paged_row(kv, r, base + i0 + x, (uint32_t)HS_DEVERR_LOC, &bad);
          if (src < 0 || src == to[x]) to[x] = -1;
          if (to[x] >= 0 && col < cols) v[x] = *(const uint4*)(kv.base + src * kv.rec + (int64_t)col * 16);
        }
      }
    }
#pragma unroll
    for (int x = 0; x < kKeepBatch; ++x)
      if (to[x] >= 0 && col < cols) *(uint4*)(kv.base + to[x] * kv.rec + (int64_t)col * 16) = v[x];
  }
  if (threadIdx.x == 0) report(kv.err, bad);
}

// 2^256 / (2 pi), lowest word first
constexpr uint64_t kOverTwoPi[4] = {0x7f9458eaf7aef158ull, 0x36d8a5664f10e410ull, 0x7f09d5f47d4d3770ull, 0x28be60db9391054aull};

bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0; }

}  // namespace

extern "C" int hs_rope_turns(const double* h_inv_freq, int n, uint64_t* h_turns) {
  if (n < 0 || (n > 0 && (h_inv_freq == nullptr || h_turns == nullptr))) return HS_ERR_ARG;
  for (int i = 0; i < n; ++i) {
    if (!(fabs(h_inv_freq[i]) < 0x1p32)) return HS_ERR_ARG;
    // |f| = m 2^e with an integer m < 2^53, e <= -21: f / (2 pi) 2^64 = m C 2^(e - 192), to the nearest
    int e = 0;
    const uint64_t m = (uint64_t)ldexp(frexp(fabs(h_inv_freq[i]), &e), 53);
    e -= 53;
    uint64_t p[6] = {0, 0, 0, 0, 0, 0};  // m C, below 2^307
    unsigned __int128 carry = 0;
    for (int w = 0; w < 4; ++w) {
      carry += (unsigned __int128)m * kOverTwoPi[w];
      p[w] = (uint64_t)carry;
      carry >>= 64;
    }
    p[4] = (uint64_t)carry;
    const int sh = 192 - e;  // >= 213
    uint64_t t = 0;
    if (sh < 320) {
      const int w = sh >> 6, b = sh & 63;
      t = b == 0 ? p[w] : (p[w] >> b) | (p[w + 1] << (64 - b));
      t += (b == 0 ? p[w - 1] >> 63 : p[w] >> (b - 1)) & 1u;
    }
    h_turns[i] = h_inv_freq[i] < 0 ? 0ull - t : t;
  }
  return HS_OK;
}

extern "C" int hs_append_rotated(const hs_config* cfg, const hs_paged_kv* kv, const hs_append_args* args,
                                 void* stream) {
  int rc = hs_check_shape(cfg);
  if (rc == HS_OK) rc = hs_check_paged(cfg, kv);
  if (rc != HS_OK) return rc;
  if (args == nullptr || args->num_tokens < 0) return HS_ERR_ARG;
  const hs_append_args& g = *args;
  const bool mla = cfg->layout == HS_LAYOUT_MLA;
  if (g.num_tokens == 0) return HS_OK;
  if (g.d_cu == nullptr || g.d_start == nullptr || !hs_aligned(g.d_cu, 4) || !hs_aligned(g.d_start, 8) ||
      !hs_aligned(g.d_rope_pos, 8))
    return HS_ERR_ARG;
  if (g.d_k == nullptr || (g.d_v == nullptr) != mla) return HS_ERR_ARG;
  if (!hs_aligned(g.d_k, 16) || !stride_ok(g.k_token_stride) || !stride_ok(g.k_head_stride)) return HS_ERR_ARG;
  if (!mla && (!hs_aligned(g.d_v, 16) || !stride_ok(g.v_token_stride) || !stride_ok(g.v_head_stride))) return HS_ERR_ARG;
  if (g.rotary_dim < 0 || g.rotary_dim % 16 != 0 || g.rotary_offset < 0 || g.rotary_offset % 8 != 0 ||
      g.rotary_offset > cfg->head_dim_qk - g.rotary_dim || (g.interleaved != 0 && g.interleaved != 1))
    return HS_ERR_ARG;
  if (g.rotary_dim > 0 && (g.d_turns == nullptr || !hs_aligned(g.d_turns, 8))) return HS_ERR_ARG;
  if (g.d_q != nullptr) {
    if (g.d_q_out == nullptr || !hs_aligned(g.d_q, 16) || !hs_aligned(g.d_q_out, 16) || !stride_ok(g.q_token_stride) ||
        !stride_ok(g.q_head_stride) || !stride_ok(g.q_out_token_stride) || !stride_ok(g.q_out_head_stride))
      return HS_ERR_ARG;
    if ((g.q_out_token_stride == 0 && g.num_tokens > 1) || (g.q_out_head_stride == 0 && cfg->num_q_heads > 1))
      return HS_ERR_ARG;  // every query would be written over the others
    if (g.q_dim != cfg->head_dim_qk && (g.q_dim != g.rotary_dim || g.q_dim == 0)) return HS_ERR_ARG;
  }
  HsOnDevice on(kv->cuda_device);
  if (!on.ok) return HS_ERR_CUDA;
  AppendArgs a{};
  a.kv = hs_paged_rows(cfg, kv);
  a.cu = g.d_cu;
  a.start = g.d_start;
  a.rope_pos = g.d_rope_pos;
  a.k = (const uint16_t*)g.d_k;
  a.v = (const uint16_t*)g.d_v;
  a.q = (const uint16_t*)g.d_q;
  a.q_out = (uint16_t*)g.d_q_out;
  a.turns = g.d_turns;
  a.kts = g.k_token_stride;
  a.khs = g.k_head_stride;
  a.vts = g.v_token_stride;
  a.vhs = g.v_head_stride;
  a.qts = g.q_token_stride;
  a.qhs = g.q_head_stride;
  a.ots = g.q_out_token_stride;
  a.ohs = g.q_out_head_stride;
  a.R = cfg->num_requests;
  a.N = g.num_tokens;
  a.Hkv = cfg->num_kv_heads;
  a.Hq = cfg->num_q_heads;
  a.dqk = cfg->head_dim_qk;
  a.dv = mla ? 0 : cfg->head_dim_v;
  a.half = g.rotary_dim / 2;
  a.k_off = g.rotary_offset;
  a.q_off = g.q_dim == cfg->head_dim_qk ? g.rotary_offset : 0;
  a.q_dim = g.q_dim;
  a.interleaved = g.interleaved;
  const size_t smem = (size_t)kAppTokens * a.half * sizeof(float2);
  const cudaError_t e = hs_launch_pdl(k_append_rotated, dim3((a.N + kAppTokens - 1) / kAppTokens), dim3(kAppThreads), smem,
                                      (cudaStream_t)stream, a);
  return e == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

extern "C" int hs_keep_path(const hs_config* cfg, const hs_paged_kv* kv, const int64_t* d_len, const int32_t* d_path,
                            int path_len, const int32_t* d_count, void* stream) {
  int rc = hs_check_shape(cfg);
  if (rc == HS_OK) rc = hs_check_paged(cfg, kv);
  if (rc != HS_OK) return rc;
  if (path_len < 0 || path_len > HS_MAX_TREE_NODES) return HS_ERR_ARG;
  if (path_len == 0) return HS_OK;
  if (d_len == nullptr || d_path == nullptr || d_count == nullptr || !hs_aligned(d_len, 8) || !hs_aligned(d_path, 4) ||
      !hs_aligned(d_count, 4))
    return HS_ERR_ARG;
  HsOnDevice on(kv->cuda_device);
  if (!on.ok) return HS_ERR_CUDA;
  const PagedRows p = hs_paged_rows(cfg, kv);
  const int cols = (int)(p.rec / 16);
  const cudaError_t e = hs_launch_pdl(k_keep_path, dim3((cols + kKeepThreads - 1) / kKeepThreads, cfg->num_requests),
                                      dim3(kKeepThreads), 0, (cudaStream_t)stream, p, d_len, d_path, path_len, d_count);
  return e == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

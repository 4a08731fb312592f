// Append to a paged cache with the norms of queries and keys and the rotation, by one or several axes of positions, in
// one pass.
//
// A head x of d values becomes  y_i = x_i w_i / sqrt(sum_j x_j^2 / d + eps)  and then each of its rotary pairs turns by
// the angle of that pair's axis: phi_j = pos[axis_j] * inv_freq_j, reduced in integers as in hs_spec.cu.  Squares are summed,
// and everything up to the one rounding at the end is done, in 32 bits.
// A token's record and queries are read once and written once: device memory bounds the large calls, latency the small.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "hs_append.cuh"

namespace {

// A head lies over a group of 4 to 32 neighbouring lanes (a power of two), a unit of two vectors each, so that the sum of its
// squares is a few shuffles; heads of more than 32 units (the latent's 36) have a second unit a lane.  The heads of
// a kind (keys, values, queries) of all tokens of a CTA stand one behind the other, 32 / group of them a warp.

constexpr int kThreads = 256;
constexpr int kTokens = 4;  // tokens of a CTA at most

struct Kind {
  const uint16_t* src;
  int64_t ts, hs;      // strides in values
  Div heads;
  int lanes;           // log2 of a head's lanes
  int units, dim, half, off;  // half: rotary pairs (0: none), off: the first rotary value
  int norm;            // the first values that are normed, a multiple of 8; 0: none
  const void* w;       // weights [norm] or [heads][norm]
  int64_t whs;
  int wide;            // weights of 32 bits, else bf16
  int first;           // the kind's first warp task
};

struct NormArgs {
  PagedRows kv;
  const int32_t* cu;
  const int64_t* start;
  const int64_t* rope_pos;
  const uint64_t* turns;
  const uint8_t* axis;  // of each pair, or null: 0
  uint16_t* q_out;
  int64_t ots, ohs;
  int R, N, dqk, dv, half, interleaved, axes;
  float eps;
  Kind kind[3];         // keys, values, queries
  int tasks, per_cta, tokens;
  Div angles;
};

// Unit u of a head: its first value, the distance to its second vector (0: none), and each vector's first pair (-1: not turned)
struct Place {
  int d, second, j, j2;
};
__device__ __forceinline__ Place place_of(const Kind& k, int u, int interleaved) {
  Place p;
  p.j = p.j2 = -1;
  if (k.half == 0 || interleaved) {
    p.d = 16 * u;
    p.second = p.d + 8 < k.dim ? 8 : 0;
    const int j = (p.d - k.off) >> 1;  // d and off are multiples of 8: a vector is rotary or it is not
    if (p.d >= k.off && j < k.half) p.j = j;
    if (p.d + 8 >= k.off && j + 4 < k.half) p.j2 = j + 4;
  } else if (8 * u < k.half) {
    p.d = k.off + 8 * u;
    p.second = k.half;
    p.j = 8 * u;
  } else {
    const int v = 16 * u - 2 * k.half, gap = 2 * k.half;
    p.d = v + (v >= k.off ? gap : 0);
    p.second = v + 8 < k.dim - gap ? v + 8 + (v + 8 >= k.off ? gap : 0) - p.d : 0;
  }
  return p;
}

__device__ __forceinline__ float squares(const Vec8& v) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) s = fmaf(hi(v.w[i]), hi(v.w[i]), fmaf(lo(v.w[i]), lo(v.w[i]), s));
  return s;
}
__device__ __forceinline__ void widen(const Vec8& v, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = lo(v.w[i]);
    x[2 * i + 1] = hi(v.w[i]);
  }
}
__device__ __forceinline__ Vec8 narrow(const float (&x)[8]) {
  return Vec8{{pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]), pack(x[6], x[7])}};
}
// times r and the weights from value d on
__device__ __forceinline__ void scale(float (&x)[8], const Kind& k, int h, int d, float r) {
  const int64_t at = (int64_t)h * k.whs + d;
  float w[8];
  if (k.wide) {
    const float4 a = *(const float4*)((const float*)k.w + at), b = *(const float4*)((const float*)k.w + at + 4);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  } else {
    widen(ld8((const uint16_t*)k.w + at), w);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
}
// the four pairs (x0, x1), (x2, x3), ... by c, s of each
__device__ __forceinline__ void turn_inside(float (&x)[8], const float2* cs) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 c = cs[i];
    const float p = x[2 * i], r = x[2 * i + 1];
    x[2 * i] = p * c.x - r * c.y;
    x[2 * i + 1] = r * c.x + p * c.y;
  }
}

// PER: units of a lane.  FLIGHT: heads whose loads are on their way at once.
template <int PER, int FLIGHT>
__global__ void __launch_bounds__(kThreads) k_append_normed(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) float2 s_cs[];  // [tokens][half] cosine and sine of each pair
  __shared__ int64_t s_row[kTokens], s_pos[kTokens][HS_MAX_AXES];
  __shared__ int s_live[kTokens];
  hs_pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.N - t0);
  for (int w = warp; w < nt; w += kThreads / 32) {  // a warp a token
    const int t = t0 + w;
    const int64_t given = a.rope_pos != nullptr && lane < a.axes ? a.rope_pos[(int64_t)t * a.axes + lane] : 0;
    const int x = request_of_token(a.cu, a.R, t, lane);
    const int c0 = a.cu[x], c1 = a.cu[x + 1];
    const bool live = c0 <= t && t < c1;
    const int64_t pos = a.start[x] + ((int64_t)t - c0);
    if (lane == 0) {
      uint32_t bad = 0u;
      s_row[w] = live ? paged_row(a.kv, x, pos, (uint32_t)HS_DEVERR_APPEND, &bad) : -1;
      s_live[w] = live;
      if (blockIdx.y == 0) report(a.kv.err, bad);
    }
    if (lane < a.axes) s_pos[w][lane] = a.rope_pos != nullptr ? given : pos;
  }
  __syncthreads();
  for (uint32_t i = tid; i < (uint32_t)(nt * a.half); i += kThreads) {
    const uint32_t t = a.angles(i), j = i - t * a.angles.d;
    const int x = a.axis != nullptr ? min((int)a.axis[j], a.axes - 1) : 0;
    const uint64_t turns = (uint64_t)s_pos[t][x] * a.turns[j];
    float s, c;
    sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
    s_cs[i] = make_float2(c, s);
  }
  __syncthreads();
  const int end = min(a.tasks, (int)(blockIdx.y + 1) * a.per_cta);
#pragma unroll 1
  for (int task0 = (int)blockIdx.y * a.per_cta + warp; task0 < end; task0 += FLIGHT * (kThreads / 32)) {
    Vec8 x[FLIGHT][PER], y[FLIGHT][PER];
    float sum[FLIGHT];
    // the loads of all heads in hand
#pragma unroll
    for (int f = 0; f < FLIGHT; ++f) {
      const int task = task0 + f * (kThreads / 32);
      sum[f] = 0.f;
      if (task >= end) continue;
      const int kn = (task >= a.kind[1].first) + (task >= a.kind[2].first);
      const Kind& k = a.kind[kn];
      const uint32_t slot = (uint32_t)(task - k.first) * 32u + lane, row = slot >> k.lanes, t = k.heads(row), h = row - t * k.heads.d;
      const bool on = t < (uint32_t)nt && (kn == 2 ? s_live[t] != 0 : s_row[t] >= 0);
#pragma unroll
      for (int p = 0; p < PER; ++p) {
        const int u = (int)(slot & ((1u << k.lanes) - 1u)) + (p << 5);
        if (!on || u >= k.units) continue;
        const Place at = place_of(k, u, a.interleaved);
        const uint16_t* src = k.src + (int64_t)(t0 + (int)t) * k.ts + (int64_t)h * k.hs + at.d;
        x[f][p] = ld8(src);
        if (at.second != 0) y[f][p] = ld8(src + at.second);
      }
    }
#pragma unroll
    for (int f = 0; f < FLIGHT; ++f) {
      const int task = task0 + f * (kThreads / 32);
      if (task >= end) continue;
      const int kn = (task >= a.kind[1].first) + (task >= a.kind[2].first);
      const Kind& k = a.kind[kn];
      const uint32_t slot = (uint32_t)(task - k.first) * 32u + lane, row = slot >> k.lanes, t = k.heads(row), h = row - t * k.heads.d;
      const bool on = t < (uint32_t)nt && (kn == 2 ? s_live[t] != 0 : s_row[t] >= 0);
      float r = 1.f;
      if (k.norm != 0) {  // the same for the whole warp
#pragma unroll
        for (int p = 0; p < PER; ++p) {
          const int u = (int)(slot & ((1u << k.lanes) - 1u)) + (p << 5);
          if (!on || u >= k.units) continue;
          const Place at = place_of(k, u, a.interleaved);
          if (at.d < k.norm) sum[f] += squares(x[f][p]);
          if (at.second != 0 && at.d + at.second < k.norm) sum[f] += squares(y[f][p]);
        }
#pragma unroll 1
        for (int o = 1; o < 1 << k.lanes; o <<= 1) sum[f] += __shfl_xor_sync(0xffffffffu, sum[f], o);
        r = rsqrtf(sum[f] / (float)k.norm + a.eps);
      }
      if (!on) continue;
      uint16_t* dst = kn == 2 ? a.q_out + (int64_t)(t0 + (int)t) * a.ots + (int64_t)h * a.ohs
                              : (uint16_t*)(a.kv.base + s_row[t] * a.kv.rec) + (int)h * (a.dqk + a.dv) + (kn == 1 ? a.dqk : 0);
      const float2* cs = s_cs + t * a.half;
#pragma unroll
      for (int p = 0; p < PER; ++p) {
        const int u = (int)(slot & ((1u << k.lanes) - 1u)) + (p << 5);
        if (u >= k.units) continue;
        const Place at = place_of(k, u, a.interleaved);
        if (k.norm != 0 || at.j >= 0 || at.j2 >= 0) {
          float v[8], w[8];
          widen(x[f][p], v);
          widen(y[f][p], w);
          if (at.d < k.norm) scale(v, k, h, at.d, r);
          if (at.second != 0 && at.d + at.second < k.norm) scale(w, k, h, at.d + at.second, r);
          if (a.interleaved) {
            if (at.j >= 0) turn_inside(v, cs + at.j);
            if (at.j2 >= 0) turn_inside(w, cs + at.j2);
          } else if (at.j >= 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 c = cs[at.j + i];
              const float v0 = v[i], w0 = w[i];
              v[i] = v0 * c.x - w0 * c.y;
              w[i] = w0 * c.x + v0 * c.y;
            }
          }
          x[f][p] = narrow(v);
          y[f][p] = narrow(w);
        }
        st8(dst + at.d, x[f][p]);
        if (at.second != 0) st8(dst + at.d + at.second, y[f][p]);
      }
    }
  }
}

int log2_up(int n) {
  int b = 0;
  while ((1 << b) < n) ++b;
  return b;
}

}  // namespace

extern "C" int hs_append_normed(const hs_config* cfg, const hs_paged_kv* kv, const hs_append_args* args,
                                const hs_norm_args* norm, void* stream) {
  const int rc = check_append(cfg, kv, args);
  if (rc != HS_OK) return rc;
  if (norm == nullptr) return HS_ERR_ARG;
  const hs_append_args& g = *args;
  const hs_norm_args& n = *norm;
  const bool mla = cfg->layout == HS_LAYOUT_MLA;
  if (g.num_tokens == 0) return HS_OK;
  if (n.axes < 1 || n.axes > HS_MAX_AXES || (n.axes > 1 && (n.d_axis == nullptr || g.d_rope_pos == nullptr))) return HS_ERR_ARG;
  for (int q = 0; q < 2; ++q) {
    const void* w = q ? n.d_q_weight : n.d_k_weight;
    const int type = q ? n.q_weight_type : n.k_weight_type;
    const int64_t hs = q ? n.q_weight_head_stride : n.k_weight_head_stride;
    if (w == nullptr) continue;
    if (!hs_aligned(w, 16) || (type != HS_WEIGHT_BF16 && type != HS_WEIGHT_FP32) || !stride_ok(hs)) return HS_ERR_ARG;
    if (!(n.eps > 0.f) || !isfinite(n.eps)) return HS_ERR_ARG;
    // a latent's queries are products of the key's up-projection: a norm over them has no meaning there
    if (q && (g.d_q == nullptr || mla || g.q_dim != cfg->head_dim_qk)) return HS_ERR_ARG;
  }
  HsOnDevice on(kv->cuda_device);
  if (!on.ok) return HS_ERR_CUDA;
  NormArgs a{};
  a.kv = hs_paged_rows(cfg, kv);
  a.cu = g.d_cu;
  a.start = g.d_start;
  a.rope_pos = g.d_rope_pos;
  a.turns = g.d_turns;
  a.axis = n.axes > 1 ? n.d_axis : nullptr;
  a.q_out = (uint16_t*)g.d_q_out;
  a.ots = g.q_out_token_stride;
  a.ohs = g.q_out_head_stride;
  a.R = cfg->num_requests;
  a.N = g.num_tokens;
  a.dqk = cfg->head_dim_qk;
  a.dv = mla ? 0 : cfg->head_dim_v;
  a.half = g.rotary_dim / 2;
  a.interleaved = g.interleaved;
  a.axes = n.axes;
  a.eps = n.eps;
  a.angles = div_by(a.half);
  int most = 0, heads = 0;  // units of a head, heads of a token
  for (int x = 0; x < 3; ++x) {
    Kind& k = a.kind[x];
    const int H = x == 0 ? cfg->num_kv_heads : x == 1 ? (mla ? 0 : cfg->num_kv_heads) : (g.d_q != nullptr ? cfg->num_q_heads : 0);
    k.src = (const uint16_t*)(x == 0 ? g.d_k : x == 1 ? g.d_v : g.d_q);
    k.ts = x == 0 ? g.k_token_stride : x == 1 ? g.v_token_stride : g.q_token_stride;
    k.hs = x == 0 ? g.k_head_stride : x == 1 ? g.v_head_stride : g.q_head_stride;
    k.dim = x == 0 ? a.dqk : x == 1 ? a.dv : g.q_dim;
    k.half = x == 1 ? 0 : a.half;
    k.off = x == 0 || (x == 2 && g.q_dim == cfg->head_dim_qk) ? g.rotary_offset : 0;
    k.w = x == 0 ? n.d_k_weight : x == 2 ? n.d_q_weight : nullptr;
    k.wide = (x == 0 ? n.k_weight_type : n.q_weight_type) == HS_WEIGHT_FP32;
    k.whs = x == 0 ? n.k_weight_head_stride : n.q_weight_head_stride;
    k.norm = k.w == nullptr ? 0 : mla ? cfg->head_dim_v : k.dim;
    k.heads = div_by(H);
    k.units = H > 0 ? head_units(k.dim, k.half, a.interleaved) : 0;
    k.lanes = log2_up(k.units < 32 ? k.units : 32);
    if (k.units > most) most = k.units;
    heads += H;
  }
  auto tasks_of = [&](int x, int tokens) {
    const Kind& k = a.kind[x];
    return k.units == 0 ? 0 : (int)((((int64_t)tokens * k.heads.d << k.lanes) + 31) >> 5);
  };
  auto tasks = [&](int tokens) { return tasks_of(0, tokens) + tasks_of(1, tokens) + tasks_of(2, tokens); };
  // as many tokens a CTA, and as many CTAs a token, as in hs_append_rotated
  a.tokens = kTokens;
  while (a.tokens > 1 && a.N < kMinCtas * a.tokens) a.tokens >>= 1;
  a.kind[1].first = tasks_of(0, a.tokens);
  a.kind[2].first = a.kind[1].first + tasks_of(1, a.tokens);
  a.tasks = tasks(a.tokens);
  const int ctas = (int)(((int64_t)a.N + a.tokens - 1) / a.tokens);
  int shares = 1;
  while (shares < 64 && (int64_t)ctas * shares < 2 * kSmsHint && a.tasks / shares > kThreads / 32) shares *= 2;
  a.per_cta = (a.tasks + shares - 1) / shares;
  const size_t smem = (size_t)a.tokens * a.half * sizeof(float2);
  const dim3 grid(ctas, shares), block(kThreads);
  const cudaError_t e = most > 32 ? hs_launch_pdl(k_append_normed<2, 1>, grid, block, smem, (cudaStream_t)stream, a)
                                  : hs_launch_pdl(k_append_normed<1, 2>, grid, block, smem, (cudaStream_t)stream, a);
  return e == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

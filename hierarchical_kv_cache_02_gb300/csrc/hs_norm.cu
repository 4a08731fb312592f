// Append to a paged cache with the norms of queries and keys and the rotation, by one or several axes of positions, in
// one pass.
//
// A head x of d values becomes  y_i = x_i w_i / sqrt(sum_j x_j^2 / d + eps)  and then each of its rotary pairs turns by
// the angle of that pair's axis: phi_j = pos[axis_j] * inv_freq_j, reduced in integers as in hs_spec.cu.  Squares are summed,
// and everything up to the one rounding at the end is done, in 32 bits.
// A token's record and queries are read once and written once: device memory bounds the large calls, latency the small.  16384
// tokens of 32 + 8 + 8 heads of 128 take 68.6 us, 5.9 TB/s, 8191 of 64 + 1 latent heads 29.4 (5.2), 6001 of three axes 33.5 (5.1), 16 4.5.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "hs_append.cuh"

namespace {

// A head lies over a group of 1 to 32 neighbouring lanes (a power of two), a unit of two vectors each, so that the sum of its
// squares is a few shuffles; heads of more than 32 units (the latent's 36) have a second unit a lane.  The heads of a kind
// (keys, values, queries) stand one behind the other, 32 / group of them a warp, and a warp does the same heads of one token
// after the other, so that places and weights are found once: what a token costs then is its loads, about 110 instructions a
// warp, its stores.  The loads go to shared memory, kAhead tokens ahead, each lane's to places of its own (in registers there is
// room for two tokens: 91 us instead of 73 on 16384 tokens of 32 + 8 + 8 heads of 128, when that was tried).  A CTA takes a run of
// tokens, finds their records' places first and the sines and cosines a few tokens ahead.

constexpr int kMaxWarps = 12;
constexpr int kRun = 64;    // tokens of a CTA at most
constexpr int kStage = 8;   // tokens whose angles are at hand; two stages
constexpr int kCtas = 2;    // CTAs of kMaxWarps an SM
constexpr int kAhead = 4;   // units of a lane on their way

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
  float per;           // 1 / norm
  int first;           // the kind's first warp among a token's
  int head_rec, to;    // keys and values: where a head's begin in the record
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
  int R, N, half, interleaved, axes;
  float eps;
  Kind kind[3];         // keys, values (a latent: the values behind its normed ones, where they are apart), queries
  int tasks, run;       // warps of a token, tokens of a CTA
  Div angles;
};

// Unit u of a head: its first value, the distance to its second vector (0: none), and each vector's first pair (-1: not turned).
// Neighbouring units have neighbouring vectors, the first ones and the second ones: a warp's accesses are whole lines (with a
// unit's two vectors side by side, half sectors: 96 us instead of 68 on 16384 tokens of 32 + 8 + 8 heads, interleaved).
struct Place {
  int d, second, j, j2;
};
__device__ __forceinline__ Place place_of(const Kind& k, int u, int interleaved) {
  Place p;
  p.j = p.j2 = -1;
  const bool pairs = k.half != 0 && !interleaved;
  if (pairs && 8 * u < k.half) {
    p.d = k.off + 8 * u;
    p.second = k.half;
    p.j = 8 * u;
    return p;
  }
  // of the vectors that are not turned with others: all, or (gap) those around the rotary ones
  const int gap = pairs ? 2 * k.half : 0, vecs = (k.dim - gap) >> 3, v = pairs ? u - (k.half >> 3) : u, w = v + ((vecs + 1) >> 1);
  p.d = 8 * v + (8 * v >= k.off ? gap : 0);
  p.second = w < vecs ? 8 * w + (8 * w >= k.off ? gap : 0) - p.d : 0;
  if (!pairs && k.half != 0) {
    const int j = (p.d - k.off) >> 1, j2 = (8 * w - k.off) >> 1;  // d and off are multiples of 8: a vector is rotary or it is not
    if (p.d >= k.off && j < k.half) p.j = j;
    if (p.second != 0 && 8 * w >= k.off && j2 < k.half) p.j2 = j2;
  }
  return p;
}

// Two 32-bit values at a time.
struct Two {
  float x, y;
};
__device__ __forceinline__ Two mul(Two a, Two b) {
  Two r;
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\t"
      "mul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
  Two r;
  asm("{\n\t.reg .b64 p, q, s;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmov.b64 s, {%6, %7};\n\t"
      "fma.rn.f32x2 p, p, q, s;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ Two wide(uint32_t w) { return Two{lo(w), hi(w)}; }

// 8 weights from value d on
__device__ __forceinline__ void weights(const Kind& k, int h, int d, Two (&w)[4]) {
  const int64_t at = (int64_t)h * k.whs + d;
  if (k.wide) {
    const float4 a = *(const float4*)((const float*)k.w + at), b = *(const float4*)((const float*)k.w + at + 4);
    w[0] = Two{a.x, a.y}, w[1] = Two{a.z, a.w}, w[2] = Two{b.x, b.y}, w[3] = Two{b.z, b.w};
  } else {
    const Vec8 v = ld8((const uint16_t*)k.w + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = wide(v.w[i]);
  }
}
// the four pairs of neighbours by their cosines and sines
__device__ __forceinline__ void turn_inside(Two (&x)[4], const float* c, const float* s) {
  const float4 cc = *(const float4*)c, ss = *(const float4*)s;
  const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const Two p = x[i];
    x[i].x = p.x * cv[i] - p.y * sv[i];
    x[i].y = p.y * cv[i] + p.x * sv[i];
  }
}

// What a lane does of every token: unit p of its head.
struct Mine {
  Place at;
  bool there;
  Two wx[4], wy[4];  // weights of its two vectors
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ Vec8 lds8(uint32_t at) {
  Vec8 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]) : "r"(at) : "memory");
  return v;
}

// PER: units of a lane.
template <int PER>
__global__ void __launch_bounds__(32 * kMaxWarps, PER == 1 ? kCtas : 1) k_append_normed(const __grid_constant__ NormArgs a) {
  constexpr int kDepth = kAhead / PER;           // tokens on their way
  extern __shared__ __align__(16) float s_cs[];  // [2][2][kStage][half]: stage, cosines and sines; then the warps' rings
  __shared__ int64_t s_row[kRun], s_pos[kRun][HS_MAX_AXES];
  __shared__ uint8_t s_live[kRun];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int t0 = blockIdx.x * a.run, nt = min(a.run, a.N - t0), half = a.half;
  const int task = (int)blockIdx.y * warps + warp;
  const int kn = (task >= a.kind[1].first) + (task >= a.kind[2].first);
  const Kind& k = a.kind[kn];
  const int u0 = lane & ((1 << k.lanes) - 1), h = ((task - k.first) * 32 + lane) >> k.lanes;
  const bool on = task < a.tasks && h < (int)k.heads.d;
  const int norm = k.norm, lanes = 1 << k.lanes, to = h * k.head_rec + k.to;
  const float per = k.per;
  const int64_t ts = k.ts;
  const uint16_t* src = k.src + (int64_t)t0 * ts + (int64_t)h * k.hs;
  hs_pdl_wait();
  Mine mine[PER];
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    Mine& m = mine[p];
    m.there = on && u0 + 32 * p < k.units;
    m.at = place_of(k, u0 + 32 * p, a.interleaved);
#pragma unroll
    for (int i = 0; i < 4; ++i) m.wx[i] = m.wy[i] = Two{1.f, 1.f};
    if (m.there && m.at.d < norm) weights(k, h, m.at.d, m.wx);
    if (m.there && m.at.second != 0 && m.at.d + m.at.second < norm) weights(k, h, m.at.d + m.at.second, m.wy);
  }
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(s_cs + 4 * kStage * half) + (uint32_t)(warp * kAhead * 1024 + lane * 16);
  auto load = [&](int t) {
    if (t < nt) {
      const uint16_t* from = src + (int64_t)t * ts;
#pragma unroll
      for (int p = 0; p < PER; ++p) {
        const uint32_t to = ring + (uint32_t)((t % kDepth * PER + p) * 1024);
        if (mine[p].there) copy16(to, from + mine[p].at.d);
        if (mine[p].there && mine[p].at.second != 0) copy16(to + 512u, from + mine[p].at.d + mine[p].at.second);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int t = 0; t < kDepth; ++t) load(t);
  for (int w = tid; w < nt; w += blockDim.x) {  // a thread a token
    const int t = t0 + w;
    int x = 0;
    for (int n = a.R; n > 1;) {  // the last request whose first token is not behind t
      const int before = n >> 1;
      if (a.cu[x + before] <= t) x += before;
      n -= before;
    }
    const int c0 = a.cu[x], c1 = a.cu[x + 1];
    const bool live = c0 <= t && t < c1;
    const int64_t pos = a.start[x] + ((int64_t)t - c0);
    uint32_t bad = 0u;
    s_row[w] = live ? paged_row(a.kv, x, pos, (uint32_t)HS_DEVERR_APPEND, &bad) : -1;
    s_live[w] = live;
    if (blockIdx.y == 0) report(a.kv.err, bad);
    for (int i = 0; i < a.axes; ++i) s_pos[w][i] = a.rope_pos != nullptr ? a.rope_pos[(int64_t)t * a.axes + i] : pos;
  }
  __syncthreads();
  auto one = [&](int t, const float* c, const float* s) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    Vec8 rx[PER], ry[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const uint32_t from = ring + (uint32_t)((t % kDepth * PER + p) * 1024);
      rx[p] = lds8(from);
      ry[p] = lds8(from + 512u);
    }
    Two r = {1.f, 1.f};
    if (norm != 0) {
      Two sum[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
      for (int p = 0; p < PER; ++p) {
        const Mine& m = mine[p];
        if (m.there && m.at.d < norm)
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i] = fma(wide(rx[p].w[i]), wide(rx[p].w[i]), sum[i]);
        if (m.there && m.at.second != 0 && m.at.d + m.at.second < norm)
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i] = fma(wide(ry[p].w[i]), wide(ry[p].w[i]), sum[i]);
      }
      float all = ((sum[0].x + sum[1].x) + (sum[2].x + sum[3].x)) + ((sum[0].y + sum[1].y) + (sum[2].y + sum[3].y));
#pragma unroll
      for (int o = 1; o < 32; o <<= 1)
        if (o < lanes) all += __shfl_xor_sync(0xffffffffu, all, o);
      r.x = r.y = rsqrtf(fmaf(all, per, a.eps));
    }
    if (kn == 2 ? !s_live[t] : s_row[t] < 0) {
      load(t + kDepth);
      return;
    }
    uint16_t* dst = kn == 2 ? a.q_out + (int64_t)(t0 + t) * a.ots + (int64_t)h * a.ohs
                            : (uint16_t*)(a.kv.base + s_row[t] * a.kv.rec) + to;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const Mine& m = mine[p];
      if (!m.there) continue;
      Vec8 x = rx[p], y = ry[p];
      if (norm != 0 || m.at.j >= 0 || m.at.j2 >= 0) {
        Two v[4], w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = wide(x.w[i]);
          w[i] = wide(y.w[i]);
        }
        if (m.at.d < norm)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = mul(v[i], mul(r, m.wx[i]));
        if (m.at.d + m.at.second < norm)
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = mul(w[i], mul(r, m.wy[i]));
        if (a.interleaved) {
          if (m.at.j >= 0) turn_inside(v, c + m.at.j, s + m.at.j);
          if (m.at.j2 >= 0) turn_inside(w, c + m.at.j2, s + m.at.j2);
        } else if (m.at.j >= 0) {
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const int from = (m.at.j >> 1) + (i >> 1) * (half >> 1);
            const float4 cc = *(const float4*)(c + from), ss = *(const float4*)(s + from);
            const Two ck[2] = {{cc.x, cc.y}, {cc.z, cc.w}}, sk[2] = {{ss.x, ss.y}, {ss.z, ss.w}};
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const Two b = v[i + n], e = w[i + n];
              v[i + n] = fma(e, Two{-sk[n].x, -sk[n].y}, mul(b, ck[n]));
              w[i + n] = fma(b, sk[n], mul(e, ck[n]));
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x.w[i] = pack(v[i].x, v[i].y);
          y.w[i] = pack(w[i].x, w[i].y);
        }
      }
      st8(dst + m.at.d, x);
      if (m.at.second != 0) st8(dst + m.at.d + m.at.second, y);
    }
    load(t + kDepth);  // into the place that was read, by the lane that read it
  };
#pragma unroll 1
  for (int b = 0; b < nt; b += kStage) {
    // the angles of this stage; the stage before last has been read by all
    float* c = s_cs + (b / kStage & 1) * 2 * kStage * half;
    float* s = c + kStage * half;
    const int m = min(kStage, nt - b);
    for (uint32_t i = tid; i < (uint32_t)(m * half); i += blockDim.x) {
      const uint32_t t = a.angles(i), j = i - t * a.angles.d;
      const int x = a.axis != nullptr ? min((int)a.axis[j], a.axes - 1) : 0;
      const uint64_t turns = (uint64_t)s_pos[b + t][x] * a.turns[j];
      // half form: a lane takes 8 neighbouring pairs; the first four of all lanes lie together, then the second
      const uint32_t to = a.interleaved ? i : t * half + (j >> 3) * 4u + (j & 3u) + (j & 4u ? (uint32_t)half >> 1 : 0u);
      sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s[to], &c[to]);
    }
    __syncthreads();
#pragma unroll 1
    for (int t = 0; t < m; ++t) one(b + t, c + t * half, s + t * half);
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
  a.half = g.rotary_dim / 2;
  a.interleaved = g.interleaved;
  a.axes = n.axes;
  a.eps = n.eps;
  a.angles = div_by(a.half);
  const int dqk = cfg->head_dim_qk, dv = cfg->head_dim_v;
  // a latent's normed values and its rotary tail are heads of their own: the first are 32 units then
  const bool apart = mla && n.d_k_weight != nullptr && g.rotary_offset >= dv && dv < dqk;
  int most = 0;  // units of a head
  for (int x = 0; x < 3; ++x) {
    Kind& k = a.kind[x];
    const bool tail = x == 1 && apart;
    const int H = x == 0 || tail ? cfg->num_kv_heads : x == 1 ? (mla ? 0 : cfg->num_kv_heads) : (g.d_q != nullptr ? cfg->num_q_heads : 0);
    k.src = (const uint16_t*)(x == 0 ? g.d_k : x == 1 ? (tail ? (const uint16_t*)g.d_k + dv : g.d_v) : g.d_q);
    k.ts = x == 0 || tail ? g.k_token_stride : x == 1 ? g.v_token_stride : g.q_token_stride;
    k.hs = x == 0 || tail ? g.k_head_stride : x == 1 ? g.v_head_stride : g.q_head_stride;
    k.dim = x == 0 ? (apart ? dv : dqk) : x == 1 ? (tail ? dqk - dv : dv) : g.q_dim;
    k.half = (x == 0 && apart) || (x == 1 && !tail) ? 0 : a.half;
    k.off = tail ? g.rotary_offset - dv : x == 0 || (x == 2 && g.q_dim == dqk) ? g.rotary_offset : 0;
    k.w = x == 0 ? n.d_k_weight : x == 2 ? n.d_q_weight : nullptr;
    k.wide = (x == 0 ? n.k_weight_type : n.q_weight_type) == HS_WEIGHT_FP32;
    k.whs = x == 0 ? n.k_weight_head_stride : n.q_weight_head_stride;
    k.norm = k.w == nullptr ? 0 : mla ? dv : k.dim;
    k.per = k.norm > 0 ? 1.f / (float)k.norm : 0.f;
    k.head_rec = mla ? dqk : dqk + dv;
    k.to = tail ? dv : x == 1 ? dqk : 0;
    k.heads = div_by(H);
    k.units = H > 0 ? head_units(k.dim, k.half, a.interleaved) : 0;
    k.lanes = log2_up(k.units < 32 ? k.units : 32);
    if (k.units > most) most = k.units;
  }
  for (int x = 0; x < 3; ++x) {
    a.kind[x].first = a.tasks;
    if (a.kind[x].units > 0) a.tasks += (int)((((int64_t)a.kind[x].heads.d << a.kind[x].lanes) + 31) >> 5);
  }
  // the warps of a token over as few CTAs as hold them, evenly; runs so long that the CTAs fill the SMs once
  const int shares = (a.tasks + kMaxWarps - 1) / kMaxWarps, warps = (a.tasks + shares - 1) / shares;
  const int64_t room = (int64_t)kSmsHint * (kCtas * kMaxWarps / warps);
  const int64_t full = ((int64_t)a.N * shares + room * kRun - 1) / (room * kRun);  // or as often as it takes
  a.run = (int)(((int64_t)a.N * shares + room * full - 1) / (room * full));
  const size_t smem = 4 * (size_t)kStage * a.half * sizeof(float) + (size_t)warps * kAhead * 1024;
  static bool done[64];
  if (kv->cuda_device >= 64 || !done[kv->cuda_device]) {
    const int top = 4 * kStage * 288 * (int)sizeof(float) + kMaxWarps * kAhead * 1024;
    if (hs_raise_smem_limit(k_append_normed<1>, top) != cudaSuccess || hs_raise_smem_limit(k_append_normed<2>, top) != cudaSuccess)
      return HS_ERR_CUDA;
    if (kv->cuda_device < 64) done[kv->cuda_device] = true;
  }
  const dim3 grid((unsigned)(((int64_t)a.N + a.run - 1) / a.run), shares), block(32 * warps);
  const cudaError_t e = most > 32 ? hs_launch_pdl(k_append_normed<2>, grid, block, smem, (cudaStream_t)stream, a)
                                  : hs_launch_pdl(k_append_normed<1>, grid, block, smem, (cudaStream_t)stream, a);
  return e == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

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

// A CTA takes a few tokens: their records' places and the sines and cosines, shared by all heads, first; then
// units of two 16-byte vectors, two of them in flight per thread at 40 registers (six CTAs an SM).  Few tokens
// spread over many CTAs, each with a share of every token's units.  16384 tokens of 32 + 8 + 8 heads of 128:
// 65.7 us, 6.1 TB/s (four units in flight at 64 registers 73.6 us, one 68.1; 8 or 16 tokens a CTA 72 and 83 us, one 74;
// all loads issued before the places are known, into registers, 75: spills).  Latents, 8191 tokens of 576 and 64 queries'
// 64 rotary values each: 31.3 us, 4.9 TB/s; 4 tokens are 2.3 rounds of a CTA's 512 units there, and 87 heads, which fill
// three, move 4.66 TB/s where 64 heads move 4.03 (single calls, caches cold).

constexpr int kAppThreads = 256;
constexpr int kAppTokens = 4;   // tokens of a CTA at most
constexpr int kAppFlight = 2;   // units a thread loads before it stores

// i / d by a multiplication with ceil(2^32 / d): exact while i * d < 2^32
struct Div {
  uint32_t d, m;
  __device__ __forceinline__ uint32_t operator()(uint32_t i) const { return d == 1u ? i : __umulhi(i, m); }
};

struct AppendArgs {
  PagedRows kv;
  const int32_t* cu;
  const int64_t* start;
  const int64_t* rope_pos;
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  const uint64_t* turns;
  int64_t kts, khs, vts, vhs, qts, qhs, ots, ohs;  // strides in values
  int R, N, dqk, dv;                               // dv = 0: the record is the key alone (shared latent)
  int half, k_off, q_off, q_dim, interleaved;      // half = rotary_dim / 2
  int kn, vn, per_cta, tokens;                     // units of a token's keys and values, units and tokens of a CTA
  Div all, kh, vh, qh, angles;                     // units of a token, of a head of each kind; pairs
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

// four neighbouring pairs (cs: 16-byte aligned, as a multiple of four pairs)
__device__ __forceinline__ void turn(Vec8& v, const float2* cs) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const float4 c = *(const float4*)(cs + i);
    const float p0 = lo(v.w[i]), r0 = hi(v.w[i]), p1 = lo(v.w[i + 1]), r1 = hi(v.w[i + 1]);
    v.w[i] = pack(p0 * c.x - r0 * c.y, r0 * c.x + p0 * c.y);
    v.w[i + 1] = pack(p1 * c.z - r1 * c.w, r1 * c.z + p1 * c.w);
  }
}

// Units of one head, two vectors of 8 values each.  Half form: unit u < half / 8 turns values 8u.. with their
// partners half further on; the rest of the head, before and behind the rotary values, is copied, two vectors a
// unit.  Interleaved: unit u holds values 16u.., each vector turned when it is a rotary one.
int head_units(int dim, int half, int interleaved) {
  return interleaved ? (dim + 15) / 16 : half / 8 + (dim - 2 * half + 15) / 16;
}

// One unit: where it reads and writes, and how it turns.
struct Unit {
  const uint16_t* src;  // null: nothing to do
  uint16_t* dst;
  int second;           // values to the second vector, 0: none
  int cs, cs2;          // first pair of each vector in the table of sines and cosines, -1: copied
};

__global__ void __launch_bounds__(kAppThreads, 6) k_append_rotated(AppendArgs a) {
  extern __shared__ __align__(16) float2 s_cs[];   // [tokens][half] cosine and sine of each pair
  __shared__ int64_t s_row[kAppTokens], s_pos[kAppTokens];  // record row (-1: not stored), angle position
  __shared__ int s_live[kAppTokens];
  hs_pdl_wait();
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.N - t0);
  for (int w = tid >> 5; w < nt; w += kAppThreads / 32) {  // a warp a token
    const int lane = tid & 31, t = t0 + w;
    const int64_t given = a.rope_pos != nullptr ? a.rope_pos[t] : 0;
    // the last request whose first token is not behind t: 32 places of the rest are looked at at a time
    int x = 0, n = a.R;
    while (n > 1) {
      const int step = (n + 31) >> 5, at = lane * step;
      const bool before = at < n && a.cu[x + at] <= t;
      const int c = max(__popc(__ballot_sync(0xffffffffu, before)) - 1, 0);
      x += c * step;
      n = min(step, n - c * step);
    }
    if (lane == 0) {
      const int c0 = a.cu[x], c1 = a.cu[x + 1];
      const int64_t st = a.start[x];
      const bool live = c0 <= t && t < c1;
      int64_t row = -1, pos = 0;
      if (live) {
        uint32_t bad = 0u;
        pos = st + ((int64_t)t - c0);
        row = paged_row(a.kv, x, pos, (uint32_t)HS_DEVERR_APPEND, &bad);
        if (blockIdx.y == 0) report(a.kv.err, bad);
        if (a.rope_pos != nullptr) pos = given;
      }
      s_live[w] = live;
      s_row[w] = row;
      s_pos[w] = pos;
    }
  }
  __syncthreads();
  for (uint32_t i = tid; i < (uint32_t)(nt * a.half); i += kAppThreads) {
    const uint32_t t = a.angles(i), j = i - t * a.angles.d;
    const uint64_t turn = (uint64_t)s_pos[t] * a.turns[j];
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    s_cs[i] = make_float2(c, s);
  }
  __syncthreads();
  const int head_rec = a.dqk + a.dv;
  const uint32_t end = min((uint32_t)(nt * (int)a.all.d), (blockIdx.y + 1) * (uint32_t)a.per_cta);
  for (uint32_t i0 = blockIdx.y * (uint32_t)a.per_cta + tid; i0 < end; i0 += kAppFlight * kAppThreads) {
    Unit un[kAppFlight];
    Vec8 x[kAppFlight], y[kAppFlight];
#pragma unroll
    for (int f = 0; f < kAppFlight; ++f) {
      const uint32_t i = i0 + f * kAppThreads;
      Unit& n = un[f];
      n.src = nullptr;
      if (i >= end) continue;
      const uint32_t t = a.tokens == 1 ? 0u : a.all(i), w = i - t * a.all.d;
      const int64_t tok = t0 + (int)t;
      int u, off, dim;
      bool value = false;
      if (w < (uint32_t)a.kn) {
        if (s_row[t] < 0) continue;
        const uint32_t h = a.kh(w);
        u = (int)(w - h * a.kh.d);
        off = a.k_off;
        dim = a.dqk;
        n.src = a.k + tok * a.kts + (int64_t)h * a.khs;
        n.dst = (uint16_t*)(a.kv.base + s_row[t] * a.kv.rec) + (int)h * head_rec;
      } else if (w < (uint32_t)(a.kn + a.vn)) {
        if (s_row[t] < 0) continue;
        const uint32_t v = w - a.kn, h = a.vh(v);
        u = (int)(v - h * a.vh.d);
        off = 0;
        dim = a.dv;
        value = true;
        n.src = a.v + tok * a.vts + (int64_t)h * a.vhs;
        n.dst = (uint16_t*)(a.kv.base + s_row[t] * a.kv.rec) + (int)h * head_rec + a.dqk;
      } else {
        if (!s_live[t]) continue;
        const uint32_t v = w - a.kn - a.vn, h = a.qh(v);
        u = (int)(v - h * a.qh.d);
        off = a.q_off;
        dim = a.q_dim;
        n.src = a.q + tok * a.qts + (int64_t)h * a.qhs;
        n.dst = a.q_out + tok * a.ots + (int64_t)h * a.ohs;
      }
      int d;  // the unit's first value
      n.cs = n.cs2 = -1;
      if (!value && a.interleaved) {
        // d and off are multiples of 8: a vector is rotary or it is not
        d = 16 * u;
        n.second = d + 8 < dim ? 8 : 0;
        const int j = (d - off) >> 1;
        if (d >= off && j < a.half) n.cs = (int)t * a.half + j;
        if (d + 8 >= off && j + 4 < a.half) n.cs2 = (int)t * a.half + j + 4;
      } else if (!value && 8 * u < a.half) {
        d = off + 8 * u;
        n.second = a.half;
        n.cs = (int)t * a.half + 8 * u;
      } else {  // copied
        const int gap = value ? 0 : 2 * a.half, from = value ? dim : off, v = 16 * u - (value ? 0 : 2 * a.half);
        d = v + (v >= from ? gap : 0);
        n.second = v + 8 < dim - gap ? v + 8 + (v + 8 >= from ? gap : 0) - d : 0;
      }
      n.src += d;
      n.dst += d;
      x[f] = ld8(n.src);
      if (n.second != 0) y[f] = ld8(n.src + n.second);
    }
#pragma unroll
    for (int f = 0; f < kAppFlight; ++f) {
      const Unit& n = un[f];
      if (n.src == nullptr) continue;
      if (!a.interleaved && n.cs >= 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 c = *(const float4*)&s_cs[n.cs + 2 * i];  // two pairs: cosine, sine, cosine, sine
          const float a0 = lo(x[f].w[i]), a1 = hi(x[f].w[i]), b0 = lo(y[f].w[i]), b1 = hi(y[f].w[i]);
          x[f].w[i] = pack(a0 * c.x - b0 * c.y, a1 * c.z - b1 * c.w);
          y[f].w[i] = pack(b0 * c.x + a0 * c.y, b1 * c.z + a1 * c.w);
        }
      } else {
        if (n.cs >= 0) turn(x[f], s_cs + n.cs);
        if (n.cs2 >= 0) turn(y[f], s_cs + n.cs2);
      }
      st8(n.dst, x[f]);
      if (n.second != 0) st8(n.dst + n.second, y[f]);
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
  __shared__ int64_t s_src[HS_MAX_TREE_NODES], s_dst[HS_MAX_TREE_NODES];  // source -1: stays
  hs_pdl_wait();
  const int r = blockIdx.y;
  const int given = count[r];
  const int64_t base = len[r];
  const int n = min(max(given, 0), path_len);
  uint32_t bad = n != given ? (uint32_t)HS_DEVERR_LOC : 0u;
  for (int i = threadIdx.x; i < n; i += kKeepThreads) {
    const int p = path[(int64_t)r * path_len + i];
    int64_t src = -1, dst = -1;
    if (p < i) {
      bad |= (uint32_t)HS_DEVERR_LOC;
    } else if (p > i) {
      src = paged_row(kv, r, base + p, (uint32_t)HS_DEVERR_LOC, &bad);
      dst = paged_row(kv, r, base + i, (uint32_t)HS_DEVERR_LOC, &bad);
    } else {
      paged_row(kv, r, base + p, (uint32_t)HS_DEVERR_LOC, &bad);  // stays where it is, but has to be somewhere
    }
    s_src[i] = dst < 0 ? -1 : src;
    s_dst[i] = dst;
  }
  if (blockIdx.x == 0) report(kv.err, bad);
  __syncthreads();
  const int64_t col = ((int64_t)blockIdx.x * kKeepThreads + threadIdx.x) * 16;
  if (col >= kv.rec) return;
  for (int i0 = 0; i0 < n; i0 += kKeepBatch) {
    uint4 v[kKeepBatch];
#pragma unroll
    for (int x = 0; x < kKeepBatch; ++x)
      if (i0 + x < n && s_src[i0 + x] >= 0) v[x] = *(const uint4*)(kv.base + s_src[i0 + x] * kv.rec + col);
#pragma unroll
    for (int x = 0; x < kKeepBatch; ++x)
      if (i0 + x < n && s_src[i0 + x] >= 0) *(uint4*)(kv.base + s_dst[i0 + x] * kv.rec + col) = v[x];
  }
}

// 2^256 / (2 pi), lowest word first
constexpr uint64_t kOverTwoPi[4] = {0x7f9458eaf7aef158ull, 0x36d8a5664f10e410ull, 0x7f09d5f47d4d3770ull, 0x28be60db9391054aull};

constexpr int kMinCtas = 456;

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
    // no two queries may be written over each other: one stride has to step over all that the other spans
    const int64_t n = g.num_tokens, hq = cfg->num_q_heads, ts = g.q_out_token_stride, hs = g.q_out_head_stride, d = g.q_dim;
    const bool by_token = (hq == 1 || hs >= d) && (n == 1 || ts >= (hq - 1) * hs + d);
    const bool by_head = (n == 1 || ts >= d) && (hq == 1 || hs >= (n - 1) * ts + d);
    if (!by_token && !by_head) return HS_ERR_ARG;
    // in place, every thread reads what it writes only where both have the same strides
    if (g.d_q == g.d_q_out && ((n > 1 && g.q_token_stride != ts) || (hq > 1 && g.q_head_stride != hs))) return HS_ERR_ARG;
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
  a.dqk = cfg->head_dim_qk;
  a.dv = mla ? 0 : cfg->head_dim_v;
  a.half = g.rotary_dim / 2;
  a.k_off = g.rotary_offset;
  a.q_off = g.q_dim == cfg->head_dim_qk ? g.rotary_offset : 0;
  a.q_dim = g.q_dim;
  a.interleaved = g.interleaved;
  const int ku = head_units(a.dqk, a.half, a.interleaved), vu = (a.dv + 15) / 16;
  const int qu = g.d_q != nullptr ? head_units(g.q_dim, a.half, a.interleaved) : 0;
  a.kn = cfg->num_kv_heads * ku;
  a.vn = cfg->num_kv_heads * vu;
  const int units = a.kn + a.vn + cfg->num_q_heads * qu;
  auto div = [](int d) { return Div{(uint32_t)(d > 0 ? d : 1), d > 1 ? (uint32_t)((0x100000000ull + d - 1) / d) : 0u}; };
  a.all = div(units);
  a.kh = div(ku);
  a.vh = div(vu);
  a.qh = div(qu);
  a.angles = div(a.half);
  // kAppTokens tokens a CTA while that leaves three CTAs an SM, fewer else; then every token's units are shared by
  // several CTAs until the GPU is filled or a share is below a quarter of one round (16 tokens: 3.2 us; a CTA a token
  // 6.2 us).  A CTA of several tokens has fewer than 2^16 units (see Div; of one token nothing is divided by them).
  a.tokens = kAppTokens;
  while (a.tokens > 1 && (a.N < kMinCtas * a.tokens || units * a.tokens >= 65536)) a.tokens >>= 1;
  const int ctas = (int)(((int64_t)a.N + a.tokens - 1) / a.tokens);
  int shares = 1;
  while (shares < 64 && (int64_t)ctas * shares < 2 * kSmsHint && units * a.tokens / shares > kAppFlight * kAppThreads / 4)
    shares *= 2;
  a.per_cta = (units * a.tokens + shares - 1) / shares;
  const size_t smem = (size_t)a.tokens * a.half * sizeof(float2);
  const cudaError_t e = hs_launch_pdl(k_append_rotated, dim3(ctas, shares), dim3(kAppThreads), smem, (cudaStream_t)stream, a);
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

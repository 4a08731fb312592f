// What the appends to a paged cache have in common: vectors of bf16, units of a head, the checks of their arguments.
#pragma once

#include <cuda_bf16.h>

#include "hs_paged.cuh"

namespace {

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

// Units of one head, two vectors of 8 values each.  Half form: unit u < half / 8 turns values 8u.. with their
// partners half further on; the rest of the head, before and behind the rotary values, is copied, two vectors a
// unit.  Interleaved: unit u holds values 16u.., each vector turned when it is a rotary one.
inline int head_units(int dim, int half, int interleaved) {
  return interleaved ? (dim + 15) / 16 : half / 8 + (dim - 2 * half + 15) / 16;
}

inline bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0; }

inline int check_append(const hs_config* cfg, const hs_paged_kv* kv, const hs_append_args* args) {
  int rc = hs_check_shape(cfg);
  if (rc == HS_OK) rc = hs_check_paged(cfg, kv);
  if (rc != HS_OK) return rc;
  if (args == nullptr || args->num_tokens < 0) return HS_ERR_ARG;
  const hs_append_args& g = *args;
  const bool mla = cfg->layout == HS_LAYOUT_MLA;
  if (g.num_tokens == 0) return HS_OK;  // the rest of the arguments is not looked at
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
  return HS_OK;
}

}  // namespace

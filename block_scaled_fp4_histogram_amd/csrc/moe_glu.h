// The gated block's activation and its gradient on fp32 values, for the epilogues
// of the products and the elementwise gradient (moe_glu.hip).
#pragma once

#include "moe_device.h"
#include "moe_mm.h"

namespace moe {

// Clamps that let NaN through.
__device__ __forceinline__ float clamp_above(float v, float l) { return v > l ? l : v; }
__device__ __forceinline__ float clamp_both(float v, float l) { return v > l ? l : v < -l ? -l : v; }

// sigmoid(x) and 1 - sigmoid(x) from e = exp(-|x|), which never overflows: 1 / (1 + e)
// and e / (1 + e), whichever sign x has.  exp2 takes the product's rounding error
// as a correction, so e keeps its precision at large |x| as well; at 150 it is 0.  NaN
// stays NaN in both.
struct Sigmoid {
  float s, r;
};
__device__ __forceinline__ Sigmoid sigmoid2(float x) {
  constexpr float kLog2e = 1.44269502f, kLow = 1.92596303e-8f, kLn2 = 0.693147182f;
  const float n = -clamp_above(fabsf(x), 150.0f), hi = n * kLog2e, lo = fmaf(n, kLow, fmaf(n, kLog2e, -hi));
  float e = __builtin_amdgcn_exp2f(hi);
  e = fmaf(e, lo * kLn2, e);
  const float q = __builtin_amdgcn_rcpf(1.0f + e), p = e * q;
  return x >= 0.0f ? Sigmoid{q, p} : Sigmoid{p, q};
}

// tanh(y) and 1 - tanh^2(y) from s = sigmoid(2 y): s - (1 - s), or where these come near each
// other y + y^3 q(y^2), q fitted to (tanh(y) / y - 1) / y^2 up to 0.625 (within 2^-27), and
// 4 s (1 - s), which keeps its precision where the tanh rounds to 1.
struct Tanh {
  float t, d;
};
__device__ __forceinline__ Tanh tanh2(float y) {
  const Sigmoid s = sigmoid2(2.0f * y);
  const float z = y * y;
  const float q = fmaf(z, fmaf(z, fmaf(z, fmaf(z, -5.717041902e-3f, 2.065058425e-2f), -5.374349654e-2f), 1.333149076e-1f), -3.333328366e-1f);
  return Tanh{fabsf(y) < 0.625f ? fmaf(y * z, q, y) : s.s - s.r, 4.0f * s.s * s.r};
}

// act(gate, up): gate sigmoid(alpha gate) (up + beta) after the limit, or SiTU,
// silu(4 tanh(gate / 4)) 25 tanh(up / 25).
__device__ __forceinline__ float glu_act(float gate, float up, const GluForm &f) {
  if (f.act == ACT_SITU) {
    const float t = 4.0f * tanhf(0.25f * gate);
    return t * sigmoid2(t).s * (25.0f * tanhf(0.04f * up));
  }
  if (f.has_limit) {
    gate = clamp_above(gate, f.limit);
    up = clamp_both(up, f.limit);
  }
  return gate * sigmoid2(f.alpha * gate).s * (up + f.beta);
}

// Its gradient times dh, and the value.  Beyond the limit a branch has none; at it
// the clamp is the identity.
__device__ __forceinline__ void glu_grad(float dh, float gate, float up, const GluForm &f, float &d_gate, float &d_up,
                                         float &h) {
  float g_in = 1.0f, u_in = 1.0f, alpha = f.alpha, beta = f.beta;
  bool g_out = false, u_out = false;
  if (f.act == ACT_SITU) {               // the same with alpha 1 on the capped branches, by the chain rule
    const Tanh tg = tanh2(0.25f * gate), tu = tanh2(0.04f * up);
    gate = 4.0f * tg.t, up = 25.0f * tu.t;
    g_in = tg.d, u_in = tu.d;
  } else if (f.has_limit) {
    g_out = gate > f.limit, u_out = fabsf(up) > f.limit;
    gate = clamp_above(gate, f.limit);
    up = clamp_both(up, f.limit);
  }
  const Sigmoid s = sigmoid2(alpha * gate);
  const float a = gate * s.s, u = up + beta;
  h = a * u;
  d_up = u_out ? 0.0f : dh * a * u_in;
  // (gate s (1 - s) before alpha: where alpha gate passes the range, it is 0)
  d_gate = g_out ? 0.0f : dh * u * fmaf(alpha, gate * (s.s * s.r), s.s) * g_in;
}

template <int TYPE>
__device__ __forceinline__ float glu_elem(uint32_t d, int h) {
  const uint32_t u = h ? d >> 16 : d & 0xFFFFu;
  return TYPE == MM_BF16 ? bf16_to_f32(u) : (float)__builtin_bit_cast(_Float16, (uint16_t)u);
}
template <int TYPE>
__device__ __forceinline__ uint32_t glu_pack(float lo, float hi) {
  if (TYPE == MM_BF16) return pack_bf16x2(lo, hi);
  return __builtin_bit_cast(uint32_t, v2h{(_Float16)lo, (_Float16)hi});
}

// Eight columns from c of row r: dh in d0, d1, the projections from memory, their
// gradient (and h where it is wanted) to memory, rounded once each.
template <int TYPE>
__device__ __forceinline__ void glu_back8(const GluForm &f, int I, const void *pre, void *d_pre, void *h_out, long r,
                                          int c, v4f d0, v4f d1) {
  const long at = r * 2 * I + c;
  const v4i vg = *(const v4i *)((const uint16_t *)pre + at + f.gate0);
  const v4i vu = *(const v4i *)((const uint16_t *)pre + at + f.up0);
  v4i og, ou, oh;
#pragma unroll
  for (int k = 0; k < 4; k++) {
    float g[2], u[2], h[2];
#pragma unroll
    for (int j = 0; j < 2; j++)
      glu_grad(k < 2 ? d0[2 * k + j] : d1[2 * k - 4 + j], glu_elem<TYPE>(vg[k], j), glu_elem<TYPE>(vu[k], j), f, g[j], u[j], h[j]);
    og[k] = glu_pack<TYPE>(g[0], g[1]);
    ou[k] = glu_pack<TYPE>(u[0], u[1]);
    oh[k] = glu_pack<TYPE>(h[0], h[1]);
  }
  *(v4i *)((uint16_t *)d_pre + at + f.gate0) = og;
  *(v4i *)((uint16_t *)d_pre + at + f.up0) = ou;
  if (h_out) *(v4i *)((uint16_t *)h_out + r * I + c) = oh;
}

}  // namespace moe

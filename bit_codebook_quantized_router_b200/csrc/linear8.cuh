// What the kernels of the int8 products share.
#pragma once

#include "q4_api_internal.h"
#include "q4_common.cuh"

namespace q4 {

// Every kernel of the int8 calls lets the next one of the stream start early
// and waits itself, before its first access, for the kernels in front
// (griddepcontrol): launches and prologues overlap.  Only in a chain inside one
// call are weights read before that wait, since elsewhere the kernel in front
// may be the one that writes them; so a product lets the next one start only
// after its own wait, when what was in front of the call is done.
struct LinArgs {
  const int8_t* x;       // [T][ldx]
  const float* xs;       // [T]
  const int8_t* w;       // [N][ldw], gated: [2 N][ldw], the gate's rows first
  const float* ws;       // [N], gated: [2 N]
  const float* bias;     // [N] or null
  void* out;             // [T][ldo], bf16 or fp32
  int32_t* status;       // or null
  long long ldx, ldw, ldo;
  int T, N, K;
  int out_f32;
  int chained;           // behind a kernel of the same call: the weights may be read before it is done
#ifdef MOE_Q4_DEBUG
  uint64_t limit_ns;     // test support, moe_q4_debug_withhold
  int withheld, late;
#endif
};

// What turns a sum into a value: (sum * x_scale) * w_scale, each product rounded
// (__fmul_rn, and packed products in wide_kernel: none is contracted with a bias
// behind it), the same bits in every kernel.  Not x_scale * w_scale first, which
// leaves fp32's range where the result does not: the sum, below 2^31, is a whole
// number, so its product with a small x_scale loses nothing that the result would
// keep; one with an x_scale of 2^96 and more could overflow, so those are taken
// down by 2^64 and the value brought up again, both exact.
constexpr float kScaleBig = 0x1p96f, kScaleDown = 0x1p-64f, kScaleUp = 0x1p64f;

struct RowFactor {
  float s;   // x_scale, or x_scale * kScaleDown
  bool up;   // the latter
};

__device__ __forceinline__ RowFactor row_factor(float xs) {
  const bool up = fabsf(xs) >= kScaleBig;
  return {up ? xs * kScaleDown : xs, up};
}

__device__ __forceinline__ float scaled(int acc, RowFactor x, float ws) {
  const float v = __fmul_rn(__fmul_rn((float)acc, x.s), ws);
  return x.up ? __fmul_rn(v, kScaleUp) : v;
}

// silu(g) u = g / (1 + e^-g) u, each operation rounded to fp32 as silu_mul's are
// but without the cost of its division: an approximate quotient q is corrected
// by its exact remainder (Markstein, IBM J. Res. Dev. 34, 1990), which rounds
// correctly except within about 2^-20 of an ulp beside a tie.  The reciprocal is
// taken of a quarter of the denominator, so that it is a normal number while e^-g
// is finite (to g = -88.7; then the quotient is 0).  So h, rounded to
// bf16, is silu_mul's.  Measured, MLP of 600 tokens, H = 2048, I = 1024, and of
// 2048, H = 6144, I = 2048: 0.4 and 0.9 us more than silu_mul_fast (of 18.3 and
// 62.2), whose error grows with |g|; silu_mul 5.1 and 2.6 us more.
__device__ __forceinline__ float swiglu(float g, float u) {
  const float d = 1.0f + expf(-g);
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(0.25f * d));
  y *= 0.25f;
  const float q = g * y, silu = fmaf(fmaf(-d, q, g), y, q);
  return __fmul_rn(d == INFINITY ? g * 0.0f : silu, u);
}

__device__ __forceinline__ void store_out(const LinArgs& a, long long t, int n, float v) {
  if (a.out_f32)
    reinterpret_cast<float*>(a.out)[t * a.ldo + n] = v;
  else
    reinterpret_cast<__nv_bfloat16*>(a.out)[t * a.ldo + n] = __float2bfloat16_rn(v);
}

}  // namespace q4

// linear8_tc.cu: products on the tensor cores, for a moderate number of
// tokens (K split over a cluster) and for many (CTA pairs).
int q4_launch_linear_mid(const q4::LinArgs& a, bool gated, cudaStream_t s);
int q4_launch_linear_wide(const q4::LinArgs& a, bool gated, cudaStream_t s);
constexpr int kLinearMidTokens = 128;  // the most that q4_launch_linear_mid takes

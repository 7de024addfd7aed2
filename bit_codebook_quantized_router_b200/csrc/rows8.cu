// Rows to int8 codes with one scale a row, alone (moe_q4_quant_rows) and
// behind the residual's addition and the root-mean-square norm
// (moe_q4_add_norm).
//
// A row p of K values gets m = max |p|, scale = m / 127 and the codes
//   q_i = the whole number nearest to 127 p_i / m, a tie to the even one,
// of the exact quotient.  The norm's row is p = r * weight with r = x +
// residual as the residual is stored; its factor 1/sqrt(mean r^2 + eps) is
// positive and common to the row, so the codes do not need it: they come from
// p, whose products are exact for a bf16 residual and weight, and only the
// scale and the bf16 output carry the factor.  So the codes do not depend on
// the order in which the squares are summed, and the square sum and the
// maximum come out of one pass over the row with one reduction.
//
// Exact quotient: 127 / m and its product with p are each rounded once, so
// the product is within 127 * 2^-23 < 2e-5 of the quotient; one whose distance
// from its nearest whole number is below 0.4999 has the quotient's rounding.
// For the others (2 in 10,000) the sign of 127 |p| - h m, h the half between
// the two candidates, decides: both products are taken as a rounded value and
// its exact remainder, the values' difference is exact (they are within a
// factor of 2), and so is the remainders' (at most 508 units of the smaller
// operand's last place), so the sign is that of the exact difference.
#include <type_traits>

#include "q4_api_internal.h"
#include "q4_common.cuh"

namespace q4 {

namespace {

struct RowArgs {
  const void* x;
  const void* res;      // residual in, null: none
  void* res_out;        // residual out (given with res)
  const void* weight;   // norm only, null: all ones
  __nv_bfloat16* out;   // norm only, null: not wanted
  int8_t* q;            // null: not wanted (then scale is null too)
  float* scale;
  long long ldx, ldr, ldro, ldo, ldq;
  int T, H;
  int weight_f32;
  float eps;
};

struct NoRes {};  // residual type of a call without one

template <int VEC>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float v[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    v[0] = __bfloat162float(*p);
  }
}

template <int VEC>
__device__ __forceinline__ void load_vec(const float* p, float v[VEC]) {
  if constexpr (VEC == 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    v[0] = *p;
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int VEC>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float v[VEC]) {
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  else
    *p = __float2bfloat16_rn(v[0]);
}

template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float v[VEC]) {
  if constexpr (VEC == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *p = v[0];
  }
}

// The first n (1..VEC) values; the others 0.
template <int VEC, typename T>
__device__ __forceinline__ void load_part(const T* p, float v[VEC], int n) {
  if (n >= VEC) {
    load_vec<VEC>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      v[i] = 0.0f;
      if (i < n) load_vec<1>(p + i, v + i);
    }
  }
}

template <int VEC, typename T>
__device__ __forceinline__ void store_part(T* p, const float v[VEC], int n) {
  if (n >= VEC) {
    store_vec<VEC>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i < n) store_vec<1>(p + i, v + i);
  }
}

__device__ __forceinline__ float to_type(float v, const float*) { return v; }
__device__ __forceinline__ float to_type(float v, const __nv_bfloat16*) {
  return __bfloat162float(__float2bfloat16_rn(v));
}

// What a row's reduction gives every thread of it.
struct RowScale {
  float rstd;   // 1 without a norm
  float scale;  // the row's scale
  float up;     // a power of two that brings m near 1 where 127 / m or 127 m could leave fp32's range
  float m;      // max |p| * up
  float inv;    // 127 / m, 0 for a row of zeros
  bool bad;     // a value is not finite, or the squares' sum is not
};

__device__ __forceinline__ RowScale row_scale(float m, float sum, bool norm, int H, float eps) {
  RowScale s;
  s.bad = !(m < INFINITY) || (norm && !(sum < INFINITY));
  s.rstd = norm ? rsqrtf(sum / (float)H + eps) : 1.0f;
  s.scale = norm ? m * s.rstd / 127.0f : m / 127.0f;
  s.up = m < 0x1p-60f ? 0x1p100f : (m > 0x1p60f ? 0x1p-100f : 1.0f);
  s.m = m * s.up;
  s.inv = s.m > 0.0f ? 127.0f / s.m : 0.0f;
  if (s.bad) {
    s.rstd = __uint_as_float(0x7fc00000u);
    s.scale = s.rstd;
  }
  return s;
}

// max of |a| and m, NaN if either is.
__device__ __forceinline__ float max_abs(float m, float a) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(m), "f"(fabsf(a)));
  return d;
}

// The rounding of 127 p / m where r = p (127 / m), rounded, is within 1e-4 of
// a half (see above).
__device__ __forceinline__ float near_half(float p, float r, float m) {
  const float a = fabsf(p), lo = floorf(fabsf(r)), h = lo + 0.5f;
  const float pa = 127.0f * a, pb = h * m;
  const float d = (pa - pb) + (fmaf(127.0f, a, -pa) - fmaf(h, m, -pb));
  const float odd = lo - 2.0f * floorf(0.5f * lo);
  return copysignf(lo + (d > 0.0f ? 1.0f : (d < 0.0f ? 0.0f : odd)), p);
}

// The codes of p as the low bytes of c.
template <int VEC>
__device__ __forceinline__ void codes(const float p[VEC], const RowScale& s, uint32_t c[VEC]) {
  constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number, ties to even
  float r[VEC], t[VEC], far = 0.0f;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    r[i] = p[i] * s.inv;
    t[i] = r[i] + kRound;
    far = fmaxf(far, fabsf(r[i] - (t[i] - kRound)));
  }
  if (far > 0.4999f) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (fabsf(r[i] - (t[i] - kRound)) > 0.4999f) t[i] = near_half(p[i], r[i], s.m) + kRound;
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) c[i] = __float_as_uint(t[i]);
}

// p as it stands in registers, brought near 1 (rarely) or to zeros (a bad row).
template <int VEC>
__device__ __forceinline__ void ready(float p[VEC], const RowScale& s) {
  if (s.bad || s.up != 1.0f) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = s.bad ? 0.0f : p[i] * s.up;
  }
}

template <int VEC>
__device__ __forceinline__ void store_codes(int8_t* q, const float p[VEC], const RowScale& s, int n) {
  uint32_t c[VEC];
  codes<VEC>(p, s, c);
  if constexpr (VEC == 8) {
    if (n >= VEC) {
      uint2 w;
      w.x = prmt(prmt(c[0], c[1], 0x0040), prmt(c[2], c[3], 0x0040), 0x5410);
      w.y = prmt(prmt(c[4], c[5], 0x0040), prmt(c[6], c[7], 0x0040), 0x5410);
      *reinterpret_cast<uint2*>(q) = w;
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    if (i < n) q[i] = (int8_t)(c[i] & 0xff);
}

// The row's values r: x, or the residual as it is stored (and here it is).
template <typename XT, typename RT, int VEC>
__device__ __forceinline__ void take(const RowArgs& a, long long row, int i, int n, float r[VEC]) {
  load_part<VEC>(reinterpret_cast<const XT*>(a.x) + row * a.ldx + i, r, n);
  if constexpr (!std::is_same<RT, NoRes>::value) {
    float o[VEC];
    load_part<VEC>(reinterpret_cast<const RT*>(a.res) + row * a.ldr + i, o, n);
    RT* to = reinterpret_cast<RT*>(a.res_out) + row * a.ldro + i;
#pragma unroll
    for (int j = 0; j < VEC; ++j) r[j] += o[j];
    if constexpr (VEC == 8 && std::is_same<RT, __nv_bfloat16>::value) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = pack_bf16(r[2 * j], r[2 * j + 1]);
        r[2 * j] = __uint_as_float(w[j] << 16);
        r[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
      if (n >= VEC)
        *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
      else
        store_part<VEC>(to, r, n);
    } else {
      store_part<VEC>(to, r, n);
#pragma unroll
      for (int j = 0; j < VEC; ++j) r[j] = to_type(r[j], (const RT*)nullptr);
    }
  }
}

template <int VEC>
__device__ __forceinline__ void times_weight(const RowArgs& a, int i, int n, float p[VEC]) {
  if (!a.weight) return;
  float w[VEC];
  if (a.weight_f32)
    load_part<VEC>(reinterpret_cast<const float*>(a.weight) + i, w, n);
  else
    load_part<VEC>(reinterpret_cast<const __nv_bfloat16*>(a.weight) + i, w, n);
#pragma unroll
  for (int j = 0; j < VEC; ++j) p[j] *= w[j];
}

__device__ __forceinline__ float warp_max(float m) {
  // magnitudes compare as their bits do, a NaN above infinity
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m) & 0x7fffffffu));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Sum and maximum over the CTA's threads, or over a warp's when WARP; every
// thread gets them (the same bits: both trees are symmetric).
template <bool WARP, bool NORM>
__device__ __forceinline__ void reduce(float& m, float& sum) {
  m = warp_max(m);
  if (NORM) sum = warp_sum(sum);
  if constexpr (!WARP) {
    __shared__ float2 part[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) part[warp] = make_float2(m, sum);
    __syncthreads();
    const float2 v = lane < (int)(blockDim.x >> 5) ? part[lane] : make_float2(0.0f, 0.0f);
    m = warp_max(v.x);
    if (NORM) sum = warp_sum(v.y);
  }
}

// One row a CTA (or a warp), held in registers: NV vectors of VEC values a
// thread, vector v of thread i at i + v * threads.
template <typename XT, typename RT, bool NORM, int VEC, int NV, bool WARP>
__global__ void __launch_bounds__(1024) row_kernel(const __grid_constant__ RowArgs a) {
  const int threads = WARP ? 32 : blockDim.x;
  const int me = WARP ? threadIdx.x & 31 : threadIdx.x;
  const long long row = WARP ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= a.T) return;
  float p[NV][VEC];
  float sum = 0.0f, m = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = (me + v * threads) * VEC, n = a.H - i;
    if (n > 0) {
      take<XT, RT, VEC>(a, row, i, n, p[v]);
      if constexpr (NORM) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum = fmaf(p[v][j], p[v][j], sum);
        times_weight<VEC>(a, i, n, p[v]);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) m = max_abs(m, p[v][j]);
    }
  }
  reduce<WARP, NORM>(m, sum);
  const RowScale s = row_scale(m, sum, NORM, a.H, a.eps);
  if (me == 0 && a.scale) a.scale[row] = s.scale;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = (me + v * threads) * VEC, n = a.H - i;
    if (n <= 0) break;
    if (NORM && a.out) {
      float o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = p[v][j] * s.rstd;
      store_part<VEC>(a.out + row * a.ldo + i, o, n);
    }
    if (a.q) {
      ready<VEC>(p[v], s);
      store_codes<VEC>(a.q + row * a.ldq + i, p[v], s, n);
    }
  }
}

// Rows that do not fit the registers: a CTA a row, two passes over it (the
// second finds it in L2).  A thread reads in the second pass what it read or
// wrote in the first, so out may be x and res_out may be res or x.
template <typename XT, typename RT, bool NORM>
__global__ void __launch_bounds__(1024) row_loop_kernel(const __grid_constant__ RowArgs a) {
  const long long row = blockIdx.x;
  float sum = 0.0f, m = 0.0f;
  for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
    float p[1];
    take<XT, RT, 1>(a, row, i, 1, p);
    if constexpr (NORM) {
      sum = fmaf(p[0], p[0], sum);
      times_weight<1>(a, i, 1, p);
    }
    m = max_abs(m, p[0]);
  }
  reduce<false, NORM>(m, sum);
  const RowScale s = row_scale(m, sum, NORM, a.H, a.eps);
  if (threadIdx.x == 0 && a.scale) a.scale[row] = s.scale;
  for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
    float p[1];
    if constexpr (std::is_same<RT, NoRes>::value)
      load_vec<1>(reinterpret_cast<const XT*>(a.x) + row * a.ldx + i, p);
    else
      load_vec<1>(reinterpret_cast<const RT*>(a.res_out) + row * a.ldro + i, p);
    if constexpr (NORM) {
      times_weight<1>(a, i, 1, p);
      if (a.out) a.out[row * a.ldo + i] = __float2bfloat16_rn(p[0] * s.rstd);
    }
    if (a.q) {
      ready<1>(p, s);
      store_codes<1>(a.q + row * a.ldq + i, p, s, 1);
    }
  }
}

template <typename XT, typename RT, bool NORM, int VEC, int NV>
cudaError_t launch_rows(const RowArgs& a, int threads, cudaStream_t s) {
  if (threads <= 32)
    row_kernel<XT, RT, NORM, VEC, NV, true><<<(unsigned)(((long long)a.T + 3) / 4), 128, 0, s>>>(a);
  else
    row_kernel<XT, RT, NORM, VEC, NV, false><<<a.T, threads, 0, s>>>(a);
  return cudaGetLastError();
}

bool aligned(const void* p, long long ld, int esize, int vec_bytes) {
  return ((uintptr_t)p & (vec_bytes - 1)) == 0 && (ld * esize) % vec_bytes == 0;
}

int esize(int type) { return type == MOE_Q4_F32 ? 4 : 2; }

template <typename XT, typename RT, bool NORM>
int launch(const RowArgs& a, bool vec, cudaStream_t s) {
  const int V = vec ? 8 : 1;
  const int units = (a.H + V - 1) / V;
  // vectors a thread: one while the rows are too few to fill the card (a row's
  // latency counts), else as many as keep the row's CTA near 256 threads
  int nv = 1;
  const int most = 4;
  while (nv < most && (units > 1024 * nv || (a.T >= 296 && units > 256 * nv))) nv *= 2;
  cudaError_t e;
  if (units > 1024 * nv) {
    row_loop_kernel<XT, RT, NORM><<<a.T, 1024, 0, s>>>(a);
    e = cudaGetLastError();
  } else {
    const int threads = ((units + nv - 1) / nv + 31) / 32 * 32;
    if (vec)
      e = nv == 1   ? launch_rows<XT, RT, NORM, 8, 1>(a, threads, s)
          : nv == 2 ? launch_rows<XT, RT, NORM, 8, 2>(a, threads, s)
                    : launch_rows<XT, RT, NORM, 8, 4>(a, threads, s);
    else
      e = nv == 1   ? launch_rows<XT, RT, NORM, 1, 1>(a, threads, s)
          : nv == 2 ? launch_rows<XT, RT, NORM, 1, 2>(a, threads, s)
                    : launch_rows<XT, RT, NORM, 1, 4>(a, threads, s);
  }
  return e == cudaSuccess ? MOE_Q4_OK : MOE_Q4_ECUDA;
}

bool row_type(int t) { return t == MOE_Q4_BF16 || t == MOE_Q4_F32; }

bool elem_aligned(const void* p, int type) { return ((uintptr_t)p & (esize(type) - 1)) == 0; }

}  // namespace

}  // namespace q4

using namespace q4;

extern "C" int moe_q4_quant_rows(const void* x, int x_type, long long ldx, int T, int K, int8_t* q, long long ldq,
                                 float* scale, void* stream) {
  if (!row_type(x_type) || T < 0 || K < 1 || ldx < K || ldq < K) return MOE_Q4_EINVAL;
  if (T == 0) return MOE_Q4_OK;
  if (!x || !q || !scale || !elem_aligned(x, x_type) || ((uintptr_t)scale & 3)) return MOE_Q4_EINVAL;
  RowArgs a = {};
  a.x = x, a.ldx = ldx;
  a.q = q, a.ldq = ldq, a.scale = scale;
  a.T = T, a.H = K;
  const bool vec = aligned(x, ldx, esize(x_type), 16) && aligned(q, ldq, 1, 8);
  const cudaStream_t s = (cudaStream_t)stream;
  return x_type == MOE_Q4_F32 ? launch<float, NoRes, false>(a, vec, s)
                              : launch<__nv_bfloat16, NoRes, false>(a, vec, s);
}

extern "C" int moe_q4_add_norm(const void* x, int x_type, long long ldx, const void* residual, int residual_type,
                               long long ldr, void* residual_out, long long ldro, const void* weight,
                               int weight_type, float eps, int T, int H, void* out, long long ldo, int8_t* q,
                               long long ldq, float* scale, void* stream) {
  if (!row_type(x_type) || T < 0 || H < 1 || ldx < H || !(eps > 0.0f) || !(eps < INFINITY)) return MOE_Q4_EINVAL;
  if (residual && (!row_type(residual_type) || ldr < H || ldro < H)) return MOE_Q4_EINVAL;
  if (weight && !row_type(weight_type)) return MOE_Q4_EINVAL;
  if ((out && ldo < H) || (q && ldq < H)) return MOE_Q4_EINVAL;
  if ((residual == nullptr) != (residual_out == nullptr) || (q == nullptr) != (scale == nullptr))
    return MOE_Q4_EINVAL;
  if (T == 0) return MOE_Q4_OK;
  if (!x || (!out && !q) || (out && out == residual_out)) return MOE_Q4_EINVAL;
  if (!elem_aligned(x, x_type) || (residual && (!elem_aligned(residual, residual_type) ||
                                                !elem_aligned(residual_out, residual_type))) ||
      (weight && !elem_aligned(weight, weight_type)) || ((uintptr_t)out & 1) || ((uintptr_t)scale & 3))
    return MOE_Q4_EINVAL;
  RowArgs a = {};
  a.x = x, a.ldx = ldx;
  a.res = residual, a.ldr = ldr;
  a.res_out = residual_out, a.ldro = ldro;
  a.weight = weight, a.weight_f32 = weight_type == MOE_Q4_F32;
  a.out = (__nv_bfloat16*)out, a.ldo = ldo;
  a.q = q, a.ldq = ldq, a.scale = scale;
  a.T = T, a.H = H, a.eps = eps;
  bool vec = aligned(x, ldx, esize(x_type), 16) && aligned(weight, 0, 1, 16) && (!out || aligned(out, ldo, 2, 16)) &&
             (!q || aligned(q, ldq, 1, 8));
  if (residual)
    vec = vec && aligned(residual, ldr, esize(residual_type), 16) &&
          aligned(residual_out, ldro, esize(residual_type), 16);
  const cudaStream_t s = (cudaStream_t)stream;
  typedef __nv_bfloat16 bf;
  if (x_type == MOE_Q4_F32) {
    if (!residual) return launch<float, NoRes, true>(a, vec, s);
    return residual_type == MOE_Q4_F32 ? launch<float, float, true>(a, vec, s) : launch<float, bf, true>(a, vec, s);
  }
  if (!residual) return launch<bf, NoRes, true>(a, vec, s);
  return residual_type == MOE_Q4_F32 ? launch<bf, float, true>(a, vec, s) : launch<bf, bf, true>(a, vec, s);
}

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
// The others (2 in 10,000) are divided in 64 bits, where 127 p is exact and a
// quotient that is no tie is at least 2^-25 from one.
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
  float inv;    // 127 / m, of the row scaled by 2^100 when tiny
  float m;      // max |p|, scaled likewise
  float scale;  // the row's scale
  bool bad;     // a value is not finite, or the squares' sum is not
  bool tiny;    // m below 2^-100: 127 / m could overflow
};

constexpr float kTiny = 0x1p-100f, kTinyUp = 0x1p100f;

__device__ __forceinline__ RowScale row_scale(uint32_t m_bits, float sum, bool norm, int H, float eps) {
  RowScale s;
  s.m = __uint_as_float(m_bits);
  s.bad = m_bits >= 0x7f800000u || (norm && !(sum < INFINITY));
  s.rstd = norm ? rsqrtf(sum / (float)H + eps) : 1.0f;
  s.scale = norm ? s.m * s.rstd / 127.0f : s.m / 127.0f;
  s.tiny = s.m < kTiny;
  if (s.tiny) s.m *= kTinyUp;
  s.inv = s.m > 0.0f ? 127.0f / s.m : 0.0f;
  if (s.bad) {
    s.rstd = __uint_as_float(0x7fc00000u);
    s.scale = s.rstd;
    s.inv = 0.0f;
    s.tiny = false;
  }
  return s;
}

__device__ __noinline__ float code_by_division(float p, float m) {
  return (float)rint((double)p * 127.0 / (double)m);
}

// The code of p as the low byte of the result.
__device__ __forceinline__ uint32_t code_of(float p, float inv, float m) {
  constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number, ties to even
  const float r = p * inv;
  float t = r + kRound;
  if (fabsf(r - (t - kRound)) > 0.4999f) t = code_by_division(p, m) + kRound;
  return __float_as_uint(t);
}

template <int VEC>
__device__ __forceinline__ void store_codes(int8_t* q, const float p[VEC], const RowScale& s, int n) {
  uint32_t c[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const float v = s.bad ? 0.0f : (s.tiny ? p[i] * kTinyUp : p[i]);
    c[i] = code_of(v, s.inv, s.m);
  }
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

// r (the residual as stored, or x), and p = r * weight.
template <typename XT, typename RT, bool NORM, int VEC>
__device__ __forceinline__ void take(const RowArgs& a, long long row, int i, int n, float r[VEC], float p[VEC]) {
  load_part<VEC>(reinterpret_cast<const XT*>(a.x) + row * a.ldx + i, r, n);
  if constexpr (!std::is_same<RT, NoRes>::value) {
    float o[VEC];
    load_part<VEC>(reinterpret_cast<const RT*>(a.res) + row * a.ldr + i, o, n);
#pragma unroll
    for (int j = 0; j < VEC; ++j) r[j] = to_type(r[j] + o[j], (const RT*)nullptr);
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) p[j] = r[j];
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

// Sum and maximum over the CTA's threads, or over a warp's when WARP; every
// thread gets them (the same bits: both trees are symmetric).
template <bool WARP>
__device__ __forceinline__ void reduce(uint32_t& m_bits, float& sum) {
  m_bits = __reduce_max_sync(0xffffffffu, m_bits);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if constexpr (!WARP) {
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
      s_sum[warp] = sum;
      s_max[warp] = m_bits;
    }
    __syncthreads();
    const bool has = lane < (int)(blockDim.x >> 5);
    sum = has ? s_sum[lane] : 0.0f;
    m_bits = __reduce_max_sync(0xffffffffu, has ? s_max[lane] : 0u);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
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
  float sum = 0.0f;
  uint32_t m_bits = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = (me + v * threads) * VEC, n = a.H - i;
    if (n > 0) {
      float r[VEC];
      take<XT, RT, NORM, VEC>(a, row, i, n, r, p[v]);
      if constexpr (!std::is_same<RT, NoRes>::value)
        store_part<VEC>(reinterpret_cast<RT*>(a.res_out) + row * a.ldro + i, r, n);
      if constexpr (NORM) {
        times_weight<VEC>(a, i, n, p[v]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum = fmaf(r[j], r[j], sum);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) m_bits = max(m_bits, __float_as_uint(p[v][j]) & 0x7fffffffu);
    }
  }
  reduce<WARP>(m_bits, sum);
  const RowScale s = row_scale(m_bits, sum, NORM, a.H, a.eps);
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
    if (a.q) store_codes<VEC>(a.q + row * a.ldq + i, p[v], s, n);
  }
}

// Rows that do not fit the registers: a CTA a row, two passes over it (the
// second finds it in L2).  A thread reads in the second pass what it read or
// wrote in the first, so out may be x and res_out may be res or x.
template <typename XT, typename RT, bool NORM>
__global__ void __launch_bounds__(1024) row_loop_kernel(const __grid_constant__ RowArgs a) {
  const long long row = blockIdx.x;
  float sum = 0.0f;
  uint32_t m_bits = 0;
  for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
    float r[1], p[1];
    take<XT, RT, NORM, 1>(a, row, i, 1, r, p);
    if constexpr (!std::is_same<RT, NoRes>::value) reinterpret_cast<RT*>(a.res_out)[row * a.ldro + i] = RT(r[0]);
    if constexpr (NORM) {
      times_weight<1>(a, i, 1, p);
      sum = fmaf(r[0], r[0], sum);
    }
    m_bits = max(m_bits, __float_as_uint(p[0]) & 0x7fffffffu);
  }
  reduce<false>(m_bits, sum);
  const RowScale s = row_scale(m_bits, sum, NORM, a.H, a.eps);
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
    if (a.q) store_codes<1>(a.q + row * a.ldq + i, p, s, 1);
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

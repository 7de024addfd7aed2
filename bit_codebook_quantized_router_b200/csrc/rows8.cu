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
// (rows8.cuh has the arithmetic.)
#include <type_traits>

#include "rows8.cuh"

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
  int exact;            // the values' products with the weight have 16-bit significands
  float eps;
};

// The stream's next kernel may start at once (those that read these results
// wait themselves), and this one waits for the kernels in front.
__device__ __forceinline__ void begin() {
  pdl_trigger();
  pdl_wait();
}

template <typename K>
cudaError_t start(K kernel, const RowArgs& a, long long grid, int threads, int smem, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

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

template <int VEC>
__device__ __forceinline__ void store_codes(int8_t* q, const float p[VEC], const RowScale& s, bool exact, int n) {
  uint32_t c[VEC];
  codes<VEC>(p, s, exact, c);
  if constexpr (VEC == 8) {
    if (n >= VEC) {
      *reinterpret_cast<uint2*>(q) = pack_codes(c);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    if (i < n) q[i] = (int8_t)(c[i] & 0xff);
}

// r += o, stored as the residual at `to` and left as it is stored.
template <typename RT, int VEC>
__device__ __forceinline__ void add_residual(float r[VEC], const float o[VEC], RT* to, int n) {
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

// One value of the row: x, or the residual as it is stored (and here it is).
template <typename XT, typename RT>
__device__ __forceinline__ void take(const RowArgs& a, long long row, int i, float r[1]) {
  load_vec<1>(reinterpret_cast<const XT*>(a.x) + row * a.ldx + i, r);
  if constexpr (!std::is_same<RT, NoRes>::value) {
    float o[1];
    load_vec<1>(reinterpret_cast<const RT*>(a.res) + row * a.ldr + i, o);
    add_residual<RT, 1>(r, o, reinterpret_cast<RT*>(a.res_out) + row * a.ldro + i, 1);
  }
}

// A vector of 8 bf16 values, n of them in the row, to a slot: what lies past
// the row is filled with zeros and not read.
__device__ __forceinline__ void copy_vector(uint4* to, const __nv_bfloat16* from, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
               "l"(from), "r"(2 * min(n, 8))
               : "memory");
}

template <int VEC>
__device__ __forceinline__ void times_weight(const RowArgs& a, int i, int n, float p[VEC]) {
  if (!a.weight) return;
  float w[VEC];
  if (a.weight_f32)
    load_part<VEC>(reinterpret_cast<const float*>(a.weight) + i, w, n);
  else
    load_part<VEC>(reinterpret_cast<const __nv_bfloat16*>(a.weight) + i, w, n);
  if constexpr (VEC == 8) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) split(mul(f2(p[j], p[j + 1]), f2(w[j], w[j + 1])), p[j], p[j + 1]);
  } else {
    p[0] *= w[0];
  }
}

// The squares of p added to sum, p times the weight, its largest magnitude
// into m.
template <bool NORM, int VEC>
__device__ __forceinline__ void gather_row(const RowArgs& a, int i, int n, float p[VEC], float& sum, float& m) {
  if constexpr (VEC == 8) {
    if constexpr (NORM) {
      F2 q = mul(f2(p[0], p[1]), f2(p[0], p[1]));
#pragma unroll
      for (int j = 2; j < 8; j += 2) q = fma(f2(p[j], p[j + 1]), f2(p[j], p[j + 1]), q);
      float u, v;
      split(q, u, v);
      sum += u + v;
      times_weight<VEC>(a, i, n, p);
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) m = max_abs(m, p[j], p[j + 1]);
  } else {
    if constexpr (NORM) {
      sum = fmaf(p[0], p[0], sum);
      times_weight<VEC>(a, i, n, p);
    }
    m = max_abs(m, p[0], p[0]);
  }
}

// What the row's scale makes of p: the bf16 output and the codes.
template <bool NORM, int VEC>
__device__ __forceinline__ void put_row(const RowArgs& a, long long row, int i, int n, float p[VEC],
                                        const RowScale& s) {
  if (NORM && a.out) {
    float y[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) y[j] = p[j] * s.rstd;
    store_part<VEC>(a.out + row * a.ldo + i, y, n);
  }
  if (a.q) {
    ready<VEC>(p, s);
    store_codes<VEC>(a.q + row * a.ldq + i, p, s, a.exact, n);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Sum and maximum over the CTA's threads, or over a warp's when WARP; every
// thread gets them (the same bits: both trees are symmetric).
// `buf` alternates between a CTA's calls.
template <bool WARP, bool NORM>
__device__ __forceinline__ void reduce(float& m, float& sum, int buf) {
  m = warp_max(m);
  if (NORM) sum = warp_sum(sum);
  if constexpr (!WARP) {
    __shared__ float2 part[2][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) part[buf][warp] = make_float2(m, sum);
    __syncthreads();
    const float2 v = lane < (int)(blockDim.x >> 5) ? part[buf][lane] : make_float2(0.0f, 0.0f);
    m = warp_max(v.x);
    if (NORM) sum = warp_sum(v.y);
  }
}

// bf16 rows on 16-byte boundaries, THREADS threads a row (32: a warp, four rows
// a CTA), NV vectors of 8 values a thread, vector v of thread i at
// 8 (i + v * THREADS).  A CTA takes further rows, and the next one is on its way
// to shared memory (cp.async, each thread to slots of its own) while this one
// is reduced and written: the card's bandwidth needs more bytes under way than
// the registers of a row in work leave room for.  Measured at 8192 rows of
// 6144, residual and norm: 76 us (5.9 TB/s), rows read into registers with
// nothing ahead 99 us; two to four rows ahead 75 to 82 us.  4096 rows of 6144
// to codes alone: 15.3 us against 21.8.
template <bool RES, bool NORM, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS == 32 ? 128 : THREADS, THREADS == 32 ? 8 : 1024 / THREADS)
    row_kernel(const __grid_constant__ RowArgs a) {
  begin();
  typedef __nv_bfloat16 bf;
  constexpr bool kWarp = THREADS == 32;
  constexpr int kCta = kWarp ? 128 : THREADS;
  extern __shared__ uint4 slots[];  // [NV][x, residual][threads of the CTA]
  const int me = kWarp ? threadIdx.x & 31 : threadIdx.x;
  long long row = kWarp ? (long long)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  const long long step = (long long)gridDim.x * (kWarp ? 4 : 1);
  uint4* const slot = slots + threadIdx.x;
  auto fetch = [&](long long t) {
    if (t < a.T) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = (me + v * THREADS) * 8, n = a.H - i;
        if (n > 0) {
          copy_vector(slot + v * (1 + RES) * kCta, reinterpret_cast<const bf*>(a.x) + t * a.ldx + i, n);
          if (RES)
            copy_vector(slot + (v * (1 + RES) + 1) * kCta, reinterpret_cast<const bf*>(a.res) + t * a.ldr + i, n);
        }
      }
    }
  };
  fetch(row);
  for (int turn = 0; row < a.T; row += step, turn ^= 1) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    float p[NV][8];
    float sum = 0.0f, m = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = (me + v * THREADS) * 8, n = a.H - i;
      if (n > 0) {
        const uint4* x = slot + v * (1 + RES) * kCta;
        unpack(x[0], p[v]);
        if constexpr (RES) {
          float r[8];
          unpack(x[kCta], r);
          add_residual<bf, 8>(p[v], r, reinterpret_cast<bf*>(a.res_out) + row * a.ldro + i, n);
        }
        gather_row<NORM, 8>(a, i, n, p[v], sum, m);
      }
    }
    // (in place, a row's results go where only that row was read)
    fetch(row + step);
    reduce<kWarp, NORM>(m, sum, turn);
    const RowScale s = row_scale(m, sum, NORM, a.H, a.eps);
    if (me == 0 && a.scale) a.scale[row] = s.scale;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = (me + v * THREADS) * 8, n = a.H - i;
      if (n > 0) put_row<NORM, 8>(a, row, i, n, p[v], s);
    }
  }
}

// The same straight from memory, NV vectors a thread, a CTA a row: few rows,
// where one row's latency counts, and rows of fp32.
template <typename XT, typename RT, bool NORM, int NV>
__global__ void __launch_bounds__(1024) direct_row_kernel(const __grid_constant__ RowArgs a) {
  begin();
  const long long row = blockIdx.x;
  float p[NV][8];
  float sum = 0.0f, m = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = (threadIdx.x + v * blockDim.x) * 8, n = a.H - i;
    if (n > 0) {
      load_part<8>(reinterpret_cast<const XT*>(a.x) + row * a.ldx + i, p[v], n);
      if constexpr (!std::is_same<RT, NoRes>::value) {
        float r[8];
        load_part<8>(reinterpret_cast<const RT*>(a.res) + row * a.ldr + i, r, n);
        add_residual<RT, 8>(p[v], r, reinterpret_cast<RT*>(a.res_out) + row * a.ldro + i, n);
      }
      gather_row<NORM, 8>(a, i, n, p[v], sum, m);
    }
  }
  reduce<false, NORM>(m, sum, 0);
  const RowScale s = row_scale(m, sum, NORM, a.H, a.eps);
  if (threadIdx.x == 0 && a.scale) a.scale[row] = s.scale;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = (threadIdx.x + v * blockDim.x) * 8, n = a.H - i;
    if (n > 0) put_row<NORM, 8>(a, row, i, n, p[v], s);
  }
}

// Rows on other boundaries, value by value: a CTA a row, NV values a thread.
template <typename XT, typename RT, bool NORM, int NV>
__global__ void __launch_bounds__(1024) odd_row_kernel(const __grid_constant__ RowArgs a) {
  begin();
  const long long row = blockIdx.x;
  float p[NV][1];
  float sum = 0.0f, m = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = threadIdx.x + v * blockDim.x;
    if (i < a.H) {
      take<XT, RT>(a, row, i, p[v]);
      gather_row<NORM, 1>(a, i, 1, p[v], sum, m);
    }
  }
  reduce<false, NORM>(m, sum, 0);
  const RowScale s = row_scale(m, sum, NORM, a.H, a.eps);
  if (threadIdx.x == 0 && a.scale) a.scale[row] = s.scale;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = threadIdx.x + v * blockDim.x;
    if (i < a.H) put_row<NORM, 1>(a, row, i, 1, p[v], s);
  }
}

// Rows that fit neither: a CTA a row, two passes over it (the second finds it
// in L2).  A thread reads in the second pass what it read or wrote in the
// first, so out may be x and res_out may be res or x.
template <typename XT, typename RT, bool NORM>
__global__ void __launch_bounds__(1024) row_loop_kernel(const __grid_constant__ RowArgs a) {
  begin();
  const long long row = blockIdx.x;
  float sum = 0.0f, m = 0.0f;
  for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
    float p[1];
    take<XT, RT>(a, row, i, p);
    gather_row<NORM, 1>(a, i, 1, p, sum, m);
  }
  reduce<false, NORM>(m, sum, 0);
  const RowScale s = row_scale(m, sum, NORM, a.H, a.eps);
  if (threadIdx.x == 0 && a.scale) a.scale[row] = s.scale;
  for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
    float p[1];
    if constexpr (std::is_same<RT, NoRes>::value)
      load_vec<1>(reinterpret_cast<const XT*>(a.x) + row * a.ldx + i, p);
    else
      load_vec<1>(reinterpret_cast<const RT*>(a.res_out) + row * a.ldro + i, p);
    if constexpr (NORM) times_weight<1>(a, i, 1, p);
    put_row<NORM, 1>(a, row, i, 1, p, s);
  }
}

int sm_count() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms = 148;
  return sms;
}

template <bool RES, bool NORM, int NV, int THREADS>
cudaError_t launch_rows(const RowArgs& a, cudaStream_t s) {
  constexpr int cta = THREADS == 32 ? 128 : THREADS, per = cta / THREADS, smem = NV * (1 + RES) * 16 * cta;
  const auto kernel = row_kernel<RES, NORM, NV, THREADS>;
  // twice the CTAs that fit an SM (1,024 threads): the second half fills in
  // where SMs get ahead
  const long long groups = ((long long)a.T + per - 1) / per, grid = min(groups, 2ll * (1024 / cta) * sm_count());
  if (smem > 47 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return cudaErrorInvalidValue;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess)
    return cudaErrorInvalidValue;
  return start(kernel, a, grid, cta, smem, s);
}

bool aligned(const void* p, long long ld, int esize, int vec_bytes) {
  return ((uintptr_t)p & (vec_bytes - 1)) == 0 && (ld * esize) % vec_bytes == 0;
}

int esize(int type) { return type == MOE_Q4_F32 ? 4 : 2; }

template <typename XT, typename RT, bool NORM>
int launch(const RowArgs& a, bool vec, cudaStream_t s) {
  constexpr bool res = !std::is_same<RT, NoRes>::value;
  constexpr bool half = std::is_same<XT, __nv_bfloat16>::value && !std::is_same<RT, float>::value;
  const int units = vec ? (a.H + 7) / 8 : a.H;  // vectors, or values, of a row
  // two rows an SM and more: the card's bandwidth counts, else a row's latency
  // (8 rows of 6144: 3.4 us with a thread for each vector, 3.7 by row_kernel)
  const bool many = a.T >= 296;
  if (half && vec && many && units <= 4096) {
    if constexpr (half) {
      // three or four vectors a thread where the row has them (fewer threads
      // meet in the reduction, and more rows are in work: 8192 rows of 2048
      // values 12.3 us with 64 x 4, 15.5 with 256 x 1)
      const cudaError_t e = units <= 32     ? launch_rows<res, NORM, 1, 32>(a, s)
                            : units <= 128  ? launch_rows<res, NORM, 4, 32>(a, s)
                            : units <= 192  ? launch_rows<res, NORM, 3, 64>(a, s)
                            : units <= 256  ? launch_rows<res, NORM, 4, 64>(a, s)
                            : units <= 384  ? launch_rows<res, NORM, 3, 128>(a, s)
                            : units <= 512  ? launch_rows<res, NORM, 4, 128>(a, s)
                            : units <= 768  ? launch_rows<res, NORM, 3, 256>(a, s)
                            : units <= 1024 ? launch_rows<res, NORM, 4, 256>(a, s)
                                            : launch_rows<res, NORM, 4, 1024>(a, s);
      return e == cudaSuccess ? MOE_Q4_OK : MOE_Q4_ECUDA;
    }
  }
  cudaError_t e;
  if (units > 4096) {
    e = start(row_loop_kernel<XT, RT, NORM>, a, a.T, 1024, 0, s);
  } else {
    // fp32 (twice the bytes a vector, so enough are under way): 8192 rows of
    // 6144 with an fp32 residual 113 us (6.7 TB/s) with two vectors a thread,
    // 118 with four, 151 with one.  Unaligned rows in number: four values a thread,
    // 2000 rows of 2047 codes 8.3 us (one or two 12.4), 8000 of 601 9.8 (13.4)
    const int nv = units > 2048 || (!vec && many && units > 512) ? 4 : (units > 1024 || (many && units > 256) ? 2 : 1);
    const int threads = ((units + nv - 1) / nv + 31) / 32 * 32;
    if (vec && nv == 1)
      e = start(direct_row_kernel<XT, RT, NORM, 1>, a, a.T, threads, 0, s);
    else if (vec && nv == 2)
      e = start(direct_row_kernel<XT, RT, NORM, 2>, a, a.T, threads, 0, s);
    else if (vec)
      e = start(direct_row_kernel<XT, RT, NORM, 4>, a, a.T, threads, 0, s);
    else if (nv == 1)
      e = start(odd_row_kernel<XT, RT, NORM, 1>, a, a.T, threads, 0, s);
    else if (nv == 2)
      e = start(odd_row_kernel<XT, RT, NORM, 2>, a, a.T, threads, 0, s);
    else
      e = start(odd_row_kernel<XT, RT, NORM, 4>, a, a.T, threads, 0, s);
  }
  return e == cudaSuccess ? MOE_Q4_OK : MOE_Q4_ECUDA;
}

constexpr int kMaxRow = 1 << 30;  // values of a row (positions in 32 bits)

bool row_type(int t) { return t == MOE_Q4_BF16 || t == MOE_Q4_F32; }

bool elem_aligned(const void* p, int type) { return ((uintptr_t)p & (esize(type) - 1)) == 0; }

}  // namespace

}  // namespace q4

using namespace q4;

extern "C" int moe_q4_quant_rows(const void* x, int x_type, long long ldx, int T, int K, int8_t* q, long long ldq,
                                 float* scale, void* stream) {
  if (!row_type(x_type) || T < 0 || K < 1 || ldx < K || ldq < K) return MOE_Q4_EINVAL;
  if (K > kMaxRow) return MOE_Q4_ENOTSUP;
  if (T == 0) return MOE_Q4_OK;
  if (!x || !q || !scale || !elem_aligned(x, x_type) || ((uintptr_t)scale & 3)) return MOE_Q4_EINVAL;
  RowArgs a = {};
  a.x = x, a.ldx = ldx;
  a.q = q, a.ldq = ldq, a.scale = scale;
  a.T = T, a.H = K, a.exact = x_type == MOE_Q4_BF16;
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
  if (H > kMaxRow) return MOE_Q4_ENOTSUP;
  if (T == 0) return MOE_Q4_OK;
  if (!x || (!out && !q) || (out && out == residual_out)) return MOE_Q4_EINVAL;
  // in place: a row's results have to go where that row, and no other, was read
  if (residual && residual_out == residual && T > 1 && ldro != ldr) return MOE_Q4_EINVAL;
  if (residual && residual_out == x && (residual_type != x_type || (T > 1 && ldro != ldx))) return MOE_Q4_EINVAL;
  if (out && out == x && (x_type != MOE_Q4_BF16 || (T > 1 && ldo != ldx))) return MOE_Q4_EINVAL;
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
  a.exact = (residual ? residual_type : x_type) == MOE_Q4_BF16 && (!weight || weight_type == MOE_Q4_BF16);
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

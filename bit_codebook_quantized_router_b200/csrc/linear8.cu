// Products of int8 rows and int8 weights with a scale for each row and each
// channel, and the SwiGLU MLP made of two of them.
//
//   y[t][n] = x_scale[t] * w_scale[n] * sum_k x[t][k] w[n][k]  (+ bias[n])
//
// The sums are taken in int32 and are exact: |x w| <= 2^14, so K up to
// 131,071 cannot overflow, and they do not depend on the order or on how K is
// split.  The one rounding of a sum is its conversion to fp32; its products with
// the two scales are one each, and the result's type is the last.
#include "linear8.cuh"

namespace q4 {

namespace {

constexpr int kMaxK = 131071;          // 2^14 * K < 2^31
constexpr int kMaxRows = 1 << 30;      // tokens or channels of a product (tile arithmetic in 32 bits)
constexpr int kFewTokens = 16;         // the most that few_kernel takes

// D += A(16x32, int8, row) * B(32x8, int8, col), int32.
__device__ __forceinline__ void mma_s8(int c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first n (1 to 15) bytes at p (16-byte aligned), and zeros.
__device__ __noinline__ uint4 load_some(const int8_t* p, int n) {
  uint32_t lo = 0, tail = 0;
  uint2 d = make_uint2(0, 0);
  if (n & 8) d = *reinterpret_cast<const uint2*>(p);
  if (n & 4) lo = *reinterpret_cast<const uint32_t*>(p + (n & 8));
  if (n & 2) tail = *reinterpret_cast<const uint16_t*>(p + (n & 12));
  if (n & 1) tail |= (uint32_t)(uint8_t)p[n & 14] << (8 * (n & 2));
  const uint32_t e = n & 4 ? lo : tail, f = n & 4 ? tail : 0;
  return n & 8 ? make_uint4(d.x, d.y, e, f) : make_uint4(e, f, 0, 0);
}

// 16 bytes of a weight row: read once, so not kept in L1, and through the
// coherent path.  The kernel in front may write the weights while this one is
// already resident (outside a chain they are read after its wait), and the
// read-only path is for what does not change in a kernel's whole life.
__device__ __forceinline__ uint4 load_weight(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// The 16 bytes of a row at k, zeros past its end K (nothing is read there).
__device__ __forceinline__ uint4 load_row16(const int8_t* row, int k, int K) {
  if (k + 16 <= K) return *reinterpret_cast<const uint4*>(row + k);
  return k < K ? load_some(row + k, K - k) : make_uint4(0, 0, 0, 0);
}

// The same of a weight row; what lies between the rows in the 16 bytes that
// hold its end is taken as it is (it meets the tokens' zeros), but nothing is
// read behind the last row.
__device__ __forceinline__ uint4 load_weight16(const int8_t* row, int k, int K, bool last) {
  return k < K && !last ? load_weight(row + k) : load_row16(row, k, K);
}

// Few tokens: 16 weight rows a CTA (8 gate and 8 up rows when GATED), 8 NT
// tokens, K split over the warps in segments of 128 bytes.  The weights go from
// memory to the registers of the MMA with no stop: lane (g, t) holds 16 bytes
// of rows g and g + 8 at byte 16 t of each half of a segment, which are the A
// operands of two MMAs once K is permuted the same way in the tokens' rows.
// The loads of U segments are under way before the first product, and in a
// chain the first ones before the kernel in front is done.
// Measured, N = K = 6144 from memory: 1 token 7.9 us (4.8 TB/s with the launch),
// 8 tokens 8.4, 16 tokens 9.8; the memory's bandwidth and the launch bound it.
// Three CTAs an SM (85 registers): with two, 384 CTAs take two turns (9.2 us).
template <int NT, int U, bool GATED>
__global__ void __launch_bounds__(256, NT <= 2 || (NT == 4 && U == 1) ? 3 : 1) few_kernel(const __grid_constant__ LinArgs a) {
  extern __shared__ int s_acc[];  // [warps][8 NT][16]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int n0 = blockIdx.x * (GATED ? 8 : 16);
  const int ra = min(n0 + g, a.N - 1);
  const int rb = GATED ? a.N + ra : min(n0 + g + 8, a.N - 1);
  const int8_t* wa = a.w + ra * a.ldw;
  const int8_t* wb = a.w + rb * a.ldw;
  const int full = a.K / 128;  // whole segments
  int acc[NT][4] = {};

  auto load_x = [&](int n, int k, bool whole) {
    const int t = 8 * n + g;
    if (t >= a.T) return make_uint4(0, 0, 0, 0);
    // (no read-only path: the rows may be written while this kernel is resident)
    if (whole) return *reinterpret_cast<const uint4*>(a.x + t * a.ldx + k);
    return load_row16(a.x + t * a.ldx, k, a.K);
  };
  auto product = [&](int n, uint4 p, uint4 q, uint4 x) {
    mma_s8(acc[n], p.x, q.x, p.y, q.y, x.x, x.y);
    mma_s8(acc[n], p.z, q.z, p.w, q.w, x.z, x.w);
  };
  uint4 va[U][2], vb[U][2];
  auto load_w = [&](int sg) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (sg + u * warps) * 128 + h * 64 + 16 * t4;
        va[u][h] = load_weight(wa + k);
        vb[u][h] = load_weight(wb + k);
      }
  };
  int sg = warp;
  const bool some = sg + (U - 1) * warps < full;
  if (some && a.chained) load_w(sg);
  pdl_wait();
  pdl_trigger();
  if (some && !a.chained) load_w(sg);
  if (some)
    for (;;) {
      uint4 x[U][2][NT];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < NT; ++n) x[u][h][n] = load_x(n, (sg + u * warps) * 128 + h * 64 + 16 * t4, true);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < NT; ++n) product(n, va[u][h], vb[u][h], x[u][h][n]);
      sg += U * warps;
      if (sg + (U - 1) * warps >= full) break;
      load_w(sg);
    }
  for (; sg < full; sg += warps)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = sg * 128 + h * 64 + 16 * t4;
      const uint4 p = load_weight(wa + k), q = load_weight(wb + k);
#pragma unroll
      for (int n = 0; n < NT; ++n) product(n, p, q, load_x(n, k, true));
    }
  // the rest, in halves of a segment, from the warps on that had fewest
  const int rest = (warp + warps - full % warps) % warps;
  for (int k = full * 128 + rest * 64 + 16 * t4; k < a.K + 16 * t4; k += warps * 64) {
    const uint4 p = load_weight16(wa, k, a.K, !GATED && ra == a.N - 1);
    const uint4 q = load_weight16(wb, k, a.K, rb == (GATED ? 2 * a.N : a.N) - 1);
#pragma unroll
    for (int n = 0; n < NT; ++n) product(n, p, q, load_x(n, k, false));
  }

#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s_acc[(warp * 8 * NT + 8 * n + 2 * t4 + (i & 1)) * 16 + g + 8 * (i >> 1)] = acc[n][i];
  __syncthreads();
  constexpr int kRows = GATED ? 8 : 16;
  for (int i = threadIdx.x; i < 8 * NT * kRows; i += blockDim.x) {
    const int t = i / kRows, r = i % kRows, n = n0 + r;
    if (t >= a.T || n >= a.N) continue;
    int v = 0, u = 0;
    for (int w = 0; w < warps; ++w) {
      v += s_acc[(w * 8 * NT + t) * 16 + r];
      if (GATED) u += s_acc[(w * 8 * NT + t) * 16 + r + 8];
    }
    const RowFactor xs = row_factor(a.xs[t]);
    float y = scaled(v, xs, a.ws[n]);
    if (GATED)
      y = swiglu(y, scaled(u, xs, a.ws[a.N + n]));
    else if (a.bias)
      y += a.bias[n];
    store_out(a, t, n, y);
  }
}

template <int NT, int U, bool GATED>
cudaError_t start_few(const LinArgs& a, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.N + (GATED ? 7 : 15)) / (GATED ? 8 : 16));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 8 * 8 * NT * 16 * 4;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_kernel<NT, U, GATED>, a);
}

long long few_ctas(const LinArgs& a, bool gated) { return ((long long)a.N + (gated ? 7 : 15)) / (gated ? 8 : 16); }

template <bool GATED>
int launch_few(const LinArgs& a, cudaStream_t s) {
  const cudaError_t e = a.T <= 8    ? start_few<1, 2, GATED>(a, s)
                        : a.T <= 16 ? start_few<2, 2, GATED>(a, s)
                        : a.T > 32  ? start_few<8, 1, GATED>(a, s)
                        : few_ctas(a, GATED) <= 296 ? start_few<4, 2, GATED>(a, s)
                                                    : start_few<4, 1, GATED>(a, s);
  return e == cudaSuccess ? MOE_Q4_OK : MOE_Q4_ECUDA;
}

// few_kernel or the tensor cores' kernels (one launch of those is 3 us longer,
// and their time grows less with tokens): up to 16 tokens always; to 64 where
// the tokens' rows, which every CTA reads, are short and the CTAs fit the card
// at once (three an SM with one segment at a time or two up to 32 tokens, one
// beyond).  Measured, us, few_kernel and mid_kernel: 32 tokens, N = K = 2048 3.4
// and 7.6; N = 6144, K = 512 3.9 and 5.2; N = K = 6144 13.8 and 12.1; 64 tokens,
// N = K = 2048 5.5 and 7.6; N = 2048, K = 4096 9.6 and 7.9; N = 6144, K = 512
// 8.3 and 6.3.
bool few_tokens(const LinArgs& a, bool gated) {
  if (a.T <= kFewTokens) return true;
  const long long ctas = few_ctas(a, gated), rows = (long long)a.T * a.K;
  if (a.T <= 32) return rows <= (ctas <= 296 ? 131072 : 32768) && ctas <= 444;
  return a.T <= 64 && rows <= 131072 && ctas <= 148;
}

int launch_linear(const LinArgs& a, bool gated, cudaStream_t s) {
  if (few_tokens(a, gated)) return gated ? launch_few<true>(a, s) : launch_few<false>(a, s);
  // mid_kernel's K over a cluster, or wide_kernel's pairs: to 64 tokens always
  // the first, to 128 where K is long.  Measured at 96 tokens, us, mid_kernel
  // and wide_kernel: N = K = 6144 15.2 and 18.0; N = 512, K = 6144 7.8 and 16.5;
  // N = 1003, K = 1990 6.5 and 9.2; N = K = 600 6.2 and 5.3.
  if (a.T <= 64 || (a.T <= kLinearMidTokens && a.K >= 1536)) return q4_launch_linear_mid(a, gated, s);
  return q4_launch_linear_wide(a, gated, s);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Workspace of the MLP: h bf16 [T][ldh] | its codes int8 [T][ldq] | their scales f32 [T].
struct MlpLayout {
  size_t h, q, scale, end;
  long long ldh, ldq;
};

MlpLayout mlp_layout(int I, int T) {
  MlpLayout o;
  o.ldh = ((long long)I + 7) / 8 * 8;
  o.ldq = ((long long)I + 15) / 16 * 16;
  size_t p = 0;
  o.h = p;
  p = up256(p + sizeof(__nv_bfloat16) * (size_t)T * o.ldh);
  o.q = p;
  p = up256(p + (size_t)T * o.ldq);
  o.scale = p;
  p = up256(p + sizeof(float) * (size_t)T);
  o.end = p;
  return o;
}

bool rows16(const void* p, long long ld) { return p && ((uintptr_t)p & 15) == 0 && ld % 16 == 0; }
bool floats(const void* p) { return p && ((uintptr_t)p & 3) == 0; }

int mlp_check(const moe_q4_mlp* m) {
  if (!m || m->H < 1 || m->I < 1 || m->ld_gate_up < m->H || m->ld_down < m->I) return MOE_Q4_EINVAL;
  if (m->H > kMaxK || m->I > kMaxK) return MOE_Q4_ENOTSUP;
  if (!rows16(m->gate_up, m->ld_gate_up) || !rows16(m->down, m->ld_down) || !floats(m->gate_up_scale) ||
      !floats(m->down_scale))
    return MOE_Q4_EINVAL;
  return MOE_Q4_OK;
}

}  // namespace

}  // namespace q4

using namespace q4;

extern "C" int moe_q4_linear_i8(const int8_t* x, long long ldx, const float* x_scale, const int8_t* w, long long ldw,
                                const float* w_scale, const float* bias, int T, int N, int K, void* out,
                                int out_type, long long ldo, int32_t* status, void* stream) {
  if (T < 0 || N < 1 || K < 1 || ldx < K || ldw < K || ldo < N) return MOE_Q4_EINVAL;
  if (out_type != MOE_Q4_BF16 && out_type != MOE_Q4_F32) return MOE_Q4_EINVAL;
  if (K > kMaxK || T > kMaxRows || N > kMaxRows) return MOE_Q4_ENOTSUP;
  if (T == 0) return MOE_Q4_OK;
  if (!rows16(x, ldx) || !rows16(w, ldw) || !floats(x_scale) || !floats(w_scale) || ((uintptr_t)bias & 3) || !out ||
      ((uintptr_t)out & (out_type == MOE_Q4_F32 ? 3 : 1)) || ((uintptr_t)status & 3))
    return MOE_Q4_EINVAL;
  const LinArgs a = {x, x_scale, w, w_scale, bias, out, status, ldx, ldw, ldo, T, N, K, out_type == MOE_Q4_F32};
  return launch_linear(a, false, (cudaStream_t)stream);
}

extern "C" size_t moe_q4_mlp_i8_workspace(const moe_q4_mlp* mlp, int T) {
  if (T < 1 || mlp_check(mlp) != MOE_Q4_OK) return 0;
  return mlp_layout(mlp->I, T).end;
}

extern "C" int moe_q4_mlp_i8(const moe_q4_mlp* mlp, const int8_t* x, long long ldx, const float* x_scale, int T,
                             void* out, int out_type, long long ldo, int32_t* status, void* ws, size_t ws_bytes,
                             void* stream) {
  int rc = mlp_check(mlp);
  if (rc != MOE_Q4_OK) return rc;
  if (T < 0 || ldx < mlp->H || ldo < mlp->H || (out_type != MOE_Q4_BF16 && out_type != MOE_Q4_F32))
    return MOE_Q4_EINVAL;
  if (T > kMaxRows) return MOE_Q4_ENOTSUP;
  if (T == 0) return MOE_Q4_OK;
  if (!rows16(x, ldx) || !floats(x_scale) || !out || ((uintptr_t)out & (out_type == MOE_Q4_F32 ? 3 : 1)) ||
      ((uintptr_t)status & 3))
    return MOE_Q4_EINVAL;
  const MlpLayout o = mlp_layout(mlp->I, T);
  if (!ws || ((uintptr_t)ws & 255) || ws_bytes < o.end) return MOE_Q4_EWORKSPACE;
  char* p = (char*)ws;
  const cudaStream_t s = (cudaStream_t)stream;
  const LinArgs gu = {x, x_scale, mlp->gate_up, mlp->gate_up_scale, nullptr, p + o.h, status, ldx, mlp->ld_gate_up,
                      o.ldh, T, mlp->I, mlp->H, 0};
  rc = launch_linear(gu, true, s);
  if (rc != MOE_Q4_OK) return rc;
  const LinArgs dn = {(const int8_t*)(p + o.q), (const float*)(p + o.scale), mlp->down, mlp->down_scale, nullptr, out,
                     status, o.ldq, mlp->ld_down, ldo, T, mlp->H, mlp->I, out_type == MOE_Q4_F32, 1};
  // h's codes in a launch of their own also for few tokens: 9.6 us in three
  // launches (8 tokens, H = 6144, I = 512), 10.5 with every CTA of the down
  // product making them itself; 1 token, I = 2048 11.6 and 11.75
  rc = moe_q4_quant_rows(p + o.h, MOE_Q4_BF16, o.ldh, T, mlp->I, (int8_t*)(p + o.q), o.ldq, (float*)(p + o.scale),
                         stream);
  return rc == MOE_Q4_OK ? launch_linear(dn, false, s) : rc;
}

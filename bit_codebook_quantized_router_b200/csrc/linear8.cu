// Products of int8 rows and int8 weights with a scale for each row and each
// channel, and the SwiGLU MLP made of two of them.
//
//   y[t][n] = x_scale[t] * w_scale[n] * sum_k x[t][k] w[n][k]  (+ bias[n])
//
// The sums are taken in int32 and are exact: |x w| <= 2^14, so K up to
// 131,071 cannot overflow, and they do not depend on the order or on how K is
// split.  The one rounding of a sum is its conversion to fp32; the product of
// the scales and the result's are one each, and the result's type is the last.
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

// The 16 bytes of a row at k, zeros past the row's end K (nothing is read there).
__device__ __forceinline__ uint4 load_row16(const int8_t* row, int k, int K) {
  if (k + 16 <= K) return ldg_nc(row + k);
  uint32_t v[4] = {0, 0, 0, 0};
  for (int i = 0; k + i < K; ++i) v[i >> 2] |= (uint32_t)(uint8_t)row[k + i] << (8 * (i & 3));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// U segments of 128 bytes of the rows at wa and wb, `stride` apart: every load
// is under way before the first product.
template <int NT, int U>
__device__ __forceinline__ void few_step(const LinArgs& a, const int8_t* wa, const int8_t* wb, int sg, int stride, int g,
                                         int t4, int acc[NT][4]) {
  uint4 va[U][2], vb[U][2], b[U][2][NT];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = (sg + u * stride) * 128 + h * 64 + 16 * t4;
      va[u][h] = ldg_stream(wa + k);
      vb[u][h] = ldg_stream(wb + k);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int t = 8 * n + g;
        b[u][h][n] = t < a.T ? ldg_nc(a.x + t * a.ldx + k) : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 p = va[u][h], q = vb[u][h], x = b[u][h][n];
        mma_s8(acc[n], p.x, q.x, p.y, q.y, x.x, x.y);
        mma_s8(acc[n], p.z, q.z, p.w, q.w, x.z, x.w);
      }
}

// Few tokens: 16 weight rows a CTA (8 gate and 8 up rows when GATED), 8 NT
// tokens, K split over the warps in segments of 128 bytes.  The weights go from
// memory to the registers of the MMA with no stop: lane (g, t) holds 16 bytes
// of rows g and g + 8 at byte 16 t of the segment, which are the A operands of
// two MMAs once K is permuted the same way in the tokens' rows.
template <int NT, int U, bool GATED>
__global__ void __launch_bounds__(256) few_kernel(const __grid_constant__ LinArgs a) {
  extern __shared__ int s_acc[];  // [warps][8 NT][16]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int n0 = blockIdx.x * (GATED ? 8 : 16);
  const int ra = min(n0 + g, a.N - 1);
  const int rb = GATED ? a.N + ra : min(n0 + g + 8, a.N - 1);
  const int8_t* wa = a.w + ra * a.ldw;
  const int8_t* wb = a.w + rb * a.ldw;
  int acc[NT][4] = {};
  const int full = a.K / 128;  // whole segments of 128 bytes
  int sg = warp;
  for (; sg + (U - 1) * warps < full; sg += U * warps) few_step<NT, U>(a, wa, wb, sg, warps, g, t4, acc);
  for (; sg < full; sg += warps) few_step<NT, 1>(a, wa, wb, sg, warps, g, t4, acc);
  for (int k = full * 128 + warp * 64 + 16 * t4; k < a.K + 16 * t4; k += warps * 64) {
    const uint4 va = load_row16(wa, k, a.K), vb = load_row16(wb, k, a.K);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = 8 * n + g;
      const uint4 b = t < a.T ? load_row16(a.x + t * a.ldx, k, a.K) : make_uint4(0, 0, 0, 0);
      mma_s8(acc[n], va.x, vb.x, va.y, vb.y, b.x, b.y);
      mma_s8(acc[n], va.z, vb.z, va.w, vb.w, b.z, b.w);
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s_acc[(warp * 8 * NT + 8 * n + 2 * t4 + (i & 1)) * 16 + g + 8 * (i >> 1)] = acc[n][i];
  __syncthreads();
  constexpr int kRows = GATED ? 8 : 16;
  for (int i = threadIdx.x; i < 8 * NT * kRows; i += blockDim.x) {
    const int col = i / kRows, r = i % kRows, t = col, n = n0 + r;
    if (t >= a.T || n >= a.N) continue;
    int v = 0, u = 0;
    for (int w = 0; w < warps; ++w) {
      v += s_acc[(w * 8 * NT + col) * 16 + r];
      if (GATED) u += s_acc[(w * 8 * NT + col) * 16 + r + 8];
    }
    float y = scaled(v, a.xs[t], a.ws[n]);
    if (GATED)
      y = silu_mul(y, scaled(u, a.xs[t], a.ws[a.N + n]));
    else if (a.bias)
      y += a.bias[n];
    store_out(a, t, n, y);
  }
}

int launch_few(const LinArgs& a, bool gated, cudaStream_t s) {
  const int rows = gated ? 8 : 16, nt = a.T <= 8 ? 1 : 2;
  const unsigned grid = (a.N + rows - 1) / rows;
  const int smem = 8 * 8 * nt * 16 * 4;
  if (nt == 1) {
    if (gated)
      few_kernel<1, 3, true><<<grid, 256, smem, s>>>(a);
    else
      few_kernel<1, 3, false><<<grid, 256, smem, s>>>(a);
  } else {
    if (gated)
      few_kernel<2, 2, true><<<grid, 256, smem, s>>>(a);
    else
      few_kernel<2, 2, false><<<grid, 256, smem, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? MOE_Q4_OK : MOE_Q4_ECUDA;
}

int launch_linear(const LinArgs& a, bool gated, cudaStream_t s) {
  if (a.T <= kFewTokens) return launch_few(a, gated, s);
  if (a.T <= kLinearMidTokens) return q4_launch_linear_mid(a, gated, s);
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
  if (rc == MOE_Q4_OK)
    rc = moe_q4_quant_rows(p + o.h, MOE_Q4_BF16, o.ldh, T, mlp->I, (int8_t*)(p + o.q), o.ldq, (float*)(p + o.scale),
                           stream);
  if (rc != MOE_Q4_OK) return rc;
  const LinArgs dn = {(const int8_t*)(p + o.q), (const float*)(p + o.scale), mlp->down, mlp->down_scale, nullptr, out,
                      status, o.ldq, mlp->ld_down, ldo, T, mlp->H, mlp->I, out_type == MOE_Q4_F32};
  return launch_linear(dn, false, s);
}

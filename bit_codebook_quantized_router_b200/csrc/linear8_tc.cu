// Int8 products on the 5th-generation tensor cores (tcgen05, kind::i8, int32
// accumulators in TMEM), for moderate and large numbers of tokens.
//
// mid_kernel, up to 256 tokens: the weights' bytes bound it.  The MMA's M is
// 128 weight rows and its N all the tokens, so each weight is read once; K is
// split over the CTAs of a cluster so that every SM streams weights.  The
// partial sums are int32, so adding them is exact in any order: each CTA
// sends the columns that another owns to that CTA's shared memory, and each
// finishes its own columns.  No workspace and one launch.
//
// wide_kernel, more tokens: pairs of CTAs (cta_group::2) multiply 256 tokens
// by 256 weight rows, each CTA holding 128 rows of both operands, so a pair
// reads half of what two CTAs with tiles of 128 x 256 would; persistent, with
// two accumulators, so that one tile's results leave while the next is
// multiplied.
//
// Both read operands by TMA into the 128-byte-swizzle K-major layout, in
// k-steps of 128 bytes; what lies past a row, a matrix or K arrives as zeros.
// For the SwiGLU a tile holds as many rows of the gate as of the up
// projection.  Every wait is bounded; one that gives up records
// MOE_Q4_ETIMEOUT.
#include <cuda.h>

#include "linear8.cuh"
#include "sm100.cuh"

namespace q4 {

using namespace sm100;

namespace {

constexpr int kBK = 128;               // bytes of K per stage
constexpr int kTile = 128 * kBK;       // 128 rows of a stage
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kEpiWarp0 = 2;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kSmemLimit = 227 * 1024;
constexpr int kSmemExtra = 2048;       // alignment and barriers

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// On an abandoned wait: record it and let the copies in flight land before
// the shared memory goes away.
__device__ __forceinline__ void give_up(int32_t* status, uint64_t* full, int stages) {
  record_error(status, MOE_Q4_ETIMEOUT);
  for (int s = 0; s < stages; ++s)
    for (uint32_t par = 0; par < 2; ++par) {
      volatile int quick = 0;
      mbar_wait(&full[s], par, &quick, 20000000ull);
    }
}

// ---- up to 256 tokens -----------------------------------------------------------

struct MidPlan {
  int bn;       // tokens, rounded up to 16
  int stages;   // ring stages
  int ksteps;   // k-steps of 128 in K
};

template <bool GATED>
__global__ void __launch_bounds__(kThreads, 1)
    mid_kernel(const __grid_constant__ LinArgs a, const __grid_constant__ MidPlan p,
               const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const int S = p.stages, b_tile = p.bn * kBK;
  uint8_t* sA = smem;              // [S][128][128 B] weights
  uint8_t* sB = sA + S * kTile;    // [S][bn][128 B] tokens
  uint64_t* full = reinterpret_cast<uint64_t*>(sB + S * b_tile);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = gridDim.y, rank = blockIdx.y;  // the cluster's CTAs share blockIdx.x
  const int n0 = blockIdx.x * (GATED ? 64 : 128);
  const int k_lo = (int)((long long)p.ksteps * rank / splits);
  const int k_hi = (int)((long long)p.ksteps * (rank + 1) / splits);
  uint32_t cols = 32;
  while (cols < (uint32_t)p.bn) cols *= 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      for (int ks = k_lo; ks < k_hi; ++ks, ++it) {
        const int s = it % S;
        if (!mbar_wait(&empty[s], ((it / S) & 1) ^ 1, abort_flag, kWaitNs)) break;
        mbar_arrive_expect_tx(&full[s], kTile + b_tile);
        if (GATED) {
          tma_load_2d(sA + s * kTile, &tm_w, &full[s], ks * kBK, n0);
          tma_load_2d(sA + s * kTile + kTile / 2, &tm_w, &full[s], ks * kBK, a.N + n0);
        } else {
          tma_load_2d(sA + s * kTile, &tm_w, &full[s], ks * kBK, n0);
        }
        tma_load_2d(sB + s * b_tile, &tm_x, &full[s], ks * kBK, 0);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = umma_idesc_s8(128, p.bn);
      int it = 0;
      bool ok = true;
      for (int ks = k_lo; ks < k_hi; ++ks, ++it) {
        const int s = it % S;
        if (!(ok = mbar_wait(&full[s], (it / S) & 1, abort_flag, kWaitNs))) break;
        tc_fence_after();
        const uint64_t da = umma_desc_sw128(smem_u32(sA + s * kTile));
        const uint64_t db = umma_desc_sw128(smem_u32(sB + s * b_tile));
#pragma unroll
        for (int kk = 0; kk < kBK / 32; ++kk)  // 32 bytes of K per MMA
          umma_s8<false>(tmem, da + 2 * kk, db + 2 * kk, idesc, (it | kk) != 0);
        umma_commit(&empty[s]);
      }
      umma_commit(acc_full);
      mbar_wait(acc_full, 0, abort_flag, kWaitNs);
    }
  }
  __syncthreads();
  // every copy has been read by an MMA and every MMA is done (or the wait for
  // it was given up): the ring's memory is free, here and, past the barrier,
  // in every CTA of the cluster
  if (threadIdx.x == 0 && *abort_flag) give_up(a.status, full, S);
  __syncthreads();
  cluster_arrive();
  cluster_wait();

  // send: columns [own * r, own * (r + 1)) to CTA r as [src][column][128]
  const int own = (p.bn + splits - 1) / splits;
  const uint32_t inbox = smem_u32(smem) + (uint32_t)rank * own * 512;
  tc_fence_after();
  if (warp >= kEpiWarp0) {
    const int quad = warp & 3, half = (warp - kEpiWarp0) >> 2, row = quad * 32 + lane;
    const uint32_t tb = tmem + ((uint32_t)(quad * 32) << 16);
    for (int c0 = half * 8; c0 < p.bn; c0 += 16) {
      uint32_t v[8];
      tmem_ld8_nowait(tb + c0, v);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = c0 + j, to = c / own;
        cluster_st32(cluster_addr(inbox + ((c - to * own) * 128 + row) * 4, to), (int)v[j]);
      }
    }
  }
  tc_fence_before();
  cluster_arrive();
  cluster_wait();

  // finish this CTA's columns
  const int* box = reinterpret_cast<const int*>(smem);
  constexpr int kRows = GATED ? 64 : 128;
  const int c_lo = rank * own, c_n = min(own, a.T - c_lo);
  for (int i = threadIdx.x; i < c_n * kRows; i += kThreads) {
    const int c = i / kRows, r = i % kRows, n = n0 + r, t = c_lo + c;
    if (n >= a.N) continue;
    int v = 0, u = 0;
    for (int src = 0; src < splits; ++src) {
      v += box[(src * own + c) * 128 + r];
      if (GATED) u += box[(src * own + c) * 128 + 64 + r];
    }
    float y = scaled(v, a.xs[t], a.ws[n]);
    if (GATED)
      y = silu_mul(y, scaled(u, a.xs[t], a.ws[a.N + n]));
    else if (a.bias)
      y += a.bias[n];
    store_out(a, t, n, y);
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, cols);
  }
}

// ---- many tokens ----------------------------------------------------------------

constexpr int kWideStages = 6;
constexpr int kWideSmem = kWideStages * 2 * kTile + kSmemExtra;

template <bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    wide_kernel(const __grid_constant__ LinArgs a, const __grid_constant__ CUtensorMap tm_x,
                const __grid_constant__ CUtensorMap tm_w) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sA = smem;                       // [stages][128][128 B] tokens
  uint8_t* sB = sA + kWideStages * kTile;   // [stages][128][128 B] weights
  uint64_t* full = reinterpret_cast<uint64_t*>(sB + kWideStages * kTile);  // the even CTA's: both CTAs' copies
  uint64_t* empty = full + kWideStages;
  uint64_t* acc_full = empty + kWideStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2], the even CTA's
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kWideStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int m_tiles = (a.T + 255) / 256;
  constexpr int kBN = GATED ? 128 : 256;  // output columns of a tile
  const int n_tiles = (a.N + kBN - 1) / kBN;
  const int total = m_tiles * n_tiles;
  const int ksteps = (a.K + kBK - 1) / kBK;
  const int first = blockIdx.x / 2, step = gridDim.x / 2;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int tile = first; tile < total && ok; tile += step) {
        const int m = tile % m_tiles, n = tile / m_tiles;
        const int ya = m * 256 + rank * 128;
        const int yb = GATED ? rank * a.N + n * 128 : n * 256 + rank * 128;
        for (int ks = 0; ks < ksteps; ++ks, ++it) {
          const int s = it % kWideStages;
          if (!(ok = mbar_wait(&empty[s], ((it / kWideStages) & 1) ^ 1, abort_flag, kWaitNs))) break;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 4 * kTile);
          const uint32_t bar = cluster_addr(smem_u32(&full[s]), 0);
          tma_load_2d_pair(sA + s * kTile, &tm_x, bar, ks * kBK, ya);
          tma_load_2d_pair(sB + s * kTile, &tm_w, bar, ks * kBK, yb);
        }
      }
      // the last MMAs' arrivals at this CTA's barriers, so that none comes after its end
      for (int j = 0; j < kWideStages && ok; ++j, ++it)
        ok = mbar_wait(&empty[it % kWideStages], ((it / kWideStages) & 1) ^ 1, abort_flag, kWaitNs);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = umma_idesc_s8(256, 256);
      uint32_t it = 0, use = 0;
      bool ok = true;
      for (int tile = first; tile < total && ok; tile += step, ++use) {
        const int buf = use & 1;
        if (!(ok = mbar_wait(&acc_empty[buf], ((use >> 1) & 1) ^ 1, abort_flag, kWaitNs))) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * 256;
        for (int ks = 0; ks < ksteps; ++ks, ++it) {
          const int s = it % kWideStages;
          if (!(ok = mbar_wait(&full[s], (it / kWideStages) & 1, abort_flag, kWaitNs))) break;
          tc_fence_after();
          const uint64_t da = umma_desc_sw128(smem_u32(sA + s * kTile));
          const uint64_t db = umma_desc_sw128(smem_u32(sB + s * kTile));
#pragma unroll
          for (int kk = 0; kk < kBK / 32; ++kk)
            umma_s8<true>(d, da + 2 * kk, db + 2 * kk, idesc, (ks | kk) != 0);
          umma_commit_pair(&empty[s]);
        }
        if (ok) umma_commit_pair(&acc_full[buf]);
      }
    }
  } else {
    const int quad = warp & 3, half = (warp - kEpiWarp0) >> 2;
    const int es = a.out_f32 ? 4 : 2;
    const bool vec = ((uintptr_t)a.out & 15) == 0 && (a.ldo * es) % 16 == 0;
    uint32_t use = 0;
    for (int tile = first; tile < total; tile += step, ++use) {
      const int m = tile % m_tiles, n0 = tile / m_tiles * kBN;
      const int buf = use & 1;
      if (!mbar_wait_warp(&acc_full[buf], (use >> 1) & 1, abort_flag, kWaitNs)) break;
      tc_fence_after();
      const long long t = (long long)m * 256 + rank * 128 + quad * 32 + lane;
      const float xs = t < a.T ? a.xs[t] : 0.0f;
      const uint32_t tb = tmem + ((uint32_t)(quad * 32) << 16) + buf * 256;
      for (int c0 = half * (kBN / 2); c0 < (half + 1) * (kBN / 2); c0 += 16) {
        uint32_t v[16], u[16];
        __syncwarp();  // (rows past T skip the stores below)
        tmem_ld16_nowait(tb + c0, v);
        if (GATED) tmem_ld16_nowait(tb + 128 + c0, u);
        tmem_wait_ld();
        const int n = n0 + c0;
        float y[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int nj = min(n + j, a.N - 1);
          y[j] = scaled((int)v[j], xs, a.ws[nj]);
          if (GATED)
            y[j] = silu_mul(y[j], scaled((int)u[j], xs, a.ws[a.N + nj]));
          else if (a.bias)
            y[j] += a.bias[nj];
        }
        if (t >= a.T) {
        } else if (vec && n + 16 <= a.N) {
          if (a.out_f32) {
            float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + t * a.ldo + n);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
          } else {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
              w[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + t * a.ldo + n);
            o[0] = make_uint4(w[0], w[1], w[2], w[3]);
            o[1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (n + j < a.N) store_out(a, t, n + j, y[j]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_u32(&acc_empty[buf]), 0));
    }
  }

  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) give_up(a.status, full, kWideStages);
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// int8 rows of `cols` bytes, `ld` apart: boxes of 128 bytes x box_rows rows, 128-byte swizzle
bool map_rows(CUtensorMap* map, const int8_t* base, uint64_t cols, uint64_t rows, uint64_t ld, uint32_t box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {ld};
  cuuint32_t box[2] = {(cuuint32_t)kBK, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms = 148;
  return sms;
}

template <bool GATED>
int launch_mid(const LinArgs& a, cudaStream_t s) {
  MidPlan p;
  p.bn = (a.T + 15) / 16 * 16;
  p.ksteps = (a.K + kBK - 1) / kBK;
  const int tiles = GATED ? (a.N + 63) / 64 : (a.N + 127) / 128;
  // K split until every SM has a CTA, at most a portable cluster of 8, and two k-steps each
  int splits = 1;
  const int sms = sm_count();
  while (splits < 8 && tiles * (splits + 1) <= sms && p.ksteps >= 2 * (splits + 1)) ++splits;
  const int stage = kTile + p.bn * kBK;
  p.stages = (kSmemLimit - kSmemExtra) / stage;
  if (p.stages > 10) p.stages = 10;
  const int most = (p.ksteps + splits - 1) / splits;
  // the ring is also the inbox of the partial sums, 512 bytes a column and source
  const int box = splits * ((p.bn + splits - 1) / splits) * 512;
  if (p.stages > most) p.stages = most;
  if (p.stages * stage < box) p.stages = (box + stage - 1) / stage;
  const int smem = p.stages * stage + kSmemExtra;
  if (smem > kSmemLimit) return MOE_Q4_ECUDA;
  CUtensorMap tx, tw;
  if (!map_rows(&tx, a.x, a.K, a.T, a.ldx, p.bn) ||
      !map_rows(&tw, a.w, a.K, GATED ? 2ull * a.N : a.N, a.ldw, GATED ? 64 : 128))
    return MOE_Q4_ECUDA;
  if (cudaFuncSetAttribute(mid_kernel<GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) != cudaSuccess)
    return MOE_Q4_ECUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = splits;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles, splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mid_kernel<GATED>, a, p, tx, tw) == cudaSuccess ? MOE_Q4_OK : MOE_Q4_ECUDA;
}

template <bool GATED>
int launch_wide(const LinArgs& a, cudaStream_t s) {
  const long long tiles = (((long long)a.T + 255) / 256) * ((a.N + (GATED ? 127 : 255)) / (GATED ? 128 : 256));
  if (tiles > 0x3fffffff) return MOE_Q4_ENOTSUP;
  CUtensorMap tx, tw;
  if (!map_rows(&tx, a.x, a.K, a.T, a.ldx, 128) ||
      !map_rows(&tw, a.w, a.K, GATED ? 2ull * a.N : a.N, a.ldw, 128))
    return MOE_Q4_ECUDA;
  if (cudaFuncSetAttribute(wide_kernel<GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kWideSmem) != cudaSuccess)
    return MOE_Q4_ECUDA;
  const int pairs = sm_count() / 2;
  const int grid = 2 * (int)(tiles < pairs ? tiles : pairs);
  wide_kernel<GATED><<<grid, kThreads, kWideSmem, s>>>(a, tx, tw);
  return cudaGetLastError() == cudaSuccess ? MOE_Q4_OK : MOE_Q4_ECUDA;
}

}  // namespace

}  // namespace q4

int q4_launch_linear_mid(const q4::LinArgs& a, bool gated, cudaStream_t s) {
  return gated ? q4::launch_mid<true>(a, s) : q4::launch_mid<false>(a, s);
}

int q4_launch_linear_wide(const q4::LinArgs& a, bool gated, cudaStream_t s) {
  return gated ? q4::launch_wide<true>(a, s) : q4::launch_wide<false>(a, s);
}

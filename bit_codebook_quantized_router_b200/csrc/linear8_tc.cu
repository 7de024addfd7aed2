// Int8 products on the 5th-generation tensor cores (tcgen05, kind::i8, int32
// accumulators in TMEM), for moderate and large numbers of tokens.
//
// mid_kernel, up to 128 tokens: the weights' bytes bound it.  The MMA's M is 128
// weight rows and its N all the tokens, so each weight is read once; K is split
// over the CTAs of a cluster, two CTAs an SM to 64 tokens, so that every SM
// streams weights.
// The partial sums are int32, so adding them is exact in any order: each CTA
// sends the columns that another owns to that CTA's shared memory, and each
// finishes its own columns.  No workspace and one launch.  Measured, N = K =
// 6144 from memory: 17 tokens 10.5 us, 64 tokens 12.5 (3.1 TB/s with the
// launch), 128 tokens 16.5.  At 64 the weights arrive from 2.4 to 8.5-10 us of a
// CTA's life, the exchange and the last step take 3.  With the weights as the MMA's N = 256 and the tokens as
// its M, 64 tokens took 22 us: twice the sums to exchange, by half the warps.
//
// wide_kernel, more tokens: pairs of CTAs (cta_group::2) multiply 256 tokens
// by 256 weight rows, each CTA holding 128 rows of both operands, so a pair
// reads half of what two CTAs with tiles of 128 x 256 would; persistent, with
// two accumulators, so that one tile's results leave while the next is
// multiplied.  An MMA of 256 x 256 x 32 takes 129 cycles (128 is the units'
// rate); one of a single CTA, 128 rows, takes 170 whatever its N.  Measured:
// 8192 tokens, N = K = 6144 200 us, 3.1 POP/s (1.88 times the measured bf16
// rate; at 4096 tokens, 102 us, the tensor pipe is busy 85% of the time that SMs
// are); 2048 tokens 53 us; 256 tokens, K = 2048 9.6-9.9 us.  A tile's
// results take 4 us to leave, hidden but for the last tile's; staging them in
// shared memory for whole lines or for TMA stores was no faster end to end
// (2048 tokens, K = 2048: 23.6 us as it is, 25.2 to 26.0 so).
//
// Both read operands by TMA into the 128-byte-swizzle K-major layout, in
// k-steps of 128 bytes; what lies past a row, a matrix or K arrives as zeros.
// For the SwiGLU a tile holds as many rows of the gate as of the up
// projection.  Every wait is bounded; one that gives up records
// MOE_Q4_ETIMEOUT.
#include <cuda.h>

#include "linear8.cuh"
#include "rows8.cuh"
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
constexpr int kSmemExtra = 2048;       // alignment and barriers
constexpr int kMidStages = 8;

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// The waits' limit, and in the debug build what a test withholds to make one
// run out (moe_q4_debug_withhold).
#ifdef MOE_Q4_DEBUG
__device__ __forceinline__ uint64_t wait_ns(const LinArgs& a) { return a.limit_ns; }
__device__ __forceinline__ bool withheld(const LinArgs& a, int block) { return block == a.withheld && !a.late; }
__device__ __forceinline__ void send_late(const LinArgs& a, int block) {
  if (block != a.withheld || !a.late) return;
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 4 * a.limit_ns) __nanosleep(1000);
}
#else
__device__ __forceinline__ constexpr uint64_t wait_ns(const LinArgs&) { return kWaitNs; }
__device__ __forceinline__ constexpr bool withheld(const LinArgs&, int) { return false; }
__device__ __forceinline__ void send_late(const LinArgs&, int) {}
#endif

// The status word of calls that were given none.
__device__ int32_t common_status;

__device__ __forceinline__ void record_timeout(const LinArgs& a) {
  record_error(a.status ? a.status : &common_status, MOE_Q4_ETIMEOUT);
}

// On an abandoned wait: record it and let the copies in flight land before
// the shared memory goes away.
__device__ __forceinline__ void give_up(const LinArgs& a, uint64_t* full, int stages) {
  record_timeout(a);
  for (int s = 0; s < stages; ++s)
    for (uint32_t par = 0; par < 2; ++par) {
      volatile int quick = 0;
      mbar_wait(&full[s], par, &quick, 20000000ull);
    }
}

// ---- up to 128 tokens -----------------------------------------------------------

struct MidPlan {
  int bn;       // tokens, rounded up to 16
  int own;      // columns that a CTA of the cluster finishes (a multiple of 8)
  int stages;   // ring stages
  int ksteps;   // k-steps of 128 in K
  int inbox;    // byte offset of the other CTAs' partial sums, behind the ring
};

template <bool GATED>
__global__ void __launch_bounds__(kThreads)
    mid_kernel(const __grid_constant__ LinArgs a, const __grid_constant__ MidPlan p,
               const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint64_t full[kMidStages], empty[kMidStages], acc_full[1], in_full[1];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word, in_abort_word;
  __shared__ RowFactor s_xs[kLinearMidTokens];
  volatile int* abort_flag = &abort_word;
  volatile int* in_abort = &in_abort_word;
  uint8_t* smem = align1024(smem_raw);
  const int S = p.stages, b_tile = p.bn * kBK;
  uint8_t* sA = smem;              // [S][128][128 B] weights
  uint8_t* sB = sA + S * kTile;    // [S][bn][128 B] tokens

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = gridDim.y, rank = blockIdx.y;  // the cluster's CTAs share blockIdx.x
  const int n0 = blockIdx.x * (GATED ? 64 : 128);
  const int k_lo = (int)((long long)p.ksteps * rank / splits);
  const int k_hi = (int)((long long)p.ksteps * (rank + 1) / splits);
  uint32_t cols = 32;
  while (cols < (uint32_t)p.bn) cols *= 2;
  auto load_w = [&](int ks, int s) {
    mbar_arrive_expect_tx(&full[s], kTile + b_tile);
    tma_load_2d(sA + s * kTile, &tm_w, &full[s], ks * kBK, n0);
    if (GATED) tma_load_2d(sA + s * kTile + kTile / 2, &tm_w, &full[s], ks * kBK, a.N + n0);
  };
  const int block = blockIdx.x * splits + rank;
  auto load_x = [&](int ks, int s) {
    if (ks != k_lo || !withheld(a, block)) tma_load_2d(sB + s * b_tile, &tm_x, &full[s], ks * kBK, 0);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(in_full, splits * kEpiWarps);
    *abort_flag = *in_abort = 0;
    fence_mbar_init();
    // the ring's first loads, before anything is set up beside them; in a
    // chain the weights' before the kernel in front is done with the tokens
    if (!a.chained) pdl_wait();
    for (int i = 0; i < S && k_lo + i < k_hi; ++i) {
      load_w(k_lo + i, i);
      if (!a.chained) load_x(k_lo + i, i);
    }
    if (a.chained) {
      pdl_wait();
      for (int i = 0; i < S && k_lo + i < k_hi; ++i) load_x(k_lo + i, i);
    }
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(&tmem_slot, cols);
    tmem_relinquish();
  }
  // what the results are scaled with, while the sums are made
  const int c_lo = rank * p.own, c_n = min(p.own, a.T - c_lo);
  const int et = threadIdx.x - 32 * kEpiWarp0;  // epilogue thread: one weight row, every second (fourth) column
  constexpr int kRows = GATED ? 64 : 128;
  const int n = n0 + (et & (kRows - 1));
  float wscale = 0.0f, uscale = 0.0f, bias = 0.0f;
  pdl_wait();  // (before these loads: it waits for them)
  if (et >= 0 && n < a.N) {
    wscale = a.ws[n];
    if (GATED) uscale = a.ws[a.N + n];
    if (!GATED && a.bias) bias = a.bias[n];
  }
  tc_fence_before();
  __syncthreads();
  pdl_trigger();  // (once this CTA has its tensor memory: the next kernel's CTAs may ask for all that is left)
  cluster_arrive_relaxed();  // this CTA's barriers are ready (waited for before anything is sent)
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      int it = S;
      for (int ks = k_lo + S; ks < k_hi; ++ks, ++it) {
        const int s = it % S;
        if (!mbar_wait(&empty[s], ((it / S) & 1) ^ 1, abort_flag, wait_ns(a))) break;
        load_w(ks, s);
        load_x(ks, s);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = umma_idesc_s8(128, p.bn);
      int it = 0;
      for (int ks = k_lo; ks < k_hi; ++ks, ++it) {
        const int s = it % S;
        if (!mbar_wait(&full[s], (it / S) & 1, abort_flag, wait_ns(a))) break;
        tc_fence_after();
        const uint64_t da = umma_desc_sw128(smem_u32(sA + s * kTile));
        const uint64_t db = umma_desc_sw128(smem_u32(sB + s * b_tile));
#pragma unroll
        for (int kk = 0; kk < kBK / 32; ++kk)  // 32 bytes of K per MMA
          umma_s8<false>(tmem, da + 2 * kk, db + 2 * kk, idesc, (it | kk) != 0);
        umma_commit(&empty[s]);
      }
      umma_commit(acc_full);
      mbar_wait(acc_full, 0, abort_flag, wait_ns(a));
    }
  } else if (et < c_n) {
    s_xs[et] = row_factor(a.xs[c_lo + et]);
  }
  __syncthreads();
  // every MMA is done, or a wait was given up
  if (threadIdx.x == 0 && *abort_flag) give_up(a, full, S);
  __syncwarp();
  cluster_wait();
  tc_fence_after();
  // The second barrier of the cluster: no CTA ends, and its shared memory with
  // it, before every other has sent, whatever wait was given up.
  if (warp < kEpiWarp0) {
    cluster_arrive_relaxed();
  } else {
    send_late(a, block);
    // send: columns [own * r, own * (r + 1)) to CTA r as [src][column][128
    // rows], a warp 128 consecutive bytes at a time (16 bytes a lane at a row's
    // pitch measured slower, 17.1 against 14.6 us at 64 tokens and 6144 x 6144,
    // and so did bulk copies of what was gathered here first, 15.6)
    const int quad = warp & 3, half = (warp - kEpiWarp0) >> 2, row = quad * 32 + lane;
    const uint32_t tb = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t inbox = smem_u32(smem) + p.inbox;
    const uint32_t mine = inbox + (rank * p.own * 128 + row) * 4;
    for (int c0 = half * 16; c0 < p.bn; c0 += 32) {
      uint32_t v[16];
      tmem_ld16_nowait(tb + c0, v);
      tmem_wait_ld();
#pragma unroll
      for (int h = 0; h < 16; h += 8) {
        const int to = (c0 + h) / p.own;
        const uint32_t at = cluster_addr(mine + (c0 + h - to * p.own) * 512, to);
#pragma unroll
        for (int j = 0; j < 8; ++j) cluster_st32(at + j * 512, v[h + j]);
      }
    }
    __syncwarp();
    if (lane < splits) mbar_arrive_cluster(cluster_addr(smem_u32(in_full), lane));
    __syncwarp();
    cluster_arrive_relaxed();  // (the arrivals in front waited for what was sent)
    tc_fence_before();

    // finish this CTA's columns, four at a time, once all their sums are here
    // (a CTA that gave a wait up sends what it has all the same, so this wait is
    // longer than those, and has a flag of its own)
    if (!mbar_wait_warp<true>(in_full, 0, in_abort, 3 * wait_ns(a))) *abort_flag = 1;
    if (n < a.N) {
      constexpr int kStep = 32 * kEpiWarps / kRows;
      const uint32_t box = inbox + (et & (kRows - 1)) * 4;
      for (int c0 = et / kRows; c0 < c_n; c0 += 4 * kStep) {
        int v[4] = {}, u[4] = {};
        for (int src = 0; src < splits; ++src)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t at = box + (src * p.own + min(c0 + j * kStep, c_n - 1)) * 512;
            v[j] += (int)lds32(at);
            if (GATED) u[j] += (int)lds32(at + 256);
          }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = c0 + j * kStep;
          if (c >= c_n) break;
          const RowFactor xs = s_xs[c];
          float y = scaled(v[j], xs, wscale);
          if (GATED)
            y = swiglu(y, scaled(u[j], xs, uscale));
          else if (a.bias)
            y += bias;
          store_out(a, c_lo + c, n, y);
        }
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) record_timeout(a);
  cluster_wait();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, cols);
  }
}

// ---- many tokens ----------------------------------------------------------------

constexpr int kWideStages = 6;
constexpr int kWideRow = 17;  // floats of a staged row of 16
constexpr int kWideSmem = kWideStages * 2 * kTile + kSmemExtra + 2 * 512 * 4 + kEpiWarps * 32 * kWideRow * 4;

// How the output's rows can be written: 32 bytes at a time, 16, or as they come.
__device__ __forceinline__ int out_align(const LinArgs& a) {
  const unsigned long long es = a.out_f32 ? 4 : 2, b = (uintptr_t)a.out | (a.ldo * es);
  return b % 32 == 0 ? 32 : (b % 16 == 0 ? 16 : 1);
}

__device__ __forceinline__ void store32(void* p, const uint32_t w[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 16 values of row t from column n, one row a lane (t >= a.T: nothing).
// A row's values leave in whole sectors where its alignment allows; else they
// go through shared memory, so that lanes write along the rows.
__device__ __forceinline__ void store_row16(const LinArgs& a, int align, float* stage, long long t, int n,
                                            const float y[16]) {
  const int lane = threadIdx.x & 31;
  if (align > 1 && n + 16 <= a.N) {
    if (t >= a.T) return;
    uint32_t w[16];
    int words;
    char* p;
    if (a.out_f32) {
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(y[j]);
      p = reinterpret_cast<char*>(reinterpret_cast<float*>(a.out) + t * a.ldo + n);
      words = 16;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      p = reinterpret_cast<char*>(reinterpret_cast<__nv_bfloat16*>(a.out) + t * a.ldo + n);
      words = 8;
    }
#pragma unroll
    for (int j = 0; j < 16; j += 8) {
      if (j >= words) break;
      if (align == 32) {
        store32(p + 4 * j, w + j);
      } else {
        reinterpret_cast<uint4*>(p + 4 * j)[0] = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
        reinterpret_cast<uint4*>(p + 4 * j)[1] = make_uint4(w[j + 4], w[j + 5], w[j + 6], w[j + 7]);
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) stage[lane * kWideRow + j] = y[j];
  __syncwarp();
  const int c = lane & 15;
  if (n + c < a.N)
#pragma unroll 8
    for (int r = lane >> 4; r < 32; r += 2)
      if (t - lane + r < a.T) store_out(a, t - lane + r, n + c, stage[r * kWideRow + c]);
  __syncwarp();
}

// SPLIT > 1: a cluster of SPLIT pairs has one tile; each pair multiplies a part
// of K and finishes a part of the columns, with the others' int32 sums of them
// (exact, so the result's bits are those of the unsplit kernel), which they send
// to its ring once it is done with.
template <bool GATED, int BN, int SPLIT>
__global__ void __cluster_dims__(2 * SPLIT, 1, 1) __launch_bounds__(kThreads, 1)
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
  uint64_t* ready = acc_empty + 2;           // SPLIT: the others' rings are done with
  uint64_t* in_full = ready + 1;             // SPLIT: the others' sums are here
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(in_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* s_scale = reinterpret_cast<float*>(sB + kWideStages * kTile + 512);  // [2][256] the columns' scales
  float* s_bias = s_scale + 512;                                              // [2][256] and biases
  float* s_rows = s_bias + 512;                                               // [epilogue warps][32][kWideRow]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank() & 1, part = SPLIT > 1 ? (int)cluster_rank() >> 1 : 0, lead = 2 * part;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kWideStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    if (SPLIT > 1) {
      mbar_init(ready, SPLIT - 1);
      mbar_init(in_full, (SPLIT - 1) * kEpiWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 2 * BN);
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int m_tiles = (a.T + 255) / 256;
  constexpr int kBN = GATED ? BN / 2 : BN;  // output columns of a tile
  const int n_tiles = (a.N + kBN - 1) / kBN;
  const int total = m_tiles * n_tiles;
  const int all = (a.K + kBK - 1) / kBK, k_lo = all * part / SPLIT, ksteps = all * (part + 1) / SPLIT - k_lo;
  const int first = blockIdx.x / (2 * SPLIT), step = gridDim.x / (2 * SPLIT);

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true, filled = !a.chained;
      auto load_x = [&](int s, uint32_t bar, int ks, int y, bool first) {
        if (!first || !withheld(a, blockIdx.x)) tma_load_2d_pair(sA + s * kTile, &tm_x, bar, (k_lo + ks) * kBK, y);
      };
      if (!a.chained) pdl_wait();
      for (int tile = first; tile < total && ok; tile += step) {
        const int m = tile % m_tiles, n = tile / m_tiles;
        const int ya = m * 256 + rank * 128;
        const int yb = GATED ? rank * a.N + n * kBN : n * BN + rank * (BN / 2);
        for (int ks = 0; ks < ksteps; ++ks, ++it) {
          const int s = it % kWideStages;
          if (!(ok = mbar_wait(&empty[s], ((it / kWideStages) & 1) ^ 1, abort_flag, wait_ns(a)))) break;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (kTile + BN / 2 * kBK));
          const uint32_t bar = cluster_addr(smem_u32(&full[s]), lead);
          tma_load_2d_pair(sB + s * kTile, &tm_w, bar, (k_lo + ks) * kBK, yb);
          // in a chain the ring's first weights are asked for before the
          // kernel in front is done with the tokens (elsewhere step by step:
          // weights first costs 1 us)
          if (!filled) {
            if ((int)it + 1 < min(kWideStages, ksteps)) continue;
            pdl_wait();
            for (int i = 0; i < ks; ++i) load_x(i, cluster_addr(smem_u32(&full[i]), lead), i, ya, i == 0);
            filled = true;
          }
          load_x(s, bar, ks, ya, it == 0);
        }
      }
      // the last MMAs' arrivals at this CTA's barriers, so that none comes after its end
      for (int j = 0; j < kWideStages && ok; ++j, ++it)
        ok = mbar_wait(&empty[it % kWideStages], ((it / kWideStages) & 1) ^ 1, abort_flag, wait_ns(a));
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      pdl_wait();  // (so that the waits' limits do not count the kernel in front, however long it runs)
      const uint32_t idesc = umma_idesc_s8(256, BN);
      uint32_t it = 0, use = 0;
      bool ok = true;
      for (int tile = first; tile < total && ok; tile += step, ++use) {
        const int buf = use & 1;
        if (!(ok = mbar_wait(&acc_empty[buf], ((use >> 1) & 1) ^ 1, abort_flag, wait_ns(a)))) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * BN;
        for (int ks = 0; ks < ksteps; ++ks, ++it) {
          const int s = it % kWideStages;
          if (!(ok = mbar_wait(&full[s], (it / kWideStages) & 1, abort_flag, wait_ns(a)))) break;
          tc_fence_after();
          const uint64_t da = umma_desc_sw128(smem_u32(sA + s * kTile));
          const uint64_t db = umma_desc_sw128(smem_u32(sB + s * kTile));
#pragma unroll
          for (int kk = 0; kk < kBK / 32; ++kk)
            umma_s8<true>(d, da + 2 * kk, db + 2 * kk, idesc, (ks | kk) != 0);
          umma_commit_pair(&empty[s], lead);
        }
        if (ok) umma_commit_pair(&acc_full[buf], lead);
      }
      // the last tiles' arrivals from the pair's other CTA, so that none comes
      // after this one's end
      for (uint32_t u = use > 2 ? use - 2 : 0; u < use && ok; ++u)
        ok = mbar_wait(&acc_empty[u & 1], (u >> 1) & 1, abort_flag, wait_ns(a));
    }
  } else {
    const int quad = warp & 3, half = (warp - kEpiWarp0) >> 2, e = threadIdx.x - 32 * kEpiWarp0;
    const int align = out_align(a);
    pdl_wait();
    pdl_trigger();  // (after the wait: the next kernels of a chain read weights at once)
    float* stage = s_rows + (warp - kEpiWarp0) * 32 * kWideRow;
    uint32_t use = 0;
    bool lost = false;
    for (int tile = first; tile < total; tile += step, ++use) {
      const int m = tile % m_tiles, n0 = tile / m_tiles * kBN;
      const int buf = use & 1;
      // the columns' scales, while the tile is multiplied (a buffer is written
      // again two tiles later, past the barrier of the tile between)
      {
        const int n = n0 + (e & (kBN - 1));
        float* sc = s_scale + buf * 256;
        if (e < BN) sc[e] = n < a.N ? a.ws[GATED && e >= kBN ? a.N + n : n] : 0.0f;
        if (!GATED && e < BN) s_bias[buf * 256 + e] = a.bias && n < a.N ? a.bias[n] : 0.0f;
      }
      const long long t = (long long)m * 256 + rank * 128 + quad * 32 + lane;
      const RowFactor xf = row_factor(t < a.T ? a.xs[t] : 0.0f);
      named_bar(1, 32 * kEpiWarps);
      // (a warp whose wait was given up still meets the others at the barrier)
      if (lost || (lost = !mbar_wait_warp(&acc_full[buf], (use >> 1) & 1, abort_flag, wait_ns(a)))) continue;
      tc_fence_after();
      const uint32_t tb = tmem + ((uint32_t)(quad * 32) << 16) + buf * BN;
      constexpr int kOwn = kBN / SPLIT, kCols = kOwn / 2;  // columns of this pair, of this warp
      constexpr int kPlanes = GATED ? 2 : 1;
      // [SPLIT - 1][kPlanes][kOwn / 4][128 rows][4 columns]: a warp writes and reads 512 consecutive bytes
      const uint32_t inbox = smem_u32(sA) + (quad * 32 + lane) * 16;
      if (SPLIT > 1) {
        // this CTA's ring is free; once the others' are, their columns' sums go there
        if (e < SPLIT && e != part) mbar_arrive_cluster(cluster_addr(smem_u32(ready), 2 * e + rank));
        if ((lost = !mbar_wait_warp<true>(ready, 0, abort_flag, wait_ns(a)))) continue;
#pragma unroll
        for (int d = 1; d < SPLIT; ++d) {
          const int to = (part + d) % SPLIT;
          const uint32_t at = cluster_addr(inbox + (d - 1) * kPlanes * kOwn * 512, 2 * to + rank);
#pragma unroll
          for (int pl = 0; pl < kPlanes; ++pl)
#pragma unroll
            for (int c = 0; c < kCols; c += 16) {
              uint32_t w[16];
              tmem_ld16_nowait(tb + pl * kBN + to * kOwn + half * kCols + c, w);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; j += 4) cluster_st128(at + (pl * kOwn + half * kCols + c + j) * 512, w + j);
            }
        }
        __syncwarp();
        if (lane < SPLIT && lane != part) mbar_arrive_cluster(cluster_addr(smem_u32(in_full), 2 * lane + rank));
        __syncwarp();
        if ((lost = !mbar_wait_warp<true>(in_full, 0, abort_flag, wait_ns(a)))) continue;
      }
      uint32_t v[2][16], u[2][16];
      auto load = [&](int i) {
        const int c = part * kOwn + half * kCols + i * 16;
        tmem_ld16_nowait(tb + c, v[i & 1]);
        if (GATED) tmem_ld16_nowait(tb + kBN + c, u[i & 1]);
      };
      load(0);
#pragma unroll
      for (int i = 0; i < kCols / 16; ++i) {
        tmem_wait_ld();
        if (i + 1 < kCols / 16) {
          load(i + 1);
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_u32(&acc_empty[buf]), lead));
        }
        if (SPLIT > 1) {
#pragma unroll
          for (int src = 0; src < SPLIT - 1; ++src)
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const uint32_t at = inbox + (src * kPlanes * kOwn + half * kCols + i * 16 + j) * 512;
              auto add = [](uint32_t d[4], uint4 w) { d[0] += w.x, d[1] += w.y, d[2] += w.z, d[3] += w.w; };
              add(v[i & 1] + j, lds32x4(at));
              if (GATED) add(u[i & 1] + j, lds32x4(at + kOwn * 512));
            }
        }
        const int c = part * kOwn + half * kCols + i * 16;
        const float* sc = s_scale + buf * 256 + c;
        const float* sb = s_bias + buf * 256 + c;
        const F2 xs2 = f2(xf.s, xf.s);
        float y[16];
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          // (as scaled(), two at a time)
          const float4 w = *reinterpret_cast<const float4*>(sc + j);
          const uint32_t* q = v[i & 1] + j;
          split(mul(mul(f2((float)(int)q[0], (float)(int)q[1]), xs2), f2(w.x, w.y)), y[j], y[j + 1]);
          split(mul(mul(f2((float)(int)q[2], (float)(int)q[3]), xs2), f2(w.z, w.w)), y[j + 2], y[j + 3]);
          if (xf.up)
#pragma unroll
            for (int h = 0; h < 4; ++h) y[j + h] = __fmul_rn(y[j + h], kScaleUp);
          if (GATED) {
            const float4 g = *reinterpret_cast<const float4*>(sc + kBN + j);
            const uint32_t* p = u[i & 1] + j;
            float z[4];
            split(mul(mul(f2((float)(int)p[0], (float)(int)p[1]), xs2), f2(g.x, g.y)), z[0], z[1]);
            split(mul(mul(f2((float)(int)p[2], (float)(int)p[3]), xs2), f2(g.z, g.w)), z[2], z[3]);
            if (xf.up)
#pragma unroll
              for (int h = 0; h < 4; ++h) z[h] = __fmul_rn(z[h], kScaleUp);
#pragma unroll
            for (int h = 0; h < 4; ++h) y[j + h] = swiglu(y[j + h], z[h]);
          } else if (a.bias) {
            const float4 b = *reinterpret_cast<const float4*>(sb + j);
            y[j] += b.x, y[j + 1] += b.y, y[j + 2] += b.z, y[j + 3] += b.w;
          }
        }
        store_row16(a, align, stage, t, n0 + c, y);
        __syncwarp();
      }
    }
  }

  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) give_up(a, full, kWideStages);
  __syncthreads();
  cluster_arrive_relaxed();  // (a release would wait for the results' stores)
  cluster_wait();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * BN);
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
  const int stage = kTile + p.bn * kBK;
  // two CTAs an SM where their rings and inboxes fit (to 64 tokens), else one
  const int an_sm = p.bn <= 64 ? 2 : 1, room = an_sm == 2 ? 108 * 1024 : 216 * 1024;
  // K split in two, four or eight while the CTAs fit the card at once (clusters
  // leave an eighth of it unused, at one CTA an SM those of eight a fifth) and
  // keep two k-steps
  const long long slots = an_sm * sm_count();
  int splits = 1;
  while (splits < 8 && 2ll * splits * tiles <= (splits == 4 && an_sm == 1 ? slots * 4 / 5 : slots * 7 / 8) && p.ksteps >= 4 * splits)
    splits *= 2;
  p.own = (p.bn / 8 + splits - 1) / splits * 8;
  const int most = (p.ksteps + splits - 1) / splits, box = splits * p.own * 512;
  p.stages = min(min(most, kMidStages), (room - box) / stage);
  p.inbox = p.stages * stage;
  const int smem = p.inbox + box + 1024;
  CUtensorMap tx, tw;
  if (!map_rows(&tx, a.x, a.K, a.T, a.ldx, p.bn) ||
      !map_rows(&tw, a.w, a.K, GATED ? 2ull * a.N : a.N, a.ldw, GATED ? 64 : 128))
    return MOE_Q4_ECUDA;
  if (cudaFuncSetAttribute(mid_kernel<GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024) !=
          cudaSuccess ||
      cudaFuncSetAttribute(mid_kernel<GATED>, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess)
    return MOE_Q4_ECUDA;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = splits;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles, splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, mid_kernel<GATED>, a, p, tx, tw) == cudaSuccess ? MOE_Q4_OK : MOE_Q4_ECUDA;
}

template <bool GATED, int BN, int SPLIT>
int launch_wide(const LinArgs& a, cudaStream_t s) {
  constexpr int cols = GATED ? BN / 2 : BN;
  const long long tiles = (((long long)a.T + 255) / 256) * ((a.N + cols - 1) / cols);
  if (tiles > 0x3fffffff) return MOE_Q4_ENOTSUP;
  CUtensorMap tx, tw;
  if (!map_rows(&tx, a.x, a.K, a.T, a.ldx, 128) ||
      !map_rows(&tw, a.w, a.K, GATED ? 2ull * a.N : a.N, a.ldw, BN / 2))
    return MOE_Q4_ECUDA;
  const auto kernel = wide_kernel<GATED, BN, SPLIT>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWideSmem) != cudaSuccess)
    return MOE_Q4_ECUDA;
  const int pairs = sm_count() / 2;
  const int grid = SPLIT > 1 ? 2 * SPLIT * (int)tiles : 2 * (int)(tiles < pairs ? tiles : pairs);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kWideSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, tx, tw) == cudaSuccess ? MOE_Q4_OK : MOE_Q4_ECUDA;
}

template <bool GATED>
int launch_wide(const LinArgs& a, cudaStream_t s) {
  // A k-step takes 0.26 to 0.28 us whatever the tile's width (the MMA's 256 rows
  // bound it), so tiles are wide; narrower ones are for products whose tiles
  // leave SMs idle: each then writes fewer results (T = 256, N = 6144,
  // K = 2048: 12.6 us with 256 columns, 11.9 with 128, 14.8 with 64 in two
  // turns; N = K = 512: 8.0, 6.6 and 5.8).
  const long long m = (a.T + 255) / 256, sms = sm_count(), pairs = sms / 2, n = GATED ? 2ll * a.N : a.N;
  const long long t128 = m * ((n + 127) / 128), t256 = m * ((n + 255) / 256);
  // A long K is split over the pairs of a cluster where the clusters fit the
  // card at once (32 of four CTAs, 15 of eight): the exchange of the sums costs
  // what 10 to 20 k-steps do.  Measured at 256 tokens, us, unsplit and split:
  // N = 2048 in tiles of 128 over two pairs, K = 2048 8.0 and 8.1, K = 2560 9.1
  // and 8.7, K = 4096 12.9 and 10.8; N = 6144 in tiles of 256, K = 2560 11.1 and
  // 12.0, K = 4096 14.8 and 14.0 (N = 8192 15.0 and 15.1), K = 6144 19.0 and
  // 16.5; N = 512 over two and four pairs, K = 3584 9.5 and 9.8, K = 5120 11.3
  // and 10.6, K = 8192 14.7 and 12.4.
  if (a.K >= 5120 && 8 * t256 <= sms * 5 / 6) return launch_wide<GATED, 256, 4>(a, s);
  if (a.K >= 2560 && 4 * t128 <= sms * 8 / 9) return launch_wide<GATED, 128, 2>(a, s);
  if (a.K >= 4096 && 4 * t256 <= sms * 8 / 9) return launch_wide<GATED, 256, 2>(a, s);
  if (m * ((n + 63) / 64) <= pairs) return launch_wide<GATED, 64, 1>(a, s);
  if (m * ((n + 127) / 128) <= pairs) return launch_wide<GATED, 128, 1>(a, s);
  return launch_wide<GATED, 256, 1>(a, s);
}

}  // namespace

}  // namespace q4

extern "C" int moe_q4_i8_status(void* stream) {
  void* word = nullptr;
  if (cudaGetSymbolAddress(&word, q4::common_status) != cudaSuccess) return MOE_Q4_ECUDA;
  const int rc = moe_q4_read_status(static_cast<const int32_t*>(word), stream);
  if (rc == MOE_Q4_ETIMEOUT && cudaMemsetAsync(word, 0, sizeof(int32_t), (cudaStream_t)stream) != cudaSuccess)
    return MOE_Q4_ECUDA;
  return rc;
}

#ifdef MOE_Q4_DEBUG
static uint64_t debug_limit_ns = q4::kWaitNs;
static int debug_block = -1, debug_late = 0;

// Test support, this build only: from now on the products of this file limit
// their device waits to limit_us (1 .. 2,000,000; the release build's is the
// last), and block `block` of each launch (-1: none) never asks for its first
// tokens or, with `late` (to 128 tokens), sends its partial sums only after four
// limits, so that waits run out.  Not for calls from several threads.
extern "C" MOE_Q4_API int moe_q4_debug_withhold(int block, int late, unsigned limit_us) {
  if (block < -1 || limit_us == 0 || limit_us > 2000000u) return MOE_Q4_EINVAL;
  debug_block = block, debug_late = late, debug_limit_ns = (uint64_t)limit_us * 1000ull;
  return MOE_Q4_OK;
}

static q4::LinArgs with_debug(q4::LinArgs a) {
  a.limit_ns = debug_limit_ns, a.withheld = debug_block, a.late = debug_late;
  return a;
}
#else
static const q4::LinArgs& with_debug(const q4::LinArgs& a) { return a; }
#endif

int q4_launch_linear_mid(const q4::LinArgs& a, bool gated, cudaStream_t s) {
  return gated ? q4::launch_mid<true>(with_debug(a), s) : q4::launch_mid<false>(with_debug(a), s);
}

int q4_launch_linear_wide(const q4::LinArgs& a, bool gated, cudaStream_t s) {
  return gated ? q4::launch_wide<true>(with_debug(a), s) : q4::launch_wide<false>(with_debug(a), s);
}

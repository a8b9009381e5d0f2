// y = residual + act(x W + b), or with a gate
// y = residual + act(x Wg + bg) * (x W + b): bf16 operands, fp32 sums in TMEM,
// everything after the product in fp32, one rounding to y's type.
//
// "Flash-dLLM: I/O-Aware KV Caching and Parallel Decoding for Fast,
// Memory-Efficient Diffusion LLMs" (ai4snews summary), paragraph 1, covers a
// layer up to the attention output. These are the layer's other products (the
// projections of a single-token step, the feed-forward block), read with the
// conventions of Wqkv (y = x W, W row-major).
//
// Two kernels:
//   wide_kernel, for many rows, bound by the tensor cores. A pair of CTAs
//     (cta_group::2) computes 256 rows x 256 columns: 128 rows of x and half
//     of the columns of W are staged by each, so that each SM reads 64 bytes
//     of shared memory a cycle where a tile of its own would take 96. With a
//     gate the even CTA stages 128 columns of W and the odd one the same 128
//     of Wg: the accumulator then holds both products of an output side by
//     side and the epilogue needs no exchange. Persistent pairs; two
//     accumulators of 256 TMEM columns, so that the epilogue of a tile runs
//     under the products of the next.
//   narrow_kernel, for few rows, bound by the bytes of W. The product is
//     taken transposed, W's columns on the 128 rows of the instruction and
//     the 16 .. 128 rows of x on its N side, so that no part of it is
//     padding to 128 rows. Tiles of 64 to 256 columns, whose depth is split
//     over a cluster of one to eight CTAs, are chosen to give as many SMs
//     as possible an equal part of W; the partial sums meet in
//     shared memory, each CTA adding up its share of the rows in the order of
//     the ranks (the same result every time, no workspace).
// Both start under the tail of the launch before them (dependent launch): the
// barriers, the TMEM and the tensor maps are ready when its results are.
//
// Measured on one B200, device time of launches back to back: wide, 8192 rows, 4096 ->
// 12288 with gelu: 579 to 640 us (1420 to 1290 TFLOP/s, as the power limit leaves);
// gated, 1536 rows: 189 to 199 us (1640 to 1560 TFLOP/s, tensor pipe 95 % active), 224
// to 232 in minutes of such calls; 1001 rows, 1304 -> 2696: 16.0 us, of which 7 are fill
// and epilogue. Narrow, one row, 4096 -> 4096: 9.8 us (3.4 TB/s); to 12288: 20.1 us
// (5.0 TB/s); gated, 32 rows: 36.9 us (5.5 TB/s).
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "fdllm.h"
#include "fdllm_internal.h"
#include "host_api.h"
#include "ptx_serve.cuh"
#include "serve_internal.h"

namespace fdllm {
namespace {

constexpr int BK = 64;                   // depth of a stage: one 128-byte span
constexpr int BOX = BK * 64 * 2;         // a box of W: 64 K rows x 64 columns, 8 KB

// ---------------------------------------------------------------- epilogue arithmetic
__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {
    case FDLLM_ACT_RELU: return x > 0.f ? x : (x == x ? 0.f : x);
    case FDLLM_ACT_SILU: {
      // e = exp(-|x|) as a square: exp(x / 2) is a normal number down to x = -174,
      // so x e keeps its bits where e itself would not. The divisor is in [1, 2],
      // where the fast quotient is good to two steps.
      const float t = expf(-0.5f * fabsf(x)), e = t * t;
      return __fdividef(x < 0.f ? x * t * t : x, 1.f + e);
    }
    case FDLLM_ACT_GELU: return 0.5f * x * (1.f + erff(x * 0.7071067811865476f));
    case FDLLM_ACT_GELU_TANH:
      return 0.5f * x * (1.f + tanhf(0.7978845608028654f * fmaf(0.044715f * x * x, x, x)));
  }
  return x;
}

// N values: the choice once, not for each of them.
template <int N>
__device__ __forceinline__ void activate_all(float* v, int act) {
  if (act == FDLLM_ACT_RELU) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = activate(v[e], FDLLM_ACT_RELU);
  } else if (act == FDLLM_ACT_SILU) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = activate(v[e], FDLLM_ACT_SILU);
  } else if (act == FDLLM_ACT_GELU) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = activate(v[e], FDLLM_ACT_GELU);
  } else if (act == FDLLM_ACT_GELU_TANH) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = activate(v[e], FDLLM_ACT_GELU_TANH);
  }
}

__device__ __forceinline__ float bias_at(const void* p, int i, int f32) {
  return f32 ? reinterpret_cast<const float*>(p)[i]
             : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

// A bounded wait without side effects, and one that marks the CTA and reports
// when it (or another wait of the CTA) gives up. The producer and the issuer
// pass here once a stage on one thread, so a completed barrier costs one probe.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, const LinearArgs& a) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!ptx::mbar_try_wait(bar, parity))
    if (clock64() - t0 > a.wait_cycles) return false;
  return true;
}

__device__ __forceinline__ bool lin_wait(int* abort, uint64_t* bar, uint32_t parity,
                                         const LinearArgs& a) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (*reinterpret_cast<volatile int*>(abort)) return false;
    if (clock64() - t0 > a.wait_cycles) {
      atomicExch(abort, 1);
      if (a.status) atomicExch(reinterpret_cast<int*>(a.status), (int)FDLLM_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// Bytes to come for a stage, and the arrival that completes it with them (of the
// first one withheld where a test wants its wait to run out: fdllm_inject_tile_timeout).
__device__ __forceinline__ void expect(uint64_t* full, uint32_t bytes, bool first,
                                       const LinearArgs& a) {
  if (first && a.withhold) ptx::mbar_expect_tx(full, bytes);
  else ptx::mbar_arrive_expect_tx(full, bytes);
}

// A place in a ring of stages; `parity` is that of its current pass.
struct Ring {
  int s = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      parity ^= 1;
    }
  }
};

// ---------------------------------------------------------------- many rows
constexpr int W_THREADS = 320;           // TMA, MMA and eight epilogue warps
constexpr int W_EPI = 8;
constexpr int W_STAGES = 6;
constexpr int W_STAGE = 32 * 1024;       // 128 rows of x, 128 columns of W
constexpr int W_COLS = 256;              // accumulator columns
constexpr int W_OUT = 4096;              // a warp's store tile: 32 rows x 128 bytes
constexpr int W_SMEM = W_STAGES * W_STAGE + W_EPI * W_OUT + 1024;
constexpr int W_GROUP = 8;               // row tiles whose pairs share W columns in L2

struct WideCtrl {
  uint64_t full[W_STAGES];               // both CTAs' loads; used in the even CTA
  uint64_t empty[W_STAGES];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];                 // both CTAs' epilogues; used in the even CTA
  uint64_t drained;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void tile_at(int t, int mt, int nt, int& m, int& n) {
  const int width = W_GROUP * nt;
  const int g = t / width, r = t - g * width;
  const int rows = min(mt - g * W_GROUP, W_GROUP);
  n = r / rows;
  m = g * W_GROUP + (r - n * rows);
}

template <bool kGate>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(W_THREADS, 1)
    wide_kernel(const __grid_constant__ CUtensorMap tmap_x,
                const __grid_constant__ CUtensorMap tmap_w,
                const __grid_constant__ CUtensorMap tmap_g,
                const __grid_constant__ CUtensorMap tmap_y, const LinearArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ WideCtrl ctrl;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  constexpr int OUT_COLS = kGate ? 128 : 256;
  const int mt = (a.rows + 255) / 256, nt = (a.n_out + OUT_COLS - 1) / OUT_COLS;
  const int tiles = mt * nt, pairs = gridDim.x / 2;
  const int nkb = (a.n_in + BK - 1) / BK;
  if (tid == 0) {
    for (int s = 0; s < W_STAGES; ++s) {
      ptx::mbar_init(&ctrl.full[s], 1);
      ptx::mbar_init(&ctrl.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&ctrl.acc_full[b], 1);
      ptx::mbar_init(&ctrl.acc_empty[b], 2 * W_EPI);
    }
    ptx::mbar_init(&ctrl.drained, 1);
    ctrl.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(&ctrl.tmem_base, 2 * W_COLS);
    ptx::tmem_relinquish_pair();
  }
  ptx::wait_primary();
  ptx::launch_dependents();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync_warps();                   // both CTAs' barriers exist
  ptx::tc_fence_after();
  const uint32_t tmem = ctrl.tmem_base;

  if (warp == 0) {
    if (ptx::elect_one()) {
      const CUtensorMap* tw = kGate && rank == 1 ? &tmap_g : &tmap_w;
      const uint32_t full0 = ptx::mapa_shared(ptx::smem_u32(&ctrl.full[0]), 0);
      const uint32_t ring = ptx::smem_u32(smem);
      int it = 0;
      Ring at;
      bool ok = true;
      for (int t = blockIdx.x / 2; t < tiles && ok; t += pairs) {
        int m, n;
        tile_at(t, mt, nt, m, n);
        const int row = m * 256 + (int)rank * 128;
        const int col = kGate ? n * 128 : n * 256 + (int)rank * 128;
        for (int k = 0; k < nkb * BK; k += BK, ++it, at.next(W_STAGES)) {
          if (it >= W_STAGES && !lin_wait(&ctrl.abort, &ctrl.empty[at.s], at.parity ^ 1, a)) {
            ok = false;
            break;
          }
          const uint32_t st = ring + at.s * W_STAGE, bar = full0 + at.s * 8;
          if (rank == 0) expect(&ctrl.full[at.s], 2 * W_STAGE, it == 0, a);
          ptx::tma_load_2d_pair(st, &tmap_x, k, row, bar);
          ptx::tma_load_2d_pair(st + 16384, tw, col, k, bar);
          ptx::tma_load_2d_pair(st + 16384 + BOX, tw, col + 64, k, bar);
        }
      }
      // the last copies of both CTAs have landed before either exits, also
      // after a timeout
      if (rank == 0)
        for (int i = it > W_STAGES ? it - W_STAGES : 0; i < it; ++i)
          wait_for(&ctrl.full[i % W_STAGES], (i / W_STAGES) & 1, a);
    }
  } else if (warp == 1) {
    if (rank == 0 && ptx::elect_one()) {
      constexpr uint32_t idesc = ptx::idesc_bf16_f32(256, W_COLS, false, true);
      // x: K-major rows of 128 bytes, 8-row groups 1024 bytes apart; W:
      // N-major, 64-column boxes 8 KB apart, 16 K rows = 2 KB
      const uint64_t xh = ptx::smem_desc_sw128(0, 16, 1024), wh = ptx::smem_desc_sw128(0, BOX, 1024);
      const uint32_t ring = ptx::smem_u32(smem);
      int i = 0;
      Ring at;
      bool ok = true;
      for (int t = blockIdx.x / 2; t < tiles && ok; t += pairs, ++i) {
        const int b = i & 1;
        if (i >= 2 && !lin_wait(&ctrl.abort, &ctrl.acc_empty[b], ((i >> 1) - 1) & 1, a)) break;
        ptx::tc_fence_after();
        const uint32_t acc = tmem + b * W_COLS;
        for (int kb = 0; kb < nkb; ++kb, at.next(W_STAGES)) {
          if (!lin_wait(&ctrl.abort, &ctrl.full[at.s], at.parity, a)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t st = ring + at.s * W_STAGE;
          const uint64_t xd = ptx::desc_at(xh, st), wd = ptx::desc_at(wh, st + 16384);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            ptx::umma_f16_pair(acc, xd + kk * 2, wd + kk * 128, idesc, (kb | kk) != 0 ? 1u : 0u);
          ptx::umma_commit_pair(&ctrl.empty[at.s]);
        }
        if (ok) ptx::umma_commit_pair(&ctrl.acc_full[b]);
      }
      // no product is in flight when TMEM is freed
      ptx::umma_commit_pair(&ctrl.drained);
      wait_for(&ctrl.drained, 0, a);
    }
  } else {
    // a warp: 32 rows (its TMEM lane quadrant) x half of the columns
    const int quad = warp & 3, half = (warp - 2) >> 2;
    uint8_t* out = smem + W_STAGES * W_STAGE + (warp - 2) * W_OUT;
    const uint32_t out_u = ptx::smem_u32(out);
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    int i = 0;
    for (int t = blockIdx.x / 2; t < tiles; t += pairs, ++i) {
      const int b = i & 1;
      int m, n;
      tile_at(t, mt, nt, m, n);
      const int row0 = m * 256 + (int)rank * 128 + quad * 32;
      // The residual comes a round ahead, by rows, four lanes a row, and changes
      // lanes where the output will lie (1001 rows, 1304 -> 2696: 16.0 us; 16.8 in
      // the round that needs it, 16.9 with a lane for a row).
      uint4 res[4];
      auto bring = [&](int c) {
        const int col = n * OUT_COLS + half * (OUT_COLS / 2) + c + (lane & 3) * 8;
        const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(a.residual) + col;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = row0 + q * 8 + (lane >> 2);
          res[q] = make_uint4(0u, 0u, 0u, 0u);
          if (r < a.rows && col < a.n_out) res[q] = *reinterpret_cast<const uint4*>(p + r * a.ldr);
        }
      };
      if (a.residual) bring(0);
      if (!__all_sync(0xffffffffu, lin_wait(&ctrl.abort, &ctrl.acc_full[b], (i >> 1) & 1, a)))
        break;
      ptx::tc_fence_after();
      const uint32_t acc = tmem + b * W_COLS + lane_base + half * (OUT_COLS / 2);
#pragma unroll 1
      for (int c = 0; c < OUT_COLS / 2; c += 32) {
        const int col = n * OUT_COLS + half * (OUT_COLS / 2) + c;
        // the store tile: 128-byte rows, 16-byte chunks swizzled by the row; a
        // bf16 row takes the columns of two rounds
        const bool second = !a.out_f32 && (c & 32);
        auto chunk = [&](int r, int q) {
          return reinterpret_cast<uint4*>(out + r * 128 + (((q + (second ? 4 : 0)) ^ (r & 7)) * 16));
        };
        float v[32], g[kGate ? 32 : 1];
        ptx::tmem_ld32(acc + c, v);
        if constexpr (kGate) ptx::tmem_ld32(acc + 128 + c, g);
        ptx::tmem_ld_wait();
        if (c + 32 == OUT_COLS / 2) {    // the accumulator is in registers: the next tile's
          ptx::tc_fence_before();        // products may overwrite it
          __syncwarp();
          if (lane == 0)
            ptx::mbar_arrive_remote(ptx::mapa_shared(ptx::smem_u32(&ctrl.acc_empty[b]), 0));
        }
        const int bc = min(col + lane, a.n_out - 1);
        if (a.bias) {
          const float bl = bias_at(a.bias, bc, a.bias_f32);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] += __shfl_sync(0xffffffffu, bl, e);
        }
        if constexpr (kGate) {
          if (a.bias_gate) {
            const float bg = bias_at(a.bias_gate, bc, a.bias_f32);
#pragma unroll
            for (int e = 0; e < 32; ++e) g[e] += __shfl_sync(0xffffffffu, bg, e);
          }
        }
        if constexpr (kGate) {
          activate_all<32>(g, a.act);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] *= g[e];
        } else {
          activate_all<32>(v, a.act);
        }
        if (!second) {
          if (lane == 0) ptx::tma_store_wait_read<0>();
          __syncwarp();
        }
        if (a.residual) {
#pragma unroll
          for (int q = 0; q < 4; ++q) *chunk(q * 8 + (lane >> 2), lane & 3) = res[q];
          if (c + 32 < OUT_COLS / 2) bring(c + 32);
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 w = *chunk(lane, q);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[8 * q + 2 * e] += __uint_as_float(ws[e] << 16);
              v[8 * q + 2 * e + 1] += __uint_as_float(ws[e] & 0xffff0000u);
            }
          }
          __syncwarp();                  // (an fp32 row overwrites its neighbours' chunks)
        }
        if (a.out_f32) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(out + lane * 128 + ((q ^ (lane & 7)) * 16)) =
                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *chunk(lane, q) =
                make_uint4(ptx::pack_bf16(v[8 * q], v[8 * q + 1]),
                           ptx::pack_bf16(v[8 * q + 2], v[8 * q + 3]),
                           ptx::pack_bf16(v[8 * q + 4], v[8 * q + 5]),
                           ptx::pack_bf16(v[8 * q + 6], v[8 * q + 7]));
        }
        if (a.out_f32 || second) {
          ptx::fence_async_shared();
          __syncwarp();
          const int col0 = a.out_f32 ? col : col - 32;
          if (lane == 0) {
            if (row0 < a.rows && col0 < a.n_out) ptx::tma_store_2d(&tmap_y, out_u, col0, row0);
            ptx::tma_store_commit();
          }
        }
      }
    }
    if (lane == 0) ptx::tma_store_wait_all();
  }
  ptx::tc_fence_before();
  __syncthreads();
  // the even CTA's last arrival at the odd one's barriers, behind all the others
  if (warp == 1 && rank == 1) wait_for(&ctrl.drained, 0, a);
  ptx::cluster_sync_warps();                   // the peer's loads, arrivals and products are done too
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc_pair(tmem, 2 * W_COLS);
}

// ---------------------------------------------------------------- few rows
constexpr int N_EPI = 16;                // epilogue warps: with few, the sums at the end wait on
                                         // the latency of every instruction
constexpr int N_THREADS = 32 * (2 + N_EPI);
constexpr int N_STAGES = 16;             // at most
constexpr int N_RING = 208 * 1024;
constexpr int N_SMEM = N_RING + BOX + 1024;   // an odd last box may be read past the ring

// How the columns and the depth are dealt: tiles of `width` columns (64, 128,
// 192 or 256: a box that starts off a 128-byte line reads two lines a row),
// each by a cluster of `split` CTAs.
struct NarrowPlan {
  int width, split, stages;
  int blocked;     // W's tensor map counts whole 64-column blocks
  int parts_at;    // where the ranks' sums meet: 0, the ring's place, or behind it
};

// Rows that a rank finishes: a multiple of 8 (accumulator columns are read
// eight at a time).
__host__ __device__ constexpr int narrow_share(int rows, int split) {
  return (rows + 8 * split - 1) / (8 * split) * 8;
}

// Bytes of the sums that meet in a rank.
__host__ __device__ constexpr int narrow_parts(int rows, int split, bool gate, int boxes) {
  return split * narrow_share(rows, split) * 512 * (gate ? 2 : 1) * ((boxes + 1) / 2);
}

// Bytes of a stage: `boxes` 64-column boxes of W (and of Wg), N rows of x.
__host__ __device__ constexpr int narrow_stage(int boxes, bool gate, int n) {
  return boxes * BOX * (gate ? 2 : 1) + n * BK * 2;
}

struct NarrowCtrl {
  uint64_t full[N_STAGES];
  uint64_t empty[N_STAGES];
  uint64_t done;
  uint32_t tmem_base;
  int abort;
};

// (Results after a wait that gave up are wrong, and reported as such.)
template <bool kGate, int N>
__global__ void __launch_bounds__(N_THREADS, 1)
    narrow_kernel(const __grid_constant__ CUtensorMap tmap_x,
                  const __grid_constant__ CUtensorMap tmap_w,
                  const __grid_constant__ CUtensorMap tmap_g, const LinearArgs a,
                  const NarrowPlan plan) {
  constexpr int P = kGate ? 2 : 1;
  constexpr int COLS = 2 * P * N < 32 ? 32 : 2 * P * N;   // two blocks of 128 columns of W
  extern __shared__ uint8_t smem_raw[];
  __shared__ NarrowCtrl ctrl;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = plan.split, stages = plan.stages;
  const int rank = blockIdx.x % split, n0 = blockIdx.x / split * plan.width, m0 = blockIdx.y * N;
  const int width = min(plan.width, a.n_out - n0);
  const int boxes = plan.blocked ? plan.width / 64 : (width + 63) / 64, blocks = (boxes + 1) / 2;
  const int stage_bytes = narrow_stage(plan.width / 64, kGate, N);
  const int g_at = boxes * BOX, x_at = g_at * P;
  const int rows = min(N, a.rows - m0);
  const int nkb_all = (a.n_in + BK - 1) / BK;
  const int kb0 = nkb_all * rank / split, nkb = nkb_all * (rank + 1) / split - kb0;
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(&ctrl.full[s], 1);
      ptx::mbar_init(&ctrl.empty[s], 1);
    }
    ptx::mbar_init(&ctrl.done, 1);
    ctrl.abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmap_w);
    if (kGate) ptx::prefetch_tmap(&tmap_g);
    ptx::prefetch_tmap(&tmap_x);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&ctrl.tmem_base, COLS);
    ptx::tmem_relinquish();
  }
  if (plan.parts_at) ptx::cluster_arrive_warps();   // this CTA runs: others may write to it
  ptx::wait_primary();
  ptx::launch_dependents();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ctrl.tmem_base;

  if (warp == 0) {
    if (ptx::elect_one()) {
      const uint32_t ring = ptx::smem_u32(smem);
      const uint32_t bytes = x_at + N * BK * 2;
      int issued = 0, k = kb0 * BK;
      Ring at;
      for (; issued < nkb; ++issued, k += BK, at.next(stages)) {
        if (issued >= stages && !lin_wait(&ctrl.abort, &ctrl.empty[at.s], at.parity ^ 1, a))
          break;
        uint64_t* bar = &ctrl.full[at.s];
        const uint32_t st = ring + at.s * stage_bytes;
        expect(bar, bytes, issued == 0, a);
        if (plan.blocked) {              // all boxes of a matrix in one copy
          ptx::tma_load_3d_at(st, &tmap_w, 0, k, n0 >> 6, bar);
          if (kGate) ptx::tma_load_3d_at(st + g_at, &tmap_g, 0, k, n0 >> 6, bar);
        } else {
          for (int j = 0; j < boxes; ++j) {
            ptx::tma_load_2d_at(st + j * BOX, &tmap_w, n0 + 64 * j, k, bar);
            if (kGate) ptx::tma_load_2d_at(st + g_at + j * BOX, &tmap_g, n0 + 64 * j, k, bar);
          }
        }
        ptx::tma_load_2d_at(st + x_at, &tmap_x, k, m0, bar);
      }
      // every copy has landed before the ring is reused, also after a timeout
      for (int kb = issued > stages ? issued - stages : 0; kb < issued; ++kb)
        wait_for(&ctrl.full[kb % stages], (kb / stages) & 1, a);
    }
  } else if (warp == 1) {
    if (ptx::elect_one()) {
      constexpr uint32_t idesc = ptx::idesc_bf16_f32(128, N, true, false);
      const uint64_t xh = ptx::smem_desc_sw128(0, 16, 1024), wh = ptx::smem_desc_sw128(0, BOX, 1024);
      const uint32_t ring = ptx::smem_u32(smem);
      Ring at;
      for (int kb = 0; kb < nkb; ++kb, at.next(stages)) {
        if (!lin_wait(&ctrl.abort, &ctrl.full[at.s], at.parity, a)) break;
        ptx::tc_fence_after();
        const uint32_t st = ring + at.s * stage_bytes;
        const uint64_t xd = ptx::desc_at(xh, st + x_at), wd = ptx::desc_at(wh, st);
        const uint64_t gd = ptx::desc_at(wh, st + g_at);
        // a block of an odd number of boxes reads 64 columns that belong to
        // something else: they end in accumulator rows that nothing reads
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
          const uint32_t acc = (kb | kk) != 0 ? 1u : 0u;
          ptx::umma_f16_ss(tmem, wd + kk * 128, xd + kk * 2, idesc, acc);
          if (kGate) ptx::umma_f16_ss(tmem + N, gd + kk * 128, xd + kk * 2, idesc, acc);
        }
        if (blocks > 1) {
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint32_t acc = (kb | kk) != 0 ? 1u : 0u;
            ptx::umma_f16_ss(tmem + P * N, wd + kk * 128 + 2 * BOX / 16, xd + kk * 2, idesc, acc);
            if (kGate)
              ptx::umma_f16_ss(tmem + P * N + N, gd + kk * 128 + 2 * BOX / 16, xd + kk * 2, idesc,
                               acc);
          }
        }
        ptx::umma_commit(&ctrl.empty[at.s]);
      }
      ptx::umma_commit(&ctrl.done);
      wait_for(&ctrl.done, 0, a);   // no product is in flight when TMEM is freed
    }
  } else {
    if (a.residual) {                    // this rank's rows are on the way when they are needed
      const int r0 = rank * narrow_share(rows, split);
      const int lines = (width + 63) / 64;
      for (int i = tid - 64; i < min(rows - r0, narrow_share(rows, split)) * lines; i += 32 * N_EPI)
        ptx::prefetch_l2(reinterpret_cast<const __nv_bfloat16*>(a.residual) +
                         (int64_t)(m0 + r0 + i / lines) * a.ldr + n0 + i % lines * 64);
    }
    lin_wait(&ctrl.abort, &ctrl.done, 0, a);
    __syncwarp();
    ptx::tc_fence_after();
  }

  // Rank r finishes the rows [r share, (r + 1) share): every rank writes its
  // part of them into that rank's memory, [source rank][product][row][column]:
  // behind the ring when it is small, else over it, when all are done with theirs.
  // Then all warps add the parts up in the order of the ranks, two columns a
  // lane. The loops stay rolled: this runs once a CTA, so unrolled
  // instructions would be fetched for nothing.
  const int share = narrow_share(rows, split);
  const int ld = blocks * 128;
  if (plan.parts_at) ptx::cluster_wait_warps();
  else if (split > 1) ptx::cluster_sync_warps();   // every rank's ring is idle
  const uint32_t parts = ptx::smem_u32(smem) + plan.parts_at;
  if (warp >= 2) {
    const int quad = warp & 3, c = quad * 32 + lane;
    const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16);
    const int groups = (rows + 15) / 16;
#pragma unroll 1
    for (int i = (warp - 2) >> 2; i < blocks * P * groups; i += N_EPI / 4) {
      const int bp = i / groups, r = (i - bp * groups) * 16;
      float v[16];
      ptx::tmem_ld16(taddr + bp * N + r, v);
      ptx::tmem_ld_wait();
#pragma unroll
      for (int h = 0; h < 16; h += 8) {
        const int to = min((r + h) / share, split - 1);
        const uint32_t at =
            ptx::mapa_shared(parts, to) +
            (((rank * P + bp % P) * share + r + h - to * share) * ld + bp / P * 128 + c) * 4;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (r + h + e < rows) ptx::st_cluster_f32(at + e * ld * 4, v[h + e]);
      }
    }
  }
  if (split > 1) ptx::cluster_sync_warps();    // every part has arrived
  else __syncthreads();
  {
    constexpr int U = 4;                 // a row's pieces of 64 columns
    const int r0 = rank * share, mine = min(rows, r0 + share) - r0;
    const int n = n0 + lane * 2;
    const uint32_t product = share * ld * 4, part = P * product;
#pragma unroll 1
    for (int r = warp; r < mine; r += 2 + N_EPI) {
      const int64_t row = m0 + r0 + r;
      uint32_t at = parts + (r * ld + lane * 2) * 4;
      float v[P][2 * U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = u * 64 + lane * 2 < width;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const void* bias = p ? a.bias_gate : a.bias;
          v[p][2 * u] = bias && in ? bias_at(bias, n + u * 64, a.bias_f32) : 0.f;
          v[p][2 * u + 1] = bias && in ? bias_at(bias, n + u * 64 + 1, a.bias_f32) : 0.f;
        }
      }
#pragma unroll 1
      for (int src = 0; src < split; ++src, at += part)
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u * 64 < width) {
#pragma unroll
            for (int p = 0; p < P; ++p) {
              const float2 t = ptx::ld_shared_f32x2(at + p * product + u * 256);
              v[p][2 * u] += t.x;
              v[p][2 * u + 1] += t.y;
            }
          }
      activate_all<2 * U>(v[P - 1], a.act);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u * 64 + lane * 2 < width) {
          float2 y = make_float2(v[P - 1][2 * u], v[P - 1][2 * u + 1]);
          if (kGate) {
            y.x *= v[0][2 * u];
            y.y *= v[0][2 * u + 1];
          }
          if (a.residual) {
            const float2 t = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(
                reinterpret_cast<const __nv_bfloat16*>(a.residual) + row * a.ldr + n + u * 64));
            y.x += t.x;
            y.y += t.y;
          }
          if (a.out_f32)
            *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.y) + row * a.ldy + n + u * 64) = y;
          else
            *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(a.y) +
                                               row * a.ldy + n + u * 64) =
                __floats2bfloat162_rn(y.x, y.y);
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, COLS);
}

// ---------------------------------------------------------------- host
// A row-major matrix [rows][cols] with row stride ld, in boxes of box_rows
// rows and 128 bytes (128-byte swizzle); zeros outside.
bool encode(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, int64_t ld,
            uint32_t box_rows, bool f32 = false) {
  EncodeTiledFn fn = get_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * (f32 ? 4 : 2)};
  cuuint32_t box[2] = {f32 ? 32u : 64u, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// W in 3 dimensions (column of a 64-column block, K row, block), in boxes of
// BK rows of `blocks` blocks; the blocks of a box lie 8 KB apart.
bool encode_blocks(CUtensorMap* map, const void* base, uint64_t n_in, uint64_t n_out,
                   uint32_t blocks) {
  EncodeTiledFn fn = get_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {64, n_in, n_out / 64};
  cuuint64_t strides[2] = {n_out * 2, 128};
  cuuint32_t box[3] = {64, BK, blocks};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Call {
  const LinearArgs& a;
  const void* x;
  int64_t ldx;
  const void* w;
  const void* w_gate;
  int sms;
  cudaStream_t stream;
};

template <bool kGate>
cudaError_t launch_wide(const Call& c) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(wide_kernel<kGate>), W_SMEM, done);
  if (e != cudaSuccess) return e;
  const LinearArgs& a = c.a;
  CUtensorMap tx, tw, tg, ty;
  if (!encode(&tx, c.x, a.rows, a.n_in, c.ldx, 128) ||
      !encode(&tw, c.w, a.n_in, a.n_out, a.n_out, BK) ||
      !encode(&tg, kGate ? c.w_gate : c.w, a.n_in, a.n_out, a.n_out, BK) ||
      !encode(&ty, a.y, a.rows, a.n_out, a.ldy, 32, a.out_f32))
    return cudaErrorInvalidValue;
  const long long tiles =
      (long long)((a.rows + 255) / 256) * ((a.n_out + (kGate ? 127 : 255)) / (kGate ? 128 : 256));
  const int pairs = (int)(tiles < c.sms / 2 ? tiles : c.sms / 2);
  return launch_early(wide_kernel<kGate>, dim3(2 * pairs), W_THREADS, W_SMEM, 1, c.stream, tx, tw, tg,
                      ty, a);
}

// Clusters of `split` CTAs (one CTA an SM) that are resident at once: a
// cluster stays inside a group of SMs, so large ones leave some SMs over.
int clusters_at_once(int split, int sms) {
  return split == 1 ? sms : split == 2 ? sms / 2 : split == 4 ? sms * 33 / 148 : sms * 15 / 148;
}

// The plan of the least modelled time for row tiles of N, and that time in
// us. A CTA's stage costs its products (39 cycles an instruction up to 64 rows,
// 64 for 128, at 1.9 GHz) or its bytes; the epilogue 8 us for 128 x
// 128 outputs; another round of CTAs 12 us. The constants order the plans
// rather than predict them: over 78 shapes (1 to 4096 rows, depths of 512 to
// 12288) measured with every plan, the chosen one took 1.7 % longer than the
// best on average, 17 % at most.
NarrowPlan plan_narrow(const LinearArgs& a, bool gate, int N, int sms, double& best_us) {
  const int mt = (a.rows + N - 1) / N, nkb = (a.n_in + BK - 1) / BK;
  const int rows = a.rows < N ? a.rows : N, P = gate ? 2 : 1;
  const double product = (N == 128 ? 64 : 39) * 4 * P / 1900.0;
  NarrowPlan best = {256, 1, 0, 0, 0};
  best_us = 1e30;
  for (int split = 1; split <= 8; split *= 2) {
    if (split > 1 && nkb < 2 * split) break;
    const int at_once = clusters_at_once(split, sms);
    if (at_once < 1) break;
    for (int boxes = 1; boxes <= 4; ++boxes) {
      const int width = 64 * boxes, blocks = (boxes + 1) / 2;
      if (narrow_parts(rows, split, gate, boxes) > N_RING) continue;
      const long long clusters = (long long)((a.n_out + width - 1) / width) * mt;
      const double waves = (double)((clusters + at_once - 1) / at_once);
      const double bytes = narrow_stage(boxes, gate, N) / 250e3;
      const double stage = blocks * product > bytes ? blocks * product : bytes;
      const double us = 4.5 + (waves - 1) * 12.0 + waves * ((nkb + split - 1) / split) * stage +
                        7.9 / 128 * rows * blocks * P / split;
      if (us < best_us) {
        best_us = us;
        best.width = width;
        best.split = split;
      }
    }
  }
  const int stage = narrow_stage(best.width / 64, gate, N);
  // up to 32 KB of parts have a place of their own: no wait for the other ranks
  // before they are written (one row, 1024 -> 1024: 4.1 us instead of 4.6; 12 rows,
  // 8192 -> 1024: 8.0 instead of 9.2)
  const int parts = narrow_parts(rows, best.split, gate, best.width / 64);
  const int room = best.split > 1 && parts <= 32 * 1024 ? N_RING - parts : N_RING;
  best.stages = room / stage < N_STAGES ? room / stage : N_STAGES;
  if (room < N_RING) best.parts_at = best.stages * stage;
  return best;
}

// The same for the kernel for many rows.
double wide_us(const LinearArgs& a, bool gate, int sms) {
  const int cols = gate ? 128 : 256, pairs = sms / 2;
  const long long tiles = (long long)((a.rows + 255) / 256) * ((a.n_out + cols - 1) / cols);
  return 7.0 + (double)((tiles + pairs - 1) / pairs) * ((a.n_in + BK - 1) / BK * 0.29 + 1.0);
}

template <bool kGate, int N>
cudaError_t launch_narrow(const Call& c, NarrowPlan plan) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(narrow_kernel<kGate, N>), N_SMEM, done);
  if (e != cudaSuccess) return e;
  const LinearArgs& a = c.a;
  // whole blocks only: the last tile's boxes may lie past the last block, but
  // not a block past the end of W
  plan.blocked = a.n_out % 64 == 0;
  CUtensorMap tx, tw, tg;
  const uint32_t boxes = (uint32_t)plan.width / 64;
  auto encode_w = [&](CUtensorMap* map, const void* w) {
    return plan.blocked ? encode_blocks(map, w, a.n_in, a.n_out, boxes)
                        : encode(map, w, a.n_in, a.n_out, a.n_out, BK);
  };
  if (!encode(&tx, c.x, a.rows, a.n_in, c.ldx, N) || !encode_w(&tw, c.w) ||
      (kGate && !encode_w(&tg, c.w_gate)))
    return cudaErrorInvalidValue;
  const dim3 grid((unsigned)((a.n_out + plan.width - 1) / plan.width * plan.split),
                  (unsigned)((a.rows + N - 1) / N));
  return launch_early(narrow_kernel<kGate, N>, grid, N_THREADS, N_SMEM, plan.split, c.stream, tx, tw,
                      kGate ? tg : tw, a, plan);
}

// Up to 64 rows only the row tile that holds them. Beyond, tiles of 64 or 128
// rows give few outputs to more SMs than the pairs' tiles do (300 rows, 4096 ->
// 1024: 11.7 us against 26.4; 512 rows, 2048 -> 2048: 12.4 against 17.6), until
// there are tiles enough (256 rows, 4096 -> 12288: 35.2 us against 29.9).
template <bool kGate>
cudaError_t launch(const Call& c) {
  const int rows = c.a.rows;
  double us, other;
  if (rows <= 16) return launch_narrow<kGate, 16>(c, plan_narrow(c.a, kGate, 16, c.sms, us));
  if (rows <= 32) return launch_narrow<kGate, 32>(c, plan_narrow(c.a, kGate, 32, c.sms, us));
  const NarrowPlan plan = plan_narrow(c.a, kGate, 64, c.sms, us);
  if (rows <= 64) return launch_narrow<kGate, 64>(c, plan);
  const double wide = wide_us(c.a, kGate, c.sms);
  const bool fits = rows <= 65535 * 64;  // row tiles are the grid's y
  if constexpr (!kGate) {                // two products of 128 rows: no room for the exchange
    const NarrowPlan plan128 = plan_narrow(c.a, kGate, 128, c.sms, other);
    if (other <= us && other <= wide && fits) return launch_narrow<kGate, 128>(c, plan128);
  }
  return us <= wide && fits ? launch_narrow<kGate, 64>(c, plan) : launch_wide<kGate>(c);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, const void* x, int64_t ldx, const void* w,
                          const void* w_gate, int sms, cudaStream_t stream) {
  const Call c{a, x, ldx, w, w_gate, sms, stream};
  return a.gated ? launch<true>(c) : launch<false>(c);
}

}  // namespace fdllm

// Declarations shared by the host side (serve_api.cu) and the kernels of the
// single-token serving operators: block planning, decode attention and the
// linear map.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include <utility>

#include "fdllm_internal.h"

namespace fdllm {

// Launch that may begin under the tail of the launch before it on the stream
// (the kernel itself waits for that one's results before it reads anything);
// cluster > 1: in clusters of so many CTAs along x.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, int smem, int cluster,
                         cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// n / d for 0 <= n < 2^31 and 1 <= d < 2^31 as a multiply and a shift
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication"): with 2^(l-1) < d <= 2^l and
// m = floor(2^32 (2^l - d) / d) + 1, n / d = (hi32(m n) + n) >> l; the sum
// stays below 2^32 because n < 2^31.
struct FastDiv {
  uint32_t d, m, l;
  static FastDiv of(uint32_t d) {
    FastDiv f{d, 0, 0};
    while ((1ull << f.l) < d) ++f.l;
    f.m = (uint32_t)(((1ull << 32) * ((1ull << f.l) - d)) / d + 1);
    return f;
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int div(int n) const {
    return (int)((__umulhi(m, (uint32_t)n) + (uint32_t)n) >> l);
  }
#endif
};

// Bound of the kernels' waits, in cycles of the SM clock: about a second.
constexpr long long kWaitCycles = 2000000000ll;

// ---------------------------------------------------------------- block planning
constexpr int kMaxPlanBatch = 16384;   // 12 bytes of shared memory per request

struct PlanArgs {
  const int32_t* seq_lens;
  const int32_t* new_lens;    // plan: new tokens; release: tokens kept
  int32_t* table;
  int32_t* free_pages;        // plan: read; release: written
  const int32_t* n_free;
  int batch, max_blocks, num_pages, capacity;
  FastDiv ps;
  int32_t* cu_rows;
  int32_t* positions;
  int32_t* slots;
  int64_t* slot_map;
  int32_t* row_seq;
  int32_t* seq_lens_out;
  int32_t* granted;
  int32_t* n_free_out;
  int32_t* headroom;          // null: not wanted
  int32_t* seq_positions;     // and these
  int32_t* seq_slots;
  int32_t* status;
  int vec;                    // the row outputs are 16-byte aligned
};

cudaError_t launch_plan_blocks(const PlanArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_release_blocks(const PlanArgs& a, int sms, cudaStream_t stream);

// ---------------------------------------------------------------- decode attention
constexpr int kDecodeHeads = 8;        // query heads of one key head that a work unit carries

struct DecodeArgs {
  const void* q;
  const void* k;              // null: nothing is written to the cache
  const void* v;
  const int32_t* positions;   // null without RoPE and with slots
  const int32_t* slots;       // null: slot = position
  const double* rope_cos;     // null: no rotation
  const double* rope_sin;
  void* k_pool;               // already at the layer's slice
  void* v_pool;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* starts;      // null: 0
  void* out;
  float* lse;                 // null: not wanted
  float* part;                // workspace
  unsigned long long* begun;  // behind the parts (see kBegun)
  int32_t* status;
  long long wait_cycles;      // bound of a wait
  int withhold;               // the first tile of every CTA is not said to be there (for tests)
  int batch, n_heads, n_kv_heads, group, head_chunks, units_per_seq;
  int max_blocks, num_pages, max_position, in_f32, out_bf16;
  FastDiv ps;
  float scale;
  int64_t q_stride, k_stride, v_stride;   // elements
  int resident;               // CTAs of the attention grid that run at once
  int ctas;                   // CTAs of the grid: an upper bound of the shares of work
  FastDiv resident_div, ctas_div;
  int unit_heads;             // query heads of a unit, at most
  int kv_at;                  // where the new row's k and v lie behind a unit's q, bytes; 0: no
                              // room for them
  int rope_at;                // where the cosines and sines lie
  int slot_bytes;             // all of them
  int box;                    // quarters of a tile in one load
};

// CTAs of the attention grid at most, and the workspace that their partial
// results take.
int decode_ctas(int sms);
size_t decode_workspace_bytes(int group, int head_dim, int sms);
cudaError_t launch_decode_attention(const DecodeArgs& a, int head_dim, bool f32, int sms,
                                    cudaStream_t stream);

// ---------------------------------------------------------------- linear
struct LinearArgs {
  const void* bias;
  const void* bias_gate;
  const void* residual;       // bf16
  void* y;
  int32_t* status;
  int rows, n_in, n_out;
  int act, gated, bias_f32, out_f32;
  int64_t ldr, ldy;           // elements
  int withhold;               // the first stage of every CTA is not said to be there (for tests)
  long long wait_cycles;      // bound of a wait
};

cudaError_t launch_linear(const LinearArgs& a, const void* x, int64_t ldx, const void* w,
                          const void* w_gate, int sms, cudaStream_t stream);

}  // namespace fdllm

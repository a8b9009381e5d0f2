// Host side of the single-token serving operators declared in
// include/fdllm.h: argument checks and launches. No call here allocates,
// synchronises or throws.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fdllm.h"
#include "host_api.h"
#include "serve_internal.h"

using namespace fdllm;

namespace {

struct Span {
  uintptr_t b, e;
  Span(const void* p, uint64_t bytes)
      : b(reinterpret_cast<uintptr_t>(p)), e(b + (p ? (uintptr_t)bytes : 0)) {}
  bool meets(const Span& o) const { return b < o.e && o.b < e; }
};

template <int N, int M>
bool any_meet(const Span (&outs)[N], const Span (&ins)[M]) {
  for (int i = 0; i < N; ++i) {
    for (int j = 0; j < M; ++j)
      if (outs[i].meets(ins[j])) return true;
    for (int j = i + 1; j < N; ++j)
      if (outs[i].meets(outs[j])) return true;
  }
  return false;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool is_dtype(int32_t d) { return d == FDLLM_BF16 || d == FDLLM_F32; }
uint64_t size_of(int32_t d) { return d == FDLLM_F32 ? 4 : 2; }

// Set by fdllm_inject_tile_timeout for this thread's next call: the bound of the
// waits in ns, 0: nothing.
thread_local int64_t g_inject_wait_ns = 0;

template <typename Args>
void bound_waits(Args& a) {
  a.withhold = g_inject_wait_ns > 0;
  a.wait_cycles = g_inject_wait_ns > 0 ? 2 * g_inject_wait_ns : kWaitCycles;
  g_inject_wait_ns = 0;
}

int sms_here() {
  const int n = sm_count();
  return n > 0 ? n : 148;
}

// The sizes that fdllm_plan_blocks and fdllm_release_blocks share.
fdllm_status check_plan(const char* what, int32_t batch, int32_t mb, int32_t ps, int32_t np) {
  if (batch <= 0 || mb <= 0 || ps <= 0 || np <= 0)
    return fail(FDLLM_ERR_INVALID_ARG, "%s: sizes must be positive", what);
  if (batch > kMaxPlanBatch)
    return fail(FDLLM_ERR_UNSUPPORTED, "%s: batch %d > %d", what, batch, kMaxPlanBatch);
  const int64_t blocks = (int64_t)batch * mb + 1;
  if (blocks >= (1ll << 31) || blocks * ps >= (1ll << 31) || (int64_t)np * ps >= (1ll << 31))
    return fail(FDLLM_ERR_UNSUPPORTED, "%s: 2^31 or more slots", what);
  return FDLLM_OK;
}

}  // namespace

extern "C" {

fdllm_status fdllm_plan_blocks(int32_t batch, int32_t max_blocks, int32_t page_size,
                               int32_t num_pages, int32_t capacity, const int32_t* seq_lens,
                               const int32_t* new_lens, int32_t* block_table,
                               const int32_t* free_pages, const int32_t* n_free, int32_t* cu_rows,
                               int32_t* positions, int32_t* slots, int32_t* row_seq,
                               int64_t* slot_map, int32_t* seq_lens_out, int32_t* granted,
                               int32_t* n_free_out, int32_t* headroom, int32_t* status, void* stream) {
  return fdllm_plan_step(batch, max_blocks, page_size, num_pages, capacity, seq_lens, new_lens,
                         block_table, free_pages, n_free, cu_rows, positions, slots, row_seq,
                         slot_map, seq_lens_out, granted, n_free_out, headroom, nullptr, nullptr,
                         status, stream);
}

fdllm_status fdllm_plan_step(int32_t batch, int32_t max_blocks, int32_t page_size,
                             int32_t num_pages, int32_t capacity, const int32_t* seq_lens,
                             const int32_t* new_lens, int32_t* block_table,
                             const int32_t* free_pages, const int32_t* n_free, int32_t* cu_rows,
                             int32_t* positions, int32_t* slots, int32_t* row_seq,
                             int64_t* slot_map, int32_t* seq_lens_out, int32_t* granted,
                             int32_t* n_free_out, int32_t* headroom, int32_t* seq_positions,
                             int32_t* seq_slots, int32_t* status, void* stream) {
  NvtxRange nvtx_range("fdllm_plan_blocks");
  fdllm_status st = check_plan("plan_blocks", batch, max_blocks, page_size, num_pages);
  if (st != FDLLM_OK) return st;
  if (capacity < 0) return fail(FDLLM_ERR_INVALID_ARG, "plan_blocks: negative capacity");
  if (capacity > (1 << 30))
    return fail(FDLLM_ERR_UNSUPPORTED, "plan_blocks: capacity %d > 2^30", capacity);
  if (!seq_lens || !new_lens || !block_table || !free_pages || !n_free || !cu_rows ||
      !seq_lens_out || !granted || !n_free_out ||
      (capacity > 0 && (!positions || !slots || !row_seq || !slot_map)))
    return fail(FDLLM_ERR_INVALID_ARG, "plan_blocks: null pointer");
  const uint64_t nb = (uint64_t)batch * 4, nc = (uint64_t)capacity * 4;
  const Span outs[] = {{block_table, nb * max_blocks}, {cu_rows, nb + 4}, {positions, nc},
                       {slots, nc}, {row_seq, nc}, {slot_map, 2 * nc}, {seq_lens_out, nb},
                       {granted, nb}, {n_free_out, 4}, {headroom, 4}, {seq_positions, nb},
                       {seq_slots, nb}};
  const Span ins[] = {{seq_lens, nb}, {new_lens, nb}, {free_pages, (uint64_t)num_pages * 4},
                      {n_free, 4}, {status, 4}};
  for (const Span& s : outs)
    if (s.b & 3) return fail(FDLLM_ERR_INVALID_ARG, "plan_blocks: misaligned pointer");
  for (const Span& s : ins)
    if (s.b & 3) return fail(FDLLM_ERR_INVALID_ARG, "plan_blocks: misaligned pointer");
  if (!aligned(slot_map, 8)) return fail(FDLLM_ERR_INVALID_ARG, "plan_blocks: misaligned slot_map");
  if (any_meet(outs, ins))
    return fail(FDLLM_ERR_INVALID_ARG, "plan_blocks: an output overlaps another argument");
  PlanArgs a = {};
  a.seq_lens = seq_lens;
  a.new_lens = new_lens;
  a.table = block_table;
  a.free_pages = const_cast<int32_t*>(free_pages);
  a.n_free = n_free;
  a.batch = batch;
  a.max_blocks = max_blocks;
  a.num_pages = num_pages;
  a.capacity = capacity;
  a.ps = FastDiv::of((uint32_t)page_size);
  a.cu_rows = cu_rows;
  a.positions = positions;
  a.slots = slots;
  a.slot_map = slot_map;
  a.row_seq = row_seq;
  a.seq_lens_out = seq_lens_out;
  a.granted = granted;
  a.n_free_out = n_free_out;
  a.headroom = headroom;
  a.seq_positions = seq_positions;
  a.seq_slots = seq_slots;
  a.status = status;
  a.vec = aligned(positions, 16) && aligned(slots, 16) && aligned(row_seq, 16) &&
          aligned(slot_map, 16);
  cudaError_t e = launch_plan_blocks(a, sms_here(), reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "plan_blocks: launch");
  set_launch_count(1);
  return FDLLM_OK;
}

fdllm_status fdllm_release_blocks(int32_t batch, int32_t max_blocks, int32_t page_size,
                                  int32_t num_pages, const int32_t* seq_lens,
                                  const int32_t* keep_lens, const int32_t* block_table,
                                  int32_t* free_pages, const int32_t* n_free,
                                  int32_t* seq_lens_out, int32_t* n_free_out, int32_t* status,
                                  void* stream) {
  NvtxRange nvtx_range("fdllm_release_blocks");
  fdllm_status st = check_plan("release_blocks", batch, max_blocks, page_size, num_pages);
  if (st != FDLLM_OK) return st;
  if (!seq_lens || !keep_lens || !block_table || !free_pages || !n_free || !seq_lens_out ||
      !n_free_out)
    return fail(FDLLM_ERR_INVALID_ARG, "release_blocks: null pointer");
  const uint64_t nb = (uint64_t)batch * 4;
  const Span outs[] = {{free_pages, (uint64_t)num_pages * 4}, {seq_lens_out, nb}, {n_free_out, 4}};
  const Span ins[] = {{seq_lens, nb}, {keep_lens, nb}, {block_table, nb * max_blocks}, {n_free, 4},
                      {status, 4}};
  for (const Span& s : outs)
    if (s.b & 3) return fail(FDLLM_ERR_INVALID_ARG, "release_blocks: misaligned pointer");
  for (const Span& s : ins)
    if (s.b & 3) return fail(FDLLM_ERR_INVALID_ARG, "release_blocks: misaligned pointer");
  if (any_meet(outs, ins))
    return fail(FDLLM_ERR_INVALID_ARG, "release_blocks: an output overlaps another argument");
  PlanArgs a = {};
  a.seq_lens = seq_lens;
  a.new_lens = keep_lens;
  a.table = const_cast<int32_t*>(block_table);
  a.free_pages = free_pages;
  a.n_free = n_free;
  a.batch = batch;
  a.max_blocks = max_blocks;
  a.num_pages = num_pages;
  a.ps = FastDiv::of((uint32_t)page_size);
  a.seq_lens_out = seq_lens_out;
  a.n_free_out = n_free_out;
  a.status = status;
  cudaError_t e = launch_release_blocks(a, sms_here(), reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "release_blocks: launch");
  set_launch_count(1);
  return FDLLM_OK;
}

int64_t fdllm_decode_workspace_bytes(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim) {
  if (n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads || head_dim <= 0 || head_dim > 128 ||
      head_dim % 32)
    return -1;
  return (int64_t)decode_workspace_bytes(n_heads / n_kv_heads, head_dim, sms_here());
}

fdllm_status fdllm_decode_attention(const fdllm_decode* d, int32_t layer, const void* q,
                                    const void* k, const void* v, const int32_t* positions,
                                    const int32_t* slots, const double* rope_cos,
                                    const double* rope_sin, void* k_pool, void* v_pool,
                                    const int32_t* block_table, const int32_t* seq_lens,
                                    const int32_t* starts, void* out, float* lse, void* workspace,
                                    int64_t workspace_bytes, int32_t* status, void* stream) {
  NvtxRange nvtx_range("fdllm_decode_attention");
  if (!d) return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: null shape");
  if (d->batch <= 0 || d->n_heads <= 0 || d->n_kv_heads <= 0 || d->n_layers <= 0 ||
      d->num_pages <= 0 || d->page_size <= 0 || d->max_blocks_per_seq <= 0)
    return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: sizes must be positive");
  if (!is_dtype(d->dtype) || !is_dtype(d->in_dtype) || !is_dtype(d->out_dtype))
    return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: unknown dtype");
  if (d->head_dim <= 0 || d->head_dim > 128 || d->head_dim % 32)
    return fail(FDLLM_ERR_UNSUPPORTED, "decode_attention: head_dim %d is not 32, 64, 96 or 128",
                d->head_dim);
  if (d->n_heads % d->n_kv_heads)
    return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: n_heads %d is no multiple of n_kv_heads %d",
                d->n_heads, d->n_kv_heads);
  if (layer < 0 || layer >= d->n_layers)
    return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: layer %d outside [0, %d)", layer,
                d->n_layers);
  if (!(d->scale > 0.f) || !std::isfinite(d->scale))
    return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: scale must be finite and > 0");
  if ((double)d->n_layers * d->num_pages * d->n_kv_heads * d->page_size >= 2147483648.0)
    return fail(FDLLM_ERR_UNSUPPORTED, "decode_attention: pool has 2^31 or more slot rows");
  if (((int64_t)d->max_blocks_per_seq + 1) * d->page_size >= (1ll << 31))
    return fail(FDLLM_ERR_UNSUPPORTED, "decode_attention: 2^31 or more slots a sequence");
  const int group = d->n_heads / d->n_kv_heads;
  const int chunks = (group + kDecodeHeads - 1) / kDecodeHeads;
  if ((double)d->batch * d->n_heads >= 2147483648.0)
    return fail(FDLLM_ERR_UNSUPPORTED, "decode_attention: batch * heads too large");
  const int tile = d->dtype == FDLLM_F32 ? 32 : 64;
  if ((double)d->batch * d->n_kv_heads * chunks *
          ((double)d->max_blocks_per_seq * d->page_size / tile + 2) >= 2147418112.0)
    return fail(FDLLM_ERR_UNSUPPORTED, "decode_attention: 2^31 or more tiles of %d slots", tile);
  if (!q || !k_pool || !v_pool || !block_table || !seq_lens || !out || !workspace)
    return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: null pointer");
  if (!k != !v) return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: k and v go together");
  if (!rope_cos != !rope_sin)
    return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: rope_cos and rope_sin go together");
  if (rope_cos && (!positions || d->max_position <= 0))
    return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: RoPE needs positions and max_position");
  if (k && !slots && !positions)
    return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: k needs slots or positions");
  const uint64_t in = size_of(d->in_dtype);
  const int64_t hq = (int64_t)d->n_heads * d->head_dim, hk = (int64_t)d->n_kv_heads * d->head_dim;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_pool, 16) ||
      !aligned(v_pool, 16) || !aligned(out, 16) || !aligned(workspace, 16) ||
      !aligned(rope_cos, 16) || !aligned(rope_sin, 16) || !aligned(lse, 4) ||
      !aligned(positions, 4) || !aligned(slots, 4) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(starts, 4) || !aligned(status, 4))
    return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: misaligned pointer");
  if (d->batch > 1 && (d->q_stride < hq || (k && (d->k_stride < hk || d->v_stride < hk))))
    return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: a row stride is shorter than its row");
  if ((d->q_stride * in) % 16 || (k && ((d->k_stride * in) % 16 || (d->v_stride * in) % 16)))
    return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: row strides must be multiples of 16 bytes");
  const int64_t need = fdllm_decode_workspace_bytes(d->n_heads, d->n_kv_heads, d->head_dim);
  if (workspace_bytes < need)
    return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: workspace of %lld bytes, %lld needed",
                (long long)workspace_bytes, (long long)need);
  const uint64_t rows = (uint64_t)d->batch, slice = (uint64_t)d->num_pages * d->n_kv_heads *
                                                    d->page_size * d->head_dim * size_of(d->dtype);
  const uint64_t pool = slice * d->n_layers;
  {
    const Span outs[] = {{k_pool, pool}, {v_pool, pool}, {out, rows * hq * size_of(d->out_dtype)},
                         {lse, rows * d->n_heads * 4}, {workspace, (uint64_t)need}, {status, 4}};
    const Span ins[] = {{q, ((rows - 1) * d->q_stride + hq) * in},
                        {k, ((rows - 1) * d->k_stride + hk) * in},
                        {v, ((rows - 1) * d->v_stride + hk) * in},
                        {positions, rows * 4}, {slots, rows * 4}, {seq_lens, rows * 4},
                        {starts, rows * 4}, {block_table, rows * d->max_blocks_per_seq * 4},
                        {rope_cos, (uint64_t)std::max(d->max_position, 0) * d->head_dim * 4},
                        {rope_sin, (uint64_t)std::max(d->max_position, 0) * d->head_dim * 4}};
    if (any_meet(outs, ins))
      return fail(FDLLM_ERR_INVALID_ARG, "decode_attention: an output overlaps another argument");
  }
  DecodeArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.positions = positions;
  a.slots = slots;
  a.rope_cos = rope_cos;
  a.rope_sin = rope_sin;
  a.k_pool = reinterpret_cast<uint8_t*>(k_pool) + slice * layer;
  a.v_pool = reinterpret_cast<uint8_t*>(v_pool) + slice * layer;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.starts = starts;
  a.out = out;
  a.lse = lse;
  a.part = reinterpret_cast<float*>(workspace);
  a.begun = reinterpret_cast<unsigned long long*>(reinterpret_cast<uint8_t*>(workspace) + need - 16);
  a.status = status;
  a.batch = d->batch;
  a.n_heads = d->n_heads;
  a.n_kv_heads = d->n_kv_heads;
  a.group = group;
  a.head_chunks = chunks;
  a.units_per_seq = d->n_kv_heads * chunks;
  a.max_blocks = d->max_blocks_per_seq;
  a.num_pages = d->num_pages;
  a.max_position = d->max_position;
  a.in_f32 = d->in_dtype == FDLLM_F32;
  a.out_bf16 = d->out_dtype == FDLLM_BF16;
  a.ps = FastDiv::of((uint32_t)d->page_size);
  a.scale = d->scale;
  a.q_stride = d->q_stride;
  a.k_stride = d->k_stride;
  a.v_stride = d->v_stride;
  a.unit_heads = group < kDecodeHeads ? group : kDecodeHeads;
  bound_waits(a);
  cudaError_t e = launch_decode_attention(a, d->head_dim, d->dtype == FDLLM_F32, sms_here(),
                                          reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "decode_attention: launch");
  set_launch_count(2);
  return FDLLM_OK;
}

fdllm_status fdllm_inject_tile_timeout(int64_t wait_ns) {
  if (wait_ns < 0 || wait_ns > 1000000000)
    return fail(FDLLM_ERR_INVALID_ARG, "inject_tile_timeout: wait of %lld ns outside [0, 10^9]",
                (long long)wait_ns);
  g_inject_wait_ns = wait_ns;
  return FDLLM_OK;
}

fdllm_status fdllm_linear(const fdllm_linear_shape* s, const void* x, const void* w,
                          const void* bias, const void* w_gate, const void* bias_gate,
                          const void* residual, void* y, int32_t* status, void* stream) {
  NvtxRange nvtx_range("fdllm_linear");
  if (!s) return fail(FDLLM_ERR_INVALID_ARG, "linear: null shape");
  if (s->rows < 0 || s->n_in <= 0 || s->n_out <= 0)
    return fail(FDLLM_ERR_INVALID_ARG, "linear: rows >= 0, n_in > 0 and n_out > 0 required");
  if (s->n_in % 8 || s->n_out % 8)
    return fail(FDLLM_ERR_UNSUPPORTED, "linear: n_in %d and n_out %d must be multiples of 8",
                s->n_in, s->n_out);
  if (s->rows > (1 << 23) || s->n_in > (1 << 20) || s->n_out > (1 << 20))
    return fail(FDLLM_ERR_UNSUPPORTED, "linear: rows > 2^23, or n_in or n_out > 2^20");
  if (s->act < FDLLM_ACT_NONE || s->act > FDLLM_ACT_GELU_TANH)
    return fail(FDLLM_ERR_INVALID_ARG, "linear: unknown activation %d", s->act);
  if (!is_dtype(s->bias_dtype) || !is_dtype(s->out_dtype))
    return fail(FDLLM_ERR_INVALID_ARG, "linear: unknown dtype");
  if (bias_gate && !w_gate) return fail(FDLLM_ERR_INVALID_ARG, "linear: bias_gate without w_gate");
  if (s->rows == 0) {
    set_launch_count(0);
    return FDLLM_OK;
  }
  if (!x || !w || !y) return fail(FDLLM_ERR_INVALID_ARG, "linear: null pointer");
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 16) || !aligned(w_gate, 16) ||
      !aligned(bias_gate, 16) || !aligned(residual, 16) || !aligned(y, 16) || !aligned(status, 4))
    return fail(FDLLM_ERR_INVALID_ARG, "linear: pointers must be 16-byte aligned");
  const uint64_t out = size_of(s->out_dtype);
  if (s->ldx < s->n_in || s->ldy < s->n_out || (residual && s->ldr < s->n_out))
    return fail(FDLLM_ERR_INVALID_ARG, "linear: a row stride is shorter than its row");
  if (s->ldx % 8 || (s->ldy * out) % 16 || (residual && s->ldr % 8))
    return fail(FDLLM_ERR_INVALID_ARG, "linear: row strides must be multiples of 16 bytes");
  if (s->ldx >= (1ll << 32) || s->ldy >= (1ll << 32) || (residual && s->ldr >= (1ll << 32)))
    return fail(FDLLM_ERR_UNSUPPORTED, "linear: row stride of 2^32 elements or more");
  {
    const uint64_t r = (uint64_t)s->rows, wb = (uint64_t)s->n_in * s->n_out * 2;
    const uint64_t bb = (uint64_t)s->n_out * size_of(s->bias_dtype);
    const bool in_place = residual == y && residual && s->ldr == s->ldy && out == 2;
    const Span outs[] = {{y, ((r - 1) * s->ldy + s->n_out) * out}, {status, 4}};
    const Span ins[] = {{x, ((r - 1) * s->ldx + s->n_in) * 2}, {w, wb}, {w_gate, wb}, {bias, bb},
                        {bias_gate, bb},
                        {in_place ? nullptr : residual, ((r - 1) * s->ldr + s->n_out) * 2}};
    if (any_meet(outs, ins))
      return fail(FDLLM_ERR_INVALID_ARG, "linear: y overlaps another argument");
  }
  LinearArgs a = {};
  a.bias = bias;
  a.bias_gate = bias_gate;
  a.residual = residual;
  a.y = y;
  a.status = status;
  a.rows = s->rows;
  a.n_in = s->n_in;
  a.n_out = s->n_out;
  a.act = s->act;
  a.gated = w_gate != nullptr;
  a.bias_f32 = s->bias_dtype == FDLLM_F32;
  a.out_f32 = s->out_dtype == FDLLM_F32;
  a.ldr = s->ldr;
  a.ldy = s->ldy;
  bound_waits(a);
  cudaError_t e = launch_linear(a, x, s->ldx, w, w_gate, sms_here(),
                                reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "linear: launch");
  set_launch_count(1);
  return FDLLM_OK;
}

}  // extern "C"

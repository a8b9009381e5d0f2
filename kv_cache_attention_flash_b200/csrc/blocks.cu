// Block tables and slot maps from request lengths, on the GPU.
//
// "Flash-dLLM: I/O-Aware KV Caching and Parallel Decoding for Fast,
// Memory-Efficient Diffusion LLMs" (ai4snews summary), paragraph 1: a block
// table aligns the query rows of sequences in different stages with their
// pages. These kernels keep that table: they take pages from a free list for
// the tokens that a step adds, list the step's rows, and give pages back.
//
// With ps slots a page, held_b = ceil(len_b / ps) and
// need_b = ceil((len_b + new_b) / ps) - held_b, request b's pages are the
// free list's entries n_free - 1 - (before_b + j), j < need_b, where before_b
// is the sum of need over the earlier requests: a prefix sum decides every
// page, so no atomics and no order of arrival are involved. A second prefix
// sum, over new_b, places the rows.
//
// Bound: a decode step (32 requests) is launch latency; a step of long
// prompts writes 20 bytes a row. One launch: every CTA makes both sums of all
// requests for itself (8 bytes a request from L2, at most 64 requests a
// thread) and keeps them in shared memory, which costs less than a second
// launch or a wait between CTAs; then the rows and the pages are spread over
// the grid, each finding its request by bisection in shared memory. A thread
// takes four consecutive rows: one bisection and 16-byte stores, and all four
// page numbers on the way at once (a decode step's rows belong to four requests:
// 3.7 us a launch of 32 requests where one load after the other took 4.7). A
// million rows of prompts take 9.7 us, 2.2 TB/s of stores.
#include <cstdint>

#include "fdllm.h"
#include "fdllm_internal.h"
#include "ptx_serve.cuh"
#include "serve_internal.h"

namespace fdllm {
namespace {

constexpr int PT = 256;     // threads of a CTA
constexpr int ROWS = 4;     // rows of a thread

struct Request {
  int len;       // tokens held (0 where the lengths make no sense)
  int rows;      // plan: new tokens
  int held;      // pages held
  int need;      // plan: pages to take; release: pages to give back
  bool bad;
};

__device__ __forceinline__ void report(int32_t* status) {
  if (status) atomicExch(reinterpret_cast<int*>(status), (int)FDLLM_ERR_DEVICE_BOUNDS);
}

template <bool kRelease>
__device__ __forceinline__ Request request(const PlanArgs& a, int b) {
  Request r;
  const int len = a.seq_lens[b], n = a.new_lens[b];
  const int top = a.max_blocks * (int)a.ps.d;        // < 2^31: checked on the host
  r.bad = len < 0 || len > top || n < 0 || (!kRelease && n > top - len);
  r.len = r.bad ? 0 : len;
  const int m = r.bad ? 0 : n;
  r.held = a.ps.div(r.len + (int)a.ps.d - 1);
  if (kRelease) {
    r.rows = m < r.len ? m : r.len;                  // tokens kept
    r.need = r.held - a.ps.div(r.rows + (int)a.ps.d - 1);
  } else {
    r.rows = m;
    r.need = a.ps.div(r.len + m + (int)a.ps.d - 1) - r.held;
  }
  return r;
}

// Exclusive sum of v over the CTA's threads; total in `all`.
__device__ __forceinline__ long long block_scan(long long v, long long& all) {
  __shared__ long long warp_sum[PT / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  if (lane == 31) warp_sum[warp] = s;
  __syncthreads();
  long long before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < PT / 32; ++w) {
    const long long t = warp_sum[w];
    if (w < warp) before += t;
    all += t;
  }
  __syncthreads();
  return before + s - v;
}

// The last b in [0, n) with first[b] <= x (first[0] = 0 <= x): the request
// that x falls to, empty requests passed over.
__device__ __forceinline__ int find(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int free_count(const PlanArgs& a) {
  const int n = *a.n_free;
  const int m = n < 0 ? 0 : (n > a.num_pages ? a.num_pages : n);
  if (m != n && blockIdx.x == 0 && threadIdx.x == 0) report(a.status);
  return m;
}

// (Six CTAs fit an SM: the next launch's three start beside this one's; with five
// a million rows take 12.7 us instead of 9.7.)
__global__ void __launch_bounds__(PT, 6) plan_kernel(const PlanArgs a) {
  extern __shared__ int smem[];
  const int B = a.batch, tid = threadIdx.x;
  ptx::wait_primary();
  ptx::launch_dependents();
  int* cu = smem;               // [B + 1] rows before request b
  int* pages = cu + B + 1;      // [B + 1] pages taken before it
  int* lens = pages + B + 1;    // [B] its length; negative (~length): not granted
  const int n_free = free_count(a);

  // both sums: each thread a run of consecutive requests
  const int each = (B + PT - 1) / PT;
  const int b0 = min(tid * each, B), b1 = min(b0 + each, B);
  long long mine = 0;
  Request only;                 // of a thread with one request: kept
  for (int b = b0; b < b1; ++b) {
    only = request<false>(a, b);
    mine += ((long long)only.rows << 32) + only.need;
  }
  long long all;
  long long at = block_scan(mine, all);
  const int total_rows = (int)(all >> 32), total_pages = (int)(all & 0xffffffff);
  int taken = 0, asked = 0;     // pages that the granted ones of this run end at: taken, asked for
  for (int b = b0; b < b1; ++b) {
    const Request r = each == 1 ? only : request<false>(a, b);
    const int row0 = (int)(at >> 32), page0 = (int)(at & 0xffffffff);
    const bool ok = !r.bad && (r.need == 0 || page0 + r.need <= n_free);
    cu[b] = row0;
    pages[b] = page0;
    lens[b] = ok ? r.len : ~r.len;
    if (ok && r.need > 0) taken = page0 + r.need;
    if (ok) asked = page0 + r.need;
    at += ((long long)r.rows << 32) + r.need;
    if (blockIdx.x == 0) {
      a.cu_rows[b] = row0;
      a.seq_lens_out[b] = ok ? r.len + r.rows : a.seq_lens[b];
      a.granted[b] = ok ? 1 : 0;
      const bool row = ok && r.rows > 0;
      if (a.seq_positions) a.seq_positions[b] = row ? r.len + r.rows - 1 : 0;
      if (a.seq_slots) a.seq_slots[b] = row ? r.len + r.rows - 1 : -1;
      if (r.bad) report(a.status);
    }
  }
  if (tid == 0) {
    cu[B] = total_rows;
    pages[B] = total_pages;
    if (blockIdx.x == 0) {
      a.cu_rows[B] = total_rows;
      if (total_rows > a.capacity) report(a.status);
    }
  }
  if (blockIdx.x == 0) {
    __shared__ int most[2][PT / 32];
    const int m = __reduce_max_sync(0xffffffffu, taken), n = __reduce_max_sync(0xffffffffu, asked);
    if ((tid & 31) == 0) {
      most[0][tid >> 5] = m;
      most[1][tid >> 5] = n;
    }
    __syncthreads();
    if (tid == 0) {
      int t = 0, u = 0;
      for (int w = 0; w < PT / 32; ++w) {
        t = max(t, most[0][w]);
        u = max(u, most[1][w]);
      }
      *a.n_free_out = n_free - t;
      if (a.headroom) *a.headroom = n_free - u;
    }
  }
  __syncthreads();

  // the new entries of the table, by the last threads first: the first ones have
  // the rows to do
  const int step = gridDim.x * PT;
  const int n_pages = min(total_pages, n_free);
  // (page counts reach 2^31 - 2, from where a step leaves int)
  for (uint32_t at_page = step - 1 - (blockIdx.x * PT + tid); at_page < (uint32_t)n_pages; at_page += step) {
    const int p = (int)at_page, b = find(pages, B, p);
    if (lens[b] < 0) continue;
    const int id = a.free_pages[n_free - 1 - p];
    const bool ok = id >= 0 && id < a.num_pages;
    if (!ok) report(a.status);
    const int held = a.ps.div(lens[b] + (int)a.ps.d - 1);
    a.table[(int64_t)b * a.max_blocks + held + p - pages[b]] = ok ? id : -1;
  }

  // the rows; pages come from the free list, not from the table entries that
  // another CTA may be writing
  const int n_rows = min(total_rows, a.capacity);
  for (int r0 = (blockIdx.x * PT + tid) * ROWS; r0 < n_rows; r0 += step * ROWS) {
    int pos[ROWS], slot[ROWS], seq[ROWS], id[ROWS], off[ROWS];
    const int* from[ROWS];      // where the page number is, null: the row before's
    long long map[ROWS];
    int b = find(cu, B, r0);
    int last_b = -1, last_j = -1;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int r = r0 + i;
      if (r < n_rows)
        while (r >= cu[b + 1]) ++b;
      const bool ok = lens[b] >= 0 && r < n_rows;
      const int len = lens[b] >= 0 ? lens[b] : ~lens[b];
      pos[i] = len + r - cu[b];
      seq[i] = b;
      slot[i] = ok ? pos[i] : -1;
      const int j = a.ps.div(ok ? pos[i] : 0);
      off[i] = pos[i] - j * (int)a.ps.d;
      from[i] = nullptr;
      if (ok && (b != last_b || j != last_j)) {
        const int held = a.ps.div(len + (int)a.ps.d - 1);
        from[i] = j < held ? a.table + (int64_t)b * a.max_blocks + j
                           : a.free_pages + n_free - 1 - (pages[b] + j - held);
        last_b = b;
        last_j = j;
      }
    }
    // (the loads do not wait on one another: four requests' rows in a step of
    // single tokens)
#pragma unroll
    for (int i = 0; i < ROWS; ++i) id[i] = from[i] ? *from[i] : -1;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (from[i]) {
        if (id[i] < 0 || id[i] >= a.num_pages) {
          id[i] = -1;
          report(a.status);
        }
      } else if (i > 0) {
        id[i] = id[i - 1];
      }
      map[i] = slot[i] >= 0 && id[i] >= 0 ? (long long)id[i] * a.ps.d + off[i] : -1;
    }
    if (a.vec && r0 + ROWS <= n_rows) {
      *reinterpret_cast<int4*>(a.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(a.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.row_seq + r0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
      longlong2* m = reinterpret_cast<longlong2*>(a.slot_map + r0);
      m[0] = make_longlong2(map[0], map[1]);
      m[1] = make_longlong2(map[2], map[3]);
    } else {
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
        if (r0 + i < n_rows) {
          a.positions[r0 + i] = pos[i];
          a.slots[r0 + i] = slot[i];
          a.row_seq[r0 + i] = seq[i];
          a.slot_map[r0 + i] = map[i];
        }
    }
  }
}

// Pages past the kept tokens go onto the free list, request by request, in
// the table's order.
__global__ void __launch_bounds__(PT) release_kernel(const PlanArgs a) {
  extern __shared__ int smem[];
  const int B = a.batch, tid = threadIdx.x;
  ptx::wait_primary();
  ptx::launch_dependents();
  int* pages = smem;            // [B + 1] pages given back before request b
  int* kept = pages + B + 1;    // [B] pages it keeps
  const int n_free = free_count(a);
  const int each = (B + PT - 1) / PT;
  const int b0 = min(tid * each, B), b1 = min(b0 + each, B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += request<true>(a, b).need;
  long long all;
  long long at = block_scan(mine, all);
  const int total = (int)all;
  for (int b = b0; b < b1; ++b) {
    const Request r = request<true>(a, b);
    pages[b] = (int)at;
    kept[b] = r.held - r.need;
    at += r.need;
    if (blockIdx.x == 0) {
      a.seq_lens_out[b] = r.bad ? a.seq_lens[b] : r.rows;
      if (r.bad) report(a.status);
    }
  }
  const int room = a.num_pages - n_free;
  if (tid == 0) {
    pages[B] = total;
    if (blockIdx.x == 0) {
      *a.n_free_out = n_free + min(total, room);
      if (total > room) report(a.status);
    }
  }
  __syncthreads();
  const int n = min(total, room);
  for (uint32_t at_page = blockIdx.x * PT + tid; at_page < (uint32_t)n; at_page += gridDim.x * PT) {
    const int p = (int)at_page, b = find(pages, B, p);
    const int id = a.table[(int64_t)b * a.max_blocks + kept[b] + p - pages[b]];
    const bool ok = id >= 0 && id < a.num_pages;
    if (!ok) report(a.status);
    a.free_pages[n_free + p] = ok ? id : -1;
  }
}

template <typename K>
cudaError_t launch(K kernel, const PlanArgs& a, int words, long long items, int sms,
                   std::atomic<uint64_t>& done, cudaStream_t stream) {
  const int bytes = words * (int)sizeof(int);
  if (bytes > 48 * 1024) {
    cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kernel),
                                (3 * kMaxPlanBatch + 2) * (int)sizeof(int), done);
    if (e != cudaSuccess) return e;
  }
  const long long want = (items + PT - 1) / PT;
  // Three CTAs an SM at most: prompts of 509 requests, a million rows, take 9.7
  // us (two: 10.9; five, whose sums cost more than they bring: 10.3), pages of
  // 1000 requests given back 4.0 (4.1; 6.3).
  const int most = 3 * sms;
  const int grid = (int)(want < 1 ? 1 : (want > most ? most : want));
  return launch_early(kernel, dim3((unsigned)grid), PT, bytes, 1, stream, a);
}

}  // namespace

cudaError_t launch_plan_blocks(const PlanArgs& a, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  return launch(plan_kernel, a, 3 * a.batch + 2, ((long long)a.capacity + ROWS - 1) / ROWS, sms,
                done, stream);
}

cudaError_t launch_release_blocks(const PlanArgs& a, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const long long most = (long long)a.batch * a.max_blocks;
  return launch(release_kernel, a, 2 * a.batch + 1, (most < a.num_pages ? most : a.num_pages) / 2,
                sms, done, stream);
}

}  // namespace fdllm

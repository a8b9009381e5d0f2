// Attention of one new token a sequence over the paged cache, with the
// token's RoPE and its cache write.
//
// "Flash-dLLM: I/O-Aware KV Caching and Parallel Decoding for Fast,
// Memory-Efficient Diffusion LLMs" (ai4snews summary), paragraph 1: RoPE, the
// cache write and the paged attention of a step share a kernel. This is that
// step for a single row a sequence, whose products are already projected:
//
//   q' = R(p) q,  k' = R(p) k,  cache[slot] = (k', v)
//   s_j = scale q' . K_j  over the visible slots j,
//   out = sum_j e^(s_j - m) V_j / sum_j e^(s_j - m),  lse = m + ln sum_j e^(s_j - m)
//
// in one pass over K and V: each warp carries a running maximum m, sum l and
// O, rescaled when m grows.
//
// Bound: the visible K and V are read once, so HBM bandwidth; a query head
// shares its key head's bytes with up to seven others. What follows from it:
//   - Split over the length. The work of all (sequence, key head, up to 8
//     query heads) units is cut into tiles of 64 (bf16) or 32 (fp32) slots,
//     put in one line and dealt in equal contiguous shares, so that every CTA
//     streams the same number of bytes whatever the lengths are. A share holds
//     at most one unit's tail and one unit's head besides whole units; those
//     leave (m, l, O) in the workspace, and a second launch joins them in the
//     order of the shares (no atomics: the same result every time). It starts
//     under the first one's tail (dependent launch).
//   - Two CTAs an SM, each a loading warp and four computing ones. The loading
//     warp walks the line, looks pages up and keeps three tiles (96 KB at
//     head_dim 128) under way, whole pages of K and V by TMA, so that HBM sees
//     16 KB requests; it also brings each unit's q, cosines and sines, and
//     writes down for each tile what the others need to know. They take a
//     quarter of a tile's slots each and meet only where a unit ends. (One-warp
//     CTAs that each streamed 16-slot tiles of their own met nowhere and were
//     7 % slower on long sequences: 4 KB requests.) Pages that do not hold
//     whole runs of 16 (8) slots are gathered row by row in 16-byte copies.
//   - Where units are many, up to four times as many shares as CTAs run at once,
//     of eight tiles at least, taken over from the grid as CTAs get on: SMs do
//     not stream at one speed.
//   - bf16 products by m16n8k16 warp MMAs: eight heads are far too few rows
//     for tcgen05's 128, and the bytes bound them (the tensor pipe is active in
//     a fifth of the cycles, ncu). The cache's rows are the A operand (16 slots, then
//     16 dimensions), the heads B's eight columns; each fp32 value of q and
//     then of P enters as a bf16 pair hi + lo, a product each, which keeps 16
//     bits of it. Every thread holds two heads, whose statistics, scores and O
//     need no exchange but a transpose of P. fp32 caches use fp32 FMAs.
//   - q and k are rotated in fp64 (angles of far positions); k is rounded to
//     the cache's type once, q is not rounded. Both come with the unit's first
//     tile and are rotated by all computing warps; the new row waits in shared
//     memory for the tile that it belongs to.
//
// Measured on one B200, both launches, back to back, head_dim 128: two sequences
// of 120 to 131 thousand slots, 8 key heads: 157 to 159 us (6.5 TB/s, the rate of a
// copy); 32 of 256 to 1024 slots, 32 key heads: 60.7 us (5.5 TB/s; an end of a unit
// costs a CTA's computing warps 1.5 us); one of 768: 8.5 to 8.8 us (latency); fp32, 61
// sequences, pages of 6, head_dim 96: 48.6 us (4.4 TB/s; row copies and fp32 FMAs);
// fp32, 16 of 1024 to 4096, 8 key heads, pages of 64: 56 us with one head each and 59
// with four (6.0 and 5.7 TB/s), 91 with eight (3.7 TB/s: one CTA an SM, and FMAs).
// K and V are read once for every eight heads of a key head: four sequences of 60 to
// 66 thousand slots, one key head: 31 us with 8 heads, 37 with 16, 69 with 32.
#include <cuda_bf16.h>

#include <cstdint>

#include "fdllm.h"
#include "fdllm_internal.h"
#include "host_api.h"
#include "ptx_serve.cuh"
#include "serve_index.h"
#include "serve_internal.h"

namespace fdllm {
namespace {

constexpr int NH = kDecodeHeads;
constexpr int WARPS = 4;                // computing warps
// Loading warps: one issues tile loads; row-by-row copies take four, a quarter
// of a tile each (one took 90 us where four took 70;
// two take as long as four but for short rows: 26.7 us against 25.6 at head_dim 32).
constexpr int loaders(bool rows) { return rows ? WARPS : 1; }
constexpr int JT = 256;                 // threads of the joining CTA
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <bool kF32, int D>
struct Shape {
  using T = typename std::conditional<kF32, float, __nv_bfloat16>::type;
  static constexpr int SIZE = kF32 ? 4 : 2;
  static constexpr int KS = kF32 ? 8 : 16;              // slots of a warp's quarter
  static constexpr int TILE = KS * WARPS;
  static constexpr int ROW = D * SIZE;                  // bytes of a row
  static constexpr int CH = ROW / 16;                   // its 16-byte chunks
  // A quarter's rows lie as a tile load writes them: pieces of PB bytes of all
  // KS rows one after another, chunks swizzled within 128 (64) bytes, so that
  // equal chunks of eight consecutive rows are in different banks.
  static constexpr int PB = ROW % 128 == 0 ? 128 : 64;
  static constexpr int QUARTER = KS * ROW;
  static constexpr int V = WARPS * QUARTER;             // from a quarter's K rows to its V rows
  static constexpr int STAGE = 2 * V;
  static constexpr int STAGES = D <= 64 ? 4 : 3;
  static constexpr int OROW = D + 8;                    // floats between rotated heads of q
  static_assert(KS * CH % 32 == 0, "whole warps of chunks");
  static_assert(NH * D * 4 <= QUARTER, "a warp's O fits its part of a consumed tile");
  static __device__ __forceinline__ int at(int row, int chunk) {
    constexpr int CPP = PB / 16;
    return chunk / CPP * (KS * PB) + row * PB +
           (chunk % CPP ^ (PB == 128 ? row & 7 : row >> 1 & 3)) * 16;
  }
};

// A sequence as every kernel here sees it.
struct Seq {
  int first, len;     // visible slots [first, len)
  int slot;           // where the new row goes, -1: nowhere
  int pos;
  int tile0, tiles;   // its tiles; at least one, so that an empty one is answered too
  bool bad;
};

template <int TILE>
__device__ __forceinline__ Seq seq_of(const DecodeArgs& a, int b) {
  Seq s;
  const int top = a.max_blocks * (int)a.ps.d;
  s.len = a.seq_lens[b];
  s.first = a.starts ? max(a.starts[b], 0) : 0;
  s.pos = a.positions ? a.positions[b] : 0;
  s.slot = -1;
  s.bad = s.len < 0 || s.len > top;
  if (a.rope_cos) s.bad |= s.pos < 0 || s.pos >= a.max_position;
  if (a.k) {
    s.slot = a.slots ? max(a.slots[b], -1) : s.pos;
    s.bad |= s.slot >= top || (!a.slots && s.pos < 0);
  }
  if (s.bad) {
    s.len = 0;
    s.slot = -1;
  }
  s.first = min(s.first, s.len);
  s.tile0 = s.first / TILE;
  s.tiles = tiles_of(s.first, s.len, TILE);
  return s;
}

__device__ __forceinline__ void report(int32_t* status) {
  if (status) atomicExch(reinterpret_cast<int*>(status), (int)FDLLM_ERR_DEVICE_BOUNDS);
}

// The shares of a line of `total` tiles (fewer than 2^31): the first `more` of
// q + 1 tiles, the others of q. As many as CTAs run at once; where the grid has
// more CTAs (they are taken over one by one), as many as that, but of eight
// tiles at least. Divided by constants of the launch, with the host's
// multipliers: a division takes over 100 cycles, and nothing else goes on
// before the first load.
struct Shares {
  int total, q, more;
  __device__ __forceinline__ Shares(const DecodeArgs& a, int n) : total(n), q(1), more(0) {
    if (n <= a.resident) return;
    q = a.resident_div.div(n);
    more = n - q * a.resident;
    if (q < 8 || a.ctas == a.resident) return;
    q = a.ctas_div.div(n);
    more = n - q * a.ctas;
    if (q < 8) q = 8, more = 0;         // (the last one may be short)
  }
  __device__ __forceinline__ int begin(int i) const { return i * q + min(i, more); }
  __device__ __forceinline__ int end(int i) const { return min(begin(i + 1), total); }
  __device__ __forceinline__ int with(int tile) const {
    const int first = more * (q + 1);
    return tile < first ? (uint32_t)tile / (uint32_t)(q + 1)
                        : more + (uint32_t)(tile - first) / (uint32_t)q;
  }
};

// What the computing warps know of a tile.
struct Tile {
  uint32_t seen[WARPS];                 // visible slots of each quarter, one bit each
  int flags;
  int b, hk, chunk;                     // its unit
  int slot;                             // of the new row
  int row;                              // of the pool for it, -1: another unit writes it there
  int key0;
  int part;                             // partial result that its segment leaves, if not whole
};
constexpr int kFirst = 1;               // first tile of its segment: q is in the stage's slot
constexpr int kLast = 2;                // last tile of its segment
constexpr int kWhole = 4;               // the segment is a whole unit
constexpr int kRow = 8;                 // first tile: the new row is this segment's to make
constexpr int kNew = 16;                // and is one of this tile's
constexpr int kBad = 32;                // the sequence's metadata is out of range
constexpr int kStop = 64;               // no tile: the work is done

// The joining launch starts under the first one's tail, and reads the lengths
// (for which parts there are) while it waits. Its own wait would make them
// visible, but ends with the first launch. So one thread of the first launch,
// past its wait for what came before, releases this mark, and a joining warp that
// acquires it may read on; one that does not find it waits first. The joining
// launch takes the mark off again. (1 x 768: 8.5 us; 9.7 with the wait first.)
constexpr unsigned long long kBegun = 0x64c0de5eb8f3a127ull;

template <int STAGES>
struct Ctrl {
  uint64_t full[STAGES];                // a tile has come: 33 arrivals of a loading warp
  uint64_t empty[STAGES];               // it is consumed: one arrival a warp
  uint64_t took;                        // the answer in `answer` has arrived
  uint64_t met;                         // the computing warps meet, and
  uint64_t met_loaders;                 // the loading warps
  alignas(16) uint8_t answer[16];
  Tile tile[STAGES];
  float m[2][WARPS][NH];                // of a segment, by turns
  float l[2][WARPS][NH];
};

// 32 sequences of the line, one a lane, kept by a warp: what a batch of up to
// 32 needs is read once. A larger one is walked through, 32 at a time, by every
// loading warp (for the line's length, then for its share's place) and every
// joining one, which short sequences do not cover: 1000 of up to 1024 slots, 8 key
// heads, 510 us (6.2 TB/s), of up to 128 slots 136 us, of up to 16 slots 110 us.
template <int TILE>
struct Window {
  Seq own;
  int b0, base;       // its first sequence and the tiles before that
  int n, sum;         // this lane's tiles, and the sums up to it
  __device__ __forceinline__ void read(const DecodeArgs& a, int b, int before) {
    const int lane = threadIdx.x & 31;
    b0 = b;
    base = before;
    own = seq_of<TILE>(a, min(b + lane, a.batch - 1));
    n = b + lane < a.batch ? own.tiles * a.units_per_seq : 0;
    sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += t;
    }
  }
  __device__ __forceinline__ int end() const { return base + __shfl_sync(0xffffffffu, sum, 31); }
  // Up to the last window; the line's tiles.
  __device__ __forceinline__ int read_all(const DecodeArgs& a) {
    read(a, 0, 0);
    while (b0 + 32 < a.batch) read(a, b0 + 32, end());
    return end();
  }
  // To the window that tile lo of the line falls to.
  __device__ __forceinline__ void find(const DecodeArgs& a, int lo) {
    if (lo < base) read(a, 0, 0);
    for (int e = end(); lo >= e && b0 + 32 < a.batch; e = end()) read(a, b0 + 32, e);
  }
  __device__ __forceinline__ Seq get(const DecodeArgs& a, int b) {
    if (b >= b0 + 32) read(a, b0 + 32, end());
    const int i = b - b0;
    Seq s;
    s.first = __shfl_sync(0xffffffffu, own.first, i);
    s.len = __shfl_sync(0xffffffffu, own.len, i);
    s.slot = __shfl_sync(0xffffffffu, own.slot, i);
    s.pos = __shfl_sync(0xffffffffu, own.pos, i);
    s.tile0 = __shfl_sync(0xffffffffu, own.tile0, i);
    s.tiles = __shfl_sync(0xffffffffu, own.tiles, i);
    s.bad = __shfl_sync(0xffffffffu, (int)own.bad, i);
    return s;
  }
};

// A place in the line of tiles.
template <int TILE>
struct Cursor {
  Window<TILE> w;
  Seq s;
  int b, u, t;        // sequence, unit of it, tile of the unit
  int hk, chunk;      // the unit's key head and its part of the query heads
  __device__ __forceinline__ void open(const DecodeArgs& a, int lo) {
    w.find(a, lo);
    const int i = __ffs(__ballot_sync(0xffffffffu, lo < w.base + w.sum)) - 1;
    const int tile = lo - w.base - __shfl_sync(0xffffffffu, w.sum - w.n, i);
    b = w.b0 + i;
    s = w.get(a, b);
    u = (uint32_t)tile / (uint32_t)s.tiles;
    t = tile - u * s.tiles;
    hk = a.head_chunks == 1 ? u : u / a.head_chunks;
    chunk = u - hk * a.head_chunks;
  }
  __device__ __forceinline__ void next_unit(const DecodeArgs& a) {
    t = 0;
    if (++chunk == a.head_chunks) {
      chunk = 0;
      ++hk;
    }
    if (++u < a.units_per_seq) return;
    u = hk = 0;
    if (++b < a.batch) s = w.get(a, b);
  }
};

__device__ __forceinline__ double load_in(const void* p, int64_t i, bool f32) {
  return f32 ? (double)reinterpret_cast<const float*>(p)[i]
             : (double)__bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ void put(__nv_bfloat16* p, double x) { *p = ptx::double_to_bf16(x); }
__device__ __forceinline__ void put(float* p, double x) { *p = (float)x; }

__device__ __forceinline__ void write_out2(const DecodeArgs& a, int64_t at, float x, float y) {
  if (a.out_bf16)
    *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(a.out) + at) =
        __floats2bfloat162_rn(x, y);
  else
    *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out) + at) = make_float2(x, y);
}

__device__ __forceinline__ float inverse(float l) { return l > 0.f ? 1.f / l : (l == l ? 0.f : l); }

// m: the largest score in steps of log2. Nothing seen: l = 0 and -inf. A NaN
// score leaves m as it is (-inf when every score is one) and l NaN, which stays.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : fmaf(m, kLn2, logf(l));
}

// Floats of a partial result: O of each head, then m, then l, each 16-byte
// aligned as a whole.
__host__ __device__ constexpr int part_floats(int heads, int head_dim) {
  return heads * (head_dim + 4);
}

// Values d and d + D / 2 of a row of q or k, rotated. cs: D / 2 cosines, then
// the sines, or null.
struct Pair {
  double x, y;
};
template <int D>
__device__ __forceinline__ Pair rotated(const void* row, const double* cs, int d, bool f32) {
  const double x = load_in(row, d, f32), y = load_in(row, d + D / 2, f32);
  if (!cs) return {x, y};
  const double c = cs[d], n = cs[D / 2 + d];
  return {x * c - y * n, y * c + x * n};
}

// ---------------------------------------------------------------- a warp's arithmetic
// bf16 cache: S and O by warp MMAs (see the header).
template <bool kF32, int D, int HT>
struct Warp;

template <int D, int HT>
struct Warp<false, D, HT> {
  using S = Shape<false, D>;
  uint32_t q[D / 16][4];    // hi and lo of dimensions 2t, 2t+1, then of 2t+8, 2t+9; head g
  float o[D / 16][4];       // dimensions g and g + 8 of heads 2t and 2t + 1
  float m[2], l[2];         // of heads 2t and 2t + 1; l: of this thread's slots alone

  // qf: the unit's rotated q, [head][OROW].
  __device__ __forceinline__ void open(const float* qf, int heads) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float2 x = make_float2(0.f, 0.f);
        if (g < heads) x = *reinterpret_cast<const float2*>(qf + g * S::OROW + kk * 16 + j * 8 + 2 * t);
        ptx::split_bf16(x.x, x.y, q[kk][2 * j], q[kk][2 * j + 1]);
      }
#pragma unroll
    for (int n = 0; n < D / 16; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  // The 32 dimensions i, of every piece in turn: the swizzle is an exclusive
  // or within a piece's row, so the chunks' addresses are too.
  template <int P>
  __device__ __forceinline__ void scores(float (&hi)[4], float (&lo)[4], uint32_t ka, int i) {
    if constexpr (P < S::ROW / S::PB) {
      uint32_t r[4];
      const int kk = P * (S::PB / 32) + i;
      ptx::ldmatrix4<P * S::KS * S::PB>(r, ka);
      ptx::mma_bf16(hi, r, q[kk][0], q[kk][2]);
      ptx::mma_bf16(lo, r, q[kk][1], q[kk][3]);
      scores<P + 1>(hi, lo, ka, i);
    }
  }
  template <int P>
  __device__ __forceinline__ void outputs(const uint32_t (&p)[4], uint32_t va, int i) {
    if constexpr (P < S::ROW / S::PB) {
      uint32_t r[4];
      const int n = P * (S::PB / 32) + i;
      ptx::ldmatrix4_trans<S::V + P * S::KS * S::PB>(r, va);
      ptx::mma_bf16(o[n], r, p[0], p[1]);
      ptx::mma_bf16(o[n], r, p[2], p[3]);
      outputs<P + 1>(p, va, i);
    }
  }

  __device__ __forceinline__ void step(const uint8_t* stage, uint32_t seen, float c, const float*,
                                       float*) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const int mi = lane >> 3, mr = lane & 7;
    const uint32_t base = ptx::smem_u32(stage);
    const uint32_t ka = base + S::at((mi & 1) * 8 + mr, mi >> 1);
    const uint32_t va = base + S::at((mi >> 1) * 8 + mr, mi & 1);
    float s[4] = {}, s2[4] = {};        // slots g and g + 8 of heads 2t and 2t + 1
#pragma unroll
    for (int i = 0; i < S::PB / 32; ++i) scores<0>(s, s2, ka ^ (i * 32), i);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] += s2[i];
    if (seen != (1u << S::KS) - 1) {
      if (!(seen >> g & 1)) s[0] = s[1] = -INFINITY;
      if (!(seen >> (g + 8) & 1)) s[2] = s[3] = -INFINITY;
    }
    float top[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], d));
      top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], d));
    }
    if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
      float f[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float mn = fmaxf(m[j], top[j]);
        f[j] = mn == -INFINITY ? 1.f : ptx::ex2((m[j] - mn) * c);
        m[j] = mn;
        l[j] *= f[j];
      }
#pragma unroll
      for (int n = 0; n < D / 16; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][i] *= f[i & 1];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float mc = m[j] == -INFINITY ? 0.f : m[j] * c;
      s[j] = ptx::ex2(fmaf(s[j], c, -mc));
      s[j + 2] = ptx::ex2(fmaf(s[j + 2], c, -mc));
      l[j] += s[j] + s[j + 2];
    }
    uint32_t p[4];                      // hi of slots 0-7 and 8-15, then lo
    ptx::split_bf16(s[0], s[1], p[0], p[2]);
    ptx::split_bf16(s[2], s[3], p[1], p[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = ptx::transpose8(p[i]);
#pragma unroll
    for (int i = 0; i < S::PB / 32; ++i) outputs<0>(p, va ^ (i * 32), i);
  }

  // O of each head to buf [head][D], m and l to the control block.
  __device__ __forceinline__ void close(float* buf, float* ms, float* ls, int heads) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float sum = l[j];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      const int h = 2 * t + j;
      if (h < heads) {
#pragma unroll
        for (int n = 0; n < D / 16; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) buf[h * D + n * 16 + 8 * e + g] = o[n][j + 2 * e];
        if (g == 0) {
          ms[h] = m[j];
          ls[h] = sum;
        }
      }
    }
  }
};

// fp32 cache, up to HT (1, 4 or 8) heads: lane l scores slot l % 8 over the
// quarter l / 8 of the dimensions. With four heads the quarters' sums are
// exchanged so that each lane ends with the whole score of one head (the
// quarter's number; of two with eight heads), and a softmax step of all heads
// costs what one head's would. For O a lane owns four dimensions (lanes beyond
// D / 4 take other slots of the stage).
template <int D, int HT>
struct Warp<true, D, HT> {
  using S = Shape<true, D>;
  static constexpr int OWN = D / 4;                 // lanes that cover a row
  static constexpr int SETS = 32 / OWN;             // slots taken side by side
  static constexpr int HL = HT == 8 ? 2 : 1;        // heads whose scores a lane holds
  float4 o[HT];
  float m[HL], l[HL];                               // l: of this lane's slots alone

  __device__ __forceinline__ void open(const float*, int) {
#pragma unroll
    for (int h = 0; h < HT; ++h) o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int h = 0; h < HL; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
    }
  }

  __device__ __forceinline__ void step(const uint8_t* stage, uint32_t seen, float c,
                                       const float* qf, float* ps) {
    const int lane = threadIdx.x & 31, key = lane & 7, part = lane >> 3;
    float s[HT];
#pragma unroll
    for (int h = 0; h < HT; ++h) s[h] = 0.f;
    const float* qp = qf + part * 4;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const int ch = i * 4 + part;
      const float4 k = *reinterpret_cast<const float4*>(stage + S::at(key, ch));
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        const float4 q = *reinterpret_cast<const float4*>(qp + h * S::OROW + i * 16);
        s[h] = fmaf(k.x, q.x, fmaf(k.y, q.y, fmaf(k.z, q.z, fmaf(k.w, q.w, s[h]))));
      }
    }
    const bool vis = (seen >> key) & 1;
    float f[HL];
    bool grew = false;
#pragma unroll
    for (int j = 0; j < HL; ++j) {
      float v;
      if constexpr (HT == 1) {
        v = s[0] + __shfl_xor_sync(0xffffffffu, s[0], 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
      } else {
        const float* x = s + 4 * j;
        const bool up = part & 2, odd = part & 1;
        const float a = (up ? x[2] : x[0]) + __shfl_xor_sync(0xffffffffu, up ? x[0] : x[2], 16);
        const float b = (up ? x[3] : x[1]) + __shfl_xor_sync(0xffffffffu, up ? x[1] : x[3], 16);
        v = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
      }
      if (!vis) v = -INFINITY;
      float top = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
      const float mn = fmaxf(m[j], top);
      f[j] = mn == -INFINITY ? 1.f : ptx::ex2((m[j] - mn) * c);
      grew |= mn != m[j];
      const float mc = mn == -INFINITY ? 0.f : mn * c;
      const float p = ptx::ex2(fmaf(v, c, -mc));
      m[j] = mn;
      l[j] = fmaf(l[j], f[j], p);
      if (HT > 1 || part == 0) ps[key * HT + (HT > 1 ? 4 * j + part : 0)] = p;
    }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        const float fh = __shfl_sync(0xffffffffu, f[h / 4], (h % 4) * 8);
        o[h].x *= fh, o[h].y *= fh, o[h].z *= fh, o[h].w *= fh;
      }
    }
    __syncwarp();
    const int own = lane % OWN, set = lane / OWN;
    if (set < SETS) {
#pragma unroll
      for (int j = 0; j < S::KS; j += SETS) {
        const float4 v = *reinterpret_cast<const float4*>(stage + S::V + S::at(j + set, own));
        const float* pj = ps + (j + set) * HT;
        float p[HT];
        if constexpr (HT == 1) {
          p[0] = pj[0];
        } else {
#pragma unroll
          for (int h = 0; h < HT; h += 4)
            *reinterpret_cast<float4*>(p + h) = *reinterpret_cast<const float4*>(pj + h);
        }
#pragma unroll
        for (int h = 0; h < HT; ++h) {
          o[h].x = fmaf(p[h], v.x, o[h].x);
          o[h].y = fmaf(p[h], v.y, o[h].y);
          o[h].z = fmaf(p[h], v.z, o[h].z);
          o[h].w = fmaf(p[h], v.w, o[h].w);
        }
      }
    }
  }

  __device__ __forceinline__ void close(float* buf, float* ms, float* ls, int heads) {
    const int lane = threadIdx.x & 31, own = lane % OWN, set = lane / OWN;
#pragma unroll
    for (int j = 0; j < HL; ++j) {
      float sum = l[j];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      const int h = HT == 1 ? 0 : 4 * j + (lane >> 3);
      if ((lane & 7) == 0 && h < heads && (HT > 1 || lane == 0)) {
        ms[h] = m[j];
        ls[h] = sum;
      }
    }
#pragma unroll
    for (int h = 0; h < HT; ++h) {
      float4 v = o[h];
      if (SETS > 1) {
#pragma unroll
        for (int d = OWN; d < 32; d <<= 1) {
          v.x += __shfl_xor_sync(0xffffffffu, v.x, d);
          v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
          v.z += __shfl_xor_sync(0xffffffffu, v.z, d);
          v.w += __shfl_xor_sync(0xffffffffu, v.w, d);
        }
      }
      if (set == 0 && h < heads) *reinterpret_cast<float4*>(buf + h * D + own * 4) = v;
    }
  }
};

// ---------------------------------------------------------------- the shares
// Waits for an arrival, for a second at most; reported if `said`.
__device__ __forceinline__ bool wait_arrival(uint64_t* bar, uint32_t parity, const DecodeArgs& a,
                                             bool said = true) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!ptx::mbar_try_wait(bar, parity))
    if (clock64() - t0 > a.wait_cycles) {
      if (said && a.status)
        atomicExch(reinterpret_cast<int*>(a.status), (int)FDLLM_ERR_TIMEOUT);
      return false;
    }
  return true;
}

// Warps meet at `bar` (its count is theirs); bounded as every wait here, so
// that none is held up by another that gave up.
__device__ __forceinline__ bool meet(uint64_t* bar, uint32_t& phase, const DecodeArgs& a) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar);
  const bool ok = __all_sync(0xffffffffu, wait_arrival(bar, phase & 1, a));
  ++phase;
  __syncwarp();
  return ok;
}

// The arrivals of a loading warp at a stage's barrier: each lane's once its
// copies are there, and one that releases what the warp has stored for the tile
// (an arrival that waits for copies orders copies, not stores).
__device__ __forceinline__ void publish(uint64_t* full, bool withhold = false) {
  ptx::cp_async_arrive(full);
  __syncwarp();
  if ((threadIdx.x & 31) == 0 && !withhold) ptx::mbar_arrive(full);
}

// A loading warp: walks the shares, brings every tile (by rows: its quarter of
// it) and, the first of them, the unit's q.
template <bool kF32, int D, bool kRows>
__device__ __forceinline__ void load_tiles(const DecodeArgs& a, const CUtensorMap* tmap_k,
                                           const CUtensorMap* tmap_v,
                                           Ctrl<Shape<kF32, D>::STAGES>& ctrl, uint8_t* ring,
                                           uint8_t* slots) {
  using S = Shape<kF32, D>;
  const int lane = threadIdx.x & 31, loader = (threadIdx.x >> 5) - WARPS;
  const bool first = loader == 0;
  // The line of tiles, and this CTA's first share of it.
  Cursor<S::TILE> at;
  const int total = at.w.read_all(a);
  const Shares shares(a, total);
  int share = blockIdx.x;
  // One request for another share is always under way while there are more
  // than run at once.
  bool asked = shares.begin(share) < total && shares.begin(a.resident) < total;
  uint32_t answers = 0, meetings = 0;
  int stage = 0;
  uint32_t round = 0;                   // passes through the ring
  bool ok = true;                       // no wait has given up
  auto next_stage = [&] {
    if (++stage == S::STAGES) {
      stage = 0;
      ++round;
    }
  };
  auto wait_empty = [&] {
    if (round > 0 && ok)
      ok = __all_sync(0xffffffffu, wait_arrival(&ctrl.empty[stage], (round - 1) & 1, a));
    __syncwarp();
  };
  while (ok && shares.begin(share) < total) {
    if (asked && lane == 0 && first) {
      ptx::fence_async_shared();
      ptx::mbar_arrive_expect_tx(&ctrl.took, 16);
      ptx::take_cta(ctrl.answer, &ctrl.took);
    }
    const int lo = shares.begin(share);
    int left = shares.end(share) - lo;
    at.open(a, lo);
    bool first_segment = true;
    while (ok && left > 0) {
      // a segment: the tiles of one unit in this share
      const int seg = min(left, at.s.tiles - at.t);
      const int heads = min(NH, a.group - at.chunk * NH);
      int flags = kFirst | (seg == at.s.tiles ? kWhole : 0) | (at.s.bad ? kBad : 0);
      if (at.s.bad && at.t == 0 && lane == 0 && first) report(a.status);
      // The new row: made with the segment that sees it, or that begins the
      // unit when none does.
      const bool seen_slot = at.s.slot >= at.s.first && at.s.slot < at.s.len;
      const int new_tile = seen_slot ? at.s.slot / S::TILE - at.s.tile0 - at.t : -1;
      if (at.s.slot >= 0 && (seen_slot ? new_tile >= 0 && new_tile < seg : at.t == 0 && at.chunk == 0))
        flags |= kRow;
      for (int i = 0; i < seg; ++i) {
        const int key0 = (at.s.tile0 + at.t + i) * S::TILE;
        // runs: lane w < 4 looks up quarter w; by rows: lane r < KS row r of
        // this warp's quarter (the lanes beyond stay inside the tile: a slot
        // behind the last tile may be past 2^31)
        const int key = key0 + (kRows ? loader * S::KS + min(lane, S::KS - 1)
                                      : min(lane, WARPS - 1) * S::KS);
        int row = -1;
        uint32_t seen = 0;              // runs: of quarter `lane`
        bool want = lane < S::KS && key < at.s.len && key >= at.s.first;
        if (!kRows) {
          const int f = min(max(at.s.first - key, 0), S::KS), n = min(max(at.s.len - key, 0), S::KS);
          seen = lane < WARPS && n > f ? ((1u << n) - 1) & ~((1u << f) - 1) : 0;
          want = seen;
        }
        if (want) {
          const int j = a.ps.div(key);
          const int id = a.block_table[(int64_t)at.b * a.max_blocks + j];
          if (id >= 0 && id < a.num_pages)
            // the pool holds fewer than 2^31 rows
            row = (id * a.n_kv_heads + at.hk) * (int)a.ps.d + key - j * (int)a.ps.d;
          else
            report(a.status);
        }
        const int f = flags | (i == seg - 1 ? kLast : 0) | (i == new_tile ? kNew : 0);
        int new_at = -1;
        if (first && f & kRow && at.chunk == 0) {
          const int j = a.ps.div(at.s.slot);
          const int id = a.block_table[(int64_t)at.b * a.max_blocks + j];
          if (id >= 0 && id < a.num_pages)
            new_at = (id * a.n_kv_heads + at.hk) * (int)a.ps.d + at.s.slot - j * (int)a.ps.d;
          else if (lane == 0)
            report(a.status);
        }
        wait_empty();
        if (!ok) break;
        const uint32_t dst = ptx::smem_u32(ring) + stage * S::STAGE;
        uint64_t* bar = &ctrl.full[stage];
        Tile* tile = &ctrl.tile[stage];
        if constexpr (!kRows) {
          if (row < 0) seen = 0;
          if (lane < WARPS) tile->seen[lane] = seen;
          // Boxes of a.box quarters. All rows of one come, the new row's old
          // contents and what is not visible among them: neither is used (see
          // the computing warps).
          const uint32_t real = __ballot_sync(0xffffffffu, seen != 0);
          int bytes = 0;
          for (int w = 0; w < WARPS; w += a.box)
            if (real >> w & ((1u << a.box) - 1)) bytes += 2 * a.box * S::QUARTER;
          if (lane == 0 && bytes) ptx::mbar_expect_tx(bar, bytes);
          __syncwarp();
          for (int w = 0; w < WARPS; w += a.box) {
            const uint32_t any = real >> w & ((1u << a.box) - 1);
            if (!any) continue;
            // (the box's first quarter may be hidden: its row follows from another's)
            const int by = w + __ffs(any) - 1;
            const int r = __shfl_sync(0xffffffffu, row, by) - (by - w) * S::KS;
            if (ptx::elect_one()) {
              ptx::tma_load_4d_at(dst + w * S::QUARTER, tmap_k, 0, 0, 0, r / S::KS, bar);
              ptx::tma_load_4d_at(dst + S::V + w * S::QUARTER, tmap_v, 0, 0, 0, r / S::KS, bar);
            }
            __syncwarp();
          }
        } else {
          seen = __ballot_sync(0xffffffffu, row >= 0);
          if (lane == 0) tile->seen[loader] = seen;
          if (key == at.s.slot) row = -1;              // the new row is not read
          const uint32_t to = dst + loader * S::QUARTER;
#pragma unroll
          for (int e = 0; e < S::KS * S::CH / 32; ++e) {
            const int ch = e * 32 + lane;
            const int r = ch / S::CH, cc = ch % S::CH;
            const int src = __shfl_sync(0xffffffffu, row, r);
            const int64_t off = (int64_t)max(src, 0) * S::ROW + cc * 16;
            ptx::cp_async16(to + S::at(r, cc), reinterpret_cast<const uint8_t*>(a.k_pool) + off,
                            src >= 0);
            ptx::cp_async16(to + S::V + S::at(r, cc),
                            reinterpret_cast<const uint8_t*>(a.v_pool) + off, src >= 0);
          }
        }
        if (first && f & kFirst && !at.s.bad) {
          // the unit's q, the new row's k and v (where there is room), cosines
          // and sines come along
          const int size = a.in_f32 ? 4 : 2;
          const uint32_t to = ptx::smem_u32(slots) + stage * a.slot_bytes;
          auto bring = [&](uint32_t at_byte, const void* from, int64_t element, int bytes) {
            const uint8_t* p = reinterpret_cast<const uint8_t*>(from) + element * size;
            for (int e = lane * 16; e < bytes; e += 512) ptx::cp_async16(to + at_byte + e, p + e, true);
          };
          bring(0, a.q, (int64_t)at.b * a.q_stride + (int64_t)(at.hk * a.group + at.chunk * NH) * D,
                heads * D * size);
          if (f & kRow && a.kv_at) {
            bring(a.kv_at, a.k, (int64_t)at.b * a.k_stride + (int64_t)at.hk * D, D * size);
            bring(a.kv_at + D * size, a.v, (int64_t)at.b * a.v_stride + (int64_t)at.hk * D, D * size);
          }
          if (a.rope_cos)
#pragma unroll
            for (int e = lane; e < D / 2; e += 32) {
              const double* t = e < D / 4 ? a.rope_cos : a.rope_sin;
              ptx::cp_async16(to + a.rope_at + e * 16,
                              t + (int64_t)at.s.pos * (D / 2) + (e < D / 4 ? e : e - D / 4) * 2, true);
            }
        }
        if (lane == 0 && first) {
          tile->flags = f;
          tile->b = at.b;
          tile->hk = at.hk;
          tile->chunk = at.chunk;
          tile->slot = at.s.slot;
          tile->row = new_at;
          tile->key0 = key0;
          tile->part = 2 * share + (first_segment ? 0 : 1);
        }
        // (withheld where a test wants the wait for it to run out: fdllm_inject_tile_timeout)
        publish(bar, a.withhold && round == 0 && stage == 0);
        flags &= ~(kFirst | kRow);
        next_stage();
      }
      first_segment = false;
      left -= seg;
      at.next_unit(a);
    }
    if (!asked) break;
    // (a wait that gives up ends the work, and is reported; the answer is waited
    // for all the same, it comes into this CTA's memory)
    ok = __all_sync(0xffffffffu, wait_arrival(&ctrl.took, answers & 1, a)) && ok;
    ++answers;
    share = ok ? ptx::taken_cta(ctrl.answer) : -1;
    // every loading warp has read the answer before the next request
    if (kRows) ok = meet(&ctrl.met_loaders, meetings, a) && ok;
    else __syncwarp();
    if (share < 0) break;
  }
  wait_empty();
  if (ok) {
    if (lane == 0 && first) ctrl.tile[stage].flags = kStop;
    publish(&ctrl.full[stage]);
  }
  // No copy is under way when this warp leaves: the computing warps may have given
  // up before it. (After a wait that gave up here the next stage may hold one too.)
  ptx::cp_async_wait_all();
  if (lane != 0) return;
#pragma unroll 1
  for (int s = 0; s < S::STAGES; ++s) {
    const int pass = last_pass(s, stage, (int)round);
    if (pass >= 0 && !(ok && s == stage)) wait_arrival(&ctrl.full[s], pass & 1, a, false);
  }
}

template <bool kF32, int D, int HT, bool kRows>
__global__ void __launch_bounds__(32 * (WARPS + loaders(kRows)), 2) decode_kernel(
    const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
    const DecodeArgs a) {
  using S = Shape<kF32, D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* slots = ring + S::STAGES * S::STAGE;
  __shared__ Ctrl<S::STAGES> ctrl;
  // q, rotated: room for the unit's heads; of an fp32 cache, which reads it with
  // every tile, at a fixed place (61 sequences, 3 heads a key head: 53.3 us instead of 56.5)
  __shared__ __align__(16) float q_fixed[kF32 ? HT * S::OROW : 4];
  float* qf = kF32 ? q_fixed : reinterpret_cast<float*>(slots + S::STAGES * a.slot_bytes);
  // the new row's K and V
  __shared__ __align__(16) typename S::T fresh[2 * D];
  __shared__ __align__(16) float ps[kF32 ? WARPS * S::KS * HT : 4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < S::STAGES; ++i) {
      ptx::mbar_init(&ctrl.full[i], 33 * loaders(kRows));
      ptx::mbar_init(&ctrl.empty[i], WARPS);
    }
    ptx::mbar_init(&ctrl.took, 1);
    ptx::mbar_init(&ctrl.met, WARPS);
    ptx::mbar_init(&ctrl.met_loaders, loaders(kRows));
    ptx::fence_mbar_init();
    if (!kRows) {
      ptx::prefetch_tmap(&tmap_k);
      ptx::prefetch_tmap(&tmap_v);
    }
  }
  ptx::wait_primary();
  ptx::launch_dependents();
  ptx::fence_async_global();
  __syncthreads();
  if (warp >= WARPS) {
    load_tiles<kF32, D, kRows>(a, &tmap_k, &tmap_v, ctrl, ring, slots);
    return;
  }
  if (blockIdx.x == 0 && tid == 0) ptx::st_release_gpu(a.begun, kBegun);

  const float c = a.scale * kLog2e;
  float* my_ps = kF32 ? ps + warp * S::KS * HT : ps;
  Warp<kF32, D, HT> w;
  int stage = 0, turn = 0;
  uint32_t phase = 0, meetings = 0;
#pragma unroll 1
  while (true) {
    // a tile that does not come within a second ends the work, reported
    if (!__all_sync(0xffffffffu, wait_arrival(&ctrl.full[stage], phase, a))) break;
    __syncwarp();
    const Tile* tile = &ctrl.tile[stage];
    const int flags = tile->flags;
    if (flags & kStop) break;
    const uint32_t seen = tile->seen[warp];
    uint8_t* rows = ring + stage * S::STAGE + warp * S::QUARTER;
    const int heads = min(NH, a.group - tile->chunk * NH);
    if (flags & kFirst) {
      // q and the new k are rotated once, by all four warps (they are past the
      // last unit: they have met since)
      const uint8_t* slot = slots + stage * a.slot_bytes;
      const double* cs =
          a.rope_cos ? reinterpret_cast<const double*>(slot + a.rope_at) : nullptr;
      const int size = a.in_f32 ? 4 : 2;
      const int real = flags & kBad ? 0 : heads, made = kF32 ? HT : real;
      for (int e = tid; e < (made + (flags & kRow ? 1 : 0)) * (D / 2); e += 32 * WARPS) {
        const int h = e / (D / 2), d = e % (D / 2);
        if (h < made) {
          const Pair x = h < real ? rotated<D>(slot + h * D * size, cs, d, a.in_f32) : Pair{0., 0.};
          qf[h * S::OROW + d] = (float)x.x;
          qf[h * S::OROW + d + D / 2] = (float)x.y;
          continue;
        }
        const uint8_t *k = slot + a.kv_at, *v = k + D * size;
        if (!a.kv_at) {                  // no room beside q: from where they are
          k = reinterpret_cast<const uint8_t*>(a.k) +
              ((int64_t)tile->b * a.k_stride + (int64_t)tile->hk * D) * size;
          v = reinterpret_cast<const uint8_t*>(a.v) +
              ((int64_t)tile->b * a.v_stride + (int64_t)tile->hk * D) * size;
        }
        const Pair x = rotated<D>(k, cs, d, a.in_f32);
        const Pair y = rotated<D>(v, nullptr, d, a.in_f32);
        put(&fresh[d], x.x);
        put(&fresh[d + D / 2], x.y);
        put(&fresh[D + d], y.x);
        put(&fresh[D + d + D / 2], y.y);
        if (tile->row >= 0) {
          typename S::T* kc = reinterpret_cast<typename S::T*>(a.k_pool) + (int64_t)tile->row * D;
          typename S::T* vc = reinterpret_cast<typename S::T*>(a.v_pool) + (int64_t)tile->row * D;
          kc[d] = fresh[d];
          kc[d + D / 2] = fresh[d + D / 2];
          vc[d] = fresh[D + d];
          vc[d + D / 2] = fresh[D + d + D / 2];
        }
      }
      if (!meet(&ctrl.met, meetings, a)) break;
      w.open(qf, real);
    }
    bool wrote = false;                 // to the stage
    if (!kRows && seen && seen != (1u << S::KS) - 1) {
      // V rows that are not visible: whatever the page holds there must not
      // meet a probability of zero as a NaN
      for (int e = lane; e < S::KS * S::CH; e += 32)
        if (!(seen >> (e / S::CH) & 1))
          *reinterpret_cast<uint4*>(rows + S::V + S::at(e / S::CH, e % S::CH)) =
              make_uint4(0u, 0u, 0u, 0u);
      wrote = true;
      __syncwarp();
    }
    if (flags & kNew) {
      // in place of what the cache held
      const int r = tile->slot - tile->key0 - warp * S::KS;
      if (r >= 0 && r < S::KS && (seen >> r & 1)) {
        for (int e = lane; e < 2 * S::CH; e += 32)
          *reinterpret_cast<uint4*>(rows + (e < S::CH ? 0 : S::V) + S::at(r, e % S::CH)) =
              reinterpret_cast<const uint4*>(fresh)[e];
        wrote = true;
        __syncwarp();
      }
    }
    if (seen) w.step(rows, seen, c, qf, my_ps);
    if (flags & kLast) {
      // The warps' parts meet in the consumed stage, each thread adding up
      // some pairs of dimensions; the stage is released when all have read.
      __syncwarp();
      w.close(reinterpret_cast<float*>(rows), ctrl.m[turn][warp], ctrl.l[turn][warp], heads);
      wrote = true;
      if (!meet(&ctrl.met, meetings, a)) break;
      const int64_t head0 = (int64_t)tile->b * a.n_heads + tile->hk * a.group + tile->chunk * NH;
      float* part = a.part + (int64_t)tile->part * part_floats(a.unit_heads, D);
      const float* buf = reinterpret_cast<const float*>(ring + stage * S::STAGE);
      for (int e = tid; e < heads * (D / 2); e += 32 * WARPS) {
        const int h = e / (D / 2), d = e % (D / 2) * 2;
        float m = ctrl.m[turn][0][h];
#pragma unroll
        for (int v = 1; v < WARPS; ++v) m = fmaxf(m, ctrl.m[turn][v][h]);
        float x = 0.f, y = 0.f, l = 0.f;
#pragma unroll
        for (int v = 0; v < WARPS; ++v) {
          const float mv = ctrl.m[turn][v][h];
          const float f = mv == -INFINITY ? 0.f : ptx::ex2((mv - m) * c);
          const float2 t = *reinterpret_cast<const float2*>(buf + v * (S::QUARTER / 4) + h * D + d);
          l = fmaf(f, ctrl.l[turn][v][h], l);
          x = fmaf(f, t.x, x);
          y = fmaf(f, t.y, y);
        }
        if (flags & kWhole) {
          const float inv = inverse(l);
          write_out2(a, (head0 + h) * D + d, x * inv, y * inv);
          if (d == 0 && a.lse) a.lse[head0 + h] = lse_of(m * c, l);
        } else {
          *reinterpret_cast<float2*>(part + h * D + d) = make_float2(x, y);
          if (d == 0) {
            part[a.unit_heads * D + h] = m * c;
            part[a.unit_heads * (D + 1) + h] = l;
          }
        }
      }
      turn ^= 1;
    }
    if (wrote) ptx::fence_async_shared();   // before the next tile load into the stage
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&ctrl.empty[stage]);
    if (++stage == S::STAGES) {
      stage = 0;
      phase ^= 1;
    }
  }
}

// Joins (in the order of the shares within a warp, then of the warps) the parts
// of heads whose unit lies in more than one share: JW warps a
// head, each taking every JW-th part, a lane four dimensions.
template <bool kF32, int D, int JW>
__global__ void __launch_bounds__(JT) join_kernel(const DecodeArgs a) {
  using S = Shape<kF32, D>;
  __shared__ float ms[JT / 32], ls[JT / 32];
  __shared__ __align__(16) float4 os[JW > 1 ? JW : 1][JW > 1 ? D / 4 : 1];
  const int tid = threadIdx.x, warp = JW > 1 ? tid >> 5 : 0, lane = tid & 31;
  const int64_t q_head = JW > 1 ? blockIdx.x : (int64_t)blockIdx.x * (JT / 32) + (tid >> 5);
  const bool real = q_head < (int64_t)a.batch * a.n_heads;
  const int b = real ? (int)(q_head / a.n_heads) : 0, head = (int)(q_head - (int64_t)b * a.n_heads);
  const int hk = head / a.group, g = head - hk * a.group;
  const int u = hk * a.head_chunks + g / NH, h = g % NH;
  if (__any_sync(0xffffffffu, ptx::ld_acquire_gpu(a.begun) != kBegun)) ptx::wait_primary();
  int before = 0;
  Window<S::TILE> line;
  line.read(a, 0, 0);
  while (true) {
    const int i = b - line.b0;
    const int upto = __shfl_sync(0xffffffffu, line.base + line.sum - line.n, i & 31);
    if (i >= 0 && i < 32) before = upto;
    if (line.b0 + 32 >= a.batch) break;
    line.read(a, line.b0 + 32, line.end());
  }
  const int total = line.end();
  const int tiles = seq_of<S::TILE>(a, b).tiles;
  const int t0 = before + u * tiles;
  const Shares shares(a, total);
  const int c0 = shares.with(t0), c1 = shares.with(t0 + tiles - 1);
  // the first part is its share's only or last segment, the others are first
  const bool at_front = shares.begin(c0) == t0;
  ptx::wait_primary();
  ptx::launch_dependents();
  if (blockIdx.x == 0 && tid == 0) *a.begun = 0;
  if (!real || c0 == c1) return;        // JW > 1: the same for the whole CTA
  auto part = [&](int c) {
    return a.part + (int64_t)(2 * c + (c == c0 && !at_front ? 1 : 0)) * part_floats(a.unit_heads, D);
  };
  const int m_at = a.unit_heads * D + h, l_at = m_at + a.unit_heads;
  // One pass, four parts at a time (their loads do not wait on one another).
  constexpr int N = 4;
  float m = -INFINITY, l = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float f, const float4& t) {
    x.x = fmaf(f, t.x, x.x);
    x.y = fmaf(f, t.y, x.y);
    x.z = fmaf(f, t.z, x.z);
    x.w = fmaf(f, t.w, x.w);
  };
  for (int c = c0 + warp; c <= c1; c += N * JW) {
    float pm[N], pl[N];
    float4 px[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool in = c + i * JW <= c1;
      const float* p = part(in ? c + i * JW : c);
      pm[i] = in ? p[m_at] : -INFINITY;
      pl[i] = p[l_at];
      px[i] = lane < D / 4 ? *reinterpret_cast<const float4*>(p + h * D + lane * 4)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float mn = fmaxf(fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])), m);
    const float f = m == -INFINITY ? 0.f : ptx::ex2(m - mn);
    m = mn;
    l *= f;
    x.x *= f, x.y *= f, x.z *= f, x.w *= f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (c + i * JW <= c1) {
        // (an empty part adds zeros; one whose scores are all NaN has no maximum
        // either, and its NaN stays)
        const float fi = pm[i] == -INFINITY ? 0.f : ptx::ex2(pm[i] - mn);
        l = fmaf(fi, pl[i], l);
        add(fi, px[i]);
      }
    }
  }
  if constexpr (JW > 1) {
    if (lane == 0) {
      ms[warp] = m;
      ls[warp] = l;
    }
    if (lane < D / 4) os[warp][lane] = x;
    __syncthreads();
    if (warp != 0) return;
    m = ms[0];
#pragma unroll
    for (int w = 1; w < JW; ++w) m = fmaxf(m, ms[w]);
    l = 0.f;
    x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < JW; ++w) {
      const float f = ms[w] == -INFINITY ? 0.f : ptx::ex2(ms[w] - m);
      l = fmaf(f, ls[w], l);
      if (lane < D / 4) add(f, os[w][lane]);
    }
  }
  const float inv = inverse(l);
  if (lane < D / 4) {
    write_out2(a, q_head * D + lane * 4, x.x * inv, x.y * inv);
    write_out2(a, q_head * D + lane * 4 + 2, x.z * inv, x.w * inv);
  }
  if (lane == 0 && a.lse) a.lse[q_head] = lse_of(m, l);
}

// The layer's slice of a pool in 4 dimensions (element of a piece, row of a
// quarter, piece, quarter), in boxes of `box` quarters.
template <bool kF32, int D>
bool encode_pool(CUtensorMap* map, const void* base, uint64_t rows, int box) {
  using S = Shape<kF32, D>;
  EncodeTiledFn fn = get_encode_fn();
  if (!fn) return false;
  constexpr cuuint32_t piece = S::PB / S::SIZE;
  cuuint64_t dims[4] = {piece, S::KS, D / piece, rows / S::KS};
  cuuint64_t strides[3] = {S::ROW, S::PB, S::QUARTER};
  cuuint32_t boxes[4] = {piece, S::KS, D / piece, (cuuint32_t)box};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, kF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<void*>(base), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            S::PB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kF32, int D, int HT, bool kRows>
cudaError_t launch(const DecodeArgs& a, int sms, cudaStream_t stream) {
  using S = Shape<kF32, D>;
  static std::atomic<uint64_t> done{0};
  constexpr int fixed = S::STAGES * S::STAGE + 1024;
  cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(decode_kernel<kF32, D, HT, kRows>),
                              fixed + S::STAGES * ((NH + 2) * D * 4 + D * 8) + NH * S::OROW * 4, done);
  if (e != cudaSuccess) return e;
  DecodeArgs b = a;
  b.box = a.ps.d % (4 * S::KS) == 0 ? 4 : a.ps.d % (2 * S::KS) == 0 ? 2 : 1;
  constexpr int own =
      sizeof(Ctrl<S::STAGES>) + 2 * S::ROW + (kF32 ? HT * S::OROW + WARPS * S::KS * HT : 8) * 4;
  const int rotated = kF32 ? 0 : a.unit_heads * S::OROW * 4;
  const int row = D * (a.in_f32 ? 4 : 2), q_bytes = a.unit_heads * row;
  auto lay_out = [&](bool both) {         // of a slot; whether two CTAs fit an SM
    b.kv_at = both ? q_bytes : 0;
    b.rope_at = q_bytes + (both ? 2 * row : 0);
    b.slot_bytes = b.rope_at + (a.rope_cos ? D * 8 : 0);
    return 2 * (fixed + S::STAGES * b.slot_bytes + rotated + own + 1024) <= 228 * 1024;
  };
  // (One CTA an SM remains for fp32 q of 8 heads a key head at head_dim 128: over a
  // bf16 cache of 8 key heads, 32 sequences of 512 to 2048 slots, 53.0 us instead of
  // the 44.6 of bf16 q, 2 of 60 to 66 thousand 88.3 instead of 84.0; and for fp32
  // caches of 5 to 8 heads.)
  const bool two = lay_out(a.k != nullptr) || lay_out(false);
  b.resident = two ? 2 * sms : sms;
  const int bytes = fixed + S::STAGES * b.slot_bytes + rotated;
  // As many units as CTAs (a switch now and then, at a different pace on every
  // SM): up to four shares a CTA and, since a unit then has few parts, a warp a
  // head to join them: 61.6 us instead of 64.0 for 1024 units of 4 to 16 tiles,
  // 43.9 instead of 46.2 for 320 of 20. Fewer, longer ones: equal shares even out
  // by themselves and leave fewer parts, 64.0 us instead of 68.3 for 160 units of
  // 70 tiles, 158 instead of 191 for 16 of 2000.
  const bool many = (double)a.batch * a.units_per_seq >= b.resident;
  b.ctas = many ? decode_ctas(sms) : b.resident;
  // no more CTAs than the longest possible line has shares for
  const double most = (double)a.batch * a.units_per_seq *
                      (((double)a.max_blocks * a.ps.d + S::TILE - 1) / S::TILE + 1);
  if (most / 8 < b.ctas) b.ctas = most / 8 < b.resident ? b.resident : (int)(most / 8);
  if (most < b.ctas) b.ctas = (int)most;
  b.resident_div = FastDiv::of((uint32_t)b.resident);
  b.ctas_div = FastDiv::of((uint32_t)b.ctas);
  CUtensorMap tk = {}, tv = {};
  const uint64_t rows = (uint64_t)a.num_pages * a.n_kv_heads * a.ps.d;
  if (!kRows && (!encode_pool<kF32, D>(&tk, a.k_pool, rows, b.box) ||
                 !encode_pool<kF32, D>(&tv, a.v_pool, rows, b.box)))
    return cudaErrorInvalidValue;
  e = launch_early(decode_kernel<kF32, D, HT, kRows>, dim3((unsigned)b.ctas),
                   32 * (WARPS + loaders(kRows)), bytes, 1, stream, tk, tv, b);
  if (e != cudaSuccess) return e;
  // (A warp a head needs no shared memory: its CTAs fit beside the last ones
  // above.)
  const unsigned heads = (unsigned)a.batch * (unsigned)a.n_heads;
  if (many)
    return launch_early(join_kernel<kF32, D, 1>, dim3((heads + JT / 32 - 1) / (JT / 32)), JT, 0, 1,
                        stream, b);
  return launch_early(join_kernel<kF32, D, JT / 32>, dim3(heads), JT, 0, 1, stream, b);
}

// fp32 caches: the arithmetic for one, four or eight heads of a key head (one
// of the three is the least that covers the unit; 3 heads at four's cost).
template <int D, bool kRows>
cudaError_t launch_for(const DecodeArgs& a, bool f32, int sms, cudaStream_t stream) {
  if (!f32) return launch<false, D, NH, kRows>(a, sms, stream);
  if (a.group == 1) return launch<true, D, 1, kRows>(a, sms, stream);
  if (a.group <= 4) return launch<true, D, 4, kRows>(a, sms, stream);
  return launch<true, D, NH, kRows>(a, sms, stream);
}

// Tile loads where a page holds whole runs of a quarter's slots, else rows.
template <int D>
cudaError_t launch_for(const DecodeArgs& a, bool f32, int sms, cudaStream_t stream) {
  return a.ps.d % (f32 ? Shape<true, D>::KS : Shape<false, D>::KS) == 0
             ? launch_for<D, false>(a, f32, sms, stream)
             : launch_for<D, true>(a, f32, sms, stream);
}

}  // namespace

int decode_ctas(int sms) { return 8 * sms; }

size_t decode_workspace_bytes(int group, int head_dim, int sms) {
  const int heads = group < NH ? group : NH;
  return (size_t)decode_ctas(sms) * 2 * part_floats(heads, head_dim) * sizeof(float) + 16;
}

cudaError_t launch_decode_attention(const DecodeArgs& a, int head_dim, bool f32, int sms,
                                    cudaStream_t stream) {
  switch (head_dim) {
    case 32: return launch_for<32>(a, f32, sms, stream);
    case 64: return launch_for<64>(a, f32, sms, stream);
    case 96: return launch_for<96>(a, f32, sms, stream);
    case 128: return launch_for<128>(a, f32, sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fdllm

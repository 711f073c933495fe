// What the paged caches' kernels have in common, whatever form their codes have:
// the shape of a cache, the division of attention's work over workgroups, the
// join of shared tiles, and the checks of a call.
//
// A form's attention is a core: a type with
//   Elem, kDim, kRows      the query's type, the head's dims, the rows of a tile
//   kThreads, kResident    threads of a workgroup, and how many of them a CU is to hold
//                          (bounds the registers of a lane)
//   Shared                 its shared memory
//   rows(A, sh, b, h, first, c0, c1, part, stats)
// where rows() computes the rows first .. first + kRows - 1 of request b and
// key/value head h over the chunks c0 .. c1 - 1 by a workgroup; with part null these
// are all the tokens, and the rows are written, else their sums go to part and stats.
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <string>
#include <utility>

#include "xfer.h"

namespace xfer {

void set_error(int code, const std::string& msg);  // conn.cpp

namespace {

int fail(int code, const std::string& msg) {
  set_error(code, msg);
  return code;
}

int hip_fail(hipError_t e, const char* what) {
  set_error(XFER_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
  return XFER_ERR_HIP;
}

template <typename Fn, typename Args>
hipError_t launch(Fn fn, const Args& a, dim3 grid, int block, hipStream_t s) {
  void* kargs[] = {const_cast<Args*>(&a)};
  return hipLaunchKernel(reinterpret_cast<const void*>(fn), grid, dim3(block), kargs, 0, s);
}

// ------------------------------------------------------------------- shape
struct Shape {
  uint64_t block_bytes;
  uint32_t T, H, D, blocks;
  uint32_t log2T;
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16_t;
typedef _Float16 fp16_t;
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 fp16x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------ attend
// A tile of rows whose tokens several workgroups share, from w on to `last`.
struct Begun {
  int32_t request;  // -1: there is none
  uint32_t tile, last, pad;
};

// The same value in every lane, known to the compiler as such.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t uniform(uint64_t v) {
  return static_cast<uint64_t>(uniform(static_cast<uint32_t>(v >> 32))) << 32 |
         uniform(static_cast<uint32_t>(v));
}

struct AttendArgs {
  const uint8_t* cache;
  const void* query;
  void* out;
  float* lse;
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* starts;
  // A launch whose workgroups share the tokens out evenly (flat > 0):
  Begun* begun;     // [flat] the tile that a workgroup begins and does not finish
  float* part;      // [workgroups][2][tile rows][D] sums of weighted values of begun tiles
  float* stats;     // [workgroups][2][tile rows][2] their maxima and sums of weights
  int64_t query_row, query_head, out_row, out_head, table_stride;
  int32_t batch, rows, heads, width;
  uint32_t group;         // query heads of one key/value head
  uint32_t flat;          // workgroups of one key/value head, 0: one per tile of rows
  uint32_t packed;        // tile numbers of one key/value head (flat == 0 and 0: a grid of requests and tiles)
  float scale2;           // scale * log2(e): weights are powers of two
  Shape s;
};

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 fp16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(fp16x8 a, fp16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

constexpr int kAttendWaves = 4;
constexpr int kChunk = 64;  // tokens a wave takes at once

// The rows of one request and key/value head that a workgroup computes.
struct RowTile {
  int64_t start;  // first packed row of the request
  int64_t ahead;  // tokens before its first row's own (negative: rows that see nothing)
  int32_t seen;   // tokens that the tile's last row sees
  uint32_t rows;  // rows times group
};

// Rows of request b that there are (a start below 0 has none).
__device__ __forceinline__ uint32_t rows_of(const AttendArgs& A, uint32_t b) {
  const int64_t start = A.starts[b], end = min<int64_t>(A.starts[b + 1], A.rows);
  return start < 0 || end <= start ? 0u : static_cast<uint32_t>(end - start) * A.group;
}

__device__ __forceinline__ RowTile row_tile(const AttendArgs& A, uint32_t b, uint32_t first,
                                            uint32_t tile_rows) {
  RowTile r;
  r.start = A.starts[b];
  const int64_t queries = static_cast<int64_t>(A.starts[b + 1]) - r.start, length = A.lengths[b];
  const int64_t held = min<int64_t>(length, static_cast<int64_t>(A.width) * A.s.T);
  r.ahead = length - queries;
  r.rows = rows_of(A, b);
  const uint32_t last = min(r.rows, first + tile_rows);
  r.seen = 0;
  if (last > first)
    r.seen = static_cast<int32_t>(
        max<int64_t>(0, min<int64_t>(held, r.ahead + (last - 1) / A.group + 1)));
  r.seen = __builtin_amdgcn_readfirstlane(r.seen);  // (the same in every lane)
  r.rows = __builtin_amdgcn_readfirstlane(r.rows);
  return r;
}

// Request b's tiles of rows and, for each of them, units of work: chunks of
// its tokens (one at least, so that every row is written).  A tile that sees
// fewer tokens has units that hold nothing.
struct Units {
  uint32_t tiles, chunks;
  __device__ uint64_t all() const { return static_cast<uint64_t>(tiles) * chunks; }
};

__device__ __forceinline__ Units units_of(const AttendArgs& A, uint32_t b, uint32_t tile_rows) {
  const int64_t held = min<int64_t>(A.lengths[b], static_cast<int64_t>(A.width) * A.s.T);
  const uint32_t chunks = (static_cast<uint32_t>(max<int64_t>(1, held)) + kChunk - 1) / kChunk;
  return Units{(rows_of(A, b) + tile_rows - 1) / tile_rows, chunks};
}

// A lane's blocks in a chunk: as the holder of scores and values of tokens
// 16g .. (-1: none), and as a loader of key lines (line n is token 16 (n / 4) +
// 4t + n % 4; any block where there is none).
struct Place {
  int32_t mine, line;
  // (seen > 0; the entries of tokens past it are those of the last)
  __device__ __forceinline__ void look(const AttendArgs& A, const int32_t* table, uint32_t t0,
                                       uint32_t seen, uint32_t g, uint32_t n) {
    mine = table[min(t0 + 16 * g, seen - 1) >> A.s.log2T];
    line = table[min(t0 + 16 * (n >> 2), seen - 1) >> A.s.log2T];
  }
  __device__ __forceinline__ void settle(const AttendArgs& A, uint32_t t0, uint32_t seen, uint32_t g) {
    if (static_cast<uint32_t>(mine) >= A.s.blocks || t0 + 16 * g >= seen) mine = -1;
    if (static_cast<uint32_t>(line) >= A.s.blocks) line = 0;
  }
};

// A load of the cache.  ONCE: no other workgroup reads the same bytes, so the caches need not keep them.
template <bool ONCE, typename V>
__device__ __forceinline__ V fetch(const uint8_t* p) {
  if constexpr (ONCE)
    return __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
  else
    return *reinterpret_cast<const V*>(p);
}

// One workgroup per tile of rows and key/value head.  The last tiles see most
// tokens and are begun first: with 32 heads of 128 over 8, 8 requests of 3000 to
// 3900 tokens, 700 to 3000 of them new, take 1290 us and not 1390.
template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kResident) attend_kernel(AttendArgs A) {
  __shared__ typename C::Shared sh;
  const uint32_t h = blockIdx.x % A.s.H, b = blockIdx.x / A.s.H;
  const uint32_t tiles = units_of(A, b, C::kRows).tiles;
  for (uint32_t y = blockIdx.y; y < tiles; y += gridDim.y)
    C::rows(A, sh, b, h, (tiles - 1 - y) * C::kRows, 0, ~0u, nullptr, nullptr);
}

// Tiles numbered through the packed rows: with R rows a tile, request b's begin at
// number first(b) = starts[b] * group / R + b, which leaves it as many as it can
// need.  The request of number k, by a search with a lane per candidate: one trip
// to memory for 64 requests, two for 4096.  (Starts outside the rows count as at
// their ends, as rows_of has it.)
__device__ __forceinline__ uint32_t first_tile(const AttendArgs& A, uint32_t b, uint32_t tile_rows) {
  const uint32_t row = static_cast<uint32_t>(min(max(A.starts[b], 0), A.rows));
  return row * A.group / tile_rows + b;
}

__device__ __forceinline__ uint32_t request_of(const AttendArgs& A, uint32_t k, uint32_t tile_rows) {
  const uint32_t lane = threadIdx.x & 63u;
  uint32_t lo = 0, n = A.batch;
  while (n > 1) {
    const uint32_t step = (n + 63) / 64, at = lane * step;
    const bool there = at < n && first_tile(A, lo + at, tile_rows) <= k;
    const uint32_t pos = max(static_cast<uint32_t>(__popcll(__ballot(there))), 1u) - 1;
    lo += pos * step;
    n = min(step, n - pos * step);
  }
  return uniform(lo);
}

// As attend_kernel, a workgroup per number and key/value head.
template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kResident) attend_packed_kernel(AttendArgs A) {
  constexpr uint32_t kRows = C::kRows;
  __shared__ typename C::Shared sh;
  const uint32_t h = blockIdx.x % A.s.H;
  for (uint32_t k = blockIdx.x / A.s.H; k < A.packed; k += gridDim.x / A.s.H) {
    const uint32_t b = request_of(A, k, kRows), y = uniform(k - first_tile(A, b, kRows));
    const uint32_t tiles = units_of(A, b, kRows).tiles;
    if (y < tiles)  // (a number may be one that its request, or none, does not need)
      C::rows(A, sh, b, h, (tiles - 1 - y) * kRows, 0, ~0u, nullptr, nullptr);
  }
}

// The chunks of all requests and tiles in one line, cut into equal shares for
// as many workgroups per key/value head as the GPU holds: requests of very
// different lengths, or few long ones, keep every CU busy to the end.  Every tile
// of a request counts all of its chunks, those past the tile's last row too:
// shares are even where few rows follow many tokens, while for a whole prompt
// half of the units are skipped, most of them at its front.  A workgroup writes
// the tiles that lie whole in its share and leaves the sums of at most two others,
// the first and the last, to join_kernel.  Every workgroup sums up the requests'
// units for itself.
template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kResident) attend_flat_kernel(AttendArgs A) {
  constexpr uint32_t kThreads = C::kThreads, kWaves = kThreads / 64, kRows = C::kRows;
  __shared__ typename C::Shared sh;
  __shared__ uint64_t s_pre[kThreads], s_wave[kWaves];
  const uint32_t h = blockIdx.x % A.s.H, w = blockIdx.x / A.s.H, tid = threadIdx.x;
  const uint32_t batch = A.batch, seg = (batch + kThreads - 1) / kThreads;
  const uint32_t b0 = min(batch, tid * seg), b1 = min(batch, b0 + seg);
  uint64_t sum = 0;
  for (uint32_t b = b0; b < b1; ++b) sum += units_of(A, b, kRows).all();
  uint64_t run = sum;  // inclusive over the wave's lanes
  for (uint32_t d = 1; d < 64; d <<= 1) {
    const uint64_t o = __shfl_up(static_cast<unsigned long long>(run), d);
    if ((tid & 63u) >= d) run += o;
  }
  if ((tid & 63u) == 63u) s_wave[tid >> 6] = run;
  __syncthreads();
  uint64_t pre = run - sum, all = 0;
  for (uint32_t k = 0; k < kWaves; ++k) {
    if (k < (tid >> 6)) pre += s_wave[k];
    all += s_wave[k];
  }
  s_pre[tid] = pre;
  __syncthreads();
  all = uniform(all);
  const uint64_t flat = min<uint64_t>(A.flat, all);  // (so every share holds a unit)
  if (h == 0 && tid == 0) A.begun[w].request = -1;
  if (w >= flat) return;
  const uint64_t lo = all * w / flat, hi = all * (w + 1) / flat;
  uint32_t first = 0, last = kThreads;  // the last segment that begins at or before lo
  while (last - first > 1) {
    const uint32_t mid = (first + last) / 2;
    if (s_pre[mid] <= lo)
      first = mid;
    else
      last = mid;
  }
  uint32_t b = uniform(first) * seg;
  uint64_t u = lo, at = uniform(s_pre[first]);  // the unit to do, the request's first
  Units q = units_of(A, b, kRows);
  for (;;) {
    while (at + q.all() <= u && b + 1 < batch) {  // (u < all: a request with units follows)
      at = uniform(at + q.all());
      q = units_of(A, ++b, kRows);
    }
    q.chunks = uniform(q.chunks);
    const uint32_t y = uniform(static_cast<uint32_t>((u - at) / q.chunks));
    const uint64_t begin = at + static_cast<uint64_t>(y) * q.chunks, end = begin + q.chunks;
    const uint64_t to = min(hi, end);
    const bool whole = begin >= lo && end <= hi;
    if (end > hi && begin >= lo && h == 0 && tid == 0)
      A.begun[w] = Begun{static_cast<int32_t>(b), y, static_cast<uint32_t>((end * flat - 1) / all), 0};
    const uint32_t slot = (blockIdx.x * 2 + (begin >= lo ? 1 : 0)) * kRows;
    C::rows(A, sh, b, h, y * kRows, static_cast<uint32_t>(u - begin), static_cast<uint32_t>(to - begin),
            whole ? nullptr : A.part + static_cast<uint64_t>(slot) * C::kDim, A.stats + slot * 2);
    u = to;
    if (u == hi) return;
  }
}

constexpr int kJoinThreads = 256;

// Joins the sums of the tiles that several workgroups shared: workgroup (w, h)
// that of the tile which share w begins and later ones go on with, D / 4
// threads for a row, the shares in order, so the result does not depend on
// when they were done.  Bound by latency: 4.6 us behind 64 requests' decode
// step, 9.4 where 2 long ones are spread over 512 workgroups, 6.8 for chunks in tiles of 32
// rows, 15 in tiles of 128.
template <typename E, int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttendArgs A) {
  constexpr uint32_t kWide = D / 4, kGroups = kJoinThreads / kWide, kRows = ROWS;
  const uint32_t w = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, d = tid % kWide;
  const Begun t = A.begun[w];
  if (t.request < 0 || tid >= kGroups * kWide) return;
  const uint32_t rows = rows_of(A, t.request);
  const int64_t start = A.starts[t.request];
  const uint32_t r = blockIdx.z * kGroups + tid / kWide, i = t.tile * kRows + r;
  if (r >= kRows || i >= rows) return;
  // the first share's second place, the later ones' first
  const uint64_t p0 = (static_cast<uint64_t>(w * A.s.H + h) * 2 + 1) * kRows + r;
  const uint64_t step = 2ull * A.s.H * kRows, p1 = p0 - kRows + step;
  float top = -INFINITY, sum = 0.0f;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr uint32_t kTake = 8;  // shares taken together: their loads are in flight at once
  for (uint32_t k0 = 0; k0 <= t.last - w; k0 += kTake) {
    float m[kTake], l[kTake];
    f32x4 v[kTake];
#pragma unroll
    for (uint32_t k = 0; k < kTake; ++k) {
      const bool there = k0 + k <= t.last - w;
      const uint64_t p = k0 + k == 0 || !there ? p0 : p1 + (k0 + k - 1) * step;
      m[k] = there ? A.stats[p * 2] : -INFINITY;
      l[k] = there ? A.stats[p * 2 + 1] : 0.0f;
      v[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (there) v[k] = *reinterpret_cast<const f32x4*>(A.part + p * D + 4 * d);
    }
    const float was = top;
#pragma unroll
    for (uint32_t k = 0; k < kTake; ++k) top = fmaxf(top, m[k]);
    const float base = top == -INFINITY ? 0.0f : top;
    const float keep = __builtin_amdgcn_exp2f(was - base);
    sum *= keep;
    o *= keep;
#pragma unroll
    for (uint32_t k = 0; k < kTake; ++k) {
      const float f = __builtin_amdgcn_exp2f(m[k] - base);
      sum += l[k] * f;
      o += v[k] * f;
    }
  }
  const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
  const int64_t row = start + i / A.group;
  const uint32_t head = h * A.group + i % A.group;
  E v[4];
  for (int k = 0; k < 4; ++k) v[k] = static_cast<E>(o[k] * inv);
  __builtin_memcpy(static_cast<E*>(A.out) + row * A.out_row + head * A.out_head + 4 * d, v, 8);
  if (d == 0 && A.lse)
    A.lse[row * A.heads + head] = (top + __builtin_amdgcn_logf(sum)) * 0.69314718055994531f;
}

using AttendFn = void (*)(AttendArgs);
struct AttendKernels {
  AttendFn attend, packed, flat, join;
  int threads;  // of a workgroup but of join's
};

// The kernels of a core; P: the core of the tiles that are numbered.
template <class C, class P, bool SHARED>
AttendKernels attend_kernels() {
  if constexpr (SHARED)
    return {attend_kernel<C>, attend_packed_kernel<P>, attend_flat_kernel<C>,
            join_kernel<typename C::Elem, C::kDim, C::kRows>, C::kThreads};
  else
    return {attend_kernel<C>, attend_packed_kernel<P>, nullptr, nullptr, C::kThreads};
}

// The launch of a call: rows of a workgroup's tile, and how the work is shared.
struct AttendPlan {
  int tile;
  uint32_t tiles;  // of a request
  uint32_t flat;   // AttendArgs::flat
  uint32_t packed; // AttendArgs::packed
};

constexpr int64_t kEmptyWorkgroups = 16384;

// The workspace: the begun tiles, their sums and the sums' statistics.
struct AttendWork {
  size_t begun, part, stats;
  size_t all() const { return begun + part + stats; }
};

AttendWork attend_work(const Shape& s, const xfer_attend& q, const AttendPlan& p) {
  if (!p.flat) return AttendWork{0, 0, 0};
  const size_t tiles = size_t(p.flat) * s.H * 2 * size_t(p.tile);
  return AttendWork{size_t(p.flat) * sizeof(Begun), tiles * s.D * sizeof(float),
                    tiles * 2 * sizeof(float)};
}

// ------------------------------------------------------------------ checks
constexpr int kMaxHeads = 1024;
constexpr uint64_t kMaxGrid = (1u << 24) - 1;  // workgroups of 256 threads: 2^32 threads at most

int shape_of(const xfer_cache_shape* g, const char* who, Shape* out) {
  if (!g) return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": NULL shape");
  if (g->block_tokens != 16 && g->block_tokens != 32 && g->block_tokens != 64)
    return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": block_tokens must be 16, 32 or 64");
  if (g->kv_heads < 1 || g->kv_heads > kMaxHeads)
    return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": kv_heads must be 1..1024");
  if (g->head_dim != 64 && g->head_dim != 96 && g->head_dim != 128 && g->head_dim != 192 &&
      g->head_dim != 256)
    return fail(XFER_ERR_INVALID_ARG,
                std::string(who) + ": head_dim must be 64, 96, 128, 192 or 256");
  if (g->blocks < 1 || int64_t(g->blocks) * g->block_tokens > 0x7FFFFFFFll)
    return fail(XFER_ERR_INVALID_ARG,
                std::string(who) + ": blocks must be >= 1 and hold at most 2^31 - 1 tokens");
  out->T = uint32_t(g->block_tokens);
  out->log2T = out->T == 16 ? 4 : out->T == 32 ? 5 : 6;
  out->H = uint32_t(g->kv_heads);
  out->D = uint32_t(g->head_dim);
  out->blocks = uint32_t(g->blocks);
  out->block_bytes = 0;  // (of the form of the codes)
  return XFER_OK;
}

// The shape of a cache of 8 bits: codes, and a float pair of scales for each head.
int shape8_of(const xfer_cache_shape* g, const char* who, Shape* out) {
  const int rc = shape_of(g, who, out);
  if (rc) return rc;
  out->block_bytes = 2ull * out->H * out->T * out->D + ((8ull * out->H + 127) & ~127ull);
  return XFER_OK;
}

// Whether vectors of `inner` elements, n0 times n1 of them with strides s0 and s1,
// may share elements: they do not where the vectors of one dimension follow one
// another and those of the other lie behind them all.
bool vectors_overlap(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t inner) {
  typedef __int128 wide;
  wide a = s0 < 0 ? -wide(s0) : wide(s0), b = s1 < 0 ? -wide(s1) : wide(s1);
  if (n0 <= 1 || (n1 > 1 && a > b)) {
    std::swap(n0, n1);
    std::swap(a, b);
  }
  if (n0 <= 1) return false;
  return a < inner || (n1 > 1 && b < a * (n0 - 1) + inner);
}

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// The checks of a call's sizes (s: its shape, checked).
int attend_args(const Shape& s, const xfer_attend* q, const char* who) {
  if (!q) return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": NULL arguments");
  if (q->batch < 0 || q->rows < 0 || q->table_width < 0 || q->table_stride < q->table_width)
    return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": need batch, rows and table_width >= 0 "
                                                         "and table_stride >= table_width");
  if (q->heads < 1 || q->heads > 16 * kMaxHeads || uint32_t(q->heads) % s.H)
    return fail(XFER_ERR_INVALID_ARG,
                std::string(who) + ": heads must be a multiple of kv_heads, at most 16384");
  if (int64_t(q->rows) * q->heads > 0x7FFFFFFFll)
    return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": rows * heads must stay below 2^31");
  if (uint64_t(q->batch) * uint64_t(s.H) > kMaxGrid)
    return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": batch * kv_heads must stay below 2^24");
  if (q->dtype != XFER_BF16 && q->dtype != XFER_FP16)
    return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": dtype must be BF16 or FP16");
  if (!(q->scale > 0.0f) || !(q->scale <= 3.402823466e38f))
    return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": scale must be positive and finite");
  if (q->max_query < 0 || q->max_length < 0)
    return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": max_query and max_length must be >= 0");
  return XFER_OK;
}

// A call of attention: its checks, its workspace, its launches.  p: the launch's shape;
// pick(dtype, p): its kernels.
template <typename Pick>
int attend_call(const Shape& s, const void* cache, const xfer_attend* q, const AttendPlan& p, Pick pick,
                void* stream, const char* who) {
  if (!cache || !q->query || !q->out || !q->lengths || !q->starts ||
      (q->table_width > 0 && !q->table))
    return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": NULL buffer with rows to compute");
  if (!aligned(cache, 16) || !aligned(q->query, 2) || !aligned(q->out, 2) || !aligned(q->lse, 4) ||
      !aligned(q->table, 4) || !aligned(q->lengths, 4) || !aligned(q->starts, 4))
    return fail(XFER_ERR_INVALID_ARG,
                std::string(who) + ": the cache must be 16-byte aligned, the others by their type");
  if (vectors_overlap(q->rows, q->out_row, q->heads, q->out_head, s.D))
    return fail(XFER_ERR_INVALID_ARG,
                std::string(who) + ": the rows and heads of out must not overlap");
  AttendArgs a;
  a.s = s;
  a.cache = static_cast<const uint8_t*>(cache);
  a.query = q->query;
  a.out = q->out;
  a.lse = q->lse;
  a.table = q->table;
  a.lengths = q->lengths;
  a.starts = q->starts;
  a.query_row = q->query_row;
  a.query_head = q->query_head;
  a.out_row = q->out_row;
  a.out_head = q->out_head;
  a.table_stride = q->table_stride;
  a.batch = q->batch;
  a.rows = q->rows;
  a.heads = q->heads;
  a.width = q->table_width;
  a.group = uint32_t(q->heads) / a.s.H;
  a.scale2 = q->scale * 1.44269504088896341f;
  a.flat = p.flat;
  a.packed = p.packed;
  const AttendWork work = attend_work(a.s, *q, p);
  if (p.flat && (!q->workspace || q->workspace_bytes < work.all() || !aligned(q->workspace, 16)))
    return fail(XFER_ERR_INVALID_ARG,
                std::string(who) + ": the workspace must hold " + who + "_workspace() bytes, 16-byte aligned");
  uint8_t* mem = static_cast<uint8_t*>(q->workspace);
  a.begun = reinterpret_cast<Begun*>(mem);
  a.part = reinterpret_cast<float*>(mem + work.begun);
  a.stats = reinterpret_cast<float*>(mem + work.begun + work.part);
  const AttendKernels k = pick(q->dtype, p);
  const hipStream_t on = static_cast<hipStream_t>(stream);
  hipError_t e;
  if (p.flat) {
    e = launch(k.flat, a, dim3(p.flat * a.s.H), k.threads, on);
    if (e == hipSuccess) {
      const uint32_t rows = uint32_t(kJoinThreads) / (a.s.D / 4);  // of a join workgroup
      e = launch(k.join, a, dim3(p.flat, a.s.H, (uint32_t(p.tile) + rows - 1) / rows), kJoinThreads, on);
    }
  } else if (p.packed) {
    const uint64_t most = kMaxGrid * 256 / uint64_t(k.threads) / a.s.H;
    e = launch(k.packed, a, dim3(uint32_t(std::min<uint64_t>(p.packed, most)) * a.s.H), k.threads, on);
  } else {
    e = launch(k.attend, a, dim3(uint32_t(q->batch) * a.s.H, p.tiles), k.threads, on);
  }
  if (e != hipSuccess) return hip_fail(e, (std::string(who) + " launch").c_str());
  return XFER_OK;
}

}  // namespace
}  // namespace xfer

// gfx950 kernels of the paged 8-bit cache: block plans, stores and attention.
// Their entry points (xfer_cache_*) are at the end of the file.
//
// A cache is a pool of blocks, each one record of bytes that a connection can
// move as it is (xfer_run_blocks): per key/value head the key codes [T][D],
// then the value codes [D][T], and behind the heads a float pair of scales per
// head, padded to 128 bytes.  A code is an e4m3 number and stands for code x
// scale, a power of two: dequantising and rescaling by it are exact, and an
// e4m3 number, which has an exponent of its own, gains nothing from a finer
// scale.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <string>

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
  __device__ uint64_t key_at(uint32_t block, uint32_t h) const {
    return block * block_bytes + static_cast<uint64_t>(2u * h) * T * D;
  }
  __device__ uint64_t value_at(uint32_t block, uint32_t h) const {
    return key_at(block, h) + static_cast<uint64_t>(T) * D;
  }
  __device__ uint64_t scales_at(uint32_t block, uint32_t h) const {
    return block * block_bytes + 2ull * H * T * D + 8u * h;
  }
};

// -------------------------------------------------------------------- plan
struct PlanArgs {
  const int32_t* cached;
  const int32_t* added;
  int32_t* table;
  const int32_t* free_blocks;
  int32_t* slots;
  int32_t* positions;
  int32_t* starts;
  int32_t* lengths;
  int32_t* counts;
  int64_t table_stride;
  int32_t batch, width, nfree, T, rows, per_wg;
};

constexpr int kPlanThreads = 256;
constexpr int kPlanEach = 4;  // requests a thread scans
constexpr int kPlanTile = kPlanThreads * kPlanEach;

// Largest i in [0, n) with a[i] <= x; a[0] <= x.
__device__ __forceinline__ int last_at_most(const int64_t* a, int n, int64_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Request i holds held_i = ceil(cached_i / T) blocks and needs
// ceil((cached_i + added_i) / T); with f_i and s_i the sums of the new blocks
// and of the added tokens over the requests before it, new block k of i is
// free_blocks[f_i + k], and its token j is packed row s_i + j.
//
// One launch and no word passes between workgroups: every workgroup scans all
// requests, a tile of 1024 at a time, and serves its own range of rows and its
// own share of new blocks by a search in the scanned sums.  The lengths are a
// few KiB that every workgroup finds in the L2, so scanning them again costs
// less than a second launch or a hand-off would.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs A) {
  __shared__ int64_t s_tok[kPlanTile + 1], s_blk[kPlanTile + 1];
  __shared__ int32_t s_cached[kPlanTile];
  __shared__ int64_t w_tok[kPlanThreads / 64], w_blk[kPlanThreads / 64], w_lost[kPlanThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t T = A.T;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * A.per_wg;
  const int64_t row1 = min<int64_t>(A.rows, row0 + A.per_wg);
  int64_t carry_tok = 0, carry_blk = 0, lost = 0;
  for (int b0 = 0; b0 < A.batch; b0 += kPlanTile) {
    const int cnt = min(kPlanTile, A.batch - b0);
    int64_t tok[kPlanEach], blk[kPlanEach], sum_tok = 0, sum_blk = 0;
#pragma unroll
    for (int i = 0; i < kPlanEach; ++i) {
      const int r = tid * kPlanEach + i;
      const int64_t c = r < cnt ? max(A.cached[b0 + r], 0) : 0;
      const int64_t a = r < cnt ? max(A.added[b0 + r], 0) : 0;
      s_cached[r] = static_cast<int32_t>(c);
      tok[i] = sum_tok;
      blk[i] = sum_blk;
      sum_tok += a;
      sum_blk += (c + a + T - 1) / T - (c + T - 1) / T;
    }
    int64_t inc_tok = sum_tok, inc_blk = sum_blk;  // inclusive over the wave's lanes
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t t = __shfl_up(inc_tok, d), k = __shfl_up(inc_blk, d);
      if (lane >= d) {
        inc_tok += t;
        inc_blk += k;
      }
    }
    if (lane == 63) {
      w_tok[wave] = inc_tok;
      w_blk[wave] = inc_blk;
    }
    __syncthreads();
    int64_t at_tok = carry_tok + inc_tok - sum_tok, at_blk = carry_blk + inc_blk - sum_blk;
    for (int w = 0; w < wave; ++w) {
      at_tok += w_tok[w];
      at_blk += w_blk[w];
    }
#pragma unroll
    for (int i = 0; i < kPlanEach; ++i) {
      s_tok[tid * kPlanEach + i] = at_tok + tok[i];
      s_blk[tid * kPlanEach + i] = at_blk + blk[i];
    }
    for (int w = 0; w < kPlanThreads / 64; ++w) {
      carry_tok += w_tok[w];
      carry_blk += w_blk[w];
    }
    if (tid == 0) {
      s_tok[kPlanTile] = carry_tok;
      s_blk[kPlanTile] = carry_blk;
    }
    __syncthreads();
    // (entries past cnt repeat the totals, so [i + 1] is right for every request)
    if (blockIdx.x == 0) {
      for (int i = tid; i < cnt; i += kPlanThreads) {
        const int64_t c = s_cached[i], len = c + s_tok[i + 1] - s_tok[i];
        const int64_t held = (c + T - 1) / T;
        A.starts[b0 + i] = static_cast<int32_t>(s_tok[i]);
        A.lengths[b0 + i] = static_cast<int32_t>(len);
        const int64_t reach = min<int64_t>(A.width, held + max<int64_t>(0, A.nfree - s_blk[i]));
        lost += max<int64_t>(0, len - max<int64_t>(c, reach * T));
      }
    }
    // new blocks
    for (int64_t x = s_blk[0] + static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;
         x < min<int64_t>(carry_blk, A.nfree); x += static_cast<int64_t>(gridDim.x) * kPlanThreads) {
      const int i = last_at_most(s_blk, cnt, x);
      const int64_t page = (s_cached[i] + T - 1) / T + x - s_blk[i];
      if (page < A.width) A.table[(b0 + i) * A.table_stride + page] = A.free_blocks[x];
    }
    // rows
    for (int64_t n = max(row0, s_tok[0]) + tid; n < min(row1, carry_tok); n += kPlanThreads) {
      const int i = last_at_most(s_tok, cnt, n);
      const int64_t pos = s_cached[i] + n - s_tok[i], page = pos / T;
      const int64_t held = (s_cached[i] + T - 1) / T, take = s_blk[i] + page - held;
      int64_t id = -1;
      if (page < A.width) {
        if (page < held)
          id = A.table[(b0 + i) * A.table_stride + page];
        else if (take < A.nfree)
          id = A.free_blocks[take];
      }
      const int64_t slot = id < 0 ? -1 : id * T + pos % T;
      A.slots[n] = slot > 0x7FFFFFFF ? -1 : static_cast<int32_t>(slot);
      A.positions[n] = static_cast<int32_t>(pos);
    }
    __syncthreads();
  }
  for (int64_t n = max(row0, carry_tok) + tid; n < row1; n += kPlanThreads) {
    A.slots[n] = -1;
    A.positions[n] = -1;
  }
  if (blockIdx.x == 0) {
    for (int d = 1; d < 64; d <<= 1) lost += __shfl_xor(lost, d);
    if (lane == 0) w_lost[wave] = lost;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kPlanThreads / 64; ++w) lost += w_lost[w];
      A.starts[A.batch] = static_cast<int32_t>(carry_tok);
      A.counts[0] = static_cast<int32_t>(carry_blk);
      A.counts[1] = static_cast<int32_t>(lost);
    }
  }
}

// ------------------------------------------------------------------- store
struct StoreArgs {
  uint8_t* cache;
  const void* key;
  const void* value;
  int64_t key_row, key_head, value_row, value_head;  // strides in elements
  const int32_t* slots;
  int32_t rows;
  Shape s;
};

typedef __bf16 bf16_t;
typedef _Float16 fp16_t;

// Smallest power of two, 2^-118 at least, that brings amax (finite) to 448 =
// 1.75 * 2^8 or below.  amax = (1 + m / 2^23) * 2^(x - 127) from its bits; a
// subnormal amax falls under the floor.
__device__ __forceinline__ float scale_of(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, -118) + 127) << 23);
}

// The reciprocal of a power of two within 2^-118 .. 2^120.
__device__ __forceinline__ float power_inverse(float s) {
  return __uint_as_float((254u << 23) - __float_as_uint(s));
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.0f;  // infinities and NaN count for nothing
}

// Nearest e4m3 code of x (|x| <= 448 but for rounding errors of none: the
// scale is a power of two); what is not finite becomes NaN.
__device__ __forceinline__ uint8_t code_of(float x) {
  if (!(fabsf(x) <= 448.0f)) return 0x7F;
  return static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(x, 0.0f, 0, false));
}

__device__ __forceinline__ float value_of(uint8_t c) {
  return __builtin_amdgcn_cvt_f32_fp8(c, 0);
}

constexpr int kStoreThreads = 128;

// A run is the rows that fall into one block: consecutive slots that do not
// pass its end.  The workgroup of a run's first row and one head finds the
// largest magnitude of the run's keys (values), settles the block's scale,
// rounds the earlier tokens' codes again if it grew and writes the run's.
template <typename E>
__global__ void __launch_bounds__(kStoreThreads) store_kernel(StoreArgs A) {
  __shared__ float s_max[kStoreThreads / 64];
  const int32_t n = blockIdx.x;
  const uint32_t h = blockIdx.y, T = A.s.T, D = A.s.D, tid = threadIdx.x;
  const int32_t slot = A.slots[n];
  if (slot < 0 || static_cast<uint32_t>(slot) / T >= A.s.blocks) return;
  const uint32_t block = static_cast<uint32_t>(slot) / T, off = static_cast<uint32_t>(slot) % T;
  if (off > 0 && n > 0 && A.slots[n - 1] == slot - 1) return;
  uint32_t cnt = 1;
  while (n + static_cast<int32_t>(cnt) < A.rows && off + cnt < T &&
         A.slots[n + cnt] == slot + static_cast<int32_t>(cnt))
    ++cnt;
  for (int side = 0; side < 2; ++side) {
    const E* src = side ? static_cast<const E*>(A.value) + n * A.value_row + h * A.value_head
                        : static_cast<const E*>(A.key) + n * A.key_row + h * A.key_head;
    const int64_t row = side ? A.value_row : A.key_row;
    uint8_t* codes = A.cache + (side ? A.s.value_at(block, h) : A.s.key_at(block, h));
    float* held = reinterpret_cast<float*>(A.cache + A.s.scales_at(block, h)) + side;
    const uint32_t st = side ? 1u : D, sd = side ? T : 1u;  // code strides of a token and a dim
    float amax = 0.0f;
    for (uint32_t i = tid; i < cnt * D; i += kStoreThreads)
      amax = fmaxf(amax, finite_abs(static_cast<float>(src[(i / D) * row + i % D])));
    for (int d = 1; d < 64; d <<= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
    __syncthreads();
    if ((tid & 63u) == 0) s_max[tid >> 6] = amax;
    __syncthreads();
    for (int w = 0; w < kStoreThreads / 64; ++w) amax = fmaxf(amax, s_max[w]);
    float scale = scale_of(amax);
    if (off > 0) {
      const float was = *held;
      if (scale > was) {
        const float f = was * power_inverse(scale);
        for (uint32_t i = tid; i < off * D; i += kStoreThreads) {
          uint8_t* c = codes + (i / D) * st + (i % D) * sd;
          *c = code_of(value_of(*c) * f);
        }
      } else {
        scale = was;
      }
    }
    const float inv = power_inverse(scale);
    for (uint32_t i = tid; i < cnt * D; i += kStoreThreads)
      codes[(off + i / D) * st + (i % D) * sd] =
          code_of(static_cast<float>(src[(i / D) * row + i % D]) * inv);
    __syncthreads();  // every thread has read the old scale
    if (tid == 0) *held = scale;
  }
}

// ------------------------------------------------------------------ attend
struct AttendArgs {
  const uint8_t* cache;
  const void* query;
  void* out;
  float* lse;
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* starts;
  int64_t query_row, query_head, out_row, out_head, table_stride;
  int32_t batch, rows, heads, width;
  float scale;
  Shape s;
};

constexpr int kAttendThreads = 256;

// Row n of request b sees the tokens 0 .. length_b - (rows of b) + its place.
// One workgroup per row and head, tokens in chunks of a thread each, with a
// running maximum m and sum l: o = sum p v / l, p = exp(score - m).
template <typename E>
__global__ void __launch_bounds__(kAttendThreads) attend_kernel(AttendArgs A) {
  __shared__ float s_q[256], s_p[kAttendThreads], s_red[kAttendThreads / 64];
  __shared__ int64_t s_block[kAttendThreads];
  const int32_t n = blockIdx.x;
  const uint32_t hq = blockIdx.y, T = A.s.T, D = A.s.D, tid = threadIdx.x;
  const uint32_t h = hq / (A.heads / A.s.H);
  int lo = 0, hi = A.batch;  // last request that starts at or before n
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (A.starts[mid] <= n) lo = mid; else hi = mid;
  }
  const int32_t r0 = A.starts[lo], r1 = A.starts[lo + 1];
  if (n < r0 || n >= r1) return;  // a row of no request
  const int64_t len = min<int64_t>(max(A.lengths[lo], 0), static_cast<int64_t>(A.width) * T);
  const int64_t seen = min<int64_t>(len, static_cast<int64_t>(A.lengths[lo]) - (r1 - r0) + (n - r0) + 1);
  const E* q = static_cast<const E*>(A.query) + n * A.query_row + hq * A.query_head;
  if (tid < D) s_q[tid] = static_cast<float>(q[tid]);
  float m = -INFINITY, l = 0.0f, acc = 0.0f;
  for (int64_t t0 = 0; t0 < seen; t0 += kAttendThreads) {
    const int64_t t = t0 + tid;
    int64_t block = -1;
    if (t < seen) {
      const int32_t id = A.table[lo * A.table_stride + t / T];
      if (static_cast<uint32_t>(id) < A.s.blocks) block = id;
    }
    __syncthreads();
    float x = -INFINITY;
    if (block >= 0) {
      const uint8_t* k = A.cache + A.s.key_at(block, h) + (t % T) * D;
      const float ks = *reinterpret_cast<const float*>(A.cache + A.s.scales_at(block, h));
      x = 0.0f;
      for (uint32_t d = 0; d < D; ++d) x += s_q[d] * value_of(k[d]);
      x *= ks * A.scale;
    }
    s_block[tid] = block;
    float top = x;
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    if ((tid & 63u) == 0) s_red[tid >> 6] = top;
    __syncthreads();
    for (int w = 0; w < kAttendThreads / 64; ++w) top = fmaxf(top, s_red[w]);
    top = fmaxf(m, top);
    const float base = top == -INFINITY ? 0.0f : top;
    const float keep = expf(m - base);
    m = top;
    const float p = block >= 0 ? expf(x - base) : 0.0f;
    s_p[tid] = p;
    __syncthreads();
    l *= keep;
    acc *= keep;
    const int cnt = static_cast<int>(min<int64_t>(kAttendThreads, seen - t0));
    for (int i = 0; i < cnt; ++i) {
      if (s_block[i] < 0) continue;
      l += s_p[i];
      if (tid < D) {
        const uint8_t* v = A.cache + A.s.value_at(s_block[i], h);
        const float vs = *reinterpret_cast<const float*>(A.cache + A.s.scales_at(s_block[i], h) + 4);
        acc += s_p[i] * value_of(v[tid * T + (t0 + i) % T]) * vs;
      }
    }
  }
  E* o = static_cast<E*>(A.out) + n * A.out_row + hq * A.out_head;
  if (tid < D) o[tid] = static_cast<E>(l != 0.0f ? acc / l : 0.0f);
  if (tid == 0 && A.lse) A.lse[static_cast<int64_t>(n) * A.heads + hq] = m + logf(l);
}

// ------------------------------------------------------------------ checks
constexpr int kMaxHeads = 1024;

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
  out->H = uint32_t(g->kv_heads);
  out->D = uint32_t(g->head_dim);
  out->blocks = uint32_t(g->blocks);
  out->block_bytes = 2ull * out->H * out->T * out->D + ((8ull * out->H + 127) & ~127ull);
  return XFER_OK;
}

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

}  // namespace
}  // namespace xfer

using namespace xfer;

extern "C" int xfer_cache_block_bytes(const xfer_cache_shape* shape, size_t* bytes) {
  Shape s;
  const int rc = shape_of(shape, "xfer_cache_block_bytes", &s);
  if (rc) return rc;
  if (!bytes) return fail(XFER_ERR_INVALID_ARG, "xfer_cache_block_bytes: NULL bytes");
  *bytes = size_t(s.block_bytes);
  return XFER_OK;
}

extern "C" int xfer_cache_plan(const int32_t* cached, const int32_t* added, int batch,
                               int32_t* table, int64_t table_stride, int table_width,
                               const int32_t* free_blocks, int nfree, int block_tokens,
                               int32_t* slots, int32_t* positions, int rows, int32_t* starts,
                               int32_t* lengths, int32_t* counts, void* stream) {
  if (batch < 0 || rows < 0 || nfree < 0 || table_width < 0 || table_stride < table_width)
    return fail(XFER_ERR_INVALID_ARG,
                "xfer_cache_plan: need batch, rows, nfree and table_width >= 0 and table_stride >= "
                "table_width");
  if (block_tokens != 16 && block_tokens != 32 && block_tokens != 64)
    return fail(XFER_ERR_INVALID_ARG, "xfer_cache_plan: block_tokens must be 16, 32 or 64");
  if (!starts || !counts || (batch > 0 && (!cached || !added || !lengths)) ||
      (batch > 0 && table_width > 0 && !table) || (nfree > 0 && !free_blocks) ||
      (rows > 0 && (!slots || !positions)))
    return fail(XFER_ERR_INVALID_ARG, "xfer_cache_plan: NULL array");
  for (const void* p : {static_cast<const void*>(cached), static_cast<const void*>(added),
                        static_cast<const void*>(table), static_cast<const void*>(free_blocks),
                        static_cast<const void*>(slots), static_cast<const void*>(positions),
                        static_cast<const void*>(starts), static_cast<const void*>(lengths),
                        static_cast<const void*>(counts)})
    if (!aligned(p, 4))
      return fail(XFER_ERR_INVALID_ARG, "xfer_cache_plan: arrays must be 4-byte aligned");
  PlanArgs a{cached, added,  table,  free_blocks,  slots, positions,   starts, lengths,
             counts, table_stride, batch, table_width, nfree, block_tokens, rows,  0};
  // About 1024 rows or 256 requests a workgroup.
  const int grid = std::max(1, std::min(1024, std::max((rows + 1023) / 1024, (batch + 255) / 256)));
  a.per_wg = (rows + grid - 1) / grid;
  const hipError_t e =
      launch(plan_kernel, a, dim3(uint32_t(grid)), kPlanThreads, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "xfer_cache_plan launch");
  return XFER_OK;
}

extern "C" int xfer_cache_store(const xfer_cache_shape* shape, void* cache, const void* key,
                                int64_t key_row, int64_t key_head, const void* value,
                                int64_t value_row, int64_t value_head, int dtype,
                                const int32_t* slots, int rows, void* stream) {
  StoreArgs a;
  const int rc = shape_of(shape, "xfer_cache_store", &a.s);
  if (rc) return rc;
  if (dtype != XFER_BF16 && dtype != XFER_FP16 && dtype != XFER_FP32)
    return fail(XFER_ERR_INVALID_ARG, "xfer_cache_store: unknown dtype");
  if (rows < 0) return fail(XFER_ERR_INVALID_ARG, "xfer_cache_store: rows must be >= 0");
  if (rows == 0) return XFER_OK;
  if (!cache || !key || !value || !slots)
    return fail(XFER_ERR_INVALID_ARG, "xfer_cache_store: NULL buffer with rows to store");
  const size_t size = dtype == XFER_FP32 ? 4 : 2;
  if (!aligned(cache, 16) || !aligned(slots, 4) || !aligned(key, size) || !aligned(value, size))
    return fail(XFER_ERR_INVALID_ARG,
                "xfer_cache_store: the cache must be 16-byte aligned, the others by their type");
  a.cache = static_cast<uint8_t*>(cache);
  a.key = key;
  a.value = value;
  a.key_row = key_row;
  a.key_head = key_head;
  a.value_row = value_row;
  a.value_head = value_head;
  a.slots = slots;
  a.rows = rows;
  const dim3 grid(uint32_t(rows), a.s.H);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = dtype == XFER_BF16   ? launch(store_kernel<bf16_t>, a, grid, kStoreThreads, s)
                       : dtype == XFER_FP16 ? launch(store_kernel<fp16_t>, a, grid, kStoreThreads, s)
                                            : launch(store_kernel<float>, a, grid, kStoreThreads, s);
  if (e != hipSuccess) return hip_fail(e, "xfer_cache_store launch");
  return XFER_OK;
}

namespace {

int attend_args(const xfer_cache_shape* shape, const xfer_attend* q, const char* who, Shape* s) {
  const int rc = shape_of(shape, who, s);
  if (rc) return rc;
  if (!q) return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": NULL arguments");
  if (q->batch < 0 || q->rows < 0 || q->table_width < 0 || q->table_stride < q->table_width)
    return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": need batch, rows and table_width >= 0 "
                                                         "and table_stride >= table_width");
  if (q->heads < 1 || q->heads > 16 * kMaxHeads || q->heads % shape->kv_heads)
    return fail(XFER_ERR_INVALID_ARG,
                std::string(who) + ": heads must be a multiple of kv_heads, at most 16384");
  if (q->dtype != XFER_BF16 && q->dtype != XFER_FP16)
    return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": dtype must be BF16 or FP16");
  if (!(q->scale > 0.0f) || !(q->scale <= 3.402823466e38f))
    return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": scale must be positive and finite");
  if (q->max_query < 0 || q->max_length < 0)
    return fail(XFER_ERR_INVALID_ARG, std::string(who) + ": max_query and max_length must be >= 0");
  return XFER_OK;
}

}  // namespace

extern "C" int xfer_cache_attend_workspace(const xfer_cache_shape* shape, const xfer_attend* q,
                                           size_t* bytes) {
  Shape s;
  const int rc = attend_args(shape, q, "xfer_cache_attend_workspace", &s);
  if (rc) return rc;
  if (!bytes) return fail(XFER_ERR_INVALID_ARG, "xfer_cache_attend_workspace: NULL bytes");
  *bytes = 0;
  return XFER_OK;
}

extern "C" int xfer_cache_attend(const xfer_cache_shape* shape, const void* cache,
                                 const xfer_attend* q, void* stream) {
  AttendArgs a;
  const int rc = attend_args(shape, q, "xfer_cache_attend", &a.s);
  if (rc) return rc;
  if (q->rows == 0 || q->batch == 0) return XFER_OK;
  if (!cache || !q->query || !q->out || !q->lengths || !q->starts ||
      (q->table_width > 0 && !q->table))
    return fail(XFER_ERR_INVALID_ARG, "xfer_cache_attend: NULL buffer with rows to compute");
  if (!aligned(cache, 16) || !aligned(q->query, 2) || !aligned(q->out, 2) || !aligned(q->lse, 4) ||
      !aligned(q->table, 4) || !aligned(q->lengths, 4) || !aligned(q->starts, 4))
    return fail(XFER_ERR_INVALID_ARG,
                "xfer_cache_attend: the cache must be 16-byte aligned, the others by their type");
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
  a.scale = q->scale;
  const dim3 grid(uint32_t(q->rows), uint32_t(q->heads));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = q->dtype == XFER_BF16
                           ? launch(attend_kernel<bf16_t>, a, grid, kAttendThreads, s)
                           : launch(attend_kernel<fp16_t>, a, grid, kAttendThreads, s);
  if (e != hipSuccess) return hip_fail(e, "xfer_cache_attend launch");
  return XFER_OK;
}

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
#include "cache_common.h"

#include <math.h>
#include <string.h>

#include <type_traits>

namespace xfer {
namespace {

// -------------------------------------------------------------------- form
__device__ __forceinline__ uint64_t key_at(const Shape& s, uint32_t block, uint32_t h) {
  return block * s.block_bytes + static_cast<uint64_t>(2u * h) * s.T * s.D;
}
__device__ __forceinline__ uint64_t value_at(const Shape& s, uint32_t block, uint32_t h) {
  return key_at(s, block, h) + static_cast<uint64_t>(s.T) * s.D;
}
__device__ __forceinline__ uint64_t scales_at(const Shape& s, uint32_t block, uint32_t h) {
  return block * s.block_bytes + 2ull * s.H * s.T * s.D + 8u * h;
}

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
// own share of new blocks by a search in the scanned sums; the last one writes
// what belongs to requests and counts instead.  The lengths are a
// few KiB that every workgroup finds in the L2, so scanning them again costs
// less than a second launch or a hand-off would.  Bound by the chain lengths ->
// scan -> search -> stores: 5.3 us for 64 requests of a token, 11 for 1000
// prompts of 1 to 1200 tokens (a launch that does nothing: 3.6).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs A) {
  __shared__ int64_t s_tok[kPlanTile + 1], s_blk[kPlanTile + 1];
  __shared__ int32_t s_cached[kPlanTile];
  __shared__ int64_t w_tok[kPlanThreads / 64], w_blk[kPlanThreads / 64], w_lost[kPlanThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t T = A.T;
  const uint32_t servers = gridDim.x - 1;
  const bool books = blockIdx.x == servers;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * A.per_wg;
  const int64_t row1 = books ? row0 : min<int64_t>(A.rows, row0 + A.per_wg);
  int64_t carry_tok = 0, carry_blk = 0, lost = 0;
  for (int64_t b0 = 0; b0 < A.batch; b0 += kPlanTile) {
    const int cnt = static_cast<int>(min<int64_t>(kPlanTile, A.batch - b0));
    int64_t tok[kPlanEach], blk[kPlanEach], sum_tok = 0, sum_blk = 0;
    // The block that a request's last token is in, where its new ones go on with
    // it, and how many do: lost too if the table lacks it.
    int32_t last[kPlanEach], more[kPlanEach];
#pragma unroll
    for (int i = 0; i < kPlanEach; ++i) {
      const int r = tid * kPlanEach + i;
      const int64_t c = r < cnt ? max(A.cached[b0 + r], 0) : 0;
      const int64_t a = r < cnt ? max(A.added[b0 + r], 0) : 0;
      s_cached[r] = static_cast<int32_t>(c);
      const int64_t held = (c + T - 1) / T;
      last[i] = 0;
      more[i] = static_cast<int32_t>(min(a, held * T - c));
      if (books && more[i] > 0 && held <= A.width)
        last[i] = A.table[(b0 + r) * A.table_stride + held - 1];  // (no workgroup writes held entries)
      tok[i] = sum_tok;
      blk[i] = sum_blk;
      sum_tok += a;
      sum_blk += (c + a + T - 1) / T - held;
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
    if (books) {
      for (int i = tid; i < cnt; i += kPlanThreads) {
        const int64_t c = s_cached[i], len = c + s_tok[i + 1] - s_tok[i];
        const int64_t held = (c + T - 1) / T;
        A.starts[b0 + i] = static_cast<int32_t>(s_tok[i]);
        A.lengths[b0 + i] = static_cast<int32_t>(len);
        const int64_t reach = min<int64_t>(A.width, held + max<int64_t>(0, A.nfree - s_blk[i]));
        lost += max<int64_t>(0, len - max<int64_t>(c, reach * T));
      }
#pragma unroll
      for (int i = 0; i < kPlanEach; ++i)
        if (last[i] < 0) lost += more[i];
      __syncthreads();
      continue;
    }
    // new blocks
    for (int64_t x = s_blk[0] + static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;
         x < min<int64_t>(carry_blk, A.nfree); x += static_cast<int64_t>(servers) * kPlanThreads) {
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
  if (books) {
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
  uint32_t tile, wg_heads;  // rows whose runs, and heads, a workgroup looks after
  Shape s;
};

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

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Element j of eight packed in words.
template <typename E>
__device__ __forceinline__ float element(const uint32_t* w, uint32_t j) {
  if constexpr (sizeof(E) == 4) {
    return __uint_as_float(w[j]);
  } else {
    const uint16_t b = static_cast<uint16_t>(w[j / 2] >> (16 * (j % 2)));
    return static_cast<float>(__builtin_bit_cast(E, b));
  }
}

// Bits of the 16-bit types' infinity: the magnitudes' bits are ordered as they
// are, those that are not finite last.
template <typename E>
constexpr uint32_t infinity_bits() {
  return __is_same(E, bf16_t) ? 0x7F80u : 0x7C00u;
}

// Groups of four places that a wave holds at once.
constexpr uint32_t store_groups(int d, int t) {
  const uint32_t fit = d <= 64 ? 8 : d <= 128 ? 4 : 2, all = t / 4;
  return fit < all ? fit : all;
}

constexpr int kStoreWaves = 4;

__device__ __forceinline__ float wave_max(float x) {
  for (int d = 1; d < 64; d <<= 1) x = fmaxf(x, __shfl_xor(x, d));
  return x;
}

typedef int16_t i16x2 __attribute__((ext_vector_type(2)));

// The codes of elements 4q .. 4q + 3 of eight packed in words, divided by
// scale (a power of two), the first lowest.  The conversion divides and rounds
// to nearest even in one step.
template <typename E>
__device__ __forceinline__ uint32_t codes_of(const uint32_t* w, uint32_t q, float scale) {
  i16x2 r = {0, 0};
  if constexpr (__is_same(E, bf16_t)) {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, w[2 * q]), scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, w[2 * q + 1]), scale, true);
  } else if constexpr (__is_same(E, fp16_t)) {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, __builtin_bit_cast(fp16x2, w[2 * q]), scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, __builtin_bit_cast(fp16x2, w[2 * q + 1]), scale, true);
  } else {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __uint_as_float(w[4 * q]), __uint_as_float(w[4 * q + 1]), scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __uint_as_float(w[4 * q + 2]), __uint_as_float(w[4 * q + 3]), scale, true);
  }
  return __builtin_bit_cast(uint32_t, r);
}

// NaN in the places of a word of codes whose elements are not finite.
template <typename E>
__device__ __forceinline__ uint32_t with_nans(uint32_t codes, const uint32_t* w, uint32_t q) {
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j)
    if (!(fabsf(element<E>(w, 4 * q + j)) <= 3.402823466e38f))
      codes = (codes & ~(0xFFu << (8 * j))) | 0x7Fu << (8 * j);
  return codes;
}

// Byte j of the four words, as word j.
__device__ __forceinline__ void transpose(const uint32_t (&w)[4], uint32_t (&out)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  out[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// A run is the rows that fall into one block: consecutive slots that do not
// pass its end, places off .. end - 1, from row n on.  The keys or the values of
// one run and head are an item: its largest magnitude is found, the block's
// scale settled, the earlier tokens' codes rounded again if the scale grew, and
// the run's written.
//
// A lane holds four consecutive places of a block times eight dims (col): the
// keys go out as eight bytes per place, the values, which the cache holds
// transposed, as a word of four places per dim.  64 / (D / 8) groups of four
// places fit a wave at once (TG): a pass.  WV waves take an item, each its share
// of the block's passes, and exchange their magnitudes through shared memory
// (every wave of the workgroup must then be in the same call).  With several
// waves the rows of 16-bit types stay in registers between the two looks at
// them; one wave loads them again, which its short runs bear.
template <typename E, int D, int T, int WV>
__device__ __forceinline__ void store_item(const StoreArgs& A, float* s_max, int32_t n, uint32_t block,
                                           uint32_t off, uint32_t end, uint32_t h, uint32_t side) {
  constexpr uint32_t W = D / 8;
  constexpr uint32_t TG = store_groups(D, T), P = T / (4 * TG) / WV;
  constexpr bool kKeep = P == 1 || (sizeof(E) == 2 && WV > 1);
  constexpr uint32_t kSpan = 4 * TG;  // places of a pass
  struct Row8 {
    uint32_t w[2 * sizeof(E)];
  };
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const uint32_t tg = lane % TG, col = lane / TG;
  const bool active = col < W;
  const uint32_t base = wave % WV * P * kSpan;  // the wave's first place
  float* held = reinterpret_cast<float*>(A.cache + scales_at(A.s, block, h)) + side;
  const int64_t row_stride = side ? A.value_row : A.key_row;
  // (of place 0, which may lie before the rows: only places of the run are read)
  const E* src = static_cast<const E*>(side ? A.value : A.key) +
                 (static_cast<int64_t>(n) - off) * row_stride +
                 static_cast<int64_t>(h) * (side ? A.value_head : A.key_head) + 8 * col;
  auto load_pass = [&](uint32_t p, Row8 (&x)[4]) {
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t place = base + kSpan * p + 4 * tg + i;
      x[i] = Row8{};
      if (active && place >= off && place < end) __builtin_memcpy(&x[i], src + place * row_stride, sizeof(x[i]));
    }
  };
  Row8 x[kKeep ? P : 1][4];
  const float was = off ? *held : 0.0f;
  // visit(p, rows) for the passes that hold places of the run, their rows
  // loaded by then: all at once if they are kept, else one after the other.
  auto each_pass = [&](bool loaded, auto&& visit) {
    if constexpr (kKeep) {
      if (!loaded) {
#pragma unroll
        for (uint32_t p = 0; p < P; ++p)
          if (base + kSpan * (p + 1) > off && base + kSpan * p < end) load_pass(p, x[p]);
      }
#pragma unroll
      for (uint32_t p = 0; p < P; ++p)
        if (base + kSpan * (p + 1) > off && base + kSpan * p < end) visit(p, x[p]);
    } else {
#pragma clang loop unroll(disable)
      for (uint32_t p = 0; p < P; ++p) {
        if (base + kSpan * (p + 1) <= off || base + kSpan * p >= end) continue;
        load_pass(p, x[0]);
        visit(p, x[0]);
      }
    }
  };
  uint8_t* codes = A.cache + (side ? value_at(A.s, block, h) : key_at(A.s, block, h));
  float amax = 0.0f;
  bool strange = false;  // some element is not finite
  if constexpr (sizeof(E) == 2) {
    // two magnitudes at a time by their bits; what is not finite is left
    // out in a second look, if there is any
    u16x2 top = {0, 0};
    each_pass(false, [&](uint32_t, Row8 (&y)[4]) {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i)
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
          asm volatile("" : "+v"(y[i].w[j]));  // (kept as it came, not widened)
          top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, y[i].w[j] & 0x7FFF7FFFu));
        }
    });
    uint32_t most = max<uint32_t>(top[0], top[1]);
    strange = __ballot(most >= infinity_bits<E>()) != 0;
    if (strange) {
      most = 0;
      each_pass(true, [&](uint32_t, Row8 (&y)[4]) {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t w = y[i].w[j], lo = w & 0x7FFFu, hi = w >> 16 & 0x7FFFu;
            if (lo < infinity_bits<E>()) most = max(most, lo);
            if (hi < infinity_bits<E>()) most = max(most, hi);
          }
      });
    }
    amax = static_cast<float>(__builtin_bit_cast(E, static_cast<uint16_t>(most)));
  } else {
    each_pass(false, [&](uint32_t, Row8 (&y)[4]) {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i)
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
          const float v = element<E>(y[i].w, j);
          amax = fmaxf(amax, finite_abs(v));
          strange |= !(fabsf(v) <= 3.402823466e38f);
        }
    });
    strange = __ballot(strange) != 0;
  }
  amax = wave_max(amax);
  if constexpr (WV > 1) {
    if (lane == 0) s_max[wave] = amax;
    __syncthreads();
#pragma unroll
    for (uint32_t w = 0; w < WV; ++w) amax = fmaxf(amax, s_max[wave / WV * WV + w]);
    __syncthreads();  // (also: every wave has read the old scale)
  }
  float scale = scale_of(amax);
  const bool grew = off && scale > was;
  if (off && !grew) scale = was;
  const float again = grew ? was * power_inverse(scale) : 1.0f;
#pragma clang loop unroll_count(kKeep ? P : 1)
  for (uint32_t p = 0; p < P; ++p) {
    if (base + kSpan * p >= end || (base + kSpan * (p + 1) <= off && !grew)) continue;
    const uint32_t first = base + kSpan * p + 4 * tg;
    if constexpr (!kKeep) load_pass(p, x[0]);
    uint32_t lo[4], hi[4];  // the codes of dims 0 .. 3 and 4 .. 7 of each place
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const Row8& r = x[kKeep ? p : 0][i];
      lo[i] = codes_of<E>(r.w, 0, scale);
      hi[i] = codes_of<E>(r.w, 1, scale);
      if (strange) {
        lo[i] = with_nans<E>(lo[i], r.w, 0);
        hi[i] = with_nans<E>(hi[i], r.w, 1);
      }
    }
    if (!active) continue;
    if (side == 0) {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t place = first + i;
        uint8_t* c = codes + place * D + 8 * col;
        if (place >= off && place < end) {
          *reinterpret_cast<u32x2*>(c) = u32x2{lo[i], hi[i]};
        } else if (place < off && grew) {
          for (uint32_t j = 0; j < 8; ++j) c[j] = code_of(value_of(c[j]) * again);
        }
      }
    } else if (first >= off && first + 4 <= end) {
      // four places by eight dims to eight words of four places
      uint32_t v[2][4];
      transpose(lo, v[0]);
      transpose(hi, v[1]);
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j)
        *reinterpret_cast<uint32_t*>(codes + (8 * col + j) * T + first) = v[j / 4][j % 4];
    } else {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t place = first + i;
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
          uint8_t* c = codes + (8 * col + j) * T + place;
          if (place >= off && place < end)
            *c = static_cast<uint8_t>((j < 4 ? lo[i] : hi[i]) >> (8 * (j % 4)));
          else if (place < off && grew)
            *c = code_of(value_of(*c) * again);
        }
      }
    }
  }
  if (lane == 0 && wave % WV == 0) *held = scale;
}

// A workgroup looks after the runs that begin in its tile of rows, for its
// heads.  Runs that take more than one pass are done one after the other by all
// waves, a pass each, and keep many loads in flight; shorter ones, such as a
// decode step's single tokens, go to a wave each.  161 MB read and written for
// 26k tokens of 29 prompts take 45 us (3.6 TB/s; a copy 32): a workgroup waits
// for its slots, then its rows, then the largest magnitude.  Asking for the next
// item's rows ahead changed nothing, other orders of heads and rows 47 to 55.
template <typename E, int D, int T>
__global__ void __launch_bounds__(kStoreWaves * 64) store_kernel(StoreArgs A) {
  constexpr uint32_t kSpan = 4 * store_groups(D, T), kPasses = T / kSpan;
  constexpr uint32_t WV = kPasses < kStoreWaves ? kPasses : kStoreWaves;
  __shared__ float s_max[kStoreWaves];
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // (known to be uniform)
  const uint32_t groups = (A.s.H + A.wg_heads - 1) / A.wg_heads;  // the heads of a tile side by side
  const int32_t n0 = static_cast<int32_t>(blockIdx.x / groups * A.tile);
  const uint32_t h0 = blockIdx.x % groups * A.wg_heads, items = min(A.wg_heads, A.s.H - h0) * 2;
  // The slots of the tile's rows and of those that a run from there may reach.
  auto slot_at = [&](int32_t n) { return n >= 0 && n < A.rows ? A.slots[n] : -1; };
  const int32_t near = slot_at(n0 + static_cast<int32_t>(lane)), before = slot_at(n0 - 1);
  const int32_t last = __shfl_up(near, 1);
  const bool begins = lane < A.tile && near >= 0 && static_cast<uint32_t>(near) / T < A.s.blocks &&
                      (near % T == 0 || (lane ? last : before) != near - 1);
  const uint64_t runs = __ballot(begins);
  if (runs == 0) return;
  const int32_t far = A.tile + T > 65 ? slot_at(n0 + 64 + static_cast<int32_t>(lane)) : -1;
  // each(long, f) calls f(row, block, off, end) for the runs of more than one pass, or the others.
  auto each = [&](bool longer, auto&& f) {
    for (uint64_t left = runs; left; left &= left - 1) {
      const int32_t r = __builtin_ctzll(left);  // the run's first row in the tile
      const int32_t slot = __builtin_amdgcn_readlane(near, r);
      const uint32_t off = static_cast<uint32_t>(slot) % T, at = r + lane;
      const int32_t close = __shfl(near, at & 63), wide = __shfl(far, at & 63);
      const bool goes_on =
          off + lane < T && (at < 64 ? close : wide) == slot + static_cast<int32_t>(lane);
      const uint64_t stops = ~__ballot(goes_on);
      const uint32_t end = off + (stops ? __builtin_ctzll(stops) : 64u);
      if (((end - 1) / kSpan > off / kSpan) == longer) f(n0 + r, static_cast<uint32_t>(slot) / T, off, end);
    }
  };
  if constexpr (kPasses > 1)
    each(true, [&](int32_t n, uint32_t block, uint32_t off, uint32_t end) {
      for (uint32_t k = wave / WV; k < items; k += kStoreWaves / WV)
        store_item<E, D, T, WV>(A, s_max, n, block, off, end, h0 + k / 2, k % 2);
    });
  uint32_t turn = 0;
  each(false, [&](int32_t n, uint32_t block, uint32_t off, uint32_t end) {
    for (uint32_t k = 0; k < items; ++k)
      if (turn++ % kStoreWaves == wave)
        store_item<E, D, T, 1>(A, s_max, n, block, off, end, h0 + k / 2, k % 2);
  });
}

using StoreFn = void (*)(StoreArgs);

template <typename E, int D>
StoreFn pick_store_tokens(uint32_t t) {
  return t == 16 ? store_kernel<E, D, 16> : t == 32 ? store_kernel<E, D, 32> : store_kernel<E, D, 64>;
}

template <typename E>
StoreFn pick_store(uint32_t d, uint32_t t) {
  switch (d) {
    case 64: return pick_store_tokens<E, 64>(t);
    case 96: return pick_store_tokens<E, 96>(t);
    case 128: return pick_store_tokens<E, 128>(t);
    case 192: return pick_store_tokens<E, 192>(t);
    default: return pick_store_tokens<E, 256>(t);
  }
}

// ------------------------------------------------------------------ attend
template <typename E>
struct Vec8;
template <>
struct Vec8<bf16_t> {
  typedef bf16x8 type;
};
template <>
struct Vec8<fp16_t> {
  typedef fp16x8 type;
};

// Eight e4m3 codes times scale, exactly (a power of two, in range).
__device__ __forceinline__ void widen(uint32_t lo, uint32_t hi, float scale, bf16x8& r) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  r = bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ void widen(uint32_t lo, uint32_t hi, float scale, fp16x8& r) {
  const fp16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, scale, false);
  const fp16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, scale, true);
  const fp16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, scale, false);
  const fp16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, scale, true);
  r = fp16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The dims of lane group g in step k of 32: sixteen-byte loads of the keys
// serve two steps where D allows.
template <int D>
__device__ __forceinline__ uint32_t key_dim(uint32_t k, uint32_t g) {
  if constexpr (D % 64 == 0)
    return 64 * (k / 2) + 16 * g + 8 * (k % 2);
  else
    return 32 * k + 8 * g;
}

// A chunk's value codes and the scales of the lane's block.
template <int D, bool ONCE>
struct Values {
  u32x4 w[D / 16];
  float key_scale, value_scale;
  __device__ __forceinline__ void load(const AttendArgs& A, const Place& at, uint32_t t0, uint32_t h,
                                       uint32_t g, uint32_t n) {
    const uint32_t block = max(at.mine, 0), T = A.s.T;
    const uint8_t* p = A.cache + value_at(A.s, block, h) + n * T + ((t0 + 16 * g) & (T - 1));
    const float* s = reinterpret_cast<const float*>(A.cache + scales_at(A.s, block, h));
    key_scale = s[0];
    value_scale = s[1];
#pragma unroll
    for (int e = 0; e < D / 16; ++e) w[e] = fetch<ONCE, u32x4>(p + 16 * e * T);
  }
};

// Workgroups a CU is to hold: bounds the registers of a lane (four waves of 512
// / this).  Two with two tiles of 128 measured 118 us where one took 187 (chunks of
// 8 requests), 1135 and 1650 (8 prompts of 3000 tokens); three with one tile of 128
// were no faster.
constexpr int attend_resident(int d, int nr) {
  return nr == 2 ? (d <= 128 ? 2 : 1) : d == 64 ? 3 : d <= 192 ? 2 : 1;
}

template <int D, bool ONCE>
struct Keys {
  static constexpr bool kWide = D % 64 == 0;
  u32x4 w[4][kWide ? D / 64 : 1];
  u32x2 d[4][kWide ? 1 : D / 32];
  __device__ __forceinline__ void load(const AttendArgs& A, const Place& at, uint32_t t0, uint32_t h,
                                       uint32_t g, uint32_t n) {
    const uint32_t tk = t0 + 16 * (n >> 2);
    const uint8_t* p = A.cache + key_at(A.s, at.line, h) +
                       ((tk & (A.s.T - 1)) + (n & 3u)) * D + (kWide ? 16 : 8) * g;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if constexpr (kWide) {
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
          w[t][j] = fetch<ONCE, u32x4>(p + 4 * t * D + 64 * j);
      } else {
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
          d[t][j] = fetch<ONCE, u32x2>(p + 4 * t * D + 32 * j);
      }
    }
  }
  __device__ __forceinline__ uint32_t lo(int t, int k) const {
    if constexpr (kWide)
      return w[t][k / 2][k % 2 * 2];
    else
      return d[t][k][0];
  }
  __device__ __forceinline__ uint32_t hi(int t, int k) const {
    if constexpr (kWide)
      return w[t][k / 2][k % 2 * 2 + 1];
    else
      return d[t][k][1];
  }
};

// NaN for each of the dims d .. d + 3 in which one of the tokens t0 .. last
// has a NaN code, 0 for the others.  Rarely run, so it is a plain loop.
__device__ __forceinline__ f32x4 seen_nans(const AttendArgs& A, const int32_t* table,
                                                       uint32_t h, int32_t t0, int32_t last,
                                                       uint32_t d) {
  f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma clang loop unroll(disable)
  for (int32_t t = t0; t <= last; ++t) {
    const int32_t id = table[t >> A.s.log2T];
    if (static_cast<uint32_t>(id) >= A.s.blocks) continue;
    const uint8_t* v = A.cache + value_at(A.s, id, h) + (t & (A.s.T - 1));
#pragma clang loop unroll(disable)
    for (uint32_t k = 0; k < 4; ++k)
      if ((v[static_cast<uint64_t>(d + k) * A.s.T] & 0x7F) == 0x7F) r[k] = NAN;
  }
  return r;
}

// The weights of a chunk's scores and their product with the values.  MASK:
// some row does not see some token of the chunk.
template <bool MASK, int DT, int NR>
__device__ __forceinline__ void weigh(const AttendArgs& A, f32x4 (&s)[NR][4], f32x4 (&acc)[NR][DT],
                                      float (&m)[NR], float (&l)[NR], const u32x4 (&vc)[DT],
                                      const int32_t (&limit)[NR], float mul, float vs,
                                      int32_t seen_all, int32_t tg, int32_t bg, uint32_t& nans) {
  bf16x8 p[NR][2], p2[NR][2];
#pragma unroll
  for (int x = 0; x < NR; ++x) {
    const int32_t seen = bg < 0 ? 0 : limit[x] - tg + 1;  // of this lane's sixteen tokens
    float top = -INFINITY;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v = s[x][t][r] * mul;
        if (MASK && 4 * t + r >= seen) v = -INFINITY;
        s[x][t][r] = v;
        top = fmaxf(top, v);
      }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    // The reference m follows the maximum only when that is 8 above it, so most
    // chunks leave the accumulators alone: weights reach 256 at most, and the
    // same powers of two leave sums and accumulators in the end.
    const bool grows = top > m[x] + 8.0f;
    const float next = grows ? top : m[x], base = next == -INFINITY ? 0.0f : next;
    const float keep = grows ? __builtin_amdgcn_exp2f(m[x] - base) : 1.0f;
    m[x] = next;
    float sum = 0.0f;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float w = __builtin_amdgcn_exp2f(s[x][t][r] - base);
        sum += w;
        const bf16_t first = static_cast<bf16_t>(w);
        p[x][t >> 1][(t & 1) * 4 + r] = first;
        p2[x][t >> 1][(t & 1) * 4 + r] = static_cast<bf16_t>(w - static_cast<float>(first));
      }
    l[x] = l[x] * keep + sum;
    if (__ballot(grows) != 0) {
#pragma unroll
      for (int e = 0; e < DT; ++e) acc[x][e] *= keep;
    }
  }
  // Codes of tokens that no row sees are cleared: they may be anything, and 0
  // times NaN is NaN.
  uint32_t mask[4];
  if constexpr (MASK) {
    const int32_t held = bg < 0 ? 0 : seen_all - tg;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int left = held - 4 * w;
      mask[w] = left <= 0 ? 0u : left >= 4 ? ~0u : (1u << (8 * left)) - 1u;
    }
  }
#pragma unroll
  for (int e = 0; e < DT; ++e) {
    u32x4 v = vc[e];
    if constexpr (MASK) {
      u32x4 nan;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        v[w] &= mask[w];
        nan[w] = (((v[w] & 0x7F7F7F7Fu) + 0x01010101u) >> 7) & 0x01010101u;
      }
      // A NaN among the others reaches the rows that see its token and no
      // other: it is taken out here and looked for again in memory at the end.
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        nans |= nan[w];
        v[w] &= ~(nan[w] * 0xFFu);
      }
    }
    bf16x8 a, z;
    widen(v[0], v[1], vs, a);
    widen(v[2], v[3], vs, z);
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      acc[x][e] = mfma(a, p[x][0], acc[x][e]);
      acc[x][e] = mfma(z, p[x][1], acc[x][e]);
      acc[x][e] = mfma(a, p2[x][0], acc[x][e]);
      acc[x][e] = mfma(z, p2[x][1], acc[x][e]);
    }
  }
}

// Row i of a request and key/value head is query row i / group, head i %
// group of the group.  A workgroup computes NR tiles of 16 rows of one request
// and key/value head over a range of the tokens: its waves take chunks of 64
// tokens in turn, each with a reference m, which the running maximum may pass
// by 8, a sum l and an accumulator of its own, and join them at the end:
//   p_t = 2^(s_t - m), l = sum p_t, acc = sum p_t v_t, out = acc / l,
// the scores s_t in units of log 2.
//
// Both products run on the 16x16x32 matrix instruction with the cache's codes
// as the left operand, straight from the loads: no shared memory, no
// transposing.  S^T = K Q^T takes 16 tokens by 16 rows a time.  In its result
// lane (g, n) = (lane / 16, lane % 16) holds row n and the tile's lines 4g + r,
// so which token sits at line 4g + r of tile t is chosen as 16g + 4t + r: over
// the four tiles of a chunk a lane then holds the sixteen consecutive tokens
// 16g .. 16g + 15 of its row.  Those are what O^T = V^T P^T wants from it: its
// right operand takes eight consecutive tokens of row n from lane (g, n), and
// its left operand eight consecutive tokens of dim 16e + n, which the cache
// holds together as V^T.  Sixteen tokens never pass a block's end, so a lane
// has one block, one key scale and one value scale per chunk: the key scale
// goes into the scores' multiplier, the value scale into the widening of the
// codes to bfloat16, where both are exact.
//
// Weights multiply the values as bfloat16 whatever the query's type: code times
// scale needs its range.  One such number would be off by up to 2^-8 of the
// weight, which shows beside the output's own rounding (and is far above it
// where values cancel), so a weight goes in two parts, the rounded one and the
// rounded rest (off by 2^-16), at one more product each.  The codes are widened
// although there are matrix instructions for 8 bits: those align a sum's
// products to the largest with about 13 bits, which on random wide exponents
// was off by 2^-12.5 of the sum of magnitudes (bfloat16's form 2.5 x 2^-24).
//
// What bounds it: memory where there are few rows (64 requests of 500 .. 8000
// tokens, 8 heads of 128, group 4: 360 MB in 80 us, 4.5 TB/s; 2 of 65k .. 131k,
// group 8: 402 MB in 82 us, 4.9 TB/s; a read alone reaches 6.3), each piece's
// first trip to memory and the join making up the rest; the instructions that
// widen, weigh and rescale where there are many (8 requests with up to 600 rows
// each after up to 5000 tokens: 34.5 GFLOP in 107 us, 322 TFLOP/s, of which the
// weights' second parts take 10 us); the chain table -> codes -> products for
// short ones (300 tokens: 8 us).
template <int D, int NR>
struct AttendShared {  // 19 to 84 KiB
  u32x4 q[NR][D / 32][64];  // the rows' queries, in the order of the matrix operand
  float acc[kAttendWaves][16][D + 4];
  float m[kAttendWaves][NR * 16], l[kAttendWaves][NR * 16];
};

// The rows first .. first + 16 NR - 1 of request b and key/value head h over
// the chunks c0 .. c1 - 1, by a workgroup.  part null: these are all the
// tokens, and the rows are written; else their sums go to part and stats.
template <typename E, int D, int NR, bool ONCE>
__device__ __forceinline__ void attend_rows(const AttendArgs& A, AttendShared<D, NR>& sh, uint32_t b,
                                            uint32_t h, uint32_t first, uint32_t c0, uint32_t c1,
                                            float* part, float* stats) {
  typedef typename Vec8<E>::type E8;
  constexpr int KL = D / 32;  // steps of 32 dims
  constexpr int DT = D / 16;  // tiles of dims
  const uint32_t lane = threadIdx.x & 63u, n = lane & 15u, g = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // (known to be uniform)
  const int32_t* table = A.table + static_cast<int64_t>(b) * A.table_stride;
  const RowTile rt = row_tile(A, b, first, NR * 16);
  c1 = min(c1, (static_cast<uint32_t>(rt.seen) + kChunk - 1) / kChunk);

  // The first chunk's table entries, then its keys and values, are asked for
  // before anything is waited for: each is a trip to memory.
  // Waves with no chunk ask too, for the last block or, where no token is seen
  // and the table may be empty, for whichever the first entry of starts names
  // (any word will do, settle puts it in range): behind a branch around these
  // loads every wait of the loop would be one for all of them.
  const uint32_t seen_all = uniform(static_cast<uint32_t>(rt.seen)), reach = max(seen_all, 1u);
  if (seen_all == 0) table = A.starts;
  uint32_t c = c0 + wave, nans = 0;
  Keys<D, ONCE> keys;
  Values<D, ONCE> vals;
  Place at, next;
  constexpr uint32_t kNext = kAttendWaves * kChunk;  // tokens from a wave's chunk to its next
  at.look(A, table, c * kChunk, reach, g, n);
  next.look(A, table, c * kChunk + kNext, reach, g, n);
  __builtin_amdgcn_sched_barrier(0);

  // Queries: lane (g, n) takes row n's dims in the order of its key loads.
  // They wait in shared memory, the same for every wave, which frees the
  // registers that decide how many waves a CU holds.
  constexpr int QL = (KL + kAttendWaves - 1) / kAttendWaves;
  int32_t limit[NR];        // last token that the row sees
  int32_t least = rt.seen;  // the first of them
  u32x4 q[NR][QL];
#pragma unroll
  for (int x = 0; x < NR; ++x) {
    const uint32_t i = first + x * 16 + n;
    const int64_t j = i / A.group, row = rt.start + j;
    const bool there = i < rt.rows;
    limit[x] = there ? static_cast<int32_t>(max<int64_t>(-1, min<int64_t>(rt.seen - 1, rt.ahead + j))) : -1;
    const E* p = static_cast<const E*>(A.query) + row * A.query_row +
                 static_cast<int64_t>(h * A.group + i % A.group) * A.query_head;
#pragma unroll
    for (int k = 0; k < QL; ++k) {
      q[x][k] = u32x4{0u, 0u, 0u, 0u};
      const uint32_t step = wave + k * kAttendWaves;
      if (there && step < KL) __builtin_memcpy(&q[x][k], p + key_dim<D>(step, g), 16);
    }
    if (there) least = min(least, limit[x]);  // (other rows hold zeros and go nowhere)
  }
  at.settle(A, c * kChunk, seen_all, g);
  keys.load(A, at, c * kChunk, h, g, n);
  __builtin_amdgcn_sched_barrier(0);
  vals.load(A, at, c * kChunk, h, g, n);
#pragma unroll
  for (int x = 0; x < NR; ++x)
#pragma unroll
    for (int k = 0; k < QL; ++k)
      if (wave + k * kAttendWaves < KL) sh.q[x][wave + k * kAttendWaves][lane] = q[x][k];
  for (int d = 1; d < 16; d <<= 1) least = min(least, __shfl_xor(least, d));
  least = __builtin_amdgcn_readfirstlane(least);
  __syncthreads();

  float m[NR], l[NR];
  f32x4 acc[NR][DT];
#pragma unroll
  for (int x = 0; x < NR; ++x) {
    m[x] = -INFINITY;
    l[x] = 0.0f;
#pragma unroll
    for (int e = 0; e < DT; ++e) acc[x][e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // A chunk's keys are loaded while the chunk before is still at its weights
  // and values, its values as soon as those are done.  Loads return in the
  // order they were asked for, so its table entries come a step earlier yet,
  // ahead of the values of the chunk before: waiting for them waits for no
  // codes.  The last step loads too (the last block again, near at hand): a
  // branch around the loads would make every wait after it one for all of
  // them.
  auto step = [&](auto masked) {
    const uint32_t t0 = c * kChunk, tg = t0 + 16 * g, ahead = t0 + kNext;
    const int32_t bg = at.mine;
    f32x4 s[NR][4];
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int t = 0; t < 4; ++t) s[x][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < KL; ++k) {
      E8 b8[NR];
#pragma unroll
      for (int x = 0; x < NR; ++x) b8[x] = __builtin_bit_cast(E8, sh.q[x][k][lane]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        E8 a;
        widen(keys.lo(t, k), keys.hi(t, k), 1.0f, a);
#pragma unroll
        for (int x = 0; x < NR; ++x) s[x][t] = mfma(a, b8[x], s[x][t]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    next.settle(A, ahead, seen_all, g);
    keys.load(A, next, ahead, h, g, n);
    __builtin_amdgcn_sched_barrier(0);
    // (the scales of a block that is not the request's: anything)
    const float ks = bg < 0 ? 1.0f : vals.key_scale, vs = bg < 0 ? 1.0f : vals.value_scale;
    weigh<decltype(masked)::value, DT, NR>(A, s, acc, m, l, vals.w, limit, ks * A.scale2, vs,
                                           seen_all, tg, bg, nans);
    __builtin_amdgcn_sched_barrier(0);
    at = next;
    next.look(A, table, ahead + kNext, seen_all, g, n);
    vals.load(A, at, ahead, h, g, n);
    c += kAttendWaves;
  };
  // Chunks that every row sees whole, up to the first that is not; then the rest.
  const uint32_t whole = min(c1, static_cast<uint32_t>(least + 1) / kChunk);
  while (c < whole && __ballot(at.mine < 0) == 0) step(std::false_type());
  const uint32_t rest = c;
  while (c < c1) step(std::true_type());
  const bool any_nan = __ballot(nans != 0) != 0;

  // Join the waves.
#pragma unroll
  for (int x = 0; x < NR; ++x) {
    l[x] += __shfl_xor(l[x], 16);
    l[x] += __shfl_xor(l[x], 32);
    if (g == 0) {
      sh.m[wave][x * 16 + n] = m[x];
      sh.l[wave][x * 16 + n] = l[x];
    }
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < NR; ++x) {
    float top = sh.m[0][x * 16 + n];
    for (int w = 1; w < kAttendWaves; ++w) top = fmaxf(top, sh.m[w][x * 16 + n]);
    const float base = top == -INFINITY ? 0.0f : top;
    const float f = __builtin_amdgcn_exp2f(m[x] - base);
#pragma unroll
    for (int e = 0; e < DT; ++e)
      *reinterpret_cast<f32x4*>(&sh.acc[wave][n][16 * e + 4 * g]) = acc[x][e] * f;
    if (any_nan) {
#pragma clang loop unroll(disable)
      for (uint32_t i = 0; i < DT * ((c1 - rest + kAttendWaves - 1) / kAttendWaves); ++i) {
        const uint32_t d = 16 * (i % DT) + 4 * g;
        const int32_t t0 = (rest + i / DT * kAttendWaves) * kChunk;
        f32x4* o = reinterpret_cast<f32x4*>(&sh.acc[wave][n][d]);
        *o += seen_nans(A, table, h, t0, min(t0 + kChunk - 1, limit[x]), d);
      }
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < 16 * (D / 4); i += kAttendWaves * 64) {
      const uint32_t r = i / (D / 4), d = i % (D / 4) * 4, ri = first + x * 16 + r;
      const int64_t row = rt.start + ri / A.group;
      if (ri >= rt.rows) continue;
      float top = sh.m[0][x * 16 + r], sum = 0.0f;
      for (int w = 1; w < kAttendWaves; ++w) top = fmaxf(top, sh.m[w][x * 16 + r]);
      const float base = top == -INFINITY ? 0.0f : top;
      f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int w = 0; w < kAttendWaves; ++w) {
        sum += sh.l[w][x * 16 + r] * __builtin_amdgcn_exp2f(sh.m[w][x * 16 + r] - base);
        o += *reinterpret_cast<const f32x4*>(&sh.acc[w][r][d]);
      }
      const uint32_t head = h * A.group + ri % A.group;
      const int64_t at = row * A.heads + head;
      if (part == nullptr) {
        const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
        E v[4];
        for (int k = 0; k < 4; ++k) v[k] = static_cast<E>(o[k] * inv);
        __builtin_memcpy(static_cast<E*>(A.out) + row * A.out_row + head * A.out_head + d, v, 8);
        if (d == 0 && A.lse)
          A.lse[at] = (top + __builtin_amdgcn_logf(sum)) * 0.69314718055994531f;
      } else {
        *reinterpret_cast<f32x4*>(part + (x * 16 + r) * D + d) = o;
        if (d == 0) {
          stats[(x * 16 + r) * 2] = top;
          stats[(x * 16 + r) * 2 + 1] = sum;
        }
      }
    }
    __syncthreads();
  }
}

template <typename E, int D, int NR, bool ONCE>
struct Core {
  typedef E Elem;
  typedef AttendShared<D, NR> Shared;
  static constexpr int kDim = D, kRows = NR * 16, kThreads = kAttendWaves * 64;
  static constexpr int kResident = attend_resident(D, NR);
  static __device__ __forceinline__ void rows(const AttendArgs& A, Shared& sh, uint32_t b, uint32_t h,
                                              uint32_t first, uint32_t c0, uint32_t c1, float* part,
                                              float* stats) {
    attend_rows<E, D, NR, ONCE>(A, sh, b, h, first, c0, c1, part, stats);
  }
};



template <typename E, int D>
AttendKernels pick_attend_rows(int nr, bool once) {
  if constexpr (D != 192) {
    if (nr == 2) return attend_kernels<Core<E, D, 2, false>, Core<E, D, 2, false>, (2 * D <= 256)>();
  }
  return once ? attend_kernels<Core<E, D, 1, true>, Core<E, D, 1, false>, true>()
              : attend_kernels<Core<E, D, 1, false>, Core<E, D, 1, false>, true>();
}

template <typename E>
AttendKernels pick_attend(uint32_t d, int nr, bool once) {
  switch (d) {
    case 64: return pick_attend_rows<E, 64>(nr, once);
    case 96: return pick_attend_rows<E, 96>(nr, once);
    case 128: return pick_attend_rows<E, 128>(nr, once);
    case 192: return pick_attend_rows<E, 192>(nr, once);
    default: return pick_attend_rows<E, 256>(nr, once);
  }
}

AttendPlan attend_plan(const Shape& s, const xfer_attend& q) {
  AttendPlan p;
  const int64_t group = q.heads / int(s.H);
  int64_t most = q.max_query ? std::min(q.max_query, q.rows) : q.rows;
  if (!q.max_query && q.rows <= q.batch) most = 1;
  const int64_t rows = most * group;
  // Two tiles of rows share the widened codes and halve the reads, but two of 192
  // or 256 leave a CU one workgroup, and no registers for sharing.  One against
  // two (us, drafts with 12 heads over 2, the others with 32 over 8): heads of 192:
  // 48 requests of 3 to 5 rows 27 / 42, 256 of them 58 / 52, 8 with 1 to 600 rows
  // after up to 4400 tokens 208 / 438, 2 prompts of 1000 99 / 120, 8 of 3000 2060 /
  // 2210.  Heads of 256: 48 drafts 39 / 48, a prompt of 100 12.6 / 16.8 (200 tiles),
  // 256 drafts 86 / 63 (1024), 2 prompts of 1000 208 / 151 (4000), 8 with up to 600
  // rows 439 / 548, 8 prompts of 3000 4140 / 2770.
  int nr = rows <= 16 || s.D == 192 ? 1 : 2;
  if (s.D == 256 && q.batch * int64_t(s.H) * ((rows + 15) / 16) <= 1024) nr = 1;
  p.tile = nr * 16;
  p.tiles = uint32_t(std::min<int64_t>(65535, (rows + nr * 16 - 1) / (nr * 16)));
  const int64_t width = int64_t(q.table_width) * s.T;
  const int64_t tokens = q.max_length ? std::min<int64_t>(q.max_length, width) : width;
  const int64_t chunks = std::max<int64_t>(1, (tokens + kChunk - 1) / kChunk);
  const int64_t wgs = int64_t(q.batch) * s.H * p.tiles;
  // Tiles that the packed rows can have, and so workgroups of one head (first_tile).
  const int64_t numbers = int64_t(q.rows) * group / (nr * 16) + q.batch;
  const int64_t resident = 256 * attend_resident(int(s.D), nr);  // workgroups on 256 CUs
  // Sharing costs a second launch and about 8 us; it pays where few workgroups
  // would be left with long requests.  Measured at 8 key/value heads of 128,
  // group 4, one workgroup per tile against shared (us): 1 request of 1024
  // tokens 14 / 16, of 2048 21 / 17, of 16384 120 / 23; 32 requests of 2048
  // 31 / 38, of 4096 52 / 60, of 410 .. 4096 42 / 38, of 8192 95 / 104, of 820 ..
  // 8192 75 / 56; 128 requests of 400 .. 5000 109 / 97, 1024 of them 656 / 679, of
  // 100 .. 12000 913 / 865, of 4200 1352 / 1399: single rows gain where lengths
  // differ and lose a twentieth where they do not.  Many rows, as workgroups for
  // each one that is resident: 0.6 (3 requests of up to 200 rows) 76 / 69, 2.9 (8
  // of up to 600) 326 / 185, 3.9 (1 of 2000 after 3000 tokens) 247 / 289, 8.2 (1
  // whole prompt of 4200) 285 / 427, 9.2 (32 of up to 600) 668 / 537, 66 (8 whole
  // prompts of 4200) 2089 / 3806; heads of 64, 16 (32 of up to 600) 456 / 521.  So
  // from 12 on there are enough of them, whatever the lengths.
  p.flat = p.packed = 0;
  const bool enough = most > 1 && numbers * s.H > 12 * resident;
  if (!enough && chunks >= (wgs <= 128 ? 24 : 64) && int(s.D) * nr <= 256) {
    // As many workgroups as are resident at once, eight chunks each at least.
    p.flat = uint32_t(std::max<int64_t>(
        1, std::min<int64_t>(resident / s.H, chunks * q.batch * p.tiles / 8)));
  }
  // Where one request may have most of the rows, a grid of requests and tiles is
  // mostly empty: 2000 workgroups that find nothing to do take 1 us, and hold up
  // those behind them.  Numbers through the packed rows leave those out, at a
  // search in each workgroup.  Grid against numbers (us): 1024 requests of 16 rows
  // and 64 tokens, no hints, 9260 / 330; 2000 rows beside 63 single ones 343 / 88;
  // 60 requests of 8 rows and 300 tokens, no hints, 29.7 / 26.6 (28k empty
  // workgroups), with heads of 256 28.7 / 34.7 (10k).
  if (!p.flat && wgs > numbers * s.H + kEmptyWorkgroups) p.packed = uint32_t(numbers);
  return p;
}

}  // namespace
}  // namespace xfer

using namespace xfer;

extern "C" int xfer_cache_block_bytes(const xfer_cache_shape* shape, size_t* bytes) {
  Shape s;
  const int rc = shape8_of(shape, "xfer_cache_block_bytes", &s);
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
  // (in 64 bits: rows and batch may be 2^31 - 1)
  const int64_t grid = std::max<int64_t>(
      1, std::min<int64_t>(1024, std::max((int64_t(rows) + 1023) / 1024, (int64_t(batch) + 255) / 256)));
  a.per_wg = int32_t((rows + grid - 1) / grid);
  const hipError_t e =
      launch(plan_kernel, a, dim3(uint32_t(grid) + 1), kPlanThreads, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "xfer_cache_plan launch");
  return XFER_OK;
}

extern "C" int xfer_cache_store(const xfer_cache_shape* shape, void* cache, const void* key,
                                int64_t key_row, int64_t key_head, const void* value,
                                int64_t value_row, int64_t value_head, int dtype,
                                const int32_t* slots, int rows, void* stream) {
  StoreArgs a;
  const int rc = shape8_of(shape, "xfer_cache_store", &a.s);
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
  // Rows of a workgroup's tile: a decode step wants a workgroup per token, a
  // prompt one per block, and the lengths of runs are not known here.  Tiles of
  // 1, 8 and T rows take, with 8 heads of 128, bfloat16 and blocks of 16 (64), in
  // us: 256 single tokens 10, 19, 11 (13, 24, 138), 1024 of them 21, 25, 23 (27,
  // 32, 144), 4096 60, 63, 66 (138, 145, 174); a prompt of 500 tokens 10, 9, 9 (24,
  // 10, 13), of 2000 23, 11, 10 (28, 15, 13), of 4000 37, 15, 12 (41, 23, 15), 26k of
  // prompts 152, 67, 46 (150, 83, 47: 3.4 TB/s read and written, waiting for memory).
  a.tile = rows <= 256 ? 1 : rows <= 2048 ? 8 : a.s.T;
  a.wg_heads = a.tile == 1 ? 2 : 1;
  const uint32_t tiles = (uint32_t(rows) + a.tile - 1) / a.tile;
  const uint64_t wgs = uint64_t(tiles) * ((a.s.H + a.wg_heads - 1) / a.wg_heads);
  if (wgs > kMaxGrid)
    return fail(XFER_ERR_INVALID_ARG, "xfer_cache_store: too many rows times heads for one call");
  const dim3 grid(static_cast<uint32_t>(wgs));
  const StoreFn fn = dtype == XFER_BF16   ? pick_store<bf16_t>(a.s.D, a.s.T)
                     : dtype == XFER_FP16 ? pick_store<fp16_t>(a.s.D, a.s.T)
                                          : pick_store<float>(a.s.D, a.s.T);
  const hipError_t e = launch(fn, a, grid, kStoreWaves * 64, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "xfer_cache_store launch");
  return XFER_OK;
}

extern "C" int xfer_cache_attend_workspace(const xfer_cache_shape* shape, const xfer_attend* q,
                                           size_t* bytes) {
  Shape s;
  int rc = shape8_of(shape, "xfer_cache_attend_workspace", &s);
  if (!rc) rc = attend_args(s, q, "xfer_cache_attend_workspace");
  if (rc) return rc;
  if (!bytes) return fail(XFER_ERR_INVALID_ARG, "xfer_cache_attend_workspace: NULL bytes");
  *bytes = attend_work(s, *q, attend_plan(s, *q)).all();
  return XFER_OK;
}

extern "C" int xfer_cache_attend(const xfer_cache_shape* shape, const void* cache,
                                 const xfer_attend* q, void* stream) {
  Shape s;
  int rc = shape8_of(shape, "xfer_cache_attend", &s);
  if (!rc) rc = attend_args(s, q, "xfer_cache_attend");
  if (rc) return rc;
  if (q->rows == 0 || q->batch == 0) return XFER_OK;
  // With one tile a request no other workgroup reads the same tokens (but for
  // requests that share blocks), and loads that leave the caches alone serve long
  // even reads better (us, with against without): 64 single rows over 4000 tokens
  // each, 8 heads of 128, 92 / 99; 2 over 65k and 131k 84 / 92; 128 over 3500, heads
  // of 64, 76 / 85.  Where latency counts they lose: 48 over 100 .. 3000, heads of
  // 256, 42.6 / 38.4; 100 over 300, heads of 192, 17.3 / 15.2.
  const auto pick = [&](int dtype, const AttendPlan& p) {
    const int nr = p.tile / 16;
    const bool once = p.tiles == 1;
    return dtype == XFER_BF16 ? pick_attend<bf16_t>(s.D, nr, once) : pick_attend<fp16_t>(s.D, nr, once);
  };
  return attend_call(s, cache, q, attend_plan(s, *q), pick, stream, "xfer_cache_attend");
}

// gfx950 kernels of the paged 4-bit cache: stores and attention, and the reading
// back of either cache.  Their entry points (xfer_mxcache_*, xfer_cache_load) are at
// the end of the file.
//
// A block is one record of bytes: per key/value head the key codes, then the value
// codes, T * D / 2 bytes each, and behind the heads a byte of scale for each head,
// side (key, value), 32 dims and token, [H][2][D / 32][T], padded to 128 bytes.  A
// code is an e2m1 number, a scale byte s stands for 2^(s - 127), 255 for 32 dims
// of which some are not finite.  So a token's codes and scales are its own:
// storing one never touches another's, whatever the order of the rows, and
// nothing is rounded twice.
//
// Keys lie as [T][D / 2], dim 2j in the lower half of byte j: sixteen bytes are 32 dims
// of a token, a quarter of a head of 128, which a lane loads at once and widens with one scale for
// four products of 32 dims.  Values lie in parts of 128, 64 or 32 dims as
// D is made of (96 = 64 + 32, 192 = 128 + 64): a sixteenth of the part's dims, b = 4,
// 2 or 1 bytes, of u = 16 / b tokens together, [T / u][16][u][b].  A lane then loads
// sixteen tokens of its dims in pieces of sixteen bytes, and one scale serves all
// dims that it has of a token.
#include "cache_common.h"

#include <math.h>

#include <type_traits>

namespace xfer {
namespace {

// -------------------------------------------------------------------- form
// The parts that the dims of a head are divided into.
constexpr int part_count(int d) { return d == 64 || d == 128 ? 1 : 2; }
constexpr int part_dims(int d, int p) {
  return p == 0 ? (d >= 128 ? 128 : 64) : d == 96 ? 32 : d == 192 ? 64 : 128;
}
constexpr int part_at(int d, int p) { return p == 0 ? 0 : part_dims(d, 0); }

__device__ __forceinline__ uint64_t keys4_at(const Shape& s, uint32_t block, uint32_t h) {
  return block * s.block_bytes + static_cast<uint64_t>(h) * s.T * s.D;
}
__device__ __forceinline__ uint64_t values4_at(const Shape& s, uint32_t block, uint32_t h) {
  return keys4_at(s, block, h) + s.T * s.D / 2;
}
// Of a side's dims 32 * group .. 32 * group + 31.
__device__ __forceinline__ uint64_t scales4_at(const Shape& s, uint32_t block, uint32_t h, uint32_t side,
                                               uint32_t group) {
  return block * s.block_bytes + static_cast<uint64_t>(s.H) * s.T * s.D +
         ((2 * h + side) * (s.D / 32) + group) * s.T;
}

int shape4_of(const xfer_cache_shape* g, const char* who, Shape* out) {
  const int rc = shape_of(g, who, out);
  if (rc) return rc;
  const uint64_t codes = uint64_t(out->H) * out->T * out->D;
  out->block_bytes = codes + ((codes / 16 + 127) & ~127ull);
  return XFER_OK;
}

// The power of two that a byte of w (0 the lowest) stands for; NaN for 255, as
// the conversions take it.
__device__ __forceinline__ float power_of(uint32_t w, uint32_t byte) {
  return __uint_as_float((w >> (8 * byte) & 255u) << 23);
}

// The two numbers of a byte of w, times scale: exact in bfloat16 and float for
// the scales of a cache, rounded to nearest even in float16.
__device__ __forceinline__ bf16x2 two_bf16(uint32_t w, int byte, float scale) {
  switch (byte) {
    case 0: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
    case 1: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
    case 2: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
    default: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  }
}
template <typename E>
__device__ __forceinline__ void eight_of(uint32_t w, float scale, E (&out)[8]) {
  if constexpr (__is_same(E, bf16_t)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x2 p = two_bf16(w, j, scale);
      out[2 * j] = p[0];
      out[2 * j + 1] = p[1];
    }
  } else if constexpr (__is_same(E, fp16_t)) {
    const fp16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 0);
    const fp16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 1);
    const fp16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 2);
    const fp16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 3);
    const E all[8] = {a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    __builtin_memcpy(out, all, sizeof(all));
  } else {
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0);
    const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
    const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2);
    const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
    const E all[8] = {a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    __builtin_memcpy(out, all, sizeof(all));
  }
}

// Byte j of the four words, as word j.
__device__ __forceinline__ void transpose(const uint32_t (&w)[4], uint32_t (&out)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u);
  const uint32_t b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
  const uint32_t d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  out[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// ------------------------------------------------------------------- store
struct Store4Args {
  uint8_t* cache;
  const void* key;
  const void* value;
  int64_t key_row, key_head, value_row, value_head;  // strides in elements
  const int32_t* slots;
  int32_t rows;
  Shape s;
};

// Exponent of the smallest power of two, 2^-118 to 2^125, that brings a magnitude
// (its bits, finite) to 7 = 1.75 * 2^2 or below.
__device__ __forceinline__ int exponent_of(uint32_t bits) {
  const int e = static_cast<int>(bits >> 23) - 127 - 2 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, -118), 125);
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Largest of x in four neighbouring lanes.
__device__ __forceinline__ uint32_t max_of_four(uint32_t x) {
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0xB1, 0xF, 0xF, true)));
  return max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x4E, 0xF, 0xF, true)));
}

// Eight neighbouring dims of a row.
template <typename E>
struct Piece {
  uint32_t w[2 * sizeof(E)];

  // Bits of the largest magnitude, as a float's (magnitudes are ordered as their
  // bits are, those that are not finite last).
  __device__ __forceinline__ uint32_t largest() const {
    if constexpr (sizeof(E) == 4) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, w[j] & 0x7FFFFFFFu);
      return m;
    } else {
      u16x2 m = {0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[j] & 0x7FFF7FFFu));
      const uint16_t most = max(m[0], m[1]);
      return __float_as_uint(static_cast<float>(__builtin_bit_cast(E, most)));
    }
  }
  // Their codes, dim j in bits 4j ..: divided by scale (a power of two) and rounded to
  // nearest even in one step, at most 6.
  __device__ __forceinline__ uint32_t codes(float scale) const {
    uint32_t r = 0;
    if constexpr (__is_same(E, bf16_t)) {
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w[0]), scale, 0);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w[1]), scale, 1);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w[2]), scale, 2);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w[3]), scale, 3);
    } else if constexpr (__is_same(E, fp16_t)) {
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(fp16x2, w[0]), scale, 0);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(fp16x2, w[1]), scale, 1);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(fp16x2, w[2]), scale, 2);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(fp16x2, w[3]), scale, 3);
    } else {
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(w[0]), __uint_as_float(w[1]), scale, 0);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(w[2]), __uint_as_float(w[3]), scale, 1);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(w[4]), __uint_as_float(w[5]), scale, 2);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(w[6]), __uint_as_float(w[7]), scale, 3);
    }
    return r;
  }
};

// Offset of dims 8 * piece .. of token t among a head's value codes: unit i of the
// value_units(piece) that eight dims are in.
template <int D>
__device__ __forceinline__ uint32_t value_unit_at(uint32_t T, uint32_t piece, uint32_t i, uint32_t t) {
  const uint32_t d = 8 * piece, p = part_count(D) > 1 && d >= part_dims(D, 0) ? 1 : 0;
  const uint32_t at = p ? part_at(D, 1) : 0, dims = p ? part_dims(D, 1) : part_dims(D, 0);
  const uint32_t b = dims / 32, u = 16 / b, n = (d - at) / (dims / 16) + i;
  return T * at / 2 + t / u * 256 + n * 16 + t % u * b;
}

constexpr int kStoreThreads = 256, kStoreEach = 2, kStoreRows = 16;

// A thread takes eight dims of one head and side of a row: four neighbours have
// the 32 that share a scale.  Rows are taken in tiles of 16, a head and side of all
// of them after the other, so that what one workgroup writes of neighbouring tokens
// fills whole lines; a workgroup takes the next kStoreEach * 256 pieces of eight.
//
// What bounds it is memory: the rows of 29 prompts, 54 M numbers of 16 bits, are stored in
// 23 us where they lie in the Infinity Cache (5.9 TB/s read and written).  New data, stored and
// read back by load_kernel, take 55 us for 272 MB, 5.0 TB/s (a large copy: 5.3).  Row by row the store
// alone took 30 (values of four tokens share a line, scales of 64: 63 MB written for
// 29), with one piece a thread both 54 and not 50 on data near at hand.
template <typename E, int D>
__global__ void __launch_bounds__(kStoreThreads) store4_kernel(Store4Args A) {
  constexpr uint32_t W = D / 8, kSide = kStoreRows * W;  // pieces of a row, of a tile's head and side
  const uint32_t tile_pieces = 2 * A.s.H * kSide;
  const uint64_t base = static_cast<uint64_t>(blockIdx.x) * (kStoreThreads * kStoreEach);
  const uint64_t tile0 = base / tile_pieces;
  const uint32_t rest = static_cast<uint32_t>(base - tile0 * tile_pieces) + threadIdx.x;
  Piece<E> all[kStoreEach];
  int32_t slots[kStoreEach];
  uint32_t where[kStoreEach];  // side and head
#pragma unroll
  for (int i = 0; i < kStoreEach; ++i) {
    const uint32_t q = rest + i * kStoreThreads, ahead = q / tile_pieces, c = q - ahead * tile_pieces;
    const uint32_t r = c / W % kStoreRows, piece = c % W;
    const uint32_t side = c / kSide >= A.s.H ? 1 : 0, h = c / kSide - side * A.s.H;
    const uint64_t row = (tile0 + ahead) * kStoreRows + r, last = static_cast<uint64_t>(A.rows) - 1;
    where[i] = 2 * h + side;
    slots[i] = A.slots[min(row, last)];  // (rows past the end are read as the last and dropped)
    if (row > last) slots[i] = -1;
    const E* src = static_cast<const E*>(side ? A.value : A.key) +
                   static_cast<int64_t>(min(row, last)) * (side ? A.value_row : A.key_row) +
                   static_cast<int64_t>(h) * (side ? A.value_head : A.key_head) + 8 * piece;
    __builtin_memcpy(&all[i], src, sizeof(all[i]));
  }
#pragma unroll
  for (int i = 0; i < kStoreEach; ++i) {
    const Piece<E>& x = all[i];
    const int32_t slot = slots[i];
    const uint32_t side = where[i] & 1, h = where[i] >> 1, piece = (rest + i * kStoreThreads) % W;
    const uint32_t most = max_of_four(x.largest());
    const uint32_t block = static_cast<uint32_t>(slot) >> A.s.log2T, t = static_cast<uint32_t>(slot) & (A.s.T - 1);
    if (slot < 0 || block >= A.s.blocks) continue;
    const bool fine = most < 0x7F800000u;
    const uint32_t e = fine ? static_cast<uint32_t>(exponent_of(most) + 127) : 255u;
    const uint32_t codes = fine ? x.codes(__uint_as_float(e << 23)) : 0u;
    if (side == 0) {
      *reinterpret_cast<uint32_t*>(A.cache + keys4_at(A.s, block, h) + t * (D / 2) + 4 * piece) = codes;
    } else {
      uint8_t* v = A.cache + values4_at(A.s, block, h);
      if (D >= 128 && (D != 192 || piece < 16)) {
        *reinterpret_cast<uint32_t*>(v + value_unit_at<D>(A.s.T, piece, 0, t)) = codes;
      } else if (D != 96 || piece < 8) {
        *reinterpret_cast<uint16_t*>(v + value_unit_at<D>(A.s.T, piece, 0, t)) = static_cast<uint16_t>(codes);
        *reinterpret_cast<uint16_t*>(v + value_unit_at<D>(A.s.T, piece, 1, t)) = static_cast<uint16_t>(codes >> 16);
      } else {
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
          v[value_unit_at<D>(A.s.T, piece, k, t)] = static_cast<uint8_t>(codes >> (8 * k));
      }
    }
    if (piece % 4 == 0) A.cache[scales4_at(A.s, block, h, side, piece / 4) + t] = static_cast<uint8_t>(e);
  }
}

using Store4Fn = void (*)(Store4Args);

template <typename E>
Store4Fn pick_store4(uint32_t d) {
  switch (d) {
    case 64: return store4_kernel<E, 64>;
    case 96: return store4_kernel<E, 96>;
    case 128: return store4_kernel<E, 128>;
    case 192: return store4_kernel<E, 192>;
    default: return store4_kernel<E, 256>;
  }
}

// -------------------------------------------------------------------- load
struct LoadArgs {
  const uint8_t* cache;
  void* key;
  void* value;
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* starts;
  int64_t key_row, key_head, value_row, value_head, table_stride;
  int32_t batch, rows, width;
  uint32_t numbers;  // of tiles
  Shape s;
};

constexpr int kLoadThreads = 256, kLoadEach = 2, kLoadShare = kLoadThreads * kLoadEach;
constexpr int kLoadTile = 16;  // tokens, the first a multiple of it

// Tiles numbered through the packed rows: request b's begin at number first(b) =
// starts[b] / 16 + 2 b.  Its rows, n of them, touch (n + 14) / 16 + 1 tiles at most, which
// is n / 16 + 2 or less.
__device__ __forceinline__ uint32_t first_load(const LoadArgs& A, uint32_t b) {
  return static_cast<uint32_t>(min(max(A.starts[b], 0), A.rows)) / kLoadTile + 2 * b;
}

// Four tokens' codes of eight dims of one side, and their scales.
template <int BITS, int D>
struct Quad;

template <int D>
struct Quad<4, D> {
  uint32_t w[4], s;
  __device__ __forceinline__ void load(const Shape& S, const uint8_t* cache, uint32_t block, uint32_t h,
                                       uint32_t side, uint32_t piece, uint32_t t) {
    s = *reinterpret_cast<const uint32_t*>(cache + scales4_at(S, block, h, side, piece / 4) + t);
    if (side == 0) {
      const uint8_t* k = cache + keys4_at(S, block, h) + t * (D / 2) + 4 * piece;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint32_t*>(k + j * (D / 2));
      return;
    }
    const uint8_t* v = cache + values4_at(S, block, h);
    if (D >= 128 && (D != 192 || piece < 16)) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(v + value_unit_at<D>(S.T, piece, 0, t));
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = x[j];
    } else if (D != 96 || piece < 8) {
      const u32x2 a = *reinterpret_cast<const u32x2*>(v + value_unit_at<D>(S.T, piece, 0, t));
      const u32x2 b = *reinterpret_cast<const u32x2*>(v + value_unit_at<D>(S.T, piece, 1, t));
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = __builtin_amdgcn_perm(b[j / 2], a[j / 2], j % 2 ? 0x07060302u : 0x05040100u);
    } else {
      uint32_t x[4];
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
        x[j] = *reinterpret_cast<const uint32_t*>(v + value_unit_at<D>(S.T, piece, j, t));
      transpose(x, w);
    }
  }
  template <typename E>
  __device__ __forceinline__ void rows(int j, E (&out)[8]) const {
    eight_of<E>(w[j], power_of(s, j), out);
  }
};

template <int D>
struct Quad<8, D> {
  uint32_t w[4][2];
  float s;
  __device__ __forceinline__ void load(const Shape& S, const uint8_t* cache, uint32_t block, uint32_t h,
                                       uint32_t side, uint32_t piece, uint32_t t) {
    const uint8_t* p = cache + block * S.block_bytes;
    s = reinterpret_cast<const float*>(p + 2ull * S.H * S.T * D)[2 * h + side];
    p += (2ull * h + side) * S.T * D;
    if (side == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x2 x = *reinterpret_cast<const u32x2*>(p + (t + j) * D + 8 * piece);
        w[j][0] = x[0];
        w[j][1] = x[1];
      }
      return;
    }
    uint32_t x[2][4], y[4];
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k)
      x[k / 4][k % 4] = *reinterpret_cast<const uint32_t*>(p + (8 * piece + k) * S.T + t);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      transpose(x[i], y);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j][i] = y[j];
    }
  }
  template <typename E>
  __device__ __forceinline__ void rows(int j, E (&out)[8]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t x = w[j][i];
      if constexpr (__is_same(E, bf16_t)) {
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, s, false);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, s, true);
        const E all[4] = {a[0], a[1], b[0], b[1]};
        __builtin_memcpy(out + 4 * i, all, sizeof(all));
      } else if constexpr (__is_same(E, fp16_t)) {
        const fp16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, s, false);
        const fp16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, s, true);
        const E all[4] = {a[0], a[1], b[0], b[1]};
        __builtin_memcpy(out + 4 * i, all, sizeof(all));
      } else {
        const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(x, s, false);
        const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(x, s, true);
        const E all[4] = {a[0], a[1], b[0], b[1]};
        __builtin_memcpy(out + 4 * i, all, sizeof(all));
      }
    }
  }
};

// A workgroup takes a tile of a request's tokens and, of the tile's keys and values,
// its share: a thread twice four tokens of eight dims at a time, neighbours the
// neighbouring dims, so that rows are written in long pieces.  (A block outside the
// cache is read as block 0, and its rows are zeros: a branch around the loads would
// make the second wait for the first.)
//
// What bounds it is memory, four fifths of it the rows written: 24 prefixes of up to 9001 tokens
// from 4 bits, 300 MB, take 61 us (4.9 TB/s) of new data and 52 (5.7) of data in the Infinity
// Cache, 17 of up to 12001 from 8, 255 MB, 73 (3.5) and 53 (4.8).  With one load a thread in
// flight the latter take 20 and 9 us more.
template <int BITS, typename E, int D>
__global__ void __launch_bounds__(kLoadThreads) load_kernel(LoadArgs A) {
  constexpr uint32_t W = D / 8;
  const uint32_t lane = threadIdx.x & 63u;
  for (uint32_t k = blockIdx.x; k < A.numbers; k += gridDim.x) {
    // the last request that begins at or before number k, by a lane per candidate
    uint32_t b = 0, n = A.batch;
    while (n > 1) {
      const uint32_t step = (n + 63) / 64, at = lane * step;
      const bool there = at < n && first_load(A, b + at) <= k;
      const uint32_t pos = max(static_cast<uint32_t>(__popcll(__ballot(there))), 1u) - 1;
      b += pos * step;
      n = min(step, n - pos * step);
    }
    b = uniform(b);
    const int64_t start = A.starts[b], end = min<int64_t>(A.starts[b + 1], A.rows);
    if (start < 0 || end <= start) continue;
    // row start holds token ahead (it may be negative: then there is none)
    const int64_t ahead = static_cast<int64_t>(A.lengths[b]) - (static_cast<int64_t>(A.starts[b + 1]) - start);
    const int64_t tile = (ahead >> 4) + (k - first_load(A, b));
    if (tile * kLoadTile >= ahead + (end - start)) continue;
    const int64_t t0 = tile * kLoadTile, page = t0 >> A.s.log2T;
    int32_t block = -1;
    if (t0 >= 0 && page < A.width) block = A.table[b * A.table_stride + page];
    if (static_cast<uint32_t>(block) >= A.s.blocks) block = -1;
    const uint32_t off = static_cast<uint32_t>(t0) & (A.s.T - 1);
    const uint32_t side_pieces = A.s.H * W, all = 2 * 4 * side_pieces;
    const uint32_t from = max(block, 0);
    for (uint32_t i0 = blockIdx.y * kLoadShare + threadIdx.x; i0 < all; i0 += gridDim.y * kLoadShare) {
      Quad<BITS, D> q[kLoadEach];
#pragma unroll
      for (int z = 0; z < kLoadEach; ++z) {
        const uint32_t i = min(i0 + z * kLoadThreads, all - 1);
        const uint32_t quad = i / side_pieces & 3u, side = i / side_pieces >> 2, c = i % side_pieces;
        q[z].load(A.s, A.cache, from, c / W, side, c % W, off + 4 * quad);
      }
#pragma unroll
      for (int z = 0; z < kLoadEach; ++z) {
        const uint32_t i = i0 + z * kLoadThreads;
        if (i >= all) continue;
        const uint32_t quad = i / side_pieces & 3u, side = i / side_pieces >> 2, c = i % side_pieces;
        const uint32_t h = c / W, piece = c % W;
        E* out = static_cast<E*>(side ? A.value : A.key) +
                 static_cast<int64_t>(h) * (side ? A.value_head : A.key_head) + 8 * piece;
        const int64_t stride = side ? A.value_row : A.key_row;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t row = start + t0 + 4 * quad + j - ahead;
          if (row < start || row >= end) continue;
          E x[8] = {};
          if (block >= 0) q[z].rows(j, x);
          __builtin_memcpy(out + row * stride, x, sizeof(x));
        }
      }
    }
  }
}

using LoadFn = void (*)(LoadArgs);

template <int BITS, typename E>
LoadFn pick_load_dim(uint32_t d) {
  switch (d) {
    case 64: return load_kernel<BITS, E, 64>;
    case 96: return load_kernel<BITS, E, 96>;
    case 128: return load_kernel<BITS, E, 128>;
    case 192: return load_kernel<BITS, E, 192>;
    default: return load_kernel<BITS, E, 256>;
  }
}

template <int BITS>
LoadFn pick_load(uint32_t d, int dtype) {
  return dtype == XFER_BF16   ? pick_load_dim<BITS, bf16_t>(d)
         : dtype == XFER_FP16 ? pick_load_dim<BITS, fp16_t>(d)
                              : pick_load_dim<BITS, float>(d);
}

// ------------------------------------------------------------------ attend
// Step k of 32 dims of the score product takes dims key4_dim(k, g) .. + 7 from lane
// group g: a part's steps follow one another in the lane's load of it.
template <int D>
__device__ __forceinline__ uint32_t key4_dim(uint32_t k, uint32_t g) {
  const uint32_t p = part_count(D) > 1 && k >= part_dims(D, 0) / 32 ? 1 : 0;
  const uint32_t at = p ? part_at(D, 1) : 0, dims = p ? part_dims(D, 1) : part_dims(D, 0);
  return at + dims / 4 * g + 8 * (k - at / 32);
}

template <bool ONCE, int WORDS>
__device__ __forceinline__ void fetch_words(const uint8_t* p, uint32_t* w) {
  if constexpr (WORDS == 4) {
    const u32x4 x = fetch<ONCE, u32x4>(p);
    for (int i = 0; i < 4; ++i) w[i] = x[i];
  } else if constexpr (WORDS == 2) {
    const u32x2 x = fetch<ONCE, u32x2>(p);
    for (int i = 0; i < 2; ++i) w[i] = x[i];
  } else {
    w[0] = fetch<ONCE, uint32_t>(p);
  }
}

// f(part, its number as a constant) for every part of D.
template <int D, typename F>
__device__ __forceinline__ void each_part(F&& f) {
  f(std::integral_constant<int, 0>());
  if constexpr (part_count(D) > 1) f(std::integral_constant<int, 1>());
}

// A chunk's key codes and scales: tile t's line n of a lane.
template <int D, bool ONCE>
struct Keys4 {
  uint32_t w[4][D / 32];
  u32x4 s[part_count(D)];
  __device__ __forceinline__ void load(const AttendArgs& A, const Place& at, uint32_t t0, uint32_t h,
                                       uint32_t g, uint32_t n) {
    const uint32_t block = at.line, tk = (t0 + 16 * (n >> 2)) & (A.s.T - 1);
    const uint8_t* k = A.cache + keys4_at(A.s, block, h) + (tk + (n & 3u)) * (D / 2);
    const uint8_t* x = A.cache + scales4_at(A.s, block, h, 0, 0) + tk;
    each_part<D>([&](auto part) {
      constexpr int p = part.value, dims = part_dims(D, p), from = part_at(D, p);
#pragma unroll
      for (int t = 0; t < 4; ++t)
        fetch_words<ONCE, dims / 32>(k + 4 * t * (D / 2) + from / 2 + dims / 8 * g, &w[t][from / 32]);
      s[p] = fetch<ONCE, u32x4>(x + (from / 32 + g * (dims / 32) / 4) * A.s.T);
    });
  }
};

// A chunk's value codes and scales: sixteen tokens of a lane.
template <int D, bool ONCE>
struct Values4 {
  u32x4 w[D / 32];
  u32x4 s[part_count(D)];
  __device__ __forceinline__ void load(const AttendArgs& A, const Place& at, uint32_t t0, uint32_t h,
                                       uint32_t g, uint32_t n) {
    const uint32_t block = max(at.mine, 0), T = A.s.T, t = (t0 + 16 * g) & (T - 1);
    const uint8_t* v = A.cache + values4_at(A.s, block, h) + n * 16;
    const uint8_t* x = A.cache + scales4_at(A.s, block, h, 1, 0) + t;
    each_part<D>([&](auto part) {
      constexpr int p = part.value, dims = part_dims(D, p), from = part_at(D, p), b = dims / 32;
#pragma unroll
      for (int i = 0; i < b; ++i)
        w[from / 32 + i] = fetch<ONCE, u32x4>(v + T * from / 2 + t * b * 16 + i * 256);
      s[p] = fetch<ONCE, u32x4>(x + (from / 32 + n * b / 16) * T);
    });
  }
};

// Which of the parts' 32 dims that a lane holds results of have a token t0 .. last whose
// values are not finite: NaN for those, else 0.  Rarely run, so it is a plain loop.
template <int D>
__device__ __forceinline__ void seen_nans4(const AttendArgs& A, const int32_t* table, uint32_t h, int32_t t0,
                                           int32_t last, uint32_t g, float (&r)[part_count(D)]) {
#pragma clang loop unroll(disable)
  for (int32_t t = t0; t <= last; ++t) {
    const int32_t id = table[t >> A.s.log2T];
    if (static_cast<uint32_t>(id) >= A.s.blocks) continue;
    each_part<D>([&](auto part) {
      constexpr int p = part.value, dims = part_dims(D, p), from = part_at(D, p);
      const uint32_t group = from / 32 + g * (dims / 32) / 4;
      if (A.cache[scales4_at(A.s, id, h, 1, group) + (t & (A.s.T - 1))] == 255) r[p] = NAN;
    });
  }
}

// A float16 query as the sum of two bfloat16 numbers, exactly: it has 11 significant
// bits, the rounded one takes 8 of them.
__device__ __forceinline__ void two_parts(u32x4 q, u32x4& hi, u32x4& lo) {
  const fp16x8 x = __builtin_bit_cast(fp16x8, q);
  bf16x8 a, b;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float v = static_cast<float>(x[j]);
    a[j] = static_cast<bf16_t>(v);
    b[j] = static_cast<bf16_t>(fabsf(v) <= 65504.0f ? v - static_cast<float>(a[j]) : 0.0f);
  }
  hi = __builtin_bit_cast(u32x4, a);
  lo = __builtin_bit_cast(u32x4, b);
}

__device__ __forceinline__ bf16x8 widen4(uint32_t w, float scale) {
  bf16x8 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bf16x2 p = two_bf16(w, j, scale);
    r[2 * j] = p[0];
    r[2 * j + 1] = p[1];
  }
  return r;
}

// The largest of x in the four lanes n, n + 16, n + 32, n + 48.
__device__ __forceinline__ float max_of_groups(float x) {
  const uint32_t a = __float_as_uint(x);
  const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  x = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
  const uint32_t b = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The weights of a chunk's scores s, in units of 1 / mul, as two bfloat16 numbers each:
// p the rounded ones, p2 the rounded rests.  Maxima m, sums l and accumulators acc go
// along.  MASK: some row does not see some token of the chunk; limit: the last token
// that each row sees; tg: the lane's first of sixteen; bg: their block (below 0: none).
template <bool MASK, int DT>
__device__ __forceinline__ void weights_of(f32x4 (&s)[4], f32x4 (&acc)[DT], float (&m),
                                           float (&l), const int32_t (&limit), float mul,
                                           int32_t tg, int32_t bg, bf16x8 (&p)[2],
                                           bf16x8 (&p2)[2]) {
  const int32_t seen = bg < 0 ? 0 : limit - tg + 1;  // of this lane's sixteen tokens
  float top = -INFINITY;
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float v = s[t][r] * mul;
      if (MASK && 4 * t + r >= seen) v = -INFINITY;
      s[t][r] = v;
      top = fmaxf(top, v);
    }
  top = max_of_groups(top);
  // The reference m follows the maximum only when that is 8 above it, so most
  // chunks leave the accumulators alone: weights reach 256 at most, and the
  // same powers of two leave sums and accumulators in the end.
  const bool grows = top > m + 8.0f;
  const float next = grows ? top : m, base = next == -INFINITY ? 0.0f : next;
  const float keep = grows ? __builtin_amdgcn_exp2f(m - base) : 1.0f;
  m = next;
  float sum = 0.0f;
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float w = __builtin_amdgcn_exp2f(s[t][r] - base);
      sum += w;
      const bf16_t first = static_cast<bf16_t>(w);
      p[t >> 1][(t & 1) * 4 + r] = first;
      p2[t >> 1][(t & 1) * 4 + r] = static_cast<bf16_t>(w - static_cast<float>(first));
    }
  l = l * keep + sum;
  if (__ballot(grows) != 0) {
#pragma unroll
    for (int e = 0; e < DT; ++e) acc[e] *= keep;
  }
}

// The thread's number, of which nothing that follows is worked out before a loop around the
// caller: registers would have to hold it.
__device__ __forceinline__ uint32_t thread_here() {
  uint32_t tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  return tid;
}

// Writes the sixteen rows first .. of a request from what each wave of the workgroup
// has of them: its sums of weighted values acc, relative to the rows' largest maximum
// already, and its maxima m and sums l, `stride` from a wave's to the next's.  part
// null: the rows of out and lse, else their sums to part and stats.
template <typename E, int D>
__device__ __forceinline__ void write_rows(const AttendArgs& A, const float (&acc)[kAttendWaves][16][D + 4],
                                           const float* m, const float* l, uint32_t stride,
                                           const RowTile& rt, uint32_t h, uint32_t first, float* part,
                                           float* stats) {
  for (uint32_t i = thread_here(); i < 16 * (D / 4); i += kAttendWaves * 64) {
    const uint32_t r = i / (D / 4), d = i % (D / 4) * 4, ri = first + r;
    const int64_t row = rt.start + ri / A.group;
    if (ri >= rt.rows) continue;
    float top = m[r], sum = 0.0f;
    for (int w = 1; w < kAttendWaves; ++w) top = fmaxf(top, m[w * stride + r]);
    const float base = top == -INFINITY ? 0.0f : top;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int w = 0; w < kAttendWaves; ++w) {
      sum += l[w * stride + r] * __builtin_amdgcn_exp2f(m[w * stride + r] - base);
      o += *reinterpret_cast<const f32x4*>(&acc[w][r][d]);
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
      *reinterpret_cast<f32x4*>(part + r * D + d) = o;
      if (d == 0) {
        stats[r * 2] = top;
        stats[r * 2 + 1] = sum;
      }
    }
  }
}

// The product of a chunk's weights p + p2 with the values.  A byte of codes gives two
// dims of a token, the left operand wants eight tokens of a dim: two bytes of
// neighbouring tokens, each widened with its own scale, and the halves put together.
template <int D>
__device__ __forceinline__ void weigh4(const u32x4 (&w)[D / 32], const u32x4 (&vs)[part_count(D)],
                                       const bf16x8 (&p)[2], const bf16x8 (&p2)[2],
                                       f32x4 (&acc)[D / 16]) {
  each_part<D>([&](auto part) {
    constexpr int pt = part.value, dims = part_dims(D, pt), from = part_at(D, pt), b = dims / 32;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float scale[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) scale[k] = power_of(vs[pt][2 * s + k / 4], k % 4);
#pragma unroll
      for (int j = 0; j < b; ++j) {
        u32x4 even, odd;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t c[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int byte = (8 * s + 2 * k + i) * b + j;
            c[i] = __builtin_bit_cast(
                uint32_t, two_bf16(w[from / 32 + byte / 16][byte / 4 % 4], byte % 4, scale[2 * k + i]));
          }
          even[k] = __builtin_amdgcn_perm(c[1], c[0], 0x05040100u);
          odd[k] = __builtin_amdgcn_perm(c[1], c[0], 0x07060302u);
        }
        const bf16x8 a = __builtin_bit_cast(bf16x8, even), z = __builtin_bit_cast(bf16x8, odd);
        f32x4& e = acc[from / 16 + 2 * j];
        f32x4& o = acc[from / 16 + 2 * j + 1];
        e = mfma(a, p[s], e);
        o = mfma(z, p[s], o);
        e = mfma(a, p2[s], e);
        o = mfma(z, p2[s], o);
        if constexpr (D >= 192) __builtin_amdgcn_sched_barrier(0);
      }
    }
  });
}

// The scales of tokens that no row sees are replaced by 1, as they may be anything and 0
// times infinity or NaN is NaN; so are the NaN of the others, which reach the rows
// that see their token and no other: they are looked for again in memory at the end.
__device__ __forceinline__ void mask_scales(u32x4& v, int32_t held, uint32_t& nans) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int left = held - 4 * w;
    const uint32_t mask = left <= 0 ? 0u : left >= 4 ? ~0u : (1u << (8 * left)) - 1u;
    const uint32_t nan = (((v[w] & 0x7F7F7F7Fu) + 0x01010101u) & v[w] & 0x80808080u & mask) >> 7;
    nans |= nan;
    const uint32_t keep = mask & ~(nan * 0xFFu);
    v[w] = (v[w] & keep) | (0x7F7F7F7Fu & ~keep);
  }
}

template <typename E, int D>
struct Shared4 {
  static constexpr int kQueries = __is_same(E, fp16_t) ? 2 : 1;  // bfloat16 numbers of one
  union {
    u32x4 q[kQueries][D / 32][64];  // the rows' queries, in the order of the matrix operand
    float acc[kAttendWaves][16][D + 4];
  };
  float m[kAttendWaves][16], l[kAttendWaves][16];
};

constexpr int attend4_resident(int d) { return d <= 96 ? 3 : 2; }

// Attention as over 8-bit codes (cache.hip's kernels have its mathematics: which token
// sits where, one running maximum and sum a wave, weights in two bfloat16 numbers):
// S^T = K Q^T and O^T = V^T P^T on the 16x16x32 matrix instruction, the cache's codes
// the left operand, waves that take chunks of 64 tokens in turn.  What differs: scales
// belong to a token's 32 dims, so keys and values are widened with them to
// bfloat16, exactly; a float16 query goes in two bfloat16 numbers, exactly, since
// keys need bfloat16's range; a lane's result tile e of a part holds dims b' n + e, the
// b' dims that its sixteen-byte pieces have of each token.
template <typename E, int D, bool ONCE>
struct Core4 {
  typedef E Elem;
  typedef Shared4<E, D> Shared;
  static constexpr int kDim = D, kRows = 16, kThreads = kAttendWaves * 64;
  static constexpr int kResident = attend4_resident(D);

  static __device__ __forceinline__ void rows(const AttendArgs& A, Shared& sh, uint32_t b, uint32_t h,
                                              uint32_t first, uint32_t c0, uint32_t c1, float* part,
                                              float* stats) {
    constexpr int KL = D / 32, DT = D / 16, NQ = Shared::kQueries;
    const uint32_t tid = thread_here(), lane = tid & 63u, n = lane & 15u, g = lane >> 4;
    const uint32_t wave = uniform(tid >> 6);
    const int32_t* table = A.table + static_cast<int64_t>(b) * A.table_stride;
    const RowTile rt = row_tile(A, b, first, kRows);
    c1 = min(c1, (static_cast<uint32_t>(rt.seen) + kChunk - 1) / kChunk);

    // (waves with no chunk load too, any block: behind a branch around the loads every
    // wait of the loop would be one for all of them)
    const uint32_t seen_all = uniform(static_cast<uint32_t>(rt.seen)), reach = max(seen_all, 1u);
    if (seen_all == 0) table = A.starts;
    uint32_t c = c0 + wave, nans = 0;
    Keys4<D, ONCE> keys;
    Values4<D, ONCE> vals;
    Place at, next;
    constexpr uint32_t kNext = kAttendWaves * kChunk;  // tokens from a wave's chunk to its next
    at.look(A, table, c * kChunk, reach, g, n);
    next.look(A, table, c * kChunk + kNext, reach, g, n);
    __builtin_amdgcn_sched_barrier(0);

    constexpr int QL = (KL + kAttendWaves - 1) / kAttendWaves;
    int32_t limit;            // last token that the row sees
    int32_t least = rt.seen;  // the first of them
    u32x4 q[QL];
    const uint32_t i = first + n;
    const int64_t j = i / A.group, row = rt.start + j;
    const bool there = i < rt.rows;
    limit = there ? static_cast<int32_t>(max<int64_t>(-1, min<int64_t>(rt.seen - 1, rt.ahead + j))) : -1;
    const E* p = static_cast<const E*>(A.query) + row * A.query_row +
                 static_cast<int64_t>(h * A.group + i % A.group) * A.query_head;
#pragma unroll
    for (int k = 0; k < QL; ++k) {
      q[k] = u32x4{0u, 0u, 0u, 0u};
      const uint32_t step = wave + k * kAttendWaves;
      if (there && step < KL) __builtin_memcpy(&q[k], p + key4_dim<D>(step, g), 16);
    }
    if (there) least = min(least, limit);  // (other rows hold zeros and go nowhere)
    at.settle(A, c * kChunk, seen_all, g);
    keys.load(A, at, c * kChunk, h, g, n);
    __builtin_amdgcn_sched_barrier(0);
    vals.load(A, at, c * kChunk, h, g, n);
#pragma unroll
    for (int k = 0; k < QL; ++k) {
      const uint32_t step = wave + k * kAttendWaves;
      if (step >= KL) continue;
      if constexpr (NQ == 2) {
        u32x4 hi, lo;
        two_parts(q[k], hi, lo);
        sh.q[0][step][lane] = hi;
        sh.q[NQ - 1][step][lane] = lo;
      } else {
        sh.q[0][step][lane] = q[k];
      }
    }
    for (int d = 1; d < 16; d <<= 1) least = min(least, __shfl_xor(least, d));
    least = __builtin_amdgcn_readfirstlane(least);
    __syncthreads();

    float m, l;
    f32x4 acc[DT];
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < DT; ++e) acc[e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // The order of loads is that of the 8-bit codes: the next chunk's keys once this
    // one's scores are done, its values once this one's are used up.
    auto step = [&](auto masked) {
      constexpr bool MASK = decltype(masked)::value;
      const uint32_t t0 = c * kChunk, tg = t0 + 16 * g, ahead = t0 + kNext;
      const int32_t bg = at.mine;
      f32x4 s[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) s[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < KL; ++k) {
        constexpr int kFirst = part_dims(D, 0) / 32;
        const int pt = k < kFirst ? 0 : part_count(D) - 1;
        bf16x8 b8[NQ];
#pragma unroll
        for (int i = 0; i < NQ; ++i)
          b8[i] = __builtin_bit_cast(bf16x8, sh.q[i][k][lane]);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const bf16x8 a = widen4(keys.w[t][k], power_of(keys.s[pt][t], n & 3u));
#pragma unroll
          for (int i = NQ - 1; i >= 0; --i)
            s[t] = mfma(a, b8[i], s[t]);
        }
        if constexpr (D >= 192) __builtin_amdgcn_sched_barrier(0);  // (or registers run out)
      }
      __builtin_amdgcn_sched_barrier(0);
      next.settle(A, ahead, seen_all, g);
      keys.load(A, next, ahead, h, g, n);
      __builtin_amdgcn_sched_barrier(0);
      bf16x8 p[2], p2[2];
      weights_of<MASK, DT>(s, acc, m, l, limit, A.scale2, tg, bg, p, p2);
      if constexpr (MASK) {
        const int32_t held = bg < 0 ? 0 : static_cast<int32_t>(seen_all) - static_cast<int32_t>(tg);
#pragma unroll
        for (int k = 0; k < part_count(D); ++k) mask_scales(vals.s[k], held, nans);
      }
      weigh4<D>(vals.w, vals.s, p, p2, acc);
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
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
      sh.m[wave][n] = m;
      sh.l[wave][n] = l;
    }
    __syncthreads();  // (and no wave needs the queries any more)
    float top = sh.m[0][n];
    for (int w = 1; w < kAttendWaves; ++w) top = fmaxf(top, sh.m[w][n]);
    const float f = __builtin_amdgcn_exp2f(m - (top == -INFINITY ? 0.0f : top));
    float nan[part_count(D)] = {};
    if (any_nan) {
#pragma clang loop unroll(disable)
      for (uint32_t i = rest; i < c1; i += kAttendWaves)
        seen_nans4<D>(A, table, h, i * kChunk, min(static_cast<int32_t>(i * kChunk) + kChunk - 1, limit), g, nan);
    }
    // result tile e of a part, row 4g + r of it: dim dims / 16 * (4g + r) + e
    each_part<D>([&](auto pt) {
      constexpr int k = pt.value, wide = part_dims(D, k) / 16, from = part_at(D, k);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < wide; ++e)
          sh.acc[wave][n][from + wide * (4 * g + r) + e] = acc[from / 16 + e][r] * f + nan[k];
    });
    __syncthreads();
    write_rows<E, D>(A, sh.acc, &sh.m[0][0], &sh.l[0][0], 16, rt, h, first, part, stats);
    __syncthreads();
  }
};

// ---------------------------------------------------------- attend, many rows
// Where a request has many rows, every wave takes 16 NR of them, a tile of rows is
// four waves', and its keys and values are widened once for all of them: wave t
// widens tile t of the keys, and half of the dims of half of the tokens' values, and
// writes the left operands to shared memory, each lane's sixteen bytes where it will
// read them.
//
// Weights of bfloat16 queries are held as those of few rows' attention: two bfloat16 numbers
// (off by 2^-16), relative to a reference that they are 256 times at most.
//
// Those of float16 queries, and keys and values, are float16 numbers where the chunk's scale
// bytes lie in 104 .. 135: code * 2^e is one, exactly, for e from -23 to 8, and queries stay as
// they are.  A rounded weight is then off by half a step, 2^-11 of itself, or by 2^-25
// where it is below float16's normal numbers, 2^-32 of the row's largest: maxima
// lie 7 to 15 powers of two above the reference, so weights reach 2^15.  A second number takes the
// rest (2^-22).  Other chunks take bfloat16 numbers, in a pass of their own behind the first: a
// store of zeros has a scale byte of 9, and with one such token in each request 5 prompts take
// 144 us; 246 where all behind it went on in bfloat16 numbers, 132 without it.  If no chunk is of
// float16 numbers the first pass is in vain (270 and not 248).  (In one pass registers spill: the
// accumulators are held twice where two loops may each follow the other.)
//
// Tried: one float16 number for bfloat16 queries.  Chunks take 76 us so and 87 with two numbers,
// which cost as much in either type; but where values cancel the output is off by far more than
// its own rounding, and whether a row is would depend on the call around it.
//
// What bounds it is instructions: with one number a weight a chunk of 64 tokens and 128 rows of 128
// dims took about 4300 cycles (widening 800, scores 770, weights 1170, products 630, loads and
// barriers the rest); the second number's products are 630 more.  8 chunks of prompts over up to
// 5000 tokens take 86 us, 5 prompts of up to 2900 tokens 123.  Tried and slower: the next chunk
// widened between this one's products (in the same wave), eight waves in two halves that take turns
// at widening and multiplying (88 and 235 us, where four took 81 and 179).
constexpr int wide_tiles(int d) { return d <= 128 ? 2 : 1; }    // of 16 rows, of a wave
constexpr int wide_buffers(int d) { return d <= 128 ? 2 : 1; }  // of widened chunks

template <typename E, int D, int NR>
struct WideShared {
  static constexpr int kKeys = 4 * (D / 32), kValues = 2 * (D / 16);
  union {
    u32x4 tile[wide_buffers(D)][kKeys + kValues][64];
    Shared4<E, D> few;
  };
  uint32_t nans[kAttendWaves];  // whether a wave met a value that is not a number
};

// Whether all of a word's four scales lie within 104 .. 135 (2^-23 .. 2^8): 24 is added to each
// byte, and its upper three bits are 100 then.
__device__ __forceinline__ bool float16_scales(uint32_t w) {
  return ((((w & 0x7F7F7F7Fu) + 0x18181818u) ^ (w & 0x80808080u)) & 0xE0E0E0E0u) == 0x80808080u;
}

__device__ __forceinline__ fp16x2 two_fp16(uint32_t w, int byte, float scale) {
  switch (byte) {
    case 0: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 0);
    case 1: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 1);
    case 2: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 2);
    default: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 3);
  }
}
template <bool HALF>
__device__ __forceinline__ uint32_t two_of(uint32_t w, int byte, float scale) {
  if constexpr (HALF)
    return __builtin_bit_cast(uint32_t, two_fp16(w, byte, scale));
  else
    return __builtin_bit_cast(uint32_t, two_bf16(w, byte, scale));
}
template <bool HALF>
__device__ __forceinline__ f32x4 mfma_of(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (HALF)
    return mfma(__builtin_bit_cast(fp16x8, a), __builtin_bit_cast(fp16x8, b), c);
  else
    return mfma(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c);
}

// The power of two that byte k of w stands for, in one instruction.
template <int K>
__device__ __forceinline__ float power_at(uint32_t w) {
  uint32_t r;
  if constexpr (K == 0)
    asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_0"
        : "=v"(r)
        : "v"(23u), "v"(w));
  else if constexpr (K == 1)
    asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_1"
        : "=v"(r)
        : "v"(23u), "v"(w));
  else if constexpr (K == 2)
    asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_2"
        : "=v"(r)
        : "v"(23u), "v"(w));
  else
    asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_3"
        : "=v"(r)
        : "v"(23u), "v"(w));
  return __uint_as_float(r);
}

// What a wave widens of a chunk, as loaded, and the scales that decide how.
template <int D>
struct WideCodes {
  static constexpr int kAll = (D / 32 + 3) / 4;  // words of a lane that hold all of a side's scales
  uint32_t k[D / 32], v[D / 16];
  uint32_t ks[part_count(D)], vs[part_count(D)][2];
  uint32_t all[2][kAll];

  // Where a lane loads within a block: chunks begin at multiples of 64 tokens, so it is the same for all.
  struct From {
    uint32_t key[part_count(D)], key_scale[part_count(D)], value[part_count(D)];
    uint32_t value_scale[part_count(D)], all[kAll];
    uint32_t side;  // bytes from a head's scales of keys to its values'
    __device__ __forceinline__ From(const AttendArgs& A, uint32_t h, uint32_t g, uint32_t n, uint32_t wave) {
      const uint32_t T = A.s.T, tk = 16 * (n >> 2) & (T - 1), tv = 16 * g & (T - 1), s = wave >> 1;
      const uint32_t tn = tk + 4 * wave + (n & 3u), codes = h * T * D, scales = A.s.H * T * D + 2 * h * (D / 32) * T;
      side = D / 32 * T;
      each_part<D>([&](auto part) {
        constexpr int p = part.value, dims = part_dims(D, p), at = part_at(D, p), b = dims / 32;
        key[p] = codes + tn * (D / 2) + at / 2 + dims / 8 * g;
        key_scale[p] = scales + (at / 32 + g * b / 4) * T + tn;
        // (sixteen tokens of a lane are b pieces of sixteen bytes, 256 bytes apart)
        value[p] = codes + T * D / 2 + T * at / 2 + tv * b * 16 + n * 16 + (b == 1 ? 8 * s : 128 * b * s);
        value_scale[p] = scales + side + (at / 32 + n * b / 16) * T + tv + 8 * s;
      });
#pragma unroll
      for (int i = 0; i < kAll; ++i) all[i] = scales + min(4 * i + g, D / 32 - 1u) * T + tk + 4 * (n & 3u);
    }
  };

  template <bool QUERIES16>  // (whose keys' scales are asked about too)
  __device__ __forceinline__ void load(const AttendArgs& A, const Place& at, const From& from) {
    const uint32_t bytes = static_cast<uint32_t>(A.s.block_bytes);
    const uint8_t* kb = A.cache + static_cast<uint64_t>(static_cast<uint32_t>(at.line)) * bytes;
    const uint8_t* vb = A.cache + static_cast<uint64_t>(static_cast<uint32_t>(max(at.mine, 0))) * bytes;
    each_part<D>([&](auto part) {
      constexpr int p = part.value, dims = part_dims(D, p), at = part_at(D, p), b = dims / 32;
      fetch_words<false, b>(kb + from.key[p], &k[at / 32]);
      ks[p] = kb[from.key_scale[p]];
      const uint8_t* q = vb + from.value[p];  // (eight tokens of b bytes)
      if constexpr (b == 4) {
        fetch_words<false, 4>(q, &v[at / 16]);
        fetch_words<false, 4>(q + 256, &v[at / 16 + 4]);
      } else {
        fetch_words<false, 2 * b>(q, &v[at / 16]);
      }
      fetch_words<false, 2>(vb + from.value_scale[p], vs[p]);
    });
    if constexpr (QUERIES16) {
#pragma unroll
      for (int i = 0; i < kAll; ++i)
#pragma unroll
        for (int side = 0; side < 2; ++side)
          all[side][i] = *reinterpret_cast<const uint32_t*>(kb + from.all[i] + side * from.side);
    }
  }

  // Whether all scales of tokens that some row sees are float16's.  mine: the block of the lane's sixteen
  // tokens from 16 g on (below 0: none, and no row sees them; what was loaded in their place is of block 0).
  __device__ __forceinline__ bool float16(uint32_t t0, uint32_t seen, uint32_t n, int32_t mine) const {
    bool ok = true;
    const int32_t left = static_cast<int32_t>(seen) - static_cast<int32_t>(t0 + 16 * (n >> 2) + 4 * (n & 3u));
    const bool none = (__ballot(mine < 0) >> (16 * (n >> 2)) & 1) != 0;
    const uint32_t mask = none || left <= 0 ? 0u : left >= 4 ? ~0u : (1u << (8 * left)) - 1u;
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll
      for (int i = 0; i < kAll; ++i) ok &= float16_scales((all[side][i] & mask) | (0x7F7F7F7Fu & ~mask));
    return __ballot(ok) == ~0ull;
  }

  // Replaces, as mask_scales, the scales of values that no row sees (held: tokens from the
  // lane's sixteen on that some row does), and NaN where HALF has none.
  template <bool HALF>
  __device__ __forceinline__ void mask(uint32_t wave, int32_t held, uint32_t& nans) {
    if (HALF && __ballot(held < 16) == 0) return;
    const int32_t left = held - 8 * static_cast<int32_t>(wave >> 1);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int more = left - 4 * w;
      const uint32_t seen = more <= 0 ? 0u : more >= 4 ? ~0u : (1u << (8 * more)) - 1u;
#pragma unroll
      for (int p = 0; p < part_count(D); ++p) {
        uint32_t x = vs[p][w], keep = seen;
        if constexpr (!HALF) {
          const uint32_t nan = (((x & 0x7F7F7F7Fu) + 0x01010101u) & x & 0x80808080u & seen) >> 7;
          nans |= nan;
          keep &= ~(nan * 0xFFu);
        }
        vs[p][w] = (x & keep) | (0x7F7F7F7Fu & ~keep);
      }
    }
  }

  // Writes the operands of the values' dims that the wave's half of each token's bytes holds.
  template <bool HALF, int SECOND>
  __device__ __forceinline__ void widen_values(u32x4 (*out)[64], uint32_t lane) const {
    each_part<D>([&](auto part) {
      constexpr int p = part.value, dims = part_dims(D, p), at = part_at(D, p), b = dims / 32;
      constexpr int kBytes = b == 4 ? 2 : 1, kFirst = b == 1 ? 0 : SECOND * kBytes;
      if constexpr (b == 1 && SECOND) {
        return;  // (one byte serves both)
      } else {
        const float scale[8] = {power_at<0>(vs[p][0]), power_at<1>(vs[p][0]), power_at<2>(vs[p][0]),
                                power_at<3>(vs[p][0]),
                                power_at<0>(vs[p][1]), power_at<1>(vs[p][1]), power_at<2>(vs[p][1]),
                                power_at<3>(vs[p][1])};
#pragma unroll
        for (int j = 0; j < kBytes; ++j) {
          u32x4 even, odd;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at0 = 2 * i * b + kFirst + j, at1 = at0 + b;
            const uint32_t c0 = two_of<HALF>(v[at / 16 + at0 / 4], at0 % 4, scale[2 * i]);
            const uint32_t c1 = two_of<HALF>(v[at / 16 + at1 / 4], at1 % 4, scale[2 * i + 1]);
            even[i] = __builtin_amdgcn_perm(c1, c0, 0x05040100u);
            odd[i] = __builtin_amdgcn_perm(c1, c0, 0x07060302u);
          }
          out[at / 16 + 2 * (kFirst + j)][lane] = even;
          out[at / 16 + 2 * (kFirst + j) + 1][lane] = odd;
        }
      }
    });
  }

  // Writes the operands of the wave's share.
  template <bool HALF>
  __device__ __forceinline__ void widen(u32x4 (*tile)[64], uint32_t lane, uint32_t wave, int32_t held,
                                        uint32_t& nans) {
    constexpr int KL = D / 32, DT = D / 16;
#pragma unroll
    for (int j = 0; j < KL; ++j) {
      constexpr int kFirst = part_dims(D, 0) / 32;
      const float scale = power_of(ks[j < kFirst ? 0 : part_count(D) - 1], 0);
      u32x4 a;
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = two_of<HALF>(k[j], i, scale);
      tile[wave * KL + j][lane] = a;
    }
    mask<HALF>(wave, held, nans);
    u32x4(*out)[64] = tile + 4 * KL + (wave >> 1) * DT;
    if (wave & 1u)
      widen_values<HALF, 1>(out, lane);
    else
      widen_values<HALF, 0>(out, lane);
  }
};

template <typename W>
__device__ __forceinline__ uint32_t two_in_word(W a, W b) {
  typedef W pair __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, pair{a, b});
}

template <typename E, int D, int NR>
struct Wide {
  typedef E Elem;
  typedef Core4<E, D, false> Few;
  typedef WideShared<E, D, NR> Shared;
  static constexpr int kDim = D, kRows = 64 * NR, kThreads = kAttendWaves * 64, kResident = 2;
  static constexpr bool kHalfQueries = __is_same(E, fp16_t);
  // What a lane's weights of a chunk may add up to before the reference follows the row's largest, how many
  // powers of two above the reference that must be then, and how many it is afterwards.
  static constexpr float kMost = kHalfQueries ? 32768.0f : 256.0f, kGrows = kHalfQueries ? 8.0f : 4.0f;
  static constexpr float kAbove = kHalfQueries ? 7.0f : 0.0f;
  static constexpr int KL = D / 32, DT = D / 16, NB = wide_buffers(D);

  // Units of work of a tile of `rows` rows that sees `chunks` chunks: a chunk, or four where the
  // waves of few rows' attention take one each, and two for what a tile takes besides
  // (its queries, its first loads, its result).  With shares of equal chunks 5 prompts of up
  // to 2900 tokens take 178 us in shares and with these 150; four units and not two: 153.
  static constexpr uint32_t kFixed = 2;
  static __device__ __forceinline__ uint32_t unit(uint32_t rows) { return rows <= 16 ? kAttendWaves : 1; }
  static __device__ __forceinline__ uint32_t units(uint32_t rows, uint32_t chunks) {
    return kFixed + (chunks + unit(rows) - 1) / unit(rows);
  }

  static __device__ __forceinline__ void rows(const AttendArgs& A, Shared& sh, uint32_t b, uint32_t h,
                                              uint32_t first, uint32_t u0, uint32_t u1, float* part,
                                              float* stats) {
    const uint32_t here = min(rows_of(A, b) - first, static_cast<uint32_t>(kRows));
    const uint32_t c0 = (max(u0, kFixed) - kFixed) * unit(here);
    const uint32_t c1 = u1 == ~0u ? u1 : (max(u1, kFixed) - kFixed) * unit(here);
    if (here <= 16)
      Few::rows(A, sh.few, b, h, first, c0, c1, part, stats);
    else
      many(A, sh, b, h, first, c0, c1, part, stats);
  }

  static __device__ __forceinline__ void many(const AttendArgs& A, Shared& sh, uint32_t b, uint32_t h,
                                              uint32_t first, uint32_t c0, uint32_t c1, float* part,
                                              float* stats) {
    const uint32_t tid = thread_here(), lane = tid & 63u, n = lane & 15u, g = lane >> 4;
    const uint32_t wave = uniform(tid >> 6);
    const int32_t* table = A.table + static_cast<int64_t>(b) * A.table_stride;
    const RowTile rt = row_tile(A, b, first, kRows);
    const uint32_t seen = uniform(static_cast<uint32_t>(rt.seen));
    c1 = min(c1, (seen + kChunk - 1) / kChunk);

    // the wave's rows
    const uint32_t mine = first + wave * (16 * NR);
    int32_t limit[NR];        // last token that the row sees
    int32_t least = 0x7FFFFFFF, last = -1;  // the first and last of them
    u32x4 q[NR][KL];
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      const uint32_t i = mine + x * 16 + n;
      const int64_t j = i / A.group, row = rt.start + j;
      const bool there = i < rt.rows;
      limit[x] = there ? static_cast<int32_t>(max<int64_t>(-1, min<int64_t>(rt.seen - 1, rt.ahead + j))) : -1;
      const E* p = static_cast<const E*>(A.query) + row * A.query_row +
                   static_cast<int64_t>(h * A.group + i % A.group) * A.query_head;
#pragma unroll
      for (int k = 0; k < KL; ++k) {
        q[x][k] = u32x4{0u, 0u, 0u, 0u};
        if (there) __builtin_memcpy(&q[x][k], p + key4_dim<D>(k, g), 16);
      }
      if (there) least = min(least, limit[x]);
      last = max(last, limit[x]);
    }
    for (int d = 1; d < 16; d <<= 1) {
      least = min(least, __shfl_xor(least, d));
      last = max(last, __shfl_xor(last, d));
    }
    least = __builtin_amdgcn_readfirstlane(least);
    last = __builtin_amdgcn_readfirstlane(last);

    float m[NR], l[NR];
    f32x4 acc[NR][DT];
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      m[x] = mine + x * 16 + n < rt.rows ? -INFINITY : 0.0f;  // (rows that are not there need no reference)
      l[x] = 0.0f;
#pragma unroll
      for (int e = 0; e < DT; ++e) acc[x][e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    uint32_t nans = 0;

    if (c0 < c1) {  // (so seen > 0)
      const typename WideCodes<D>::From from(A, h, g, n, wave);
      uint32_t odd0 = ~0u, odd1 = 0, turn = 0;  // chunks that are not of float16 numbers lie in odd0 .. odd1 - 1
      // The chunks c .. end - 1 that are of float16 numbers (HALF), or those that are not: the next
      // chunk's codes are loaded while one is computed, and widened behind it, into the other
      // buffer where there are two.
      auto run = [&](auto float16, uint32_t c, uint32_t end) {
        constexpr bool HALF = decltype(float16)::value;
        WideCodes<D> codes;
        Place at, next, then;  // of the chunk that codes hold, and the two behind it
        at.look(A, table, c * kChunk, seen, g, n);
        next.look(A, table, (c + 1) * kChunk, seen, g, n);
        at.settle(A, c * kChunk, seen, g);
        codes.template load<kHalfQueries>(A, at, from);
        for (; c < end; ++c) {
          const uint32_t t0 = c * kChunk;
          const int32_t tg = t0 + 16 * g, bg = at.mine;
          u32x4(*tile)[64] = sh.tile[NB == 2 ? turn & 1u : 0];
          const bool here = !kHalfQueries || codes.float16(t0, seen, n, bg) == HALF;  // (the same for all waves)
          if (here) {
            if constexpr (NB == 1) __syncthreads();
            uint32_t to = lane;
            asm volatile("" : "+v"(to));  // (as `own` below)
            codes.template widen<HALF>(tile, to, wave, bg < 0 ? 0 : static_cast<int32_t>(seen) - tg, nans);
            __syncthreads();
            ++turn;
          } else if (HALF) {
            odd0 = min(odd0, c);
            odd1 = c + 1;
          }
          next.settle(A, t0 + kChunk, seen, g);
          codes.template load<kHalfQueries>(A, next, from);
          then.look(A, table, t0 + 2 * kChunk, seen, g, n);
          __builtin_amdgcn_sched_barrier(0);
          if (here && static_cast<int32_t>(t0) <= last) {
            f32x4 s[NR][4];
#pragma unroll
            for (int x = 0; x < NR; ++x)
#pragma unroll
              for (int t = 0; t < 4; ++t) s[x][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            // Operands are asked for two products' pairs ahead: keys' tiles 2 (i % 2) and + 1 of
            // step i / 2, then the values' two steps of dims' tile i - 2 KL.
            u32x4 ops[3][2];
            uint32_t own = lane;
            asm volatile("" : "+v"(own));  // (addresses are not to be kept from chunk to chunk)
            auto ask = [&](int i) {
#pragma unroll
              for (int j = 0; j < 2; ++j)
                ops[i % 3][j] = i < 2 * KL ? tile[(2 * (i & 1) + j) * KL + i / 2][own]
                                           : tile[4 * KL + j * DT + i - 2 * KL][own];
            };
            ask(0);
            ask(1);
#pragma unroll
            for (int i = 0; i < 2 * KL; ++i) {
              ask(i + 2);
              __builtin_amdgcn_sched_barrier(0);
              u32x4 hi[NR], lo[NR];
#pragma unroll
              for (int x = 0; x < NR; ++x) {
                hi[x] = q[x][i / 2];
                if constexpr (kHalfQueries && !HALF) {
                  asm volatile("" : "+v"(hi[x]));  // (not to be kept in two parts from chunk to chunk)
                  two_parts(hi[x], hi[x], lo[x]);
                }
              }
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 0; x < NR; ++x) {
                  f32x4& to = s[x][2 * (i & 1) + j];
                  if constexpr (kHalfQueries && !HALF) to = mfma_of<false>(ops[i % 3][j], lo[x], to);
                  to = mfma_of<HALF>(ops[i % 3][j], hi[x], to);
                }
              __builtin_amdgcn_sched_barrier(0);
            }
            if (static_cast<int32_t>(t0 + kChunk - 1) > least || __ballot(bg < 0) != 0) {
#pragma unroll
              for (int x = 0; x < NR; ++x) {
                const int32_t sees = bg < 0 ? 0 : limit[x] - tg + 1;  // of this lane's sixteen tokens
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                  for (int r = 0; r < 4; ++r)
                    if (4 * t + r >= sees) s[x][t][r] = -INFINITY;
              }
            }
            typedef typename std::conditional<HALF, fp16_t, bf16_t>::type W;
            u32x4 p[2][NR][2];  // the rounded weights, and the rounded rests
            // The reference m follows the row's largest score when a chunk's weights of a lane
            // add up to more than kMost, or when there is none yet; they are worked out again then.
            // (a whole number: what is rescaled by it stays exact)
            //
            // A score times scale2 is not rounded before m is taken from it, but the maximum that m
            // follows is; where floats lie so far apart that this shows (2^20: 2^-5 at most), all
            // are rounded first, or a weight could be any power of two.
#pragma unroll
            for (int x = 0; x < NR; ++x) {
              constexpr float kFar = 1048576.0f;
              bool again = __ballot(!(fabsf(m[x]) < kFar)) != 0;
              float mul = A.scale2;
              for (;;) {
                if (again) {
                  float top = -INFINITY;
#pragma unroll
                  for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) top = fmaxf(top, s[x][t][r]);
                  top = max_of_groups(top) * A.scale2;
                  const bool grows = top > m[x] + kGrows;
                  const float was = m[x];
                  if (grows) m[x] = __builtin_floorf(top) - kAbove;
                  const float keep = grows ? __builtin_amdgcn_exp2f(was - m[x]) : 1.0f;
                  l[x] *= keep;
#pragma unroll
                  for (int e = 0; e < DT; ++e) acc[x][e] *= keep;
                  if (__ballot(fabsf(m[x]) >= kFar && m[x] != -INFINITY) != 0) {
                    mul = 1.0f;
#pragma unroll
                    for (int t = 0; t < 4; ++t) s[x][t] *= A.scale2;
                  }
                }
                const float base = m[x] == -INFINITY ? 0.0f : -m[x];
                float sum[2] = {0.0f, 0.0f};
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                  for (int r = 0; r < 4; r += 2) {
                    const float w0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x][t][r], mul, base));
                    const float w1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x][t][r + 1], mul, base));
                    sum[0] += w0;
                    sum[1] += w1;
                    const int i = (t & 1) * 2 + r / 2;
                    const W f0 = static_cast<W>(w0), f1 = static_cast<W>(w1);
                    p[0][x][t >> 1][i] = two_in_word(f0, f1);
                    p[1][x][t >> 1][i] = two_in_word(static_cast<W>(w0 - static_cast<float>(f0)),
                                                     static_cast<W>(w1 - static_cast<float>(f1)));
                  }
                const float more = sum[0] + sum[1];
                if (!again && __ballot(more > kMost) != 0) {
                  again = true;
                  continue;
                }
                l[x] += more;
                break;
              }
              __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int e = 0; e < DT; ++e) {
              if (e + 2 < DT) ask(2 * KL + e + 2);
              __builtin_amdgcn_sched_barrier(0);
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                  for (int x = 0; x < NR; ++x)
                    acc[x][e] = mfma_of<HALF>(ops[(2 * KL + e) % 3][j], p[i][x][j], acc[x][e]);
              __builtin_amdgcn_sched_barrier(0);
            }
          }
          at = next;
          next = then;
        }
      };
      if constexpr (kHalfQueries) {
        run(std::true_type(), c0, c1);
        if (odd0 < odd1) run(std::false_type(), odd0, odd1);
      } else {
        run(std::false_type(), c0, c1);
      }
    }
    // (a wave's own share of the values' NaN tells of them all: their tokens are looked for again)
    const bool some = __ballot(nans != 0) != 0;
    if (lane == 0) sh.nans[wave] = some;
    __syncthreads();
    bool any_nan = false;
    for (int w = 0; w < kAttendWaves; ++w) any_nan |= sh.nans[w] != 0;
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      const uint32_t i = mine + x * 16 + n;
      float nan[part_count(D)] = {};
      if (any_nan)
        seen_nans4<D>(A, table, h, c0 * kChunk, min(static_cast<int32_t>(c1 * kChunk) - 1, limit[x]), g, nan);
      float sum = l[x] + __shfl_xor(l[x], 16);
      sum += __shfl_xor(sum, 32);
      if (i >= rt.rows) continue;
      const int64_t row = rt.start + i / A.group;
      const uint32_t head = h * A.group + i % A.group;
      const float inv = part ? 1.0f : sum != 0.0f ? 1.0f / sum : 0.0f;
      const uint32_t r0 = wave * (16 * NR) + x * 16 + n;  // in the tile
      if (g == 0) {
        if (part) {
          stats[2 * r0] = m[x];
          stats[2 * r0 + 1] = sum;
        } else if (A.lse) {
          A.lse[row * A.heads + head] = (m[x] + __builtin_amdgcn_logf(sum)) * 0.69314718055994531f;
        }
      }
      each_part<D>([&](auto pt) {
        constexpr int k = pt.value, wide = part_dims(D, k) / 16, from = part_at(D, k);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t d = from + wide * (4 * g + r);
          float o[wide];
#pragma unroll
          for (int e = 0; e < wide; ++e) o[e] = acc[x][from / 16 + e][r] * inv + nan[k];
          if (part) {
            __builtin_memcpy(part + r0 * D + d, o, sizeof(o));
          } else {
            E v[wide];
#pragma unroll
            for (int e = 0; e < wide; ++e) v[e] = static_cast<E>(o[e]);
            __builtin_memcpy(static_cast<E*>(A.out) + row * A.out_row + head * A.out_head + d, v, sizeof(v));
          }
        }
      });
    }
    __syncthreads();
  }
};

// The units of tile number k of a core's tiles (0: no tile has it), and which tile that is.
template <class C>
struct Numbered {
  uint32_t b, y, units;
  __device__ __forceinline__ void look(const AttendArgs& A, uint32_t k) {  // (b set: the request)
    y = k - first_tile(A, b, C::kRows);
    const uint32_t rows = rows_of(A, b), first = y * C::kRows;
    units = 0;
    if (y >= (rows + C::kRows - 1) / C::kRows) return;
    const uint32_t here = min(rows - first, static_cast<uint32_t>(C::kRows));
    const int64_t length = A.lengths[b], held = min<int64_t>(length, static_cast<int64_t>(A.width) * A.s.T);
    const int64_t ahead = length - (static_cast<int64_t>(A.starts[b + 1]) - A.starts[b]);
    const int64_t sees = max<int64_t>(1, min<int64_t>(held, ahead + (first + here - 1) / A.group + 1));
    units = C::units(here, static_cast<uint32_t>((sees + kChunk - 1) / kChunk));
  }
  // To number k from one before it.
  __device__ __forceinline__ void advance(const AttendArgs& A, uint32_t k) {
    while (b + 1 < static_cast<uint32_t>(A.batch) && first_tile(A, b + 1, C::kRows) <= k) ++b;
    look(A, k);
  }
};

// As attend_flat_kernel, but the line holds what each tile sees, so shares are even for
// whole prompts too: every workgroup adds up all tiles, a thread its run of numbers.
template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kResident) attend_wide_kernel(AttendArgs A) {
  constexpr uint32_t kThreads = C::kThreads, kRows = C::kRows;
  __shared__ typename C::Shared sh;
  __shared__ uint64_t s_pre[kThreads], s_wave[kThreads / 64];
  const uint32_t h = blockIdx.x % A.s.H, w = blockIdx.x / A.s.H, tid = threadIdx.x;
  const uint32_t seg = (A.packed + kThreads - 1) / kThreads;
  const uint32_t k0 = min(A.packed, tid * seg), k1 = min(A.packed, k0 + seg);
  Numbered<C> t;
  uint64_t sum = 0;
  if (k0 < k1) {
    uint32_t lo = 0, hi = A.batch;  // the last request that begins at or before k0
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) / 2;
      if (first_tile(A, mid, kRows) <= k0)
        lo = mid;
      else
        hi = mid;
    }
    t.b = lo;
    for (uint32_t k = k0; k < k1; ++k) {
      t.advance(A, k);
      sum += t.units;
    }
  }
  uint64_t run = sum;  // inclusive over the wave's lanes
  for (uint32_t d = 1; d < 64; d <<= 1) {
    const uint64_t o = __shfl_up(static_cast<unsigned long long>(run), d);
    if ((tid & 63u) >= d) run += o;
  }
  if ((tid & 63u) == 63u) s_wave[tid >> 6] = run;
  __syncthreads();
  uint64_t pre = run - sum, all = 0;
  for (uint32_t i = 0; i < kThreads / 64; ++i) {
    if (i < (tid >> 6)) pre += s_wave[i];
    all += s_wave[i];
  }
  s_pre[tid] = pre;
  __syncthreads();
  all = uniform(all);
  const uint64_t flat = min<uint64_t>(A.flat, all);  // (so every share holds a unit)
  if (h == 0 && tid == 0) A.begun[w].request = -1;
  if (w >= flat) return;
  const uint64_t lo = uniform(all * w / flat), hi = uniform(all * (w + 1) / flat);
  uint32_t from = 0, to = kThreads;  // the last run that begins at or before lo
  while (to - from > 1) {
    const uint32_t mid = (from + to) / 2;
    if (s_pre[mid] <= lo)
      from = mid;
    else
      to = mid;
  }
  uint32_t k = uniform(from) * seg;
  uint64_t u = lo, at = uniform(s_pre[from]);  // the unit to do, the number's first
  Numbered<C> now;
  now.b = request_of(A, k, kRows);
  now.look(A, k);
  for (;;) {
    uint32_t units = uniform(now.units);
    while (at + units <= u && k + 1 < A.packed) {  // (u < all: a number with units follows)
      at = uniform(at + units);
      now.advance(A, ++k);
      now.b = uniform(now.b);
      units = uniform(now.units);
    }
    const uint32_t b = uniform(now.b), y = uniform(now.y);
    const uint64_t end = uniform(at + units), stop = uniform(min(hi, end));
    const bool whole = at >= lo && end <= hi;
    if (end > hi && at >= lo && h == 0 && tid == 0) {
      uint64_t sum_here = all;
      asm volatile("" : "+s"(sum_here));  // (nothing for its division is to be kept from before the loop)
      A.begun[w] = Begun{static_cast<int32_t>(b), y, static_cast<uint32_t>((end * flat - 1) / sum_here), 0};
    }
    const uint32_t slot = (blockIdx.x * 2 + (at >= lo ? 1 : 0)) * kRows;
    C::rows(A, sh, b, h, y * kRows, static_cast<uint32_t>(u - at), static_cast<uint32_t>(stop - at),
            whole ? nullptr : A.part + static_cast<uint64_t>(slot) * C::kDim, A.stats + slot * 2);
    u = stop;
    if (u == hi) return;
  }
}

template <class C>
AttendKernels wide_kernels() {
  return {attend_kernel<C>, attend_packed_kernel<C>, attend_wide_kernel<C>,
          join_kernel<typename C::Elem, C::kDim, C::kRows>, C::kThreads};
}

template <typename E, int D>
AttendKernels pick_attend4_rows(int tile, bool once) {
  if (tile > 16) return wide_kernels<Wide<E, D, wide_tiles(D)>>();
  return once ? attend_kernels<Core4<E, D, true>, Core4<E, D, false>, true>()
              : attend_kernels<Core4<E, D, false>, Core4<E, D, false>, true>();
}

template <typename E>
AttendKernels pick_attend4(uint32_t d, int tile, bool once) {
  switch (d) {
    case 64: return pick_attend4_rows<E, 64>(tile, once);
    case 96: return pick_attend4_rows<E, 96>(tile, once);
    case 128: return pick_attend4_rows<E, 128>(tile, once);
    case 192: return pick_attend4_rows<E, 192>(tile, once);
    default: return pick_attend4_rows<E, 256>(tile, once);
  }
}

// Which kernel computes a call's rows, and how it is cut up.  Times are of 32 heads
// over 8, 128 dims, unless they say otherwise.
AttendPlan attend4_plan(const Shape& s, const xfer_attend& q) {
  AttendPlan p;
  const int64_t group = q.heads / int(s.H);
  int64_t most = q.max_query ? std::min(q.max_query, q.rows) : q.rows;
  if (!q.max_query && q.rows <= q.batch) most = 1;
  const int64_t rows = most * group;
  const int d = int(s.D);
  const int64_t width = int64_t(q.table_width) * s.T;
  const int64_t tokens = q.max_length ? std::min<int64_t>(q.max_length, width) : width;
  const int64_t chunks = std::max<int64_t>(1, (tokens + kChunk - 1) / kChunk);
  // Tiles of 16 rows until there is work for many rows' tiles, two of whose workgroups a CU
  // holds: 14 chunks of 128 rows for each of 512 workgroups, or 12 of 64 rows of wide heads (units are
  // chunks of 16 rows).  16 requests of 15 rows over 2000 tokens take 23 us so and 39 with many
  // rows' tiles, 2 of 1000 over 1000 take 57 and 43.  They cost more per row the wider the
  // heads.  A request that fills half of one of those tiles or less stays with them in any case: 64
  // requests over 500 to 8000 tokens take 57 and 71 with 28 rows of 128 dims, 126 and 144 with 60, 173
  // and 150 with 80; with 60 rows of 256 dims 234 and 186.
  const int64_t units = int64_t(q.rows) * group / 16 * s.H * chunks;
  const bool wide = rows > 32 * wide_tiles(d) && units > 512 * (d <= 128 ? 14 * 8 : 12 * 4);
  p.tile = wide ? 64 * wide_tiles(d) : 16;
  p.tiles = uint32_t(std::min<int64_t>(65535, (rows + p.tile - 1) / p.tile));
  const int64_t wgs = int64_t(q.batch) * s.H * p.tiles;
  const int64_t numbers = int64_t(q.rows) * group / p.tile + q.batch;
  const int64_t resident = 256 * (wide ? 2 : attend4_resident(d));
  // Equal shares of all work cost a join of the tiles that they cut, a workgroup per tile leaves the device
  // waiting for the longest tile.  Many rows: that one takes `chunks` (1.6 us each), while a
  // share of equal ones takes half of its part of all chunks, as tiles of a prompt see half of
  // its tokens, and 19 chunks' time (30 us) for the join and what its tiles begin with: 8 chunks of
  // prompts up to 5000 tokens take 96 us in shares and 165 by tiles, 5 prompts up to 2900 tokens 150
  // and 127, 2 of 1000 tokens 66 and 43.  Few rows: a join takes as long as 24 chunks in four waves, or
  // 64 where 128 workgroups or more overlap the longest, and is not worth it where each place of the
  // device has 12 tiles to even out: 64 requests of up to 8000 tokens take 57 and 76, 48 of up to 3000
  // (12 heads over 2) 24 and 19.
  const int64_t share = int64_t(q.rows) * group / p.tile * s.H * chunks / resident;
  const bool shares = wide ? chunks > share / 2 + 19
                           : chunks >= (wgs <= 128 ? 24 : 64) && !(most > 1 && numbers * s.H > 12 * resident);
  p.flat = p.packed = 0;
  if (shares)
    p.flat = uint32_t(std::max<int64_t>(
        1, std::min<int64_t>(resident / s.H, chunks * q.batch * p.tiles / 8)));
  const bool sparse = wgs > numbers * s.H + kEmptyWorkgroups || int64_t(q.batch) * s.H > int64_t(kMaxGrid);
  if (wide ? p.flat > 0 || sparse : !p.flat && sparse) p.packed = uint32_t(numbers);
  return p;
}

}  // namespace
}  // namespace xfer

using namespace xfer;

extern "C" int xfer_mxcache_block_bytes(const xfer_cache_shape* shape, size_t* bytes) {
  Shape s;
  const int rc = shape4_of(shape, "xfer_mxcache_block_bytes", &s);
  if (rc) return rc;
  if (!bytes) return fail(XFER_ERR_INVALID_ARG, "xfer_mxcache_block_bytes: NULL bytes");
  *bytes = size_t(s.block_bytes);
  return XFER_OK;
}

extern "C" int xfer_mxcache_store(const xfer_cache_shape* shape, void* cache, const void* key,
                                  int64_t key_row, int64_t key_head, const void* value,
                                  int64_t value_row, int64_t value_head, int dtype,
                                  const int32_t* slots, int rows, void* stream) {
  Store4Args a;
  const int rc = shape4_of(shape, "xfer_mxcache_store", &a.s);
  if (rc) return rc;
  if (dtype != XFER_BF16 && dtype != XFER_FP16 && dtype != XFER_FP32)
    return fail(XFER_ERR_INVALID_ARG, "xfer_mxcache_store: unknown dtype");
  if (rows < 0) return fail(XFER_ERR_INVALID_ARG, "xfer_mxcache_store: rows must be >= 0");
  if (rows == 0) return XFER_OK;
  if (!cache || !key || !value || !slots)
    return fail(XFER_ERR_INVALID_ARG, "xfer_mxcache_store: NULL buffer with rows to store");
  const size_t size = dtype == XFER_FP32 ? 4 : 2;
  if (!aligned(cache, 16) || !aligned(slots, 4) || !aligned(key, size) || !aligned(value, size))
    return fail(XFER_ERR_INVALID_ARG,
                "xfer_mxcache_store: the cache must be 16-byte aligned, the others by their type");
  a.cache = static_cast<uint8_t*>(cache);
  a.key = key;
  a.value = value;
  a.key_row = key_row;
  a.key_head = key_head;
  a.value_row = value_row;
  a.value_head = value_head;
  a.slots = slots;
  a.rows = rows;
  const uint64_t tiles = (uint64_t(rows) + kStoreRows - 1) / kStoreRows;
  const uint64_t pieces = tiles * kStoreRows * a.s.H * 2 * (a.s.D / 8);
  const uint64_t each = kStoreThreads * kStoreEach, wgs = (pieces + each - 1) / each;
  if (wgs > kMaxGrid)
    return fail(XFER_ERR_INVALID_ARG, "xfer_mxcache_store: too many rows times heads for one call");
  const Store4Fn fn = dtype == XFER_BF16   ? pick_store4<bf16_t>(a.s.D)
                      : dtype == XFER_FP16 ? pick_store4<fp16_t>(a.s.D)
                                           : pick_store4<float>(a.s.D);
  const hipError_t e = launch(fn, a, dim3(uint32_t(wgs)), kStoreThreads, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "xfer_mxcache_store launch");
  return XFER_OK;
}

namespace {

// Whether the vectors of `inner` elements, n0 times n1 of them with strides s0 and s1, of two places share
// elements; the second's are `apart` elements behind the first's.  A vector of one is x + r s0 behind one
// of the other for an r between -n0 and n0, x = apart + h s1 for an h between -n1 and n1: it
// is asked of every h whether the r's that come nearest to x + r s0 = 0 are near enough.
bool places_overlap(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t inner, int64_t apart) {
  typedef __int128 wide;
  const wide reach = (n0 - 1) * (s0 < 0 ? -wide(s0) : wide(s0)) + (n1 - 1) * (s1 < 0 ? -wide(s1) : wide(s1)) + inner;
  if (apart >= reach || -wide(apart) >= reach) return false;  // (separate tensors, mostly)
  if (n1 > n0) {
    std::swap(n0, n1);
    std::swap(s0, s1);
  }
  for (int64_t h = 1 - n1; h < n1; ++h) {
    const wide x = wide(apart) + wide(h) * s1;
    const wide near = s0 ? -x / s0 : 0;
    for (wide r = near - 1; r <= near + 1; ++r) {
      const wide at = std::min<wide>(std::max<wide>(r, 1 - n0), n0 - 1), off = x + at * s0;
      if (off < inner && -off < inner) return true;
    }
  }
  return false;
}

int load_call(const Shape& s, int bits, const void* cache, const xfer_load* q, void* stream, const char* who) {
  const std::string w(who);
  if (!q) return fail(XFER_ERR_INVALID_ARG, w + ": NULL arguments");
  if (q->batch < 0 || q->rows < 0 || q->table_width < 0 || q->table_stride < q->table_width)
    return fail(XFER_ERR_INVALID_ARG,
                w + ": need batch, rows and table_width >= 0 and table_stride >= table_width");
  if (q->batch > 0x7FFFFFF)
    return fail(XFER_ERR_INVALID_ARG, w + ": batch must stay below 2^27");
  if (q->dtype != XFER_BF16 && q->dtype != XFER_FP16 && q->dtype != XFER_FP32)
    return fail(XFER_ERR_INVALID_ARG, w + ": unknown dtype");
  if (q->rows == 0 || q->batch == 0) return XFER_OK;
  if (!cache || !q->key || !q->value || !q->lengths || !q->starts || (q->table_width > 0 && !q->table))
    return fail(XFER_ERR_INVALID_ARG, w + ": NULL buffer with rows to read back");
  const size_t size = q->dtype == XFER_FP32 ? 4 : 2;
  if (!aligned(cache, 16) || !aligned(q->key, size) || !aligned(q->value, size) || !aligned(q->table, 4) ||
      !aligned(q->lengths, 4) || !aligned(q->starts, 4))
    return fail(XFER_ERR_INVALID_ARG, w + ": the cache must be 16-byte aligned, the others by their type");
  if (vectors_overlap(q->rows, q->key_row, s.H, q->key_head, s.D) ||
      vectors_overlap(q->rows, q->value_row, s.H, q->value_head, s.D))
    return fail(XFER_ERR_INVALID_ARG, w + ": the rows and heads of an output must not overlap");
  if ((q->rows == 1 || q->key_row == q->value_row) && (s.H == 1 || q->key_head == q->value_head) &&
      places_overlap(q->rows, q->key_row, s.H, q->key_head, s.D,
                     (int64_t(reinterpret_cast<uintptr_t>(q->value)) - int64_t(reinterpret_cast<uintptr_t>(q->key))) /
                         int64_t(size)))
    return fail(XFER_ERR_INVALID_ARG, w + ": the key's and the value's output must not overlap");
  LoadArgs a;
  a.cache = static_cast<const uint8_t*>(cache);
  a.key = q->key;
  a.value = q->value;
  a.table = q->table;
  a.lengths = q->lengths;
  a.starts = q->starts;
  a.key_row = q->key_row;
  a.key_head = q->key_head;
  a.value_row = q->value_row;
  a.value_head = q->value_head;
  a.table_stride = q->table_stride;
  a.batch = q->batch;
  a.rows = q->rows;
  a.width = q->table_width;
  a.numbers = uint32_t(q->rows) / kLoadTile + 2u * uint32_t(q->batch);
  a.s = s;
  const uint32_t units = 2 * 4 * s.H * (s.D / 8), shares = (units + kLoadShare - 1) / kLoadShare;
  const LoadFn fn = bits == 8 ? pick_load<8>(s.D, q->dtype) : pick_load<4>(s.D, q->dtype);
  const uint32_t most = uint32_t(kMaxGrid / shares);
  const hipError_t e = launch(fn, a, dim3(std::min(a.numbers, most), shares), kLoadThreads,
                              static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, (w + " launch").c_str());
  return XFER_OK;
}

}  // namespace

extern "C" int xfer_mxcache_load(const xfer_cache_shape* shape, const void* cache, const xfer_load* args,
                                 void* stream) {
  Shape s;
  const int rc = shape4_of(shape, "xfer_mxcache_load", &s);
  return rc ? rc : load_call(s, 4, cache, args, stream, "xfer_mxcache_load");
}

extern "C" int xfer_cache_load(const xfer_cache_shape* shape, const void* cache, const xfer_load* args,
                               void* stream) {
  Shape s;
  const int rc = shape8_of(shape, "xfer_cache_load", &s);
  return rc ? rc : load_call(s, 8, cache, args, stream, "xfer_cache_load");
}

extern "C" int xfer_mxcache_attend_workspace(const xfer_cache_shape* shape, const xfer_attend* q,
                                             size_t* bytes) {
  Shape s;
  int rc = shape4_of(shape, "xfer_mxcache_attend_workspace", &s);
  if (!rc) rc = attend_args(s, q, "xfer_mxcache_attend_workspace");
  if (rc) return rc;
  if (!bytes) return fail(XFER_ERR_INVALID_ARG, "xfer_mxcache_attend_workspace: NULL bytes");
  *bytes = attend_work(s, *q, attend4_plan(s, *q)).all();
  return XFER_OK;
}

extern "C" int xfer_mxcache_attend(const xfer_cache_shape* shape, const void* cache,
                                   const xfer_attend* q, void* stream) {
  Shape s;
  int rc = shape4_of(shape, "xfer_mxcache_attend", &s);
  if (!rc) rc = attend_args(s, q, "xfer_mxcache_attend");
  if (rc) return rc;
  if (q->rows == 0 || q->batch == 0) return XFER_OK;
  const auto pick = [&](int dtype, const AttendPlan& p) {
    const bool once = p.tiles == 1;
    return dtype == XFER_BF16 ? pick_attend4<bf16_t>(s.D, p.tile, once) : pick_attend4<fp16_t>(s.D, p.tile, once);
  };
  return attend_call(s, cache, q, attend4_plan(s, *q), pick, stream, "xfer_mxcache_attend");
}

// Device helpers shared by the grouped products (experts.hip, blocks.hip):
// finding a block's expert and output tile from the device array of token
// offsets, and 16-byte accesses of rows of any alignment.
//
// Offsets are device data that the host never reads, so a launch has as many
// blocks as any offsets could need and every block works out its own tile.
// Whatever the offsets hold, the kernels stay inside the caller's buffers:
// every value is clamped to 0..tokens and to at least the largest value
// before it.
#pragma once

#include "internal.h"

namespace dmuon {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

#define DMUON_LDS __attribute__((address_space(3)))

// One expert's rows begin..end of the token dimension.
struct GroupSpan {
  int expert, begin, end;
};

__device__ __forceinline__ int wave_scan_max(int v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (int(threadIdx.x & 63) >= d) v = o > v ? o : v;
  }
  return v;
}
__device__ __forceinline__ int wave_scan_sum(int v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (int(threadIdx.x & 63) >= d) v += o;
  }
  return v;
}

// Sixty-four experts' spans, one per lane, and the running count of row
// tiles: expert base + lane has rows lo..hi and row tiles before..upto.
struct GroupChunk {
  int lo, hi, before, upto;
};
__device__ __forceinline__ GroupChunk group_chunk(const int32_t* offsets, int experts, int tokens, int tile_rows,
                                                  int base, int carry_row, int carry_tiles) {
  const int lane = threadIdx.x & 63;
  int v = 0;
  if (base + lane < experts) {
    v = offsets[base + lane + 1];
    v = v < 0 ? 0 : v > tokens ? tokens : v;
  }
  if (v < carry_row) v = carry_row;
  GroupChunk c;
  c.hi = wave_scan_max(v);
  const int up = __shfl_up(c.hi, 1);
  c.lo = lane ? up : carry_row;
  const int n = (c.hi - c.lo + tile_rows - 1) / tile_rows;
  c.upto = carry_tiles + wave_scan_sum(n);
  c.before = c.upto - n;
  return c;
}

__device__ __forceinline__ int first_row(const int32_t* offsets, int tokens) {
  const int v = offsets[0];
  return v < 0 ? 0 : v > tokens ? tokens : v;
}

// Number of row tiles of all experts.
__device__ __forceinline__ int group_tiles(const int32_t* offsets, int experts, int tokens, int tile_rows) {
  int row = first_row(offsets, tokens), tiles = 0;
  for (int base = 0; base < experts; base += 64) {
    const GroupChunk c = group_chunk(offsets, experts, tokens, tile_rows, base, row, tiles);
    row = __builtin_amdgcn_readlane(c.hi, 63);
    tiles = __builtin_amdgcn_readlane(c.upto, 63);
  }
  return tiles;
}

// The expert of row tile `tile` (0 <= tile < group_tiles) and the tile's
// first row; every lane of the wave gets the same answer.
__device__ __forceinline__ GroupSpan group_of_tile(const int32_t* offsets, int experts, int tokens, int tile_rows,
                                                   int tile, int* row0) {
  int row = first_row(offsets, tokens), tiles = 0;
  for (int base = 0; base < experts; base += 64) {
    const GroupChunk c = group_chunk(offsets, experts, tokens, tile_rows, base, row, tiles);
    const uint64_t hit = __ballot(c.upto > tile);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      GroupSpan g;
      g.expert = base + l;
      g.begin = __builtin_amdgcn_readlane(c.lo, l);
      g.end = __builtin_amdgcn_readlane(c.hi, l);
      *row0 = g.begin + (tile - __builtin_amdgcn_readlane(c.before, l)) * tile_rows;
      return g;
    }
    row = __builtin_amdgcn_readlane(c.hi, 63);
    tiles = __builtin_amdgcn_readlane(c.upto, 63);
  }
  *row0 = 0;
  return GroupSpan{0, 0, 0};
}

// The rows of one expert.
__device__ __forceinline__ GroupSpan group_of_expert(const int32_t* offsets, int experts, int tokens, int expert) {
  int row = first_row(offsets, tokens);
  for (int base = 0; base < experts; base += 64) {
    const GroupChunk c = group_chunk(offsets, experts, tokens, 1, base, row, 0);
    if (expert < base + 64) {
      GroupSpan g;
      g.expert = expert;
      g.begin = __builtin_amdgcn_readlane(c.lo, expert - base);
      g.end = __builtin_amdgcn_readlane(c.hi, expert - base);
      return g;
    }
    row = __builtin_amdgcn_readlane(c.hi, 63);
  }
  return GroupSpan{0, 0, 0};
}

// Block -> position in the tile order (fewer than 2^31 tiles).  The hardware
// deals blocks to the 8 XCDs in turn; runs of up to 32 consecutive tiles (as
// many blocks as an XCD runs at once) go to one XCD, so that they share
// operand panels in its L2.  Of every `even` consecutive tiles each XCD gets its
// share: all tiles, or those of one expert where experts' tiles differ in
// length (fp32 weight gradient of 24 very uneven experts of 1000 x 515, 3001 rows:
// 76 to 69 us).  A grid of grouped_grid(bound) blocks reaches every position below any
// total <= bound; blocks past the total are idle.
__device__ __forceinline__ uint32_t xcd_position(uint32_t block, uint32_t even) {
  uint32_t run = (even + kNumXcd - 1) / kNumXcd;
  if (run > 32) run = 32;
  if (run < 1) run = 1;
  const uint32_t x = block % kNumXcd, s = block / kNumXcd;
  return ((s / run) * kNumXcd + x) * run + s % run;
}
inline int64_t grouped_grid(int64_t bound) { return (bound + 2 * 32 * kNumXcd - 1) / (32 * kNumXcd) * (32 * kNumXcd); }

// Position -> (row tile, column tile) of a grid of tiles: eight row tiles
// together, so the 32 blocks of an XCD cover 8 x 4 tiles.
__device__ __forceinline__ void tile_of_position(uint32_t p, uint32_t mt, uint32_t nt, int* tm, int* tn) {
  const uint32_t sg = p / (8 * nt);
  const uint32_t left = mt - sg * 8;
  const uint32_t gm = left < 8 ? left : 8;
  const uint32_t q = p - sg * 8 * nt;
  const uint32_t col = q / gm;
  *tm = int(sg * 8 + (q - col * gm));
  *tn = int(col);
}

// Two fp32 values rounded to nearest-even bf16, packed (first in the low half).
__device__ __forceinline__ uint32_t pack2_bf16(float a, float b) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Sixteen bytes from p, of which the first `valid` elements of EB bytes are
// inside the row; the others read as zero.  VEC: p is 16-byte aligned and
// `valid` is either <= 0 or a whole chunk.  Without VEC a chunk that ends
// past the row is read element by element, nothing past the row is touched.
template <int EB, bool VEC>
__device__ __forceinline__ u32x4_t load_chunk(const char* p, int valid) {
  u32x4_t v = {0, 0, 0, 0};
  if constexpr (VEC) {
    if (valid > 0) v = *reinterpret_cast<const u32x4_t*>(p);
  } else {
    struct __attribute__((packed, aligned(EB))) Any { u32x4_t v; };
    if (valid >= 16 / EB) {
      v = reinterpret_cast<const Any*>(p)->v;
    } else {
#pragma unroll
      for (int j = 0; j < 16 / EB; ++j) {
        uint32_t e = 0;
        if (j < valid) {
          if constexpr (EB == 1) e = reinterpret_cast<const uint8_t*>(p)[j];
          else if constexpr (EB == 2) e = reinterpret_cast<const uint16_t*>(p)[j];
          else e = reinterpret_cast<const uint32_t*>(p)[j];
        }
        v[j * EB / 4] |= e << (8 * ((j * EB) & 3));
      }
    }
  }
  return v;
}

// Buffer descriptor of `bytes` bytes at `base` (raw buffer, no stride), in
// scalar registers; a lane whose offset is outside reads zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t slab_rsrc(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint64_t u = (uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(uint32_t(a >> 32))))) << 32) |
                     uint32_t(__builtin_amdgcn_readfirstlane(int(uint32_t(a))));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(u), static_cast<short>(0),
                                           __builtin_amdgcn_readfirstlane(int(bytes)), 0x00020000);
}
constexpr uint32_t kSlabAll = 0x7ffffff0u;   // range of a descriptor whose lanes are masked by their offsets
constexpr uint32_t kOutside = 0x80000000u;   // an offset outside every descriptor
// Buffer load into LDS: lane l writes bytes 16l..16l+15 of the 1 KB at `lds`.
__device__ __forceinline__ void slab_load_lds(__amdgpu_buffer_rsrc_t rsrc, char* lds, uint32_t offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (DMUON_LDS void*)lds, 16, int(offset), 0, 0, 0);
}

// Two 16 x 16 blocks of bf16 results side by side, at `row` of the lane's own
// row (lane % 16); the lane holds columns 4g .. 4g + 3 of both, g = lane / 16.
// Neighbouring sixteen lanes trade words first, so that a lane writes 16 bytes
// and a row's four lanes 64: half as many requests to the L2 as with 8 bytes
// per lane (weight gradient of 8 experts 14336 x 4096, 8192 rows: 956 to 880 us;
// block-scaled 8192^3: 564 to 540 us).  Any alignment.  Every lane of the wave has to call.
__device__ __forceinline__ void store_pair(uint16_t* row, const f32x4_t& left, const f32x4_t& right, int g, bool write) {
  uint32_t x[2], y[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // the odd sixteens of the left block's words for the even ones of the right
    const auto t = __builtin_amdgcn_permlane16_swap(pack2_bf16(left[2 * h], left[2 * h + 1]),
                                                    pack2_bf16(right[2 * h], right[2 * h + 1]), false, false);
    x[h] = t[0];
    y[h] = t[1];
  }
  struct __attribute__((packed, aligned(2))) Any { u32x4_t v; };
  if (write) reinterpret_cast<Any*>(row + 16 * (g & 1) + 8 * (g >> 1))->v = u32x4_t{x[0], x[1], y[0], y[1]};
}

// Four consecutive results of a row, of which first..n-1 are written.  Whole groups go
// out in one store at any element's alignment (fp32 rows of 515: 49 MB took
// 44 us in single elements).
template <typename OutT>
__device__ __forceinline__ void store4(OutT* row, int col, int n, bool accumulate, const float (&x)[4],
                                       int first = 0) {
  if (col >= n) return;
  float v[4] = {x[0], x[1], x[2], x[3]};
  OutT* p = row + col;
  if (col >= first && col + 4 <= n) {
    if constexpr (sizeof(OutT) == 4) {
      struct __attribute__((packed, aligned(4))) Any { f32x4_t v; };
      Any* q = reinterpret_cast<Any*>(p);
      f32x4_t o = {v[0], v[1], v[2], v[3]};
      if (accumulate) o += q->v;
      q->v = o;
    } else {
      struct __attribute__((packed, aligned(2))) Any { u32x2_t v; };
      Any* q = reinterpret_cast<Any*>(p);
      if (accumulate) {
        const u32x2_t old = q->v;
        v[0] += bf16_lo(old[0]);
        v[1] += bf16_hi(old[0]);
        v[2] += bf16_lo(old[1]);
        v[3] += bf16_hi(old[1]);
      }
      q->v = u32x2_t{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])};
    }
    return;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (col + r < first || col + r >= n) continue;
    if constexpr (sizeof(OutT) == 4) {
      p[r] = accumulate ? p[r] + v[r] : v[r];
    } else {
      if (accumulate) v[r] += bf16_lo(p[r]);
      p[r] = static_cast<OutT>(pack2_bf16(v[r], 0.f));
    }
  }
}

}  // namespace dmuon

// Staging of 8-bit operands through registers into LDS, rows of 128 k (blocks.hip,
// int8.hip): any alignment, four waves.
#pragma once

#include "bigtile.h"
#include "skinny.h"

namespace dmuon {

constexpr int kStageThreads = 256;

// One thread's share of an operand's stage of 128 k: TILE / 32 chunks.
template <int TILE, bool VEC>
__device__ __forceinline__ void load_stage(const char* base, int64_t ld, int rows, int64_t k0, int64_t k,
                                           u32x4_t (&v)[TILE / 32]) {
  const int t = threadIdx.x;
#pragma unroll
  for (int q = 0; q < TILE / 32; ++q) {
    const int r = (t >> 3) + 32 * q, c = (t & 7) * 16;
    const int64_t left = k - k0 - c;
    v[q] = load_chunk<1, VEC>(base + r * ld + k0 + c, r < rows ? int(left > 16 ? 16 : left) : 0);
  }
}
template <int TILE>
__device__ __forceinline__ void write_stage(char* lds, const u32x4_t (&v)[TILE / 32]) {
  const int t = threadIdx.x;
#pragma unroll
  for (int q = 0; q < TILE / 32; ++q)
    *reinterpret_cast<u32x4_t*>(lds + row_slot((t >> 3) + 32 * q, t & 7)) = v[q];
}
// A lane's 16 bytes of half h (64 k) of row r0 + lane % 16.
__device__ __forceinline__ u32x4_t read_half(const char* lds, int r0, int h) {
  const int lane = threadIdx.x & 63;
  return *reinterpret_cast<const u32x4_t*>(lds + row_slot(r0 + (lane & 15), 4 * h + (lane >> 4)));
}
// A lane's 32 bytes of row r0 + lane % 16: chunks lane / 16 and lane / 16 + 4.
// Which k a lane holds does not matter as long as both operands agree.
__device__ __forceinline__ i32x8_t read_frag(const char* lds, int r0) {
  const int lane = threadIdx.x & 63;
  union { u32x4_t h[2]; i32x8_t v; } u;
  u.h[0] = *reinterpret_cast<const u32x4_t*>(lds + row_slot(r0 + (lane & 15), lane >> 4));
  u.h[1] = *reinterpret_cast<const u32x4_t*>(lds + row_slot(r0 + (lane & 15), 4 + (lane >> 4)));
  return u.v;
}

}  // namespace dmuon

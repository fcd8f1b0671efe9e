// 8-bit floating point with one fp32 scale per block of 128: quantisation,
// its inverse, and the matrix product of quantised operands.
//
// Quantising a block (block_rows x 128 values; 1 x 128 for activations and
// gradients, 128 x 128 for weights):
//   scale = max(amax / 448 (e4m3) or 57344 (e5m2), 2^-126),  q = rne(x * (1 / scale))
// in fp32, so amax maps to the format's largest value and nothing overflows.
// The maximum is taken over the bit patterns of |x|, in which NaN > Inf > any
// number: a block with a NaN or an Inf gets a non-finite scale and decodes to
// NaN, and no other block notices.
//
// Product: c[i][j] = sum over blocks kb of  sa[i][kb] sb[j/bs][kb] *
// (sum over the block's 128 k of a[i][k] b[j][k]); the scales are constant
// within a block of k, so each block's sum is one matrix-instruction result
// that is scaled in fp32 and added to an fp32 accumulator.
//   - results rounded to bf16: v_mfma_f32_16x16x128_f8f6f4, one instruction
//     per 16 x 16 x 128 block.  It adds eight consecutive products at a time,
//     each cut toward zero at 2^-13 of the power of two of the largest of its
//     eight, and joins the eights in fp32 (measured with single small products
//     beside large ones that cancel; a subnormal operand counts as the format's
//     smallest normal number there, a product of zero not at all).  So a result is off
//     by less than 7 * 2^-13 of the largest product of every eight.  A sum about as large as its
//     products hides that behind its bf16 rounding: over 8192 x 14336 x 4096 the
//     error's norm is 0.00166 of the result's with either sum, and 2 % of the
//     results lie more than half a step off.  Where large products cancel it
//     is the larger of the two (measured: up to 2^-11.3 of a block's largest
//     product), once per call when calls accumulate in bf16.
//   - fp32 results: the operands are widened to bf16 (exact for both
//     formats) and go through v_mfma_f32_16x16x32_bf16, which keeps fp32
//     sums, at half the rate.
#include "bigtile.h"
#include "skinny.h"
#include "stage8.h"

namespace dmuon {
namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

constexpr int kBlk = 128;         // values per scale along a row
constexpr float kScaleMin = 0x1p-126f;

template <bool E5M2>
__device__ __forceinline__ uint32_t to_q8x4(float a, float b, float c, float d) {
  int w = 0;
  if constexpr (E5M2) {
    w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
  } else {
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  }
  return uint32_t(w);
}

__device__ __forceinline__ float block_scale(uint32_t amax_bits, float max_value) {
  const float amax = __uint_as_float(amax_bits);
  const float s = amax / max_value;
  return s < kScaleMin ? kScaleMin : s;   // a NaN stays
}

// ---- quantisation -----------------------------------------------------------

// A vector at an address of any alignment: the memory system takes it in one
// store, odd row lengths included (8191 x 14335 with both copies: 345 us when
// such rows were written byte by byte, 178 so).
template <typename V>
struct __attribute__((packed, aligned(1))) AnyAddress { V v; };
struct __attribute__((packed, aligned(2))) AnyHalf { u32x4_t v; };
struct __attribute__((packed, aligned(4))) AnyFloat { f32x4_t v; };

// Eight values of a row as they were loaded.  keep() makes the compiler forget
// what it derived from them: bf16 is widened again at each use instead of
// holding 64 floats per thread (75 registers and six waves per SIMD instead
// of 171 and two; 8192 x 14336, both copies: 107 us instead of 118, 4.4 TB/s).
template <bool F32>
struct Eight {
  u32x4_t w[F32 ? 2 : 1];
  template <bool VEC>
  __device__ __forceinline__ void load(const char* p, int valid) {
    if constexpr (F32) {
      w[0] = load_chunk<4, VEC>(p, valid);
      w[1] = load_chunk<4, VEC>(p + 16, valid - 4);
    } else {
      w[0] = load_chunk<2, VEC>(p, valid);
    }
  }
  __device__ __forceinline__ float operator()(int e) const {
    if constexpr (F32) return __uint_as_float(w[e >> 2][e & 3]);
    else return (e & 1) ? bf16_hi(w[0][e >> 1]) : bf16_lo(w[0][e >> 1]);
  }
  __device__ __forceinline__ void keep() {
    if constexpr (!F32) asm volatile("" : "+v"(w[0]));
  }
};

// One 128 x 128 tile per block of 256 threads.  Thread (g, c) = (t / 16, t % 16)
// holds columns 8c..8c+7 of rows 4g..4g+3 and 64+4g..64+4g+3: sixteen lanes
// cover a row of 128 (its maximum is four shuffles), and four rows of a
// column pack into one word for the transposed copy, which is turned through
// LDS.  Bound by HBM: 8192 x 14336 in both orientations 107 us (4.4 TB/s), 8 x
// 1024 x 4096 with 128 x 128 blocks 20 us (5.1 TB/s).
template <bool F32, bool E5M2>
__global__ void __launch_bounds__(256, 4)
quantize_kernel(QuantArgs P) {
  __shared__ uint32_t row_max[kBlk], col_max[kBlk];
  __shared__ uint32_t tr[kBlk][33];       // [column][four rows per word], one word of padding
  const int t = threadIdx.x, g = t >> 4, c = t & 15;
  const int rb = int((P.rows + kBlk - 1) / kBlk), cb = int((P.cols + kBlk - 1) / kBlk);
  const int by = int(blockIdx.x) / cb, bx = int(blockIdx.x) - by * cb;
  const int64_t batch = blockIdx.z;
  const int64_t r0 = int64_t(by) * kBlk, c0 = int64_t(bx) * kBlk;
  const int rows = int(P.rows - r0 < kBlk ? P.rows - r0 : kBlk);
  const int cols = int(P.cols - c0 < kBlk ? P.cols - c0 : kBlk);
  constexpr int EB = F32 ? 4 : 2;
  constexpr float kMax = E5M2 ? 57344.f : 448.f;
  const char* x = static_cast<const char*>(P.x) + (batch * P.x_stride + r0 * P.ldx + c0) * EB;
  Eight<F32> v[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int r = 4 * g + (q & 3) + 64 * (q >> 2);
    const int valid = r < rows ? cols - 8 * c : 0;
    const char* p = x + (r * P.ldx + 8 * c) * EB;
    if (P.vec_x) v[q].template load<true>(p, valid);
    else v[q].template load<false>(p, valid);
  }
  float rinv[8];      // 1 / scale of each of the thread's rows
  uint32_t rmax[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = __float_as_uint(v[q](e)) & 0x7fffffffu;
      m = b > m ? b : m;
    }
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) {
      const uint32_t o = __shfl_xor(m, d);
      m = o > m ? o : m;
    }
    rmax[q] = m;
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q].keep();
  float binv = 0.f;
  if (P.block_rows == kBlk) {
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) m = rmax[q] > m ? rmax[q] : m;
    if (c == 0) row_max[g] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) m = row_max[i] > m ? row_max[i] : m;
    const float s = block_scale(m, kMax);
    binv = 1.f / s;
    if (t == 0) {
      if (P.scale) P.scale[(batch * rb + by) * cb + bx] = s;
      if (P.scale_t) P.scale_t[(batch * cb + bx) * rb + by] = s;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) rinv[q] = binv;
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float s = block_scale(rmax[q], kMax);
      rinv[q] = 1.f / s;
      const int r = 4 * g + (q & 3) + 64 * (q >> 2);
      if (c == 0 && r < rows && P.scale) P.scale[(batch * P.rows + r0 + r) * cb + bx] = s;
    }
  }
  if (P.q) {
    uint8_t* q0 = P.q + batch * P.rows * P.cols + r0 * P.cols + c0;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int r = 4 * g + (q & 3) + 64 * (q >> 2);
      if (r >= rows || 8 * c >= cols) continue;
      const u32x2_t w = {to_q8x4<E5M2>(v[q](0) * rinv[q], v[q](1) * rinv[q], v[q](2) * rinv[q], v[q](3) * rinv[q]),
                         to_q8x4<E5M2>(v[q](4) * rinv[q], v[q](5) * rinv[q], v[q](6) * rinv[q], v[q](7) * rinv[q])};
      uint8_t* p = q0 + r * P.cols + 8 * c;
      if (8 * c + 8 <= cols) {
        reinterpret_cast<AnyAddress<u32x2_t>*>(p)->v = w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (8 * c + e < cols) p[e] = uint8_t(w[e >> 2] >> (8 * (e & 3)));
      }
    }
  }
  if (!P.qt) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q].keep();
  // the transposed copy: its rows are the columns here, its blocks run along
  // the rows here
  float cinv[8];
  if (P.block_rows == kBlk) {
#pragma unroll
    for (int e = 0; e < 8; ++e) cinv[e] = binv;
  } else {
    if (t < kBlk) col_max[t] = 0;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t m = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t b = __float_as_uint(v[q](e)) & 0x7fffffffu;
        m = b > m ? b : m;
      }
#pragma unroll
      for (int d = 16; d < 64; d <<= 1) {
        const uint32_t o = __shfl_xor(m, d);
        m = o > m ? o : m;
      }
      if ((t & 63) < 16) atomicMax(&col_max[8 * c + e], m);   // four waves; a maximum does not depend on the order
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) cinv[e] = 1.f / block_scale(col_max[8 * c + e], kMax);
    if (t < cols && P.scale_t)
      P.scale_t[(batch * P.cols + c0 + t) * rb + by] = block_scale(col_max[t], kMax);
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q].keep();
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      tr[8 * c + e][g + 16 * h] = to_q8x4<E5M2>(v[4 * h](e) * cinv[e], v[4 * h + 1](e) * cinv[e],
                                                v[4 * h + 2](e) * cinv[e], v[4 * h + 3](e) * cinv[e]);
  __syncthreads();
  uint8_t* qt0 = P.qt + batch * P.rows * P.cols + c0 * P.rows + r0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {     // eight lanes write one column's 128 bytes
    const int col = (t >> 3) + 32 * i, part = (t & 7) * 16;
    if (col >= cols || part >= rows) continue;
    u32x4_t w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = tr[col][part / 4 + e];
    uint8_t* p = qt0 + col * P.rows + part;
    if (part + 16 <= rows) {
      reinterpret_cast<AnyAddress<u32x4_t>*>(p)->v = w;
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (part + e < rows) p[e] = uint8_t(w[e >> 2] >> (8 * (e & 3)));
    }
  }
}

template <bool E5M2>
__device__ __forceinline__ float from_q8(uint32_t b) {
  if constexpr (E5M2) return __builtin_amdgcn_cvt_f32_bf8(int(b), 0);
  else return __builtin_amdgcn_cvt_f32_fp8(int(b), 0);
}

// q * scale in fp32, and for bf16 that rounded again, as plain fp32 code has it (at
// most 2^-24 of a value more than half a bf16 step); one block per 128 columns x
// 16 rows.
template <bool F32, bool E5M2>
__global__ void __launch_bounds__(256)
dequantize_kernel(QuantArgs P) {
  const int t = threadIdx.x;
  const int cb = int((P.cols + kBlk - 1) / kBlk);
  const int by = int(blockIdx.x) / cb, bx = int(blockIdx.x) - by * cb;
  const int64_t batch = blockIdx.z;
  const int64_t r = int64_t(by) * 16 + (t >> 4), c = int64_t(bx) * kBlk + (t & 15) * 8;
  if (r >= P.rows || c >= P.cols) return;
  const int64_t rb = P.block_rows == kBlk ? (P.rows + kBlk - 1) / kBlk : P.rows;
  const int64_t sr = P.block_rows == kBlk ? r / kBlk : r;
  const float s = P.scale[(batch * rb + sr) * cb + bx];
  const uint8_t* q = P.q + (batch * P.rows + r) * P.cols + c;
  const int64_t at = batch * P.x_stride + r * P.ldx + c;
  const int n = int(P.cols - c < 8 ? P.cols - c : 8);
  u32x2_t w = {0, 0};
  if (n == 8) {
    w = reinterpret_cast<const AnyAddress<u32x2_t>*>(q)->v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) w[e >> 2] |= uint32_t(q[e]) << (8 * (e & 3));
  }
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = from_q8<E5M2>(w[e >> 2] >> (8 * (e & 3)) & 0xff) * s;
  if constexpr (F32) {
    float* x = static_cast<float*>(P.x_out) + at;
    if (n == 8) {
      reinterpret_cast<AnyFloat*>(x)[0].v = f32x4_t{v[0], v[1], v[2], v[3]};
      reinterpret_cast<AnyFloat*>(x)[1].v = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) x[e] = v[e];
    }
  } else {
    uint16_t* x = static_cast<uint16_t*>(P.x_out) + at;
    const u32x4_t h = {pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]), pack2_bf16(v[6], v[7])};
    if (n == 8) {
      reinterpret_cast<AnyHalf*>(x)->v = h;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) x[e] = uint16_t(h[e >> 1] >> (16 * (e & 1)));
    }
  }
}

// ---- product ----------------------------------------------------------------

template <bool E5M2>
__device__ __forceinline__ bf16x2_t widen2(int w, bool hi) {
  if constexpr (E5M2)
    return hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.f, true)
              : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.f, false);
  else
    return hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true)
              : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false);
}
// Eight of a fragment's values (words 2p and 2p + 1) as bf16.
template <bool E5M2>
__device__ __forceinline__ bf16x8_t widen8(const i32x8_t& f, int p) {
  union { bf16x2_t h[4]; bf16x8_t v; } u;
  u.h[0] = widen2<E5M2>(f[2 * p], false);
  u.h[1] = widen2<E5M2>(f[2 * p], true);
  u.h[2] = widen2<E5M2>(f[2 * p + 1], false);
  u.h[3] = widen2<E5M2>(f[2 * p + 1], true);
  return u.v;
}

// Sum over one block of 128 k of a 16 x 16 piece, B first: the lane holds row
// lane % 16 of A's rows and four consecutive ones of B's.
template <bool A5, bool B5, bool EXACT>
__device__ __forceinline__ f32x4_t block_product(const i32x8_t& fb, const i32x8_t& fa) {
  f32x4_t p = {0.f, 0.f, 0.f, 0.f};
  if constexpr (EXACT) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<B5>(fb, q), widen8<A5>(fa, q), p, 0, 0, 0);
  } else {
    p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, fa, p, B5 ? 1 : 0, A5 ? 1 : 0, 0, 0, 0, 0);
  }
  return p;
}

// Tiles of 128 or 64, four waves in 2 x 2, operands staged through registers
// (one stage in flight, four with 64-tiles: a second one of the larger tile
// costs the two blocks per CU that its registers allow) and a two-slot LDS
// ring; any alignment.  fp32 results: every wave widens its fragments once per
// stage, 4096 x 4096 x 8190 takes 368 us, 747 TFLOP/s.
template <bool A5, bool B5, bool BROWS, bool VEC, int TILE, typename OutT>
__global__ void __launch_bounds__(kStageThreads, 2)
block_matmul_kernel(BlockArgs P) {
  constexpr bool EXACT = sizeof(OutT) == 4;
  constexpr int OPB = TILE * kBlk, D = TILE == 64 ? 4 : 1, F = TILE / 32;
  __shared__ __attribute__((aligned(1024))) char smem[4 * OPB];
  __shared__ __attribute__((aligned(16))) float scales[2][2 * TILE];     // A's rows, B's rows
  const uint32_t nt = (uint32_t(P.n) + TILE - 1) / TILE;
  uint32_t mt;
  if (P.offsets) mt = group_tiles(P.offsets, P.experts, int(P.m), TILE);
  else mt = (uint32_t(P.m) + TILE - 1) / TILE;
  const uint32_t pos = xcd_position(blockIdx.x, mt * nt);
  if (pos >= mt * nt) return;
  int tm, tn, row0, end, e = 0;
  tile_of_position(pos, mt, nt, &tm, &tn);
  if (P.offsets) {
    const GroupSpan g = group_of_tile(P.offsets, P.experts, int(P.m), TILE, tm, &row0);
    end = g.end;
    e = g.expert;
  } else {
    row0 = tm * TILE;
    end = int(P.m);
  }
  const int64_t j0 = int64_t(tn) * TILE;
  const int rows = end - row0 < TILE ? end - row0 : TILE;
  const int cols = int(P.n - j0 < TILE ? P.n - j0 : TILE);
  const int kb = int((P.k + kBlk - 1) / kBlk);
  const char* a = static_cast<const char*>(P.a) + row0 * P.lda;
  const char* b = static_cast<const char*>(P.b) + e * P.b_stride + j0 * P.ldb;
  // this thread's scale of a stage: the first TILE threads A's rows, the next B's
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const float* sp = nullptr;
  if (t < TILE) {
    if (t < rows) sp = P.a_scale + (int64_t(row0) + t) * kb;
  } else if (t - TILE < cols && t < 2 * TILE) {
    const int64_t brows = BROWS ? P.n : (P.n + kBlk - 1) / kBlk;
    sp = P.b_scale + (e * brows + (BROWS ? j0 + t - TILE : j0 / kBlk)) * kb;
  }
  const int wm = (wave >> 1) * (TILE / 2), wn = (wave & 1) * (TILE / 2);
  f32x4_t acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  u32x4_t va[D][TILE / 32], vb[D][TILE / 32];
  float vs[D];
  auto load = [&](int st, int d) {
    if (st < kb) {
      load_stage<TILE, VEC>(a, P.lda, rows, int64_t(st) * kBlk, P.k, va[d]);
      load_stage<TILE, VEC>(b, P.ldb, cols, int64_t(st) * kBlk, P.k, vb[d]);
      vs[d] = sp ? sp[st] : 0.f;
    }
  };
  auto write = [&](int st, int d) {
    if (st < kb) {
      write_stage<TILE>(smem + (st & 1) * 2 * OPB, va[d]);
      write_stage<TILE>(smem + (st & 1) * 2 * OPB + OPB, vb[d]);
      if (t < 2 * TILE) scales[st & 1][t] = vs[d];
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, d);
  write(0, 0);
  load(D, 0);
  for (int base = 0; base < kb; base += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int st = base + d;
      if (st >= kb) break;
      const char* cur = smem + (st & 1) * 2 * OPB;
      const float* sc = scales[st & 1];
      __syncthreads();
      write(st + 1, (d + 1) % D);
      load(st + 1 + D, (d + 1) % D);
      f32x4_t sb[F];
      if constexpr (BROWS) {
#pragma unroll
        for (int j = 0; j < F; ++j) sb[j] = *reinterpret_cast<const f32x4_t*>(sc + TILE + wn + 16 * j + 4 * (lane >> 4));
      }
      float sa[F];
#pragma unroll
      for (int i = 0; i < F; ++i) {
        sa[i] = sc[wm + 16 * i + (lane & 15)];
        if constexpr (!BROWS) sa[i] *= sc[TILE];   // the tile's columns share one scale
      }
      auto add = [&](int i, int j, const f32x4_t& p) {
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(BROWS ? sa[i] * sb[j][r] : sa[i], p[r], acc[i][j][r]);
      };
      i32x8_t fb[F];
#pragma unroll
      for (int j = 0; j < F; ++j) fb[j] = read_frag(cur + OPB, wn + 16 * j);
      if constexpr (EXACT) {
        // every fragment is widened once
        bf16x8_t wb[F][4];
#pragma unroll
        for (int j = 0; j < F; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) wb[j][q] = widen8<B5>(fb[j], q);
#pragma unroll
        for (int i = 0; i < F; ++i) {
          const i32x8_t fa = read_frag(cur, wm + 16 * i);
          f32x4_t p[F];
#pragma unroll
          for (int j = 0; j < F; ++j) p[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const bf16x8_t wa = widen8<A5>(fa, q);
#pragma unroll
            for (int j = 0; j < F; ++j) p[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j][q], wa, p[j], 0, 0, 0);
          }
#pragma unroll
          for (int j = 0; j < F; ++j) add(i, j, p[j]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < F; ++i) {
          const i32x8_t fa = read_frag(cur, wm + 16 * i);
#pragma unroll
          for (int j = 0; j < F; ++j) add(i, j, block_product<A5, B5, false>(fb[j], fa));
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < F; ++i) {
    const int r = wm + 16 * i + (lane & 15);
    if (r >= rows) continue;
    OutT* row = static_cast<OutT*>(P.c) + (int64_t(row0) + r) * P.ldc + j0;
#pragma unroll
    for (int j = 0; j < F; ++j) {
      const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      store4<OutT>(row, wn + 16 * j + 4 * (lane >> 4), cols, P.accumulate, v);
    }
  }
}

// ---- product, 256 x 256 tiles --------------------------------------------------
//
// The tile of bigtile.h with eight waves (2 in rows x 4 in columns, 128 x 64
// each): every block's result is scaled on the vector unit before it joins the
// sum, so the accumulators have to be vector registers, of which a wave has
// 256; two waves per SIMD let one wave's vector work run beside the other's
// matrix instructions.  A stage is 128 k, one block of scales.  The loads of
// the next stage go out over the first half of a stage's row blocks; the one
// barrier of a stage stands behind its last matrix instructions, and the next
// stage's first fragments are read while those run.  Persistent blocks, as in
// bigtile.h; a tile has an even number of stages.  8192^3: 527 to 540 us, 2.04 to
// 2.09 PFLOP/s; 8192 x 14336 x 4096: 467 us.
constexpr int kWaves8 = 8;
constexpr int kThreads8 = kWaves8 * 64;

struct BlockTile {
  const char* a;
  const char* b;
  const char* sa;
  const char* sb;
  char* c;
  int rows, cols;      // of C from the corner on; 0 rows: no tile
};

// The stream of a wave's loads: per stage four 1 KB pieces of each operand and
// 64 scales (waves 0-3: of A's rows, 4-7: of B's).  Past the last tile (no
// rows) the loads read nothing.
struct BlockStream {
  uint32_t at_a[4], at_b[4], at_scale;
  int first_k, lda, ldb, kb, k;
  bool per_block;          // 128 of this wave's rows share a scale
  const char* pa;
  const char* pb;
  const char* ps;
  int rows_a, rows_b, rows_s, st;
  __amdgpu_buffer_rsrc_t ra, rb, rs;
  uint32_t outside;

  __device__ __forceinline__ void init(int lda_, int ldb_, int k_, bool b_rows, int wave, int lane) {
    lda = lda_;
    ldb = ldb_;
    k = k_;
    kb = (k + kBlk - 1) / kBlk;
    per_block = wave >= 4 && !b_rows;
    first_k = ((lane & 7) ^ (((wave * 8 + (lane >> 3)) >> 1) & 7)) * 16;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t r = (wave + 8 * q) * 8 + (lane >> 3);
      at_a[q] = r * uint32_t(lda) + first_k;
      at_b[q] = r * uint32_t(ldb) + first_k;
    }
    const int r = (wave & 3) * 64 + lane;
    at_scale = uint32_t(per_block ? r >> 7 : r) * uint32_t(kb) * 4u;
  }
  __device__ __forceinline__ void start(const BlockTile& t, int wave) {
    pa = t.a;
    pb = t.b;
    ps = wave < 4 ? t.sa : t.sb;
    rows_a = t.rows;
    rows_b = t.rows > 0 ? t.cols : 0;
    rows_s = wave < 4 ? rows_a : per_block ? (rows_b + 127) >> 7 : rows_b;
    st = 0;
  }
  // Descriptors of the next stage's loads, then its nine loads one by one.
  __device__ __forceinline__ void prepare() {
    const int rest = k - st * kBlk;
    const int left = rest < 0 ? 0 : rest < kBlk ? rest : kBlk;      // of this stage's k
    const bool none = left == 0 || rows_a == 0;
    ra = slab_rsrc(pa, none ? 0u : uint32_t(rows_a - 1) * uint32_t(lda) + uint32_t(left));
    rb = slab_rsrc(pb, none ? 0u : uint32_t(rows_b - 1) * uint32_t(ldb) + uint32_t(left));
    rs = slab_rsrc(ps, none ? 0u : (uint32_t(rows_s - 1) * uint32_t(kb) + uint32_t(kb - st)) * 4u);
    outside = first_k < left ? 0u : kOutside;
    pa += kBlk;
    pb += kBlk;
    ps += 4;
    ++st;
  }
  __device__ __forceinline__ void load(int n, char* slot, float* scales, int wave) const {
    if (n == 8)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (DMUON_LDS void*)(scales + wave * 64), 4, int(at_scale), 0, 0, 0);
    else if (n & 1)
      slab_load_lds(rb, slot + kBigOp + (wave + 8 * (n >> 1)) * 1024, at_b[n >> 1] | outside);
    else
      slab_load_lds(ra, slot + (wave + 8 * (n >> 1)) * 1024, at_a[n >> 1] | outside);
  }
};

__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(7 << 4);      // vmcnt(0) lgkmcnt(0)
  plain_barrier();
}

template <bool A5, bool B5, bool BROWS>
struct BlockBig {
  char* const slot0;
  char* const slot1;
  float* const sc0;
  float* const sc1;
  const BigGroups* const groups;
  const int lane0, wave;
  uint32_t mt, nt, pos;
  BigPlan plan;
  BlockTile w, nw;
  BlockStream loads;
  int kb;

  __device__ __forceinline__ BlockBig(char* s0, char* s1, float* c0, float* c1, const BigGroups* g)
      : slot0(s0), slot1(s1), sc0(c0), sc1(c1), groups(g), lane0(threadIdx.x & 63), wave(uniform(threadIdx.x >> 6)) {}

  // The kernel's arguments, read again at each use (BlockArgs is its only parameter).
  static __device__ __forceinline__ const BlockArgs& args() {
    auto* p = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const BlockArgs*)p;
  }
  __device__ __forceinline__ void find(uint32_t p, BlockTile* t) const {
    t->rows = 0;
    t->cols = 1;
    uint32_t tile;
    int part;
    if (p >= plan.end || !plan.locate(p, &tile, &part)) return;
    const BlockArgs& P = args();
    int tm, tn, row0, end, e = 0;
    tile_of_position(tile, mt, nt, &tm, &tn);
    if (P.offsets) {
      e = groups->expert_of(P.experts, tm);
      row0 = uniform(groups->rows[e]) + (tm - uniform(groups->tiles[e])) * kBig;
      end = uniform(groups->rows[e + 1]);
    } else {
      row0 = tm * kBig;
      end = int(P.m);
    }
    const int64_t j0 = int64_t(tn) * kBig, n_scales = BROWS ? P.n : (P.n + kBlk - 1) / kBlk;
    int rows = end - row0 < kBig ? end - row0 : kBig;
    row0 += plan.cut(part, &rows);
    if (rows <= 0) return;
    t->rows = uniform(rows);
    t->cols = uniform(int(P.n - j0 < kBig ? P.n - j0 : kBig));
    t->a = uniform_ptr(static_cast<const char*>(P.a) + row0 * P.lda);
    t->b = uniform_ptr(static_cast<const char*>(P.b) + e * P.b_stride + j0 * P.ldb);
    t->sa = uniform_ptr(reinterpret_cast<const char*>(P.a_scale + int64_t(row0) * kb));
    t->sb = uniform_ptr(reinterpret_cast<const char*>(P.b_scale + (e * n_scales + (BROWS ? j0 : 2 * tn)) * kb));
    t->c = uniform_ptr(static_cast<char*>(P.c) + (row0 * P.ldc + j0) * 2);
  }
  __device__ __forceinline__ i32x8_t frag(const char* slot, int operand, int b, int lane) const {
    union { u32x4_t h[2]; i32x8_t v; } u;
    u.h[0] = *reinterpret_cast<const u32x4_t*>(slot + (operand + b * 2048 + row_slot(lane & 15, lane >> 4)));
    u.h[1] = *reinterpret_cast<const u32x4_t*>(slot + (operand + b * 2048 + row_slot(lane & 15, 4 + (lane >> 4))));
    return u.v;
  }
  // Loads issued before row block i of NI: all nine within the first half.
  static constexpr int kLoadsAt(int i, int ni) { return i * 18 / ni < 9 ? i * 18 / ni : 9; }

  // B's fragments and scales of a stage, and the first row block's of A.
  struct Frags {
    i32x8_t b[4], a[2];
    f32x4_t sb[4];
    float sa[2], sb_all;
  };
  __device__ __forceinline__ void read_first(const char* slot, const float* sc, int lane, Frags& f) const {
    const int wm = wave >> 2, wn = wave & 3;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f.b[j] = frag(slot, kBigOp, 4 * wn + j, lane);
      if constexpr (BROWS) f.sb[j] = *reinterpret_cast<const f32x4_t*>(sc + kBig + 64 * wn + 16 * j + 4 * (lane >> 4));
    }
    f.sb_all = BROWS ? 1.f : sc[kBig + 64 * wn];
    f.a[0] = frag(slot, 0, wm, lane);
    f.sa[0] = sc[16 * wm + (lane & 15)] * f.sb_all;
  }
  // One stage from `slot`, whose first fragments are in registers, with the
  // loads of the stage after into `to` spread over its row blocks.  Behind the
  // last row block's matrix instructions a barrier (the next stage has landed,
  // this one is read) and the next stage's first reads.
  template <int NI>
  __device__ __forceinline__ void multiply(const char* slot, const float* sc, char* to, float* to_sc, Frags& f,
                                           f32x4_t (&acc)[NI][4]) {
    const int lane = here(lane0), wm = wave >> 2, wv = here_scalar(wave);
    loads.prepare();
    // row block i's matrix instructions go out before row block i - 1's
    // results are scaled and added; the scheduling barriers keep it at that
    // (two row blocks of results in registers)
    f32x4_t p[2][4];
    auto add = [&](int i) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][j][r] = fmaf(BROWS ? f.sa[i & 1] * f.sb[j][r] : f.sa[i & 1], p[i & 1][j][r], acc[i][j][r]);
      // here and not later: the compiler would keep the results for the next stage
      asm volatile("" : "+v"(acc[i][0]), "+v"(acc[i][1]), "+v"(acc[i][2]), "+v"(acc[i][3]));
    };
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) p[i & 1][j] = block_product<A5, B5, false>(f.b[j], f.a[i & 1]);
      if (i > 0) add(i - 1);
      if (i + 1 < NI) {
        f.a[(i + 1) & 1] = frag(slot, 0, 2 * (i + 1) + wm, lane);
        f.sa[(i + 1) & 1] = sc[32 * (i + 1) + 16 * wm + (lane & 15)] * f.sb_all;
      }
#pragma unroll
      for (int n = kLoadsAt(i, NI); n < kLoadsAt(i + 1, NI); ++n) loads.load(n, to, to_sc, wv);
      __builtin_amdgcn_sched_barrier(0);
    }
    stage_barrier();
    if constexpr (BROWS) {
      // the last row block still needs this stage's scales
      add(NI - 1);
      __builtin_amdgcn_sched_barrier(0);
      read_first(to, to_sc, lane, f);
    } else {
      static_assert(NI % 2 == 0, "the last row block's scale is in sa[1]");
      read_first(to, to_sc, lane, f);
      add(NI - 1);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  template <int NI>
  __device__ __forceinline__ void tile() {
    f32x4_t acc[NI][4];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const int stages = (kb + 1) / 2 * 2;
    Frags f;
    read_first(slot0, sc0, here(lane0), f);
    for (int st = 0; st < stages; st += 2) {
      multiply<NI>(slot0, sc0, slot1, sc1, f, acc);
      if (st + 2 >= stages) loads.start(nw, wave);
      multiply<NI>(slot1, sc1, slot0, sc0, f, acc);
    }
    store<NI>(acc);
  }
  template <int NI>
  __device__ __forceinline__ void store(const f32x4_t (&acc)[NI][4]) {
    const BlockArgs& P = args();
    const int lane = here(lane0);
    const int64_t ldc = P.ldc;
    const bool accumulate = P.accumulate;
    const int g = lane >> 4, col0 = 64 * (wave & 3);
    const bool plain = !accumulate && w.cols == kBig;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = 32 * i + 16 * (wave >> 2) + (lane & 15);
      uint16_t* row = reinterpret_cast<uint16_t*>(w.c) + int64_t(r) * ldc + col0;
      if (plain) {
#pragma unroll
        for (int j = 0; j < 4; j += 2) store_pair(row + 16 * j, acc[i][j], acc[i][j + 1], g, r < w.rows);
      } else if (r < w.rows) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
          store4<uint16_t>(row, 16 * j + 4 * g, w.cols - col0, accumulate, v);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  __device__ __forceinline__ void run(BigGroups* g) {
    {
      const BlockArgs& P = args();
      kb = int((P.k + kBlk - 1) / kBlk);
      nt = (uint32_t(P.n) + kBig - 1) / kBig;
      if (P.offsets) {
        g->build(P.offsets, P.experts, int(P.m));
        mt = uniform(g->tiles[P.experts]);
      } else {
        mt = (uint32_t(P.m) + kBig - 1) / kBig;
      }
      plan.make(mt * nt, true);
      loads.init(int(P.lda), int(P.ldb), int(P.k), BROWS, wave, lane0);
    }
    const uint32_t grid = gridDim.x, per = grid / kNumXcd;
    pos = grid % kNumXcd ? blockIdx.x : (blockIdx.x % kNumXcd) * per + blockIdx.x / kNumXcd;
    find(pos, &w);
    if (w.rows <= 0) return;
    loads.start(w, wave);
    loads.prepare();
#pragma unroll
    for (int n = 0; n < 9; ++n) loads.load(n, slot0, sc0, wave);
    stage_barrier();
    while (true) {
      pos += grid;
      find(pos, &nw);
      if (w.rows > 128) tile<8>();
      else if (w.rows > 64) tile<4>();
      else tile<2>();
      if (nw.rows <= 0) break;
      w = nw;
    }
    wait_loads<0>();
  }
};

template <bool A5, bool B5, bool BROWS>
__global__ void __launch_bounds__(kThreads8)
block_matmul_big_kernel(BlockArgs P) {
  __shared__ BigSlot slot0, slot1;
  __shared__ float sc0[2 * kBig], sc1[2 * kBig];
  __shared__ BigGroups groups;
  BlockBig<A5, B5, BROWS> run(slot0.data, slot1.data, sc0, sc1, &groups);
  run.run(&groups);
}

template <bool A5, bool B5, bool BROWS>
void launch_matmul_big(const BlockArgs& P, unsigned blocks, hipStream_t stream) {
  hipLaunchKernelGGL((block_matmul_big_kernel<A5, B5, BROWS>), dim3(blocks), dim3(kThreads8), 0, stream, P);
}

// ---- product, few rows ----------------------------------------------------------

// Formats and block rows are run-time values here: the branches on them are
// uniform, and memory bounds the kernel.
template <bool EXACT>
__device__ __forceinline__ f32x4_t block_product_of(const i32x8_t& fb, const i32x8_t& fa, bool a5, bool b5) {
  if (a5) return b5 ? block_product<true, true, EXACT>(fb, fa) : block_product<true, false, EXACT>(fb, fa);
  return b5 ? block_product<false, true, EXACT>(fb, fa) : block_product<false, false, EXACT>(fb, fa);
}

template <bool EXACT>
struct BlockSkinny : SkinnyFloat {
  const float* sa;      // of the tile's first row; kb per row
  const float* sb;      // of the tile's first column, or of its 128 columns
  int64_t kb;
  bool a5, b5, b_rows;

  template <int MB, int NB>
  __device__ __forceinline__ void step(int s, int lane, int rows, int cols, const SkinnyFrag (&b)[NB],
                                       const SkinnyFrag (&a)[MB], f32x4_t (&acc)[NB][MB]) const {
    float x[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const int t = 16 * m + (lane & 15);
      x[m] = sa[(t < rows ? t : rows - 1) * kb + s];
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      f32x4_t w;
      if (b_rows) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * n + 4 * (lane >> 4) + r;
          w[r] = sb[(j < cols ? j : cols - 1) * kb + s];
        }
      } else {
        const float all = sb[s];
        w = f32x4_t{all, all, all, all};
      }
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const f32x4_t p = block_product_of<EXACT>(__builtin_bit_cast(i32x8_t, b[n]), __builtin_bit_cast(i32x8_t, a[m]),
                                                  a5, b5);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[n][m][r] = fmaf(x[m] * w[r], p[r], acc[n][m][r]);
      }
    }
  }
};

template <int MB, int NB, int W, typename OutT>
__global__ void __launch_bounds__(64 * W)
block_skinny_kernel(BlockArgs P, int a5, int b5, int b_rows) {
  __shared__ __attribute__((aligned(16))) float sums[W * MB * NB * 256];
  const uint32_t nt = (uint32_t(P.n) + 16 * NB - 1) / (16 * NB);
  const uint32_t tm = blockIdx.x / nt, tn = blockIdx.x - tm * nt;
  int row0 = int(tm) * 16 * MB, end = int(P.m), e = 0;
  if (P.offsets) {
    const GroupSpan g = group_of_tile(P.offsets, P.experts, int(P.m), 16 * MB, tm, &row0);
    end = g.end;
    e = g.expert;
  }
  if (row0 >= end) return;
  const int64_t j0 = int64_t(tn) * (16 * NB), kb = (P.k + kBlk - 1) / kBlk;
  const int64_t b_scales = b_rows ? P.n : (P.n + kBlk - 1) / kBlk;
  BlockSkinny<sizeof(OutT) == 4> op;
  op.sa = P.a_scale + int64_t(row0) * kb;
  op.sb = P.b_scale + (e * b_scales + (b_rows ? j0 : j0 / kBlk)) * kb;
  op.kb = kb;
  op.a5 = a5;
  op.b5 = b5;
  op.b_rows = b_rows;
  skinny_block<decltype(op), MB, NB, W, OutT>(op, static_cast<const char*>(P.a) + row0 * P.lda, P.lda,
                                              static_cast<const char*>(P.b) + e * P.b_stride + j0 * P.ldb, P.ldb,
                                              static_cast<OutT*>(P.c) + row0 * P.ldc + j0, P.ldc,
                                              end - row0 < 16 * MB ? end - row0 : 16 * MB,
                                              int(P.n - j0 < 16 * NB ? P.n - j0 : 16 * NB), P.k, P.accumulate,
                                              sums);
}

int64_t skinny_blocks(const BlockArgs& P, int mb, int nb) {
  const int64_t used = P.offsets ? (P.experts < P.m ? P.experts : P.m) : 1;
  return (P.m / (16 * mb) + used) * ((P.n + 16 * nb - 1) / (16 * nb));
}
template <int MB, int NB, typename OutT>
hipError_t launch_skinny(const BlockArgs& P, int a5, int b5, int b_rows, hipStream_t stream) {
  const int64_t blocks = skinny_blocks(P, MB, NB);
  const dim3 grid(static_cast<unsigned>(blocks));
  if constexpr (skinny_sixteen(MB, NB, sizeof(OutT) == 4)) {
    if (blocks < kSkinnyWide) {
      hipLaunchKernelGGL((block_skinny_kernel<MB, NB, 16, OutT>), grid, dim3(1024), 0, stream, P, a5, b5, b_rows);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((block_skinny_kernel<MB, NB, 8, OutT>), grid, dim3(512), 0, stream, P, a5, b5, b_rows);
  return hipGetLastError();
}
template <int MB, int NB>
hipError_t launch_skinny(const BlockArgs& P, int a5, int b5, int b_rows, bool f32, hipStream_t stream) {
  return f32 ? launch_skinny<MB, NB, float>(P, a5, b5, b_rows, stream)
             : launch_skinny<MB, NB, uint16_t>(P, a5, b5, b_rows, stream);
}

template <bool A5, bool B5, bool BROWS, typename OutT>
void launch_matmul(const BlockArgs& P, bool vec, bool small, dim3 grid, hipStream_t stream) {
  const dim3 block(kStageThreads);
  if (small) {
    if (vec) hipLaunchKernelGGL((block_matmul_kernel<A5, B5, BROWS, true, 64, OutT>), grid, block, 0, stream, P);
    else hipLaunchKernelGGL((block_matmul_kernel<A5, B5, BROWS, false, 64, OutT>), grid, block, 0, stream, P);
  } else {
    if (vec) hipLaunchKernelGGL((block_matmul_kernel<A5, B5, BROWS, true, 128, OutT>), grid, block, 0, stream, P);
    else hipLaunchKernelGGL((block_matmul_kernel<A5, B5, BROWS, false, 128, OutT>), grid, block, 0, stream, P);
  }
}
template <bool A5, bool B5>
void launch_matmul_fmt(const BlockArgs& P, bool brows, bool f32, bool vec, bool small, dim3 grid, hipStream_t stream) {
  if (brows) {
    if (f32) launch_matmul<A5, B5, true, float>(P, vec, small, grid, stream);
    else launch_matmul<A5, B5, true, uint16_t>(P, vec, small, grid, stream);
  } else {
    if (f32) launch_matmul<A5, B5, false, float>(P, vec, small, grid, stream);
    else launch_matmul<A5, B5, false, uint16_t>(P, vec, small, grid, stream);
  }
}

}  // namespace

hipError_t launch_quantize(const QuantArgs& P, int x_dtype, int q_dtype, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((P.cols + kBlk - 1) / kBlk * ((P.rows + kBlk - 1) / kBlk)), 1,
                  static_cast<unsigned>(P.batch));
  const bool f32 = x_dtype == DT_F32, e5 = q_dtype == DT_E5M2;
  if (f32 && e5) hipLaunchKernelGGL((quantize_kernel<true, true>), grid, dim3(256), 0, stream, P);
  else if (f32) hipLaunchKernelGGL((quantize_kernel<true, false>), grid, dim3(256), 0, stream, P);
  else if (e5) hipLaunchKernelGGL((quantize_kernel<false, true>), grid, dim3(256), 0, stream, P);
  else hipLaunchKernelGGL((quantize_kernel<false, false>), grid, dim3(256), 0, stream, P);
  return hipGetLastError();
}

hipError_t launch_dequantize(const QuantArgs& P, int x_dtype, int q_dtype, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((P.cols + kBlk - 1) / kBlk * ((P.rows + 15) / 16)), 1,
                  static_cast<unsigned>(P.batch));
  const bool f32 = x_dtype == DT_F32, e5 = q_dtype == DT_E5M2;
  if (f32 && e5) hipLaunchKernelGGL((dequantize_kernel<true, true>), grid, dim3(256), 0, stream, P);
  else if (f32) hipLaunchKernelGGL((dequantize_kernel<true, false>), grid, dim3(256), 0, stream, P);
  else if (e5) hipLaunchKernelGGL((dequantize_kernel<false, true>), grid, dim3(256), 0, stream, P);
  else hipLaunchKernelGGL((dequantize_kernel<false, false>), grid, dim3(256), 0, stream, P);
  return hipGetLastError();
}

hipError_t launch_block_matmul(const BlockArgs& P, int a_dtype, int b_dtype, bool brows, bool f32, bool vec,
                               hipStream_t stream) {
  const int64_t used = P.offsets ? (P.experts < P.m ? P.experts : P.m) : 1;
  const int64_t big = (P.m / kBig + used) * ((P.n + kBig - 1) / kBig);
  // 256-tiles from 192 on (2048 x 4096 x 4096, 128 of them: 62 us so, 57 in
  // 128-tiles); offsets of a tile's rows within 31 bits.  With few rows per expert
  // too: both kernels then only read the weights (one row per expert, from HBM,
  // these tiles and the few-rows kernel: 8 experts of 14336 x 4096 128 and 118 us,
  // 16 of 4096 x 4096 73 and 71, 64 of 2048 x 2048 67 and 84, 32 of 4096 x 512 22 and 58)
  const bool fits = P.lda <= kMaxBigPitch && P.ldb <= kMaxBigPitch && P.experts <= kBigExperts;
  if (vec && !f32 && fits && big >= 192) {
    const unsigned blocks = static_cast<unsigned>(big < kBigBlocks ? big : kBigBlocks);
    const int which = (a_dtype == DT_E5M2 ? 4 : 0) + (b_dtype == DT_E5M2 ? 2 : 0) + (brows ? 1 : 0);
    switch (which) {
      case 0: launch_matmul_big<false, false, false>(P, blocks, stream); break;
      case 1: launch_matmul_big<false, false, true>(P, blocks, stream); break;
      case 2: launch_matmul_big<false, true, false>(P, blocks, stream); break;
      case 3: launch_matmul_big<false, true, true>(P, blocks, stream); break;
      case 4: launch_matmul_big<true, false, false>(P, blocks, stream); break;
      case 5: launch_matmul_big<true, false, true>(P, blocks, stream); break;
      case 6: launch_matmul_big<true, true, false>(P, blocks, stream); break;
      default: launch_matmul_big<true, true, true>(P, blocks, stream); break;
    }
    return hipGetLastError();
  }
  const int a5 = a_dtype == DT_E5M2, b5 = b_dtype == DT_E5M2;
  if (vec && skinny_blocks(P, 1, 1) <= kMaxSkinnyBlocks) {
    // at most 16, or 32, rows per expert on average
    const int64_t experts = P.offsets ? P.experts : 1;
    if (P.m <= 16 * experts) {
      if (skinny_blocks(P, 1, 2) >= kSkinnyWide) return launch_skinny<1, 2>(P, a5, b5, brows, f32, stream);
      return launch_skinny<1, 1>(P, a5, b5, brows, f32, stream);
    }
    if (P.m <= 32 * experts) return launch_skinny<2, 2>(P, a5, b5, brows, f32, stream);
  }
  // 64-tiles where 128-tiles would give fewer than one per CU: 2048 x 2560 x
  // 1000 with fp32 results takes 35 us in 128-tiles, 41 in 64-tiles; 265 x 464 x 3584
  // takes 38 us in 128-tiles, 16 in 64-tiles
  auto tiles = [&](int64_t t) { return (P.m / t + used) * ((P.n + t - 1) / t); };
  const bool small = tiles(128) < 256 && tiles(64) <= kMaxSkinnyBlocks;
  const dim3 grid(static_cast<unsigned>(grouped_grid(tiles(small ? 64 : 128))));
  if (a_dtype == DT_E5M2) {
    if (b_dtype == DT_E5M2) launch_matmul_fmt<true, true>(P, brows, f32, vec, small, grid, stream);
    else launch_matmul_fmt<true, false>(P, brows, f32, vec, small, grid, stream);
  } else {
    if (b_dtype == DT_E5M2) launch_matmul_fmt<false, true>(P, brows, f32, vec, small, grid, stream);
    else launch_matmul_fmt<false, false>(P, brows, f32, vec, small, grid, stream);
  }
  return hipGetLastError();
}

}  // namespace dmuon

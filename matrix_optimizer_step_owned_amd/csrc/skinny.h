// Products of few rows with whole weight matrices (serving): C[t][j] = sum_k
// A[t][k] B[j][k] for at most 16 MB rows t of one expert, both operands with
// contiguous k, bf16, 8-bit blocks or 8-bit integers.
//
// The weights are read once and bound everything, so nothing is staged: a block
// takes 16 NB rows of B, its W waves split k between them, and a lane loads its
// fragment of a matrix instruction straight into registers, 32 of the 128
// bytes that a row has in one step (two 16-byte loads; the four lanes of a row
// take whole lines).  Four steps are in flight per wave.  A comes from L2.  The
// waves' sums are added in LDS in wave order, so results are deterministic.
#pragma once

#include "grouped.h"

namespace dmuon {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct SkinnyFrag {
  u32x4_t h[2];
};

// 32 bytes of the 128 from byte `at` of a row of `bytes` bytes on: those at 16 g and
// at 64 + 16 g; bytes past the row read as zero.
__device__ __forceinline__ SkinnyFrag skinny_load(const char* row, int64_t at, int64_t bytes, int g) {
  SkinnyFrag f;
  f.h[0] = u32x4_t{0, 0, 0, 0};
  f.h[1] = u32x4_t{0, 0, 0, 0};
  const int64_t rest = bytes - at;
  const int left = rest < 0 ? 0 : rest > 128 ? 128 : int(rest);
  if (16 * g < left) f.h[0] = *reinterpret_cast<const u32x4_t*>(row + at + 16 * g);
  if (64 + 16 * g < left) f.h[1] = *reinterpret_cast<const u32x4_t*>(row + at + 64 + 16 * g);
  return f;
}

// Op: Acc, the accumulators' type (four floats or ints); load(row, byte, row's bytes, g) a
// fragment; step(...) adds one step's products; finish(sums, row, first column,
// columns) turns a lane's four sums into results.
struct SkinnyFloat {
  using Acc = f32x4_t;
  static __device__ __forceinline__ SkinnyFrag load(const char* row, int64_t at, int64_t bytes, int g) {
    return skinny_load(row, at, bytes, g);
  }
  __device__ __forceinline__ f32x4_t finish(const f32x4_t& v, int, int, int) const { return v; }
};
template <class Op, int MB, int NB, int W, typename OutT>
__device__ __forceinline__ void skinny_block(const Op& op, const char* a, int64_t lda, const char* b, int64_t ldb,
                                             OutT* c, int64_t ldc, int rows, int cols, int64_t row_bytes,
                                             bool accumulate, float* sums) {
  constexpr int U = 4;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  using Acc = typename Op::Acc;
  Acc acc[NB][MB];
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int m = 0; m < MB; ++m) acc[n][m] = Acc{0, 0, 0, 0};
  const int steps = int((row_bytes + 127) / 128);
  // rows past the end read the last one: their results are not stored
  const char* bp[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int j = 16 * n + r;
    bp[n] = b + (j < cols ? j : cols - 1) * ldb;
  }
  const char* ap[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int t = 16 * m + r;
    ap[m] = a + (t < rows ? t : rows - 1) * lda;
  }
  for (int s0 = wave * U; s0 < steps; s0 += W * U) {
    SkinnyFrag fb[U][NB], fa[U][MB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = int64_t(s0 + u) * 128;
#pragma unroll
      for (int n = 0; n < NB; ++n) fb[u][n] = Op::load(bp[n], at, row_bytes, g);
#pragma unroll
      for (int m = 0; m < MB; ++m) fa[u][m] = Op::load(ap[m], at, row_bytes, g);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + u < steps) op.template step<MB, NB>(s0 + u, lane, rows, cols, fb[u], fa[u], acc);
    }
  }
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int m = 0; m < MB; ++m)
      *reinterpret_cast<Acc*>(sums + ((wave * NB * MB + n * MB + m) * 64 + lane) * 4) = acc[n][m];
  __syncthreads();
  for (int q = wave; q < NB * MB; q += W) {
    Acc sum = *reinterpret_cast<const Acc*>(sums + (q * 64 + lane) * 4);
#pragma unroll
    for (int w = 1; w < W; ++w) sum += *reinterpret_cast<const Acc*>(sums + ((w * NB * MB + q) * 64 + lane) * 4);
    const int n = q / MB, t = 16 * (q % MB) + r;
    if (t < rows) {
      const f32x4_t v = op.finish(sum, t, 16 * n + 4 * g, cols);
      const float x[4] = {v[0], v[1], v[2], v[3]};
      store4<OutT>(c + t * ldc, 16 * n + 4 * g, cols, accumulate, x);
    }
  }
}

// Blocks of one launch: fewer than 2^32 threads.
constexpr int64_t kMaxSkinnyBlocks = int64_t(1) << 23;

// Two blocks of 16 columns per block halve the reads of A, which come from L2
// but take the same load path as the weights; worth it while enough blocks remain.
constexpr int64_t kSkinnyWide = 256;

// Waves per block: eight (7 x 14336 x 4096 in 8 bits, 448 blocks: 15.2 us, 15.7
// with four), and sixteen for fewer blocks than CUs of the smallest form (4 rows
// of 1024 x 14336, weights from HBM: bf16 22.2 us against 23.1 with eight, 8-bit
// 14.5 against 15.8).  Sixteen waves leave a lane 128 registers, which the larger
// forms and those with fp32 results exceed: they then keep up to 215 in scratch
// memory (17 rows of 4096 x 4096, sixteen and eight waves: bf16 35.5 and 17.3 us,
// 8-bit 34.2 and 11.2, with fp32 results 34.0 and 12.9).
constexpr bool skinny_sixteen(int mb, int nb, bool f32) { return mb * nb == 1 && !f32; }

}  // namespace dmuon

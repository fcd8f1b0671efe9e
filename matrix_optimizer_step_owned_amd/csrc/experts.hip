// Matrix products of experts with ragged token counts.
//
// Tokens are sorted by expert: expert e has rows offsets[e] .. offsets[e+1]
// of x (tokens x k), y and dy (tokens x n); its weights are w[e] (n x k).
//   forward          y[t]  = w[e] x[t]                 sums over k
//   input gradient   dx[t] = w[e]^T dy[t]              sums over n
//   weight gradient  dw[e] = sum over its t of dy[t] x[t]^T
// One form C[i][j] = sum_s A(i, s) B(j, s) covers the three; they differ in
// which operand's rows run along the summed index:
//   forward:         A = x rows      (s contiguous), B = w rows    (s contiguous)
//   input gradient:  A = dy rows     (s contiguous), B = w columns (j contiguous)
//   weight gradient: A = dy columns  (i contiguous), B = x columns (j contiguous)
//
// bf16 operands go through v_mfma_f32_16x16x32_bf16 with fp32 accumulators.
// A contiguous-s operand sits in LDS as rows of 64 s (128 bytes) and a lane
// reads its eight s of one row with one 16-byte read; the other kind sits as
// 64 rows of 128 i and is read through the LDS transpose read
// (ds_read_b64_tr_b16: sixteen lanes name a 4 x 16 piece by rows and each
// receives one column of four), two reads for eight s.  So no operand is
// transposed in memory.  Both LDS layouts are swizzled so that a read covers
// all 64 banks once.  fp32 operands go through v_mfma_f32_32x32x2_f32.
#include <type_traits>

#include "bigtile.h"
#include "skinny.h"

namespace dmuon {
namespace {

constexpr int kTile = 128;        // edge of the larger tile
constexpr int kSmallTile = 64;
constexpr int kStage = 64;        // bf16: summed indices per LDS stage
constexpr int kThreads = 256;     // four waves, 2 x 2 quadrants of the tile
// Stages of operands in flight in registers: four for the small tile (16
// registers a stage), two for the larger one.  A stage's arithmetic takes
// 0.1 to 0.5 us and a load 1 us or more, so with one stage in flight a few
// tiles with a long sum ran at a load's latency per stage.
constexpr int depth_of(int tile) { return tile == kTile ? 2 : 4; }

// What one block works on: rows/cols of C that exist from the tile's corner
// on, the length of the sum, and the corner's operand and result addresses.
struct Work {
  const char* a;
  const char* b;
  char* c;
  int rows, cols, sum;
  int64_t lda, ldb, ldc;   // bytes per row as stored
  int row0, col0;          // rows and columns of C that the tile before writes
};

// A last tile of columns that would end inside a 16-byte chunk starts a few
// columns earlier, inside the tile before, so that it ends with a whole chunk:
// element by element such chunks took 1.6 times as long (fp32 weight gradient
// of 3000 rows, 1024 x 511: 138 us against 82 with 512 columns).  Returns the
// columns gained.
__device__ __forceinline__ int whole_chunks(const char** p, int* extent, int64_t before, int eb) {
  const int n = 16 / eb, d = before > 0 ? (n - *extent % n) % n : 0;
  *p -= d * eb;
  *extent += d;
  return d;
}

template <int OP, bool VEC>
__device__ __forceinline__ bool find_work(const ExpertArgs& P, int tile_m, int tile_n, int eb, int out_eb, Work* w) {
  w->row0 = w->col0 = 0;
  int tm, tn;
  if constexpr (OP == OP_WEIGHT) {
    const uint32_t mt = (uint32_t(P.n) + tile_m - 1) / tile_m, nt = (uint32_t(P.k) + tile_n - 1) / tile_n;
    const uint32_t total = mt * nt * P.experts, pos = xcd_position(blockIdx.x, mt * nt);
    if (pos >= total) return false;
    const uint32_t e = pos / (mt * nt);
    tile_of_position(pos - e * mt * nt, mt, nt, &tm, &tn);
    const GroupSpan g = group_of_expert(P.offsets, P.experts, P.tokens, e);
    const int64_t i0 = int64_t(tm) * tile_m, j0 = int64_t(tn) * tile_n;
    w->sum = g.end - g.begin;
    if (w->sum == 0 && P.accumulate) return false;   // left as it is
    w->rows = int(P.n - i0 < tile_m ? P.n - i0 : tile_m);
    w->cols = int(P.k - j0 < tile_n ? P.k - j0 : tile_n);
    w->lda = P.ld_n * eb;
    w->ldb = P.ld_k * eb;
    w->ldc = P.ldw * out_eb;
    w->a = static_cast<const char*>(P.a) + g.begin * w->lda + i0 * eb;
    w->b = static_cast<const char*>(P.b) + g.begin * w->ldb + j0 * eb;
    w->c = static_cast<char*>(P.c) + e * P.w_stride * out_eb + i0 * w->ldc + j0 * out_eb;
    if constexpr (!VEC) {
      w->row0 = whole_chunks(&w->a, &w->rows, i0, eb);
      w->col0 = whole_chunks(&w->b, &w->cols, j0, eb);
      w->c -= w->row0 * w->ldc + w->col0 * out_eb;
    }
  } else {
    const int64_t cols = OP == OP_FORWARD ? P.n : P.k;
    const uint32_t nt = (uint32_t(cols) + tile_n - 1) / tile_n;
    const uint32_t mt = group_tiles(P.offsets, P.experts, P.tokens, tile_m);
    const uint32_t pos = xcd_position(blockIdx.x, mt * nt);
    if (pos >= mt * nt) return false;
    tile_of_position(pos, mt, nt, &tm, &tn);
    int row0;
    const GroupSpan g = group_of_tile(P.offsets, P.experts, P.tokens, tile_m, tm, &row0);
    const int64_t j0 = int64_t(tn) * tile_n;
    w->rows = g.end - row0 < tile_m ? g.end - row0 : tile_m;
    w->cols = int(cols - j0 < tile_n ? cols - j0 : tile_n);
    w->sum = int(OP == OP_FORWARD ? P.k : P.n);
    w->lda = (OP == OP_FORWARD ? P.ld_k : P.ld_n) * eb;
    w->ldb = P.ldw * eb;
    w->ldc = (OP == OP_FORWARD ? P.ld_n : P.ld_k) * out_eb;
    w->a = static_cast<const char*>(P.a) + row0 * w->lda;
    w->b = static_cast<const char*>(P.b) + g.expert * P.w_stride * eb + (OP == OP_FORWARD ? j0 * w->ldb : j0 * eb);
    w->c = static_cast<char*>(P.c) + row0 * w->ldc + j0 * out_eb;
    if constexpr (!VEC && OP == OP_INPUT) {
      w->col0 = whole_chunks(&w->b, &w->cols, j0, eb);
      w->c -= w->col0 * out_eb;
    }
  }
  return true;
}

// ---- bf16 -------------------------------------------------------------------

// LDS offset of the 32-byte unit u (16 columns) of row s, rows of TILE columns:
// the eight rows that half a wave's transpose read touches (s & 3 and bit 3)
// go to eight different pieces of the 256 bytes that the banks hold.
template <int TILE>
__device__ __forceinline__ int col_slot(int s, int u) {
  if constexpr (TILE == 128) return s * 256 + ((u ^ ((s & 3) | ((s >> 1) & 4))) << 5);
  else return s * 128 + ((u ^ (((s >> 1) & 1) | ((s >> 2) & 2))) << 5);
}

// One thread's share of an operand's stage: TILE / 32 chunks of 16 bytes.
template <int TILE, bool COLS, bool VEC>
__device__ __forceinline__ void load_stage(const char* base, int64_t ld, int extent, int s0, int sum,
                                           u32x4_t (&v)[TILE / 32]) {
  const int t = threadIdx.x;
  constexpr int PER = TILE / 8;          // chunks per row of columns
#pragma unroll
  for (int q = 0; q < TILE / 32; ++q) {
    if constexpr (COLS) {   // row s, columns 8c..
      const int s = s0 + t / PER + kThreads / PER * q, c = (t % PER) * 8;
      v[q] = load_chunk<2, VEC>(base + s * ld + c * 2, s < sum ? extent - c : 0);
    } else {                // row r, s 8c..
      const int r = (t >> 3) + 32 * q, c = (t & 7) * 8;
      v[q] = load_chunk<2, VEC>(base + r * ld + (s0 + c) * 2, r < extent ? sum - s0 - c : 0);
    }
  }
}
template <int TILE, bool COLS>
__device__ __forceinline__ void write_stage(char* lds, const u32x4_t (&v)[TILE / 32]) {
  const int t = threadIdx.x;
  constexpr int PER = TILE / 8;
#pragma unroll
  for (int q = 0; q < TILE / 32; ++q) {
    const int at = COLS ? col_slot<TILE>(t / PER + kThreads / PER * q, (t % PER) >> 1) + (t & 1) * 16
                        : row_slot((t >> 3) + 32 * q, t & 7);
    *reinterpret_cast<u32x4_t*>(lds + at) = v[q];
  }
}
// A lane's fragment: row (or column) r0 + lane % 16, s = 32 step + 8 (lane / 16) ..
template <int TILE, bool COLS>
__device__ __forceinline__ bf16x8_t read_frag(const char* lds, int r0, int step) {
  const int lane = threadIdx.x & 63;
  if constexpr (COLS) {
    typedef short s16x4_t __attribute__((ext_vector_type(4)));
    const int s = 32 * step + 8 * (lane >> 4) + ((lane & 15) >> 2);
    const char* p = lds + col_slot<TILE>(s, r0 >> 4) + (lane & 3) * 8;
    const char* q = lds + col_slot<TILE>(s + 4, r0 >> 4) + (lane & 3) * 8;
    union { s16x4_t h[2]; bf16x8_t v; } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DMUON_LDS s16x4_t*)p);
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DMUON_LDS s16x4_t*)q);
    return u.v;
  } else {
    return *reinterpret_cast<const bf16x8_t*>(lds + row_slot(r0 + (lane & 15), 4 * step + (lane >> 4)));
  }
}

// Bound by a stage's latency where tiles are few and by the LDS reads where
// they are many (each wave reads its operands' 64 or 32 rows itself): 8 experts
// of 1200 x 1004, 4096 rows, forward 40 us, 246 TFLOP/s; one expert of 2048 x
// 2048, 4096 rows, 50 us, 690 TFLOP/s.
template <int OP, bool VEC, int TILE, typename OutT>
__global__ void __launch_bounds__(kThreads)
expert_bf16_kernel(ExpertArgs P) {
  constexpr bool CA = OP == OP_WEIGHT, CB = OP != OP_FORWARD;
  constexpr int OPB = TILE * kStage * 2, D = depth_of(TILE), F = TILE / 32;
  __shared__ __attribute__((aligned(1024))) char smem[4 * OPB];
  Work w;
  if (!find_work<OP, VEC>(P, TILE, TILE, 2, sizeof(OutT), &w)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = (wave >> 1) * (TILE / 2), wn = (wave & 1) * (TILE / 2);
  f32x4_t acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int stages = (w.sum + kStage - 1) / kStage;
  u32x4_t va[D][TILE / 32], vb[D][TILE / 32];
  auto load = [&](int st, int d) {
    if (st < stages) {
      load_stage<TILE, CA, VEC>(w.a, w.lda, w.rows, st * kStage, w.sum, va[d]);
      load_stage<TILE, CB, VEC>(w.b, w.ldb, w.cols, st * kStage, w.sum, vb[d]);
    }
  };
  auto write = [&](int st, int d) {
    if (st < stages) {
      write_stage<TILE, CA>(smem + (st & 1) * 2 * OPB, va[d]);
      write_stage<TILE, CB>(smem + (st & 1) * 2 * OPB + OPB, vb[d]);
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, d);
  write(0, 0);
  load(D, 0);
  for (int base = 0; base < stages; base += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int st = base + d;
      if (st >= stages) break;
      const char* cur = smem + (st & 1) * 2 * OPB;
      __syncthreads();   // stage st is written; everyone has read stage st - 1
      write(st + 1, (d + 1) % D);
      load(st + 1 + D, (d + 1) % D);
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        bf16x8_t fa[F], fb[F];
#pragma unroll
        for (int i = 0; i < F; ++i) fa[i] = read_frag<TILE, CA>(cur, wm + 16 * i, step);
#pragma unroll
        for (int j = 0; j < F; ++j) fb[j] = read_frag<TILE, CB>(cur + OPB, wn + 16 * j, step);
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int j = 0; j < F; ++j)
            // B first: the lane then holds row lane % 16 and four consecutive columns
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < F; ++i) {
    const int r = wm + 16 * i + (lane & 15);
    if (r < w.row0 || r >= w.rows) continue;
    OutT* row = reinterpret_cast<OutT*>(w.c + r * w.ldc);
#pragma unroll
    for (int j = 0; j < F; ++j) {
      const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      store4<OutT>(row, wn + 16 * j + 4 * (lane >> 4), w.cols, P.accumulate, v, w.col0);
    }
  }
}

// ---- bf16, 256 x 256 tiles ----------------------------------------------------

// Tiles and stages of an expert product for the 256-tile loop (bigtile.h).
template <int OP, typename OutT_>
struct ExpertBig {
  using OutT = OutT_;
  static constexpr bool kColsA = OP == OP_WEIGHT, kColsB = OP != OP_FORWARD;
  static constexpr bool kShort = OP != OP_WEIGHT;     // rows of weights seldom end inside a tile

  const BigGroups* G;
  uint32_t mt, nt;

  // The kernel's arguments, read again at each use instead of held in scalar
  // registers over the loop (ExpertArgs is the kernel's only parameter).
  static __device__ __forceinline__ const ExpertArgs& args() {
    auto* p = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const ExpertArgs*)p;
  }
  __device__ __forceinline__ uint32_t start(BigGroups* g) {
    const ExpertArgs& P = args();
    G = g;
    g->build(P.offsets, P.experts, P.tokens);
    if constexpr (OP == OP_WEIGHT) {
      mt = (uint32_t(P.n) + kBig - 1) / kBig;
      nt = (uint32_t(P.k) + kBig - 1) / kBig;
      return mt * nt * P.experts;
    } else {
      mt = uniform(g->tiles[P.experts]);
      nt = (uint32_t(OP == OP_FORWARD ? P.n : P.k) + kBig - 1) / kBig;
      return mt * nt;
    }
  }
  __device__ __forceinline__ void find(uint32_t pos, BigWork* w) const {
    const ExpertArgs& P = args();
    int tm, tn;
    if constexpr (OP == OP_WEIGHT) {
      const uint32_t e = pos / (mt * nt);
      tile_of_position(pos - e * mt * nt, mt, nt, &tm, &tn);
      const int lo = uniform(G->rows[e]), hi = uniform(G->rows[e + 1]);
      const int64_t i0 = int64_t(tm) * kBig, j0 = int64_t(tn) * kBig;
      w->sum = hi - lo;
      w->rows = int(P.n - i0 < kBig ? P.n - i0 : kBig);
      w->cols = int(P.k - j0 < kBig ? P.k - j0 : kBig);
      w->lda = int(P.ld_n * 2);
      w->ldb = int(P.ld_k * 2);
      w->ldc = int(P.ldw * int(sizeof(OutT)));
      w->a = static_cast<const char*>(P.a) + lo * (P.ld_n * 2) + i0 * 2;
      w->b = static_cast<const char*>(P.b) + lo * (P.ld_k * 2) + j0 * 2;
      w->c = static_cast<char*>(P.c) + e * P.w_stride * int(sizeof(OutT)) + i0 * w->ldc + j0 * int(sizeof(OutT));
    } else {
      const int64_t cols = OP == OP_FORWARD ? P.n : P.k;
      tile_of_position(pos, mt, nt, &tm, &tn);
      const int e = G->expert_of(P.experts, tm);
      const int row0 = uniform(G->rows[e]) + (tm - uniform(G->tiles[e])) * kBig;
      const int end = uniform(G->rows[e + 1]);
      const int64_t j0 = int64_t(tn) * kBig;
      w->rows = end - row0 < kBig ? end - row0 : kBig;
      w->cols = int(cols - j0 < kBig ? cols - j0 : kBig);
      w->sum = int(OP == OP_FORWARD ? P.k : P.n);
      w->lda = int((OP == OP_FORWARD ? P.ld_k : P.ld_n) * 2);
      w->ldb = int(P.ldw * 2);
      w->ldc = int((OP == OP_FORWARD ? P.ld_n : P.ld_k) * 2);
      w->a = static_cast<const char*>(P.a) + int64_t(row0) * w->lda;
      w->b = static_cast<const char*>(P.b) + e * P.w_stride * 2 + (OP == OP_FORWARD ? j0 * w->ldb : j0 * 2);
      w->c = static_cast<char*>(P.c) + int64_t(row0) * w->ldc + j0 * 2;
    }
  }
};

// 8192^3: 1.40 to 1.45 PFLOP/s in all three directions, the board at its power
// cap.  8 experts of 14336 x 4096, 8192 even rows: forward 903 us, input gradient
// 756 (long sums), weight gradient 875 (short sums); uneven ones (deviation 0.5 of
// the logarithm) 875, 857 and 887.  Runs differ by 5 % with the clock under the cap
// (the uneven forward took 823 in another).
template <int OP, typename OutT>
__global__ void __launch_bounds__(kBigThreads)
expert_bf16_big_kernel(ExpertArgs P) {
  __shared__ BigSlot slot0, slot1;
  __shared__ BigGroups groups;
  ExpertBig<OP, OutT> op;
  BigRun<ExpertBig<OP, OutT>> run(op, slot0.data, slot1.data, P.accumulate);
  run.run(&groups);
}

// ---- bf16, few rows per expert (forward) ---------------------------------------

struct ExpertSkinny {
  template <int MB, int NB>
  __device__ __forceinline__ void step(int, int, int, int, const SkinnyFrag (&b)[NB], const SkinnyFrag (&a)[MB],
                                       f32x4_t (&acc)[NB][MB]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int m = 0; m < MB; ++m)
          acc[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, b[n].h[h]),
                                                              __builtin_bit_cast(bf16x8_t, a[m].h[h]), acc[n][m], 0, 0, 0);
  }
};

// Row tiles of 16 MB rows by column tiles of 16 NB.
template <int MB, int NB, int W>
__global__ void __launch_bounds__(64 * W)
expert_skinny_kernel(ExpertArgs P) {
  __shared__ __attribute__((aligned(16))) float sums[W * MB * NB * 256];
  const uint32_t nt = (uint32_t(P.n) + 16 * NB - 1) / (16 * NB);
  const uint32_t tm = blockIdx.x / nt, tn = blockIdx.x - tm * nt;
  int row0;
  const GroupSpan g = group_of_tile(P.offsets, P.experts, P.tokens, 16 * MB, tm, &row0);
  if (row0 >= g.end) return;                // past the last tile
  const int64_t j0 = int64_t(tn) * (16 * NB);
  skinny_block<ExpertSkinny, MB, NB, W, uint16_t>(
      ExpertSkinny{}, static_cast<const char*>(P.a) + row0 * P.ld_k * 2, P.ld_k * 2,
      static_cast<const char*>(P.b) + (g.expert * P.w_stride + j0 * P.ldw) * 2, P.ldw * 2,
      static_cast<uint16_t*>(P.c) + row0 * P.ld_n + j0, P.ld_n, g.end - row0 < 16 * MB ? g.end - row0 : 16 * MB,
      int(P.n - j0 < 16 * NB ? P.n - j0 : 16 * NB), P.k * 2, false, sums);
}

int64_t skinny_blocks(const ExpertArgs& P, int mb, int nb) {
  const int64_t used = P.experts < P.tokens ? P.experts : P.tokens;
  return (P.tokens / (16 * mb) + used) * ((P.n + 16 * nb - 1) / (16 * nb));
}
template <int MB, int NB>
hipError_t launch_skinny(const ExpertArgs& P, hipStream_t stream) {
  const int64_t blocks = skinny_blocks(P, MB, NB);
  const dim3 grid(static_cast<unsigned>(blocks));
  if constexpr (skinny_sixteen(MB, NB, false)) {
    if (blocks < kSkinnyWide) {
      hipLaunchKernelGGL((expert_skinny_kernel<MB, NB, 16>), grid, dim3(1024), 0, stream, P);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((expert_skinny_kernel<MB, NB, 8>), grid, dim3(512), 0, stream, P);
  return hipGetLastError();
}

// ---- fp32 -------------------------------------------------------------------

constexpr int kStageF = 16;                               // summed indices per stage
constexpr int pitch_f(int tile) { return tile + 4; }      // words per LDS row (one s, TILE rows)

template <int TILE, bool COLS, bool VEC>
__device__ __forceinline__ void load_stage_f(const char* base, int64_t ld, int extent, int s0, int sum,
                                             u32x4_t (&v)[TILE / 64]) {
  const int t = threadIdx.x;
  constexpr int PER = TILE / 4;
#pragma unroll
  for (int q = 0; q < TILE / 64; ++q) {
    if constexpr (COLS) {
      const int s = s0 + t / PER + kThreads / PER * q, c = (t % PER) * 4;
      v[q] = load_chunk<4, VEC>(base + s * ld + c * 4, s < sum ? extent - c : 0);
    } else {
      const int r = (t >> 2) + 64 * q, c = (t & 3) * 4;
      v[q] = load_chunk<4, VEC>(base + r * ld + (s0 + c) * 4, r < extent ? sum - s0 - c : 0);
    }
  }
}
template <int TILE, bool COLS>
__device__ __forceinline__ void write_stage_f(float* lds, const u32x4_t (&v)[TILE / 64]) {
  const int t = threadIdx.x;
  constexpr int PER = TILE / 4;
#pragma unroll
  for (int q = 0; q < TILE / 64; ++q) {
    if constexpr (COLS) {
      *reinterpret_cast<u32x4_t*>(lds + (t / PER + kThreads / PER * q) * pitch_f(TILE) + (t % PER) * 4) = v[q];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        lds[((t & 3) * 4 + e) * pitch_f(TILE) + (t >> 2) + 64 * q] = __uint_as_float(v[q][e]);
    }
  }
}

// Bound by the fp32 matrix instructions for whole tiles and long sums (weight
// gradient of 4096 x 4096, 3000 rows: 906 us, 111 of the 154 TFLOP/s that a large
// library product reaches), by 0.4 us per stage where a CU has one tile.
template <int OP, bool VEC, int TILE>
__global__ void __launch_bounds__(kThreads)
expert_f32_kernel(ExpertArgs P) {
  constexpr bool CA = OP == OP_WEIGHT, CB = OP != OP_FORWARD;
  constexpr int OPW = kStageF * pitch_f(TILE), D = depth_of(TILE), F = TILE / 64;
  __shared__ __attribute__((aligned(16))) float smem[4 * OPW];
  Work w;
  if (!find_work<OP, VEC>(P, TILE, TILE, 4, 4, &w)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = (wave >> 1) * (TILE / 2), wn = (wave & 1) * (TILE / 2);
  f32x16_t acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  const int stages = (w.sum + kStageF - 1) / kStageF;
  u32x4_t va[D][TILE / 64], vb[D][TILE / 64];
  auto load = [&](int st, int d) {
    if (st < stages) {
      load_stage_f<TILE, CA, VEC>(w.a, w.lda, w.rows, st * kStageF, w.sum, va[d]);
      load_stage_f<TILE, CB, VEC>(w.b, w.ldb, w.cols, st * kStageF, w.sum, vb[d]);
    }
  };
  auto write = [&](int st, int d) {
    if (st < stages) {
      write_stage_f<TILE, CA>(smem + (st & 1) * 2 * OPW, va[d]);
      write_stage_f<TILE, CB>(smem + (st & 1) * 2 * OPW + OPW, vb[d]);
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, d);
  write(0, 0);
  load(D, 0);
  for (int base = 0; base < stages; base += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int st = base + d;
      if (st >= stages) break;
      const float* cur = smem + (st & 1) * 2 * OPW;
      __syncthreads();
      write(st + 1, (d + 1) % D);
      load(st + 1 + D, (d + 1) % D);
#pragma unroll
      for (int s = 0; s < kStageF; s += 2) {
        float fa[F], fb[F];
#pragma unroll
        for (int i = 0; i < F; ++i) {
          fa[i] = cur[(s + (lane >> 5)) * pitch_f(TILE) + wm + 32 * i + (lane & 31)];
          fb[i] = cur[OPW + (s + (lane >> 5)) * pitch_f(TILE) + wn + 32 * i + (lane & 31)];
        }
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int j = 0; j < F; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fb[j], fa[i], acc[i][j], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < F; ++i) {
    const int r = wm + 32 * i + (lane & 31);
    if (r < w.row0 || r >= w.rows) continue;
    float* row = reinterpret_cast<float*>(w.c + r * w.ldc);
#pragma unroll
    for (int j = 0; j < F; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float v[4] = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
        store4<float>(row, wn + 32 * j + 8 * g + 4 * (lane >> 5), w.cols, P.accumulate, v, w.col0);
      }
  }
}

template <int OP, int TILE>
hipError_t launch_tiles(const ExpertArgs& P, int64_t tiles, int dtype, int out_dtype, bool vec, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(grouped_grid(tiles))), block(kThreads);
  if (dtype == DT_F32) {
    if (vec) hipLaunchKernelGGL((expert_f32_kernel<OP, true, TILE>), grid, block, 0, stream, P);
    else hipLaunchKernelGGL((expert_f32_kernel<OP, false, TILE>), grid, block, 0, stream, P);
    return hipGetLastError();
  }
  if constexpr (OP == OP_WEIGHT) {
    if (out_dtype == DT_F32) {
      if (vec) hipLaunchKernelGGL((expert_bf16_kernel<OP, true, TILE, float>), grid, block, 0, stream, P);
      else hipLaunchKernelGGL((expert_bf16_kernel<OP, false, TILE, float>), grid, block, 0, stream, P);
      return hipGetLastError();
    }
  }
  if (vec) hipLaunchKernelGGL((expert_bf16_kernel<OP, true, TILE, uint16_t>), grid, block, 0, stream, P);
  else hipLaunchKernelGGL((expert_bf16_kernel<OP, false, TILE, uint16_t>), grid, block, 0, stream, P);
  return hipGetLastError();
}

constexpr int64_t kMaxSmallTiles = int64_t(1) << 23;    // fewer than 2^32 threads

// Tiles of edge t that any offsets could need.
template <int OP>
int64_t tile_bound(const ExpertArgs& P, int64_t t) {
  if (OP == OP_WEIGHT) return int64_t(P.experts) * ((P.n + t - 1) / t) * ((P.k + t - 1) / t);
  const int64_t used = P.experts < P.tokens ? P.experts : P.tokens;   // experts with a partial tile
  return (P.tokens / t + used) * (((OP == OP_FORWARD ? P.n : P.k) + t - 1) / t);
}

template <int OP>
hipError_t launch_op(const ExpertArgs& P, int dtype, int out_dtype, bool vec, hipStream_t stream) {
  // 256-tiles from half a tile per CU on: 8 experts of 2048 x 2048, 2048 rows,
  // take 35 us so and 38 in 128-tiles, their weight gradient 30 and 46.  Experts
  // with few rows come here too, down to one: both kernels then only read the
  // weights, and neither is ahead everywhere (forward, one row per expert,
  // weights from HBM, these tiles and the few-rows kernel: 8 experts of 14336 x 4096
  // 165 and 177 us, 8 of 8192 x 8192 182 and 210, 32 of 4096 x 512 28 and 35, but 16
  // of 4096 x 4096 125 and 105, 64 of 2048 x 2048 134 and 93); with eight rows and
  // more the tiles stay as they are and the other grows by 3 to 20 %.
  const int64_t big = tile_bound<OP>(P, kBig);
  if (dtype == DT_BF16 && vec && big >= 128 && P.experts <= kBigExperts) {
    const dim3 grid(static_cast<unsigned>(big < kBigBlocks ? big : kBigBlocks)), block(kBigThreads);
    if constexpr (OP == OP_WEIGHT) {
      if (out_dtype == DT_F32) {
        hipLaunchKernelGGL((expert_bf16_big_kernel<OP, float>), grid, block, 0, stream, P);
        return hipGetLastError();
      }
    }
    hipLaunchKernelGGL((expert_bf16_big_kernel<OP, uint16_t>), grid, block, 0, stream, P);
    return hipGetLastError();
  }
  if constexpr (OP == OP_FORWARD) {
    // too few tiles to fill the GPU and at most 16, or 32, rows per expert on
    // average: one 4096 x 4096 expert takes 54 us for 4 rows in 128-tiles,
    // 10 us here (weights from HBM)
    if (dtype == DT_BF16 && vec && skinny_blocks(P, 1, 1) <= kMaxSkinnyBlocks) {
      if (P.tokens <= 16 * int64_t(P.experts)) {
        if (skinny_blocks(P, 1, 2) >= kSkinnyWide) return launch_skinny<1, 2>(P, stream);
        return launch_skinny<1, 1>(P, stream);
      }
      if (P.tokens <= 32 * int64_t(P.experts)) return launch_skinny<2, 2>(P, stream);
    }
  }
  // 64-tiles where 128-tiles would leave CUs idle: fewer than one per CU, or,
  // for the weight gradient, whose tiles are as long as their experts' rows,
  // fewer than 64 per expert.  With 256 tiles (weight gradient of one expert
  // 2048 x 2048, 4096 rows) 128-tiles take 63 us, 64-tiles 78;  fp32 forward of 294 rows over 64 experts of
  // 16 x 640: 54 us in 128-tiles, 20 in 64-tiles; fp32 weight gradient of 3001
  // uneven rows over 24 experts of 1000 x 515: 196 and 96 us before
  // whole_chunks and store4's vectors, 72 with them.
  const int64_t tiles = tile_bound<OP>(P, kTile), small = tile_bound<OP>(P, kSmallTile);
  const bool few = tiles < 256 || (OP == OP_WEIGHT && tiles < 64 * int64_t(P.experts));
  if (few && small <= kMaxSmallTiles) return launch_tiles<OP, kSmallTile>(P, small, dtype, out_dtype, vec, stream);
  return launch_tiles<OP, kTile>(P, tiles, dtype, out_dtype, vec, stream);
}

}  // namespace

hipError_t launch_expert_product(int op, const ExpertArgs& P, int dtype, int out_dtype, bool vec, hipStream_t stream) {
  switch (op) {
    case OP_FORWARD: return launch_op<OP_FORWARD>(P, dtype, out_dtype, vec, stream);
    case OP_INPUT: return launch_op<OP_INPUT>(P, dtype, out_dtype, vec, stream);
    default: return launch_op<OP_WEIGHT>(P, dtype, out_dtype, vec, stream);
  }
}

}  // namespace dmuon

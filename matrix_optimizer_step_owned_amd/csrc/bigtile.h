// The 256 x 256 tile loop of the expert products in bf16 and of the products of
// 8-bit integers, whose stages have the same bytes: 128 k in place of 64, and
// v_mfma_i32_16x16x64_i8 in place of v_mfma_f32_16x16x32_bf16, which takes as long.
// Sums count in units of two bytes.
//
// C[i][j] = sum_s A(i, s) B(j, s), one block of four waves per CU.  A wave
// computes 128 x 128 of the tile (16 x 16 blocks, of the rows every second
// one), 256 accumulation registers; 256 x 256 is the smallest tile
// whose operands the load path delivers as fast as the matrix cores use them
// (64 KB per 2048 cycles of matrix instructions).  Operands stream through a
// two-slot LDS ring (128 KB) by direct-to-LDS loads of 64 s per stage.
//
// A stage is four quarters of 32 matrix instructions (two steps of 32 s, two
// halves of the row blocks).  The fragments of both steps have registers of
// their own: step 1's are read under quarter 0, the next stage's step 0 under
// quarter 3.  A barrier after quarter 0 frees the stage's slot for the stage
// after next, whose 16 loads per wave go out over the next four quarters (6, 6,
// 2, 2); a barrier after quarter 2 makes the next stage visible.  So a load
// has about one and a half stages to land, which covers an L2 miss: with one
// barrier and one stage of room the same tile ran at 0.8 of this rate.
//
// Blocks are persistent and the stream of stages runs on from a block's tile
// to its next one, so neither the first loads of a tile nor the stores of the
// one before are waited for.  A short tile (at most 128 or 64 rows: the last
// rows of an expert) computes fewer row blocks.
#pragma once

#include <type_traits>

#include "grouped.h"

namespace dmuon {

constexpr int kBig = 256;
constexpr int kBigThreads = 256;
constexpr int kBigOp = kBig * 128;        // bytes of one operand in a stage
constexpr int kBigBlocks = 256;           // one per CU
constexpr int kBigExperts = 1024;         // most experts whose rows fit the LDS table

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// LDS offset of 16-byte chunk c of row r, rows of 128 bytes: sixteen rows'
// chunks cover all 64 banks.
__device__ __forceinline__ int row_slot(int r, int c) { return r * 128 + ((c ^ ((r >> 1) & 7)) << 4); }
// LDS offset of the 32-byte unit u (16 columns of 2 bytes) of row s, rows of
// 256 columns: the eight rows that half a wave's transpose read touches (s & 3
// and bit 3) go to eight different units.
__device__ __forceinline__ int big_col_slot(int s, int u) { return s * 512 + ((u ^ ((s & 3) | ((s >> 1) & 4))) << 5); }

// The same value, as one that the compiler cannot compute anything from ahead
// of this point: addresses derived from it are formed again where they are
// used instead of being kept in registers over the whole loop.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

__device__ __forceinline__ int here_scalar(int v) {
  asm volatile("" : "+s"(v));
  return v;
}

// Every expert's first row and first row tile (entry `experts`: the ends).
struct BigGroups {
  int rows[kBigExperts + 1], tiles[kBigExperts + 1];

  __device__ __forceinline__ void build(const int32_t* offsets, int experts, int tokens) {
    if (threadIdx.x < 64) {
      const int lane = threadIdx.x;
      int row = first_row(offsets, tokens), n = 0;
      for (int base = 0; base < experts; base += 64) {
        const GroupChunk c = group_chunk(offsets, experts, tokens, kBig, base, row, n);
        if (base + lane < experts) {
          rows[base + lane] = c.lo;
          tiles[base + lane] = c.before;
        }
        row = __builtin_amdgcn_readlane(c.hi, 63);
        n = __builtin_amdgcn_readlane(c.upto, 63);
      }
      if (lane == 0) {
        rows[experts] = row;
        tiles[experts] = n;
      }
    }
    __syncthreads();
  }
  // The expert of a row tile: the last one whose first tile is at most `tile`
  // (experts without rows have the next one's first tile).
  __device__ __forceinline__ int expert_of(int experts, int tile) const {
    int lo = 0, hi = experts - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (uniform(tiles[mid]) <= tile) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
};

// Which tiles a block takes.  Whole rounds of the grid first, every block one
// tile; what is left behind them is split by rows where that gives more blocks
// something to do.  A half or a quarter of the rows needs all of B's loads and
// so takes about 0.75 or 0.6 of a tile's time (block-scaled, 16 uneven experts
// of 4096 x 2048, 8192 rows: 123 to 109 us together with store_pair).
struct BigPlan {
  uint32_t full, left, end;    // positions of whole rounds; parts behind them; past the last position
  int split;                   // a part has 256 >> split rows

  __device__ __forceinline__ void make(uint32_t tiles, bool may_split) {
    const uint32_t grid = gridDim.x;
    full = tiles / grid * grid;
    left = tiles - full;
    split = !may_split ? 0 : 4 * left <= grid ? 2 : 2 * left <= grid ? 1 : 0;
    left <<= split;
    end = left ? full + grid : full;
  }
  // False where the position has nothing.
  __device__ __forceinline__ bool locate(uint32_t p, uint32_t* tile, int* part) const {
    *tile = p;
    *part = -1;               // all of the tile
    if (p < full) return true;
    uint32_t i = p - full;
    if (gridDim.x == kBigBlocks) {    // dealt to the XCDs in turn, four at a time
      const uint32_t per = kBigBlocks / kNumXcd, x = i / per, k = i % per;
      i = ((k >> 2) * kNumXcd + x) * 4 + (k & 3);
    }
    *tile = full + (i >> split);
    *part = int(i & ((1u << split) - 1));
    return i < left;
  }
  // First row of a part, and its rows out of the tile's.
  __device__ __forceinline__ int cut(int part, int* rows) const {
    if (part < 0) return 0;
    const int most = kBig >> split, skip = part * most;
    *rows = *rows - skip < most ? *rows - skip : most;
    return skip;
  }
};

// One tile: rows / cols of C that exist from its corner on, the length of
// the sum in elements, addresses of the corner (bytes, row strides in bytes).
struct BigWork {
  const char* a;
  const char* b;
  char* c;
  int lda, ldb, ldc;
  int rows, cols, sum;
};

// Moves a tile's description to scalar registers (the divisions that found it
// run on the vector unit).
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  return int64_t((uint64_t(uint32_t(uniform(int(uint64_t(v) >> 32)))) << 32) | uint32_t(uniform(int(uint32_t(v)))));
}
template <class T>
__device__ __forceinline__ T* uniform_ptr(T* p) {   // of global memory
  typedef __attribute__((address_space(1))) T* G;
  return (T*)reinterpret_cast<G>(uniform64(reinterpret_cast<int64_t>(p)));
}
__device__ __forceinline__ void to_scalar(BigWork* w) {
  w->a = uniform_ptr(w->a);
  w->b = uniform_ptr(w->b);
  w->c = uniform_ptr(w->c);
  w->lda = uniform(w->lda);
  w->ldb = uniform(w->ldb);
  w->ldc = uniform(w->ldc);
  w->rows = uniform(w->rows);
  w->cols = uniform(w->cols);
  w->sum = uniform(w->sum);
}

// The ring's two slots are variables of their own, and every access names its
// slot statically: the compiler then knows that a fragment read does not
// touch what the loads in flight write (else it waits for them before every
// transpose read).
struct BigSlot {
  __attribute__((aligned(1024))) char data[2 * kBigOp];
};

constexpr int kBigStage = 64;             // s per stage
constexpr int64_t kMaxBigPitch = int64_t(1) << 23;   // bytes: offsets of a tile's rows within 31 bits

// The stream of one operand's loads: sixteen-byte pieces of a stage, eight
// per lane, an eighth of the operand's rows apart, at fixed offsets (the row
// stride is the same for every tile) from a base that moves with the stage.
// The descriptor is scalar; its range cuts off what lies past the tile's last
// row or the sum's end.  Columns past the tile's are read where they lie
// inside the operand: they only reach results that are not stored.
template <bool COLS>
struct BigLoads {
  __amdgpu_buffer_rsrc_t rsrc;
  const char* p;
  uint32_t step;
  uint32_t at[8];
  uint32_t outside;       // !COLS: the lane's chunk lies past the sum's end
  int first_s;            // !COLS: the lane's first s within a stage
  int left, ld, extent;

  __device__ __forceinline__ void init(int ld_, int wave, int lane) {
    ld = ld_;
    step = COLS ? uint32_t(kBigStage) * uint32_t(ld) : 128u;
    first_s = ((lane & 7) ^ (((wave * 8 + (lane >> 3)) >> 1) & 7)) * 8;   // the same for every piece
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if constexpr (COLS) {
        const int s = (wave + 4 * q) * 2 + (lane >> 5);
        const int unit = ((lane & 31) >> 1) ^ ((s & 3) | ((s >> 1) & 4));
        at[q] = uint32_t(s) * uint32_t(ld) + (unit * 16 + (lane & 1) * 8) * 2;
      } else {
        at[q] = uint32_t((wave + 4 * q) * 8 + (lane >> 3)) * uint32_t(ld) + first_s * 2;
      }
    }
  }
  __device__ __forceinline__ void aim() {
    // a stage past the sum (left <= 0) reads nothing
    const int in = left < 0 ? 0 : left < kBigStage ? left : kBigStage;
    uint32_t range;
    if constexpr (COLS) {
      range = in == 0 ? 0u : uint32_t(in - 1) * uint32_t(ld) + uint32_t(extent) * 2;
    } else {
      range = in == 0 ? 0u : uint32_t(extent - 1) * uint32_t(ld) + uint32_t(in) * 2;
      outside = first_s < left ? 0u : kOutside;
    }
    rsrc = slab_rsrc(p, range);
  }
  __device__ __forceinline__ void start(const char* base, int extent_, int sum) {
    p = base;
    extent = extent_;
    left = sum;
    aim();
  }
  __device__ __forceinline__ void next() {
    p += step;
    left -= kBigStage;
    aim();
  }
  __device__ __forceinline__ void load(int q, char* lds, int wave) const {
    slab_load_lds(rsrc, lds + (wave + 4 * q) * 1024, COLS ? at[q] : at[q] | outside);
  }
};

// Workgroup barrier without a memory fence (a fence would wait for every
// direct-to-LDS load in flight); the waits that a barrier needs stand before
// it, in the gfx9 encoding.
__device__ __forceinline__ void plain_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }   // lgkmcnt(0)
template <int N>
__device__ __forceinline__ void wait_loads() {                                       // vmcnt(N)
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// The matrix instructions are asm statements with the accumulator as a tied
// operand in accumulation registers, so that each accumulator stays in place
// (with the builtin the register allocator moves them about and spills).
// The compiler does not see their latency: accumulators are only read behind
// settle(), and written (clear()) well before a matrix instruction.
__device__ __forceinline__ void big_mfma(f32x4_t& acc, const bf16x8_t& b, const bf16x8_t& a) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}
typedef int i32x4_t __attribute__((ext_vector_type(4)));
// Sixteen 8-bit integers per lane and operand, int32 sums.
__device__ __forceinline__ void big_mfma(i32x4_t& acc, const bf16x8_t& b, const bf16x8_t& a) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}
#define DMUON_ACC8(i) \
  "+a"(acc[i][0]), "+a"(acc[i][1]), "+a"(acc[i][2]), "+a"(acc[i][3]), "+a"(acc[i][4]), "+a"(acc[i][5]), \
      "+a"(acc[i][6]), "+a"(acc[i][7])
template <int NI, typename Acc>
__device__ __forceinline__ void settle(Acc (&acc)[NI][8]) {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" : DMUON_ACC8(0));
#pragma unroll
  for (int i = 1; i < NI; ++i) asm volatile("" : DMUON_ACC8(i));
  __builtin_amdgcn_sched_barrier(0);
}
template <int NI, typename Acc>
__device__ __forceinline__ void clear(Acc (&acc)[NI][8]) {
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = Acc{0, 0, 0, 0};
  // opaque from here on, so that no zero is formed again next to its use
#pragma unroll
  for (int i = 0; i < NI; ++i) asm volatile("s_nop 0" : DMUON_ACC8(i));
  asm volatile("s_nop 3" : DMUON_ACC8(0));
  __builtin_amdgcn_sched_barrier(0);
}
#undef DMUON_ACC8

// Writes one tile: the lane holds row lane % 16 and columns 4 (lane / 16) .. of
// every block.  bf16 results trade words with the neighbouring sixteen lanes
// first, so that a lane writes 16 bytes and a row's four lanes 64: with 8 bytes
// each the L2's requests for 32 bytes bound the stores.
template <typename OutT, int NI>
__device__ __forceinline__ void store_tile(const BigWork& w, const f32x4_t (&acc)[NI][8], bool accumulate,
                                           int wave, int lane) {
  const int wm = wave >> 1, wn = wave & 1, g = lane >> 4;
  const bool plain = !accumulate && w.cols == kBig;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = 32 * i + 16 * wm + (lane & 15);
    OutT* row = reinterpret_cast<OutT*>(w.c + int64_t(r) * w.ldc) + 128 * wn;
    if (plain) {
      if constexpr (sizeof(OutT) == 4) {
        if (r < w.rows) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
            store4<OutT>(row, 16 * j + 4 * g, 128, false, v);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; j += 2)
          store_pair(row + 16 * j, acc[i][j], acc[i][j + 1], g, r < w.rows);
      }
    } else if (r < w.rows) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        store4<OutT>(row, 16 * j + 4 * g, w.cols - 128 * wn, accumulate, v);
      }
    }
    __builtin_amdgcn_sched_barrier(0);   // one row of blocks at a time
  }
}

// Zeros over one tile.
template <typename OutT>
__device__ __forceinline__ void store_zeros(const BigWork& w, int wave, int lane) {
  for (int r = wave; r < w.rows; r += kBigThreads / 64)
    for (int c = lane; c < w.cols; c += 64) reinterpret_cast<OutT*>(w.c + int64_t(r) * w.ldc)[c] = 0;
}

// What most operators share: fp32 accumulators that are stored as they are.
template <typename OutT_>
struct BigPlain {
  using OutT = OutT_;
  using Acc = f32x4_t;
  using Work = BigWork;
  static __device__ __forceinline__ void skip(BigWork*, int) {}
  static __device__ __forceinline__ void to_scalar(BigWork*) {}
  template <int NI>
  static __device__ __forceinline__ void store(const BigWork& w, const f32x4_t (&acc)[NI][8], bool accumulate, int wave,
                                               int lane) {
    store_tile<OutT>(w, acc, accumulate, wave, lane);
  }
};

// The tiles of one block.  Op: kColsA / kColsB (operand kinds), kShort (short
// tiles happen), OutT, Acc (accumulators), Work (BigWork and what the operator
// adds), start(groups) -> number of tiles, find(position, work), skip(work, rows)
// and to_scalar(work) for what it adds, store(work, accumulators, ...).
template <class Op>
struct BigRun {
  using OutT = typename Op::OutT;
  using Acc = typename Op::Acc;
  using Work = typename Op::Work;
  static constexpr bool kA = Op::kColsA, kB = Op::kColsB;

  Op& op;
  char* const slot0;
  char* const slot1;
  const bool accumulate;
  const int lane0, wave;
  uint32_t pos;
  BigPlan plan;
  Work w, nw;                    // present tile, next one (sum 0: none)
  BigLoads<kA> la;               // the stage whose loads are being issued
  BigLoads<kB> lb;
  int loads_left;                // stages of its tile after it
  bf16x8_t fa[2][8], fb[2][8];   // fragments of steps 0 and 1

  __device__ __forceinline__ BigRun(Op& o, char* s0, char* s1, bool acc_)
      : op(o), slot0(s0), slot1(s1), accumulate(acc_), lane0(threadIdx.x & 63),
        wave(uniform(threadIdx.x >> 6)) {}

  // Every tile has an even number of stages; a stage past the sum reads zeros.
  static __device__ __forceinline__ int stages_of(int sum) { return (sum + 2 * kBigStage - 1) / (2 * kBigStage) * 2; }

  // Tile or part of one at position p.
  __device__ __forceinline__ void find(uint32_t p, Work* t) const {
    uint32_t tile;
    int part;
    if (!plan.locate(p, &tile, &part)) {
      t->sum = 0;
      t->rows = 0;
      return;
    }
    op.find(tile, t);
    if constexpr (Op::kShort) {
      const int skip = plan.cut(part, &t->rows);
      t->a += int64_t(skip) * t->lda;
      t->c += int64_t(skip) * t->ldc;
      Op::skip(t, skip);
      if (t->rows <= 0) t->sum = t->rows = 0;
    }
  }
  // The block's first tile from position p on that has anything to sum.
  // Tiles without are written here: zeros, or nothing when accumulating.
  __device__ __forceinline__ void find_from(uint32_t p, Work* t) {
    t->sum = 0;
    t->rows = t->cols = 1;       // of no tile: loads that read nothing
    for (; p < plan.end; p += gridDim.x) {
      find(p, t);
      to_scalar(t);
      Op::to_scalar(t);
      if (t->sum > 0) break;
      if (!accumulate) store_zeros<OutT>(*t, wave, here(lane0));
      t->sum = 0;
      t->rows = t->cols = 1;
    }
    pos = p;
  }
  __device__ __forceinline__ void load_tile(const BigWork& t) {
    la.start(t.a, t.rows, t.sum);
    lb.start(t.b, t.cols, t.sum);
    loads_left = stages_of(t.sum) - 1;
  }
  // On to the next stage's loads: of the present tile, then of the next one.
  // Past the last tile they read nothing (a sum of 0), into slots that nobody
  // reads: so the counts of loads in flight are the same everywhere.
  __device__ __forceinline__ void load_next() {
    if (loads_left > 0) {
      --loads_left;
      la.next();
      lb.next();
    } else {
      load_tile(nw);
    }
  }
  // Load n of the sixteen of a stage: A's and B's pieces in turn.
  template <int SLOT>
  __device__ __forceinline__ void load(int n, int wv) const {
    char* at = SLOT ? slot1 : slot0;
    if (n & 1) lb.load(n >> 1, at + kBigOp, wv);
    else la.load(n >> 1, at, wv);
  }
  // Eight s of 16-row block b of an operand: s = 32 step + 8 (lane / 16) ..
  template <bool COLS>
  static __device__ __forceinline__ bf16x8_t frag(const char* slot, int operand, int b, int step, int lane) {
    if constexpr (COLS) {
      typedef short s16x4_t __attribute__((ext_vector_type(4)));
      const int s = 8 * (lane >> 4) + ((lane & 15) >> 2);
      const int at = operand + big_col_slot(s, b & 7) + (lane & 3) * 8 + (b >> 3) * 256 + step * 32 * 512;
      union { s16x4_t h[2]; bf16x8_t v; } u;
      // one index from the slot's own variable: a longer chain of offsets
      // loses what the compiler knows about it
      u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DMUON_LDS s16x4_t*)(slot + at));
      u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DMUON_LDS s16x4_t*)(slot + (at + 4 * 512)));
      return u.v;
    } else {
      return *reinterpret_cast<const bf16x8_t*>(slot + (operand + b * 2048 + row_slot(lane & 15, 4 * step + (lane >> 4))));
    }
  }
  // Fragment r of a step: B's eight, then A's NI.
  template <int SET, int SLOT>
  __device__ __forceinline__ void read(int r, int lane) {
    const char* slot = SLOT ? slot1 : slot0;
    if (r < 8) fb[SET][r] = frag<kB>(slot, kBigOp, 8 * (wave & 1) + r, SET, lane);
    else fa[SET][r - 8] = frag<kA>(slot, 0, 2 * (r - 8) + (wave >> 1), SET, lane);
  }
  // One quarter in a fixed order: the matrix instructions of half HALF of step
  // SET; fragments of set RSET (none if < 0) from RSLOT spread over the first
  // 1/RPART of them; loads L0 .. L1 - 1 of the running stage into LSLOT spread
  // over all of them.
  template <int NI, int SET, int HALF, int RSET, int RSLOT, int RPART, int LSLOT, int L0, int L1>
  __device__ __forceinline__ void quarter(Acc (&acc)[NI][8], int lane, int wv) {
    constexpr int NM = NI / 2 * 8, NR = RSET < 0 ? 0 : 8 + NI, LIM = NM / RPART, NL = L1 - L0;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      big_mfma(acc[HALF * (NI / 2) + m / 8][m % 8], fb[SET][m % 8], fa[SET][HALF * (NI / 2) + m / 8]);
      if constexpr (NR > 0) {
        if (m < LIM) {
#pragma unroll
          for (int r = m * NR / LIM; r < (m + 1) * NR / LIM; ++r) read<RSET < 0 ? 0 : RSET, RSLOT>(r, lane);
        }
      }
      if constexpr (NL > 0) {
#pragma unroll
        for (int l = m * NL / NM; l < (m + 1) * NL / NM; ++l) load<LSLOT>(L0 + l, wv);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // One stage in SLOT; its step 0 is in registers.
  template <int NI, int SLOT>
  __device__ __forceinline__ void stage(Acc (&acc)[NI][8]) {
    const int lane = here(lane0), wv = here_scalar(wave);
    quarter<NI, 0, 0, 1, SLOT, 2, SLOT ^ 1, 14, 16>(acc, lane, wv);
    wait_lds();
    plain_barrier();              // SLOT is read
    load_next();
    quarter<NI, 0, 1, -1, 0, 1, SLOT, 0, 6>(acc, lane, wv);
    quarter<NI, 1, 0, -1, 0, 1, SLOT, 6, 12>(acc, lane, wv);
    wait_loads<12>();
    plain_barrier();              // the next stage has landed
    // (behind the tile's last stage these are the next tile's, read again there:
    // a branch around them would make the compiler copy accumulators)
    quarter<NI, 1, 1, 0, SLOT ^ 1, 1, SLOT, 12, 14>(acc, lane, wv);
  }
  // The present tile, its first stage in slot 0 and visible.
  template <int NI>
  __device__ __forceinline__ void tile() {
    Acc acc[NI][8];
    clear(acc);
    const int stages = stages_of(w.sum);
    const int lane = here(lane0);
#pragma unroll
    for (int r = 0; r < 8 + NI; ++r) read<0, 0>(r, lane);
    __builtin_amdgcn_sched_barrier(0);
    for (int st = 0; st < stages; st += 2) {
      stage<NI, 0>(acc);
      stage<NI, 1>(acc);
    }
    settle(acc);
    op.template store<NI>(w, acc, accumulate, wave, here(lane0));
  }
  __device__ __forceinline__ void run(BigGroups* groups) {
    plan.make(op.start(groups), Op::kShort);
    // a full round of blocks covers gridDim consecutive positions, each XCD a
    // run of them (blocks go to the XCDs in turn)
    const uint32_t grid = gridDim.x, per = grid / kNumXcd;
    find_from(grid % kNumXcd ? blockIdx.x : (blockIdx.x % kNumXcd) * per + blockIdx.x / kNumXcd, &w);
    if (w.sum <= 0) return;
    nw = w;
    la.init(w.lda, wave, lane0);
    lb.init(w.ldb, wave, lane0);
    load_tile(w);
#pragma unroll
    for (int n = 0; n < 16; ++n) load<0>(n, wave);
    load_next();
#pragma unroll
    for (int n = 0; n < 14; ++n) load<1>(n, wave);
    wait_loads<14>();
    plain_barrier();
    while (true) {
      find_from(pos + grid, &nw);
      if (!Op::kShort || w.rows > 128) tile<8>();
      else if (w.rows > 64) tile<4>();
      else tile<2>();
      if (nw.sum <= 0) break;
      w = nw;
    }
    wait_loads<0>();      // nothing may land in LDS that is no longer ours
  }
};

}  // namespace dmuon

// A whole layer of experts for a few tokens (serving), two kernels:
//   h[t, e] = g[t, e] * silu(G[e] x[t]) * (U[e] x[t])          layer_in
//   y[t]    = sum over the token's experts e of  D[e] h[t, e]  layer_out
// with G and U the two halves of the rows of w_in[e] (2n x k), D = w_out[e] (k x n)
// and g the token's gate of that expert.  Weights are bf16, or 8-bit integers
// with a scale per output channel, which become bf16 in registers (exactly).
// Sums are fp32 over v_mfma_f32_16x16x32_bf16.  h is an operand of the second
// product as the sum of two bf16 values, its rounding and the rounding of what
// that left (2^-17 of it is lost): one alone would add as much error as the
// rounding of y (2.4e-3 in place of 1.7e-3 of y's norm), and the second costs
// matrix instructions that the weights' loads hide.  y is rounded once.
//
// Every touched expert's weights are read once and bound everything.  So, as in
// skinny.h, nothing is staged: lanes load their fragments straight into
// registers, 32 of the 128 bytes that a row has in one step, waves split the
// sum and add up in LDS in wave order.  Which experts are touched is device
// data: layer_in has blocks for as many experts as there can be and each finds
// its own from the ids.  In layer_out a block keeps its 16 output columns for
// all tokens and runs over the touched experts, so that no sum crosses blocks: a
// token that did not pick the expert has zeros in place of h.
#include "skinny.h"

namespace dmuon {
namespace {

constexpr int kLayerWaves = 8;
constexpr int kLayerThreads = kLayerWaves * 64;

// Sixteen bytes of a row at p, of which `left` bytes are inside; elements of EB bytes.
template <int EB, bool VEC>
__device__ __forceinline__ u32x4_t chunk_of(const char* p, int64_t left) {
  return load_chunk<EB, VEC>(p, left < 0 ? 0 : left > 16 ? 16 / EB : int(left) / EB);
}

__device__ __forceinline__ f32x4_t multiply(const bf16x8_t& b, const bf16x8_t& a, const f32x4_t& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
}

// Eight 8-bit integers as bf16, which holds them exactly: a byte plus 128 is
// converted without its sign.
__device__ __forceinline__ bf16x8_t widen(uint32_t lo, uint32_t hi) {
  u32x4_t v;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t u = (h ? hi : lo) ^ 0x80808080u;
    uint32_t f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __float_as_uint(float((u >> (8 * e)) & 0xffu) - 128.f);
    v[2 * h] = __builtin_amdgcn_perm(f[1], f[0], 0x07060302u);
    v[2 * h + 1] = __builtin_amdgcn_perm(f[3], f[2], 0x07060302u);
  }
  return __builtin_bit_cast(bf16x8_t, v);
}

// One step (128 bytes of a weight row) of the weights and of the rows that they
// multiply: a bf16 row has 128 bytes of it, or 256 with 8-bit weights.
struct WeightStep {
  u32x4_t h[2];
};
template <bool I8>
struct RowStep {
  u32x4_t h[I8 ? 4 : 2];
};
template <bool I8, bool VEC>
__device__ __forceinline__ WeightStep load_weight(const char* row, int64_t at, int64_t bytes, int g) {
  WeightStep w;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t o = at + 64 * h + 16 * g;
    w.h[h] = chunk_of<I8 ? 1 : 2, VEC>(row + o, bytes - o);
  }
  return w;
}
// `at`, `bytes`: of the weight row.
template <bool I8, bool VEC>
__device__ __forceinline__ RowStep<I8> load_row(const char* row, int64_t at, int64_t bytes, int g) {
  RowStep<I8> x;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t o = at + 64 * h + 16 * g;
    if constexpr (I8) {
      x.h[2 * h] = chunk_of<2, VEC>(row + 2 * o, 2 * (bytes - o));
      x.h[2 * h + 1] = chunk_of<2, VEC>(row + 2 * o + 16, 2 * (bytes - o) - 16);
    } else {
      x.h[h] = chunk_of<2, VEC>(row + o, bytes - o);
    }
  }
  return x;
}
// acc[m] += one step's products with MB blocks of rows; the weights are widened once.
template <bool I8, int MB>
__device__ __forceinline__ void add_step(const WeightStep& w, const RowStep<I8> (&x)[MB], f32x4_t (&acc)[MB]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (I8) {
      const bf16x8_t a = widen(w.h[h][0], w.h[h][1]), b = widen(w.h[h][2], w.h[h][3]);
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        acc[m] = multiply(a, __builtin_bit_cast(bf16x8_t, x[m].h[2 * h]), acc[m]);
        acc[m] = multiply(b, __builtin_bit_cast(bf16x8_t, x[m].h[2 * h + 1]), acc[m]);
      }
    } else {
#pragma unroll
      for (int m = 0; m < MB; ++m)
        acc[m] = multiply(__builtin_bit_cast(bf16x8_t, w.h[h]), __builtin_bit_cast(bf16x8_t, x[m].h[h]), acc[m]);
    }
  }
}

// Set of the touched experts: one bit each.  Ids outside 0 .. experts - 1 are
// nobody's.  All threads of the block call it; a barrier behind it is the caller's.
struct Touched {
  uint32_t bits[kLayerExperts / 32];
  __device__ __forceinline__ void build(const LayerArgs& P) {
    for (int i = threadIdx.x; i < kLayerExperts / 32; i += kLayerThreads) bits[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < P.tokens * P.top_k; i += kLayerThreads) {
      const uint32_t id = uint32_t(P.ids[i]);
      if (id < uint32_t(P.experts)) atomicOr(&bits[id >> 5], 1u << (id & 31));
    }
  }
};

// The rows of one expert: the tokens that picked it, in their order.
struct ExpertRows {
  int expert, count;         // -1: no such expert
  int token[kLayerTokens], pick[kLayerTokens];
  float gate[kLayerTokens];
};

// The slot-th touched expert and its rows, found by one wave.  A token that
// picked an expert twice has one row, with the sum of its gates.
__device__ __forceinline__ void find_rows(const LayerArgs& P, const Touched& set, int slot, ExpertRows* out) {
  static_assert(kLayerExperts / 32 <= 128 && kLayerTokens <= 64, "two words and one token per lane");
  const int lane = threadIdx.x & 63;
  const uint32_t a = set.bits[2 * lane], b = set.bits[2 * lane + 1];
  const int n = __popc(a) + __popc(b), upto = wave_scan_sum(n);
  const uint64_t hit = __ballot(upto > slot);
  int expert = -1;
  if (hit) {
    const int l = __builtin_ctzll(hit);
    int left = slot - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(n, l));
    uint64_t word = (uint64_t(uint32_t(__builtin_amdgcn_readlane(int(b), l))) << 32) |
                    uint32_t(__builtin_amdgcn_readlane(int(a), l));
    for (; left > 0; --left) word &= word - 1;
    expert = 64 * l + __builtin_ctzll(word);
  }
  int pick = -1;
  float gate = 0.f;
  if (lane < P.tokens && expert >= 0) {
    for (int j = 0; j < P.top_k; ++j) {
      if (P.ids[lane * P.top_k + j] != expert) continue;
      if (pick < 0) pick = j;
      gate += P.gates[lane * P.top_k + j];
    }
  }
  const uint64_t rows = __ballot(pick >= 0);
  if (pick >= 0) {
    const int i = __popcll(rows & ((uint64_t(1) << lane) - 1));
    out->token[i] = lane;
    out->pick[i] = pick;
    out->gate[i] = gate;
  }
  if (lane == 0) {
    out->expert = expert;
    out->count = __popcll(rows);
  }
}

// Rows of h, elements: both parts one behind the other, whole 16-byte chunks.
__device__ __forceinline__ int64_t part_of(int64_t n) { return (n + 7) / 8 * 8; }

// Sixteen columns of h (16 rows of G and of U) of one expert.
template <bool I8, bool VEC, int MB>
__global__ void __launch_bounds__(kLayerThreads)
layer_in_kernel(LayerArgs P) {
  constexpr int U = I8 ? 2 : 4;
  __shared__ Touched set;
  __shared__ ExpertRows rows;
  __shared__ __attribute__((aligned(16))) float sums[kLayerWaves * 2 * MB * 256];
  const uint32_t nt = (uint32_t(P.n) + 15) / 16;
  const int slot = int(blockIdx.x / nt), tn = int(blockIdx.x - uint32_t(slot) * nt);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  set.build(P);
  __syncthreads();
  if (wave == 0) find_rows(P, set, slot, &rows);
  __syncthreads();
  const int e = __builtin_amdgcn_readfirstlane(rows.expert), count = __builtin_amdgcn_readfirstlane(rows.count);
  if (e < 0) return;
  const int r = lane & 15, g = lane >> 4;
  const int cols = int(P.n - 16 * tn < 16 ? P.n - 16 * tn : 16);
  const int64_t bytes = P.k * (I8 ? 1 : 2), part = part_of(P.n);
  const int steps = int((bytes + 127) / 128);
  // columns past the end read the last one: their results are not stored
  const int64_t j = 16 * int64_t(tn) + (r < cols ? r : cols - 1);
  const char* wp[2];
  wp[0] = static_cast<const char*>(P.w_in) + (e * P.in_stride + j * P.ld_in) * (I8 ? 1 : 2);
  wp[1] = wp[0] + P.n * P.ld_in * (I8 ? 1 : 2);
  for (int r0 = 0; r0 < count; r0 += 16 * MB) {
    const char* xp[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const int i = r0 + 16 * m + r;
      xp[m] = static_cast<const char*>(P.x) + rows.token[i < count ? i : count - 1] * P.ldx * 2;
    }
    f32x4_t acc[2][MB];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int m = 0; m < MB; ++m) acc[n][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int s0 = wave * U; s0 < steps; s0 += kLayerWaves * U) {
      WeightStep w[U][2];
      RowStep<I8> x[U][MB];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t at = int64_t(s0 + u) * 128;
#pragma unroll
        for (int n = 0; n < 2; ++n) w[u][n] = load_weight<I8, VEC>(wp[n], at, bytes, g);
#pragma unroll
        for (int m = 0; m < MB; ++m) x[u][m] = load_row<I8, VEC>(xp[m], at, bytes, g);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int n = 0; n < 2; ++n) add_step<I8, MB>(w[u][n], x[u], acc[n]);
    }
    if (r0 > 0) __syncthreads();      // the sums of the rows before are read
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int m = 0; m < MB; ++m)
        *reinterpret_cast<f32x4_t*>(sums + ((wave * 2 * MB + n * MB + m) * 64 + lane) * 4) = acc[n][m];
    __syncthreads();
    if (wave < MB) {
      f32x4_t v[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        v[n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kLayerWaves; ++w)
          v[n] += *reinterpret_cast<const f32x4_t*>(sums + ((w * 2 * MB + n * MB + wave) * 64 + lane) * 4);
      }
      const int i = r0 + 16 * wave + r;
      if (i < count) {
        const float gate = rows.gate[i];
        float x[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float a = v[0][q], b = v[1][q];
          if constexpr (I8) {
            const int64_t c = 16 * int64_t(tn) + (4 * g + q < cols ? 4 * g + q : cols - 1);
            a *= P.in_scale[e * 2 * P.n + c];
            b *= P.in_scale[e * 2 * P.n + P.n + c];
          }
          x[q] = gated(a, b) * gate;
        }
        uint16_t* h = P.h + (int64_t(rows.token[i]) * P.top_k + rows.pick[i]) * 2 * part + 16 * int64_t(tn);
        store4<uint16_t>(h, 4 * g, cols, false, x);
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] -= bf16_lo(pack2_bf16(x[q], 0.f));
        store4<uint16_t>(h + part, 4 * g, cols, false, x);
      }
    }
  }
}

// Sixteen columns of y for all tokens.  The waves take (expert, four steps of
// its rows) in turn.
template <bool I8, bool VEC, int MB>
__global__ void __launch_bounds__(kLayerThreads)
layer_out_kernel(LayerArgs P) {
  constexpr int U = I8 ? 2 : 4;
  __shared__ Touched set;
  __shared__ uint16_t experts[kLayerExperts];
  __shared__ int total;
  __shared__ int16_t ids[kLayerTokens * kLayerPicks];
  __shared__ __attribute__((aligned(16))) float sums[kLayerWaves * MB * 256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  set.build(P);
  for (int i = threadIdx.x; i < P.tokens * P.top_k; i += kLayerThreads) {
    const uint32_t id = uint32_t(P.ids[i]);
    ids[i] = id < uint32_t(P.experts) ? int16_t(id) : int16_t(-1);
  }
  __syncthreads();
  if (wave == 0) {
    uint64_t word = (uint64_t(set.bits[2 * lane + 1]) << 32) | set.bits[2 * lane];
    const int n = __popcll(word), upto = wave_scan_sum(n);
    for (int i = upto - n; word; ++i, word &= word - 1) experts[i] = uint16_t(64 * lane + __builtin_ctzll(word));
    if (lane == 63) total = upto;
  }
  __syncthreads();
  const int r = lane & 15, g = lane >> 4;
  const int64_t c0 = 16 * int64_t(blockIdx.x);
  const int cols = int(P.k - c0 < 16 ? P.k - c0 : 16);
  const int64_t bytes = P.n * (I8 ? 1 : 2), part = part_of(P.n);
  const int steps = int((bytes + 127) / 128), units = (steps + U - 1) / U;
  const int64_t j = c0 + (r < cols ? r : cols - 1);
  f32x4_t acc[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int all = __builtin_amdgcn_readfirstlane(total) * units;
  for (int i = wave; i < all; i += kLayerWaves) {
    const int slot = i / units, s0 = (i - slot * units) * U;
    const int e = __builtin_amdgcn_readfirstlane(experts[slot]);
    const char* wp = static_cast<const char*>(P.w_out) + (e * P.out_stride + j * P.ld_out) * (I8 ? 1 : 2);
    const char* hp[MB];
    bool has[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const int t = 16 * m + r;
      int pick = -1;
      if (t < P.tokens)
        for (int q = P.top_k - 1; q >= 0; --q)
          if (ids[t * P.top_k + q] == e) pick = q;
      has[m] = pick >= 0;
      hp[m] = reinterpret_cast<const char*>(P.h + (int64_t(t) * P.top_k + (pick < 0 ? 0 : pick)) * 2 * part);
    }
    WeightStep w[U];
    RowStep<I8> x[U][2][MB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = int64_t(s0 + u) * 128;
      w[u] = load_weight<I8, VEC>(wp, at, bytes, g);
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int m = 0; m < MB; ++m)
          x[u][q][m] = load_row<I8, VEC>(hp[m] + q * part * 2, at, has[m] ? bytes : 0, g);
    }
    f32x4_t p[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) p[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < 2; ++q) add_step<I8, MB>(w[u], x[u][q], p);
    // only the expert's own tokens: a weight that is not finite is nobody else's
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float s = 1.f;
      if constexpr (I8) s = P.out_scale[e * P.k + c0 + (4 * g + q < cols ? 4 * g + q : cols - 1)];
#pragma unroll
      for (int m = 0; m < MB; ++m) acc[m][q] = has[m] ? fmaf(s, p[m][q], acc[m][q]) : acc[m][q];
    }
  }
#pragma unroll
  for (int m = 0; m < MB; ++m)
    *reinterpret_cast<f32x4_t*>(sums + ((wave * MB + m) * 64 + lane) * 4) = acc[m];
  __syncthreads();
  if (wave < MB) {
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kLayerWaves; ++w)
      v += *reinterpret_cast<const f32x4_t*>(sums + ((w * MB + wave) * 64 + lane) * 4);
    const int t = 16 * wave + r;
    if (t < P.tokens) {
      const float x[4] = {v[0], v[1], v[2], v[3]};
      store4<uint16_t>(static_cast<uint16_t*>(P.y) + t * P.ldy + c0, 4 * g, cols, false, x);
    }
  }
}

template <bool I8, bool VEC>
hipError_t launch_in(const LayerArgs& P, hipStream_t stream) {
  const int64_t picks = int64_t(P.tokens) * P.top_k, slots = picks < P.experts ? picks : P.experts;
  const dim3 grid(static_cast<unsigned>(slots * ((P.n + 15) / 16))), block(kLayerThreads);
  if (P.tokens <= 16) hipLaunchKernelGGL((layer_in_kernel<I8, VEC, 1>), grid, block, 0, stream, P);
  else hipLaunchKernelGGL((layer_in_kernel<I8, VEC, 2>), grid, block, 0, stream, P);
  return hipGetLastError();
}
template <bool I8, bool VEC>
hipError_t launch_out(const LayerArgs& P, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((P.k + 15) / 16)), block(kLayerThreads);
  if (P.tokens <= 16) hipLaunchKernelGGL((layer_out_kernel<I8, VEC, 1>), grid, block, 0, stream, P);
  else if (P.tokens <= 32) hipLaunchKernelGGL((layer_out_kernel<I8, VEC, 2>), grid, block, 0, stream, P);
  else hipLaunchKernelGGL((layer_out_kernel<I8, VEC, 4>), grid, block, 0, stream, P);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_in(const LayerArgs& P, bool vec, hipStream_t stream) {
  if (P.in_scale) return vec ? launch_in<true, true>(P, stream) : launch_in<true, false>(P, stream);
  return vec ? launch_in<false, true>(P, stream) : launch_in<false, false>(P, stream);
}
hipError_t launch_layer_out(const LayerArgs& P, bool vec, hipStream_t stream) {
  if (P.in_scale) return vec ? launch_out<true, true>(P, stream) : launch_out<true, false>(P, stream);
  return vec ? launch_out<false, true>(P, stream) : launch_out<false, false>(P, stream);
}

}  // namespace dmuon

// Argument checks shared by the entry points of the products and the 8-bit
// operators (products.hip, products8.hip): limits, alignment, overlaps.
#pragma once

#include <initializer_list>
#include <string>

#include "internal.h"

namespace dmuon {

constexpr int64_t kMaxDim = int64_t(1) << 22;       // features, row strides
constexpr int64_t kMaxRows = int64_t(1) << 30;      // tokens
constexpr int64_t kMaxStride = int64_t(1) << 44;    // between experts' weights or a batch's matrices
constexpr int32_t kMaxExperts = 65536;
constexpr int64_t kMaxNumel = int64_t(1) << 42;     // elements of a tensor
constexpr int64_t kMaxInt8Sum = 131071;             // products of two 8-bit integers that an int32 holds
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 4096;   // blocks of 256 threads in one launch

inline int bad(const std::string& msg) { return set_last_error(DMUON_ERR_INVALID_ARG, msg); }

inline bool real_dtype(int32_t dt) { return dt == DT_F32 || dt == DT_BF16; }
inline bool q8_dtype(int32_t dt) { return dt == DT_E4M3 || dt == DT_E5M2; }
inline int64_t size_of(int32_t dt) { return dt == DT_F32 ? 4 : dt == DT_BF16 ? 2 : 1; }
inline int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

struct Span {
  const void* p;
  int64_t bytes;      // from the first to one past the last
  const char* name;
};

// The written buffers (the first `nout`) must not overlap each other or anything read.
inline int check_spans(std::initializer_list<Span> spans, int nout) {
  int i = 0;
  for (const Span& a : spans) {
    if (i++ >= nout) break;
    if (!a.p || a.bytes <= 0) continue;
    int j = 0;
    for (const Span& b : spans) {
      if (j++ < i || !b.p || b.bytes <= 0) continue;
      const uintptr_t al = reinterpret_cast<uintptr_t>(a.p), bl = reinterpret_cast<uintptr_t>(b.p);
      if (al < bl + uintptr_t(b.bytes) && bl < al + uintptr_t(a.bytes))
        return set_last_error(DMUON_ERR_ALIASING, std::string(a.name) + " overlaps " + b.name);
    }
  }
  return DMUON_OK;
}

inline int hip_status(hipError_t e, const char* what) {
  return e == hipSuccess ? DMUON_OK
                         : set_last_error(DMUON_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

inline int64_t product_flops(int64_t m, int64_t n, int64_t k) {
  const double f = 2.0 * double(m) * double(n) * double(k);   // beyond int64 for the largest allowed sizes
  return f < 9e18 ? static_cast<int64_t>(f) : INT64_MAX;
}

inline int64_t rows_bytes(int64_t rows, int64_t ld, int64_t cols, int64_t size) {
  return rows <= 0 ? 0 : ((rows - 1) * ld + cols) * size;
}

}  // namespace dmuon

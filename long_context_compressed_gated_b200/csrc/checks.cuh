// checks.cuh - host-side argument checks shared by the entry points of the C ABI.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>
#include <initializer_list>

#include "common.cuh"

namespace csa {

// Records e for csa_last_cuda_error() and returns the status to hand back.
int cuda_fail(cudaError_t e);
// Streaming multiprocessors of the current device (queried once per device).
int sm_count();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename... P>
int check_ptrs(P... ps) {
  const void* arr[] = {static_cast<const void*>(ps)...};
  for (const void* p : arr) {
    if (p == nullptr) return CSA_ERR_INVALID_ARG;
    if (!aligned16(p)) return CSA_ERR_MISALIGNED;
  }
  return CSA_OK;
}

inline int check_opt(const void* p) { return (p != nullptr && !aligned16(p)) ? CSA_ERR_MISALIGNED : CSA_OK; }

inline int check_ws(void* ws, size_t bytes, size_t need) {
  if (ws == nullptr || bytes < need) return CSA_ERR_WORKSPACE;
  if (!aligned16(ws)) return CSA_ERR_MISALIGNED;
  return CSA_OK;
}

inline int* status_word(void* ws) { return static_cast<int*>(ws); }

inline bool valid_odtype(int t) { return t == CSA_BF16 || t == CSA_F32; }

// Rows of a page of the paged cache: a power of two, 16 .. 256.
inline bool valid_page(int page) { return page >= 16 && page <= 256 && (page & (page - 1)) == 0; }

// The arguments of a position rotation (rope.cu).
int check_rotation(int d, const double* inv_freq, int rot_start, int rot_dim, int rot_style, float eps);

// Bytes from the first to the last element of T token rows, `stride` elements apart.
inline size_t span(int64_t T, int64_t stride, int heads, int d, int dtype) {
  return T > 0 && heads > 0 ? (size_t)((T - 1) * stride + (int64_t)heads * d) * (dtype == CSA_BF16 ? 2 : 4) : 0;
}

// Whether two ranges of bytes share one.
inline bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return an > 0 && bn > 0 && x < y + bn && y < x + an;
}

// A range of bytes, and whether one shares a byte with any of some others (null pointers share none).
struct Bytes {
  const void* p;
  size_t n;
};
inline bool overlap_any(Bytes a, std::initializer_list<Bytes> others) {
  for (const Bytes& b : others)
    if (a.p != nullptr && b.p != nullptr && overlap(a.p, a.n, b.p, b.n)) return true;
  return false;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace csa

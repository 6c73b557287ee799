// Host-side argument validation shared by the C entry points of libmuon.
#pragma once
#include <cstddef>
#include <cstdint>

#include "muon.h"

namespace muon {

// Host validation of a Newton-Schulz-only matrix list and its hyper-parameters
// (null pointers, enums, flags, eps, shapes, leading dimensions, dtypes, alignment,
// aliasing). Makes no CUDA call. Every Newton-Schulz entry point uses it, so the
// same arguments get the same status from each of them.
muon_status_t validate_ns(const muon_ns_matrix_t* mats, int n, const muon_hparams_t* hp);

// The current device and its SM count; MUON_ERR_UNSUPPORTED when it is not sm_100.
muon_status_t current_device(int* dev, int* num_sms);

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte.
inline bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

// Bytes from the first to the last element of a rows x cols matrix (0 without rows).
inline size_t matrix_span(int64_t rows, int64_t cols, int64_t ld, size_t elem) {
  return rows < 1 ? 0 : (static_cast<size_t>(rows - 1) * static_cast<size_t>(ld) +
                         static_cast<size_t>(cols)) * elem;
}

}  // namespace muon

// 8-bit activation checkpoints: int8 values with one power-of-two scale per row and group
// of 32 columns (muon_act8_t).
//
//   amax = max |x| of the group, E = max(floor(log2 amax) - 6, -126)
//   q = clamp(rne(x 2^-E), -127, 127)          restored: q 2^E
//
// E is read off the exponent bits of amax, and both scalings are by powers of two, so the
// only rounding is the one to an integer. A power of two rather than amax / 127 costs up to
// one bit of q; in return q 2^E has 7 significant bits and a consumer that feeds a bf16
// matrix instruction restores it without a second rounding.
//
// Memory bound: store reads x and writes 1 + 1/32 bytes per element, restore the reverse.
// A thread owns 8 consecutive columns (one or two 16-byte loads, one 8-byte store) of kUnits
// rows, all loaded first; four neighbouring lanes hold a group (two shuffles for amax).
// 16384 x 5632 in bf16: store 65 us (4.3 TB/s, still the instructions: about 10 per element),
// restore 48 us (5.8 TB/s).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <memory>
#include <new>

#include "act8.cuh"
#include "muon.h"
#include "ptx.cuh"
#include "validate.h"

namespace muon {
namespace {

// Items of one launch: kernel parameters stay below 32 KB, and a short list takes the form
// with short ones, whose launch costs the host a microsecond less.
constexpr int kItemsPerLaunch = 128, kFewItems = 4;
constexpr int kThreads = 256;
constexpr int kUnits = 4;                // rows a thread handles
constexpr int64_t kMaxCols = int64_t(1) << 26;

template <int kItems>
struct Act8Launch {
  muon_act8_t a[kItems];
  int32_t block_base[kItems + 1];
  int32_t n;
};
static_assert(sizeof(Act8Launch<kItemsPerLaunch>) < 32000, "kernel parameter space");

// How a block covers a matrix: `span` units (whole groups of four, so that a group's lanes stay
// together) of each row, one of `chunks` equal parts of it, in `rows` rows at a time, kUnits
// times. A thread keeps its columns and steps down the rows, so that it divides once.
struct Cover {
  int32_t chunks, span, rows;
};

__host__ __device__ inline Cover cover_of(int64_t cols) {
  const int32_t units = static_cast<int32_t>((cols + 31) / 32 * 4);
  Cover c;
  c.chunks = (units + kThreads - 1) / kThreads;
  c.span = ((units + c.chunks - 1) / c.chunks + 3) / 4 * 4;
  c.rows = kThreads / c.span;
  return c;
}

inline int64_t blocks_of(const muon_act8_t& a) {
  const Cover c = cover_of(a.cols);
  return (a.rows + kUnits * c.rows - 1) / (kUnits * c.rows) * c.chunks;
}

template <int kItems>
__device__ __forceinline__ int find_item(const Act8Launch<kItems>& L) {
  int lo = 0, hi = L.n - 1;  // the item of this block: last base <= blockIdx.x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (L.block_base[mid] <= static_cast<int>(blockIdx.x)) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// This thread's columns [col, col + 8) and its rows row, row + step, ..; live(u): in the matrix.
struct Place {
  int64_t row, rows;
  int32_t col, step, cols;
  __device__ __forceinline__ bool live(int u) const { return row + u * step < rows; }
  __device__ __forceinline__ bool whole() const { return col + 8 <= cols; }
};

__device__ __forceinline__ Place place_of(const muon_act8_t& a, int block) {
  const Cover c = cover_of(a.cols);
  const int rb = block / c.chunks, chunk = block - rb * c.chunks;
  const int rt = static_cast<int>(threadIdx.x) / c.span, ct = static_cast<int>(threadIdx.x) - rt * c.span;
  Place p;
  p.step = c.rows;
  p.cols = static_cast<int32_t>(a.cols);
  p.col = (chunk * c.span + ct) * 8;
  p.row = static_cast<int64_t>(rb) * (kUnits * c.rows) + rt;
  p.rows = rt < c.rows && p.col < p.cols ? a.rows : 0;
  return p;
}

// The 8 values of a unit as they are in memory (BF16: 4 words, F32: 8); columns past the matrix
// read as 0.
template <bool kBf16>
__device__ __forceinline__ void load_unit(const void* X, int64_t off, const Place& t, int u, bool vec,
                                          uint32_t (&w)[kBf16 ? 4 : 8]) {
#pragma unroll
  for (int i = 0; i < (kBf16 ? 4 : 8); ++i) w[i] = 0;
  if (!t.live(u)) return;
  if (kBf16) {
    const uint16_t* p = static_cast<const uint16_t*>(X) + off;
    if (vec && t.whole()) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t.col + i < t.cols) w[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
    }
  } else {
    const uint32_t* p = static_cast<const uint32_t*>(X) + off;
    if (vec && t.whole()) {
      const uint4 v0 = __ldcs(reinterpret_cast<const uint4*>(p)), v1 = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
      w[0] = v0.x; w[1] = v0.y; w[2] = v0.z; w[3] = v0.w;
      w[kBf16 ? 0 : 4] = v1.x; w[kBf16 ? 0 : 5] = v1.y; w[kBf16 ? 0 : 6] = v1.z; w[kBf16 ? 0 : 7] = v1.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t.col + i < t.cols) w[kBf16 ? 0 : i] = p[i];
    }
  }
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// Two signed 16-bit numbers clamped to [-127, 127].
__device__ __forceinline__ uint32_t clamp127_s16x2(uint32_t x) {
  uint32_t r;
  asm("min.s16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x007F007Fu));
  asm("max.s16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0xFF81FF81u));
  return r;
}

// Stores rows u0 .. u0 + kCount - 1 of the thread: all loads first.
template <bool kBf16, int kCount>
__device__ __forceinline__ void store_units(const muon_act8_t& a, const Place& t, bool vec, int u0) {
  uint32_t w[kCount][kBf16 ? 4 : 8];
  const int64_t row0 = t.row + u0 * t.step, off0 = row0 * a.ld_x + t.col, step_x = t.step * a.ld_x;
#pragma unroll
  for (int u = 0; u < kCount; ++u) load_unit<kBf16>(a.X, off0 + u * step_x, t, u0 + u, vec, w[u]);
  int8_t* q = a.q + row0 * a.ld_q + t.col;
  uint8_t* ex = a.exps + row0 * a.ld_e + (t.col >> 5);
  const int64_t step_q = t.step * a.ld_q, step_e = t.step * a.ld_e;
#pragma unroll
  for (int u = 0; u < kCount; ++u, q += step_q, ex += step_e) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = __uint_as_float(!kBf16 ? w[u][kBf16 ? 0 : i] : (i & 1) ? w[u][i >> 1] & 0xFFFF0000u : w[u][i >> 1] << 16);
    uint32_t top = 0;  // magnitudes compare as integers, NaN above infinity
    if (kBf16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max_u16x2(top, w[u][i] & 0x7FFF7FFFu);
      top = max(top & 0xFFFF0000u, top << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, w[u][kBf16 ? 0 : i] & 0x7FFFFFFFu);
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int be = static_cast<int>(top >> 23);
    const uint32_t byte = be == 255 ? 255u : static_cast<uint32_t>(max(be - 6, 1));
    // 2^-E; a group with a NaN or an infinity stores zeros under byte 255
    const float inv = byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
    // Adding 1.5 * 2^23 to the (exact) product rounds half to even and leaves the integer, at most
    // 128, in the low bits (a conversion instruction runs at a quarter of the rate); the clamp
    // then takes two of them at a time.
    uint32_t v[8], pk[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(fmaf(x[i], inv, 12582912.f));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      pk[i] = __byte_perm(clamp127_s16x2(__byte_perm(v[4 * i], v[4 * i + 1], 0x5410)),
                          clamp127_s16x2(__byte_perm(v[4 * i + 2], v[4 * i + 3], 0x5410)), 0x6420);
      if (byte == 255u) pk[i] = 0;
    }
    if (!t.live(u0 + u)) continue;
    if (t.whole()) {
      *reinterpret_cast<uint2*>(q) = make_uint2(pk[0], pk[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t.col + i < t.cols) q[i] = static_cast<int8_t>(pk[i >> 2] >> (8 * (i & 3)));
    }
    if ((threadIdx.x & 3) == 0) *ex = static_cast<uint8_t>(byte);
  }
}

__device__ __forceinline__ bool rows_aligned(const muon_act8_t& a) {
  const int64_t elem = a.dtype == MUON_BF16 ? 2 : 4;
  return reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && (a.ld_x * elem) % 16 == 0;
}

template <int kItems>
__global__ void __launch_bounds__(kThreads, 5) act8_store_kernel(const __grid_constant__ Act8Launch<kItems> L) {
  const int it = find_item(L);
  const muon_act8_t& a = L.a[it];
  const Place t = place_of(a, static_cast<int>(blockIdx.x) - L.block_base[it]);
  const bool vec = rows_aligned(a);
  if (a.dtype == MUON_BF16) {
    store_units<true, kUnits>(a, t, vec, 0);
  } else {
    store_units<false, kUnits / 2>(a, t, vec, 0);
    store_units<false, kUnits / 2>(a, t, vec, kUnits / 2);
  }
}

template <int kItems>
__global__ void __launch_bounds__(kThreads) act8_restore_kernel(const __grid_constant__ Act8Launch<kItems> L) {
  const int it = find_item(L);
  const muon_act8_t& a = L.a[it];
  const Place t = place_of(a, static_cast<int>(blockIdx.x) - L.block_base[it]);
  const bool vec = rows_aligned(a);
  uint2 w[kUnits];
  uint32_t byte[kUnits];
  const int8_t* q = a.q + t.row * a.ld_q + t.col;
  const uint8_t* ex = a.exps + t.row * a.ld_e + (t.col >> 5);
  const int64_t step_q = t.step * a.ld_q, step_e = t.step * a.ld_e;
#pragma unroll
  for (int u = 0; u < kUnits; ++u, q += step_q, ex += step_e) {
    w[u] = make_uint2(0, 0);
    byte[u] = 1;
    if (!t.live(u)) continue;
    if (t.whole()) {
      w[u] = __ldcs(reinterpret_cast<const uint2*>(q));
    } else {
      uint32_t pk[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t.col + i < t.cols) pk[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(q[i])) << (8 * (i & 3));
      w[u] = make_uint2(pk[0], pk[1]);
    }
    byte[u] = *ex;
  }
  int64_t off = t.row * a.ld_x + t.col;
  const int64_t step_x = t.step * a.ld_x;
#pragma unroll
  for (int u = 0; u < kUnits; ++u, off += step_x) {
    if (!t.live(u)) continue;
    const uint32_t sc = act8_scale2(byte[u]);
    uint32_t y[4];  // bf16 pairs
    act8_restore4(w[u].x, sc, sc, &y[0], &y[1]);
    act8_restore4(w[u].y, sc, sc, &y[2], &y[3]);
    const bool whole = vec && t.whole();
    if (a.dtype == MUON_BF16) {
      uint16_t* p = static_cast<uint16_t*>(a.X) + off;
      if (whole) {
        *reinterpret_cast<uint4*>(p) = make_uint4(y[0], y[1], y[2], y[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (t.col + i < t.cols) p[i] = static_cast<uint16_t>(y[i >> 1] >> (16 * (i & 1)));
      }
    } else {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float((i & 1) ? y[i >> 1] & 0xFFFF0000u : y[i >> 1] << 16);
      float* p = static_cast<float*>(a.X) + off;
      if (whole) {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (t.col + i < t.cols) p[i] = x[i];
      }
    }
  }
}

size_t span_x(const muon_act8_t& a) {
  return matrix_span(a.rows, a.cols, a.ld_x, a.dtype == MUON_BF16 ? 2 : 4);
}
size_t span_q(const muon_act8_t& a) { return matrix_span(a.rows, a.cols, a.ld_q, 1); }
size_t span_e(const muon_act8_t& a) { return matrix_span(a.rows, (a.cols + 31) / 32, a.ld_e, 1); }

muon_status_t validate_act8(const muon_act8_t* items, int n, bool store) {
  if (n < 0 || (n > 0 && items == nullptr)) return MUON_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    const muon_act8_t& a = items[i];
    if (a.dtype != MUON_F32 && a.dtype != MUON_BF16) return MUON_ERR_DTYPE;
    const int64_t groups = (a.cols + 31) / 32;
    if (a.rows < 0 || a.cols < 1 || a.cols > kMaxCols || a.ld_x < a.cols || a.ld_q < a.cols ||
        a.ld_e < groups || a.ld_q % 16 || a.ld_e % 16)
      return MUON_ERR_SHAPE;
    // every byte offset stays far inside 63 bits
    const int64_t lim = int64_t(1) << 40;
    if (a.rows > lim || a.ld_x > lim || a.ld_q > lim || a.ld_e > lim) return MUON_ERR_SHAPE;
    if (a.rows > 0 && (a.ld_x > (lim << 1) / a.rows || a.ld_q > (lim << 1) / a.rows)) return MUON_ERR_SHAPE;
    if (a.rows > 0 && a.ld_e > (lim << 1) / a.rows) return MUON_ERR_SHAPE;
    if (a.rows == 0) continue;
    if (a.X == nullptr || a.q == nullptr || a.exps == nullptr) return MUON_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a.X) % (a.dtype == MUON_BF16 ? 2 : 4) ||
        reinterpret_cast<uintptr_t>(a.q) % 16 || reinterpret_cast<uintptr_t>(a.exps) % 16)
      return MUON_ERR_INVALID_ARG;
  }
  // Nothing written (store: q and exps, restore: X) overlaps anything else: in the order of their
  // starts, nothing begins before the end of what is written before it, and nothing written
  // before the end of anything.
  struct Range {
    uintptr_t lo, hi;
    bool written;
  };
  Range few[3 * kFewItems];
  std::unique_ptr<Range[]> many(n > kFewItems ? new (std::nothrow) Range[3 * static_cast<size_t>(n)] : nullptr);
  Range* const r = n > kFewItems ? many.get() : few;
  if (r == nullptr) return MUON_ERR_CUDA;  // out of host memory
  size_t count = 0;
  for (int i = 0; i < n; ++i) {
    const muon_act8_t& a = items[i];
    if (a.rows == 0) continue;
    const auto x = reinterpret_cast<uintptr_t>(a.X), q = reinterpret_cast<uintptr_t>(a.q),
               e = reinterpret_cast<uintptr_t>(a.exps);
    r[count++] = {x, x + span_x(a), !store};
    r[count++] = {q, q + span_q(a), store};
    r[count++] = {e, e + span_e(a), store};
  }
  std::sort(r, r + count, [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t end = 0, end_written = 0;
  for (size_t i = 0; i < count; ++i) {
    if (r[i].lo < (r[i].written ? end : end_written)) return MUON_ERR_ALIAS;
    end = std::max(end, r[i].hi);
    if (r[i].written) end_written = std::max(end_written, r[i].hi);
  }
  return MUON_OK;
}

template <int kItems>
muon_status_t launch_act8(const muon_act8_t* items, int n, bool store, cudaStream_t st) {
  Act8Launch<kItems> L;
  L.n = n;
  int64_t blocks = 0;
  for (int i = 0; i < n; ++i) {
    L.a[i] = items[i];
    L.block_base[i] = static_cast<int32_t>(blocks);
    blocks += blocks_of(items[i]);
  }
  L.block_base[n] = static_cast<int32_t>(blocks);
  if (blocks == 0) return MUON_OK;
  if (store) act8_store_kernel<kItems><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(L);
  else act8_restore_kernel<kItems><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(L);
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

muon_status_t run_act8(const muon_act8_t* items, int n, bool store, void* stream) {
  const muon_status_t v = validate_act8(items, n, store);
  if (v != MUON_OK || n == 0) return v;
  int dev = 0, sms = 0;
  const muon_status_t d = current_device(&dev, &sms);
  if (d != MUON_OK) return d;
  for (int i = 0; i < n; ++i)  // nothing runs unless every launch fits its grid
    if (blocks_of(items[i]) > (int64_t(1) << 30) / kItemsPerLaunch) return MUON_ERR_SHAPE;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n <= kFewItems) return launch_act8<kFewItems>(items, n, store, st);
  for (int i0 = 0; i0 < n; i0 += kItemsPerLaunch) {
    const muon_status_t s =
        launch_act8<kItemsPerLaunch>(items + i0, n - i0 < kItemsPerLaunch ? n - i0 : kItemsPerLaunch, store, st);
    if (s != MUON_OK) return s;
  }
  return MUON_OK;
}

}  // namespace
}  // namespace muon

extern "C" MUON_API muon_status_t muon_act8_store(const muon_act8_t* items, int n, void* stream) {
  return muon::run_act8(items, n, true, stream);
}

extern "C" MUON_API muon_status_t muon_act8_restore(const muon_act8_t* items, int n, void* stream) {
  return muon::run_act8(items, n, false, stream);
}

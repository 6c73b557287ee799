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
// A thread owns units of 8 consecutive columns (one or two 16-byte loads, one 8-byte store),
// four neighbouring lanes a group (two shuffles for amax); kUnits units a thread keep as
// many loads in flight.
#include <cuda_runtime.h>

#include <cstdint>

#include "muon.h"
#include "ptx.cuh"
#include "validate.h"

namespace muon {
namespace {

constexpr int kItemsPerLaunch = 128;  // kernel parameters stay below 32 KB
constexpr int kThreads = 256;
constexpr int kUnits = 4;
constexpr int kUnitsPerBlock = kThreads * kUnits;
constexpr int64_t kMaxCols = int64_t(1) << 26;

struct Act8Launch {
  muon_act8_t a[kItemsPerLaunch];
  int32_t block_base[kItemsPerLaunch + 1];
  int32_t n;
};
static_assert(sizeof(Act8Launch) < 32000, "kernel parameter space");

// Units of a row: whole groups of four, so that a group's lanes stay together.
__host__ __device__ inline int64_t units_per_row(int64_t cols) { return (cols + 31) / 32 * 4; }

struct Unit {
  int64_t row;
  int32_t col;     // first column
  bool live;       // inside the matrix's rows
};

__device__ __forceinline__ int find_item(const Act8Launch& L) {
  int lo = 0, hi = L.n - 1;  // the item of this block: last base <= blockIdx.x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (L.block_base[mid] <= static_cast<int>(blockIdx.x)) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ Unit unit_at(const muon_act8_t& a, int64_t row0, uint32_t rem0,
                                        uint32_t upr, int u) {
  const uint32_t r = rem0 + u * kThreads + threadIdx.x;
  const uint32_t dr = r / upr;
  Unit t;
  t.row = row0 + dr;
  t.col = static_cast<int32_t>(r - dr * upr) * 8;
  t.live = t.row < a.rows;
  return t;
}

// The 8 values of a unit as fp32; columns past the matrix read as 0.
__device__ __forceinline__ void load_unit(const muon_act8_t& a, const Unit& t, bool vec,
                                          float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = 0.f;
  if (!t.live || t.col >= a.cols) return;
  const int64_t off = t.row * a.ld_x + t.col;
  if (a.dtype == MUON_BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(a.X) + off;
    if (vec && t.col + 8 <= a.cols) {
      const uint4 w = __ldcs(reinterpret_cast<const uint4*>(p));
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t.col + i < a.cols) x[i] = bf16_to_f32(p[i]);
    }
  } else {
    const float* p = static_cast<const float*>(a.X) + off;
    if (vec && t.col + 8 <= a.cols) {
      const float4 v0 = __ldcs(reinterpret_cast<const float4*>(p));
      const float4 v1 = __ldcs(reinterpret_cast<const float4*>(p) + 1);
      x[0] = v0.x; x[1] = v0.y; x[2] = v0.z; x[3] = v0.w;
      x[4] = v1.x; x[5] = v1.y; x[6] = v1.z; x[7] = v1.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t.col + i < a.cols) x[i] = p[i];
    }
  }
}

__device__ __forceinline__ bool rows_aligned(const muon_act8_t& a) {
  const int64_t elem = a.dtype == MUON_BF16 ? 2 : 4;
  return reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && (a.ld_x * elem) % 16 == 0;
}

__global__ void __launch_bounds__(kThreads) act8_store_kernel(const __grid_constant__ Act8Launch L) {
  const int it = find_item(L);
  const muon_act8_t& a = L.a[it];
  const uint32_t upr = static_cast<uint32_t>(units_per_row(a.cols));
  const int64_t base = static_cast<int64_t>(blockIdx.x - L.block_base[it]) * kUnitsPerBlock;
  const int64_t row0 = base / upr;
  const uint32_t rem0 = static_cast<uint32_t>(base - row0 * upr);
  const bool vec = rows_aligned(a);
  float x[kUnits][8];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) load_unit(a, unit_at(a, row0, rem0, upr, u), vec, x[u]);
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const Unit t = unit_at(a, row0, rem0, upr, u);
    uint32_t top = 0;  // magnitudes compare as integers, NaN above infinity
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[u][i]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int be = static_cast<int>(top >> 23);
    const uint32_t byte = be == 255 ? 255u : static_cast<uint32_t>(max(be - 6, 1));
    // 2^-E; a group with a NaN or an infinity stores zeros under byte 255
    const float inv = byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
    uint32_t pk[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int q = __float2int_rn(x[u][i] * inv);
      q = byte == 255u ? 0 : min(max(q, -127), 127);
      pk[i >> 2] |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * (i & 3));
    }
    if (!t.live || t.col >= a.cols) continue;
    int8_t* q = a.q + t.row * a.ld_q + t.col;
    if (t.col + 8 <= a.cols) {
      *reinterpret_cast<uint2*>(q) = make_uint2(pk[0], pk[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t.col + i < a.cols) q[i] = static_cast<int8_t>(pk[i >> 2] >> (8 * (i & 3)));
    }
    if ((threadIdx.x & 3) == 0) a.exps[t.row * a.ld_e + (t.col >> 5)] = static_cast<uint8_t>(byte);
  }
}

__global__ void __launch_bounds__(kThreads) act8_restore_kernel(const __grid_constant__ Act8Launch L) {
  const int it = find_item(L);
  const muon_act8_t& a = L.a[it];
  const uint32_t upr = static_cast<uint32_t>(units_per_row(a.cols));
  const int64_t base = static_cast<int64_t>(blockIdx.x - L.block_base[it]) * kUnitsPerBlock;
  const int64_t row0 = base / upr;
  const uint32_t rem0 = static_cast<uint32_t>(base - row0 * upr);
  const bool vec = rows_aligned(a);
  uint2 w[kUnits];
  uint32_t byte[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const Unit t = unit_at(a, row0, rem0, upr, u);
    w[u] = make_uint2(0, 0);
    byte[u] = 1;
    if (!t.live || t.col >= a.cols) continue;
    const int8_t* q = a.q + t.row * a.ld_q + t.col;
    if (t.col + 8 <= a.cols) {
      w[u] = __ldcs(reinterpret_cast<const uint2*>(q));
    } else {
      uint32_t pk[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t.col + i < a.cols) pk[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(q[i])) << (8 * (i & 3));
      w[u] = make_uint2(pk[0], pk[1]);
    }
    byte[u] = a.exps[t.row * a.ld_e + (t.col >> 5)];
  }
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const Unit t = unit_at(a, row0, rem0, upr, u);
    if (!t.live || t.col >= a.cols) continue;
    const float s = __uint_as_float(byte[u] << 23);  // byte 0: zero, byte 255: infinity, times 0 NaN
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = static_cast<float>(static_cast<int8_t>((i < 4 ? w[u].x : w[u].y) >> (8 * (i & 3)))) * s;
    const int64_t off = t.row * a.ld_x + t.col;
    const bool whole = vec && t.col + 8 <= a.cols;
    if (a.dtype == MUON_BF16) {
      uint16_t* p = static_cast<uint16_t*>(a.X) + off;
      if (whole) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                  pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (t.col + i < a.cols) p[i] = f32_to_bf16(x[i]);
      }
    } else {
      float* p = static_cast<float*>(a.X) + off;
      if (whole) {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (t.col + i < a.cols) p[i] = x[i];
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
  for (int i = 0; i < n; ++i) {
    const muon_act8_t& a = items[i];
    for (int j = 0; j < n; ++j) {
      const muon_act8_t& b = items[j];
      const void* bp[3] = {b.X, b.q, b.exps};
      const size_t bs[3] = {span_x(b), span_q(b), span_e(b)};
      for (int k = 0; k < 3; ++k) {
        // store writes q and exps, restore writes X; a buffer does not overlap itself
        if (store) {
          if (!(i == j && k == 1) && ranges_overlap(a.q, span_q(a), bp[k], bs[k])) return MUON_ERR_ALIAS;
          if (!(i == j && k == 2) && ranges_overlap(a.exps, span_e(a), bp[k], bs[k])) return MUON_ERR_ALIAS;
        } else if (!(i == j && k == 0) && ranges_overlap(a.X, span_x(a), bp[k], bs[k])) {
          return MUON_ERR_ALIAS;
        }
      }
    }
  }
  return MUON_OK;
}

muon_status_t run_act8(const muon_act8_t* items, int n, bool store, void* stream) {
  const muon_status_t v = validate_act8(items, n, store);
  if (v != MUON_OK || n == 0) return v;
  int dev = 0, sms = 0;
  const muon_status_t d = current_device(&dev, &sms);
  if (d != MUON_OK) return d;
  for (int i = 0; i < n; ++i)  // nothing runs unless every launch fits its grid
    if (units_per_row(items[i].cols) * items[i].rows / kUnitsPerBlock >
        (int64_t(1) << 30) / kItemsPerLaunch)
      return MUON_ERR_SHAPE;
  for (int i0 = 0; i0 < n; i0 += kItemsPerLaunch) {
    Act8Launch L;
    L.n = n - i0 < kItemsPerLaunch ? n - i0 : kItemsPerLaunch;
    int64_t blocks = 0;
    for (int i = 0; i < L.n; ++i) {
      L.a[i] = items[i0 + i];
      L.block_base[i] = static_cast<int32_t>(blocks);
      blocks += (units_per_row(L.a[i].cols) * L.a[i].rows + kUnitsPerBlock - 1) / kUnitsPerBlock;
    }
    L.block_base[L.n] = static_cast<int32_t>(blocks);
    if (blocks == 0) continue;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (store) act8_store_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(L);
    else act8_restore_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(L);
    if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
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

// Weight gradients from 8-bit activation checkpoints (muon_weight_grad_t):
//   dW_g[o, i] (+)= sum over the tokens t of group g of dY[t, o] q[t, i] 2^E[t, i/32]
//
// Simple form: a block computes a 64 x 64 tile of one group's gradient from tiles of 16
// tokens in shared memory, 4 x 4 outputs a thread, in fp32 on the CUDA cores.
#include <cuda_runtime.h>

#include <cstdint>

#include "muon.h"
#include "ptx.cuh"
#include "validate.h"

namespace muon {
namespace {

constexpr int kTile = 64, kTok = 16;

__device__ __forceinline__ float wg_scale(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u)
                      : byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

// Token range of group g, clamped to the tensor.
__device__ __forceinline__ void group_range(const muon_weight_grad_t& a, int g, int64_t* lo, int64_t* hi) {
  if (a.offsets == nullptr) {
    *lo = 0;
    *hi = a.tokens;
    return;
  }
  const int64_t b = a.offsets[g], e = a.offsets[g + 1];
  *lo = b < 0 ? 0 : b > a.tokens ? a.tokens : b;
  *hi = e < 0 ? 0 : e > a.tokens ? a.tokens : e;
  if (*hi < *lo) *hi = *lo;
}

__global__ void __launch_bounds__(256) wgrad_simple_kernel(const __grid_constant__ muon_weight_grad_t a) {
  __shared__ float sy[kTok][kTile + 1], sx[kTok][kTile + 1];
  const int g = blockIdx.z;
  const int64_t o0 = static_cast<int64_t>(blockIdx.y) * kTile, i0 = static_cast<int64_t>(blockIdx.x) * kTile;
  int64_t lo, hi;
  group_range(a, g, &lo, &hi);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  const uint16_t* dY = static_cast<const uint16_t*>(a.dY);
  for (int64_t t0 = lo; t0 < hi; t0 += kTok) {
    for (int j = threadIdx.x; j < kTok * kTile; j += 256) {
      const int r = j / kTile, c = j % kTile;
      const int64_t t = t0 + r;
      sy[r][c] = t < hi && o0 + c < a.out ? bf16_to_f32(dY[t * a.ld_dy + o0 + c]) : 0.f;
      sx[r][c] = t < hi && i0 + c < a.in
                     ? a.q[t * a.ld_q + i0 + c] * wg_scale(a.exps[t * a.ld_e + (i0 + c) / 32]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kTok; ++r)
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[y][x] = fmaf(sy[r][ty + 16 * y], sx[r][tx + 16 * x], acc[y][x]);
    __syncthreads();
  }
  for (int y = 0; y < 4; ++y)
    for (int x = 0; x < 4; ++x) {
      const int64_t o = o0 + ty + 16 * y, i = i0 + tx + 16 * x;
      if (o >= a.out || i >= a.in) continue;
      const int64_t at = g * a.stride_w + o * a.ld_w + i;
      if (a.w_dtype == MUON_F32) {
        float* p = static_cast<float*>(a.dW) + at;
        *p = a.accumulate ? *p + acc[y][x] : acc[y][x];
      } else {
        uint16_t* p = static_cast<uint16_t*>(a.dW) + at;
        *p = f32_to_bf16(a.accumulate ? bf16_to_f32(*p) + acc[y][x] : acc[y][x]);
      }
    }
}

muon_status_t validate_weight_grad(const muon_weight_grad_t* p) {
  if (p == nullptr) return MUON_ERR_INVALID_ARG;
  const muon_weight_grad_t& a = *p;
  if (a.w_dtype != MUON_F32 && a.w_dtype != MUON_BF16) return MUON_ERR_DTYPE;
  const int64_t lim = int64_t(1) << 31;
  if (a.tokens < 0 || a.out < 1 || a.in < 1 || a.groups < 1 || a.tokens >= lim || a.out >= lim ||
      a.in >= lim || a.groups > 65535 || a.out * a.in >= lim)
    return MUON_ERR_SHAPE;
  if (a.ld_dy < a.out || a.ld_q < a.in || a.ld_e < (a.in + 31) / 32 || a.ld_w < a.in ||
      a.ld_dy >= lim || a.ld_q >= lim || a.ld_e >= lim || a.ld_w >= lim ||
      a.ld_dy % 8 || a.ld_q % 16 || a.ld_e % 4)
    return MUON_ERR_SHAPE;
  if (a.groups > 1 && (a.stride_w < (a.out - 1) * a.ld_w + a.in || a.stride_w >= (int64_t(1) << 44)))
    return MUON_ERR_SHAPE;
  if (a.accumulate != 0 && a.accumulate != 1) return MUON_ERR_INVALID_ARG;
  if (a.dW == nullptr || (a.groups > 1 && a.offsets == nullptr)) return MUON_ERR_INVALID_ARG;
  const size_t we = a.w_dtype == MUON_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(a.dW) % we || reinterpret_cast<uintptr_t>(a.offsets) % 4 ||
      reinterpret_cast<uintptr_t>(a.status_dev) % 4)
    return MUON_ERR_INVALID_ARG;
  if (a.tokens > 0) {
    if (a.dY == nullptr || a.q == nullptr || a.exps == nullptr) return MUON_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a.dY) % 16 || reinterpret_cast<uintptr_t>(a.q) % 16 ||
        reinterpret_cast<uintptr_t>(a.exps) % 4)
      return MUON_ERR_INVALID_ARG;
  }
  const int64_t gs = a.groups > 1 ? a.stride_w : 0;
  const size_t span_w = (static_cast<size_t>(a.groups - 1) * gs) * we + matrix_span(a.out, a.in, a.ld_w, we);
  if (ranges_overlap(a.dW, span_w, a.dY, matrix_span(a.tokens, a.out, a.ld_dy, 2)) ||
      ranges_overlap(a.dW, span_w, a.q, matrix_span(a.tokens, a.in, a.ld_q, 1)) ||
      ranges_overlap(a.dW, span_w, a.exps, matrix_span(a.tokens, (a.in + 31) / 32, a.ld_e, 1)) ||
      (a.offsets != nullptr && ranges_overlap(a.dW, span_w, a.offsets, (a.groups + 1) * size_t(4))) ||
      (a.status_dev != nullptr && ranges_overlap(a.dW, span_w, a.status_dev, 4)))
    return MUON_ERR_ALIAS;
  return MUON_OK;
}

}  // namespace
}  // namespace muon

extern "C" MUON_API size_t muon_weight_grad_workspace_size(const muon_weight_grad_t* a) {
  (void)a;
  return 0;
}

extern "C" MUON_API muon_status_t muon_weight_grad(const muon_weight_grad_t* a, void* workspace,
                                                   size_t ws_bytes, void* stream) {
  using namespace muon;
  (void)workspace;
  (void)ws_bytes;
  const muon_status_t v = validate_weight_grad(a);
  if (v != MUON_OK) return v;
  int dev = 0, sms = 0;
  const muon_status_t d = current_device(&dev, &sms);
  if (d != MUON_OK) return d;
  const int64_t ti = (a->out + kTile - 1) / kTile, tj = (a->in + kTile - 1) / kTile;
  if (ti > 65535) return MUON_ERR_SHAPE;
  wgrad_simple_kernel<<<dim3(tj, ti, a->groups), 256, 0, static_cast<cudaStream_t>(stream)>>>(*a);
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

// Host validation and device helpers shared by the forward and the backward pass.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "muon.h"
#include "umma.cuh"

namespace muon {

// Host checks of an attention call (no CUDA call); backward: the gradients' tensors too.
muon_status_t validate_attention(const muon_attention_t* a, bool backward);

// Two fp32 values rounded to bf16, the first in the low half, in one instruction.
__device__ __forceinline__ uint32_t round_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One sequence's rows and keys, clamped to the tensors.
struct SeqRange {
  int32_t q0, m;  // first query row, queries
  int32_t k0, n;  // first key, keys
};

__device__ __forceinline__ int32_t clamp_offset(const int32_t* off, int i, int32_t tokens) {
  const int32_t v = __ldg(off + i);
  return v < 0 ? 0 : v > tokens ? tokens : v;
}

__device__ __forceinline__ SeqRange seq_range(const muon_attention_t& a, int s) {
  const int32_t qt = static_cast<int32_t>(a.q_tokens), kt = static_cast<int32_t>(a.k_tokens);
  SeqRange r{0, qt, 0, kt};
  // (a single sequence may have either of the two)
  if (a.q_offsets != nullptr) {
    r.q0 = clamp_offset(a.q_offsets, s, qt);
    r.m = clamp_offset(a.q_offsets, s + 1, qt) - r.q0;
  }
  if (a.k_offsets != nullptr) {
    r.k0 = clamp_offset(a.k_offsets, s, kt);
    r.n = clamp_offset(a.k_offsets, s + 1, kt) - r.k0;
  }
  if (r.m < 0) r.m = 0;
  if (r.n < 0) r.n = 0;
  return r;
}

// The sequence of block t of `slots`, and the first row (or, by_keys, key) of its tile of `rows`;
// every warp calls it whole. A tile that starts past its sequence's end has no work.
//
// Up to 32 sequences, one to a lane: tiles in the order of falling level, a tile's level being
// its index (by_keys: counted from the last), which is what a causal tile's work grows with, so
// that the long tiles start first. With c(l) tiles of level l and above, block t has the level l
// with c(l + 1) <= t < c(l), found by bisection with one warp sum a step.
// More sequences: sequence s owns the slots from off[s] / rows + s on, which is enough for its
// ceil(len / rows) tiles (floor(e / rows) - floor(b / rows) + 1 >= ceil((e - b) / rows)), so a
// block finds it by bisection over the offsets, without a prefix sum or a table.
__device__ __forceinline__ SeqRange find_tile(const muon_attention_t& a, bool by_keys, int rows, int t, int slots,
                                              int lane, int* row0) {
  const int32_t* off = by_keys ? a.k_offsets : a.q_offsets;
  const int32_t tokens = static_cast<int32_t>(by_keys ? a.k_tokens : a.q_tokens);
  if (off == nullptr) {
    *row0 = (by_keys ? t : slots - 1 - t) * rows;
    return seq_range(a, 0);
  }
  if (a.n_seq <= 32) {
    SeqRange r{0, 0, 0, 0};
    if (lane < a.n_seq) r = seq_range(a, lane);
    const int tiles = ((by_keys ? r.n : r.m) + rows - 1) / rows;
    auto count = [&](int l) { return __reduce_add_sync(0xffffffffu, tiles > l ? tiles - l : 0); };
    int lo = 0, hi = __reduce_max_sync(0xffffffffu, tiles);  // count(hi) = 0
    if (count(0) <= t) {
      *row0 = 0x7FFFFFFF;  // past the last tile
      return r;
    }
    int above = 0;  // count(hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1, c = count(mid);
      if (c > t) {
        lo = mid;
      } else {
        hi = mid;
        above = c;
      }
    }
    unsigned have = __ballot_sync(0xffffffffu, tiles > lo);
    for (int k = t - above; k > 0; --k) have &= have - 1;  // the (t - above)-th of these sequences
    const int s = __ffs(have) - 1;
    r.q0 = __shfl_sync(0xffffffffu, r.q0, s);
    r.m = __shfl_sync(0xffffffffu, r.m, s);
    r.k0 = __shfl_sync(0xffffffffu, r.k0, s);
    r.n = __shfl_sync(0xffffffffu, r.n, s);
    const int mine = __shfl_sync(0xffffffffu, tiles, s);
    *row0 = (by_keys ? mine - 1 - lo : lo) * rows;
    return r;
  }
  if (!by_keys) t = slots - 1 - t;
  int lo = 0, hi = a.n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (clamp_offset(off, mid, tokens) / rows + mid <= t) lo = mid; else hi = mid - 1;
  }
  // slots below the first sequence's (its offset may be past 0) have no tile
  const int tile = t - (clamp_offset(off, lo, tokens) / rows + lo);
  *row0 = tile < 0 ? 0x7FFFFFFF : tile * rows;
  return seq_range(a, lo);
}

// Writes W accumulator columns (W / 8 16-byte units) of a warp's 32 rows, times each lane's f
// (0: zeros, whatever the accumulator holds), as bf16: through `tile`, a shared-memory tile of
// 128 rows x 64-column chunks that the warp's rows are free in (128B swizzle), so that
// neighbouring lanes write neighbouring bytes. (Straight from the accumulator every lane writes
// another row: 32 lines an instruction, 5000 cycles for two 128 x 128 results.)
// out: row 0 of the warp, column col0; `rows` of its rows exist, columns of `dim`.
template <int W>
__device__ __forceinline__ void store_rows(uint32_t taddr, uint8_t* tile, int w, int lane, int col0, float f, bool zero,
                                           uint16_t* out, int64_t ld, int rows, int dim) {
  constexpr int kUnits = W / 8, kStep = 32 / kUnits;  // rows a warp writes at a time
  const int row = w * 32 + lane, u0 = col0 / 8;
  uint32_t v[W / 32][32];
  if (!zero) {
#pragma unroll
    for (int c = 0; c < W / 32; ++c) tmem_ld32(taddr + c * 32, v[c]);
    tmem_wait_ld();
  }
  if (zero || f == 0.f) {
#pragma unroll
    for (int c = 0; c < W / 32; ++c)
#pragma unroll
      for (int e = 0; e < 32; ++e) v[c][e] = 0;
  }
#pragma unroll
  for (int c = 0; c < W / 32; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t pk[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        pk[k] = round_bf16x2(__uint_as_float(v[c][8 * e + 2 * k]) * f, __uint_as_float(v[c][8 * e + 2 * k + 1]) * f);
      const int u = u0 + c * 4 + e;
      *reinterpret_cast<uint4*>(tile + (u >> 3) * (128 * 128) + row * 128 + (((u & 7) ^ (row & 7)) << 4)) =
          make_uint4(pk[0], pk[1], pk[2], pk[3]);
    }
  __syncwarp();
  const int r0 = lane / kUnits, u = u0 + lane % kUnits;
  const uint8_t* src = tile + (u >> 3) * (128 * 128) + w * 32 * 128;
  uint16_t* dst = out + r0 * ld + (lane % kUnits) * 8;
  if (u * 8 < dim) {
#pragma unroll
    for (int i = 0; i < 32 / kStep; ++i) {
      const int r = r0 + i * kStep;
      if (r < rows)
        *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src + r * 128 + (((u & 7) ^ (r & 7)) << 4));
      dst += kStep * ld;
    }
  }
}

// Tensor map of tokens x heads x head_dim, boxes of 64 columns of one head x `rows` tokens
// (128B swizzle; columns past head_dim and tokens past the tensor read as zeros). Without
// tokens the map is left alone and must not be used.
bool encode_heads_map(CUtensorMap* out, const muon_heads_t& t, int64_t tokens, int heads, int dim, int rows);

inline int64_t tile_slots(const int32_t* off, int n_seq, int64_t tokens, int rows) {
  return off == nullptr ? (tokens + rows - 1) / rows : tokens / rows + n_seq;
}

cudaError_t launch_attention_forward(const muon_attention_t& a, int dev, cudaStream_t st);
// delta: heads x q_tokens floats of scratch, written by the first kernel, read by the second.
cudaError_t launch_attention_backward(const muon_attention_t& a, float* delta, int dev, cudaStream_t st);

}  // namespace muon

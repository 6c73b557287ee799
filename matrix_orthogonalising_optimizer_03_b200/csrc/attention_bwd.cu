// Backward pass of softmax attention over packed sequences (muon_attention_backward). The
// probabilities are recomputed from the forward pass's log-sum-exp:
//   P = exp(S - lse), delta_i = o_i . dout_i, dS = P (dout V^T - delta)
//   dV = P^T dout, dK = scale dS^T Q, dQ = scale dS K
//
// Two kernels, each of whose outputs is summed by one CTA in a fixed order, so that equal
// calls give equal bits: one per 128 query rows for dQ (and delta), one per 128 keys for dK
// and dV, over all query heads of the key head. S and dout V^T are computed in both: seven
// products instead of five, against fp32 atomics on dQ, whose order changes its sums.
// A thread owns 32 elements of one lane's row. P and dS are rounded to bf16 (at most 2^-8 relative,
// errors of either sign; where a block's whole sum is one product of blocks of 128 it also adds the
// product with the rounding's rest, see kExact) and written back over the scores they came from, where the next product takes them as
// its tensor-memory operand; the transposes that dV and dK need cost nothing, because the second
// kernel computes S^T = K Q^T and (dout V^T)^T = V dout^T to begin with.
// Head dimension 128: 128 x 128 scores at a time, 16 warps, one block on an SM. Per 128 x 128
// scores the products take 1536 cycles (dQ) and 2048 (dK, dV) at the full rate; measured 2420 and
// 3440 over the whole kernels (8192 tokens, causal, 16 heads on 4: 311 and 434 us), the tensor core
// active 66 and 63 % of the time. An M = 128 product whose operands both come
// from shared memory runs at 0.84 of the rate for N = 128, as it reads 8 KB per 64 cycles; the
// rest is the chain product - exponential - product of a block.
// Head dimension 64, large grids: 128 x 64 scores at a time, 8 warps, two blocks on an SM, whose
// chains, starts and ends (about 8000 cycles of a block) overlap. With 128 x 128 scores and one
// block, sequences of 1 to 2311 tokens, 12 heads, took 146 us instead of 112. The exponentials
// alone, taken in both kernels, are 1024 cycles per 128 x 128 scores of each, the products 1280
// and 1536 (S and dP at half of the rate with 64 columns).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "attention.h"
#include "muon.h"
#include "umma.cuh"

namespace muon {
namespace {

constexpr int kRows = 128;            // rows of a dQ tile, keys of a tile of dK and dV
constexpr float kLog2e = 1.4426950408889634f;

// W: keys (dQ) or rows (dK, dV) of a block. With 64 of them, head dimension 64 needs half of the
// tensor memory and of the shared memory, and two thread blocks share an SM.
template <int HD, int W>
struct BwdCfg {
  static constexpr int kCols = W;
  static constexpr int kParts = kCols / 32;                // 32 columns a thread
  static constexpr int kCompute = 4 * kParts;              // warps that compute
  static constexpr int kThreads = 32 * (4 + kCompute);     // and 4 that move and issue
  // Thread blocks on an SM. Two of 384 threads have 80 registers a thread at launch, of which the
  // four warps that move and issue leave some to the others: 128 x 64 + 256 x 88 is the same total.
  static constexpr int kPerSm = W == 64 ? 2 : 1;
  static constexpr uint32_t kTmem = 512 / kPerSm;
  // A thread block whose whole sum is one product (dQ: its rows see at most 128 keys; dK and dV: 128
  // rows of one query head see its keys) also takes the rest of the rounding of P and dS
  // (store_operand): errors of 0.0017 instead of 0.0024. Two blocks an SM leave no registers for it
  // (it spilled: 107 -> 119 us): there a short sequence is off by as much as a long one.
  static constexpr bool kExact = kPerSm == 1;
  static constexpr int kTile = kRows * HD * 2;
  static constexpr int kBlock = kCols * HD * 2;
  static constexpr int kRing3 = 3, kRing2 = 2;  // the operand of two chains, and of one
  static constexpr int kOffRing3 = 2 * kTile;
  static constexpr int kOffRing2 = kOffRing3 + kRing3 * kBlock;
  static constexpr int kOffVec = kOffRing2 + kRing2 * kBlock;  // lse and delta of a block of rows
  static constexpr int kVecBytes = 2 * kCols * 4;
  // Blocks of 128 rows of head dimension 64 leave tensor memory for a second S in the kernel of dK
  // and dV, so that the next block's scores are computed during this block's softmax; it then
  // needs lse and delta of three blocks.
  static constexpr bool kTwoS = HD == 64 && W == 128;
  static constexpr int kVecs = kTwoS ? 3 : 2;
  static constexpr int kOffBar = kOffVec + kVecs * kVecBytes;
  static constexpr int kSmemBytes = kOffBar + 512;
  static_assert(kParts * kRows * 4 <= 2 * kVecBytes, "exchange of the parts of delta");
  static_assert(2 * kRows * HD * 4 <= kOffVec, "sums shared by a cluster");
  static_assert(kPerSm * (kSmemBytes + 1024) <= 228 * 1024, "shared memory");
};

struct BwdParams {
  CUtensorMap tq, tk, tv, tdo;
  muon_attention_t a;
  float* delta;
};

__device__ __forceinline__ bool wait_all(uint64_t* bar, int phase, volatile int* abort_flag) {
  const bool got = __all_sync(0xffffffffu, mbar_wait(bar, static_cast<uint32_t>(phase & 1), abort_flag));
  tc_fence_after();
  return got;
}

// Loads kR rows of one head by boxes of HD rows.
template <int HD, int kR>
__device__ __forceinline__ void load_boxes(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int head, int token) {
#pragma unroll
  for (int c = 0; c < HD / 64; ++c)
#pragma unroll
    for (int b = 0; b < kR; b += HD) tma_load_3d(dst + (c * kR + b) * 128, map, bar, c * 64, head, token + b);
}

template <int HD, int W>
__device__ __forceinline__ void load_block(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int head, int token) {
  mbar_expect_tx(bar, BwdCfg<HD, W>::kBlock);
  load_boxes<HD, W>(dst, map, bar, head, token);
}

// Zeros the rows from `live` on of a block in shared memory (one warp): another sequence's rows
// that a product would sum over, with factors of zero but perhaps NaN themselves.
template <int HD, int W>
__device__ __forceinline__ void clear_rows(uint8_t* block, int live, int lane) {
  for (int e = live * 8 + lane; e < W * 8; e += 32)
#pragma unroll
    for (int c = 0; c < HD / 64; ++c)
      *reinterpret_cast<uint4*>(block + c * (W * 128) + e * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

// D = A B^T over the head dimension: a tile and a block in shared memory, both K-major.
template <int HD, int W>
__device__ __forceinline__ void product_ss(uint32_t d, uint32_t a_addr, uint32_t b_addr) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, W, false);
  const uint32_t ad = desc_lo(a_addr, 16), bd = desc_lo(b_addr, 16);
#pragma unroll
  for (int k = 0; k < HD / 16; ++k) {
    const uint32_t c = k >> 2, in = (k & 3) * 2;
    umma_f16_lo(d, ad + c * (kRows * 8) + in, bd + c * (W * 8) + in, kDescHi, idesc, k != 0);
  }
}

// D (+)= A B over the rows or keys of a block: A bf16 in tensor memory (each 32 of them in the
// first 16 of the 32 columns they came from), B an MN-major block in shared memory.
template <int HD, int W>
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a_tmem, uint32_t b_addr, bool accumulate, bool exact) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, HD, true);
  const uint32_t bd = desc_lo(b_addr, W * 128);
#pragma unroll
  for (int k = 0; k < W / 16; ++k)
    umma_f16_ts_lo(d, a_tmem + (k >> 1) * 32 + (k & 1) * 8, bd + 128u * k, kDescHi, idesc, accumulate || k != 0);
  if (exact)  // and the rest of A, see store_operand
#pragma unroll
    for (int k = 0; k < W / 16; ++k)
      umma_f16_ts_lo(d, a_tmem + (k >> 1) * 32 + (k & 1) * 8 + 16, bd + 128u * k, kDescHi, idesc, true);
}

// Writes 32 values as bf16 into the first 16 columns of a thread's 32, where product_ts takes them;
// with `exact`, what their rounding left as bf16 into the other 16.
__device__ __forceinline__ void store_operand(uint32_t taddr, const uint32_t (&x)[32], bool exact) {
  uint32_t pk[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) pk[e] = round_bf16x2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
  tmem_st16(taddr, pk);
  if (exact) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      pk[e] = round_bf16x2(__uint_as_float(x[2 * e]) - __uint_as_float(pk[e] << 16),
                           __uint_as_float(x[2 * e + 1]) - __uint_as_float(pk[e] & 0xFFFF0000u));
    tmem_st16(taddr + 16, pk);
  }
  tmem_wait_st();
}

// Whether the probability of a row's lone key is 1 up to the rounding of its exponent (lse in units
// of log 2, rounded a few times). Then o is the key's v and dS = 0: taken so, dQ of such a row is
// zero to the last bit, not the difference of two sums of o . dout. (Not so where a caller passes
// the lse of more keys than these.)
__device__ __forceinline__ bool is_one(float p, float lse) {
  return fabsf(p - 1.f) <= fmaf(fabsf(lse), 0x1p-21f, 0x1p-21f);
}

// ------------------------------------------------------------------ dQ and delta
// Chain A: S_j = Q K_j^T (two buffers), dQ += dS_j K_j.  Chain B: dP_j = dout V_j^T.
template <int HD, int W>
__global__ void __launch_bounds__(BwdCfg<HD, W>::kThreads, BwdCfg<HD, W>::kPerSm) attention_dq_kernel(const __grid_constant__ BwdParams P) {
  using C = BwdCfg<HD, W>;
  const muon_attention_t& a = P.a;
  const int heads = a.heads, head = static_cast<int>(blockIdx.x % heads);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  int row0;
  const SeqRange r = find_tile(a, false, kRows, static_cast<int>(blockIdx.x / heads), static_cast<int>(gridDim.x / heads),
                               lane, &row0);
  if (row0 >= r.m) return;
  const int shift = r.n - r.m;  // causal: row i sees keys j <= i + shift
  const int keys = a.causal ? min(r.n, min(row0 + kRows, r.m) + shift) : r.n;
  const int n = keys > 0 ? (keys + C::kCols - 1) / C::kCols : 0;  // key blocks

  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* k_full = q_full + 1;    // ring of K blocks
  uint64_t* k_empty = k_full + 3;
  uint64_t* v_full = k_empty + 3;   // ring of V blocks
  uint64_t* v_empty = v_full + 2;
  uint64_t* s_full = v_empty + 2;   // per block parity
  uint64_t* dp_full = s_full + 2;
  uint64_t* dp_read = dp_full + 1;
  uint64_t* ds_full = dp_read + 1;  // per block parity
  uint64_t* turn = ds_full + 2;     // per half of the parts and lane quarter: exponentials done
  uint64_t* done = turn + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t *sq = smem, *sdo = smem + C::kTile, *sk = smem + C::kOffRing3, *sv = smem + C::kOffRing2;
  const int kvh = head / (heads / a.kv_heads);

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < 3; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&ds_full[s], C::kCompute);
    }
    for (int e = 0; e < 8; ++e) mbar_init(&turn[e], 2);
    mbar_init(dp_full, 1);
    mbar_init(dp_read, C::kCompute);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    // the first blocks are on their way before the other warps are set up
    mbar_expect_tx(q_full, 2 * C::kTile);
    load_boxes<HD, kRows>(sq, &P.tq, q_full, head, r.q0 + row0);
    load_boxes<HD, kRows>(sdo, &P.tdo, q_full, head, r.q0 + row0);
    if (n > 0) {
      load_block<HD, W>(sk, &P.tk, &k_full[0], kvh, r.k0);
      load_block<HD, W>(sv, &P.tv, &v_full[0], kvh, r.k0);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  constexpr uint32_t kDp = 2 * C::kCols, kDq = 3 * C::kCols;  // columns of dP and dQ; S at kCols (j & 1)
  bool ok = true;
  if (C::kPerSm == 2 && warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");  // see kPerSm

  if (warp == 0) {
    if (lane == 0) {
      int kl = n > 0, vl = kl;
      for (int j = 1; j < n; ++j) {
        ok = mbar_wait(&k_empty[j % 3], static_cast<uint32_t>((j / 3) & 1) ^ 1u, abort_flag);
        if (!ok) break;
        load_block<HD, W>(sk + j % 3 * C::kBlock, &P.tk, &k_full[j % 3], kvh, r.k0 + j * C::kCols);
        ++kl;
        ok = mbar_wait(&v_empty[j & 1], static_cast<uint32_t>((j >> 1) & 1) ^ 1u, abort_flag);
        if (!ok) break;
        load_block<HD, W>(sv + (j & 1) * C::kBlock, &P.tv, &v_full[j & 1], kvh, r.k0 + j * C::kCols);
        ++vl;
      }
      // never leave with bulk copies still landing in shared memory
      mbar_wait(q_full, 0, nullptr);
      for (int j = kl > 3 ? kl - 3 : 0; j < kl; ++j) mbar_wait(&k_full[j % 3], static_cast<uint32_t>((j / 3) & 1), nullptr);
      for (int j = vl > 2 ? vl - 2 : 0; j < vl; ++j) mbar_wait(&v_full[j & 1], static_cast<uint32_t>((j >> 1) & 1), nullptr);
    }
  } else if (warp == 1) {
    if (n > 0) {
      auto score = [&](int j) {  // S_j; the buffer's dS_{j-2} went into a product issued before
        if (!wait_all(&k_full[j % 3], j / 3, abort_flag)) return false;
        const int live = r.n - j * C::kCols;
        if (live < C::kCols) clear_rows<HD, W>(sk + j % 3 * C::kBlock, live, lane);
        if (elect_one()) {
          product_ss<HD, W>(tmem + (j & 1) * C::kCols, smem_u32(sq), smem_u32(sk) + j % 3 * C::kBlock);
          umma_commit(&s_full[j & 1]);
        }
        return true;
      };
      ok = wait_all(q_full, 0, abort_flag) && score(0) && (n < 2 || score(1));
      for (int j = 0; j < n && ok; ++j) {
        ok = wait_all(&ds_full[j & 1], j >> 1, abort_flag);
        if (!ok) break;
        if (elect_one()) {
          product_ts<HD, W>(tmem + kDq, tmem + (j & 1) * C::kCols, smem_u32(sk) + j % 3 * C::kBlock, j > 0, C::kExact && n == 1);
          umma_commit(&k_empty[j % 3]);
          if (j + 1 == n) umma_commit(done);
        }
        if (j + 2 < n) ok = score(j + 2);
      }
      ok = ok && wait_all(done, 0, abort_flag);  // never leave with products still running
    }
  } else if (warp == 2) {
    if (n > 0) {
      ok = wait_all(q_full, 0, abort_flag);
      for (int j = 0; j < n && ok; ++j) {
        ok = wait_all(&v_full[j & 1], j >> 1, abort_flag) && (j == 0 || wait_all(dp_read, j - 1, abort_flag));
        if (ok && elect_one()) {
          product_ss<HD, W>(tmem + kDp, smem_u32(sdo), smem_u32(sv) + (j & 1) * C::kBlock);
          umma_commit(dp_full);
          umma_commit(&v_empty[j & 1]);
        }
      }
      ok = ok && wait_all(dp_full, n - 1, abort_flag);
    }
  } else if (warp >= 4) {
    if (C::kPerSm == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
    const int w = warp & 3, part = (warp - 4) >> 2;     // lane quarter, and 32 of a block's keys
    const int row = row0 + w * 32 + lane;               // within the sequence
    const bool live = row < r.m;
    const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
    const int64_t token = r.q0 + row, vec = static_cast<int64_t>(head) * a.q_tokens + token;
    // delta = o . dout: the threads of a row sum a share of the columns each, dout from its tile in
    // shared memory
    float lse = INFINITY;  // of rows without keys, or none: P = 0
    float sum[4] = {};
    {
      constexpr int kUnits = HD / 8 / C::kParts;
      uint4 o[kUnits];
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.o.ptr) + token * a.o.ld + head * a.o.head);
#pragma unroll
      for (int c = 0; c < kUnits; ++c)
        o[c] = live && (part * kUnits + c) * 8 < a.head_dim ? __ldg(src + part * kUnits + c) : make_uint4(0, 0, 0, 0);
      if (live) {
        const float l = __ldg(a.lse + vec);
        if (l != -INFINITY) lse = l * kLog2e;
      }
      ok = wait_all(q_full, 0, abort_flag);
      const int rt = w * 32 + lane;
#pragma unroll
      for (int c = 0; c < kUnits; ++c) {
        const int u = part * kUnits + c;
        const uint4 g = *reinterpret_cast<const uint4*>(sdo + (u >> 3) * (kRows * 128) + rt * 128 + (((u & 7) ^ (rt & 7)) << 4));
        const uint32_t xs[4] = {o[c].x, o[c].y, o[c].z, o[c].w}, ys[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum[e] = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), sum[e]);
          sum[e] = fmaf(__uint_as_float(xs[e] & 0xFFFF0000u), __uint_as_float(ys[e] & 0xFFFF0000u), sum[e]);
        }
      }
    }
    float* exchange = reinterpret_cast<float*>(smem + C::kOffVec) + w * 32 + lane;
    exchange[part * kRows] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    named_barrier(1, 32 * C::kCompute);
    float delta = exchange[0] + exchange[kRows];
    if (C::kParts > 2) delta += exchange[2 * kRows] + exchange[3 * kRows];
    if (live && part == 0) P.delta[vec] = delta;
    const float sl = a.scale * kLog2e;
    for (int j = 0; j < n && ok; ++j) {
      ok = wait_all(&s_full[j & 1], j >> 1, abort_flag);
      if (!ok) break;
      const uint32_t ts = tmem + lanes + (j & 1) * C::kCols + part * 32;
      uint32_t s[32], p[32];
      tmem_ld32(ts, s);
      tmem_wait_ld();
      // keys of this part of the block that the row sees
      const int vis = min(r.n, a.causal ? row + shift + 1 : r.n) - j * C::kCols - part * 32;
      const bool masked = __any_sync(0xffffffffu, vis < 32);
      // With one block on the SM, two of the four warps of a scheduler take turns with the other two
      // at the exponentials: one pair's other work overlaps the other's. (Two blocks overlap by
      // themselves: 408 us with turns, 398 without, 8192 tokens, 12 heads of 64, causal.)
      const int grp = part >> 1;
      if (C::kPerSm == 1 && (grp == 1 || j > 0)) ok = wait_all(&turn[4 * (1 - grp) + w], grp == 1 ? j : j - 1, abort_flag);
      if (!ok) break;
#pragma unroll
      for (int e = 0; e < 32; ++e) s[e] = __float_as_uint(ex2(fmaf(__uint_as_float(s[e]), sl, -lse)));
      if (j == 0 && part == 0 && vis == 1 && is_one(__uint_as_float(s[0]), lse)) s[0] = 0;
      __syncwarp();
      if (C::kPerSm == 1 && lane == 0) mbar_arrive(&turn[4 * grp + w]);
      ok = wait_all(dp_full, j, abort_flag);
      if (!ok) break;
      tmem_ld32(tmem + lanes + kDp + part * 32, p);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dp_read);
#pragma unroll
      for (int e = 0; e < 32; ++e) s[e] = __float_as_uint(__uint_as_float(s[e]) * (__uint_as_float(p[e]) - delta));
      if (masked) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (e >= vis) s[e] = 0;
      }
      store_operand(ts, s, C::kExact && n == 1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ds_full[j & 1]);
    }
    if (ok && n > 0) ok = wait_all(done, 0, abort_flag);
    // staged where Q was: its products are complete
    if (part < HD / 32)
      store_rows<32>(tmem + lanes + kDq + part * 32, sq, w, lane, part * 32, a.scale, n == 0,
                     static_cast<uint16_t*>(a.dq.ptr) + (r.q0 + row0 + w * 32) * a.dq.ld + head * a.dq.head + part * 32, a.dq.ld,
                     ok ? r.m - row0 - w * 32 : 0, a.head_dim);
    tc_fence_before();
  }
  if (!ok && lane == 0) {
    set_error(a.status_dev, MUON_ERR_TIMEOUT);
    *abort_flag = 1;
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// ------------------------------------------------------------------ dK and dV
// Sums shared by a cluster: dV and dK of a key tile in fp32, 128 rows x HD each, over the block's
// shared memory from its start (its products are complete). 16-byte units are swizzled by the row.
template <int HD>
__device__ __forceinline__ uint32_t sum_offset(int tensor, int row, int unit) {
  return static_cast<uint32_t>(((tensor * kRows + row) * (HD / 4) + (unit ^ (row & 7))) * 16);
}

// A thread's share of its row: kShare columns of dV or dK, from `col` on.
template <int HD, int kShare>
__device__ __forceinline__ void leave_sums(uint8_t* smem, uint32_t taddr, int tensor, int col, int row, bool zero) {
#pragma unroll
  for (int c = 0; c < kShare; c += 32) {
    uint32_t v[32];
    if (!zero) {
      tmem_ld32(taddr + col + c, v);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = 0;
    }
#pragma unroll
    for (int e = 0; e < 32; e += 4)
      *reinterpret_cast<uint4*>(smem + sum_offset<HD>(tensor, row, (col + c + e) / 4)) =
          make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
  }
}

__device__ __forceinline__ float4 load_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// Adds rows rank * 128 / split .. of both tensors over the cluster's blocks, in their order, and
// writes them: thread t of 32 kCompute takes 8 columns at a time. Of the tile's rows `rows` exist.
template <int HD, int W>
__device__ __forceinline__ void join_sums(const uint8_t* smem, const muon_attention_t& a, int split, int rank, int t, int kvh,
                                          int64_t token0, int rows) {
  const int mine = kRows / split, total = 2 * mine * (HD / 8);
  for (int i = t; i < total; i += 32 * BwdCfg<HD, W>::kCompute) {
    const int u = i % (HD / 8), row = rank * mine + i / (HD / 8) % mine, tensor = i / (HD / 8) / mine;
    if (row >= rows || u * 8 >= a.head_dim) continue;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    for (int c = 0; c < split; ++c) {
      const uint32_t base = peer_addr(smem, static_cast<uint32_t>(c));
      const float4 p = load_cluster_f4(base + sum_offset<HD>(tensor, row, 2 * u));
      const float4 q = load_cluster_f4(base + sum_offset<HD>(tensor, row, 2 * u + 1));
      x.x += p.x; x.y += p.y; x.z += p.z; x.w += p.w;
      y.x += q.x; y.y += q.y; y.z += q.z; y.w += q.w;
    }
    const float f = tensor == 0 ? 1.f : a.scale;
    const muon_heads_t& out = tensor == 0 ? a.dv : a.dk;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out.ptr) + (token0 + row) * out.ld + kvh * out.head + u * 8) =
        make_uint4(round_bf16x2(x.x * f, x.y * f), round_bf16x2(x.z * f, x.w * f), round_bf16x2(y.x * f, y.y * f),
                   round_bf16x2(y.z * f, y.w * f));
  }
}

// S^T_j = K Q_j^T, dP^T_j = V dout_j^T, dV += P^T_j dout_j, dK += dS^T_j Q_j.
// Block j runs over the row tiles that see the keys, head after head. With several query heads to
// a key head and few tiles, a cluster shares the heads (dkv_split): each block leaves its sums in
// its shared memory, and each then adds a share of the rows over all blocks, in their order.
template <int HD, int W>
__global__ void __launch_bounds__(BwdCfg<HD, W>::kThreads, BwdCfg<HD, W>::kPerSm) attention_dkv_kernel(const __grid_constant__ BwdParams P) {
  using C = BwdCfg<HD, W>;
  const muon_attention_t& a = P.a;
  const int split = static_cast<int>(cluster_num_ctas()), rank = static_cast<int>(cluster_cta_rank());
  const int block = static_cast<int>(blockIdx.x) / split;
  const int kvh = block % a.kv_heads, per = a.heads / a.kv_heads / split;
  const int head0 = (kvh * split + rank) * per;  // this block's query heads: head0 .. head0 + per - 1
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  int key0;
  const SeqRange r = find_tile(a, true, kRows, block / a.kv_heads, static_cast<int>(gridDim.x) / split / a.kv_heads, lane, &key0);
  if (key0 >= r.n) return;
  const int shift = r.n - r.m;
  const int tile0 = a.causal ? max(0, key0 - shift) / C::kCols : 0;  // the first block of rows that sees a key
  const int tiles = max(0, (r.m + C::kCols - 1) / C::kCols - tile0), n = tiles * per;

  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_full = kv_full + 1;    // ring of Q blocks: landed
  uint64_t* q_ready = q_full + 3;    // and with rows past the sequence cleared, lse and delta in place
  uint64_t* q_empty = q_ready + 3;
  uint64_t* do_full = q_empty + 3;   // ring of dout blocks
  uint64_t* do_ready = do_full + 2;
  uint64_t* do_empty = do_ready + 2;
  uint64_t* s_full = do_empty + 2;   // per block parity (two S), as p_full
  uint64_t* p_full = s_full + 2;
  uint64_t* dp_full = p_full + 2;
  uint64_t* ds_full = dp_full + 1;
  uint64_t* done = ds_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t *sk = smem, *sv = smem + C::kTile, *sq = smem + C::kOffRing3, *sdo = smem + C::kOffRing2;

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < 3; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_ready[s], 1);
      mbar_init(&q_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&do_full[s], 1);
      mbar_init(&do_ready[s], 1);
      mbar_init(&do_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], C::kCompute);
    }
    mbar_init(dp_full, 1);
    mbar_init(ds_full, C::kCompute);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    // the first blocks are on their way before the other warps are set up
    if (n > 0) {
      mbar_expect_tx(kv_full, 2 * C::kTile);
      load_boxes<HD, kRows>(sk, &P.tk, kv_full, kvh, r.k0 + key0);
      load_boxes<HD, kRows>(sv, &P.tv, kv_full, kvh, r.k0 + key0);
      load_block<HD, W>(sq, &P.tq, &q_full[0], head0, r.q0 + tile0 * C::kCols);
      load_block<HD, W>(sdo, &P.tdo, &do_full[0], head0, r.q0 + tile0 * C::kCols);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  constexpr uint32_t kDp = C::kCols, kDv = 2 * C::kCols, kDk = kDv + HD;  // columns; S at 0, and behind them (two S)
  // the S of block j, and barriers that may complete for the next block before this one's wait
  auto s_col = [](int j) { return C::kTwoS && (j & 1) ? kDk + HD : 0u; };
  auto s_par = [](int j) { return C::kTwoS ? j & 1 : 0; };
  auto s_phase = [](int j) { return C::kTwoS ? j >> 1 : j; };
  bool ok = true;
  if (C::kPerSm == 2 && warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");  // see kPerSm

  if (warp == 0) {
    if (lane == 0 && n > 0) {
      int ql = 1, dl = 1, h = head0, t = tile0;
      if (++t == tile0 + tiles) t = tile0, ++h;
      for (int j = 1; j < n; ++j) {
        ok = mbar_wait(&q_empty[j % 3], static_cast<uint32_t>((j / 3) & 1) ^ 1u, abort_flag);
        if (!ok) break;
        load_block<HD, W>(sq + j % 3 * C::kBlock, &P.tq, &q_full[j % 3], h, r.q0 + t * C::kCols);
        ++ql;
        ok = mbar_wait(&do_empty[j & 1], static_cast<uint32_t>((j >> 1) & 1) ^ 1u, abort_flag);
        if (!ok) break;
        load_block<HD, W>(sdo + (j & 1) * C::kBlock, &P.tdo, &do_full[j & 1], h, r.q0 + t * C::kCols);
        ++dl;
        if (++t == tile0 + tiles) t = tile0, ++h;
      }
      // never leave with bulk copies still landing in shared memory
      mbar_wait(kv_full, 0, nullptr);
      for (int j = ql > 3 ? ql - 3 : 0; j < ql; ++j) mbar_wait(&q_full[j % 3], static_cast<uint32_t>((j / 3) & 1), nullptr);
      for (int j = dl > 2 ? dl - 2 : 0; j < dl; ++j) mbar_wait(&do_full[j & 1], static_cast<uint32_t>((j >> 1) & 1), nullptr);
    }
  } else if (warp == 1) {
    // One issuer keeps the order dV_j, S_{j+1} (two S: S_{j+2}), dK_j, dP_{j+1}: S_{j+1} is what the
    // softmax waits for next. Issued by two warps, the two chains share the tensor core evenly and S_{j+1} came 600
    // cycles later.
    if (n > 0) {
      auto score = [&](int j) {  // S^T_j; the P^T before it in these columns went into an earlier product
        if (!wait_all(&q_ready[j % 3], j / 3, abort_flag)) return false;
        if (elect_one()) {
          product_ss<HD, W>(tmem + s_col(j), smem_u32(sk), smem_u32(sq) + j % 3 * C::kBlock);
          umma_commit(&s_full[s_par(j)]);
        }
        return true;
      };
      auto dprob = [&](int j) {  // dP^T_j; dS^T_{j-1} over it went into a product issued before
        if (!wait_all(&do_ready[j & 1], j >> 1, abort_flag)) return false;
        if (elect_one()) {
          product_ss<HD, W>(tmem + kDp, smem_u32(sv), smem_u32(sdo) + (j & 1) * C::kBlock);
          umma_commit(dp_full);
        }
        return true;
      };
      ok = wait_all(kv_full, 0, abort_flag) && score(0) && dprob(0) && (!C::kTwoS || n < 2 || score(1));
      for (int j = 0; j < n && ok; ++j) {
        ok = wait_all(&p_full[s_par(j)], s_phase(j), abort_flag);
        if (!ok) break;
        if (elect_one()) {
          product_ts<HD, W>(tmem + kDv, tmem + s_col(j), smem_u32(sdo) + (j & 1) * C::kBlock, j > 0, C::kExact && n == 1);
          umma_commit(&do_empty[j & 1]);
        }
        constexpr int ahead = C::kTwoS ? 2 : 1;
        if (j + ahead < n) ok = score(j + ahead);
        ok = ok && wait_all(ds_full, j, abort_flag);
        if (!ok) break;
        if (elect_one()) {
          product_ts<HD, W>(tmem + kDk, tmem + kDp, smem_u32(sq) + j % 3 * C::kBlock, j > 0, C::kExact && n == 1);
          umma_commit(&q_empty[j % 3]);
          if (j + 1 == n) umma_commit(done);
        }
        if (j + 1 < n) ok = dprob(j + 1);
      }
      ok = ok && wait_all(done, 0, abort_flag);  // never leave with products still running
    }
  } else if (warp == 3) {
    // Stages what the copies do not bring: lse (times log2 e) and delta of the block's rows, and
    // zeros over the rows past the sequence. Such rows, and rows that see no key, get lse = inf:
    // P = 0.
    int h = head0, t = tile0;
    for (int j = 0; j < n; ++j) {
      const int live = r.m - t * C::kCols;
      const int64_t at = static_cast<int64_t>(h) * a.q_tokens + r.q0 + t * C::kCols;
      float l[C::kParts], d[C::kParts];
#pragma unroll
      for (int e = 0; e < C::kParts; ++e) {
        const int i = e * 32 + lane;
        const float x = i < live ? __ldg(a.lse + at + i) : -INFINITY;
        l[e] = x == -INFINITY ? INFINITY : x * kLog2e;
        d[e] = i < live ? P.delta[at + i] : 0.f;
      }
      // With two of these vectors, block j - 2 is done with its own once its last product is
      // complete; with three, the copy of Q_j came after that of block j - 3.
      ok = wait_all(&q_full[j % 3], j / 3, abort_flag) &&
           (C::kVecs == 3 || j < 2 || wait_all(&q_empty[(j - 2) % 3], (j - 2) / 3, abort_flag));
      if (!ok) break;
      float* v = reinterpret_cast<float*>(smem + C::kOffVec + j % C::kVecs * C::kVecBytes);
#pragma unroll
      for (int e = 0; e < C::kParts; ++e) {
        v[e * 32 + lane] = l[e];
        v[C::kCols + e * 32 + lane] = d[e];
      }
      if (live < C::kCols) clear_rows<HD, W>(sq + j % 3 * C::kBlock, live, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_ready[j % 3]);
      ok = wait_all(&do_full[j & 1], j >> 1, abort_flag);
      if (!ok) break;
      if (live < C::kCols) clear_rows<HD, W>(sdo + (j & 1) * C::kBlock, live, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&do_ready[j & 1]);
      if (++t == tile0 + tiles) t = tile0, ++h;
    }
  } else if (warp >= 4) {
    if (C::kPerSm == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
    const int w = warp & 3, part = (warp - 4) >> 2;     // lane quarter, and 32 of a block's rows
    const int key = key0 + w * 32 + lane;               // within the sequence
    const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
    const float sl = a.scale * kLog2e;
    int t = tile0;
    for (int j = 0; j < n; ++j) {
      ok = wait_all(&q_ready[j % 3], j / 3, abort_flag) && wait_all(&s_full[s_par(j)], s_phase(j), abort_flag);
      if (!ok) break;
      const float4* lse = reinterpret_cast<const float4*>(smem + C::kOffVec + j % C::kVecs * C::kVecBytes) + part * 8;
      const float4* dlt = lse + C::kCols / 4;
      const uint32_t ts = tmem + lanes + s_col(j) + part * 32, tp = tmem + lanes + kDp + part * 32;
      uint32_t s[32], p[32];
      tmem_ld32(ts, s);
      tmem_wait_ld();
      // the first row of this part of the block that sees the key (rows are columns here)
      const int first = a.causal ? key - shift - t * C::kCols - part * 32 : 0;
      // and those, [lone, lone_end), that see key 0 alone (is_one)
      const int lone = (a.causal ? max(0, -shift) : 0) - t * C::kCols - part * 32;
      const int lone_end = key0 > 0 ? -1 : (r.n == 1 ? r.m : a.causal ? 1 - shift : 0) - t * C::kCols - part * 32;
      if (++t == tile0 + tiles) t = tile0;
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 l = lse[e / 4];
        s[e] = __float_as_uint(ex2(fmaf(__uint_as_float(s[e]), sl, -l.x)));
        s[e + 1] = __float_as_uint(ex2(fmaf(__uint_as_float(s[e + 1]), sl, -l.y)));
        s[e + 2] = __float_as_uint(ex2(fmaf(__uint_as_float(s[e + 2]), sl, -l.z)));
        s[e + 3] = __float_as_uint(ex2(fmaf(__uint_as_float(s[e + 3]), sl, -l.w)));
      }
      if (__any_sync(0xffffffffu, first > 0)) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (e < first) s[e] = 0;
      }
      store_operand(ts, s, C::kExact && n == 1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[s_par(j)]);
      if (lone < 32 && lone_end > max(lone, 0)) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (e >= lone && e < lone_end && is_one(__uint_as_float(s[e]), reinterpret_cast<const float*>(lse)[e])) s[e] = 0;
      }
      ok = wait_all(dp_full, j, abort_flag);
      if (!ok) break;
      tmem_ld32(tp, p);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 d = dlt[e / 4];
        s[e] = __float_as_uint(__uint_as_float(s[e]) * (__uint_as_float(p[e]) - d.x));
        s[e + 1] = __float_as_uint(__uint_as_float(s[e + 1]) * (__uint_as_float(p[e + 1]) - d.y));
        s[e + 2] = __float_as_uint(__uint_as_float(s[e + 2]) * (__uint_as_float(p[e + 2]) - d.z));
        s[e + 3] = __float_as_uint(__uint_as_float(s[e + 3]) * (__uint_as_float(p[e + 3]) - d.w));
      }
      store_operand(tp, s, C::kExact && n == 1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_full);
    }
    if (ok && n > 0) ok = wait_all(done, 0, abort_flag);
    // half of the parts write dV, half dK
    constexpr int kShare = 2 * HD / C::kParts;
    const int tensor = part / (C::kParts / 2), col = part % (C::kParts / 2) * kShare;
    const uint32_t acc = tmem + lanes + (tensor == 0 ? kDv : kDk);
    if (split > 1) {
      leave_sums<HD, kShare>(smem, acc, tensor, col, w * 32 + lane, n == 0);
    } else {
      // staged where V and K were: their products are complete
      const muon_heads_t& out = tensor == 0 ? a.dv : a.dk;
      store_rows<kShare>(acc + col, tensor == 0 ? sv : sk, w, lane, col, tensor == 0 ? 1.f : a.scale, n == 0,
                         static_cast<uint16_t*>(out.ptr) + (r.k0 + key0 + w * 32) * out.ld + kvh * out.head + col, out.ld,
                         ok ? r.n - key0 - w * 32 : 0, a.head_dim);
    }
    tc_fence_before();
  }
  if (!ok && lane == 0) {
    set_error(a.status_dev, MUON_ERR_TIMEOUT);
    *abort_flag = 1;
  }
  __syncthreads();
  if (split > 1) {
    cluster_sync_all();
    if (warp >= 4)
      join_sums<HD, W>(smem, a, split, rank, static_cast<int>(threadIdx.x) - 128, kvh, r.k0 + key0, r.n - key0);
    cluster_sync_all();  // nobody leaves while its sums are read
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// Blocks that share a key tile's query heads: as many (a power of two that divides them, at most
// 4: a block takes a whole SM, and larger clusters leave SMs of a GPC over) as it takes to give
// every SM three blocks. Few key heads would otherwise leave SMs idle, and the long tiles of a
// causal sequence make them wait; more blocks only repeat the loads of K and V and the joins.
// The whole backward pass at 8192 tokens, causal, split against not: 4 query heads on 1 key head
// 218 against 504 us, 16 on 4 757 against 759 us (head dimension 96: 798 against 738).
int dkv_split(const muon_attention_t& a, int64_t grid) {
  int split = 1;
  while (split < 4 && (a.heads / a.kv_heads) % (2 * split) == 0 && grid * split < 3 * 148) split *= 2;
  return split;
}

// Head dimension 64: blocks of 64 columns, two of them on an SM, where a grid gives every SM more
// than two; else blocks of 128, whose chain is shorter per column. Both kernels of causal
// sequences, 64 against 128 columns: 4096 tokens and 8 heads (264 blocks) 125 against 93 us, 12 heads
// (396) 134 against 142, 24 heads (792) 229 against 257.
bool narrow(int64_t grid) { return grid > 2 * 148; }

template <class C>
cudaError_t launch(void (*kernel)(BwdParams), std::atomic<uint64_t>& attr_devices, const BwdParams& P, int dev, int64_t grid,
                   int cluster, cudaStream_t st) {
  static_assert(C::kSmemBytes <= 227 * 1024, "shared memory");
  // function attributes are per device: set them once on each device
  const uint64_t bit = dev < 64 ? (uint64_t{1} << dev) : 0;
  if (bit == 0 || !(attr_devices.load(std::memory_order_acquire) & bit)) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e == cudaSuccess && C::kPerSm > 1)  // all of the SM's memory, so that two blocks fit
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    attr_devices.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, P);
}

template <int HD, int W>
cudaError_t launch_dq(const BwdParams& P, int dev, int64_t grid, cudaStream_t st) {
  static std::atomic<uint64_t> attr_devices{0};
  return launch<BwdCfg<HD, W>>(attention_dq_kernel<HD, W>, attr_devices, P, dev, grid, 1, st);
}

template <int HD, int W>
cudaError_t launch_dkv(const BwdParams& P, int dev, int64_t grid, int split, cudaStream_t st) {
  static std::atomic<uint64_t> attr_devices{0};
  return launch<BwdCfg<HD, W>>(attention_dkv_kernel<HD, W>, attr_devices, P, dev, grid * split, split, st);
}

}  // namespace

cudaError_t launch_attention_backward(const muon_attention_t& a, float* delta, int dev, cudaStream_t st) {
  BwdParams P;
  std::memset(&P, 0, sizeof(P));
  P.a = a;
  P.delta = delta;
  const int box = a.head_dim <= 64 ? 64 : 128;
  if (!encode_heads_map(&P.tq, a.q, a.q_tokens, a.heads, a.head_dim, box) ||
      !encode_heads_map(&P.tdo, a.dout, a.q_tokens, a.heads, a.head_dim, box) ||
      !encode_heads_map(&P.tk, a.k, a.k_tokens, a.kv_heads, a.head_dim, box) ||
      !encode_heads_map(&P.tv, a.v, a.k_tokens, a.kv_heads, a.head_dim, box))
    return cudaErrorInvalidValue;
  const int64_t grid_q = tile_slots(a.q_offsets, a.n_seq, a.q_tokens, kRows) * a.heads;
  const int64_t grid_k = tile_slots(a.k_offsets, a.n_seq, a.k_tokens, kRows) * a.kv_heads;
  if (grid_q >= (int64_t(1) << 31) || grid_k >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  if (a.q_tokens > 0) {
    const cudaError_t e = a.head_dim > 64  ? launch_dq<128, 128>(P, dev, grid_q, st)
                          : narrow(grid_q) ? launch_dq<64, 64>(P, dev, grid_q, st)
                                           : launch_dq<64, 128>(P, dev, grid_q, st);
    if (e != cudaSuccess) return e;
  }
  if (a.k_tokens == 0) return cudaSuccess;
  const int split = dkv_split(a, grid_k);
  return a.head_dim > 64          ? launch_dkv<128, 128>(P, dev, grid_k, split, st)
         : narrow(grid_k * split) ? launch_dkv<64, 64>(P, dev, grid_k, split, st)
                                  : launch_dkv<64, 128>(P, dev, grid_k, split, st);
}

}  // namespace muon

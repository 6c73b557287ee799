// Forward pass of softmax attention over packed sequences, with the log-sum-exp of every row
// and the largest logit of every head (muon_attention_forward).
//
// One pass over the keys with a running maximum and sum per row. A block owns 128 query rows of
// one head:
//   S = Q K^T (fp32 in tensor memory), P = exp2(S scale log2 e - m) as bf16 in tensor memory,
//   O += P V with P as the tensor-memory operand
// Warps: 0 TMA producer (Q once, then K and V blocks through a ring), 1 MMA issuer, 4-7 the
// softmax, one thread per row. Two blocks share an SM (256 columns of tensor memory and half of
// the shared memory each): one's softmax, start and end overlap the other's products. (Two tiles
// in one block of 256 rows, taking turns, needed 10 to 20 % longer for head dimension 128 and
// short sequences, 5 % less for 64.) The next key block's S is computed while this one's softmax
// runs; how tensor memory allows that differs by head dimension (FwdCfg).
// m is the row's running maximum, moved only when a block exceeds it by more than 2^8 in the
// exponent: until then P stays below 2^8 and nothing overflows (fp32 sums, bf16 P), and the
// accumulator, which a thread would have to read and write back, is left alone. P is rounded
// to bf16 for the product (at most 2^-8 relative, errors of either sign); the row's sum adds the
// unrounded values.
// Bounds, per 128 keys of both blocks: head dimension 128 by the products, 2048 cycles at the full
// rate (S, with both operands in shared memory and 64 columns, runs at half of it; 3300 measured
// in a full round of blocks, 1040 to 1110 TFLOP/s at 8191 tokens, 12 heads); head dimension 64 by the exponentials, 16 per cycle and
// SM, 2048 cycles (3160 measured: the sums, maxima and transfers of two softmax warps to a
// scheduler do not all hide behind them; moving exponentials to the FMA pipe made it slower).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "attention.h"
#include "muon.h"
#include "ns_tc.h"
#include "umma.cuh"

namespace muon {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

bool encode_heads_map(CUtensorMap* out, const muon_heads_t& t, int64_t tokens, int heads, int dim, int rows) {
  if (tokens == 0) return true;
  const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  // strides of axes of one element are never used, and may be anything
  const int64_t head = heads > 1 ? t.head : dim, ld = tokens > 1 ? t.ld : dim;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(head) * 2, static_cast<cuuint64_t>(ld) * 2};
  cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, t.ptr, dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

constexpr int kRows = 128;          // query rows of a block
constexpr int kThreads = 256;
constexpr float kLazy = 8.f;        // the running maximum moves when exceeded by this (log2)

template <int HD>
struct FwdCfg {
  // Half of the tensor memory, 256 columns, beside the accumulator's HD:
  //   128: S in blocks of 64 keys, two buffers, P over the buffer it came from
  //   64:  S in blocks of 128 keys, one buffer, and P in columns of its own
  // Either way the next block's S is computed while this block's softmax runs.
  static constexpr bool kOwnP = HD == 64;
  static constexpr int kKeys = kOwnP ? 128 : 64;      // keys of a block
  static constexpr int kHalves = kKeys / 64;          // P is handed over by 64 keys
  static constexpr int kQBytes = kRows * HD * 2;
  static constexpr int kQChunk = kRows * 128;         // bytes of 64 columns of Q
  static constexpr int kKvBytes = kKeys * HD * 2;
  static constexpr int kKvChunk = kKeys * 128;
  static constexpr int kStages = 5;                   // K and V blocks in flight
  static constexpr int kOffKv = kQBytes;
  static constexpr int kOffBar = kOffKv + kStages * kKvBytes;
  static constexpr int kSmemBytes = kOffBar + 256;
  static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two blocks share an SM");
  static constexpr uint32_t kO = 128;                 // first accumulator column
  static constexpr uint32_t kP = kO + HD;             // P of its own: 64 columns
  __host__ __device__ static constexpr uint32_t s_col(int j) { return kOwnP ? 0 : (j & 1) * 64; }
  __host__ __device__ static constexpr uint32_t p_col(int j) { return kOwnP ? kP : s_col(j); }
};

struct FwdParams {
  CUtensorMap tq, tk, tv;
  muon_attention_t a;
};

// Raises *p to v: positive floats order as integers, negative ones in reverse as unsigned.
// The result does not depend on the order of the calls; NaN changes nothing. (-0 is taken as +0:
// as an integer it would be below everything.)
__device__ __forceinline__ void atomic_max_float(float* p, float v) {
  v += 0.f;
  if (v >= 0.f) atomicMax(reinterpret_cast<int*>(p), __float_as_int(v));
  else if (v < 0.f) atomicMin(reinterpret_cast<unsigned*>(p), __float_as_uint(v));
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 2) attention_fwd_kernel(const __grid_constant__ FwdParams P) {
  using C = FwdCfg<HD>;
  const muon_attention_t& a = P.a;
  const int heads = a.heads;
  const int head = static_cast<int>(blockIdx.x % heads);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  int row0;
  const SeqRange r = find_tile(a, false, kRows, static_cast<int>(blockIdx.x / heads),
                               static_cast<int>(gridDim.x / heads), lane, &row0);
  if (row0 >= r.m) return;
  const int shift = r.n - r.m;  // causal: row i sees keys j <= i + shift
  const int keys = a.causal ? min(r.n, min(row0 + kRows, r.m) + shift) : r.n;
  const int n = keys > 0 ? (keys + C::kKeys - 1) / C::kKeys : 0;  // key blocks

  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // ring of K and V blocks
  uint64_t* empty = full + C::kStages;
  uint64_t* q_full = empty + C::kStages;
  // A barrier that may complete for block j + 1 before block j has been waited for exists once
  // per block parity.
  uint64_t* s_full = q_full + 1;   // per block parity: S is complete
  uint64_t* s_read = s_full + 2;   // S is in registers (own P)
  uint64_t* p_full = s_read + 1;   // per half (own P) or block parity: 64 keys of P are in place
  uint64_t* o_full = p_full + 2;   // per block parity: the product with V is complete
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_full + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert(8 * (2 * C::kStages + 8) + 8 <= 256, "barrier region");
  const int kvh = head / (heads / a.kv_heads);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(s_read, 4);
    for (int e = 0; e < 2; ++e) {
      mbar_init(&s_full[e], 1);
      mbar_init(&p_full[e], 4);
      mbar_init(&o_full[e], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    // Q and the first K block are on their way before the other warps are set up
    if (n > 0) {
      mbar_expect_tx(q_full, C::kQBytes);
      for (int c = 0; c < HD / 64; ++c)
        tma_load_3d(smem + c * C::kQChunk, &P.tq, q_full, c * 64, head, r.q0 + row0);
      mbar_expect_tx(&full[0], C::kKvBytes);
      for (int c = 0; c < HD / 64; ++c)
        tma_load_3d(smem + C::kOffKv + c * C::kKvChunk, &P.tk, &full[0], c * 64, kvh, r.k0);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  // Ring positions of the K and V blocks, in the order of use: K_{j+1} before V_j.
  auto pos_k = [&](int j) { return j == 0 ? 0 : 2 * j - 1; };
  auto pos_v = [&](int j) { return j + 1 < n ? 2 * j + 2 : 2 * n - 1; };

  // Registers: 256 x 128 at launch; 128 x 56 + 128 x 200 is the same total.
  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0 && n > 0) {
      bool ok = true;
      int loads = 1, j[2] = {1, 0};  // the next K and V block; K_0 is under way
      for (int t = 1; t < 2 * n; ++t) {
        const int s = t % C::kStages;
        const bool is_v = j[1] < n && t == pos_v(j[1]);
        if (!mbar_wait(&empty[s], static_cast<uint32_t>((t / C::kStages) & 1) ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        uint8_t* dst = smem + C::kOffKv + s * C::kKvBytes;
        const int key = r.k0 + (is_v ? j[1]++ : j[0]++) * C::kKeys;
        mbar_expect_tx(&full[s], C::kKvBytes);
        for (int c = 0; c < HD / 64; ++c)
          tma_load_3d(dst + c * C::kKvChunk, is_v ? &P.tv : &P.tk, &full[s], c * 64, kvh, key);
        ++loads;
      }
      if (!ok) {
        set_error(a.status_dev, MUON_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // never leave with bulk copies still landing in shared memory
      mbar_wait(q_full, 0, nullptr);
      for (int t = loads > C::kStages ? loads - C::kStages : 0; t < loads; ++t)
        mbar_wait(&full[t % C::kStages], static_cast<uint32_t>((t / C::kStages) & 1), nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (n > 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, C::kKeys, false), idesc_o = idesc_bf16_f32(128, HD, true);
      const uint32_t base = smem_u32(smem), qd = desc_lo(base, 16);
      const uint32_t to = tmem + C::kO;
      auto slot_of = [&](int t) { return t % C::kStages; };
      auto wait_bar = [&](uint64_t* bar, int phase) {
        const bool got = __all_sync(0xffffffffu, mbar_wait(bar, static_cast<uint32_t>(phase & 1), abort_flag));
        tc_fence_after();
        return got;
      };
      // S = Q K_j^T, then K_j is free. The buffer is: read (own P), or the P of two blocks ago,
      // whose product was issued before.
      auto qk = [&](int j) {
        const int t = pos_k(j);
        if (!wait_bar(&full[slot_of(t)], t / C::kStages)) return false;
        if (C::kOwnP && j > 0 && !wait_bar(s_read, j - 1)) return false;
        if (elect_one()) {
          const uint32_t kd = desc_lo(base + C::kOffKv + slot_of(t) * C::kKvBytes, 16);
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {
            const uint32_t in = (k & 3) * 2, c = k >> 2;
            umma_f16_lo(tmem + C::s_col(j), qd + c * (C::kQChunk >> 4) + in, kd + c * (C::kKvChunk >> 4) + in,
                        kDescHi, idesc_s, k != 0);
          }
          umma_commit(&s_full[j & 1]);
          umma_commit(&empty[slot_of(t)]);
        }
        return true;
      };
      auto pv = [&](int j) {  // O += P V_j, by halves of the keys as P arrives, then V_j is free
        const int t = pos_v(j), s = slot_of(t), live = r.n - j * C::kKeys;
        if (!wait_bar(&full[s], t / C::kStages)) return false;
        if (live < C::kKeys) {
          // keys past the sequence have probability 0, and their V must not be NaN
          uint8_t* v = smem + C::kOffKv + s * C::kKvBytes;
          for (int e = live * 8 + lane; e < C::kKeys * 8; e += 32)
#pragma unroll
            for (int c = 0; c < HD / 64; ++c)
              *reinterpret_cast<uint4*>(v + c * C::kKvChunk + e * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        const uint32_t vd = desc_lo(base + C::kOffKv + s * C::kKvBytes, C::kKvChunk);
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h) {
          if (!(C::kOwnP ? wait_bar(&p_full[h], j) : wait_bar(&p_full[j & 1], j >> 1))) return false;
          if (elect_one()) {
#pragma unroll
            for (int k = 4 * h; k < 4 * h + 4; ++k)
              umma_f16_ts_lo(to, tmem + C::p_col(j) + k * 8, vd + 128u * k, kDescHi, idesc_o, (j | k) != 0);
            if (h == C::kHalves - 1) {
              umma_commit(&o_full[j & 1]);
              umma_commit(&empty[s]);
            }
          }
        }
        return true;
      };
      bool ok = wait_bar(q_full, 0) && qk(0);
      for (int j = 0; j < n && ok; ++j) ok = (j + 1 >= n || qk(j + 1)) && pv(j);
      // never leave with products still running
      ok = ok && wait_bar(&o_full[(n - 1) & 1], (n - 1) >> 1);
      if (!ok && lane == 0) {
        set_error(a.status_dev, MUON_ERR_TIMEOUT);
        *abort_flag = 1;
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax, one thread per row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int w = warp & 3;
    const int row = row0 + w * 32 + lane;  // within the sequence
    const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
    const uint32_t to = tmem + lanes + C::kO;
    constexpr int kParts = C::kKeys / 32;
    const float sl = a.scale * 1.4426950408889634f;
    float top = -INFINITY;            // largest logit so far, unscaled
    float ref = 0.f;                  // the exponent's reference, scaled
    float sum = 0.f;
    bool ok = true;
    auto wait_o = [&](int j) {  // the product of block j is complete
      const bool got = __all_sync(0xffffffffu, mbar_wait(&o_full[j & 1], static_cast<uint32_t>((j >> 1) & 1), abort_flag));
      tc_fence_after();
      return got;
    };
    for (int j = 0; j < n; ++j) {
      if (!__all_sync(0xffffffffu, mbar_wait(&s_full[j & 1], static_cast<uint32_t>((j >> 1) & 1), abort_flag))) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t s[kParts][32];
#pragma unroll
      for (int c = 0; c < kParts; ++c) tmem_ld32(tmem + lanes + C::s_col(j) + c * 32, s[c]);
      tmem_wait_ld();
      if (C::kOwnP) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_read);
      }
      // keys of this block that the row sees
      const int vis = min(r.n, a.causal ? row + shift + 1 : r.n) - j * C::kKeys;
      if (__any_sync(0xffffffffu, vis < C::kKeys)) {
#pragma unroll
        for (int c = 0; c < kParts; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (c * 32 + e >= vis) s[c][e] = 0xFF800000u;
      }
      float m[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 32; e += 2)
#pragma unroll
        for (int c = 0; c < kParts; ++c)
          m[2 * (c & 1) + (e / 2 & 1)] = max3(m[2 * (c & 1) + (e / 2 & 1)], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
      top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
      // (a row whose logits so far are all -inf: below any that follow, yet finite)
      const float want = top == -INFINITY ? -3e38f : top * sl;
      if (j == 0) {
        ref = want;
      } else {
        // The product that read the columns P goes to is complete (long ago).
        const int jp = j - (C::kOwnP ? 1 : 2);
        if (jp >= 0) {
          ok = wait_o(jp);
          if (!ok) break;
        }
        const bool move = want > ref + kLazy;
        if (__any_sync(0xffffffffu, move)) {
          if (!C::kOwnP) {  // and so is the one before this block: O may be rescaled
            ok = wait_o(j - 1);
            if (!ok) break;
          }
          const float f = move ? ex2(ref - want) : 1.f;
          if (move) ref = want;
          sum *= f;
#pragma unroll
          for (int c = 0; c < HD / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(to + c * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(to + c * 32, o);
          }
        }
      }
      float add[4] = {sum, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < C::kHalves; ++h) {
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int c = 2 * h + (e >> 4), k = 2 * (e & 15);
          const float p0 = ex2(fmaf(__uint_as_float(s[c][k]), sl, -ref));
          const float p1 = ex2(fmaf(__uint_as_float(s[c][k + 1]), sl, -ref));
          add[2 * (e & 1)] += p0;
          add[2 * (e & 1) + 1] += p1;
          pk[e] = round_bf16x2(p0, p1);
        }
        tmem_st32(tmem + lanes + C::p_col(j) + h * 32, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[C::kOwnP ? h : j & 1]);
      }
      sum = (add[0] + add[1]) + (add[2] + add[3]);
    }
    if (!ok && lane == 0) {
      set_error(a.status_dev, MUON_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    if (n > 0 && ok) {
      ok = wait_o(n - 1);
      if (!ok && lane == 0) set_error(a.status_dev, MUON_ERR_TIMEOUT);
    }
    const bool live = row < r.m, seen = top > -INFINITY || sum != 0.f;
    const float inv = seen ? 1.f / sum : 0.f;  // 0: the row is written as zeros
    // staged where Q was: its products are complete
    store_rows<HD>(to, smem, w, lane, 0, inv, n == 0,
                   static_cast<uint16_t*>(a.o.ptr) + static_cast<int64_t>(r.q0 + row0 + w * 32) * a.o.ld + head * a.o.head,
                   a.o.ld, ok ? r.m - row0 - w * 32 : 0, a.head_dim);
    if (live && ok)
      a.lse[static_cast<int64_t>(head) * a.q_tokens + r.q0 + row] =
          seen ? (ref + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    if (a.s_max != nullptr) {
      float best = live && ok ? top : -INFINITY;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
      if (lane == 0 && best > -INFINITY) atomic_max_float(a.s_max + head, best * a.scale);
    }
    tc_fence_before();
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

template <int HD>
cudaError_t launch(const FwdParams& P, int dev, int64_t grid, cudaStream_t st) {
  // the shared-memory opt-in is a per-device attribute: set it once on each device
  static std::atomic<uint64_t> attr_devices{0};
  const uint64_t bit = dev < 64 ? (uint64_t{1} << dev) : 0;
  if (bit == 0 || !(attr_devices.load(std::memory_order_acquire) & bit)) {
    cudaError_t e = cudaFuncSetAttribute(attention_fwd_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         FwdCfg<HD>::kSmemBytes);
    if (e == cudaSuccess)  // all of the SM's memory, so that two blocks fit
      e = cudaFuncSetAttribute(attention_fwd_kernel<HD>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    attr_devices.fetch_or(bit, std::memory_order_acq_rel);
  }
  attention_fwd_kernel<HD><<<static_cast<unsigned>(grid), kThreads, FwdCfg<HD>::kSmemBytes, st>>>(P);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_forward(const muon_attention_t& a, int dev, cudaStream_t st) {
  FwdParams P;
  std::memset(&P, 0, sizeof(P));
  P.a = a;
  const int keys = a.head_dim <= 64 ? FwdCfg<64>::kKeys : FwdCfg<128>::kKeys;
  if (!encode_heads_map(&P.tq, a.q, a.q_tokens, a.heads, a.head_dim, kRows) ||
      !encode_heads_map(&P.tk, a.k, a.k_tokens, a.kv_heads, a.head_dim, keys) ||
      !encode_heads_map(&P.tv, a.v, a.k_tokens, a.kv_heads, a.head_dim, keys))
    return cudaErrorInvalidValue;
  const int64_t grid = tile_slots(a.q_offsets, a.n_seq, a.q_tokens, kRows) * a.heads;
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  return a.head_dim <= 64 ? launch<64>(P, dev, grid, st) : launch<128>(P, dev, grid, st);
}

}  // namespace muon

// Weight gradients from 8-bit activation checkpoints (muon_weight_grad_t):
//   dW_g[o, i] (+)= sum over the tokens t of group g of dY[t, o] q[t, i] 2^E[t, i/32]
//
// A GEMM whose reduction axis is the outer axis of both operands. dY is taken as it lies in
// memory: an MN-major tile (64 columns x 64 tokens a chunk, 128B swizzle) as the B operand of
// tcgen05.mma. X^T is the A operand and lives in tensor memory, where a lane is a column of X
// and a 32-bit column two consecutive tokens: ldmatrix transposes 16 x 16 bytes of q on the
// way to the registers in just the fragment that tcgen05.st takes, so the restored tile never
// passes through shared memory. (The first form restored into a shared-memory operand: 16 KB
// written and 16 KB read per k-block and CTA, 80 KB of shared-memory traffic in all against
// 128 B a cycle, which held it at 850 cycles a k-block where the MMAs need 512.)
// q 2^E has 7 significant bits and is exact in bf16, so every product dY q 2^E is exact and
// sums are fp32 in tensor memory.
//
// Tile 256 (in) x N = 128, 256 or 384 (out) per CTA pair (cta_group::2): each CTA restores its
// 128 columns of X and loads its N / 2 columns of dY, so a restored element serves N output
// rows. Persistent, one CTA per SM, warps:
//   0      TMA producer: per 64-token k-block 8 to 24 KB of dY, 8 KB of q and 1 KB of exponents,
//          into a ring of 8 stages (N = 384: 4)
//   1      TMEM allocator and (first CTA) MMA issuer
//   2-13   restore, three teams that take the k-blocks in turn; the last k-block of a group also
//          clears the rows past its end in both operands, so that a neighbouring group's NaN
//          cannot reach this one's sums
//   14-21  epilogue: a lane is a column of dW's row, so the accumulator's registers are
//          written in whole 128-byte rows at any alignment, without a transpose
// Split of the work: groups of several matrices are dealt in runs of tiles of equal work; other
// tiles go to the 74 CTA pairs in whole rounds, and those left over for the last round are split
// along the tokens into as many parts as keep all pairs busy, whose fp32 partial sums a second
// kernel adds in order (no atomics).
// Bound by the products and their operands for long groups (130 us for 5632 x 2048 from 8192
// tokens, 1450 TFLOP/s, at the full clock; 161 us under the power cap), by restoring X at 128
// rows, and by start and epilogue for short groups.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "act8.cuh"
#include "muon.h"
#include "ns_tc.h"
#include "umma.cuh"
#include "validate.h"

namespace muon {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace {

constexpr int kIn = 256;                      // tile columns (in) of a CTA pair
constexpr int kTok = 64;                      // tokens per k-block
constexpr int kQBytes = 128 * kTok;           // a CTA's stored X columns of one k-block
constexpr int kEBytesRow = 16;                // exponents of 512 columns, the smallest TMA row
constexpr int kEBytes = kEBytesRow * kTok;
constexpr int kTeams = 3, kTeamWarps = 4;     // restore teams take k-blocks in turn
constexpr int kRestoreWarps = kTeams * kTeamWarps, kEpiWarps = 8;
constexpr int kFirstEpi = 2 + kRestoreWarps;
constexpr int kThreads = 32 * (2 + kRestoreWarps + kEpiWarps);
constexpr int kXCols = kTok / 2;              // columns of one stage
constexpr int kPairs = 74;                    // CTA pairs of a B200 (148 SMs)

constexpr int kMaxBalanced = 128;             // groups whose lengths every block adds up

// N: tile rows (out) of a CTA pair, half of them from each CTA's dY columns. Tensor memory holds
// 256 / N accumulators (one of 256 or 384 columns) and, behind them, the stages of X^T.
template <int N>
struct WgradCfg {
  static constexpr int kAcc = N >= 256 ? 1 : 256 / N;
  static constexpr int kTmemX = kAcc * N;     // first column of the X^T stages
  static constexpr int kStages = (512 - kTmemX) / kXCols;
  static constexpr int kYBytes = N / 2 * kTok * 2;
  static constexpr int kOffE = kYBytes + kQBytes;
  static constexpr int kStageBytes = kOffE + kEBytes;
  static constexpr int kOffBar = kStages * kStageBytes;
  static constexpr int kSmemBytes = kOffBar + 256 + 1024;
  static_assert(kSmemBytes <= 227 * 1024 && kStageBytes % 1024 == 0, "shared memory");
  static_assert(kStages >= kTeams, "a team stays within one round of the ring");
};

// How the tiles are dealt: `whole` tiles by one unit each, the `left` ones by `splits` units.
struct WgradSplit {
  int32_t n;                 // tile rows: 384, 256 or 128
  int32_t tile_kb;           // what a tile costs beside its k-blocks, in k-blocks
  int32_t tiles_o, tiles_i;
  int32_t splits;
  int32_t balance;           // tiles dealt in contiguous runs of equal k-blocks
  int64_t whole, left;
  int64_t units;
  size_t part_bytes;
};

// What a tile of N rows costs a pair: cycles per k-block (measured on long groups: at 128 rows
// the restoring of X is the limit, above the products are), and what its start and an epilogue
// that nothing hides add.
struct TileCost {
  int n;
  double per_kb, fixed;
};
constexpr TileCost kCosts[3] = {{384, 950., 5500.}, {256, 700., 4500.}, {128, 560., 2500.}};

// Picks the tile height and the split of the last round by the cost of the longest pair's tiles;
// partial sums and the second launch cost about 7000 cycles. High tiles restore X for more rows;
// low ones waste less of a small or ragged `out`.
WgradSplit split_of(const muon_weight_grad_t& a) {
  const int64_t kb = (a.tokens / a.groups + kTok - 1) / kTok;  // of a mean group
  WgradSplit best{};
  double best_cost = 0;
  for (const TileCost& t : kCosts) {
    const int n = t.n;
    const double per_kb = t.per_kb, fixed = t.fixed;
    WgradSplit s{};
    s.n = n;
    s.tile_kb = static_cast<int32_t>(fixed / per_kb);
    s.tiles_o = static_cast<int32_t>((a.out + n - 1) / n);
    s.tiles_i = static_cast<int32_t>((a.in + kIn - 1) / kIn);
    s.part_bytes = static_cast<size_t>(n) * kIn * 4;
    const int64_t tiles = static_cast<int64_t>(s.tiles_o) * s.tiles_i * a.groups;
    for (int split = 0; split < 2; ++split) {
      s.whole = tiles;
      s.left = 0;
      s.splits = 1;
      double cost = static_cast<double>((tiles + kPairs - 1) / kPairs) * (kb * per_kb + fixed);
      if (split) {
        s.whole = tiles / kPairs * kPairs;
        s.left = tiles - s.whole;
        if (s.left == 0) break;
        int64_t parts = kPairs / s.left;
        if (parts > kb / 4) parts = kb / 4;  // at least 4 k-blocks each
        if (parts < 2) break;
        s.splits = static_cast<int32_t>(parts);
        cost = static_cast<double>(s.whole / kPairs) * (kb * per_kb + fixed) +
               (kb + parts - 1) / parts * per_kb + fixed + 7000.;
      }
      s.units = s.whole + s.left * s.splits;
      s.balance = s.splits == 1 && a.groups > 1 && a.groups <= kMaxBalanced && tiles > kPairs;
      if (best.n == 0 || cost < best_cost) {
        best = s;
        best_cost = cost;
      }
    }
  }
  return best;
}

struct WgradParams {
  CUtensorMap ty, tq, te;
  muon_weight_grad_t a;
  WgradSplit s;
  float* parts;
};

// Token range of group g, clamped to the tensor.
__device__ __forceinline__ void group_range(const muon_weight_grad_t& a, int g, int* lo, int* hi) {
  const int tokens = static_cast<int>(a.tokens);
  if (a.offsets == nullptr) {
    *lo = 0;
    *hi = tokens;
    return;
  }
  const int b = __ldg(a.offsets + g), e = __ldg(a.offsets + g + 1);
  *lo = min(max(b, 0), tokens);
  *hi = max(min(max(e, 0), tokens), *lo);
}

// Arrives on the first CTA's mbarrier. What it signals is read by the tensor core from this
// CTA's own shared memory, behind the writer's proxy fence; no generic access of the other CTA
// depends on it, so the default (CTA) scope is enough. A cluster-scope release here flushed
// this CTA's traffic on every k-block: 1300 cycles against 260.
__device__ __forceinline__ void mbar_arrive_peer(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// One unit of work: a tile, its tokens [t0, t1) and, for a split tile, where its sum goes.
struct Job {
  int g, o0, i0;    // group, first row and column of the tile
  int t0, t1, nkb;  // tokens and k-blocks
  int part;         // partial sum, or -1: dW
};

template <int N>
__device__ __forceinline__ Job job_of(const WgradParams& P, uint32_t u) {
  Job j;
  uint32_t t = u, split = 0;
  const uint32_t whole = static_cast<uint32_t>(P.s.whole), splits = static_cast<uint32_t>(P.s.splits);
  j.part = -1;
  if (u >= whole) {
    const uint32_t r = (u - whole) / splits;
    split = u - whole - r * splits;
    t = whole + r;
    j.part = static_cast<int>(u - whole);
  }
  const uint32_t ti = static_cast<uint32_t>(P.s.tiles_i), per = static_cast<uint32_t>(P.s.tiles_o) * ti;
  j.g = static_cast<int>(t / per);
  const uint32_t rem = t - static_cast<uint32_t>(j.g) * per;
  j.o0 = static_cast<int>(rem / ti) * N;
  j.i0 = static_cast<int>(rem % ti) * kIn;
  int lo, hi;
  group_range(P.a, j.g, &lo, &hi);
  if (j.part >= 0) {
    const uint32_t kb = static_cast<uint32_t>(hi - lo + kTok - 1) / kTok;  // at most 2^25, splits at most 74
    const uint32_t b0 = kb * split / splits, b1 = kb * (split + 1) / splits;
    if (static_cast<int>(b1) * kTok < hi - lo) hi = lo + static_cast<int>(b1) * kTok;
    lo += static_cast<int>(b0) * kTok;
  }
  j.t0 = lo;
  j.t1 = hi;
  j.nkb = (hi - lo + kTok - 1) / kTok;
  return j;
}

// The tiles [u[0], u[1]) of CTA pair `pair` out of `pairs`, by one warp: tiles in order, each
// weighing its k-blocks and tile_kb, and dealt to the pair in whose share of the total weight
// its middle lies. A router's groups differ in length: dealt in turn, 64 experts of 0 to 1487
// tokens left the busiest pair with 1.6 times the mean, dealt so with 1.2.
__device__ __forceinline__ void balanced_range(const WgradParams& P, int pair, int pairs, int lane, uint32_t* u) {
  const int groups = P.a.groups;
  const int per = P.s.tiles_o * P.s.tiles_i;  // below 2^24: a float holds it
  int w[kMaxBalanced / 32];  // all loads first
#pragma unroll
  for (int c = 0; c < kMaxBalanced / 32; ++c) {
    const int g = c * 32 + lane;
    int lo = 0, hi = 0;
    if (g < groups) group_range(P.a, g, &lo, &hi);
    w[c] = g < groups ? (hi - lo + kTok - 1) / kTok + P.s.tile_kb : 0;
  }
  // in fp32: every pair computes the same numbers, and rounds monotonically, so that one's end
  // is the next one's start
  uint32_t mine = 0;
#pragma unroll
  for (int c = 0; c < kMaxBalanced / 32; ++c) mine += w[c];
  const float total = static_cast<float>(__reduce_add_sync(0xffffffffu, mine));
  const float share[2] = {total * pair / pairs, total * (pair + 1) / pairs};
  uint32_t before = 0, count[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < kMaxBalanced / 32; ++c) {
    if (c * 32 >= groups) break;
    uint32_t upto = w[c];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const float base = static_cast<float>(before + upto - w[c]);
    before += __shfl_sync(0xffffffffu, upto, 31);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // tiles of the group whose middle base + (i + 1/2) w / per lies before the share's end
      const float n = w[c] == 0 ? 0.f : ceilf((share[e] - base) * per / w[c] - 0.5f);
      count[e] += static_cast<uint32_t>(fminf(fmaxf(n, 0.f), w[c] == 0 ? 0.f : static_cast<float>(per)));
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) count[e] = __reduce_add_sync(0xffffffffu, count[e]);
  if (lane == 0) {
    u[0] = count[0];
    u[1] = pair + 1 == pairs ? static_cast<uint32_t>(P.s.units) : count[1];
  }
}

// Two 16 x 16 byte matrices, transposed: lanes 0-15 and 16-31 give their rows' addresses.
// Lane l gets of each matrix the rows 4 (l % 4) .. + 3 of column l / 4 and of column l / 4 + 8.
__device__ __forceinline__ void ldmatrix_b8_x2_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// 16 lanes x 32 columns of tensor memory; register 4 n + i holds, for lane l of the warp,
// column 8 n + 2 (l % 4) + (i & 1) of row l / 4 + 8 (i >> 1).
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// D (both CTAs' tensor memory) (+)= A (both CTAs' tensor memory, M split) * B (both CTAs'
// shared memory, N split)^T.
__device__ __forceinline__ void umma_f16_pair_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
      : "memory");
}

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(uint16_t* p, float x) { *p = f32_to_bf16(x); }

// Up to 32 rows of one column, ld apart: the lanes of a warp write 32 neighbours of each row.
template <class T>
__device__ __forceinline__ void write_rows(T* p, int64_t ld, int n, bool accumulate, uint32_t (&v)[32]) {
  if (accumulate) {
    T old[32];
    const T* q = p;
#pragma unroll
    for (int i = 0; i < 32; ++i, q += ld) old[i] = i < n ? *q : T(0);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + widen(old[i]));
  }
#pragma unroll
  for (int i = 0; i < 32; ++i, p += ld)
    if (i < n) put(p, __uint_as_float(v[i]));
}

// The row of the tile that chunk c (64 columns of dY) of a CTA starts at: a product takes the
// first half of its N rows from the first CTA and the second half from the other.
template <int N>
__device__ __forceinline__ int chunk_row(int rank, int c) {
  return N > 256 && c == 2 ? 256 + rank * 64 : rank * (N < 256 ? N / 2 : 128) + 64 * c;
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1) wgrad_kernel(const __grid_constant__ WgradParams P) {
  using C = WgradCfg<N>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // this CTA's loads have landed
  uint64_t* ready = full + C::kStages;   // first CTA's: both CTAs' operands are in place
  uint64_t* empty = ready + C::kStages;  // the MMAs have read the stage
  uint64_t* tfull = empty + C::kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* range = tmem_slot + 2;    // this pair's units
  static_assert(8 * (3 * C::kStages + 5) + 16 <= 256, "barrier region");

  const muon_weight_grad_t& a = P.a;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_cta_rank());

  if (threadIdx.x == 32 * kFirstEpi && a.tokens > 0) {
    tma_prefetch(&P.tq);
    tma_prefetch(&P.te);
    tma_prefetch(&P.ty);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&ready[s], 2 * kTeamWarps);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kAcc; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kEpiWarps);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  if (warp == 2 && P.s.balance) balanced_range(P, blockIdx.x >> 1, gridDim.x >> 1, lane, range);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  griddep_launch_dependents();  // the join, where there is one, waits for this grid's end
  const uint32_t unit0 = P.s.balance ? range[0] : blockIdx.x >> 1;
  const uint32_t unit1 = P.s.balance ? range[1] : static_cast<uint32_t>(P.s.units);
  const uint32_t stride = P.s.balance ? 1 : gridDim.x >> 1;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    int s = 0;
    uint32_t par = 0, loads = 0;
    bool ok = true;
    for (uint32_t u = unit0; u < unit1 && ok; u += stride) {
      const Job j = job_of<N>(P, u);
      const int i = j.i0 + rank * 128;
      for (int kb = 0; kb < j.nkb; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], par ^ 1u, abort_flag));
        if (!ok) break;
        if (elect_one()) {
          uint8_t* st = smem + s * C::kStageBytes;
          const int t = j.t0 + kb * kTok;
          mbar_expect_tx(&full[s], C::kStageBytes);
          tma_load_3d(st + C::kYBytes, &P.tq, &full[s], i, t, 0);
          tma_load_3d(st + C::kOffE, &P.te, &full[s], i / 512 * kEBytesRow, t, 0);
#pragma unroll
          for (int c = 0; c < N / 128; ++c)
            tma_load_3d(st + c * (64 * kTok * 2), &P.ty, &full[s], j.o0 + chunk_row<N>(rank, c), t, 0);
        }
        ++loads;
        if (++s == C::kStages) s = 0, par ^= 1u;
      }
    }
    if (!ok && lane == 0) {
      set_error(a.status_dev, MUON_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    // never leave with bulk copies still landing in shared memory
    for (uint32_t r = loads > C::kStages ? loads - C::kStages : 0; r < loads; ++r)
      mbar_wait(&full[r % C::kStages], (r / C::kStages) & 1u, nullptr);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      // A from tensor memory, B MN-major; 384 rows are two products, of 256 and 128
      constexpr uint32_t idesc = idesc_bf16_f32(256, N < 256 ? N : 256, true), idesc2 = idesc_bf16_f32(256, 128, true);
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool got = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
        tc_fence_after();
        return got;
      };
      int s = 0, it = 0;
      uint32_t par = 0;
      bool ok = true;
      for (uint32_t u = unit0; u < unit1 && ok; u += stride) {
        const Job j = job_of<N>(P, u);
        if (j.nkb == 0) continue;
        const int acc = it % C::kAcc;
        ok = wait(&tempty[acc], static_cast<uint32_t>((it / C::kAcc) & 1) ^ 1u);
        ++it;
        const uint32_t d = tmem + acc * N;
        for (int kb = 0; kb < j.nkb && ok; ++kb) {
          ok = wait(&ready[s], par);
          if (!ok) break;
          if (elect_one()) {
            const uint32_t bd = desc_lo(smem_u32(smem) + s * C::kStageBytes, 64 * kTok * 2);
            const uint32_t at = tmem + C::kTmemX + s * kXCols;
#pragma unroll
            for (int kk = 0; kk < kTok / 16; ++kk)  // 16 tokens: 8 columns, 2 KB of a chunk
            {
              umma_f16_pair_ts(d, at + 8u * kk, bd + 128u * kk, idesc, (kb | kk) != 0 ? 1u : 0u);
              if (N > 256)
                umma_f16_pair_ts(d + 256, at + 8u * kk, bd + ((2 * 64 * kTok * 2) >> 4) + 128u * kk, idesc2,
                                 (kb | kk) != 0 ? 1u : 0u);
            }
            umma_commit_pair(smem_u32(&empty[s]));
            umma_commit_pair(peer_addr(&empty[s], 1));
            if (kb + 1 == j.nkb) {
              umma_commit_pair(smem_u32(&tfull[acc]));
              umma_commit_pair(peer_addr(&tfull[acc], 1));
            }
          }
          if (++s == C::kStages) s = 0, par ^= 1u;
        }
      }
      if (!ok && lane == 0) {
        set_error(a.status_dev, MUON_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // never leave with products still running
      if (elect_one()) umma_commit_pair(smem_u32(done));
      __syncwarp();
      mbar_wait(done, 0, nullptr);
    }
  } else if (warp < kFirstEpi) {
    // ------------------------------------------------------------ restore
    // A team's warp owns the 32 columns of X of its tensor-memory lane quarter: one group of
    // the checkpoint. Its exponents go through ldmatrix as well: row g of the transposed
    // exponent tile holds group g, whose bytes a shuffle hands to the lanes of their tokens.
    const int team = (warp - 2) / kTeamWarps, w = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
    uint32_t q0 = 0;  // k-blocks of the units before this one
    bool ok = true;
    for (uint32_t u = unit0; u < unit1 && ok; u += stride) {
      const Job j = job_of<N>(P, u);
      const int grp = ((j.i0 + rank * 128) / 32 + w) % kEBytesRow;  // within a stage's exponent row
      const int src = (grp & 7) * 4 + (lane & 3);
      for (int kb = static_cast<int>((team + kTeams - q0 % kTeams) % kTeams); kb < j.nkb; kb += kTeams) {
        const uint32_t q = q0 + kb;
        const int s = static_cast<int>(q % C::kStages);
        // A team does not see every k-block, and copies may land out of order: the parity of `full`
        // alone could still be the one before the stage's previous copy. That copy has landed once
        // the products that read it are complete. (They are at most one phase ahead: the team's
        // own previous copy was issued after those of the round before.)
        const uint32_t round = q / C::kStages;
        const bool landed = (round == 0 || mbar_wait(&empty[s], (round - 1) & 1u, abort_flag)) &&
                            mbar_wait(&full[s], round & 1u, abort_flag);
        if (!__all_sync(0xffffffffu, landed)) {
          ok = false;
          if (lane == 0) {
            set_error(a.status_dev, MUON_ERR_TIMEOUT);
            *abort_flag = 1;
          }
          break;
        }
        uint8_t* st = smem + s * C::kStageBytes;
        const int live = j.t1 - (j.t0 + kb * kTok);  // tokens of the group from this k-block on
        uint32_t sc[4][2];  // scales of tokens 16 b + 4 (lane % 4) + {0, 1}, {2, 3}
#pragma unroll
        for (int b = 0; b < 4; b += 2) {
          uint32_t e[4];
          ldmatrix_b8_x2_trans(smem_u32(st + C::kOffE + (16 * b + lane) * kEBytesRow), e);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x0 = __shfl_sync(0xffffffffu, e[2 * h], src), x1 = __shfl_sync(0xffffffffu, e[2 * h + 1], src);
            const uint32_t x = grp < 8 ? x0 : x1;
            sc[b + h][0] = __byte_perm(x, 0, 0x4140) << 7;
            sc[b + h][1] = __byte_perm(x, 0, 0x4342) << 7;
          }
        }
        if (live < kTok) {
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int t = 16 * b + 4 * (lane & 3) + 2 * h;
              sc[b][h] &= (t < live ? 0xFFFFu : 0u) | (t + 1 < live ? 0xFFFF0000u : 0u);
            }
          // the dY of tokens past the group: zeros too
          for (int t = live + w; t < kTok; t += kTeamWarps)
#pragma unroll
            for (int c = 0; c < N / 128; ++c)
              *reinterpret_cast<uint32_t*>(st + c * (64 * kTok * 2) + t * 128 + lane * 4) = 0;
          fence_proxy_async_smem();
        }
        uint32_t x[2][16];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int t = 16 * b + (lane & 15);
          uint32_t v[4];
          ldmatrix_b8_x2_trans(smem_u32(st + C::kYBytes + t * 128 + (((2 * w + (lane >> 4)) ^ (t & 7)) << 4)), v);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            act8_restore4(v[2 * h], sc[b][0], sc[b][1], &x[h][4 * b], &x[h][4 * b + 1]);
            act8_restore4(v[2 * h + 1], sc[b][0], sc[b][1], &x[h][4 * b + 2], &x[h][4 * b + 3]);
          }
        }
        const uint32_t at = tmem + C::kTmemX + s * kXCols + lanes;
        tmem_st_16x256b_x4(at, x[0]);
        tmem_st_16x256b_x4(at + (16u << 16), x[1]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) mbar_arrive(&ready[s]);
          else mbar_arrive_peer(peer_addr(&ready[s], 0));
        }
      }
      q0 += j.nkb;
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int w = warp & 3;                              // the TMEM lane quarter this warp may access
    const int half = (warp - kFirstEpi) / 4 * (N / 2);   // and its half of the tile's rows of dW
    int it = 0;
    bool ok = true;
    for (uint32_t u = unit0; u < unit1 && ok; u += stride) {
      const Job j = job_of<N>(P, u);
      if (j.nkb == 0 && (j.part >= 0 || a.accumulate)) continue;
      const int acc = it % C::kAcc;
      if (j.nkb > 0) {
        // Every other wait is for one k-block or one epilogue, this one for a tile: its limit grows
        // with the k-blocks (470 to 950 cycles each; a tile of 4.3 million outlasts the fixed part).
        const long long limit = kWaitLimitCycles + 4096LL * j.nkb;
        if (!__all_sync(0xffffffffu,
                        mbar_wait(&tfull[acc], static_cast<uint32_t>((it / C::kAcc) & 1), abort_flag, limit))) {
          ok = false;
          if (lane == 0) {
            set_error(a.status_dev, MUON_ERR_TIMEOUT);
            *abort_flag = 1;
          }
          break;
        }
        ++it;
        tc_fence_after();
      }
      const int c0 = rank * 128 + w * 32 + lane, col = j.i0 + c0;
      const int rows = min(N / 2, static_cast<int>(a.out) - j.o0 - half);
#pragma unroll 1
      for (int c = 0; c < N / 64; ++c) {
        uint32_t v[32];
        __syncwarp();  // lanes past the last column skip the stores: the load takes the warp whole
        if (j.nkb > 0) {
          tmem_ld32(tmem + (static_cast<uint32_t>(w * 32) << 16) + static_cast<uint32_t>(acc * N + half + c * 32), v);
          tmem_wait_ld();
          if (c == N / 64 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (rank == 0) mbar_arrive(&tempty[acc]);
              else mbar_arrive_peer(peer_addr(&tempty[acc], 0));
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0;
        }
        const int n = rows - c * 32;
        if (col >= a.in || n <= 0) continue;
        if (j.part >= 0) {
          float* p = P.parts + static_cast<int64_t>(j.part) * (N * kIn) + (half + c * 32) * kIn + c0;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < n) p[i * kIn] = __uint_as_float(v[i]);
        } else {
          const int64_t at = j.g * a.stride_w + (j.o0 + half + c * 32) * a.ld_w + col;
          if (a.w_dtype == MUON_F32) write_rows(static_cast<float*>(a.dW) + at, a.ld_w, n, a.accumulate != 0, v);
          else write_rows(static_cast<uint16_t*>(a.dW) + at, a.ld_w, n, a.accumulate != 0, v);
        }
      }
    }
  }

  __syncthreads();
  cluster_sync_all();  // no cross-CTA signal or TMEM access outstanding
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Adds the partial sums of the split tiles in order: a block per 4 rows of a tile, a thread per
// 4 columns of one row, kBatch partial sums in flight.
template <int N>
__global__ void __launch_bounds__(kIn) wgrad_join_kernel(const __grid_constant__ WgradParams P) {
  constexpr int kBatch = 10;
  const muon_weight_grad_t& a = P.a;
  const int64_t r = blockIdx.x / (N / 4);
  const int row = blockIdx.x % (N / 4) * 4 + threadIdx.x / 64, c0 = threadIdx.x % 64 * 4;
  const Job j = job_of<N>(P, static_cast<uint32_t>(P.s.whole + r * P.s.splits));
  int lo, hi;
  group_range(a, j.g, &lo, &hi);
  const int64_t o = j.o0 + row;
  const int kb = (hi - lo + kTok - 1) / kTok, splits = P.s.splits, cols = static_cast<int>(a.in) - j.i0 - c0;
  if (o >= a.out || cols <= 0) return;
  griddep_wait();  // the partial sums are complete
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* p = P.parts + r * splits * (N * kIn) + row * kIn + c0;
  for (int s0 = 0; s0 < splits; s0 += kBatch) {
    float4 v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int s = s0 + b;
      // a part without tokens has no partial sum (every part has some if there are k-blocks enough)
      const uint32_t ukb = static_cast<uint32_t>(kb);
      const bool have = s < splits && (kb >= splits || ukb * s / splits != ukb * (s + 1) / splits);
      v[b] = have ? __ldcs(reinterpret_cast<const float4*>(p + static_cast<int64_t>(s) * (N * kIn)))
                  : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      sum.x += v[b].x;
      sum.y += v[b].y;
      sum.z += v[b].z;
      sum.w += v[b].w;
    }
  }
  const float x[4] = {sum.x, sum.y, sum.z, sum.w};
  const int64_t at = j.g * a.stride_w + o * a.ld_w + j.i0 + c0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= cols) break;
    if (a.w_dtype == MUON_F32) {
      float* w = static_cast<float*>(a.dW) + at + i;
      put(w, a.accumulate ? *w + x[i] : x[i]);
    } else {
      uint16_t* w = static_cast<uint16_t*>(a.dW) + at + i;
      put(w, a.accumulate ? widen(*w) + x[i] : x[i]);
    }
  }
}

// Tensor map of one operand: tokens x cols, boxes of `row` bytes x 64 tokens, with the 128B
// swizzle for rows of 128 bytes (the third axis has one entry, its stride is never used).
bool encode_tokens_map(CUtensorMap* out, CUtensorMapDataType type, int elem, int row, const void* base,
                       int64_t cols, int64_t tokens, int64_t ld) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(tokens), 1};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * elem), static_cast<cuuint64_t>(ld * elem)};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(row / elem), kTok, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode(out, type, 3, const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE,
                row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

muon_status_t validate_weight_grad(const muon_weight_grad_t* p) {
  if (p == nullptr) return MUON_ERR_INVALID_ARG;
  const muon_weight_grad_t& a = *p;
  if (a.w_dtype != MUON_F32 && a.w_dtype != MUON_BF16) return MUON_ERR_DTYPE;
  const int64_t lim = int64_t(1) << 31;
  // (tokens up to the end of a k-block, rows and columns up to the end of a tile stay below 2^31)
  if (a.tokens < 0 || a.out < 1 || a.in < 1 || a.groups < 1 || a.tokens > lim - kTok || a.out > lim - 512 ||
      a.in > lim - 512 || a.groups > 65535 || a.out * a.in >= lim)
    return MUON_ERR_SHAPE;
  if (a.ld_dy < a.out || a.ld_q < a.in || a.ld_e < (a.in + 31) / 32 || a.ld_w < a.in ||
      a.ld_dy >= lim || a.ld_q >= lim || a.ld_e >= lim || a.ld_w >= lim ||
      a.ld_dy % 8 || a.ld_q % 16 || a.ld_e % 16)
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
        reinterpret_cast<uintptr_t>(a.exps) % 16)
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

template <int N>
cudaError_t launch_wgrad(const WgradParams& P, int dev, int sms, cudaStream_t st) {
  using C = WgradCfg<N>;
  // the shared-memory opt-in is a per-device attribute: set it once on each device
  static std::atomic<uint64_t> attr_devices{0};
  const uint64_t bit = dev < 64 ? (uint64_t{1} << dev) : 0;
  if (bit == 0 || !(attr_devices.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(wgrad_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_devices.fetch_or(bit, std::memory_order_acq_rel);
  }
  const int64_t pairs = P.s.units < sms / 2 ? P.s.units : sms / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, wgrad_kernel<N>, P);
  if (e != cudaSuccess || P.s.left == 0) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(P.s.left * (N / 4)), 1, 1);
  cfg.blockDim = dim3(kIn, 1, 1);
  cfg.dynamicSmemBytes = 0;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, wgrad_join_kernel<N>, P);
}

}  // namespace
}  // namespace muon

extern "C" MUON_API size_t muon_weight_grad_workspace_size(const muon_weight_grad_t* a) {
  using namespace muon;
  if (validate_weight_grad(a) != MUON_OK) return 0;
  const WgradSplit s = split_of(*a);
  return static_cast<size_t>(s.left * s.splits) * s.part_bytes;
}

extern "C" MUON_API muon_status_t muon_weight_grad(const muon_weight_grad_t* a, void* workspace,
                                                   size_t ws_bytes, void* stream) {
  using namespace muon;
  const muon_status_t v = validate_weight_grad(a);
  if (v != MUON_OK) return v;
  WgradParams P;
  std::memset(&P, 0, sizeof(P));
  P.a = *a;
  P.s = split_of(*a);
  if (P.s.units >= (int64_t(1) << 31)) return MUON_ERR_SHAPE;
  const size_t need = static_cast<size_t>(P.s.left * P.s.splits) * P.s.part_bytes;
  if (need > 0 && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 || ws_bytes < need))
    return MUON_ERR_WORKSPACE;
  P.parts = static_cast<float*>(workspace);
  int dev = 0, sms = 0;
  const muon_status_t d = current_device(&dev, &sms);
  if (d != MUON_OK) return d;
  if (a->tokens > 0 &&
      !(encode_tokens_map(&P.ty, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, 128, a->dY, a->out, a->tokens, a->ld_dy) &&
        encode_tokens_map(&P.tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 128, a->q, a->in, a->tokens, a->ld_q) &&
        encode_tokens_map(&P.te, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, kEBytesRow, a->exps, (a->in + 31) / 32, a->tokens,
                          a->ld_e)))
    return MUON_ERR_CUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = P.s.n == 384   ? launch_wgrad<384>(P, dev, sms, st)
                        : P.s.n == 256 ? launch_wgrad<256>(P, dev, sms, st)
                                       : launch_wgrad<128>(P, dev, sms, st);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

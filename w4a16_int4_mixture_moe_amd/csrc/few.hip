// A whole MoE layer for a few tokens in two kernels, no routing buffers:
//
//   h[t, e]  = bf16(silu(x_t . Wg_e) * (x_t . Wu_e))            few_gate_up_kernel
//   y[t]     = bf16(sum over t's local experts of w[t, e] (W2_e . h[t, e]))   few_down_kernel
//
// for INT4 weights with bf16 group-32 scales or MXFP4 weights, bf16
// activations, fp32 accumulation.  At a few tokens the time is the weight
// stream of the touched experts plus launches, so: every touched expert's
// weights are read once per block of 16 of its rows, straight into registers
// in operand order; there is no align kernel, no combine kernel and no
// partial sum in memory.
//
// Measured on MI355X (whole calls, graph replays; bytes are the touched
// experts' weights and scales; a 2 GiB copy 4.9 TB/s): 16 tokens on an INT4
// EP8 share (48 of 384 experts, H 7168, I 2048) 107 us where the routing
// touches 17 experts (421 MB, 3.9 TB/s), 84 us over routings that touch 12.8;
// 37 tokens x 16 on an MXFP4 share of 112 of 896 experts, 47 touched, 221 us
// (1111 MB, 5.0 TB/s); one token on a TP8 slice (I 256) 18 us, MXFP4 19 us
// over many routings, of which the weights' bytes are 5.  HBM bounds the MXFP4
// call.  The INT4 one keeps the vector units busy (issue 61 % of the time in
// gate/up, 46 % in down; the dequantisation takes 17 instructions for 8
// weights) and reads 1.15 times its bytes: each wave's ring asks for up to D
// chunks past its last one.  The single token is two kernels of dependent
// loads (10.1 + 7.0 us): ids, block search, then the first weight.
//
// Both weight layouts give lane l = 16 g + i the 32 consecutive K of row i
// that scale block 4 c + g covers, eight codes a word, so one dequantised
// word is a v_mfma_f32_16x16x32_bf16 operand and only the dequantisation
// differs: (q - 8) s rounded to bf16 for INT4 (dequant8), and for MXFP4
// gfx950's v_cvt_scalef32_pk_bf16_fp4, exact (an E2M1 value times a power of
// two is a bf16 number).
//
// Rows.  An expert's tokens are a 64-bit mask (at most 64 tokens), so a token
// that lists an expert twice is one row, whose weights add up; the rows are
// taken 16 at a time in token order, each such block is one MFMA operand, and
// a block's weights are read once.  Every workgroup of the first kernel works
// the blocks out for itself from the ids (one read of them, then LDS), so no
// launch goes before it; it leaves them in the workspace for the second.
#include <algorithm>
#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"
#include "tile_common.hpp"

namespace w4a16 {

namespace {

constexpr int kFewWaves = 8;
constexpr int kFewThreads = kFewWaves * kWave;
static_assert(kFewMaxSlots == 2 * kFewThreads && kFewMaxTokens <= 64, "two slots a thread, a bit a token");
// workgroups of the gate/up kernel, two on each of 256 CUs: with a workgroup
// for every (slot, tile pair) instead, those with nothing to do held the CUs
// for as long as the others took (139 -> 101 us on the INT4 share above)
constexpr int kFewGroups = 512;
// The down kernel takes two column tiles a workgroup (a deeper ring, one
// workgroup per CU, half the work a block costs besides its weights) where
// that leaves most CUs a workgroup and each wave several units.  Measured on
// MI355X, whole call, one / two tiles: 16 tokens on an INT4 EP8 share 93.8 /
// 88.8 us, 37 x 16 on an MXFP4 share 278 / 264 us; but one token on a TP8
// slice 19.4 / 22.9 us (each wave then has two units).
constexpr int kFewWideDown = 192;
constexpr int kFewWideUnits = 512;

// ---- the two weight kinds: K chunk c of one packed 16-row tile

struct Int4Weights {
  __device__ static __forceinline__ int64_t scale_tile_bytes(int KC) { return (int64_t)((KC + 1) / 2) * (kWave * 4); }
  __device__ static __forceinline__ uint32_t load_scale(gptr_t tile, int c, int lane) {
    return gload_u32(tile + (int64_t)(c >> 1) * (kWave * 4) + lane * 4);
  }
  DequantMasks masks;
  __device__ __forceinline__ Int4Weights() : masks(make_dequant_masks()) {}
  __device__ __forceinline__ void operands(const u32x4_t& w, uint32_t sw, int c, bf16x8_t (&A)[4]) const {
    const float s = __builtin_bit_cast(float, (c & 1) ? (sw & 0xFFFF0000u) : (sw << 16));
#pragma unroll
    for (int j = 0; j < 4; ++j) A[j] = dequant8(w[j], s, -1032.0f * s, 0.0625f * s, -72.0f * s, masks);
  }
};

struct Mxfp4Weights {
  __device__ static __forceinline__ int64_t scale_tile_bytes(int KC) { return (int64_t)KC * kWave; }
  __device__ static __forceinline__ uint32_t load_scale(gptr_t tile, int c, int lane) {
    return *reinterpret_cast<const __attribute__((address_space(1))) uint8_t*>(tile + (int64_t)c * kWave + lane);
  }
  __device__ __forceinline__ void operands(const u32x4_t& w, uint32_t sb, int, bf16x8_t (&A)[4]) const {
    const float s = __builtin_bit_cast(float, sb << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) A[j] = mxfp4_to_bf16x8(w[j], s);
  }
};

// 32 bf16 of K chunk c for this lane (block g of the chunk) as four operand
// words.  Always four loads: a load that a lane or a branch may skip would
// make the compiler count fewer loads in flight and wait too early.  Lanes
// past the block's rows read its first row, which only reaches columns that
// nothing reads; lanes past K (a ragged last chunk) read the row's start, and
// clear_tail makes zeros of that before it is used.
__device__ __forceinline__ void load_rows(gptr_t row, int c, int g, int K, bf16x8_t (&B)[4]) {
  const int k = c * kChunk + g * kGroup;
  const gptr_t p = row + (k < K ? k * 2 : 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) B[j] = __builtin_bit_cast(bf16x8_t, gload_u32x4(p + 16 * j));
}

__device__ __forceinline__ void clear_tail(int c, int g, int K, bf16x8_t (&B)[4]) {
  if ((c + 1) * kChunk <= K) return;                    // the same for the whole wave
  const bool in = c * kChunk + g * kGroup < K;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const u32x4_t v = __builtin_bit_cast(u32x4_t, B[j]);
    B[j] = __builtin_bit_cast(bf16x8_t, in ? v : u32x4_t{0u, 0u, 0u, 0u});
  }
}

// ------------------------------------------------------------ gate / up

struct GateUpSmem {
  unsigned long long tokens[kFewMaxExperts];            // of each expert held here, one bit each
  uint32_t wave_sum[kFewWaves];
  FewBlock block[kFewMaxSlots];
  uint8_t count[kFewMaxSlots];                          // rows of each block
  uint8_t token[kFewMaxSlots][16];                      // their tokens
  f32x4_t red[2][kFewWaves][2][kWave];
};

// The blocks of rows, from the ids: numbered by expert, then by token.
// Returns their number.
__device__ __forceinline__ int find_blocks(const FewParams& p, GateUpSmem& sm) {
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int S = p.T * p.topk;
  static_assert(kFewMaxExperts == 2 * kFewThreads, "two experts a thread");
  uint32_t expert[2];                                   // id - first: from E upwards, not held here
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = tid + q * kFewThreads;
    expert[q] = i < S ? (uint32_t)p.topk_ids[i] - (uint32_t)p.first : ~0u;
    sm.tokens[i] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q)
    if (expert[q] < (uint32_t)p.E)                      // bits, not a sum: the order of the updates is nothing
      atomicOr(&sm.tokens[expert[q]], 1ull << ((tid + q * kFewThreads) / p.topk));
  __syncthreads();
  // blocks (high half) and rows (low half) of the experts before this thread's two
  unsigned long long mask[2];
  uint32_t own[2], before = 0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    mask[q] = sm.tokens[2 * tid + q];
    const uint32_t rows = __popcll(mask[q]);
    own[q] = (rows + 15) / 16 << 16 | rows;
    before += own[q];
  }
  const uint32_t both = before;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const uint32_t v = __shfl_up(before, d);
    if (lane >= d) before += v;
  }
  if (lane == kWave - 1) sm.wave_sum[wave] = before;
  before -= both;
  __syncthreads();
  uint32_t total = 0;
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w) {
    if (w < wave) before += sm.wave_sum[w];
    total += sm.wave_sum[w];
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    int b = before >> 16, row = before & 0xFFFF;
    unsigned long long m = mask[q];
    for (int left = __popcll(m); left > 0; left -= 16, ++b) {
      const int n = min(left, 16);
      sm.block[b] = FewBlock{2 * tid + q, row};
      sm.count[b] = (uint8_t)n;
      for (int r = 0; r < n; ++r, ++row, m &= m - 1) sm.token[b][r] = (uint8_t)__builtin_ctzll(m);
    }
    before += own[q];
  }
  __syncthreads();
  return (int)(__builtin_amdgcn_readfirstlane(total) >> 16);
}

// A barrier for LDS alone: the loads in flight for later chunks stay in
// flight (__syncthreads waits for every one of them).
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// step(0), step(1), ..., step(D - 1), the index a compile-time constant (a
// ring of registers takes no other).  A loop over whole turns of the ring
// with its only exit at the end: with an exit after every step the compiler
// waited for all loads once a turn.
template <int D, int I = 0, typename Step>
__device__ __forceinline__ void ring_turn(Step&& step) {
  if constexpr (I < D) {
    step(std::integral_constant<int, I>{});
    ring_turn<D, I + 1>(step);
  }
}

// Items (block, tile pair), dealt round robin: 16 gate and 16 up columns of
// the block's rows over all of K, the waves splitting the K chunks; their
// sums meet in LDS in wave order, and the waves take turns finishing.  A wave
// sees its chunks of all its items as one sequence and keeps D of them in
// flight across the items' ends.
// PARTS = 2 (few items): an item is half a pair, rows 8 h .. 8 h + 7 of the
// gate and the up tile as the two halves of one operand, so twice as many
// workgroups share the dequantisation.
template <typename Weights, int PARTS, int D, int kPerCU>
__global__ __launch_bounds__(kFewThreads, 2 * kPerCU) void few_gate_up_kernel(const FewParams p) {
  __shared__ GateUpSmem sm;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int g = lane >> 4;
  const int blocks = find_blocks(p, sm);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.blocks = blocks;
  constexpr int R = 2 / PARTS;                          // operands a chunk
  const int pairs = p.I / kRowTile * PARTS;             // items of a block
  const int total = blocks * pairs, grid = gridDim.x;
  if ((int)blockIdx.x >= total) return;
  const int items = (total - 1 - (int)blockIdx.x) / grid + 1;
  const int KC = p.KC1;
  const int c0 = (int)((int64_t)wave * KC / kFewWaves);
  const int share = (int)((int64_t)(wave + 1) * KC / kFewWaves) - c0;
  const int nc = max(share, 1);                         // a wave without a chunk loads one and adds nothing
  const gptr_t xbase = uniform_ptr(p.x);
  const Weights weights;

  // the chunk to load next
  gptr_t wbase[R], sbase[R], xrow;
  int half = 0, next = 0, next_item = blockIdx.x;
  auto seek = [&](int item) {
    const int b = item / pairs, pair = item - b * pairs;
    const int expert = __builtin_amdgcn_readfirstlane(sm.block[b].expert);
    const int r = (lane & 15) < (int)sm.count[b] ? lane & 15 : 0;
    xrow = xbase + (int64_t)sm.token[b][r] * p.H * 2;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t tile = (int64_t)expert * (p.I / 8) + 2 * (pair / PARTS) + r;
      wbase[r] = uniform_ptr(p.w1 + tile * KC * (kWave * 16));
      sbase[r] = uniform_ptr(p.s1 + tile * Weights::scale_tile_bytes(KC));
    }
    half = pair % PARTS * 8;
  };
  // this lane's row of the operand: its own of each tile, or row half + l % 8
  // of the gate (l % 16 < 8) or the up tile, which follows it
  const bool up = PARTS == 2 && (lane & 8);
  const int64_t w_up = up ? (int64_t)KC * (kWave * 16) : 0, s_up = up ? Weights::scale_tile_bytes(KC) : 0;
  u32x4_t w[D][R];
  uint32_t sw[D][R];
  bf16x8_t x[D][4];
  auto issue = [&](auto st_) {
    constexpr int st = decltype(st_)::value;
    const int c = c0 + next;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int from = PARTS == 2 ? (lane & 0x37) + half : lane;
      w[st][r] = gload_u32x4(wbase[r] + (int64_t)c * (kWave * 16) + (w_up + from * 16));
      sw[st][r] = Weights::load_scale(sbase[r] + s_up, c, from);
    }
    load_rows(xrow, c, g, p.H, x[st]);
    __builtin_amdgcn_sched_barrier(0);
    if (++next == nc) {                                 // past the last item its chunks come again, not used
      next = 0;
      next_item += grid;
      if (next_item < total) seek(next_item);
    }
  };

  f32x4_t acc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  int c = 0, n = 0;
  // the item's last chunk is done: two buffers and one barrier an item (the
  // buffer written here was last read before the previous item's barrier)
  auto finish = [&]() {
    f32x4_t (&red)[kFewWaves][2][kWave] = sm.red[n & 1];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      red[wave][r][lane] = acc[r];
      acc[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    lds_barrier();
    if (wave != n % kFewWaves) return;
    const int item = blockIdx.x + n * grid;
    const int b = item / pairs, pair = item - b * pairs;
    const int r = lane & 15;
    const bool valid = r < (int)sm.count[b];
    const FewBlock blk = sm.block[b];
    if (pair == 0 && lane < 16) {
      // the block for the down kernel: each row's token and its weight for the expert
      FewRow row{-1, 0.f};
      if (valid) {
        row.token = sm.token[b][r];
        const int32_t* ids = p.topk_ids + row.token * p.topk;
        const float* wts = p.topk_weights + row.token * p.topk;
#pragma unroll 4
        for (int j = 0; j < p.topk; ++j) {
          const float wt = wts[j];
          row.weight += ids[j] == p.first + blk.expert ? wt : 0.f;
        }
      }
      p.rows[b * 16 + r] = row;
      if (lane == 0) p.plan[b] = blk;
    }
    // columns 4 g .. 4 g + 3 of gate and up; of half a pair: the gate's in
    // lanes g = 0, 1 and the up's in g = 2, 3
    if (!valid || (PARTS == 2 && g >= 2)) return;
    f32x4_t gu[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int from = lane + (PARTS == 2 ? 32 * r : 0), q = PARTS == 2 ? 0 : r;
      gu[r] = red[0][q][from];
#pragma unroll
      for (int v = 1; v < kFewWaves; ++v) gu[r] += red[v][q][from];
    }
    // one rounding, to the bf16 the down product's operand holds
    uint2 o;
    o.x = pack_bf16x2(silu_mul(gu[0][0], gu[1][0]), silu_mul(gu[0][1], gu[1][1]));
    o.y = pack_bf16x2(silu_mul(gu[0][2], gu[1][2]), silu_mul(gu[0][3], gu[1][3]));
    *reinterpret_cast<uint2*>(p.h + (int64_t)(blk.h_row + r) * p.I + pair * (kRowTile / PARTS) + 4 * g) = o;
  };
  seek(blockIdx.x);
  ring_turn<D>(issue);
  for (int left = items * nc; left > 0; left -= D) ring_turn<D>([&](auto st_) {
    constexpr int st = decltype(st_)::value;            // steps past the last chunk finish nothing
    clear_tail(c0 + c, g, p.H, x[st]);
    if (share > 0)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      bf16x8_t A[4];
      weights.operands(w[st][r], sw[st][r], c0 + c, A);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[j], x[st][j], acc[r], 0, 0, 0);
    }
    issue(st_);
    if (++c == nc) {
      c = 0;
      if (n < items) finish();
      ++n;
    }
  });
}

// ------------------------------------------------------------ down

// Workgroup n: 16 NT output columns of every token.  The (block, K chunk)
// units of all blocks are split evenly over the waves, which keep D of theirs
// in flight; a wave adds each of its blocks' rows, times the row's weight, to
// its totals (token t in column t % 16 of total t / 16), and the waves'
// totals meet in LDS in wave order.
constexpr int kStage = 16;                              // blocks staged at a time

template <int MT, int NT>
struct DownSmem {
  FewRow rows[kFewWaves][kStage * 16];                  // of each wave's next blocks
  FewBlock block[kFewWaves][kStage];
  f32x4_t red[kFewWaves][NT * MT][kWave];
};

template <typename Weights, int MT, int NT, int D, int kPerCU>
__global__ __launch_bounds__(kFewThreads, 2 * kPerCU) void few_down_kernel(const FewParams p) {
  __shared__ DownSmem<MT, NT> sm;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int KC = p.KC2;
  const int64_t units = (int64_t)*p.blocks * KC;
  const int u0 = (int)(wave * units / kFewWaves), u1 = (int)((wave + 1) * units / kFewWaves);
  const int g = lane >> 4, col = lane & 15;
  const int tiles = p.H / kRowTile;
  const int nt = NT * (int)blockIdx.x;                  // the first of the workgroup's tiles
  const gptr_t hbase = uniform_ptr(p.h);
  const Weights weights;
  f32x4_t tot[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int t = 0; t < MT; ++t) tot[i][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (u0 < u1) {
    const int last = (u1 - 1) / KC;
    int blk = u0 / KC, next = u0 - blk * KC;            // the unit to load next
    int staged = blk;                                   // blocks [staged, staged + kStage) are in LDS
    gptr_t wbase[NT], sbase[NT], hrow;
    FewRow row;
    // the wave's own part of LDS: its accesses stay in order, no barrier
    auto stage = [&]() {
      const int n = min(kStage, last + 1 - staged);
      for (int i = lane; i < n * 16; i += kWave) sm.rows[wave][i] = p.rows[staged * 16 + i];
      if (lane < n) sm.block[wave][lane] = p.plan[staged + lane];
      __builtin_amdgcn_wave_barrier();
    };
    auto seek = [&]() {
      if (blk == staged + kStage) {
        staged = blk;
        __builtin_amdgcn_wave_barrier();
        stage();
      }
      row = sm.rows[wave][(blk - staged) * 16 + col];
      const FewBlock block = sm.block[wave][blk - staged];
      const int64_t tile0 = (int64_t)__builtin_amdgcn_readfirstlane(block.expert) * tiles;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        wbase[i] = uniform_ptr(p.w2 + (tile0 + nt + i) * KC * (kWave * 16));
        sbase[i] = uniform_ptr(p.s2 + (tile0 + nt + i) * Weights::scale_tile_bytes(KC));
      }
      hrow = hbase + (int64_t)(block.h_row + (row.token >= 0 ? col : 0)) * p.I * 2;
    };
    stage();
    u32x4_t w[D][NT];
    uint32_t sw[D][NT];
    FewRow rows[D];
    bf16x8_t x[D][4];
    auto issue = [&](auto st_) {
      constexpr int st = decltype(st_)::value;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        w[st][i] = gload_u32x4(wbase[i] + (int64_t)next * (kWave * 16) + lane * 16);
        sw[st][i] = Weights::load_scale(sbase[i], next, lane);
      }
      load_rows(hrow, next, g, p.I, x[st]);
      rows[st] = row;
      __builtin_amdgcn_sched_barrier(0);
      if (++next == KC) {                               // past the last block its chunks come again, not used
        next = 0;
        if (blk < last) {
          ++blk;
          seek();
        }
      }
    };
    seek();
    ring_turn<D>(issue);
    f32x4_t acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    int u = u0, c = u0 % KC;
    while (u < u1) ring_turn<D>([&](auto st_) {
      constexpr int st = decltype(st_)::value;          // units past the last add nothing
      clear_tail(c, g, p.I, x[st]);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        bf16x8_t A[4];
        weights.operands(w[st][i], sw[st][i], c, A);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[j], x[st][j], acc[i], 0, 0, 0);
      }
      const FewRow mine = rows[st];
      issue(st_);
      if (++u > u1) return;
      if (++c == KC || u == u1) {                       // the block's (or the wave's) last chunk
        c = 0;
        const int n = __popcll(__ballot(mine.token >= 0)) / 4;
        for (int r = 0; r < n; ++r) {                   // valid rows come first
          const int t = __builtin_amdgcn_readlane(mine.token, r);
          const float wt = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, mine.weight), r));
          f32x4_t v[NT];
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) v[i][q] = wt * __shfl(acc[i][q], 16 * g + r);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int q = 0; q < 4; ++q) tot[i][m][q] += 16 * m + col == t ? v[i][q] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
    });
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) sm.red[wave][i * MT + m][lane] = tot[i][m];
  __syncthreads();
  if (wave >= NT * MT) return;                          // one wave for each (tile, 16 tokens)
  f32x4_t y = sm.red[0][wave][lane];
#pragma unroll
  for (int v = 1; v < kFewWaves; ++v) y += sm.red[v][wave][lane];
  const int t = 16 * (wave % MT) + col;
  const int tile = nt + wave / MT;
  if (t >= p.T) return;
  uint2 o;
  o.x = pack_bf16x2(y[0], y[1]);
  o.y = pack_bf16x2(y[2], y[3]);
  *reinterpret_cast<uint2*>(p.out + (int64_t)t * p.H + tile * kRowTile + 4 * g) = o;
}

template <typename Weights>
hipError_t launch_kind(const FewParams& p, hipStream_t stream) {
  // for as many blocks as there are slots: which of them are held here only
  // the device knows, so a share counts more items than it will have
  const int64_t items = (int64_t)p.I / kRowTile * p.T * p.topk;
  const dim3 up((unsigned)std::min<int64_t>(items, kFewGroups)), down(p.H / kRowTile), block(kFewThreads);
  // halves of pairs where twice the items still fit one workgroup per CU:
  // one token on a TP8 slice (128 items) 19.5 -> 18.3 us a call; 256 items
  // 23.6 -> 29.2 us, so not there
  if (items <= kFewGroups / 4)
    hipLaunchKernelGGL((few_gate_up_kernel<Weights, 2, 7, 1>), dim3((unsigned)(2 * items)), block, 0, stream, p);
  else
    hipLaunchKernelGGL((few_gate_up_kernel<Weights, 1, 3, 2>), up, block, 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.H / kRowTile >= 2 * kFewWideDown && (int64_t)p.T * p.topk * p.KC2 >= kFewWideUnits) {
    const dim3 half(p.H / kRowTile / 2);                // H, a K of the gate/up weight, is a multiple of 32
    if (p.T <= 16)
      hipLaunchKernelGGL((few_down_kernel<Weights, 1, 2, 6, 1>), half, block, 0, stream, p);
    else if (p.T <= 32)
      hipLaunchKernelGGL((few_down_kernel<Weights, 2, 2, 6, 1>), half, block, 0, stream, p);
    else
      hipLaunchKernelGGL((few_down_kernel<Weights, 4, 2, 5, 1>), half, block, 0, stream, p);
  } else if (p.T <= 16) {
    hipLaunchKernelGGL((few_down_kernel<Weights, 1, 1, 3, 2>), down, block, 0, stream, p);
  } else if (p.T <= 32) {
    hipLaunchKernelGGL((few_down_kernel<Weights, 2, 1, 3, 2>), down, block, 0, stream, p);
  } else {
    hipLaunchKernelGGL((few_down_kernel<Weights, 4, 1, 3, 2>), down, block, 0, stream, p);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few_tokens(bool mxfp4, const FewParams& p, hipStream_t stream) {
  return mxfp4 ? launch_kind<Mxfp4Weights>(p, stream) : launch_kind<Int4Weights>(p, stream);
}

}  // namespace w4a16

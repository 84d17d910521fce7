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
// Both weight layouts give lane l = 16 g + i the 32 consecutive K of row i
// that scale block 4 c + g covers, eight codes a word, so one dequantised
// word is a v_mfma_f32_16x16x32_bf16 operand and only the dequantisation
// differs: (q - 8) s rounded to bf16 for INT4 (dequant8), and for MXFP4
// gfx950's v_cvt_scalef32_pk_bf16_fp4, exact (an E2M1 value times a power of
// two is a bf16 number).
//
// Rows.  The routed slots of expert e are taken 16 at a time in slot order;
// the first slot of each such block is its leader and stands for the block.
// A token that lists an expert twice is one row whose weights add up.
#include "device_common.hpp"
#include "launch.hpp"
#include "tile_common.hpp"

namespace w4a16 {

namespace {

constexpr int kFewWaves = 8;
constexpr int kFewThreads = kFewWaves * kWave;
constexpr int kSlotWords = kFewMaxSlots / kWave;       // ballot words over the slots
static_assert(kFewMaxSlots == 2 * kFewThreads, "two slots a thread");

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
// words; zeros where `on` is false
__device__ __forceinline__ void load_rows(gptr_t row, int c, bool on, bf16x8_t (&B)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (on) v = gload_u32x4(row + (int64_t)c * (kChunk * 2) + 16 * j);
    B[j] = __builtin_bit_cast(bf16x8_t, v);
  }
}

// ------------------------------------------------------------ gate / up

struct GateUpSmem {
  unsigned long long match[kSlotWords];                 // slots of this expert, one bit each
  int row[16];                                          // slot of each column, -1 = none
  f32x4_t red[kFewWaves][2][kWave];
};

// Workgroup (tile pair, slot): if the slot leads a block of its expert, the
// block's 16 gate and 16 up columns over all of K, the waves splitting the K
// chunks; their sums meet in LDS in wave order.  The workgroups of pair 0
// also leave the block's rows and weights for the down kernel.
template <typename Weights>
__global__ __launch_bounds__(kFewThreads) void few_gate_up_kernel(const FewParams p) {
  constexpr int KB = 4;                                 // chunks in flight per wave
  __shared__ GateUpSmem sm;
  const int pair = blockIdx.x, s = blockIdx.y;
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int S = p.T * p.topk;
  const int id = p.topk_ids[s];
  const int expert = __builtin_amdgcn_readfirstlane(id - p.first);
  if ((unsigned)expert >= (unsigned)p.E) {              // not held here
    if (pair == 0 && tid == 0) p.leader[s] = 0;
    return;
  }
  // this expert's slots, the first of each token only
  bool hit[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = tid + q * kFewThreads;
    hit[q] = i < S && p.topk_ids[i] == id;
    if (hit[q])
      for (int j = i - i % p.topk; j < i; ++j)
        if (p.topk_ids[j] == id) hit[q] = false;
    const unsigned long long m = __ballot(hit[q]);
    if (lane == 0) sm.match[q * kFewWaves + wave] = m;
  }
  if (tid < 16) sm.row[tid] = -1;
  __syncthreads();
  auto position = [&](int i) {                          // slots of this expert before slot i
    int n = 0;
    for (int q = 0; q < i / kWave; ++q) n += __popcll(sm.match[q]);
    return n + __popcll(sm.match[i / kWave] & ((1ull << (i % kWave)) - 1ull));
  };
  const int rank = position(s);
  const bool lead = ((sm.match[s / kWave] >> (s % kWave)) & 1ull) && rank % 16 == 0;
  if (!lead) {
    if (pair == 0 && tid == 0) p.leader[s] = 0;
    return;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q)
    if (hit[q]) {
      const int i = tid + q * kFewThreads;
      const int n = position(i) - rank;
      if (n >= 0 && n < 16) sm.row[n] = i;
    }
  __syncthreads();
  const int slot = sm.row[lane & 15];
  if (pair == 0 && tid < 16) {
    float w = 0.f;
    if (slot >= 0) {
      const int i0 = slot - slot % p.topk;
      for (int j = i0; j < i0 + p.topk; ++j)
        if (p.topk_ids[j] == id) w += p.topk_weights[j];
    }
    p.rows[s * 16 + tid] = FewRow{slot, w};
    if (tid == 0) p.leader[s] = 1;
  }

  const int KC = p.KC1;
  const int c0 = (int)((int64_t)wave * KC / kFewWaves), c1 = (int)((int64_t)(wave + 1) * KC / kFewWaves);
  gptr_t wbase[2], sbase[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int64_t tile = (int64_t)expert * (p.I / 8) + 2 * pair + r;
    wbase[r] = uniform_ptr(p.w1 + tile * KC * (kWave * 16)) + lane * 16;
    sbase[r] = uniform_ptr(p.s1 + tile * Weights::scale_tile_bytes(KC));
  }
  const int g = lane >> 4;
  const gptr_t xrow = uniform_ptr(p.x) + (int64_t)(max(slot, 0) / p.topk) * p.H * 2 + g * 64;
  const Weights weights;
  f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  for (int cb = c0; cb < c1; cb += KB) {
    u32x4_t w[KB][2];
    uint32_t sw[KB][2];
    bf16x8_t x[KB][4];
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int c = min(cb + i, c1 - 1);               // past c1: a repeated load, multiplied by zeros
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        w[i][r] = gload_u32x4(wbase[r] + (int64_t)c * (kWave * 16));
        sw[i][r] = Weights::load_scale(sbase[r], c, lane);
      }
      load_rows(xrow, c, slot >= 0 && cb + i < c1 && c * kChunk + g * kGroup < p.H, x[i]);
    }
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      if (cb + i >= c1) break;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        bf16x8_t A[4];
        weights.operands(w[i][r], sw[i][r], cb + i, A);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[j], x[i][j], acc[r], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) sm.red[wave][r][lane] = acc[r];
  __syncthreads();
  if (wave != 0 || slot < 0) return;
  f32x4_t gu[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    gu[r] = sm.red[0][r][lane];
#pragma unroll
    for (int v = 1; v < kFewWaves; ++v) gu[r] += sm.red[v][r][lane];
  }
  // one rounding, to the bf16 the down product's operand holds
  uint2 o;
  o.x = pack_bf16x2(silu_mul(gu[0][0], gu[1][0]), silu_mul(gu[0][1], gu[1][1]));
  o.y = pack_bf16x2(silu_mul(gu[0][2], gu[1][2]), silu_mul(gu[0][3], gu[1][3]));
  *reinterpret_cast<uint2*>(p.h + (int64_t)slot * p.I + pair * kRowTile + 4 * g) = o;
}

// ------------------------------------------------------------ down

template <int MT>
struct DownSmem {
  unsigned long long lead[kSlotWords];
  int list[kFewMaxSlots];                               // leaders in slot order
  f32x4_t red[kFewWaves][MT][kWave];
};

// Workgroup n: 16 output columns of every token.  The (block, K chunk) units
// of all blocks are split evenly over the waves; a wave adds each of its
// blocks' rows, times the row's weight, to its totals (token t in column
// t % 16 of total t / 16), and the waves' totals meet in LDS in wave order.
template <typename Weights, int MT>
__global__ __launch_bounds__(kFewThreads) void few_down_kernel(const FewParams p) {
  constexpr int KB = 4;                                 // units in flight per wave
  __shared__ DownSmem<MT> sm;
  const int nt = blockIdx.x;
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int S = p.T * p.topk;
  bool lead[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = tid + q * kFewThreads;
    lead[q] = i < S && p.leader[i] != 0;
    const unsigned long long m = __ballot(lead[q]);
    if (lane == 0) sm.lead[q * kFewWaves + wave] = m;
  }
  __syncthreads();
  int blocks = 0;
#pragma unroll
  for (int q = 0; q < kSlotWords; ++q) {
    const unsigned long long m = sm.lead[q];
    if (q % kFewWaves == wave && lead[q / kFewWaves])
      sm.list[blocks + __popcll(m & ((1ull << lane) - 1ull))] = tid + (q / kFewWaves) * kFewThreads;
    blocks += __popcll(m);
  }
  blocks = __builtin_amdgcn_readfirstlane(blocks);
  __syncthreads();

  const int KC = p.KC2;
  const int64_t units = (int64_t)blocks * KC;
  const int u0 = (int)(wave * units / kFewWaves), u1 = (int)((wave + 1) * units / kFewWaves);
  const int g = lane >> 4, col = lane & 15;
  const gptr_t hbase = uniform_ptr(p.h);
  const Weights weights;
  f32x4_t tot[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) tot[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int ub = u0; ub < u1; ub += KB) {
    u32x4_t w[KB];
    uint32_t sw[KB];
    FewRow row[KB];
    int chunk[KB];
    bf16x8_t x[KB][4];
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int u = min(ub + i, u1 - 1);               // past u1: a repeated load, not used
      const int blk = u / KC;
      chunk[i] = u - blk * KC;
      const int s = __builtin_amdgcn_readfirstlane(sm.list[blk]);
      const int64_t tile = (int64_t)(p.topk_ids[s] - p.first) * (p.H / kRowTile) + nt;
      w[i] = gload_u32x4(uniform_ptr(p.w2 + (tile * KC + chunk[i]) * (kWave * 16)) + lane * 16);
      sw[i] = Weights::load_scale(uniform_ptr(p.s2 + tile * Weights::scale_tile_bytes(KC)), chunk[i], lane);
      row[i] = p.rows[s * 16 + col];
    }
#pragma unroll
    for (int i = 0; i < KB; ++i)
      load_rows(hbase + (int64_t)max(row[i].slot, 0) * p.I * 2 + g * 64, chunk[i],
                row[i].slot >= 0 && chunk[i] * kChunk + g * kGroup < p.I, x[i]);
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      if (ub + i >= u1) break;
      bf16x8_t A[4];
      weights.operands(w[i], sw[i], chunk[i], A);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[j], x[i][j], acc, 0, 0, 0);
      if (chunk[i] == KC - 1 || ub + i == u1 - 1) {     // the block's (or the wave's) last chunk
        const int token = row[i].slot / p.topk;         // of this lane's column, where slot >= 0
        const int rows = __popcll(__ballot(row[i].slot >= 0)) / 4;
        for (int r = 0; r < rows; ++r) {                // valid rows come first
          const int t = __builtin_amdgcn_readlane(token, r);
          const float wt = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, row[i].weight), r));
          f32x4_t v;
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = __shfl(acc[q], 16 * g + r);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            if (m == t / 16 && col == t % 16) tot[m] += wt * v;
        }
        acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) sm.red[wave][m][lane] = tot[m];
  __syncthreads();
  if (wave >= MT) return;
  f32x4_t y = sm.red[0][wave][lane];
#pragma unroll
  for (int v = 1; v < kFewWaves; ++v) y += sm.red[v][wave][lane];
  const int t = 16 * wave + col;
  if (t >= p.T) return;
  uint2 o;
  o.x = pack_bf16x2(y[0], y[1]);
  o.y = pack_bf16x2(y[2], y[3]);
  *reinterpret_cast<uint2*>(p.out + (int64_t)t * p.H + nt * kRowTile + 4 * g) = o;
}

template <typename Weights>
hipError_t launch_kind(const FewParams& p, hipStream_t stream) {
  const dim3 up(p.I / kRowTile, p.T * p.topk), down(p.H / kRowTile), block(kFewThreads);
  hipLaunchKernelGGL(few_gate_up_kernel<Weights>, up, block, 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.T <= 16)
    hipLaunchKernelGGL((few_down_kernel<Weights, 1>), down, block, 0, stream, p);
  else if (p.T <= 32)
    hipLaunchKernelGGL((few_down_kernel<Weights, 2>), down, block, 0, stream, p);
  else
    hipLaunchKernelGGL((few_down_kernel<Weights, 4>), down, block, 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few_tokens(bool mxfp4, const FewParams& p, hipStream_t stream) {
  return mxfp4 ? launch_kind<Mxfp4Weights>(p, stream) : launch_kind<Int4Weights>(p, stream);
}

}  // namespace w4a16

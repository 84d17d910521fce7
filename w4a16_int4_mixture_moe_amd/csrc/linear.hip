// One INT4 weight for all rows (a layer's shared projection), with low-rank
// adapters beside it or without: rows in the order of their adapters
// (AdapterParams::order), so that a 16-row tile mixes few of them; results go
// back to the rows' own places.
//
// Up to 64 rows, and more where whole tiles would leave most CUs idle: one or
// two weight tiles a workgroup, its eight waves splitting K (split_product).
// Otherwise the general 64-row tile or, with K a multiple of 128, the prefill
// tiles.
#include <type_traits>

#include "adapter.hpp"
#include "adapter_launch.hpp"
#include "device_common.hpp"
#include "gemm_tile.hpp"
#include "launch.hpp"
#include "prefill_tile.hpp"
#include "tile_common.hpp"

namespace w4a16 {

namespace {

constexpr int kSplitWaves = 8;

template <int MT, int NT, int EPI>
__global__ __launch_bounds__(kSplitWaves * kWave) void linear_split_kernel(const GemmParams p, const AdapterParams q) {
  __shared__ __attribute__((aligned(16))) AdapterSmem<SplitSmem<MT, NT, kSplitWaves>, 16 * MT> sm;
  // the blocks of one pair of weight tiles next to each other: they read the same weights
  const int mb = blockIdx.x % p.grid_blocks, nt = blockIdx.x / p.grid_blocks;
  setup_adapter_rows<MT, kSplitWaves, kRouteDense, EPI>(p, q, mb, sm);
  clear_low(sm);
  __syncthreads();
  f32x4_t acc[NT][1];
  split_product<MT, NT, kSplitWaves>(p, q, sm, 0, nt, acc);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (wave >= MT) return;
  store_tiles<1, NT, EPI>(p, sm.out + 16 * wave, NT * nt, 1u, acc);
}

template <int MT, int NR, int EPI>
__global__ __launch_bounds__(4 * kWave) void linear_tile_kernel(const GemmParams p, const AdapterParams q) {
  constexpr int NW = 4;
  __shared__ __attribute__((aligned(16))) AdapterSmem<TileSmem<MT>, 16 * MT> sm;
  int mb, nt;
  if (!block_of(p, blockIdx.x, p.n_tiles, mb, nt)) return;
  setup_adapter_rows<MT, NW, kRouteDense, EPI>(p, q, mb, sm);
  __syncthreads();
  const int rt_base = nt * (NW * NR) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) * NR;
  run_tile<MT, NR, NW, 2>(
      p, static_cast<TileSmem<MT>&>(sm), 0, nt, active_tiles<MT>(sm), 0, p.KC,
      [&](f32x4_t(&acc)[NR][MT], auto na) { start_from_adapters<MT, NR, decltype(na)::value>(p, q, sm, 0, rt_base, acc); },
      [&](const f32x4_t(&acc)[NR][MT], uint32_t tm) { store_tiles<MT, NR, EPI>(p, sm.out, rt_base, tm, acc); });
}

template <int MT, int NR, int NW, int EPI>
__global__ __launch_bounds__(NW * kWave, 8 / NW) void linear_prefill_kernel(const GemmParams p, const AdapterParams q) {
  using C = PfCfg<MT, NR, NW>;
  __shared__ __attribute__((aligned(16))) AdapterSmem<PfSmem<C::BM>, C::BM> sm;
  int mb, nt;
  if (!block_of(p, blockIdx.x, p.n_tiles, mb, nt)) return;
  setup_adapter_rows<MT, NW, kRouteDense, EPI>(p, q, mb, sm);
  __syncthreads();
  const int rt_base = nt * (NW * NR) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) * NR;
  pf_run<C, false>(
      p, static_cast<PfSmem<C::BM>&>(sm), 0, nt, nt + 1, active_tiles<MT>(sm),
      [&](auto& acc, auto na, int) { start_from_adapters<MT, NR, decltype(na)::value>(p, q, sm, 0, rt_base, acc); },
      [&](const auto& acc, uint32_t tm, int) { store_tiles<MT, NR, EPI>(p, sm.out, rt_base, tm, acc); });
}

typedef void (*LinearKernel)(const GemmParams, const AdapterParams);

constexpr int64_t kTileMinWorkgroups = 256;     // one a CU

hipError_t launch(LinearKernel k, GemmParams p, const AdapterParams& q, int rows, int tiles, int waves, bool split,
                  hipStream_t stream) {
  p.grid_blocks = (int32_t)((q.rows + rows - 1) / rows);
  p.n_tiles = (p.NT + tiles - 1) / tiles;
  p.xcd_group = split ? 0 : xcd_group_for(1, p.n_tiles);
  const int64_t grid = split ? (int64_t)p.grid_blocks * p.n_tiles : grid_of(p, p.n_tiles);
  if (grid > INT32_MAX / (waves * kWave)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(k, dim3((unsigned)grid), dim3(waves * kWave), 0, stream, p, q);
  return hipGetLastError();
}

template <int EPI>
hipError_t launch_of(const GemmParams& p, const AdapterParams& q, hipStream_t stream) {
  constexpr int ONE = EPI == kEpiSilu ? 2 : 1;
  const int64_t T = q.rows;
  auto grid = [&](int rows, int tiles) { return (T + rows - 1) / rows * ((p.NT + tiles - 1) / tiles); };
  if (T <= 16) return launch(linear_split_kernel<1, ONE, EPI>, p, q, 16, ONE, kSplitWaves, true, stream);
  if (T <= 32) return launch(linear_split_kernel<2, 2, EPI>, p, q, 32, 2, kSplitWaves, true, stream);
  if (grid(64, 8) < kTileMinWorkgroups)
    return launch(linear_split_kernel<4, 2, EPI>, p, q, 64, 2, kSplitWaves, true, stream);
  if (p.K % kChunk == 0) {
    if (grid(256, 16) >= kTileMinWorkgroups)
      return launch(linear_prefill_kernel<16, 2, 8, EPI>, p, q, 256, 16, 8, false, stream);
    if (grid(128, 16) >= kTileMinWorkgroups)
      return launch(linear_prefill_kernel<8, 4, 4, EPI>, p, q, 128, 16, 4, false, stream);
  }
  return launch(linear_tile_kernel<4, 2, EPI>, p, q, 64, 8, 4, false, stream);
}

}  // namespace

hipError_t launch_linear(int epilogue, const GemmParams& p, const AdapterParams& q, hipStream_t stream) {
  if (q.rows <= 0) return hipSuccess;
  return epilogue == kEpiSilu ? launch_of<kEpiSilu>(p, q, stream) : launch_of<kEpiStore>(p, q, stream);
}

}  // namespace w4a16

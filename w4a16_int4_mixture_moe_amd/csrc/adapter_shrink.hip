// The first half of a low-rank adapter as a launch of its own (adapter_shrink.hpp).
#include <algorithm>

#include "adapter_launch.hpp"
#include "adapter_shrink.hpp"
#include "device_common.hpp"

namespace w4a16 {

namespace {

__global__ __launch_bounds__(kShrinkThreads, 2) void adapter_shrink_kernel(const ShrinkParams p, const ShrinkGrid grid) {
  shrink_block<4>(p, grid, blockIdx.x);
}

constexpr int64_t kShrinkItems = 2048;          // waves that keep 1024 SIMDs busy
constexpr int kShrinkMaxSlices = 16;

}  // namespace

// K is cut where the 64-row tiles alone leave waves idle, not below four chunks a slice
int shrink_slices(int64_t positions, int32_t width, int32_t KC) {
  const int64_t items = (positions + kShrinkRows - 1) / kShrinkRows * ((width + kShrinkWidth - 1) / kShrinkWidth);
  const int64_t want = (kShrinkItems + std::max<int64_t>(items, 1) - 1) / std::max<int64_t>(items, 1);
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, kShrinkMaxSlices, KC / 4}));
}

hipError_t shrink_grid(const ShrinkParams& p, ShrinkGrid* out) {
  ShrinkGrid grid;
  if (p.ad.L > kMaxAdapters) return hipErrorInvalidValue;
  if (p.order != nullptr && (p.sorted_ids != nullptr || p.positions > kOrderMaxRows)) return hipErrorInvalidValue;
  const int64_t tiles = (p.positions + kShrinkRows - 1) / kShrinkRows;
  grid.parts = (p.ad.slices * p.ad.rank + kShrinkWidth - 1) / kShrinkWidth;
  const int64_t per = tiles * p.ad.ks * grid.parts;
  grid.z = (int32_t)std::max<int64_t>(1, std::min<int64_t>({2 * kShrinkItems / per, kShrinkRows, p.positions}));
  grid.items = per * grid.z;
  const int64_t blocks = (grid.items + kShrinkWaves - 1) / kShrinkWaves + (p.order != nullptr);
  if (blocks > INT32_MAX / kShrinkThreads) return hipErrorInvalidConfiguration;
  grid.blocks = (int32_t)blocks;
  *out = grid;
  return hipSuccess;
}

hipError_t launch_adapter_shrink(const ShrinkParams& p, hipStream_t stream) {
  if (p.positions <= 0 || p.ad.L <= 0) return hipSuccess;
  ShrinkGrid grid;
  const hipError_t e = shrink_grid(p, &grid);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(adapter_shrink_kernel, dim3((unsigned)grid.blocks), dim3(kShrinkThreads), 0, stream, p, grid);
  return hipGetLastError();
}

}  // namespace w4a16

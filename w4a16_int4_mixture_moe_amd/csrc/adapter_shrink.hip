// The first half of a low-rank adapter (adapter.hpp): h_i = s_a A_a x_i in
// fp32 for every row i that has an adapter a, of an expert e where the rows
// are routed (A [L][E][S r][K], S r rows of K).
//
// Few rows are bound by reading A (S r K bf16 of each adapter in use), many by
// reading x.  A wave takes 64 consecutive rows, one slice of K and up to 32
// rows of A; it gathers the rows that share an (adapter, expert) by ballot,
// 16 of them make one v_mfma_f32_16x16x32_bf16 operand against 16 rows of A,
// and each such group is one pass over the slice.  So an A is read once for
// every 64 rows that use it however the requests are mixed, nothing is
// sorted first, and no wave waits for another: sums of one row from different
// slices of K go to different planes of h, which the product's start adds in
// slice order.
//
// Per 128-wide chunk of K lane l = 16 g + i holds 32 consecutive K (64 bytes,
// four 16-byte loads) of row i of A and of x; both sides take the chunk's K in
// the same order.
#include <algorithm>
#include <type_traits>

#include "adapter_launch.hpp"
#include "device_common.hpp"
#include "launch.hpp"

namespace w4a16 {

namespace {

constexpr int kShrinkWaves = 4;
constexpr int kShrinkThreads = kShrinkWaves * kWave;
constexpr int kShrinkRows = 64;                 // positions of a wave
constexpr int kShrinkWidth = 32;                // rows of A of a wave
constexpr int kMaxAdapters = 1024;

struct ShrinkGrid {
  int32_t tiles, z, parts;      // 64-row tiles, waves that share a tile's adapters, parts of A's rows
  int64_t items;
};

// 32 K of this lane's 64 bytes of chunk c; zeros past K
__device__ __forceinline__ void load_k(gptr_t row, int c, int g, int K, bf16x8_t (&v)[4]) {
  const int k = c * kChunk + g * kGroup;
  const gptr_t p = row + (k < K ? k * 2 : 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = __builtin_bit_cast(bf16x8_t, gload_u32x4(p + 16 * j));
}

__device__ __forceinline__ void clear_past(int c, int g, int K, bf16x8_t (&v)[4]) {
  if ((c + 1) * kChunk <= K) return;
  const bool in = c * kChunk + g * kGroup < K;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const u32x4_t b = __builtin_bit_cast(u32x4_t, v[j]);
    v[j] = __builtin_bit_cast(bf16x8_t, in ? b : u32x4_t{0u, 0u, 0u, 0u});
  }
}

// the slice [c0, c1) of 16 M rows of x against 32 rows of A, KB chunks in flight
template <int M, int KB>
__device__ __forceinline__ void shrink_pass(const ShrinkParams& p, const gptr_t (&arow)[2], const gptr_t (&xrow)[M],
                                            int c0, int c1, bool both, f32x4_t (&acc)[M][2]) {
  const int g = (threadIdx.x & (kWave - 1)) >> 4;
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[m][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int cb = c0; cb < c1; cb += KB) {
    bf16x8_t a[KB][2][4], x[KB][M][4];
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int c = min(cb + i, c1 - 1);                // past the slice: loaded again, not used
      load_k(arow[0], c, g, p.K, a[i][0]);
      if (both) load_k(arow[1], c, g, p.K, a[i][1]);
#pragma unroll
      for (int m = 0; m < M; ++m) load_k(xrow[m], c, g, p.K, x[i][m]);
    }
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int c = cb + i;
      if (c >= c1) break;
      clear_past(c, g, p.K, a[i][0]);
      if (both) clear_past(c, g, p.K, a[i][1]);
#pragma unroll
      for (int m = 0; m < M; ++m) clear_past(c, g, p.K, x[i][m]);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int m = 0; m < M; ++m) {
          acc[m][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i][0][q], x[i][m][q], acc[m][0], 0, 0, 0);
          if (both) acc[m][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i][1][q], x[i][m][q], acc[m][1], 0, 0, 0);
        }
    }
  }
}

// The rows in order of their adapters, rows without one last: what makes a
// product's 16-row tiles hold few adapters each.  Rows of one adapter come in
// any order (a row's result does not depend on where it stands).
__device__ __forceinline__ void order_rows(const ShrinkParams& p) {
  __shared__ int start[kMaxAdapters + 1];
  const int L = p.ad.L, T = (int)p.positions;
  for (int b = threadIdx.x; b <= L; b += kShrinkThreads) start[b] = 0;
  __syncthreads();
  auto bucket = [&](int t) {
    const int a = p.ad.ids[t];
    return (unsigned)a < (unsigned)L ? a : L;
  };
  for (int t = threadIdx.x; t < T; t += kShrinkThreads) atomicAdd(&start[bucket(t)], 1);
  __syncthreads();
  if (threadIdx.x < kWave) {                            // exclusive sums, a run of buckets a lane
    const int per = (L + kWave) / kWave;
    const int b0 = min((int)threadIdx.x * per, L + 1), b1 = min(b0 + per, L + 1);
    int own = 0;
    for (int b = b0; b < b1; ++b) own += start[b];
    int incl = own;
    for (int d = 1; d < kWave; d *= 2) {
      const int v = __shfl_up(incl, d);
      if ((int)threadIdx.x >= d) incl += v;
    }
    int run = incl - own;
    for (int b = b0; b < b1; ++b) {
      const int n = start[b];
      start[b] = run;
      run += n;
    }
  }
  __syncthreads();
  for (int t = threadIdx.x; t < T; t += kShrinkThreads) p.order[atomicAdd(&start[bucket(t)], 1)] = t;
}

__global__ __launch_bounds__(kShrinkThreads, 2) void adapter_shrink_kernel(const ShrinkParams p, const ShrinkGrid grid) {
  int block = blockIdx.x;
  if (p.order != nullptr) {
    if (block == 0) {
      order_rows(p);
      return;
    }
    --block;
  }
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t item = (int64_t)block * kShrinkWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (item >= grid.items) return;
  const AdapterParams& q = p.ad;
  const int part = (int)(item % grid.parts);
  int64_t left = item / grid.parts;
  const int z = (int)(left % grid.z);
  left /= grid.z;
  const int ks = (int)(left % q.ks);
  const int64_t pos = (left / q.ks) * kShrinkRows + lane;

  // this lane's row: its (adapter, expert), row of x and row of h
  int key = -1, x_row = 0, h_row = 0;
  if (p.sorted_ids != nullptr) {
    const int64_t end = min(p.positions, (int64_t)*p.num_tokens_padded);
    if (pos < end) {
      const int s = p.sorted_ids[pos];
      const int e = p.expert_ids[pos >> p.block_shift];
      if ((unsigned)s < (unsigned)p.sentinel && (unsigned)e < (unsigned)q.E) {
        const int a = q.ids[s / q.topk];
        if ((unsigned)a < (unsigned)q.L) key = a * q.E + e;
        x_row = p.a_row_div > 0 ? s / p.a_row_div : (int)pos;
        h_row = s;
      }
    }
  } else if (pos < p.positions) {
    const int a = q.ids[pos];
    if ((unsigned)a < (unsigned)q.L) key = a;
    x_row = (int)pos;
    h_row = (int)pos;
  }

  const int width = q.slices * q.rank;
  const int i = lane & 15, g = lane >> 4;
  const int c0 = (int)((int64_t)ks * p.KC / q.ks), c1 = (int)((int64_t)(ks + 1) * p.KC / q.ks);
  const int j0 = part * kShrinkWidth;
  const bool both = j0 + 16 < width;
  float* const plane = q.h + (int64_t)ks * q.rows * width;
  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (kWave - lane);
  uint64_t rest = __ballot(key >= 0);
  for (int d = 0; rest; d = d + 1 == grid.z ? 0 : d + 1) {
    const int k = __builtin_amdgcn_readlane(key, __builtin_ctzll(rest));
    const uint64_t same = __ballot(key == k);
    rest &= ~same;
    if (d != z) continue;
    const int n = __popcll(same);
    // lane j learns the lane of the group's j-th row (a permutation: the others fill the places after them)
    const int place = (same >> lane) & 1 ? __popcll(same & below) : n + __popcll(~same & below);
    const int from = __builtin_amdgcn_ds_permute(place * 4, lane);
    const uint16_t* const base = q.a + (int64_t)k * width * p.K;
    gptr_t arow[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) arow[j] = uniform_ptr(base) + (int64_t)min(j0 + 16 * j + i, width - 1) * p.K * 2;
    float s = 1.f;
    if (q.scale != nullptr) s = q.scale[k / q.E];
    auto rows = [&](int m0, auto tiles, auto chunks) {
      constexpr int M = decltype(tiles)::value, KB = decltype(chunks)::value;
      gptr_t xrow[M];
      int out[M];
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int r = 16 * (m0 + m) + i;
        const int src = __shfl(from, r < n ? r : 0);
        xrow[m] = uniform_ptr(p.x) + (int64_t)__shfl(x_row, src) * p.K * 2;
        out[m] = __shfl(h_row, src);
        if (r >= n) out[m] = -1;
      }
      f32x4_t acc[M][2];
      shrink_pass<M, KB>(p, arow, xrow, c0, c1, both, acc);
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = j0 + 16 * j + 4 * g;
          if (out[m] >= 0 && r < width)
            *reinterpret_cast<f32x4_t*>(plane + (int64_t)out[m] * width + r) = s * acc[m][j];
        }
    };
    if (n > 16) {
      for (int m0 = 0; 16 * m0 < n; m0 += 2) rows(m0, std::integral_constant<int, 2>{}, std::integral_constant<int, 1>{});
    } else {
      rows(0, std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{});
    }
  }
}

constexpr int64_t kShrinkItems = 2048;          // waves that keep 1024 SIMDs busy
constexpr int kShrinkMaxSlices = 8;

}  // namespace

// K is cut where the 64-row tiles alone leave waves idle, not below four chunks a slice
int shrink_slices(int64_t positions, int32_t width, int32_t KC) {
  const int64_t items = (positions + kShrinkRows - 1) / kShrinkRows * ((width + kShrinkWidth - 1) / kShrinkWidth);
  const int64_t want = (kShrinkItems + std::max<int64_t>(items, 1) - 1) / std::max<int64_t>(items, 1);
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, kShrinkMaxSlices, KC / 4}));
}

hipError_t launch_adapter_shrink(const ShrinkParams& p, hipStream_t stream) {
  if (p.positions <= 0 || p.ad.L <= 0) return hipSuccess;
  if (p.ad.L > kMaxAdapters) return hipErrorInvalidValue;
  ShrinkGrid grid;
  const int64_t tiles = (p.positions + kShrinkRows - 1) / kShrinkRows;
  grid.parts = (p.ad.slices * p.ad.rank + kShrinkWidth - 1) / kShrinkWidth;
  const int64_t per = tiles * p.ad.ks * grid.parts;
  grid.z = (int32_t)std::max<int64_t>(1, std::min<int64_t>({2 * kShrinkItems / per, kShrinkRows, p.positions}));
  grid.tiles = (int32_t)tiles;
  grid.items = per * grid.z;
  ShrinkParams q = p;
  if (q.order != nullptr && (p.sorted_ids != nullptr || p.positions > kOrderMaxRows)) return hipErrorInvalidValue;
  const int64_t blocks = (grid.items + kShrinkWaves - 1) / kShrinkWaves + (q.order != nullptr);
  if (blocks > INT32_MAX / kShrinkThreads) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(adapter_shrink_kernel, dim3((unsigned)blocks), dim3(kShrinkThreads), 0, stream, q, grid);
  return hipGetLastError();
}

}  // namespace w4a16

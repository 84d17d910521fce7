// A4W4 tile of 128 rows x 256 weight rows for the grouped layouts: MXFP4
// activations x MXFP4 weights in v_mfma_scale_f32_16x16x128_f8f6f4.
//
// Per 128-wide K chunk a workgroup needs 8 KB of activation codes, 16 KB of
// weight codes and 1.5 KB of scales for 4 x 32 MFMAs of 16 cycles.  Everything
// goes HBM -> LDS by LDS-DMA, three chunks deep, and from there to the
// matrix unit, so no register holds data in flight and two workgroups (two
// waves per SIMD) share a CU: 128 accumulator registers a wave, 76.5 KB of
// LDS a workgroup.  (With the activations through registers and one chunk
// ahead, as the general tile does it, a chunk took as long as its loads.)
//
// LDS holds whole operand fragments: fragment f is the 64 lanes' 16 bytes in
// lane order, which is how one LDS-DMA instruction writes and one
// conflict-free ds_read_b128 reads it.  The packed weights are fragments
// already; of the activations, lane l fetches the 16 bytes of block l / 16 of
// its row l % 16.  Scales: a dword (four blocks) per row, a byte per lane of
// each weight tile; both are read as the byte the lane's operand wants.
//
// One barrier a chunk.  A wave waits until its own part of chunk c has landed
// (its loads complete in order: at most the next chunk's may be in flight),
// then the barrier says that everyone's has and that everyone is done with
// chunk c - 1, whose buffer takes chunk c + 2.  The barrier is the bare
// instruction behind a wait for this wave's LDS reads: __syncthreads, or a
// fence, would wait for every load (an LDS-DMA counts as a write to LDS).
// Nothing is requested past the last chunk, so no DMA outlives the workgroup.
#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"
#include "tile_common.hpp"

namespace w4a16 {

namespace {

constexpr int kMT = 8, kNR = 4, kNW = 4;            // token tiles, weight tiles per wave, waves
constexpr int kTiles = kNR * kNW;                   // weight tiles per workgroup
constexpr int kStages = 3;
constexpr int kThreads = kNW * kWave;

typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct Stage {
  u32x4_t w[kTiles][kWave];                         // weight fragments
  u32x4_t x[kMT][kWave];                            // activation fragments
  uint8_t ws[kTiles][kWave];                        // weight scales, a byte per lane
  uint32_t xs[16 * kMT];                            // activation scales, four blocks per row
};

struct TileSmemMx {
  Stage stage[kStages];
  int row[16 * kMT];
  int out[16 * kMT];
  float w[16 * kMT];
};

typedef __attribute__((address_space(3))) void* lds_ptr_t;

__device__ __forceinline__ void dma16(gptr_t src, lds_ptr_t dst) { __builtin_amdgcn_global_load_lds(src, dst, 16, 0, 0); }
__device__ __forceinline__ void dma4(gptr_t src, lds_ptr_t dst) { __builtin_amdgcn_global_load_lds(src, dst, 4, 0, 0); }

// At most n of this wave's loads still in flight.
template <int n>
__device__ __forceinline__ void wait_loads() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14));
}

// This wave's LDS reads have ended and every wave is here; loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));   // lgkmcnt(0) alone
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// LDS-DMA instructions a wave issues per chunk: 4 weight fragments, 2
// activation fragments, 4 tiles' scales, 64 rows' scales
constexpr int kLoads = kTiles / kNW + kMT / kNW + 2;

template <int NA>
__device__ __forceinline__ void tile_mainloop(const GemmParams& p, TileSmemMx& sm, int expert, int nt,
                                              f32x4_t (&acc)[kNR][kMT]) {
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int KC = p.KC;
  const uint32_t kb = (uint32_t)p.K / 2, ks = (uint32_t)p.K / 32;
  const int spare = sm.row[0];                      // padding reads the block's first row, which is valid
  auto row_of = [&](int i) { return (uint32_t)(sm.row[i] >= 0 ? sm.row[i] : spare); };

  // sources: weight tiles wave, wave + 4, ...; token tiles wave and wave + 4
  gptr_t wsrc[kNR];
#pragma unroll
  for (int i = 0; i < kNR; ++i) {
    const int64_t tile = (int64_t)expert * p.w_tiles + min(nt * kTiles + wave + kNW * i, p.NT - 1);
    wsrc[i] = uniform_ptr(p.packed_w + tile * KC * kWave);
  }
  // scales of tiles 4 wave .. 4 wave + 3, 16 lanes each
  const gptr_t wssrc = uniform_ptr(p.packed_s) +
                       ((int64_t)expert * p.w_tiles + min(nt * kTiles + 4 * wave + (lane >> 4), p.NT - 1)) * KC * kWave +
                       4 * (lane & 15);
  const gptr_t xbase = uniform_ptr(p.a);
  uint32_t xoff[kMT / kNW];
#pragma unroll
  for (int i = 0; i < kMT / kNW; ++i)
    xoff[i] = row_of(16 * (wave + kNW * i) + (lane & 15)) * kb + 16u * (uint32_t)(lane >> 4);
  const gptr_t xsbase = uniform_ptr(p.a_scale);
  // 64 rows' scales a wave, so each half is fetched twice (the same bytes to
  // the same place): masking half the lanes off would end the basic block, and
  // the compiler then sinks every MFMA of the loop behind its last barrier
  const int xsrow = 64 * (wave & 1);
  const uint32_t xsoff = row_of(xsrow + lane) * ks;

  auto issue = [&](int c, int slot) {
    Stage& s = sm.stage[slot];
#pragma unroll
    for (int i = 0; i < kNR; ++i)
      dma16(wsrc[i] + (int64_t)c * (kWave * 16) + lane * 16, (lds_ptr_t)&s.w[wave + kNW * i][0]);
#pragma unroll
    for (int i = 0; i < kMT / kNW; ++i) dma16(xbase + (int64_t)c * 64 + xoff[i], (lds_ptr_t)&s.x[wave + kNW * i][0]);
    dma4(wssrc + (int64_t)c * kWave, (lds_ptr_t)&s.ws[4 * wave][0]);
    dma4(xsbase + (int64_t)c * 4 + xsoff, (lds_ptr_t)&s.xs[xsrow]);
  };
  auto compute = [&](int slot) {
    const Stage& s = sm.stage[slot];
    u32x4_t A[kNR];
    uint32_t as[kNR];
#pragma unroll
    for (int r = 0; r < kNR; ++r) {
      A[r] = s.w[kNR * wave + r][lane];
      as[r] = s.ws[kNR * wave + r][lane];
    }
    const uint8_t* xs = reinterpret_cast<const uint8_t*>(&s.xs[0]) + 4 * (lane & 15) + (lane >> 4);
    u32x4_t B = s.x[0][lane];
    uint32_t bs = xs[0];
#pragma unroll
    for (int t = 0; t < NA; ++t) {
      u32x4_t Bn = B;
      uint32_t bn = bs;
      if (t + 1 < NA) {
        Bn = s.x[t + 1][lane];
        bn = xs[64 * (t + 1)];
      }
      const i32x8_t b = {(int)B[0], (int)B[1], (int)B[2], (int)B[3], 0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < kNR; ++r) {
        const i32x8_t a = {(int)A[r][0], (int)A[r][1], (int)A[r][2], (int)A[r][3], 0, 0, 0, 0};
        acc[r][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[r][t], 4, 4, 0, (int)as[r], 0, (int)bs);
      }
      B = Bn;
      bs = bn;
      __builtin_amdgcn_sched_barrier(0);            // one tile read ahead, no more: the registers are full
    }
  };

  static_assert(kStages == 3, "the waits below keep one later chunk in flight");
  issue(0, 0);
  if (KC > 1) issue(1, 1);
  // chunk c: landed; its buffer's predecessor free; ask for chunk c + 2; multiply
  auto step = [&](int c, int slot, int ahead) {
    wait_loads<kLoads>();
    lds_barrier();
    issue(c + 2, ahead);
    __builtin_amdgcn_sched_barrier(0);
    compute(slot);
  };
  int c = 0;
  for (; c + 4 < KC; c += 3) {
    step(c, 0, 2);
    step(c + 1, 1, 0);
    step(c + 2, 2, 1);
  }
  // at most four chunks are left, c is a multiple of 3; the last two ask for nothing
  for (int slot = 0; c < KC; ++c, slot = slot == 2 ? 0 : slot + 1) {
    if (c + 1 < KC)
      wait_loads<kLoads>();
    else
      wait_loads<0>();
    lds_barrier();
    if (c + 2 < KC) issue(c + 2, slot == 0 ? 2 : slot - 1);
    __builtin_amdgcn_sched_barrier(0);
    compute(slot);
  }
}

template <int ROUTE>
__global__ __launch_bounds__(kThreads, 2) void mx_tile_kernel(const GemmParams p) {
  __shared__ __attribute__((aligned(16))) TileSmemMx sm;
  int mb, nt;
  if (!block_of(p, blockIdx.x, p.n_tiles, mb, nt)) return;
  const int expert = setup_rows<kMT, kNW, ROUTE, kEpiStore>(p, mb, sm);
  if (expert < 0) return;
  __syncthreads();
  const uint32_t tmask = active_tiles<kMT>(sm);
  // token tiles run: the active prefix rounded up to an even count (an extra
  // tile of padding rows reads a valid row and is never stored)
  auto go = [&](auto na) {
    constexpr int NA = decltype(na)::value;
    f32x4_t acc[kNR][kMT];
#pragma unroll
    for (int r = 0; r < kNR; ++r)
#pragma unroll
      for (int t = 0; t < kMT; ++t) acc[r][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    tile_mainloop<NA>(p, sm, expert, nt, acc);
    epilogue<kMT, kNR, kNW, kEpiStore>(p, sm, nt, (1u << NA) - 1u, acc);
  };
  const int na = 32 - __clz(tmask);
  if (na <= 2) go(std::integral_constant<int, 2>{});
  else if (na <= 4) go(std::integral_constant<int, 4>{});
  else if (na <= 6) go(std::integral_constant<int, 6>{});
  else go(std::integral_constant<int, 8>{});
}

}  // namespace

hipError_t launch_mx_tile(int route, const GemmParams& p, hipStream_t stream) {
  GemmParams q = p;
  q.n_tiles = (p.NT + kTiles - 1) / kTiles;
  q.xcd_group = 0;
  const int64_t grid = grid_of(q, q.n_tiles);
  if (grid <= 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidConfiguration;
  if (route == kRouteContiguous)
    hipLaunchKernelGGL(mx_tile_kernel<kRouteContiguous>, dim3((unsigned)grid), dim3(kThreads), 0, stream, q);
  else
    hipLaunchKernelGGL(mx_tile_kernel<kRouteMasked>, dim3((unsigned)grid), dim3(kThreads), 0, stream, q);
  return hipGetLastError();
}

}  // namespace w4a16

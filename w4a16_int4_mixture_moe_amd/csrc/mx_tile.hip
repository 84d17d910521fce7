// A4W4 tile of 128 rows x 256 weight rows for the grouped layouts: MXFP4
// activations x MXFP4 weights in v_mfma_scale_f32_16x16x128_f8f6f4.
//
// Per 128-wide K chunk a workgroup needs 8 KB of activation codes, 16 KB of
// weight codes and 1.5 KB of scales for 4 x 32 MFMAs of 16 cycles.  Everything
// goes HBM -> LDS by LDS-DMA, three chunks deep, and from there to the
// matrix unit, so no register holds data in flight and two workgroups (two
// waves per SIMD) share a CU: 128 accumulator registers a wave, 76.5 KB of
// LDS a workgroup.  Measured on MI355X (N 4096, K 7168, graph replays):
// 16384 rows of 48 experts, 44 of them with rows, 361 us, 2.7 PFLOP/s on
// valid rows; all rows one expert's 274 us, 3.5 PFLOP/s; masked decode, 576
// rows of 48 experts, 132 - 142 us, 5.1 - 5.5 TB/s of weights and rows.  What
// bounds it: with one expert, whose 80 MB stay in the last-level cache, the
// LDS-DMA stream (without the MFMAs 252 us before the order of the fetches
// below, without the DMA 185 us; MFMA busy 47 %), with many experts that
// stream and the requests beyond the L2s (1.78 GB, 4.9 TB/s, the weights' part
// of them from HBM; MFMA busy 33 %), in decode the HBM.  Tried and slower: the
// operands through registers, two chunks ahead (472 against 378 us); 256 rows
// by 256 weight rows on eight waves, one workgroup per CU, three chunks ahead
// (436 against 363 us); every request of a chunk in one go (376 against 375 us).
//
// LDS holds whole operand fragments of 1 KB, one LDS-DMA instruction each.
// The packed weights are fragments in lane order already.  Of the
// activations, lane l fetches 16 of the 64 bytes of row l / 4 of the tile, so
// that neighbouring lanes share a row (with row l % 16, the operand's own
// order, every lane was a request of its own: the rows alone took a third of
// the time); block b of row r lands in place b of the row's four, or 3 - b
// where bit 2 of r is set, so that the lanes a b128 read serves together
// (not sixteen in a row) fall on different banks.  Scales: four blocks' bytes
// per row, a byte per lane of each weight tile; both are read as the byte the
// lane's operand wants.  Bank conflicts (SQ_LDS_BANK_CONFLICT, the prefill
// case above) take 4 % of the CUs' cycles, about two for each read of the row
// scales, which lie 16 bytes apart; with places b ^ (r / 4) they took 12 %.
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
constexpr int kAhead = 2;                           // token tiles whose LDS reads run ahead of their MFMAs

typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct Stage {
  u32x4_t w[kTiles][kWave];                         // weight fragments
  u32x4_t x[kMT][kWave];                            // activation fragments
  uint8_t ws[kTiles][kWave];                        // weight scales, a byte per lane
};

struct TileSmemMx {
  Stage stage[kStages];
  union {                                           // activation scales
    u32x4_t four[2][16 * kMT];                      // a row's 16 bytes of four chunks, two groups of chunks
    uint32_t one[kStages][kNW][kWave];              // a row's 4 bytes of a chunk: 32 rows a wave (and 32 copies)
  } xs;
  union {
    int row[16 * kMT];                              // activation row per block row, -1 = padding
    int out[16 * kMT];                              // output row: the same in both grouped layouts
  };
};
// two workgroups fit the 160 KB of a CU in its units of 1280 bytes
static_assert((sizeof(TileSmemMx) + 1279) / 1280 * 1280 * 2 <= 160 * 1024, "two workgroups per CU");

typedef __attribute__((address_space(3))) void* lds_ptr_t;

__device__ __forceinline__ void dma16(gptr_t src, lds_ptr_t dst) { __builtin_amdgcn_global_load_lds(src, dst, 16, 0, 0); }
__device__ __forceinline__ void dma4(gptr_t src, lds_ptr_t dst) { __builtin_amdgcn_global_load_lds(src, dst, 4, 0, 0); }

// At most n of this wave's loads still in flight.
template <int n>
__device__ __forceinline__ void wait_loads() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14));
}

// Activation fragments in LDS: the row of its tile and the block that lane l
// fetches, and where the operand's lane l (row l % 16, block l / 16) finds its
// 16 bytes.
__device__ __forceinline__ int fetch_row(int lane) { return lane >> 2; }
__device__ __forceinline__ int place_swap(int row) { return row & 4 ? 3 : 0; }
__device__ __forceinline__ uint32_t fetch_block(int lane) { return (uint32_t)((lane & 3) ^ place_swap(lane >> 2)); }
__device__ __forceinline__ int operand_at(int lane) { return 4 * (lane & 15) + ((lane >> 4) ^ place_swap(lane)); }

// This wave's LDS reads have ended and every wave is here; loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));   // lgkmcnt(0) alone
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// FOUR: K is a multiple of 512 and the scales lie on 16 bytes, so a row's
// come 16 bytes (four chunks) at a time: every row is a cache line of its own to the address
// unit, and fetched chunk by chunk they kept it busier (82 % of the time) than
// everything else together.
template <int NA, bool FOUR>
__device__ __forceinline__ void tile_mainloop(const GemmParams& p, TileSmemMx& sm, int expert, int nt,
                                              f32x4_t (&acc)[kNR][kMT]) {
  // LDS-DMA instructions a wave issues per chunk: 4 weight fragments, 1 or 2
  // activation fragments, 4 tiles' scales (and, not FOUR, 32 rows' scales)
  constexpr int XF = (NA + kNW - 1) / kNW;
  constexpr int kLoads = kNR + XF + 1 + (FOUR ? 0 : 1);
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
  uint32_t xoff[XF];
#pragma unroll
  for (int i = 0; i < XF; ++i)
    xoff[i] = row_of(16 * (wave + kNW * i) + fetch_row(lane)) * kb + 16u * fetch_block(lane);
  const gptr_t xsbase = uniform_ptr(p.a_scale);
  // no lane or wave is masked off in the loop: a branch there would end its
  // basic block, and the compiler then sinks the MFMAs behind the last
  // barrier.  So waves 2 and 3 fetch the 64 rows' groups of waves 0 and 1
  // again, and the upper half of a wave copies of its first row's dword.
  const int xs0 = FOUR ? 64 * (wave & 1) : 32 * wave;
  const uint32_t xsoff = row_of(FOUR ? xs0 + lane : xs0 + (lane < 32 ? lane : 0)) * ks;

  const int at = operand_at(lane);
  // instruction i (of kLoads) of chunk c
  auto issue = [&](int i, int c, int slot) {
    Stage& s = sm.stage[slot];
    if (i < kNR)
      dma16(wsrc[i] + (int64_t)c * (kWave * 16) + lane * 16, (lds_ptr_t)&s.w[wave + kNW * i][0]);
    else if (i < kNR + XF)
      dma16(xbase + (int64_t)c * 64 + xoff[i - kNR], (lds_ptr_t)&s.x[wave + kNW * (i - kNR)][0]);
    else if (i == kNR + XF)
      dma4(wssrc + (int64_t)c * kWave, (lds_ptr_t)&s.ws[4 * wave][0]);
    else
      dma4(xsbase + (int64_t)c * 4 + xsoff, (lds_ptr_t)&sm.xs.one[slot][wave][0]);
  };
  auto issue_all = [&](int c, int slot) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) issue(i, c, slot);
  };
  auto issue_four = [&](int group) {
    dma16(xsbase + (int64_t)min(group, KC / 4 - 1) * 16 + xsoff, (lds_ptr_t)&sm.xs.four[group & 1][xs0]);
  };
  // chunk c; the requests of a later one (more: chunk `ask`, buffer `to`) go
  // out one after each tile's MFMAs, since an LDS-DMA takes the address unit
  // some 40 cycles
  auto compute = [&](int c, int slot, auto more, int ask, int to) {
    constexpr bool MORE = decltype(more)::value;
    const Stage& s = sm.stage[slot];
    u32x4_t A[kNR];
    uint32_t as[kNR];
#pragma unroll
    for (int r = 0; r < kNR; ++r) {
      A[r] = s.w[kNR * wave + r][lane];
      as[r] = s.ws[kNR * wave + r][lane];
    }
    // the scale byte of (row 16 t + l % 16, block l / 16)
    const uint8_t* xs = FOUR ? reinterpret_cast<const uint8_t*>(&sm.xs.four[(c >> 2) & 1][lane & 15]) + 4 * (c & 3)
                             : reinterpret_cast<const uint8_t*>(&sm.xs.one[slot][0][lane & 15]);
    xs += lane >> 4;
    auto xs_at = [&](int t) { return FOUR ? 256 * t : 256 * (t / 2) + 64 * (t % 2); };
    // kAhead tiles of reads in flight: a read takes about as long as the MFMAs
    // of two or three tiles
    u32x4_t B[kAhead + 1];
    uint32_t bs[kAhead + 1];
#pragma unroll
    for (int t = 0; t < kAhead && t < NA; ++t) {
      B[t] = s.x[t][at];
      bs[t] = xs[xs_at(t)];
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < NA; ++t) {
      if (t + kAhead < NA) {
        B[(t + kAhead) % (kAhead + 1)] = s.x[t + kAhead][at];
        bs[(t + kAhead) % (kAhead + 1)] = xs[xs_at(t + kAhead)];
      }
      const u32x4_t v = B[t % (kAhead + 1)];
      const i32x8_t b = {(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < kNR; ++r) {
        const i32x8_t a = {(int)A[r][0], (int)A[r][1], (int)A[r][2], (int)A[r][3], 0, 0, 0, 0};
        acc[r][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[r][t], 4, 4, 0, (int)as[r], 0,
                                                                     (int)bs[t % (kAhead + 1)]);
      }
      __builtin_amdgcn_sched_barrier(0);            // no more reads ahead: the registers are full
      if (MORE && t < kLoads) issue(t, ask, to);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = NA; i < kLoads; ++i)
      if (MORE) issue(i, ask, to);
  };

  static_assert(kStages == 3, "the waits below keep one later chunk in flight");
  auto after = [](int slot) { return slot == kStages - 1 ? 0 : slot + 1; };
  if constexpr (FOUR) issue_four(0);
  issue_all(0, 0);
  if (KC > 1) issue_all(1, 1);
  int c = 0, slot = 0;
  // Chunk c has landed and its predecessor's buffer is free: fill that with
  // chunk c + 2, multiply.  newer: this wave's loads issued after chunk c's.
  auto step = [&](auto newer, auto group) {
    wait_loads<decltype(newer)::value>();
    lds_barrier();
    if constexpr (decltype(group)::value) issue_four(c / 4 + 1);
    __builtin_amdgcn_sched_barrier(0);
    compute(c, slot, std::true_type{}, c + 2, after(after(slot)));
    ++c;
    slot = after(slot);
  };
  auto last = [&](auto newer) {
    wait_loads<decltype(newer)::value>();
    lds_barrier();
    compute(c, slot, std::false_type{}, 0, 0);
    ++c;
    slot = after(slot);
  };
  using N0 = std::integral_constant<int, 0>;
  using N1 = std::integral_constant<int, kLoads>;
  using N2 = std::integral_constant<int, kLoads + 1>;   // and the next four chunks' scales, one step old
  using Yes = std::true_type;
  using No = std::false_type;
  if constexpr (FOUR) {                             // KC is a multiple of 4
    while (c + 4 < KC) {
      step(N1{}, Yes{});
      step(N2{}, No{});
      step(N1{}, No{});
      step(N1{}, No{});
    }
    step(N1{}, Yes{});                              // the last group's scales again, so that the count holds
    step(N2{}, No{});
    last(N1{});
    last(N0{});
  } else {
    while (c + 2 < KC) step(N1{}, No{});
    if (c + 1 < KC) last(N1{});
    last(N0{});
  }
}

template <int ROUTE>
__global__ __launch_bounds__(kThreads, 2) void mx_tile_kernel(const GemmParams p) {
  __shared__ __attribute__((aligned(16))) TileSmemMx sm;
  const int mb = blockIdx.x / p.n_tiles, nt = blockIdx.x - mb * p.n_tiles;
  const int expert = setup_rows<kMT, kNW, ROUTE, kEpiStore>(p, mb, sm);
  if (expert < 0) return;
  __syncthreads();
  const uint32_t tmask = active_tiles<kMT>(sm);
  // token tiles run: the active prefix, above one rounded up to an even count (an extra
  // tile of padding rows reads a valid row and is never stored)
  auto go = [&](auto na) {
    constexpr int NA = decltype(na)::value;
    f32x4_t acc[kNR][kMT];
#pragma unroll
    for (int r = 0; r < kNR; ++r)
#pragma unroll
      for (int t = 0; t < kMT; ++t) acc[r][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (p.KC % 4 == 0 && (reinterpret_cast<uintptr_t>(p.a_scale) & 15) == 0)
      tile_mainloop<NA, true>(p, sm, expert, nt, acc);
    else
      tile_mainloop<NA, false>(p, sm, expert, nt, acc);
    epilogue<kMT, kNR, kNW, kEpiStore>(p, sm, nt, (1u << NA) - 1u, acc);
  };
  const int na = 32 - __clz(tmask);
  if (na <= 1) go(std::integral_constant<int, 1>{});
  else if (na <= 2) go(std::integral_constant<int, 2>{});
  else if (na <= 4) go(std::integral_constant<int, 4>{});
  else if (na <= 6) go(std::integral_constant<int, 6>{});
  else go(std::integral_constant<int, 8>{});
}

}  // namespace

hipError_t launch_mx_tile(int route, const GemmParams& p, hipStream_t stream) {
  GemmParams q = p;
  q.n_tiles = (p.NT + kTiles - 1) / kTiles;
  // Block after block: a block's N tiles go to the eight XCDs in turn, so each
  // XCD reads every block's rows and its own share of the N tiles.  (Runs of 2
  // to 8 blocks with all their N tiles on one XCD, which reads the rows once,
  // measured no faster: 16384 rows of 48 experts 358 - 404 us against 360.)
  const int64_t grid = (int64_t)p.grid_blocks * q.n_tiles;
  if (grid <= 0) return hipSuccess;
  if (grid > UINT32_MAX / kThreads) return hipErrorInvalidConfiguration;   // threads past 32 bits wrap, without an error
  if (route == kRouteContiguous)
    hipLaunchKernelGGL(mx_tile_kernel<kRouteContiguous>, dim3((unsigned)grid), dim3(kThreads), 0, stream, q);
  else
    hipLaunchKernelGGL(mx_tile_kernel<kRouteMasked>, dim3((unsigned)grid), dim3(kThreads), 0, stream, q);
  return hipGetLastError();
}

}  // namespace w4a16

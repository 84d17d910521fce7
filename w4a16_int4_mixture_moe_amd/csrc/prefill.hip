// Prefill-side W4A16 MoE GEMM tiles for gfx950: 128 routed rows x 256 weight
// rows per workgroup (four waves, two workgroups per CU), or 256 routed rows x
// 256 weight rows (eight waves, one workgroup per CU; an expert of up to 256
// rows then streams its weights once).  The description below is the
// 128-row tile's; the 256-row one gives each wave two weight tiles of all
// sixteen token tiles instead of four of eight, which leaves registers for a
// software-pipelined step (see pf_mainloop).
//
// Why a separate kernel.  Large routed blocks are MFMA-bound, and on gfx950
// what limits the MFMA rate in this GEMM is the LDS and register traffic per
// MFMA, not the MFMA unit.  Each wave here owns four 16-row weight tiles
// (64 weight rows) and all eight 16-row token tiles of the block, so every
// activation fragment read from LDS feeds four MFMAs, and the dequantised
// weights (VALU work, subtract-then-scale of the Chord post's "H200 and
// Blackwell indexed decode" section) are amortised over 128 rows.  The
// accumulators (4 x 8 MFMA tiles, 128 registers) stay in ordinary VGPRs and
// the whole wave fits 256 registers, so two workgroups (two waves per SIMD)
// share a CU.  (One eight-wave workgroup of 512 weight rows per CU, which
// stages each activation chunk once for twice the weight rows, measured 3-19 %
// slower: its eight waves meet at every chunk barrier together, where two
// independent workgroups cover each other's waits.)  That needs the
// activation staging to cost no registers: the
// block's rows are copied HBM -> LDS with global_load_lds_dwordx4 (16 bytes
// per lane, straight into LDS), one 128-wide K chunk ahead of the MFMAs,
// double buffered.
//
// LDS layout.  A staged chunk is 128 rows x 256 bytes (128 bf16 of K).  The
// LDS-DMA writes each instruction's 64 lanes to 1 KB of consecutive LDS (four
// rows), so rows cannot be padded; instead the sixteen 16-byte granules of
// row r are permuted, granule q at position q ^ swz(r) with
// swz(r) = (r % 4) ^ (12 if bit 2 of r is set).  The MFMA operand read of
// lane l (row 16 t + l % 16, granule 4 (l / 16) + j) is then free of bank
// conflicts.  Measured on MI355X with SQ_LDS_BANK_CONFLICT (a wave's
// ds_read_b128 takes 4 LDS cycles when linear): q ^ swz(r) 4 cycles;
// q ^ (r % 16), q ^ (r % 8), and 272-byte padded rows 8 cycles each.  gfx950
// serves the 64 lanes of a b128 read 16 at a time, and the lanes that share
// a cycle are not a run of 16 consecutive lanes (that model would make
// q ^ (r % 16) conflict-free); swz was chosen to be conflict-free under every
// lane grouping and 64-bank mapping consistent with a set of measured read
// patterns, and measured so.
//
// Arithmetic is that of moe_gemm_kernel: the same packed weights and scales,
// dequant8, v_mfma_f32_16x16x32_bf16 with the weights as the A operand, K
// chunks in order and the four 32-wide MFMA steps of a chunk in order, so the
// outputs are bit-identical to the general kernel's tile configurations
// (only the tile whose waves split K sums in another order).  K must be a
// multiple of 128 (the DMA copies whole chunks; other K use the general
// kernel).
#include <type_traits>

#include "device_common.hpp"
#include "gemm_tile.hpp"
#include "launch.hpp"
#include "prefill_tile.hpp"
#include "tile_common.hpp"

namespace w4a16 {

namespace {

// One workgroup per (routed block, group of n_loop consecutive N tiles);
// n_loop > 1 only when K fits the two LDS buffers.
// (Template arguments are the tile's sizes rather than its PfCfg so that the
// kernel's name in a trace reads like the general kernel's.)
template <int MT, int NR, int NW, int ROUTE, int EPI, bool LOOP>
__global__ __launch_bounds__(NW * kWave, 8 / NW) void moe_gemm_prefill_kernel(const GemmParams p, int n_loop) {
  using C = PfCfg<MT, NR, NW>;
  __shared__ __attribute__((aligned(16))) PfSmem<C::BM> sm;
  // work item (routed block, N-tile group), block-major (consecutive
  // workgroups, the N tiles of one block, go to different XCDs) unless the
  // block has few groups (block_of).  Measured against orders that keep a
  // block's sixteen N tiles on one XCD (its activation rows then come from
  // HBM once): all sixteen side by side there, 4.8x slower (one L2 serving
  // the same lines to sixteen CUs at once); spread over time (N-tile-major),
  // 1-8 % slower.
  const int groups = (p.n_tiles + n_loop - 1) / n_loop;
  int mb, g;
  if (!block_of(p, blockIdx.x, groups, mb, g)) return;
  const int nt0 = g * n_loop;
  const int expert = setup_rows<C::MT, C::NW, ROUTE, EPI>(p, mb, sm);
  if (expert < 0) return;
  __syncthreads();
  pf_run<C, LOOP>(p, sm, expert, nt0, min(nt0 + n_loop, p.n_tiles), active_tiles<C::MT>(sm),
                  [](auto& acc, auto na, int) { ZeroStart{}(acc, na); },
                  [&](const auto& acc, uint32_t tm, int nt) { epilogue<C::MT, C::NR, C::NW, EPI>(p, sm, nt, tm, acc); });
}

typedef void (*PfKernel)(const GemmParams, int);

template <class C, bool LOOP>
PfKernel pick_prefill_of(int route, int epi) {
  if (route == kRouteIndexed) {
    if (epi == kEpiStore) return moe_gemm_prefill_kernel<C::MT, C::NR, C::NW, kRouteIndexed, kEpiStore, LOOP>;
    if (epi == kEpiWeighted) return moe_gemm_prefill_kernel<C::MT, C::NR, C::NW, kRouteIndexed, kEpiWeighted, LOOP>;
    if (epi == kEpiSilu) return moe_gemm_prefill_kernel<C::MT, C::NR, C::NW, kRouteIndexed, kEpiSilu, LOOP>;
    return nullptr;
  }
  if (epi != kEpiStore) return nullptr;
  if (route == kRouteContiguous) return moe_gemm_prefill_kernel<C::MT, C::NR, C::NW, kRouteContiguous, kEpiStore, LOOP>;
  if (route == kRouteMasked) return moe_gemm_prefill_kernel<C::MT, C::NR, C::NW, kRouteMasked, kEpiStore, LOOP>;
  return nullptr;
}

// The prefill tile of a configuration (m_tiles, nr, waves), or nullptr; the
// N-tile loop exists for the narrow tile only.
PfKernel pick_prefill(int m_tiles, int nr, int waves, int route, int epi, bool loop) {
  if (m_tiles == PfNarrow::MT && nr == PfNarrow::NR && waves == PfNarrow::NW)
    return loop ? pick_prefill_of<PfNarrow, true>(route, epi) : pick_prefill_of<PfNarrow, false>(route, epi);
  if (m_tiles == PfWide::MT && nr == PfWide::NR && waves == PfWide::NW && !loop)
    return pick_prefill_of<PfWide, false>(route, epi);
  return nullptr;
}

}  // namespace

bool prefill_applies(int route, int epilogue, int m_tiles, int nr, int waves, int stages, const GemmParams& p) {
  return stages == 2 && p.K % kChunk == 0 && p.split <= 1 &&
         pick_prefill(m_tiles, nr, waves, route, epilogue, false) != nullptr;
}

// N tiles per workgroup.  With K of at most two chunks (K <= 256, the down
// projection of a TP8 share) a block's 128 activation rows (64 KB at K = 256)
// outweigh an N tile's weights (36 KB with scales), and every N tile's
// workgroup fetches them again; a workgroup that keeps them in LDS and runs
// several N tiles fetches them once.  As many tiles per workgroup as keep the
// grid at kPfLoopMinWorkgroups or more (the routed-block bound counts every
// block).  Measured on MI355X, TP8 T = 4096 down + combine in four passes of
// seven N tiles: one tile per workgroup 541 us; 2, 3, 7 tiles 513, 501,
// 515 us; 4 tiles (two workgroups per block) 684 us.
constexpr int64_t kPfLoopMinWorkgroups = 1536;

int prefill_n_loop(const GemmParams& p, int m_tiles) {
  if (p.KC > 2 || m_tiles != PfNarrow::MT) return 1;
  int best = 1;
  for (int l = 2; l <= p.n_tiles; ++l)
    if ((int64_t)p.grid_blocks * ((p.n_tiles + l - 1) / l) >= kPfLoopMinWorkgroups) best = l;
  return best;
}

hipError_t launch_gemm_prefill(int route, int epilogue, int m_tiles, int nr, int waves, const GemmParams& p,
                               hipStream_t stream) {
  const int n_loop = prefill_n_loop(p, m_tiles);
  const PfKernel k = pick_prefill(m_tiles, nr, waves, route, epilogue, n_loop > 1);
  if (k == nullptr || p.K % kChunk) return hipErrorInvalidValue;
  const int groups = (p.n_tiles + n_loop - 1) / n_loop;
  GemmParams q = p;
  q.xcd_group = xcd_group_for(1, groups);
  const int64_t grid = grid_of(q, groups);
  if (grid <= 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(k, dim3((unsigned)grid), dim3(waves * kWave), 0, stream, q, n_loop);
  return hipGetLastError();
}

}  // namespace w4a16

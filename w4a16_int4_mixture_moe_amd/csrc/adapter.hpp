// Low-rank adapters of many requests beside an INT4 product:
//
//   y_i = W x_i + s_a B_a (A_a x_i),  a = ids[token of row i],  none where a is outside [0, L)
//
// A kernel of its own leaves h_i = s_a A_a x_i in fp32 (adapter_shrink.hip);
// the product's accumulators start from B_a h_i, so the sum is rounded once,
// by the epilogue, and y is neither written nor read twice.
//
// The start is one v_mfma_f32_16x16x32_bf16 for 16 ranks: h is fp32, and its
// two leading bf16 parts (h = hi + lo up to 2^-17 of it; one bf16 part alone
// would cost the adapter's term as much as the output's own rounding) take the
// instruction's two K halves, both against the same 16 ranks of B:
//   K 0 .. 15   hi of ranks 16 c .. 16 c + 15
//   K 16 .. 31  lo of the same
// Lane l = 16 g + i supplies row i of B's 16-row tile, or row i of h's 16-row
// tile, at ranks 16 c + 8 (g % 2) .. + 7, hi for g < 2 and lo for the others.
//
// A 16-row tile may mix adapters.  Each of them multiplies the whole tile, the
// other rows' h replaced by zero; a row then takes the product of its own
// adapter by selection, not by the sum alone, as an infinity or a NaN in one
// request's B times that zero would reach the other requests.
#pragma once
#include "adapter_launch.hpp"
#include "device_common.hpp"
#include "launch.hpp"
#include "tile_common.hpp"

namespace w4a16 {

constexpr int kNoAdapter = -1;    // a row without one
constexpr int kNoRow = -2;        // padding

// a kernel's shared memory, with each block row's adapter and row of h
template <class Base, int BM>
struct AdapterSmem : Base {
  int ad[BM];
  int slot[BM];
};

__device__ __forceinline__ int adapter_of(const AdapterParams& q, int token) {
  if (q.ids == nullptr) return kNoAdapter;
  const int a = q.ids[token];
  return (unsigned)a < (unsigned)q.L ? a : kNoAdapter;
}

// setup_rows, and the rows' adapters.  kRouteDense: row p.order[position] (or
// the position itself) of one weight.
template <int MT, int NW, int ROUTE, int EPI, typename Smem>
__device__ __forceinline__ int setup_adapter_rows(const GemmParams& p, const AdapterParams& q, int mb, Smem& sm) {
  constexpr int BM = 16 * MT;
  if constexpr (ROUTE == kRouteIndexed) {
    const int expert = setup_rows<MT, NW, ROUTE, EPI>(p, mb, sm);
    if (expert < 0) return expert;
    for (int i = threadIdx.x; i < BM; i += NW * kWave) {
      const int s = p.sorted_ids[mb * BM + i];
      const bool v = (unsigned)s < (unsigned)p.sentinel;
      sm.slot[i] = v ? s : -1;
      sm.ad[i] = v ? adapter_of(q, s / q.topk) : kNoRow;
    }
    return expert;
  } else {
    for (int i = threadIdx.x; i < BM; i += NW * kWave) {
      const int pos = mb * BM + i;
      const bool v = pos < q.rows;
      const int row = v ? (q.order ? q.order[pos] : pos) : -1;
      sm.row[i] = row;
      sm.out[i] = row;
      sm.slot[i] = row;
      sm.ad[i] = v ? adapter_of(q, row) : kNoRow;
    }
    return 0;
  }
}

// this lane's part of a row of h at rank k0 of one slice of A's rows: the sum
// over the slices of K, then its hi or lo bf16 part
__device__ __forceinline__ bf16x8_t h_operand(const AdapterParams& q, int slot, int slice, int k0, bool lo) {
  const int width = q.slices * q.rank;
  const float* src = q.h + (int64_t)slot * width + slice * q.rank + k0;
  f32x4_t v[2] = {*reinterpret_cast<const f32x4_t*>(src), *reinterpret_cast<const f32x4_t*>(src + 4)};
  for (int k = 1; k < q.ks; ++k) {
    src += q.rows * width;
    v[0] += *reinterpret_cast<const f32x4_t*>(src);
    v[1] += *reinterpret_cast<const f32x4_t*>(src + 4);
  }
  bf16x8_t r;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = v[e / 4][e % 4];
    const __bf16 hi = (__bf16)x;
    const float rest = x - (float)hi;                   // NaN where hi is infinite: hi stands alone there
    r[e] = lo ? (__bf16)(rest == rest ? rest : 0.f) : hi;
  }
  return r;
}

__device__ __forceinline__ bf16x8_t zero_operand() { return __builtin_bit_cast(bf16x8_t, u32x4_t{0u, 0u, 0u, 0u}); }

// B_a h of weight tiles rt_base + r < NR and row tiles t < NA, 16 ranks at a
// time: add(t, r, own, y) with y to be added to the lanes whose row is this
// adapter's (own).  Waves that share the tiles deal the (row tile, adapter)
// pairs among them: `step` waves, this one taking every step-th from `first`.
template <int NR, int NA, typename Smem, typename Add>
__device__ __forceinline__ void adapter_products(const GemmParams& p, const AdapterParams& q, const Smem& sm, int expert,
                                                 int rt_base, int first, int step, Add&& add) {
  constexpr int U = 4;                                  // adapters whose B is in flight together
  if (q.L == 0) return;
  const int lane = threadIdx.x & (kWave - 1);
  const int i = lane & 15, g = lane >> 4;
  const bool lo = g >= 2;
  const int chunks = (q.rank + 15) / 16;
  // row i of each weight tile in B, and the slice of h it multiplies
  int64_t brow[NR];
  int slice[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int n = q.n0 + logical_tile(p, min(rt_base + r, p.NT - 1)) * kRowTile;
    slice[r] = q.slices == 2 && n >= q.N / 2 ? 1 : 0;
    brow[r] = (int64_t)(n + i) * q.rank;
  }
  const int64_t per_adapter = (int64_t)q.E * q.N * q.rank, of_expert = (int64_t)expert * q.N * q.rank;
  int turn = 0;
#pragma unroll
  for (int t = 0; t < NA; ++t) {
    const int mine = sm.ad[16 * t + i];
    const uint32_t any = (uint32_t)__ballot(mine >= 0) & 0xFFFFu;
    if (!any) continue;
    const int slot = sm.slot[16 * t + i];
    const int h_row = mine >= 0 ? slot : sm.slot[16 * t + __builtin_ctz(any)];
    uint32_t rest = any;
    while (rest) {
      int a[U];
      int n = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // the next adapter that is this wave's; none left: -1
        a[u] = kNoAdapter;
        while (rest && a[u] < 0) {
          const int next = __builtin_amdgcn_readlane(mine, __builtin_ctz(rest));
          rest &= ~(uint32_t)__ballot(mine == next);
          if (turn == first) {
            a[u] = next;
            ++n;
          }
          turn = turn + 1 == step ? 0 : turn + 1;
        }
      }
      if (n == 0) break;
      for (int c = 0; c < chunks; ++c) {
        const int k0 = 16 * c + 8 * (g & 1);
        const bool in = k0 < q.rank;
        const int k = in ? k0 : 0;
        bf16x8_t b[U][NR];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u < n) {
            const uint16_t* base = q.b + (int64_t)a[u] * per_adapter + of_expert + k;
#pragma unroll
            for (int r = 0; r < NR; ++r) b[u][r] = *reinterpret_cast<const bf16x8_t*>(base + brow[r]);
          }
        bf16x8_t h[2];
        h[0] = h_operand(q, h_row, 0, k, lo);
        if (q.slices == 2) h[1] = h_operand(q, h_row, 1, k, lo);
        else h[1] = h[0];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u < n) {
            const bool own = mine == a[u];
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              const bf16x8_t bv = in ? b[u][r] : zero_operand();
              const bf16x8_t hv = own && in ? (slice[r] ? h[1] : h[0]) : zero_operand();
              add(t, r, own, __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv, hv, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0));
            }
          }
      }
    }
  }
}

// acc = the adapters' products (zero past row tile NA, and for rows without an adapter)
template <int MT, int NR, int NA, typename Smem>
__device__ __forceinline__ void start_from_adapters(const GemmParams& p, const AdapterParams& q, const Smem& sm,
                                                    int expert, int rt_base, f32x4_t (&acc)[NR][MT]) {
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[r][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  adapter_products<NR, NA>(p, q, sm, expert, rt_base, 0, 1, [&](int t, int r, bool own, const f32x4_t& y) {
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[r][t][v] += own ? y[v] : 0.f;
  });
}

// The epilogue of weight tiles rt_base .. rt_base + NR - 1: as `epilogue`, but
// SiLU(gate) * up of the fp32 sums (one rounding, at the store).
template <int MT, int NR, int EPI, typename Out>
__device__ __forceinline__ void store_tiles(const GemmParams& p, const Out& out_row, int rt_base, uint32_t tmask,
                                            const f32x4_t (&acc)[NR][MT]) {
  static_assert(EPI == kEpiStore || (EPI == kEpiSilu && NR % 2 == 0), "gate and up tiles in pairs");
  const int lane = threadIdx.x & (kWave - 1);
  const int nr_valid = min(NR, p.NT - rt_base);
  constexpr int STEP = EPI == kEpiSilu ? 2 : 1;
  const int64_t ld = p.N / STEP;
#pragma unroll
  for (int r = 0; r < NR; r += STEP) {
    if (r >= nr_valid) continue;
    const int tile = EPI == kEpiSilu ? (rt_base + r) >> 1 : logical_tile(p, rt_base + r);
    const int n = tile * kRowTile + 4 * (lane >> 4);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      if (!((tmask >> t) & 1u)) continue;
      const int orow = out_row[16 * t + (lane & 15)];
      if (orow < 0) continue;
      f32x4_t y = acc[r][t];
      if constexpr (EPI == kEpiSilu)
#pragma unroll
        for (int v = 0; v < 4; ++v) y[v] = silu_mul(y[v], acc[r + 1][t][v]);
      uint2 o;
      o.x = pack_bf16x2(y[0], y[1]);
      o.y = pack_bf16x2(y[2], y[3]);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + orow * ld + n) = o;
    }
  }
}

template <int MT, int NR, int NW, int EPI, typename Smem>
__device__ __forceinline__ void adapter_epilogue(const GemmParams& p, const Smem& sm, int nt, uint32_t tmask,
                                                 const f32x4_t (&acc)[NR][MT]) {
  if constexpr (EPI == kEpiWeighted) {
    epilogue<MT, NR, NW, EPI>(p, sm, nt, tmask, acc);
  } else {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    store_tiles<MT, NR, EPI>(p, sm.out, nt * (NW * NR) + wave * NR, tmask, acc);
  }
}

// Few rows: NT weight tiles of 16 MT rows a workgroup, its NW waves splitting
// K and dealing the adapters; chunks go straight into registers, and the
// partial sums meet in LDS, in wave order.  The adapters' products have a place
// of their own there, since which wave takes one depends on the other rows of
// the tile, and a row's sum must not.
template <int MT, int NT, int NW>
struct SplitSmem {
  int row[16 * MT];
  int out[16 * MT];
  float w[16 * MT];
  f32x4_t red[NW][MT][NT][kWave];
  f32x4_t low[MT][NT][kWave];           // the adapters' products
};

// acc[r][0] = token tile `wave` of weight tile NT nt + r, in waves below MT
template <int MT, int NT, int NW, typename Smem>
__device__ __forceinline__ void split_product(const GemmParams& p, const AdapterParams& q, Smem& sm, int expert, int nt,
                                              f32x4_t (&tot)[NT][1]) {
  static_assert(MT <= NW, "a wave for every token tile");
  constexpr int KB = MT == 4 ? 2 : MT == 2 ? 4 : 8 / NT;   // chunks in flight per wave
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int g = lane >> 4;
  const int KC = p.KC;
  const int c0 = (int)((int64_t)wave * KC / NW), c1 = (int)((int64_t)(wave + 1) * KC / NW);
  gptr_t wbase[NT], sbase[NT], xrow[MT];
#pragma unroll
  for (int r = 0; r < NT; ++r) {
    const int64_t tile = (int64_t)expert * p.w_tiles + min(NT * nt + r, p.NT - 1);
    wbase[r] = uniform_ptr(p.packed_w + tile * KC * kWave) + lane * 16;
    sbase[r] = uniform_ptr(p.packed_s + tile * ((KC + 1) / 2) * kWave) + lane * 4;
  }
  // rows past the block's read its first row, for columns that nothing stores
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int r = sm.row[16 * t + (lane & 15)];
    xrow[t] = uniform_ptr(p.a) + (int64_t)(r >= 0 ? r : sm.row[0]) * p.K * 2;
  }
  const DequantMasks masks = make_dequant_masks();
  u32x4_t w[KB][NT];
  uint32_t sw[KB][NT];
  bf16x8_t x[KB][MT][4];
  auto issue = [&](int cb) {
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int c = max(min(cb + i, c1 - 1), 0);        // past the wave's chunks: loaded again, not used
      const int k = c * kChunk + g * kGroup;
#pragma unroll
      for (int r = 0; r < NT; ++r) {
        w[i][r] = gload_u32x4(wbase[r] + (int64_t)c * (kWave * 16));
        sw[i][r] = gload_u32(sbase[r] + (int64_t)(c >> 1) * (kWave * 4));
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[i][t][j] = __builtin_bit_cast(bf16x8_t, gload_u32x4(xrow[t] + (k < p.K ? k * 2 : 0) + 16 * j));
    }
  };
  f32x4_t acc[NT][MT];
#pragma unroll
  for (int r = 0; r < NT; ++r)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[r][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  issue(c0);
  __builtin_amdgcn_sched_barrier(0);                    // the first chunks are under way while the adapters' parts are found
  adapter_products<NT, MT>(p, q, sm, expert, NT * nt, wave, NW, [&](int t, int r, bool own, const f32x4_t& y) {
    if (own) sm.low[t][r][lane] += y;                   // a row's adapter is one wave's
  });
  for (int cb = c0; cb < c1; cb += KB) {
    if (cb > c0) issue(cb);
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int c = cb + i;
      if (c >= c1) break;
      const bool in = c * kChunk + g * kGroup < p.K;    // a ragged last chunk: zeros past K
#pragma unroll
      for (int r = 0; r < NT; ++r) {
        const float s = __builtin_bit_cast(float, (c & 1) ? (sw[i][r] & 0xFFFF0000u) : (sw[i][r] << 16));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8_t A = dequant8(w[i][r][j], s, -1032.0f * s, 0.0625f * s, -72.0f * s, masks);
#pragma unroll
          for (int t = 0; t < MT; ++t)
            acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, in ? x[i][t][j] : zero_operand(), acc[r][t], 0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int r = 0; r < NT; ++r) sm.red[wave][t][r][lane] = acc[r][t];
  __syncthreads();
  if (wave >= MT) return;
#pragma unroll
  for (int r = 0; r < NT; ++r) {
    tot[r][0] = sm.red[0][wave][r][lane];
#pragma unroll
    for (int v = 1; v < NW; ++v) tot[r][0] += sm.red[v][wave][r][lane];
    tot[r][0] += sm.low[wave][r][lane];
  }
}

// before the barrier that follows the rows' setup
template <int MT, int NT, int NW>
__device__ __forceinline__ void clear_low(SplitSmem<MT, NT, NW>& sm) {
  f32x4_t* low = &sm.low[0][0][0];
  for (int i = threadIdx.x; i < MT * NT * kWave; i += NW * kWave) low[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
}

}  // namespace w4a16

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
#include <type_traits>

#include "adapter_launch.hpp"
#include "device_common.hpp"
#include "gemm_tile.hpp"
#include "launch.hpp"
#include "prefill_tile.hpp"
#include "ring.hpp"
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

// A row's h in LDS, 64 ranks at a time: 16 granules of 8 bf16, granule 4 j + g
// what lane group g supplies to instruction j (16 ranks: two granules of hi,
// two of lo).
constexpr int kHRanks = 64;

__device__ __forceinline__ bf16x8_t zero_operand() { return __builtin_bit_cast(bf16x8_t, u32x4_t{0u, 0u, 0u, 0u}); }

// Ranks r0 .. of every row of the block that has an adapter: the sum over the
// slices of K, split in two bf16 parts; zeros past the rank.  place(slice,
// row, granule) is the granule's address.  The caller synchronises.
// IP groups of 8 ranks a thread and KP slices of each in flight together.
template <int BM, int NTHR, int IP, int KP, typename Smem, typename Place>
__device__ __forceinline__ void stage_h(const AdapterParams& q, const Smem& sm, int r0, Place&& place) {
  const int width = q.slices * q.rank;
  const int64_t plane = q.rows * width;
  const int left = min(q.rank - r0, kHRanks);
  const int eights = (left + 15) / 16 * 2;                // groups of 8 ranks, whole instructions
  const int items = BM * q.slices * eights;
  for (int it0 = threadIdx.x; it0 < items; it0 += IP * NTHR) {
    int row[IP], slice[IP], e[IP];
    const float* src[IP];
    f32x4_t v[IP][2];
#pragma unroll
    for (int n = 0; n < IP; ++n) {
      const int it = min(it0 + n * NTHR, items - 1);      // past the last: the last again
      const int rest = it / eights;
      e[n] = it - rest * eights;
      slice[n] = rest / BM;
      row[n] = rest - slice[n] * BM;
      // rows without an adapter: any address of h, for values that are never used
      const bool in = sm.ad[row[n]] >= 0 && 8 * e[n] < left;
      src[n] = q.h + (in ? (int64_t)sm.slot[row[n]] * width + slice[n] * q.rank + r0 + 8 * e[n] : 0);
      v[n][0] = v[n][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    for (int k0 = 0; k0 < q.ks; k0 += KP) {               // past the last slice: the last again, not added
      f32x4_t w[KP][IP][2];
#pragma unroll
      for (int k = 0; k < KP; ++k)
#pragma unroll
        for (int n = 0; n < IP; ++n) {
          const float* from = src[n] + min(k0 + k, q.ks - 1) * plane;
          w[k][n][0] = *reinterpret_cast<const f32x4_t*>(from);
          w[k][n][1] = *reinterpret_cast<const f32x4_t*>(from + 4);
        }
#pragma unroll
      for (int k = 0; k < KP; ++k)
        if (k0 + k < q.ks)
#pragma unroll
          for (int n = 0; n < IP; ++n) {
            v[n][0] += w[k][n][0];
            v[n][1] += w[k][n][1];
          }
    }
#pragma unroll
    for (int n = 0; n < IP; ++n) {
      if (sm.ad[row[n]] < 0) continue;
      if (8 * e[n] >= left) v[n][0] = v[n][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      bf16x8_t hi, lo;
      split_bf16(v[n], hi, lo);
      *place(slice[n], row[n], e[n] / 2 * 4 + (e[n] & 1)) = hi;
      *place(slice[n], row[n], e[n] / 2 * 4 + (e[n] & 1) + 2) = lo;
    }
  }
}

// The same from a packed h, IP granules a thread in flight.
template <int BM, int NTHR, int IP, typename Smem, typename Place>
__device__ __forceinline__ void stage_packed_h(const AdapterParams& q, const Smem& sm, int r0, Place&& place) {
  const int all = (q.rank + 15) / 16 * 4, from = r0 / 16 * 4;   // a row's granules, and the first of these ranks
  const int count = min(all - from, kHRanks / 4);
  const int items = BM * q.slices * count;
  for (int it0 = threadIdx.x; it0 < items; it0 += IP * NTHR) {
    u32x4_t v[IP];
    int row[IP], slice[IP], at[IP];
#pragma unroll
    for (int n = 0; n < IP; ++n) {
      const int it = min(it0 + n * NTHR, items - 1);      // past the last: the last again
      const int rest = it / count;
      at[n] = it - rest * count;
      slice[n] = rest / BM;
      row[n] = rest - slice[n] * BM;
      const int64_t src = sm.ad[row[n]] >= 0 ? ((int64_t)sm.slot[row[n]] * q.slices + slice[n]) * all + from + at[n] : 0;
      v[n] = *reinterpret_cast<const u32x4_t*>(q.packed + src * 8);
    }
#pragma unroll
    for (int n = 0; n < IP; ++n)
      if (sm.ad[row[n]] >= 0) *place(slice[n], row[n], at[n]) = __builtin_bit_cast(bf16x8_t, v[n]);
  }
}

// What a wave multiplies its h by: row i of each of its weight tiles in B, and
// the slice of h that the tile takes.
template <int NR>
struct AdapterTiles {
  int64_t row[NR];
  int slice[NR];
  __device__ __forceinline__ AdapterTiles(const GemmParams& p, const AdapterParams& q, int rt_base) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int n = q.n0 + logical_tile(p, min(rt_base + r, p.NT - 1)) * kRowTile;
      slice[r] = q.slices == 2 && n >= q.N / 2 ? 1 : 0;
      row[r] = (int64_t)(n + (threadIdx.x & 15)) * q.rank;
    }
  }
};

// this lane's operand of B at instruction j of ranks r0 ..; zeros past the rank
__device__ __forceinline__ bf16x8_t b_operand(const AdapterParams& q, const uint16_t* base, int64_t row, int k) {
  const bf16x8_t v = *reinterpret_cast<const bf16x8_t*>(base + row + (k < q.rank ? k : 0));
  return k < q.rank ? v : zero_operand();
}

// acc = B_a h of the wave's weight tiles and row tiles t < NA (zero past it,
// and for rows without an adapter).  h goes through LDS, then the adapters of
// the block are taken in rising order: an adapter's B once for all row tiles
// that hold it.  at(slice, row, granule): see stage_h; that memory is free
// before the call and after it (both synchronise).  PACKS: h may be packed.
template <int MT, int NR, int NW, int NA, bool PACKS, typename Smem, typename Place>
__device__ __forceinline__ void start_from_adapters(const GemmParams& p, const AdapterParams& q, const Smem& sm,
                                                    int expert, int rt_base, f32x4_t (&acc)[NR][MT], Place&& at) {
  constexpr int U = MT >= 8 ? 2 : 4;
  // decode tiles stream weights with as many waves as their registers allow, and a block of theirs holds few adapters:
  // nothing ahead
  constexpr int SETS = MT >= 4 ? 2 : 1;
  auto clear = [&]() {
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[r][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  };
  if (q.L == 0) return clear();
  const int lane = threadIdx.x & (kWave - 1);
  const int i = lane & 15, g = lane >> 4;
  const AdapterTiles<NR> tiles(p, q, rt_base);
  const int64_t per_adapter = (int64_t)q.E * q.N * q.rank, of_expert = (int64_t)expert * q.N * q.rank;
  int mine[NA];
#pragma unroll
  for (int t = 0; t < NA; ++t) mine[t] = sm.ad[16 * t + i];
  // the least adapter above a
  auto next_after = [&](int a) {
    int best = INT32_MAX;
#pragma unroll
    for (int t = 0; t < NA; ++t) best = mine[t] > a ? min(best, mine[t]) : best;
#pragma unroll
    for (int m = 1; m < 16; m *= 2) best = min(best, __shfl_xor(best, m));
    return __builtin_amdgcn_readfirstlane(best);
  };
  const int first = next_after(-1);
  if (first == INT32_MAX) return clear();               // the whole block, so every wave
  // the first ranks before the accumulators take their registers
  const bool packed = PACKS && q.packed != nullptr;
  if (packed) stage_packed_h<16 * MT, NW * kWave, 16>(q, sm, 0, at);
  else stage_h<16 * MT, NW * kWave, MT >= 4 ? 2 : 1, 4>(q, sm, 0, at);
  clear();
  for (int r0 = 0; r0 < q.rank; r0 += kHRanks) {
    if (r0 > 0) {
      __syncthreads();
      if (packed) stage_packed_h<16 * MT, NW * kWave, 4>(q, sm, r0, at);
      else stage_h<16 * MT, NW * kWave, 1, 2>(q, sm, r0, at);
    }
    __syncthreads();
    const int steps = (min(q.rank - r0, kHRanks) + 15) / 16;
    // (adapter, instruction) after (adapter, instruction): U of them, with two sets the next U on their way
    int a = first, j = 0;
    int ua[SETS][U], uj[SETS][U];
    bf16x8_t b[SETS][U][NR];
    auto request = [&](auto set_) {
      constexpr int set = decltype(set_)::value;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        ua[set][u] = a;
        uj[set][u] = j;
        if (a == INT32_MAX) continue;
        const uint16_t* base = q.b + (int64_t)a * per_adapter + of_expert;
#pragma unroll
        for (int r = 0; r < NR; ++r) b[set][u][r] = b_operand(q, base, tiles.row[r], r0 + 16 * j + 8 * (g & 1));
        if (++j == steps) {
          j = 0;
          a = next_after(a);
        }
      }
    };
    auto use = [&](auto set_) {
      constexpr int set = decltype(set_)::value;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (ua[set][u] == INT32_MAX) continue;
#pragma unroll
        for (int t = 0; t < NA; ++t) {
          const bool own = mine[t] == ua[set][u];
          if (!__ballot(own)) continue;
          const bf16x8_t h0 = *at(0, 16 * t + i, 4 * uj[set][u] + g);
          const bf16x8_t h1 = q.slices == 2 ? *at(1, 16 * t + i, 4 * uj[set][u] + g) : h0;
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const f32x4_t y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[set][u][r], tiles.slice[r] ? h1 : h0,
                                                                      f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[r][t][v] += own ? y[v] : 0.f;
          }
        }
      }
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, SETS - 1>;
    if constexpr (SETS == 1) {
      while (a != INT32_MAX) {
        request(I0{});
        use(I0{});
      }
      continue;
    }
    request(I0{});
    while (true) {
      const bool more = a != INT32_MAX;
      if (more) request(I1{});
      use(I0{});
      if (!more) break;
      const bool again = a != INT32_MAX;
      if (again) request(I0{});
      use(I1{});
      if (!again) break;
    }
  }
  __syncthreads();
}

// addresses in the general tile's two activation buffers (rows padded by 16
// bytes) and in the prefill tiles' (granules permuted by row): a slice each
template <int MT>
__device__ __forceinline__ bf16x8_t* h_place(TileSmem<MT>& sm, int slice, int row, int granule) {
  return reinterpret_cast<bf16x8_t*>(&sm.xs[slice][row][8 * granule]);
}
template <int BM>
__device__ __forceinline__ bf16x8_t* h_place(PfSmem<BM>& sm, int slice, int row, int granule) {
  const int at = granule ^ (row & 3) ^ (row & 4 ? 12 : 0);
  return reinterpret_cast<bf16x8_t*>(&sm.xs[slice][row * kChunk + 8 * at]);
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

// Few rows: NW / MT waves for each of a block's MT row tiles, which deal the
// tile's adapters among them.  The products have a place of their own in LDS,
// since which wave takes one depends on the other rows of the tile, and a row's
// sum must not.
template <int MT, int NT>
struct LowSmem {
  f32x4_t low[MT][NT][kWave];                // the adapters' products
  uint16_t h[2][16 * MT][2 * kHRanks + 8];   // 272-byte rows
};

// before the barrier that follows the rows' setup
template <int MT, int NT, int NW>
__device__ __forceinline__ void clear_low(LowSmem<MT, NT>& sm) {
  f32x4_t* low = &sm.low[0][0][0];
  for (int i = threadIdx.x; i < MT * NT * kWave; i += NW * kWave) low[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
}

// A barrier for LDS alone: loads in flight stay in flight.
__device__ __forceinline__ void lds_only_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Lane l = 16 g + i of a chunk's packed words holds row i's K 32 g .. 32 g + 31,
// word j the 8 from 32 g + 8 j.  An activation row is loaded 64 bytes at a time
// by four lanes side by side, so instruction j of its operand is K 32 j + 8 g
// there (64 bytes in one lane would touch 64 cache lines a load, for 16 bytes
// of each).  So the words change places instead, 4 x 4 over lane groups and
// words: word j of group g <-> word g of group j.
__device__ __forceinline__ void transpose_words(u32x4_t& w) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  w = u32x4_t{c[0], c[1], d[0], d[1]};
}

// ... and every lane needs the scales of all four groups
__device__ __forceinline__ u32x4_t spread_scales(uint32_t s) {
  const auto a = __builtin_amdgcn_permlane32_swap(s, s, false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[1], a[1], false, false);
  return u32x4_t{b[0], b[1], c[0], c[1]};
}

// The adapters' products of row tile wave % MT into sm.low, U instructions' B in
// flight together, the first ones while h is on its way.  (Synchronises by LDS
// alone: loads under way stay under way.)
template <int MT, int NT, int NW, typename Smem>
__device__ __forceinline__ void deal_adapters(const GemmParams& p, const AdapterParams& q, Smem& sm, int expert, int rt_base) {
  constexpr int U = 8 / NT;
  constexpr int P = NW / MT;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int i = lane & 15, g = lane >> 4;
  const int t = wave % MT;
  const AdapterTiles<NT> tiles(p, q, rt_base);
  const int64_t per_adapter = (int64_t)q.E * q.N * q.rank, of_expert = (int64_t)expert * q.N * q.rank;
  const int mine = sm.ad[16 * t + i];
  const uint32_t rows = (uint32_t)__ballot(mine >= 0) & 0xFFFFu;
  f32x4_t low[NT];
#pragma unroll
  for (int r = 0; r < NT; ++r) low[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  bool took = false;                                    // this wave has the lane's row
  for (int r0 = 0; r0 < q.rank; r0 += kHRanks) {
    const int steps = (min(q.rank - r0, kHRanks) + 15) / 16;
    // (adapter, instruction) after (adapter, instruction) of every P-th adapter
    uint32_t rest = rows;
    int turn = 0, a = kNoAdapter, j = steps;
    int ua[U], uj[U], n;
    bf16x8_t b[U][NT];
    auto request = [&]() {
      n = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (j == steps) {
          a = kNoAdapter;
          while (rest && a < 0) {
            const int next = __builtin_amdgcn_readlane(mine, __builtin_ctz(rest));
            rest &= ~(uint32_t)__ballot(mine == next);
            if (turn == wave / MT) a = next;
            turn = turn + 1 == P ? 0 : turn + 1;
          }
          j = 0;
        }
        ua[u] = a;
        uj[u] = j;
        if (a < 0) {
          j = steps;
          continue;
        }
        const uint16_t* base = q.b + (int64_t)a * per_adapter + of_expert;
#pragma unroll
        for (int r = 0; r < NT; ++r) b[u][r] = b_operand(q, base, tiles.row[r], r0 + 16 * j + 8 * (g & 1));
        ++j;
        n = u + 1;
      }
    };
    request();
    if (r0 > 0) lds_only_barrier();
    stage_h<16 * MT, NW * kWave, 2, 4>(q, sm, r0, [&](int slice, int row, int granule) {
      return reinterpret_cast<bf16x8_t*>(&sm.h[slice][row][8 * granule]);
    });
    lds_only_barrier();
    while (n > 0) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < n) {
          const bool own = mine == ua[u];
          took = took || own;
          const bf16x8_t h0 = *reinterpret_cast<const bf16x8_t*>(&sm.h[0][16 * t + i][8 * (4 * uj[u] + g)]);
          const bf16x8_t h1 =
              q.slices == 2 ? *reinterpret_cast<const bf16x8_t*>(&sm.h[1][16 * t + i][8 * (4 * uj[u] + g)]) : h0;
#pragma unroll
          for (int r = 0; r < NT; ++r) {
            const f32x4_t y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[u][r], tiles.slice[r] ? h1 : h0,
                                                                      f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
            for (int v = 0; v < 4; ++v) low[r][v] += own ? y[v] : 0.f;
          }
        }
      if (n < U) break;
      request();
    }
  }
  if (took)
#pragma unroll
    for (int r = 0; r < NT; ++r) sm.low[t][r][lane] = low[r];
}

// 16 rows on a small grid: NT weight tiles a workgroup, its NW waves splitting
// K; chunks go straight into registers, and the partial sums meet in LDS, in
// wave order.
template <int NT, int NW>
struct SplitSmem : LowSmem<1, NT> {
  int row[16];
  int out[16];
  float w[16];
  f32x4_t red[NW][NT][kWave];
};

// tot[r][0] = weight tile NT nt + r, in wave 0.  D: chunks in flight per wave.
template <int NT, int NW, int D, typename Smem>
__device__ __forceinline__ void split_product(const GemmParams& p, const AdapterParams& q, Smem& sm, int expert, int nt,
                                              f32x4_t (&tot)[NT][1]) {
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int g = lane >> 4;
  const int KC = p.KC;
  const int c0 = (int)((int64_t)wave * KC / NW), c1 = (int)((int64_t)(wave + 1) * KC / NW);
  gptr_t wbase[NT], sbase[NT];
#pragma unroll
  for (int r = 0; r < NT; ++r) {
    const int64_t tile = (int64_t)expert * p.w_tiles + min(NT * nt + r, p.NT - 1);
    wbase[r] = uniform_ptr(p.packed_w + tile * KC * kWave);
    sbase[r] = uniform_ptr(p.packed_s + tile * ((KC + 1) / 2) * kWave);
  }
  const gptr_t xbase = uniform_ptr(p.a);
  // rows past the block's read its first row, for columns that nothing stores
  const int own_row = sm.row[lane & 15];
  const uint32_t xoff = (uint32_t)(own_row >= 0 ? own_row : sm.row[0]) * (uint32_t)(p.K * 2) + 16 * g;
  const DequantMasks masks = make_dequant_masks();
  u32x4_t w[D][NT];
  uint32_t sw[D][NT];
  u32x4_t x[D][4];
  auto issue = [&](auto st_, int c) {
    constexpr int st = decltype(st_)::value;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      w[st][r] = gload_u32x4(wbase[r] + (int64_t)c * (kWave * 16) + lane * 16);
      sw[st][r] = gload_u32(sbase[r] + (int64_t)(c >> 1) * (kWave * 4) + lane * 4);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) x[st][j] = gload_u32x4(xbase + (c * kChunk + 32 * j) * 2 + xoff);
    __builtin_amdgcn_sched_barrier(0);
  };
  f32x4_t acc[NT];
#pragma unroll
  for (int r = 0; r < NT; ++r) acc[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](auto st_, int c) {
    constexpr int st = decltype(st_)::value;
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      transpose_words(w[st][r]);
      const u32x4_t scales = spread_scales((c & 1) ? (sw[st][r] & 0xFFFF0000u) : (sw[st][r] << 16));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t sbits = scales[j];
        const float s = __builtin_bit_cast(float, sbits);
        const bf16x8_t A = dequant8(w[st][r][j], s, -1032.0f * s, 0.0625f * s, -72.0f * s, masks);
        acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, __builtin_bit_cast(bf16x8_t, x[st][j]), acc[r], 0, 0, 0);
      }
    }
  };
  const int last = max(c1 - 1, 0);
  ring_steps<D>([&](auto st_) { issue(st_, min(c0 + decltype(st_)::value, last)); });
  if (q.L > 0) deal_adapters<1, NT, NW>(p, q, sm, expert, NT * nt);   // while the first chunks are under way
  ring_run<D>(c0, c1, multiply, issue);
#pragma unroll
  for (int r = 0; r < NT; ++r) sm.red[wave][r][lane] = acc[r];
  lds_only_barrier();
  if (wave > 0) return;
#pragma unroll
  for (int r = 0; r < NT; ++r) {
    tot[r][0] = sm.red[0][r][lane];
#pragma unroll
    for (int v = 1; v < NW; ++v) tot[r][0] += sm.red[v][r][lane];
    tot[r][0] += sm.low[0][r][lane];
  }
}

}  // namespace w4a16

// Router: gate logits [T, E] -> the top-k experts of each token and their
// weights, what moe_align and the few-token layer start from.
//
//   softmax   p_e = exp(l_e - m) / sum_e' exp(l_e' - m); order by l_e
//   sigmoid   s_e = 1 / (1 + exp(-l_e));  order by s_e + b_e, or by l_e
//             without a bias (s is strictly increasing)
// The weights are p or s of the chosen experts (never the bias), divided by
// their sum where `renormalize` asks for it, times `scale`.  An expert whose
// logit (or bias) is -inf or NaN is masked; a slot for which no expert is
// left gets id -1 and weight 0.
//
// A group of L lanes holds one token, V = ceil(E / L) keys a lane (expert
// i L + lane, so loads are coalesced).  What bounds a long batch is the
// number of vector instructions a token, not its bytes, so the k winners are
// not taken out one by one:
//   1. each lane's maximum; the k-th largest of those L maxima is a lower
//      bound of the k-th largest key (k rounds of a DPP maximum over the
//      group, equal maxima leaving together);
//   2. every expert at or above the bound is appended to a list in LDS: k
//      of them and a few more (L sum_{i<k} 1 / (L - i) expected: 11 at k = 8,
//      L = 16; 18 at k = 16, L = 64);
//   3. each listed expert counts the listed ones that come before it (larger
//      key, or equal and lower index): its rank, whatever the list's order.
// A list that overflows is made once more above its own k-th key; if it
// overflows again (many equal keys) k passes over the row take its place.
//
// Order with a bias.  s_e + b_e in 32 bits carries an error of a few 2^-24,
// enough to swap two experts that nearly tie.  The list's bound is lowered by
// that error, and where two of its keys are closer than it the group ranks
// the list again by s_e + b_e in 64 bits.
#include <algorithm>
#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"

namespace w4a16 {

namespace {

constexpr int kRouteThreads = 256;
constexpr float kMaxFinite = 3.402823466e+38f;

// +inf counts as the largest finite value; a NaN stays one
template <typename T>
__device__ __forceinline__ float logit_value(T v) {
  const float x = (float)v;
  return x > kMaxFinite ? kMaxFinite : x;
}

// a buffer of bytes, bounds checked by the load (zero past its end)
constexpr int kRawBuffer = 0x00027000;

template <typename T>
__device__ __forceinline__ float buffer_value(__amdgpu_buffer_rsrc_t buffer, uint32_t at) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t v = __builtin_amdgcn_raw_buffer_load_b32(buffer, at, 0, 0);
    return __builtin_bit_cast(float, v);
  } else {
    const uint16_t v = __builtin_amdgcn_raw_buffer_load_b16(buffer, at, 0, 0);
    return (float)__builtin_bit_cast(T, v);
  }
}

template <int kCtrl>
__device__ __forceinline__ float max_dpp(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, 0xF, 0xF, false);
  return fmaxf(v, __builtin_bit_cast(float, o));
}

// maximum over the group of L lanes, in each of them: rotations within rows
// of 16 lanes, then (L = 64) rows and halves exchanged
template <int L>
__device__ __forceinline__ float group_max(float v) {
  v = max_dpp<0x121>(v);
  v = max_dpp<0x122>(v);
  v = max_dpp<0x124>(v);
  v = max_dpp<0x128>(v);
  if constexpr (L == 64) {
    const uint32_t a = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    const uint32_t r0 = r[0], r1 = r[1];
    const uint32_t b = __builtin_bit_cast(uint32_t, fmaxf(__builtin_bit_cast(float, r0), __builtin_bit_cast(float, r1)));
    const auto q = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const uint32_t q0 = q[0], q1 = q[1];
    v = fmaxf(__builtin_bit_cast(float, q0), __builtin_bit_cast(float, q1));
  }
  return v;
}

template <int kCtrl>
__device__ __forceinline__ double add_dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, kCtrl, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), kCtrl, 0xF, 0xF, false);
  return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// sum over the group, the same bits in each of its lanes: neighbours, pairs
// (quad_perm), mirrored halves and rows, then (L = 64) rows
template <int L>
__device__ __forceinline__ double group_sum(double v) {
  v = add_dpp<0xB1>(v);
  v = add_dpp<0x4E>(v);
  v = add_dpp<0x141>(v);
  v = add_dpp<0x140>(v);
#pragma unroll
  for (int m = 16; m < L; m *= 2) v += __shfl_xor(v, m);
  return v;
}

// sum over the lanes of the group before this one (row_shr 1, 2, 4, 8 inside
// a row; then the rows before)
template <int L>
__device__ __forceinline__ int group_prefix(int v) {
  int s = v;
  s += __builtin_amdgcn_update_dpp(0, s, 0x111, 0xF, 0xF, true);
  s += __builtin_amdgcn_update_dpp(0, s, 0x112, 0xF, 0xF, true);
  s += __builtin_amdgcn_update_dpp(0, s, 0x114, 0xF, 0xF, true);
  s += __builtin_amdgcn_update_dpp(0, s, 0x118, 0xF, 0xF, true);
  if constexpr (L == 64) {
    const int a = __builtin_amdgcn_readlane(s, 15), b = __builtin_amdgcn_readlane(s, 31);
    const int c = __builtin_amdgcn_readlane(s, 47);
    const int row = (threadIdx.x % 64) / 16;
    s += (row > 0 ? a : 0) + (row > 1 ? b : 0) + (row > 2 ? c : 0);
  }
  return s - v;
}

// Weights before their division and scale: exp(x) of x <= 0, and
// 1 / (1 + exp(-x)) without overflow at either end.  Evaluated in 32 bits,
// within a few 2^-24, down to exp(-80); below that in 64, since an fp32 result
// would soon be a subnormal of fewer bits (2 % off at exp(-100)), which a
// division by a small sum or a large scale brings back into range.
constexpr float kExp32 = -80.f;

__device__ __forceinline__ double exp_weight(float x) {
  if (x < kExp32) return exp((double)x);
  return (double)expf(x);
}

__device__ __forceinline__ double sigmoid_weight(float x) {
  if (x < kExp32) return exp((double)x);                // 1 + exp(x) is 1 in 64 bits
  const float z = expf(-fabsf(x));
  return (double)((x >= 0.f ? 1.f : z) / (1.f + z));
}

// the same within 2^-22 absolutely (exp and reciprocal instructions; the
// exponent's rounding moves the result by at most |x| e^-|x| 2^-24 more)
__device__ __forceinline__ float sigmoid_key(float x) { return __builtin_amdgcn_rcpf(1.f + __expf(-x)); }

// keys of two experts further apart than this are in true order: each is off
// by at most 2^-22 (sigmoid) + half a unit of the sum
__device__ __forceinline__ float key_error(float c) { return 0x1p-21f + 0x1p-23f * (fabsf(c) + 1.f); }

__device__ __forceinline__ double exact_key(float x, float b) {
  return fmin(1.0 / (1.0 + exp(-(double)x)) + (double)b, 1.7976931348623157e308);
}

struct RouteArgs {
  const void* logits;
  int64_t row_stride;          // elements between rows
  const float* bias;           // sigmoid only, or NULL
  int32_t T, E, topk;
  int32_t renorm;
  float scale;
  int32_t* ids;
  float* weights;
};

// A listed expert as one number, larger = earlier in order of choice: the
// key's bits in rising order (-0 as +0), then the expert, lower first.
__device__ __forceinline__ uint64_t listed_as(float key, int expert) {
  const uint32_t u = __builtin_bit_cast(uint32_t, key + 0.f);
  const uint32_t up = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return (uint64_t)up << 32 | (uint32_t)~expert;
}
__device__ __forceinline__ int listed_expert(uint64_t c) { return (int)~(uint32_t)c; }
__device__ __forceinline__ float listed_key(uint64_t c) {
  const uint32_t up = (uint32_t)(c >> 32);
  return __builtin_bit_cast(float, up ^ ((uint32_t)((int32_t)~up >> 31) | 0x80000000u));
}

// in order of choice: larger key first, the lower expert of equals
template <typename K>
__device__ __forceinline__ bool before(K a, int ea, K b, int eb) { return a > b || (a == b && ea < eb); }

template <int L>
struct RouteSmem {
  static constexpr int G = kRouteThreads / L;      // tokens per workgroup
  static constexpr int CAP = 2 * (L < 32 ? 16 : L);  // listed experts a token, at most
  uint64_t list[G][CAP + 4];                        // read four at a time, zeros behind the last
  float logit[G][CAP];                              // with a bias
  float sorted[G][CAP];                             // with a bias: the keys in order
  float kth[G];                                     // of an overflowing list
  double exact[G][CAP];
  int count[G];
};

template <typename T, int L, int V, bool kSigmoid>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(const RouteArgs p) {
  using Smem = RouteSmem<L>;
  constexpr int OWN = Smem::CAP / L;                // listed experts a lane looks after
  __shared__ Smem sm;
  const int g = threadIdx.x / L, l = threadIdx.x % L;
  // groups past the last token follow it and store nothing
  const int64_t t0 = (int64_t)blockIdx.x * Smem::G;
  const int follow = (int)min((int64_t)g, p.T - 1 - t0);
  const bool real = follow == g;
  const int64_t t = t0 + follow;
  // the workgroup's rows: a uniform base and 32-bit offsets (the launcher
  // bounds the stride).  Read as a buffer that ends with the last row's E
  // values: offsets are constants added by the load, and what a lane reads
  // past its row is in the buffer, or zero, and masked below.
  const T* rows = static_cast<const T*>(p.logits) + t0 * p.row_stride;
  const uint32_t row0 = (uint32_t)follow * (uint32_t)p.row_stride;
  const uint32_t held = (uint32_t)min((int64_t)Smem::G, p.T - t0) - 1u;   // rows of the workgroup, less one
  const uint32_t extent = (held * (uint32_t)p.row_stride + (uint32_t)p.E) * (uint32_t)sizeof(T);
  const bool biased = kSigmoid && p.bias != nullptr;

  // keys; -inf: masked or past E
  float x[V], key[V];
  const auto row_buffer = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(rows), 0, extent, kRawBuffer);
  const uint32_t lane0 = (row0 + l) * (uint32_t)sizeof(T);
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = buffer_value<T>(row_buffer, lane0 + i * L * (uint32_t)sizeof(T));
  double sum = 0.0;
  float m = -INFINITY;
  if (biased) {
    // an infinite logit needs no clamp here (its score is 1); a NaN bias
    // makes a NaN key, which loses every comparison below
    const auto bias_buffer = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(p.bias), 0, 4u * (uint32_t)p.E, kRawBuffer);
    float b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = buffer_value<float>(bias_buffer, (uint32_t)l * 4u + i * L * 4u);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float c = sigmoid_key(x[i]) + b[i];
      key[i] = i * L + l < p.E && x[i] > -INFINITY ? (c > kMaxFinite ? kMaxFinite : c) : -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      key[i] = i * L + l < p.E && x[i] > -INFINITY ? fminf(x[i], kMaxFinite) : -INFINITY;   // a NaN compares false
  }
#pragma unroll
  for (int i = 0; i < V; ++i) m = fmaxf(m, key[i]);
  const float top = group_max<L>(m);
  if (!kSigmoid && !p.renorm) {                     // softmax over every live expert
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] > -INFINITY) sum += (double)expf(key[i] - top);
    sum = group_sum<L>(sum);
  }

  // the k-th largest lane maximum
  float bound = top;
  {
    float rest = m;
    for (int j = 1; j < p.topk; ++j) {
      rest = rest == bound ? -INFINITY : rest;
      bound = group_max<L>(rest);
    }
  }
  if (biased) bound -= key_error(bound);
  bound = fmaxf(bound, -kMaxFinite);                // fewer lanes than k hold an expert: every live one (NaN: as well)
  int expert[OWN], rank[OWN], listed, n;
  uint64_t own[OWN];
  float logit[OWN];
  // the list, and the ranks in it.  Where it overflows, the k-th of the listed
  // is a higher bound: once more with that.
  for (bool again = false;; again = true) {
    int mine = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) mine += key[i] >= bound ? 1 : 0;
    int at = group_prefix<L>(mine);
    if (l == L - 1) sm.count[g] = at + mine;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] >= bound) {
        if (at < Smem::CAP) {
          sm.list[g][at] = listed_as(key[i], i * L + l);
          if (biased) sm.logit[g][at] = x[i];
        }
        ++at;
      }
    __builtin_amdgcn_wave_barrier();
    listed = sm.count[g];
    n = min(listed, Smem::CAP);
    if (l < 4) sm.list[g][n + l] = 0;               // comes before nothing
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < OWN; ++q) {
      own[q] = sm.list[g][l + q * L];
      expert[q] = l + q * L < n ? listed_expert(own[q]) : -1;
      logit[q] = biased ? sm.logit[g][l + q * L] : listed_key(own[q]);
      rank[q] = 0;
    }
    auto count = [&](auto owned) {
      constexpr int Q = decltype(owned)::value;
      for (int j = 0; j < n; j += 4) {
        uint64_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = sm.list[g][j + i];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int q = 0; q < Q; ++q) rank[q] += c[i] > own[q] ? 1 : 0;
      }
    };
    if (__ballot(n > L)) count(std::integral_constant<int, OWN>{});   // any group of the wave
    else count(std::integral_constant<int, 1>{});
    if (again || !__ballot(listed > Smem::CAP)) break;
    if (listed > Smem::CAP) {
#pragma unroll
      for (int q = 0; q < OWN; ++q)
        if (rank[q] == p.topk - 1) sm.kth[g] = listed_key(own[q]);
    }
    __builtin_amdgcn_wave_barrier();
    if (listed > Smem::CAP) {
      const float k = sm.kth[g];
      bound = fmaxf(bound, biased ? k - key_error(k) : k);
    }
  }
  bool close = false;
  if (biased) {
    // neighbours in order: where any two are close, two neighbours are
#pragma unroll
    for (int q = 0; q < OWN; ++q)
      if (expert[q] >= 0) sm.sorted[g][rank[q]] = listed_key(own[q]);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < OWN; ++q)
      if (expert[q] >= 0 && rank[q] + 1 < n) {
        const float k = listed_key(own[q]), next = sm.sorted[g][rank[q] + 1];
        close = close || k - next <= fmaxf(key_error(k), key_error(next));
      }
  }
  if (biased && __ballot(close)) {                  // any group of the wave
    double exact[OWN];
#pragma unroll
    for (int q = 0; q < OWN; ++q) {
      exact[q] = -HUGE_VAL;
      if (expert[q] >= 0) {
        exact[q] = exact_key(logit[q], p.bias[expert[q]]);
        sm.exact[g][l + q * L] = exact[q];
      }
      rank[q] = 0;
    }
    __builtin_amdgcn_wave_barrier();
    for (int j = 0; j < n; ++j) {
      const double c = sm.exact[g][j];
      const int e = listed_expert(sm.list[g][j]);
#pragma unroll
      for (int q = 0; q < OWN; ++q) rank[q] += before(c, e, exact[q], expert[q]) ? 1 : 0;
    }
  }
  if (__ballot(listed > Smem::CAP)) {
    // more equal keys than the list holds: k passes, each the best after the last
    double last = HUGE_VAL;
    int last_e = -1;
    int found[OWN];
#pragma unroll
    for (int q = 0; q < OWN; ++q) found[q] = -1;
    for (int j = 0; j < p.topk; ++j) {
      double best = -HUGE_VAL;
      int best_e = p.E;
      for (int e = l; e < p.E; e += L) {
        const float v = logit_value(rows[row0 + e]);
        const float b = biased ? p.bias[e] : 0.f;
        if (!(v > -INFINITY && b > -INFINITY)) continue;
        const double c = biased ? exact_key(v, b) : (double)v;
        if (before(last, last_e, c, e) && before(c, e, best, best_e)) {
          best = c;
          best_e = e;
        }
      }
#pragma unroll
      for (int s = 1; s < L; s *= 2) {
        const double c = __shfl_xor(best, s);
        const int e = __shfl_xor(best_e, s);
        if (before(c, e, best, best_e)) {
          best = c;
          best_e = e;
        }
      }
      last = best;
      last_e = best_e;
#pragma unroll
      for (int q = 0; q < OWN; ++q)
        if (j == l + q * L && best > -HUGE_VAL) found[q] = best_e;
    }
    if (listed > Smem::CAP) {
#pragma unroll
      for (int q = 0; q < OWN; ++q) {
        expert[q] = found[q];
        rank[q] = found[q] >= 0 ? l + q * L : p.topk;
        if (found[q] >= 0) logit[q] = logit_value(rows[row0 + found[q]]);
      }
    }
  }

  // weights of the chosen, each by the lane that ranked it; sums in 64 bits
  double w[OWN], chosen = 0.0;
#pragma unroll
  for (int q = 0; q < OWN; ++q) {
    w[q] = 0.0;
    if (expert[q] >= 0 && rank[q] < p.topk) w[q] = kSigmoid ? sigmoid_weight(logit[q]) : exp_weight(logit[q] - top);
    chosen += w[q];
  }
  if (p.renorm) sum = group_sum<L>(chosen) + (kSigmoid ? 1e-20 : 0.0);
  if (!real) return;
  const bool divide = !kSigmoid || p.renorm;
#pragma unroll
  for (int q = 0; q < OWN; ++q) {
    if (expert[q] >= 0 && rank[q] < p.topk) {
      p.ids[t * p.topk + rank[q]] = expert[q];
      p.weights[t * p.topk + rank[q]] = (float)((divide ? w[q] / sum : w[q]) * (double)p.scale);
    }
  }
  // slots for which no expert was left (an overflowing list never leaves any)
  for (int j = n + l; j < p.topk; j += L) {
    p.ids[t * p.topk + j] = -1;
    p.weights[t * p.topk + j] = 0.f;
  }
}

// Lanes per token: 16 lanes share every instruction of the search with three
// other tokens, 64 lanes finish a token sooner; a 16-lane list stays short
// only while k is well below 16; and past 512 experts 16 lanes hold more keys,
// logits and biases than their registers do.  Measured on MI355X, graph
// replays (an empty launch is about 4.5 us), 64 / 16 lanes, us:
//                                  4096 tokens   6144        8192        16384
//   256 experts  sigmoid+bias k 8    7.0 /  7.4   9.3 /  7.9  10.2 /  7.8  16.6 /  9.5
//   384          sigmoid+bias k 8    7.5 /  8.4   9.6 /  9.2  11.0 /  9.1  17.9 / 11.5
//   384          sigmoid+bias k 10   8.1 / 10.1  10.1 /  9.5  12.2 / 10.1  19.7 / 12.7
//   384     bf16 softmax      k 8    6.6 /  6.3   7.9 /  6.7   9.3 /  6.8  14.8 /  8.4
//   384     bf16 softmax      k 10   7.1 /  8.8   8.7 /  9.1  10.4 /  9.2  16.7 / 11.3
//   512          sigmoid+bias k 8    7.9 /  9.4   9.7 / 10.2  11.3 / 10.2  19.2 / 16.5
//   640          sigmoid+bias k 8    9.0 / 11.8  10.8 / 19.9  13.1 / 20.3  22.2 / 40.7
//   640     fp32 softmax      k 8    7.3 /  8.3   9.0 /  9.4  10.4 /  9.2  17.7 / 17.3
//  1024          sigmoid+bias k 8    9.5 / 13.2  11.6 / 23.4  14.3 / 23.4  24.6 / 48.4
//  1024     bf16 softmax      k 8    7.6 /  8.9   9.2 / 12.4  11.0 / 13.3  18.0 / 17.4
// and 384 experts, sigmoid + bias, 8192 tokens, top 12 13.0 / 12.8, top 14
// 14.4 / 62 (lists that overflow twice).  (Taking the k winners out one by
// one, 64 lanes: 16384 tokens 25 us.  A 16-lane list that went straight to k
// passes when it overflowed: 8192 tokens top 10 81 us.)  What 16384 tokens
// spend: about 880 vector instructions a wave of four tokens, whose issue
// fills half of the kernel's 10.5 - 12 us, and the chains of the rounds and of the
// list in LDS for the rest.
constexpr int kNarrowMaxTopk = 10;
constexpr int kNarrowMinTokens = 6144;
constexpr int kNarrowMaxExperts = 512;

// Threads of one launch are counted in 32 bits, and a grid past them wraps
// without an error: 2^26 tokens of 64 lanes would be no workgroup at all.
// Longer batches go in pieces, each far below.
constexpr int kLaunchTokens = 1 << 24;

template <typename T, bool kSigmoid>
hipError_t launch_piece(const RouteArgs& a, int lanes, hipStream_t stream) {
  const int v = (a.E + lanes - 1) / lanes;
  const int per = kRouteThreads / lanes;
  const dim3 grid((unsigned)((a.T + per - 1) / per)), block(kRouteThreads);
  // keys per lane rounded up to a built width
#define W4A16_ROUTE_CASE(L_, V_)                                                         \
  if (lanes == L_ && v <= V_) {                                                          \
    hipLaunchKernelGGL((route_kernel<T, L_, V_, kSigmoid>), grid, block, 0, stream, a);  \
    return hipGetLastError();                                                            \
  }
  W4A16_ROUTE_CASE(16, 8) W4A16_ROUTE_CASE(16, 16) W4A16_ROUTE_CASE(16, 24) W4A16_ROUTE_CASE(16, 32)
  W4A16_ROUTE_CASE(64, 2) W4A16_ROUTE_CASE(64, 4) W4A16_ROUTE_CASE(64, 6) W4A16_ROUTE_CASE(64, 8)
  W4A16_ROUTE_CASE(64, 14) W4A16_ROUTE_CASE(64, 16)
#undef W4A16_ROUTE_CASE
  return hipErrorInvalidValue;
}

template <typename T, bool kSigmoid>
hipError_t launch_typed(const RouteArgs& a, hipStream_t stream) {
  const bool narrow = a.topk <= kNarrowMaxTopk && a.T >= kNarrowMinTokens && a.E <= kNarrowMaxExperts;
  for (int64_t t = 0; t < a.T; t += kLaunchTokens) {
    RouteArgs piece = a;
    piece.logits = static_cast<const T*>(a.logits) + t * a.row_stride;
    piece.T = (int32_t)std::min((int64_t)kLaunchTokens, a.T - t);
    piece.ids = a.ids + t * a.topk;
    piece.weights = a.weights + t * a.topk;
    const hipError_t e = launch_piece<T, kSigmoid>(piece, narrow ? 16 : 64, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_route(const void* logits, int dtype, int64_t row_stride, const float* bias, int32_t T, int32_t E,
                        int32_t topk, int sigmoid, int renorm, float scale, int32_t* ids, float* weights,
                        hipStream_t stream) {
  const RouteArgs a{logits, row_stride, bias, T, E, topk, renorm, scale, ids, weights};
  switch (2 * dtype + (sigmoid ? 1 : 0)) {
    case 0: return launch_typed<float, false>(a, stream);
    case 1: return launch_typed<float, true>(a, stream);
    case 2: return launch_typed<__bf16, false>(a, stream);
    case 3: return launch_typed<__bf16, true>(a, stream);
    case 4: return launch_typed<_Float16, false>(a, stream);
    case 5: return launch_typed<_Float16, true>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace w4a16

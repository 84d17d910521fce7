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
// One wave per token.  Lane l holds experts [l V, l V + V) in registers as
// order-preserving 32-bit integers, so the wave's maximum is four DPP steps
// and four lane reads, and the winner of equal keys -- the lowest expert --
// is the lowest set bit of a ballot.  k rounds; a round costs about 3 V + 20
// instructions.  The bytes that have to move are the logits, read once; each
// row is read by one wave, and the weights are worked out by lanes 0 .. k - 1
// at the end.
//
// Order with a bias.  s_e + b_e in 32 bits carries an error of a few 2^-24,
// enough to swap two experts that nearly tie.  After k + 1 rounds the gaps
// between consecutive winners are compared with that error's bound; where one
// is too small the wave forms s_e + b_e in 64 bits for the candidates (every
// expert whose 32-bit key could be among the top k) and picks again from
// those.  About one token in a hundred takes that path at 384 experts.
#include "device_common.hpp"
#include "launch.hpp"

namespace w4a16 {

namespace {

constexpr int kRouteWaves = 4;      // tokens per workgroup
constexpr float kMaxFinite = 3.402823466e+38f;

template <typename T>
__device__ __forceinline__ float logit_value(const T* p);
template <>
__device__ __forceinline__ float logit_value<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float logit_value<_Float16>(const _Float16* p) { return (float)*p; }
template <>
__device__ __forceinline__ float logit_value<__bf16>(const __bf16* p) { return (float)*p; }

// Ordered key of a value that is not NaN: u < v as integers exactly when
// a < b as floats; -0 counts as +0.  0 is below every value's key.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __builtin_bit_cast(float, u ^ ((uint32_t)((int32_t)~u >> 31) | 0x80000000u));
}

template <int kCtrl>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, false));
}

// maximum over the wave, in every lane (a scalar): rotate within rows of 16
// lanes (row_ror 1, 2, 4, 8), then the four rows
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max_dpp<0x121>(v);
  v = max_dpp<0x122>(v);
  v = max_dpp<0x124>(v);
  v = max_dpp<0x128>(v);
  const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
  const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
  return max(max(a, b), max(c, d));
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < kWave; m *= 2) v += __shfl_xor(v, m);
  return v;
}

__device__ __forceinline__ double wave_max_f64(double v) {
#pragma unroll
  for (int m = 1; m < kWave; m *= 2) v = fmax(v, __shfl_xor(v, m));
  return v;
}

// 1 / (1 + exp(-x)), without overflow at either end
__device__ __forceinline__ float sigmoid32(float x) {
  const float z = expf(-fabsf(x));
  return (x >= 0.f ? 1.f : z) / (1.f + z);
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

template <typename T, int V, bool kSigmoid>
__global__ __launch_bounds__(kRouteWaves * kWave) void route_kernel(const RouteArgs p) {
  extern __shared__ double exact_keys[];                  // kRouteWaves x 64 V, only with a bias
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (t >= p.T) return;                                   // whole waves; the workgroup never synchronises
  const T* row = static_cast<const T*>(p.logits) + t * p.row_stride;
  const int e0 = lane * V;
  const bool biased = kSigmoid && p.bias != nullptr;

  // masked experts: key 0; a +inf logit counts as the largest finite value
  float x[V], b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = min(e0 + i, p.E - 1);
    x[i] = logit_value<T>(row + e);
    b[i] = 0.f;
    if (biased) b[i] = p.bias[e];
  }
  uint32_t key[V];
  float top = -kMaxFinite;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool live = e0 + i < p.E && x[i] > -INFINITY && b[i] > -INFINITY;   // false for NaN
    const float v = fminf(x[i], kMaxFinite);
    key[i] = 0u;
    if (live) {
      key[i] = ordered(biased ? fminf(sigmoid32(v) + b[i], kMaxFinite) : v);
      top = fmaxf(top, v);
    }
  }
  if (!kSigmoid && !p.renorm) {                            // softmax over every live expert
    top = from_ordered(wave_max(ordered(top)));
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i]) sum += (double)expf(fminf(x[i], kMaxFinite) - top);
    sum = wave_sum(sum);
  }

  // k rounds; lane j keeps the j-th winner.  With a bias one round more, and
  // the smallest gap between neighbours against the error of their keys.
  int win = -1;
  uint32_t prev = 0;
  bool close = false;
  uint32_t threshold = 1u;
  const int rounds = p.topk + (biased ? 1 : 0);
  for (int j = 0; j < rounds; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = max(m, key[i]);
    const uint32_t best = wave_max(m);
    if (best == 0u) break;                                 // no live expert left
    if (biased) {
      const float c = from_ordered(best), a = from_ordered(prev);
      // each key: the sigmoid within 2^-22, the sum within half a unit
      const float err = 0x1p-21f + 0x1p-23f * fmaxf(fabsf(c), fabsf(a));
      close = close || (j > 0 && !(a - c > err));
      threshold = ordered(c - err);
      if (j == p.topk) break;                              // only its gap was wanted
    }
    const int src = __builtin_ctzll(__ballot(m == best));
    int slot = V - 1;
#pragma unroll
    for (int i = V - 2; i >= 0; --i) slot = key[i] == best ? i : slot;
    const int e = __builtin_amdgcn_readlane(e0 + slot, src);
    if (lane == j) win = e;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane == src && i == slot) key[i] = 0u;
    prev = best;
  }

  if (biased && close) {
    // The winners of the rounds above were taken out of `key`; the keys are
    // formed again in 64 bits for every expert that can be among the top k.
    double* mine = exact_keys + wave * (kWave * V) + lane * V;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool live = e0 + i < p.E && x[i] > -INFINITY && b[i] > -INFINITY;
      const float v = fminf(x[i], kMaxFinite);
      double c = -HUGE_VAL;
      if (live && ordered(fminf(sigmoid32(v) + b[i], kMaxFinite)) >= threshold)
        c = fmin(1.0 / (1.0 + exp(-(double)v)) + (double)b[i], 1.7976931348623157e308);
      mine[i] = c;
    }
    win = -1;
    for (int j = 0; j < p.topk; ++j) {
      double m = mine[0];
      int slot = 0;
      for (int i = 1; i < V; ++i) {
        const double c = mine[i];
        if (c > m) {
          m = c;
          slot = i;
        }
      }
      const double best = wave_max_f64(m);
      if (best == -HUGE_VAL) break;
      const int src = __builtin_ctzll(__ballot(m == best));
      const int e = __builtin_amdgcn_readlane(e0 + slot, src);
      if (lane == j) win = e;
      if (lane == src) mine[slot] = -HUGE_VAL;             // read again by this lane only
    }
  }

  // weights of the winners, lane j's own; sums in 64 bits
  float w = 0.f;
  if constexpr (kSigmoid) {
    if (win >= 0) w = sigmoid32(fminf(logit_value<T>(row + win), kMaxFinite));
    if (p.renorm) sum = wave_sum((double)w) + 1e-20;
  } else {
    float v = -kMaxFinite;
    if (win >= 0) v = fminf(logit_value<T>(row + win), kMaxFinite);
    // the first winner holds the largest logit
    const float first = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 0));
    if (win >= 0) w = expf(v - first);
    if (p.renorm) sum = wave_sum((double)w);
  }
  if (lane < p.topk) {
    const bool divide = !kSigmoid || p.renorm;
    const double q = win < 0 ? 0.0 : (divide ? (double)w / sum : (double)w) * (double)p.scale;
    p.ids[t * p.topk + lane] = win;
    p.weights[t * p.topk + lane] = (float)q;
  }
}

template <typename T, bool kSigmoid>
hipError_t launch_typed(const RouteArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), block(kRouteWaves * kWave);
  const int v = (a.E + kWave - 1) / kWave;
  // experts per lane rounded up to a built width
#define W4A16_ROUTE_CASE(V_)                                                                              \
  if (v <= V_) {                                                                                          \
    const size_t lds = a.bias != nullptr ? sizeof(double) * kRouteWaves * kWave * V_ : 0;                  \
    hipLaunchKernelGGL((route_kernel<T, V_, kSigmoid>), grid, block, lds, stream, a);                      \
    return hipGetLastError();                                                                             \
  }
  W4A16_ROUTE_CASE(1) W4A16_ROUTE_CASE(2) W4A16_ROUTE_CASE(4) W4A16_ROUTE_CASE(6) W4A16_ROUTE_CASE(8)
  W4A16_ROUTE_CASE(12) W4A16_ROUTE_CASE(14) W4A16_ROUTE_CASE(16)
#undef W4A16_ROUTE_CASE
  return hipErrorInvalidValue;
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

// Router with scores, balance bias and expert groups (gfx950).
//
// Of a token with logits l and E experts in G groups of E / G:
//   s_e = softmax(l)_e or sigmoid(l_e);   v_e = s_e + b_e
//   group score = sum of the group's best 1 or 2 values v; the best top_groups
//   groups stay;  ids = the k largest v there, ties to the lower index;
//   w_j = s_{id_j} [/ sum of the k], times scale.
// An expert is masked where its logit is -inf or NaN, or its bias; masked
// experts and those of dropped groups come last, by index, with weight 0, so
// that a token always has k different experts.
//
// Precision.  The order of two experts is decided by v in binary64: a
// prefill batch compares millions of neighbouring values, and in binary32
// (2^-24 around 1) some of them change places.  A candidate's key is the
// order-preserving pattern of the binary64 value with its lowest 10 bits
// replaced by the expert (1023 - e), so values nearer than 2^-42 of their
// size count as equal.  Without a bias v has the logits' order and the key is
// made of the logit itself.  Group scores are binary64 sums.  The k weights of
// a token are formed in binary64 and rounded once to binary32.
//
// Work.  The bytes are T * E logits, read once; what bounds the kernel is
// vector work: with a bias (or groups by two values) one binary64
// exponential for every logit (about the issue rate of binary32 on this
// chip, two registers a value), the sort of each lane's keys, and k rounds of
// a maximum over a token's lanes.  16 lanes share a token (four tokens a
// wave) or, for few tokens or more than 256 experts, the whole wave.
#include "common.hpp"
#include "dtype.hpp"
#include "kernels.hpp"
#include "route.hpp"

namespace nvfp4 {

namespace {

constexpr float kF32Max = 3.402823466e38f;
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float load_logit(const void* p, int dtype, int64_t i) {
  if (dtype == MOE_F32) return F32::get(p, i);
  return dtype == MOE_BF16 ? Bf16::get(p, i) : F16::get(p, i);
}

// NaN counts as masked, +inf as the largest finite value.
__device__ __forceinline__ float clean(float v) { return v >= kNegInf ? fminf(v, kF32Max) : kNegInf; }

__device__ __forceinline__ double sigmoid64(float v) { return 1.0 / (1.0 + exp(-static_cast<double>(v))); }

// Key of a binary64 value: its order-preserving pattern, the expert in the
// lowest 10 bits.  Finite values have a nonzero high word.
__device__ __forceinline__ uint64_t value_key(double v, int e) {
  uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  u = (u >> 63) ? ~u : (u | 0x8000000000000000ull);
  return (u & ~1023ull) | static_cast<uint64_t>(1023 - e);
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
  const uint64_t lo = dpp_u32<CTRL>(static_cast<uint32_t>(u)), hi = dpp_u32<CTRL>(static_cast<uint32_t>(u >> 32));
  return __longlong_as_double(static_cast<long long>((hi << 32) | lo));
}
__device__ __forceinline__ double row16_sum64(double v) {
  v += dpp_f64<kDppXor1>(v);
  v += dpp_f64<kDppXor2>(v);
  v += dpp_f64<kDppRor4>(v);
  v += dpp_f64<kDppRor8>(v);
  return v;
}
template <bool WAVE>
__device__ __forceinline__ double token_sum64(double v) {
  v = row16_sum64(v);
  if constexpr (WAVE) {
    v += __shfl_xor(v, 16, kWave);
    v += __shfl_xor(v, 32, kWave);
  }
  return v;
}
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, dpp_f32<kDppXor1>(v));
  v = fmaxf(v, dpp_f32<kDppXor2>(v));
  v = fmaxf(v, dpp_f32<kDppRor4>(v));
  v = fmaxf(v, dpp_f32<kDppRor8>(v));
  return v;
}
template <bool WAVE>
__device__ __forceinline__ float token_max(float v) {
  if constexpr (WAVE) return wave_max(v);
  else return row16_max(v);
}

// (best, second) of two such pairs
__device__ __forceinline__ void merge_best(double& a1, double& a2, double b1, double b2) {
  const double lo = fmin(a1, b1);
  a1 = fmax(a1, b1);
  a2 = fmax(fmax(a2, b2), lo);
}

}  // namespace

// Lanes of one token: 16 (four tokens a wave) or the wave; lane gl holds
// experts gl, gl + L, ... (KPL of them).
template <int KPL, bool WAVE>
__global__ __launch_bounds__(256) void moe_route_scores_kernel(RouteParams q) {
  constexpr int L = WAVE ? kWave : 16;
  constexpr int kTok = 256 / L;
  extern __shared__ double s_route[];  // [kTok][E] values and [kTok][kMaxRouteGroups] group scores (G > 1)
  const int lane = threadIdx.x & (kWave - 1), gl = lane & (L - 1), lt = threadIdx.x / L;
  const int E = q.E, k = q.k, G = q.groups;
  const int64_t t_own = static_cast<int64_t>(blockIdx.x) * kTok + lt;
  const int64_t t = min(t_own, static_cast<int64_t>(q.T) - 1);  // past the end: the last token again, not stored
  const bool softmax = q.score == MOE_SCORE_SOFTMAX;
  const bool has_bias = q.bias != nullptr;

  float v[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) v[i] = load_logit(q.logits, q.dtype, t * q.ld + min(gl + L * i, E - 1));
  uint32_t open = 0;  // bit i: expert gl + L i may be chosen
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    v[i] = gl + L * i < E ? clean(v[i]) : kNegInf;
    open |= (v[i] > kNegInf ? 1u : 0u) << i;
  }
  float m = v[0];
#pragma unroll
  for (int i = 1; i < KPL; ++i) m = fmaxf(m, v[i]);
  m = token_max<WAVE>(m);
  if (!(m > kNegInf)) m = 0.0f;  // no expert at all: every exponential below is 0

  // values in binary64 where the order or the groups need them
  const bool values = has_bias || (G > 1 && q.group_best == 2);
  double val[KPL];
  double z = 0.0;  // the softmax sum, where it is needed
  if (values) {
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      val[i] = softmax ? exp(static_cast<double>(v[i]) - static_cast<double>(m)) : sigmoid64(v[i]);
    if (softmax && (has_bias || !q.renormalize)) {
#pragma unroll
      for (int i = 0; i < KPL; ++i) z += val[i];
      z = token_sum64<WAVE>(z);
    }
    if (has_bias) {
      const double rz = softmax && z > 0.0 ? 1.0 / z : 1.0;
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        const float b = clean(q.bias[min(gl + L * i, E - 1)]);
        if (!(b > kNegInf)) open &= ~(1u << i);
        val[i] = val[i] * rz + static_cast<double>(b);
      }
    }
  } else {
    if (softmax && !q.renormalize) {
      // (binary32 exponentials: they only scale the weights and order nothing)
#pragma unroll
      for (int i = 0; i < KPL; ++i) z += static_cast<double>(expf(v[i] - m));
      z = token_sum64<WAVE>(z);
    }
#pragma unroll
    for (int i = 0; i < KPL; ++i) val[i] = static_cast<double>(v[i]);  // groups by the largest logit
  }

  if (G > 1) {
    const int gs = E / G;
    double* sv = s_route + static_cast<int64_t>(lt) * E;
    double* sg = s_route + static_cast<int64_t>(kTok) * E + lt * kMaxRouteGroups;
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if (gl + L * i < E) sv[gl + L * i] = (open >> i) & 1 ? val[i] : static_cast<double>(kNegInf);
    __syncthreads();
    // P lanes a group (a power of two), L / P groups at a time
    int P = L;
    while (P > 1 && P * G > L) P >>= 1;
    const int sub = gl & (P - 1), per = L / P;
    for (int g0 = 0; g0 < G; g0 += per) {
      const int g = g0 + gl / P;
      double b1 = static_cast<double>(kNegInf), b2 = b1;
      if (g < G)
        for (int j = sub; j < gs; j += P) merge_best(b1, b2, sv[g * gs + j], static_cast<double>(kNegInf));
      for (int d = 1; d < P; d <<= 1) {
        const double o1 = __shfl_xor(b1, d, kWave), o2 = __shfl_xor(b2, d, kWave);
        merge_best(b1, b2, o1, o2);
      }
      if (g < G && sub == 0)
        sg[g] = q.group_best == 2 && b2 > static_cast<double>(kNegInf) ? b1 + b2 : b1;
    }
    __syncthreads();
    uint64_t kept = 0;
    for (int g0 = 0; g0 < G; g0 += L) {
      const int g = g0 + gl;
      const double mine = g < G ? sg[g] : static_cast<double>(kNegInf);
      int rank = 0;
      for (int h = 0; h < G; ++h) {
        const double o = sg[h];
        rank += (o > mine || (o == mine && h < g)) ? 1 : 0;
      }
      const uint64_t b = __ballot(g < G && rank < q.top_groups);
      kept |= WAVE ? b : (((b >> (lane & 48)) & 0xFFFFull) << g0);
    }
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int e = min(gl + L * i, E - 1);
      const int g = static_cast<int>((static_cast<uint32_t>(e) * q.group_magic) >> 20);  // e / gs
      if (!((kept >> g) & 1)) open &= ~(1u << i);
    }
  }

  // keys: closed experts have a zero high word and go by index
  uint64_t cand[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int e = gl + L * i;
    const uint64_t key = has_bias ? value_key(val[i], e) : route_key(v[i], e);
    const uint64_t last = has_bias ? static_cast<uint64_t>(2047 - e) : static_cast<uint32_t>(~e);
    cand[i] = e < E ? ((open >> i) & 1 ? key : last) : 0ull;
  }
  sort_keys_desc<KPL>(cand);
  uint64_t mine = 0, top = 0;
  if (k <= 8)
    select_rounds<KPL, 8, WAVE>(cand, k, gl, mine, top);
  else
    select_rounds<KPL, kMaxTopK, WAVE>(cand, k, gl, mine, top);

  // slot gl < k
  const int id = gl >= k ? 0 : has_bias ? 1023 - static_cast<int>(mine & 1023) : key_expert(mine);
  const bool on = gl < k && (mine >> 32) != 0;
  const float lv = on ? clean(load_logit(q.logits, q.dtype, t * q.ld + id)) : kNegInf;
  double w;
  if (softmax) {
    // normalized over the k: relative to their own largest, which may lie far
    // below the row's where a bias or the groups decide
    float ref = m;
    if (q.renormalize) {
      ref = row16_max(lv);
      if (!(ref > kNegInf)) ref = 0.0f;
    }
    w = exp(static_cast<double>(lv) - static_cast<double>(ref));
    if (!q.renormalize && z > 0.0) w /= z;
  } else {
    w = on ? sigmoid64(lv) : 0.0;
  }
  if (q.renormalize) {
    const double sum = row16_sum64(w);
    if (sum > 0.0) w /= sum;
  }
  if (gl < k && t_own < q.T) {
    q.ids[t * k + gl] = id;
    q.weights[t * k + gl] = static_cast<float>(w * static_cast<double>(q.scale));
  }
}

template <int KPL, bool WAVE>
static void launch_scores(const RouteParams& q, hipStream_t s) {
  constexpr int kTok = 256 / (WAVE ? kWave : 16);
  const size_t lds = q.groups > 1 ? static_cast<size_t>(kTok) * (q.E + kMaxRouteGroups) * sizeof(double) : 0;
  moe_route_scores_kernel<KPL, WAVE><<<static_cast<unsigned>((q.T + kTok - 1) / kTok), 256, lds, s>>>(q);
}

hipError_t launch_route_scores(const RouteParams& q, hipStream_t s) {
  if (q.E > 256 || q.T <= kRouteWaveTokens) {
    if (q.E <= 64) launch_scores<1, true>(q, s);
    else if (q.E <= 128) launch_scores<2, true>(q, s);
    else if (q.E <= 256) launch_scores<4, true>(q, s);
    else if (q.E <= 512) launch_scores<8, true>(q, s);
    else launch_scores<16, true>(q, s);
  } else {
    if (q.E <= 16) launch_scores<1, false>(q, s);
    else if (q.E <= 32) launch_scores<2, false>(q, s);
    else if (q.E <= 64) launch_scores<4, false>(q, s);
    else if (q.E <= 128) launch_scores<8, false>(q, s);
    else launch_scores<16, false>(q, s);
  }
  return hipGetLastError();
}

}  // namespace nvfp4

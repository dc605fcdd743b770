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
// (2^-24 around 1) some of them change places.  Ten bits of a candidate hold
// the expert, which takes 2^-42 of a value's size; scores are off by at most
// 2^-42 of theirs (exp64, recip64, the sum), so values that differ by less than
// 2^-40 of the larger of score and bias may change places.  Experts of equal
// logits and biases have equal values, the same in every batch.  Without a bias
// v has the logits' order and the candidate is made of the logit itself.  Group
// scores are binary64 sums.  The k weights of a token are formed in binary64 and
// rounded once to binary32 (a softmax sum of binary32 exponentials would put them up
// to 10 roundings off and saves little: 16384 tokens of 256 experts 9.2 us for 10.2).
//
// Work.  The bytes are T * E logits, read once; what bounds the kernel is
// vector work: with a bias (or groups by two values) one binary64
// exponential for every logit, the sort of each lane's candidates, and k
// rounds of a maximum over a token's lanes.  16 lanes share a token (four
// tokens a wave) or, for few tokens or more than 432 experts, the whole wave; a
// lane's experts are consecutive, so that groups of whole lanes are reduced in
// registers (through LDS: 2.7 us more of the 18.5).  16384 tokens of 256 experts
// take 15.2 us with bias and groups (1610 vector instructions for four tokens),
// 7.4 without (floor of the bytes: 3.7); one token of 128 experts 2.9 us, 64 of 256
// in groups 4.7 (replayed; single calls take 16.1 and 5.0).
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
// Values first .. first + KPL - 1 of a row of E; past the end the last one again.
template <typename T, int KPL>
__device__ __forceinline__ void load_row(float (&v)[KPL], const void* p, int64_t row, int first, int E) {
  if (first + KPL <= E) {
    // consecutive: wide loads at any address
    typename T::Word w[KPL];
    __builtin_memcpy(w, static_cast<const char*>(p) + (row + first) * T::kBytes, sizeof(w));
#pragma unroll
    for (int i = 0; i < KPL; ++i) v[i] = T::value(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < KPL; ++i) v[i] = T::get(p, row + min(first + i, E - 1));
  }
}

// NaN counts as masked, +inf as the largest finite value.
__device__ __forceinline__ float clean(float v) { return v >= kNegInf ? fminf(v, kF32Max) : kNegInf; }

// exp(x) in binary64 to 2^-46 of it, x in [-1200, 709]: x = n ln 2 + r with |r| <=
// ln 2 / 2, ln 2 subtracted in two parts of which n times the first is exact (W. J.
// Cody and W. Waite, "Software Manual for the Elementary Functions", 1980), e^r by
// its series to r^11 (the rest, r^12 / 12!, is below 2^-46.6 of it).  Below -708 with
// the absolute error of a subnormal number, 0 below -745.
__device__ __forceinline__ double exp64(double x) {
  const double n = __builtin_rint(x * 1.4426950408889634);
  const double r = __builtin_fma(n, -1.9082149292705877e-10, __builtin_fma(n, -0.693147180369123816490, x));
  double p = 1.0 / 39916800.0;
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_amdgcn_ldexp(p, static_cast<int>(n));
}
// The same for any x: above 709 the value there.
__device__ __forceinline__ double exp64_any(double x) { return exp64(fmin(fmax(x, -1200.0), 709.0)); }
// 1 / d for d >= 1, finite, to 2^-45 of it: the hardware's reciprocal (within
// 2^-23) and one Newton step.
__device__ __forceinline__ double recip64(double d) {
  const double y = __builtin_amdgcn_rcp(d);
  return __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
}
// sigmoid(v), beyond 709 the value there
__device__ __forceinline__ double sigmoid64(float v) {
  return recip64(1.0 + exp64(-static_cast<double>(__builtin_amdgcn_fmed3f(v, -709.0f, 709.0f))));
}

// A candidate as one binary64 number: the value with its lowest 10 bits
// replaced so that of equal values the lower expert's number is the larger.
// Its order is the numbers' own, so a comparator of the sort is one maximum
// and one minimum.  Masked experts come behind every value (|value| <= 2
// FLT_MAX), by index.
constexpr double kMasked = -0x1p1000;
__device__ __forceinline__ double candidate(double v, int e) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  const uint32_t low = (u >> 63) ? static_cast<uint32_t>(e) : static_cast<uint32_t>(1023 - e);
  return __longlong_as_double(static_cast<long long>((u & ~1023ull) | low));
}
__device__ __forceinline__ int candidate_expert(double c) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(c));
  const int low = static_cast<int>(u & 1023);
  return (u >> 63) ? low : 1023 - low;
}

template <int CTRL>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t u) {
  // (every lane has a source under these controls: no value to keep)
  const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, 0xF, 0xF, true));
  const uint64_t hi =
      static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, 0xF, 0xF, true));
  return (hi << 32) | lo;
}
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  return __longlong_as_double(static_cast<long long>(dpp_u64<CTRL>(static_cast<uint64_t>(__double_as_longlong(v)))));
}
// The mirrors reach a lane of the other half, where every lane has the same sum:
// each step adds the same two numbers in both of its lanes, so the sum is the
// same bits in all 16.
__device__ __forceinline__ double row16_sum64(double v) {
  v += dpp_f64<kDppXor1>(v);
  v += dpp_f64<kDppXor2>(v);
  v += dpp_f64<kDppHalfMirror>(v);
  v += dpp_f64<kDppMirror>(v);
  return v;
}
// The lanes of a token: a 16-lane row, or the wave, whose rows meet by register
// swaps (short; the vector ALU does them) or by shuffles through LDS (long;
// they leave it free).
enum class Lanes { kRow, kSwap, kShuffle };

// A lane's value and its partner's, 16 or 32 lanes away, in either order.
template <Lanes LANES, int PAIR>
__device__ __forceinline__ void lane_pair64(uint64_t u, uint64_t& a, uint64_t& b) {
  if constexpr (LANES == Lanes::kSwap) {
    uint32_t al, bl, ah, bh;
    lane_pair<PAIR>(static_cast<uint32_t>(u), al, bl);
    lane_pair<PAIR>(static_cast<uint32_t>(u >> 32), ah, bh);
    a = (static_cast<uint64_t>(ah) << 32) | al;
    b = (static_cast<uint64_t>(bh) << 32) | bl;
  } else {
    a = u;
    b = __shfl_xor(static_cast<unsigned long long>(u), PAIR, kWave);
  }
}
template <Lanes LANES, int PAIR>
__device__ __forceinline__ void lane_pair64(double v, double& a, double& b) {
  uint64_t x, y;
  lane_pair64<LANES, PAIR>(static_cast<uint64_t>(__double_as_longlong(v)), x, y);
  a = __longlong_as_double(static_cast<long long>(x));
  b = __longlong_as_double(static_cast<long long>(y));
}
// The sum of a token's exponentials e, each in [0, 1], as whole multiples of
// 2^-52 (the lowest bit of 1 + e; at e = 1 the pattern goes on into the next
// binade).  Whole numbers add up the same in any order, so every lane has the
// same bits, and so has the same token in another batch, where other lanes hold
// its experts: experts of equal logits and biases have equal values everywhere.
// Off by at most 2^-53 a term, 2^-43 of a sum of 1024 (it is at least 1 with any
// expert).
template <Lanes LANES, int KPL>
__device__ __forceinline__ double exp_sum(const double (&e)[KPL]) {
  constexpr uint64_t kOne = 0x3FF0000000000000ull;
  uint64_t u = 0;
#pragma unroll
  for (int i = 0; i < KPL; ++i) u += static_cast<uint64_t>(__double_as_longlong(1.0 + e[i]));
  u += dpp_u64<kDppXor1>(u);
  u += dpp_u64<kDppXor2>(u);
  u += dpp_u64<kDppHalfMirror>(u);
  u += dpp_u64<kDppMirror>(u);
  if constexpr (LANES != Lanes::kRow) {
    uint64_t a, b;
    lane_pair64<LANES, 16>(u, a, b);
    lane_pair64<LANES, 32>(a + b, a, b);
    u = a + b;
  }
  u -= kOne * static_cast<uint64_t>(KPL * (LANES == Lanes::kRow ? 16 : kWave));
  return 0x1p-52 * static_cast<double>(u);
}
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, dpp_f32<kDppXor1>(v));
  v = fmaxf(v, dpp_f32<kDppXor2>(v));
  v = fmaxf(v, dpp_f32<kDppRor4>(v));
  v = fmaxf(v, dpp_f32<kDppRor8>(v));
  return v;
}
template <Lanes LANES>
__device__ __forceinline__ float token_max(float v) {
  if constexpr (LANES != Lanes::kRow) return wave_max(v);
  else return row16_max(v);
}

template <Lanes LANES>
__device__ __forceinline__ double token_max64(double v) {
  v = fmax(v, dpp_f64<kDppXor1>(v));
  v = fmax(v, dpp_f64<kDppXor2>(v));
  v = fmax(v, dpp_f64<kDppRor4>(v));
  v = fmax(v, dpp_f64<kDppRor8>(v));
  if constexpr (LANES != Lanes::kRow) {
    double a, b;
    lane_pair64<LANES, 16>(v, a, b);
    lane_pair64<LANES, 32>(fmax(a, b), a, b);
    v = fmax(a, b);
  }
  return v;
}

// Batcher's odd-even merge sort (see route.hpp), largest first.  Its passes and
// the selection's rounds are template steps: a loop that the compiler leaves
// rolled indexes the list by chains of selects.
template <int N, int P, int D>
__device__ __forceinline__ void sort_pass(double (&c)[N]) {
#pragma unroll
  for (int a = D % P; a + D < N; ++a) {
    if ((a - D % P) / D % 2 == 0 && a / (2 * P) == (a + D) / (2 * P)) {
      const double hi = fmax(c[a], c[a + D]), lo = fmin(c[a], c[a + D]);
      c[a] = hi;
      c[a + D] = lo;
    }
  }
  if constexpr (D > 1) sort_pass<N, P, D / 2>(c);
  else if constexpr (2 * P < N) sort_pass<N, 2 * P, 2 * P>(c);
}
template <int N>
__device__ __forceinline__ void sort_desc64(double (&c)[N]) {
  if constexpr (N > 1) sort_pass<N, 1, 1>(c);
}

// The k selection rounds over the lanes' sorted lists, as select_rounds in
// route.hpp: lane j keeps round j's candidate.
template <int N, int KMAX, Lanes LANES, int J>
__device__ __forceinline__ void select_round(double (&c)[N], int k, int gl, double& mine) {
  if (J < k) {
    const double best = token_max64<LANES>(c[0]);
    mine = gl == J ? best : mine;
    const bool pop = c[0] == best;
    constexpr int kShift = N < KMAX - 1 - J ? N : KMAX - 1 - J;  // entries that can still become a head
#pragma unroll
    for (int i = 0; i < kShift; ++i) c[i] = pop ? (i + 1 < N ? c[i + 1] : 2.0 * kMasked) : c[i];
    if constexpr (J + 1 < KMAX) select_round<N, KMAX, LANES, J + 1>(c, k, gl, mine);
  }
}
template <int N, int KMAX, Lanes LANES>
__device__ __forceinline__ double select64(double (&c)[N], int k, int gl) {
  double mine = kMasked;
  select_round<N, KMAX, LANES, 0>(c, k, gl, mine);
  return mine;
}

// Orders a wave's own LDS writes before its reads (a token's lanes are in one
// wave; LDS works in order).
__device__ __forceinline__ void wave_lds_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// one more value to (best, second)
__device__ __forceinline__ void add_best(double& a1, double& a2, double v) {
  a2 = fmax(a2, fmin(a1, v));
  a1 = fmax(a1, v);
}
// (best, second) of two such pairs
__device__ __forceinline__ void merge_best(double& a1, double& a2, double b1, double b2) {
  const double lo = fmin(a1, b1);
  a1 = fmax(a1, b1);
  a2 = fmax(fmax(a2, b2), lo);
}
template <int CTRL>
__device__ __forceinline__ void merge_dpp(double& a1, double& a2) {
  merge_best(a1, a2, dpp_f64<CTRL>(a1), dpp_f64<CTRL>(a2));
}
template <Lanes LANES, int PAIR>
__device__ __forceinline__ void merge_pair(double& a1, double& a2) {
  double x1, y1, x2, y2;
  lane_pair64<LANES, PAIR>(a1, x1, y1);
  lane_pair64<LANES, PAIR>(a2, x2, y2);
  merge_best(x1, x2, y1, y2);
  a1 = x1;
  a2 = x2;
}
// The pairs of P consecutive lanes (a power of two) merged in each of them.  The
// mirrors reach a lane of the other half, where every lane has the same pair.
template <Lanes LANES>
__device__ __forceinline__ void merge_lanes(double& a1, double& a2, int P) {
  if (P > 1) merge_dpp<kDppXor1>(a1, a2);
  if (P > 2) merge_dpp<kDppXor2>(a1, a2);
  if (P > 4) merge_dpp<kDppHalfMirror>(a1, a2);
  if (P > 8) merge_dpp<kDppMirror>(a1, a2);
  if constexpr (LANES != Lanes::kRow) {
    if (P > 16) merge_pair<LANES, 16>(a1, a2);
    if (P > 32) merge_pair<LANES, 32>(a1, a2);
  }
}

}  // namespace

// Lanes of one token: 16 (four tokens a wave) or the wave; lane gl holds
// experts KPL gl .. KPL gl + KPL - 1.  BIAS: ranked by value, else by logit.
// A masked expert's value is -inf from the point where it is known to be.
template <int KPL, Lanes LANES, bool BIAS>
__global__ __launch_bounds__(256) void moe_route_scores_kernel(RouteParams q) {
  constexpr bool WAVE = LANES != Lanes::kRow;
  constexpr int L = WAVE ? kWave : 16;
  constexpr int kTok = 256 / L;
  constexpr double kNegInf64 = -__builtin_inf();
  extern __shared__ double s_route[];  // [kTok][kMaxRouteGroups] group scores, then [kTok][E + L] values (G > 1)
  const int lane = threadIdx.x & (kWave - 1), gl = lane & (L - 1), lt = threadIdx.x / L;
  const int E = q.E, k = q.k, G = q.groups;
  const int64_t t_own = block_id() * kTok + lt;
  const int64_t t = min(t_own, static_cast<int64_t>(q.T) - 1);  // past the end: the last token again, not stored
  const bool softmax = q.score == MOE_SCORE_SOFTMAX;

  float v[KPL];
  const int first = KPL * gl;
  if (q.dtype == MOE_F32) load_row<F32, KPL>(v, q.logits, t * q.ld, first, E);
  else if (q.dtype == MOE_BF16) load_row<Bf16, KPL>(v, q.logits, t * q.ld, first, E);
  else load_row<F16, KPL>(v, q.logits, t * q.ld, first, E);
  float b[BIAS ? KPL : 1];
  if constexpr (BIAS) load_row<F32, KPL>(b, q.bias, 0, first, E);
#pragma unroll
  for (int i = 0; i < KPL; ++i) v[i] = first + i < E ? clean(v[i]) : kNegInf;
  float m = 0.0f;  // the largest logit; 0 without any, where every exponential is 0
  if (softmax) {
    m = v[0];
#pragma unroll
    for (int i = 1; i < KPL; ++i) m = fmaxf(m, v[i]);
    m = token_max<LANES>(m);
    m = m > kNegInf ? m : 0.0f;
  }

  // What the experts (BIAS) and groups are ranked by: values in binary64, or
  // (groups by their largest value without a bias) the logits themselves.
  double val[KPL];
  double z = 0.0;  // the softmax sum, where it is needed
  const bool sums = softmax && (BIAS || !q.renormalize);
  if (BIAS || (G > 1 && q.group_best == 2)) {
    if (softmax) {
#pragma unroll
      for (int i = 0; i < KPL; ++i) val[i] = exp64(fmax(static_cast<double>(v[i]) - static_cast<double>(m), -1200.0));
      if (sums) z = exp_sum<LANES>(val);
    } else {
#pragma unroll
      for (int i = 0; i < KPL; ++i) val[i] = sigmoid64(v[i]);
    }
    if constexpr (BIAS) {
      const double rz = softmax ? recip64(fmax(z, 1.0)) : 1.0;  // (z >= 1 where there is any expert)
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        const float bi = clean(b[i]);
        if (!(bi > kNegInf)) v[i] = kNegInf;
        val[i] = __builtin_fma(val[i], rz, static_cast<double>(bi));
      }
    }
#pragma unroll
    for (int i = 0; i < KPL; ++i) val[i] = v[i] > kNegInf ? val[i] : kNegInf64;
  } else {
    if (sums) {
#pragma unroll
      for (int i = 0; i < KPL; ++i) val[i] = exp64(fmax(static_cast<double>(v[i]) - static_cast<double>(m), -1200.0));
      z = exp_sum<LANES>(val);
    }
#pragma unroll
    for (int i = 0; i < KPL; ++i) val[i] = static_cast<double>(v[i]);
  }

  if (G > 1) {
    const int gs = E / G;
    double* sg = s_route + lt * kMaxRouteGroups;
    // Best two values of each group.  Where a group is a power of two of whole
    // lanes they come from the lanes' registers; else from LDS, a lane's
    // values one double further apart so that lanes start on different banks.
    if (q.group_lanes > 0) {
      double b1 = val[0], b2 = kNegInf64;
#pragma unroll
      for (int i = 1; i < KPL; ++i) add_best(b1, b2, val[i]);
      merge_lanes<LANES>(b1, b2, q.group_lanes);
      const int g = gl / q.group_lanes;
      if (gl % q.group_lanes == 0 && g < G) sg[g] = q.group_best == 2 && b2 > kNegInf64 ? b1 + b2 : b1;
    } else {
      double* sv = s_route + kTok * kMaxRouteGroups + static_cast<int64_t>(lt) * (E + L);
#pragma unroll
      for (int i = 0; i < KPL; ++i)
        if (first + i < E) sv[first + i + gl] = val[i];
      wave_lds_fence();
      // P lanes a group (a power of two), L / P groups at a time
      int P = L;
      while (P > 1 && P * G > L) P >>= 1;
      const int sub = gl & (P - 1), per = L / P;
      for (int g0 = 0; g0 < G; g0 += per) {
        const int g = g0 + gl / P;
        double b1 = kNegInf64, b2 = kNegInf64;
        if (g < G) {
          for (int j = sub; j < gs; j += 4 * P) {  // four reads in flight; past the end: not counted
            double x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int e = g * gs + min(j + u * P, gs - 1);
              x[u] = sv[e + e / KPL];
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) add_best(b1, b2, j + u * P < gs ? x[u] : kNegInf64);
          }
        }
        merge_lanes<LANES>(b1, b2, P);
        if (g < G && sub == 0) sg[g] = q.group_best == 2 && b2 > kNegInf64 ? b1 + b2 : b1;
      }
    }
    wave_lds_fence();
    // a group's rank among all; kept where it is below top_groups
    const auto kept = [&](int g) {
      const double mine = sg[g];
      int rank = 0;
      for (int h0 = 0; h0 < G; h0 += 4) {
        double o[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) o[u] = sg[min(h0 + u, G - 1)];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          rank += h0 + u < G && (o[u] > mine || (o[u] == mine && h0 + u < g)) ? 1 : 0;
      }
      return rank < q.top_groups;
    };
    if (q.group_lanes > 0) {
      const bool keep = kept(min(gl / q.group_lanes, G - 1));  // all of the lane's experts are in one group
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        v[i] = keep ? v[i] : kNegInf;
        val[i] = keep ? val[i] : kNegInf64;
      }
    } else {
      uint64_t mask = 0;
      for (int g0 = 0; g0 < G; g0 += L) {
        const int g = g0 + gl;
        const uint64_t ballot = __ballot(g < G && kept(min(g, G - 1)));
        mask |= WAVE ? ballot : (((ballot >> (lane & 48)) & 0xFFFFull) << g0);
      }
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        const int g = static_cast<int>((static_cast<uint32_t>(min(first + i, E - 1)) * q.group_magic) >> 20);  // e / gs
        const bool keep = (mask >> g) & 1;
        v[i] = keep ? v[i] : kNegInf;
        val[i] = keep ? val[i] : kNegInf64;
      }
    }
  }

  double cand[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int e = first + i;
    const double rank = BIAS ? val[i] : static_cast<double>(v[i]);
    cand[i] = e < E ? candidate(v[i] > kNegInf ? rank : kMasked, e) : 2.0 * kMasked;
  }
  sort_desc64<KPL>(cand);
  const double mine = k <= 8 ? select64<KPL, 8, LANES>(cand, k, gl) : select64<KPL, kMaxTopK, LANES>(cand, k, gl);

  // slot gl < k
  const int id = gl < k ? candidate_expert(mine) : 0;
  const bool on = gl < k && mine > 0.5 * kMasked;
  const float lv = on ? clean(load_logit(q.logits, q.dtype, t * q.ld + id)) : kNegInf;
  // Weights.  Normalized over the k they are formed relative to the largest of
  // their logits (softmax) or, below 0, of their scores (sigmoid): with c that
  // logit, e^-c / (1 + e^-l) = 1 / (e^c + e^(c - l)), so that they are exact
  // however far below the row's largest the k lie.
  float ref = softmax ? m : 0.0f;
  if (q.renormalize) {
    const float most = row16_max(lv);
    ref = most > kNegInf ? (softmax ? most : fminf(most, 0.0f)) : 0.0f;
  }
  const double c = static_cast<double>(ref), l = static_cast<double>(lv);
  double w = softmax ? exp64_any(l - c) : recip64(exp64_any(c) + exp64_any(c - l));
  w = on ? w : 0.0;
  if (q.renormalize) {
    const double sum = row16_sum64(w);
    if (sum > 0.0) w /= sum;
  } else if (softmax && z > 0.0) {
    w /= z;
  }
  if (gl < k && t_own < q.T) {
    q.ids[t * k + gl] = id;
    q.weights[t * k + gl] = static_cast<float>(w * static_cast<double>(q.scale));
  }
}

template <int KPL, Lanes LANES>
static void launch_scores(RouteParams q, hipStream_t s) {
  constexpr int L = LANES == Lanes::kRow ? 16 : kWave, kTok = 256 / L;
  const int gs = q.E / q.groups, lanes = gs / KPL;
  const bool whole = gs % KPL == 0 && (lanes & (lanes - 1)) == 0;
  q.group_lanes = q.groups > 1 && whole ? lanes : 0;
  const size_t doubles = q.groups <= 1 ? 0 : kTok * (kMaxRouteGroups + (whole ? 0 : q.E + L));
  const dim3 blocks = grid_of((static_cast<int64_t>(q.T) + kTok - 1) / kTok);
  if (q.bias) moe_route_scores_kernel<KPL, LANES, true><<<blocks, 256, doubles * sizeof(double), s>>>(q);
  else moe_route_scores_kernel<KPL, LANES, false><<<blocks, 256, doubles * sizeof(double), s>>>(q);
}

// Few tokens wait for each step of their chain, many for the vector ALU (1000
// experts with a bias, k = 16: 64 tokens 7.2 us by swaps, 8.1 by shuffles; 16384
// 57.8 and 54.0).
template <int KPL>
static void launch_wave_scores(const RouteParams& q, hipStream_t s) {
  if (q.T <= kRouteWaveTokens) launch_scores<KPL, Lanes::kSwap>(q, s);
  else launch_scores<KPL, Lanes::kShuffle>(q, s);
}

// Most experts of which 16 lanes hold a token (their values for the groups,
// [16][E + 16] doubles, and the group scores within 64 KB of LDS).
constexpr int kRouteRowExperts = 432;
static_assert(8 * 16 * (kMaxRouteGroups + kRouteRowExperts + 16) <= 64 * 1024, "a block's groups and values");

hipError_t launch_route_scores(const RouteParams& q, hipStream_t s) {
  // A whole wave a token where 16 lanes would hold many experts each and the
  // batch does not fill the chip (256 experts in groups with a bias: 1 token
  // 4.4 us, with 16 lanes 6.3; 2048: 5.9 and 6.9; 4096: 8.7 and 7.0.  300, k = 16:
  // 2048 tokens 5.7 and 5.8, 4096 8.7 and 5.8, 16384 26.2 and 12.0; 384 in groups
  // with a bias 7.9 and 12.8, 12.7 and 13.2, 37.7 and 34.2).
  if (q.E > kRouteRowExperts || (q.E > 128 && q.T <= kRouteWaveTokens)) {
    if (q.E <= 256) launch_scores<4, Lanes::kSwap>(q, s);
    else if (q.E <= 320) launch_scores<5, Lanes::kSwap>(q, s);
    else if (q.E <= 512) launch_wave_scores<8>(q, s);
    else launch_wave_scores<16>(q, s);
  } else {
    // (16384 tokens of 160 experts in two groups, k = 16: 10 a lane 10.9 us, 16 a lane
    // 16.0; 192 in groups with a bias: 12 a lane 12.4, 16 a lane 18.8)
    if (q.E <= 16) launch_scores<1, Lanes::kRow>(q, s);
    else if (q.E <= 32) launch_scores<2, Lanes::kRow>(q, s);
    else if (q.E <= 64) launch_scores<4, Lanes::kRow>(q, s);
    else if (q.E <= 128) launch_scores<8, Lanes::kRow>(q, s);
    else if (q.E <= 160) launch_scores<10, Lanes::kRow>(q, s);
    else if (q.E <= 192) launch_scores<12, Lanes::kRow>(q, s);
    else if (q.E <= 256) launch_scores<16, Lanes::kRow>(q, s);
    else if (q.E <= 320) launch_scores<20, Lanes::kRow>(q, s);
    else launch_scores<32, Lanes::kRow>(q, s);
  }
  return hipGetLastError();
}

}  // namespace nvfp4

// Router building blocks shared by the forward's prologues and the router with
// scores, groups and bias: candidate keys, reductions over a token's lanes, the
// per-lane sort and the selection rounds.
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace nvfp4 {

// ---------------------------------------------------------------------------
// Router reductions.  A candidate is the 64-bit key (order-preserving bits of
// the logit) << 32 | ~expert, so the larger key is the larger logit and, on
// equal logits, the smaller expert index.  -0.0 is keyed as +0.0: a binary32
// comparison finds the two equal, so their tie also goes to the smaller
// index.  Reductions over a 16-lane DPP row use quad permutes (xor 1, xor 2)
// and row rotates (4, 8), one instruction each.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t route_key(float v, int e) {
  const uint32_t u = __float_as_uint(v) == 0x80000000u ? 0u : __float_as_uint(v);
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return (static_cast<uint64_t>(o) << 32) | static_cast<uint32_t>(~e);
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ int key_expert(uint64_t k) { return static_cast<int>(~static_cast<uint32_t>(k)); }

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(v)));
}

// The largest key over a 16-lane DPP row, or over the wave, as two 32-bit
// maxima: of the high words (the ordered logits), then of the low words
// (~expert) of the lanes whose high word is that maximum.  The pair is the
// lexicographic, i.e. 64-bit, maximum; each DPP step is a single max with a
// DPP operand (the 64-bit form takes two moves, a compare and two selects).
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
  v = max(v, dpp_u32<kDppXor1>(v));
  v = max(v, dpp_u32<kDppXor2>(v));
  v = max(v, dpp_u32<kDppRor4>(v));
  v = max(v, dpp_u32<kDppRor8>(v));
  return v;
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = row16_max_u32(v);
  uint32_t a, b;
  lane_pair<16>(v, a, b);
  v = max(a, b);
  lane_pair<32>(v, a, b);
  return max(a, b);
}
template <bool WAVE>
__device__ __forceinline__ uint64_t key_max(uint64_t k) {
  const uint32_t h = static_cast<uint32_t>(k >> 32), l = static_cast<uint32_t>(k);
  const uint32_t mh = WAVE ? wave_max_u32(h) : row16_max_u32(h);
  const uint32_t tl = h == mh ? l : 0u;
  const uint32_t ml = WAVE ? wave_max_u32(tl) : row16_max_u32(tl);
  return (static_cast<uint64_t>(mh) << 32) | ml;
}
// (the association, and so the rounding, depends on the lane: a slot's weight
// is normalized by the sum its own lane forms)
__device__ __forceinline__ float row16_sum(float v) {
  v += dpp_f32<kDppXor1>(v);
  v += dpp_f32<kDppXor2>(v);
  v += dpp_f32<kDppRor4>(v);
  v += dpp_f32<kDppRor8>(v);
  return v;
}

// ---------------------------------------------------------------------------
// Router: the k largest logits of one token, ties to the smaller expert
// index, slots in descending order; weights = exp(l_j - l_0) normalized over
// the k slots (the softmax over all experts restricted to the chosen k).
// Keys order the logits as binary32 compares do (-0 as +0) and, on equal
// values, put the smaller expert first.
//
// Both routers below first sort each lane's keys (largest first) with
// Batcher's odd-even merge sorting network (K. E. Batcher, "Sorting networks
// and their applications", AFIPS 1968), so that each of the k selection
// rounds only takes the maximum of the lanes' heads and pops the winning
// lane's list.  Keys are unique (the expert index is part of them).  Slot j
// ends in lane j of the token's lanes, and its weight is normalized by the
// row-16 sum over the first 16 of them, so both routers give the same ids
// and the same weights.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void key_cx(uint64_t& a, uint64_t& b) {
  const bool sw = b > a;
  const uint64_t hi = sw ? b : a, lo = sw ? a : b;
  a = hi;
  b = lo;
}

template <int N>
__device__ __forceinline__ void sort_keys_desc(uint64_t (&c)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int d = p; d >= 1; d >>= 1)
#pragma unroll
      for (int j = d % p; j + d < N; j += 2 * d)
#pragma unroll
        for (int i = 0; i < d; ++i)
          if (i + j + d < N && (i + j) / (2 * p) == (i + j + d) / (2 * p)) key_cx(c[i + j], c[i + j + d]);
}

// The k selection rounds over the lanes' sorted lists (KMAX >= k rounds at
// most): each round takes the largest head over the 16-lane row (or the
// wave) and pops it from the lane that held it; lane j keeps round j's key.
// After round j at most KMAX - 1 - j more pops follow, so only that many
// leading entries of a list can still become its head and only those are
// shifted.
template <int N, int KMAX, bool WAVE>
__device__ __forceinline__ void select_rounds(uint64_t (&cand)[N], int k, int lane, uint64_t& mine,
                                              uint64_t& top) {
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    if (j < k) {
      const uint64_t best = key_max<WAVE>(cand[0]);
      if (j == 0) top = best;
      mine = lane == j ? best : mine;
      const bool pop = cand[0] == best;  // this lane held the winner
#pragma unroll
      for (int i = 0; i < N && i + 1 < KMAX - j; ++i) cand[i] = pop ? (i + 1 < N ? cand[i + 1] : 0ull) : cand[i];
    }
  }
}

}  // namespace nvfp4

// Attention of a batch's new tokens over the 8-bit key-value cache (gfx950).
//
//   x_j = scale log2(e) q . k_j,  m = max x_j,  p_j = 2^(x_j - m)
//   o = sum p_j v_j / sum p_j       over the keys j that the token sees
// in one pass over the keys: running maximum and sum in binary32, the output's sums
// rescaled when the maximum grows.
//
// Operands.  Both products run on v_mfma_f32_16x16x32_f16.  A code is exact in fp16;
// q is scaled by one power of two a tile (its largest value in [2^14, 2^15)), which
// is exact for fp16 and bf16 values within 2^29 of it.  The keys' scales multiply
// the scores.  The values' scales s multiply the probabilities: the weight
// p s 2^14 / u is rounded to fp16 (11 bits, the one rounding of this kernel that is
// not binary32), u the largest s so far, so that weights stay in [0, 2^14] and keep
// their 11 bits down to 2^-28 of the largest; the sums are kept in units of u 2^-14.
//
// The score product is formed transposed, keys x rows: a lane then has four
// consecutive keys of one row, which is the operand the output product (channels x
// rows) takes, with the values stored in that order of keys.  Probabilities never
// leave the registers, and a row's maximum and sum are over four lanes.
//
// Rows: the call's tokens times the query heads that share a kv head, row r = token
// r / G, head r % G.  A work item is a tile of rows of one entry and kv head over one
// piece of the keys; pieces are made where there are too few tiles for the chip and
// joined by a second kernel, in order.
#include <algorithm>
#include <climits>

#include "kernels.hpp"
#include "kv_cache.hpp"

namespace nvfp4 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kUnit = 0x1p14f;      // weights are up to this
constexpr float kLeastUnit = 0x1p-100f;  // and u at least this
constexpr float kNone = -__builtin_huge_valf();

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

struct AttnParams {
  KvParams c;
  const void* q;
  void* out;
  int64_t ldq, ldq_head, ldo, ldo_head;  // elements
  float scale;
  int group, window, bf16;
  // which entries: rows (tokens times group) in (rows_above, rows_most]
  int rows_above, rows_most;
  // keys are cut into pieces of at least least_steps steps, about `target` of all tiles
  // together (0: never cut)
  int target, least_steps;
  KvJoin* joins;      // of tiles in pieces, *join_count of them
  int* join_count;
  float* part;        // [slot][rows of a tile][D] sums, then
  float* part_ml;     // [slot][rows of a tile][2] maximum and sum
};

struct Work {
  KvEntry e;
  int entry, head, tile, tiles, pieces, piece, slot;
};

// Keys as steps of STEP tokens: those of full pages, then the tail's.  A step's tokens
// lie at keys first(s) ..; the last step of the full pages may reach behind them.
template <int STEP>
struct Steps {
  int full_keys, full_steps;
  __device__ Steps(int total, int shift) {
    full_keys = total >> shift << shift;
    full_steps = (full_keys + STEP - 1) / STEP;
  }
  __device__ int of(int key) const { return key < full_keys ? key / STEP : full_steps + (key - full_keys) / STEP; }
  __device__ int first(int s) const { return s < full_steps ? s * STEP : full_keys + (s - full_steps) * STEP; }
};

// The first and the last key that the rows [r, r + count) of an entry see.
__device__ __forceinline__ void seen(const AttnParams& a, const KvEntry& e, int r, int count, int& lo, int& hi) {
  lo = a.window ? max(0, e.len + r / a.group - a.window + 1) : 0;
  hi = e.len + (r + count - 1) / a.group;
}

// Steps of the widest tile of an entry (an upper bound).
template <int STEP, int BM>
__device__ __forceinline__ int entry_steps(const AttnParams& a, const KvEntry& e) {
  const Steps<STEP> st(e.total(), a.c.shift);
  const int all = st.of(e.total() - 1) + 1;
  return a.window ? min(all, (a.window + BM / a.group) / STEP + 4) : all;
}

// Which work item a block has (false: none).  Every block computes the same cut of
// the batch: the number of pieces of each entry, and from their sums where its own
// index falls.  The sums hold blocks, pieces of cut tiles and cut tiles, each without
// the factor of the kv heads, in 40, 12 and 12 bits: with target <= 1024 there are at
// most 2048 pieces of cut tiles.
template <int THREADS, int STEP, int BM>
__device__ __forceinline__ bool find_work(const AttnParams& a, Work& w) {
  __shared__ uint64_t buf[2][THREADS / kWave];
  __shared__ int found[4];
  const KvParams& p = a.c;
  const int per = (p.entries + THREADS - 1) / THREADS;
  const int i0 = threadIdx.x * per, i1 = min(i0 + per, p.entries);
  auto tiles_of = [&](const KvEntry& e) {
    const int64_t rows = int64_t{e.n} * a.group;
    return rows > a.rows_above && rows <= a.rows_most ? static_cast<int>((rows + BM - 1) / BM) : 0;
  };
  uint64_t own = 0, total;
  if (a.target) {
    for (int i = i0; i < i1; ++i) {
      const KvEntry e = kv_entry(p, i);
      const int t = tiles_of(e);
      if (t) own += static_cast<uint64_t>(t) * entry_steps<STEP, BM>(a, e);
    }
  }
  int piece_steps = INT_MAX;
  if (a.target) {
    block_scan<THREADS>(own, buf[0], total);
    const uint64_t n = (total * p.heads + a.target - 1) / a.target;
    piece_steps = uniform(static_cast<int>(min(max(n, static_cast<uint64_t>(a.least_steps)), uint64_t{INT_MAX / 2})));
  }
  auto count_of = [&](const KvEntry& e, int tiles) -> uint64_t {
    if (!tiles) return 0;
    const int pieces = a.target ? (entry_steps<STEP, BM>(a, e) + piece_steps - 1) / piece_steps : 1;
    const uint64_t blocks = static_cast<uint64_t>(tiles) * pieces;
    return blocks << 24 | (pieces > 1 ? blocks << 12 | static_cast<uint64_t>(tiles) : 0);
  };
  own = 0;
  for (int i = i0; i < i1; ++i) {
    const KvEntry e = kv_entry(p, i);
    own += count_of(e, tiles_of(e));
  }
  if (threadIdx.x == 0) found[0] = -1;
  uint64_t at = block_scan<THREADS>(own, buf[1], total) - own;
  // (entries that share tokens can need more blocks than there are: such a call does nothing)
  const bool fits = (total >> 24) * p.heads <= gridDim.x;
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.target)
    *a.join_count = fits ? static_cast<int>(total & 4095) * p.heads : 0;
  if (!fits) return false;
  const uint64_t want = blockIdx.x / p.heads;
  if (want >= at >> 24 && want < (at + own) >> 24) {
    for (int i = i0; i < i1; ++i) {
      const KvEntry e = kv_entry(p, i);
      const uint64_t c = count_of(e, tiles_of(e));
      if (want < (at + c) >> 24) {
        found[0] = i;
        found[1] = static_cast<int>(want - (at >> 24));
        found[2] = static_cast<int>(at >> 12 & 4095);
        found[3] = static_cast<int>(at & 4095);
        break;
      }
      at += c;
    }
  }
  __syncthreads();
  w.entry = uniform(found[0]);
  if (w.entry < 0) return false;
  const int index = uniform(found[1]);
  w.e = kv_entry(p, w.entry);
  w.head = blockIdx.x % p.heads;
  w.tiles = tiles_of(w.e);
  w.pieces = a.target ? (entry_steps<STEP, BM>(a, w.e) + piece_steps - 1) / piece_steps : 1;
  // the last rows see the most keys: their tiles first
  w.tile = w.tiles - 1 - index / w.pieces;
  w.piece = index % w.pieces;
  w.slot = (uniform(found[2]) + index) * p.heads + w.head;
  if (w.pieces > 1 && w.piece == 0 && threadIdx.x == 0) {
    const int r0 = w.tile * BM;
    KvJoin j;
    j.first = w.e.first;
    j.row = r0;
    j.rows = min(BM, w.e.n * a.group - r0);
    j.head = w.head;
    j.slot = w.slot;
    j.pieces = w.pieces;
    j.stride = p.heads;
    a.joins[(found[3] + index / w.pieces) * p.heads + w.head] = j;
  }
  return true;
}

// The steps of a work item: its piece of those that its rows see.
template <int STEP>
__device__ __forceinline__ void piece_steps(const Steps<STEP>& st, const Work& w, int lo, int hi, int& s0, int& s1) {
  const int a = st.of(lo), n = st.of(hi) + 1 - a;
  const int per = (n + w.pieces - 1) / w.pieces;
  s0 = a + min(n, w.piece * per);
  s1 = a + min(n, w.piece * per + per);
}

template <bool MAX>
__device__ __forceinline__ float over_groups(float v) {  // over the four lanes of a row
  uint32_t x, y;
  lane_pair<16>(__float_as_uint(v), x, y);
  v = MAX ? fmaxf(__uint_as_float(x), __uint_as_float(y)) : __uint_as_float(x) + __uint_as_float(y);
  lane_pair<32>(__float_as_uint(v), x, y);
  return MAX ? fmaxf(__uint_as_float(x), __uint_as_float(y)) : __uint_as_float(x) + __uint_as_float(y);
}

// A wave's 16 MR rows: operands, running maximum, sum (of the lane's own keys) and
// output sums (channels 16 f + 4 (lane / 16) + i of row lane % 16).
template <int D, int MR>
struct Rows {
  half8 q[MR][D / 32];
  float m[MR], l[MR];
  f32x4 o[MR][D / 16];
  float u, inv;      // unit, kUnit / u
  float c;           // scale log2(e) over q's power of two
  int lo[MR], hi[MR];  // keys that the lane's row sees: lo <= key < hi
  int all_lo, all_hi;  // keys that every row sees

  // Rows [r0, r0 + 16 MR) of the entry, of which `rows` exist.
  __device__ __forceinline__ void load(const AttnParams& a, const KvEntry& e, int head, int r0, int rows) {
    const int lane = threadIdx.x & (kWave - 1);
    u32x4 raw[MR][D / 32];
#pragma unroll
    for (int r = 0; r < MR; ++r) {
      const int row = r0 + 16 * r + lane % 16, token = row / a.group;
      const int64_t at = (e.first + token) * a.ldq + (head * a.group + row % a.group) * a.ldq_head;
      const char* p = static_cast<const char*>(a.q) + (at + 16 * (lane / 16)) * 2;
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
        raw[r][k] = row < rows ? *reinterpret_cast<const u32x4*>(p + (64 * (k / 2) + 8 * (k % 2)) * 2) : u32x4{};
      hi[r] = e.len + min(token, (rows - 1) / a.group) + 1;
      lo[r] = a.window ? max(0, hi[r] - a.window) : 0;
      m[r] = kNone;
      l[r] = 0.0f;
#pragma unroll
      for (int f = 0; f < D / 16; ++f) o[r][f] = f32x4{};
    }
    const int last = min(r0 + 16 * MR, rows) - 1;
    all_hi = e.len + r0 / a.group + 1;
    all_lo = a.window ? max(0, e.len + last / a.group + 1 - a.window) : 0;
    u = kLeastUnit;
    inv = kUnit / kLeastUnit;
    // the largest finite magnitude of the tile, as bits
    uint32_t top = 0;
    auto widen = [&](uint32_t w, float& x, float& y) {
      if (a.bf16) Bf16::unpack(w, x, y);
      else F16::unpack(w, x, y);
    };
#pragma unroll
    for (int r = 0; r < MR; ++r)
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x, y;
          widen(raw[r][k][i], x, y);
          const uint32_t bx = __float_as_uint(x) & 0x7fffffffu, by = __float_as_uint(y) & 0x7fffffffu;
          top = max(top, max(bx < 0x7f800000u ? bx : 0u, by < 0x7f800000u ? by : 0u));
        }
    top = __float_as_uint(wave_max(__uint_as_float(top)));
    const int exp = max(static_cast<int>(top >> 23) - 127 - 14, -126);
    const float mul = __uint_as_float(static_cast<uint32_t>(127 - exp) << 23);
    c = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + exp) << 23);
#pragma unroll
    for (int r = 0; r < MR; ++r)
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x, y;
          widen(raw[r][k][i], x, y);
          q[r][k][2 * i] = static_cast<_Float16>(x * mul);
          q[r][k][2 * i + 1] = static_cast<_Float16>(y * mul);
        }
  }

  // One step: 16 NB keys from key0 on.  key(b, k): a key operand, value(t, f): a value
  // operand of 32 keys, ks / vs[b][i]: scales (of a block's four keys of this lane, or
  // one for the block); ok[b]: whether the block's page is one.  masked: not every
  // row sees every key.
  template <int NB, int SC, typename Key, typename Value>
  __device__ __forceinline__ void step(int key0, bool masked, const float (&ks)[NB][SC], const float (&vs)[NB][SC],
                                       const bool (&ok)[NB], Key key, Value value) {
    const int g4 = (threadIdx.x & (kWave - 1)) / 16 * 4;
    f32x4 s[MR][NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int r = 0; r < MR; ++r) s[r][b] = f32x4{};
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const half8 x = key(b, k);
#pragma unroll
        for (int r = 0; r < MR; ++r) s[r][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, q[r][k], s[r][b], 0, 0, 0);
      }
    }
    // a larger unit
    float top = u;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < SC; ++i) top = fmaxf(top, vs[b][i]);
    if (__ballot(top > u)) {
      top = over_groups<true>(top);
      const float down = u / top;
      u = top;
      inv = kUnit / top;
#pragma unroll
      for (int r = 0; r < MR; ++r)
#pragma unroll
        for (int f = 0; f < D / 16; ++f) o[r][f] *= down;
    }
    half8 w[MR][NB / 2];
#pragma unroll
    for (int r = 0; r < MR; ++r) {
      float top_x = kNone;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = s[r][b][i] * (ks[b][SC == 1 ? 0 : i] * c);
          if (masked) {
            const int at = key0 + 16 * b + g4 + i;
            x = ok[b] && at >= lo[r] && at < hi[r] ? x : kNone;
          }
          s[r][b][i] = x;
          top_x = fmaxf(top_x, x);
        }
      if (__ballot(top_x > m[r])) {
        const float now = fmaxf(m[r], over_groups<true>(top_x));
        const float down = __builtin_amdgcn_exp2f(m[r] - (now == kNone ? 0.0f : now));
        m[r] = now;
        l[r] *= down;
#pragma unroll
        for (int f = 0; f < D / 16; ++f) o[r][f] *= down;
      }
      const float base = m[r] == kNone ? 0.0f : m[r];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = __builtin_amdgcn_exp2f(s[r][b][i] - base);
          l[r] += e;
          float v = e * (vs[b][SC == 1 ? 0 : i] * inv);
          if (masked) v = s[r][b][i] == kNone ? 0.0f : v;  // (a scale that is NaN stays out of sight)
          w[r][b / 2][b % 2 * 4 + i] = static_cast<_Float16>(v);
        }
    }
#pragma unroll
    for (int t = 0; t < NB / 2; ++t)
#pragma unroll
      for (int f = 0; f < D / 16; ++f) {
        const half8 x = value(t, f);
#pragma unroll
        for (int r = 0; r < MR; ++r) o[r][f] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, w[r][t], o[r][f], 0, 0, 0);
      }
  }

  // Sums over a row's lanes, outputs in their own unit.
  __device__ __forceinline__ void finish() {
    const float unit = u / kUnit;
#pragma unroll
    for (int r = 0; r < MR; ++r) {
      l[r] = over_groups<false>(l[r]);
#pragma unroll
      for (int f = 0; f < D / 16; ++f) o[r][f] *= unit;
    }
  }
};

// Where row r of an entry writes its output.
__device__ __forceinline__ int64_t out_at(const AttnParams& a, int first, int head, int row) {
  return (first + row / a.group) * a.ldo + (head * a.group + row % a.group) * a.ldo_head;
}

__device__ __forceinline__ void put8(const AttnParams& a, int64_t at, const float (&v)[8]) {
  if (a.bf16) store8<Bf16>(a.out, at, v);
  else store8<F16>(a.out, at, v);
}

// Few rows: the kernel reads the cache once and is bound by that.  Each of a block's
// waves takes every fourth step of the piece, its codes straight to registers, the
// next step's loads in flight while one is computed; the four results meet in LDS.
constexpr int kStreamWaves = 4, kStreamThreads = kStreamWaves * kWave;
template <int D, int MR>
constexpr int stream_blocks_of_step = D * MR <= 128 ? 4 : 2;

template <int D, int MR>
__global__ __launch_bounds__(kStreamThreads, D * MR >= 256 ? 1 : 2) void kv_stream_kernel(AttnParams a) {
  constexpr int NB = stream_blocks_of_step<D, MR>, STEP = 16 * NB, NU = D / 64, BM = 16 * MR;
  constexpr int kBatch = kWave / NB;  // steps whose pages a wave looks up together
  extern __shared__ __align__(16) float lds[];
  const KvParams& p = a.c;
  Work w;
  if (!find_work<kStreamThreads, STEP, BM>(a, w)) return;
  const KvEntry& e = w.e;
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
  const int r0 = w.tile * BM, rows = e.n * a.group;
  int lo, hi, s0, s1;
  seen(a, e, r0, min(BM, rows - r0), lo, hi);
  const Steps<STEP> st(e.total(), p.shift);
  piece_steps<STEP>(st, w, lo, hi, s0, s1);

  Rows<D, MR> t;
  t.load(a, e, w.head, r0, rows);

  struct Codes {
    u32x4 k[NB][NU], v[NB][NU];
  };
  const int64_t page_bytes = int64_t{p.P} * p.D;
  const int mine = wave < s1 - s0 ? (s1 - s0 - wave + kStreamWaves - 1) / kStreamWaves : 0;  // steps of this wave
  const int of_codes = max(0, min(mine, (min(s1, st.full_steps) - s0 - wave + kStreamWaves - 1) / kStreamWaves));
  for (int b0 = 0; b0 < of_codes; b0 += kBatch) {
    // lane NB j + b: block b of this wave's step b0 + j
    const int key = (s0 + wave + (b0 + lane / NB) * kStreamWaves) * STEP + 16 * (lane % NB);
    int id = -1;
    if (b0 + lane / NB < of_codes && key < st.full_keys) id = kv_page(p, w.entry, key >> p.shift);
    float ks_lane = 0.0f, vs_lane = 0.0f;
    if (id >= 0) {
      ks_lane = p.scales[kv_page_at(p, id, 0, w.head)];
      vs_lane = p.scales[kv_page_at(p, id, 1, w.head)];
    }
    auto fetch = [&](Codes& x, int j) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int page = max(__builtin_amdgcn_readlane(id, j * NB + b), 0);
        const int in_page = ((s0 + wave + (b0 + j) * kStreamWaves) * STEP + 16 * b) & (p.P - 1);
        const uint8_t* k = p.codes + kv_page_at(p, page, 0, w.head) * page_bytes + in_page * D;
        const uint8_t* v = k + p.heads * page_bytes;
#pragma unroll
        for (int c = 0; c < NU; ++c) {
          x.k[b][c] = *reinterpret_cast<const u32x4*>(k + c * 1024 + lane * 16);
          x.v[b][c] = *reinterpret_cast<const u32x4*>(v + c * 1024 + lane * 16);
        }
      }
    };
    auto compute = [&](const Codes& x, int j) {
      float ks[NB][1], vs[NB][1];
      bool ok[NB], all = true;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        ok[b] = __builtin_amdgcn_readlane(id, j * NB + b) >= 0;
        all = all && ok[b];
        ks[b][0] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ks_lane), j * NB + b));
        vs[b][0] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(vs_lane), j * NB + b));
      }
      const int key0 = (s0 + wave + (b0 + j) * kStreamWaves) * STEP;
      const bool masked = !all || key0 < t.all_lo || key0 + STEP > t.all_hi;
      t.template step<NB, 1>(
          key0, masked, ks, vs, ok,
          [&](int b, int k) { return kv_codes8(x.k[b][k / 2][k % 2 * 2], x.k[b][k / 2][k % 2 * 2 + 1]); },
          [&](int h, int f) { return kv_codes8(x.v[2 * h][f / 4][f % 4], x.v[2 * h + 1][f / 4][f % 4]); });
    };
    const int n = min(kBatch, of_codes - b0);
    Codes x, y;
    fetch(x, 0);
    int j = 0;
    for (; j + 2 <= n; j += 2) {
      fetch(y, j + 1);
      compute(x, j);
      if (j + 2 < n) fetch(x, j + 2);
      compute(y, j + 1);
    }
    if (j < n) compute(x, j);
  }

  // the tail's steps
  for (int i = of_codes; i < mine; ++i) {
    const int s = s0 + wave + i * kStreamWaves, key0 = st.first(s), in_tail = key0 - st.full_keys;
    const int64_t at = kv_page_at(p, e.slot, 0, w.head);
    const char* k = reinterpret_cast<const char*>(p.tails + at * page_bytes);
    const char* v = reinterpret_cast<const char*>(p.tails + (at + p.heads) * page_bytes);
    float ks[NB][4], vs[NB][4];
    bool ok[NB];
    int unit[NB];  // (a block behind the page is out of sight; its operands are the page's first)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      ok[b] = in_tail + 16 * b < p.P;
      const int block = ok[b] ? in_tail / 16 + b : 0;
      unit[b] = block * NU;
      const f32x4 x = *reinterpret_cast<const f32x4*>(p.tail_scales + at * p.P + block * 16 + lane / 16 * 4);
      const f32x4 y = *reinterpret_cast<const f32x4*>(p.tail_scales + (at + p.heads) * p.P + block * 16 + lane / 16 * 4);
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4) {
        const bool in = ok[b] && key0 + 16 * b + lane / 16 * 4 + i4 < e.total();
        ks[b][i4] = in ? x[i4] : 0.0f;
        vs[b][i4] = in ? y[i4] : 0.0f;
      }
    }
    t.template step<NB, 4>(
        key0, true, ks, vs, ok,
        [&](int b, int c) { return *reinterpret_cast<const half8*>(k + (unit[b] * 2 + c) * 1024 + lane * 16); },
        [&](int h, int f) {
          typedef _Float16 half4 __attribute__((ext_vector_type(4)));
          const int in = f / 4 * 2048 + f % 4 / 2 * 1024 + lane * 16 + f % 2 * 8;
          const half4 x = *reinterpret_cast<const half4*>(v + unit[2 * h] * 2048 + in);
          const half4 y = *reinterpret_cast<const half4*>(v + unit[2 * h + 1] * 2048 + in);
          return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        });
  }
  t.finish();

  // the waves' results of a row together, in their order
  constexpr int LD = D + 4;  // (a row starts four banks behind the one before)
  float* sums = lds;
  float* ml = lds + kStreamWaves * 16 * LD;
#pragma unroll
  for (int r = 0; r < MR; ++r) {
    if (r) __syncthreads();
#pragma unroll
    for (int f = 0; f < D / 16; ++f)
      *reinterpret_cast<f32x4*>(sums + (wave * 16 + lane % 16) * LD + 16 * f + lane / 16 * 4) = t.o[r][f];
    if (lane < 16) {
      ml[(wave * 16 + lane) * 2] = t.m[r];
      ml[(wave * 16 + lane) * 2 + 1] = t.l[r];
    }
    __syncthreads();
    for (int item = threadIdx.x; item < 16 * D / 8; item += kStreamThreads) {
      const int row = item / (D / 8), d = item % (D / 8) * 8, at_row = r0 + 16 * r + row;
      if (at_row >= rows) continue;
      float m = kNone, l = 0.0f, f[kStreamWaves], v[8] = {};
#pragma unroll
      for (int i = 0; i < kStreamWaves; ++i) m = fmaxf(m, ml[(i * 16 + row) * 2]);
#pragma unroll
      for (int i = 0; i < kStreamWaves; ++i) {
        f[i] = __builtin_amdgcn_exp2f(ml[(i * 16 + row) * 2] - (m == kNone ? 0.0f : m));
        l += f[i] * ml[(i * 16 + row) * 2 + 1];
      }
#pragma unroll
      for (int i = 0; i < kStreamWaves; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += f[i] * sums[(i * 16 + row) * LD + d + j];
      if (w.pieces == 1) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= inv;
        put8(a, out_at(a, e.first, w.head, at_row) + d, v);
      } else {
        const int64_t at = int64_t{w.slot} * BM + 16 * r + row;
        store8<F32>(a.part, at * D + d, v);
        if (d == 0) {
          a.part_ml[at * 2] = m;
          a.part_ml[at * 2 + 1] = l;
        }
      }
    }
  }
}

// Many rows: eight waves of 16 MR rows each share every step's keys and values, which
// are made fp16 once, on their way into LDS.
constexpr int kTileWaves = 8, kTileThreads = kTileWaves * kWave;
template <int D>
constexpr int tile_frags = D <= 128 ? 2 : 1;

template <int D>
struct TileLds {
  half8 k[4][D / 32][kWave];   // [block of 16 keys][32 channels][lane]
  half8 v[2][D / 16][kWave];   // [32 keys][16 channels][lane]
  float ks[64], vs[64];
  int bad[4];
};

template <int D>
__global__ __launch_bounds__(kTileThreads, 2) void kv_tile_kernel(AttnParams a) {
  constexpr int MR = tile_frags<D>, BM = 16 * MR * kTileWaves, STEP = 64, NB = 4, NU = D / 64;
  typedef _Float16 half4 __attribute__((ext_vector_type(4)));
  extern __shared__ __align__(16) char raw_lds[];
  TileLds<D>* lds = reinterpret_cast<TileLds<D>*>(raw_lds);
  const KvParams& p = a.c;
  Work w;
  if (!find_work<kTileThreads, STEP, BM>(a, w)) return;
  const KvEntry& e = w.e;
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
  const int t0 = w.tile * BM, rows = e.n * a.group, r0 = t0 + wave * 16 * MR;
  int lo, hi, s0, s1;
  seen(a, e, t0, min(BM, rows - t0), lo, hi);
  const Steps<STEP> st(e.total(), p.shift);
  piece_steps<STEP>(st, w, lo, hi, s0, s1);
  const bool some = r0 < rows;  // this wave has rows
  int wave_lo = 0, wave_hi = -1;
  if (some) seen(a, e, r0, min(16 * MR, rows - r0), wave_lo, wave_hi);

  Rows<D, MR> t;
  t.load(a, e, w.head, r0, rows);

  // Staging: this wave brings block `block` of 16 keys (waves 0 to 3: keys, 4 to 7:
  // values) of a step into LDS; its scales come with it.
  const int block = wave % 4, which = wave / 4;
  const int64_t page_bytes = int64_t{p.P} * p.D;
  auto page_of = [&](int s) {  // the page of this wave's block in step s, -1 outside the full pages
    const int key = st.first(s) + 16 * block;
    return s < min(s1, st.full_steps) && key < st.full_keys ? kv_page(p, w.entry, key >> p.shift) : -1;
  };
  u32x4 st_raw[2 * NU];
  float st_scale = 0.0f;
  bool st_ok = false;
  auto fetch = [&](int s, int page) {
    const int key0 = st.first(s) + 16 * block;
    if (s < st.full_steps) {
      const int64_t at = kv_page_at(p, max(page, 0), which, w.head);
      const uint8_t* src = p.codes + at * page_bytes + (key0 & (p.P - 1)) * D + lane * 16;
#pragma unroll
      for (int c = 0; c < NU; ++c) st_raw[c] = *reinterpret_cast<const u32x4*>(src + c * 1024);
      st_scale = p.scales[at];
      st_ok = page >= 0;
    } else {
      const int64_t at = kv_page_at(p, e.slot, which, w.head);
      st_ok = key0 - st.full_keys < p.P;
      const int in_tail = st_ok ? key0 - st.full_keys : 0;
      const char* src = reinterpret_cast<const char*>(p.tails + at * page_bytes + in_tail * D) + lane * 16;
#pragma unroll
      for (int c = 0; c < 2 * NU; ++c) st_raw[c] = *reinterpret_cast<const u32x4*>(src + c * 1024);
      st_scale = p.tail_scales[at * p.P + in_tail + lane % 16];
      if (key0 + lane % 16 >= e.total()) st_scale = 0.0f;
    }
  };
  auto stage = [&](int s, TileLds<D>& to) {
    if (which == 0) {
#pragma unroll
      for (int c = 0; c < NU; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          to.k[block][2 * c + h][lane] = s < st.full_steps ? kv_codes8(st_raw[c][2 * h], st_raw[c][2 * h + 1])
                                                           : __builtin_bit_cast(half8, st_raw[2 * c + h]);
    } else {
#pragma unroll
      for (int c = 0; c < NU; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const half8 x = s < st.full_steps ? kv_codes8(st_raw[c][2 * h], st_raw[c][2 * h + 1])
                                            : __builtin_bit_cast(half8, st_raw[2 * c + h]);
#pragma unroll
          for (int f = 0; f < 2; ++f)
            reinterpret_cast<half4*>(&to.v[block / 2][4 * c + 2 * h + f][lane])[block % 2] =
                f ? __builtin_shufflevector(x, x, 4, 5, 6, 7) : __builtin_shufflevector(x, x, 0, 1, 2, 3);
        }
    }
    if (lane < 16) (which ? to.vs : to.ks)[16 * block + lane] = st_ok ? st_scale : 0.0f;
    if (which == 0 && lane == 0) to.bad[block] = !st_ok;
  };

  int page = page_of(s0);
  if (s0 < s1) {
    fetch(s0, page);
    page = page_of(s0 + 1);
    stage(s0, lds[0]);
  }
  __syncthreads();
  for (int s = s0; s < s1; ++s) {
    TileLds<D>& now = lds[(s - s0) & 1];
    const bool more = s + 1 < s1;
    if (more) {
      fetch(s + 1, page);
      page = page_of(s + 2);
    }
    const int key0 = st.first(s);
    if (some && key0 <= wave_hi && key0 + STEP > wave_lo) {
      float ks[NB][4], vs[NB][4];
      bool ok[NB], all = true;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(now.ks + 16 * b + lane / 16 * 4);
        const f32x4 y = *reinterpret_cast<const f32x4*>(now.vs + 16 * b + lane / 16 * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ks[b][i] = x[i];
          vs[b][i] = y[i];
        }
        ok[b] = !now.bad[b];
        all = all && ok[b];
      }
      const bool masked = !all || key0 < t.all_lo || key0 + STEP > t.all_hi;
      auto key = [&](int b, int k) { return now.k[b][k][lane]; };
      auto value = [&](int h, int f) { return now.v[h][f][lane]; };
      t.template step<NB, 4>(key0, masked, ks, vs, ok, key, value);
    }
    if (more) stage(s + 1, lds[(s + 1 - s0) & 1]);
    __syncthreads();
  }
  t.finish();
  if (!some) return;
#pragma unroll
  for (int r = 0; r < MR; ++r) {
    const int row = r0 + 16 * r + lane % 16;
    if (row >= rows) continue;
    if (w.pieces == 1) {
      const float inv = t.l[r] == 0.0f ? 0.0f : 1.0f / t.l[r];
      const int64_t at = out_at(a, e.first, w.head, row) + lane / 16 * 4;
#pragma unroll
      for (int f = 0; f < D / 16; ++f) {
        const float v[4] = {t.o[r][f][0] * inv, t.o[r][f][1] * inv, t.o[r][f][2] * inv, t.o[r][f][3] * inv};
        if (a.bf16) store4_any<Bf16>(a.out, at + 16 * f, v);
        else store4_any<F16>(a.out, at + 16 * f, v);
      }
    } else {
      const int64_t at = int64_t{w.slot} * BM + row - t0;
#pragma unroll
      for (int f = 0; f < D / 16; ++f)
        *reinterpret_cast<f32x4*>(a.part + at * D + 16 * f + lane / 16 * 4) = t.o[r][f];
      if (lane < 16) {
        a.part_ml[at * 2] = t.m[r];
        a.part_ml[at * 2 + 1] = t.l[r];
      }
    }
  }
}

// Pieces of a row joined in their order.  A block takes every gridDim.y-th row of a cut
// tile: a thread four channels of every LANES-th piece.
constexpr int kJoinThreads = 256;

template <int D>
__global__ __launch_bounds__(kJoinThreads) void kv_join_kernel(AttnParams a, int bm) {
  constexpr int CH = D / 4, GROUPS = kJoinThreads / CH;
  __shared__ float top[kJoinThreads / kWave], sum[GROUPS][D + 4], sum_l[GROUPS];
  if (static_cast<int>(blockIdx.x) >= *a.join_count) return;
  const KvJoin j = a.joins[blockIdx.x];
  const int ch = threadIdx.x % CH, group = threadIdx.x / CH;
  for (int row = blockIdx.y; row < j.rows; row += gridDim.y) {
    auto at = [&](int piece) { return (int64_t{j.slot} + int64_t{piece} * j.stride) * bm + row; };
    float m = kNone;
    for (int i = threadIdx.x; i < j.pieces; i += kJoinThreads) m = fmaxf(m, a.part_ml[at(i) * 2]);
    m = wave_max(m);
    __syncthreads();
    if (threadIdx.x % kWave == 0) top[threadIdx.x / kWave] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoinThreads / kWave; ++i) m = fmaxf(m, top[i]);
    const float base = m == kNone ? 0.0f : m;
    f32x4 v{};
    float l = 0.0f;
    if (group < GROUPS) {
      for (int i = group; i < j.pieces; i += GROUPS) {
        const float f = __builtin_amdgcn_exp2f(a.part_ml[at(i) * 2] - base);
        l += f * a.part_ml[at(i) * 2 + 1];
        v += f * *reinterpret_cast<const f32x4*>(a.part + at(i) * D + 4 * ch);
      }
      *reinterpret_cast<f32x4*>(&sum[group][4 * ch]) = v;
      if (ch == 0) sum_l[group] = l;
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int i = 1; i < GROUPS; ++i) {
        v += *reinterpret_cast<const f32x4*>(&sum[i][4 * ch]);
        l += sum_l[i];
      }
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const float out[4] = {v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
      const int64_t to = out_at(a, j.first, j.head, j.row + row) + 4 * ch;
      if (a.bf16) store4_any<Bf16>(a.out, to, out);
      else store4_any<F16>(a.out, to, out);
    }
  }
}

// --- host ------------------------------------------------------------------------

// How a call is run.  An entry of more rows than a stream tile has goes to the tile
// kernel; the host knows rows only where every entry has one token or there is one
// entry, else both kernels run, each on its entries.
struct Cut {
  bool use;
  int bm, target, least_steps, rows_above, rows_most;
  int64_t tiles, slots, joins;  // upper bounds, kv heads included
  int64_t blocks() const { return target + tiles; }
};
struct Plan {
  Cut stream, tile;
  int mr;
};

// Keys below which a sequence stays in one piece and no join is launched.
constexpr int64_t kWholeKeys = 1024;

Cut make_cut(const KvParams& p, int group, int bm, int step, int target, int least_steps) {
  Cut c{};
  c.use = true;
  c.bm = bm;
  c.rows_most = INT_MAX;
  const int64_t rows = int64_t{p.tokens} * group;
  c.tiles = (p.cu ? rows / bm + std::min(p.entries, p.tokens) : int64_t{p.entries} * ((group + bm - 1) / bm)) * p.heads;
  const int64_t keys = int64_t{p.width} << p.shift, steps = keys / step + 2;
  if (keys <= kWholeKeys || (p.entries == 1 && rows / bm * p.heads >= target)) return c;
  c.target = target;
  c.least_steps = least_steps;
  c.slots = std::min(int64_t{2} * target, c.tiles * ((steps + least_steps - 1) / least_steps));
  c.joins = std::min(int64_t{target}, c.tiles);
  return c;
}

template <int D>
Plan make_plan(const KvParams& p, int group) {
  Plan x{};
  x.mr = group > 16 || (p.cu && p.tokens > p.entries) ? 2 : 1;
  const int most = 32, rows = static_cast<int>(std::min(int64_t{p.tokens} * group, int64_t{INT_MAX}));
  const bool stream = !p.cu || rows <= most, tile = !stream && p.entries == 1;
  if (!tile) x.stream = make_cut(p, group, 16 * x.mr, 16 * (x.mr == 1 ? stream_blocks_of_step<D, 1> : stream_blocks_of_step<D, 2>), 1024, 8);
  if (!stream) x.tile = make_cut(p, group, 16 * tile_frags<D> * kTileWaves, 64, 256, 8);
  if (!tile && !stream) x.stream.rows_most = x.tile.rows_above = most;
  return x;
}

struct Area {
  int64_t count, joins, part, ml, end;
};
Area area(const Cut& c, int D, int64_t at) {
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  Area a{};
  a.count = at;
  a.end = at;
  if (!c.use || !c.target) return a;
  a.joins = up(a.count + 4);
  a.part = up(a.joins + c.joins * static_cast<int64_t>(sizeof(KvJoin)));
  a.ml = up(a.part + c.slots * c.bm * D * 4);
  a.end = up(a.ml + c.slots * c.bm * 8);
  return a;
}

AttnParams with(const KvAttention& k, const Cut& c, const Area& at, char* ws) {
  AttnParams a{};
  a.c = k.c;
  a.q = k.q;
  a.out = k.out;
  a.ldq = k.ldq;
  a.ldq_head = k.ldq_head;
  a.ldo = k.ldo;
  a.ldo_head = k.ldo_head;
  a.scale = k.scale;
  a.group = k.group;
  a.window = k.window;
  a.bf16 = k.dtype == MOE_BF16;
  a.rows_above = c.rows_above;
  a.rows_most = c.rows_most;
  a.target = c.target;
  a.least_steps = c.least_steps;
  if (c.target) {
    a.join_count = reinterpret_cast<int*>(ws + at.count);
    a.joins = reinterpret_cast<KvJoin*>(ws + at.joins);
    a.part = reinterpret_cast<float*>(ws + at.part);
    a.part_ml = reinterpret_cast<float*>(ws + at.ml);
  }
  return a;
}

template <typename K>
hipError_t allow_lds(K kernel, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int D>
hipError_t join(const AttnParams& a, const Cut& c, hipStream_t s) {
  if (!c.target) return hipSuccess;
  const int64_t rows = std::max<int64_t>(1, std::min<int64_t>(c.bm, 2048 / c.joins));
  kv_join_kernel<D><<<dim3(c.joins, rows), kJoinThreads, 0, s>>>(a, c.bm);
  return hipGetLastError();
}

template <int D, int MR>
hipError_t run_stream(const AttnParams& a, const Cut& c, hipStream_t s) {
  constexpr int kLds = (kStreamWaves * 16 * (D + 4) + kStreamWaves * 16 * 2) * 4;
  static const hipError_t allowed = allow_lds(kv_stream_kernel<D, MR>, kLds);
  if (allowed != hipSuccess) return allowed;
  kv_stream_kernel<D, MR><<<c.blocks(), kStreamThreads, kLds, s>>>(a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : join<D>(a, c, s);
}

template <int D>
hipError_t run(const KvAttention& k, char* ws, hipStream_t s) {
  const Plan x = make_plan<D>(k.c, k.group);
  const Area sa = area(x.stream, D, 0), ta = area(x.tile, D, sa.end);
  if (x.tile.use) {
    constexpr int kLds = 2 * sizeof(TileLds<D>);
    static const hipError_t allowed = allow_lds(kv_tile_kernel<D>, kLds);
    if (allowed != hipSuccess) return allowed;
    const AttnParams a = with(k, x.tile, ta, ws);
    kv_tile_kernel<D><<<x.tile.blocks(), kTileThreads, kLds, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess) e = join<D>(a, x.tile, s);
    if (e != hipSuccess) return e;
  }
  if (!x.stream.use) return hipSuccess;
  const AttnParams a = with(k, x.stream, sa, ws);
  return x.mr == 1 ? run_stream<D, 1>(a, x.stream, s) : run_stream<D, 2>(a, x.stream, s);
}

template <int D>
int64_t bytes(const KvParams& p, int group, int64_t* blocks) {
  const Plan x = make_plan<D>(p, group);
  *blocks = std::max(x.stream.use ? x.stream.blocks() : 0, x.tile.use ? x.tile.blocks() : 0);
  return area(x.tile, D, area(x.stream, D, 0).end).end;
}

}  // namespace

int64_t kv_attention_bytes(const KvParams& p, int group, int64_t* blocks) {
  return p.D == 64    ? bytes<64>(p, group, blocks)
         : p.D == 128 ? bytes<128>(p, group, blocks)
         : p.D == 192 ? bytes<192>(p, group, blocks)
                      : bytes<256>(p, group, blocks);
}

hipError_t launch_kv_attention(const KvAttention& k, void* workspace, hipStream_t s) {
  char* ws = static_cast<char*>(workspace);
  return k.c.D == 64 ? run<64>(k, ws, s) : k.c.D == 128 ? run<128>(k, ws, s) : k.c.D == 192 ? run<192>(k, ws, s) : run<256>(k, ws, s);
}

}  // namespace nvfp4

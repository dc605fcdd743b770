// Attention of a batch's new tokens over the 8-bit key-value cache (gfx950).
//
//   x_j = scale log2(e) q . k_j,  m = max x_j,  p_j = 2^(x_j - m)
//   o = sum p_j v_j / sum p_j       over the keys j that the token sees
// in one pass over the keys: running maximum and sum in binary32, the output's sums
// rescaled when the maximum grows.
//
// Operands.  Both products run on v_mfma_f32_16x16x32_f16.  A code is exact in fp16;
// a bf16 q is scaled by one power of two a tile (its largest value in [2^14, 2^15)),
// which is exact for values within 2^29 of it.  The keys' scales multiply the scores.
// The values' scales s multiply the probabilities: the weight p s 2^11 / u is rounded to
// fp16 (11 bits: fp16 results are then as far from the exact ones as one rounding to fp16,
// 2.1e-4 for 2.0e-4 in the 2-norm; the one rounding here that is not binary32), u the
// largest s so far.  Weights are at most 2^15 and keep their 11 bits down to 2^-25 of the
// largest; the sums are kept in units of u 2^-11.
//
// The score product is formed transposed, keys x rows: a lane then has four
// consecutive keys of one row, which is the operand the output product (channels x
// rows) takes, with the values stored in that order of keys.  Probabilities never
// leave the registers, and a row's maximum and sum are over four lanes.
//
// Rows: the call's tokens times the query heads that share a kv head, row r = token
// r / G, head r % G.  A work item is a tile of rows of one entry and kv head over one
// piece of the keys; pieces are made where there are too few tiles for the chip and
// joined by a second kernel, in order.  Which tiles and pieces there are is worked out by
// every block from the lengths on the device, so that a captured step follows them.
#include <algorithm>
#include <atomic>
#include <climits>

#include "kernels.hpp"
#include "kv_cache.hpp"

namespace nvfp4 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -__builtin_huge_valf();
// A running maximum is kept while weights stay within 2^4 of its own, so that the
// output's sums are rescaled a few times instead of at every second step; fp16 holds
// 2^11 times that.
constexpr float kSlack = 4.0f;
constexpr float kUnit = 0x1p11f;
constexpr float kLeastUnit = 0x1p-100f;   // of u
constexpr float kLeastScale = 0x1p-126f;  // of a page's scales, as this kernel uses them

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
  uint32_t blocks;
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

// Tiles of an entry, none if its rows are another kernel's.
template <int BM>
__device__ __forceinline__ int entry_tiles(const AttnParams& a, const KvEntry& e) {
  const int rows = e.n * a.group;
  return rows > a.rows_above && rows <= a.rows_most ? (rows + BM - 1) / BM : 0;
}

// Steps of a piece, from the sum of tiles x steps over all entries (binary32, in an order
// that is every block's; one step more than the quotient covers its rounding).
__device__ __forceinline__ int steps_of_piece(const AttnParams& a, float total) {
  const float n = total * static_cast<float>(a.c.heads) / static_cast<float>(a.target) * 1.0001f + 1.0f;
  return max(a.least_steps, static_cast<int>(fminf(n, 0x1p30f)));
}

struct Count {
  uint32_t blocks, cut;  // cut: pieces of cut tiles << 12 | cut tiles; both without the factor of the kv heads
  int pieces;
};
__device__ __forceinline__ Count entry_blocks(const AttnParams& a, int tiles, int steps, int piece_steps) {
  Count c{0, 0, 1};
  if (!tiles) return c;
  if (a.target) c.pieces = (steps + piece_steps - 1) / piece_steps;
  const uint64_t n = static_cast<uint64_t>(tiles) * c.pieces;
  c.blocks = static_cast<uint32_t>(min(n, uint64_t{1} << 25));
  // (with target <= 1024 the pieces of cut tiles are at most 2048 in all)
  if (c.pieces > 1) c.cut = c.blocks << 12 | static_cast<uint32_t>(tiles);
  return c;
}

__device__ __forceinline__ float wave_total(float v) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// Which work item a block has (false: none).  Every block computes the same cut of
// the batch: the number of pieces of each entry, and from their sums where its own
// index falls.  Up to 256 entries every wave does so by itself, up to four entries a
// lane, without a barrier; more are the block's together.
template <int THREADS, int STEP, int BM>
__device__ __forceinline__ bool find_work(const AttnParams& a, uint32_t block, Work& w) {
  const KvParams& p = a.c;
  const int lane = threadIdx.x & (kWave - 1);
  const uint32_t want = block / p.heads;
  w.head = block % p.heads;
  if (!a.target && !p.cu) {  // every entry has one token, every tile one block
    const uint32_t tiles = (a.group + BM - 1) / BM;
    w.entry = want / tiles;
    w.e = kv_entry(p, w.entry);
    w.tiles = tiles;
    w.tile = want % tiles;
    w.pieces = 1;
    w.piece = w.slot = 0;
    return w.e.n > 0;
  }
  uint32_t total_blocks, total_cut;
  int index, cut_before;
  if (p.entries <= 4 * kWave) {
    const int per = (p.entries + kWave - 1) / kWave;
    KvEntry e[4];
    int tiles[4], steps[4];
    float work = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = lane * per + k;
      e[k] = KvEntry{};
      tiles[k] = steps[k] = 0;
      if (k < per && i < p.entries) {
        e[k] = kv_entry(p, i);
        tiles[k] = entry_tiles<BM>(a, e[k]);
        if (tiles[k]) steps[k] = entry_steps<STEP, BM>(a, e[k]);
        work += static_cast<float>(tiles[k]) * static_cast<float>(steps[k]);
      }
    }
    const int piece_steps = a.target ? steps_of_piece(a, wave_total(work)) : 0;
    Count c[4];
    uint32_t blocks = 0, cut = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      c[k] = entry_blocks(a, tiles[k], steps[k], piece_steps);
      blocks += c[k].blocks;
      cut += c[k].cut;
    }
    uint32_t at = wave_scan(blocks), cut_at = a.target ? wave_scan(cut) : 0;
    total_blocks = __builtin_amdgcn_readlane(at, kWave - 1);
    total_cut = __builtin_amdgcn_readlane(cut_at, kWave - 1);
    at -= blocks;
    cut_at -= cut;
    const uint64_t here = __ballot(want - at < blocks);
    const int from = here ? __builtin_ctzll(here) : 0;
    w.entry = here ? 0 : -1;
    // the lane's entry among its four
    int mine = 0;
    uint32_t in = want - at;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (mine == k && in >= c[k].blocks) {
        in -= c[k].blocks;
        cut_at += c[k].cut;
        mine = k + 1;
      }
    }
    KvEntry x = e[0];
    int t = tiles[0], n = c[0].pieces;
#pragma unroll
    for (int k = 1; k < 4; ++k)
      if (mine == k) {
        x = e[k];
        t = tiles[k];
        n = c[k].pieces;
      }
    if (here) w.entry = from * per + __builtin_amdgcn_readlane(mine, from);
    w.e.len = __builtin_amdgcn_readlane(x.len, from);
    w.e.n = __builtin_amdgcn_readlane(x.n, from);
    w.e.first = __builtin_amdgcn_readlane(x.first, from);
    w.e.slot = __builtin_amdgcn_readlane(x.slot, from);
    w.tiles = __builtin_amdgcn_readlane(t, from);
    w.pieces = __builtin_amdgcn_readlane(n, from);
    index = __builtin_amdgcn_readlane(in, from);
    cut_before = __builtin_amdgcn_readlane(cut_at, from);
  } else {
    __shared__ uint64_t buf[2][THREADS / kWave];
    __shared__ float sum[THREADS / kWave];
    __shared__ int found[3];
    const int per = (p.entries + THREADS - 1) / THREADS;
    const int i0 = threadIdx.x * per, i1 = min(i0 + per, p.entries);
    int piece_steps = 0;
    if (a.target) {
      float work = 0.0f;
      for (int i = i0; i < i1; ++i) {
        const KvEntry e = kv_entry(p, i);
        const int t = entry_tiles<BM>(a, e);
        if (t) work += static_cast<float>(t) * static_cast<float>(entry_steps<STEP, BM>(a, e));
      }
      work = wave_total(work);
      if (lane == 0) sum[threadIdx.x / kWave] = work;
      __syncthreads();
      work = 0.0f;
      for (int i = 0; i < THREADS / kWave; ++i) work += sum[i];
      piece_steps = steps_of_piece(a, work);
    }
    auto count_of = [&](int i, KvEntry& e, int& t) {
      e = kv_entry(p, i);
      t = entry_tiles<BM>(a, e);
      return entry_blocks(a, t, t ? entry_steps<STEP, BM>(a, e) : 0, piece_steps);
    };
    KvEntry e;
    int t;
    uint64_t own = 0, total;
    for (int i = i0; i < i1; ++i) {
      const Count c = count_of(i, e, t);
      own += static_cast<uint64_t>(c.blocks) << 24 | c.cut;
    }
    if (threadIdx.x == 0) found[0] = -1;
    uint64_t at = block_scan<THREADS>(own, buf[0], total) - own;
    total_blocks = static_cast<uint32_t>(min(total >> 24, uint64_t{UINT32_MAX}));
    total_cut = static_cast<uint32_t>(total & 0xffffff);
    if (want >= at >> 24 && want < (at + own) >> 24) {
      for (int i = i0; i < i1; ++i) {
        const Count c = count_of(i, e, t);
        if (want < (at >> 24) + c.blocks) {
          found[0] = i;
          found[1] = static_cast<int>(want - (at >> 24));
          found[2] = static_cast<int>(at & 0xffffff);
          break;
        }
        at += static_cast<uint64_t>(c.blocks) << 24 | c.cut;
      }
    }
    __syncthreads();
    w.entry = uniform(found[0]);
    index = cut_before = 0;
    if (w.entry >= 0) {
      w.pieces = uniform(count_of(w.entry, w.e, w.tiles).pieces);
      index = uniform(found[1]);
      cut_before = uniform(found[2]);
    }
  }
  // (entries that share tokens can need more blocks than there are: such a call does nothing)
  const bool fits = static_cast<uint64_t>(total_blocks) * p.heads <= a.blocks;
  if (a.target && block == 0 && threadIdx.x == 0)
    *a.join_count = fits ? static_cast<int>(total_cut & 4095) * p.heads : 0;
  if (!fits || w.entry < 0) return false;
  // the last rows see the most keys: their tiles first
  w.tile = w.tiles - 1 - index / w.pieces;
  w.piece = index % w.pieces;
  w.slot = ((cut_before >> 12) + index) * p.heads + w.head;
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
    a.joins[((cut_before & 4095) + index / w.pieces) * p.heads + w.head] = j;
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

// The tail's tokens have scales of their own, powers of two.  A block of 16 gets the largest
// as its scale; the values are brought to it (a token of 2^-28 of the block's largest
// keeps its 11 bits), so that the products see the same thing as in a page.
__device__ __forceinline__ float row_max(float v) {  // over 16 lanes (a NaN is none)
  v = fmaxf(v, __uint_as_float(dpp_u32<kDppXor1>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp_u32<kDppXor2>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp_u32<kDppHalfMirror>(__float_as_uint(v))));
  return fmaxf(v, __uint_as_float(dpp_u32<kDppMirror>(__float_as_uint(v))));
}
__device__ __forceinline__ float relative(float scale, float block) {  // 0 for a NaN and for none
  return scale > 0.0f ? scale / block : 0.0f;
}
__device__ __forceinline__ float nan_mark(float k, float v) {  // 0, or NaN if either is
  return k != k || v != v ? __uint_as_float(0x7fc00000u) : 0.0f;
}

// A wave's 16 MR rows: operands, running maximum, sum (of the lane's own keys) and
// output sums (channels 16 f + 4 (lane / 16) + i of row lane % 16).
template <int D, int MR>
struct Rows {
  half8 q[MR][D / 32];
  float m[MR], l[MR];
  f32x4 o[MR][D / 16];
  float u, inv;        // unit, kUnit / u
  float c;             // |scale| log2(e) over q's power of two
  int lo[MR], hi[MR];  // keys that the lane's row sees: lo <= key < hi
  int all_lo, all_hi;  // keys that every row sees

  struct Raw {
    u32x4 x[MR][D / 32];
  };

  // Rows [r0, r0 + 16 MR) of the entry, of which `rows` exist: the loads of q, and what
  // needs no memory.
  __device__ __forceinline__ void issue(Raw& raw, const AttnParams& a, const KvEntry& e, int head, int r0, int rows) {
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int r = 0; r < MR; ++r) {
      const int row = r0 + 16 * r + lane % 16, token = row / a.group;
      const int64_t at = (e.first + token) * a.ldq + (head * a.group + row % a.group) * a.ldq_head;
      const char* p = static_cast<const char*>(a.q) + (at + 16 * (lane / 16)) * 2;
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
        raw.x[r][k] = row < rows ? *reinterpret_cast<const u32x4*>(p + (64 * (k / 2) + 8 * (k % 2)) * 2) : u32x4{};
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
  }

  // fp16 operands; the scale's sign is q's (the largest score is then the largest product).
  __device__ __forceinline__ void prepare(const Raw& raw, const AttnParams& a) {
    c = fabsf(a.scale) * kLog2e;
    if (!a.bf16) {
      const uint32_t keep = a.scale == 0.0f ? 0u : ~0u, flip = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
      for (int r = 0; r < MR; ++r)
#pragma unroll
        for (int k = 0; k < D / 32; ++k) q[r][k] = __builtin_bit_cast(half8, (raw.x[r][k] & keep) ^ flip);
      return;
    }
    // The largest finite magnitude of the tile: with 0x80 added to its bits an infinity or a
    // NaN is a negative number to the signed maximum.
    typedef short short2v __attribute__((ext_vector_type(2)));
    short2v most = {0, 0};
#pragma unroll
    for (int r = 0; r < MR; ++r)
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = raw.x[r][k][i] & 0x7fff7fffu;
          most = __builtin_elementwise_max(most, __builtin_bit_cast(short2v, w) + short2v{0x80, 0x80});
        }
    const float top = wave_max(static_cast<float>(max(most[0], most[1])));
    const int exp = max((max(static_cast<int>(top) - 0x80, 0) >> 7) - 127 - 14, -126);
    const float sign = a.scale < 0.0f ? -1.0f : a.scale > 0.0f ? 1.0f : 0.0f;
    const float mul = sign * __uint_as_float(static_cast<uint32_t>(127 - exp) << 23);
    c *= __uint_as_float(static_cast<uint32_t>(127 + exp) << 23);
#pragma unroll
    for (int r = 0; r < MR; ++r)
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          typedef float f32x2 __attribute__((ext_vector_type(2)));
          const half2v h = __builtin_convertvector((f32x2{bf16_lo(raw.x[r][k][i]) * mul, bf16_hi(raw.x[r][k][i]) * mul}), half2v);
          q[r][k][2 * i] = h[0];
          q[r][k][2 * i + 1] = h[1];
        }
  }

  // One step, 16 NB keys, in three parts.  s: products of q and the keys.  key(b, k): a
  // key operand, of block b of 16 keys and 32 channels.
  template <int NB, typename Key>
  __device__ __forceinline__ void scores(f32x4 (&s)[MR][NB], Key key) const {
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
  }

  // The largest score of a lane's four keys in each block.
  template <int NB>
  __device__ __forceinline__ void tops(const f32x4 (&s)[MR][NB], float (&top)[MR][NB]) const {
#pragma unroll
    for (int r = 0; r < MR; ++r)
#pragma unroll
      for (int b = 0; b < NB; ++b) top[r][b] = fmaxf(fmaxf(s[r][b][0], s[r][b][1]), fmaxf(s[r][b][2], s[r][b][3]));
  }

  // Scores out of sight: of keys before or behind what a row sees, of a block whose page is
  // none (ok[b] false).  mark: 0, or NaN where a key or its value is NaN.  Only for
  // steps that have such keys.
  template <int NB>
  __device__ __forceinline__ void mask(f32x4 (&s)[MR][NB], int key0, const bool (&ok)[NB], const f32x4 (&mark)[NB]) const {
    const int g4 = (threadIdx.x & (kWave - 1)) / 16 * 4;
#pragma unroll
    for (int r = 0; r < MR; ++r)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = key0 + 16 * b + g4 + i;
          s[r][b][i] = ok[b] && at >= lo[r] && at < hi[r] ? s[r][b][i] + mark[b][i] : kNone;
        }
  }

  // w: weights 2^(x - m) s_v kUnit / u of the values' codes; maxima, sums, units.  ks, vs:
  // the scales of each block of 16 keys.  The values' factor goes into the exponent: a
  // weight costs one fma, one exponential, one addition and half a conversion, and a
  // block's weights are divided by their factor in their sum.
  template <int NB>
  __device__ __forceinline__ void weights(const f32x4 (&s)[MR][NB], const float (&tops)[MR][NB], half8 (&w)[MR][NB / 2],
                                          const float (&ks)[NB], const float (&vs)[NB]) {
    float top = vs[0];
#pragma unroll
    for (int b = 1; b < NB; ++b) top = fmaxf(top, vs[b]);
    if (__ballot(top > u)) {
      const float down = u / top;
      u = top;
      inv = kUnit / top;
#pragma unroll
      for (int r = 0; r < MR; ++r)
#pragma unroll
        for (int f = 0; f < D / 16; ++f) o[r][f] *= down;
    }
    // Scales of nothing but zeros, and those far below the unit (2^-60: fp16 has lost
    // their weights), are raised, so that no factor is zero.
    const float least = fmaxf(u * 0x1p-60f, kLeastScale);
    float kc[NB], log_f[NB], one_f[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float f = fmaxf(vs[b], least) * inv;
      kc[b] = fmaxf(ks[b] * c, kLeastScale);
      log_f[b] = __builtin_amdgcn_logf(f);
      one_f[b] = __builtin_amdgcn_rcpf(f);
    }
    float top_x[MR];
    bool grows = false;
#pragma unroll
    for (int r = 0; r < MR; ++r) {
      top_x[r] = kNone;
#pragma unroll
      for (int b = 0; b < NB; ++b) top_x[r] = fmaxf(top_x[r], tops[r][b] * kc[b]);
      grows = grows || top_x[r] > m[r] + kSlack;
    }
    if (__ballot(grows)) {
#pragma unroll
      for (int r = 0; r < MR; ++r) {
        const float now = fmaxf(m[r], over_groups<true>(top_x[r]));
        const float down = __builtin_amdgcn_exp2f(m[r] - (now == kNone ? 0.0f : now));
        m[r] = now;
        l[r] *= down;
#pragma unroll
        for (int f = 0; f < D / 16; ++f) o[r][f] *= down;
      }
    }
#pragma unroll
    for (int r = 0; r < MR; ++r) {
      const float base = m[r] == kNone ? 0.0f : m[r];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const float off = log_f[b] - base;
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][b][i], kc[b], off));
        l[r] += ((e[0] + e[1]) + (e[2] + e[3])) * one_f[b];
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const half2v h = __builtin_convertvector((f32x2{e[i], e[i + 1]}), half2v);
          w[r][b / 2][b % 2 * 4 + i] = h[0];
          w[r][b / 2][b % 2 * 4 + i + 1] = h[1];
        }
      }
    }
  }

  // The weights times the values.  value(t, f): a value operand, of 32 keys and 16 channels.
  template <int NB, typename Value>
  __device__ __forceinline__ void outputs(const half8 (&w)[MR][NB / 2], Value value) {
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

using GlobalBytes = __attribute__((address_space(1))) uint8_t;
using GlobalPiece = __attribute__((address_space(1))) u32x4;

// Where row r of an entry writes its output.
__device__ __forceinline__ int64_t out_at(const AttnParams& a, int first, int head, int row) {
  return (first + row / a.group) * a.ldo + (head * a.group + row % a.group) * a.ldo_head;
}

__device__ __forceinline__ void put8(const AttnParams& a, int64_t at, const float (&v)[8]) {
  if (a.bf16) store8<Bf16>(a.out, at, v);
  else store8<F16>(a.out, at, v);
}

// Few rows: the kernel reads the cache once and is bound by that.  Each of a block's
// NW waves takes every NW-th step of the piece, its codes straight to registers, the
// next step's loads in flight while one is computed; the results meet in LDS.  Steps of 32
// keys, their code once in the kernel: a call of one short sequence is bound by the way
// through memory to instructions and codes (600 tokens, 2 kv heads: 9.1 us, with steps of 64
// keys unrolled twice 12.1), and a CU has twelve waves of loads in flight (64 sequences of
// up to 8192 tokens, 8 kv heads, 8 query heads each, D = 128: 119 us, 5.3 TB/s; with
// steps of 64 and eight waves 131; with sixteen waves, which spill, 201).  One sequence of 131001 tokens, 4
// kv heads: 26.6 us, 5.0 TB/s, in 512 pieces; in 768 29, in 1024 31.
constexpr int stream_waves_of_simd(int D, int MR, int NW) {
  return NW > 4 ? 2 : D * MR <= 128 ? 3 : D * MR <= 256 ? 2 : 1;
}

template <int D, int MR, int NW>
__device__ __forceinline__ void stream_block(const AttnParams& a, uint32_t index, float* lds) {
  constexpr int NB = 2, STEP = 16 * NB, NU = D / 64, BM = 16 * MR;
  constexpr int kBatch = kWave / NB;  // steps whose pages a wave looks up together
  const KvParams& p = a.c;
  Work w;
  if (!find_work<NW * kWave, STEP, BM>(a, index, w)) return;
  const KvEntry& e = w.e;
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
  const int r0 = w.tile * BM, rows = e.n * a.group;
  int lo, hi, s0, s1;
  seen(a, e, r0, min(BM, rows - r0), lo, hi);
  const Steps<STEP> st(e.total(), p.shift);
  piece_steps<STEP>(st, w, lo, hi, s0, s1);

  const int64_t page_bytes = int64_t{p.P} * p.D;
  // This wave's steps: every NW-th of the pages', and the tail's from the last wave on.
  const int codes = min(s1, st.full_steps) - s0, tail0 = max(s0, st.full_steps);
  const int of_codes = wave < codes ? (codes - wave + NW - 1) / NW : 0;

  // A batch of steps' pages.  Lane NB j + b: block b of this wave's step b0 + j.
  int id = -1;
  float ks_lane = 0.0f, vs_lane = 0.0f;
  auto look_up = [&](int b0) {
    const int key = (s0 + wave + (b0 + lane / NB) * NW) * STEP + 16 * (lane % NB);
    id = -1;
    ks_lane = vs_lane = 0.0f;
    if (b0 + lane / NB < of_codes && key < st.full_keys) id = kv_page(p, w.entry, key >> p.shift);
    if (id >= 0) {
      ks_lane = p.scales[kv_page_at(p, id, 0, w.head)];
      vs_lane = p.scales[kv_page_at(p, id, 1, w.head)];
    }
  };
  struct Codes {
    u32x4 k[NB][NU], v[NB][NU];
  };
  auto fetch = [&](Codes& x, int b0, int j) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int page = max(__builtin_amdgcn_readlane(id, j * NB + b), 0);
      const int in_page = ((s0 + wave + (b0 + j) * NW) * STEP + 16 * b) & (p.P - 1);
      const uint8_t* k = p.codes + kv_page_at(p, page, 0, w.head) * page_bytes + in_page * D;
      const uint8_t* v = k + p.heads * page_bytes;
#pragma unroll
      for (int c = 0; c < NU; ++c) {
        x.k[b][c] = *reinterpret_cast<const u32x4*>(k + c * 1024 + lane * 16);
        x.v[b][c] = *reinterpret_cast<const u32x4*>(v + c * 1024 + lane * 16);
      }
    }
  };

  // q's loads go out first, then the way to the first codes, then q is prepared
  Rows<D, MR> t;
  typename Rows<D, MR>::Raw raw;
  t.issue(raw, a, e, w.head, r0, rows);
  Codes x;
  if (of_codes) {
    look_up(0);
    fetch(x, 0, 0);
  }
  t.prepare(raw, a);

  f32x4 s[MR][NB];
  float tops[MR][NB];
  half8 wt[MR][NB / 2];
  for (int b0 = 0; b0 < of_codes; b0 += kBatch) {
    if (b0) {
      look_up(b0);
      fetch(x, b0, 0);
    }
    const int n = min(kBatch, of_codes - b0);
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      Codes y = x;
      if (j + 1 < n) fetch(x, b0, j + 1);
      float ks[NB], vs[NB];
      f32x4 mark[NB];
      bool ok[NB], plain = true;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        ok[b] = __builtin_amdgcn_readlane(id, j * NB + b) >= 0;
        ks[b] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ks_lane), j * NB + b));
        vs[b] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(vs_lane), j * NB + b));
        mark[b] = f32x4{} + nan_mark(ks[b], vs[b]);
        plain = plain && ok[b] && nan_mark(ks[b], vs[b]) == 0.0f;
      }
      const int key0 = (s0 + wave + (b0 + j) * NW) * STEP;
      t.template scores<NB>(s, [&](int b, int k) { return kv_codes8(y.k[b][k / 2][k % 2 * 2], y.k[b][k / 2][k % 2 * 2 + 1]); });
      if (!plain || key0 < t.all_lo || key0 + STEP > t.all_hi) t.template mask<NB>(s, key0, ok, mark);
      t.template tops<NB>(s, tops);
      t.template weights<NB>(s, tops, wt, ks, vs);
      t.template outputs<NB>(wt, [&](int h, int f) { return kv_codes8(y.v[2 * h][f / 4][f % 4], y.v[2 * h + 1][f / 4][f % 4]); });
    }
  }

  // the tail's steps
#pragma unroll 1
  for (int i = tail0 + NW - 1 - wave; i < s1; i += NW) {
    const int key0 = st.first(i), in_tail = key0 - st.full_keys;
    const int64_t at = kv_page_at(p, e.slot, 0, w.head);
    const char* k = reinterpret_cast<const char*>(p.tails + at * page_bytes) + lane * 16;
    const char* v = k + p.heads * page_bytes * 2;
    half8 xk[NB][2 * NU], xv[NB][2 * NU];
    float ks[NB], vs[NB];
    f32x4 mark[NB];
    bool ok[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      // (a block behind the page is out of sight; its operands are the page's first)
      ok[b] = in_tail + 16 * b < p.P;
      const int block = ok[b] ? in_tail / 16 + b : 0;
#pragma unroll
      for (int c = 0; c < 2 * NU; ++c) {
        xk[b][c] = *reinterpret_cast<const half8*>(k + (block * 2 * NU + c) * 1024);
        xv[b][c] = *reinterpret_cast<const half8*>(v + (block * 2 * NU + c) * 1024);
      }
      const int valid = e.total() - key0 - 16 * b;  // tokens of the block
      const float* k16 = p.tail_scales + at * p.P + block * 16;
      const float* v16 = k16 + static_cast<int64_t>(p.heads) * p.P;
      const float k_own = lane % 16 < valid ? k16[lane % 16] : 0.0f, v_own = lane % 16 < valid ? v16[lane % 16] : 0.0f;
      ks[b] = row_max(k_own);
      vs[b] = row_max(v_own);
      const float k_rel = relative(k_own, ks[b]), v_lane = relative(v_own, vs[b]), nan = nan_mark(k_own, v_own);
      float v_rel[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v_rel[j] = __shfl(v_lane, lane / 16 * 4 + j);
        mark[b][j] = __shfl(nan, lane / 16 * 4 + j);
      }
#pragma unroll
      for (int c = 0; c < 2 * NU; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          xk[b][c][j] = static_cast<_Float16>(static_cast<float>(xk[b][c][j]) * k_rel);
          xv[b][c][j] = static_cast<_Float16>(static_cast<float>(xv[b][c][j]) * v_rel[j % 4]);
        }
    }
    t.template scores<NB>(s, [&](int b, int c) { return xk[b][c]; });
    t.template mask<NB>(s, key0, ok, mark);
    t.template tops<NB>(s, tops);
    t.template weights<NB>(s, tops, wt, ks, vs);
    t.template outputs<NB>(wt, [&](int h, int f) {
      const half8 x0 = xv[2 * h][f / 2], x1 = xv[2 * h + 1][f / 2];
      return f % 2 ? __builtin_shufflevector(x0, x1, 4, 5, 6, 7, 12, 13, 14, 15) : __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 8, 9, 10, 11);
    });
  }
  t.finish();

  // the waves' results of a row together, in their order
  constexpr int LD = D + 4;  // (a row starts four banks behind the one before)
  float* sums = lds;
  float* ml = lds + NW * 16 * LD;
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
    for (int item = threadIdx.x; item < 16 * D / 8; item += NW * kWave) {
      const int row = item / (D / 8), d = item % (D / 8) * 8, at_row = r0 + 16 * r + row;
      if (at_row >= rows) continue;
      float m = kNone, l = 0.0f, f[NW], v[8] = {};
#pragma unroll
      for (int i = 0; i < NW; ++i) m = fmaxf(m, ml[(i * 16 + row) * 2]);
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        f[i] = __builtin_amdgcn_exp2f(ml[(i * 16 + row) * 2] - (m == kNone ? 0.0f : m));
        l += f[i] * ml[(i * 16 + row) * 2 + 1];
      }
#pragma unroll
      for (int i = 0; i < NW; ++i)
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

template <int D, int MR, int NW>
__global__ __launch_bounds__(NW * kWave, (stream_waves_of_simd(D, MR, NW))) void kv_stream_kernel(AttnParams a) {
  extern __shared__ __align__(16) float stream_lds[];
  stream_block<D, MR, NW>(a, blockIdx.x, stream_lds);
}

// Many rows: eight waves of 16 MR rows each share every step's keys and values, which
// are made fp16 once, on their way into LDS.
constexpr int kTileWaves = 8, kTileThreads = kTileWaves * kWave;
template <int D>
constexpr int tile_frags = D <= 128 ? 2 : 1;

template <int D>
struct TileLds {
  half8 k[4][D / 32][kWave];  // [block of 16 keys][32 channels][lane]
  half8 v[2][D / 16][kWave];  // [32 keys][16 channels][lane]
};
// Scales of a step's blocks, keys' and values'; the keys' is -1 where a block's page is
// none.  Marks of the tail's tokens: NaN for one with a NaN, else 0.  Written two or three
// steps ahead, a scale read during the products before it is used: four places.
struct TileScales {
  f32x4 of[4][2];
  float mark[4][2][64];
};

template <int D>
__device__ __forceinline__ void tile_block(const AttnParams& a, uint32_t index, char* raw_lds) {
  constexpr int MR = tile_frags<D>, BM = 16 * MR * kTileWaves, STEP = 64, NB = 4, NU = D / 64;
  typedef _Float16 half4 __attribute__((ext_vector_type(4)));
  TileLds<D>* lds = reinterpret_cast<TileLds<D>*>(raw_lds);
  TileScales& steps = *reinterpret_cast<TileScales*>(lds + 2);
  const KvParams& p = a.c;
  Work w;
  if (!find_work<kTileThreads, STEP, BM>(a, index, w)) return;
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
  typename Rows<D, MR>::Raw raw;
  t.issue(raw, a, e, w.head, r0, rows);

  // Staging: this wave brings block `block` of 16 keys (waves 0 to 3: keys, 4 to 7:
  // values) of a step into LDS; its scales come with it.
  const int block = wave % 4, which = wave / 4;
  const int64_t page_bytes = int64_t{p.P} * p.D;
  // Where the block is and its scale, of 64 steps, a lane each.  Vector loads, since a
  // barrier waits for scalar ones; complete addresses, since a step has no time for them.
  int from = 0;
  float scales = 0.0f;
  uint64_t sources = 0;
  auto look_up = [&](int s) {
    const int key = st.first(s + lane) + 16 * block;
    from = s;
    if (s + lane < st.full_steps) {
      const int id = s + lane < s1 && key < st.full_keys ? kv_page(p, w.entry, key >> p.shift) : -1;
      const int64_t at = kv_page_at(p, max(id, 0), which, w.head);
      scales = id >= 0 ? p.scales[at] : which ? 0.0f : -1.0f;
      sources = reinterpret_cast<uint64_t>(p.codes + at * page_bytes + (key & (p.P - 1)) * D);
    } else {
      // a block of the tail has the largest scale of its tokens
      sources = reinterpret_cast<uint64_t>(p.codes);
      scales = which ? 0.0f : -1.0f;
      if (s + lane < s1 && key - st.full_keys < p.P) {
        const float* x = p.tail_scales + kv_page_at(p, e.slot, which, w.head) * p.P + (key - st.full_keys);
        const int n = min(16, e.total() - key);
        scales = 0.0f;
        for (int i = 0; i < n; ++i) scales = fmaxf(scales, x[i]);
      }
    }
  };
  auto tell = [&](int s) {  // step s's scale, and its marks, to the others
    if (s - from < kWave) {
      const float scale = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(scales), s - from));
      if (lane == 0) reinterpret_cast<float*>(&steps.of[s & 3][which])[block] = scale;
    }
    const int in_tail = (s - st.full_steps) * STEP + 16 * block + lane;
    if (s >= st.full_steps && s < s1 && lane < 16)
      steps.mark[s & 3][which][16 * block + lane] =
          st.full_keys + in_tail < e.total()
              ? nan_mark(p.tail_scales[kv_page_at(p, e.slot, which, w.head) * p.P + in_tail], 0.0f)
              : 0.0f;
  };
  // (loaded for every step, from the first page where there are no codes: a load under a
  // condition would be waited for where the two ways meet)
  u32x4 st_raw[NU];
  auto fetch = [&](int s) {
    if (s - from >= kWave) look_up(s);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(sources), s - from);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(sources >> 32), s - from);
    // (an address made of integers is none of global memory to the compiler unless told,
    // and a barrier waits for loads that may be LDS's)
    const GlobalBytes* src = reinterpret_cast<const GlobalBytes*>(static_cast<uint64_t>(hi) << 32 | lo);
#pragma unroll
    for (int c = 0; c < NU; ++c) st_raw[c] = *reinterpret_cast<const GlobalPiece*>(src + (c * 1024 + lane * 16));
  };
  // What the wave brings in of step s: fp16 operands, from the codes that were fetched or
  // from the tail.
  auto convert = [&](int s, half8 (&x)[2 * NU]) {
    if (s < st.full_steps || s >= s1) {
#pragma unroll
      for (int c = 0; c < 2 * NU; ++c) x[c] = kv_codes8(st_raw[c / 2][c % 2 * 2], st_raw[c / 2][c % 2 * 2 + 1]);
    } else {
      const int key0 = st.first(s) + 16 * block;
      const int64_t at = kv_page_at(p, e.slot, which, w.head);
      const int in_tail = key0 - st.full_keys < p.P ? key0 - st.full_keys : 0;
      const char* src = reinterpret_cast<const char*>(p.tails + at * page_bytes + in_tail * D) + lane * 16;
      float token = p.tail_scales[at * p.P + in_tail + lane % 16];
      if (key0 + lane % 16 >= e.total()) token = 0.0f;
      const float own = relative(token, row_max(token));
      // of the lane's eight values' tokens: one (keys) or four, twice (values)
      float rel[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) rel[i] = which ? __shfl(own, lane / 16 * 4 + i) : own;
#pragma unroll
      for (int c = 0; c < 2 * NU; ++c) {
        x[c] = *reinterpret_cast<const half8*>(src + c * 1024);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c][i] = static_cast<_Float16>(static_cast<float>(x[c][i]) * rel[i % 4]);
      }
    }
  };
  // Into LDS: a key operand is a lane's eight values; a value operand has four of one block
  // of 16 keys and four of the next.  The same instructions for both.
  const int part_step = which ? 2048 : 1024, half_step = which ? 1024 : 8;
  const int part_first = which ? static_cast<int>(sizeof(lds->k)) + block / 2 * (D / 16) * 1024 + lane * 16 + block % 2 * 8
                               : block * (D / 32) * 1024 + lane * 16;
  auto put = [&](const half8 (&x)[2 * NU], TileLds<D>& to) {
    char* at = reinterpret_cast<char*>(&to) + part_first;
#pragma unroll
    for (int c = 0; c < 2 * NU; ++c) {
      *reinterpret_cast<half4*>(at + c * part_step) = __builtin_shufflevector(x[c], x[c], 0, 1, 2, 3);
      *reinterpret_cast<half4*>(at + c * part_step + half_step) = __builtin_shufflevector(x[c], x[c], 4, 5, 6, 7);
    }
  };

  const int ahead = which ? 1 : 2;
  if (s0 < s1) {
    look_up(s0);
    fetch(s0);
  }
  t.prepare(raw, a);
  if (s0 < s1) {
    tell(s0);
    for (int i = 0; i < ahead; ++i) {
      half8 x[2 * NU];
      convert(s0 + i, x);
      put(x, lds[i]);
      fetch(s0 + i + 1);
      tell(s0 + i + 1);
    }
  }
  // A step is its softmax and then the matrix products (its outputs and the next step's
  // scores) with a part of a later step brought in between them.  There is one barrier a
  // step: waves 0 to 3 have it before the softmax, waves 4 to 7, which share the SIMDs with
  // them, before the products.  So in every interval between barriers one half begins with
  // the softmax and the other with the products, and both the vector and the matrix units
  // have work; the products go first where both want to issue.  Chunks of 4096 tokens at 4096
  // (kv heads 8, 4 query heads each, D = 128, two sequences) take 687 us, 0.98 PFLOP/s; without the
  // two orders 1186 us, without the priority 909 us.
  // (In the interval of step s's products its values and the keys of s + 1 are read, and the
  // values of s + 1 and the keys of s + 2 written: each has two places.  The last products
  // read keys of a step that is not there: whatever scores they give are not used.)
  if (s0 < s1) {
    f32x4 sc[MR][NB];
    float tops[MR][NB];
    half8 wt[MR][NB / 2];
    lds_barrier();
    if (some) t.template scores<NB>(sc, [&](int b, int k) { return lds[0].k[b][k][lane]; });
    f32x4 ks4 = steps.of[s0 & 3][0], vs4 = steps.of[s0 & 3][1];
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      TileLds<D>& now = lds[(s - s0) & 1];
      TileLds<D>& next = lds[(s - s0 + 1) & 1];
      __builtin_amdgcn_s_setprio(0);
      if (!which) lds_barrier();
      if (some) {
        const int key0 = st.first(s);
        float ks[NB], vs[NB];
        uint32_t odd = 0;  // (a negative number and a NaN are above every scale, as bits)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          ks[b] = ks4[b];
          vs[b] = vs4[b];
          odd = max(odd, max(__float_as_uint(ks[b]), __float_as_uint(vs[b])));
        }
        t.template tops<NB>(sc, tops);
        if (static_cast<uint32_t>(uniform(odd)) >= 0x7f800000u || s >= st.full_steps || key0 < t.all_lo ||
            key0 + STEP > t.all_hi) {
          bool ok[NB];
          f32x4 mark[NB];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            ok[b] = !(ks[b] < 0.0f);
            if (s < st.full_steps)
              mark[b] = f32x4{} + nan_mark(ks[b], vs[b]);
            else
              mark[b] = *reinterpret_cast<const f32x4*>(steps.mark[s & 3][0] + 16 * b + lane / 16 * 4) +
                        *reinterpret_cast<const f32x4*>(steps.mark[s & 3][1] + 16 * b + lane / 16 * 4);
          }
          t.template mask<NB>(sc, key0, ok, mark);
          t.template tops<NB>(sc, tops);
        }
        t.template weights<NB>(sc, tops, wt, ks, vs);
      }
      if (which) lds_barrier();
      __builtin_amdgcn_s_setprio(2);
      half8 x[2 * NU];
      convert(s + ahead, x);
      fetch(s + ahead + 1);
      tell(s + ahead + 1);
      ks4 = steps.of[(s + 1) & 3][0];
      vs4 = steps.of[(s + 1) & 3][1];
      put(x, which ? next : now);
      if (some) {
        t.template outputs<NB>(wt, [&](int h, int f) { return now.v[h][f][lane]; });
        t.template scores<NB>(sc, [&](int b, int k) { return next.k[b][k][lane]; });
        // Operands are read kAhead before their products: left to itself the compiler reads two
        // and waits (a read takes about 130 cycles, its products 16 MR).
        constexpr int kReads = D / 4, kAhead = 8;
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
        for (int i = 0; i < kReads - kAhead; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, MR, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, kAhead * MR, 0);
      }
    }
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

template <int D>
__global__ __launch_bounds__(kTileThreads, 2) void kv_tile_kernel(AttnParams a) {
  extern __shared__ __align__(16) char tile_lds[];
  tile_block<D>(a, blockIdx.x, tile_lds);
}

// Entries of many and of few rows together, each kind by its blocks: one launch, and neither
// waits for the other (9 entries, 501 tokens at most, D = 64: in two launches 12 us more).
template <int D, int MR>
__global__ __launch_bounds__(kTileThreads, 2) void kv_mixed_kernel(AttnParams many, AttnParams few) {
  extern __shared__ __align__(16) char mixed_lds[];
  if (blockIdx.x < many.blocks) tile_block<D>(many, blockIdx.x, mixed_lds);
  else stream_block<D, MR, kTileWaves>(few, blockIdx.x - many.blocks, reinterpret_cast<float*>(mixed_lds));
}

// Pieces of a row joined in their order.  One wave a row, or where there are few rows the
// block's four (SPLIT) for one, each with a quarter of the pieces; a lane has four channels.
constexpr int kJoinThreads = 256, kJoinWaves = kJoinThreads / kWave;

template <int D, int SPLIT>
__global__ __launch_bounds__(kJoinThreads) void kv_join_kernel(AttnParams a, int bm, int joins, AttnParams b, int b_bm) {
  constexpr int CH = D / 4, PER = kWave / CH, ROWS = kJoinWaves / SPLIT;  // PER pieces at once
  __shared__ f32x4 sums[kJoinWaves][CH];
  __shared__ float sums_l[kJoinWaves];
  int index = blockIdx.x;
  if (index >= joins) {
    index -= joins;
    a.joins = b.joins;
    a.join_count = b.join_count;
    a.part = b.part;
    a.part_ml = b.part_ml;
    bm = b_bm;
  }
  if (index >= *a.join_count) return;
  const KvJoin j = a.joins[index];
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
  const int ch = lane % CH, sub = lane / CH;
  for (int r = blockIdx.y * ROWS; r < j.rows; r += gridDim.y * ROWS) {
    const int row = r + wave / SPLIT;
    const bool in = row < j.rows;
    auto at = [&](int piece) { return (int64_t{j.slot} + int64_t{piece} * j.stride) * bm + row; };
    float m = kNone, l = 0.0f;
    f32x4 v{};
    if (in) {
      for (int i = lane; i < j.pieces; i += kWave) m = fmaxf(m, a.part_ml[at(i) * 2]);
    }
    m = wave_max(m);
    const float base = m == kNone ? 0.0f : m;
    if (in && sub < PER) {
#pragma unroll 8
      for (int i = wave % SPLIT * PER + sub; i < j.pieces; i += SPLIT * PER) {
        const float f = __builtin_amdgcn_exp2f(a.part_ml[at(i) * 2] - base);
        l += f * a.part_ml[at(i) * 2 + 1];
        v += f * *reinterpret_cast<const f32x4*>(a.part + at(i) * D + 4 * ch);
      }
    }
#pragma unroll
    for (int d = CH; d < kWave && PER > 1; d *= 2) {
      l += __shfl_xor(l, d);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += __shfl_xor(v[i], d);
    }
    if constexpr (SPLIT > 1) {
      __syncthreads();
      if (lane < CH) sums[wave][lane] = v;
      if (lane == 0) sums_l[wave] = l;
      __syncthreads();
      if (wave % SPLIT == 0 && lane < CH) {
#pragma unroll
        for (int i = 1; i < SPLIT; ++i) {
          v += sums[wave + i][lane];
          l += sums_l[wave + i];
        }
      }
    }
    if (in && wave % SPLIT == 0 && lane < CH) {
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
  int64_t tiles, slots, joins, blocks;  // upper bounds, kv heads included
};
struct Plan {
  Cut stream, tile;
  int mr;
};

// Keys below which a sequence stays in one piece and no join is launched.
constexpr int64_t kWholeKeys = 1024;

Cut make_cut(const KvParams& p, int group, int bm, int step, int target, int least_steps, int rows_above, int rows_most) {
  Cut c{};
  c.use = true;
  c.bm = bm;
  c.rows_above = rows_above;
  c.rows_most = rows_most;
  const int64_t rows = int64_t{p.tokens} * group, entries = std::min(p.entries, p.tokens);
  c.tiles = p.cu ? rows / bm + entries : entries * ((group + bm - 1) / bm);
  c.tiles = std::min(c.tiles, entries * ((int64_t{rows_most} + bm - 1) / bm)) * p.heads;
  c.blocks = c.tiles;
  const int64_t keys = int64_t{p.width} << p.shift, most = (keys / step + 2 + least_steps - 1) / least_steps;
  if (keys <= kWholeKeys || (p.entries == 1 && rows / bm * p.heads >= target)) return c;
  c.target = target;
  c.least_steps = least_steps;
  c.blocks = std::min(target + c.tiles, c.tiles * most);
  c.slots = std::min(int64_t{2} * target, c.tiles * most);
  c.joins = std::min(int64_t{target}, c.tiles);
  return c;
}

template <int D>
Plan make_plan(const KvParams& p, int group) {
  Plan x{};
  // Entries of up to three tiles are the stream kernel's: a tile of the other has eight
  // waves, of which they would keep two or three busy (64 entries of 8 tokens, 8 heads a kv head, at
  // 8000 tokens: 206 us, by the other 442).  Tiles of 32 rows where the entries have between
  // 16 and 96 on average, and 256 registers hold them; else those of few rows are likely
  // single tokens (9 entries, 501 tokens at most, 3 heads a kv head: 35 us, with tiles of 32 rows 37).
  const int all = INT_MAX / 2;
  const int64_t rows = int64_t{p.tokens} * group, entries = std::max(1, std::min(p.entries, p.tokens));
  const int frags = D <= 128 && rows > 16 * entries && rows <= 96 * entries ? 2 : 1, most = 48 * frags;
  const bool stream = !p.cu || rows <= 32, tile = !stream && p.entries == 1, both = !stream && !tile;
  x.mr = stream ? (group > 16 || (p.cu && p.tokens > p.entries) ? 2 : 1) : frags;
  // (blocks at once: two a CU of four waves, one of eight)
  if (!tile)
    x.stream = make_cut(p, group, 16 * x.mr, 32, both ? 256 : 512, 16, 0, both ? most : all);
  if (!stream) x.tile = make_cut(p, group, 16 * tile_frags<D> * kTileWaves, 64, 256, 8, both ? most : 0, all);
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
  a.blocks = static_cast<uint32_t>(c.blocks);
  if (c.target) {
    a.join_count = reinterpret_cast<int*>(ws + at.count);
    a.joins = reinterpret_cast<KvJoin*>(ws + at.joins);
    a.part = reinterpret_cast<float*>(ws + at.part);
    a.part_ml = reinterpret_cast<float*>(ws + at.ml);
  }
  return a;
}

// Lets a kernel use `bytes` of dynamic LDS, once a device (devices past the mask's 64 on
// every call).
template <typename K>
hipError_t allow_lds(K kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t{1} << dev : 0;
  if (bit != 0 && (done.load(std::memory_order_relaxed) & bit) != 0) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Joins of one or (b) two kinds of blocks.
template <int D>
hipError_t join(const AttnParams& a, const Cut& c, const AttnParams& b, const Cut& d, hipStream_t s) {
  if (!c.target && !d.target) return hipSuccess;
  if (!c.target) return join<D>(b, d, a, c, s);
  const int64_t joins = c.joins + (d.target ? d.joins : 0), rows = c.rows_most < c.bm ? c.rows_most : c.bm;
  if (joins * rows >= 1024) {
    const int64_t y = std::max<int64_t>(1, std::min<int64_t>((rows + 3) / 4, 8192 / joins));
    kv_join_kernel<D, 1><<<dim3(joins, y), kJoinThreads, 0, s>>>(a, c.bm, c.joins, b, d.bm);
  } else {
    kv_join_kernel<D, kJoinWaves><<<dim3(joins, rows), kJoinThreads, 0, s>>>(a, c.bm, c.joins, b, d.bm);
  }
  return hipGetLastError();
}

constexpr int stream_lds_bytes(int D, int NW) { return (NW * 16 * (D + 4) + NW * 16 * 2) * 4; }
template <int D>
constexpr int tile_lds_bytes = 2 * sizeof(TileLds<D>) + sizeof(TileScales);

template <int D, int MR, int NW>
hipError_t run_stream(const AttnParams& a, hipStream_t s) {
  constexpr int kLds = stream_lds_bytes(D, NW);
  static std::atomic<uint64_t> done{0};
  const hipError_t e = allow_lds(kv_stream_kernel<D, MR, NW>, kLds, done);
  if (e != hipSuccess) return e;
  kv_stream_kernel<D, MR, NW><<<a.blocks, NW * kWave, kLds, s>>>(a);
  return hipGetLastError();
}

template <int D>
hipError_t run(const KvAttention& k, char* ws, hipStream_t s) {
  const Plan x = make_plan<D>(k.c, k.group);
  const Area sa = area(x.stream, D, 0), ta = area(x.tile, D, sa.end);
  const AttnParams few = with(k, x.stream, sa, ws), many = with(k, x.tile, ta, ws);
  hipError_t e;
  if (x.tile.use && x.stream.use) {
    constexpr int kLds = std::max(tile_lds_bytes<D>, stream_lds_bytes(D, kTileWaves));
    const auto launch = [&](auto kernel, std::atomic<uint64_t>& done) {
      const hipError_t set = allow_lds(kernel, kLds, done);
      if (set != hipSuccess) return set;
      kernel<<<many.blocks + few.blocks, kTileThreads, kLds, s>>>(many, few);
      return hipGetLastError();
    };
    static std::atomic<uint64_t> done[2];
    if constexpr (D <= 128) e = x.mr == 2 ? launch(kv_mixed_kernel<D, 2>, done[1]) : launch(kv_mixed_kernel<D, 1>, done[0]);
    else e = launch(kv_mixed_kernel<D, 1>, done[0]);
  } else if (x.tile.use) {
    static std::atomic<uint64_t> done{0};
    e = allow_lds(kv_tile_kernel<D>, tile_lds_bytes<D>, done);
    if (e != hipSuccess) return e;
    kv_tile_kernel<D><<<many.blocks, kTileThreads, tile_lds_bytes<D>, s>>>(many);
    e = hipGetLastError();
  } else if (x.mr == 2) {
    e = run_stream<D, 2, 4>(few, s);
  } else {
    e = x.stream.target || few.blocks > 256 ? run_stream<D, 1, 4>(few, s) : run_stream<D, 1, 8>(few, s);
  }
  return e != hipSuccess ? e : join<D>(many, x.tile, few, x.stream, s);
}

template <int D>
int64_t bytes(const KvParams& p, int group, int64_t* blocks) {
  const Plan x = make_plan<D>(p, group);
  *blocks = x.stream.blocks + x.tile.blocks;
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

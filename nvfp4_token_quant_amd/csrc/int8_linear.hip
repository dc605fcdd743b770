// 8-bit integer linear product with scales for each token and channel (gfx950).
//
//   quantize: s = RN(amax / 127), q = RNE(x * RN(127 / amax)) of a row
//   product:  out[m, n] = sa[m] sb[n] sum_k a[m, k] b[n, k] + bias[n]
// The sum is exact in int32 for K < 2^31 / 128^2.  In binary32 it is rounded,
// multiplied by the rounded product of its scales and, in one rounding, added to
// the bias; that is rounded to the output's type.
#include <algorithm>
#include <atomic>
#include <iterator>
#include <type_traits>

#include "common.hpp"
#include "dtype.hpp"
#include "kernels.hpp"

namespace nvfp4 {

namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// Rows whose largest magnitude is below 2^-119 quantize as zero rows: there
// 127 / amax would leave the binary32 range.
constexpr float kMinAmax = 0x1p-119f;

// Eight codes as two dwords, the first column in the lowest byte.
__device__ __forceinline__ u32x2 pack_codes(const float (&f)[8], float inv) {
  u32x2 r = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // |x inv| <= 127 (1 + 2^-23): the clamp only bounds a row with an infinity or a
    // NaN, whose codes mean nothing
    const int q = static_cast<int>(__builtin_amdgcn_fmed3f(__builtin_rintf(f[j] * inv), -127.0f, 127.0f));
    r[j / 4] |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * (j % 4));
  }
  return r;
}

// Eight columns of a row as binary32, 0 past the end.  VEC: cols a multiple of
// 8, rows 16-byte aligned; else pieces at any address, and the row's last one
// value by value.
template <typename T, bool VEC>
__device__ __forceinline__ void load_piece(float (&f)[8], const void* row, int64_t c, int64_t cols) {
  Raw8<T> raw;
  if constexpr (VEC) {
    load8<T>(raw, row, min(c, cols - 8));  // unconditional, so that all pieces' loads are in flight together
    to_f32<T>(raw, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = c < cols ? f[j] : 0.0f;
  } else if (c + 8 <= cols) {
    load8_any<T>(raw, row, c);
    to_f32<T>(raw, f);
  } else if (c < cols) {
    // (unconditional loads, in flight together)
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = T::get(row, min(c + j, cols - 1));
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = c + j < cols ? f[j] : 0.0f;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.0f;
  }
}

// The larger of two magnitudes, NaN if one is.
__device__ __forceinline__ float amax(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float amax8(const float (&f)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = amax(m, fabsf(f[j]));
  return m;
}
// The wave's largest magnitude, NaN if one is: bit patterns of magnitudes are
// ordered as they are, infinity and NaN last.
__device__ __forceinline__ float wave_amax(float m) {
  uint32_t v = __float_as_uint(m) & 0x7FFFFFFFu;
  v = max(v, dpp_u32<kDppXor1>(v));
  v = max(v, dpp_u32<kDppXor2>(v));
  v = max(v, dpp_u32<kDppHalfMirror>(v));
  v = max(v, dpp_u32<kDppMirror>(v));
  uint32_t a, b;
  lane_pair<16>(v, a, b);
  lane_pair<32>(max(a, b), a, b);
  return __uint_as_float(max(a, b));
}
// A row's factor and scale from its largest magnitude.  A row with an infinity or
// a NaN has the scale NaN, and so have its products.
struct RowScale {
  float inv, scale;
  __device__ explicit RowScale(float am) {
    const bool some = am >= kMinAmax && am <= 3.402823466e38f;
    inv = some ? 127.0f / am : 0.0f;
    scale = some ? am / 127.0f : am < kMinAmax ? 1.0f : __builtin_nanf("");
  }
};

}  // namespace

// TPR threads a row (64: four rows a block, 256: one), NC pieces of eight
// columns a thread, held in registers between the maximum and the codes, so
// that the row is read once.  The codes of a row end on a 16-byte piece,
// filled with zeros.  Bound by memory: 16384 x 7168 bf16 67 us (5.3 TB/s).
template <typename T, bool VEC, int TPR, int NC>
__global__ __launch_bounds__(256) void int8_quantize_kernel(const void* __restrict__ x, int64_t rows, int cols,
                                                            int64_t ld, int8_t* __restrict__ codes,
                                                            int64_t ld_codes, float* __restrict__ scales) {
  __shared__ float s_am[4];
  const int lt = threadIdx.x % TPR;
  const int64_t row = block_id() * (256 / TPR) + threadIdx.x / TPR;
  if (row >= rows) return;  // whole waves, and no barrier where a block holds several rows
  const void* xrow = static_cast<const char*>(x) + row * ld * T::kBytes;
  const int cols16 = (cols + 15) / 16 * 16;
  float f[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) load_piece<T, VEC>(f[i], xrow, 8 * (lt + TPR * i), cols);
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) am = amax(am, amax8(f[i]));
  am = wave_amax(am);
  if constexpr (TPR > kWave) {
    if ((threadIdx.x & (kWave - 1)) == 0) s_am[threadIdx.x / kWave] = am;
    __syncthreads();
    am = amax(amax(s_am[0], s_am[1]), amax(s_am[2], s_am[3]));
  }
  const RowScale rs(am);
  int8_t* crow = codes + row * ld_codes;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = 8 * (lt + TPR * i);
    if (c < cols16) *reinterpret_cast<u32x2*>(crow + c) = pack_codes(f[i], rs.inv);
  }
  if (lt == 0) scales[row] = rs.scale;
}

// Longer rows: one block a row, two passes over it.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void int8_quantize_long_kernel(const void* __restrict__ x, int64_t rows,
                                                                 int64_t cols, int64_t ld, int8_t* __restrict__ codes,
                                                                 int64_t ld_codes, float* __restrict__ scales) {
  __shared__ float s_am[4];
  const int64_t row = block_id();
  if (row >= rows) return;
  const void* xrow = static_cast<const char*>(x) + row * ld * T::kBytes;
  const int64_t cols16 = (cols + 15) / 16 * 16;
  float am = 0.0f;
  for (int64_t c = 8 * static_cast<int64_t>(threadIdx.x); c < cols; c += 8 * 256) {
    float f[8];
    load_piece<T, VEC>(f, xrow, c, cols);
    am = amax(am, amax8(f));
  }
  am = wave_amax(am);
  if ((threadIdx.x & (kWave - 1)) == 0) s_am[threadIdx.x / kWave] = am;
  __syncthreads();
  am = amax(amax(s_am[0], s_am[1]), amax(s_am[2], s_am[3]));
  const RowScale rs(am);
  for (int64_t c = 8 * static_cast<int64_t>(threadIdx.x); c < cols16; c += 8 * 256) {
    float f[8];
    load_piece<T, VEC>(f, xrow, c, cols);
    *reinterpret_cast<u32x2*>(codes + row * ld_codes + c) = pack_codes(f, rs.inv);
  }
  if (threadIdx.x == 0) scales[row] = rs.scale;
}

template <typename T, bool VEC>
static void launch_quantize_width(const void* x, int64_t rows, int64_t cols, int64_t ld, int8_t* codes,
                                  int64_t ld_codes, float* scales, hipStream_t s) {
  const int64_t cols16 = (cols + 15) / 16 * 16;
  const int c = static_cast<int>(cols);
  const dim3 g1 = grid_of(rows), g4 = grid_of((rows + 3) / 4);
  if (cols16 <= 512)
    int8_quantize_kernel<T, VEC, 64, 1><<<g4, 256, 0, s>>>(x, rows, c, ld, codes, ld_codes, scales);
  else if (cols16 <= 1024)
    int8_quantize_kernel<T, VEC, 64, 2><<<g4, 256, 0, s>>>(x, rows, c, ld, codes, ld_codes, scales);
  else if (cols16 <= 2048)
    int8_quantize_kernel<T, VEC, 256, 1><<<g1, 256, 0, s>>>(x, rows, c, ld, codes, ld_codes, scales);
  else if (cols16 <= 4096)
    int8_quantize_kernel<T, VEC, 256, 2><<<g1, 256, 0, s>>>(x, rows, c, ld, codes, ld_codes, scales);
  else if (cols16 <= 8192)
    int8_quantize_kernel<T, VEC, 256, 4><<<g1, 256, 0, s>>>(x, rows, c, ld, codes, ld_codes, scales);
  else if (cols16 <= 16384)
    int8_quantize_kernel<T, VEC, 256, 8><<<g1, 256, 0, s>>>(x, rows, c, ld, codes, ld_codes, scales);
  else
    int8_quantize_long_kernel<T, VEC><<<g1, 256, 0, s>>>(x, rows, cols, ld, codes, ld_codes, scales);
}

template <typename T>
static void launch_quantize_type(const void* x, int64_t rows, int64_t cols, int64_t ld, int8_t* codes,
                                 int64_t ld_codes, float* scales, hipStream_t s) {
  const bool vec = cols % 8 == 0 && (ld * T::kBytes) % 16 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
  if (vec) launch_quantize_width<T, true>(x, rows, cols, ld, codes, ld_codes, scales, s);
  else launch_quantize_width<T, false>(x, rows, cols, ld, codes, ld_codes, scales, s);
}

hipError_t launch_int8_quantize_rows(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld,
                                     int8_t* codes, int64_t ld_codes, float* scales, hipStream_t s) {
  if (dtype == MOE_BF16) launch_quantize_type<Bf16>(x, rows, cols, ld, codes, ld_codes, scales, s);
  else if (dtype == MOE_F16) launch_quantize_type<F16>(x, rows, cols, ld, codes, ld_codes, scales, s);
  else launch_quantize_type<F32>(x, rows, cols, ld, codes, ld_codes, scales, s);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Product.  Weight rows are MFMA operand A (16 channels x 64 k), token rows
// operand B (64 k x 16 tokens): lane l holds 16 k of channel or token l % 16,
// and of the result token l % 16, channels 4 (l / 16) + 0..3.  k may be
// assigned to lanes in any order that both operands share.
// ---------------------------------------------------------------------------

// The sum times its scales, plus the bias, in binary32: the same steps in every
// kernel (one rounding of product and bias), so that a token's result does not
// depend on the batch that it comes with.
__device__ __forceinline__ float scaled(float acc, float s, bool has_bias, float bias) {
  return has_bias ? __builtin_fmaf(acc, s, bias) : acc * s;
}
// Whether a product of scales is a normal number: its rounding is then half a
// step, else (smallest rows and channels: 2^-126 x 1e-4) it has lost bits that
// the result would have.
__device__ __forceinline__ bool scale_in_range(float s) {
  return fabsf(s) >= 0x1p-126f && fabsf(s) <= 3.402823466e38f;
}
// The factors acc and s = sa * sb where s may be out of range: s of the scales'
// fractions (with the bits of sa * sb where that is in range), their exponents
// shared between the two factors.
__device__ __forceinline__ void factors_far(float& acc, float& s, float sa, float sb) {
  s = __builtin_amdgcn_frexp_mantf(sa) * __builtin_amdgcn_frexp_mantf(sb);
  const int e = __builtin_amdgcn_frexp_expf(sa) + __builtin_amdgcn_frexp_expf(sb);
  const int es = min(max(e, -120), 120);
  s = ldexpf(s, es);
  acc = ldexpf(acc, e - es);
}

// out[m, n]; sa: token m's scale
__device__ __forceinline__ void store_one(const Int8GemmParams& p, int m, int n, int acc, float sa) {
  const float sb = p.sb[n];
  float a = static_cast<float>(acc), s = sa * sb;
  if (!scale_in_range(s)) factors_far(a, s, sa, sb);
  const float f = scaled(a, s, p.bias != nullptr, p.bias ? p.bias[n] : 0.0f);
  const int64_t at = static_cast<int64_t>(m) * p.ldo + n;
  if (p.dtype == MOE_BF16) Bf16::put(p.out, at, f);
  else if (p.dtype == MOE_F16) F16::put(p.out, at, f);
  else F32::put(p.out, at, f);
}

// kDotLoads loads of a whole kilobyte of a channel's row are in flight together.
constexpr int kDotLoads = 8;

__device__ __forceinline__ int wave_sum_i32(int v) {
  v += static_cast<int>(dpp_u32<kDppXor1>(static_cast<uint32_t>(v)));
  v += static_cast<int>(dpp_u32<kDppXor2>(static_cast<uint32_t>(v)));
  v += static_cast<int>(dpp_u32<kDppHalfMirror>(static_cast<uint32_t>(v)));
  v += static_cast<int>(dpp_u32<kDppMirror>(static_cast<uint32_t>(v)));
  uint32_t a, b;
  lane_pair<16>(static_cast<uint32_t>(v), a, b);
  v = static_cast<int>(a) + static_cast<int>(b);
  lane_pair<32>(static_cast<uint32_t>(v), a, b);
  return static_cast<int>(a) + static_cast<int>(b);
}

// One token: a wave a channel, products of four bytes at a time in the vector
// ALU (a tile of matrix instructions would be a sixteenth full).  Every block
// keeps the row's codes in LDS; with an unquantized row x of type T it makes
// them itself, behind the loads of its waves' first channels, by the steps of
// the quantization kernel (two launches cost more than the work: 7168 x 2048
// 8.1 us in two kernels, 4.5 in one).
constexpr int kTokenThreads = 512;
static_assert(kTokenThreads * 8 * 8 == kLinearTokenMaxK, "eight pieces of a row a thread at most");

struct Codes {};  // the row is p.a, its scale p.sa[0]

// Eight codes at column c of the row, 0 from K on.  The row's last 16-byte
// piece lies inside its leading dimension.
__device__ __forceinline__ u32x2 load_codes8(const int8_t* row, int c, int K) {
  u32x2 v = *reinterpret_cast<const u32x2*>(row + min(c, (K + 15) / 16 * 16 - 8));
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int left = K - c - 4 * j;  // bytes of this dword before K
    if (left < 4) v[j] = left <= 0 ? 0u : v[j] & ((1u << (8 * left)) - 1u);
  }
  return v;
}

template <typename T, int NC>
__global__ __launch_bounds__(kTokenThreads) void int8_token_kernel(Int8GemmParams p, const void* __restrict__ x) {
  extern __shared__ __align__(16) uint8_t s_codes[];  // the row's codes, zeros up to a whole kilobyte
  __shared__ float s_am[kTokenThreads / kWave];
  constexpr int W = kTokenThreads / kWave;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int last = (p.K - 1) / 16 * 16;
  int64_t n = static_cast<int64_t>(blockIdx.x) * W + wave;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * W;
  // a chunk: kDotLoads kilobytes of a channel's row (past its end the last
  // piece again, times zero)
  const auto load = [&](i32x4 (&b)[kDotLoads], int64_t ch, int c0) {
    const int8_t* row = p.b + min(ch, static_cast<int64_t>(p.N) - 1) * p.ldb;
#pragma unroll
    for (int i = 0; i < kDotLoads; ++i) b[i] = *reinterpret_cast<const i32x4*>(row + min(c0 + 1024 * i + 16 * lane, last));
  };
  const int kib = (p.K + 1023) / 1024 * 1024;
  i32x4 b[kDotLoads];
  float scale;
  if constexpr (std::is_same_v<T, Codes>) {
    u32x2 q[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) q[i] = load_codes8(p.a, 8 * (tid + kTokenThreads * i), p.K);
    load(b, n, 0);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = 8 * (tid + kTokenThreads * i);
      if (c < kib) *reinterpret_cast<u32x2*>(s_codes + c) = q[i];
    }
    scale = p.sa[0];
  } else {
    float f[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) load_piece<T, false>(f[i], x, 8 * (tid + kTokenThreads * i), p.K);
    load(b, n, 0);
    float am = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) am = amax(am, amax8(f[i]));
    am = wave_amax(am);
    if (lane == 0) s_am[wave] = am;
    lds_barrier();  // (the channels' loads stay in flight)
#pragma unroll
    for (int w = 0; w < W; ++w) am = amax(am, s_am[w]);
    const RowScale rs(am);
    scale = rs.scale;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = 8 * (tid + kTokenThreads * i);
      if (c < kib) *reinterpret_cast<u32x2*>(s_codes + c) = pack_codes(f[i], rs.inv);
    }
  }
  lds_barrier();
  for (; n < p.N; n += stride) {
    int acc = 0;
    for (int c0 = 0; c0 < p.K; c0 += 1024 * kDotLoads) {
#pragma unroll
      for (int i = 0; i < kDotLoads; ++i) {
        if (c0 + 1024 * i < p.K) {
          const i32x4 a = *reinterpret_cast<const i32x4*>(s_codes + c0 + 1024 * i + 16 * lane);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_sdot4(a[j], b[i][j], acc, false);
        }
      }
      // the next chunk, of this channel or the next
      if (c0 + 1024 * kDotLoads < p.K) load(b, n, c0 + 1024 * kDotLoads);
      else if (n + stride < p.N) load(b, n + stride, 0);
    }
    acc = wave_sum_i32(acc);
    if (lane == 0) store_one(p, 0, static_cast<int>(n), acc, scale);
  }
}

// ---------------------------------------------------------------------------
// Tiled product for many tokens.  A block of WM x WN waves computes BM = 16 FM
// WM tokens by BN = 16 FN WN channels; K goes by in steps of 128 bytes through
// two LDS buffers.
//
// Copies go from global memory straight to LDS, one instruction for 8 rows of
// 128 bytes (whole lines).  The 16-byte pieces of a row are permuted by a key
// of the row, so that the eight lanes of an LDS read that take the same piece
// of different rows touch different banks (no conflict counted; a 1 KB read
// takes 4 cycles).  Token fragments are read from LDS kAhead ahead of their
// MFMAs, across the step's barrier too: the last kAhead fragments of a step are
// in registers when its buffer is handed back.  A buffer comes back in two
// parts: behind a barrier in the middle of the step the channel rows and the
// token rows of the first four groups, which everybody has read by then, and
// behind its end the rest, so that copies start one and a half steps and one
// step before they are needed (one buffer at a time, at the end of the step:
// 8192^3 of zeros 412 us, in two parts 370).
//
// What bounds it: on operands like activations and weights the chip's power.
// 8192^3 takes 449 us (2450 TOP/s; of zeros 370, without the copies 384), 4096 x
// 7168 x 7168 176 to 212 us from one card to another (448 tiles on 256 CUs), a
// library's product alone, measured beside it, 462 and 195 to 236.  Four waves of
// twice the tile each (128 x 128) took 576 us of zeros: one wave a SIMD hides
// nothing.  Bands of 4 token tiles an XCD: 1% over 8; tiles in block order
// instead: 5% slower.
//
// Fragment f of a wave's channels holds channels 4 FN (r / 4) + 4 f + r % 4
// (r its row), so a lane ends with 4 FN consecutive channels of a token and
// stores them as whole 16-byte pieces.
// ---------------------------------------------------------------------------
constexpr int kStepBytes = 128;
constexpr int64_t kMaxTileLd = int64_t(1) << 22;  // 256 rows within 31-bit offsets
constexpr int kAhead = 3;

template <int FN>
__device__ __forceinline__ int channel_key(int row) { return (row & 3) | ((row / (4 * FN) & 1) << 2); }

// Origin of this block's tile, false past the last: each XCD (block % 8) takes a contiguous run of
// tiles, ordered in bands of 4 token tiles, so that the blocks that share an
// L2 share operands.
template <int BM, int BN>
__device__ __forceinline__ bool tile_origin(int mtiles, int ntiles, int& m0, int& n0) {
  const int total = mtiles * ntiles;
  if (block_id() >= total) return false;
  const int block = static_cast<int>(block_id()), x = block & 7;
  const int id = x * (total / 8) + min(x, total % 8) + (block >> 3);
  const int band = id / (4 * ntiles), in_band = id - band * 4 * ntiles;
  const int bh = min(4, mtiles - 4 * band);
  m0 = (4 * band + in_band % bh) * BM;
  n0 = in_band / bh * BN;
  return true;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t code_rsrc(const int8_t* base, int64_t bytes) {
  // dword 3 = 0x00020000: 32-bit data format, no swizzle (raw buffer)
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(base), static_cast<short>(0),
                                           static_cast<int>(bytes), 0x00020000);
}

// In the last step (columns c0 .. of a K that is no multiple of 128): zeros for
// the bytes of the BM token rows in LDS from K on.
template <int BM, int THREADS>
__device__ __forceinline__ void clear_behind(uint8_t* rows, int c0, int K) {
  for (int i = threadIdx.x; i < BM * 8; i += THREADS) {
    const int c = c0 + 16 * ((i & 7) ^ (i >> 3 & 7));
    i32x4* at = reinterpret_cast<i32x4*>(rows + 16 * i);
    i32x4 v = *at;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int left = K - c - 4 * j;
      if (left < 4) v[j] = left <= 0 ? 0 : v[j] & static_cast<int32_t>((1u << (8 * left)) - 1u);
    }
    *at = v;
  }
  lds_barrier();
}

// Lane's part of the result: tokens t0 + 16 m, channels n0 .. n0 + 4 FN - 1.
template <typename T, int FM, int FN, bool FAR>
__device__ __forceinline__ void store_rows(const Int8GemmParams& p, const i32x4 (&acc)[FN][FM], int t0, int n0,
                                           const float (&sa)[FM], const float (&sb)[4 * FN],
                                           const float (&bias)[4 * FN]) {
#pragma unroll
  for (int m = 0; m < FM; ++m) {
    const int t = t0 + 16 * m;
    if (t >= p.M) continue;
    const int64_t row = static_cast<int64_t>(t) * p.ldo;
#pragma unroll
    for (int f = 0; f < FN; f += 2) {
      constexpr int kP = FN == 1 ? 4 : 8;  // channels of a store
      float v[kP];
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        float a = static_cast<float>(acc[f + i / 4][m][i % 4]), s = sa[m] * sb[4 * f + i];
        if constexpr (FAR) factors_far(a, s, sa[m], sb[4 * f + i]);
        v[i] = scaled(a, s, p.bias != nullptr, bias[4 * f + i]);
      }
      const int n = n0 + 4 * f;
      if (n + kP <= p.N) {
        if constexpr (FN == 1) store4_any<T>(p.out, row + n, v);
        else store8_any<T>(p.out, row + n, v);
      } else {
#pragma unroll
        for (int i = 0; i < kP; ++i)
          if (n + i < p.N) T::put(p.out, row + n + i, v[i]);
      }
    }
  }
}

template <typename T, int FM, int FN>
__device__ __forceinline__ void store_tile(const Int8GemmParams& p, const i32x4 (&acc)[FN][FM], int t0, int n0) {
  // (rows and vectors start anywhere: global memory is read and written in
  // 16-byte pieces at any address; value by value 777 x 1003 x 1999 took 10.5 us,
  // so 9.2)
  float sa[FM], sb[4 * FN], bias[4 * FN] = {};
#pragma unroll
  for (int m = 0; m < FM; ++m) sa[m] = p.sa[min(t0 + 16 * m, p.M - 1)];
  if (n0 <= p.N - 4 * FN) {
    __builtin_memcpy(sb, p.sb + n0, sizeof(sb));
    if (p.bias) __builtin_memcpy(bias, p.bias + n0, sizeof(bias));
  } else {
#pragma unroll
    for (int i = 0; i < 4 * FN; ++i) {
      const int n = min(n0 + i, p.N - 1);
      sb[i] = p.sb[n];
      if (p.bias) bias[i] = p.bias[n];
    }
  }
  // One wave's products of scales are hardly ever out of range, so the question
  // is asked once, of the smallest and the largest.
  float a0 = fabsf(sa[0]), a1 = a0, b0 = fabsf(sb[0]), b1 = b0;
#pragma unroll
  for (int m = 1; m < FM; ++m) {
    a0 = fminf(a0, fabsf(sa[m]));
    a1 = fmaxf(a1, fabsf(sa[m]));
  }
#pragma unroll
  for (int i = 1; i < 4 * FN; ++i) {
    b0 = fminf(b0, fabsf(sb[i]));
    b1 = fmaxf(b1, fabsf(sb[i]));
  }
  if (__any(!scale_in_range(a0 * b0) || !scale_in_range(a1 * b1)))
    store_rows<T, FM, FN, true>(p, acc, t0, n0, sa, sb, bias);
  else
    store_rows<T, FM, FN, false>(p, acc, t0, n0, sa, sb, bias);
}

template <int WM, int WN, int FM, int FN>
__global__ __launch_bounds__(64 * WM * WN)
__attribute__((amdgpu_waves_per_eu(WM * WN / 4, WM * WN / 4))) void int8_tiled_kernel(Int8GemmParams p, int mtiles,
                                                                                  int ntiles) {
  constexpr int W = WM * WN, BM = 16 * FM * WM, BN = 16 * FN * WN;
  constexpr int kStage = (BM + BN) * kStepBytes;
  constexpr int NC = (BM + BN) / 8 / W;  // copy instructions of a wave and step
  constexpr int NCA = BM / 8 / W;        // the token rows' part of them
  constexpr int NI = 2 * FM;             // token fragments of a step
  static_assert((BM / 8) % W == 0 && (BN / 8) % W == 0, "whole copies of each operand");
  static_assert(FM > kAhead && FN % 2 == 0, "the window stays inside a half step");
  extern __shared__ __align__(1024) uint8_t s_tile[];  // 2 * kStage
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int r = lane & 15, g = lane >> 4;

  int m0, n0;
  if (!tile_origin<BM, BN>(mtiles, ntiles, m0, n0)) return;

  // copies: instruction u of this wave fills LDS rows 8 (wave + W u) .. + 7 of
  // the stage (token rows, then channel rows); lane l the piece l % 8 of row
  // l / 8.  Rows behind the last one read that one again (never stored).
  const int K16 = (p.K + 15) / 16 * 16;
  const int mrows = min(BM, p.M - m0), nrows = min(BN, p.N - n0);
  const __amdgpu_buffer_rsrc_t rsa = code_rsrc(p.a + m0 * p.lda, (mrows - 1) * p.lda + K16);
  const __amdgpu_buffer_rsrc_t rsb = code_rsrc(p.b + n0 * p.ldb, (nrows - 1) * p.ldb + K16);
  const int slot = lane & 7, sub = lane >> 3;
  int off[NC];
#pragma unroll
  for (int u = 0; u < NC; ++u) {
    const int row = 8 * (wave + W * u) + sub;
    off[u] = u < NCA ? min(row, mrows - 1) * static_cast<int>(p.lda) + 16 * (slot ^ (row & 7))
                     : min(row - BM, nrows - 1) * static_cast<int>(p.ldb) + 16 * (slot ^ channel_key<FN>(row - BM));
  }
  const int S = (p.K + kStepBytes - 1) / kStepBytes;
  const bool ragged = p.K % kStepBytes != 0;
  // in the last step a piece behind K reads the row's last one instead (cleared
  // below): the bytes to go back, for the token and the channel rows (whose
  // keys do not depend on u)
  static_assert(W % FN == 0, "a wave's channel rows of all its copies have one key");
  const int past = kStepBytes * (S - 1) - (K16 - 16);
  const int back_a = max(0, past + 16 * (slot ^ sub));
  const int back_b = max(0, past + 16 * (slot ^ channel_key<FN>(8 * wave + sub)));
  const auto copy = [&](int s, uint8_t* stage, int u) {
    const int o = off[u] - (s == S - 1 ? (u < NCA ? back_a : back_b) : 0);
    auto* d = (__attribute__((address_space(3))) void*)(stage + 1024 * (wave + W * u));
    __builtin_amdgcn_raw_ptr_buffer_load_lds(u < NCA ? rsa : rsb, d, 16, o, kStepBytes * s, 0, 0);
  };

  // fragment reads: token row 16 m + r, channel row 4 FN (r / 4) + 4 f + r % 4;
  // the second half's piece number differs in bit 2
  const int wm = wave / WN, wn = wave % WN;
  const int crow = 16 * FN * wn + 4 * FN * (r >> 2) + (r & 3);
  const int xbase = (16 * FM * wm + r) * kStepBytes + 16 * (g ^ (r & 7));
  const int wbase = (BM + crow) * kStepBytes + 16 * (g ^ channel_key<FN>(crow));
  i32x4 acc[FN][FM];
#pragma unroll
  for (int f = 0; f < FN; ++f)
#pragma unroll
    for (int m = 0; m < FM; ++m) acc[f][m] = i32x4{0, 0, 0, 0};
  i32x4 x[kAhead + 1], w[2][FN];
  // fragment i of a step: four token groups in the first half, the same four
  // in the second, then the other four
  static_assert(FM == 8, "two groups of four");
  const auto half_of = [](int i) { return i / 4 % 2; };
  const auto group_of = [](int i) { return 4 * (i / 8) + i % 4; };
  const auto read_x = [&](const uint8_t* stage, int i) {
    return *reinterpret_cast<const i32x4*>(stage + (xbase ^ (64 * half_of(i))) + 16 * kStepBytes * group_of(i));
  };
  const auto read_w = [&](const uint8_t* stage, int h, int f) {
    return *reinterpret_cast<const i32x4*>(stage + (wbase ^ (64 * h)) + 4 * kStepBytes * f);
  };
#pragma unroll
  for (int u = 0; u < NC; ++u) copy(0, s_tile, u);
#pragma unroll
  for (int u = 0; u < NC; ++u) copy(min(1, S - 1), s_tile + kStage, u);
  wait_vmcnt<NC>();
  lds_barrier();
  if (S == 1 && ragged) clear_behind<BM, 64 * W>(s_tile, kStepBytes * (S - 1), p.K);
#pragma unroll
  for (int f = 0; f < FN; ++f) w[0][f] = read_w(s_tile, 0, f);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) x[i] = read_x(s_tile, i);

  const auto mma = [&](int i) {
    const int m = group_of(i);
#pragma unroll
    for (int f0 = 0; f0 < FN; ++f0) {
      // there and back, so that two MFMAs in a row always share an operand
      // (the chip's power bounds this kernel: 8192^3 454 -> 449 us)
      const int f = i % 2 ? FN - 1 - f0 : f0;
      acc[f][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[half_of(i)][f], x[i % (kAhead + 1)], acc[f][m], 0, 0, 0);
    }
  };
  static_assert(NI == 16 && NI % (kAhead + 1) == 0 && kAhead <= 4, "the window's slots repeat every step");
  // Copies of the rows that are read by the middle of a step (all channel
  // rows, the token rows of the first four groups), and of the others.
  static_assert(W == FM, "a copy of each wave fills the rows of four groups");
  constexpr int kEarly = NC - NCA + NCA / 2;
  static_assert(NCA == 4 && kEarly <= NI / 2 - kAhead + 1, "one copy between the MFMAs of two fragments");
  const auto early = [&](int j) { return j < NC - NCA ? NCA + j : 2 * (j - (NC - NCA)); };
  // One step on buffer `cur`, whose first kAhead token and first-half channel
  // fragments are in registers.  Behind its middle barrier the early rows'
  // copies of step s + 2 go into `cur`, behind its end the others'.  In the
  // last steps the copies and the reads of the next step are of data that
  // nothing uses.
  const auto step = [&](int s, uint8_t* cur, uint8_t* nxt) {
    const int sn = min(s + 2, S - 1);
#pragma unroll
    for (int i = 0; i < NI / 2; ++i) {
      x[(i + kAhead) % (kAhead + 1)] = read_x(cur, i + kAhead);
      if (i < FN) w[1][i] = read_w(cur, 1, i);
      mma(i);
    }
#pragma unroll
    for (int i = 0; i < NI / 2; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS reads
      if (i < FN) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, FN, 0);  // MFMAs
    }
    __builtin_amdgcn_sched_barrier(0);
    // the early rows' reads have returned in every wave: their MFMAs are issued
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = NI / 2; i < NI - kAhead; ++i) {
      x[(i + kAhead) % (kAhead + 1)] = read_x(cur, i + kAhead);
      mma(i);
#pragma unroll
      for (int j = 0; j < kEarly; ++j)
        if (j * (NI / 2 - kAhead) / kEarly == i - NI / 2) copy(sn, cur, early(j));
    }
#pragma unroll
    for (int i = NI / 2; i < NI - kAhead; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, FN / 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);  // copies
      if (i == NI / 2) __builtin_amdgcn_sched_group_barrier(0x010, kEarly - (NI / 2 - kAhead), 0);
      __builtin_amdgcn_sched_group_barrier(0x008, FN / 2, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<kEarly>();
    lds_barrier();  // step s + 1 has landed; every wave has read step s
    if (ragged && s + 2 == S) clear_behind<BM, 64 * W>(nxt, kStepBytes * (S - 1), p.K);
#pragma unroll
    for (int f = 0; f < FN; ++f) w[0][f] = read_w(nxt, 0, f);
#pragma unroll
    for (int i = NI - kAhead; i < NI; ++i) {
      mma(i);
      x[(i + kAhead) % (kAhead + 1)] = read_x(nxt, i + kAhead - NI);
      if (i - (NI - kAhead) < NCA / 2) copy(sn, cur, 2 * (i - (NI - kAhead)) + 1);
    }
    __builtin_amdgcn_sched_group_barrier(0x100, FN, 0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, FN / 2, 0);
      if (i < NCA / 2) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, FN / 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  int s = 0;
  for (; s + 1 < S; s += 2) {
    step(s, s_tile, s_tile + kStage);
    step(s + 1, s_tile + kStage, s_tile);
  }
  if (s < S) step(s, s_tile, s_tile + kStage);
  wait_vmcnt<0>();  // no copy may land in LDS after the block has ended

  const int t0 = m0 + 16 * FM * wm + r, nl = n0 + 16 * FN * wn + 4 * FN * g;
  if (p.dtype == MOE_BF16) store_tile<Bf16, FM, FN>(p, acc, t0, nl);
  else if (p.dtype == MOE_F16) store_tile<F16, FM, FN>(p, acc, t0, nl);
  else store_tile<F32, FM, FN>(p, acc, t0, nl);
}

// Tokens with little to quantize, two to 16 of them (linear_few_tokens): the product from
// the unquantized rows in one kernel.  Every block quantizes the rows for itself,
// by the steps of the quantization kernel, behind the loads of its first tile's
// weights, and keeps the codes in LDS; its eight waves take every eighth step of a
// tile of 16 channels, weights straight to registers, and their sums meet in LDS.
// The quantizing in every block costs what the launch of a second kernel does at
// about 32768 values (4 x 4096 x 7168: 9.9 us in one, 10.3 in two; 16 x 8192 x 2048
// 12.0 and 7.9), so the rule is half of that: 8 x 4096 x 2048 4.8 and 6.0, 2 x 4096 x
// 7168 8.9 and 10.2, 16 x 128 x 1024 4.5 and 5.7, 2 x 65536 x 4096 53 and 60.
// Of more tokens a block takes 16 (linear_few_tiles): 512 x 256 x 512 5.3 us, in two
// kernels 6.7; with more tiles than fit the chip at once it loses (1024 x 256 x 512
// 8.9 and 7.3).
// TWO: a wave quantizes rows `wave` and `wave + 8`; else 4, 2 or 1 of the eight
// waves share a row.  Rows in LDS are 16 bytes more than a multiple of 128 apart
// (16 lanes that read the same piece of 16 rows touch all banks).
constexpr int kFewThreads = 512, kFewWaves = kFewThreads / kWave, kFewPieces = 4;
constexpr int kFewSteps = kLinearFewMaxK / kStepBytes / kFewWaves;
static_assert(kLinearFewColumns == kFewThreads * 8 * kFewPieces, "all rows' columns are in the block's pieces");

template <typename T, bool TWO>
__global__ __launch_bounds__(kFewThreads) void int8_few_kernel(Int8GemmParams p, const void* __restrict__ x,
                                                               int64_t ldx) {
  extern __shared__ __align__(16) uint8_t s_codes[];  // [M][ls]
  __shared__ float s_am[kFewWaves], s_scale[16];
  __shared__ i32x4 s_sum[kFewWaves - 1][kWave];
  const int lane = threadIdx.x & (kWave - 1), r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int m0 = 16 * static_cast<int>(blockIdx.y);  // this block's rows
  x = static_cast<const char*>(x) + m0 * ldx * T::kBytes;
  p.out = static_cast<char*>(p.out) + m0 * p.ldo * (p.dtype == MOE_F32 ? 4 : 2);
  p.M = min(p.M - m0, 16);
  const int S = (p.K + kStepBytes - 1) / kStepBytes, ls = S * kStepBytes + 16;
  int last = (p.K - 1) / 16 * 16;
  const int tiles = static_cast<int>((static_cast<int64_t>(p.N) + 15) / 16);
  const auto load = [&](i32x4 (&b)[kFewSteps][2], int tile) {  // past K: the last piece again, times zero
    const int8_t* row = p.b + min(static_cast<int64_t>(tile) * 16 + r, static_cast<int64_t>(p.N) - 1) * p.ldb;
#pragma unroll
    for (int i = 0; i < kFewSteps; ++i) {
      const int c = (wave + kFewWaves * i) * kStepBytes + 16 * g;
      if (wave + kFewWaves * i < S) {
        b[i][0] = *reinterpret_cast<const i32x4*>(row + min(c, last));
        b[i][1] = *reinterpret_cast<const i32x4*>(row + min(c + 64, last));
      }
    }
  };

  const int share = TWO || p.M > 4 ? 1 : p.M > 2 ? 2 : 4;  // waves of a row
  const auto row_of = [&](int i) { return TWO ? wave + kFewWaves * (i / (kFewPieces / 2)) : wave / share; };
  const auto col_of = [&](int i) {
    return 8 * (lane + kWave * (TWO ? i % (kFewPieces / 2) : wave % share + share * i));
  };
  float f[kFewPieces][8];
#pragma unroll
  for (int i = 0; i < kFewPieces; ++i)
    load_piece<T, false>(f[i], static_cast<const char*>(x) + min(row_of(i), p.M - 1) * ldx * T::kBytes, col_of(i), p.K);
  int tile = blockIdx.x;
  i32x4 b[kFewSteps][2];
  load(b, tile);
  float am[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kFewPieces; ++i) {
    const int u = TWO && i >= kFewPieces / 2 ? 1 : 0;
    am[u] = amax(am[u], amax8(f[i]));
  }
  am[0] = wave_amax(am[0]);
  if constexpr (TWO) {
    am[1] = wave_amax(am[1]);
  } else {
    if (lane == 0) s_am[wave] = am[0];
    lds_barrier();  // (the weights' loads stay in flight)
    for (int j = 0; j < share; ++j) am[0] = amax(am[0], s_am[wave / share * share + j]);
  }
#pragma unroll
  for (int i = 0; i < kFewPieces; ++i) {
    const RowScale rs(am[TWO && i >= kFewPieces / 2 ? 1 : 0]);
    const int row = row_of(i), c = col_of(i);
    if (row < p.M && c < S * kStepBytes) *reinterpret_cast<u32x2*>(s_codes + row * ls + c) = pack_codes(f[i], rs.inv);
    if (row < p.M && c == 0) s_scale[row] = rs.scale;
  }
  lds_barrier();

  Int8GemmParams q = p;
  q.sa = s_scale;
  const uint8_t* xrow = s_codes + min(r, p.M - 1) * ls + 16 * g;
  for (; tile < tiles; tile += gridDim.x) {
    i32x4 acc[1][1] = {{i32x4{0, 0, 0, 0}}};
#pragma unroll
    for (int i = 0; i < kFewSteps; ++i) {
      const int step = wave + kFewWaves * i;
      if (step < S) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc[0][0] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
              b[i][h], *reinterpret_cast<const i32x4*>(xrow + step * kStepBytes + 64 * h), acc[0][0], 0, 0, 0);
      }
    }
    asm volatile("" : "+s"(last));  // (the columns formed again here: the store needs the registers)
    if (tile + static_cast<int>(gridDim.x) < tiles) load(b, tile + gridDim.x);
    if (wave > 0) s_sum[wave - 1][lane] = acc[0][0];
    lds_barrier();
    if (wave == 0) {
#pragma unroll
      for (int w = 0; w < kFewWaves - 1; ++w) acc[0][0] += s_sum[w][lane];
      if (p.dtype == MOE_BF16) store_tile<Bf16, 1, 1>(q, acc, r, 16 * tile + 4 * g);
      else if (p.dtype == MOE_F16) store_tile<F16, 1, 1>(q, acc, r, 16 * tile + 4 * g);
      else store_tile<F32, 1, 1>(q, acc, r, 16 * tile + 4 * g);
    }
    lds_barrier();  // the sums may be written again
  }
}

// Lets a kernel use `bytes` of dynamic LDS.  The attribute belongs to the
// current device: set once per device (devices past the mask's 64 set it on
// every call).
static hipError_t allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t{1} << dev : 0;
  if (bit != 0 && (done.load(std::memory_order_relaxed) & bit) != 0) return hipSuccess;
  e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// The same product for tiles that fill the chip with less work each: a ring of
// NS stages (NS - 1 of them in flight).  KG groups of WM x WN waves share a
// tile: group kg takes the steps kg, kg + KG, ... (a stage holds one for each
// group), so that a CU with one block still has two waves a SIMD to hide the
// reads of one behind the MFMAs of the other; the groups' sums meet in LDS.
template <int WM, int WN, int FM, int FN, int KG, int NS, int BLOCKS>
__global__ __launch_bounds__(64 * WM * WN * KG)
__attribute__((amdgpu_waves_per_eu(WM * WN * KG * BLOCKS / 4))) void int8_ring_kernel(Int8GemmParams p, int mtiles,
                                                                                      int ntiles) {
  constexpr int W = WM * WN, BM = 16 * FM * WM, BN = 16 * FN * WN;
  constexpr int kPart = (BM + BN) * kStepBytes, kStage = KG * kPart;
  constexpr int NC = (BM + BN) / 8 / W, NCA = BM / 8 / W;
  static_assert((BM / 8) % W == 0 && (BN / 8) % W == 0 && (FN == 1 || FN % 2 == 0), "whole copies of each operand");
  static_assert((NS - 2) * NC < 64 && (KG - 1) * BM * BN * 4 <= NS * kStage, "the groups' sums fit the ring");
  extern __shared__ __align__(1024) uint8_t s_tile[];  // NS * kStage
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave % W;
  const int kg = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / (kWave * W));
  const int r = lane & 15, g = lane >> 4;
  int m0, n0;
  if (!tile_origin<BM, BN>(mtiles, ntiles, m0, n0)) return;

  // copies and fragments as in the kernel above
  const int K16 = (p.K + 15) / 16 * 16;
  const int mrows = min(BM, p.M - m0), nrows = min(BN, p.N - n0);
  const __amdgpu_buffer_rsrc_t rsa = code_rsrc(p.a + m0 * p.lda, (mrows - 1) * p.lda + K16);
  const __amdgpu_buffer_rsrc_t rsb = code_rsrc(p.b + n0 * p.ldb, (nrows - 1) * p.ldb + K16);
  const int slot = lane & 7, sub = lane >> 3;
  const int S = (p.K + kStepBytes - 1) / kStepBytes;
  const bool ragged = p.K % kStepBytes != 0;
  int off[NC], back[NC];  // back: what a piece behind K goes back in the last step
#pragma unroll
  for (int u = 0; u < NC; ++u) {
    const int row = 8 * (wave + W * u) + sub;
    const int col = 16 * (slot ^ (u < NCA ? row & 7 : channel_key<FN>(row - BM)));
    off[u] = (u < NCA ? min(row, mrows - 1) * static_cast<int>(p.lda)
                      : min(row - BM, nrows - 1) * static_cast<int>(p.ldb)) + col;
    back[u] = max(0, kStepBytes * (S - 1) + col - (K16 - 16));
  }
  const auto copy = [&](int round, int at) {  // this group's step of a round into stage `at`
    const int s = min(round * KG + kg, S - 1);
    uint8_t* part = s_tile + at * kStage + kg * kPart;
#pragma unroll
    for (int u = 0; u < NC; ++u) {
      const int o = off[u] - (s == S - 1 ? back[u] : 0);
      auto* d = (__attribute__((address_space(3))) void*)(part + 1024 * (wave + W * u));
      __builtin_amdgcn_raw_ptr_buffer_load_lds(u < NCA ? rsa : rsb, d, 16, o, kStepBytes * s, 0, 0);
    }
  };
  const int wm = wave / WN, wn = wave % WN;
  const int crow = 16 * FN * wn + 4 * FN * (r >> 2) + (r & 3);
  const int xbase = (16 * FM * wm + r) * kStepBytes + 16 * (g ^ (r & 7));
  const int wbase = (BM + crow) * kStepBytes + 16 * (g ^ channel_key<FN>(crow));
  i32x4 acc[FN][FM];
#pragma unroll
  for (int f = 0; f < FN; ++f)
#pragma unroll
    for (int m = 0; m < FM; ++m) acc[f][m] = i32x4{0, 0, 0, 0};

  const int rounds = (S + KG - 1) / KG;
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) copy(i, i);
  int at = 0;  // stage of this round
  for (int i = 0; i < rounds; ++i) {
    wait_vmcnt<(NS - 2) * NC>();
    lds_barrier();  // the round has landed; every wave has read the one before
    if (ragged && i == rounds - 1)
      clear_behind<BM, 64 * W * KG>(s_tile + at * kStage + (S - 1) % KG * kPart, kStepBytes * (S - 1), p.K);
    copy(i + NS - 1, at == 0 ? NS - 1 : at - 1);
    if (i * KG + kg < S) {
      const uint8_t* cur = s_tile + at * kStage + kg * kPart;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        i32x4 x[FM], w[FN];
#pragma unroll
        for (int f = 0; f < FN; ++f)
          w[f] = *reinterpret_cast<const i32x4*>(cur + (wbase ^ (64 * h)) + 4 * kStepBytes * f);
#pragma unroll
        for (int m = 0; m < FM; ++m)
          x[m] = *reinterpret_cast<const i32x4*>(cur + (xbase ^ (64 * h)) + 16 * kStepBytes * m);
#pragma unroll
        for (int m = 0; m < FM; ++m)
#pragma unroll
          for (int f = 0; f < FN; ++f)
            acc[f][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[f], x[m], acc[f][m], 0, 0, 0);
      }
    }
    at = at == NS - 1 ? 0 : at + 1;
  }
  wait_vmcnt<0>();  // no copy may land in LDS after the block has ended, or in the sums
  if constexpr (KG > 1) {
    lds_barrier();
    i32x4* sums = reinterpret_cast<i32x4*>(s_tile);  // [KG - 1][W][FN * FM][64]
    if (kg > 0) {
#pragma unroll
      for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int m = 0; m < FM; ++m) sums[(((kg - 1) * W + wave) * FN * FM + f * FM + m) * kWave + lane] = acc[f][m];
    }
    lds_barrier();
    if (kg > 0) return;
#pragma unroll
    for (int k = 0; k < KG - 1; ++k)
#pragma unroll
      for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int m = 0; m < FM; ++m) acc[f][m] += sums[((k * W + wave) * FN * FM + f * FM + m) * kWave + lane];
  }
  const int t0 = m0 + 16 * FM * wm + r, nl = n0 + 16 * FN * wn + 4 * FN * g;
  if (p.dtype == MOE_BF16) store_tile<Bf16, FM, FN>(p, acc, t0, nl);
  else if (p.dtype == MOE_F16) store_tile<F16, FM, FN>(p, acc, t0, nl);
  else store_tile<F32, FM, FN>(p, acc, t0, nl);
}

template <int WM, int WN, int FM, int FN, int KG, int NS, int BLOCKS>
static hipError_t launch_ring(const Int8GemmParams& p, hipStream_t s) {
  constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN;
  constexpr int kLds = NS * KG * (BM + BN) * kStepBytes;
  static_assert(kLds * BLOCKS <= 160 * 1024, "the blocks of a CU share its LDS");
  const int64_t mt = (static_cast<int64_t>(p.M) + BM - 1) / BM, nt = (static_cast<int64_t>(p.N) + BN - 1) / BN;
  if (mt * nt > INT32_MAX) return hipErrorInvalidConfiguration;
  const auto kernel = int8_ring_kernel<WM, WN, FM, FN, KG, NS, BLOCKS>;
  static std::atomic<uint64_t> lds_set{0};
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), kLds, lds_set);
  if (e != hipSuccess) return e;
  kernel<<<grid_of(mt * nt), 64 * WM * WN * KG, kLds, s>>>(p, static_cast<int>(mt), static_cast<int>(nt));
  return hipGetLastError();
}

template <int WM, int WN, int FM, int FN>
static hipError_t launch_tiled(const Int8GemmParams& p, hipStream_t s) {
  constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN;
  constexpr int kLds = 2 * (BM + BN) * kStepBytes;
  const int64_t mt = (static_cast<int64_t>(p.M) + BM - 1) / BM, nt = (static_cast<int64_t>(p.N) + BN - 1) / BN;
  if (mt * nt > INT32_MAX) return hipErrorInvalidConfiguration;
  static std::atomic<uint64_t> lds_set{0};
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(int8_tiled_kernel<WM, WN, FM, FN>), kLds, lds_set);
  if (e != hipSuccess) return e;
  int8_tiled_kernel<WM, WN, FM, FN><<<grid_of(mt * nt), 64 * WM * WN, kLds, s>>>(
      p, static_cast<int>(mt), static_cast<int>(nt));
  return hipGetLastError();
}

template <typename T>
static void launch_token(const Int8GemmParams& p, const void* x, hipStream_t s) {
  // two blocks a CU; a wave takes several channels where there are more
  const unsigned blocks = static_cast<unsigned>(std::min((p.N + 7) / 8, 512));
  const size_t lds = static_cast<size_t>((p.K + 1023) / 1024 * 1024);
  if (p.K <= kLinearTokenMaxK / 4) int8_token_kernel<T, 2><<<blocks, kTokenThreads, lds, s>>>(p, x);
  else int8_token_kernel<T, 8><<<blocks, kTokenThreads, lds, s>>>(p, x);
}

// How long `tiles` take where `slots` run at once, in units of one round: the
// mean of the whole rounds and of the share of work, since the chip's CUs
// drift apart over several rounds.
static double rounds(int64_t tiles, int64_t slots) {
  const double t = static_cast<double>(tiles) / static_cast<double>(slots);
  return 0.5 * (static_cast<double>((tiles + slots - 1) / slots) + (t > 1.0 ? t : 1.0));
}

int choose_int8_kernel(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb) {
  if (M == 1 && K <= kLinearTokenMaxK) return 0;
  // Rows far apart: a tile's rows are addressed with 32-bit byte offsets, and
  // these tiles have the fewest.
  if (lda > kMaxTileLd || ldb > kMaxTileLd) return 2;
  // What a round of each tile takes, in microseconds: for each 128 bytes of K and
  // for the rest (first loads, sums, output), where every tile has a CU to itself
  // and (_full) where there are more tiles than CUs.  Fitted to 61 sizes of 17 to 16384 tokens;
  // on 70 others the choice costs 1% over the best of the eight in the mean (with
  // times for each 128 bytes alone 7% on the 61; 1340 x 7552 x 192 21.6 us for 13.5).
  static constexpr struct { int bm, bn, slots; double step, rest, step_full, rest_full; } kTiles[] = {
      {16, 16, 256, 0.026, 0.73, 0.051, 1.8},  {16, 32, 512, 0.05, 0.55, 0.13, 1.45},
      {32, 32, 512, 0.13, 0.6, 0.186, 1.95},   {64, 32, 256, 0.145, 1.45, 0.163, 2.6},
      {64, 64, 256, 0.226, 1.4, 0.262, 2.5},   {128, 128, 256, 0.58, 3.7, 0.66, 5.1},
      {128, 128, 512, 0.70, 1.4, 1.0, 3.5},    {256, 256, 256, 1.27, 5.3, 1.6, 5.3}};
  const double steps = static_cast<double>((K + kStepBytes - 1) / kStepBytes);
  double cost[std::size(kTiles)];
  for (size_t i = 0; i < std::size(kTiles); ++i) {
    const auto& t = kTiles[i];
    const int64_t tiles = ((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
    cost[i] = tiles <= 256 ? steps * t.step + t.rest : (steps * t.step_full + t.rest_full) * rounds(tiles, t.slots);
  }
  return 1 + static_cast<int>(std::min_element(std::begin(cost), std::end(cost)) - std::begin(cost));
}

hipError_t launch_int8_matmul(const Int8GemmParams& p, hipStream_t s) {
  switch (choose_int8_kernel(p.M, p.N, p.K, p.lda, p.ldb)) {
    case 0: launch_token<Codes>(p, nullptr, s); return hipGetLastError();
    case 1: return launch_ring<1, 1, 1, 1, 8, 4, 1>(p, s);
    case 2: return launch_ring<1, 1, 1, 2, 4, 3, 2>(p, s);
    case 3: return launch_ring<1, 1, 2, 2, 4, 2, 2>(p, s);
    case 4: return launch_ring<2, 1, 2, 2, 4, 3, 1>(p, s);
    case 5: return launch_ring<2, 2, 2, 2, 2, 4, 1>(p, s);
    case 6: return launch_ring<2, 2, 4, 4, 2, 2, 1>(p, s);
    case 7: return launch_ring<2, 4, 4, 2, 1, 2, 2>(p, s);
    default: return launch_tiled<2, 4, 8, 4>(p, s);
  }
}

template <typename T>
static void launch_few(const Int8GemmParams& p, const void* x, int64_t ldx, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>(std::min((static_cast<int64_t>(p.N) + 15) / 16, int64_t{512}));
  const dim3 grid(blocks, (p.M + 15) / 16);
  const size_t lds = static_cast<size_t>(std::min(p.M, 16)) * ((p.K + kStepBytes - 1) / kStepBytes * kStepBytes + 16);
  if (p.M > kFewWaves) int8_few_kernel<T, true><<<grid, kFewThreads, lds, s>>>(p, x, ldx);
  else int8_few_kernel<T, false><<<grid, kFewThreads, lds, s>>>(p, x, ldx);
}

hipError_t launch_int8_few(const Int8GemmParams& p, const void* x, int64_t ldx, int x_dtype, hipStream_t s) {
  if (x_dtype == MOE_BF16) launch_few<Bf16>(p, x, ldx, s);
  else if (x_dtype == MOE_F16) launch_few<F16>(p, x, ldx, s);
  else launch_few<F32>(p, x, ldx, s);
  return hipGetLastError();
}

hipError_t launch_int8_token(const Int8GemmParams& p, const void* x, int x_dtype, hipStream_t s) {
  if (x_dtype == MOE_BF16) launch_token<Bf16>(p, x, s);
  else if (x_dtype == MOE_F16) launch_token<F16>(p, x, s);
  else launch_token<F32>(p, x, s);
  return hipGetLastError();
}

}  // namespace nvfp4

// 8-bit integer linear product with scales for each token and channel (gfx950).
//
//   quantize: s = RN(amax / 127), q = RNE(x * RN(127 / amax)) of a row
//   product:  out[m, n] = sa[m] sb[n] sum_k a[m, k] b[n, k] + bias[n]
// The sum is exact in int32 for K < 2^31 / 128^2; it is converted to binary32
// once, scaled there and rounded once to the output's type.
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
    // |x inv| <= 127 (1 + 2^-23): the clamp only bounds a row with inf or NaN
    const int q = static_cast<int>(__builtin_amdgcn_fmed3f(__builtin_rintf(f[j] * inv), -127.0f, 127.0f));
    r[j / 4] |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * (j % 4));
  }
  return r;
}

template <typename T, bool VEC>
__device__ __forceinline__ void load_piece(float (&f)[8], const void* row, int64_t c, int64_t cols) {
  if constexpr (VEC) {
    Raw8<T> raw;
    load8<T>(raw, row, min(c, cols - 8));
    to_f32<T>(raw, f);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = T::get(row, min(c + j, cols - 1));
  }
}
// columns past the end count as 0
template <bool VEC>
__device__ __forceinline__ void clear_tail(float (&f)[8], int64_t c, int64_t cols) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if ((VEC ? c : c + j) >= cols) f[j] = 0.0f;
}

__device__ __forceinline__ float amax8(const float (&f)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
  return m;
}

}  // namespace

// TPR threads a row (64: four rows a block, 256: one), NC pieces of eight
// columns a thread, held in registers between the maximum and the codes, so
// that the row is read once.  The codes of a row end on a 16-byte piece,
// filled with zeros.
template <typename T, bool VEC, int TPR, int NC>
__global__ __launch_bounds__(256) void int8_quantize_kernel(const void* __restrict__ x, int64_t rows, int cols,
                                                            int64_t ld, int8_t* __restrict__ codes,
                                                            int64_t ld_codes, float* __restrict__ scales) {
  __shared__ float s_am[4];
  const int lt = threadIdx.x % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / TPR) + threadIdx.x / TPR;
  if (row >= rows) return;  // whole waves, and no barrier where a block holds several rows
  const void* xrow = static_cast<const char*>(x) + row * ld * T::kBytes;
  const int cols16 = (cols + 15) / 16 * 16;
  float f[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) load_piece<T, VEC>(f[i], xrow, 8 * (lt + TPR * i), cols);
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    clear_tail<VEC>(f[i], 8 * (lt + TPR * i), cols);
    am = fmaxf(am, amax8(f[i]));
  }
  am = wave_max(am);
  if constexpr (TPR > kWave) {
    if ((threadIdx.x & (kWave - 1)) == 0) s_am[threadIdx.x / kWave] = am;
    __syncthreads();
    am = fmaxf(fmaxf(s_am[0], s_am[1]), fmaxf(s_am[2], s_am[3]));
  }
  const bool some = am >= kMinAmax;
  const float inv = some ? 127.0f / am : 0.0f;
  int8_t* crow = codes + row * ld_codes;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = 8 * (lt + TPR * i);
    if (c < cols16) *reinterpret_cast<u32x2*>(crow + c) = pack_codes(f[i], inv);
  }
  if (lt == 0) scales[row] = some ? am / 127.0f : 1.0f;
}

// Longer rows: one block a row, two passes over it.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void int8_quantize_long_kernel(const void* __restrict__ x, int64_t cols,
                                                                 int64_t ld, int8_t* __restrict__ codes,
                                                                 int64_t ld_codes, float* __restrict__ scales) {
  __shared__ float s_am[4];
  const int64_t row = blockIdx.x;
  const void* xrow = static_cast<const char*>(x) + row * ld * T::kBytes;
  const int64_t cols16 = (cols + 15) / 16 * 16;
  float am = 0.0f;
  for (int64_t c = 8 * static_cast<int64_t>(threadIdx.x); c < cols; c += 8 * 256) {
    float f[8];
    load_piece<T, VEC>(f, xrow, c, cols);
    am = fmaxf(am, amax8(f));  // a column read twice changes no maximum
  }
  am = wave_max(am);
  if ((threadIdx.x & (kWave - 1)) == 0) s_am[threadIdx.x / kWave] = am;
  __syncthreads();
  am = fmaxf(fmaxf(s_am[0], s_am[1]), fmaxf(s_am[2], s_am[3]));
  const bool some = am >= kMinAmax;
  const float inv = some ? 127.0f / am : 0.0f;
  for (int64_t c = 8 * static_cast<int64_t>(threadIdx.x); c < cols16; c += 8 * 256) {
    float f[8];
    load_piece<T, VEC>(f, xrow, c, cols);
    clear_tail<VEC>(f, c, cols);
    *reinterpret_cast<u32x2*>(codes + row * ld_codes + c) = pack_codes(f, inv);
  }
  if (threadIdx.x == 0) scales[row] = some ? am / 127.0f : 1.0f;
}

template <typename T, bool VEC>
static void launch_quantize_width(const void* x, int64_t rows, int64_t cols, int64_t ld, int8_t* codes,
                                  int64_t ld_codes, float* scales, hipStream_t s) {
  const int64_t cols16 = (cols + 15) / 16 * 16;
  const int c = static_cast<int>(cols);
  const unsigned g1 = static_cast<unsigned>(rows), g4 = static_cast<unsigned>((rows + 3) / 4);
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
    int8_quantize_long_kernel<T, VEC><<<g1, 256, 0, s>>>(x, cols, ld, codes, ld_codes, scales);
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

// out[m, n] for n .. n + 3 (those below N) of token m.
__device__ __forceinline__ void store_scaled(const Int8GemmParams& p, int m, int n, const i32x4& acc) {
  const float sa = p.sa[m];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= p.N) break;
    float f = static_cast<float>(acc[i]) * (sa * p.sb[n + i]);
    if (p.bias) f += p.bias[n + i];
    const int64_t at = static_cast<int64_t>(m) * p.ldo + n + i;
    if (p.dtype == MOE_BF16) Bf16::put(p.out, at, f);
    else if (p.dtype == MOE_F16) F16::put(p.out, at, f);
    else F32::put(p.out, at, f);
  }
}

// 16 bytes of a row at column c, zero from column K on.  The row's last
// 16-byte piece lies inside its leading dimension.
__device__ __forceinline__ i32x4 load_k16(const int8_t* row, int c, int K) {
  i32x4 v = *reinterpret_cast<const i32x4*>(row + min(c, (K - 1) / 16 * 16));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int left = K - c - 4 * j;  // bytes of this dword before K
    if (left < 4) v[j] = left <= 0 ? 0 : v[j] & static_cast<int32_t>((1u << (8 * left)) - 1u);
  }
  return v;
}

// 16 channels by 16 MT tokens a block; its waves take K in steps of 128, every
// W-th step each, and add their sums through LDS.
template <int MT, int W>
__global__ __launch_bounds__(64 * W) void int8_stream_kernel(Int8GemmParams p) {
  __shared__ i32x4 s_acc[W > 1 ? W : 1][MT][kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int r = lane & 15, g = lane >> 4;
  const int nt = (p.N + 15) / 16;
  const int n0 = static_cast<int>(blockIdx.x % nt) * 16, m0 = static_cast<int>(blockIdx.x / nt) * (16 * MT);
  const int8_t* brow = p.b + static_cast<int64_t>(min(n0 + r, p.N - 1)) * p.ldb;
  const int8_t* arow[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) arow[t] = p.a + static_cast<int64_t>(min(m0 + 16 * t + r, p.M - 1)) * p.lda;
  i32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = i32x4{0, 0, 0, 0};
  const int full = p.K / 128;
  for (int s = wave; s < full; s += W) {
    const int c = 128 * s + 32 * g;
    const i32x4 b0 = *reinterpret_cast<const i32x4*>(brow + c), b1 = *reinterpret_cast<const i32x4*>(brow + c + 16);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const i32x4 a0 = *reinterpret_cast<const i32x4*>(arow[t] + c);
      const i32x4 a1 = *reinterpret_cast<const i32x4*>(arow[t] + c + 16);
      acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b0, a0, acc[t], 0, 0, 0);
      acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b1, a1, acc[t], 0, 0, 0);
    }
  }
  if (p.K % 128 != 0 && full % W == wave) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = 128 * full + 32 * g + 16 * h;
      const i32x4 b = load_k16(brow, c, p.K);
#pragma unroll
      for (int t = 0; t < MT; ++t)
        acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b, load_k16(arow[t], c, p.K), acc[t], 0, 0, 0);
    }
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int t = 0; t < MT; ++t) s_acc[wave][t][lane] = acc[t];
    __syncthreads();
    for (int t = wave; t < MT; t += W) {
      i32x4 sum = s_acc[0][t][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) sum += s_acc[w][t][lane];
      const int m = m0 + 16 * t + r;
      if (m < p.M) store_scaled(p, m, n0 + 4 * g, sum);
    }
  } else {
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int m = m0 + 16 * t + r;
      if (m < p.M) store_scaled(p, m, n0 + 4 * g, acc[t]);
    }
  }
}

hipError_t launch_int8_matmul(const Int8GemmParams& p, hipStream_t s) {
  const int64_t nt = (static_cast<int64_t>(p.N) + 15) / 16, mt = p.M <= 16 ? 1 : (static_cast<int64_t>(p.M) + 63) / 64;
  if (nt * mt > INT32_MAX) return hipErrorInvalidConfiguration;
  if (p.M <= 16) int8_stream_kernel<1, 4><<<static_cast<unsigned>(nt), 256, 0, s>>>(p);
  else int8_stream_kernel<4, 4><<<static_cast<unsigned>(nt * mt), 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace nvfp4

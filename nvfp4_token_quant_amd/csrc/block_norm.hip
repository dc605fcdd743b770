// Norms after and before a block with its gate and residual (gfx950).
//
//   r' = res_scale r + out_scale act(gate) N_after(y),   h = N_before(r')
//   N(v) = (v - mean) / sqrt(mean((v - mean)^2) + eps) * (weight + offset) + bias
// with mean = 0 for the RMS norm, act the identity or the sigmoid.  h is taken
// of the binary32 r', before r' is rounded to its own type.
//
// One pass: y, r and the gate are read once, r' and h written once (five
// values of T * H, which bound the kernel at large T).  A row stays in the
// registers of the threads that share it, as binary32; the statistics are
// two-step for the layer norm (mean, then squares of the differences), which
// binary32 needs where the mean is large against the spread.  All loads of a
// row, weights included, are issued before the first reduction, so that a
// single row (decode) waits for memory once.
#include "common.hpp"
#include "dtype.hpp"
#include "kernels.hpp"

namespace nvfp4 {

namespace {

__device__ __forceinline__ float wave_sum(float v) {
  v += __uint_as_float(dpp_u32<kDppXor1>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u32<kDppXor2>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u32<kDppHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u32<kDppMirror>(__float_as_uint(v)));
  uint32_t a, b;
  lane_pair<16>(__float_as_uint(v), a, b);
  v = __uint_as_float(a) + __uint_as_float(b);
  lane_pair<32>(__float_as_uint(v), a, b);
  return __uint_as_float(a) + __uint_as_float(b);
}

// Sum over the TPR threads of a row, the same in each of them.  buf: one LDS
// slot a wave, not used by another reduction of the kernel.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* buf) {
  v = wave_sum(v);
  if constexpr (TPR > kWave) {
    const int wave = threadIdx.x / kWave;
    if ((threadIdx.x & (kWave - 1)) == 0) buf[wave] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < TPR / kWave; ++w) v += buf[w];
  }
  return v;
}

// Eight consecutive values at column c of a row: VEC reads whole 16-byte
// pieces (cols a multiple of 8, rows 16-byte aligned), else one by one; 0 past
// the end, which every step below keeps 0.
template <typename T, bool VEC>
struct Piece {
  Raw8<T> raw;
  __device__ __forceinline__ void load(const void* row, int c, int cols) {
    if (c < cols) load8<T>(raw, row, c);
  }
  __device__ __forceinline__ void get(float (&f)[8], int c, int cols) const {
    to_f32<T>(raw, f);
    if (c >= cols) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    }
  }
};
template <typename T>
struct Piece<T, false> {
  float v[8];
  __device__ __forceinline__ void load(const void* row, int c, int cols) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < cols ? T::get(row, c + j) : 0.0f;
  }
  __device__ __forceinline__ void get(float (&f)[8], int, int) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = v[j];
  }
};

template <typename T>
__device__ __forceinline__ const void* row_at(const void* p, int64_t elements) {
  return static_cast<const char*>(p) + elements * T::kBytes;
}

// N(v) in place on the row's pieces.  w, b: the loaded weight and bias.
template <typename T, bool VEC, int TPR, int NC>
__device__ __forceinline__ void apply_norm(float (&v)[NC][8], const NormParams& n, const Piece<T, VEC> (&w)[NC],
                                           const Piece<T, VEC> (&b)[NC], int lt, int cols, float* buf0,
                                           float* buf1) {
  const float inv_n = 1.0f / static_cast<float>(cols);
  if (n.kind == MOE_NORM_LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[i][j];
    const float mean = row_sum<TPR>(s, buf0) * inv_n;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = 8 * (lt + TPR * i) + (VEC ? 0 : j);
        v[i][j] = c < cols ? v[i][j] - mean : 0.0f;
      }
  }
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) q = __builtin_fmaf(v[i][j], v[i][j], q);
  const float inv = 1.0f / sqrtf(row_sum<TPR>(q, buf1) * inv_n + n.eps);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = 8 * (lt + TPR * i);
    float f[8];
    if (n.weight) {
      w[i].get(f, c, cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= inv * (f[j] + n.offset);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= inv;
    }
    if (n.bias) {
      b[i].get(f, c, cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] += f[j];
    }
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void put_piece(void* row, int c, int cols, const float (&f)[8]) {
  if constexpr (VEC) {
    if (c < cols) store8<T>(row, c, f);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < cols) T::put(row, c + j, f[j]);
  }
}

}  // namespace

// TPR threads a row, NC pieces of eight columns a thread.
template <typename T, typename R, bool VEC, int TPR, int NC>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void block_norm_kernel(BlockNormParams p) {
  constexpr int kThreads = TPR > 256 ? TPR : 256;
  __shared__ float s_red[4][kThreads / kWave];
  const int lt = threadIdx.x % TPR;
  const int cols = p.cols;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
  if (row >= p.rows) return;  // whole waves, and no barrier where a block holds several rows

  Piece<R, VEC> pr[NC];
  Piece<T, VEC> py[NC], pg[NC], wa[NC], ba[NC], wb[NC], bb[NC];
  const void* rrow = row_at<R>(p.r, row * p.ld_r);
  const void* yrow = row_at<T>(p.y, p.y ? row * p.ld_y : 0);
  const void* grow = row_at<T>(p.gate, p.gate ? row * p.ld_gate : 0);
  const bool wide_gate = p.gate && p.gate_cols != 1;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = 8 * (lt + TPR * i);
    pr[i].load(rrow, c, cols);
    if (p.y) py[i].load(yrow, c, cols);
  }
  float g1 = p.gate && !wide_gate ? T::get(grow, 0) : 1.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = 8 * (lt + TPR * i);
    if (wide_gate) pg[i].load(grow, c, cols);
    if (p.after.weight) wa[i].load(p.after.weight, c, cols);
    if (p.after.bias) ba[i].load(p.after.bias, c, cols);
    if (p.before.weight) wb[i].load(p.before.weight, c, cols);
    if (p.before.bias) bb[i].load(p.before.bias, c, cols);
  }

  float v[NC][8];
  if (p.y) {
#pragma unroll
    for (int i = 0; i < NC; ++i) py[i].get(v[i], 8 * (lt + TPR * i), cols);
    if (p.after.kind >= 0)
      apply_norm<T, VEC, TPR, NC>(v, p.after, wa, ba, lt, cols, s_red[0], s_red[1]);
    if (p.gate && p.gate_sigmoid && !wide_gate) g1 = 1.0f / (1.0f + expf(-g1));
    g1 *= p.out_scale;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float f[8];
      pr[i].get(f, 8 * (lt + TPR * i), cols);
      if (wide_gate) {
        float g[8];
        pg[i].get(g, 8 * (lt + TPR * i), cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= p.gate_sigmoid ? 1.0f / (1.0f + expf(-g[j])) : g[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = p.res_scale * f[j] + g1 * v[i][j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      pr[i].get(v[i], 8 * (lt + TPR * i), cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= p.res_scale;
    }
  }
  if (p.r_out) {
    void* orow = static_cast<char*>(p.r_out) + row * p.ld_r_out * R::kBytes;
#pragma unroll
    for (int i = 0; i < NC; ++i) put_piece<R, VEC>(orow, 8 * (lt + TPR * i), cols, v[i]);
  }
  if (p.h) {
    apply_norm<T, VEC, TPR, NC>(v, p.before, wb, bb, lt, cols, s_red[2], s_red[3]);
    void* hrow = static_cast<char*>(p.h) + row * p.ld_h * T::kBytes;
#pragma unroll
    for (int i = 0; i < NC; ++i) put_piece<T, VEC>(hrow, 8 * (lt + TPR * i), cols, v[i]);
  }
}

template <typename T, typename R, bool VEC>
static void launch_norm_width(const BlockNormParams& p, hipStream_t s) {
  const auto grid = [&](int rows_per_block) {
    return static_cast<unsigned>((p.rows + rows_per_block - 1) / rows_per_block);
  };
  if (p.cols <= 512) block_norm_kernel<T, R, VEC, 64, 1><<<grid(4), 256, 0, s>>>(p);
  else if (p.cols <= 1024) block_norm_kernel<T, R, VEC, 64, 2><<<grid(4), 256, 0, s>>>(p);
  else if (p.cols <= 2048) block_norm_kernel<T, R, VEC, 256, 1><<<grid(1), 256, 0, s>>>(p);
  else if (p.cols <= 4096) block_norm_kernel<T, R, VEC, 256, 2><<<grid(1), 256, 0, s>>>(p);
  else if (p.cols <= 8192) block_norm_kernel<T, R, VEC, 256, 4><<<grid(1), 256, 0, s>>>(p);
  else if (p.cols <= 16384) block_norm_kernel<T, R, VEC, 1024, 2><<<grid(1), 1024, 0, s>>>(p);
  else if (p.cols <= 32768) block_norm_kernel<T, R, VEC, 1024, 4><<<grid(1), 1024, 0, s>>>(p);
  else block_norm_kernel<T, R, VEC, 1024, 8><<<grid(1), 1024, 0, s>>>(p);
}

template <typename T, typename R>
static void launch_norm_types(const BlockNormParams& p, bool vec, hipStream_t s) {
  if (vec) launch_norm_width<T, R, true>(p, s);
  else launch_norm_width<T, R, false>(p, s);
}

hipError_t launch_block_norm(const BlockNormParams& p, int dtype, int residual_dtype, bool vec, hipStream_t s) {
  if (dtype == MOE_F32) launch_norm_types<F32, F32>(p, vec, s);
  else if (dtype == MOE_BF16 && residual_dtype == MOE_F32) launch_norm_types<Bf16, F32>(p, vec, s);
  else if (dtype == MOE_BF16) launch_norm_types<Bf16, Bf16>(p, vec, s);
  else if (residual_dtype == MOE_F32) launch_norm_types<F16, F32>(p, vec, s);
  else launch_norm_types<F16, F16>(p, vec, s);
  return hipGetLastError();
}

}  // namespace nvfp4

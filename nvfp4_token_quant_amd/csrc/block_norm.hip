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
// single row (decode) waits for memory once.  16384 rows of 7168 (bf16, binary32
// residual) take 252 us, 5.6 TB/s; one row 3.8 us, most of it the launch, one
// trip to memory and the reductions.
#include "common.hpp"
#include "dtype.hpp"
#include "kernels.hpp"

namespace nvfp4 {

// Batches of at most this many rows give a row of 513 to 1024 columns two waves.
constexpr int kFewNormRows = 2048;

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
// slot a wave, not used by another reduction of the kernel.  Where a block
// holds several rows of more than a wave, every thread of it calls this.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* buf) {
  v = wave_sum(v);
  if constexpr (TPR > kWave) {
    const int wave = threadIdx.x / kWave;
    if ((threadIdx.x & (kWave - 1)) == 0) buf[wave] = v;
    __syncthreads();
    const float* row = buf + threadIdx.x / TPR * (TPR / kWave);
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < TPR / kWave; ++w) v += row[w];
  }
  return v;
}

// A thread's part of a row of T: NC pieces of eight consecutive columns, piece
// i at column 8 (lt + TPR i).  VEC: cols is a multiple of 8 and rows start at
// multiples of 16 bytes; else pieces are read at any address, and the first
// cols % 8 threads hold one column each of the rest.  Columns that a thread
// does not have are 0, and every step below keeps them 0.
template <bool VEC, int NC>
using Own = float[8 * NC + (VEC ? 0 : 1)];

template <typename T, bool VEC, int TPR, int NC>
struct Part {
  Raw8<T> piece[NC];
  float rest;
  template <bool ALIGNED>
  __device__ __forceinline__ void load_pieces(const void* row, int lt, int cols) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = 8 * (lt + TPR * i);
      if (c + 8 <= cols) {
        if constexpr (ALIGNED) load8<T>(piece[i], row, c);
        else load8_any<T>(piece[i], row, c);
      }
    }
  }
  __device__ __forceinline__ void load(const void* row, int lt, int cols) {
    load_pieces<VEC>(row, lt, cols);
    if (!VEC && lt < cols % 8) rest = T::get(row, cols / 8 * 8 + lt);
  }
  __device__ __forceinline__ void get(Own<VEC, NC>& f, int lt, int cols) const {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const bool own = 8 * (lt + TPR * i) + 8 <= cols;
      float v[8];
      to_f32<T>(piece[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[8 * i + j] = own ? v[j] : 0.0f;
    }
    if constexpr (!VEC) f[8 * NC] = lt < cols % 8 ? rest : 0.0f;
  }
};

template <typename T, bool VEC, int TPR, int NC>
__device__ __forceinline__ void put_part(void* row, int lt, int cols, const Own<VEC, NC>& f) {
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = 8 * (lt + TPR * i);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = f[8 * i + j];
    if (c + 8 <= cols) {
      if constexpr (VEC) store8<T>(row, c, v);
      else store8_any<T>(row, c, v);
    }
  }
  if constexpr (!VEC) {
    if (lt < cols % 8) T::put(row, cols / 8 * 8 + lt, f[8 * NC]);
  }
}

template <typename T>
__device__ __forceinline__ const void* row_at(const void* p, int64_t elements) {
  return static_cast<const char*>(p) + elements * T::kBytes;
}

// Up to two pieces a thread, everything a row needs is loaded before its first
// reduction (binary32: with two pieces the weights, for which the registers do
// not reach, where they are used: two rows of 15331 columns 7.2 us, else 10.0).
// With more the registers hold the row, and the rest is loaded where it is used:
// two pieces at a time where all of them would spill (1024 rows of 65536 bf16, eight
// pieces: 294 us, all at a time 516; four pieces of bf16 together are 5% faster
// than two).
template <int NC>
constexpr bool kRowFirst = NC <= 2;
template <typename T, int NC>
constexpr bool kWeightsFirst = NC * T::kBytes <= 4;

// f(j, x) for each of a thread's columns j with its value x: of a loaded part,
// or of a row.
template <bool LOADED, typename T, bool VEC, int TPR, int NC, typename F>
__device__ __forceinline__ void with_part(const Part<T, VEC, TPR, NC>& part, const void* row, int lt, int cols, F f) {
  constexpr int N = 8 * NC + (VEC ? 0 : 1);
  if constexpr (LOADED) {
    float x[N];
    part.get(x, lt, cols);
#pragma unroll
    for (int j = 0; j < N; ++j) f(j, x[j]);
  } else {
    constexpr int kTogether = NC * T::kBytes > 8 ? 2 : NC;
    Part<T, true, TPR, kTogether> some;
#pragma unroll
    for (int i = 0; i < NC; i += kTogether) {
      float x[8 * kTogether];
      some.template load_pieces<VEC>(row, lt + TPR * i, cols);
      some.get(x, lt + TPR * i, cols);
#pragma unroll
      for (int j = 0; j < 8 * kTogether; ++j) f(8 * i + j, x[j]);
      if constexpr (NC > kTogether) __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (!VEC) f(8 * NC, lt < cols % 8 ? T::get(row, cols / 8 * 8 + lt) : 0.0f);
  }
}

// N(v) in place.  w, b: the loaded weight and bias (kWeightsFirst).
template <typename T, bool VEC, int TPR, int NC>
__device__ __forceinline__ void apply_norm(Own<VEC, NC>& v, const NormParams& n,
                                           Part<T, VEC, TPR, NC>& w, Part<T, VEC, TPR, NC>& b, int lt, int cols,
                                           float* buf0, float* buf1) {
  constexpr int N = 8 * NC + (VEC ? 0 : 1);
  const float inv_n = 1.0f / static_cast<float>(cols);
  if (n.kind == MOE_NORM_LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) s += v[j];
    const float mean = row_sum<TPR>(s, buf0) * inv_n;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const bool own = j < 8 * NC ? 8 * (lt + TPR * (j / 8)) + 8 <= cols : lt < cols % 8;
      v[j] = own ? v[j] - mean : 0.0f;
    }
  }
  float q = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) q = __builtin_fmaf(v[j], v[j], q);
  const float inv = 1.0f / sqrtf(row_sum<TPR>(q, buf1) * inv_n + n.eps);
  constexpr bool kLoaded = kWeightsFirst<T, NC>;
  if (n.weight) {
    with_part<kLoaded>(w, n.weight, lt, cols, [&](int j, float x) { v[j] *= inv * (x + n.offset); });
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] *= inv;
  }
  if (n.bias) with_part<kLoaded>(b, n.bias, lt, cols, [&](int j, float x) { v[j] += x; });
}

__device__ __forceinline__ float sigmoid32(float g) { return 1.0f / (1.0f + expf(-g)); }

}  // namespace

// TPR threads a row, NC pieces of eight columns a thread.
template <typename T, typename R, bool VEC, int TPR, int NC>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void block_norm_kernel(BlockNormParams p) {
  constexpr int kThreads = TPR > 256 ? TPR : 256;
  constexpr int N = 8 * NC + (VEC ? 0 : 1);
  __shared__ float s_red[4][kThreads / kWave];
  const int lt = threadIdx.x % TPR;
  const int cols = p.cols;
  const int64_t row_own = block_id() * (kThreads / TPR) + threadIdx.x / TPR;
  const bool active = row_own < p.rows;
  const int64_t row = active ? row_own : p.rows - 1;  // past the end: the last row again, not stored

  Part<R, VEC, TPR, NC> pr;
  Part<T, VEC, TPR, NC> py, pg, wa, ba, wb, bb;
  const void* grow = row_at<T>(p.gate, p.gate ? row * p.ld_gate : 0);
  const bool wide_gate = p.gate && p.gate_cols != 1;
  const void* rrow = row_at<R>(p.r, row * p.ld_r);
  if (kRowFirst<NC> || !p.y) pr.load(rrow, lt, cols);
  if (p.y) py.load(row_at<T>(p.y, row * p.ld_y), lt, cols);
  float g1 = p.gate && !wide_gate ? T::get(grow, 0) : 1.0f;
  if (kRowFirst<NC> && wide_gate) pg.load(grow, lt, cols);
  if constexpr (kWeightsFirst<T, NC>) {
    if (p.after.weight) wa.load(p.after.weight, lt, cols);
    if (p.after.bias) ba.load(p.after.bias, lt, cols);
    if (p.before.weight) wb.load(p.before.weight, lt, cols);
    if (p.before.bias) bb.load(p.before.bias, lt, cols);
  }

  float v[N];
  if (p.y) {
    py.get(v, lt, cols);
    if (p.after.kind >= 0) apply_norm<T, VEC, TPR, NC>(v, p.after, wa, ba, lt, cols, s_red[0], s_red[1]);
    if (p.gate && p.gate_sigmoid && !wide_gate) g1 = sigmoid32(g1);
    g1 *= p.out_scale;
    if (wide_gate)
      with_part<kRowFirst<NC>>(pg, grow, lt, cols,
                               [&](int j, float x) { v[j] *= p.gate_sigmoid ? sigmoid32(x) : x; });
    with_part<kRowFirst<NC>>(pr, rrow, lt, cols, [&](int j, float x) { v[j] = p.res_scale * x + g1 * v[j]; });
  } else {
    pr.get(v, lt, cols);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] *= p.res_scale;
  }
  if (p.r_out && active)
    put_part<R, VEC, TPR, NC>(static_cast<char*>(p.r_out) + row * p.ld_r_out * R::kBytes, lt, cols, v);
  if (p.h) {
    apply_norm<T, VEC, TPR, NC>(v, p.before, wb, bb, lt, cols, s_red[2], s_red[3]);
    if (active) put_part<T, VEC, TPR, NC>(static_cast<char*>(p.h) + row * p.ld_h * T::kBytes, lt, cols, v);
  }
}

template <typename T, typename R, bool VEC, int TPR, int NC>
static void launch_norm_shape(const BlockNormParams& p, hipStream_t s) {
  constexpr int kThreads = TPR > 256 ? TPR : 256;
  constexpr int kRows = kThreads / TPR;
  block_norm_kernel<T, R, VEC, TPR, NC><<<grid_of((p.rows + kRows - 1) / kRows), kThreads, 0, s>>>(p);
}

// One piece a thread up to 8192 columns: the shortest chain for a single row
// (7168 columns: 3.8 us with 1024 threads, 4.5 with 256 of four pieces) and as
// fast with many (16384 rows: 252 and 257 us).  Narrow rows share a block; in
// large batches a wave takes one of up to 1024 columns by itself, without a
// barrier (RMS, bf16, 1024 columns: 3000 rows 6.3 us, with two waves a row 6.9;
// 4096 8.0 and 8.7; 512 3.6 and 3.5.  Layer norms, binary32, 1001 columns with an
// element gate: 1027 rows 8.2 and 7.2, 4096 19.2 and 18.1, from memory 23.2 and
// 22.9).
template <typename T, typename R, bool VEC>
static void launch_norm_width(const BlockNormParams& p, hipStream_t s) {
  const int w = p.cols;
  if (w <= 512) launch_norm_shape<T, R, VEC, 64, 1>(p, s);
  else if (w <= 1024 && p.rows <= kFewNormRows) launch_norm_shape<T, R, VEC, 128, 1>(p, s);
  else if (w <= 1024) launch_norm_shape<T, R, VEC, 64, 2>(p, s);
  else if (w <= 2048) launch_norm_shape<T, R, VEC, 256, 1>(p, s);
  else if (w <= 4096) launch_norm_shape<T, R, VEC, 512, 1>(p, s);
  else if (w <= 8192) launch_norm_shape<T, R, VEC, 1024, 1>(p, s);
  else if (w <= 16384) launch_norm_shape<T, R, VEC, 1024, 2>(p, s);
  else if (w <= 32768) launch_norm_shape<T, R, VEC, 1024, 4>(p, s);
  else launch_norm_shape<T, R, VEC, 1024, 8>(p, s);
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

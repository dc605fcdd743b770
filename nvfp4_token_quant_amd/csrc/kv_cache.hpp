// The key-value cache in 8 bits: its layout, the entries of a batch, and how a
// block of a kernel finds its share of a ragged batch.
//
// A page holds P tokens of a sequence for every kv head: codes and one scale for
// the keys, codes and one scale for the values.  The tokens of a sequence's last,
// incomplete page are its tail: 16-bit values with a power of two for each token
// and head, in the sequence's slot.
//
// Codes and tails are laid out in the fragments of the 16 x 16 x 32 matrix
// instruction, so that a wave reads whole 1 KB pieces and moves no data between
// lanes.  A unit is 16 tokens x 64 channels, lane l's 16 codes together, the units
// of a page and head ordered [P / 16][D / 64].  With n = token % 16 and c = channel % 64:
//   keys    lane n + 16 (c / 16), code c % 16: the score product contracts channels,
//           and each of its two instructions a unit takes eight consecutive ones
//   values  lane c % 16 + 16 (n / 4), code 4 (c / 16) + n % 4: the output product
//           contracts tokens, in the order in which the score product leaves
//           them in the registers (four consecutive ones a lane)
// A code is kept plus 128: 0x6400 | byte is the fp16 number 1024 + byte, and one
// packed subtraction makes two codes exact fp16 operands.  In a tail the same units
// are two pieces of 64 lanes x 8 fp16 values: keys' channels c % 16 / 8 = 0 and 1,
// values' c / 32 = 0 and 1.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "dtype.hpp"

namespace nvfp4 {

struct KvParams {
  uint8_t* codes;      // [pages][2][kv heads][P D], keys then values
  float* scales;       // [pages][2][kv heads]
  _Float16* tails;     // [slots][2][kv heads][P D]
  float* tail_scales;  // [slots][2][kv heads][P]
  int64_t pages, slots;
  const int32_t* table;  // [entries, ld_table]
  const int32_t* lens;   // [entries]
  const int32_t* slot;   // [entries]
  const int32_t* cu;     // [entries + 1], or NULL: one token an entry
  int64_t ld_table;
  int width, entries, tokens;
  int heads, D, P, shift;  // kv heads; P = 1 << shift
};

// A tile of rows whose keys were cut into pieces: its rows, and where the pieces'
// sums are (slot, slot + stride, ...).
struct KvJoin {
  int first, row, rows, head, slot, pieces, stride, pad;
};

struct KvAttention {
  KvParams c;
  const void* q;
  void* out;
  int64_t ldq, ldq_head, ldo, ldo_head;
  float scale;
  int group, window, dtype;
};

// kv_cache.hip.  Blocks of an append or a read (host: they have to fit a launch).
int64_t kv_page_blocks(const KvParams& p);
hipError_t launch_kv_append(const KvParams& c, const void* k, int64_t ld_k, int64_t ld_k_head, const void* v,
                            int64_t ld_v, int64_t ld_v_head, int dtype, hipStream_t s);
hipError_t launch_kv_read(const KvParams& c, void* k, void* v, int dtype, hipStream_t s);
hipError_t launch_kv_fork(const KvParams& c, const int32_t* src, const int32_t* dst, int pairs, hipStream_t s);
// kv_attention.hip.  Bytes of the workspace, and the largest launch's blocks.
int64_t kv_attention_bytes(const KvParams& p, int group, int64_t* blocks);
hipError_t launch_kv_attention(const KvAttention& k, void* workspace, hipStream_t s);

// What a call sees of a batch's entry: n tokens behind the `len` that the sequence
// had, the first of them the call's token `first`; n = 0 for a padding entry
// (slot or length negative) and for one whose numbers lie outside the call's tensors.
struct KvEntry {
  int len, n, first, slot;
  __device__ int total() const { return len + n; }
};

__device__ __forceinline__ KvEntry kv_entry(const KvParams& p, int i) {
  KvEntry e;
  e.first = p.cu ? p.cu[i] : i;
  e.n = p.cu ? p.cu[i + 1] - e.first : 1;
  e.len = p.lens[i];
  e.slot = p.slot[i];
  const int room = p.width << p.shift;
  if (e.first < 0 || e.first > p.tokens || e.len < 0 || e.len > room || e.slot < 0 || e.slot >= p.slots) {
    e.first = e.len = e.slot = e.n = 0;
  }
  e.n = max(0, min(e.n, min(p.tokens - e.first, room - e.len)));
  return e;
}

// The page of an entry's table, -1 if it is none of the cache's.
__device__ __forceinline__ int kv_page(const KvParams& p, int entry, int number) {
  const int id = p.table[entry * p.ld_table + number];
  return id >= 0 && id < p.pages ? id : -1;
}

__device__ __forceinline__ int64_t kv_page_at(const KvParams& p, int64_t id, int which, int head) {
  return (id * 2 + which) * p.heads + head;
}

// fp16 operands of 8 codes (two dwords): 1024 + byte, less 1152.
__device__ __forceinline__ half8 kv_codes8(uint32_t a, uint32_t b) {
  const half2v bias = {static_cast<_Float16>(-1152.0f), static_cast<_Float16>(-1152.0f)};
  const half2v r0 = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, a, 0x04010400u)) + bias;
  const half2v r1 = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u)) + bias;
  const half2v r2 = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u)) + bias;
  const half2v r3 = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u)) + bias;
  return half8{r0[0], r0[1], r1[0], r1[1], r2[0], r2[1], r3[0], r3[1]};
}

__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {  // sum over the lanes up to this one
  v += __builtin_amdgcn_update_dpp(0u, v, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0u, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0u, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0u, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0u, v, 0x142, 0xA, 0xF, false);  // lane 15 and 47 of the row before
  v += __builtin_amdgcn_update_dpp(0u, v, 0x143, 0xC, 0xF, false);  // lane 31
  return v;
}

// Sum over the block's threads up to and including this one (`total`: over all).
// buf: one slot a wave; every thread calls it, and a barrier stands between two calls
// that use the same buf.
template <int THREADS>
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* buf, uint64_t& total) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const uint64_t up = __shfl_up(v, d);
    if (lane >= d) v += up;
  }
  if (lane == kWave - 1) buf[wave] = v;
  __syncthreads();
  uint64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / kWave; ++w) {
    if (w < wave) before += buf[w];
    total += buf[w];
  }
  return before + v;
}

// Pages that an entry's tokens fall on.
__device__ __forceinline__ int kv_touched(const KvParams& p, const KvEntry& e) {
  return e.n > 0 ? ((e.total() - 1) >> p.shift) - (e.len >> p.shift) + 1 : 0;
}

}  // namespace nvfp4

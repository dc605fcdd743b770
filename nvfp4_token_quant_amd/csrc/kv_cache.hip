// New tokens into the key-value cache, cached tokens back as values, and a
// sequence that continues another one (gfx950).  Layout: kv_cache.hpp.
//
// A page of a head is quantized once, from the values as they came, when its last
// token arrives: s = RN(amax / 127), q = RNE(RN(x RN(127 / amax))).  A full page
// never changes, so sequences share it, and what the cache holds does not depend
// on how the tokens came.
//
// One block takes the keys or the values of one page and head, as pieces of 4
// tokens x 8 channels a thread: rows are read and written in 16-byte pieces, and
// four tokens of a channel are one dword of the values' order.  Codes pass
// through LDS, so that a page leaves in whole 16-byte pieces too.  Bound by memory where
// there is enough of it: prompts of 4 x 8192 tokens (8 heads, D = 128, pages of 64) 56 us, 3.6
// TB/s with two trips to memory a block (five blocks a CU; six or eight, which spill, 57
// and 86), read back in 35 us, 5.8 TB/s; a decode batch of 64 sequences 5.7 and 5.0 us, of which a
// launch that does nothing takes 2.6.
#include "kernels.hpp"
#include "kv_cache.hpp"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

// (by value: a bit cast of a vector's element in place gives its first one)
__device__ __forceinline__ half2v half2_of(uint32_t w) { return __builtin_bit_cast(half2v, w); }

// The entry and the number of its touched page of a block (entry -1: none).
__device__ __forceinline__ int find_page(const KvParams& p, int index, KvEntry& e, int& number) {
  __shared__ uint64_t buf[kThreads / kWave];
  __shared__ int found[2];
  if (!p.cu) {
    e = kv_entry(p, index);
    number = e.len >> p.shift;
    return e.n > 0 ? index : -1;
  }
  if (p.entries <= 4 * kWave) {
    // every wave finds it by itself, up to four entries a lane, without a barrier
    const int lane = threadIdx.x & (kWave - 1), per = (p.entries + kWave - 1) / kWave;
    KvEntry x[4];
    uint32_t c[4], own = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = lane * per + k;
      x[k] = KvEntry{};
      if (k < per && i < p.entries) x[k] = kv_entry(p, i);
      c[k] = static_cast<uint32_t>(kv_touched(p, x[k]));
      own += c[k];
    }
    uint32_t in = static_cast<uint32_t>(index) - (wave_scan(own) - own);
    const uint64_t here = __ballot(in < own);
    if (!here) return -1;
    const int from = __builtin_ctzll(here);
    int mine = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (mine == k && in >= c[k]) {
        in -= c[k];
        mine = k + 1;
      }
#pragma unroll
    for (int k = 1; k < 4; ++k)
      if (mine == k) x[0] = x[k];
    e.len = __builtin_amdgcn_readlane(x[0].len, from);
    e.n = __builtin_amdgcn_readlane(x[0].n, from);
    e.first = __builtin_amdgcn_readlane(x[0].first, from);
    e.slot = __builtin_amdgcn_readlane(x[0].slot, from);
    number = (e.len >> p.shift) + __builtin_amdgcn_readlane(static_cast<int>(in), from);
    return from * per + __builtin_amdgcn_readlane(mine, from);
  }
  if (threadIdx.x == 0) found[0] = -1;
  const int per = (p.entries + kThreads - 1) / kThreads;
  const int a = threadIdx.x * per, b = min(a + per, p.entries);
  uint64_t own = 0, total;
  for (int i = a; i < b; ++i) own += kv_touched(p, kv_entry(p, i));
  uint64_t at = block_scan<kThreads>(own, buf, total) - own;  // (its barrier orders found[0] too)
  const uint64_t want = index;
  if (want >= at && want < at + own) {
    for (int i = a; i < b; ++i) {
      const int c = kv_touched(p, kv_entry(p, i));
      if (want < at + c) {
        found[0] = i;
        found[1] = static_cast<int>(want - at);
        break;
      }
      at += c;
    }
  }
  __syncthreads();
  const int i = __builtin_amdgcn_readfirstlane(found[0]);
  if (i < 0) return -1;
  e = kv_entry(p, i);
  number = (e.len >> p.shift) + __builtin_amdgcn_readfirstlane(found[1]);
  return i;
}

// A value of the tail: fp16 times the token's power of two.
__device__ __forceinline__ const char* tail_base(const KvParams& p, int slot, int which, int head) {
  return reinterpret_cast<const char*>(p.tails + kv_page_at(p, slot, which, head) * p.P * p.D);
}
// Bytes from a tail's start to the 8 channels from d (a multiple of 8) of a key, and
// to a channel of four tokens from t (a multiple of 4) of the values.
__device__ __forceinline__ int tail_key_at(int t, int d, int D) {
  return ((t / 16 * (D / 64) + d / 64) * 2 + d % 16 / 8) * 1024 + (t % 16 + 16 * (d % 64 / 16)) * 16;
}
__device__ __forceinline__ int tail_value_at(int t, int d, int D) {
  return ((t / 16 * (D / 64) + d / 64) * 2 + d % 64 / 32) * 1024 + (d % 16 + 16 * (t % 16 / 4)) * 16 + d % 32 / 16 * 8;
}
// The same for codes: 8 channels of a key, four tokens of a channel of the values.
__device__ __forceinline__ int code_key_at(int t, int d, int D) {
  return (t / 16 * (D / 64) + d / 64) * 1024 + (t % 16 + 16 * (d % 64 / 16)) * 16 + d % 16;
}
__device__ __forceinline__ int code_value_at(int t, int d, int D) {
  return (t / 16 * (D / 64) + d / 64) * 1024 + (d % 16 + 16 * (t % 16 / 4)) * 16 + d % 64 / 16 * 4;
}

// The tail's tokens t .. t + 3, channels d .. d + 7, as T's bits.  Only those with
// bit j of `mine` set are read.
template <typename T>
__device__ __forceinline__ void load_tail(const KvParams& p, int slot, int which, int head, int t, int d, int mine,
                                          u32x4 (&x)[4]) {
  const char* base = tail_base(p, slot, which, head);
  const float* scale = p.tail_scales + kv_page_at(p, slot, which, head) * p.P + t;
  half2v v[4][4];
  if (which == 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x4 w = mine >> j & 1 ? *reinterpret_cast<const u32x4*>(base + tail_key_at(t + j, d, p.D)) : u32x4{};
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = half2_of(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(base + tail_value_at(t, d + i, p.D));
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j][i / 2][i % 2] = half2_of(w[j / 2])[j % 2];
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!(mine >> j & 1)) continue;
    const float s = scale[j];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[j][i] = T::bits(static_cast<float>(v[j][i][0]) * s) | (T::bits(static_cast<float>(v[j][i][1]) * s) << 16);
  }
}

// The largest magnitude's bits (a NaN's or an infinity's are above every finite number's).
template <typename T>
__device__ __forceinline__ uint32_t top_bits(const u32x4& x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    T::unpack(x[i], a, b);
    m = max(m, max(__float_as_uint(a) & 0x7fffffffu, __float_as_uint(b) & 0x7fffffffu));
  }
  return m;
}

constexpr uint32_t kInfBits = 0x7f800000u;

// k, v: the new tokens, rows ld_token apart, heads ld_head.
struct AppendParams {
  KvParams c;
  const void* x[2];
  int64_t ld_token[2], ld_head[2];
};

// IT: pieces of 4 tokens x 8 channels a thread.
template <typename T, int IT>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(AppendParams a) {
  const KvParams& p = a.c;
  __shared__ uint32_t token_top[128];
  __shared__ uint32_t page_top;
  extern __shared__ __align__(16) uint8_t staged[];
  const int head = blockIdx.x % p.heads, which = blockIdx.x / p.heads % 2;
  KvEntry e;
  int number;
  const int entry = find_page(p, blockIdx.x / p.heads / 2, e, number);
  if (entry < 0) return;
  const int D = p.D, P = p.P, chunks = D / 8, tid = threadIdx.x;
  const int first_page = e.len >> p.shift;
  int start = number << p.shift;
  bool full = e.total() - start >= P;
  // The block that completes a tail also starts the next one in its place, behind
  // its own reads; the last page's block has nothing left to do.
  const bool older = (e.len & (P - 1)) != 0 && e.total() >> p.shift > first_page;
  if (older && !full) return;

  // every piece's tokens: of the call (new) or of the tail (behind a full page's start)
  u32x4 x[IT][4];
  const char* rows = static_cast<const char*>(a.x[which]) + head * a.ld_head[which] * 2;
  auto load = [&](int it) {
    const int piece = tid + it * kThreads, t = piece / chunks * 4, d = piece % chunks * 8;
    if (t >= P) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int pos = start + t + j;
      x[it][j] = u32x4{};
      if (pos >= e.len && pos < e.total())
        x[it][j] = *reinterpret_cast<const u32x4*>(rows + ((e.first + pos - e.len) * a.ld_token[which] + d) * 2);
    }
    if (full) {
      const int behind = e.len - start - t;  // tokens of the tail among the four
      if (behind > 0) load_tail<T>(p, e.slot, which, head, t, d, (1 << min(behind, 4)) - 1, x[it]);
    }
  };
#pragma unroll
  for (int it = 0; it < IT; ++it) load(it);

  if (full) {
    if (tid == 0) page_top = 0;
    uint32_t top = 0;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      if ((tid + it * kThreads) / chunks * 4 >= P) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, top_bits<T>(x[it][j]));
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
    __syncthreads();
    if (tid % kWave == 0) atomicMax(&page_top, top);
    __syncthreads();
    const uint32_t bits = page_top;
    const float amax = __uint_as_float(bits);
    const bool some = bits < kInfBits && amax >= 0x1p-119f;
    const float scale = bits >= kInfBits ? __uint_as_float(0x7fc00000u) : some ? amax / 127.0f : 0.0f;
    const float inv = some ? 127.0f / amax : 0.0f;
    const int page = kv_page(p, entry, number);
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int piece = tid + it * kThreads, t = piece / chunks * 4, d = piece % chunks * 8;
      if (t >= P) continue;
      uint32_t q[4][8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float u, v;
          T::unpack(x[it][j][i], u, v);
          q[j][2 * i] = some ? static_cast<int>(rintf(u * inv)) + 128 : 128;
          q[j][2 * i + 1] = some ? static_cast<int>(rintf(v * inv)) + 128 : 128;
        }
      }
      if (which == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x2 w = {q[j][0] | q[j][1] << 8 | q[j][2] << 16 | q[j][3] << 24,
                           q[j][4] | q[j][5] << 8 | q[j][6] << 16 | q[j][7] << 24};
          *reinterpret_cast<u32x2*>(staged + code_key_at(t + j, d, D)) = w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint32_t*>(staged + code_value_at(t, d + i, D)) =
              q[0][i] | q[1][i] << 8 | q[2][i] << 16 | q[3][i] << 24;
      }
    }
    __syncthreads();
    if (page >= 0) {
      const int64_t at = kv_page_at(p, page, which, head);
      u32x4* to = reinterpret_cast<u32x4*>(p.codes + at * P * D);
      for (int i = tid; i < P * D / 16; i += kThreads) to[i] = reinterpret_cast<const u32x4*>(staged)[i];
      if (tid == 0) p.scales[at] = scale;
    }
    if (!older || number != first_page) return;
    // the sequence's new tail, if it has one, in place of the one that was read
    start = e.total() >> p.shift << p.shift;
    if (start == e.total()) return;
    full = false;
#pragma unroll
    for (int it = 0; it < IT; ++it) load(it);
  }

  // Tokens that stay in the tail: the power of two of each from its largest channel,
  // so that the largest lies in [2^14, 2^15) and every value of T's precision within
  // 2^29 of it is exact.
  if (tid < P) token_top[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int t = (tid + it * kThreads) / chunks * 4;
    if (t >= P) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int pos = start + t + j;
      if (pos >= e.len && pos < e.total()) atomicMax(&token_top[t + j], top_bits<T>(x[it][j]));
    }
  }
  __syncthreads();
  char* base = const_cast<char*>(tail_base(p, e.slot, which, head));
  const int64_t at = kv_page_at(p, e.slot, which, head);
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int piece = tid + it * kThreads, t = piece / chunks * 4, d = piece % chunks * 8;
    if (t >= P) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int pos = start + t + j;
      if (pos < e.len || pos >= e.total()) continue;
      const uint32_t top = token_top[t + j];
      const bool some = top != 0 && top < kInfBits;
      const int exp = max(static_cast<int>(top >> 23) - 127 - 14, -126);  // (a subnormal's field is 0)
      const float inv = some ? __uint_as_float(static_cast<uint32_t>(127 - exp) << 23) : 0.0f;
      _Float16 h[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float u, v;
        T::unpack(x[it][j][i], u, v);
        h[2 * i] = static_cast<_Float16>(some ? u * inv : 0.0f);
        h[2 * i + 1] = static_cast<_Float16>(some ? v * inv : 0.0f);
      }
      if (which == 0) {
        *reinterpret_cast<half8*>(base + tail_key_at(t + j, d, D)) = half8{h[0], h[1], h[2], h[3], h[4], h[5], h[6], h[7]};
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) *reinterpret_cast<_Float16*>(base + tail_value_at(t, d + i, D) + 2 * j) = h[i];
      }
      if (d == 0)
        p.tail_scales[at * P + t + j] = top >= kInfBits ? __uint_as_float(0x7fc00000u)
                                        : some          ? __uint_as_float(static_cast<uint32_t>(exp + 127) << 23)
                                                        : 0.0f;
    }
  }
}

struct ReadParams {
  KvParams c;
  void* out[2];  // [tokens, heads, D]
};

template <typename T>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(ReadParams a) {
  const KvParams& p = a.c;
  const int head = blockIdx.x % p.heads, which = blockIdx.x / p.heads % 2;
  KvEntry e;
  int number;
  const int entry = find_page(p, blockIdx.x / p.heads / 2, e, number);
  if (entry < 0) return;
  const int D = p.D, P = p.P, chunks = D / 8, start = number << p.shift;
  const bool full = e.total() - start >= P;
  const int page = full ? kv_page(p, entry, number) : -1;
  const int64_t at = kv_page_at(p, full ? max(page, 0) : e.slot, which, head);
  const uint8_t* codes = p.codes + at * P * D;
  const float page_scale = full && page >= 0 ? p.scales[at] : 0.0f;
  for (int piece = threadIdx.x; piece < P / 4 * chunks; piece += kThreads) {
    const int t = piece / chunks * 4, d = piece % chunks * 8;
    float v[4][8];
    if (start + t + 4 <= e.len || start + t >= e.total()) continue;
    if (full) {
      if (which == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(codes + code_key_at(t + j, d, D));
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[j][i] = static_cast<float>(static_cast<int>(w[i / 4] >> 8 * (i % 4) & 255) - 128) * page_scale;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + code_value_at(t, d + i, D));
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j][i] = static_cast<float>(static_cast<int>(w >> 8 * j & 255) - 128) * page_scale;
        }
      }
    } else {
      const char* base = tail_base(p, e.slot, which, head);
      if (which == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const half8 w = *reinterpret_cast<const half8*>(base + tail_key_at(t + j, d, D));
          const float s = p.tail_scales[at * P + t + j];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] = static_cast<float>(w[i]) * s;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(base + tail_value_at(t, d + i, D));
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[j][i] = static_cast<float>(half2_of(w[j / 2])[j % 2]) * p.tail_scales[at * P + t + j];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int pos = start + t + j;
      if (pos < e.len || pos >= e.total()) continue;
      store8<T>(a.out[which], (static_cast<int64_t>(e.first + pos - e.len) * p.heads + head) * D + d, v[j]);
    }
  }
}

struct ForkParams {
  KvParams c;  // (lens and table are written)
  const int32_t *src, *dst;
};

// A pair's first block writes the table row and the length; the others copy the tail of
// one head's keys or values, in whole blocks of 16 tokens.
__global__ __launch_bounds__(kThreads) void kv_fork_kernel(ForkParams a) {
  const KvParams& p = a.c;
  const int parts = 1 + 2 * p.heads, pair = blockIdx.x / parts, part = blockIdx.x % parts;
  const int from = a.src[pair], to = a.dst[pair];
  if (from < 0 || from >= p.entries || to < 0 || to >= p.entries || from == to) return;
  const int len = p.lens[from], a_slot = p.slot[from], b_slot = p.slot[to];
  if (len < 0 || len > p.width << p.shift) return;
  if (part == 0) {
    int32_t* rows = const_cast<int32_t*>(p.table);
    for (int i = threadIdx.x; i < len >> p.shift; i += kThreads) rows[to * p.ld_table + i] = rows[from * p.ld_table + i];
    if (threadIdx.x == 0) const_cast<int32_t*>(p.lens)[to] = len;
    return;
  }
  const int tail = len & (p.P - 1);
  if (!tail || a_slot < 0 || a_slot >= p.slots || b_slot < 0 || b_slot >= p.slots || a_slot == b_slot) return;
  const int head = (part - 1) % p.heads, which = (part - 1) / p.heads;
  const int64_t x = kv_page_at(p, a_slot, which, head), y = kv_page_at(p, b_slot, which, head);
  const u32x4* s = reinterpret_cast<const u32x4*>(p.tails + x * p.P * p.D);
  u32x4* d = reinterpret_cast<u32x4*>(p.tails + y * p.P * p.D);
  const int blocks = (tail + 15) / 16;
  for (int i = threadIdx.x; i < blocks * 2 * p.D; i += kThreads) d[i] = s[i];
  if (threadIdx.x < tail) p.tail_scales[y * p.P + threadIdx.x] = p.tail_scales[x * p.P + threadIdx.x];
}

// Blocks: pages that the tokens can fall on, times heads, times keys and values.
int64_t page_blocks(const KvParams& p) {
  const int64_t pages = p.cu ? p.tokens / p.P + 2 * int64_t{min(p.entries, p.tokens)} : p.entries;
  return pages * p.heads * 2;
}

template <typename T, int IT>
hipError_t launch_append(const AppendParams& a, hipStream_t s) {
  kv_append_kernel<T, IT><<<page_blocks(a.c), kThreads, a.c.P * a.c.D, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_append_type(const AppendParams& a, hipStream_t s) {
  const int pieces = (a.c.P * a.c.D / 32 + kThreads - 1) / kThreads;
  return pieces <= 1 ? launch_append<T, 1>(a, s) : pieces <= 2 ? launch_append<T, 2>(a, s) : launch_append<T, 4>(a, s);
}

}  // namespace

int64_t kv_page_blocks(const KvParams& p) { return page_blocks(p); }

hipError_t launch_kv_append(const KvParams& c, const void* k, int64_t ld_k, int64_t ld_k_head, const void* v,
                            int64_t ld_v, int64_t ld_v_head, int dtype, hipStream_t s) {
  const AppendParams a{c, {k, v}, {ld_k, ld_v}, {ld_k_head, ld_v_head}};
  return dtype == MOE_BF16 ? launch_append_type<Bf16>(a, s) : launch_append_type<F16>(a, s);
}

hipError_t launch_kv_read(const KvParams& c, void* k, void* v, int dtype, hipStream_t s) {
  const ReadParams a{c, {k, v}};
  const int64_t blocks = page_blocks(c);
  if (dtype == MOE_BF16) kv_read_kernel<Bf16><<<blocks, kThreads, 0, s>>>(a);
  else if (dtype == MOE_F16) kv_read_kernel<F16><<<blocks, kThreads, 0, s>>>(a);
  else kv_read_kernel<F32><<<blocks, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_fork(const KvParams& c, const int32_t* src, const int32_t* dst, int pairs, hipStream_t s) {
  kv_fork_kernel<<<int64_t{1 + 2 * c.heads} * pairs, kThreads, 0, s>>>(ForkParams{c, src, dst});
  return hipGetLastError();
}

}  // namespace nvfp4

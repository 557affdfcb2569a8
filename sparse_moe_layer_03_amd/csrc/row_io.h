// Device-side access to rows of bf16 or fp32 values in chunks of 8, at any
// element alignment (this target's global loads and stores take any): the row
// kernels of the norms and of the 8-bit codes.
#pragma once

#include <type_traits>

#include "../../include/moe.h"
#include "common.h"
#include "wave.h"

namespace moe {

typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef u32x2_t u32x2_byte_t __attribute__((aligned(1)));

constexpr int kChunk = 8;  // values

// 8 values as they lie in memory.
template <typename T>
struct Raw {
  u32x4_t v[sizeof(T) / 2];
};

// v without its first n values, zeros behind.
__device__ __forceinline__ u32x4_t drop_words(u32x4_t v, int words) {
  if (words & 2) v = u32x4_t{v[2], v[3], 0u, 0u};
  if (words & 1) v = u32x4_t{v[1], v[2], v[3], 0u};
  return v;
}
__device__ __forceinline__ Raw<__bf16> drop(Raw<__bf16> r, int n) {
  u32x4_t v = drop_words(r.v[0], n >> 1);
  if (n & 1)
    v = u32x4_t{(v[0] >> 16) | (v[1] << 16), (v[1] >> 16) | (v[2] << 16), (v[2] >> 16) | (v[3] << 16),
                v[3] >> 16};
  r.v[0] = v;
  return r;
}
__device__ __forceinline__ Raw<float> drop(Raw<float> r, int n) {
  if (n & 4) {
    r.v[0] = r.v[1];
    r.v[1] = u32x4_t{0u, 0u, 0u, 0u};
  }
  const int m = n & 3;
  if (m) {
    const uint32_t w[8] = {r.v[0][0], r.v[0][1], r.v[0][2], r.v[0][3],
                           r.v[1][0], r.v[1][1], r.v[1][2], r.v[1][3]};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t one = i + 1 < 8 ? w[i + 1 < 8 ? i + 1 : 0] : 0u;
      const uint32_t two = i + 2 < 8 ? w[i + 2 < 8 ? i + 2 : 0] : 0u;
      const uint32_t three = i + 3 < 8 ? w[i + 3 < 8 ? i + 3 : 0] : 0u;
      o[i] = m == 1 ? one : m == 2 ? two : three;
    }
    r.v[0] = u32x4_t{o[0], o[1], o[2], o[3]};
    r.v[1] = u32x4_t{o[4], o[5], o[6], o[7]};
  }
  return r;
}

template <typename T>
__device__ __forceinline__ Raw<T> zero_raw() {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = u32x4_t{0u, 0u, 0u, 0u};
  return r;
}

// ONCE: rows that one kernel reads or writes once need not stay in the caches.
template <bool ONCE = false, typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
    const u32x4_any_t* q = reinterpret_cast<const u32x4_any_t*>((const char*)p + 16 * i);
    r.v[i] = ONCE ? __builtin_nontemporal_load(q) : *q;
  }
  return r;
}

// Chunk c of a row of n values, zeros behind its end: the row's last chunk is
// loaded from its last 8 values, and what it has too much in front dropped.
// WHOLE: rows of whole chunks.  (Unsigned byte offsets from the row's start,
// which is the same for all lanes, take one register; an index takes two.)
template <typename T>
__device__ __forceinline__ T* chunk_at(T* row, int c) {
  typedef typename std::conditional<std::is_const<T>::value, const char, char>::type B;
  return (T*)((B*)row + (uint32_t)c * (uint32_t)(kChunk * sizeof(T)));
}
template <bool WHOLE = false, bool ONCE = false, typename T>
__device__ __forceinline__ Raw<T> load_chunk(const T* row, int c, int n) {
  const int at = c * kChunk;
  if (WHOLE) return at < n ? load_raw<ONCE>(chunk_at(row, c)) : zero_raw<T>();
  if (at + kChunk <= n) return load_raw<ONCE>(chunk_at(row, c));
  if (at >= n) return zero_raw<T>();
  if (n >= kChunk) return drop(load_raw(row + n - kChunk), at + kChunk - n);
  T e[kChunk];
#pragma unroll
  for (int k = 0; k < kChunk; ++k) e[k] = k < n ? row[k] : (T)0.f;  // (c is 0)
  Raw<T> r;
  __builtin_memcpy(&r, e, sizeof r);
  return r;
}

__device__ __forceinline__ void floats(const Raw<__bf16>& r, float* f) { unpack16(r.v[0], f, (__bf16*)nullptr); }
__device__ __forceinline__ void floats(const Raw<float>& r, float* f) {
  unpack16(r.v[0], f, (float*)nullptr);
  unpack16(r.v[1], f + 4, (float*)nullptr);
}
__device__ __forceinline__ Raw<__bf16> raw_of(const float* f, __bf16*) {
  Raw<__bf16> r;
  r.v[0] = pack16(f, (__bf16*)nullptr);
  return r;
}
__device__ __forceinline__ Raw<float> raw_of(const float* f, float*) {
  Raw<float> r;
  r.v[0] = pack16(f, (float*)nullptr);
  r.v[1] = pack16(f + 4, (float*)nullptr);
  return r;
}

// (c begins inside the row)
template <bool WHOLE = false, bool ONCE = false, typename T>
__device__ __forceinline__ void store_chunk(T* row, int c, int n, const Raw<T>& r) {
  const int at = c * kChunk;
  if (WHOLE || at + kChunk <= n) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      u32x4_any_t* q = reinterpret_cast<u32x4_any_t*>((char*)chunk_at(row, c) + 16 * i);
      if (ONCE) __builtin_nontemporal_store(r.v[i], q);
      else *q = r.v[i];
    }
  } else {
    T e[kChunk];
    __builtin_memcpy(e, &r, sizeof r);
#pragma unroll
    for (int k = 0; k < kChunk - 1; ++k)
      if (at + k < n) row[at + k] = e[k];
  }
}

// ---- 8-bit codes

// The scale of a row whose largest magnitude has the bits `top`; NaN where the
// row holds an infinity or a NaN.
__device__ __forceinline__ float code_scale(uint32_t top) {
  if (top >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  return fmaxf(__uint_as_float(top) / 127.f, 0x1p-126f);
}

// The whole number nearest to the exact quotient x / scale, ties to even: the
// guess by the reciprocal is off by at most one, and x - q scale is exact (both
// are multiples of the finer one's last bit, and it is smaller than scale).
__device__ __forceinline__ int code_of(float x, float scale, float inv) {
  float q = rintf(x * inv);
  const float r = fmaf(-q, scale, x);
  const float twice = fabsf(r) * 2.f;
  int k = (int)q;
  if (twice > scale || (twice == scale && (k & 1))) k += r < 0.f ? -1 : 1;
  return k;
}

// The codes of a chunk; 0 in a row whose scale is NaN.
__device__ __forceinline__ u32x2_t codes_of(const float* f, float scale) {
  u32x2_t o = {0u, 0u};
  if (scale == scale) {
    const float inv = 1.f / scale;
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k >> 2] |= (uint32_t)(code_of(f[k], scale, inv) & 255) << (8 * (k & 3));
  }
  return o;
}

__device__ __forceinline__ void store_codes(int8_t* row, int c, int n, u32x2_t v) {
  const int at = c * kChunk;
  if (at + kChunk <= n) {
    *reinterpret_cast<u32x2_byte_t*>(chunk_at(row, c)) = v;
  } else {
#pragma unroll
    for (int k = 0; k < kChunk - 1; ++k)
      if (at + k < n) row[at + k] = (int8_t)(v[k >> 2] >> (8 * (k & 3)));
  }
}

__device__ __forceinline__ uint32_t magnitude(float f) { return __float_as_uint(f) & 0x7fffffffu; }

// ---- reductions over a row's threads: one wave (ALONE), or the NT threads of the
// workgroup through `s` (2 * 3 * 16 words, its halves used in turn: a half is
// written again only behind the barrier of the other one)

template <bool ALONE, int NT, int N, typename OP>
__device__ __forceinline__ void row_reduce(uint32_t (&v)[N], uint32_t* s, int& turn, OP op) {
  if constexpr (!ALONE) {
    constexpr int W = NT / kWave;
    uint32_t* at = s + (turn & 1) * 48;
    ++turn;
    if (lane_id() == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) at[k * 16 + (threadIdx.x >> 6)] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      uint32_t r = at[k * 16];
#pragma unroll
      for (int q = 1; q < W; ++q) r = op(r, at[k * 16 + q]);
      v[k] = r;
    }
  }
}
template <bool ALONE, int NT, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], uint32_t* s, int& turn) {
  uint32_t u[N];
#pragma unroll
  for (int k = 0; k < N; ++k) u[k] = __float_as_uint(wave_sum_f(v[k]));
  row_reduce<ALONE, NT, N>(u, s, turn, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  });
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = __uint_as_float(u[k]);
}
template <bool ALONE, int NT>
__device__ __forceinline__ float row_sum(float v, uint32_t* s, int& turn) {
  float a[1] = {v};
  row_sums<ALONE, NT, 1>(a, s, turn);
  return a[0];
}
template <bool ALONE, int NT>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* s, int& turn) {
  uint32_t a[1] = {wave_max_u(v)};
  row_reduce<ALONE, NT, 1>(a, s, turn, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
  return a[0];
}

}  // namespace moe

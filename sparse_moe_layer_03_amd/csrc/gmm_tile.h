// Device-side pieces that the grouped products on matrix instructions share:
// waits, descriptors, a group's rows, a tile's geometry in LDS and packed
// stores.
#pragma once

#include "../../include/moe.h"
#include "common.h"

namespace moe {

typedef __attribute__((address_space(3))) void lds_void_t;
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

constexpr int kMfmaMaxGroups = 1024;
constexpr int kCpolNT = 2;  // cache policy of a load: non-temporal
constexpr uint32_t kOutside = 0x7ffffff0u;  // a buffer offset behind every descriptor's end

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
__device__ __forceinline__ void barrier_all() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const char* uni(const char* p) {
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = (uint32_t)uni((int)(uint32_t)v), hi = (uint32_t)uni((int)(v >> 32));
  return (const char*)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t descriptor(const char* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)bytes, 0x00020000);
}

// Rows [lo, hi) of a group, inside [0, M] whatever the offsets hold.
__device__ __forceinline__ void rows_of(const int32_t* offsets, int e, int M, int& lo, int& hi) {
  const int first = offsets[e], end = offsets[e + 1];
  MOE_CHECK(0 <= first && first <= end && end <= M, MOE_CHECK_GMM_OFFSETS);
  lo = min(max(first, 0), M);
  hi = min(max(end, lo), M);
}

// The same for a group known to be one for all lanes, through the scalar
// cache: a vector load would wait behind the last tile's stores.
__device__ __forceinline__ void rows_of_uniform(const int32_t* offsets, int e, int M, int& lo, int& hi) {
  typedef const __attribute__((address_space(4))) int32_t* const_ptr_t;
  const const_ptr_t o = (const_ptr_t)(offsets + e);
  MOE_CHECK(0 <= o[0] && o[0] <= o[1] && o[1] <= M, MOE_CHECK_GMM_OFFSETS);
  lo = min(max(o[0], 0), M);
  hi = min(max(o[1], lo), M);
}

// One operand's tile geometry: W rows or columns of the output side, KS
// reduction values (64 or 32) a step.
template <bool OUT, int W, int NW, int KS>
struct Tile {
  static constexpr int RB = OUT ? W * 2 : KS * 2;  // bytes per LDS row
  static constexpr int RPI = 1024 / RB;            // LDS rows per DMA instruction
  static constexpr int BYTES = W * KS * 2;
  static constexpr int PW = BYTES / 1024 / NW;     // DMA instructions per wave and step
  // Instructions q and q + P of a wave fetch the same chunks of rows that lie
  // (P NW RPI) apart: their lane offsets differ by a wave-uniform amount.
  static constexpr int P = NW * RPI >= 16 ? 1 : 16 / (NW * RPI);  // the swizzles repeat every 16 rows
  static constexpr int NP = P < PW ? P : PW;
  static_assert(PW >= 1 && PW * NW * 1024 == BYTES, "whole instructions");
  static_assert(!OUT || W >= 128, "OUT tiles are 128 or 256 wide");
  // LDS row and logical 16-byte chunk that lane `lane` of instruction q of
  // wave `wave` fills
  static __device__ __forceinline__ int row(int q, int wave, int lane) {
    return (wave + q * NW) * RPI + lane / (RB / 16);
  }
  static __device__ __forceinline__ int chunk(int q, int wave, int lane) {
    const int r = row(q, wave, lane), slot = lane % (RB / 16);
    if (OUT) return slot ^ (flip(r) << 1);
    return slot ^ turn(r);
  }
  // OUT: half a wave's tr read covers 8 rows (b 8 + 0 .. 3, two values of b)
  // of 32 bytes, which land on 8 different 32-byte pieces of the 256 that the
  // banks span.
  static __device__ __forceinline__ int flip(int r) { return (r & 3) | ((r >> 1) & 4); }
  // RED: a 16-byte read serves 16 lanes a cycle, among them rows 0 .. 3 and
  // 12 .. 15 at one chunk with rows 4 .. 11 at the next; r ^ r >> 3, which
  // suits 16 rows of one chunk, had cost every read a second pass.
  static __device__ __forceinline__ int turn(int r) {
    if (KS == 32) return ((r >> 2) & 1) | (((r >> 1) ^ (r >> 2)) & 2);
    return (r >> 1) & 7;
  }
  // Fragments: block b covers 16 outputs, slice kk 32 reduction values.  The
  // block's wave-dependent part goes into the lane's base address, the rest
  // (with no bit in common) into constants.
  static __device__ __forceinline__ int lane_base(int lane, int b) {
    const int l16 = lane & 15, l4 = lane >> 4;
    if (OUT) {
      const int r = l4 * 8 + (l16 >> 2);
      return r * RB + ((b ^ flip(r)) << 5) + (l16 & 3) * 8;
    }
    // chunk (4 kk + l4) of row 16 b + l16, under the row's swizzle
    return (b * 16 + l16) * RB + ((l4 ^ turn(l16)) << 4);
  }
  static __device__ __forceinline__ bf16x8_t frag(const char* s, int base, int b, int kk) {
    if constexpr (OUT) {
      const char* p = s + kk * 32 * RB + (base ^ (b << 5));
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)p);
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + 4 * RB));
      return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return *reinterpret_cast<const bf16x8_t*>(s + b * 16 * RB + (base ^ (kk << 6)));
    }
  }
};

__device__ __forceinline__ uint2 bf16x4(const f32x4_t& v) {
  const uint32_t lo = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[0]) |
                      ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[1]) << 16);
  const uint32_t hi = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2]) |
                      ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[3]) << 16);
  return make_uint2(lo, hi);
}

// Two 16 x 16 blocks side by side, packed to bf16: a lane holds columns 4 l4 ..
// + 3 of both; swapping 16-lane rows between the two registers leaves it with
// 8 neighbouring columns of one block (of the first for even l4, of the
// second for odd), so that a row's 64 bytes go out in 16-byte stores (with
// 8-byte stores in 32-byte pieces the weights' gradients were written at half
// the rate).  bf16_col() is the first of the lane's columns.
__device__ __forceinline__ u32x4_t bf16x8(const f32x4_t& a, const f32x4_t& b) {
  const uint2 x = bf16x4(a), y = bf16x4(b);
  const auto lo = __builtin_amdgcn_permlane16_swap(x.x, y.x, false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(x.y, y.y, false, false);
  return u32x4_t{(uint32_t)lo[0], (uint32_t)hi[0], (uint32_t)lo[1], (uint32_t)hi[1]};
}
__device__ __forceinline__ int bf16_col(int l4) { return (l4 & 1) * 16 + (l4 >> 1) * 8; }

}  // namespace moe

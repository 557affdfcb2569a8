// Grouped bf16 matrix products on bf16 MFMAs: forward, gradient of the rows,
// gradient of the weights (the three forms of gmm_general.hip), for rows that
// are multiples of 16 bytes.
//
// The operands differ from the forward layer's in how they lie in memory.  An
// operand is RED when its reduction dimension is contiguous (a lane's 8
// reduction values are one 16-byte chunk), OUT when its output dimension is:
// the weights in the gradient of the rows, both operands in the gradient of
// the weights.  OUT tiles are brought into LDS as they lie (a step's reduction
// rows, each the tile's width) and transposed on the way to the registers by
// ds_read_b64_tr_b16: 16 lanes read 4 reduction rows x 16 columns and each
// gets one column's 4 values; two reads make an MFMA operand.  No transposed
// copy of the weights or rows exists anywhere.
//
//  * Tiles move HBM -> LDS with direct-to-LDS buffer loads.  Each tile (OUT:
//    each step) has a descriptor that ends where the group's rows or the
//    reduction end, and what lies behind reads as zero: ragged reductions and
//    short tiles need no other masking.
//  * LDS slots are swizzled through the global address a lane fetches
//    (Tile::turn, Tile::flip); no bank conflicts are left in either kind of
//    read (they had doubled the RED reads' time in LDS).
//  * Rings of stages, loads 1 to 3 steps ahead, one barrier a step.  FWD and
//    DX step by 64 (whole 128-byte lines of a RED row), two stages of a and
//    three of b; DW by 32 with four of each, since both of its operands come
//    from beyond L2 and short groups have few steps.
//  * A persistent grid walks over the tiles.  The next tile's place is worked
//    out, with scalar loads only, under this tile's first loads, and its first
//    loads go out before this tile's stores, which drain under its first
//    steps: loads wait for older stores, so stores always come last.  FWD, DX:
//    row tiles balanced in height, MFMAs for the blocks of 16 rows that exist.
//    DW: chunks of 32 neighbouring tiles go to one XCD and share its L2.
//
// Measured over 256 groups of W [1536, 4096] (3.2 GB): 8 rows a group FWD 566
// us, DX 483 us (5.7 and 6.7 TB/s: the weights' stream bounds), 256 rows 849
// and 850 us (970 TFLOP/s, both bounds near), 1024 rows 2.64 and 2.91 ms (1.25
// and 1.13 PFLOP/s; a library product of 8192^3 1.42 and 1.35).  DW: 39
// rows 0.79 ms, 256 rows 1.39 ms (592 TFLOP/s; 3.2 GB of results, which a
// plain fill writes in 0.47 ms).

#include <algorithm>
#include <type_traits>

#include "common.h"
#include "train.h"

namespace moe {

typedef __attribute__((address_space(3))) void lds_void_t;
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

constexpr int kMfmaMaxGroups = 1024;
constexpr int kCpolNT = 2;  // cache policy of a load: non-temporal
constexpr uint32_t kOutside = 0x7ffffff0u;  // a buffer offset behind every descriptor's end
enum { EPI_STORE = 0, EPI_SWIGLU = 1 };

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

template <int FORM, int EPI, typename TO, int BM, int BN, int WM, int WN, int KS, int SA, int SB>
__global__ void __launch_bounds__(64 * WM * WN, 2)
gmm_mfma_kernel(GmmArgs g) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NW = WM * WN, NT = 64 * NW;
  constexpr bool DW = FORM == MOE_GMM_DW, SW = EPI == EPI_SWIGLU;
  using TA = Tile<DW, BM, NW, KS>;
  using TB = Tile<FORM != MOE_GMM_FWD, BN, NW, KS>;
  constexpr int MB = BM / WM / 16, NB = BN / WN / 16;
  constexpr int A_PW = TA::PW, B_PW = TB::PW, PW = A_PW + B_PW;
  constexpr int HN = SW ? BN / 2 : BN;  // output columns per tile
  constexpr int MG = 4;
  constexpr int DA = SA - 1, DB = SB - 1;
  // store instructions of a tile's epilogue (16 bytes a lane)
  constexpr int NST_ALL = MB * NB * (int)sizeof(TO) / 4;
  // (vmcnt counts to 63; 0: every load waits for the stores before it)
  constexpr int NST = SW || NST_ALL + DB * PW > 63 ? 0 : NST_ALL;
  static_assert(A_PW >= 1 && B_PW >= 1 && (!SW || (NB % 2 == 0 && B_PW % 2 == 0)), "tile");
  static_assert(TB::BYTES > kMfmaMaxGroups * 4, "the groups' prefix fits a stage");

  // Rings of SA and SB stages, one array each: the compiler then sees that the
  // stage being read is not one being filled.  Loads of a are DA steps ahead,
  // those of b DB.
  static_assert(DA >= 1 && DB >= DA && SB <= 5 && SA * TA::BYTES + SB * TB::BYTES <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(1024))) char s_a0[TA::BYTES];
  __shared__ __attribute__((aligned(1024))) char s_a1[TA::BYTES];
  __shared__ __attribute__((aligned(1024))) char s_a2[SA > 2 ? TA::BYTES : 16];
  __shared__ __attribute__((aligned(1024))) char s_a3[SA > 3 ? TA::BYTES : 16];
  __shared__ __attribute__((aligned(1024))) char s_a4[SA > 4 ? TA::BYTES : 16];
  __shared__ __attribute__((aligned(1024))) char s_b0[TB::BYTES];
  __shared__ __attribute__((aligned(1024))) char s_b1[TB::BYTES];
  __shared__ __attribute__((aligned(1024))) char s_b2[SB > 2 ? TB::BYTES : 16];
  __shared__ __attribute__((aligned(1024))) char s_b3[SB > 3 ? TB::BYTES : 16];
  __shared__ __attribute__((aligned(1024))) char s_b4[SB > 4 ? TB::BYTES : 16];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uni(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane & 15, l4 = lane >> 4;
  // DW: a wave's row blocks are one stretch; else they interleave with the
  // other waves', so that a short tile loads all of them
  const int a_lane = TA::lane_base(lane, DW ? wm * MB : wm);
  const int b_lane = TB::lane_base(lane, SW ? wn * (NB / 2) : wn * NB);

  const int G = gridDim.x, bid = blockIdx.x;
  const int jt = DW ? 1 : (g.s[0].J + HN - 1) / HN;
  // FWD, DX: tiles that run together on an XCD are neighbours
  const int vid = (!DW && G % 8 == 0) ? (bid % 8) * (G / 8) + bid / 8 : bid;

  // FWD, DX: (first row tile << 10 | group) of this workgroup's next 64 tiles,
  // one per lane, and the number of tiles
  uint32_t desc = 0;
  long tiles = 0;
  auto describe = [&](int k0) {
    int* s_pref = reinterpret_cast<int*>(s_b0);
    int* s_scan = reinterpret_cast<int*>(s_b1);
    constexpr int PER = (kMfmaMaxGroups + NT - 1) / NT;
    // ascending offsets give at most this many row tiles; more are cut off
    // here and computed nowhere
    const int most = g.M / BM + g.ngroups;
    int loc[PER], run = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int e = tid * PER + k;
      if (e < g.ngroups) {
        int lo, hi;
        rows_of(g.offsets, e, g.M, lo, hi);
        run = min(run + (hi - lo + BM - 1) / BM, most + 1);
      }
      loc[k] = run;
    }
    const int base = block_inclusive_scan<NT>(run, s_scan) - run;
    if (tid == 0) s_pref[0] = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k)
      if (tid * PER + k < g.ngroups) s_pref[tid * PER + k + 1] = base + loc[k];
    __syncthreads();
    const int row_tiles = uni(s_pref[g.ngroups]);
    tiles = row_tiles <= most ? (long)row_tiles * jt : 0;
    const long t = (vid + (long)(k0 + lane) * G) / g.nsplit;
    desc = 0;
    if (t < tiles) {
      const int m = (int)(t / jt);
      int lo = 0, hi = g.ngroups - 1;  // last group with s_pref <= m
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_pref[mid] <= m) lo = mid; else hi = mid - 1;
      }
      desc = ((uint32_t)s_pref[lo] << 10) | (uint32_t)lo;
    }
    __syncthreads();
  };

  // ---- one tile's place, the same in all lanes
  struct Place {
    int e, i0, i_end, j0, split, rows;
    long row0;
    int k_lo, k_hi, r_end;  // its steps, and the end of its reduction
    int I, J;
    int64_t ldo;
    char* out;
    const char *a_base, *b_base, *b_base2;
    uint32_t a_bytes, b_bytes;  // OUT: of a row's part; RED: of the tile
    uint32_t lda2, ldb2;        // bytes between rows
    bool once;                  // no other tile reads this tile's part of b
  };
  // lane offsets of the first load instructions of each kind, in the tile
  // whose loads go out
  uint32_t a_off[TA::NP], b_off[TB::NP];

  // Tile number k of this workgroup; false behind the last one.
  auto setup = [&](int k, Place& t) -> bool {
    GmmSub sub = g.s[0];
    t.split = 0;
    if constexpr (DW) {
      auto count = [](const GmmSub& s) { return ((s.I + BM - 1) / BM) * ((s.J + BN - 1) / BN); };
      const int c0 = count(g.s[0]), c1 = g.nsub > 1 ? count(g.s[1]) : 0,
                c2 = g.nsub > 2 ? count(g.s[2]) : 0;
      const uint32_t per_group = (uint32_t)(c0 + c1 + c2);
      const uint32_t all = per_group * (uint32_t)g.ngroups * (uint32_t)g.nsplit;
      // chunks of 32 tiles deal over the XCDs (workgroup b runs on XCD b % 8);
      // a round of the grid is a multiple of 8
      const uint32_t b = (uint32_t)bid + (uint32_t)k * (uint32_t)G;
      const uint32_t x = b & 7, y = b >> 3;
      uint32_t n = ((y >> 5) * 8 + x) * 32 + (y & 31);
      // the tail's chunks may lie behind the end while later ones do not
      if (b >= (all + 255) / 256 * 256) return false;
      if (n >= all) {
        t.e = -1;
        return true;
      }
      if (g.nsplit > 1) {
        t.split = (int)(n % (uint32_t)g.nsplit);
        n /= (uint32_t)g.nsplit;
      }
      t.e = uni((int)(n / per_group));
      int local = (int)(n - (uint32_t)t.e * per_group);
      if (local >= c0) {
        local -= c0;
        sub = g.s[1];
        if (local >= c1) {
          local -= c1;
          sub = g.s[2];
        }
      }
      // bands of 4 rows of tiles, column by column
      const int nj = (sub.J + BN - 1) / BN, ni = (sub.I + BM - 1) / BM;
      const int band = local / (4 * nj), in = local - band * 4 * nj;
      const int high = min(4, ni - band * 4);
      t.i0 = (band * 4 + in % high) * BM;
      t.j0 = (in / high) * BN;
      t.i_end = min(sub.I, t.i0 + BM);
      int lo, hi;
      rows_of_uniform(g.offsets, t.e, g.M, lo, hi);
      t.row0 = lo;
      t.rows = hi - lo;
    } else {
      const long item = vid + (long)k * G;
      if (item >= tiles * g.nsplit) return false;
      long n = item;
      if (g.nsplit > 1) {
        n = item / g.nsplit;
        t.split = (int)(item - n * g.nsplit);
      }
      const uint32_t d = (uint32_t)__builtin_amdgcn_readlane((int)desc, k & 63);
      t.e = uni((int)(d & 1023u));
      int lo, hi;
      rows_of_uniform(g.offsets, t.e, g.M, lo, hi);
      t.row0 = lo;
      t.rows = hi - lo;
      // in a group: bands of MG row tiles, column by column, so that tiles
      // that run together share row and weight slices in L2
      const int mt = (t.rows + BM - 1) / BM;
      const int local = (int)(n - (long)(d >> 10) * jt);
      const int m0 = (local / (MG * jt)) * MG;
      const int mg = max(1, min(MG, mt - m0));
      const int in = local - m0 * jt;
      t.j0 = (in / mg) * HN;
      const int h = ((t.rows + mt - 1) / mt + 15) & ~15;  // balanced height
      t.i0 = (m0 + in % mg) * h;
      t.once = mt == 1;
      t.i_end = min(t.rows, t.i0 + h);
    }
    t.e = uni(t.e), t.i0 = uni(t.i0), t.i_end = uni(t.i_end), t.j0 = uni(t.j0);
    t.split = uni(t.split), t.rows = uni(t.rows), t.row0 = uni((int)t.row0);
    const int R = DW ? t.rows : g.R;
    const int steps = (R + KS - 1) / KS;
    const int per = g.nsplit > 1 ? (steps + g.nsplit - 1) / g.nsplit : steps;
    t.k_lo = min(t.split * per, steps), t.k_hi = min(steps, t.k_lo + per);
    t.r_end = min(R, t.k_hi * KS);
    t.I = sub.I, t.J = sub.J, t.ldo = sub.ldo, t.out = (char*)sub.out;
    t.lda2 = (uint32_t)sub.lda * 2, t.ldb2 = (uint32_t)sub.ldb * 2;
    // where the operands' tiles begin and end
    if constexpr (DW) {
      t.a_base = uni((const char*)sub.a + t.row0 * (int64_t)t.lda2 + (int64_t)t.i0 * 2);
      t.a_bytes = (uint32_t)min(BM, sub.I - t.i0) * 2;
    } else {
      t.a_base = uni((const char*)sub.a + (t.row0 + t.i0) * (int64_t)t.lda2);
      t.a_bytes = t.i_end > t.i0 ? (uint32_t)(t.i_end - t.i0 - 1) * t.lda2 + (uint32_t)g.R * 2 : 0u;
    }
    t.b_base2 = nullptr;
    if constexpr (FORM == MOE_GMM_FWD) {
      const int64_t at = ((int64_t)t.e * g.b_group + (int64_t)t.j0 * sub.ldb) * 2;
      t.b_base = uni((const char*)sub.b + at);
      if (SW) t.b_base2 = uni((const char*)g.b2 + at);
      t.b_bytes = (uint32_t)(min(HN, t.J - t.j0) - 1) * t.ldb2 + (uint32_t)g.R * 2;
    } else {
      const int64_t at = (FORM == MOE_GMM_DX ? (int64_t)t.e * g.b_group * 2
                                             : t.row0 * (int64_t)t.ldb2) + (int64_t)t.j0 * 2;
      t.b_base = uni((const char*)sub.b + at);
      if (FORM == MOE_GMM_DX && g.r_switch) t.b_base2 = uni((const char*)g.b2 + at);
      t.b_bytes = (uint32_t)min(BN, t.J - t.j0) * 2;
    }
    return true;
  };

  auto stage_a = [&](auto sc) -> char* {
    constexpr int N = decltype(sc)::value % SA;
    return N == 0 ? s_a0 : N == 1 ? s_a1 : N == 2 ? s_a2 : N == 3 ? s_a3 : s_a4;
  };
  auto stage_b = [&](auto sc) -> char* {
    constexpr int N = decltype(sc)::value % SB;
    return N == 0 ? s_b0 : N == 1 ? s_b1 : N == 2 ? s_b2 : N == 3 ? s_b3 : s_b4;
  };
  // Load instruction q of step ks into a stage.  What its wave-uniform part
  // adds to the lane offset goes through the scalar offset.
  auto load_a = [&](const Place& t, auto sc, int ks, int q) {
    char* dst = stage_a(sc) + (wave + q * NW) * 1024;
    const int add = (int)((uint32_t)(q - q % TA::NP) * (NW * TA::RPI) * t.lda2);
    if constexpr (DW) {
      const int left = min(KS, t.r_end - ks * KS);  // >= 1
      const auto rs = descriptor(t.a_base + (int64_t)ks * KS * t.lda2,
                                 (uint32_t)(left - 1) * t.lda2 + t.a_bytes);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)dst, 16, (int)a_off[q % TA::NP], add,
                                               0, 0);
    } else {
      const auto rs = descriptor(t.a_base, t.a_bytes);
      const int left = t.r_end - ks * KS;
      uint32_t off = a_off[q % TA::NP];
      if (left < KS) off = TA::chunk(q, wave, lane) * 8 < left ? off : kOutside;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)dst, 16, (int)off, ks * KS * 2 + add, 0,
                                               0);
    }
  };
  auto load_b1 = [&](const Place& t, auto sc, int ks, int q, auto cache) {
    constexpr int AUX = decltype(cache)::value;
    char* dst = stage_b(sc) + (wave + q * NW) * 1024;
    // SwiGLU step: gate rows fill the first half of the tile, up rows the second
    const bool second = SW && q >= B_PW / 2;
    const int h = second ? q - B_PW / 2 : q;
    const int add = (int)((uint32_t)(h - h % TB::NP) * (NW * TB::RPI) * t.ldb2);
    if constexpr (FORM == MOE_GMM_FWD) {
      const auto rs = descriptor(second ? t.b_base2 : t.b_base, t.b_bytes);
      const int left = t.r_end - ks * KS;
      uint32_t off = b_off[h % TB::NP];
      if (left < KS) off = TB::chunk(q, wave, lane) * 8 < left ? off : kOutside;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)dst, 16, (int)off, ks * KS * 2 + add, 0,
                                               AUX);
    } else {
      int r = ks * KS, end = t.r_end;
      const char* base = t.b_base;
      if (FORM == MOE_GMM_DX) {
        if (g.r_switch && r >= g.r_switch) {
          base = t.b_base2;
          r -= g.r_switch;
          end -= g.r_switch;
        }
        end = min(end, g.RB);
      }
      const int left = max(0, min(KS, end - r));  // rows of b that this step has
      const auto rs = descriptor(base + (int64_t)r * t.ldb2,
                                 left > 0 ? (uint32_t)(left - 1) * t.ldb2 + t.b_bytes : 0u);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)dst, 16, (int)b_off[h % TB::NP], add,
                                               0, AUX);
    }
  };

  // The step's b loads.  Weights that one tile reads are loaded non-temporally:
  // they need not stay in the caches (few rows per expert: 600 -> 549 us over
  // 256 experts' 3.2 GB).
  auto load_b = [&](const Place& t, auto sc, int ks) {
    if (!DW && t.once) {
#pragma unroll
      for (int q = 0; q < B_PW; ++q) load_b1(t, sc, ks, q, std::integral_constant<int, kCpolNT>{});
    } else {
#pragma unroll
      for (int q = 0; q < B_PW; ++q) load_b1(t, sc, ks, q, std::integral_constant<int, 0>{});
    }
  };

  constexpr int UNROLL = SA == SB ? SA : SA * SB;
  // A tile's first DA and DB steps, in the order in which the loop would
  // have asked for them.
  auto prologue = [&](const Place& t) {
#pragma unroll
    for (int q = 0; q < TA::NP; ++q)
      a_off[q] = (uint32_t)TA::row(q, wave, lane) * t.lda2 + TA::chunk(q, wave, lane) * 16;
#pragma unroll
    for (int q = 0; q < TB::NP; ++q)
      b_off[q] = (uint32_t)TB::row(q, wave, lane) * t.ldb2 + TB::chunk(q, wave, lane) * 16;
    auto one = [&](auto vc) {  // what step V of -DB .. -1 would load
      constexpr int V = decltype(vc)::value - DB;
      if constexpr (V + DA >= 0) {
        if (t.k_lo + V + DA < t.k_hi) {
#pragma unroll
          for (int q = 0; q < A_PW; ++q)
            load_a(t, std::integral_constant<int, V + DA>{}, t.k_lo + V + DA, q);
        }
      }
      if (t.k_lo + V + DB < t.k_hi)
        load_b(t, std::integral_constant<int, V + DB>{}, t.k_lo + V + DB);
    };
    one(std::integral_constant<int, 0>{});
    if constexpr (DB > 1) one(std::integral_constant<int, 1>{});
    if constexpr (DB > 2) one(std::integral_constant<int, 2>{});
    if constexpr (DB > 3) one(std::integral_constant<int, 3>{});
  };
  // Loads issued after the last one that a step with `behind` steps behind it
  // needs: a's of the next DA - 1 steps, and b's from (DB - DA) steps ahead on
  // (with equal leads, b's own is needed).
  auto later = [](int behind) constexpr {
    const int na = behind < DA - 1 ? behind : DA - 1;
    const int lo = DB == DA ? 1 : DB - DA, hi = behind < DB - 1 ? behind : DB - 1;
    return na * A_PW + (hi >= lo ? hi - lo + 1 : 0) * B_PW;
  };

  if constexpr (!DW) describe(0);
  Place t, next;
  if (!setup(0, t)) return;
  if (!DW || t.e >= 0) prologue(t);
  bool stored = false;  // whether the last tile's NST stores may be outstanding
  for (int k = 0;; ++k) {
    // the next tile's place, while this one's first loads are under way
    const bool early = DW || ((k + 1) & 63) != 0;  // else it is not known yet
    bool have = early && setup(k + 1, next);
    if (DW && t.e < 0) {  // a place behind the end: others may follow
      if (!have) break;
      t = next;
      if (t.e >= 0) prologue(t);
      stored = false;  // the stores are older than these loads
      continue;
    }
    f32x4_t acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // Step ks, at place N of the unrolled loop, with MBA active row blocks.  Its
    // loads have landed when at most the later ones are outstanding and, at a
    // tile's first DA steps (whose loads were issued before them), the last
    // tile's stores.
    auto step = [&](auto mbac, auto nc, int ks) {
      constexpr int MBA = decltype(mbac)::value, N = decltype(nc)::value;
      const char* sa = stage_a(nc);
      const char* sb = stage_b(nc);
      const int behind = t.k_hi - 1 - ks;
      auto wait = [&](auto extra) {
        constexpr int X = decltype(extra)::value;
        if (DB == 1 || behind >= DB - 1) wait_vm<later(DB - 1) + X>();
        else if (DB > 3 && behind == 2) wait_vm<later(DB > 3 ? 2 : 0) + X>();
        else if (DB > 2 && behind == 1) wait_vm<later(DB > 2 ? 1 : 0) + X>();
        else wait_vm<later(0) + X>();
      };
      if (stored && ks < t.k_lo + DA) wait(std::integral_constant<int, NST>{});
      else wait(std::integral_constant<int, 0>{});
      barrier_all();
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int kk = 0; kk < KS / 32; ++kk) {
        bf16x8_t fa[MBA], fb[NB];
#pragma unroll
        for (int i = 0; i < MBA; ++i) fa[i] = TA::frag(sa, a_lane, DW ? i : i * WM, kk);
#pragma unroll
        for (int j = 0; j < NB; ++j)
          fb[j] = TB::frag(sb, b_lane, SW && j >= NB / 2 ? BN / 32 + j - NB / 2 : j, kk);
        // into the stages that every wave has left at this step's barrier
        if (kk == 0 && behind >= DA) {
#pragma unroll
          for (int q = 0; q < A_PW; ++q) load_a(t, std::integral_constant<int, N + DA>{}, ks + DA, q);
        }
        if (kk == KS / 32 - 1 && behind >= DB)
          load_b(t, std::integral_constant<int, N + DB>{}, ks + DB);
#pragma unroll
        for (int i = 0; i < MBA; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
    };

    auto loop = [&](auto mbac) {
      for (int ks = t.k_lo; ks < t.k_hi; ks += UNROLL) {
        step(mbac, std::integral_constant<int, 0>{}, ks);
        if (ks + 1 >= t.k_hi) break;
        step(mbac, std::integral_constant<int, 1>{}, ks + 1);
        if constexpr (UNROLL > 2) {
          if (ks + 2 >= t.k_hi) break;
          step(mbac, std::integral_constant<int, 2>{}, ks + 2);
        }
        if constexpr (UNROLL > 3) {
          if (ks + 3 >= t.k_hi) break;
          step(mbac, std::integral_constant<int, 3>{}, ks + 3);
        }
        if constexpr (UNROLL > 4) {
          if (ks + 4 >= t.k_hi) break;
          step(mbac, std::integral_constant<int, 4>{}, ks + 4);
        }
        if constexpr (UNROLL > 5) {
          if (ks + 5 >= t.k_hi) break;
          step(mbac, std::integral_constant<int, 5>{}, ks + 5);
        }
      }
    };
    if constexpr (DW || MB == 1) {
      loop(std::integral_constant<int, MB>{});
    } else {
      // row blocks of this wave that hold rows (a wave without any still
      // loads and waits with the others, on one block that is not stored)
      const int nrb = (t.i_end - t.i0 + 15) / 16;
      const int mba = min(MB, (nrb - wm + WM - 1) / WM);
      if (mba >= 4 && MB >= 4) loop(std::integral_constant<int, MB >= 4 ? 4 : MB>{});
      else if (mba == 3 && MB >= 3) loop(std::integral_constant<int, MB >= 3 ? 3 : MB>{});
      else if (mba == 2) loop(std::integral_constant<int, 2>{});
      else loop(std::integral_constant<int, 1>{});
    }

    // ---- the next tile's first loads, before this one's stores: every wave
    // is done with the stages, and no load is outstanding
    if (early) {
      barrier_all();
      if (have && (!DW || next.e >= 0)) prologue(next);
    }

    // ---- out.  b was the MFMA's row operand: lane (l16, l4) holds columns
    // 4 l4 .. 4 l4 + 3 of row l16 of a 16 x 16 block.
    const int J = t.J;
    stored = false;
    if constexpr (SW) {
      float gates[MB];
#pragma unroll
      for (int i = 0; i < MB; ++i)
        gates[i] = g.gate[t.row0 + min(t.i0 + (i * WM + wm) * 16 + l16, t.rows - 1)];
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        // z, u -> h, dz, du, and this wave's part of <dh, h>
        const int ii = t.i0 + (i * WM + wm) * 16 + l16;
        const bool live = ii < t.i_end;
        const long p = t.row0 + min(ii, t.rows - 1);
        const float gt = gates[i];
        float sum = 0.f;
        // J is a multiple of 64 here: blocks are whole
        auto block = [&](int j, f32x4_t& dz, f32x4_t& du, f32x4_t& hs) {
          const int jj = t.j0 + (wn * (NB / 2) + j) * 16 + l4 * 4;
          f32x4_t dh = {0.f, 0.f, 0.f, 0.f};
          if (live && jj < J) dh = *reinterpret_cast<const f32x4_t*>(g.dh + p * J + jj);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float z = acc[i][j][v], u = acc[i][j + NB / 2][v];
            const float sg = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504f));
            const float si = z * sg, h = si * u, d = gt * dh[v];
            sum += dh[v] * h;
            dz[v] = d * u * (sg * (1.f + z * (1.f - sg)));
            du[v] = d * si;
            hs[v] = gt * h;
          }
        };
        if constexpr (NB / 2 >= 2) {
#pragma unroll
          for (int j = 0; j < NB / 2; j += 2) {
            f32x4_t dz[2], du[2], hs[2];
            block(j, dz[0], du[0], hs[0]);
            block(j + 1, dz[1], du[1], hs[1]);
            const u32x4_t oz = bf16x8(dz[0], dz[1]), ou = bf16x8(du[0], du[1]),
                          oh = bf16x8(hs[0], hs[1]);
            const int jj = t.j0 + (wn * (NB / 2) + j) * 16 + bf16_col(l4);
            if (live && jj < J) {
              char* o = (char*)g.dzu + (p * 2 * J + jj) * 2;
              st16(o, oz);
              st16(o + (int64_t)J * 2, ou);
              st16((char*)g.hs + (p * J + jj) * 2, oh);
            }
          }
        } else {
          f32x4_t dz, du, hs;
          block(0, dz, du, hs);
          const int jj = t.j0 + wn * 16 + l4 * 4;
          if (live && jj < J) {
            char* o = (char*)g.dzu + (p * 2 * J + jj) * 2;
            *reinterpret_cast<uint2*>(o) = bf16x4(dz);
            *reinterpret_cast<uint2*>(o + (int64_t)J * 2) = bf16x4(du);
            *reinterpret_cast<uint2*>((char*)g.hs + (p * J + jj) * 2) = bf16x4(hs);
          }
        }
        sum += __shfl_xor(sum, 16, kWave);
        sum += __shfl_xor(sum, 32, kWave);
        if (live && l4 == 0)
          g.dpart[p * (long)(((J + HN - 1) / HN) * WN) + (t.j0 / HN) * WN + wn] = sum;
      }
    } else {
      constexpr int IB = DW ? 1 : WM;                    // row blocks between a wave's blocks
      const int ib0 = DW ? wm * MB : wm;
      const int jw = t.j0 + wn * NB * 16;                // the wave's first column
      const int high = max(0, t.i_end - t.i0);           // rows of the tile
      // Stores go through a descriptor that ends with the tile's last row, so
      // that their number is the same for every tile; columns behind the last
      // one are sent outside it.
      if (g.nsplit > 1) {
        const long first = DW ? (long)t.e * t.I : t.row0;
        const auto ro = descriptor((const char*)(g.part + t.split * g.part_stride +
                                                 (first + t.i0) * J),
                                   (uint32_t)high * J * 4);
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const int jj = jw + j * 16 + l4 * 4;
            const uint32_t off = (uint32_t)((ib0 + i * IB) * 16 + l16) * J * 4 + jj * 4;
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[i][j]), ro,
                                                   jj < J ? off : kOutside, 0, 0);
          }
      } else {
        const long first = DW ? (long)t.e * g.out_group + (long)t.i0 * t.ldo : (t.row0 + t.i0) * t.ldo;
        const auto ro = descriptor(uni(t.out + first * (long)sizeof(TO)),
                                   high > 0 ? ((uint32_t)(high - 1) * (uint32_t)t.ldo + J) *
                                                  (uint32_t)sizeof(TO)
                                            : 0u);
        const uint32_t ldo_b = (uint32_t)t.ldo * (uint32_t)sizeof(TO);
        const bool add = g.accumulate;
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          const uint32_t row = (uint32_t)((ib0 + i * IB) * 16 + l16) * ldo_b;
          auto at = [&](int jj) { return jj < J ? row + (uint32_t)jj * (uint32_t)sizeof(TO) : kOutside; };
          asm volatile("" ::: "memory");  // one row block's old values at a time
          if constexpr (sizeof(TO) == 4) {
            f32x4_t old[NB];
            if (add) {
#pragma unroll
              for (int j = 0; j < NB; ++j)
                old[j] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                         ro, at(jw + j * 16 + l4 * 4), 0, 0));
#pragma unroll
              for (int j = 0; j < NB; ++j) acc[i][j] += old[j];
            }
#pragma unroll
            for (int j = 0; j < NB; ++j)
              __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[i][j]), ro,
                                                     at(jw + j * 16 + l4 * 4), 0, 0);
          } else {
            if (add) {
              uint2 old[NB];
#pragma unroll
              for (int j = 0; j < NB; ++j)
                old[j] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(
                                                       ro, at(jw + j * 16 + l4 * 4), 0, 0));
#pragma unroll
              for (int j = 0; j < NB; ++j) {
                const f32x4_t w = {__uint_as_float(old[j].x << 16),
                                   __uint_as_float(old[j].x & 0xffff0000u),
                                   __uint_as_float(old[j].y << 16),
                                   __uint_as_float(old[j].y & 0xffff0000u)};
                acc[i][j] += w;
              }
            }
            if (((J | (int)t.ldo) & 7) == 0) {  // whole 16-byte pieces
#pragma unroll
              for (int j = 0; j < NB; j += 2)
                __builtin_amdgcn_raw_buffer_store_b128(bf16x8(acc[i][j], acc[i][j + 1]), ro,
                                                       at(jw + j * 16 + bf16_col(l4)), 0, 0);
            } else {
#pragma unroll
              for (int j = 0; j < NB; ++j)
                __builtin_amdgcn_raw_buffer_store_b64(
                    __builtin_bit_cast(u32x2_t, bf16x4(acc[i][j])), ro, at(jw + j * 16 + l4 * 4), 0, 0);
            }
          }
        }
        // (the 8-byte stores are more; that only waits longer)
        stored = early && NST > 0;
      }
    }
    if (!early) {
      // the next 64 tiles' places are worked out in the stages
      wait_vm<0>();
      __syncthreads();
      describe(k + 1);
      have = setup(k + 1, next);
      if (have) prologue(next);
      stored = false;
    }
    if (!have) break;
    t = next;
  }
#endif
}

MOE_CHECK_ACCESSOR(check_word_gmm_mfma)

bool mfma_ok(int form, int dtype, int N, int K, int64_t lda, int64_t ldc) {
  if (dtype != MOE_BF16 || K % 8 != 0 || lda % 8 != 0) return false;
  // a descriptor spans at most 256 rows
  if (lda > (1 << 20) || ldc > (1 << 20)) return false;
  return form == MOE_GMM_FWD ? N % 4 == 0 && ldc % 4 == 0 : N % 8 == 0 && ldc % 8 == 0;
}

template <int FORM, int EPI, typename TO, int BM, int BN, int WM, int WN, int KS, int SA, int SB>
static int launch_tile(const GmmArgs& g, hipStream_t st) {
  const int cus = stream_cu_count(st);
  if (cus <= 0) return MOE_EHIP;
  constexpr bool DW = FORM == MOE_GMM_DW;
  constexpr int HN = EPI == EPI_SWIGLU ? BN / 2 : BN;
  long grid;
  if (DW) {
    long t = 0;
    for (int q = 0; q < g.nsub; ++q)
      t += (long)((g.s[q].I + BM - 1) / BM) * ((g.s[q].J + BN - 1) / BN);
    t *= (long)g.ngroups * g.nsplit;
    if (t >= (1l << 31)) return MOE_EUNSUPPORTED;
    constexpr int LDS = (BM * SA + BN * SB) * KS * 2;
    grid = (long)cus * (160 * 1024 / LDS < 2 ? 1 : 2) / 8 * 8;
    grid = std::max(8l, std::min(grid, (t + 255) / 256 * 256));
  } else {
    const long most = (long)(g.M / BM + (g.M < g.ngroups ? g.M : g.ngroups)) *
                      ((g.s[0].J + HN - 1) / HN) * g.nsplit;
    constexpr int LDS = (BM * SA + BN * SB) * KS * 2;
    grid = (long)cus * (160 * 1024 / LDS < 2 ? 1 : 2);
    if (grid > most) grid = most;
    if (grid > 8) grid -= grid % 8;
  }
  if (grid < 1) return MOE_OK;
  if (grid > 0x7fffffffl) return MOE_EUNSUPPORTED;
  hipLaunchKernelGGL((gmm_mfma_kernel<FORM, EPI, TO, BM, BN, WM, WN, KS, SA, SB>), dim3((unsigned)grid),
                     dim3(64 * WM * WN), 0, st, g);
  return check_launch();
}

// Tile choice.  FWD and DX go by the rows a group has on average (measured
// over 256 groups of W [1536, 4096], us):
//   rows        8    47    64   100   127   128   256
//   FWD  64x128 566  613   609  774          64-row tiles below 64 rows
//       128x128       659   669  730   748   754    then 128
//       256x256                              762   850   then 256
//   DX   64x256 483  548   564  890          256 columns: an OUT tile's rows
//       128x256       544   557  611   645          are 512 bytes of W
//       256x256                              676   850
// DW has 256 x 256 tiles, in steps of 32 (256 groups of 39 ragged rows: 847
// us, steps of 64: 1034; 128 x 128 tiles 1210) where they give three CUs of
// four a tile (the skewed layer's router, 240 tiles: 52 us, 128 x 128: 81).
// Else, and in the other forms where 256 columns leave CUs idle, 128 x 128.
template <int FORM, typename TO>
static int launch_form(const GmmArgs& g, hipStream_t st) {
  const int cus = stream_cu_count(st);
  if (cus <= 0) return MOE_EHIP;
  const long per = g.M / g.ngroups;
  long t256 = 0;  // 256 x 256 tiles, at most
  for (int q = 0; q < g.nsub; ++q)
    t256 += (long)((g.s[q].J + 255) / 256) * (FORM == MOE_GMM_DW ? (g.s[q].I + 255) / 256 : 1);
  t256 *= g.nsplit * (FORM == MOE_GMM_DW ? (long)g.ngroups
                                         : g.M / 256 + (g.M < g.ngroups ? g.M : g.ngroups));
  if constexpr (FORM == MOE_GMM_DW) {
    if (4 * t256 >= 3L * cus)
      return launch_tile<FORM, EPI_STORE, TO, 256, 256, 4, 2, 32, 4, 4>(g, st);
    return launch_tile<FORM, EPI_STORE, TO, 128, 128, 2, 2, 32, 4, 4>(g, st);
  } else {
    if (per >= 128 && t256 >= cus)
      return launch_tile<FORM, EPI_STORE, TO, 256, 256, 4, 2, 64, 2, 3>(g, st);
    if constexpr (FORM == MOE_GMM_DX) {
      if (per < 48) return launch_tile<FORM, EPI_STORE, TO, 64, 256, 1, 4, 64, 3, 3>(g, st);
      if (t256 >= cus) return launch_tile<FORM, EPI_STORE, TO, 128, 256, 2, 4, 64, 3, 3>(g, st);
    } else if (per < 64) {
      return launch_tile<FORM, EPI_STORE, TO, 64, 128, 1, 4, 64, 3, 3>(g, st);
    }
    return launch_tile<FORM, EPI_STORE, TO, 128, 128, 2, 2, 64, 2, 3>(g, st);
  }
}

int launch_gmm_mfma(int form, int out_dtype, const GmmArgs& g, hipStream_t st) {
  const bool f32 = out_dtype == MOE_F32;
  if (form == MOE_GMM_FWD)
    return f32 ? launch_form<MOE_GMM_FWD, float>(g, st) : launch_form<MOE_GMM_FWD, __bf16>(g, st);
  if (form == MOE_GMM_DX)
    return f32 ? launch_form<MOE_GMM_DX, float>(g, st) : launch_form<MOE_GMM_DX, __bf16>(g, st);
  return f32 ? launch_form<MOE_GMM_DW, float>(g, st) : launch_form<MOE_GMM_DW, __bf16>(g, st);
}

// Rows per expert decide the tile, as for the other products; the partial
// sums of dgate per row follow from it.
static int swiglu_tile(int M, int ngroups) {
  const int per = M / ngroups;
  return per >= 128 ? 256 : per >= 48 ? 128 : 64;
}

int swiglu_parts(int M, int ngroups, int f) {
  const int tile = swiglu_tile(M, ngroups);
  return tile == 256 ? ((f + 127) / 128) * 2 : ((f + 63) / 64) * (tile == 128 ? 2 : 4);
}

int launch_swiglu_mfma(const GmmArgs& g, hipStream_t st) {
  const int tile = swiglu_tile(g.M, g.ngroups);
  if (tile == 256) return launch_tile<MOE_GMM_FWD, EPI_SWIGLU, __bf16, 256, 256, 4, 2, 64, 2, 3>(g, st);
  if (tile == 128) return launch_tile<MOE_GMM_FWD, EPI_SWIGLU, __bf16, 128, 128, 2, 2, 64, 2, 3>(g, st);
  return launch_tile<MOE_GMM_FWD, EPI_SWIGLU, __bf16, 64, 128, 1, 4, 64, 3, 3>(g, st);
}

}  // namespace moe

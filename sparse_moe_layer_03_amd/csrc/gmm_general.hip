// Grouped matrix products for any sizes, row strides and element types: the
// forward product of a grouped linear map and the gradients of its rows and
// of its weights.
//
//   out[i, j] = sum_r A(i, r) B(j, r)
//     FWD  A = lhs[row, r]   B = W_e[j, r]     (r contiguous in both)
//     DX   A = lhs[row, r]   B = W_e[r, j]     (j contiguous in B)
//     DW   A = lhs[row, i]   B = rhs[row, j]   (r is the row)
//
// An operand is RED when its reduction dimension is contiguous, OUT when its
// output dimension is.  Both kinds go to LDS as they lie in memory, in their own
// type and in 16-byte chunks: RED as rows of KB bytes of the reduction, OUT as
// the step's reduction rows, each the tile's width.  bf16 operands feed
// 16x16x32 bf16 MFMAs, fp32 ones four 16x16x4 fp32 MFMAs a chunk.
//
// Rows may start at any element.  A chunk is one 16-byte load at its element's
// address (this target's global loads take any alignment); at a row's end the
// load moves back to the row's last 16 bytes and what it has too much in front
// is shifted out, and what lies behind the reduction's end is zeroed, both on
// the way into LDS and only in steps and tiles that have such an end.  Loads
// guarded element by element had run one after another: 8 us a step.
//
// The next step's chunks wait in registers while a step computes; two LDS
// stages, one barrier a step.  A workgroup walks over the tiles of all groups;
// it finds the groups from their offsets itself, so the host need not know
// them.  Tiles that run together on an XCD are neighbours.
//
// Bound by the fp32 matrix rate (157 TFLOP/s at the nominal clock) where rows
// are many: 8192 rows by [2048, 2048] in fp32 forward 589-640 us, rows'
// gradient 570, weights' gradient 593 (107 to 121 TFLOP/s, MFMAs busy for 76% of
// the cycles; a library product alone 470), in bf16 with odd rows (8191,
// 2047 x 2045) 114, 113 and 164 us.  Few rows are bound by the weights' stream:
// 64 groups of 2 rows by [2048, 2048] in fp32 167 and 182 us (5.6 TB/s).

#include <type_traits>

#include "common.h"
#include "train.h"

namespace moe {

constexpr int kGmmMaxGroups = 1024;

// 16 bytes and 4 elements at an element's address.
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
typedef f32x4_t f32x4_any_t __attribute__((aligned(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef u32x2_t u32x2_any_t __attribute__((aligned(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

// v without its first `bytes` bytes (the same in all lanes), zeros behind.
__device__ __forceinline__ u32x4_t drop(u32x4_t v, int bytes) {
  if (bytes & 8) v = u32x4_t{v[2], v[3], 0u, 0u};
  if (bytes & 4) v = u32x4_t{v[1], v[2], v[3], 0u};
  if (bytes & 2)
    v = u32x4_t{(v[0] >> 16) | (v[1] << 16), (v[1] >> 16) | (v[2] << 16), (v[2] >> 16) | (v[3] << 16),
                v[3] >> 16};
  return v;
}

// A chunk whose first `left` elements exist, element by element: rows that are
// shorter than a chunk.
template <typename T>
__device__ __forceinline__ u32x4_t few(const T* p, int left) {
  constexpr int CE = 16 / sizeof(T);
  T e[CE];
#pragma unroll
  for (int k = 0; k < CE; ++k) e[k] = k < left ? p[k] : (T)0.f;
  u32x4_t v;
  __builtin_memcpy(&v, e, 16);
  return v;
}

// Four neighbouring columns of which `left` exist, added to what is there if
// `add`.
__device__ __forceinline__ void put4(float* p, f32x4_t v, int left, bool add) {
  if (left >= 4) {
    if (add) v += *reinterpret_cast<const f32x4_any_t*>(p);
    *reinterpret_cast<f32x4_any_t*>(p) = v;
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < left) p[k] = add ? v[k] + p[k] : v[k];
  }
}
__device__ __forceinline__ void put4(__bf16* p, f32x4_t v, int left, bool add) {
  if (left >= 4) {
    if (add) {
      const u32x2_t w = *reinterpret_cast<const u32x2_any_t*>(p);
      v += f32x4_t{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u),
                   __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xffff0000u)};
    }
    __bf16 o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = (__bf16)v[k];
    *reinterpret_cast<u32x2_any_t*>(p) = __builtin_bit_cast(u32x2_t, o);
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < left) p[k] = (__bf16)(add ? v[k] + (float)p[k] : v[k]);
  }
}
template <typename TO>
__device__ __forceinline__ void put(TO* p, float v, bool add) {
  if (add) v += ElemOps<TO>::to_f(*p);
  *p = ElemOps<TO>::from_f(v);
}

// Rows [lo, hi) of a group, inside [0, M] whatever the offsets hold.
__device__ __forceinline__ void group_rows(const int32_t* offsets, int e, int M, int& lo, int& hi) {
  const int first = offsets[e], end = offsets[e + 1];
  MOE_CHECK(0 <= first && first <= end && end <= M, MOE_CHECK_GMM_OFFSETS);
  lo = min(max(first, 0), M);
  hi = min(max(end, lo), M);
}

// One operand's tile: W rows or columns of the output side, steps of KB bytes
// of a RED row, brought in by NT threads.
template <typename T, bool OUT, int W, int KB, int NT>
struct Side {
  static constexpr int CE = 16 / sizeof(T);          // elements of a chunk
  static constexpr int BK = KB / sizeof(T);          // reduction values a step
  static constexpr int RB = OUT ? W * (int)sizeof(T) : KB;  // bytes of an LDS row
  static constexpr int CPR = RB / 16, CH = W * KB / 16 / NT;
  static_assert(CH >= 1 && CH * 16 * NT == W * KB, "whole chunks");
  // A fragment: the 16 bytes that a lane gives to the MFMAs, of output l16 of
  // block b and the chunk l4 of a group of four chunks of the reduction.
  static constexpr int GROUPS = KB / 64;
  // Chunks are swizzled within their row so that a fragment's lanes meet no
  // bank twice.  RED: 16 lanes read 16 rows at a chunk.  OUT, bf16: half a wave
  // reads 32 bytes of 8 rows (0 .. 3 and 8 .. 11 of 16).  OUT, fp32: a wave reads
  // 64 bytes of rows 4 apart.
  static __device__ __forceinline__ int turn(int r) {
    if (!OUT) return KB == 128 ? (r >> 1) & 7 : r & 15;
    if (sizeof(T) == 2) {
      constexpr int SH = RB >= 256 ? 0 : RB == 128 ? 1 : 2;
      return ((((r & 3) | ((r >> 1) & 4)) >> SH) << 1) & (CPR - 1);
    }
    return (((r >> 2) & 3) << 2) & (CPR - 1);
  }
  static __device__ __forceinline__ u32x4_t frag(const char* s, int b, int group, int l16, int l4) {
    const int chunk = group * 4 + l4;
    if constexpr (!OUT) {
      return *reinterpret_cast<const u32x4_t*>(s + (b * 16 + l16) * RB + ((chunk ^ turn(l16)) << 4));
    } else if constexpr (sizeof(T) == 2) {
      const int r = chunk * 8 + (l16 >> 2);
      const char* p = s + r * RB + (((b * 2) ^ turn(r)) << 4) + (l16 & 3) * 8;
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)p);
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + 4 * RB));
      return __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int r = chunk * 4;
      const char* p = s + r * RB + (((b * 4) ^ turn(r)) << 4) + l16 * 4;
      u32x4_t v;
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = *reinterpret_cast<const uint32_t*>(p + c * RB);
      return v;
    }
  }
};

template <typename T>
__device__ __forceinline__ void multiply(const u32x4_t& b, const u32x4_t& a, f32x4_t& acc) {
  if constexpr (sizeof(T) == 2) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, b),
                                                  __builtin_bit_cast(bf16x8_t, a), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(b[c]), __uint_as_float(a[c]), acc, 0, 0, 0);
  }
}

template <typename T, typename TO, int FORM, int BM, int BN, int WM, int WN, int KB, bool FEW>
__global__ void __launch_bounds__(64 * WM * WN, WM * WN / 2)
gmm_general_kernel(GmmArgs g) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr bool DW = FORM == MOE_GMM_DW, DX = FORM == MOE_GMM_DX;
  constexpr int NT = 64 * WM * WN;
  using SA = Side<T, DW, BM, KB, NT>;
  using SB = Side<T, FORM != MOE_GMM_FWD, BN, KB, NT>;
  constexpr int CE = SA::CE, BK = SA::BK;
  constexpr int MB = BM / WM / 16, NB = BN / WN / 16;
  constexpr int BAND = 8;  // row tiles of a band
  __shared__ __attribute__((aligned(16))) char s_a[2][BM * KB];
  __shared__ __attribute__((aligned(16))) char s_b[2][BN * KB];
  __shared__ int s_pref[DW ? 1 : kGmmMaxGroups + 1];
  __shared__ int s_tmp[WM * WN];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane & 15, l4 = lane >> 4;
  auto cdiv = [](int n, int d) { return (n + d - 1) / d; };
  // tiles of the products: per row tile (FWD, DX), per group (DW)
  int n_sub[3];
#pragma unroll
  for (int q = 0; q < 3; ++q)
    n_sub[q] = q < g.nsub ? cdiv(g.s[q].J, BN) * (DW ? cdiv(g.s[q].I, BM) : 1) : 0;
  const int per = n_sub[0] + n_sub[1] + n_sub[2];

  // FWD, DX: prefix over the groups of their row tiles
  if (!DW) {
    constexpr int PER = kGmmMaxGroups / NT;
    const int most = g.M / BM + g.ngroups;  // row tiles that ascending offsets can give
    int loc[PER], run = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int e = tid * PER + k;
      if (e < g.ngroups) {
        int lo, hi;
        group_rows(g.offsets, e, g.M, lo, hi);
        run = min(run + cdiv(hi - lo, BM), most + 1);
      }
      loc[k] = run;
    }
    const int base = block_inclusive_scan<NT>(run, s_tmp) - run;
    if (tid == 0) s_pref[0] = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k)
      if (tid * PER + k < g.ngroups) s_pref[tid * PER + k + 1] = base + loc[k];
    __syncthreads();
  }
  const int row_tiles = DW ? g.ngroups : s_pref[g.ngroups];
  if (!DW && row_tiles > g.M / BM + g.ngroups) return;  // offsets not ascending
  const long items = (long)row_tiles * per * g.nsplit;
  // Workgroup b runs on XCD b % 8.  FWD, DX: an XCD walks over its own eighth
  // of the tiles.  DW: over every eighth run of 32 (few tiles: every eighth
  // tile), since a group's tiles cost what its rows are.
  const int G = gridDim.x;
  const bool spread = G % 8 == 0;
  const int xcd = spread ? (int)blockIdx.x % 8 : 0, place = spread ? (int)blockIdx.x / 8 : (int)blockIdx.x;
  const int step = spread ? G / 8 : G;
  const long first = !DW && spread ? items * xcd / 8 : 0, last = !DW && spread ? items * (xcd + 1) / 8 : items;

  const int run = items >= 8L * G ? 5 : 0;
  for (long k = place;; k += step) {
    const long item = DW && spread ? ((((k >> run) * 8 + xcd) << run) | (k & ((1 << run) - 1))) : first + k;
    if (item >= last) break;  // (grows with k)
    const long t = item / g.nsplit;
    const int split = (int)(item - t * g.nsplit);
    int e, rows, local, mt, lo, hi;
    if (DW) {
      e = (int)(t / per);
      local = (int)(t - (long)e * per);
      group_rows(g.offsets, e, g.M, lo, hi);
      rows = hi - lo;
      mt = 0;
    } else {
      const int m = (int)(t / per);
      int lo_e = 0, hi_e = g.ngroups - 1;  // last group with s_pref <= m
      while (lo_e < hi_e) {
        const int mid = (lo_e + hi_e + 1) >> 1;
        if (s_pref[mid] <= m) lo_e = mid; else hi_e = mid - 1;
      }
      e = lo_e;
      group_rows(g.offsets, e, g.M, lo, hi);
      rows = hi - lo;
      mt = cdiv(rows, BM);
      local = (int)(t - (long)s_pref[e] * per);
    }
    // which product; then bands of row tiles, column by column
    GmmSub sub = g.s[0];
    int in = local;
    const int high = DW ? 1 : mt;  // (DW: a sub's tiles lie side by side as they are)
    if (in >= n_sub[0] * high) {
      in -= n_sub[0] * high;
      sub = g.s[1];
      if (in >= n_sub[1] * high) {
        in -= n_sub[1] * high;
        sub = g.s[2];
      }
    }
    const int jt = cdiv(sub.J, BN);
    if (DW) mt = cdiv(sub.I, BM);
    const int m0 = in / (BAND * jt) * BAND;
    const int mg = max(1, min(BAND, mt - m0));
    const int at = in - m0 * jt;
    const int j0 = at / mg * BN, mi = m0 + at % mg;
    const long row0 = lo;
    // FWD, DX: row tiles of equal height
    const int h = DW ? BM : (cdiv(rows, mt) + 15) & ~15;
    const int i0 = mi * h, i_end = min(DW ? sub.I : rows, i0 + h);
    if (!DW && i0 >= rows) continue;  // heights rounded up to 16
    const int R = DW ? rows : g.R;
    // this split's range of the reduction, in pieces of 128 whatever the tile
    const int len = cdiv(cdiv(R, 128), g.nsplit) * 128;
    const int r_lo = min(split * len, R), r_hi = min(R, r_lo + len);

    const T* a = (const T*)sub.a + (DW ? row0 * sub.lda + i0 : (row0 + i0) * sub.lda);
    const long b_at = FORM == MOE_GMM_FWD ? e * g.b_group + (long)j0 * sub.ldb
                                          : (DX ? e * g.b_group : row0 * sub.ldb) + j0;
    const T* b = (const T*)sub.b + b_at;
    const int wide_a = i_end - i0, wide_b = sub.J - j0;

    // RED: rows of this thread's chunks (behind the tile's last: that one)
    auto fetch_red = [&](auto side, const T* base, long ld, int wide, int r, u32x4_t* v) {
      using S = decltype(side);
#pragma unroll
      for (int c = 0; c < S::CH; ++c) {
        const int x = tid + c * NT;
        const T* row = base + min(x / S::CPR, wide - 1) * ld;
        const int k = r + x % S::CPR * CE;
        if (FEW && r_hi < CE) v[c] = few(row + min(k, r_hi - 1), r_hi - k);
        else v[c] = *reinterpret_cast<const u32x4_any_t*>(row + min(k, r_hi - CE));
      }
    };
    // OUT: reduction rows r .. of which those before `end` exist (none: any
    // row is as good), columns of the tile
    auto fetch_out = [&](auto side, const T* base, long ld, int wide, int r, int end, u32x4_t* v) {
      using S = decltype(side);
#pragma unroll
      for (int c = 0; c < S::CH; ++c) {
        const int x = tid + c * NT;
        const T* row = base + (long)max(0, min(r + x / S::CPR, end - 1)) * ld;
        const int w = x % S::CPR * CE;
        if (FEW && wide < CE) v[c] = few(row + min(w, wide - 1), wide - w);
        else v[c] = *reinterpret_cast<const u32x4_any_t*>(row + min(w, wide - CE));
      }
    };
    auto store_red = [&](auto side, char* s, int r, u32x4_t* v) {
      using S = decltype(side);
      const bool tail = r + BK > r_hi && !(FEW && r_hi < CE);
#pragma unroll
      for (int c = 0; c < S::CH; ++c) {
        const int x = tid + c * NT, w = x / S::CPR, ch = x % S::CPR;
        if (tail) {
          const int left = r_hi - (r + ch * CE), part = r_hi % CE;
          const u32x4_t cut = drop(v[c], part ? (CE - part) * (int)sizeof(T) : 0);
          v[c] = left >= CE ? v[c] : left > 0 ? cut : u32x4_t{0u, 0u, 0u, 0u};
        }
        *reinterpret_cast<u32x4_t*>(s + w * S::RB + ((ch ^ S::turn(w)) << 4)) = v[c];
      }
    };
    auto store_out = [&](auto side, char* s, int r, int end, int wide, u32x4_t* v) {
      using S = decltype(side);
      const int part = wide % CE;
      const bool edge = part && wide < (int)(S::RB / sizeof(T)) && !(FEW && wide < CE), tail = r + BK > end;
#pragma unroll
      for (int c = 0; c < S::CH; ++c) {
        const int x = tid + c * NT, row = x / S::CPR, ch = x % S::CPR;
        if (edge) {
          const u32x4_t cut = drop(v[c], (CE - part) * (int)sizeof(T));
          v[c] = wide - ch * CE >= CE ? v[c] : cut;
        }
        if (tail) v[c] = r + row < end ? v[c] : u32x4_t{0u, 0u, 0u, 0u};
        *reinterpret_cast<u32x4_t*>(s + row * S::RB + ((ch ^ S::turn(row)) << 4)) = v[c];
      }
    };
    // DX: where the reduction's rows of b lie (see GmmArgs)
    auto b_rows = [&](int r, const T*& base, int& first, int& end) {
      base = b;
      first = r;
      end = DX ? min(r_hi, g.RB) : r_hi;
      if (DX && g.r_switch && r >= g.r_switch) {
        base = (const T*)g.b2 + b_at;
        first = r - g.r_switch;
        end = min(r_hi - g.r_switch, g.RB);
      }
    };

    u32x4_t va[SA::CH], vb[SB::CH];
    auto fetch = [&](int r) {
      if constexpr (DW) fetch_out(SA{}, a, sub.lda, wide_a, r, r_hi, va);
      else fetch_red(SA{}, a, sub.lda, wide_a, r, va);
      if constexpr (FORM == MOE_GMM_FWD) {
        fetch_red(SB{}, b, sub.ldb, wide_b, r, vb);
      } else {
        const T* base;
        int first, end;
        b_rows(r, base, first, end);
        fetch_out(SB{}, base, sub.ldb, wide_b, first, end, vb);
      }
    };
    auto store = [&](int st, int r) {
      if constexpr (DW) store_out(SA{}, s_a[st], r, r_hi, wide_a, va);
      else store_red(SA{}, s_a[st], r, va);
      if constexpr (FORM == MOE_GMM_FWD) {
        store_red(SB{}, s_b[st], r, vb);
      } else {
        const T* base;
        int first, end;
        b_rows(r, base, first, end);
        store_out(SB{}, s_b[st], first, end, wide_b, vb);
      }
    };

    // fp32: sums of 128 products in acc, their sum in tot: a long reduction
    // rounds like sqrt(128) + sqrt(n / 128) instead of sqrt(n) additions.
    constexpr int FLUSH = sizeof(T) == 4 ? 128 / BK : 0;
    f32x4_t acc[MB][NB], tot[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = tot[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // the steps with MBA of a wave's row blocks (the others hold no rows)
    auto loop = [&](auto mbac) {
      constexpr int MBA = decltype(mbac)::value;
      int st = 0, since = 0;
      for (int r = r_lo; r < r_hi; r += BK, st ^= 1) {
        store(st, r);
        __syncthreads();
        if (r + BK < r_hi) fetch(r + BK);
        // a fragment of a is read while the one before it is multiplied
        u32x4_t fa = SA::frag(s_a[st], wm, 0, l16, l4), fb[NB];
#pragma unroll
        for (int k = 0; k < SA::GROUPS; ++k) {
#pragma unroll
          for (int j = 0; j < NB; ++j) fb[j] = SB::frag(s_b[st], wn * NB + j, k, l16, l4);
#pragma unroll
          for (int i = 0; i < MBA; ++i) {
            const u32x4_t now = fa;
            if (i + 1 < MBA) fa = SA::frag(s_a[st], (i + 1) * WM + wm, k, l16, l4);
            else if (k + 1 < SA::GROUPS) fa = SA::frag(s_a[st], wm, k + 1, l16, l4);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < NB; ++j) multiply<T>(fb[j], now, acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        if (FLUSH && (++since == FLUSH || r + BK >= r_hi)) {
          since = 0;
#pragma unroll
          for (int i = 0; i < MBA; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              tot[i][j] += acc[i][j];
              acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            }
        }
      }
    };
    __syncthreads();  // the previous tile's last reads of LDS
    if (r_lo < r_hi) fetch(r_lo);
    constexpr bool HALVES = !DW && MB == 2 && BM < 128;
    if (HALVES && wide_a <= WM * 16) loop(std::integral_constant<int, HALVES ? 1 : MB>{});
    else loop(std::integral_constant<int, MB>{});

    // b was the MFMA's row operand: a lane holds columns 4 l4 .. + 3 of row l16
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int ii = i0 + (i * WM + wm) * 16 + l16;
      if (ii >= i_end) continue;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const f32x4_t v = FLUSH ? tot[i][j] : acc[i][j];
        const int jj = j0 + (wn * NB + j) * 16 + l4 * 4;
        if (jj >= sub.J) continue;
        if (g.nsplit > 1) {
          // partial outputs are compact: [split][row or group * I + i][J]
          const long prow = DW ? (long)e * sub.I + ii : row0 + ii;
          put4(g.part + split * g.part_stride + prow * sub.J + jj, v, sub.J - jj, false);
        } else {
          const long orow = DW ? (long)e * g.out_group + (long)ii * sub.ldo : (row0 + ii) * sub.ldo;
          put4((TO*)sub.out + orow + jj, v, sub.J - jj, g.accumulate);
        }
      }
    }
  }
#endif
}

// out = sum over splits (in split order) of the partial outputs.
template <typename TO, int FORM>
__global__ void __launch_bounds__(256) gmm_join_kernel(GmmArgs g) {
  const GmmSub& s = g.s[0];
  const long rows = FORM == MOE_GMM_DW ? (long)g.ngroups * s.I
                                       : min(max(g.offsets[g.ngroups], 0), g.M);
  const long first = FORM == MOE_GMM_DW ? 0 : min(max(g.offsets[0], 0), g.M);
  const long n = rows * s.J;
  for (long x = first * s.J + blockIdx.x * 256L + threadIdx.x; x < n; x += gridDim.x * 256L) {
    const long row = x / s.J;
    const int j = (int)(x - row * s.J);
    float v = 0.f;
    for (int q = 0; q < g.nsplit; ++q) v += g.part[q * g.part_stride + x];
    const long o = FORM == MOE_GMM_DW ? (row / s.I) * g.out_group + (row % s.I) * s.ldo : row * s.ldo;
    put((TO*)s.out + o + j, v, g.accumulate);
  }
}

template <typename T, typename TO, int FORM, int BM, int BN, int WM, int WN, int KB, bool FEW = false>
static int launch_general_tile(const GmmArgs& g, long items, int cus, hipStream_t st) {
  // workgroups that a CU holds: by LDS, and by the registers that the kernel
  // leaves for two workgroups of 128 x 128
  constexpr int LDS = 2 * (BM + BN) * KB + 4200;
  constexpr int FIT = 160 * 1024 / LDS < 4 ? 160 * 1024 / LDS : 4;
  long grid = (long)cus * FIT;
  grid = grid < 8 ? grid : grid / 8 * 8;
  if (grid > items) grid = (items + 7) / 8 * 8;
  hipLaunchKernelGGL((gmm_general_kernel<T, TO, FORM, BM, BN, WM, WN, KB, FEW>), dim3((unsigned)grid),
                     dim3(64 * WM * WN), 0, st, g);
  return check_launch();
}

// Tile choice.  FWD and DX go by the rows a group has on average (measured over
// 64 groups of W [2048, 2048] in fp32, [2047, 2047] in bf16, us):
//   rows               2    8   16   24   32   48   64   96  128  256
//   fp32  FWD  32x64  166  184  210  239  306  394  462  644  790 1452
//              64x64  216  260  243  259  317  350  490  636  787 1383
//             128x128 623  590  566  564  557  557  559  567  835 1384
//   bf16  FWD  32x64   99  118  121  140  169  191  223  300  375  670
//              64x64  122  156  165  160  160  167  224  277  332  554
//             128x128 153  168  170  158  158  160  161  177  235  379
// (DX alike.)  32-row tiles up to 32 rows; from 64 on, and in DW, 128 x 128 unless
// the CUs then have more to do than with 64 x 64, which run at 10/11 of the rate
// in fp32 and 10/16 in bf16 (DW, 256 rows: 1308 and 1456 us; 560 and 761).
// fp32 products that leave half the CUs idle take 32 x 32 tiles in longer steps:
// they are bound by the latency of their steps (64 rows by [511, 511]: 12.4 us,
// with 64 x 64 18 to 20; in bf16 no difference).
template <typename T, typename TO, int FORM>
static int launch_general(const GmmArgs& g, hipStream_t st) {
  // tiles go by the device's CUs, grids by the stream's: the order of a sum
  // follows from the tile, and is the same on every stream
  const int cus = device_cu_count(), own = stream_cu_count(st);
  if (cus <= 0 || own <= 0) return MOE_EHIP;
  constexpr bool DW = FORM == MOE_GMM_DW;
  auto bound = [&](long bm, long bn) {
    long n = 0;
    for (int q = 0; q < g.nsub; ++q)
      n += ((g.s[q].J + bn - 1) / bn) * (DW ? (g.s[q].I + bm - 1) / bm : 1);
    const long m = DW ? (long)g.ngroups : (long)g.M / bm + (g.M < g.ngroups ? g.M : g.ngroups);
    return n * m * g.nsplit;
  };
  // tiles to expect: half a row tile of each group stays empty
  auto expect = [&](long b) {
    const long over = g.M < g.ngroups ? g.M : g.ngroups;
    return DW ? bound(b, b) : bound(b, b) * ((g.M + b - 1) / b + over / 2) / (g.M / b + over);
  };
  if (bound(32, 32) < 1) return MOE_OK;
  // contiguous rows shorter than a chunk
  constexpr int CE = 16 / sizeof(T);
  bool few = !DW && g.R < CE;
  for (int q = 0; q < g.nsub; ++q)
    few = few || (FORM != MOE_GMM_FWD && g.s[q].J < CE) || (DW && g.s[q].I < CE);
  if (few) return launch_general_tile<T, TO, FORM, 64, 64, 2, 2, 128, true>(g, bound(64, 64), own, st);
  const int per = g.M / g.ngroups;
  if constexpr (sizeof(T) == 4) {
    if (2 * bound(64, 64) < cus)
      return launch_general_tile<T, TO, FORM, 32, 32, 2, 2, 256>(g, bound(32, 32), own, st);
  }
  if constexpr (!DW) {
    if (per < 32) return launch_general_tile<T, TO, FORM, 32, 64, 1, 4, 256>(g, bound(32, 64), own, st);
  }
  // outputs that the busiest CU computes
  auto turns = [&](long b) { return (expect(b) + cus - 1) / cus * b * b; };
  if ((DW || per >= 64) && 10 * turns(128) <= (sizeof(T) == 4 ? 11 : 16) * turns(64))
    return launch_general_tile<T, TO, FORM, 128, 128, 2, 4, 128>(g, bound(128, 128), own, st);
  return launch_general_tile<T, TO, FORM, 64, 64, 2, 2, 128>(g, bound(64, 64), own, st);
}

template <typename T, typename TO>
static int launch_general_form(int form, const GmmArgs& g, hipStream_t st) {
  if (form == MOE_GMM_FWD) return launch_general<T, TO, MOE_GMM_FWD>(g, st);
  if (form == MOE_GMM_DX) return launch_general<T, TO, MOE_GMM_DX>(g, st);
  return launch_general<T, TO, MOE_GMM_DW>(g, st);
}

int launch_gmm_general(int form, int dtype, int out_dtype, const GmmArgs& g, hipStream_t st) {
  if (dtype == MOE_F32) return launch_general_form<float, float>(form, g, st);
  if (out_dtype == MOE_F32) return launch_general_form<__bf16, float>(form, g, st);
  return launch_general_form<__bf16, __bf16>(form, g, st);
}

MOE_CHECK_ACCESSOR(check_word_gmm_general)

int launch_gmm_join(int form, int out_dtype, const GmmArgs& g, hipStream_t st) {
  const long n = (form == MOE_GMM_DW ? (long)g.ngroups * g.s[0].I : (long)g.M) * g.s[0].J;
  if (n < 1) return MOE_OK;
  const long blocks = (n + 255) / 256;
  const dim3 grid((unsigned)(blocks < 4096 ? blocks : 4096));
#define MOE_GMM_JOIN(TO, F) hipLaunchKernelGGL((gmm_join_kernel<TO, F>), grid, dim3(256), 0, st, g)
  if (form == MOE_GMM_DW) {
    if (out_dtype == MOE_F32) MOE_GMM_JOIN(float, MOE_GMM_DW);
    else MOE_GMM_JOIN(__bf16, MOE_GMM_DW);
  } else {  // FWD and DX alike
    if (out_dtype == MOE_F32) MOE_GMM_JOIN(float, MOE_GMM_FWD);
    else MOE_GMM_JOIN(__bf16, MOE_GMM_FWD);
  }
#undef MOE_GMM_JOIN
  return check_launch();
}

}  // namespace moe

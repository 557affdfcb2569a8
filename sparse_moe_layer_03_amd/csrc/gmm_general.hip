// Grouped matrix products for any sizes, row strides and element types: the
// forward product of a grouped linear map and the gradients of its rows and
// of its weights.
//
//   out[i, j] = sum_r A(i, r) B(j, r)
//     FWD  A = lhs[row, r]   B = W_e[j, r]     (r contiguous in both)
//     DX   A = lhs[row, r]   B = W_e[r, j]     (j contiguous in B)
//     DW   A = lhs[row, i]   B = rhs[row, j]   (r is the row)
//
// Both operands are brought into LDS as fp32, reduction-major (32 or 64
// values of r, each with the tile's i or j side by side), whatever their layout and
// type in memory; 16x16x4 fp32 MFMAs take one value per lane from there.  A
// product of two bf16 values is exact in fp32, so one kernel serves both
// types.  Rows of LDS are padded by 16 floats: the four r of a fragment read
// then start 16 banks apart and 64 lanes read without conflict.  The next
// step's elements wait in registers while a step computes; two LDS stages,
// one barrier a step.  Bound by the fp32 matrix rate (1/16 of bf16's).
//
// A workgroup walks over the tiles of all groups; it finds the groups from
// their offsets itself, so the host need not know them.

#include "common.h"
#include "train.h"

namespace moe {

constexpr int kGmmMaxGroups = 1024;

template <typename T>
__device__ __forceinline__ float elem(const T* p) {
  return ElemOps<T>::to_f(*p);
}

// Four neighbouring elements as floats; `left` of them exist.
template <typename T, bool VEC>
__device__ __forceinline__ f32x4_t load4(const T* p, int left) {
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  if (VEC && left >= 4) {
    if constexpr (sizeof(T) == 4) {
      v = *reinterpret_cast<const f32x4_t*>(p);
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      v[0] = __uint_as_float(w.x << 16);
      v[1] = __uint_as_float(w.x & 0xffff0000u);
      v[2] = __uint_as_float(w.y << 16);
      v[3] = __uint_as_float(w.y & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < left) v[k] = elem(p + k);
  }
  return v;
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

template <typename T, typename TO, int FORM, int BM, bool VEC>
__global__ void __launch_bounds__(256)
gmm_general_kernel(GmmArgs g) {
  constexpr int BK = BM == 32 ? 64 : 32, LDT = BM + 16, WT = BM / 2, NB = WT / 16, CH = BM * BK / 1024;
  constexpr bool A_RED = FORM != MOE_GMM_DW, B_RED = FORM == MOE_GMM_FWD;
  __shared__ __attribute__((aligned(16))) float s_a[2][BK * LDT];
  __shared__ __attribute__((aligned(16))) float s_b[2][BK * LDT];
  __shared__ int s_pref[FORM == MOE_GMM_DW ? 1 : kGmmMaxGroups + 1];
  __shared__ int s_tmp[4];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int r16 = lane & 15, q4 = lane >> 4;
  auto tiles_of = [](int n) { return (n + BM - 1) / BM; };
  // tiles of the products: per row tile (FWD, DX), per group (DW)
  int n_sub[3];
#pragma unroll
  for (int q = 0; q < 3; ++q)
    n_sub[q] = q < g.nsub ? tiles_of(g.s[q].J) * (FORM == MOE_GMM_DW ? tiles_of(g.s[q].I) : 1) : 0;
  const int per = n_sub[0] + n_sub[1] + n_sub[2];

  // FWD, DX: prefix over the groups of their row tiles
  if (FORM != MOE_GMM_DW) {
    constexpr int PER = kGmmMaxGroups / 256;
    const int most = g.M / BM + g.ngroups;  // row tiles that ascending offsets can give
    int loc[PER], run = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int e = tid * PER + k;
      if (e < g.ngroups) {
        int lo, hi;
        group_rows(g.offsets, e, g.M, lo, hi);
        run = min(run + (hi - lo + BM - 1) / BM, most + 1);
      }
      loc[k] = run;
    }
    const int base = block_inclusive_scan<256>(run, s_tmp) - run;
    if (tid == 0) s_pref[0] = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k)
      if (tid * PER + k < g.ngroups) s_pref[tid * PER + k + 1] = base + loc[k];
    __syncthreads();
  }
  const int row_tiles = FORM == MOE_GMM_DW ? g.ngroups : s_pref[g.ngroups];
  if (FORM != MOE_GMM_DW && row_tiles > g.M / BM + g.ngroups) return;  // offsets not ascending
  const long tiles = (long)row_tiles * per;
  const long items = tiles * g.nsplit;

  for (long item = blockIdx.x; item < items; item += gridDim.x) {
    const long t = item / g.nsplit;
    const int split = (int)(item - t * g.nsplit);
    const int m = (int)(t / per);
    int local = (int)(t - (long)m * per);
    GmmSub sub = g.s[0];
    if (local >= n_sub[0]) {
      local -= n_sub[0];
      sub = g.s[1];
      if (local >= n_sub[1]) {
        local -= n_sub[1];
        sub = g.s[2];
      }
    }
    const int jt = tiles_of(sub.J);
    const int tj = local % jt;
    int e, i0, rows, I, R;
    long row0;
    if (FORM == MOE_GMM_DW) {
      e = m;
      i0 = (local / jt) * BM;
      int lo, hi;
      group_rows(g.offsets, e, g.M, lo, hi);
      row0 = lo;
      rows = hi - lo;
      I = sub.I;
      R = rows;
    } else {
      int lo_e = 0, hi_e = g.ngroups - 1;  // last group with s_pref <= m
      while (lo_e < hi_e) {
        const int mid = (lo_e + hi_e + 1) >> 1;
        if (s_pref[mid] <= m) lo_e = mid; else hi_e = mid - 1;
      }
      e = lo_e;
      int lo, hi;
      group_rows(g.offsets, e, g.M, lo, hi);
      row0 = lo;
      rows = hi - lo;
      i0 = (m - s_pref[e]) * BM;
      I = rows;
      R = g.R;
    }
    const int j0 = tj * BM;
    // this split's range of the reduction, in whole steps
    const int steps = (R + BK - 1) / BK;
    const int len = (steps + g.nsplit - 1) / g.nsplit;
    const int r_lo = min(split * len, steps) * BK, r_hi = min(R, min((split + 1) * len, steps) * BK);

    const T* a = (const T*)sub.a + (A_RED ? (row0 + i0) * sub.lda : row0 * sub.lda + i0);
    const long b_at = B_RED ? e * g.b_group + (long)j0 * sub.ldb
                            : (FORM == MOE_GMM_DX ? e * g.b_group : row0 * sub.ldb) + j0;
    const T* b = (const T*)sub.b + b_at;
    const T* b2 = FORM == MOE_GMM_DX && g.r_switch ? (const T*)g.b2 + b_at : b;
    const int rb_hi = FORM == MOE_GMM_DX ? min(r_hi, g.RB) : r_hi;
    const int rb2_hi = min(r_hi, g.r_switch + g.RB);

    // Sums of 128 products in acc, their sum in tot: a long fp32 reduction
    // rounds like sqrt(128) + sqrt(n / 128) instead of sqrt(n) additions.
    constexpr int FLUSH = 128 / BK;
    f32x4_t acc[NB][NB], tot[NB][NB];
    int since = 0;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = tot[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // chunk c of this thread: four elements that lie side by side in memory
    auto fetch = [&](bool red, const T* base, long ld, int wide, int r0, int r_end, f32x4_t* v) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int x = tid + c * 256;
        if (red) {  // row x % BM, r = 4 (x / BM) ..
          const int w = x % BM, r = r0 + (x / BM) * 4;
          v[c] = w < wide ? load4<T, VEC>(base + w * ld + r, r_end - r) : f32x4_t{0.f, 0.f, 0.f, 0.f};
        } else {    // r = x / (BM / 4), columns 4 (x % (BM / 4)) ..
          const int w = (x % (BM / 4)) * 4, r = r0 + x / (BM / 4);
          v[c] = r < r_end ? load4<T, VEC>(base + r * ld + w, wide - w) : f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
      }
    };
    auto store = [&](bool red, float* s, const f32x4_t* v) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int x = tid + c * 256;
        if (red) {
          const int w = x % BM, r = (x / BM) * 4;
#pragma unroll
          for (int k = 0; k < 4; ++k) s[(r + k) * LDT + w] = v[c][k];
        } else {
          *reinterpret_cast<f32x4_t*>(&s[(x / (BM / 4)) * LDT + (x % (BM / 4)) * 4]) = v[c];
        }
      }
    };

    f32x4_t va[CH], vb[CH];
    const int wide_a = I - i0, wide_b = sub.J - j0;
    auto fetch_ab = [&](int r) {
      fetch(A_RED, a, sub.lda, wide_a, r, r_hi, va);
      if (FORM == MOE_GMM_DX && g.r_switch && r >= g.r_switch)
        fetch(B_RED, b2 - (long)g.r_switch * sub.ldb, sub.ldb, wide_b, r, rb2_hi, vb);
      else
        fetch(B_RED, b, sub.ldb, wide_b, r, rb_hi, vb);
    };
    __syncthreads();  // the previous tile's last reads of LDS
    if (r_lo < r_hi) fetch_ab(r_lo);
    int st = 0;
    for (int r = r_lo; r < r_hi; r += BK, st ^= 1) {
      store(A_RED, s_a[st], va);
      store(B_RED, s_b[st], vb);
      __syncthreads();
      if (r + BK < r_hi) fetch_ab(r + BK);
#pragma unroll
      for (int k = 0; k < BK; k += 4) {
        float fa[NB], fb[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) fa[i] = s_a[st][(k + q4) * LDT + wm * WT + i * 16 + r16];
#pragma unroll
        for (int j = 0; j < NB; ++j) fb[j] = s_b[st][(k + q4) * LDT + wn * WT + j * 16 + r16];
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fb[j], fa[i], acc[i][j], 0, 0, 0);
      }
      if (++since == FLUSH || r + BK >= r_hi) {
        since = 0;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            tot[i][j] += acc[i][j];
            acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
          }
      }
    }

    // b was the MFMA's row operand: a lane holds columns 4 q4 .. + 3 of row r16
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int ii = i0 + wm * WT + i * 16 + r16;
      if (ii >= I) continue;
      const long orow = FORM == MOE_GMM_DW ? (long)e * g.out_group + (long)ii * sub.ldo
                                           : (row0 + ii) * sub.ldo;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int jj = j0 + wn * WT + j * 16 + q4 * 4;
        if (jj >= sub.J) continue;
        if (g.nsplit > 1) {
          // partial outputs are compact: [split][row or group * I + i][J]
          const long prow = FORM == MOE_GMM_DW ? (long)e * sub.I + ii : row0 + ii;
          float* p = g.part + split * g.part_stride + prow * sub.J + jj;
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (jj + v < sub.J) p[v] = tot[i][j][v];
        } else {
          TO* p = (TO*)sub.out + orow + jj;
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (jj + v < sub.J) put(p + v, tot[i][j][v], g.accumulate);
        }
      }
    }
  }
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

template <typename T, typename TO, int FORM>
static int launch_general(bool vec, const GmmArgs& g, hipStream_t st) {
  const int cus = stream_cu_count(st);
  if (cus <= 0) return MOE_EHIP;
  auto bound = [&](long bm) {
    long n = 0;
    for (int q = 0; q < g.nsub; ++q)
      n += ((g.s[q].J + bm - 1) / bm) * (FORM == MOE_GMM_DW ? (g.s[q].I + bm - 1) / bm : 1);
    const long m = FORM == MOE_GMM_DW ? (long)g.ngroups
                                      : (long)g.M / bm + (g.M < g.ngroups ? g.M : g.ngroups);
    return n * m * g.nsplit;
  };
  // 128 x 128 tiles when they fill the chip twice over, 64 x 64 when they give
  // half the CUs one; else 32 x 32 in longer steps: a small product is bound
  // by the latency of its steps (64 tokens, reduction 512: 24.6 -> 12.4 us)
  const int bm = bound(128) >= 2L * cus ? 128 : 2 * bound(64) >= cus ? 64 : 32;
  const long items = bound(bm);
  if (items < 1) return MOE_OK;
  const long most = (long)cus * (bm == 128 ? 2 : 3);
  const dim3 grid((unsigned)(items < most ? items : most));
#define MOE_GMM_GEN(BM)                                                                          \
  if (vec)                                                                                       \
    hipLaunchKernelGGL((gmm_general_kernel<T, TO, FORM, BM, true>), grid, dim3(256), 0, st, g);  \
  else                                                                                           \
    hipLaunchKernelGGL((gmm_general_kernel<T, TO, FORM, BM, false>), grid, dim3(256), 0, st, g)
  if (bm == 128) {
    MOE_GMM_GEN(128);
  } else if (bm == 64) {
    MOE_GMM_GEN(64);
  } else {
    MOE_GMM_GEN(32);
  }
#undef MOE_GMM_GEN
  return check_launch();
}

template <typename T, typename TO>
static int launch_general_form(int form, bool vec, const GmmArgs& g, hipStream_t st) {
  if (form == MOE_GMM_FWD) return launch_general<T, TO, MOE_GMM_FWD>(vec, g, st);
  if (form == MOE_GMM_DX) return launch_general<T, TO, MOE_GMM_DX>(vec, g, st);
  return launch_general<T, TO, MOE_GMM_DW>(vec, g, st);
}

int launch_gmm_general(int form, int dtype, int out_dtype, bool vec, const GmmArgs& g,
                       hipStream_t st) {
  if (dtype == MOE_F32) return launch_general_form<float, float>(form, vec, g, st);
  if (out_dtype == MOE_F32) return launch_general_form<__bf16, float>(form, vec, g, st);
  return launch_general_form<__bf16, __bf16>(form, vec, g, st);
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

// Grouped products of 8-bit rows and weights for any sizes and strides, and the
// join of split reductions.
//
// Rows may start at any byte.  A chunk is one 16-byte load at its own address
// (this target's global loads take any alignment); at a row's end the load
// moves back to the row's last 16 bytes and what it has too much in front is
// shifted out.  The next step's chunks wait in registers while a step
// computes; two LDS stages, one barrier a step.  A workgroup walks over the
// tiles of all groups, which it finds from the offsets itself.
//
// Bound by the loads' address work beside the MFMAs: 8191 rows by [2047, 2049]
// 105 us (0.65 POP/s); 389 rows by [1001, 2049] 12.6 us in 3 ranges of K, and 4.4
// to join them.

#include <algorithm>

#include "block.h"
#include "common.h"
#include "gmm_tile.h"

namespace moe {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef u32x4_t u32x4_byte_t __attribute__((aligned(1)));
typedef f32x4_t f32x4_any_t __attribute__((aligned(4)));
typedef i32x4_t i32x4_any_t __attribute__((aligned(4)));
typedef u32x2_t u32x2_any_t __attribute__((aligned(2)));

// v without its first n bytes (1 .. 15), zeros behind.
__device__ __forceinline__ u32x4_t drop_bytes(u32x4_t v, int n) {
  uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
  if (n & 8) {
    lo = hi;
    hi = 0;
  }
  const int b = (n & 7) * 8;
  if (b) {
    lo = lo >> b | hi << (64 - b);
    hi >>= b;
  }
  return u32x4_t{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// 16 codes of a row of K from place k on, zeros behind its end.
__device__ __forceinline__ u32x4_t load_codes(const int8_t* row, int k, int K) {
  if (k + 16 <= K) return *reinterpret_cast<const u32x4_byte_t*>(row + k);
  if (k >= K) return u32x4_t{0u, 0u, 0u, 0u};
  if (K >= 16) return drop_bytes(*reinterpret_cast<const u32x4_byte_t*>(row + K - 16), k + 16 - K);
  int8_t e[16];  // (k is 0)
#pragma unroll
  for (int i = 0; i < 16; ++i) e[i] = i < K ? row[i] : (int8_t)0;
  u32x4_t v;
  __builtin_memcpy(&v, e, 16);
  return v;
}

// Four neighbouring columns of which `left` exist.
__device__ __forceinline__ void put4(float* p, f32x4_t v, int left) {
  if (left >= 4) {
    *reinterpret_cast<f32x4_any_t*>(p) = v;
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < left) p[k] = v[k];
  }
}
__device__ __forceinline__ void put4(__bf16* p, f32x4_t v, int left) {
  if (left >= 4) {
    __bf16 o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = (__bf16)v[k];
    *reinterpret_cast<u32x2_any_t*>(p) = __builtin_bit_cast(u32x2_t, o);
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < left) p[k] = (__bf16)v[k];
  }
}

// BM x BN tiles, 2 x 2 waves.
template <typename TO, int BM, int BN>
__global__ void __launch_bounds__(256, 2) i8_general_kernel(I8Args g) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NT = 256, KS = 128;
  using TA = Tile<false, BM, 4, KS / 2>;
  using TB = Tile<false, BN, 4, KS / 2>;
  constexpr int MB = BM / 32, NB = BN / 32;
  constexpr int CA = BM * KS / 16 / NT, CB = BN * KS / 16 / NT;  // chunks a thread
  __shared__ __attribute__((aligned(16))) char s_a[2][TA::BYTES], s_b[2][TB::BYTES];
  __shared__ int s_pref[kMfmaMaxGroups + 1], s_scan[NT / 64];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uni(tid >> 6), wm = wave >> 1, wn = wave & 1;
  const int l16 = lane & 15, l4 = lane >> 4;
  const int a_lane = TA::lane_base(lane, wm * MB), b_lane = TB::lane_base(lane, wn * NB);
  const int jt = (g.N + BN - 1) / BN;

  constexpr int PER = (kMfmaMaxGroups + NT - 1) / NT;
  const int most = g.M / BM + g.ngroups;
  int loc[PER], run = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int e = tid * PER + k;
    if (e < g.ngroups) {
      int lo = 0, hi = g.M;
      if (g.offsets != nullptr) rows_of(g.offsets, e, g.M, lo, hi);
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
  const long tiles = row_tiles <= most ? (long)row_tiles * jt * g.nsplit : 0;

  for (long n = blockIdx.x; n < tiles; n += gridDim.x) {
    const int split = (int)(n % g.nsplit);
    const int m = (int)(n / g.nsplit / jt), j0 = (int)(n / g.nsplit % jt) * BN;
    int e = 0, last = g.ngroups - 1;  // last group with s_pref <= m
    while (e < last) {
      const int mid = (e + last + 1) >> 1;
      if (s_pref[mid] <= m) e = mid; else last = mid - 1;
    }
    int lo = 0, hi = g.M;
    if (g.offsets != nullptr) rows_of(g.offsets, e, g.M, lo, hi);
    const int i0 = lo + (m - s_pref[e]) * BM, rows = min(BM, hi - i0), cols = min(BN, g.N - j0);
    const int steps = (g.K + KS - 1) / KS, per = (steps + g.nsplit - 1) / g.nsplit;
    const int k_lo = min(split * per, steps), k_hi = min(steps, k_lo + per);
    const int8_t* wb = g.b + ((int64_t)e * g.N + j0) * g.K;

    i32x4_t acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
    u32x4_t ra[CA], rb[CB];
    auto load = [&](int ks) {
#pragma unroll
      for (int q = 0; q < CA; ++q) {
        const int r = (tid + q * NT) / 8, k = ks * KS + (tid & 7) * 16;
        ra[q] = r < rows ? load_codes(g.a + (int64_t)(i0 + r) * g.lda, k, g.K) : u32x4_t{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int q = 0; q < CB; ++q) {
        const int r = (tid + q * NT) / 8, k = ks * KS + (tid & 7) * 16;
        rb[q] = r < cols ? load_codes(wb + (int64_t)r * g.K, k, g.K) : u32x4_t{0u, 0u, 0u, 0u};
      }
    };
    auto keep = [&](int stage) {
#pragma unroll
      for (int q = 0; q < CA; ++q) {
        const int r = (tid + q * NT) / 8;
        *reinterpret_cast<u32x4_t*>(s_a[stage] + r * KS + (((tid & 7) ^ TA::turn(r)) << 4)) = ra[q];
      }
#pragma unroll
      for (int q = 0; q < CB; ++q) {
        const int r = (tid + q * NT) / 8;
        *reinterpret_cast<u32x4_t*>(s_b[stage] + r * KS + (((tid & 7) ^ TB::turn(r)) << 4)) = rb[q];
      }
    };
    if (k_lo < k_hi) {
      load(k_lo);
      keep(0);
    }
    __syncthreads();
    for (int ks = k_lo; ks < k_hi; ++ks) {
      const int stage = (ks - k_lo) & 1;
      if (ks + 1 < k_hi) load(ks + 1);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        i32x4_t fa[MB], fb[NB];
#pragma unroll
        for (int i = 0; i < MB; ++i)
          fa[i] = __builtin_bit_cast(i32x4_t, TA::frag(s_a[stage], a_lane, i, kk));
#pragma unroll
        for (int j = 0; j < NB; ++j)
          fb[j] = __builtin_bit_cast(i32x4_t, TB::frag(s_b[stage], b_lane, j, kk));
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
      }
      if (ks + 1 < k_hi) keep(stage ^ 1);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int r = (wm * MB + i) * 16 + l16;
      if (r >= rows) continue;
      const int64_t p = i0 + r;
      const float sa = g.nsplit > 1 ? 0.f : g.sa[p];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int jj = j0 + (wn * NB + j) * 16 + l4 * 4, left = g.N - jj;
        if (left <= 0) continue;
        if (g.nsplit > 1) {
          int32_t* to = g.part + ((int64_t)split * g.M + p) * g.N + jj;
          if (left >= 4) {
            *reinterpret_cast<i32x4_any_t*>(to) = acc[i][j];
          } else {
#pragma unroll
            for (int v = 0; v < 3; ++v)
              if (v < left) to[v] = acc[i][j][v];
          }
        } else {
          f32x4_t o;
#pragma unroll
          for (int v = 0; v < 4; ++v)
            o[v] = (float)acc[i][j][v] * sa * g.sb[(int64_t)e * g.N + min(jj + v, g.N - 1)];
          put4((TO*)g.out + p * g.ldo + jj, o, left);
        }
      }
    }
  }
#endif
}

template <typename TO, int BM, int BN>
static int launch_general(const I8Args& g, hipStream_t st) {
  const int cus = stream_cu_count(st);
  if (cus <= 0) return MOE_EHIP;
  const long most = (long)(g.M / BM + std::min(g.M, g.ngroups)) * ((g.N + BN - 1) / BN) * g.nsplit;
  const long grid = std::min<long>(most, 2l * cus);
  if (grid < 1) return MOE_OK;
  hipLaunchKernelGGL((i8_general_kernel<TO, BM, BN>), dim3((unsigned)grid), dim3(256), 0, st, g);
  return check_launch();
}

int launch_i8_general(int out_dtype, const I8Args& g, hipStream_t st) {
  // 128 x 128 tiles where they fill the chip and groups have the rows: us with
  // 64 x 64 and 128 x 128, 8191 x 2047 of K 2049 185, 105; 1001 x 1001 of 1001 14,
  // 24; 64 groups, 8191 x 1001 of 1001 67, 50; 3000 x 1001 of 2049 56, 53
  const int cus = stream_cu_count(st);
  if (cus <= 0) return MOE_EHIP;
  const long t128 = (long)(g.M / 128 + std::min(g.M, g.ngroups)) * ((g.N + 127) / 128) * g.nsplit;
  const bool big = t128 >= cus && g.M / g.ngroups >= 64;
  if (out_dtype == MOE_F32)
    return big ? launch_general<float, 128, 128>(g, st) : launch_general<float, 64, 64>(g, st);
  return big ? launch_general<__bf16, 128, 128>(g, st) : launch_general<__bf16, 64, 64>(g, st);
}

// One row a workgroup: the splits' sums added (whole numbers: any order gives
// the same) and scaled.
template <typename TO>
__global__ void __launch_bounds__(256) i8_join_kernel(I8Args g) {
  int first = 0, end = g.M;
  if (g.offsets != nullptr) {
    first = min(max(g.offsets[0], 0), g.M);
    end = min(max(g.offsets[g.ngroups], first), g.M);
  }
  for (int p = first + blockIdx.x; p < end; p += gridDim.x) {
    int e = 0, last = g.ngroups - 1;  // last group that starts at or before p
    if (g.offsets != nullptr)
      while (e < last) {
        const int mid = (e + last + 1) >> 1;
        if (g.offsets[mid] <= p) e = mid; else last = mid - 1;
      }
    const float sa = g.sa[p];
    const float* sb = g.sb + (int64_t)e * g.N;
    for (int j = blockIdx.y * 256 + threadIdx.x; j < g.N; j += gridDim.y * 256) {
      int sum = 0;
#pragma unroll 4
      for (int q = 0; q < g.nsplit; ++q) sum += g.part[((int64_t)q * g.M + p) * g.N + j];
      ((TO*)g.out)[p * g.ldo + j] = ElemOps<TO>::from_f((float)sum * sa * sb[j]);
    }
  }
}

int launch_i8_join(int out_dtype, const I8Args& g, hipStream_t st) {
  const dim3 grid((unsigned)std::min(g.M, 4096), (unsigned)std::min(64, (g.N + 255) / 256));
  if (out_dtype == MOE_F32)
    hipLaunchKernelGGL(i8_join_kernel<float>, grid, dim3(256), 0, st, g);
  else
    hipLaunchKernelGGL(i8_join_kernel<__bf16>, grid, dim3(256), 0, st, g);
  return check_launch();
}

MOE_CHECK_ACCESSOR(check_word_i8_general)

}  // namespace moe

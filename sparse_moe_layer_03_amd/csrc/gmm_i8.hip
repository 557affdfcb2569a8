// Grouped products of 8-bit rows and weights on int8 MFMAs, for rows that are
// multiples of 16 bytes: with the scales of rows and output channels applied
// behind the reduction, or SwiGLU of the gate's and the up product.
//
// The 16x16x64 int8 MFMA takes 16 bytes a lane and operand and as many cycles as
// the bf16 one over half the depth: a tile has the bytes of a bf16 tile and
// twice its products, so its geometry is that of the bf16 products' forward form
// (direct-to-LDS loads, swizzled slots, rings of stages with one barrier a
// step, a persistent grid that works out the next tile and asks for its first
// stages before this tile's stores).  Sums are whole numbers, exact in 32 bits,
// and so do not depend on the split of a long reduction.
//
// With half the bytes a weight and twice the rate, loads bound it up to some 250
// rows a group, so every step issues the same number of loads and waits for
// those that it needs only (load_a below).
//
// Measured for 16384 tokens, 12 of 512 + 256 experts, d_model 6144, d_ff 2048:
// gate and up 3.5 ms (1.9 POP/s), down 2.1 ms (1.6); 65536 tokens 10.9 and 6.6 ms
// (2.4 and 2.0; a library product of 8192^3 2.1); 128 tokens 1.62 and 0.83 ms
// (6.9 TB/s).

#include <algorithm>
#include <type_traits>

#include "block.h"
#include "common.h"
#include "gmm_tile.h"

namespace moe {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef f32x4_t f32x4_any_t __attribute__((aligned(4)));

// silu(z) u: for a bf16 H by the hardware's exponential and reciprocal, some
// 2^-20 of the value off, a small part of the rounding that follows (2^-8); in 64
// bits for an fp32 H, whose codes hang on its last bits.
__device__ __forceinline__ float swiglu(float z, float u) {
  return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504f)) * u;
}
__device__ __forceinline__ double swiglu(double z, double u) { return z / (1.0 + exp(-z)) * u; }

// The rows of a group; all M where there are no offsets.
__device__ __forceinline__ void i8_rows(const int32_t* offsets, int e, int M, int& lo, int& hi) {
  if (offsets == nullptr) {
    lo = 0;
    hi = M;
  } else {
    rows_of_uniform(offsets, e, M, lo, hi);
  }
}

// SW: with b2, the tile's first half of columns are gate's, the second up's.
template <bool SW, typename TO, int BM, int BN, int WM, int WN, int SA, int SB, bool NT>
__global__ void __launch_bounds__(64 * WM * WN, 2)
gmm_i8_kernel(I8Args g) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NW = WM * WN, THREADS = 64 * NW, KS = 128;  // bytes a step
  using TA = Tile<false, BM, NW, KS / 2>;
  using TB = Tile<false, BN, NW, KS / 2>;
  constexpr int MB = BM / WM / 16, NB = BN / WN / 16;
  constexpr int A_PW = TA::PW, B_PW = TB::PW, PW = A_PW + B_PW;
  constexpr int HN = SW ? BN / 2 : BN;  // output columns per tile
  constexpr int MG = 4;
  constexpr int DA = SA - 1, DB = SB - 1;
  static_assert(TA::NP == 1 && TB::NP == 1 && (!SW || (NB % 2 == 0 && BN % 32 == 0)), "tile");
  static_assert(TB::BYTES > kMfmaMaxGroups * 4, "the groups' prefix fits a stage");
  static_assert(DA >= 1 && DB >= DA && SA <= 4 && SB <= 4 && SA * TA::BYTES + SB * TB::BYTES <= 160 * 1024,
                "LDS");
  __shared__ __attribute__((aligned(1024))) char s_a0[TA::BYTES];
  __shared__ __attribute__((aligned(1024))) char s_a1[TA::BYTES];
  __shared__ __attribute__((aligned(1024))) char s_a2[SA > 2 ? TA::BYTES : 16];
  __shared__ __attribute__((aligned(1024))) char s_a3[SA > 3 ? TA::BYTES : 16];
  __shared__ __attribute__((aligned(1024))) char s_b0[TB::BYTES];
  __shared__ __attribute__((aligned(1024))) char s_b1[TB::BYTES];
  __shared__ __attribute__((aligned(1024))) char s_b2[SB > 2 ? TB::BYTES : 16];
  __shared__ __attribute__((aligned(1024))) char s_b3[SB > 3 ? TB::BYTES : 16];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uni(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane & 15, l4 = lane >> 4;
  // a wave's row blocks interleave with the other waves', so that a short tile
  // loads all of them
  const int a_lane = TA::lane_base(lane, wm);
  const int b_lane = TB::lane_base(lane, SW ? wn * (NB / 2) : wn * NB);

  const int G = gridDim.x, bid = blockIdx.x;
  const int jt = (g.N + HN - 1) / HN;
  // tiles that run together on an XCD are neighbours
  const int vid = G % 8 == 0 ? (bid % 8) * (G / 8) + bid / 8 : bid;

  // (first row tile << 10 | group) of this workgroup's next 64 tiles, one per
  // lane, and the number of tiles
  uint32_t desc = 0;
  long tiles = 0;
  auto describe = [&](int k0) {
    int* s_pref = reinterpret_cast<int*>(s_b0);
    int* s_scan = reinterpret_cast<int*>(s_b1);
    constexpr int PER = (kMfmaMaxGroups + THREADS - 1) / THREADS;
    // ascending offsets give at most this many row tiles; more are cut off
    // here and computed nowhere
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
    const int base = block_inclusive_scan<THREADS>(run, s_scan) - run;
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
    int e, i0, i_end, j0, split, rows, row0;
    int k_lo, k_hi, r_end;  // its steps, and the end of its reduction
    const char *a_base, *b_base, *b_base2;
    uint32_t a_bytes, b_bytes;
    int once;               // no other tile reads this tile's part of b
  };
  const uint32_t lda = (uint32_t)g.lda, ldb = (uint32_t)g.K;
  // A load instruction brings RPI rows; a lane's place in them, and what chunk of
  // its row it fetches, are the same for all of a wave's instructions.
  const uint32_t chunk = (uint32_t)TA::chunk(0, wave, lane) * 16;
  // SwiGLU: a's rows lie in the tokens' order; what they are is asked for with
  // the tile's place, a tile ahead, and becomes the offsets of its loads.
  uint32_t a_off[SW ? A_PW : 1];
  int tok[SW ? A_PW : 1];
  a_off[0] = (uint32_t)(lane / (KS / 16)) * lda + chunk;
  const uint32_t b_off = (uint32_t)(lane / (KS / 16)) * ldb + chunk;

  // Tile number k of this workgroup; false behind the last one.
  auto setup = [&](int k, Place& t) -> bool {
    const long item = vid + (long)k * G;
    if (item >= tiles * g.nsplit) return false;
    long n = item;
    t.split = 0;
    if (g.nsplit > 1) {
      n = item / g.nsplit;
      t.split = (int)(item - n * g.nsplit);
    }
    const uint32_t d = (uint32_t)__builtin_amdgcn_readlane((int)desc, k & 63);
    t.e = uni((int)(d & 1023u));
    int lo, hi;
    i8_rows(g.offsets, t.e, g.M, lo, hi);
    t.row0 = uni(lo);
    t.rows = uni(hi - lo);
    // in a group: bands of MG row tiles, column by column, so that tiles that
    // run together share row and weight slices in L2
    const int mt = (t.rows + BM - 1) / BM;
    const int local = (int)(n - (long)(d >> 10) * jt);
    const int m0 = (local / (MG * jt)) * MG;
    const int mg = max(1, min(MG, mt - m0));
    const int in = local - m0 * jt;
    t.j0 = uni((in / mg) * HN);
    t.once = uni(mt == 1);
    const int h = ((t.rows + mt - 1) / mt + 15) & ~15;  // balanced height
    t.i0 = uni((m0 + in % mg) * h);
    t.i_end = uni(min(t.rows, t.i0 + h));
    t.split = uni(t.split);
    const int steps = (g.K + KS - 1) / KS;
    const int per = g.nsplit > 1 ? (steps + g.nsplit - 1) / g.nsplit : steps;
    t.k_lo = min(t.split * per, steps), t.k_hi = min(steps, t.k_lo + per);
    t.r_end = min(g.K, t.k_hi * KS);
    if constexpr (SW) {
      t.a_base = (const char*)g.a;
      t.a_bytes = g.a_bytes;
#pragma unroll
      for (int q = 0; q < A_PW; ++q) {
        const int r = t.i0 + (wave + q * NW) * TA::RPI + lane / (KS / 16);
        tok[q] = r < t.i_end ? g.tok[t.row0 + r] : -1;
      }
    } else {
      t.a_base = uni((const char*)g.a + (t.row0 + t.i0) * (int64_t)lda);
      t.a_bytes = t.i_end > t.i0 ? (uint32_t)(t.i_end - t.i0 - 1) * lda + (uint32_t)g.K : 0u;
    }
    const int64_t at = ((int64_t)t.e * g.N + t.j0) * ldb;
    t.b_base = uni((const char*)g.b + at);
    t.b_base2 = SW ? uni((const char*)g.b2 + at) : nullptr;
    t.b_bytes = (uint32_t)min(HN, g.N - t.j0) * ldb;
    return true;
  };

  auto stage_a = [&](auto sc) -> char* {
    constexpr int N = decltype(sc)::value % SA;
    return N == 0 ? s_a0 : N == 1 ? s_a1 : N == 2 ? s_a2 : s_a3;
  };
  auto stage_b = [&](auto sc) -> char* {
    constexpr int N = decltype(sc)::value % SB;
    return N == 0 ? s_b0 : N == 1 ? s_b1 : N == 2 ? s_b2 : s_b3;
  };
  // Load instruction q of step ks into a stage; what its wave-uniform part adds
  // to the lane offset goes through the scalar offset.  Steps behind the tile's
  // last one load zeros, with no memory access: so every step has the same
  // number of loads outstanding, and the compiler, which follows them through
  // the control flow, adds no waits of its own (with loads left out at the end
  // it had waited for all of them in every fourth step and more).
  auto load_a = [&](const Place& t, auto sc, int ks, int q) {
    const int i = wave + q * NW;
    const int left = t.r_end - ks * KS;
    const auto rs = descriptor(t.a_base, left > 0 ? t.a_bytes : 0u);
    uint32_t off = a_off[SW ? q : 0];
    if (left < KS) off = (int)chunk < left ? off : kOutside;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)(stage_a(sc) + i * 1024), 16, (int)off,
                                             ks * KS + (SW ? 0 : i * TA::RPI * (int)lda), 0, 0);
  };
  auto load_b1 = [&](const Place& t, auto sc, int ks, int q, auto cache) {
    constexpr int AUX = decltype(cache)::value;
    const int i = wave + q * NW;
    // SwiGLU: gate rows fill the first half of the tile, up rows the second
    const bool second = SW && i * TB::RPI >= BN / 2;
    const int r = i * TB::RPI - (second ? BN / 2 : 0);
    const int left = t.r_end - ks * KS;
    const auto rs = descriptor(second ? t.b_base2 : t.b_base, left > 0 ? t.b_bytes : 0u);
    uint32_t off = b_off;
    if (left < KS) off = (int)chunk < left ? off : kOutside;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)(stage_b(sc) + i * 1024), 16, (int)off,
                                             ks * KS + r * (int)ldb, 0, AUX);
  };
  // The step's b loads.  NT: tiles for few rows load weights that no other tile
  // reads non-temporally.
  auto load_b = [&](const Place& t, auto sc, int ks) {
    if (NT && uni(t.once) != 0) {
#pragma unroll
      for (int q = 0; q < B_PW; ++q) load_b1(t, sc, ks, q, std::integral_constant<int, kCpolNT>{});
    } else {
#pragma unroll
      for (int q = 0; q < B_PW; ++q) load_b1(t, sc, ks, q, std::integral_constant<int, 0>{});
    }
  };

  constexpr int UNROLL = SB % SA == 0 ? SB : SA * SB;
  static_assert(UNROLL <= 12, "code size");
  // A tile's first DA and DB steps, in the order in which the loop would
  // have asked for them.
  auto prologue = [&](const Place& t) {
    if constexpr (SW) {
#pragma unroll
      for (int q = 0; q < A_PW; ++q) a_off[q] = tok[q] < 0 ? kOutside : (uint32_t)tok[q] * lda + chunk;
    }
    auto one = [&](auto vc) {  // what step V of -DB .. -1 would load
      constexpr int V = decltype(vc)::value - DB;
      if constexpr (V + DA >= 0) {
#pragma unroll
        for (int q = 0; q < A_PW; ++q)
          load_a(t, std::integral_constant<int, V + DA>{}, t.k_lo + V + DA, q);
      }
      load_b(t, std::integral_constant<int, V + DB>{}, t.k_lo + V + DB);
    };
    auto each = [&](auto self, auto vc) {
      constexpr int V = decltype(vc)::value;
      if constexpr (V < DB) {
        one(vc);
        self(self, std::integral_constant<int, V + 1>{});
      }
    };
    each(each, std::integral_constant<int, 0>{});
  };
  // Loads issued after the last one that a step needs: a's of the next DA - 1
  // steps, and b's from (DB - DA) steps ahead on (with equal leads, b's own is
  // needed).
  constexpr int LATER = (DA - 1) * A_PW + (DB == DA ? DB - 1 : DA) * B_PW;
  static_assert(LATER < 64, "vmcnt");

  describe(0);
  Place t, next;
  if (!setup(0, t)) return;
  prologue(t);
  for (int k = 0;; ++k) {
    // the next tile's place, while this one's first loads are under way
    const bool early = ((k + 1) & 63) != 0;  // else it is not known yet
    bool have = early && setup(k + 1, next);
    i32x4_t acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};

    // Step ks, at place N of the unrolled loop, with MBA active row blocks.
    auto step = [&](auto mbac, auto nc, int ks) {
      constexpr int MBA = decltype(mbac)::value, N = decltype(nc)::value;
      const char* sa = stage_a(nc);
      const char* sb = stage_b(nc);
      wait_vm<LATER>();
      barrier_all();
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        i32x4_t fa[MBA], fb[NB];
#pragma unroll
        for (int i = 0; i < MBA; ++i)
          fa[i] = __builtin_bit_cast(i32x4_t, TA::frag(sa, a_lane, i * WM, kk));
#pragma unroll
        for (int j = 0; j < NB; ++j)
          fb[j] = __builtin_bit_cast(
              i32x4_t, TB::frag(sb, b_lane, SW && j >= NB / 2 ? BN / 32 + j - NB / 2 : j, kk));
        // into the stages that every wave has left at this step's barrier
        if (kk == 0) {
#pragma unroll
          for (int q = 0; q < A_PW; ++q) load_a(t, std::integral_constant<int, N + DA>{}, ks + DA, q);
        }
        if (kk == 1) load_b(t, std::integral_constant<int, N + DB>{}, ks + DB);
#pragma unroll
        for (int i = 0; i < MBA; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
    };

    auto loop = [&](auto mbac) {
      auto steps = [&](auto self, auto nc, int ks) -> bool {
        constexpr int N = decltype(nc)::value;
        step(mbac, nc, ks);
        if (ks + 1 >= t.k_hi) return false;
        if constexpr (N + 1 < UNROLL) return self(self, std::integral_constant<int, N + 1>{}, ks + 1);
        else return true;
      };
      for (int ks = t.k_lo; ks < t.k_hi; ks += UNROLL)
        if (!steps(steps, std::integral_constant<int, 0>{}, ks)) break;
    };
    if constexpr (MB == 1) {
      loop(std::integral_constant<int, MB>{});
    } else {
      // row blocks of this wave that hold rows (a wave without any still
      // loads and waits with the others, on one block that is not stored)
      const int nrb = (t.i_end - t.i0 + 15) / 16;
      const int mba = max(1, min(MB, (nrb - wm + WM - 1) / WM));
      auto pick = [&](auto self, auto nc) {
        constexpr int N = decltype(nc)::value;
        if constexpr (N == 1) loop(nc);
        else if (mba == N) loop(nc);
        else self(self, std::integral_constant<int, N - 1>{});
      };
      pick(pick, std::integral_constant<int, MB>{});
    }

    // ---- out.  b was the MFMA's row operand: lane (l16, l4) holds columns
    // 4 l4 .. 4 l4 + 3 of row l16 of a 16 x 16 block.
    const int J = g.N;
    const int jw = t.j0 + wn * (SW ? NB / 2 : NB) * 16;  // the wave's first column
    const int high = max(0, t.i_end - t.i0);             // rows of the tile
    // The scales, before the next tile's loads: a load waits for older ones only.
    constexpr int NC = SW ? NB / 2 : NB;
    float sa[MB];
    f32x4_t sb[NC], sb2[SW ? NC : 1];
    if (g.nsplit == 1) {
#pragma unroll
      for (int i = 0; i < MB; ++i)
        sa[i] = g.sa[t.row0 + min(t.i0 + (i * WM + wm) * 16 + l16, t.rows - 1)];
      const float* col = g.sb + (int64_t)t.e * J;
      const float* col2 = SW ? g.sb2 + (int64_t)t.e * J : nullptr;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int jj = min(jw + j * 16 + l4 * 4, J - 4);  // (J is a multiple of 4)
        sb[j] = *reinterpret_cast<const f32x4_any_t*>(col + jj);
        if constexpr (SW) sb2[j] = *reinterpret_cast<const f32x4_any_t*>(col2 + jj);
      }
    }
    // the next tile's first loads, before this one's stores: every wave is done
    // with the stages, and what they load has landed
    wait_vm<0>();
    if (early) {
      barrier_all();
      if (have) prologue(next);
    }
    // Stores go through a descriptor that ends with the tile's last row; columns
    // behind the last one are sent outside it.
    if (g.nsplit > 1) {
      const auto ro = descriptor(
          (const char*)(g.part + ((int64_t)t.split * g.M + t.row0 + t.i0) * J), (uint32_t)high * J * 4);
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const int jj = jw + j * 16 + l4 * 4;
          const uint32_t off = (uint32_t)((wm + i * WM) * 16 + l16) * J * 4 + jj * 4;
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[i][j]), ro,
                                                 jj < J ? off : kOutside, 0, 0);
        }
    } else {
      const auto ro = descriptor(
          uni((const char*)g.out + (int64_t)(t.row0 + t.i0) * g.ldo * (int64_t)sizeof(TO)),
          high > 0 ? ((uint32_t)(high - 1) * (uint32_t)g.ldo + J) * (uint32_t)sizeof(TO) : 0u);
      const uint32_t ldo_b = (uint32_t)g.ldo * (uint32_t)sizeof(TO);
      const bool wide = ((J | (int)g.ldo) & 7) == 0;
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const uint32_t row = (uint32_t)((wm + i * WM) * 16 + l16) * ldo_b;
        auto at = [&](int jj) { return jj < J ? row + (uint32_t)jj * (uint32_t)sizeof(TO) : kOutside; };
        f32x4_t o[NC];
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            if constexpr (!SW) {
              o[j][v] = (float)acc[i][j][v] * sa[i] * sb[j][v];
            } else if constexpr (sizeof(TO) == 4) {
              o[j][v] = (float)swiglu((double)acc[i][j][v] * (double)sa[i] * (double)sb[j][v],
                                      (double)acc[i][j + NC][v] * (double)sa[i] * (double)sb2[j][v]);
            } else {
              o[j][v] = swiglu((float)acc[i][j][v] * sa[i] * sb[j][v],
                               (float)acc[i][j + NC][v] * sa[i] * sb2[j][v]);
            }
          }
        if constexpr (sizeof(TO) == 4) {
#pragma unroll
          for (int j = 0; j < NC; ++j)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, o[j]), ro,
                                                   at(jw + j * 16 + l4 * 4), 0, 0);
        } else if (NC % 2 == 0 && wide) {  // whole 16-byte pieces
#pragma unroll
          for (int j = 0; j + 1 < NC; j += 2)
            __builtin_amdgcn_raw_buffer_store_b128(bf16x8(o[j], o[j + 1]), ro,
                                                   at(jw + j * 16 + bf16_col(l4)), 0, 0);
        } else {
#pragma unroll
          for (int j = 0; j < NC; ++j)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t, bf16x4(o[j])), ro,
                                                  at(jw + j * 16 + l4 * 4), 0, 0);
        }
      }
    }
    if (!early) {
      // the next 64 tiles' places are worked out in the stages
      wait_vm<0>();
      __syncthreads();
      describe(k + 1);
      have = setup(k + 1, next);
      if (have) prologue(next);
    }
    if (!have) break;
    t = next;
  }
#endif
}

MOE_CHECK_ACCESSOR(check_word_gmm_i8)

bool i8_mfma_ok(int N, int K, int64_t lda, int64_t ldo) {
  // 16-byte rows; a lane stores 4 neighbouring columns; a descriptor spans at
  // most 320 rows
  return K % 16 == 0 && lda % 16 == 0 && lda <= (1 << 20) && N % 4 == 0 && ldo % 4 == 0 && ldo <= (1 << 20);
}

template <bool SW, typename TO, int BM, int BN, int WM, int WN, int SA, int SB, bool NT>
static int launch_tile(const I8Args& g, hipStream_t st) {
  const int cus = stream_cu_count(st);
  if (cus <= 0) return MOE_EHIP;
  constexpr int HN = SW ? BN / 2 : BN;
  const long most = (long)(g.M / BM + std::min(g.M, g.ngroups)) * ((g.N + HN - 1) / HN) * g.nsplit;
  constexpr int LDS = (BM * SA + BN * SB) * 128;
  long grid = (long)cus * std::min(2, 160 * 1024 / LDS);
  if (grid > most) grid = most;
  if (grid > 8) grid -= grid % 8;
  if (grid < 1) return MOE_OK;
  hipLaunchKernelGGL((gmm_i8_kernel<SW, TO, BM, BN, WM, WN, SA, SB, NT>), dim3((unsigned)grid),
                     dim3(64 * WM * WN), 0, st, g);
  return check_launch();
}

// Tile choice by the rows that a group has on average (`rows`; measured over 512
// groups of W [2 x 2048, 6144] with SwiGLU, 12.9 GB of weights, ragged groups,
// us):
//   rows       8    32    64    96   128   192   224   256   288   512
//   64x256  1915  2223  2723  3321  3696
//   128x256 2123  2188  2391  2533  3034  3598
//   256x256 2209  2247  2467  2563  2676  3013  3217  3840  4367  6433
//   320x192             2666        3133  3317  3471  3718  3926  6494
// Weights that come once from HBM bound all of them at first (1915: 6.7 TB/s),
// so what counts is how far ahead they are asked for; a second row tile in a
// group loads them again from L2, which 320 rows avoid for groups just over
// 256.  Where a tile shape leaves CUs idle, smaller ones: the same products with
// 128 x 128 and 64 x 128 tiles, two workgroups on a CU.  Products without SwiGLU
// and of other K take the same rule, by this table: they were not measured over all
// shapes.  64 groups of some 340 rows, N 2048, K 1024 (256 x 256) run in 80 us where
// the operations would take 44: 8 steps a tile, and its stores with no MFMA beside them.
template <bool SW, typename TO>
static int launch_any(const I8Args& g, hipStream_t st) {
  const int cus = stream_cu_count(st);
  if (cus <= 0) return MOE_EHIP;
  const long per = g.rows / g.ngroups;
  auto tiles = [&](int bm, int bn) {
    const int hn = SW ? bn / 2 : bn;
    return (long)(g.rows / bm + std::min(g.rows, g.ngroups)) * ((g.N + hn - 1) / hn) * g.nsplit;
  };
  if (per >= 250 && per < 305 && tiles(320, 192) >= cus)
    return launch_tile<SW, TO, 320, 192, 4, 2, 2, 3, false>(g, st);
  if (per >= 112 && tiles(256, 256) >= cus) return launch_tile<SW, TO, 256, 256, 4, 2, 2, 3, false>(g, st);
  if (per >= 24) {
    if (tiles(128, 256) >= cus) return launch_tile<SW, TO, 128, 256, 2, 4, 3, 3, false>(g, st);
    if (per >= 64) return launch_tile<SW, TO, 128, 128, 2, 2, 2, 3, false>(g, st);
  } else if (tiles(64, 256) >= cus) {
    return launch_tile<SW, TO, 64, 256, 1, 8, 4, 4, true>(g, st);
  }
  return launch_tile<SW, TO, 64, 128, 1, 4, 3, 3, true>(g, st);
}

int launch_i8_mfma(int out_dtype, const I8Args& g, hipStream_t st) {
  const bool f32 = out_dtype == MOE_F32;
  if (g.b2 != nullptr) return f32 ? launch_any<true, float>(g, st) : launch_any<true, __bf16>(g, st);
  return f32 ? launch_any<false, float>(g, st) : launch_any<false, __bf16>(g, st);
}

}  // namespace moe

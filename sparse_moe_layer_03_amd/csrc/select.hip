// Selection of experts from the router's logits: softmax or sigmoid scores, a
// bias on the keys, groups of experts, top-k, renormalised gates; and the
// gradient at the logits.
//
// One wave per token, tokens in grid strides.  Lanes are dealt out to the
// groups: with G groups (rounded up to a power of two) lane l serves group
// l / L, L = 64 / G, and holds its experts l % L, l % L + L, ... in registers.
//
// The top k.  Keys are mapped to integers of the same order.  The k-th largest
// of the 64 lane maxima bounds the threshold from below (k keys reach it), so
// few keys beyond the k wanted are left; the surplus is taken off from below,
// one value a step.  (Building the threshold bit by bit from all keys takes 32
// ballots for each of a lane's keys.)  It is the way left where the surplus is
// large: few lanes in the kept groups, or keys in equal runs.
//
// Keys that fp32 cannot tell apart.  The fp32 key differs from the 64-bit one
// by less than half of `margin`; where another key lies within the margin of
// the threshold (of keys, or of group scores) the wave selects again with keys
// in 64 bits, in LDS.  That is rare: with random logits over 768 experts about
// 1 token of 1000 (softmax), 1 of 2000 (sigmoid).
//
// The kernel reads 4 bytes and spends some 10 instructions an expert; the
// gradient reads and writes 8.

#include <math.h>

#include <algorithm>

#include "block.h"
#include "common.h"

namespace moe {

constexpr int kMaxK = 16;

// ---- reductions over a wave without LDS: rows of 16 lanes by row_shr, then
// rows to rows; the result of lane 63, the same in every lane

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 0xf, false);
}
template <typename OP>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, uint32_t neutral, OP op) {
  v = op(v, dpp<0x111, 0xf>(neutral, v));  // row_shr 1
  v = op(v, dpp<0x112, 0xf>(neutral, v));
  v = op(v, dpp<0x114, 0xf>(neutral, v));
  v = op(v, dpp<0x118, 0xf>(neutral, v));
  v = op(v, dpp<0x142, 0xa>(neutral, v));  // lane 15 of rows 0, 2 to rows 1, 3
  v = op(v, dpp<0x143, 0xc>(neutral, v));  // lane 31 to rows 2, 3
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint32_t wave_min_u(uint32_t v) {
  return wave_reduce(v, ~0u, [](uint32_t a, uint32_t b) { return min(a, b); });
}
__device__ __forceinline__ float wave_max_f(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), 0xff800000u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
__device__ __forceinline__ float wave_sum_f(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), 0u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// exp(x): 2^(x log2 e) with the product's rounding error put back, off by
// about 2 steps.
__device__ __forceinline__ float exp_fast(float x) {
  constexpr float kL = 1.44269502162933349609f, kLo = 1.92596299e-8f;  // log2 e in two parts
  const float t = x * kL;
  const float rest = fmaf(x, kLo, fmaf(x, kL, -t));
  const float y = __builtin_amdgcn_exp2f(t);
  // (outside, y is 0, infinite or next to it, or NaN, and the rest may be NaN)
  return fabsf(t) < 126.f ? fmaf(y, rest * 0.693147182464599609375f, y) : y;
}

// A key mapped to an integer of the same order: NaN ranks as -inf, -0 as +0;
// above 0, which stands for "no key".
__device__ __forceinline__ uint32_t ordered(float key) {
  if (key != key) key = -INFINITY;
  const uint32_t b = __float_as_uint(key + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
__device__ __forceinline__ uint64_t ordered(double key) {
  if (key != key) key = -INFINITY;
  const uint64_t b = __double_as_longlong(key + 0.0);
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// A group's score from its two best keys: a second one of -inf (switched off, or
// none) does not count.
template <typename F>
__device__ __forceinline__ F group_score(F best, F best2, bool two) {
  return two && best != (F)INFINITY && best2 != -(F)INFINITY ? best + best2 : best;
}

__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// Everything that a token's lanes know about their place.
struct Lanes {
  int g, j, L, each, G;     // group, place in it, lanes and experts a group, groups
  uint64_t group, below;    // lanes of this group, lanes of the groups below
  __device__ __forceinline__ int expert(int i) const { return g * each + j + L * i; }
  __device__ __forceinline__ bool valid(int i) const { return g < G && j + L * i < each; }
};

// The same selection with keys in 64 bits; returns this lane's chosen slots.
// s_key: 64 keys a slot, this wave's own.
__device__ __forceinline__ uint32_t select64(const SelectArgs& a, const float* __restrict__ row,
                                          const float* s_bias, const Lanes& w, int slots,
                                          uint64_t* s_key) {
  const int lane = lane_id();
  double m = -INFINITY, inv = 0.0;
  if (a.score == MOE_SCORE_SOFTMAX) {
    for (int i = 0; i < slots; ++i)
      if (w.valid(i)) m = fmax(m, (double)row[w.expert(i)]);
    for (int o = 32; o > 0; o >>= 1) m = fmax(m, __shfl_xor(m, o, kWave));
    if (m == -INFINITY) m = 0.0;
    double sum = 0.0;
    for (int i = 0; i < slots; ++i)
      if (w.valid(i)) sum += exp((double)row[w.expert(i)] - m);
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
    inv = sum == 0.0 ? 1.0 : sum;
  }
  double b1 = -INFINITY, b2 = -INFINITY;
  for (int i = 0; i < slots; ++i) {
    uint64_t u = 0;
    if (w.valid(i)) {
      const double l = (double)row[w.expert(i)];
      const double p = a.score == MOE_SCORE_SOFTMAX ? exp(l - m) / inv : 1.0 / (1.0 + exp(-l));
      double key = p + (double)s_bias[64 * i + lane];
      if (key != key) key = -INFINITY;
      u = ordered(key);
      b2 = fmax(b2, fmin(b1, key));
      b1 = fmax(b1, key);
    }
    s_key[64 * i + lane] = u;
  }
  if (w.G > 1) {
    for (int o = 1; o < w.L; o <<= 1) {
      const double c1 = __shfl_xor(b1, o, kWave), c2 = __shfl_xor(b2, o, kWave);
      b2 = fmax(fmax(b2, c2), fmin(b1, c1));
      b1 = fmax(b1, c1);
    }
    const double s = group_score(b1, b2, a.group_best == 2);
    int rank = 0;
    for (int g = 0; g < w.G; ++g) {
      const double o = __shfl(s, g * w.L, kWave);
      rank += o > s || (o == s && g < w.g);
    }
    if (rank >= a.top_groups)
      for (int i = 0; i < slots; ++i) s_key[64 * i + lane] = 0;
  }
  uint32_t chosen = 0;
  for (int r = 0; r < a.k; ++r) {
    uint64_t best = 0;
    int id = 0x7fffffff, at = 0;
    for (int i = 0; i < slots; ++i) {
      const uint64_t u = s_key[64 * i + lane];
      if (u > best) {
        best = u;
        id = w.expert(i);
        at = i;
      }
    }
    const int mine = id;
    for (int o = 32; o > 0; o >>= 1) {
      const uint64_t ob = (uint64_t)__shfl_xor((unsigned long long)best, o, kWave);
      const int oi = __shfl_xor(id, o, kWave);
      if (ob > best || (ob == best && oi < id)) {
        best = ob;
        id = oi;
      }
    }
    if (best != 0 && id == mine) {
      chosen |= 1u << at;
      s_key[64 * at + lane] = 0;
    }
  }
  return chosen;
}

// PL: most experts that a lane holds.
template <int PL>
__global__ void __launch_bounds__(256) select_kernel(SelectArgs a) {
  __shared__ float s_bias[64 * PL];
  __shared__ float s_max[4];
  __shared__ uint64_t s_key[4][64 * PL];
  const int lane = lane_id(), wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  Lanes w;
  w.G = a.n_groups;
  w.each = a.E / a.n_groups;
  w.L = 64 >> (32 - __clz(a.n_groups - 1));  // (n_groups 1: 64)
  w.g = lane / w.L;
  w.j = lane & (w.L - 1);
  const uint64_t some = w.L == 64 ? ~0ull : (1ull << w.L) - 1;
  w.group = some << (w.g * w.L);
  w.below = (1ull << (w.g * w.L)) - 1;
  const int slots = (w.each + w.L - 1) / w.L;

  // the bias by slot and lane, and its largest finite magnitude
  float top = 0.f;
  for (int i = wave; i < PL; i += waves) {
    const float b = a.bias != nullptr && w.valid(i) ? a.bias[w.expert(i)] : 0.f;
    s_bias[64 * i + lane] = b;
    if (fabsf(b) < INFINITY) top = fmaxf(top, fabsf(b));
  }
  top = wave_max_f(top);
  if (lane == 0) s_max[wave] = top;
  __syncthreads();
  for (int q = 0; q < waves; ++q) top = fmaxf(top, s_max[q]);
  // Twice the error of an fp32 key, relative to key and bias: sigmoid, some 3
  // steps of p and one of the sum; softmax, exp's argument (l - m, at most 88
  // where p counts, off by 2^-24 of it), the sum's 40 additions and the rest.
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  const float margin = softmax ? 2e-5f : 1.5e-6f;
  const float least = 1e-36f;  // scores below fp32's normal numbers

  for (int t = blockIdx.x * waves + wave; t < a.T; t += gridDim.x * waves) {
    const float* row = a.logits + (size_t)t * a.ld;
    float p[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) p[i] = w.valid(i) ? row[w.expert(i)] : -INFINITY;
    if (softmax) {
      float m = p[0];
#pragma unroll
      for (int i = 1; i < PL; ++i) m = fmaxf(m, p[i]);
      m = wave_max_f(m);
      if (m == -INFINITY) m = 0.f;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        p[i] = exp_fast(p[i] - m);
        sum += p[i];
      }
      sum = wave_sum_f(sum);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int i = 0; i < PL; ++i) p[i] *= inv;
    } else {
#pragma unroll
      for (int i = 0; i < PL; ++i) p[i] = __builtin_amdgcn_rcpf(1.f + exp_fast(-p[i]));
    }
    uint32_t u[PL];
    float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      float key = p[i] + s_bias[64 * i + lane];
      if (!w.valid(i)) key = -INFINITY;
      u[i] = w.valid(i) ? ordered(key) : 0u;
      if (key != key) key = -INFINITY;
      b2 = fmaxf(b2, fminf(b1, key));
      b1 = fmaxf(b1, key);
    }
    bool close = false;
    if (w.G > 1) {
      for (int o = 1; o < w.L; o <<= 1) {
        const float c1 = __shfl_xor(b1, o, kWave), c2 = __shfl_xor(b2, o, kWave);
        b2 = fmaxf(fmaxf(b2, c2), fminf(b1, c1));
        b1 = fmaxf(b1, c1);
      }
      const float s = group_score(b1, b2, a.group_best == 2);
      int rank = 0;
      for (int g = 0; g < w.G; ++g) {
        const float o = __uint_as_float(lane_value(__float_as_uint(s), g * w.L));
        rank += o > s || (o == s && g < w.g);
      }
      const bool kept = w.g < w.G && rank < a.top_groups;
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (!kept) u[i] = 0u;
      // the last group that stays, and others within the margin below it
      const uint64_t last = __ballot(w.g < w.G && rank == a.top_groups - 1);
      const float cut = __uint_as_float(lane_value(__float_as_uint(s), __ffsll((unsigned long long)last) - 1));
      const float low = cut - (2.f * margin * (fabsf(cut) + 2.f * top) + least);
      close = __ballot(w.g < w.G && !kept && s >= low && s > -INFINITY) != 0;
    }
    // the k-th largest lane maximum
    uint32_t best = u[0];
#pragma unroll
    for (int i = 1; i < PL; ++i) best = max(best, u[i]);
    uint32_t thr = 0u;
    for (int b = 31; b >= 0; --b) {
      const uint32_t cand = thr | (1u << b);
      if (__popcll(__ballot(best >= cand)) >= a.k) thr = cand;
    }
    thr = max(thr, 1u);
    int count = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) count += __popcll(__ballot(u[i] >= thr));
    if (count > a.k + 8) {
      // a large surplus: the k-th largest of all keys bit by bit
      thr = 0u;
      for (int b = 31; b >= 0; --b) {
        const uint32_t cand = thr | (1u << b);
        int cnt = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i) cnt += __popcll(__ballot(u[i] >= cand));
        if (cnt >= a.k) {
          thr = cand;
          count = cnt;
        }
      }
    } else {
      // take the smallest value off while enough are left
      while (true) {
        uint32_t low = ~0u;
#pragma unroll
        for (int i = 0; i < PL; ++i) low = min(low, u[i] >= thr ? u[i] : ~0u);
        thr = wave_min_u(low);
        if (count == a.k) break;
        int same = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i) same += __popcll(__ballot(u[i] == thr));
        if (count - same < a.k) break;
        count -= same;
        ++thr;
      }
    }
    // keys within the margin of the threshold that are not above it
    const float cut = unordered(thr);
    const float low = cut - (margin * (fabsf(cut) + top) + least);
    const uint32_t reach = low > -INFINITY ? ordered(low) : thr;
    int near = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) near += __popcll(__ballot(u[i] >= reach));
    close = close || (near > a.k && cut > -INFINITY && cut < INFINITY);

    uint32_t chosen = 0;
    if (close) {
      chosen = select64(a, row, s_bias, w, slots, s_key[wave]);
    } else {
      // every key above the threshold, then those equal to it by ascending id
      int above = 0;
#pragma unroll
      for (int i = 0; i < PL; ++i) above += __popcll(__ballot(u[i] > thr));
      const int need = a.k - above;
      if (count == a.k) {
#pragma unroll
        for (int i = 0; i < PL; ++i) chosen |= u[i] >= thr ? 1u << i : 0u;
      } else {
        int before = 0;  // equal keys with a lower id: lower groups, then slots
#pragma unroll
        for (int i = 0; i < PL; ++i) before += __popcll(__ballot(u[i] == thr) & w.below);
#pragma unroll
        for (int i = 0; i < PL; ++i) {
          const uint64_t same = __ballot(u[i] == thr) & w.group;
          const int at = before + __popcll(same & lanemask_lt());
          chosen |= u[i] > thr || (u[i] == thr && at < need) ? 1u << i : 0u;
          before += __popcll(same);
        }
      }
    }

    float scale = a.scaling;
    float whole = 1.f;
    if (a.renorm) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < PL; ++i) s += chosen >> i & 1 ? p[i] : 0.f;
      whole = wave_sum_f(s) + a.eps;
    }
    int pos = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) pos += __popcll(__ballot(chosen >> i & 1) & w.below);
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const uint64_t sel = __ballot(chosen >> i & 1) & w.group;
      if (chosen >> i & 1) {
        const int o = pos + __popcll(sel & lanemask_lt());
        MOE_CHECK(w.valid(i), MOE_CHECK_ROUTE_ID);
        if (MOE_GUARD(o < a.k, MOE_CHECK_ROUTE_ID)) {
          a.idx[(size_t)t * a.k + o] = w.expert(i);
          const float f = a.renorm ? (whole == 0.f ? 0.f : p[i] / whole) : p[i];
          a.gate[(size_t)t * a.k + o] = scale * f;
        }
      }
      pos += __popcll(sel);
    }
  }
}

int launch_select(const SelectArgs& a, hipStream_t st) {
  const int cus = stream_cu_count(st);
  if (cus <= 0) return MOE_EHIP;
  int groups = 1;
  while (groups < a.n_groups) groups *= 2;
  const int lanes = 64 / groups, slots = (a.E / a.n_groups + lanes - 1) / lanes;
  // few tokens: a wave per workgroup, over more CUs
  const int waves = a.T < 4 * cus ? 1 : 4;
  const dim3 block(64 * waves);
  const dim3 grid((unsigned)std::min<long>(((long)a.T + waves - 1) / waves, (long)cus * 16));
#define MOE_SELECT(PL) hipLaunchKernelGGL(select_kernel<PL>, grid, block, 0, st, a)
  if (slots <= 1) MOE_SELECT(1);
  else if (slots <= 2) MOE_SELECT(2);
  else if (slots <= 4) MOE_SELECT(4);
  else if (slots <= 6) MOE_SELECT(6);
  else if (slots <= 8) MOE_SELECT(8);
  else if (slots <= 12) MOE_SELECT(12);
  else if (slots <= 16) MOE_SELECT(16);
  else MOE_SELECT(32);
#undef MOE_SELECT
  return check_launch();
}

// The gradient.  Every expert of the row gets -p c (softmax; c the selected
// experts' sum of p dp) or 0, the selected ones p dp more: few of the row's
// values need dp, which lies in LDS by expert, cleared again behind each token.
template <typename T, int PL>
__global__ void __launch_bounds__(256) select_bwd_kernel(SelectBwdArgs a) {
  __shared__ float s_dp[4][64 * PL];
  const int lane = lane_id(), wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  float* dp = s_dp[wave];
#pragma unroll
  for (int i = 0; i < PL; ++i) dp[lane + 64 * i] = 0.f;
  if (blockIdx.x == 0 && a.dl != nullptr) {
    if (threadIdx.x < 2) a.route_offs[threadIdx.x] = threadIdx.x ? a.T : 0;
    if ((int)threadIdx.x <= a.nsplit)
      a.split_offs[threadIdx.x] = (int)((long)threadIdx.x * a.T / a.nsplit);
  }
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  for (int t = blockIdx.x * waves + wave; t < a.T; t += gridDim.x * waves) {
    const float* row = a.logits + (size_t)t * a.ld;
    int e = -1;
    float dg = 0.f, l = -INFINITY;
    if (lane < a.k) {
      e = a.idx[(size_t)t * a.k + lane];
      dg = a.dgate[(size_t)t * a.k + lane];
      const bool inside = (unsigned)e < (unsigned)a.E;
      MOE_CHECK(inside, MOE_CHECK_DISPATCH_ID);
      if (inside) l = row[e];
      else e = -1;
    }
    float p[PL];
    float sel;  // the slots' scores
    if (softmax) {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        p[i] = lane + 64 * i < a.E ? row[lane + 64 * i] : -INFINITY;
        m = fmaxf(m, p[i]);
      }
      m = wave_max_f(m);
      if (m == -INFINITY) m = 0.f;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        p[i] = exp_fast(p[i] - m);
        sum += p[i];
      }
      sum = wave_sum_f(sum);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int i = 0; i < PL; ++i) p[i] *= inv;
      sel = e >= 0 ? exp_fast(l - m) * inv : 0.f;
    } else {
      sel = e >= 0 ? 1.f / (1.f + exp_fast(-l)) : 0.f;
    }
    float d = a.scaling * dg, c;
    if (a.renorm) {
      const float whole = wave_sum_f(sel) + a.eps;
      const float r = whole == 0.f ? 0.f : 1.f / whole;
      const float f = wave_sum_f(dg * sel) * r;
      d = lane < a.k ? a.scaling * (dg - f) * r : 0.f;
      // sum_j p_j dp_j without its cancellation: sum p (dg - f) = f (D - sum p)
      c = a.scaling * f * (a.eps * r);
    } else {
      c = wave_sum_f(sel * d);
    }
    // an expert that several slots name: the sum over them, in each
    float both = 0.f;
    for (int q = 0; q < a.k; ++q) {
      const float o = __uint_as_float(lane_value(__float_as_uint(d), q));
      both += (int)lane_value((uint32_t)e, q) == e ? o : 0.f;
    }
    if (e >= 0) dp[e] = softmax ? both : both * sel * (1.f - sel);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int x = lane + 64 * i;
      const float v = softmax ? p[i] * (dp[x] - c) : dp[x];
      if (x < a.E && a.dlogits != nullptr) a.dlogits[(size_t)t * a.E + x] = v;
      if (a.dl != nullptr && x < a.ep) {
        const float w = x < a.E ? v : 0.f;
        if constexpr (sizeof(T) == 4) {
          ((float*)a.dl)[(size_t)t * a.ep + x] = w;
        } else {
          __bf16* to = (__bf16*)a.dl + (size_t)t * 2 * a.ep;
          const __bf16 hi = (__bf16)w;
          to[x] = hi;
          to[a.ep + x] = (__bf16)(w - (float)hi);
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
    if (e >= 0) dp[e] = 0.f;
    __builtin_amdgcn_wave_barrier();
  }
}

template <typename T>
static int launch_select_bwd_t(const SelectBwdArgs& a, hipStream_t st) {
  const int cus = stream_cu_count(st);
  if (cus <= 0) return MOE_EHIP;
  const int waves = a.T < 4 * cus ? 1 : 4;
  const dim3 block(64 * waves);
  const dim3 grid((unsigned)std::min<long>(((long)a.T + waves - 1) / waves, (long)cus * 16));
  const int slots = (std::max(a.E, a.dl ? a.ep : 0) + 63) / 64;
#define MOE_SELECT_BWD(PL) hipLaunchKernelGGL((select_bwd_kernel<T, PL>), grid, block, 0, st, a)
  if (slots <= 1) MOE_SELECT_BWD(1);
  else if (slots <= 2) MOE_SELECT_BWD(2);
  else if (slots <= 4) MOE_SELECT_BWD(4);
  else if (slots <= 6) MOE_SELECT_BWD(6);
  else if (slots <= 8) MOE_SELECT_BWD(8);
  else if (slots <= 12) MOE_SELECT_BWD(12);
  else MOE_SELECT_BWD(16);
#undef MOE_SELECT_BWD
  return check_launch();
}

int launch_select_bwd(const SelectBwdArgs& a, hipStream_t st) {
  return a.halves == 2 ? launch_select_bwd_t<__bf16>(a, st) : launch_select_bwd_t<float>(a, st);
}

__global__ void __launch_bounds__(256)
logits_kernel(const float* __restrict__ partials, int nsplit, const float* __restrict__ col_bias,
              size_t n, int E, float* __restrict__ logits) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) {
    float v = partials[i];
#pragma unroll 4
    for (int q = 1; q < nsplit; ++q) v += partials[q * n + i];
    logits[i] = col_bias != nullptr ? v + col_bias[i % (unsigned)E] : v;
  }
}

int launch_logits(const float* partials, int nsplit, const float* col_bias, int T, int E,
                  float* logits, hipStream_t st) {
  const size_t n = (size_t)T * E;
  const unsigned grid = (unsigned)std::min<size_t>((n + 255) / 256, 1 << 16);
  hipLaunchKernelGGL(logits_kernel, dim3(grid), dim3(256), 0, st, partials, nsplit, col_bias, n, E,
                     logits);
  return check_launch();
}

MOE_CHECK_ACCESSOR(check_word_select)

}  // namespace moe

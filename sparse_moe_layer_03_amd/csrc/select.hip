// Selection of experts from the router's logits: softmax or sigmoid scores, a
// bias on the keys, groups of experts, top-k, renormalised gates; and the
// gradient at the logits.
//
// One wave per token, tokens in grid strides.  Lanes are dealt out to the
// groups: with G groups (rounded up to a power of two) lane l serves group
// l / L, L = 64 / G, and holds its experts l % L, l % L + L, ... in registers.
//
// The top k.  Keys are mapped to integers of the same order, and a threshold is
// built bit by bit until it parts k of them from the rest; of a lane's keys only
// the best two take part, which is nearly always enough (one pass over all
// keys shows it) and takes 2 ballots a bit instead of one for every slot.
//
// Keys that fp32 cannot tell apart.  Keys that lie closer to the last one chosen
// than fp32's error of both are computed in 64 bits and chosen from by those, and
// so are group scores.  With random logits over 768 experts that happens to about
// 1 token in some thousand; with a finite bias far beyond the scores, which the
// bound takes for any expert's, to all of them (one bias of fp32's lowest value:
// 16384 tokens 439 us instead of 38, with -inf 38).
//
// The kernel reads 4 bytes an expert.  16384 tokens over 768 experts in 8 groups:
// 38 us (50 MB), by counters 834 vector and 507 scalar instructions and 91
// branches a token; the vector ones issue for 22 of the 38 us.  Part of it is
// the loads: their descriptor goes by the wave's number, which the compiler does not
// know to be the same in all lanes, so each of the 12 loads is a loop over the
// lanes' descriptors; the rest is waiting.  128 tokens 8.6 us, of which an empty kernel takes
// 2.5, the other 6 one token's chain of dependent steps.  The gradient reads and
// writes 4 bytes an expert: 8192 tokens over 384 experts 8.7 us (25 MB), each wave
// one token whose ids, slots' logits and row are three reads one after another.

#include <math.h>

#include <algorithm>

#include "block.h"
#include "common.h"
#include "wave.h"

namespace moe {

// exp(x): 2^(x log2 e) with the product's rounding error put back, off by
// about 2 steps.
__device__ __forceinline__ float exp_fast(float x) {
  constexpr float kL = 1.44269502162933349609f, kLo = 1.92596299e-8f;  // log2 e in two parts
  const float t = x * kL;
  // (at most 2^-17 where 2^t is finite; NaN for an infinite t, which the median
  // makes finite: infinities, 0 and NaN of 2^t stay what they are)
  const float rest = fmaf(x, kLo, fmaf(x, kL, -t));
  const float some = __builtin_amdgcn_fmed3f(rest, -0x1p-16f, 0x1p-16f);
  return __builtin_amdgcn_exp2f(t) * fmaf(some, 0.693147182464599609375f, 1.f);
}

// A key mapped to an integer of the same order, above 0, which stands for "no
// key".  (A key is a score of 0 or more plus a bias: never -0.)
__device__ __forceinline__ uint32_t ordered(float key) {
  const uint32_t b = __float_as_uint(key);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
__device__ __forceinline__ uint64_t ordered(double key) {
  const uint64_t b = __double_as_longlong(key);
  return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}

// Half of a group's score from its two best keys (the sum of two finite ones may
// pass fp32's range): a second one of -inf (switched off, or none) does not count.
template <typename F>
__device__ __forceinline__ F group_score(F best, F best2, bool two) {
  const F h = (F)0.5 * best;
  return two && best != (F)INFINITY && best2 != -(F)INFINITY ? fma((F)0.5, best2, h) : h;
}

// The slots' scores (in lanes, of the logits l; none where `slot` is not set)
// divided by their sum + eps, and eps by it, for a sum so small that scores below
// fp32's normal numbers, which the kernels flush, weigh in it: with a power of 2
// of their own, down to where 64 bits hold 0.  (inv: 1 / softmax's sum; sigmoid:
// its denominator is 1 here.)
constexpr float kSmallSum = 0x1p-64f;
struct Shares {
  float f, eps;
};
__device__ __forceinline__ Shares small_shares(bool slot, float l, float m, float inv, float eps) {
  constexpr double kLog2e = 1.4426950408889634;
  const double t = fmax(((double)l - (double)m) * kLog2e, -1100.0), n = rint(t);
  const float e = __builtin_amdgcn_exp2f((float)(t - n)) * inv;
  const int k = (int)n;
  slot = slot && k >= -1074;
  const int top = (int)wave_max_u(slot ? (uint32_t)(k + 1100) : 0u) - 1100;
  const float f = slot ? ldexpf(e, k - top) : 0.f;
  const float sum = wave_sum_f(f), rest = (float)ldexp((double)eps, -top), whole = sum + rest;
  if (whole == 0.f) return Shares{0.f, 0.f};
  return Shares{f / whole, rest == 0.f ? 0.f : 1.f / (1.f + sum / rest)};  // (rest may be infinite)
}

// What a lane knows about its place.
struct Lanes {
  int g, j, L, each, G;   // group, place in it, lanes and experts a group, groups
  int slots;              // experts that it holds
  __device__ __forceinline__ int expert(int i) const { return g * each + j + L * i; }
};

// The best two keys of a group, in each of its lanes, from each lane's own.
template <int O>
__device__ __forceinline__ void group_best(float& b1, float& b2, int L) {
  if (O < L) {
    const float c1 = partner<O>(b1), c2 = partner<O>(b2);
    b2 = fmaxf(fmaxf(b2, c2), fminf(b1, c1));
    b1 = fmaxf(b1, c1);
  }
  if constexpr (O < 32) group_best<2 * O>(b1, b2, L);
}

// Scores in 64 bits.
struct Exact {
  const float* row;
  double m, sum;
  bool softmax;
  __device__ __forceinline__ double score(int e) const {
    const double l = (double)row[e];
    return softmax ? exp(l - m) / sum : 1.0 / (1.0 + exp(-l));
  }
  __device__ __forceinline__ double key(int e, float bias) const {
    const double k = score(e) + (double)bias;
    return k != k ? -INFINITY : k;
  }
};
__device__ __forceinline__ Exact exact_scores(const float* row, float m, bool softmax, const Lanes& w) {
  Exact x{row, (double)m, 1.0, softmax};
  if (softmax) {
    double sum = 0.0;
    for (int i = 0; i < w.slots; ++i) sum += exp((double)row[w.expert(i)] - x.m);
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
    x.sum = sum == 0.0 ? 1.0 : sum;
  }
  return x;
}

// Whether the lane's group stays, by scores in 64 bits.
__device__ __forceinline__ bool kept64(const SelectArgs& a, const Exact& x, const float* s_bias,
                                       const Lanes& w) {
  double b1 = -INFINITY, b2 = -INFINITY;
  for (int i = 0; i < w.slots; ++i) {
    const double k = x.key(w.expert(i), s_bias[64 * i + lane_id()]);
    b2 = fmax(b2, fmin(b1, k));
    b1 = fmax(b1, k);
  }
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
  return w.g < w.G && rank < a.top_groups;
}

// The `need` best, by keys in 64 bits, of the slots in the lanes' masks; returns
// the lane's.  key, ids: 64 each, this wave's own.
__device__ __forceinline__ uint32_t best64(uint32_t mask, int need, const float* row, float m,
                                           bool softmax, const float* s_bias, const Lanes& w,
                                           uint64_t* key, int* ids) {
  const int lane = lane_id();
  int before = 0, all = 0;  // of lower lanes, of the wave
#pragma unroll
  for (int b = 0; b < 6; ++b) {
    const uint64_t with = __ballot(__popc(mask) >> b & 1);
    before += __popcll(with & lanemask_lt()) << b;
    all += __popcll(with) << b;
  }
  // The same logit and bias in all of them: equal keys, and ids decide.
  uint32_t lo = ~0u, hi = 0u, blo = ~0u, bhi = 0u;
  for (uint32_t v = mask; v != 0; v &= v - 1) {
    const int i = __ffs(v) - 1;
    const uint32_t l = __float_as_uint(row[w.expert(i)]), b = __float_as_uint(s_bias[64 * i + lane]);
    lo = min(lo, l), hi = max(hi, l);
    blo = min(blo, b), bhi = max(bhi, b);
  }
  const bool equal = wave_min_u(lo) == wave_max_u(hi) && wave_min_u(blo) == wave_max_u(bhi);
  uint32_t chosen = 0;
  if (!equal && all <= 64) {
    // a lane for each: it counts those before it
    const Exact x = exact_scores(row, m, softmax, w);
    int pos = before;
    for (uint32_t v = mask; v != 0; v &= v - 1) {
      const int i = __ffs(v) - 1;
      key[pos] = ordered(x.key(w.expert(i), s_bias[64 * i + lane]));
      ids[pos++] = w.expert(i);
    }
    __builtin_amdgcn_wave_barrier();
    const uint64_t u = lane < all ? key[lane] : 0;
    const int id = lane < all ? ids[lane] : 0x7fffffff;
    int rank = 0;
    for (int q = 0; q < all; ++q) {
      const uint64_t o = (uint64_t)lane_value((uint32_t)(u >> 32), q) << 32 | lane_value((uint32_t)u, q);
      rank += o > u || (o == u && (int)lane_value((uint32_t)id, q) < id);
    }
    const uint64_t taken = __ballot(lane < all && rank < need);
    pos = before;
    for (uint32_t v = mask; v != 0; v &= v - 1)
      chosen |= taken >> pos++ & 1 ? v & -v : 0u;
    __builtin_amdgcn_wave_barrier();
    return chosen;
  }
  // one after another
  const Exact x = equal ? Exact{row, 0.0, 1.0, false} : exact_scores(row, m, softmax, w);
  for (int r = 0; r < need; ++r) {
    uint64_t best = 0;
    int id = 0x7fffffff;
    uint32_t bit = 0;
    for (uint32_t v = mask & ~chosen; v != 0; v &= v - 1) {
      const int i = __ffs(v) - 1;
      const uint64_t u = equal ? 1 : ordered(x.key(w.expert(i), s_bias[64 * i + lane]));
      if (u > best) {
        best = u;
        id = w.expert(i);
        bit = v & -v;
      }
      if (equal) break;  // (a lane's ids ascend)
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
    if (best != 0 && id == mine) chosen |= bit;
  }
  return chosen;
}

// PL: most experts that a lane holds.
template <int PL>
__global__ void __launch_bounds__(256, PL <= 12 ? 5 : 2) select_kernel(SelectArgs a) {
  __shared__ float s_bias[64 * PL];
  __shared__ float s_max[4];
  __shared__ uint64_t s_key[4][64];
  __shared__ int s_id[4][64];
  const int lane = lane_id(), wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  Lanes w;
  w.G = a.n_groups;
  w.each = a.E / a.n_groups;
  w.L = 64 >> (32 - __clz(a.n_groups - 1));  // (n_groups 1: 64)
  w.g = lane / w.L;
  w.j = lane & (w.L - 1);
  w.slots = w.g < w.G && w.j < w.each ? (w.each - w.j + w.L - 1) / w.L : 0;

  // A token's logits, asked for while the one before is worked on.  Slots without
  // an expert read another's, or 0 behind the row's end.
  int t = blockIdx.x * waves + wave;
  const int step = gridDim.x * waves;
  float next[PL];
  auto load = [&](int t) {
    const auto rs = __builtin_amdgcn_make_buffer_rsrc((void*)(a.logits + (size_t)t * a.ld), 0, a.E * 4,
                                                      0x00020000);
#pragma unroll
    for (int i = 0; i < PL; ++i)
      next[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, w.expert(0) * 4, i * w.L * 4, 0));
  };
  if (t < a.T) load(t);

  // the bias by slot and lane, and its largest finite magnitude
  float top = 0.f;
  for (int i = wave; i < PL; i += waves) {
    const float b = a.bias != nullptr && i < w.slots ? a.bias[w.expert(i)] : 0.f;
    s_bias[64 * i + lane] = b;
    if (fabsf(b) < INFINITY) top = fmaxf(top, fabsf(b));
  }
  top = wave_max_f(top);
  if (lane == 0) s_max[wave] = top;
  __syncthreads();
  for (int q = 0; q < waves; ++q) top = fmaxf(top, s_max[q]);
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  // Twice the error of the fp32 score next to the key `cut` (whose scores are
  // at most P = |cut| + top), and of the key's sum.  Sigmoid: some 6 steps of p.
  // Softmax: exp's argument l - m is off by 2^-24 of it, so p by p |l - m| 2^-24,
  // which grows with p up to p = P, where |l - m| <= -log P (or 1); the sum's
  // PL + 6 additions and a few steps more.
  auto margin = [&](float cut) {
    const float P = fmaxf(fabsf(cut) + top, 1e-30f);  // (its logarithm is finite)
    const float steps = softmax ? fmaxf(1.f, -0.6931472f * __builtin_amdgcn_logf(P)) + (PL + 14) : 8.f;
    return steps * 0x1p-23f * P + 1e-36f;  // (scores below fp32's normal numbers)
  };

  for (; t < a.T; t += step) {
    const float* row = a.logits + (size_t)t * a.ld;
    float p[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) p[i] = next[i];
    if (t + step < a.T) load(t + step);
    float m = 0.f, inv = 1.f;
    if (softmax) {
      m = -INFINITY;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        p[i] = i < w.slots ? p[i] : -INFINITY;
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
      inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int i = 0; i < PL; ++i) p[i] *= inv;
    } else {
#pragma unroll
      for (int i = 0; i < PL; ++i)  // (a reciprocal off by a step, which the margin counts)
        p[i] = __builtin_amdgcn_rcpf(1.f + exp_fast(-p[i]));
    }
    // keys, and the lane's best two
    uint32_t u[PL], u1 = 0u, u2 = 0u;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const float key = fmaxf(p[i] + s_bias[64 * i + lane], -INFINITY);  // (NaN: -inf)
      u[i] = i < w.slots ? ordered(key) : 0u;
      u2 = max(u2, min(u1, u[i]));
      u1 = max(u1, u[i]);
    }
    if (w.G > 1) {
      float b1 = u1 ? unordered(u1) : -INFINITY, b2 = u2 ? unordered(u2) : -INFINITY;
      group_best<1>(b1, b2, w.L);
      const float s = group_score(b1, b2, a.group_best == 2);
      int rank = 0;
      for (int g = 0; g < w.G; ++g) {
        const float o = lane_value(s, g * w.L);
        rank += o > s || (o == s && g < w.g);
      }
      bool kept = w.g < w.G && rank < a.top_groups;
      // Another group within the margin below the last one that stays: again in
      // 64 bits.  (Each of the sum's two keys has a score of at most P, and the
      // half of both margins is one.)
      const uint64_t last = __ballot(w.g < w.G && rank == a.top_groups - 1);
      const float cut = lane_value(s, __ffsll((unsigned long long)last) - 1);
      const float low = cut - margin(2.f * fabsf(cut) + top);
      if (__ballot(w.g < w.G && !kept && s >= low && s > -INFINITY) != 0)
        kept = kept64(a, exact_scores(row, m, softmax, w), s_bias, w);
#pragma unroll
      for (int i = 0; i < PL; ++i) u[i] = kept ? u[i] : 0u;
      u1 = kept ? u1 : 0u;
      u2 = kept ? u2 : 0u;
    }
    // A threshold that the lanes' best two keys reach k times: bit by bit, up to
    // the first that parts k of them from the others.  It serves all keys unless
    // a lane's third reaches it too.
    uint32_t thr = 0u;
    for (int b = 31; b >= 0; --b) {
      const uint32_t cand = thr | (1u << b);
      const int n = __popcll(__ballot(u1 >= cand)) + __popcll(__ballot(u2 >= cand));
      if (n >= a.k) thr = cand;
      if (n == a.k) break;
    }
    thr = max(thr, 1u);
    int count = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) count += __popcll(__ballot(u[i] >= thr));
    if (count != a.k) {
      // from all keys
      thr = 0u;
      for (int b = 31; b >= 0; --b) {
        const uint32_t cand = thr | (1u << b);
        int n = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i) n += __popcll(__ballot(u[i] >= cand));
        if (n >= a.k) {
          thr = cand;
          count = n;
        }
        if (n == a.k) break;
      }
    }
    // the smallest key of those, the k-th largest
    uint32_t least = ~0u;
#pragma unroll
    for (int i = 0; i < PL; ++i) least = min(least, u[i] >= thr ? u[i] : ~0u);
    least = wave_min_u(least);
    // Keys so close to it that fp32 may have them on the wrong side.  (An infinite
    // one has only equals, which go by their ids.)
    const float cut = unordered(least);
    uint32_t from = least, to = least;
    if (cut > -INFINITY && cut < INFINITY) {
      const float width = margin(cut);
      from = ordered(cut - width);
      to = ordered(cut + width);
    }
    uint32_t chosen = 0, open = 0;
    int near = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const bool at = u[i] >= from;
      near += __popcll(__ballot(at));
      chosen |= at ? 1u << i : 0u;
      open |= at && u[i] <= to ? 1u << i : 0u;
    }
    if (near > a.k) {
      int sure = 0;
      chosen &= ~open;
#pragma unroll
      for (int b = 0; b < 6; ++b) sure += __popcll(__ballot(__popc(chosen) >> b & 1)) << b;
      // (infinite keys: any finite score leaves them equal)
      chosen |= best64(open, a.k - sure, row, m, softmax, s_bias, w, s_key[wave], s_id[wave]);
    }
    // The ids into LDS, lane by lane; then a lane for each, which counts the
    // lower ones to find its place.
    int pos = 0;
#pragma unroll
    for (int b = 0; b < 5; ++b)  // (at most 16)
      pos += __popcll(__ballot(__popc(chosen) >> b & 1) & lanemask_lt()) << b;
    while (chosen != 0) {
      MOE_CHECK(pos < a.k, MOE_CHECK_ROUTE_ID);
      if (pos < a.k) s_id[wave][pos] = w.expert(__ffs(chosen) - 1);
      ++pos;
      chosen &= chosen - 1;
    }
    __builtin_amdgcn_wave_barrier();
    int id = lane < a.k ? s_id[wave][lane] : 0;
    __builtin_amdgcn_wave_barrier();
    int at = 0;
    for (int q = 0; q < a.k; ++q) at += (int)lane_value((uint32_t)id, q) < id;
    MOE_CHECK((unsigned)id < (unsigned)a.E, MOE_CHECK_ROUTE_ID);
    id = min(max(id, 0), a.E - 1);
    const float l = row[id];
    float f = softmax ? exp_fast(l - m) * inv : __builtin_amdgcn_rcpf(1.f + exp_fast(-l));
    if (a.renorm) {
      const float whole = wave_sum_f(lane < a.k ? f : 0.f) + a.eps;
      if (whole < kSmallSum) f = small_shares(lane < a.k, l, m, inv, a.eps).f;
      else f /= whole;
    }
    if (lane < a.k) {
      a.idx[(size_t)t * a.k + at] = id;
      a.gate[(size_t)t * a.k + at] = a.scaling * f;
    }
  }
}

int launch_select(const SelectArgs& a, hipStream_t st) {
  const int cus = stream_cu_count(st);
  if (cus <= 0) return MOE_EHIP;
  int groups = 1;
  while (groups < a.n_groups) groups *= 2;
  const int lanes = 64 / groups, slots = (a.E / a.n_groups + lanes - 1) / lanes;
  const int waves = 4;  // (one, over more CUs, is no faster for few tokens: 128 9.6 us, with four 9.3)
  const dim3 block(64 * waves);
  const dim3 grid((unsigned)std::min<long>(((long)a.T + waves - 1) / waves, (long)cus * 5));
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
    float sel, other = 1.f;  // the slots' scores p, and 1 - p of a sigmoid
    float m = 0.f, inv = 1.f;
    if (softmax) {
      m = -INFINITY;
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
      inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int i = 0; i < PL; ++i) p[i] *= inv;
      sel = e >= 0 ? exp_fast(l - m) * inv : 0.f;
    } else {
      const float x = exp_fast(-l);
      sel = e >= 0 ? 1.f / (1.f + x) : 0.f;
      // (not from p: for a logit of 16 it is 2 steps of p, above 17 less than one)
      other = fminf(x, 3.4028234663852886e38f) * sel;
    }
    float d = a.scaling * dg, c;
    bool small = false;  // scores' shares of D in their places, and 1 in D's
    if (a.renorm) {
      float eps = a.eps, r = 1.f;
      const float whole = wave_sum_f(sel) + eps;
      if (whole < kSmallSum) {
        const Shares s = small_shares(e >= 0, l, m, inv, eps);
        small = true;
        sel = s.f, eps = s.eps, other = 1.f;
      } else {
        r = 1.f / whole;
      }
      const float f = wave_sum_f(dg * sel) * r;
      // D (dg_j - f) = sum_i p_i (dg_j - dg_i) + eps dg_j: what dg has in common
      // over the slots falls out of the differences and leaves no rounding
      // behind (one slot and eps 0: the gate is a constant, its gradient 0)
      float apart = eps * dg;
      for (int q = 0; q < a.k; ++q) apart += lane_value(sel, q) * (dg - lane_value(dg, q));
      d = lane < a.k ? a.scaling * (apart * r) * r : 0.f;
      // sum_j p_j dp_j without its cancellation: sum p (dg - f) = f (D - sum p)
      c = a.scaling * f * (eps * r);
    } else {
      c = wave_sum_f(sel * d);
    }
    // an expert that several slots name: the sum over them, in each
    float both = 0.f;
    for (int q = 0; q < a.k; ++q) {
      const float o = lane_value(d, q);
      both += (int)lane_value((uint32_t)e, q) == e ? o : 0.f;
    }
    if (e >= 0) dp[e] = !softmax ? both * sel * other : small ? both * sel : both;
    __builtin_amdgcn_wave_barrier();
    auto put = [&](int x, float v) {
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
    };
    if (!softmax) {
#pragma unroll
      for (int i = 0; i < PL; ++i) put(lane + 64 * i, dp[lane + 64 * i]);
    } else if (!small) {
#pragma unroll
      for (int i = 0; i < PL; ++i) put(lane + 64 * i, p[i] * (dp[lane + 64 * i] - c));
    } else {
#pragma unroll
      for (int i = 0; i < PL; ++i) put(lane + 64 * i, dp[lane + 64 * i] - p[i] * c);
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
  const int waves = 4;  // (one is no faster for few tokens: 128 5.7 us, with four 5.8; 1 8.6 and 5.5)
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

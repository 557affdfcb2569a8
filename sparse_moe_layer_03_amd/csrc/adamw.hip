// AdamW over many tensors in one launch, with moments in fp32 or in 8 bits.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// Every element is read and written once: the step is bound by HBM (28 bytes
// an element for bf16 weights with a 32-bit copy, 16 with 8-bit moments).
// The list of up to 48 tensors travels in the kernel arguments, so a step
// needs no table in device memory and can be captured as it stands.  Chunks
// of 2048 elements over all tensors are dealt to the workgroups in turn; a
// thread handles 8 neighbouring elements with 16-byte accesses.  Measured over
// 402M parameters: 32-bit moments 2.26 ms, 4.99 TB/s (a plain copy runs at
// 4.9), 8-bit ones 1.36 ms, 4.75 TB/s; non-temporal accesses up to 10% slower.
//
// 8-bit moments: 256 elements (32 lanes) share a scale, their largest
// magnitude / 448, found by a butterfly over half a wave.  Codes are e4m3
// values, rounded at random between the two neighbours with the probability
// that keeps the mean: an average that moves by (1 - b2) of its distance
// each step would never leave its code under rounding to nearest.  The
// second moment is held as its root, which halves the exponents' range; the
// mean of the square is kept, for a rounding that kept the root's mean would
// raise v by the rounding's variance at every step.  Random bits: two rounds
// of xor-shift and multiply of the element's place, with constants that
// C. Wellons published for such a mixing of 32 bits.
// What a code follows from (the moments, their largest, the comparison) is
// computed operation by operation, each rounded by itself: contracted sums
// would move one code in a million, and a code is an eighth of its value.

#include <math.h>

#include "common.h"
#include "train.h"

#pragma clang fp contract(off)

namespace moe {

constexpr int kAdamTensors = 48;   // per launch: 48 * 80 bytes of kernel arguments
constexpr int kAdamThreads = 256, kAdamPer = 8, kAdamChunk = kAdamThreads * kAdamPer;
constexpr float kQMax = 448.f;     // largest e4m3 value

struct AdamTensor {
  void* param;
  const void* grad;
  float* master;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  float decay;          // weight decay
  uint32_t dtypes;      // bit 0: param is bf16, bit 1: grad is bf16
  uint32_t chunk_end;   // chunks of the tensors up to and with this one
  uint32_t pad;
};

struct AdamArgs {
  double beta1, beta2;
  float lr, eps, b1, b2, nb1, nb2;  // nb: 1 - b, rounded from the double
  uint32_t seed;
  int32_t first;                    // place in the list of tensor 0
  int32_t n_tensors;
  int32_t last;                     // this launch ends the step
  moe_adamw_state* state;
  const float* grad_scale;
  const float* lr_scale;
  AdamTensor t[kAdamTensors];
};
static_assert(sizeof(AdamArgs) <= 4096, "kernel arguments");

__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}

// b^t by repeated squaring.
__device__ double power(double b, int t) {
  double r = 1.0;
  for (; t > 0; t >>= 1, b *= b)
    if (t & 1) r *= b;
  return r;
}

// 8 elements at p + i of which `left` exist (all of them: 16-byte accesses).
__device__ __forceinline__ void load8(const float* p, int left, float* f) {
  if (left >= 8) {
    unpack16(ld16(p), f, (float*)nullptr);
    unpack16(ld16(p + 4), f + 4, (float*)nullptr);
  } else {
    for (int k = 0; k < 8; ++k) f[k] = k < left ? p[k] : 0.f;
  }
}
__device__ __forceinline__ void load8(const __bf16* p, int left, float* f) {
  if (left >= 8) {
    unpack16(ld16(p), f, (__bf16*)nullptr);
  } else {
    for (int k = 0; k < 8; ++k) f[k] = k < left ? (float)p[k] : 0.f;
  }
}
__device__ __forceinline__ void store8(float* p, int left, const float* f) {
  if (left >= 8) {
    st16(p, pack16(f, (float*)nullptr));
    st16(p + 4, pack16(f + 4, (float*)nullptr));
  } else {
    for (int k = 0; k < left; ++k) p[k] = f[k];
  }
}
__device__ __forceinline__ void store8(__bf16* p, int left, const float* f) {
  if (left >= 8) {
    st16(p, pack16(f, (__bf16*)nullptr));
  } else {
    for (int k = 0; k < left; ++k) p[k] = (__bf16)f[k];
  }
}

// 8 codes as values (not yet scaled), and back; values are e4m3 numbers, so
// the conversion is exact both ways.
__device__ __forceinline__ void load_codes(const uint8_t* p, int left, float* f) {
  uint32_t w[2] = {0u, 0u};
  if (left >= 8) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x;
    w[1] = x.y;
  } else {
    for (int k = 0; k < left; ++k) w[k >> 2] |= (uint32_t)p[k] << (8 * (k & 3));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
    f[4 * h] = lo[0];
    f[4 * h + 1] = lo[1];
    f[4 * h + 2] = hi[0];
    f[4 * h + 3] = hi[1];
  }
}
__device__ __forceinline__ void store_codes(uint8_t* p, int left, const float* f) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int x = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h], f[4 * h + 1], 0, false);
    w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2], f[4 * h + 3], x, true);
  }
  if (left >= 8) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
    for (int k = 0; k < left; ++k) p[k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
  }
}

// Largest magnitude over the 32 lanes that hold a block.  Magnitudes are
// compared as bit patterns, so a NaN wins over every number.
__device__ __forceinline__ float block_top(const float* x) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, kWave));
  return __uint_as_float(top);
}

// The e4m3 value that stands for x / scale: one of the neighbours of
// y = |x| inv, the upper one when u < (y - low) / (high - low) (SQUARE: of
// their squares).  u in [0, 1).
template <bool SQUARE>
__device__ __forceinline__ float round_code(float x, float inv, float u) {
  float y = fabsf(x) * inv;
  y = y > kQMax ? kQMax : y;  // keeps NaN
  // spacing of e4m3 at y: 2^(e - 3), e >= -6
  const int ex = max((int)(__float_as_uint(y) >> 23), 127 - 6);
  const float ulp = __uint_as_float((uint32_t)(ex - 3) << 23);
  const float rulp = __uint_as_float((uint32_t)(254 - (ex - 3)) << 23);
  const float low = floorf(y * rulp) * ulp;
  const float high = fminf(low + ulp, kQMax);
  const bool up = SQUARE ? u * (high * high - low * low) < y * y - low * low
                         : u * (high - low) < y - low;
  float q = up ? high : low;
  if (SQUARE) q = y > 0.f ? fmaxf(q, 0x1p-9f) : q;
  q = y != y ? y : q;
  return copysignf(q, x);
}

template <bool Q8>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(AdamArgs a) {
  __shared__ float s_c[2];
  __shared__ uint32_t s_base;
  const int tid = threadIdx.x;
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const bool skip = !(fabsf(gs) < INFINITY);
  const int step = a.state->step;
  if (tid == 0) {
    const int t = step + 1;
    s_c[0] = (float)(1.0 / (1.0 - power(a.beta1, t)));
    s_c[1] = (float)(1.0 / (1.0 - power(a.beta2, t)));
    s_base = mix32(a.seed + 0x9E3779B9u * (uint32_t)t);
  }
  __syncthreads();
  const float ic1 = s_c[0], ic2 = s_c[1];
  const uint32_t base = s_base;
  const float lr = a.lr_scale ? a.lr * *a.lr_scale : a.lr;
  const float sic2 = sqrtf(ic2), lrc1 = lr * ic1;
  const uint32_t chunks = skip ? 0u : a.t[a.n_tensors - 1].chunk_end;

  int at = 0;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    while (c >= a.t[at].chunk_end) ++at;
    const AdamTensor& w = a.t[at];
    const uint32_t c0 = at ? a.t[at - 1].chunk_end : 0u;
    const int64_t i = (int64_t)(c - c0) * kAdamChunk + tid * kAdamPer;
    const int left = (int)min((int64_t)8, w.n - i);  // 0 or less: none
    const bool p16 = w.dtypes & 1u, g16 = w.dtypes & 2u;
    const int64_t blk = i >> 8;

    float p[8], g[8], m[8], v[8];
    float ms = 0.f, vs = 0.f;
    if (left > 0) {
      if (w.master) load8(w.master + i, left, p);
      else if (p16) load8((const __bf16*)w.param + i, left, p);
      else load8((const float*)w.param + i, left, p);
      if (g16) load8((const __bf16*)w.grad + i, left, g);
      else load8((const float*)w.grad + i, left, g);
      if (Q8) {
        load_codes((const uint8_t*)w.m + i, left, m);
        load_codes((const uint8_t*)w.v + i, left, v);
        ms = w.m_scale[blk];
        vs = w.v_scale[blk];
      } else {
        load8((const float*)w.m + i, left, m);
        load8((const float*)w.v + i, left, v);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) p[k] = g[k] = m[k] = v[k] = 0.f;
    }
    float r[8];
    const float keep = 1.f - lr * w.decay;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float gk = g[k] * gs;
      float mk = m[k], vk = v[k];
      if (Q8) {
        mk *= ms;
        const float rv = vk * vs;
        vk = rv * rv;
      }
      mk = a.b1 * mk + a.nb1 * gk;
      vk = a.b2 * vk + a.nb2 * gk * gk;
      m[k] = mk;
      v[k] = vk;
      // The root is sqrtf: the hardware's alone takes a v below the normal
      // numbers for 0 and would leave eps in the denominator.  The reciprocal
      // is the hardware's (an ulp): its operand is at least eps >= 1e-30.
      float root;
      if (Q8) {
        r[k] = sqrtf(vk);
        root = r[k] * sic2;
      } else {
        root = sqrtf(vk * ic2);
      }
      p[k] = p[k] * keep - (mk * lrc1) * __builtin_amdgcn_rcpf(root + a.eps);
    }
    if (Q8) {
      // elements behind the tensor's end are zeros here: they leave the top alone
      const float tm = block_top(m), tv = block_top(r);
      const float im = tm > 0x1p-100f ? (1.f / tm) * kQMax : 0.f;
      const float iv = tv > 0x1p-100f ? (1.f / tv) * kQMax : 0.f;
      const uint32_t key = mix32(base + (uint32_t)(a.first + at)) + (uint32_t)i +
                           0x9E3779B9u * (uint32_t)((uint64_t)i >> 32);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t h = mix32(key + k);
        m[k] = round_code<false>(m[k], im, (float)(h & 0xffffu) * 0x1p-16f);
        r[k] = round_code<true>(r[k], iv, (float)(h >> 16) * 0x1p-16f);
      }
      if (left > 0) {
        store_codes((uint8_t*)w.m + i, left, m);
        store_codes((uint8_t*)w.v + i, left, r);
        if ((tid & 31) == 0) {
          w.m_scale[blk] = tm * (1.f / kQMax);
          w.v_scale[blk] = tv * (1.f / kQMax);
        }
      }
    } else if (left > 0) {
      store8((float*)w.m + i, left, m);
      store8((float*)w.v + i, left, v);
    }
    if (left > 0) {
      if (w.master) store8(w.master + i, left, p);
      if (p16) store8((__bf16*)w.param + i, left, p);
      else store8((float*)w.param + i, left, p);
    }
  }

  // The last workgroup of the step's last launch counts the step: every
  // workgroup has read the count before it arrives here.
  if (a.last) {
    __syncthreads();
    if (tid == 0 && atomicAdd(&a.state->arrived, 1u) == gridDim.x - 1) {
      a.state->arrived = 0;
      if (skip) a.state->skipped += 1;
      else a.state->step = step + 1;
    }
  }
}

int launch_adamw(const moe_adamw_params* hp, const moe_adamw_tensor* tensors, int n_tensors,
                 moe_adamw_state* state, const float* grad_scale, const float* lr_scale,
                 hipStream_t st) {
  const int cus = stream_cu_count(st);
  if (cus <= 0) return MOE_EHIP;
  AdamArgs a{};
  a.beta1 = hp->beta1;
  a.beta2 = hp->beta2;
  a.lr = (float)hp->lr;
  a.eps = (float)hp->eps;
  a.b1 = (float)hp->beta1;
  a.b2 = (float)hp->beta2;
  a.nb1 = (float)(1.0 - hp->beta1);
  a.nb2 = (float)(1.0 - hp->beta2);
  a.seed = hp->seed;
  a.state = state;
  a.grad_scale = grad_scale;
  a.lr_scale = lr_scale;
  for (int first = 0; first < n_tensors; first += kAdamTensors) {
    a.first = first;
    a.n_tensors = n_tensors - first < kAdamTensors ? n_tensors - first : kAdamTensors;
    a.last = first + a.n_tensors == n_tensors;
    uint64_t chunks = 0;
    for (int k = 0; k < a.n_tensors; ++k) {
      const moe_adamw_tensor& s = tensors[first + k];
      AdamTensor& d = a.t[k];
      d.param = s.param;
      d.grad = s.grad;
      d.master = s.master;
      d.m = s.m;
      d.v = s.v;
      d.m_scale = s.m_scale;
      d.v_scale = s.v_scale;
      d.n = s.n;
      d.decay = (float)s.weight_decay;
      d.dtypes = (s.param_dtype == MOE_BF16 ? 1u : 0u) | (s.grad_dtype == MOE_BF16 ? 2u : 0u);
      chunks += ((uint64_t)s.n + kAdamChunk - 1) / kAdamChunk;
      d.chunk_end = (uint32_t)chunks;  // the caller keeps the sum below 2^32
    }
    // four rounds of the 7 or 8 workgroups that a CU holds: 402M parameters with
    // 8-bit moments 1361 us (one round of 8: 1468, a workgroup per chunk: 2341),
    // with 32-bit ones 2261 (2271, 2450)
    const uint64_t most = 28ull * cus;
    const uint64_t grid = chunks < 1 ? 1 : chunks < most ? chunks : most;
    if (hp->state_bits == 8)
      hipLaunchKernelGGL(adamw_kernel<true>, dim3((unsigned)grid), dim3(kAdamThreads), 0, st, a);
    else
      hipLaunchKernelGGL(adamw_kernel<false>, dim3((unsigned)grid), dim3(kAdamThreads), 0, st, a);
    const int rc = check_launch();
    if (rc) return rc;
  }
  return MOE_OK;
}

// Elements of one launch's 48 tensors that the chunk counter can hold.
uint64_t adamw_max_elements() { return ((1ull << 32) - 2 - kAdamTensors - (1u << 20)) * kAdamChunk; }

}  // namespace moe

// The layer's backward pass beside its grouped products: SwiGLU's backward
// step, the gradients at the gates and logits, and the sum of the row
// gradients per token.  All of it moves data once and is bound by HBM; sums
// are fp32 in a fixed order, no atomics.

#include "common.h"
#include "train.h"

namespace moe {

// Grid of a kernel that has one row or token per workgroup.  A launch's x holds
// fewer than 2^32 threads (2^24 workgroups of 256), the calls take up to 2^27
// rows: they lie in planes of 2^20, one per y.  (A loop over them in the kernel
// cost token_bwd_kernel a quarter of its time: 20.6 -> 25.4 us at 4096 tokens.)
constexpr int kRowPlane = 20;
static dim3 row_grid(int n) {
  const int plane = 1 << kRowPlane;
  return dim3((unsigned)(n < plane ? n : plane), (unsigned)((n + plane - 1) >> kRowPlane));
}
__device__ __forceinline__ int grid_row() { return (int)(blockIdx.y << kRowPlane | blockIdx.x); }

// Sum over a block of 256 threads, the same in every thread.
__device__ __forceinline__ float block_sum(float v, float* s) {
  v = wave_sum(v);
  __syncthreads();
  if (lane_id() == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  return (s[0] + s[1]) + (s[2] + s[3]);
}
__device__ __forceinline__ float block_max(float v, float* s) {
  v = wave_max(v);
  __syncthreads();
  if (lane_id() == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  return fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
}

// One workgroup per FFN row of the Tk = T * top_k.
__global__ void __launch_bounds__(256)
swiglu_bwd_kernel(const float* __restrict__ zu, const float* __restrict__ dh0,
                  const float* __restrict__ gate_rows, const int32_t* __restrict__ offsets,
                  int n_ffn, int Tk, int f, float* __restrict__ dzu, float* __restrict__ hs,
                  float* __restrict__ part) {
  __shared__ float s[4];
  const int p = grid_row();
  if (p >= min(offsets[n_ffn], Tk)) return;
  const float gt = gate_rows[p];
  const float* zr = zu + (size_t)p * 2 * f;
  const float* dr = dh0 + (size_t)p * f;
  float* o = dzu + (size_t)p * 2 * f;
  float sum = 0.f;
  for (int c = threadIdx.x * 4; c < f; c += 1024) {
    const f32x4_t z = *reinterpret_cast<const f32x4_t*>(zr + c);
    const f32x4_t u = *reinterpret_cast<const f32x4_t*>(zr + f + c);
    const f32x4_t dh = *reinterpret_cast<const f32x4_t*>(dr + c);
    f32x4_t dz, du, h;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float sg = 1.f / (1.f + expf(-z[k]));
      const float si = z[k] * sg, d = gt * dh[k];
      sum += dh[k] * (si * u[k]);
      dz[k] = d * u[k] * (sg * (1.f + z[k] * (1.f - sg)));
      du[k] = d * si;
      h[k] = gt * (si * u[k]);
    }
    *reinterpret_cast<f32x4_t*>(o + c) = dz;
    *reinterpret_cast<f32x4_t*>(o + f + c) = du;
    *reinterpret_cast<f32x4_t*>(hs + (size_t)p * f + c) = h;
  }
  sum = block_sum(sum, s);
  if (threadIdx.x == 0) part[p] = sum;
}

int launch_swiglu_bwd(const float* zu, const float* dh, const float* gate_rows,
                      const int32_t* offsets, int n_ffn, int Tk, int f, float* dzu, float* hs,
                      float* dgate_part, hipStream_t st) {
  hipLaunchKernelGGL(swiglu_bwd_kernel, row_grid(Tk), dim3(256), 0, st, zu, dh, gate_rows, offsets,
                     n_ffn, Tk, f, dzu, hs, dgate_part);
  return check_launch();
}

// One wave per row, both arrays; four 16-byte pieces of each in flight a lane.
template <typename T>
__global__ void __launch_bounds__(256)
gather2_kernel(const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ gate,
               const int32_t* __restrict__ perm, const int32_t* __restrict__ offsets, int n_ffn,
               int Tk, int k, int d, T* __restrict__ xp, T* __restrict__ dyp,
               float* __restrict__ gate_rows) {
  constexpr int CE = 16 / sizeof(T), U = 4;
  const int lane = lane_id();
  const int rows = min(offsets[n_ffn], Tk);
  for (int p = blockIdx.x * 4 + (threadIdx.x >> 6); p < rows; p += gridDim.x * 4) {
    const int at = __builtin_amdgcn_readfirstlane(perm[p]);
    MOE_CHECK((unsigned)at < (unsigned)Tk, MOE_CHECK_GEMM_ROW);
    if ((unsigned)at >= (unsigned)Tk) continue;
    const size_t src = (size_t)(at / k) * d, dst = (size_t)p * d;
    if (lane == 0) gate_rows[p] = gate[at];
    const int chunks = d / CE;
    for (int c0 = lane; c0 < chunks; c0 += 64 * U) {
      u32x4_t vx[U], vy[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 64;
        if (c < chunks) vx[u] = ld16(x + src + c * CE), vy[u] = ld16(dy + src + c * CE);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 64;
        if (c < chunks) st16(xp + dst + c * CE, vx[u]), st16(dyp + dst + c * CE, vy[u]);
      }
    }
  }
}

int launch_gather2(int dtype, const void* x, const void* dy, const float* gate, const int32_t* perm,
                   const int32_t* offsets, int n_ffn, int Tk, int k, int d, void* xp, void* dyp,
                   float* gate_rows, hipStream_t st) {
  const int blocks = (int)(((long)Tk + 3) / 4);
  const dim3 grid(blocks < 8192 ? blocks : 8192);
  if (dtype == MOE_BF16)
    hipLaunchKernelGGL(gather2_kernel<__bf16>, grid, dim3(256), 0, st, (const __bf16*)x,
                       (const __bf16*)dy, gate, perm, offsets, n_ffn, Tk, k, d, (__bf16*)xp,
                       (__bf16*)dyp, gate_rows);
  else
    hipLaunchKernelGGL(gather2_kernel<float>, grid, dim3(256), 0, st, (const float*)x,
                       (const float*)dy, gate, perm, offsets, n_ffn, Tk, k, d, (float*)xp,
                       (float*)dyp, gate_rows);
  return check_launch();
}

// One workgroup per token.
template <typename T>
__global__ void __launch_bounds__(256) token_bwd_kernel(TokenArgs a) {
  constexpr int CE = 16 / sizeof(T);
  constexpr int MAXE = 1024;
  __shared__ float s[4];
  __shared__ float s_dp[MAXE];   // gradient at p, by expert
  constexpr int MAXK = 16;
  __shared__ __attribute__((aligned(16))) float s_dg[MAXK];
  __shared__ __attribute__((aligned(16))) int s_e[MAXK];
  const int t = grid_row(), tid = threadIdx.x;
  if (t >= a.T) return;
  if (t == 0 && a.logits) {
    if (tid < 2) a.route_offs[tid] = tid ? a.T : 0;
    if (tid <= a.nsplit) a.split_offs[tid] = (int)((long)tid * a.T / a.nsplit);
  }
  for (int e = tid; e < a.E; e += 256) s_dp[e] = 0.f;
  bool identity = false;
  if (tid < a.k) {
    const int e = a.idx[t * a.k + tid];
    const int row = a.inv_perm[t * a.k + tid];
    s_e[tid] = e;
    float dg = 0.f;
    const bool inside = (unsigned)row < (unsigned)(a.T * a.k);
    MOE_CHECK((unsigned)e < (unsigned)a.E, MOE_CHECK_DISPATCH_ID);
    MOE_CHECK(e >= a.n_ffn || inside, MOE_CHECK_COMBINE_ROW);
    if (e < a.n_ffn && inside)
      for (int q = 0; q < a.parts; ++q) dg += a.part[(size_t)row * a.parts + q];
    s_dg[tid] = dg;
    identity = e >= a.n_ffn;
  }
  if (__syncthreads_or(identity)) {
    const T* x = (const T*)a.x + (size_t)t * a.d;
    const T* dy = (const T*)a.dy + (size_t)t * a.d;
    float dot = 0.f;
    for (int c = tid * CE; c < a.d; c += 256 * CE) {
      float fx[CE], fd[CE];
      unpack16(ld16(x + c), fx, (T*)nullptr);
      unpack16(ld16(dy + c), fd, (T*)nullptr);
#pragma unroll
      for (int k = 0; k < CE; ++k) dot += fx[k] * fd[k];
    }
    dot = block_sum(dot, s);
    if (identity) s_dg[tid] = dot;
  }
  __syncthreads();
  if (tid < a.k) {
    a.dgate[t * a.k + tid] = s_dg[tid];
    // the sum over the slots of the expert: a caller's own selection may name
    // one twice (each of its slots writes the same sum)
    const int e = s_e[tid];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < MAXK; ++j) sum += j < a.k && s_e[j] == e ? s_dg[j] : 0.f;
    if ((unsigned)e < (unsigned)a.E) s_dp[e] = a.scaling * sum;
  }
  if (!a.logits) return;
  __syncthreads();
  const float* lg = a.logits + (size_t)t * a.E;
  float p[MAXE / 256];
  float top = -INFINITY;
#pragma unroll
  for (int q = 0; q < MAXE / 256; ++q) {
    const int e = tid + q * 256;
    p[q] = e < a.E ? lg[e] : -INFINITY;
    top = fmaxf(top, p[q]);
  }
  top = block_max(top, s);
  float sum = 0.f;
#pragma unroll
  for (int q = 0; q < MAXE / 256; ++q) {
    const int e = tid + q * 256;
    p[q] = e < a.E ? expf(p[q] - top) : 0.f;
    sum += p[q];
  }
  sum = block_sum(sum, s);
  float dot = 0.f;
#pragma unroll
  for (int q = 0; q < MAXE / 256; ++q) {
    const int e = tid + q * 256;
    p[q] /= sum;
    if (e < a.E) dot += p[q] * s_dp[e];
  }
  dot = block_sum(dot, s);
#pragma unroll
  for (int q = 0; q < MAXE / 256; ++q) {
    const int e = tid + q * 256;
    const float v = e < a.E ? p[q] * (s_dp[e] - dot) : 0.f;
    if (e < a.ep) {
      if constexpr (sizeof(T) == 4) {
        ((float*)a.dl)[(size_t)t * a.ep + e] = v;
      } else {
        __bf16* row = (__bf16*)a.dl + (size_t)t * 2 * a.ep;
        const __bf16 hi = (__bf16)v;
        row[e] = hi;
        row[a.ep + e] = (__bf16)(v - (float)hi);
      }
    }
    if (a.dlogits && e < a.E) a.dlogits[(size_t)t * a.E + e] = v;
  }
}

int launch_token_bwd(int dtype, const TokenArgs& a, hipStream_t st) {
  if (dtype == MOE_BF16)
    hipLaunchKernelGGL(token_bwd_kernel<__bf16>, row_grid(a.T), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(token_bwd_kernel<float>, row_grid(a.T), dim3(256), 0, st, a);
  return check_launch();
}

MOE_CHECK_ACCESSOR(check_word_layer_bwd)

// One workgroup per token: its FFN rows, the identity gates' share of dy and
// the router's share, summed in that order.  All of a piece's loads are issued
// before the first is added.
template <typename T, int MAXK>
__global__ void __launch_bounds__(256)
dx_kernel(const float* __restrict__ dx_rows, const T* __restrict__ dy, const float* __restrict__ dxr,
          const int32_t* __restrict__ idx, const float* __restrict__ gate,
          const int32_t* __restrict__ inv_perm, int Tn, int d, int k, int n_ffn,
          T* __restrict__ dx) {
  __shared__ int s_row[MAXK];
  __shared__ float s_gz;
  __shared__ int s_n;
  const int t = grid_row(), tid = threadIdx.x;
  if (t >= Tn) return;
  if (tid < 64) {
    int e = n_ffn, row = 0;
    float g = 0.f;
    if (tid < k) {
      e = idx[t * k + tid];
      g = gate[t * k + tid];
      row = inv_perm[t * k + tid];
      const bool inside = (unsigned)row < (unsigned)(Tn * k);
      MOE_CHECK(e >= n_ffn || inside, MOE_CHECK_COMBINE_ROW);
      if (!inside) row = 0;
    }
    const bool ffn = tid < k && e < n_ffn;
    const uint64_t fb = __ballot(ffn);
    if (ffn) s_row[__popcll(fb & lanemask_lt())] = row;
    const float gid = (tid < k && !ffn) ? g : 0.f;
    float gz = 0.f;
    for (int j = 0; j < k; ++j) gz += __shfl(gid, j, kWave);
    if (tid == 0) {
      s_n = __popcll(fb);
      s_gz = gz;
    }
  }
  __syncthreads();
  const int n = s_n;
  const float gz = s_gz;
  const bool ident = n < k;
  const size_t at = (size_t)t * d;
  for (int c = tid * 4; c < d; c += 1024) {
    f32x4_t rows[MAXK], r = {0.f, 0.f, 0.f, 0.f}, y = r;
#pragma unroll
    for (int q = 0; q < MAXK; ++q)
      if (q < n) rows[q] = *reinterpret_cast<const f32x4_t*>(dx_rows + (size_t)s_row[q] * d + c);
    if (dxr) r = *reinterpret_cast<const f32x4_t*>(dxr + at + c);
    if (ident) {
      if constexpr (sizeof(T) == 4) {
        y = *reinterpret_cast<const f32x4_t*>(dy + at + c);
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(dy + at + c);
        y = f32x4_t{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                    __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u)};
      }
    }
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < MAXK; ++q)
      if (q < n) acc += rows[q];
    if (ident) acc += gz * y;
    acc += r;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<f32x4_t*>(dx + at + c) = acc;
    } else {
      __bf16 o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = (__bf16)acc[i];
      *reinterpret_cast<uint2*>(dx + at + c) = __builtin_bit_cast(uint2, o);
    }
  }
}

int launch_dx(int dtype, const float* dx_rows, const void* dy, const float* dxr, const int32_t* idx,
              const float* gate, const int32_t* inv_perm, int T, int d, int k, int n_ffn, void* dx,
              hipStream_t st) {
#define MOE_DX(TY, MK)                                                                       \
  hipLaunchKernelGGL((dx_kernel<TY, MK>), row_grid(T), dim3(256), 0, st, dx_rows,             \
                     (const TY*)dy, dxr, idx, gate, inv_perm, T, d, k, n_ffn, (TY*)dx)
  if (dtype == MOE_BF16) {
    if (k <= 8) MOE_DX(__bf16, 8);
    else MOE_DX(__bf16, 16);
  } else {
    if (k <= 8) MOE_DX(float, 8);
    else MOE_DX(float, 16);
  }
#undef MOE_DX
  return check_launch();
}

}  // namespace moe

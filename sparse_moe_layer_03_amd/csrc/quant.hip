// 8-bit codes of rows, with a scale for each row; and which token each of the
// experts' rows is.
//
// A row is read once: it waits in registers while its largest magnitude is
// found, one wave for short rows, a workgroup for long ones (the longest are
// read twice).  The codes are those of the exact quotient, see code_of().
//
// Bound by memory: 16384 rows of 6144 in bf16 68 us (300 MB, 4.4 TB/s), 196608
// rows of 2048 184 us (1.2 GB, 6.6 TB/s), 128 rows 5.3 us.

#include <algorithm>

#include "block.h"
#include "common.h"
#include "row_io.h"

namespace moe {

// N chunks a thread, threads of one wave (ALONE) or of the workgroup; N = 0:
// any number, read twice.
template <typename T, int N, bool ALONE, int NT>
__global__ void __launch_bounds__(NT)
quantize_kernel(const T* __restrict__ x, int64_t ldx, int M, int K, int8_t* __restrict__ q,
                int64_t ldq, float* __restrict__ scale, const int32_t* __restrict__ used) {
  __shared__ uint32_t s[96];
  int turn = 0;
  const int tid = ALONE ? lane_id() : threadIdx.x, nt = ALONE ? kWave : NT;
  const int per = ALONE ? NT / kWave : 1;
  const int rows = used != nullptr ? min(max(used[0], 0), M) : M;
  for (int m = blockIdx.x * per + (ALONE ? (int)(threadIdx.x >> 6) : 0); m < rows; m += gridDim.x * per) {
    const T* row = x + m * ldx;
    int8_t* to = q + m * ldq;
    uint32_t top = 0;
    if constexpr (N > 0) {
      Raw<T> raw[N];
#pragma unroll
      for (int i = 0; i < N; ++i) raw[i] = load_chunk(row, tid + i * nt, K);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float f[8];
        floats(raw[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, magnitude(f[k]));
      }
      top = row_max<ALONE, NT>(top, s, turn);
      const float sc = code_scale(top);
      if (tid == 0) scale[m] = sc;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = tid + i * nt;
        if (c * kChunk < K) {
          float f[8];
          floats(raw[i], f);
          store_codes(to, c, K, codes_of(f, sc));
        }
      }
    } else {
      for (int c = tid; c * kChunk < K; c += nt) {
        float f[8];
        floats(load_chunk(row, c, K), f);
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, magnitude(f[k]));
      }
      top = row_max<ALONE, NT>(top, s, turn);
      const float sc = code_scale(top);
      if (tid == 0) scale[m] = sc;
      for (int c = tid; c * kChunk < K; c += nt) {
        float f[8];
        floats(load_chunk(row, c, K), f);
        store_codes(to, c, K, codes_of(f, sc));
      }
    }
  }
}

template <typename T>
static int launch_quantize_t(const T* x, int64_t ldx, int M, int K, int8_t* q, int64_t ldq,
                             float* scale, const int32_t* used, hipStream_t st) {
  const int cus = stream_cu_count(st);
  if (cus <= 0) return MOE_EHIP;
  const int chunks = (K + kChunk - 1) / kChunk;
#define MOE_QUANT(N, ALONE, NT)                                                                   \
  do {                                                                                            \
    const int per = ALONE ? NT / 64 : 1;                                                          \
    const long blocks = std::min<long>(((long)M + per - 1) / per, (long)cus * (8192 / NT));       \
    hipLaunchKernelGGL((quantize_kernel<T, N, ALONE, NT>), dim3((unsigned)blocks), dim3(NT), 0, st, x, \
                       ldx, M, K, q, ldq, scale, used);                                           \
  } while (0)
  // a wave for a row up to 1024 columns: 8192 rows of 512 6.6 us, 10.7 with a
  // workgroup; 32768 of 1024 24 and 37; of 1536 no difference.  As few threads as
  // hold a row: 8192 rows of 6144 36 us with 256, 57 with 1024
  if (chunks <= 64) MOE_QUANT(1, true, 256);
  else if (chunks <= 128) MOE_QUANT(2, true, 256);
  else if (chunks <= 256) MOE_QUANT(1, false, 256);
  else if (chunks <= 512) MOE_QUANT(2, false, 256);
  else if (chunks <= 1024) MOE_QUANT(4, false, 256);
  else if (chunks <= 4096) MOE_QUANT(4, false, 1024);
  else MOE_QUANT(0, false, 1024);
#undef MOE_QUANT
  return check_launch();
}

int launch_quantize(int dtype, const void* x, int64_t ldx, int M, int K, int8_t* q, int64_t ldq,
                    float* scale, const int32_t* used, hipStream_t st) {
  if (M == 0) return MOE_OK;
  return dtype == MOE_BF16
             ? launch_quantize_t((const __bf16*)x, ldx, M, K, q, ldq, scale, used, st)
             : launch_quantize_t((const float*)x, ldx, M, K, q, ldq, scale, used, st);
}

__global__ void __launch_bounds__(256)
row_tokens_kernel(const float* __restrict__ xs, const int32_t* __restrict__ perm,
                  const int32_t* __restrict__ offsets, int n_ffn, int Tk, int k,
                  int32_t* __restrict__ tok, float* __restrict__ row_scale) {
  const int used = min(offsets[n_ffn], Tk);
  for (int p = blockIdx.x * 256 + threadIdx.x; p < used; p += gridDim.x * 256) {
    const int a = perm[p];
    const bool inside = (unsigned)a < (unsigned)Tk;
    MOE_CHECK(inside, MOE_CHECK_GEMM_ROW);
    const int t = inside ? a / k : 0;
    tok[p] = t;
    row_scale[p] = xs[t];
  }
}

int launch_row_tokens(const float* xs, const int32_t* perm, const int32_t* offsets, int n_ffn, int Tk,
                      int k, int32_t* tok, float* row_scale, hipStream_t st) {
  const int blocks = (int)std::min<long>(((long)Tk + 255) / 256, 2048);
  hipLaunchKernelGGL(row_tokens_kernel, dim3(blocks), dim3(256), 0, st, xs, perm, offsets, n_ffn, Tk, k,
                     tok, row_scale);
  return check_launch();
}

MOE_CHECK_ACCESSOR(check_word_quant)

}  // namespace moe

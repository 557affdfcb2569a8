// Norms before and after a block with its gate and the residual's scale, and
// their gradients.
//
//   r = res_scale x + gate (y rstd(y) w_post),   h = r rstd(r) w_pre
//
// A row is read once and waits in registers through its two reductions; a wave
// serves a short row, a workgroup a long one, and both walk over their rows with
// the next row's loads in flight.  The vectors (w_post, w_pre) stay in
// registers over all rows, in their own type.  Bound by memory: 4 arrays (x,
// y, r, h) forward, 6 backward.  16384 rows of 6144 in bf16 145 us (805 MB, 5.6
// TB/s), with h's codes besides 177 and with the codes alone 150, 128 rows 5.6;
// backward 8192 rows of 4096 89 us and 12 for the sums (403 MB, 4.0 TB/s).
//
// Not bound by memory are the gradients of short and of the longest rows.  Up to
// 2048 columns there are one or two waves a SIMD, each a row group with partial
// sums of its own, whose loads and reductions nothing covers (8192 rows of 512: 29
// us, 7 of them vector issue, 50 MB and 6 for the sums).  Beyond 8192 columns a
// workgroup of 1024 threads has 128 registers a lane and the row does not fit: by
// counters 4096 rows of 16384 write 1.2 GB where dx and dy are 0.27, and load 8
// times as often, from scratch memory (spilled registers, bf16: 29 up to 8192
// columns, 215 up to 16384, 617 beyond; the forward kernel 54 beyond 16384).
//
// Backward, a row group walks over neighbouring rows and keeps its sums of
// the vectors' gradients in fp32 registers; a second kernel adds the groups'
// sums in a fixed order.  A gate row whose tokens lie in one group is written by
// that group; others leave a sum in each group that they touch, in slot 0 (the
// group's first gate row) or 1 (its last).

#include <algorithm>
#include <type_traits>

#include "block.h"
#include "common.h"
#include "row_io.h"

namespace moe {

// f(type, rows of whole chunks, rows that are not kept in the caches): arrays that
// L2 (4 MiB an XCD) cannot hold for the next kernel anyway are loaded and stored
// non-temporally (16384 rows of 6144: 153 -> 145 us; measured by itself, not with
// the router and experts that read h next).
template <typename F>
static int dispatch(const moe_norm_shape& s, F f) {
  const bool bf16 = s.dtype == MOE_BF16, whole = s.d_model % kChunk == 0;
  const bool once = (size_t)s.T * s.d_model * (bf16 ? 2 : 4) > (32u << 20);
  const std::true_type yes;
  const std::false_type no;
  if (!whole) return bf16 ? f((__bf16)0.f, no, no) : f(0.f, no, no);
  if (once) return bf16 ? f((__bf16)0.f, yes, yes) : f(0.f, yes, yes);
  return bf16 ? f((__bf16)0.f, yes, no) : f(0.f, yes, no);
}

struct NormArgs {
  const char *x, *y, *w_post, *gate, *w_pre;
  char *r, *h;
  int64_t ldx, ldy, ldr, ldh;
  int8_t* q;
  float* q_scale;
  float eps, res_scale;
  int T, d, per_gate;
};

// N chunks a thread; ALONE: one wave per row.
template <typename T, int N, bool ALONE, int NT, bool WHOLE, bool ONCE>
__global__ void __launch_bounds__(NT) norm_kernel(NormArgs a) {
  __shared__ uint32_t s[96];
  int turn = 0;
  const int tid = ALONE ? lane_id() : threadIdx.x, nt = ALONE ? kWave : NT;
  const int per = ALONE ? NT / kWave : 1;
  const int step = gridDim.x * per;
  const int d = a.d;
  const float over = 1.f / (float)d;
  const T *x = (const T*)a.x, *y = (const T*)a.y, *gate = (const T*)a.gate;
  Raw<T> wp[N], wn[N], rx[N], ry[N];
  int t = blockIdx.x * per + (ALONE ? (int)(threadIdx.x >> 6) : 0);
  if (t >= a.T) return;
  auto load = [&](int row) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (y != nullptr) ry[i] = load_chunk<WHOLE, ONCE>(y + row * a.ldy, tid + i * nt, d);
      if (x != nullptr) rx[i] = load_chunk<WHOLE, ONCE>(x + row * a.ldx, tid + i * nt, d);
    }
  };
  load(t);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (a.w_post != nullptr) wp[i] = load_chunk<WHOLE>((const T*)a.w_post, tid + i * nt, d);
    if (a.w_pre != nullptr) wn[i] = load_chunk<WHOLE>((const T*)a.w_pre, tid + i * nt, d);
  }
  for (; t < a.T; t += step) {
    Raw<T> rg[N], out[N];
    if (gate != nullptr) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        rg[i] = load_chunk<WHOLE>(gate + (size_t)(t / a.per_gate) * d, tid + i * nt, d);
    }
    float inv = 1.f;
    if (a.w_post != nullptr) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float f[8];
        floats(ry[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += f[k] * f[k];
      }
      sum = row_sum<ALONE, NT>(sum, s, turn);
      inv = 1.f / sqrtf(sum * over + a.eps);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (y != nullptr) {
        float v[8], f[8];
        floats(ry[i], v);
        if (a.w_post != nullptr) {
          floats(wp[i], f);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = v[k] * inv * f[k];
        }
        if (gate != nullptr) {
          floats(rg[i], f);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] *= f[k];
        }
        if (x != nullptr) {
          floats(rx[i], f);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = fmaf(a.res_scale, f[k], v[k]);
        }
        out[i] = raw_of(v, (T*)nullptr);
      } else {
        out[i] = rx[i];
      }
      float f[8];
      floats(out[i], f);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += f[k] * f[k];
    }
    const int next = t + step;
    if (next < a.T) load(next);
    if (a.r != nullptr) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((tid + i * nt) * kChunk < d) store_chunk<WHOLE, ONCE>((T*)a.r + t * a.ldr, tid + i * nt, d, out[i]);
    }
    if (a.w_pre != nullptr) {
      sum = row_sum<ALONE, NT>(sum, s, turn);
      inv = 1.f / sqrtf(sum * over + a.eps);
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float v[8], f[8];
        floats(out[i], v);
        floats(wn[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = v[k] * inv * f[k];
        out[i] = raw_of(v, (T*)nullptr);
        if (a.h != nullptr && (tid + i * nt) * kChunk < d)
          store_chunk<WHOLE, ONCE>((T*)a.h + t * a.ldh, tid + i * nt, d, out[i]);
        if (a.q != nullptr) {
          floats(out[i], v);
#pragma unroll
          for (int k = 0; k < 8; ++k) top = max(top, magnitude(v[k]));
        }
      }
      if (a.q != nullptr) {
        top = row_max<ALONE, NT>(top, s, turn);
        const float scale = code_scale(top);
        if (tid == 0) a.q_scale[t] = scale;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float v[8];
          floats(out[i], v);
          if ((tid + i * nt) * kChunk < d)
            store_codes(a.q + (size_t)t * d, tid + i * nt, d, codes_of(v, scale));
        }
      }
    }
  }
}

template <typename T, bool WHOLE, bool ONCE>
static int launch_norm_t(const NormArgs& a, hipStream_t st) {
  const int cus = stream_cu_count(st);
  if (cus <= 0) return MOE_EHIP;
  const int chunks = (a.d + kChunk - 1) / kChunk;
#define MOE_NORM(N, ALONE, NT)                                                                  \
  do {                                                                                          \
    const int per = ALONE ? NT / 64 : 1;                                                        \
    const long blocks = std::min<long>(((long)a.T + per - 1) / per, (long)cus * (2048 / NT));   \
    hipLaunchKernelGGL((norm_kernel<T, N, ALONE, NT, WHOLE, ONCE>), dim3((unsigned)blocks), dim3(NT), 0, st, a); \
  } while (0)
  // a wave for a row up to 1024 columns: 8192 rows of 512 10.7 us, 18.1 with a
  // workgroup; 32768 of 1024 49 and 61; of 1536 no difference
  if (chunks <= 64) MOE_NORM(1, true, 256);
  else if (chunks <= 128) MOE_NORM(2, true, 256);
  else if (chunks <= 256) MOE_NORM(1, false, 256);
  else if (chunks <= 512) MOE_NORM(2, false, 256);
  else if (chunks <= 768) MOE_NORM(3, false, 256);
  else if (chunks <= 1024) MOE_NORM(2, false, 512);
  else if (chunks <= 2048) MOE_NORM(2, false, 1024);
  else MOE_NORM(4, false, 1024);
#undef MOE_NORM
  return check_launch();
}

int launch_norm(const moe_norm_shape& s, const moe_norm_io& io, hipStream_t st) {
  if (s.T == 0) return MOE_OK;
  NormArgs a{};
  a.x = (const char*)io.x.p;
  a.y = (const char*)io.y.p;
  a.w_post = (const char*)io.w_post;
  a.gate = (const char*)io.gate;
  a.w_pre = (const char*)io.w_pre;
  a.r = (char*)io.r.p;
  a.h = (char*)io.h.p;
  a.ldx = io.x.ld;
  a.ldy = io.y.ld;
  a.ldr = io.r.ld;
  a.ldh = io.h.ld;
  a.q = io.q;
  a.q_scale = io.q_scale;
  a.eps = s.eps;
  a.res_scale = s.res_scale;
  a.T = s.T;
  a.d = s.d_model;
  a.per_gate = s.rows_per_gate;
  return dispatch(s, [&](auto type, auto whole, auto once) {
    return launch_norm_t<decltype(type), decltype(whole)::value, decltype(once)::value>(a, st);
  });
}

// ---- backward

struct NormBwdArgs {
  const char *r, *y, *w_post, *gate, *w_pre, *dr, *dh;
  char *dx, *dy, *dgate;
  int64_t ldr, ldy, lddr, lddh, lddx, lddy;
  float *p_pre, *p_post, *p_gate;  // partial sums: [groups, d], [groups, d], [groups, 2, d]
  float eps, res_scale;
  int T, d, per_gate, groups, rows;  // rows: of a group
  int accumulate;
};

template <typename T, int N, bool ALONE, int NT, bool WHOLE, bool ONCE>
__global__ void __launch_bounds__(NT, N == 1 && NT <= 512 ? 4 : 1) norm_bwd_kernel(NormBwdArgs a) {
  __shared__ uint32_t s[96];
  int turn = 0;
  const int tid = ALONE ? lane_id() : threadIdx.x, nt = ALONE ? kWave : NT;
  const int group = ALONE ? (int)(blockIdx.x * (NT / kWave) + (threadIdx.x >> 6)) : (int)blockIdx.x;
  if (group >= a.groups) return;
  const int lo = group * a.rows, hi = min(a.T, lo + a.rows);
  const int d = a.d;
  const float over = 1.f / (float)d;
  const bool pre = a.w_pre != nullptr, post = a.w_post != nullptr;
  const T *y = (const T*)a.y, *gate = (const T*)a.gate;
  float s_pre[N][8], s_post[N][8], s_gate[N][8];
  Raw<T> wp[N], wn[N], rr[N], ry[N], rdr[N], rdh[N];
  auto clear = [&](float (&v)[N][8]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = 0.f;
  };
  clear(s_pre), clear(s_post), clear(s_gate);
  // (each as soon as its registers are free: a row behind the last one is not
  // asked for)
  auto load_r = [&](int row) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = tid + i * nt;
      if (pre) {
        rr[i] = load_chunk<WHOLE, ONCE>((const T*)a.r + row * a.ldr, c, d);
        rdh[i] = load_chunk<WHOLE, ONCE>((const T*)a.dh + row * a.lddh, c, d);
      }
      if (a.dr != nullptr) rdr[i] = load_chunk<WHOLE, ONCE>((const T*)a.dr + row * a.lddr, c, d);
    }
  };
  auto load_y = [&](int row) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (y != nullptr) ry[i] = load_chunk<WHOLE, ONCE>(y + row * a.ldy, tid + i * nt, d);
  };
  if (lo < hi) {
    load_r(lo);
    load_y(lo);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (post) wp[i] = load_chunk<WHOLE>((const T*)a.w_post, tid + i * nt, d);
    if (pre) wn[i] = load_chunk<WHOLE>((const T*)a.w_pre, tid + i * nt, d);
  }
  for (int t = lo; t < hi; ++t) {
    Raw<T> rg[N];
    if (gate != nullptr) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        rg[i] = load_chunk<WHOLE>(gate + (size_t)(t / a.per_gate) * d, tid + i * nt, d);
    }
    // g, the gradient at r
    float g[N][8];
    float inv_r = 0.f, mean_r = 0.f, inv_y = 1.f;
    float sq = 0.f, dot = 0.f, sy = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (pre) {
        float r[8], h[8], w[8];
        floats(rr[i], r);
        floats(rdh[i], h);
        floats(wn[i], w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          sq += r[k] * r[k];
          dot += h[k] * w[k] * r[k];
        }
      }
      if (post) {
        float v[8];
        floats(ry[i], v);
#pragma unroll
        for (int k = 0; k < 8; ++k) sy += v[k] * v[k];
      }
    }
    if (pre || post) {
      float three[3] = {sq, dot, sy};
      row_sums<ALONE, NT, 3>(three, s, turn);
      if (pre) {
        inv_r = 1.f / sqrtf(three[0] * over + a.eps);
        mean_r = three[1] * over * inv_r * inv_r;
      }
      if (post) inv_y = 1.f / sqrtf(three[2] * over + a.eps);
    }
    float cn = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (a.dr != nullptr) {
        floats(rdr[i], g[i]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) g[i][k] = 0.f;
      }
      if (pre) {
        float r[8], h[8], w[8];
        floats(rr[i], r);
        floats(rdh[i], h);
        floats(wn[i], w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          g[i][k] += inv_r * (h[k] * w[k] - r[k] * mean_r);
          s_pre[i][k] += h[k] * (r[k] * inv_r);
        }
      }
      if (a.dx != nullptr && (tid + i * nt) * kChunk < d) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = a.res_scale * g[i][k];
        store_chunk<WHOLE, ONCE>((T*)a.dx + t * a.lddx, tid + i * nt, d, raw_of(v, (T*)nullptr));
      }
      if (y != nullptr) {
        float v[8], w[8], q[8];
        floats(ry[i], v);
        if (post) floats(wp[i], w);
        if (gate != nullptr) floats(rg[i], q);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float n = v[k] * inv_y;
          float c = g[i][k];
          if (gate != nullptr) {
            s_gate[i][k] += post ? c * n * w[k] : c * n;
            c *= q[k];
          }
          if (post) {
            s_post[i][k] += c * n;
            c *= w[k];
            cn += c * n;
          }
          g[i][k] = c;
        }
      }
    }
    if (t + 1 < hi) load_r(t + 1);
    if (y != nullptr) {
      float mean = 0.f;
      if (post) mean = row_sum<ALONE, NT>(cn, s, turn) * over;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float v[8];
        floats(ry[i], v);
        if (post) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = inv_y * (g[i][k] - v[k] * inv_y * mean);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = g[i][k];
        }
        if ((tid + i * nt) * kChunk < d)
          store_chunk<WHOLE, ONCE>((T*)a.dy + t * a.lddy, tid + i * nt, d, raw_of(v, (T*)nullptr));
      }
    }
    if (t + 1 < hi) load_y(t + 1);
    // the end of a gate row, or of this group
    if (a.dgate != nullptr) {
      const int at = t / a.per_gate;
      if (t + 1 == hi || (t + 1) / a.per_gate != at) {
        const long first = (long)at * a.per_gate, end = std::min<long>(first + a.per_gate, a.T);
        const bool whole = first >= lo && end <= hi;
        float* part = a.p_gate + ((size_t)group * 2 + (at == lo / a.per_gate ? 0 : 1)) * d;
        T* out = (T*)a.dgate + (size_t)at * d;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int c = tid + i * nt;
          if (c * kChunk >= d) continue;
          if (whole) {
            float v[8], old[8];
            if (a.accumulate) floats(load_chunk<WHOLE>((const T*)out, c, d), old);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = a.accumulate ? old[k] + s_gate[i][k] : s_gate[i][k];
            store_chunk<WHOLE>(out, c, d, raw_of(v, (T*)nullptr));
          } else {
            store_chunk<WHOLE>(part, c, d, raw_of(s_gate[i], (float*)nullptr));
          }
        }
        clear(s_gate);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = tid + i * nt;
    if (c * kChunk >= d) continue;
    if (a.p_pre != nullptr)
      store_chunk<WHOLE>(a.p_pre + (size_t)group * d, c, d, raw_of(s_pre[i], (float*)nullptr));
    if (a.p_post != nullptr)
      store_chunk<WHOLE>(a.p_post + (size_t)group * d, c, d, raw_of(s_post[i], (float*)nullptr));
  }
}

// The groups' sums added up.  Workgroups of 64 columns by 16 ranges of the
// groups.  blockIdx.y: dw_pre, dw_post, then the gate rows that several groups
// touch: gate row y, or, where there are more of them than groups, the one at
// the end of group y.
struct NormSumArgs {
  const float *p_pre, *p_post, *p_gate;
  char *dw_pre, *dw_post, *dgate;
  int T, d, per_gate, groups, rows, gates;
  int accumulate;
};

template <typename T>
__global__ void __launch_bounds__(1024) norm_sum_kernel(NormSumArgs a) {
  __shared__ float s[16][64];
  const int col = blockIdx.x * 64 + (threadIdx.x & 63), part = threadIdx.x >> 6;
  const float* from;
  T* out;
  int q0 = 0, q1 = a.groups;
  int gate = -1;
  size_t ld = a.d;
  if (blockIdx.y == 0) {
    from = a.p_pre;
    out = (T*)a.dw_pre;
  } else if (blockIdx.y == 1) {
    from = a.p_post;
    out = (T*)a.dw_post;
  } else {
    const int b = blockIdx.y - 2;
    from = a.p_gate;
    ld = 2 * (size_t)a.d;
    if (a.gates <= a.groups) {
      gate = b;
    } else {
      const long last = (long)(b + 1) * a.rows - 1;  // the group's last token
      if (last + 1 >= a.T) return;
      gate = (int)(last / a.per_gate);
    }
    const long first = (long)gate * a.per_gate, end = std::min<long>(first + a.per_gate, a.T);
    q0 = (int)(first / a.rows);
    q1 = (int)((end - 1) / a.rows) + 1;
    if (q1 - q0 < 2 || (a.gates > a.groups && b != q0)) return;  // whole, or another's
    out = (T*)a.dgate + (size_t)gate * a.d;
  }
  if (out == nullptr) return;
  float sum = 0.f;
  const int n = q1 - q0, each = (n + 15) / 16;
  const int lo = q0 + part * each, hi = std::min(q1, lo + each);
  if (col < a.d) {
    constexpr int U = 8;
    for (int q = lo; q < hi; q += U) {
      float v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u] = 0.f;
        if (q + u < hi) {
          // a group's second slot where the gate row is not its first
          const int slot = gate >= 0 && (int)((long)(q + u) * a.rows / a.per_gate) != gate ? 1 : 0;
          v[u] = from[(size_t)(q + u) * ld + (size_t)slot * a.d + col];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) sum += v[u];
    }
  }
  s[part][threadIdx.x & 63] = sum;
  __syncthreads();
  if (part == 0 && col < a.d) {
    sum = 0.f;
#pragma unroll
    for (int q = 0; q < 16; ++q) sum += s[q][threadIdx.x];
    if (a.accumulate) sum += ElemOps<T>::to_f(out[col]);
    out[col] = ElemOps<T>::from_f(sum);
  }
}

// Row groups: as many as keep the chip busy, of 4 rows or more where that leaves
// a group for each CU, since a group's sums (8 bytes a column and vector,
// written and read) weigh as much as a row.  us in bf16 with 1, 2, 4, 8 groups a
// CU (rows x columns):
//   1024 x 512    13.7  14.0  18.0  18.0     4096 x 2048    43  35.5  39.6  50
//   8192 x 512    51    33    29    33       32768 x 2048  264  172   177  176
//   32768 x 512   204   114   72    64       8192 x 4096    99   97    94  102
//   1024 x 2048   18.2  19.7  25.6  25.5     8192 x 6144   136  134   142  160
//   300 x 4096    15.9  18.9  18.7  18.7     4096 x 16384  308  331   377  485
int norm_bwd_groups(int T, int d, int cus) {
  const int most = d <= 1024 ? 4 * cus : d <= 4096 ? 2 * cus : cus;
  return std::max(1, std::min({most, T, std::max(cus, T / 4)}));
}

static size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

size_t norm_bwd_ws_bytes(const moe_norm_shape& s, int cus) {
  return 256 + 4 * up256((size_t)norm_bwd_groups(s.T, s.d_model, cus) * s.d_model * 4);
}

template <typename T, bool WHOLE, bool ONCE>
static int launch_norm_bwd_t(const NormBwdArgs& a, hipStream_t st) {
  const int chunks = (a.d + kChunk - 1) / kChunk;
#define MOE_NORM_BWD(N, ALONE, NT)                                                                 \
  do {                                                                                             \
    const int per = ALONE ? NT / 64 : 1;                                                           \
    hipLaunchKernelGGL((norm_bwd_kernel<T, N, ALONE, NT, WHOLE, ONCE>),                                        \
                       dim3((unsigned)((a.groups + per - 1) / per)), dim3(NT), 0, st, a);                                                        \
  } while (0)
  if (chunks <= 64) MOE_NORM_BWD(1, true, 256);
  else if (chunks <= 128) MOE_NORM_BWD(1, false, 128);
  else if (chunks <= 256) MOE_NORM_BWD(1, false, 256);
  else if (chunks <= 512) MOE_NORM_BWD(1, false, 512);
  else if (chunks <= 768) MOE_NORM_BWD(1, false, 768);
  else if (chunks <= 1024) MOE_NORM_BWD(1, false, 1024);
  else if (chunks <= 2048) MOE_NORM_BWD(2, false, 1024);
  else MOE_NORM_BWD(4, false, 1024);
#undef MOE_NORM_BWD
  return check_launch();
}

int launch_norm_bwd(const moe_norm_shape& s, const moe_norm_grad_io& io, void* ws, int cus,
                    hipStream_t st) {
  NormBwdArgs a{};
  a.r = (const char*)io.r.p;
  a.y = (const char*)io.y.p;
  a.w_post = (const char*)io.w_post;
  a.gate = (const char*)io.gate;
  a.w_pre = (const char*)io.w_pre;
  a.dr = (const char*)io.dr.p;
  a.dh = (const char*)io.dh.p;
  a.dx = (char*)io.dx.p;
  a.dy = (char*)io.dy.p;
  a.dgate = (char*)io.dgate;
  a.ldr = io.r.ld;
  a.ldy = io.y.ld;
  a.lddr = io.dr.ld;
  a.lddh = io.dh.ld;
  a.lddx = io.dx.ld;
  a.lddy = io.dy.ld;
  a.eps = s.eps;
  a.res_scale = s.res_scale;
  a.T = s.T;
  a.d = s.d_model;
  a.per_gate = s.rows_per_gate;
  const int most = norm_bwd_groups(s.T, s.d_model, cus);
  a.rows = std::max(1, (s.T + most - 1) / most);
  a.groups = (s.T + a.rows - 1) / a.rows;
  a.accumulate = io.accumulate != 0;
  const size_t each = up256((size_t)most * s.d_model * 4);
  float* base = (float*)ws;
  a.p_pre = io.dw_pre ? base : nullptr;
  a.p_post = io.dw_post ? base + each / 4 : nullptr;
  a.p_gate = base + each / 2;
  if (s.T > 0) {
    const int rc = dispatch(s, [&](auto type, auto whole, auto once) {
      return launch_norm_bwd_t<decltype(type), decltype(whole)::value, decltype(once)::value>(a, st);
    });
    if (rc) return rc;
  }
  NormSumArgs b{};
  b.p_pre = a.p_pre;
  b.p_post = a.p_post;
  b.p_gate = a.p_gate;
  b.dw_pre = (char*)io.dw_pre;
  b.dw_post = (char*)io.dw_post;
  b.dgate = (char*)io.dgate;
  b.T = s.T;
  b.d = s.d_model;
  b.per_gate = s.rows_per_gate;
  b.groups = a.groups;
  b.rows = a.rows;
  b.gates = (s.T + (int64_t)s.rows_per_gate - 1) / s.rows_per_gate;
  b.accumulate = a.accumulate;
  // gate rows end where groups do, or one token has each: none is shared
  const bool shared = io.dgate && a.rows % s.rows_per_gate != 0;
  const int gates = shared ? std::min(b.gates, b.groups) : 0;
  if (!io.dw_pre && !io.dw_post && gates == 0) return MOE_OK;
  const dim3 grid((unsigned)((s.d_model + 63) / 64), (unsigned)(2 + gates));
  if (s.dtype == MOE_BF16)
    hipLaunchKernelGGL(norm_sum_kernel<__bf16>, grid, dim3(1024), 0, st, b);
  else
    hipLaunchKernelGGL(norm_sum_kernel<float>, grid, dim3(1024), 0, st, b);
  return check_launch();
}

}  // namespace moe

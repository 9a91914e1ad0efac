// vocab.cu -- softmax cross entropy and distillation over a large vocabulary
// without kept logits (launchers in vocab.h, contraction in vocab_gemm.cuh).
//
// z[n][v] = inv_t * sum_k h[n][k] w[v][k].  Forward: every tile of the logits
// leaves (maximum, sum of exponentials) per row and up to 128 columns, joined
// in a fixed order into lse[n].  Backward, one piece of the vocabulary at a time:
// g[n][v] = c[n] (exp(z - lse[n]) - q[n][v]) as one to three bf16 planes into a
// buffer of the piece's width, then dh += g w and dw = g^T h.  The piece bounds
// the buffer; the logits are recomputed, never kept.
//
// Rows that take no part (no target, an empty list, weight 0 in the backward)
// are left out before the contractions: the rows that remain are gathered, in
// order, into an operand of 16-bit planes (bf16 rows as they are; fp32 rows as
// two of fp16, three of bf16, or both), and every extent follows their count on
// the device.
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "vocab.h"
#include "vocab_gemm.cuh"

namespace rlt {
namespace {

using namespace vocab_tc;

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
inline int64_t round_up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

// ------------------------------------------------------------------ teacher lists
// One warp per row: q = softmax(teacher * inv_t) over the valid slots, the
// slots sorted by id (and slot, so the order never depends on timing) in a
// bitonic network over P >= K keys in shared memory, P / 2 exchanges per stage
// spread over all lanes; empty slots go last.  some[n] = 0 when no slot
// carries weight.  The maximum is taken off before the division by the
// temperature: logits at the type's ends (masks of the lowest value) stay
// finite, so a row of nothing else is uniform, and only -inf is no weight.
template <int P>
__global__ void __launch_bounds__(128) teacher_prep_kernel(const int32_t* ids, const float* teacher, int N, int K,
                                                           int V, float inv_t, int32_t* sid, float* sq, float* slogq,
                                                           float* some) {
  griddep_enter();
  __shared__ unsigned long long keys_s[4][P];
  __shared__ float t_s[4][P];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t n = (int64_t)blockIdx.x * 4 + warp;
  if (n >= N) return;
  unsigned long long* keys = keys_s[warp];
  float* ts = t_s[warp];
  float m = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int k = lane; k < P; k += 32) {
    const int32_t id = k < K ? ids[n * K + k] : -1;
    const float t = k < K ? teacher[n * K + k] : 0.f;
    const bool ok = id >= 0 && id < V;
    if (ok) {
      nan |= isnan(t);
      m = fmaxf(m, t);
    }
    keys[k] = ((unsigned long long)(ok ? id : kNoId) << 32) | (unsigned)k;
    ts[k] = t;
  }
  m = warp_max(m);
  const bool has = m > -INFINITY || __any_sync(0xffffffffu, nan);
  __syncwarp();
#pragma unroll 1
  for (int size = 2; size <= P; size <<= 1)
#pragma unroll 1
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
#pragma unroll
      for (int p = lane; p < P / 2; p += 32) {
        const int i = ((p & ~(stride - 1)) << 1) | (p & (stride - 1)), j = i + stride;
        const unsigned long long a = keys[i], b = keys[j];
        if ((a > b) == ((i & size) == 0)) {
          keys[i] = b;
          keys[j] = a;
        }
      }
      __syncwarp();
    }
  float sum = 0.f;
#pragma unroll
  for (int k = lane; k < P; k += 32) {
    const unsigned long long key = keys[k];
    if ((int)(key >> 32) != kNoId) sum += expf((ts[(unsigned)key] - m) * inv_t);
  }
  sum = warp_sum(sum);
  const float logsum = logf(sum);
#pragma unroll
  for (int k = lane; k < P; k += 32) {
    if (k >= K) break;
    const unsigned long long key = keys[k];
    const int id = (int)(key >> 32);
    const bool on = has && id != kNoId;
    const float t = on ? (ts[(unsigned)key] - m) * inv_t : 0.f;
    sid[n * K + k] = on ? id : kNoId;
    sq[n * K + k] = on ? expf(t) / sum : 0.f;
    slogq[n * K + k] = on ? t - logsum : 0.f;
  }
  if (lane == 0) some[n] = has ? 1.f : 0.f;
}
cudaError_t teacher_prep(const int32_t* ids, const float* teacher, int N, int K, int V, float inv_t, int32_t* sid,
                         float* sq, float* slogq, float* some, cudaStream_t st) {
  const dim3 grid((unsigned)((N + 3) / 4)), block(128);
  const auto kernel = K <= 32    ? teacher_prep_kernel<32>
                      : K <= 64  ? teacher_prep_kernel<64>
                      : K <= 128 ? teacher_prep_kernel<128>
                                 : teacher_prep_kernel<256>;
  return launch_pdl(kernel, grid, block, 0, st, ids, teacher, N, K, V, inv_t, sid, sq, slogq, some);
}

// ------------------------------------------------------------------ rows
// The bf16 planes of 8 elements: x0 = bf16(x), x1 = bf16(x - x0), ...; the sum
// of three is x to 24 bits.
__device__ __forceinline__ void planes8(bf16* dst, int64_t plane, int planes, float* v) {
  for (int p = 0; p < planes; ++p) {
    store8(dst + p * plane, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] -= to_f32(from_f32<bf16>(v[j]));
  }
}
// One row by a warp, several loads in flight per lane: eight elements per lane
// (single loads where a bf16 row is not 16-byte aligned: its copy is, and
// 2-byte stores would cost more), or the lanes side by side for fp32.
template <typename T>
__device__ __forceinline__ void copy_row(const T* x, int d, bool vec, bf16* out, int64_t plane, int planes) {
  const int lane = threadIdx.x & 31;
  int done = 0;
  if (vec) {
    const int d8 = d / 8;
    done = d8 * 8;
    if constexpr (sizeof(T) == 2) {  // one plane: the bits as they are
      for (int c0 = lane; c0 < d8; c0 += 128) {
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c0 + u * 32 < d8) v[u] = reinterpret_cast<const uint4*>(x)[c0 + u * 32];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c0 + u * 32 < d8) reinterpret_cast<uint4*>(out)[c0 + u * 32] = v[u];
      }
    } else {
      for (int c0 = lane; c0 < d8; c0 += 64) {
        float v[2][8];
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (c0 + u * 32 < d8) load8(x + (c0 + u * 32) * 8, v[u]);
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (c0 + u * 32 < d8) planes8(out + (c0 + u * 32) * 8, plane, planes, v[u]);
      }
    }
  }
  if constexpr (sizeof(T) == 2) {
    for (int c0 = done + lane * 8; c0 < d; c0 += 512) {
      __align__(16) bf16 v[2][8];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = c0 + u * 256 + j;
          v[u][j] = c < d ? x[c] : from_f32<bf16>(0.f);
        }
#pragma unroll
      for (int u = 0; u < 2; ++u)  // up to seven zeros behind the row, inside its pitch
        if (c0 + u * 256 < d) *reinterpret_cast<uint4*>(out + c0 + u * 256) = *reinterpret_cast<const uint4*>(v[u]);
    }
    return;
  }
  for (int c0 = done + lane; c0 < d; c0 += 256) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = c0 + u * 32 < d ? to_f32(x[c0 + u * 32]) : 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (c0 + u * 32 >= d) continue;
      for (int p = 0; p < planes; ++p) {
        const bf16 h = from_f32<bf16>(v[u]);
        out[p * plane + c0 + u * 32] = h;
        v[u] -= to_f32(h);
      }
    }
  }
}
// One row as two fp16 planes, x * 2^e = x0 + 2^-12 x1; returns 2^(-e / 2) (e is
// even: the product of two rows' 2^-e may lie outside fp32 where that of the
// halves does not).  *least: the smallest scaled element (Least's bits) of the
// rows so far, per lane.
__device__ __forceinline__ float fp16_row(const float* x, int d, bool vec, __half* out, int64_t plane, uint32_t* least) {
  const int lane = threadIdx.x & 31;
  const int d8 = vec ? d / 8 : 0;  // groups of eight; what is left goes lane by lane
  float m = 0.f;
  for (int c0 = lane; c0 < d8; c0 += 64) {
    float v[2][8] = {};
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (c0 + u * 32 < d8) load8(x + (c0 + u * 32) * 8, v[u]);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(fabsf(v[0][j]), fabsf(v[1][j])));
  }
  for (int c0 = d8 * 8 + lane; c0 < d; c0 += 256) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = c0 + u * 32 < d ? x[c0 + u * 32] : 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) m = fmaxf(m, fabsf(v[u]));
  }
  m = warp_max(m);
  // exponent of the largest element, which goes to [2^13, 2^15); 2^e within the normal numbers
  const int top = (int)(__float_as_uint(m) >> 23) - 127;
  const int e = max(-112, min(126, 14 - top)) & ~1;
  const float up = __uint_as_float((uint32_t)(127 + e) << 23);
  for (int c0 = lane; c0 < d8; c0 += 32) {
    float v[8];
    load8(x + c0 * 8, v);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      __half2 h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float &a = v[2 * j], &b = v[2 * j + 1];
        if (p == 0) {
          a *= up;
          b *= up;
          *least = min(*least, min((__float_as_uint(a) & 0x7fffffffu) - 1u, (__float_as_uint(b) & 0x7fffffffu) - 1u));
        }
        h[j] = __floats2half2_rn(a, b);
        a = (a - __low2float(h[j])) * 4096.f;
        b = (b - __high2float(h[j])) * 4096.f;
      }
      *reinterpret_cast<uint4*>(out + p * plane + c0 * 8) = *reinterpret_cast<const uint4*>(h);
    }
  }
  for (int c0 = d8 * 8 + lane; c0 < d; c0 += 256) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = c0 + u * 32 < d ? x[c0 + u * 32] * up : 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (c0 + u * 32 >= d) continue;
      const __half h = __float2half_rn(v[u]);
      *least = min(*least, (__float_as_uint(v[u]) & 0x7fffffffu) - 1u);
      out[c0 + u * 32] = h;
      out[plane + c0 + u * 32] = __float2half_rn((v[u] - __half2float(h)) * 4096.f);
    }
  }
  return __uint_as_float((uint32_t)(127 - e / 2) << 23);
}

struct Gather {
  // rows of h that take part, in order, to `h_out`; row_of[i] -> row
  RowList list;
  const float* weight;  // backward: rows of weight 0 are left out too
  int N, V, d;
  int row_blocks, rows_per_block, pad_blocks;  // 0: h is read where it is
  const void* h;
  int64_t ld_h;
  int vec_h;
  bf16* h_out;
  int64_t h_plane;
  int32_t* row_of;
  int32_t* count;
  float *loss, *lse;    // forward: zeros for the others
  void* dh;             // backward: a zero row for the others
  int64_t ld_dh;
  int vec_dh;
  // rows of w to `w_out`
  int w_blocks;
  int blocks;           // of all three kinds; a smaller grid walks them
  const void* w;
  int64_t ld_w;
  int vec_w;
  bf16* w_out;
  int64_t w_plane;
  int64_t ld_out;
  int planes;           // bf16 planes (0: none wanted)
  // fp32: the fp16 planes and their rows' 2^(-e / 2), or null
  __half *h16, *w16;
  float *h_inv, *w_inv;
  uint32_t *h_least, *w_least;  // per block of rows of h and of w (Least)
};
// A row of h or w in all the forms wanted.
template <typename T>
__device__ __forceinline__ void convert_row(const T* x, int d, bool vec, bf16* out, int64_t plane, int planes,
                                            __half* out16, float* inv, uint32_t* least) {
  if (planes) copy_row(x, d, vec, out, plane, planes);
  if constexpr (sizeof(T) == 4) {
    if (out16) {
      const float i = fp16_row(x, d, vec, out16, plane, least);
      if ((threadIdx.x & 31) == 0) *inv = i;
    }
  }
}

// Does row n take part?  Both loads are issued whatever the first says.
__device__ __forceinline__ bool row_on(const Gather& g, int64_t n) {
  const float w = g.weight ? g.weight[n] : 1.f;
  return takes_part(g.list, n, g.V) & (w != 0.f);
}
// How many of the rows before `end` take part (every thread gets it).
__device__ __forceinline__ int count_rows(const Gather& g, int64_t end, int* red) {
  int n_on = 0;
  for (int64_t n0 = threadIdx.x; n0 < end; n0 += 256 * 8) {
    float w[8], some[8];
    int32_t id[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t n = n0 + u * 256;
      const bool in = n < end;
      w[u] = !in ? 0.f : g.weight ? g.weight[n] : 1.f;
      some[u] = in && g.list.some ? g.list.some[n] : 0.f;
      id[u] = in && !g.list.some ? g.list.ids[n] : -1;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) n_on += (w[u] != 0.f) & ((some[u] != 0.f) | (id[u] >= 0 && id[u] < g.V));
  }
  n_on = __reduce_add_sync(0xffffffffu, n_on);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = n_on;
  __syncthreads();
  int r = 0;
  for (int i = 0; i < 8; ++i) r += red[i];
  __syncthreads();
  return r;
}

// Operands of the contractions in one launch: blocks that gather rows of h
// (each counts the rows before its own), blocks that zero the rows behind the
// last one up to a multiple of 128, blocks that convert w.
template <typename T>
__device__ __forceinline__ void gather_block(const Gather& g, int b, int* red, uint32_t* least) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (b < g.row_blocks) {
    const int64_t n0 = (int64_t)b * g.rows_per_block;
    int at = count_rows(g, min((int64_t)g.N, n0), red);
    for (int64_t r = n0; r < min((int64_t)g.N, n0 + g.rows_per_block); r += 8) {
      const int64_t n = r + warp;
      const bool on = n < g.N && row_on(g, n);
      if (lane == 0) red[warp] = on;
      __syncthreads();
      int before = 0, all = 0;
      for (int i = 0; i < 8; ++i) {
        before += i < warp ? red[i] : 0;
        all += red[i];
      }
      __syncthreads();
      const int64_t i = at + before;
      at += all;
      if (on) {
        if (lane == 0) g.row_of[i] = (int32_t)n;
        convert_row(static_cast<const T*>(g.h) + n * g.ld_h, g.d, g.vec_h, g.h_out + i * g.ld_out, g.h_plane, g.planes,
                    g.h16 ? g.h16 + i * g.ld_out : nullptr, g.h_inv + i, least);
      } else if (n < g.N) {
        if (g.loss && lane == 0) {
          g.loss[n] = 0.f;
          g.lse[n] = 0.f;
        }
        if (g.dh) {
          T* o = static_cast<T*>(g.dh) + n * g.ld_dh;
          const float z[8] = {};
          if (g.vec_dh && g.d % 8 == 0)
            for (int c = lane * 8; c < g.d; c += 256) store8(o + c, z);
          else
            for (int c = lane; c < g.d; c += 32) o[c] = from_f32<T>(0.f);
        }
      }
    }
    return;
  }
  b -= g.row_blocks;
  if (b < g.pad_blocks) {
    const int count = count_rows(g, g.N, red);
    if (b == 0 && threadIdx.x == 0) *g.count = count;
    const int64_t i = (int64_t)count + b * 8 + warp;
    if (i >= (count + 127) / 128 * 128) return;
    for (int c = lane * 8; c < g.d; c += 256) {
      float v[8] = {};
      planes8(g.h_out + i * g.ld_out + c, g.h_plane, g.planes, v);
    }
    return;
  }
  b -= g.pad_blocks;
  const int64_t v = (int64_t)b * 8 + warp;
  if (v < g.V)
    convert_row(static_cast<const T*>(g.w) + v * g.ld_w, g.d, g.vec_w, g.w_out + v * g.ld_out, g.w_plane, g.planes,
                g.w16 ? g.w16 + v * g.ld_out : nullptr, g.w_inv + v, least);
}
template <typename T>
__global__ void __launch_bounds__(256, 4) gather_kernel(const Gather g) {
  griddep_enter();
  __shared__ int red[8];
  uint32_t least = 0xffffffffu;
  const int b = (int)blockIdx.x;
  gather_block<T>(g, b, red, &least);
  if (sizeof(T) == 4 && g.h_least && (b < g.row_blocks || b >= g.row_blocks + g.pad_blocks)) {
    least = __reduce_min_sync(0xffffffffu, least);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = (int)least;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 0; i < 8; ++i) least = min(least, (uint32_t)red[i]);
      if (b < g.row_blocks) g.h_least[b] = least;
      else g.w_least[b - g.row_blocks - g.pad_blocks] = least;
    }
  }
}
// The same into three bf16 planes, if two fp16 planes do not hold the rows; one
// wave of blocks.
__global__ void __launch_bounds__(256, 3) gather_again_kernel(const Gather g) {
  griddep_enter();
  __shared__ int red[8];
  __shared__ uint32_t least_s[2][8];
  uint32_t h = least_of(g.h_least, g.row_blocks, 256), w = least_of(g.w_least, g.w_blocks, 256);
  h = __reduce_min_sync(0xffffffffu, h);
  w = __reduce_min_sync(0xffffffffu, w);
  if ((threadIdx.x & 31) == 0) {
    least_s[0][threadIdx.x >> 5] = h;
    least_s[1][threadIdx.x >> 5] = w;
  }
  __syncthreads();
  for (int i = 0; i < 8; ++i) {
    h = min(h, least_s[0][i]);
    w = min(w, least_s[1][i]);
  }
  if (fp16_holds(h, w, g.d)) return;
  for (int b = (int)blockIdx.x; b < g.blocks; b += (int)gridDim.x) gather_block<float>(g, b, red, &h);
}

// Joins the statistics of a row's column groups, in a fixed order, and writes
// the row's loss.  A block has 32 rows; first lane = row and warp = group,
// then warp = row and lane = group.
__global__ void __launch_bounds__(1024) join_kernel(const float2* part, int parts, int64_t ld, int N,
                                                    const int32_t* row_of, const int32_t* count, int V, RowList list,
                                                    const float* slogq, const float* zsel, float* loss, float* lse) {
  griddep_enter();
  __shared__ float ms[32][33], ss[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int rows = count ? *count : N;
  if ((int64_t)blockIdx.x * 32 >= rows) return;
  {
    const int64_t i = (int64_t)blockIdx.x * 32 + lane;
    float m = -INFINITY, s = 0.f;
    if (i < rows) {
      for (int t0 = w; t0 < parts; t0 += 256) {
        float2 p[8];
        float mn = m;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          p[u] = t0 + u * 32 < parts ? part[(int64_t)(t0 + u * 32) * ld + i] : make_float2(-INFINITY, 0.f);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) mn = fmaxf(mn, p[u].x);
        const float ref = mn > -INFINITY ? mn : 0.f;
        s = s == 0.f ? 0.f : s * expf(m - ref);
#pragma unroll
        for (int u = 0; u < 8; ++u) s += p[u].y == 0.f ? 0.f : p[u].y * expf(p[u].x - ref);
        m = mn;
      }
    }
    ms[w][lane] = m;
    ss[w][lane] = s;
  }
  __syncthreads();
  const int64_t i = (int64_t)blockIdx.x * 32 + w;
  if (i >= rows) return;
  const int64_t n = row_of ? row_of[i] : i;
  if (!row_of && !takes_part(list, n, V)) {
    if (lane == 0) {
      loss[n] = 0.f;
      lse[n] = 0.f;
    }
    return;
  }
  const float m = ms[lane][w], s = ss[lane][w];
  const float M = warp_max(m), ref = M > -INFINITY ? M : 0.f;
  const float l = M + logf(warp_sum(s == 0.f ? 0.f : s * expf(m - ref)));
  float r = 0.f;
  if (list.q == nullptr) {
    r = zsel[n] - l;
  } else {
    for (int k = lane; k < list.K; k += 32) {
      const int64_t e = n * list.K + k;
      if (list.ids[e] != kNoId && list.q[e] != 0.f) r += list.q[e] * (slogq[e] - zsel[e] + l);
    }
    r = warp_sum(r);
  }
  if (lane == 0) {
    lse[n] = l;
    loss[n] = r;
  }
}

// out rows of the tiles whose K was split = the slabs' sum in order.
struct SlabSum {
  const float4* slab;
  int M, N, K;
  const int32_t *m_count, *k_count;
  int terms, terms2, fine_rows, units, max_splits, cg, bn;  // as in Args
  int rows_in_k;  // the rows that take part run along K (DW), not M
  const int32_t* row_of;
  void* out;
  int64_t ld;
  int accumulate, vec;
  float* acc;  // as in Args
  int acc_in, acc_out;
};
template <typename T>
__global__ void __launch_bounds__(256) slab_sum_kernel(const SlabSum a) {
  griddep_enter();
  const int M = a.m_count ? *a.m_count : a.M, K = a.k_count ? *a.k_count : a.K;
  const int tile_rows = BM * a.cg;
  Cut cut;
  const int terms = (a.rows_in_k ? K : M) <= a.fine_rows ? a.terms2 : a.terms;
  cut.init(M, a.N, K, tile_rows, a.bn, terms, a.units, a.max_splits);
  const int rows = min(M, tile_rows);  // of a tile, that exist
  const int total = cut.rest * rows * (BN / 8), tile = tile_rows * (BN / 4);
  const int64_t stride = (int64_t)cut.rest * tile;
  for (int e = (int)blockIdx.x * 256 + threadIdx.x; e < total; e += (int)gridDim.x * 256) {
    const int row = e % rows, c = e / rows % (BN / 8) * 8, rest = e / (rows * (BN / 8));
    int m, nt;
    cut.place(cut.whole + rest, kPanel / a.cg, &m, &nt);
    const int64_t i = (int64_t)m * tile_rows + row;
    const int col = nt * a.bn + c;
    if (i >= M || c >= a.bn || col >= a.N) continue;
    const float4* p = a.slab + (int64_t)rest * tile + c / 4 * tile_rows + row;
    float s[8] = {};
    for (int k0 = 0; k0 < cut.splits; k0 += 4) {
      float4 lo[4], hi[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k0 + u < cut.splits) {
          lo[u] = p[(k0 + u) * stride];
          hi[u] = p[(k0 + u) * stride + tile_rows];
        }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k0 + u < cut.splits) {
          s[0] += lo[u].x; s[1] += lo[u].y; s[2] += lo[u].z; s[3] += lo[u].w;
          s[4] += hi[u].x; s[5] += hi[u].y; s[6] += hi[u].z; s[7] += hi[u].w;
        }
    }
    if (a.acc) {
      float* p = a.acc + i * a.N + col;
      const int cols = min(8, a.N - col);
      const bool whole = cols == 8 && a.N % 4 == 0;
      if (a.acc_in) {
        if (whole) {
          float old[8];
          load8(p, old);
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] += old[j];
        } else {
          for (int j = 0; j < cols; ++j) s[j] += p[j];
        }
      }
      if (a.acc_out) {
        if (whole) store8(p, s);
        else
          for (int j = 0; j < cols; ++j) p[j] = s[j];
        continue;
      }
    }
    T* o = static_cast<T*>(a.out) + (a.row_of ? a.row_of[i] : i) * a.ld + col;
    if (a.vec && col + 8 <= a.N) {
      if (a.accumulate) {
        float old[8];
        load8(o, old);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += old[j];
      }
      store8(o, s);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < a.N) o[j] = from_f32<T>(a.accumulate ? s[j] + to_f32(o[j]) : s[j]);
    }
  }
}

// ------------------------------------------------------------------ residuals
// acc[i] (+)= sum_k resid[n][k] w[ids[n][k]]: what rounding g to bf16 took from
// dh at the row's listed ids.  Those are the entries that carry dh (the target
// has p - 1 where others have their p), and a sum near zero, of rows of w that
// point the same way, shows their rounding most: dh of bf16 operands was off by
// 1.35 to 1.57 of its own rounding with one plane of g, and is by 1.00 to 1.14
// with its listed entries whole (234 cases of d = 17 to 400); a second plane
// would cost a quarter of the backward.  One warp per row; entries whose
// residual is below 1 / (8 sqrt(K)) of the row's largest, together an eighth of
// it, are left out, so a list costs few rows of w.  Where fine_rows or fewer
// take part g has both planes and nothing is missing.
__global__ void __launch_bounds__(256) residual_kernel(RowList list, const float* resid, const int32_t* row_of,
                                                       const int32_t* count, int fine_rows, int V, const bf16* w,
                                                       int64_t ld_w, int d, float* acc, int add) {
  griddep_enter();
  __shared__ int32_t ids_s[8][256];
  __shared__ float r_s[8][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * 8 + warp;
  const int rows = *count;
  if (i >= rows) return;
  int32_t* ids = ids_s[warp];
  float* rs = r_s[warp];
  int kept = 0;
  if (rows > fine_rows) {
    const int64_t e0 = (int64_t)row_of[i] * list.K;
    int32_t id[8];
    float r[8], m = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int k = u * 32 + lane;
      id[u] = k < list.K ? list.ids[e0 + k] : -1;
      r[u] = id[u] >= 0 && id[u] < V ? resid[e0 + k] : 0.f;
      m = fmaxf(m, fabsf(r[u]));
    }
    m = warp_max(m);
    const float least = list.K == 1 ? 0.f : m * 0.125f * rsqrtf((float)list.K);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool keep = !(fabsf(r[u]) <= least);  // NaN is kept
      const unsigned in = __ballot_sync(0xffffffffu, keep);
      if (keep) {
        const int at = kept + __popc(in & ((1u << lane) - 1));
        ids[at] = id[u];
        rs[at] = r[u];
      }
      kept += __popc(in);
    }
    __syncwarp();
  }
  float* out = acc + i * d;
  const bool vec = d % 4 == 0;
  for (int c0 = lane * 8; c0 < d; c0 += 1024) {
    float s[4][8] = {};
    for (int e = 0; e < kept; ++e) {
      const bf16* row = w + (int64_t)ids[e] * ld_w;
      const float r = rs[e];
      float x[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = c0 + u * 256;
        if (c + 8 <= d) {
          load8(row + c, x[u]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[u][j] = c + j < d ? to_f32(row[c + j]) : 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[u][j] = fmaf(r, x[u][j], s[u][j]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + u * 256;
      if (vec && c + 8 <= d) {
        if (add) {
          float old[8];
          load8(out + c, old);
#pragma unroll
          for (int j = 0; j < 8; ++j) s[u][j] += old[j];
        }
        store8(out + c, s[u]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < d) out[c + j] = add ? s[u][j] + out[c + j] : s[u][j];
      }
    }
  }
}

// ------------------------------------------------------------------ few rows
// Statistics, or g, of up to 8 rows: bound by reading w once, so w goes through
// registers (16-byte loads, the next step's in flight under this one's
// products) and h through shared memory, in fp32.  A warp takes two to four
// rows of w at a time against all NB rows of h; the sums of its lanes are added by
// exchanging halves, after which lane r * NB + n holds z of w row r and h row n.
// At V = 32000, d = 2048: bf16 29, 31, 39 and 56 us for 1, 2, 4 and 8 rows
// against 33 on the tensor cores, so up to 2; fp32 53 and 79 us for 4 and 8
// against 172 (there w is first split into planes), so up to 8.
// Rows of w per group: few, so that the groups spread evenly over the warps
// (at V = 32000 four per group leave a round 38 % full), but four where each
// read of h from shared memory has to serve more products.
template <int NB>
constexpr int kFewW = NB <= 2 ? 2 : 4;
constexpr int kFewRows = 8;
int few_rows_limit(int dtype) { return dtype ? 2 : kFewRows; }
constexpr size_t kFewSmem = 200 << 10;  // h in shared memory

template <typename T>
struct Raw;
template <>
struct Raw<bf16> {
  uint4 a;
  __device__ __forceinline__ void load(const bf16* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ float get(int j) const {
    const uint32_t w = j < 2 ? a.x : j < 4 ? a.y : j < 6 ? a.z : a.w;
    return __uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16);
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p + 4));
  }
  __device__ __forceinline__ float get(int j) const {
    const float4& v = j < 4 ? a : b;
    return (j & 3) == 0 ? v.x : (j & 3) == 1 ? v.y : (j & 3) == 2 ? v.z : v.w;
  }
};

//
// fp32 rows whose statistics came from here get their g from here too (FewGrad),
// from the same sums: the tensor cores' logits lie a few 1e-7 of themselves
// towards zero, which an lse of the same logits takes out of p = exp(z - lse)
// and an exact one does not (gradients of 1 to 8 rows were off by up to 5.7e-6
// where fp32 matrix products leave 1e-6; now by 1.3e-6 at most in 400 cases).
// The backward of 8 rows, V = 32000, d = 2048 takes 457 us for 491 with the
// logits from fp16 planes, that of 8, V = 4000, d = 512 48 for 56.
struct FewGrad {
  bf16* g;  // three planes of [rows][ld], from row 0 of w on; rows up to 64 and columns up to 64 are filled with zeros
  int64_t plane, ld;
  const int32_t *row_of, *count;
  const float *lse, *weight;
  int v0;   // first row of w in the vocabulary
};
template <typename T, int NB, bool GRADIENT>
__global__ void __launch_bounds__(512, 1) few_rows_kernel(const T* h, int64_t ld_h, const T* w, int64_t ld_w, int N,
                                                          int V, int d, int vec, float scale, RowList list, int early,
                                                          float2* part, int64_t part_ld, float* zsel,
                                                          const FewGrad fg) {
  constexpr int R = kFewW<NB>;
  constexpr int U = (sizeof(T) == 2 ? 8 : 4) / R;  // groups of 256 columns per step
  extern __shared__ float4 hs[];  // [NB][2][d8]: the two halves of every group of eight
  __shared__ float2 sums[16][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d8 = (d + 7) / 8;
  const int steps = (d8 + 32 * U - 1) / (32 * U);
  const int groups = (V + R - 1) / R, stride = (int)gridDim.x * 16;
  const int g0 = warp * (int)gridDim.x + (int)blockIdx.x;
  const int total = g0 < groups ? ((groups - 1 - g0) / stride + 1) * steps : 0;
  if (!early) griddep_enter();
  Raw<T> cur[U][R], nxt[U][R];
  int f_step = 0, f_v = g0 * R;  // what is fetched next
  auto fetch = [&](Raw<T>(&x)[U][R]) {
    const int c = f_step * (32 * U) + lane;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const T* row = w + (int64_t)min(f_v + i, V - 1) * ld_w;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if ((c + u * 32) * 8 + 8 <= d) x[u][i].load(row + (c + u * 32) * 8);
    }
    if (++f_step == steps) {
      f_step = 0;
      f_v += stride * R;
    }
  };
  if (vec && total > 0) fetch(cur);
  for (int i = threadIdx.x; i < NB * d8 * 2; i += 512) {
    const int n = i / (d8 * 2), r = i - n * d8 * 2, half = r / d8, g = r - half * d8;
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = g * 8 + half * 4 + j;
      v[j] = n < N && k < d ? to_f32(h[n * ld_h + k]) : 0.f;
    }
    hs[i] = make_float4(v[0], v[1], v[2], v[3]);
  }
  if (early) griddep_enter();
  __syncthreads();
  const int n = lane % NB, r = lane / NB;  // what this lane finishes
  bool mine = lane < R * NB && n < N;
  [[maybe_unused]] float cw = 0.f, l = 0.f;
  [[maybe_unused]] bf16* g_row = nullptr;  // of row n, if it takes part
  if constexpr (GRADIENT) {
    const int count = *fg.count;
    int at = -1;
    for (int i = 0; i < count; ++i)
      if (fg.row_of[i] == n) at = i;
    mine = mine && at >= 0;
    if (mine) {
      cw = fg.weight[n] * scale;
      l = fg.lse[n];
      g_row = fg.g + at * fg.ld;
    }
    // what the products read besides: rows behind the last, columns behind V
    const int64_t thread = (int64_t)blockIdx.x * 512 + threadIdx.x, threads = (int64_t)gridDim.x * 512;
    const int chunks = (V + BK - 1) / BK * (BK / 8), rows = count > 0 ? BK - count : 0;
    for (int64_t e = thread; e < (int64_t)3 * rows * chunks; e += threads) {
      const int64_t row = e / chunks, c = e - row * chunks;
      *reinterpret_cast<uint4*>(fg.g + row / rows * fg.plane + (count + row % rows) * fg.ld + c * 8) = make_uint4(0, 0, 0, 0);
    }
    const int tail = chunks * 8 - V;
    for (int64_t e = thread; e < (int64_t)3 * count * tail; e += threads) {
      const int64_t row = e / tail;
      fg.g[row / count * fg.plane + row % count * fg.ld + V + e % tail] = from_f32<bf16>(0.f);
    }
  }
  int pos = 0, next = mine ? list.ids[(int64_t)n * list.K] : kNoId;
  float m = -INFINITY, s = 0.f;
  float acc[R * NB];
#pragma unroll
  for (int i = 0; i < R * NB; ++i) acc[i] = 0.f;
  int step = 0;
  int64_t v0 = (int64_t)g0 * R;
#pragma unroll 2
  for (int it = 0; it < total; ++it) {
    if (vec && it + 1 < total) fetch(nxt);
    if (vec) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = step * (32 * U) + u * 32 + lane;
        if (c * 8 + 8 > d) continue;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float4 lo = hs[(b * 2) * d8 + c], hi = hs[(b * 2 + 1) * d8 + c];
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const Raw<T>& x = cur[u][i];
            float& t = acc[i * NB + b];
            t = fmaf(x.get(0), lo.x, t);
            t = fmaf(x.get(1), lo.y, t);
            t = fmaf(x.get(2), lo.z, t);
            t = fmaf(x.get(3), lo.w, t);
            t = fmaf(x.get(4), hi.x, t);
            t = fmaf(x.get(5), hi.y, t);
            t = fmaf(x.get(6), hi.z, t);
            t = fmaf(x.get(7), hi.w, t);
          }
        }
      }
    }
    // rows off the 16-byte grid, and the last columns of the others: element
    // by element, the lanes side by side
    const float* hf = reinterpret_cast<const float*>(hs);
    const int k_end = min(d, (step + 1) * 256 * U);
    for (int k0 = vec ? max(step * 256 * U, d / 8 * 8) : step * 256 * U; k0 < k_end; k0 += 128) {
      float y[4][R];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int k = k0 + u * 32 + lane;
          y[u][i] = k < k_end ? to_f32(w[min(v0 + i, (int64_t)V - 1) * ld_w + k]) : 0.f;
        }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = min(k0 + u * 32 + lane, d - 1);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float hk = hf[((b * 2 + ((k >> 2) & 1)) * d8 + (k >> 3)) * 4 + (k & 3)];
#pragma unroll
          for (int i = 0; i < R; ++i) acc[i * NB + b] = fmaf(y[u][i], hk, acc[i * NB + b]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < R; ++i) cur[u][i] = nxt[u][i];
    if (++step != steps) continue;
    step = 0;
    // the group's sums over the lanes: value i ends in lane i
    __syncwarp();
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      if (off >= R * NB) {
#pragma unroll
        for (int i = 0; i < R * NB; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], off);
      } else {
        const bool upper = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < R * NB; ++i) {
          if (i < off) {
            const float send = upper ? acc[i] : acc[i + off], keep = upper ? acc[i + off] : acc[i];
            acc[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
          }
        }
      }
    }
    const int64_t v = v0 + r;
    if (mine && v < V) {
      const float z = acc[0] * scale;
      const int64_t id = GRADIENT ? v + fg.v0 : v;
      while (next < id && pos + 1 < list.K) next = list.ids[(int64_t)n * list.K + ++pos];
      if constexpr (GRADIENT) {
        float g = cw * expf(z - l);
        while (next == id) {
          g -= cw * (list.q ? list.q[(int64_t)n * list.K + pos] : 1.f);
          next = ++pos < list.K ? list.ids[(int64_t)n * list.K + pos] : kNoId;
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          const bf16 b = from_f32<bf16>(g);
          g_row[p * fg.plane + v] = b;
          g -= to_f32(b);
        }
      } else {
        while (next == id) {
          zsel[(int64_t)n * list.K + pos] = z;
          next = ++pos < list.K ? list.ids[(int64_t)n * list.K + pos] : kNoId;
        }
        const float mn = fmaxf(m, z), ref = mn > -INFINITY ? mn : 0.f;
        s = (s == 0.f ? 0.f : s * expf(m - ref)) + expf(z - ref);
        m = mn;
      }
    }
    __syncwarp();
    v0 += (int64_t)stride * R;
#pragma unroll
    for (int i = 0; i < R * NB; ++i) acc[i] = 0.f;
  }
  if constexpr (GRADIENT) return;
  sums[warp][lane] = make_float2(m, s);
  __syncthreads();
  if (warp == 0 && lane < NB && lane < N) {  // the block's statistics of row `lane`
    float M = -INFINITY, total = 0.f;
    for (int k = 0; k < 16; ++k)
      for (int i = 0; i < R; ++i) M = fmaxf(M, sums[k][i * NB + lane].x);
    const float ref = M > -INFINITY ? M : 0.f;
    for (int k = 0; k < 16; ++k)
      for (int i = 0; i < R; ++i) {
        const float2 t = sums[k][i * NB + lane];
        total += t.y == 0.f ? 0.f : t.y * expf(t.x - ref);
      }
    part[(int64_t)blockIdx.x * part_ld + lane] = make_float2(M, total);
  }
}

// ------------------------------------------------------------------ host
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// A 16-bit operand in memory: `planes` matrices [rows][cols], rows ld apart.
struct Matrix {
  const bf16* p;
  int64_t rows, cols, ld, plane;
  int planes;
};
// Boxes of box_cols (64: 128-byte swizzle, 32: 64-byte) by box_rows of one
// plane; what lies outside [rows][cols] reads as 0.
cudaError_t tensor_map(CUtensorMap* tm, const Matrix& m, int box_rows, int box_cols = BK) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  cuuint64_t dims[3] = {(cuuint64_t)m.cols, (cuuint64_t)m.rows, (cuuint64_t)m.planes};
  cuuint64_t strides[2] = {(cuuint64_t)m.ld * 2, (cuuint64_t)(m.planes > 1 ? m.plane : m.rows * m.ld) * 2};
  cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1}, step[3] = {1, 1, 1};
  const CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<bf16*>(m.p), dims, strides, box, step,
                        CU_TENSOR_MAP_INTERLEAVE_NONE,
                        box_cols == BK ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

#define VOCAB_TRY(...)                \
  do {                                \
    cudaError_t e_ = (__VA_ARGS__);   \
    if (e_ != cudaSuccess) return e_; \
  } while (0)

// Raises a kernel's shared-memory limit, once per device.
template <auto Kernel>
cudaError_t set_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  VOCAB_TRY(cudaGetDevice(&dev));
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  VOCAB_TRY(cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  done.fetch_or(bit, std::memory_order_relaxed);
  return cudaSuccess;
}

// The operands of a contraction: A, B, the gradient that GRAD writes or null,
// and the second form of A (GRAD: of the gradient) and B that some kinds may
// choose, or null.
struct Operands {
  Matrix A, B;
  const Matrix* G = nullptr;
  const Matrix *A2 = nullptr, *B2 = nullptr;
};
template <int KIND, int CG>
cudaError_t launch(const Operands& o, Args a, cudaStream_t st) {
  using C = Cfg<CG>;
  constexpr bool A_MN = KIND == DW, B_MN = KIND == DH || KIND == DW;
  CUtensorMap ta, tb, tg, ta2, tb2;
  a.stages = std::min(C::MOST_STAGES, C::PIPE / (C::A_BYTES + a.bn / CG * BK * 2));
  // (a box of rows that are not there costs as much as one of rows that are)
  a.a_rows = A_MN ? BM : (int)std::min<int64_t>(BM, round_up(a.M, 8));
  VOCAB_TRY(tensor_map(&ta, o.A, A_MN ? 64 : a.a_rows));
  VOCAB_TRY(tensor_map(&tb, o.B, B_MN ? 64 : a.bn / CG));
  if (o.G) VOCAB_TRY(tensor_map(&tg, *o.G, 32, 32));
  else tg = ta;
  if (o.A2) VOCAB_TRY(KIND == GRAD ? tensor_map(&ta2, *o.A2, 32, 32) : tensor_map(&ta2, *o.A2, A_MN ? 64 : a.a_rows));
  else ta2 = ta;
  if (o.B2) VOCAB_TRY(tensor_map(&tb2, *o.B2, B_MN ? 64 : a.bn / CG));
  else tb2 = tb;
  VOCAB_TRY((set_smem<vocab_gemm_kernel<KIND, CG>>(C::SMEM)));
  const int64_t tiles = round_up(a.M, BM * CG) / (BM * CG) * (round_up(a.N, a.bn) / a.bn) * a.max_splits;
  if (tiles == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(std::min<int64_t>(tiles, kSmCount / CG) * CG));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, vocab_gemm_kernel<KIND, CG>, ta, tb, tg, ta2, tb2, a);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Two CTAs per tile (256 rows; each loads half of the columns' operand)
// wherever there is more than one row tile.
template <int KIND>
cudaError_t contract(const Operands& o, const Args& a, cudaStream_t st) {
  return a.M > BM ? launch<KIND, 2>(o, a, st) : launch<KIND, 1>(o, a, st);
}

// Where things lie in the workspace, and how the work is cut.
struct Layout {
  size_t sid = 0, sq = 0, slogq = 0, some = 0, row_of = 0, count = 0, h = 0, w = 0, h16 = 0, w16 = 0, h_inv = 0,
         w_inv = 0, h_least = 0, w_least = 0, part = 0, zsel = 0, g = 0,
         dh = 0, dw = 0, acc = 0, resid = 0, total = 0;
  int planes = 1, terms = 1;      // bf16 planes of h and w; products of h w^T
  int g_planes = 1, g_terms = 1;  // of g, and of its products
  bool few = false, gather = true, pack_w = false;
  int64_t rows = 0;  // rows of the gathered operand, a multiple of 256
  int64_t ld = 0;    // row distance of gathered and packed operands
  int bn = BN, parts = 0, piece = 0, pieces = 0;
  int dh_splits = 1, dw_splits = 1;  // at most
  bool residuals = false;  // g may be one plane: dh gets back what rounding took from its listed entries
};

bool tma_ready(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0; }

constexpr int kMostSplits = 64;
constexpr int kFineRows = 256;  // a multiple of the rows of a tile
int cta_group(int M) { return M > BM ? 2 : 1; }
// Floats that the split sums of a product can take: split_rule makes at most
// two rounds of split tiles, and none of fewer than 32 k-blocks.
int64_t slab_floats(int64_t M, int64_t N, int64_t kblocks, int* most) {
  *most = kblocks >= 32 ? kMostSplits : 1;
  if (*most == 1) return 0;
  const int64_t n_tiles = (N + 63) / 64;  // of the narrowest
  int64_t need = 0;
  for (int cg = 1; cg <= 2; ++cg) {
    const int64_t all = (M + BM * cg - 1) / (BM * cg) * n_tiles;
    need = std::max(need, std::min<int64_t>(2 * (kSmCount / cg), all * kMostSplits) * BM * cg * BN);
  }
  return need;
}

// Columns per tile of the logits: the width whose rounds take the least time,
// a tile costing its columns and 128 more for its rows' operand and what is
// fixed (192 columns ran at 0.87 of the rate of 256).  Wide tiles where there
// are many, narrow ones where wide ones leave SMs idle: forward and backward of
// 300 rows, V = 4000, d = 1024 in 63 us for 69; 12 fp32 rows, V = 251, d = 2432
// in 155 us for 172.
int logit_columns(int64_t M, int64_t V) {
  const int cg = cta_group((int)M);
  const int64_t units = kSmCount / cg, m_tiles = (M + BM * cg - 1) / (BM * cg);
  int best = BN;
  int64_t cost = INT64_MAX;
  for (int bn = BN; bn >= 64; bn -= 64) {  // the gradient writes 64 columns at a time
    const int64_t c = (m_tiles * ((V + bn - 1) / bn) + units - 1) / units * (bn + 128);
    if (c < cost) {
      cost = c;
      best = bn;
    }
  }
  return best;
}
// Columns per tile of a product with d columns (its idle SMs take ranges of
// K): fewer than 256 where d does not fill them, 2 to 8 % of a backward at
// d = 64 to 300.
int product_columns(int64_t M, int64_t d) {
  const int step = 64 * cta_group((int)M);
  int best = BN;
  int64_t cost = INT64_MAX;
  for (int bn = BN; bn >= step; bn -= step) {
    const int64_t c = (d + bn - 1) / bn * (bn + 64);
    if (c < cost) {
      cost = c;
      best = bn;
    }
  }
  return best;
}

// Time of a product in k-blocks of a round: its whole rounds, and the last one
// as split_rule cuts it.
int64_t product_time(int64_t M, int64_t N, int64_t kblocks) {
  const int cg = cta_group((int)M), bn = product_columns(M, N), units = kSmCount / cg;
  const int64_t tiles = (M + BM * cg - 1) / (BM * cg) * ((N + bn - 1) / bn);
  const int left = (int)(tiles % units), s = left ? split_rule(left, units, (int)kblocks, kMostSplits) : 1;
  const int64_t rest = !left ? 0
                       : s == 1 ? kblocks
                                : (left * s + units - 1) / units * ((kblocks + s - 1) / s + 12) + 12;
  return tiles / units * kblocks + rest;
}

// One wave of blocks gathers rows of h, each of which counts all rows before
// its own; eight rows of w to a block.
struct RowBlocks {
  int per_block, blocks;
};
RowBlocks gather_rows(int N) {
  constexpr int kWave = 4 * kSmCount;
  const int per_block = (int)round_up(std::max(1, (N + kWave - 1) / kWave), 8);
  return {per_block, (N + per_block - 1) / per_block};
}
int w_gather_blocks(int V) { return (V + 7) / 8; }

Layout layout(const VocabLoss& p, int backward) {
  Layout L;
  auto take = [&](size_t n) {
    const size_t at = L.total;
    L.total += align256(n);
    return at;
  };
  const bool f32 = p.dtype == 0;
  L.planes = !f32 ? 1 : backward ? 3 : 0;
  L.terms = f32 ? 3 : 1;
  L.rows = round_up(std::max(p.N, 1), 256);
  L.ld = round_up(p.d, 64);  // rows on 128-byte lines
  const size_t n = (size_t)p.N;
  if (p.teacher) {
    L.sid = take(n * p.K * 4);
    L.sq = take(n * p.K * 4);
    L.slogq = take(n * p.K * 4);
    L.some = take(n * 4);
  }
  const bool few = p.N <= few_rows_limit(p.dtype) && (size_t)kFewRows * round_up(p.d, 8) * 4 <= kFewSmem;
  L.few = few && (!backward || f32);  // (of bf16 rows g is rounded far coarser than where its logits differ)
  // A forward pass over one row tile has nothing to gain from leaving rows
  // out, and its rows do not mix: it reads h where it is.
  L.gather = backward || (!L.few && (f32 || p.N > BM || !tma_ready(p.h, p.ld_h)));
  // w is read where it is whenever TMA can: rows that do not start on 128-byte
  // lines cost up to 27 % of a contraction's rate (d = 1000), but a copy on
  // every call costs more (2048 rows, V = 32000: 107 us with it, 94 without).
  L.pack_w = (backward || !L.few) && (f32 || !tma_ready(p.w, p.ld_w));
  if (L.gather) {
    L.row_of = take(n * 4);
    L.count = take(4);
    L.h = take((size_t)L.planes * L.rows * L.ld * 2);
  }
  if (L.pack_w) L.w = take((size_t)L.planes * p.V * L.ld * 2);
  if (f32 && !L.few) {
    // the forward's second form takes the fp16 planes' place
    L.h16 = take((size_t)(backward ? 2 : 3) * L.rows * L.ld * 2);
    L.w16 = take((size_t)(backward ? 2 : 3) * p.V * L.ld * 2);
    L.h_inv = take((size_t)L.rows * 4);
    L.w_inv = take((size_t)(round_up(p.V, BN) + BN) * 4);  // tiles read past V
    L.h_least = take((size_t)gather_rows(p.N).blocks * 4);
    L.w_least = take((size_t)w_gather_blocks(p.V) * 4);
  }
  const int64_t n_tiles = (p.V + BN - 1) / BN;
  L.bn = logit_columns(p.N, p.V);
  if (!backward) {
    L.parts = L.few ? (int)std::min<int64_t>(kSmCount, (p.V + 15) / 16) : 2 * ((p.V + L.bn - 1) / L.bn);
    L.part = take((size_t)L.parts * (L.few ? kFewRows : L.rows) * 8);
    L.zsel = take(n * p.K * 4);
    return L;
  }
  // g of bf16 operands is rounded to bf16 as an operand of the products, about
  // as much again as the gradients' own rounding (1.41 of it in all, over many
  // rows).  Over few rows single entries of g carry the gradients and their
  // rounding does not average: where up to kFineRows take part, a count that
  // only the device knows, a second plane takes it away, at 13 to 22 % of the
  // backward's time (64 to 256 rows, V = 32000, d = 2048).  Over more rows dh,
  // whose rows stay single, gets back what rounding took from their listed
  // entries (residual_kernel).
  L.g_planes = f32 ? 3 : p.N <= kFineRows ? 2 : 1;  // at most, and what the cut of the work reckons with
  L.g_terms = f32 ? 6 : L.g_planes;
  // The piece: at most as wide as 512 MB of g allow (256 MB was 5 % slower at
  // 16,368 rows, 1 GB no faster), at least 2048 columns, and of the next few
  // equal cuts the one whose products fill their rounds best.
  const int64_t most = std::max<int64_t>(2048, ((int64_t)512 << 20) / (L.rows * 2 * L.g_planes) / BN * BN);
  const int64_t whole = n_tiles * BN, fewest = (whole + most - 1) / most;
  int64_t best = INT64_MAX;
  for (int64_t q = fewest; q < fewest + 3; ++q) {
    const int64_t piece = round_up((whole + q - 1) / q, BN);
    if (q > fewest && piece < 2048) break;
    const int64_t pieces = (whole + piece - 1) / piece;
    const int64_t cost = pieces * (product_time(p.N, p.d, piece / BK * L.g_terms) +
                                   product_time(piece, p.d, L.rows / BK * L.g_terms) + 32);
    if (cost < best) {
      best = cost;
      L.piece = (int)piece;
      L.pieces = (int)pieces;
    }
  }
  L.g = take((size_t)(f32 ? 3 * L.rows : std::max<int64_t>(L.rows, 2 * kFineRows)) * L.piece * 2);
  L.dw = take((size_t)slab_floats(L.piece, p.d, L.rows / BK * L.g_terms, &L.dw_splits) * 4);
  L.dh = take((size_t)slab_floats(p.N, p.d, (int64_t)L.piece / BK * L.g_terms, &L.dh_splits) * 4);
  L.residuals = !f32 && p.N > kFineRows;
  if (L.residuals) L.resid = take(n * p.K * 4);
  if (L.pieces > 1 || L.residuals) L.acc = take((size_t)L.rows * p.d * 4);  // dh over the pieces, residuals
  return L;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

// What both directions start from: lists, the rows that take part, operands.
struct Prepared {
  RowList list;
  const float* slogq = nullptr;
  const int32_t *row_of = nullptr, *count = nullptr;
  const float *h_inv = nullptr, *w_inv = nullptr;
  Matrix h, w;    // of the products of g
  Matrix zh, zw;  // of the logits
  Matrix zh2, zw2;  // fp32: their second form
  Least least = {};
};

int vector_rows(const void* p, int64_t ld, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % (dtype ? 8 : 4) == 0;
}

cudaError_t prepare(const VocabLoss& p, const Layout& L, void* ws, const float* weight, float* loss, float* lse,
                    void* dh, int64_t ld_dh, Prepared* r, cudaStream_t st) {
  r->list = RowList{p.ids, nullptr, nullptr, p.K};
  if (p.teacher) {
    int32_t* sid = at<int32_t>(ws, L.sid);
    float *sq = at<float>(ws, L.sq), *slogq = at<float>(ws, L.slogq), *some = at<float>(ws, L.some);
    VOCAB_TRY(teacher_prep(p.ids, p.teacher, p.N, p.K, p.V, p.inv_t, sid, sq, slogq, some, st));
    r->list = RowList{sid, sq, some, p.K};
    r->slogq = slogq;
  }
  r->h = Matrix{static_cast<const bf16*>(p.h), p.N, p.d, p.ld_h, 0, 1};
  r->w = Matrix{static_cast<const bf16*>(p.w), p.V, p.d, p.ld_w, 0, 1};
  r->zh = r->h;
  r->zw = r->w;
  if (!L.gather && !L.pack_w) return cudaSuccess;
  Gather g{};
  g.N = p.N;
  g.V = p.V;
  g.d = p.d;
  g.ld_out = L.ld;
  g.planes = L.planes;
  if (L.gather) {
    g.list = r->list;
    g.weight = weight;
    const RowBlocks rows = gather_rows(p.N);
    g.rows_per_block = rows.per_block;
    g.row_blocks = rows.blocks;
    g.pad_blocks = 16;
    g.h = p.h;
    g.ld_h = p.ld_h;
    g.vec_h = vector_rows(p.h, p.ld_h, p.dtype);
    g.h_out = at<bf16>(ws, L.h);
    g.h_plane = L.rows * L.ld;
    g.row_of = at<int32_t>(ws, L.row_of);
    g.count = at<int32_t>(ws, L.count);
    g.loss = loss;
    g.lse = lse;
    g.dh = dh;
    g.ld_dh = ld_dh;
    g.vec_dh = dh && vector_rows(dh, ld_dh, p.dtype);
    r->row_of = g.row_of;
    r->count = g.count;
    r->zh = r->h = Matrix{g.h_out, L.rows, p.d, L.ld, g.h_plane, L.planes};
  }
  if (L.pack_w) {
    g.w_blocks = w_gather_blocks(p.V);
    g.w = p.w;
    g.ld_w = p.ld_w;
    g.vec_w = vector_rows(p.w, p.ld_w, p.dtype);
    g.w_out = at<bf16>(ws, L.w);
    g.w_plane = (int64_t)p.V * L.ld;
    r->zw = r->w = Matrix{g.w_out, p.V, p.d, L.ld, g.w_plane, L.planes};
  }
  if (p.dtype == 0 && !L.few) {
    g.h16 = at<__half>(ws, L.h16);
    g.w16 = at<__half>(ws, L.w16);
    r->h_inv = g.h_inv = at<float>(ws, L.h_inv);
    r->w_inv = g.w_inv = at<float>(ws, L.w_inv);
    r->zh = Matrix{reinterpret_cast<const bf16*>(g.h16), L.rows, p.d, L.ld, g.h_plane, 2};
    r->zw = Matrix{reinterpret_cast<const bf16*>(g.w16), p.V, p.d, L.ld, g.w_plane, 2};
    g.h_least = at<uint32_t>(ws, L.h_least);
    g.w_least = at<uint32_t>(ws, L.w_least);
    r->least = Least{g.h_least, g.w_least, g.row_blocks, g.w_blocks};
    r->zh2 = r->h;
    r->zw2 = r->w;
  }
  g.blocks = g.row_blocks + g.pad_blocks + g.w_blocks;
  const dim3 grid((unsigned)g.blocks);
  if (p.dtype) return launch_pdl(gather_kernel<bf16>, grid, dim3(256), 0, st, g);
  VOCAB_TRY(launch_pdl(gather_kernel<float>, grid, dim3(256), 0, st, g));
  if (L.planes) return cudaSuccess;
  // Forward: the bf16 planes are made only where the fp16 ones do not hold the
  // rows, in their place, by a launch that else ends at once (2 us).
  Gather g2 = g;
  g2.planes = 3;
  g2.h_out = at<bf16>(ws, L.h16);
  g2.w_out = at<bf16>(ws, L.w16);
  g2.h16 = g2.w16 = nullptr;
  r->zh2 = Matrix{g2.h_out, L.rows, p.d, L.ld, g.h_plane, 3};
  r->zw2 = Matrix{g2.w_out, p.V, p.d, L.ld, g.w_plane, 3};
  return launch_pdl(gather_again_kernel, dim3((unsigned)std::min(g.blocks, 3 * kSmCount)), dim3(256), 0, st, g2);
}
// The operands of the logits.
Operands logit_operands(const Prepared& r, const Matrix* G) {
  Operands o{r.zh, r.zw, G};
  if (r.least.n_w) {
    o.A2 = &r.zh2;
    o.B2 = &r.zw2;
  }
  return o;
}

// k-blocks per tensor-memory sum of the logits.  bf16: 16, an error of some
// 1e-6 of a logit, far below its operands' rounding.  fp32: 4, and 1 where the
// tiles are no more than a round and the extra sums are not what they wait for
// (a logit of 15 off by 12 steps of 2^-21 moved a probability, and so a
// gradient, by 5e-6).  For longer work 1 would cost 10 %.
int logit_chunk(int dtype, int64_t M, int64_t N, int bn) {
  if (dtype) return 16;
  const int cg = cta_group((int)M);
  const int64_t tiles = (M + BM * cg - 1) / (BM * cg) * ((N + bn - 1) / bn);
  return tiles <= kSmCount / cg ? 1 : 4;
}

Args args_of(const VocabLoss& p, const Layout& L, const Prepared& r) {
  Args a{};
  a.terms = L.terms;
  a.chunk = 4;
  a.least = r.least;
  a.terms2 = 6;
  a.h_inv = r.h_inv;
  a.w_inv = r.w_inv;
  a.bn = BN;
  a.max_splits = 1;
  a.list = r.list;
  a.row_of = r.row_of;
  a.scale = p.inv_t;
  return a;
}

// Statistics into part and zsel, or (fg) g of the `rows` rows of w from fg->v0 on.
template <typename T, int NB>
cudaError_t few_rows(const VocabLoss& p, const RowList& list, float2* part, float* zsel,
                     const FewGrad* fg, int rows, cudaStream_t st) {
  const size_t smem = (size_t)NB * round_up(p.d, 8) * 4;
  const int vec = vector_rows(p.w, p.ld_w, p.dtype);
  const dim3 grid((unsigned)std::min<int64_t>(kSmCount, ((int64_t)rows + 15) / 16));
  const T *h = static_cast<const T*>(p.h), *w = static_cast<const T*>(p.w);
  if constexpr (sizeof(T) == 4) {
    if (fg) {
      VOCAB_TRY((set_smem<few_rows_kernel<T, NB, true>>((int)kFewSmem)));
      return launch_pdl(few_rows_kernel<T, NB, true>, grid, dim3(512), smem, st, h, p.ld_h, w + fg->v0 * p.ld_w, p.ld_w,
                        p.N, rows, p.d, vec, p.inv_t, list, 0, part, (int64_t)kFewRows, zsel, *fg);
    }
  }
  VOCAB_TRY((set_smem<few_rows_kernel<T, NB, false>>((int)kFewSmem)));
  return launch_pdl(few_rows_kernel<T, NB, false>, grid, dim3(512), smem, st, h, p.ld_h, w, p.ld_w, p.N, rows, p.d, vec,
                    p.inv_t, list, (int)(p.teacher != nullptr), part, (int64_t)kFewRows, zsel, FewGrad{});
}
cudaError_t few_rows_of(const VocabLoss& p, const RowList& list, float2* part, float* zsel,
                        const FewGrad* fg, int rows, cudaStream_t st) {
  if (p.dtype)
    return p.N == 1 ? few_rows<bf16, 1>(p, list, part, zsel, fg, rows, st)
                    : few_rows<bf16, 2>(p, list, part, zsel, fg, rows, st);
  if (p.N == 1) return few_rows<float, 1>(p, list, part, zsel, fg, rows, st);
  if (p.N == 2) return few_rows<float, 2>(p, list, part, zsel, fg, rows, st);
  if (p.N <= 4) return few_rows<float, 4>(p, list, part, zsel, fg, rows, st);
  return few_rows<float, 8>(p, list, part, zsel, fg, rows, st);
}

// A product of g into typed rows, K split where the rule says so.
template <int KIND>
cudaError_t product(const VocabLoss& p, const Operands& o, Args a, float4* slab, void* out, int64_t ld,
                    int accumulate, cudaStream_t st) {
  const int cg = cta_group(a.M);
  a.units = kSmCount / cg;
  a.bn = product_columns(a.M, a.N);
  a.slab = slab;
  a.out = out;
  a.ld_out = ld;
  a.out_bf16 = p.dtype;
  a.accumulate = accumulate;
  a.vec = vector_rows(out, ld, p.dtype);
  VOCAB_TRY(contract<KIND>(o, a, st));
  if (a.max_splits == 1) return cudaSuccess;
  const SlabSum s{slab,  a.M,    a.N,          a.K, a.m_count, a.k_count,  a.terms,  a.terms2, a.fine_rows,
                  a.units, a.max_splits, cg, a.bn, KIND == DW, a.row_of,  out, ld,       accumulate,
                  a.vec, a.acc,  a.acc_in,     a.acc_out};
  const int64_t tiles = (a.M + BM * cg - 1) / (BM * cg) * (int64_t)((a.N + a.bn - 1) / a.bn);
  const int64_t most = std::min<int64_t>(tiles, a.units) * std::min(a.M, BM * cg) * (BN / 8);
  const dim3 grid((unsigned)std::min<int64_t>(4 * kSmCount, (most + 255) / 256));
  return p.dtype ? launch_pdl(slab_sum_kernel<bf16>, grid, dim3(256), 0, st, s)
                 : launch_pdl(slab_sum_kernel<float>, grid, dim3(256), 0, st, s);
}

}  // namespace

size_t vocab_workspace_bytes(const VocabLoss& p, int backward) { return layout(p, backward).total; }

cudaError_t vocab_forward(const VocabLoss& p, float* loss, float* lse, void* ws, cudaStream_t st) {
  if (p.N == 0) return cudaSuccess;
  const Layout L = layout(p, 0);
  Prepared r;
  VOCAB_TRY(prepare(p, L, ws, nullptr, loss, lse, nullptr, 0, &r, st));
  float2* part = at<float2>(ws, L.part);
  float* zsel = at<float>(ws, L.zsel);
  if (L.few) {
    VOCAB_TRY(few_rows_of(p, r.list, part, zsel, nullptr, p.V, st));
  } else {
    Args a = args_of(p, L, r);
    a.M = p.N;
    a.m_count = r.count;
    a.N = p.V;
    a.K = p.d;
    a.bn = L.bn;
    a.chunk = logit_chunk(p.dtype, p.N, p.V, L.bn);
    // The list kernel before this one let it start after its own wait, so h
    // and w are complete: only the epilogue waits for the lists.
    a.early = p.teacher != nullptr && !L.gather && !L.pack_w;
    a.part = part;
    a.part_ld = L.rows;
    a.zsel = zsel;
    const Operands z = logit_operands(r, nullptr);
    VOCAB_TRY(p.dtype ? contract<STATS>(z, a, st) : contract<STATS32>(z, a, st));
  }
  return launch_pdl(join_kernel, dim3((unsigned)((p.N + 31) / 32)), dim3(1024), 0, st, (const float2*)part, L.parts,
                    L.few ? (int64_t)kFewRows : L.rows, p.N, r.row_of, r.count, p.V, r.list, r.slogq,
                    (const float*)zsel, loss, lse);
}

cudaError_t vocab_backward(const VocabLoss& p, const float* lse, const float* weight, void* dh, int64_t ld_dh,
                           void* dw, int64_t ld_dw, int accumulate_dw, void* ws, cudaStream_t st) {
  const size_t e = p.dtype ? 2 : 4;
  if (p.N == 0) {
    if (!dw || accumulate_dw) return cudaSuccess;
    return cudaMemset2DAsync(dw, ld_dw * e, 0, p.d * e, p.V, st);
  }
  const Layout L = layout(p, 1);
  Prepared r;
  VOCAB_TRY(prepare(p, L, ws, weight, nullptr, nullptr, dh, ld_dh, &r, st));
  float4 *dh_slab = at<float4>(ws, L.dh), *dw_slab = at<float4>(ws, L.dw);
  // g: three planes of fp32 operands; of bf16 ones a single plane, or two of kFineRows in its place
  const Matrix G{at<bf16>(ws, L.g), L.rows, L.piece, L.piece, L.rows * L.piece, p.dtype ? 1 : 3};
  const Matrix G2{G.p, kFineRows, L.piece, L.piece, (int64_t)kFineRows * L.piece, 2};
  const Matrix* fine = p.dtype ? &G2 : nullptr;
  for (int i = 0; i < L.pieces; ++i) {
    const int v0 = i * L.piece, width = std::min(p.V - v0, L.piece);
    Args a = args_of(p, L, r);
    a.M = p.N;
    a.m_count = r.count;
    a.N = width;
    a.K = p.d;
    a.b_row = v0;
    a.lse = lse;
    a.weight = weight;
    a.bn = L.bn;
    a.chunk = logit_chunk(p.dtype, p.N, width, L.bn);
    a.fine_rows = fine ? kFineRows : 0;
    const bool last = i + 1 == L.pieces, residuals = dh && L.residuals;
    a.resid = residuals ? at<float>(ws, L.resid) : nullptr;
    Operands z = logit_operands(r, &G);
    if (fine) z.A2 = fine;
    if (L.few) {
      const FewGrad fg{const_cast<bf16*>(G.p), G.plane, G.ld, r.row_of, r.count, lse, weight, v0};
      VOCAB_TRY(few_rows_of(p, r.list, nullptr, nullptr, &fg, width, st));
    } else {
      VOCAB_TRY(p.dtype ? contract<GRAD>(z, a, st) : contract<GRAD3>(z, a, st));
    }
    Args b = args_of(p, L, r);
    b.terms = fine ? 1 : 6;
    b.terms2 = 2;
    b.fine_rows = a.fine_rows;
    // k-blocks per tensor-memory sum.  bf16 gradients: a sum's drift over 4096
    // of k (8e-6) is far below their own rounding.  Few fp32 rows: a single
    // entry of g is most of a sum, and what comes after it drifts by 8 of its
    // last places over 256 of k; there the extra sums hide behind w.
    b.chunk = p.dtype ? 64 : L.few ? 1 : 4;
    if (dh) {
      Args c = b;
      c.M = p.N;
      c.m_count = r.count;
      c.N = p.d;
      c.K = width;
      c.b_k = v0;
      c.max_splits = L.dh_splits;
      c.acc = L.pieces > 1 || residuals ? at<float>(ws, L.acc) : nullptr;
      c.acc_in = i > 0 || (residuals && last);
      c.acc_out = !last;
      if (residuals && last)
        VOCAB_TRY(launch_pdl(residual_kernel, dim3((unsigned)((p.N + 7) / 8)), dim3(256), 0, st, r.list,
                             (const float*)a.resid, r.row_of, r.count, kFineRows, p.V, r.w.p, r.w.ld, p.d, c.acc,
                             (int)(i > 0)));
      VOCAB_TRY(product<DH>(p, Operands{G, r.w, nullptr, fine}, c, dh_slab, dh, ld_dh, 0, st));
    }
    if (dw) {
      b.row_of = nullptr;
      b.M = width;
      b.N = p.d;
      b.K = p.N;
      b.k_count = r.count;
      b.max_splits = L.dw_splits;
      VOCAB_TRY(product<DW>(p, Operands{G, r.h, nullptr, fine}, b, dw_slab, static_cast<uint8_t*>(dw) + (int64_t)v0 * ld_dw * e, ld_dw,
                            accumulate_dw, st));
    }
  }
  return cudaSuccess;
}

}  // namespace rlt

// vocab.cu -- softmax cross entropy and distillation over a large vocabulary
// without kept logits (launchers in vocab.h).
//
// z[n][v] = inv_t * sum_k h[n][k] w[v][k].  Forward: every vocabulary tile
// leaves (max, sum of exponentials) per row, joined in tile order into
// lse[n].  Backward, one piece of the vocabulary at a time: g[n][v] = c[n]
// (exp(z - lse[n]) - q[n][v]) into a buffer of the piece's width, then
// dh += g w and dw = g^T h.  The piece bounds the buffer; the logits are
// recomputed, never kept.
#include <math.h>

#include <algorithm>

#include "vocab.h"

namespace rlt {
namespace {

constexpr int kTile = 64;
constexpr int kNoId = 0x7fffffff;
constexpr int kMaxK = 256;

__host__ __device__ inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// ------------------------------------------------------------------ teacher lists
// One warp per row: q = softmax(teacher * inv_t) over the valid slots, the
// slots sorted by id (and slot, so the order never depends on timing); empty
// slots go last.  some[n] = 0 when no slot carries weight.
__global__ void __launch_bounds__(128) teacher_prep_kernel(const int32_t* ids, const float* teacher, int N, int K,
                                                           int V, float inv_t, int32_t* sid, float* sq, float* slogq,
                                                           float* some) {
  griddep_enter();
  __shared__ unsigned long long keys[4][kMaxK];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t n = (int64_t)blockIdx.x * 4 + warp;
  if (n >= N) return;
  int P = 32;
  while (P < K) P <<= 1;
  float m = -INFINITY;
  bool nan = false;
  for (int k = lane; k < P; k += 32) {
    const int32_t id = k < K ? ids[n * K + k] : -1;
    const bool ok = id >= 0 && id < V;
    if (ok) {
      const float t = teacher[n * K + k] * inv_t;
      nan |= isnan(t);
      m = fmaxf(m, t);
    }
    keys[warp][k] = ((unsigned long long)(ok ? id : kNoId) << 32) | (unsigned)k;
  }
  m = warp_max(m);
  const bool any_nan = __any_sync(0xffffffffu, nan);
  const bool has = m > -INFINITY || any_nan;
  __syncwarp();
  for (int size = 2; size <= P; size <<= 1)
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      for (int i = lane; i < P; i += 32) {
        const int j = i ^ stride;
        if (j > i) {
          const unsigned long long a = keys[warp][i], b = keys[warp][j];
          const bool up = (i & size) == 0;
          if ((a > b) == up) {
            keys[warp][i] = b;
            keys[warp][j] = a;
          }
        }
      }
      __syncwarp();
    }
  float sum = 0.f;
  for (int k = lane; k < K; k += 32) {
    const unsigned long long key = keys[warp][k];
    if ((int)(key >> 32) != kNoId) sum += expf(teacher[n * K + (unsigned)key] * inv_t - m);
  }
  sum = warp_sum(sum);
  const float logsum = logf(sum);
  for (int k = lane; k < K; k += 32) {
    const unsigned long long key = keys[warp][k];
    const int id = (int)(key >> 32);
    const bool on = has && id != kNoId;
    const float t = on ? teacher[n * K + (unsigned)key] * inv_t - m : 0.f;
    sid[n * K + k] = on ? id : kNoId;
    sq[n * K + k] = on ? expf(t) / sum : 0.f;
    slogq[n * K + k] = on ? t - logsum : 0.f;
  }
  if (lane == 0) some[n] = has ? 1.f : 0.f;
}

// A row's list as the tile kernels see it.
struct RowList {
  const int32_t* ids;  // ascending when K > 1
  const float* q;      // null: 1
  const float* some;   // null: the row takes part if its one id is in [0, V)
  int K;
};
__device__ __forceinline__ bool takes_part(const RowList& r, int64_t n, int V) {
  if (r.some) return r.some[n] != 0.f;
  const int32_t id = r.ids[n];
  return id >= 0 && id < V;
}

// ------------------------------------------------------------------ contractions
// C[m][n] = sum_k A(m, k) B(n, k) in fp32 over 64 x 64 tiles.
struct Operand {
  const void* p;
  int64_t s_row, s_k;  // strides in elements
  int bf;
  __device__ __forceinline__ float at(int64_t row, int64_t k) const {
    const int64_t o = row * s_row + k * s_k;
    return bf ? __bfloat162float(static_cast<const bf16*>(p)[o]) : static_cast<const float*>(p)[o];
  }
};

__device__ __forceinline__ void tile_product(const Operand& A, const Operand& B, int64_t m0, int64_t n0, int64_t M,
                                             int64_t N, int64_t K, const float* k_mask, float (*acc)[4],
                                             float (*as)[kTile + 1], float (*bs)[kTile + 1]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int64_t k0 = 0; k0 < K; k0 += 16) {
    for (int i = threadIdx.x; i < 16 * kTile; i += 256) {
      const int kk = i & 15, r = i >> 4;
      const bool on = k0 + kk < K && (k_mask == nullptr || k_mask[k0 + kk] != 0.f);
      as[kk][r] = on && m0 + r < M ? A.at(m0 + r, k0 + kk) : 0.f;
      bs[kk][r] = on && n0 + r < N ? B.at(n0 + r, k0 + kk) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[kk][ty * 4 + i], bs[kk][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
}

// Logit tile of rows m0.. and vocabulary n0..: statistics (g null) or the
// piece's gradient g[n][v - v_base].
__global__ void __launch_bounds__(256) logits_kernel(Operand h, Operand w, int N, int V, int d, float inv_t,
                                                     RowList list, int v_base, int v_end, float2* part, float* zsel,
                                                     const float* lse, const float* c, float* g, int64_t ld_g) {
  griddep_enter();
  __shared__ float as[16][kTile + 1], bs[16][kTile + 1];
  __shared__ float tile[kTile][kTile + 1];
  const int64_t m0 = (int64_t)blockIdx.y * kTile, n0 = v_base + (int64_t)blockIdx.x * kTile;
  float acc[4][4] = {};
  tile_product(h, w, m0, n0, N, V, d, nullptr, acc, as, bs);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) tile[ty * 4 + i][tx * 4 + j] = acc[i][j] * inv_t;
  __syncthreads();
  const int64_t n = m0 + threadIdx.x;
  if (threadIdx.x >= kTile || n >= N) return;
  float* z = tile[threadIdx.x];
  const int cols = (int)min((int64_t)kTile, v_end - n0);
  if (g == nullptr) {
    float m = -INFINITY, s = 0.f;
    for (int j = 0; j < cols; ++j) m = fmaxf(m, z[j]);
    const float mm = m > -INFINITY ? m : 0.f;
    for (int j = 0; j < cols; ++j) s += expf(z[j] - mm);
    part[(int64_t)blockIdx.x * N + n] = make_float2(m, s);
    for (int k = 0; k < list.K; ++k) {
      const int64_t j = list.ids[n * list.K + k] - n0;
      if (j >= 0 && j < cols) zsel[n * list.K + k] = z[j];
    }
  } else {
    const float cn = c[n], l = lse[n];
    if (cn == 0.f) {
      for (int j = 0; j < cols; ++j) z[j] = 0.f;
    } else {
      for (int j = 0; j < cols; ++j) z[j] = cn * expf(z[j] - l);
      for (int k = 0; k < list.K; ++k) {
        const int64_t j = list.ids[n * list.K + k] - n0;
        if (j >= 0 && j < cols) z[j] -= cn * (list.q ? list.q[n * list.K + k] : 1.f);
      }
    }
    for (int j = 0; j < cols; ++j) g[n * ld_g + (n0 - v_base) + j] = z[j];
  }
}

// out[m][n] (+)= A B in the output's type, optionally through an fp32
// accumulator over the pieces (acc_in: add it; acc_out: leave it there).
__global__ void __launch_bounds__(256) product_kernel(Operand A, Operand B, int64_t M, int64_t N, int64_t K,
                                                      const float* k_mask, void* out, int64_t ld_out, int out_bf,
                                                      int accumulate, const float* acc_in, float* acc_out) {
  griddep_enter();
  __shared__ float as[16][kTile + 1], bs[16][kTile + 1];
  const int64_t m0 = (int64_t)blockIdx.y * kTile, n0 = (int64_t)blockIdx.x * kTile;
  float acc[4][4] = {};
  tile_product(A, B, m0, n0, M, N, K, k_mask, acc, as, bs);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= M || n >= N) continue;
      float x = acc[i][j];
      if (acc_in) x += acc_in[m * N + n];
      if (acc_out) {
        acc_out[m * N + n] = x;
        continue;
      }
      const int64_t o = m * ld_out + n;
      if (out_bf) {
        bf16* p = static_cast<bf16*>(out) + o;
        *p = __float2bfloat16_rn(accumulate ? x + __bfloat162float(*p) : x);
      } else {
        float* p = static_cast<float*>(out) + o;
        *p = accumulate ? x + *p : x;
      }
    }
}

// ------------------------------------------------------------------ rows
// Joins the tiles' statistics in tile order; loss of every row.
__global__ void __launch_bounds__(128) join_kernel(const float2* part, int tiles, int N, int V, RowList list,
                                                   const float* slogq, const float* zsel, float* loss, float* lse) {
  griddep_enter();
  const int64_t n = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (n >= N) return;
  if (!takes_part(list, n, V)) {
    loss[n] = 0.f;
    lse[n] = 0.f;
    return;
  }
  float m = -INFINITY;
  for (int t = 0; t < tiles; ++t) m = fmaxf(m, part[(int64_t)t * N + n].x);
  float s = 0.f;
  for (int t = 0; t < tiles; ++t) {
    const float2 p = part[(int64_t)t * N + n];
    s += p.x > -INFINITY ? p.y * expf(p.x - m) : (isnan(p.y) ? p.y : 0.f);
  }
  const float l = m + logf(s);
  lse[n] = l;
  if (list.q == nullptr) {
    loss[n] = zsel[n] - l;
    return;
  }
  float kl = 0.f;
  for (int k = 0; k < list.K; ++k) {
    const int64_t i = n * list.K + k;
    if (list.ids[i] != kNoId && list.q[i] != 0.f) kl += list.q[i] * (slogq[i] - zsel[i] + l);
  }
  loss[n] = kl;
}

// c[n] = weight * inv_t where the row takes part, exactly 0 elsewhere.
__global__ void coef_kernel(const float* weight, int N, int V, float inv_t, RowList list, float* c) {
  griddep_enter();
  const int64_t n = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (n < N) c[n] = takes_part(list, n, V) ? weight[n] * inv_t : 0.f;
}

// ------------------------------------------------------------------ layout
struct Layout {
  size_t sid = 0, sq = 0, slogq = 0, some = 0, part = 0, zsel = 0, c = 0, g = 0, dh = 0, total = 0;
  int tiles = 0, piece = 0, pieces = 0;
};
Layout layout(const VocabLoss& p, int backward) {
  Layout L;
  auto take = [&](size_t n) {
    const size_t at = L.total;
    L.total += align256(n);
    return at;
  };
  const size_t rows = (size_t)p.N;
  if (p.teacher) {
    L.sid = take(rows * p.K * 4);
    L.sq = take(rows * p.K * 4);
    L.slogq = take(rows * p.K * 4);
    L.some = take(rows * 4);
  }
  L.tiles = (p.V + kTile - 1) / kTile;
  if (!backward) {
    L.part = take(rows * L.tiles * 8);
    L.zsel = take(rows * p.K * 4);
    return L;
  }
  const size_t budget = (size_t)256 << 20;
  size_t piece = budget / (std::max<size_t>(rows, 1) * 4) / kTile * kTile;
  piece = std::max<size_t>(piece, 2048);
  L.piece = (int)std::min<size_t>(piece, (size_t)L.tiles * kTile);
  L.pieces = (p.V + L.piece - 1) / L.piece;
  L.c = take(rows * 4);
  L.g = take(rows * L.piece * 4);
  if (L.pieces > 1) L.dh = take(rows * p.d * 4);
  return L;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

#define VOCAB_TRY(...)                    \
  do {                                    \
    cudaError_t e_ = (__VA_ARGS__);       \
    if (e_ != cudaSuccess) return e_;     \
  } while (0)

// The rows' lists, prepared in the workspace where there is a teacher.
cudaError_t row_lists(const VocabLoss& p, const Layout& L, void* ws, RowList* r, cudaStream_t st) {
  *r = RowList{p.ids, nullptr, nullptr, p.K};
  if (!p.teacher) return cudaSuccess;
  int32_t* sid = at<int32_t>(ws, L.sid);
  float *sq = at<float>(ws, L.sq), *slogq = at<float>(ws, L.slogq), *some = at<float>(ws, L.some);
  VOCAB_TRY(launch_pdl(teacher_prep_kernel, dim3((unsigned)((p.N + 3) / 4)), dim3(128), 0, st, p.ids, p.teacher, p.N,
                       p.K, p.V, p.inv_t, sid, sq, slogq, some));
  *r = RowList{sid, sq, some, p.K};
  return cudaSuccess;
}

}  // namespace

size_t vocab_workspace_bytes(const VocabLoss& p, int backward) { return layout(p, backward).total; }

cudaError_t vocab_forward(const VocabLoss& p, float* loss, float* lse, void* ws, cudaStream_t st) {
  if (p.N == 0) return cudaSuccess;
  const Layout L = layout(p, 0);
  RowList list;
  VOCAB_TRY(row_lists(p, L, ws, &list, st));
  const Operand h{p.h, p.ld_h, 1, p.dtype}, w{p.w, p.ld_w, 1, p.dtype};
  float2* part = at<float2>(ws, L.part);
  float* zsel = at<float>(ws, L.zsel);
  VOCAB_TRY(launch_pdl(logits_kernel, dim3((unsigned)L.tiles, (unsigned)((p.N + kTile - 1) / kTile)), dim3(256), 0, st,
                       h, w, p.N, p.V, p.d, p.inv_t, list, 0, p.V, part, zsel, (const float*)nullptr,
                       (const float*)nullptr, (float*)nullptr, (int64_t)0));
  return launch_pdl(join_kernel, dim3((unsigned)((p.N + 127) / 128)), dim3(128), 0, st, part, L.tiles, p.N, p.V, list,
                    p.teacher ? at<float>(ws, L.slogq) : nullptr, zsel, loss, lse);
}

cudaError_t vocab_backward(const VocabLoss& p, const float* lse, const float* weight, void* dh, int64_t ld_dh,
                           void* dw, int64_t ld_dw, int accumulate_dw, void* ws, cudaStream_t st) {
  if (p.N == 0) {
    if (!dw || accumulate_dw) return cudaSuccess;
    const size_t e = p.dtype ? 2 : 4;
    return cudaMemset2DAsync(dw, ld_dw * e, 0, p.d * e, p.V, st);
  }
  const Layout L = layout(p, 1);
  RowList list;
  VOCAB_TRY(row_lists(p, L, ws, &list, st));
  float *c = at<float>(ws, L.c), *g = at<float>(ws, L.g);
  float* acc = L.pieces > 1 ? at<float>(ws, L.dh) : nullptr;
  VOCAB_TRY(launch_pdl(coef_kernel, dim3((unsigned)((p.N + 255) / 256)), dim3(256), 0, st, weight, p.N, p.V, p.inv_t,
                       list, c));
  const size_t e = p.dtype ? 2 : 4;
  const unsigned rt = (unsigned)((p.N + kTile - 1) / kTile), dt = (unsigned)((p.d + kTile - 1) / kTile);
  for (int i = 0; i < L.pieces; ++i) {
    const int v0 = i * L.piece, v1 = std::min(p.V, v0 + L.piece);
    const int64_t width = v1 - v0;
    const unsigned vt = (unsigned)((width + kTile - 1) / kTile);
    const void* w0 = static_cast<const uint8_t*>(p.w) + (int64_t)v0 * p.ld_w * e;
    VOCAB_TRY(launch_pdl(logits_kernel, dim3(vt, rt), dim3(256), 0, st, Operand{p.h, p.ld_h, 1, p.dtype},
                         Operand{p.w, p.ld_w, 1, p.dtype}, p.N, p.V, p.d, p.inv_t, list, v0, v1, (float2*)nullptr,
                         (float*)nullptr, lse, (const float*)c, g, (int64_t)L.piece));
    if (dh)
      VOCAB_TRY(launch_pdl(product_kernel, dim3(dt, rt), dim3(256), 0, st, Operand{g, L.piece, 1, 0},
                           Operand{w0, 1, p.ld_w, p.dtype}, (int64_t)p.N, (int64_t)p.d, width, (const float*)nullptr,
                           dh, ld_dh, p.dtype, 0, i > 0 ? (const float*)acc : (const float*)nullptr,
                           i + 1 < L.pieces ? acc : (float*)nullptr));
    if (dw)
      VOCAB_TRY(launch_pdl(product_kernel, dim3(dt, vt), dim3(256), 0, st, Operand{g, 1, L.piece, 0},
                           Operand{p.h, 1, p.ld_h, p.dtype}, width, (int64_t)p.d, (int64_t)p.N, (const float*)c,
                           (void*)(static_cast<uint8_t*>(dw) + (int64_t)v0 * ld_dw * e), ld_dw, p.dtype,
                           accumulate_dw, (const float*)nullptr, (float*)nullptr));
  }
  return cudaSuccess;
}

}  // namespace rlt

// vocab.cu -- softmax cross entropy and distillation over a large vocabulary
// without kept logits (launchers in vocab.h, contraction in vocab_gemm.cuh).
//
// z[n][v] = inv_t * sum_k h[n][k] w[v][k].  Forward: every tile of the logits
// leaves (maximum, sum of exponentials) per row and 128 columns, joined in
// column order into lse[n].  Backward, one piece of the vocabulary at a time:
// g[n][v] = c[n] (exp(z - lse[n]) - q[n][v]) as bf16 into a buffer of the
// piece's width, then dh += g w and dw = g^T h.  The piece bounds the buffer;
// the logits are recomputed, never kept.
//
// Rows that take no part (no target, an empty list, weight 0 in the backward)
// are left out before the contractions: the rows that remain are gathered, in
// order, into one bf16 operand, and every extent follows their count on the
// device.
#include <math.h>

#include <algorithm>

#include "vocab.h"
#include "vocab_gemm.cuh"

namespace rlt {
namespace {

using namespace vocab_tc;

constexpr int kMaxK = 256;

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
inline int64_t round_up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

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

// ------------------------------------------------------------------ rows
// The rows that take part, in order: row_of[i] -> n, pos_of[n] -> i (or -1),
// and their count.  Forward (weight null) also writes the zeros of the others.
__global__ void __launch_bounds__(1024) rows_kernel(RowList list, const float* weight, int N, int V, int32_t* row_of,
                                                    int32_t* pos_of, int32_t* count, float* loss, float* lse) {
  griddep_enter();
  __shared__ int warp_sum_s[32];
  __shared__ int base_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) base_s = 0;
  __syncthreads();
  for (int64_t n0 = 0; n0 < N; n0 += 1024) {
    const int64_t n = n0 + threadIdx.x;
    const bool on = n < N && takes_part(list, n, V) && (weight == nullptr || weight[n] != 0.f);
    const unsigned b = __ballot_sync(0xffffffffu, on);
    if (lane == 0) warp_sum_s[warp] = __popc(b);
    __syncthreads();
    const int base = base_s;
    int mine = lane < 32 ? warp_sum_s[lane] : 0;
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0);
    const int total = __reduce_add_sync(0xffffffffu, mine);
    const int at = base + before + __popc(b & ((1u << lane) - 1));
    if (n < N) {
      pos_of[n] = on ? at : -1;
      if (on) row_of[at] = (int32_t)n;
      else if (loss) {
        loss[n] = 0.f;
        lse[n] = 0.f;
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) base_s = base + total;
    __syncthreads();
  }
  if (threadIdx.x == 0) *count = base_s;
}

// 8 elements from column c of a row (zeros past d).
template <typename T>
__device__ __forceinline__ void row8(const T* row, int c, int d, bool vec, float* v) {
  if (vec && c + 8 <= d) {
    load8(row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < d ? to_f32(row[c + j]) : 0.f;
  }
}
// The bf16 planes of 8 elements: x0 = bf16(x), x1 = bf16(x - x0), ...; their
// sum is x to 24 bits.
__device__ __forceinline__ void planes8(bf16* dst, int64_t plane, int planes, float* v) {
  for (int p = 0; p < planes; ++p) {
    store8(dst + p * plane, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] -= to_f32(from_f32<bf16>(v[j]));
  }
}

// One warp per row.  out row pos_of[n] (or n) = h row n as bf16 planes; rows
// that take no part get a zero dh row instead; the 128 warps behind the last
// row write zero rows up to the next multiple of 128.
template <typename T>
__global__ void __launch_bounds__(256) gather_kernel(const T* x, int64_t ld, int64_t rows, int d, int vec,
                                                     const int32_t* pos_of, const int32_t* count, bf16* out,
                                                     int64_t ld_out, int64_t plane, int planes, T* zero,
                                                     int64_t ld_zero) {
  griddep_enter();
  const int64_t n = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (n < rows) {
    const int64_t i = pos_of ? pos_of[n] : n;
    if (i < 0) {
      if (zero)
        for (int c = lane; c < d; c += 32) zero[n * ld_zero + c] = from_f32<T>(0.f);
      return;
    }
    for (int c = lane * 8; c < d; c += 256) {
      float v[8];
      row8(x + n * ld, c, d, vec, v);
      planes8(out + i * ld_out + c, plane, planes, v);
    }
  } else if (count && n < rows + 128) {
    const int64_t i = *count + (n - rows);
    if (i >= (*count + 127) / 128 * 128) return;
    for (int c = lane * 8; c < d; c += 256) {
      float v[8] = {};
      planes8(out + i * ld_out + c, plane, planes, v);
    }
  }
}

// Joins the statistics of a row's column groups; the row's loss.  A block has
// 32 rows (x) by 32 groups of column groups (y); the order is fixed.
__global__ void __launch_bounds__(1024) join_kernel(const float2* part, int parts, int64_t ld, int N,
                                                    const int32_t* row_of, const int32_t* count, int V, RowList list,
                                                    const float* slogq, const float* zsel, float* loss, float* lse) {
  griddep_enter();
  __shared__ float ms[32][33], ss[32][33];
  const int x = threadIdx.x, y = threadIdx.y;
  const int64_t i = (int64_t)blockIdx.x * 32 + x;
  const int rows = count ? *count : N;
  const bool in = i < rows;
  float m = -INFINITY, s = 0.f;
  if (in) {
    for (int t = y; t < parts; t += 32) {
      const float2 p = part[(int64_t)t * ld + i];
      const float mn = fmaxf(m, p.x);
      const float a = m > -INFINITY ? expf(m - mn) : (isnan(s) ? s : 0.f);
      const float b = p.x > -INFINITY ? expf(p.x - mn) : (isnan(p.y) ? p.y : 0.f);
      s = s * a + p.y * b;
      m = mn;
    }
  }
  ms[y][x] = m;
  ss[y][x] = s;
  __syncthreads();
  const int64_t n = in && row_of ? row_of[i] : i;
  const bool on = in && (row_of || takes_part(list, n, V));
  float M = -INFINITY, total = 0.f;
  for (int j = 0; j < 32; ++j) M = fmaxf(M, ms[j][x]);
  for (int j = 0; j < 32; ++j) {
    const float mj = ms[j][x], sj = ss[j][x];
    total += mj > -INFINITY ? sj * expf(mj - M) : (isnan(sj) ? sj : 0.f);
  }
  const float l = M + logf(total);
  if (list.q == nullptr) {
    if (y == 0 && in) {
      lse[n] = on ? l : 0.f;
      loss[n] = on ? zsel[n] - l : 0.f;
    }
    return;
  }
  float kl = 0.f;
  if (on)
    for (int k = y; k < list.K; k += 32) {
      const int64_t e = n * list.K + k;
      if (list.ids[e] != kNoId && list.q[e] != 0.f) kl += list.q[e] * (slogq[e] - zsel[e] + l);
    }
  __syncthreads();
  ss[y][x] = kl;
  __syncthreads();
  if (y == 0 && in) {
    float r = 0.f;
    for (int j = 0; j < 32; ++j) r += ss[j][x];
    lse[n] = on ? l : 0.f;
    loss[n] = on ? r : 0.f;
  }
}

// out rows = the slabs' sum in order (a long K split over the SMs).
template <typename T>
__global__ void __launch_bounds__(256) slab_sum_kernel(const float* slab, int splits, int64_t slab_rows, int rows,
                                                       const int32_t* count, int d, const int32_t* row_of, T* out,
                                                       int64_t ld, int accumulate) {
  griddep_enter();
  const int64_t i = blockIdx.y;
  if (i >= (count ? *count : rows)) return;
  const int64_t n = row_of ? row_of[i] : i;
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= d) return;
  float s = 0.f;
  for (int k = 0; k < splits; ++k) s += slab[((int64_t)k * slab_rows + i) * d + c];
  T* o = out + n * ld + c;
  *o = from_f32<T>(accumulate ? s + to_f32(*o) : s);
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

// A bf16 operand in memory: `planes` matrices [rows][cols], rows ld apart.
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

template <int KIND, int CG>
cudaError_t launch(const Matrix& A, const Matrix& B, const Matrix* G, const Args& a, cudaStream_t st) {
  using C = Cfg<CG>;
  constexpr bool A_MN = KIND == DW, B_MN = KIND == DH || KIND == DW;
  CUtensorMap ta, tb, tg;
  VOCAB_TRY(tensor_map(&ta, A, A_MN ? 64 : BM));
  VOCAB_TRY(tensor_map(&tb, B, B_MN ? 64 : a.bn / CG));
  if (G) VOCAB_TRY(tensor_map(&tg, *G, 32, 32));
  else tg = ta;
  VOCAB_TRY(cudaFuncSetAttribute(vocab_gemm_kernel<KIND, CG>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
  const int64_t tiles = round_up(a.M, BM * CG) / (BM * CG) * (round_up(a.N, a.bn) / a.bn) * a.splits;
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, vocab_gemm_kernel<KIND, CG>, ta, tb, tg, a);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Two CTAs per tile (256 rows; each loads half of the columns' operand)
// wherever there is more than one row tile.
template <int KIND>
cudaError_t contract(const Matrix& A, const Matrix& B, const Matrix* G, const Args& a, cudaStream_t st) {
  return a.M > BM ? launch<KIND, 2>(A, B, G, a, st) : launch<KIND, 1>(A, B, G, a, st);
}

// Where things lie in the workspace, and how the work is cut.
struct Layout {
  size_t sid = 0, sq = 0, slogq = 0, some = 0, row_of = 0, pos_of = 0, count = 0, h = 0, w = 0, part = 0, zsel = 0,
         g = 0, dh = 0, dw = 0, total = 0;
  int planes = 1, terms = 1;
  bool gather = true, pack_w = false;
  int64_t rows = 0;  // rows of the gathered operand, a multiple of 256
  int64_t ld = 0;    // row distance of gathered and packed operands
  int bn = BN, n_tiles = 0, piece = 0, pieces = 0, dh_splits = 1, dw_splits = 1;
  bool dh_slab = false;
};

bool tma_ready(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0; }

// Splits of a long K for a product with too few tiles to fill the SMs, at
// least eight k-blocks each.
int split_count(int64_t tiles, int64_t kblocks) {
  if (tiles * 2 > kSmCount) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>(kSmCount / tiles, kblocks / 8));
}

Layout layout(const VocabLoss& p, int backward) {
  Layout L;
  auto take = [&](size_t n) {
    const size_t at = L.total;
    L.total += align256(n);
    return at;
  };
  const bool f32 = p.dtype == 0;
  L.planes = f32 ? 3 : 1;
  L.terms = f32 ? 6 : 1;
  L.rows = round_up(std::max(p.N, 1), 256);
  L.ld = round_up(p.d, 8);
  // A forward pass over one row tile has nothing to gain from leaving rows
  // out, and its rows do not mix: it reads h where it is.
  L.gather = f32 || backward || p.N > BM || !tma_ready(p.h, p.ld_h);
  L.pack_w = f32 || !tma_ready(p.w, p.ld_w);
  L.n_tiles = (p.V + BN - 1) / BN;
  if (!backward && p.N <= BM) {
    // One row tile: the work is reading w once.  Columns per tile so that the
    // tiles fill whole rounds of the SMs evenly.
    const int rounds = (L.n_tiles + kSmCount - 1) / kSmCount;
    L.bn = std::max(32, (int)round_up((p.V + kSmCount * rounds - 1) / (kSmCount * rounds), 16));
    L.n_tiles = (p.V + L.bn - 1) / L.bn;
  }
  const size_t n = (size_t)p.N;
  if (p.teacher) {
    L.sid = take(n * p.K * 4);
    L.sq = take(n * p.K * 4);
    L.slogq = take(n * p.K * 4);
    L.some = take(n * 4);
  }
  if (L.gather) {
    L.row_of = take(n * 4);
    L.pos_of = take(n * 4);
    L.count = take(4);
    L.h = take((size_t)L.planes * L.rows * L.ld * 2);
  }
  if (L.pack_w) L.w = take((size_t)L.planes * p.V * L.ld * 2);
  if (!backward) {
    L.part = take((size_t)2 * L.n_tiles * L.rows * 8);
    L.zsel = take(n * p.K * 4);
    return L;
  }
  // The piece: as wide as 512 MB of g allow, at least 2048 columns; equal pieces.
  const int64_t most = std::max<int64_t>(2048, ((int64_t)512 << 20) / (L.rows * 2 * L.planes) / BN * BN);
  const int64_t whole = (int64_t)L.n_tiles * BN;
  L.pieces = (int)((whole + most - 1) / most);
  L.piece = (int)round_up((whole + L.pieces - 1) / L.pieces, BN);
  L.pieces = (int)((whole + L.piece - 1) / L.piece);
  L.g = take((size_t)L.planes * L.rows * L.piece * 2);
  const int64_t dt = (p.d + BN - 1) / BN;
  L.dh_splits = split_count(L.rows / BM * dt, (int64_t)L.piece / BK * L.terms);
  L.dh_slab = L.dh_splits > 1 || L.pieces > 1;
  if (L.dh_slab) L.dh = take((size_t)L.dh_splits * L.rows * p.d * 4);
  L.dw_splits = split_count(L.piece / BM * dt, (int64_t)L.rows / BK * L.terms);
  if (L.dw_splits > 1) L.dw = take((size_t)L.dw_splits * L.piece * p.d * 4);
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
  Matrix h, w;
};

template <typename T>
cudaError_t gather_rows(const void* x, int64_t ld, int64_t rows, int d, const int32_t* pos_of, const int32_t* count,
                        bf16* out, int64_t ld_out, int64_t plane, int planes, void* zero, int64_t ld_zero,
                        cudaStream_t st) {
  const int64_t warps = rows + (count ? 128 : 0);
  const int vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && ld % (16 / (int)sizeof(T)) == 0;
  return launch_pdl(gather_kernel<T>, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, st, static_cast<const T*>(x),
                    ld, rows, d, vec, pos_of, count, out, ld_out, plane, planes, static_cast<T*>(zero), ld_zero);
}

cudaError_t prepare(const VocabLoss& p, const Layout& L, void* ws, const float* weight, float* loss, float* lse,
                    void* dh, int64_t ld_dh, Prepared* r, cudaStream_t st) {
  r->list = RowList{p.ids, nullptr, nullptr, p.K};
  if (p.teacher) {
    int32_t* sid = at<int32_t>(ws, L.sid);
    float *sq = at<float>(ws, L.sq), *slogq = at<float>(ws, L.slogq), *some = at<float>(ws, L.some);
    VOCAB_TRY(launch_pdl(teacher_prep_kernel, dim3((unsigned)((p.N + 3) / 4)), dim3(128), 0, st, p.ids, p.teacher, p.N,
                         p.K, p.V, p.inv_t, sid, sq, slogq, some));
    r->list = RowList{sid, sq, some, p.K};
    r->slogq = slogq;
  }
  r->h = Matrix{static_cast<const bf16*>(p.h), p.N, p.d, p.ld_h, 0, 1};
  r->w = Matrix{static_cast<const bf16*>(p.w), p.V, p.d, p.ld_w, 0, 1};
  if (L.gather) {
    int32_t *row_of = at<int32_t>(ws, L.row_of), *pos_of = at<int32_t>(ws, L.pos_of), *count = at<int32_t>(ws, L.count);
    VOCAB_TRY(launch_pdl(rows_kernel, dim3(1), dim3(1024), 0, st, r->list, weight, p.N, p.V, row_of, pos_of, count,
                         loss, lse));
    const int64_t plane = L.rows * L.ld;
    bf16* h = at<bf16>(ws, L.h);
    VOCAB_TRY((p.dtype ? gather_rows<bf16> : gather_rows<float>)(p.h, p.ld_h, p.N, p.d, pos_of, count, h, L.ld, plane,
                                                                 L.planes, dh, ld_dh, st));
    r->row_of = row_of;
    r->count = count;
    r->h = Matrix{h, L.rows, p.d, L.ld, plane, L.planes};
  }
  if (L.pack_w) {
    const int64_t plane = (int64_t)p.V * L.ld;
    bf16* w = at<bf16>(ws, L.w);
    VOCAB_TRY((p.dtype ? gather_rows<bf16> : gather_rows<float>)(p.w, p.ld_w, p.V, p.d, nullptr, nullptr, w, L.ld,
                                                                 plane, L.planes, nullptr, 0, st));
    r->w = Matrix{w, p.V, p.d, L.ld, plane, L.planes};
  }
  return cudaSuccess;
}

Args args_of(const VocabLoss& p, const Layout& L, const Prepared& r) {
  Args a{};
  a.terms = L.terms;
  a.chunk = p.dtype ? 16 : 4;
  a.bn = BN;
  a.splits = 1;
  a.list = r.list;
  a.row_of = r.row_of;
  a.V = p.V;
  a.scale = p.inv_t;
  return a;
}

template <typename T>
cudaError_t slab_sum(const float* slab, int splits, int64_t slab_rows, int rows, const int32_t* count, int d,
                     const int32_t* row_of, void* out, int64_t ld, int accumulate, cudaStream_t st) {
  // grid.y is bounded by the slab's own rule: few tiles, so few rows
  return launch_pdl(slab_sum_kernel<T>, dim3((unsigned)((d + 255) / 256), (unsigned)rows), dim3(256), 0, st, slab,
                    splits, slab_rows, rows, count, d, row_of, static_cast<T*>(out), ld, accumulate);
}

void typed_output(Args* a, void* out, int64_t ld, int dtype, int accumulate) {
  a->out = out;
  a->ld_out = ld;
  a->out_bf16 = dtype;
  a->accumulate = accumulate;
  a->vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0 && ld % (dtype ? 8 : 4) == 0;
}

}  // namespace

size_t vocab_workspace_bytes(const VocabLoss& p, int backward) { return layout(p, backward).total; }

cudaError_t vocab_forward(const VocabLoss& p, float* loss, float* lse, void* ws, cudaStream_t st) {
  if (p.N == 0) return cudaSuccess;
  const Layout L = layout(p, 0);
  Prepared r;
  VOCAB_TRY(prepare(p, L, ws, nullptr, loss, lse, nullptr, 0, &r, st));
  Args a = args_of(p, L, r);
  a.M = p.N;
  a.m_count = r.count;
  a.N = p.V;
  a.K = p.d;
  a.part = at<float2>(ws, L.part);
  a.part_ld = L.rows;
  a.zsel = at<float>(ws, L.zsel);
  a.bn = L.bn;
  VOCAB_TRY(contract<STATS>(r.h, r.w, nullptr, a, st));
  return launch_pdl(join_kernel, dim3((unsigned)((p.N + 31) / 32)), dim3(32, 32), 0, st, (const float2*)a.part,
                    2 * L.n_tiles, L.rows, p.N, r.row_of, r.count, p.V, r.list, r.slogq, (const float*)a.zsel, loss,
                    lse);
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
  bf16* g = at<bf16>(ws, L.g);
  float* slab = L.dh_slab ? at<float>(ws, L.dh) : nullptr;
  const int64_t g_plane = L.rows * L.piece;
  for (int i = 0; i < L.pieces; ++i) {
    const int v0 = i * L.piece, width = std::min(p.V - v0, L.piece);
    const Matrix G{g, L.rows, L.piece, L.piece, g_plane, L.planes};
    Args a = args_of(p, L, r);
    a.M = p.N;
    a.m_count = r.count;
    a.N = width;
    a.K = p.d;
    a.b_row = v0;
    a.lse = lse;
    a.weight = weight;
    VOCAB_TRY(L.planes == 1 ? contract<GRAD>(r.h, r.w, &G, a, st) : contract<GRAD3>(r.h, r.w, &G, a, st));
    if (dh) {
      const bool last = i + 1 == L.pieces;
      Args b = args_of(p, L, r);
      // bf16 gradients: the sum's drift over 4096 of k (8e-6) is far below
      // their own rounding
      if (p.dtype) b.chunk = 64;
      b.M = p.N;
      b.m_count = r.count;
      b.N = p.d;
      b.K = width;
      b.b_k = v0;
      b.splits = L.dh_splits;
      b.acc_in = i > 0 ? slab : nullptr;
      b.slab_rows = L.rows;
      if (L.dh_splits > 1 || !last) b.slab = slab;
      else typed_output(&b, dh, ld_dh, p.dtype, 0);
      VOCAB_TRY(contract<DH>(G, r.w, nullptr, b, st));
      if (last && L.dh_splits > 1)
        VOCAB_TRY((p.dtype ? slab_sum<bf16> : slab_sum<float>)(slab, L.dh_splits, L.rows, p.N, r.count, p.d, r.row_of,
                                                               dh, ld_dh, 0, st));
    }
    if (dw) {
      void* out = static_cast<uint8_t*>(dw) + (int64_t)v0 * ld_dw * e;
      Args b = args_of(p, L, r);
      b.row_of = nullptr;
      if (p.dtype) b.chunk = 64;
      b.M = width;
      b.N = p.d;
      b.K = p.N;
      b.k_count = r.count;
      b.splits = L.dw_splits;
      b.slab_rows = L.piece;
      if (L.dw_splits > 1) b.slab = at<float>(ws, L.dw);
      else typed_output(&b, out, ld_dw, p.dtype, accumulate_dw);
      VOCAB_TRY(contract<DW>(G, r.h, nullptr, b, st));
      if (L.dw_splits > 1)
        VOCAB_TRY((p.dtype ? slab_sum<bf16> : slab_sum<float>)(b.slab, L.dw_splits, L.piece, width, nullptr, p.d,
                                                               nullptr, out, ld_dw, accumulate_dw, st));
    }
  }
  return cudaSuccess;
}

}  // namespace rlt

// vocab_gemm.cuh -- the tensor-core contraction of the vocabulary operators
// (sm_100a: tcgen05.mma with fp32 accumulators in tensor memory, operands by
// TMA), persistent, with the loss fused into its epilogue.
//
//   D[m][n] = sum over terms and k of A[plane a][m][k] B[plane b][n][k]
//
// Kinds:
//   STATS  D = h w^T: per row and 128 columns, the maximum and the sum of
//          exponentials of z = D * inv_t, and z at the row's listed ids
//   GRAD   D = h w^T: g = c (exp(z - lse) - q), rounded to bf16 (one plane),
//          or to three bf16 planes whose sum is g to 2^-24 (fp32 operands)
//   DH     D = g w     (A K-major, B MN-major): fp32 partials or typed rows
//   DW     D = g^T h   (A and B MN-major): fp32 partials or typed rows
//
// fp32 operands are held as three bf16 planes x = x0 + x1 + x2 (24 bits); six
// products, the smallest first, leave out terms below 2^-24 |x||y|.
//
// A CTA has twelve warps: one issues TMA, one MMA, one owns tensor memory,
// eight drain a 128 x 256 accumulator (warps 4-7 its first 128 columns, 8-11
// the others) while the next tile's MMAs fill the second of two.
#pragma once
#include <cuda.h>

#include "common.cuh"

namespace rlt {
namespace vocab_tc {

constexpr int BM = 128, BN = 256, BK = 64;
constexpr int kThreads = 384;
constexpr int kNoId = 0x7fffffff;

enum Kind { STATS, GRAD, DH, DW };

// A row's list of (id, probability) as the kernels see it.
struct RowList {
  const int32_t* ids;  // ascending when K > 1, empty slots (kNoId) last
  const float* q;      // null: 1
  const float* some;   // null: the row takes part if its one id is in [0, V)
  int K;
};
__device__ __forceinline__ bool takes_part(const RowList& r, int64_t n, int V) {
  if (r.some) return r.some[n] != 0.f;
  const int32_t id = r.ids[n];
  return id >= 0 && id < V;
}

struct Args {
  int M, N, K;            // extents; *m_count / *k_count replace M / K where set
  const int32_t* m_count;
  const int32_t* k_count;
  int terms;              // 1 or 6 plane products
  int splits;             // K ranges, one fp32 slab each (DH, DW)
  int a_row, a_k, b_row, b_k;  // coordinate offsets of the operands
  // STATS, GRAD
  RowList list;
  const int32_t* row_of;  // compact row -> row, or null
  int V;
  float scale;            // inv_t
  float2* part;           // [2 * n_tiles][part_ld]
  int64_t part_ld;
  float* zsel;            // [rows][K]
  const float* lse;
  const float* weight;
  bf16* g;                // [planes][.][ld_g]
  int64_t ld_g, g_plane;
  int planes;
  // DH, DW
  float* slab;            // fp32 [splits][slab_rows][N]; null: typed output
  int64_t slab_rows;
  const float* acc_in;    // added first (same layout as slab), or null
  void* out;
  int64_t ld_out;
  int out_bf16, accumulate, vec;
};

template <int CG>
struct Cfg {
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_ROWS = BN / CG;
  static constexpr int B_BYTES = B_ROWS * BK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = CG == 1 ? 4 : 6;
  static constexpr int BAR_OFF = STAGES * STAGE;
  static constexpr int SMEM = BAR_OFF + 256 + 1024;
};

// Shared-memory descriptor, 128-byte swizzle: 8-row groups 1024 bytes apart;
// `lbo` is the distance of 64-element blocks along M or N (MN-major only).
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

template <int CG>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int x, int y, int z) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
        "%5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// One operand tile of ROWS rows (or columns) and 64 of k: K-major as ROWS
// rows of 128 bytes, MN-major as ROWS / 64 boxes of 64 k-rows.
template <int CG, int ROWS, bool MN>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int row, int k, int plane) {
  if constexpr (MN) {
#pragma unroll
    for (int i = 0; i < ROWS / 64; ++i) load_box<CG>(dst + i * 8192, tm, bar, row + 64 * i, k, plane);
  } else {
    load_box<CG>(dst, tm, bar, k, row, plane);
  }
}

template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// Address in CTA 0 of the pair of a shared-memory location of this CTA's layout.
__device__ __forceinline__ uint32_t in_leader(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(0));
  return r;
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// v[i] for a per-thread i, and v[i] -= x, without leaving registers.
__device__ __forceinline__ float pick(const float* v, int i) {
  float r = v[0];
#pragma unroll
  for (int j = 1; j < 32; ++j) r = j == i ? v[j] : r;
  return r;
}
__device__ __forceinline__ void sub_at(float* v, int i, float x) {
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] -= j == i ? x : 0.f;
}

// First position of a row's ascending list whose id is at least `id`.
__device__ __forceinline__ int lower_bound(const int32_t* ids, int K, int id) {
  int lo = 0, hi = K;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ids[mid] < id) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

constexpr float kLog2e = 1.4426950408889634f;

struct Tile {
  int m, n, kb0, kb1, split;
};

template <int CG>
struct Plan {
  int m_tiles, n_tiles, kb, total_kb, per_split, tiles;
  __device__ __forceinline__ void init(const Args& a) {
    const int M = a.m_count ? *a.m_count : a.M, K = a.k_count ? *a.k_count : a.K;
    m_tiles = (M + BM * CG - 1) / (BM * CG);
    n_tiles = (a.N + BN - 1) / BN;
    kb = (K + BK - 1) / BK;
    total_kb = kb * a.terms;
    per_split = (total_kb + a.splits - 1) / a.splits;
    tiles = m_tiles * n_tiles * a.splits;
  }
  // Panels of 16 row tiles, columns of tiles inside: the tiles that run
  // together share their operands in L2.
  __device__ __forceinline__ Tile at(int t) const {
    constexpr int GM = 16 / CG;
    Tile r;
    const int mn = m_tiles * n_tiles;
    r.split = t / mn;
    t -= r.split * mn;
    const int p = t / (GM * n_tiles), first = p * GM;
    const int g = min(m_tiles - first, GM);
    const int i = t - first * n_tiles;
    r.n = i / g;
    r.m = first + (i - r.n * g);
    r.kb0 = min(total_kb, r.split * per_split);
    r.kb1 = min(total_kb, r.kb0 + per_split);
    return r;
  }
};

// ---------------------------------------------------------------- epilogues
// Each handles 128 columns from `col` (within the tile's N extent) of one row
// per thread; acc(c, v) reads 32 accumulator columns.
template <typename Acc>
__device__ __forceinline__ void stats_epilogue(const Args& a, int64_t i, int64_t n, bool on, int n_tile, int half,
                                               int v0, int pos, Acc acc) {
  const float s2 = a.scale * kLog2e;
  float m = -INFINITY, s = 0.f;
  const int cols = min(128, a.N - (n_tile * BN + half * 128));
  int next = on && pos < a.list.K ? a.list.ids[n * a.list.K + pos] : kNoId;
#pragma unroll 1
  for (int c = 0; c < 128; c += 32) {
    if (c >= cols) break;
    float v[32];
    acc(c, v);
    while (next >= v0 + c && next < v0 + c + 32) {
      a.zsel[n * a.list.K + pos] = pick(v, next - v0 - c) * a.scale;
      next = ++pos < a.list.K ? a.list.ids[n * a.list.K + pos] : kNoId;
    }
    float cm = -INFINITY;
    if (c + 32 <= cols) {
#pragma unroll
      for (int j = 0; j < 32; ++j) cm = fmaxf(cm, v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        if (c + j >= cols) v[j] = -INFINITY;
        cm = fmaxf(cm, v[j]);
      }
    }
    const float mn = fmaxf(m, cm);
    const float sub = mn > -INFINITY ? mn * s2 : 0.f;
    float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 32; ++j) t[j & 3] += ex2(fmaf(v[j], s2, -sub));
    s = s * (m > -INFINITY ? ex2(fmaf(m, s2, -sub)) : (isnan(s) ? s : 0.f)) + ((t[0] + t[1]) + (t[2] + t[3]));
    m = mn;
  }
  if (on) a.part[(int64_t)(n_tile * 2 + half) * a.part_ld + i] = make_float2(m * a.scale, s);
}

template <typename Acc>
__device__ __forceinline__ void grad_epilogue(const Args& a, int64_t i, int64_t n, bool on, int n_tile, int half,
                                              int v0, int pos, Acc acc) {
  const float s2 = a.scale * kLog2e;
  const int cols = min(128, a.N - (n_tile * BN + half * 128));
  const float cw = on ? a.weight[n] * a.scale : 0.f;
  const float sub = on ? a.lse[n] * kLog2e : 0.f;
  int next = on && pos < a.list.K ? a.list.ids[n * a.list.K + pos] : kNoId;
  bf16* grow = a.g + i * a.ld_g + n_tile * BN + half * 128;
#pragma unroll 1
  for (int c = 0; c < 128; c += 32) {
    float v[32];
    acc(c, v);
    if (on) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = cw * ex2(fmaf(v[j], s2, -sub));
      while (next >= v0 + c && next < v0 + c + 32) {
        sub_at(v, next - v0 - c, cw * (a.list.q ? a.list.q[n * a.list.K + pos] : 1.f));
        next = ++pos < a.list.K ? a.list.ids[n * a.list.K + pos] : kNoId;
      }
      if (c + 32 > cols) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = c + j < cols ? v[j] : 0.f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = 0.f;
    }
#pragma unroll 1
    for (int p = 0; p < a.planes; ++p) {
      uint4* dst = reinterpret_cast<uint4*>(grow + p * a.g_plane + c);
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        w[j] = pack2(v[2 * j], v[2 * j + 1]);
        v[2 * j] -= __uint_as_float(w[j] << 16);
        v[2 * j + 1] -= __uint_as_float(w[j] & 0xFFFF0000u);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) dst[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    }
  }
}

template <typename OT>
__device__ __forceinline__ void store_row32(OT* o, float* v, int left, bool vec, bool add) {
  if (vec && left >= 32) {
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
      if (add) {
        float old[8];
        load8(o + j, old);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j + e] += old[e];
      }
      store8(o + j, v + j);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < left) o[j] = from_f32<OT>(add ? v[j] + to_f32(o[j]) : v[j]);
  }
}

template <typename Acc>
__device__ __forceinline__ void product_epilogue(const Args& a, int64_t i, int64_t n, bool on, int n_tile, int half,
                                                 int split, Acc acc) {
  const int col0 = n_tile * BN + half * 128;
  const int64_t slab = ((int64_t)split * a.slab_rows + i) * a.N + col0;
#pragma unroll 1
  for (int c = 0; c < 128; c += 32) {
    const int left = a.N - col0 - c;
    if (left <= 0) break;
    float v[32];
    acc(c, v);
    if (!on) continue;
    if (a.acc_in) {
      const float* p = a.acc_in + slab + c;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < left) v[j] += p[j];
    }
    if (a.slab) {
      store_row32(a.slab + slab + c, v, left, (a.N & 3) == 0, false);
    } else if (a.out_bf16) {
      store_row32(static_cast<bf16*>(a.out) + n * a.ld_out + col0 + c, v, left, a.vec, a.accumulate);
    } else {
      store_row32(static_cast<float*>(a.out) + n * a.ld_out + col0 + c, v, left, a.vec, a.accumulate);
    }
  }
}

// ---------------------------------------------------------------- kernel
template <int KIND, int CG>
__global__ void __launch_bounds__(kThreads, 1)
    vocab_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const Args a) {
  using C = Cfg<CG>;
  constexpr bool A_MN = KIND == DW, B_MN = KIND == DH || KIND == DW;
  constexpr int S = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(smem);
  const uint32_t bars = base + C::BAR_OFF;
  const uint32_t full = bars, empty = bars + 8 * S, acc_full = bars + 16 * S, acc_empty = acc_full + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::BAR_OFF + 16 * S + 32);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0 : cta_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(acc_full + 8 * s, 1);
      mbar_init(acc_empty + 8 * s, 8 * CG);
    }
    *abort_flag = 0;
    fence_mbar_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmA)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmB)) : "memory");
  }
  if (warp == 2) {
    if constexpr (CG == 1) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
  }
  griddep_enter();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if constexpr (CG == 2) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  Plan<CG> plan;
  plan.init(a);
  const int first = blockIdx.x / CG, step = gridDim.x / CG;

  // Products of planes for fp32 operands, smallest first: (2,0) (0,2) (1,1) (1,0) (0,1) (0,0).
  if (warp == 0 && lane == 0) {
    uint32_t it = 0;
    bool ok = true;
    for (int t = first; t < plan.tiles && ok; t += step) {
      const Tile tile = plan.at(t);
      const int row_a = tile.m * BM * CG + rank * BM + a.a_row, row_b = tile.n * BN + rank * C::B_ROWS + a.b_row;
      for (int kb = tile.kb0; kb < tile.kb1; ++kb, ++it) {
        const int term = a.terms == 1 ? 5 : kb / plan.kb;
        const int k = (a.terms == 1 ? kb : kb - term * plan.kb) * BK;
        const int plane_a = term == 0 ? 2 : (term == 2 || term == 3) ? 1 : 0;
        const int plane_b = term == 1 ? 2 : (term == 2 || term == 4) ? 1 : 0;
        const int s = it % S;
        if (!mbar_wait(empty + 8 * s, ((it / S) & 1u) ^ 1u) || *abort_flag) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        const uint32_t sa = base + s * C::STAGE, sb = sa + C::A_BYTES;
        uint32_t bar = full + 8 * s;
        if (rank == 0) mbar_arrive_expect_tx(bar, C::STAGE * CG);
        if constexpr (CG == 2) bar = in_leader(bar);
        load_tile<CG, BM, A_MN>(sa, &tmA, bar, row_a, k + a.a_k, plane_a);
        load_tile<CG, C::B_ROWS, B_MN>(sb, &tmB, bar, row_b, k + a.b_k, plane_b);
      }
    }
    if (!ok && rank == 0) {  // copies still in flight land before the CTA leaves
      for (uint32_t i = it > S ? it - S : 0; i < it; ++i) mbar_wait(full + 8 * (i % S), (i / S) & 1u);
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)A_MN << 15) | ((uint32_t)B_MN << 16) |
                               ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(BM * CG >> 4) << 24);
    uint32_t it = 0, n_acc = 0;
    bool ok = true;
    for (int t = first; t < plan.tiles && ok; t += step) {
      const Tile tile = plan.at(t);
      if (tile.kb0 == tile.kb1) continue;
      const uint32_t as = n_acc & 1u;
      if (!mbar_wait(acc_empty + 8 * as, ((n_acc >> 1) & 1u) ^ 1u) || *abort_flag) {
        *abort_flag = 1;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t d = tmem + as * BN;
      for (int kb = tile.kb0; kb < tile.kb1; ++kb, ++it) {
        const int s = it % S;
        if (!mbar_wait(full + 8 * s, (it / S) & 1u) || *abort_flag) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t sa = base + s * C::STAGE, sb = sa + C::A_BYTES;
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
          const uint64_t da = A_MN ? sdesc(sa + kk * 2048, 8192) : sdesc(sa + kk * 32, 16);
          const uint64_t db = B_MN ? sdesc(sb + kk * 2048, 8192) : sdesc(sb + kk * 32, 16);
          mma<CG>(d, da, db, idesc, kb > tile.kb0 || kk > 0);
        }
        commit<CG>(empty + 8 * s);
      }
      if (ok) commit<CG>(acc_full + 8 * as);
      ++n_acc;
    }
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    uint32_t n_acc = 0;
    const int M = a.m_count ? *a.m_count : a.M;
    for (int t = first; t < plan.tiles; t += step) {
      const Tile tile = plan.at(t);
      const int64_t i = (int64_t)tile.m * BM * CG + rank * BM + q * 32 + lane;
      bool on = i < M;
      const int64_t n = on && a.row_of ? a.row_of[i] : i;
      const int v0 = tile.n * BN + half * 128 + a.b_row;
      int pos = 0;
      if constexpr (KIND == STATS || KIND == GRAD) {
        if (on && a.list.K > 1) pos = lower_bound(a.list.ids + n * a.list.K, a.list.K, v0);
      }
      const bool any = tile.kb0 < tile.kb1;
      const uint32_t as = n_acc & 1u;
      if (any) {
        if (!mbar_wait(acc_full + 8 * as, (n_acc >> 1) & 1u) || *abort_flag) {
          *abort_flag = 1;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      }
      const uint32_t d = tmem + as * BN + lanes + half * 128;
      auto acc = [&](int c, float* v) {
        __syncwarp();
        if (any) {
          ld32(d + c, v);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.f;
        }
      };
      if constexpr (KIND == STATS) stats_epilogue(a, i, n, on, tile.n, half, v0, pos, acc);
      else if constexpr (KIND == GRAD) grad_epilogue(a, i, n, on, tile.n, half, v0, pos, acc);
      else product_epilogue(a, i, n, on, tile.n, half, tile.split, acc);
      if (any) {
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 1) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(acc_empty + 8 * as) : "memory");
          else arrive_at(in_leader(acc_empty + 8 * as));
        }
        ++n_acc;
      }
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if constexpr (CG == 2) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 2) {
    if constexpr (CG == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    else
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

}  // namespace vocab_tc
}  // namespace rlt

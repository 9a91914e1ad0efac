// vocab_gemm.cuh -- the tensor-core contraction of the vocabulary operators
// (sm_100a: tcgen05.mma with fp32 accumulators in tensor memory, operands by
// TMA), persistent, with the loss fused into its epilogue.
//
//   D[m][n] = sum over terms and k of A[plane a][m][k] B[plane b][n][k]
//
// Kinds:
//   STATS  D = h w^T: per row and up to 128 columns, the maximum and the sum
//          of exponentials of z = D * inv_t, and z at the row's listed ids
//   STATS32  the same of fp32 operands, in one of two forms
//   GRAD   D = h w^T of bf16 operands: g = c (exp(z - lse) - q), rounded to
//          bf16, or as two planes whose sum is g to 2^-16 (Args::fine_rows)
//   GRAD3  the same of fp32 operands, as three planes, g to 2^-24
//   DH     D = g w     (A K-major, B MN-major): fp32 partials or typed rows
//   DW     D = g^T h   (A and B MN-major): fp32 partials or typed rows
//
// fp32 operands are held as 16-bit planes whose products add up, smallest
// products first.
//   Logits: two fp16 planes, x * 2^e = x0 + 2^-12 x1, with e per row so that
//   the row's largest element is in [2^13, 2^15).  Three products (the two of
//   x1 are added first, then scaled).  x0 holds x to r = max(2^-11, 2^-25 / x)
//   of itself, both to max(2^-23, 2^-37 / x); the left-out product of the x1 is
//   below r_h r_w |h||w|.  The powers of two are taken back in the epilogue.
//   Logits of rows whose elements differ by more than that holds (fp16_holds):
//   three bf16 planes x = x0 + x1 + x2, 24 bits of any element (down to 2^-110;
//   2^-134 is the least that is held), six products, what is left out below
//   2^-24 |h||w|.  The conversion finds the smallest elements, the contraction
//   chooses.
//   Products of g: three bf16 planes, as above.
//
// A CTA has twelve warps: two issue TMA, one MMA, one owns tensor memory,
// eight drain a 128 x 256 accumulator (warps 4-7 its first 128 columns, 8-11
// the others) while the MMAs fill the second of two.
//
// The tensor cores add to an accumulator towards zero, an error of half a
// unit in the last place per 16 of k on average, all one way: over k = 2048
// logits came out 1e-6 short of themselves, over k = 32000 gradients 2e-5.
// So a sum stays in tensor memory for `chunk` k-blocks only; the epilogue
// warps add the chunks in registers, rounding to nearest, under the next
// chunk's MMAs.
//
// Bound by the tensor cores where there are rows enough: at 8,192 rows, V =
// 32000, d = 2048, the tensor pipe is active 95 % of the time in all four
// kinds and the power limit sets the clock (1.35 to 1.42 GHz): 651 us for
// STATS, 1.65 PFLOP/s, and 1.56 to 1.58 in the others.  Two CTAs per tile
// (256 x 256, each loads half of the columns' operand) took 8 % off a forward
// and backward of 16,368 rows against one (128 x 256).
#pragma once
#include <cuda.h>

#include "common.cuh"

namespace rlt {
namespace vocab_tc {

constexpr int BM = 128, BN = 256, BK = 64;
constexpr int kThreads = 384;
constexpr int kNoId = 0x7fffffff;

enum Kind { STATS, STATS32, GRAD, GRAD3, DH, DW };

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

// The smallest nonzero elements of scaled fp32 rows, per block of the
// conversion, as the bits of |x| less one (so that 0 is the largest).
struct Least {
  const uint32_t *h, *w;
  int n_h, n_w;
};
// This thread's share of them, four words to a load and all loads of a few
// thousand words in flight.
__device__ __forceinline__ uint32_t least_of(const uint32_t* p, int n, int threads) {
  uint32_t r = 0xffffffffu;
  const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll 4
  for (int i = threadIdx.x; i < n / 4; i += threads) {
    const uint4 v = q[i];
    r = min(r, min(min(v.x, v.y), min(v.z, v.w)));
  }
  if ((int)threadIdx.x < n % 4) r = min(r, p[n / 4 * 4 + threadIdx.x]);
  return r;
}
// Do two fp16 planes hold every product of such rows to d / 2 roundings of
// fp32, as many as a sum of d products has in any case?  With m the smallest
// element, or 2^-14 where that is more: m_h m_w >= 2^-25 / d bounds the left-out
// product by 2^-50 / (m_h m_w) <= (d / 2) 2^-24, and each operand's own error by
// 2^-37 / m <= (d / 4) 2^-24.  Rows of random numbers have it so (32,000 and
// 16,384 normal rows of 2,048: all but about 1 call in 100), rows with outliers
// 2^20 and more above the rest do not.
__device__ __forceinline__ bool fp16_holds(uint32_t h, uint32_t w, int d) {
  const float mh = h == 0xffffffffu ? 0x1p-14f : fminf(__uint_as_float(h + 1), 0x1p-14f);
  const float mw = w == 0xffffffffu ? 0x1p-14f : fminf(__uint_as_float(w + 1), 0x1p-14f);
  return mh * mw * (float)d >= 0x1p-25f;
}

struct Args {
  int M, N, K;            // extents; *m_count / *k_count replace M / K where set
  const int32_t* m_count;
  const int32_t* k_count;
  int terms;              // 1, 2, 3 or 6 plane products
  // A second form of an operand, in terms2 products, that the device chooses:
  int terms2;
  Least least;            // STATS32, GRAD3: three bf16 planes for two fp16 ones
  int fine_rows;          // GRAD, DH, DW: g is two planes, not one, where at most so many rows take part
  int chunk;              // k-blocks per tensor-memory sum (of the leading term)
  int bn;                 // columns per tile: a multiple of 64 (DH, DW: 64 per CTA) up to BN
  int stages;             // of bn's size
  int a_rows;             // rows of A that a tile loads (fewer than BM when M is: the rest are never looked at)
  int units;              // CTAs or pairs on the device
  int max_splits;         // K ranges of the last round's tiles at most (DH, DW); see split_rule
  int b_row, b_k;         // coordinate offsets of B: a piece of the vocabulary
  // STATS, GRAD
  int early;              // operands are older than the kernel before this one: loads do not wait for it
  RowList list;
  const float *h_inv, *w_inv;  // fp16 planes: 2^(-e / 2) of the rows of h and w
  const int32_t* row_of;  // compact row -> row, or null
  float scale;            // inv_t
  float2* part;           // [2 * n_tiles][part_ld]
  int64_t part_ld;
  float* zsel;            // [rows][K]
  const float* lse;
  const float* weight;
  float* resid;           // [rows][K], GRAD of one plane: what rounding took from g at the row's listed ids, or null
  // DH, DW
  float4* slab;           // [splits][last round's tiles][BN / 4][rows of a tile]: a warp's rows side by side
  float* acc;             // fp32 [rows][N]: the sum over pieces of K and what rounding took, or null
  int acc_in, acc_out;    // add what acc holds; leave the sum there
  void* out;
  int64_t ld_out;
  int out_bf16, accumulate, vec;
};

template <int CG>
struct Cfg {
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int PIPE = 196608;               // 4 or 6 stages of the largest tile, up to 12 of smaller ones
  static constexpr int MOST_STAGES = 12;
  static constexpr int OUT_OFF = PIPE;              // 8 warps x two 32 x 32 bf16 boxes
  static constexpr int BAR_OFF = OUT_OFF + 8 * 4096;
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

// One operand tile of `rows` rows (or columns) and 64 of k: K-major as rows of
// 128 bytes, MN-major as rows / 64 boxes of 64 k-rows.
template <int CG, bool MN>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int rows, int row, int k,
                                          int plane) {
  if constexpr (MN) {
    for (int i = 0; i < rows / 64; ++i) load_box<CG>(dst + i * 8192, tm, bar, row + 64 * i, k, plane);
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
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}

// 16 accumulator columns of this warp's 32 lanes.
__device__ __forceinline__ void ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
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
  int m, n, kb0, kb1;
  int split, rest;  // K range and number among the split tiles; split -1: whole
};

// Stores a 32 x 32 bf16 box (64-byte swizzle) from shared memory; what lies
// outside the map is not written.
__device__ __forceinline__ void store_box(const CUtensorMap* tm, uint32_t src, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(tm)),
      "r"(src), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// K ranges for `tiles` tiles (fewer than a round) on `units` CTAs or pairs, at
// least 16 k-blocks each: as many as fill one round, or two, whichever takes
// less time.  A range also writes a slab that is read again, about 12
// k-blocks' time (3 us), and the sum is a launch of its own.
// In whole numbers: host and device have to agree.
__host__ __device__ inline int split_rule(int tiles, int units, int kblocks, int most) {
  int best = 1, cost = kblocks;
  const int limit = kblocks / 16 < most ? kblocks / 16 : most;
  for (int rounds = 1; rounds <= 2; ++rounds) {
    const int fill = rounds * units / tiles, s = fill < limit ? fill : limit;
    if (s < 2) continue;
    const int c = (tiles * s + units - 1) / units * ((kblocks + s - 1) / s + 12) + 12;
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}

// The tiles of a product.  Whole rounds of the device take whole tiles; the
// tiles of a last, unfilled round (or of the only one) are split over K.
struct Cut {
  int m_tiles, n_tiles, kb, total_kb, whole, rest, splits, per_split, tiles;
  __device__ __forceinline__ void init(int M, int N, int K, int tile_m, int tile_n, int terms, int units, int most) {
    m_tiles = (M + tile_m - 1) / tile_m;
    n_tiles = (N + tile_n - 1) / tile_n;
    kb = (K + BK - 1) / BK;
    total_kb = kb * terms;
    const int all = m_tiles * n_tiles;
    whole = all;
    rest = 0;
    splits = 1;
    if (most > 1) {
      const int left = all % units;
      splits = left ? split_rule(left, units, total_kb, most) : 1;
      if (splits > 1) {
        rest = left;
        whole = all - left;
      }
    }
    per_split = (total_kb + splits - 1) / splits;
    tiles = whole + rest * splits;
  }
  // Panels of `gm` row tiles, columns of tiles inside: the tiles that run
  // together share their operands in L2.
  __device__ __forceinline__ void place(int t, int gm, int* m, int* n) const {
    const int p = t / (gm * n_tiles), first = p * gm;
    const int g = min(m_tiles - first, gm);
    const int i = t - first * n_tiles;
    *n = i / g;
    *m = first + (i - *n * g);
  }
};
constexpr int kPanel = 16;  // row tiles of 128 per panel

template <int CG>
struct Plan : Cut {
  __device__ __forceinline__ void init(const Args& a, int terms) {
    Cut::init(a.m_count ? *a.m_count : a.M, a.N, a.k_count ? *a.k_count : a.K, BM * CG, a.bn, terms, a.units,
              a.max_splits);
  }
  __device__ __forceinline__ Tile at(int t) const {
    Tile r;
    r.split = -1;  // whole
    r.rest = 0;
    r.kb0 = 0;
    r.kb1 = total_kb;
    if (t >= whole) {
      const int u = t - whole;
      r.split = u / rest;
      r.rest = u - r.split * rest;
      r.kb0 = min(total_kb, r.split * per_split);
      r.kb1 = min(total_kb, r.kb0 + per_split);
      t = whole + r.rest;
    }
    place(t, kPanel / CG, &r.m, &r.n);
    return r;
  }
  // End of the tensor-memory sum that starts at c0.  Of several plane products
  // all but the last add up to 2^-8 of it, and their error counts as little.
  __device__ __forceinline__ int chunk_end(const Args& a, int terms, int c0, int kb1) const {
    const int small = (terms - 1) * kb;
    if (c0 < small) return min(kb1, min(c0 + 64, small));
    return min(kb1, c0 + a.chunk);
  }
};

// ---------------------------------------------------------------- epilogues
// Each handles up to 128 columns from n_tile * bn + half * 128 of one row per
// thread, in registers.

// x *= (h w)^2 for two columns, in packed operations.
__device__ __forceinline__ void scale2(float& x0, float& x1, float h, float w0, float w1) {
  asm("{\n\t.reg .b64 x, t, h;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 h, {%2, %2};\n\tmov.b64 t, {%3, %4};\n\t"
      "mul.rn.f32x2 t, t, h;\n\tmul.rn.f32x2 x, x, t;\n\tmul.rn.f32x2 x, x, t;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(h), "f"(w0), "f"(w1));
}
// Takes the operands' powers of two back, the product of their halves twice:
// it is a normal number whatever the rows' sizes, so a sum of 0 stays 0 and
// one that fp32 holds is not lost on the way.  Columns past the matrix are
// ignored by what follows.
__device__ __forceinline__ void unscale(const Args& a, int64_t i, bool on, int v0, float (&x)[4][32]) {
  const float hi = on ? a.h_inv[i] : 0.f;
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 w = *reinterpret_cast<const float4*>(a.w_inv + v0 + c * 32 + j);
      scale2(x[c][j], x[c][j + 1], hi, w.x, w.y);
      scale2(x[c][j + 2], x[c][j + 3], hi, w.z, w.w);
    }
}

__device__ __forceinline__ void stats_epilogue(const Args& a, int64_t i, int64_t n, bool on, int n_tile, int half,
                                               int v0, int pos, float (&x)[4][32]) {
  const float s2 = a.scale * kLog2e;
  const int cols = min(min(128, a.bn - half * 128), a.N - (n_tile * a.bn + half * 128));
  int next = on && pos < a.list.K ? a.list.ids[n * a.list.K + pos] : kNoId;
  float m = -INFINITY;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    while (next >= v0 + c * 32 && next < v0 + min(c * 32 + 32, cols)) {
      a.zsel[n * a.list.K + pos] = pick(x[c], next - v0 - c * 32) * a.scale;
      next = ++pos < a.list.K ? a.list.ids[n * a.list.K + pos] : kNoId;
    }
    if (c * 32 + 32 > cols) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (c * 32 + j >= cols) x[c][j] = -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) m = fmaxf(m, x[c][j]);
  }
  // (x - m) first: one product of x less one of m would round at the size of
  // the logits, 1e-6 of a sum at logits of 15
  const float ref = m > -INFINITY ? m : 0.f;
  float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int j = 0; j < 32; ++j) t[j & 3] += ex2((x[c][j] - ref) * s2);
  if (on)
    a.part[(int64_t)(n_tile * 2 + half) * a.part_ld + i] =
        make_float2(m * a.scale, cols > 0 ? (t[0] + t[1]) + (t[2] + t[3]) : 0.f);
}

// Every warp writes its 32 rows as 32 x 32 boxes through shared memory: stores
// from the registers would touch 32 lines each.
template <int PLANES>
__device__ __forceinline__ void grad_epilogue(const Args& a, const CUtensorMap* tm, uint32_t stage, int64_t i0,
                                              int lane, int64_t n, bool on, int n_tile, int half, int v0, int pos,
                                              float (&x)[4][32]) {
  const int col0 = n_tile * a.bn + half * 128;
  const int cols = min(min(128, a.bn - half * 128), a.N - col0);
  // what is written: whole k-blocks of the products to come, zeros past N
  const int out_cols = min(min(128, a.bn - half * 128), (a.N + BK - 1) / BK * BK - col0);
  const float cw = on ? a.weight[n] * a.scale : 0.f;
  const float l = on ? a.lse[n] : 0.f;
  int next = on && pos < a.list.K ? a.list.ids[n * a.list.K + pos] : kNoId;
  const uint32_t row = (uint32_t)lane * 64, sw = (uint32_t)(lane >> 1) & 3u;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float* v = x[c];
    if (on) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = cw * ex2(fmaf(v[j], a.scale, -l) * kLog2e);
      while (next >= v0 + c * 32 && next < v0 + min(c * 32 + 32, cols)) {
        const int id = next, slot = pos;
        sub_at(v, id - v0 - c * 32, cw * (a.list.q ? a.list.q[n * a.list.K + pos] : 1.f));
        next = ++pos < a.list.K ? a.list.ids[n * a.list.K + pos] : kNoId;
        if constexpr (PLANES == 1) {
          if (a.resid) {  // of an id in several slots the last has it
            const float g = pick(v, id - v0 - c * 32);
            a.resid[n * a.list.K + slot] = next == id ? 0.f : g - to_f32(from_f32<bf16>(g));
          }
        }
      }
      if (c * 32 + 32 > cols) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = c * 32 + j < cols ? v[j] : 0.f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = 0.f;
    }
#pragma unroll
    for (int p = 0; p < PLANES; ++p) {
      if (c * 32 >= out_cols) continue;  // an even number of chunks is written: the buffers keep alternating
      const uint32_t buf = stage + (uint32_t)((c * PLANES + p) & 1) * 2048;
      if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float* u = v + j * 8 + 2 * e;
          w[e] = pack2(u[0], u[1]);
          if (p + 1 < PLANES) {
            u[0] -= __uint_as_float(w[e] << 16);
            u[1] -= __uint_as_float(w[e] & 0xFFFF0000u);
          }
        }
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + row + (((uint32_t)j ^ sw) << 4)), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3])
                     : "memory");
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) store_box(tm, buf, col0 + c * 32, (int)i0, p);
    }
  }
}

// Up to 32 columns of one row per lane, eight at a time.
template <typename OT>
__device__ __forceinline__ void store_row32(OT* o, float* v, int left, bool add) {
#pragma unroll
  for (int j = 0; j < 32; j += 8) {
    if (j + 8 <= left) {
      if (add) {
        float old[8];
        load8(o + j, old);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j + e] += old[e];
      }
      store8(o + j, v + j);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e < left) o[j + e] = from_f32<OT>(add ? v[j + e] + to_f32(o[j + e]) : v[j + e]);
    }
  }
}
// The same where rows are not 16-byte aligned: the warp's 32 rows go through shared memory and come out with the lanes along
// the columns (60 rows, V = 45885, d = 355, bf16: a backward in 194 us for 275).
// `at`: this lane's row, an offset of out; `on`: rows to write.
template <typename OT>
__device__ __forceinline__ void store_turned(OT* out, int64_t at, uint32_t on, uint32_t stage, int lane,
                                             const float* v, int left, bool add) {
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 32; ++j)
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(stage + (uint32_t)lane * 128 + (uint32_t)((j ^ lane) & 31) * 4), "f"(v[j])
                 : "memory");
  __syncwarp();
#pragma unroll 4
  for (int r = 0; r < 32; ++r) {
    const int64_t o = __shfl_sync(0xffffffffu, at, r) + lane;
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(stage + (uint32_t)r * 128 + (uint32_t)((lane ^ r) & 31) * 4));
    if (((on >> r) & 1u) && lane < left) out[o] = from_f32<OT>(add ? x + to_f32(out[o]) : x);
  }
}

template <int CG>
__device__ __forceinline__ void product_epilogue(const Args& a, uint32_t stage, int lane, int64_t i, int64_t n, bool on,
                                                 int n_tile, int half, float4* slab_row, float (&x)[4][32]) {
  const int col0 = n_tile * a.bn + half * 128;
  const int cols = min(a.bn - half * 128, a.N - col0);
  const uint32_t rows_on = __ballot_sync(0xffffffffu, on);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int left = cols - c * 32;
    if (left <= 0) return;
    float* v = x[c];
    if (slab_row) {
      if (on) {
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          slab_row[(half * 32 + c * 8 + j / 4) * (BM * CG)] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
      }
      continue;
    }
    if (a.acc) {
      const int64_t at = i * a.N + col0 + c * 32;
      if (a.acc_out) {
        if ((a.N & 3) == 0) {
          if (on) store_row32(a.acc + at, v, left, a.acc_in != 0);
        } else {
          store_turned(a.acc, at, rows_on, stage, lane, v, left, a.acc_in != 0);
        }
        continue;
      }
      if (on && a.acc_in) {
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          if (j + 8 <= left && (a.N & 3) == 0) {
            float old[8];
            load8(a.acc + at + j, old);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j + e] += old[e];
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (j + e < left) v[j + e] += a.acc[at + j + e];
          }
        }
      }
    }
    const int64_t at = n * a.ld_out + col0 + c * 32;
    if (a.vec) {
      if (on) {
        if (a.out_bf16) store_row32(static_cast<bf16*>(a.out) + at, v, left, a.accumulate);
        else store_row32(static_cast<float*>(a.out) + at, v, left, a.accumulate);
      }
    } else if (a.out_bf16) {
      store_turned(static_cast<bf16*>(a.out), at, rows_on, stage, lane, v, left, a.accumulate);
    } else {
      store_turned(static_cast<float*>(a.out), at, rows_on, stage, lane, v, left, a.accumulate);
    }
  }
}

// ---------------------------------------------------------------- kernel
template <int KIND, int CG>
__global__ void __launch_bounds__(kThreads, 1)
    vocab_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmG,
                      const __grid_constant__ CUtensorMap tmA2,  // second forms; GRAD: of G
                      const __grid_constant__ CUtensorMap tmB2, const Args a) {
  using C = Cfg<CG>;
  constexpr bool A_MN = KIND == DW, B_MN = KIND == DH || KIND == DW;
  constexpr bool kChooses = KIND == STATS32 || KIND == GRAD3;  // between two forms of fp32 operands
  constexpr bool kFine = KIND == GRAD || KIND == DH || KIND == DW;  // between two of g
  constexpr bool kSecondA = kChooses || KIND == DH || KIND == DW, kSecondB = kChooses;
  const int S = a.stages;
  const uint32_t stage_bytes = C::A_BYTES + (uint32_t)a.bn / CG * (BK * 2);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(smem);
  const uint32_t bars = base + C::BAR_OFF;
  constexpr int MS = C::MOST_STAGES;
  const uint32_t full = bars, empty = bars + 8 * MS, acc_full = bars + 16 * MS, acc_empty = acc_full + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::BAR_OFF + 16 * MS + 32);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
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
  if (!a.early) griddep_enter();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  bool second = false;
  if constexpr (kChooses) {
    __shared__ uint32_t least[2][kThreads / 32];
    uint32_t h = least_of(a.least.h, a.least.n_h, kThreads), w = least_of(a.least.w, a.least.n_w, kThreads);
    h = __reduce_min_sync(0xffffffffu, h);
    w = __reduce_min_sync(0xffffffffu, w);
    if (lane == 0) {
      least[0][warp] = h;
      least[1][warp] = w;
    }
    __syncthreads();
    h = __reduce_min_sync(0xffffffffu, least[0][min(lane, kThreads / 32 - 1)]);
    w = __reduce_min_sync(0xffffffffu, least[1][min(lane, kThreads / 32 - 1)]);
    second = __any_sync(0xffffffffu, !fp16_holds(h, w, a.K));  // a vote: uniform
  } else {
    __syncthreads();
    if constexpr (kFine) {
      const int32_t* count = KIND == DW ? a.k_count : a.m_count;  // rows that take part
      second = __any_sync(0xffffffffu, a.fine_rows > 0 && *count <= a.fine_rows);
    }
  }
  if (a.early && warp >= 4) griddep_enter();
  if constexpr (CG == 2) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  Plan<CG> plan;
  const int terms = kSecondA && second ? a.terms2 : a.terms;
  plan.init(a, terms);
  const int first = blockIdx.x / CG, step = gridDim.x / CG;

  // The loops below run in whole warps with one elected lane at work: what
  // they count is then uniform and stays in uniform registers, where TMA and
  // MMA take their operands from.  (In a branch of lane 0 alone, moving them
  // there held the MMA warp to 640 cycles per k-block, whatever its width.)
  // A wait that runs out ends its role; the others' waits then run out too.
  if (warp == 0 || warp == 3) {
    // TMA: warp 0 loads A, warp 3 loads B.
    // Products of planes go smallest first: (2,0) (0,2) (1,1) (1,0) (0,1)
    // (0,0), or the last three, or (1,0) (0,0); `planes` lists an operand's,
    // last product lowest.
    const bool is_a = warp == 0;
    const uint32_t planes = terms == 6   ? (is_a ? 0x201100u : 0x021010u)
                            : terms == 3 ? (is_a ? 0x100u : 0x010u)
                            : terms == 2 ? (is_a ? 0x10u : 0u)
                                         : 0u;
    int slot = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    const uint32_t bytes = (uint32_t)(a.a_rows * CG + a.bn) * (BK * 2);
    const int k_off = is_a ? 0 : a.b_k;
    for (int t = first; t < plan.tiles && ok; t += step) {
      const Tile tile = plan.at(t);
      const int row = is_a ? tile.m * BM * CG + rank * BM : tile.n * a.bn + rank * (a.bn / CG) + a.b_row;
      int turn = tile.kb0 / max(1, plan.kb), kt = tile.kb0 - turn * plan.kb;
      for (int kb = tile.kb0; kb < tile.kb1; ++kb) {
        if (!mbar_wait(empty + 8 * slot, phase ^ 1u)) {
          ok = false;
          break;
        }
        __syncwarp();
        const int plane = (planes >> (4 * (terms - 1 - turn))) & 15;
        const uint32_t sa = base + slot * stage_bytes;
        uint32_t bar = full + 8 * slot;
        if (elect_one()) {
          if (is_a && rank == 0) mbar_arrive_expect_tx(bar, bytes);
          if constexpr (CG == 2) bar = in_leader(bar);
          if (is_a) load_tile<CG, A_MN>(sa, kSecondA && second ? &tmA2 : &tmA, bar, BM, row, kt * BK + k_off, plane);
          else load_tile<CG, B_MN>(sa + C::A_BYTES, kSecondB && second ? &tmB2 : &tmB, bar, a.bn / CG, row, kt * BK + k_off, plane);
        }
        __syncwarp();
        issued = min(S, issued + 1);
        if (++slot == S) {
          slot = 0;
          phase ^= 1u;
        }
        if (++kt == plan.kb) {
          kt = 0;
          ++turn;
        }
      }
    }
    if (!ok && is_a && rank == 0) {  // copies still in flight land before the CTA leaves
      for (int i = issued; i > 0; --i) {  // the last `issued` slots, oldest first
        const int at = slot - i;
        mbar_wait(full + 8 * (at < 0 ? at + S : at), at < 0 ? phase ^ 1u : phase);
      }
    }
  } else if (warp == 1 && rank == 0) {
    const uint32_t idesc = (1u << 4) | (kChooses && !second ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)A_MN << 15) | ((uint32_t)B_MN << 16) |
                           ((uint32_t)(a.bn >> 3) << 17) | ((uint32_t)(BM * CG >> 4) << 24);
    int slot = 0;
    uint32_t phase = 0, n_acc = 0;
    bool ok = true;
    for (int t = first; t < plan.tiles && ok; t += step) {
      const Tile tile = plan.at(t);
      for (int c0 = tile.kb0, c1; c0 < tile.kb1 && ok; c0 = c1, ++n_acc) {
        c1 = plan.chunk_end(a, terms, c0, tile.kb1);
        const uint32_t as = n_acc & 1u;
        if (!mbar_wait(acc_empty + 8 * as, ((n_acc >> 1) & 1u) ^ 1u)) {
          ok = false;
          break;
        }
        const uint32_t d = tmem + as * BN;
        for (int kb = c0; kb < c1; ++kb) {
          if (!mbar_wait(full + 8 * slot, phase)) {
            ok = false;
            break;
          }
          __syncwarp();
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t sa = base + slot * stage_bytes, sb = sa + C::A_BYTES;
          const uint64_t da = A_MN ? sdesc(sa, 8192) : sdesc(sa, 16), db = B_MN ? sdesc(sb, 8192) : sdesc(sb, 16);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)  // the address field counts 16 bytes
              mma<CG>(d, da + kk * (A_MN ? 128 : 2), db + kk * (B_MN ? 128 : 2), idesc, kb > c0 || kk > 0);
            commit<CG>(empty + 8 * slot);
            if (kb + 1 == c1) commit<CG>(acc_full + 8 * as);
          }
          __syncwarp();
          if (++slot == S) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
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
      const int v0 = tile.n * a.bn + half * 128 + a.b_row;
      int pos = 0;
      if constexpr (KIND != DH && KIND != DW) {
        if (on && a.list.K > 1) pos = lower_bound(a.list.ids + n * a.list.K, a.list.K, v0);
      }
      float x[4][32];
      bool ok = true;
      if (tile.kb0 == tile.kb1) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) x[c][j] = 0.f;
      }
      for (int c0 = tile.kb0; c0 < tile.kb1; c0 = plan.chunk_end(a, terms, c0, tile.kb1), ++n_acc) {
        const uint32_t as = n_acc & 1u;
        if (!mbar_wait(acc_full + 8 * as, (n_acc >> 1) & 1u)) {
          ok = false;
          break;
        }
        __syncwarp();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t d = tmem + as * BN + lanes + half * 128;
        // fp16: the sum of x1's products, complete, is scaled by 2^-12 as the leading product's joins it
        float keep = 1.f;
        if constexpr (kChooses) keep = !second && c0 == (terms - 1) * plan.kb ? 1.f / 4096 : 1.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float v[16];
          ld16(d + c * 16, v);
          if (c0 == tile.kb0) {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[c >> 1][(c & 1) * 16 + j] = v[j];
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[c >> 1][(c & 1) * 16 + j] = kChooses ? fmaf(x[c >> 1][(c & 1) * 16 + j], keep, v[j]) : x[c >> 1][(c & 1) * 16 + j] + v[j];
          }
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 1) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(acc_empty + 8 * as) : "memory");
          else arrive_at(in_leader(acc_empty + 8 * as));
        }
      }
      if (!ok) break;
      if constexpr (kChooses) {
        if (!second) unscale(a, i, on, v0, x);
      }
      if constexpr (KIND == STATS || KIND == STATS32) stats_epilogue(a, i, n, on, tile.n, half, v0, pos, x);
      else if constexpr (KIND != DH && KIND != DW) {
        const uint32_t stage = base + C::OUT_OFF + (uint32_t)(warp - 4) * 4096;
        if constexpr (KIND == GRAD3) grad_epilogue<3>(a, &tmG, stage, i - lane, lane, n, on, tile.n, half, v0, pos, x);
        else if (second) grad_epilogue<2>(a, &tmA2, stage, i - lane, lane, n, on, tile.n, half, v0, pos, x);
        else grad_epilogue<1>(a, &tmG, stage, i - lane, lane, n, on, tile.n, half, v0, pos, x);
      }
      else {
        float4* slab_row = tile.split < 0 ? nullptr
                                          : a.slab + ((int64_t)tile.split * plan.rest + tile.rest) * (BM * CG * BN / 4) +
                                                rank * BM + q * 32 + lane;
        product_epilogue<CG>(a, base + C::OUT_OFF + (uint32_t)(warp - 4) * 4096, lane, i, n, on, tile.n, half, slab_row, x);
      }
    }
    if constexpr (KIND == GRAD || KIND == GRAD3) {
      if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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

// embed_grad.cu -- embedding lookup with a scale, and its gradient by sorted
// tokens (launchers in vocab.h).
//
// Lookup: out[n] = scale * emb[tok[n]]; bound by the bytes of out and of the
// rows read, eight elements per thread.
//
// Gradient: demb[v] = scale * sum of dout[n] over tok[n] = v.  The ids are
// sorted (stable, so every id's rows come in order of n); the sorted rows are
// cut into runs of equal length, so that an id that makes up a tenth of the
// batch is summed by as many thread groups as its rows need.  A group walks its run
// in registers, writes the rows of ids that begin and end inside it, and
// leaves an fp32 partial for the id that it shares with its neighbours; the
// partials are added in run order.  demb is zeroed by the SMs that have no part
// in the sort, while it runs (finding the absent rows afterwards took as long at
// N = 65,536 and 16 us more at N = 8,191, d = 512).  Bound by the bytes of
// dout and demb, each moved once; nothing is added atomically.
#include <algorithm>

#include "vocab.h"

namespace rlt {
namespace {

constexpr int kSortOne = 16384;  // ids one block sorts in shared memory
constexpr int kSortChunk = 2048;  // ids per block of the passes over more

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

template <typename T>
__device__ __forceinline__ void read8(const T* p, int left, bool vec, float* v) {
  if (vec && left >= 8) {
    load8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < left ? to_f32(p[j]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void write8(T* p, int left, bool vec, const float* v) {
  if (vec && left >= 8) {
    store8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p[j] = from_f32<T>(v[j]);
  }
}

// Eight elements as they lie in memory, so that several rows can be in flight
// before the first is converted.
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16> {
  uint4 a;
  __device__ __forceinline__ void load(const bf16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void add_to(float* s) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[2 * i] += __uint_as_float(w[i] << 16);
      s[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void add_to(float* s) const {
    s[0] += a.x; s[1] += a.y; s[2] += a.z; s[3] += a.w;
    s[4] += b.x; s[5] += b.y; s[6] += b.z; s[7] += b.w;
  }
};

// ------------------------------------------------------------------ lookup
template <typename ET, typename OT>
__global__ void __launch_bounds__(256) lookup_kernel(const ET* emb, int64_t ld_emb, int V, int d, const int32_t* tok,
                                                     int64_t N, float scale, OT* out, int64_t ld_out, int vec_e,
                                                     int vec_o) {
  griddep_enter();
  const int per_row = (d + 7) / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t n = i / per_row;
  if (n >= N) return;
  const int c = (int)(i - n * per_row) * 8;
  const int32_t id = tok[n];
  float v[8] = {};
  if (id >= 0 && id < V) {
    read8(emb + (int64_t)id * ld_emb + c, d - c, vec_e, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= scale;
  }
  write8(out + n * ld_out + c, d - c, vec_o, v);
}

// ------------------------------------------------------------------ sort
// Stable ranks of a block's items by an 8-bit digit.  Warp w owns a
// contiguous run of items, `rounds` of 32; hist[w][digit] counts them.
__device__ __forceinline__ int rank_in_warp(uint32_t* hist, int digit, bool on) {
  unsigned same = __ballot_sync(0xffffffffu, on);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const bool bit = (digit >> b) & 1;
    const unsigned v = __ballot_sync(0xffffffffu, bit);
    same &= bit ? v : ~v;
  }
  const int lane = threadIdx.x & 31;
  const int before = __popc(same & ((1u << lane) - 1));
  int base = 0;
  if (on) base = (int)hist[digit];
  __syncwarp();
  if (on && before == 0) hist[digit] += __popc(same);
  __syncwarp();
  return base + before;
}
// Turns hist[32][256] into exclusive offsets in (digit, warp) order; 1024
// threads, totals of the digits into total[256] on the way.
__device__ __forceinline__ void scan_hist(uint32_t (*hist)[256], uint32_t* total, uint32_t* warp_sums) {
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  __syncthreads();
  if (t < 256) {
    uint32_t s = 0;
    for (int i = 0; i < 32; ++i) {
      const uint32_t n = hist[i][t];
      hist[i][t] = s;
      s += n;
    }
    uint32_t incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) warp_sums[w] = incl;
    total[t] = incl - s;
  }
  __syncthreads();
  if (t < 256) {
    uint32_t b = 0;
    for (int i = 0; i < w; ++i) b += warp_sums[i];
    total[t] += b;
  }
  __syncthreads();
}

// Zeroes rows [0, V) of a matrix; block b of `blocks`, `threads` each.
// (part of parts launches, so that every launch of a sort takes a share)
struct ZeroRows {
  uint8_t* p;
  int64_t row_bytes, ld_bytes;  // multiples of the element size
  int V, elem, whole;           // whole: no gaps between rows, base 16-byte aligned
  int part, parts;
};
__device__ __forceinline__ void zero_rows(const ZeroRows& z, int b, int blocks, int threads) {
  const int64_t step = (int64_t)blocks * threads, at = (int64_t)b * threads + threadIdx.x;
  if (z.whole) {  // one stretch of memory: 16 bytes at a time, whatever its rows are
    const int64_t bytes = z.row_bytes * z.V, n = bytes / 16, end = n * (z.part + 1) / z.parts;
    int64_t i = n * z.part / z.parts + at;
    uint4* p = reinterpret_cast<uint4*>(z.p);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (; i + 3 * step < end; i += 4 * step) {
      p[i] = zero;
      p[i + step] = zero;
      p[i + 2 * step] = zero;
      p[i + 3 * step] = zero;
    }
    for (; i < end; i += step) p[i] = zero;
    if (z.part + 1 == z.parts && at < bytes % 16) z.p[n * 16 + at] = 0;
    return;
  }
  const int64_t per_row = z.row_bytes / z.elem, n = per_row * z.V, end = n * (z.part + 1) / z.parts;
  for (int64_t i = n * z.part / z.parts + at; i < end; i += step) {
    uint8_t* p = z.p + i / per_row * z.ld_bytes + i % per_row * z.elem;
    if (z.elem == 4) *reinterpret_cast<uint32_t*>(p) = 0;
    else *reinterpret_cast<uint16_t*>(p) = 0;
  }
}

// All of N <= 16384 ids in one block.  Ids outside [0, V) get key V: last.
__global__ void __launch_bounds__(1024) sort_one_kernel(const int32_t* tok, int N, int V, int passes, int32_t* key_out,
                                                        int32_t* pos_out, const ZeroRows z) {
  griddep_enter();
  if (blockIdx.x > 0) {
    zero_rows(z, (int)blockIdx.x - 1, (int)gridDim.x - 1, 1024);
    return;
  }
  extern __shared__ uint32_t sm[];
  uint32_t* keys = sm;                                                   // [16384]
  uint16_t* where = reinterpret_cast<uint16_t*>(sm + kSortOne);          // [16384]
  uint32_t(*hist)[256] = reinterpret_cast<uint32_t(*)[256]>(sm + kSortOne + kSortOne / 2);
  __shared__ uint32_t total[256], warp_sums[32];
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  const int rounds = (N + 1023) / 1024;
  const int base = w * rounds * 32;
  for (int i = t; i < N; i += 1024) {
    const int32_t id = tok[i];
    keys[i] = id >= 0 && id < V ? (uint32_t)id : (uint32_t)V;
    where[i] = (uint16_t)i;
  }
  for (int p = 0; p < passes; ++p) {
    for (int i = t; i < 32 * 256; i += 1024) (&hist[0][0])[i] = 0;
    __syncthreads();
    uint32_t k[16], rank[16];
    uint16_t q[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      if (r < rounds) {
        const int i = base + r * 32 + lane;
        const bool on = i < N;
        k[r] = on ? keys[i] : 0;
        q[r] = on ? where[i] : 0;
        rank[r] = rank_in_warp(hist[w], (k[r] >> (8 * p)) & 255, on);
      }
    }
    scan_hist(hist, total, warp_sums);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      if (r < rounds && base + r * 32 + lane < N) {
        const int digit = (k[r] >> (8 * p)) & 255;
        const uint32_t to = total[digit] + hist[w][digit] + rank[r];
        keys[to] = k[r];
        where[to] = q[r];
      }
    }
    __syncthreads();
  }
  for (int i = t; i < N; i += 1024) {
    key_out[i] = (int32_t)keys[i];
    pos_out[i] = where[i];
  }
}

// One pass over more ids, blocks of 2048: digit counts per block, then the
// scatter, whose blocks work out their own offsets from all counts.
__global__ void __launch_bounds__(1024) sort_count_kernel(const int32_t* in, int64_t N, int V, int first, int shift,
                                                          uint32_t* counts, int sort_blocks, const ZeroRows z) {
  griddep_enter();
  if ((int)blockIdx.x >= sort_blocks) {
    zero_rows(z, (int)blockIdx.x - sort_blocks, (int)gridDim.x - sort_blocks, 1024);
    return;
  }
  __shared__ uint32_t h[256];
  const int t = threadIdx.x;
  if (t < 256) h[t] = 0;
  __syncthreads();
  for (int r = 0; r < kSortChunk / 1024; ++r) {
    const int64_t i = (int64_t)blockIdx.x * kSortChunk + r * 1024 + t;
    if (i < N) {
      uint32_t k = (uint32_t)in[i];
      if (first && k >= (uint32_t)V) k = (uint32_t)V;
      atomicAdd(&h[(k >> shift) & 255], 1u);
    }
  }
  __syncthreads();
  if (t < 256) counts[(int64_t)blockIdx.x * 256 + t] = h[t];
}
__global__ void __launch_bounds__(1024) sort_scatter_kernel(const int32_t* in, const int32_t* pos_in, int64_t N, int V,
                                                            int shift, const uint32_t* counts, int32_t* out,
                                                            int32_t* pos_out, int sort_blocks, const ZeroRows z) {
  griddep_enter();
  if ((int)blockIdx.x >= sort_blocks) {
    zero_rows(z, (int)blockIdx.x - sort_blocks, (int)gridDim.x - sort_blocks, 1024);
    return;
  }
  __shared__ uint32_t hist[32][256];
  __shared__ uint32_t part_all[4][256], part_before[4][256];
  __shared__ uint32_t total[256], before[256], warp_sums[32];
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  for (int i = t; i < 32 * 256; i += 1024) (&hist[0][0])[i] = 0;
  {  // counts of all blocks, and of the earlier ones
    const int digit = t & 255, g = t >> 8;
    uint32_t all = 0, mine = 0;
    for (unsigned b = g; b < (unsigned)sort_blocks; b += 4) {
      const uint32_t n = counts[(int64_t)b * 256 + digit];
      all += n;
      if (b < blockIdx.x) mine += n;
    }
    part_all[g][digit] = all;
    part_before[g][digit] = mine;
  }
  __syncthreads();
  constexpr int R = kSortChunk / 1024;
  uint32_t k[R], rank[R];
  int32_t q[R];
  const int64_t base = (int64_t)blockIdx.x * kSortChunk + w * 32 * R;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t i = base + r * 32 + lane;
    const bool on = i < N;
    k[r] = on ? (uint32_t)in[i] : 0;
    if (pos_in == nullptr && k[r] >= (uint32_t)V) k[r] = (uint32_t)V;
    q[r] = on ? (pos_in ? pos_in[i] : (int32_t)i) : 0;
    rank[r] = rank_in_warp(hist[w], (k[r] >> shift) & 255, on);
  }
  scan_hist(hist, total, warp_sums);  // hist: the warps' offsets within a digit
  if (t < 256) {
    const uint32_t all = part_all[0][t] + part_all[1][t] + part_all[2][t] + part_all[3][t];
    uint32_t incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) warp_sums[w] = incl;
    before[t] = incl - all + part_before[0][t] + part_before[1][t] + part_before[2][t] + part_before[3][t];
  }
  __syncthreads();
  if (t < 256) {
    uint32_t b = 0;
    for (int i = 0; i < w; ++i) b += warp_sums[i];
    before[t] += b;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (base + r * 32 + lane < N) {
      const int digit = (k[r] >> shift) & 255;
      const uint32_t to = before[digit] + hist[w][digit] + rank[r];
      out[to] = (int32_t)k[r];
      pos_out[to] = q[r];
    }
  }
}

// ------------------------------------------------------------------ sums
struct Sums {
  const int32_t *key, *pos;
  int64_t N;
  int V, d, run, group;  // rows per run; threads per group, eight columns each
  int64_t runs;
  float scale;
  float* part;  // [runs][2][d]: the run's first id when it began earlier, and its last when it goes on
  int accumulate, vec_in, vec_out;
  int64_t ld_in, ld_out;
};

template <typename OT>
__device__ __forceinline__ void finish_row(const Sums& a, OT* demb, int32_t v, int c, const float* s) {
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = a.scale * s[j];
  OT* o = demb + (int64_t)v * a.ld_out + c;
  if (a.accumulate) {
    float old[8];
    read8(o, a.d - c, a.vec_out, old);
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] += old[j];
  }
  write8(o, a.d - c, a.vec_out, r);
}

template <typename GT, typename OT>
__global__ void __launch_bounds__(256, 2) sum_kernel(const GT* dout, OT* demb, const Sums a) {
  griddep_enter();
  const int c0 = (int)blockIdx.y * a.group * 8;
  __shared__ int32_t keys[8][64], rows[8][64];
  const int g = threadIdx.x / a.group, lane = threadIdx.x % a.group;
  const int64_t run = (int64_t)blockIdx.x * (256 / a.group) + g;
  const int c = c0 + lane * 8;
  const int64_t i0 = run * a.run, i1 = min(a.N, i0 + a.run);
  for (int i = lane; i < a.run; i += a.group) {
    keys[g][i] = i0 + i < i1 ? a.key[i0 + i] : -1;
    rows[g][i] = i0 + i < i1 ? a.pos[i0 + i] : 0;
  }
  __syncthreads();
  if (run >= a.runs || c >= a.d) return;
  int32_t v = keys[g][0];
  bool shared = i0 > 0 && a.key[i0 - 1] == v;  // the id began in an earlier run
  float s[8] = {};
  auto close = [&](int32_t next) {  // the id's rows are all in: its row, or its partial
    if (shared) write8(a.part + run * 2 * a.d + c, a.d - c, a.d % 4 == 0, s);
    else finish_row(a, demb, v, c, s);
    v = next;
    shared = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = 0.f;
  };
  constexpr int U = sizeof(GT) == 2 ? 16 : 8;
  const bool vec = a.vec_in && a.d - c >= 8;
  for (int i = 0; i < a.run; i += U) {
    if (vec) {
      Raw8<GT> x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int32_t k = keys[g][i + u];
        if (k >= 0 && k < a.V) x[u].load(dout + (int64_t)rows[g][i + u] * a.ld_in + c);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int32_t k = keys[g][i + u];
        if (k >= 0 && k != v) close(k);
        if (k >= 0 && k < a.V) x[u].add_to(s);
      }
    } else {
      for (int u = 0; u < U; ++u) {
        const int32_t k = keys[g][i + u];
        if (k < 0) break;
        if (k != v) close(k);
        if (k >= a.V) break;
        const GT* p = dout + (int64_t)rows[g][i + u] * a.ld_in + c;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < a.d) s[j] += to_f32(p[j]);
      }
    }
    if (v >= a.V) return;  // the ids that do not count come last
  }
  if (v >= a.V) return;
  const bool goes_on = i1 < a.N && a.key[i1] == v;
  if (shared) write8(a.part + run * 2 * a.d + c, a.d - c, a.d % 4 == 0, s);
  else if (goes_on) write8(a.part + (run * 2 + 1) * a.d + c, a.d - c, a.d % 4 == 0, s);
  else finish_row(a, demb, v, c, s);
}

// Ids that go past the run they begin in.  A block looks at eight runs and
// adds the partials of those that start such an id: 256 columns, every eighth
// run per warp, the eight warps' sums in warp order.
template <typename OT>
__global__ void __launch_bounds__(256) join_runs_kernel(OT* demb, const Sums a) {
  griddep_enter();
  __shared__ float sums[8][32][9];
  __shared__ int64_t ends[8];  // first run behind the id's last; 0: nothing to add
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t run0 = (int64_t)blockIdx.x * 8;
  {
    const int64_t run = run0 + w, i0 = run * a.run, i1 = i0 + a.run;
    int64_t end = 0;
    if (i1 < a.N) {
      const int32_t v = a.key[i1 - 1], after = a.key[i1], before = i0 > 0 ? a.key[i0 - 1] : -1;
      if (v < a.V && after == v && before != v) {
        // 32 probes at a time: the first run behind the id's last
        int64_t lo = run + 1, hi = a.runs;
        while (lo < hi) {
          const int64_t step = (hi - lo + 31) / 32, at = lo + lane * step;
          const unsigned in = __ballot_sync(0xffffffffu, at < hi && a.key[at * a.run] <= v);
          if (in == 0) break;
          const int64_t last = lo + (31 - __clz(in)) * step;  // in is a prefix of the lanes
          hi = min(hi, last + step);
          lo = last + 1;
        }
        end = lo;
      }
    }
    if (lane == 0) ends[w] = end;
  }
  __syncthreads();
  const int c = (int)blockIdx.y * 256 + lane * 8;
  const bool vec = a.d % 4 == 0;
  for (int e = 0; e < 8; ++e) {
    const int64_t run = run0 + e, end = ends[e];
    if (end == 0) continue;
    float s[8] = {};
    if (c < a.d) {
      if (w == 0) read8(a.part + (run * 2 + 1) * a.d + c, a.d - c, vec, s);
      for (int64_t r = run + 1 + w; r < end; r += 32) {
        float x[4][8] = {};
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (r + 8 * u < end) read8(a.part + (r + 8 * u) * 2 * a.d + c, a.d - c, vec, x[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] += x[u][j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[w][lane][j] = s[j];
    __syncthreads();
    if (w == 0 && c < a.d) {
      for (int k = 1; k < 8; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += sums[k][lane][j];
      finish_row(a, demb, a.key[run * a.run + a.run - 1], c, s);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host
template <typename T>
bool aligned16(const T* p, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld * (int64_t)sizeof(T) % 16 == 0;
}

template <typename ET, typename OT>
cudaError_t lookup(const void* emb_, int64_t ld_emb, int V, int d, const int32_t* tok, int N, float scale, void* out_,
                   int64_t ld_out, cudaStream_t st) {
  const ET* emb = static_cast<const ET*>(emb_);
  OT* out = static_cast<OT*>(out_);
  const int64_t blocks = ((int64_t)N * ((d + 7) / 8) + 255) / 256;
  return launch_pdl(lookup_kernel<ET, OT>, dim3((unsigned)blocks), dim3(256), 0, st, emb, ld_emb, V, d, tok,
                    (int64_t)N, scale, out, ld_out, (int)aligned16(emb, ld_emb), (int)aligned16(out, ld_out));
}

struct Layout {
  size_t key[2] = {0, 0}, pos[2] = {0, 0}, counts = 0, part = 0, total = 0;
  int passes = 0, run = 0, group = 0;
  int64_t runs = 0;
};
Layout layout(int N, int V, int d) {
  Layout L;
  auto take = [&](size_t n) {
    const size_t at = L.total;
    L.total += align256(n);
    return at;
  };
  if (N == 0) return L;
  while (L.passes < 4 && ((uint64_t)V >> (8 * L.passes)) != 0) ++L.passes;  // keys 0..V
  // Longer runs leave fewer partials, shorter ones more groups to work.  Lookup
  // and gradient at d = 2048 with runs of 16 and of 64: 44 and 59 us for 1,000
  // rows, 70 and 78 for 8,191, 93 and 90 for 16,384, 233 and 205 for 65,536.
  L.run = N <= kSortOne ? 16 : 64;
  L.runs = ((int64_t)N + L.run - 1) / L.run;
  L.group = 32;
  while (L.group < 256 && L.group * 8 < d) L.group *= 2;
  const int copies = N <= kSortOne ? 1 : 2;
  for (int i = 0; i < copies; ++i) {
    L.key[i] = take((size_t)N * 4);
    L.pos[i] = take((size_t)N * 4);
  }
  if (copies == 2) L.counts = take(((size_t)N + kSortChunk - 1) / kSortChunk * 256 * 4);
  L.part = take((size_t)L.runs * 2 * d * 4);
  return L;
}
template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

#define EMBED_TRY(...)                \
  do {                                \
    cudaError_t e_ = (__VA_ARGS__);   \
    if (e_ != cudaSuccess) return e_; \
  } while (0)

template <typename GT, typename OT>
cudaError_t gradient(const void* dout_, int64_t ld_dout, const int32_t* tok, int N, int V, int d, float scale,
                     void* demb_, int64_t ld_demb, int accumulate, void* ws, cudaStream_t st) {
  const GT* dout = static_cast<const GT*>(dout_);
  OT* demb = static_cast<OT*>(demb_);
  const Layout L = layout(N, V, d);
  int last = 0;
  ZeroRows z{};
  z.parts = N <= kSortOne ? 1 : 2 * L.passes;
  if (!accumulate) {
    z.p = reinterpret_cast<uint8_t*>(demb);
    z.elem = sizeof(OT);
    z.row_bytes = (int64_t)d * z.elem;
    z.ld_bytes = ld_demb * z.elem;
    z.V = V;
    z.whole = ld_demb == d && (reinterpret_cast<uintptr_t>(demb) & 15) == 0;
  }
  const unsigned idle = accumulate ? 0 : (unsigned)std::min<int64_t>(
      kSmCount, ((int64_t)V * d + 16383) / 16384);  // zeroing blocks, 16k elements each or more
  if (N <= kSortOne) {
    constexpr int kSmem = kSortOne * 4 + kSortOne * 2 + 32 * 256 * 4;
    EMBED_TRY(cudaFuncSetAttribute(sort_one_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
    EMBED_TRY(launch_pdl(sort_one_kernel, dim3(1 + idle), dim3(1024), kSmem, st, tok, N, V, L.passes,
                         at<int32_t>(ws, L.key[0]), at<int32_t>(ws, L.pos[0]), z));
  } else {
    const unsigned blocks = (unsigned)(((int64_t)N + kSortChunk - 1) / kSortChunk);
    uint32_t* counts = at<uint32_t>(ws, L.counts);
    const int32_t *in = tok, *pos_in = nullptr;
    for (int p = 0; p < L.passes; ++p) {
      last = p & 1;
      int32_t *out = at<int32_t>(ws, L.key[last]), *pos_out = at<int32_t>(ws, L.pos[last]);
      EMBED_TRY(launch_pdl(sort_count_kernel, dim3(blocks + idle), dim3(1024), 0, st, in, (int64_t)N, V,
                           (int)(p == 0), 8 * p, counts, (int)blocks, z));
      ++z.part;
      EMBED_TRY(launch_pdl(sort_scatter_kernel, dim3(blocks + idle), dim3(1024), 0, st, in, pos_in, (int64_t)N, V, 8 * p,
                           (const uint32_t*)counts, out, pos_out, (int)blocks, z));
      ++z.part;
      in = out;
      pos_in = pos_out;
    }
  }
  Sums a{};
  a.key = at<int32_t>(ws, L.key[last]);
  a.pos = at<int32_t>(ws, L.pos[last]);
  a.N = N;
  a.V = V;
  a.d = d;
  a.run = L.run;
  a.group = L.group;
  a.runs = L.runs;
  a.scale = scale;
  a.part = at<float>(ws, L.part);
  a.accumulate = accumulate;
  a.vec_in = aligned16(dout, ld_dout);
  a.vec_out = aligned16(demb, ld_demb);
  a.ld_in = ld_dout;
  a.ld_out = ld_demb;
  const int groups = 256 / L.group;
  const unsigned blocks = (unsigned)((L.runs + groups - 1) / groups);
  const unsigned cols = (unsigned)((d + L.group * 8 - 1) / (L.group * 8));
  EMBED_TRY(launch_pdl(sum_kernel<GT, OT>, dim3(blocks, cols), dim3(256), 0, st, dout, demb, a));
  if (L.runs == 1) return cudaSuccess;
  return launch_pdl(join_runs_kernel<OT>, dim3((unsigned)((L.runs + 7) / 8), (unsigned)((d + 255) / 256)), dim3(256), 0, st, demb, a);
}

}  // namespace

cudaError_t embed_lookup(const void* emb, int64_t ld_emb, int emb_dtype, int V, int d, const int32_t* tok, int N,
                         float scale, void* out, int64_t ld_out, int out_dtype, cudaStream_t st) {
  if (N == 0) return cudaSuccess;
  if (emb_dtype) {
    if (out_dtype) return lookup<bf16, bf16>(emb, ld_emb, V, d, tok, N, scale, out, ld_out, st);
    return lookup<bf16, float>(emb, ld_emb, V, d, tok, N, scale, out, ld_out, st);
  }
  if (out_dtype) return lookup<float, bf16>(emb, ld_emb, V, d, tok, N, scale, out, ld_out, st);
  return lookup<float, float>(emb, ld_emb, V, d, tok, N, scale, out, ld_out, st);
}

size_t embed_backward_workspace_bytes(int N, int V, int d) { return layout(N, V, d).total; }

cudaError_t embed_backward(const void* dout, int64_t ld_dout, int dout_dtype, const int32_t* tok, int N, int V, int d,
                           float scale, void* demb, int64_t ld_demb, int demb_dtype, int accumulate, void* ws,
                           cudaStream_t st) {
  if (N == 0) {
    if (accumulate) return cudaSuccess;
    const size_t e = demb_dtype ? 2 : 4;
    return cudaMemset2DAsync(demb, ld_demb * e, 0, d * e, V, st);
  }
  if (dout_dtype) {
    if (demb_dtype) return gradient<bf16, bf16>(dout, ld_dout, tok, N, V, d, scale, demb, ld_demb, accumulate, ws, st);
    return gradient<bf16, float>(dout, ld_dout, tok, N, V, d, scale, demb, ld_demb, accumulate, ws, st);
  }
  if (demb_dtype) return gradient<float, bf16>(dout, ld_dout, tok, N, V, d, scale, demb, ld_demb, accumulate, ws, st);
  return gradient<float, float>(dout, ld_dout, tok, N, V, d, scale, demb, ld_demb, accumulate, ws, st);
}

}  // namespace rlt

// embed_grad.cu -- embedding lookup with a scale, and its gradient summed in
// token order (launchers in vocab.h).
#include "vocab.h"

namespace rlt {
namespace {

template <typename ET, typename OT>
__global__ void __launch_bounds__(256) lookup_kernel(const ET* emb, int64_t ld_emb, int V, int d, const int32_t* tok,
                                                     float scale, OT* out, int64_t ld_out) {
  griddep_enter();
  const int64_t n = blockIdx.x;
  const int32_t id = tok[n];
  const bool ok = id >= 0 && id < V;
  const ET* e = emb + (int64_t)(ok ? id : 0) * ld_emb;
  for (int i = threadIdx.x; i < d; i += 256) out[n * ld_out + i] = from_f32<OT>(ok ? scale * to_f32(e[i]) : 0.f);
}

// One block per vocabulary row: scans the ids in order and adds the rows that
// carry its own.
template <typename GT, typename OT>
__global__ void __launch_bounds__(256) scan_sum_kernel(const GT* dout, int64_t ld, const int32_t* tok, int N, int d,
                                                       float scale, OT* demb, int64_t ld_demb, int accumulate) {
  griddep_enter();
  const int32_t v = (int32_t)blockIdx.x;
  __shared__ int hits[256];
  __shared__ int warp_n[8];
  for (int c0 = 0; c0 < d; c0 += 1024) {
    float s[4] = {};
    for (int n0 = 0; n0 < N; n0 += 256) {
      const int n = n0 + threadIdx.x;
      const bool hit = n < N && tok[n] == v;
      const unsigned b = __ballot_sync(0xffffffffu, hit);
      const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
      if (lane == 0) warp_n[w] = __popc(b);
      if (__syncthreads_or(hit) == 0) continue;
      int base = 0, total = 0;
      for (int i = 0; i < 8; ++i) {
        base += i < w ? warp_n[i] : 0;
        total += warp_n[i];
      }
      if (hit) hits[base + __popc(b & ((1u << lane) - 1))] = n;
      __syncthreads();
      for (int i = 0; i < total; ++i)
        for (int j = 0; j < 4; ++j) {
          const int c = c0 + j * 256 + threadIdx.x;
          if (c < d) s[j] += to_f32(dout[(int64_t)hits[i] * ld + c]);
        }
      __syncthreads();
    }
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + j * 256 + threadIdx.x;
      if (c < d) {
        OT* o = demb + (int64_t)v * ld_demb + c;
        *o = from_f32<OT>(scale * s[j] + (accumulate ? to_f32(*o) : 0.f));
      }
    }
  }
}

template <typename ET, typename OT>
cudaError_t lookup(const void* emb, int64_t ld_emb, int V, int d, const int32_t* tok, int N, float scale, void* out,
                   int64_t ld_out, cudaStream_t st) {
  return launch_pdl(lookup_kernel<ET, OT>, dim3((unsigned)N), dim3(256), 0, st, static_cast<const ET*>(emb), ld_emb, V,
                    d, tok, scale, static_cast<OT*>(out), ld_out);
}
template <typename GT, typename OT>
cudaError_t scan_sum(const void* dout, int64_t ld, const int32_t* tok, int N, int V, int d, float scale, void* demb,
                     int64_t ld_demb, int accumulate, cudaStream_t st) {
  return launch_pdl(scan_sum_kernel<GT, OT>, dim3((unsigned)V), dim3(256), 0, st, static_cast<const GT*>(dout), ld,
                    tok, N, d, scale, static_cast<OT*>(demb), ld_demb, accumulate);
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

size_t embed_backward_workspace_bytes(int, int, int) { return 0; }

cudaError_t embed_backward(const void* dout, int64_t ld_dout, int dout_dtype, const int32_t* tok, int N, int V, int d,
                           float scale, void* demb, int64_t ld_demb, int demb_dtype, int accumulate, void*,
                           cudaStream_t st) {
  if (dout_dtype) {
    if (demb_dtype) return scan_sum<bf16, bf16>(dout, ld_dout, tok, N, V, d, scale, demb, ld_demb, accumulate, st);
    return scan_sum<bf16, float>(dout, ld_dout, tok, N, V, d, scale, demb, ld_demb, accumulate, st);
  }
  if (demb_dtype) return scan_sum<float, bf16>(dout, ld_dout, tok, N, V, d, scale, demb, ld_demb, accumulate, st);
  return scan_sum<float, float>(dout, ld_dout, tok, N, V, d, scale, demb, ld_demb, accumulate, st);
}

}  // namespace rlt

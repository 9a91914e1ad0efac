// vocab.h -- launchers of the vocabulary operators: softmax cross entropy and
// distillation over z = h w^T without kept logits, and the embedding lookup
// with its gradient.  Host side, not exported; arguments are validated by the
// entry points.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace rlt {

// One loss over N rows of h [N][d] against the V rows of w [V][d] (dtype 0
// fp32, 1 bf16; rows ld_* elements apart).  Every row compares softmax(z *
// inv_t) with a short list of K vocabulary ids: its target (K = 1, teacher
// null, weight 1), or the teacher's candidates with q = softmax(teacher *
// inv_t) over the slots whose id lies in [0, V).  A row with no such slot
// takes no part.
struct VocabLoss {
  const void* h;
  int64_t ld_h;
  const void* w;
  int64_t ld_w;
  int N, V, d, dtype;
  const int32_t* ids;    // [N][K]
  const float* teacher;  // [N][K], or null
  int K;
  float inv_t;
};

// Workspace bytes of one forward (backward = 0) or backward (1) call.
size_t vocab_workspace_bytes(const VocabLoss& p, int backward);

// loss[n] = log p(target) (teacher null) or KL(q || p); lse[n] = the
// log-sum-exp of the scaled logits; both 0 for rows that take no part.
cudaError_t vocab_forward(const VocabLoss& p, float* loss, float* lse, void* ws, cudaStream_t st);

// Gradient of -sum weight[n] logp[n] (teacher null) or sum weight[n] kl[n] to
// h and w (either may be null) in the operands' type; accumulate_dw adds to
// dw, otherwise all of dw is written.
cudaError_t vocab_backward(const VocabLoss& p, const float* lse, const float* weight, void* dh, int64_t ld_dh,
                           void* dw, int64_t ld_dw, int accumulate_dw, void* ws, cudaStream_t st);

// out[n] = scale * emb[tok[n]] (a zero row for ids outside [0, V)).
cudaError_t embed_lookup(const void* emb, int64_t ld_emb, int emb_dtype, int V, int d, const int32_t* tok, int N,
                         float scale, void* out, int64_t ld_out, int out_dtype, cudaStream_t st);

// demb[v] (+)= scale * sum of dout[n] over tok[n] = v, in order of n within the
// runs that the sorted rows are cut into, then in order of the runs.
size_t embed_backward_workspace_bytes(int N, int V, int d);
cudaError_t embed_backward(const void* dout, int64_t ld_dout, int dout_dtype, const int32_t* tok, int N, int V, int d,
                           float scale, void* demb, int64_t ld_demb, int demb_dtype, int accumulate, void* ws,
                           cudaStream_t st);

}  // namespace rlt

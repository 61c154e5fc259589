// la.h -- linear attention with a decay for each head: problem description and internal launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gdnqat.h"

namespace gdn {

struct LaProblem {
  const void* q;       // bf16 [tokens, Hqk, dk]
  const void* k;       // bf16 [tokens, Hqk, dk]
  const void* v;       // bf16 [tokens, Hv, dv]
  const float* g;      // fp32 [tokens, Hv], or [Hv] (head_decay)
  const float* h0;     // fp32 [N, Hv, dk, dv] or null
  const int32_t* cu;   // device cu_seqlens or null
  void* o;             // bf16 [tokens, Hv, dv]
  float* hT;           // fp32 [N, Hv, dk, dv] or null
  int B, T, N, Hqk, Hv, dk, dv;
  float scale;
  int head_decay;
  const int32_t* cu_host;
};

struct LaGrads {
  const void* dout;    // bf16 [tokens, Hv, dv]
  const float* dhT;    // fp32 [N, Hv, dk, dv] or null (zero)
  void* dq;            // bf16 [tokens, Hqk, dk]
  void* dk;            // bf16 [tokens, Hqk, dk]
  void* dv;            // bf16 [tokens, Hv, dv]
  float* dg;           // fp32, as g
  float* dh0;          // fp32 [N, Hv, dk, dv] or null
};

size_t la_fwd_workspace(const LaProblem& p);
cudaError_t launch_la_fwd(const LaProblem& p, void* ws, cudaStream_t stream);
size_t la_bwd_workspace(const LaProblem& p);
cudaError_t launch_la_bwd(const LaProblem& p, const LaGrads& gr, void* ws, cudaStream_t stream);

cudaError_t launch_upload_i32(const int32_t* host, int32_t* device, int64_t n, cudaStream_t stream);

cudaError_t launch_la_decode(const void* q, const void* k, const void* v, const float* g, const float* state,
                             float* state_out, void* o, int N, int Hqk, int Hv, int dk, int dv, float scale,
                             int state_qdq, cudaStream_t stream);

}  // namespace gdn

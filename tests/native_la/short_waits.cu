// short_waits.cu -- test-only entries to the linear-attention kernels built with GDN_WAIT_LIMIT=0.
//
// Each CTA's warps then leave their loops at their first wait, set the status word, wait (with the usual limits)
// for copies and products in flight, free their tensor memory and exit; the device stays usable.
#include "../../fp8_state_qat_gb300/csrc/la.h"

static gdn::LaProblem problem(const la_chunk_args* a) {
  return {a->q, a->k, a->v, a->g, a->h0, nullptr, a->o, a->hT, a->B, a->T, a->N, a->Hqk, a->Hv, a->dk, a->dv,
          a->scale, 0, nullptr};
}

extern "C" int la_testing_fwd(const la_chunk_args* a, void* ws, size_t bytes, cudaStream_t stream) {
  if (!a || a->cu_seqlens || a->B != a->N || bytes < gdn::la_fwd_workspace(problem(a))) return 1;
  return gdn::launch_la_fwd(problem(a), ws, stream) == cudaSuccess ? 0 : 2;
}

extern "C" int la_testing_bwd(const la_chunk_args* a, const la_chunk_grads* g, void* ws, size_t bytes,
                              cudaStream_t stream) {
  if (!a || a->cu_seqlens || a->B != a->N || bytes < gdn::la_bwd_workspace(problem(a))) return 1;
  return gdn::launch_la_bwd(problem(a), {g->dout, g->dhT, g->dq, g->dk, g->dv, g->dg, g->dh0}, ws, stream) ==
                 cudaSuccess ? 0 : 2;
}

// la_recurrent.cu -- linear attention with a decay for each head, token by token on CUDA cores.
//
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
//
// and its gradients, with dS_t = scale q_t do_t^T + exp(g_{t+1}) dS_{t+1}:
//   dq_t = scale S_t do_t,  dk_t = dS_t v_t,  dv_t = dS_t^T k_t.
// All four are one recurrence over a state St [da x dc]: forwards out_t = s St^T a_t after
// St = e^{g_t} St + b_t c_t^T; backwards out_t = St^T a_t after St += s b_t c_t^T, then
// St *= e^{g_t}:
//   o: a = q, b = k, c = v      dq: a = do, b = v, c = k (St = S^T)
//   dv: a = k, b = q, c = do    dk: a = v, b = do, c = q (St = dS^T)
// The gradient of g: the outputs depend on g through its prefix sums gam alone, dL/dgam_t =
// q_t . dq_t - k_t . dk_t (and <hT, dhT> at the end), so dg_t sums these over all later tokens
// (in 64 bits: the two terms cancel).
//
// One CTA per (sequence, value head, 64-column slab of dc): the state stays in registers, and the
// time is the chain of T token steps.
#include "common.cuh"
#include "la.h"

namespace gdn {
namespace {

struct RecParams {
  const __nv_bfloat16 *a, *b, *c, *e;   // e: rows dotted with the outputs, or null
  int Ha, Hb, Hc, He;                   // their heads
  const float* g;
  const int32_t* cu;
  const float* s0;                      // initial state or null; element (i, j) at i * si + j * sj
  float* sT;                            // final state or null
  const float* edge_with;               // <final state, edge_with> -> edge, or null
  int si, sj;
  __nv_bfloat16* out;
  float* out32;                         // or the same in fp32
  float* dot;                           // [slab][tokens, Hv]
  float* edge;                          // [slab][N, Hv]
  int64_t tokens;
  int T, Hv, head_decay, reverse;
  float scale;
};

template <int DA>
__global__ void __launch_bounds__(128) la_rec_kernel(const RecParams p, int dc) {
  constexpr int R = DA / 8;
  const int slabs = dc / 64;
  const int slab = blockIdx.x % slabs;
  const int64_t unit = blockIdx.x / slabs;
  const int n = (int)(unit / p.Hv), h = (int)(unit % p.Hv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rg = lane >> 2, col = slab * 64 + warp * 16 + (lane & 3) * 4;
  const int64_t t0 = p.cu ? p.cu[n] : (int64_t)n * p.T;
  const int64_t len = p.cu ? p.cu[n + 1] - p.cu[n] : p.T;
  const int64_t sbase = unit * DA * dc;
  const int ha = h / (p.Hv / p.Ha), hb = h / (p.Hv / p.Hb), hc = h / (p.Hv / p.Hc);
  float s[R][4];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      s[i][j] = p.s0 ? p.s0[sbase + (int64_t)(rg + 8 * i) * p.si + (int64_t)(col + j) * p.sj] : 0.f;
  __shared__ float red[4];
  for (int64_t step = 0; step < len; ++step) {
    const int64_t t = t0 + (p.reverse ? len - 1 - step : step);
    const __nv_bfloat16* ap = p.a + (t * p.Ha + ha) * DA;
    const __nv_bfloat16* bp = p.b + (t * p.Hb + hb) * DA;
    const __nv_bfloat16* cp = p.c + (t * p.Hc + hc) * dc + col;
    const float al = expf(p.head_decay ? p.g[h] : p.g[t * p.Hv + h]);
    float cv[4], o[4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) cv[j] = bf16_to_f32(cp[j]) * (p.reverse ? p.scale : 1.f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float av = bf16_to_f32(ap[rg + 8 * i]), bv = bf16_to_f32(bp[rg + 8 * i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = fmaf(bv, cv[j], p.reverse ? s[i][j] : al * s[i][j]);
        o[j] = fmaf(s[i][j], av, o[j]);
        if (p.reverse) s[i][j] *= al;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) o[j] += __shfl_xor_sync(0xffffffffu, o[j], off);
      if (!p.reverse) o[j] *= p.scale;
    }
    if (rg == 0)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t at = (t * p.Hv + h) * dc + col + j;
        if (p.out32) p.out32[at] = o[j];
        else p.out[at] = __float2bfloat16_rn(o[j]);
      }
    if (p.e) {
      const __nv_bfloat16* ep = p.e + (t * p.He + h / (p.Hv / p.He)) * dc + col;
      float d = 0.f;
      if (rg == 0)
#pragma unroll
        for (int j = 0; j < 4; ++j) d = fmaf(o[j], bf16_to_f32(ep[j]), d);
      d = warp_sum(d);
      __syncthreads();
      if (lane == 0) red[warp] = d;
      __syncthreads();
      if (threadIdx.x == 0)
        p.dot[(int64_t)slab * p.tokens * p.Hv + t * p.Hv + h] = (red[0] + red[1]) + (red[2] + red[3]);
    }
  }
  float d = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t at = sbase + (int64_t)(rg + 8 * i) * p.si + (int64_t)(col + j) * p.sj;
      if (p.sT) p.sT[at] = s[i][j];
      if (p.edge_with) d = fmaf(s[i][j], p.edge_with[at], d);
    }
  if (p.edge) {
    d = warp_sum(d);
    __syncthreads();
    if (lane == 0) red[warp] = d;
    __syncthreads();
    if (threadIdx.x == 0)
      p.edge[slab * ((int64_t)gridDim.x / slabs) + unit] = (red[0] + red[1]) + (red[2] + red[3]);
  }
}

// dg of one (sequence, head): suffix sums of rq - rk plus the edge term, or their sum over the tokens
__global__ void la_dg_kernel(const float* rq, int nq, const float* rk, int nk, const float* edge, int ne, float* dg,
                             double* head_part, const int32_t* cu, int T, int N, int Hv, int64_t tokens) {
  const int64_t unit = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (unit >= (int64_t)N * Hv) return;
  const int n = (int)(unit / Hv), h = (int)(unit % Hv);
  const int64_t t0 = cu ? cu[n] : (int64_t)n * T, len = cu ? cu[n + 1] - cu[n] : T;
  double s = 0., all = 0.;
  for (int i = 0; i < ne; ++i) s += edge[i * (int64_t)N * Hv + unit];
  for (int64_t t = t0 + len - 1; t >= t0; --t) {
    for (int i = 0; i < nq; ++i) s += rq[i * tokens * Hv + t * Hv + h];
    for (int i = 0; i < nk; ++i) s -= rk[i * tokens * Hv + t * Hv + h];
    if (head_part) all += s;
    else dg[t * Hv + h] = (float)s;
  }
  if (head_part) head_part[unit] = all;
}
__global__ void la_dg_head_kernel(const double* part, float* dg, int N, int Hv) {
  const int h = blockIdx.x * blockDim.x + threadIdx.x;
  if (h >= Hv) return;
  double s = 0.;
  for (int n = 0; n < N; ++n) s += part[(int64_t)n * Hv + h];
  dg[h] = (float)s;
}
// the sum over the value heads of a query head
__global__ void la_group_sum_kernel(const float* x, __nv_bfloat16* y, int64_t rows, int G, int D) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= rows * D) return;
  const int64_t row = i / D, d = i % D;
  float s = 0.f;
  for (int j = 0; j < G; ++j) s += x[(row * G + j) * D + d];
  y[i] = __float2bfloat16_rn(s);
}

cudaError_t rec(const RecParams& p, int N, int da, int dc, cudaStream_t stream) {
  const int64_t ctas = (int64_t)N * p.Hv * (dc / 64);
  if (ctas == 0) return cudaSuccess;
  if (da == 64) la_rec_kernel<64><<<(unsigned)ctas, 128, 0, stream>>>(p, dc);
  else la_rec_kernel<128><<<(unsigned)ctas, 128, 0, stream>>>(p, dc);
  return cudaGetLastError();
}

struct BwdWs {
  size_t rq, rk, edge, head, part, total;
};
BwdWs bwd_ws(const LaProblem& p) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const int64_t tokens = (int64_t)p.B * p.T;
  BwdWs w;
  size_t at = 256;
  w.rq = at; at += up((size_t)tokens * p.Hv * (p.dk / 64) * 4);
  w.rk = at; at += up((size_t)tokens * p.Hv * (p.dk / 64) * 4);
  w.edge = at; at += up((size_t)p.N * p.Hv * (p.dk / 64) * 4);
  w.head = at; at += up((size_t)p.N * p.Hv * 8);
  w.part = at; at += p.Hv == p.Hqk ? 0 : up((size_t)tokens * p.Hv * p.dk * 4);
  w.total = at;
  return w;
}

}  // namespace

size_t la_fwd_workspace(const LaProblem&) { return 256; }
cudaError_t launch_la_fwd(const LaProblem& p, void* ws, cudaStream_t stream) {
  using B = const __nv_bfloat16*;
  cudaError_t e0 = cudaMemsetAsync(ws, 0, 4, stream);   // the status word
  if (e0 != cudaSuccess) return e0;
  RecParams r{};
  r.a = (B)p.q; r.b = (B)p.k; r.c = (B)p.v;
  r.Ha = r.Hb = p.Hqk; r.Hc = p.Hv; r.He = p.Hv;
  r.g = p.g; r.cu = p.cu; r.s0 = p.h0; r.sT = p.hT; r.si = p.dv; r.sj = 1;
  r.out = (__nv_bfloat16*)p.o;
  r.tokens = (int64_t)p.B * p.T; r.T = p.T; r.Hv = p.Hv; r.head_decay = p.head_decay; r.scale = p.scale;
  return rec(r, p.N, p.dk, p.dv, stream);
}

size_t la_bwd_workspace(const LaProblem& p) { return bwd_ws(p).total; }
cudaError_t launch_la_bwd(const LaProblem& p, const LaGrads& gr, void* ws, cudaStream_t stream) {
  using B = const __nv_bfloat16*;
  unsigned char* base = static_cast<unsigned char*>(ws);
  const BwdWs w = bwd_ws(p);
  const int64_t tokens = (int64_t)p.B * p.T;
  const int G = p.Hv / p.Hqk;
  float *rq = (float*)(base + w.rq), *rk = (float*)(base + w.rk), *edge = (float*)(base + w.edge);
  float* part = (float*)(base + w.part);
  double* head = (double*)(base + w.head);
  RecParams r{};
  r.g = p.g; r.cu = p.cu; r.tokens = tokens; r.T = p.T; r.Hv = p.Hv; r.head_decay = p.head_decay; r.scale = p.scale;
  auto group_sum = [&](void* out) {
    const int64_t n = tokens * p.Hqk * p.dk;
    if (n) la_group_sum_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(part, (__nv_bfloat16*)out, tokens * p.Hqk, G, p.dk);
    return cudaGetLastError();
  };
  cudaError_t e = cudaMemsetAsync(ws, 0, 4, stream);   // the status word
  if (e != cudaSuccess) return e;
  // dq
  RecParams q = r;
  q.a = (B)gr.dout; q.b = (B)p.v; q.c = (B)p.k; q.e = (B)p.q;
  q.Ha = q.Hb = p.Hv; q.Hc = q.He = p.Hqk;
  q.s0 = p.h0; q.si = 1; q.sj = p.dv; q.edge_with = gr.dhT; q.edge = edge; q.dot = rq;
  if (G > 1) q.out32 = part; else q.out = (__nv_bfloat16*)gr.dq;
  if ((e = rec(q, p.N, p.dv, p.dk, stream)) != cudaSuccess) return e;
  if (G > 1 && (e = group_sum(gr.dq)) != cudaSuccess) return e;
  // dk
  q = r;
  q.reverse = 1;
  q.a = (B)p.v; q.b = (B)gr.dout; q.c = (B)p.q; q.e = (B)p.k;
  q.Ha = q.Hb = p.Hv; q.Hc = q.He = p.Hqk;
  q.s0 = gr.dhT; q.si = 1; q.sj = p.dv; q.dot = rk;
  if (G > 1) q.out32 = part; else q.out = (__nv_bfloat16*)gr.dk;
  if ((e = rec(q, p.N, p.dv, p.dk, stream)) != cudaSuccess) return e;
  if (G > 1 && (e = group_sum(gr.dk)) != cudaSuccess) return e;
  // dv, dh0
  q = r;
  q.reverse = 1;
  q.a = (B)p.k; q.b = (B)p.q; q.c = (B)gr.dout;
  q.Ha = q.Hb = p.Hqk; q.Hc = q.He = p.Hv;
  q.s0 = gr.dhT; q.sT = gr.dh0; q.si = p.dv; q.sj = 1;
  q.out = (__nv_bfloat16*)gr.dv;
  if ((e = rec(q, p.N, p.dk, p.dv, stream)) != cudaSuccess) return e;
  const int64_t units = (int64_t)p.N * p.Hv;
  if (units)
    la_dg_kernel<<<(unsigned)((units + 31) / 32), 32, 0, stream>>>(rq, p.dk / 64, rk, p.dk / 64, edge, p.dk / 64, gr.dg,
                                                                 p.head_decay ? head : nullptr, p.cu, p.T, p.N, p.Hv,
                                                                 tokens);
  if (p.head_decay) la_dg_head_kernel<<<(unsigned)((p.Hv + 31) / 32), 32, 0, stream>>>(head, gr.dg, p.N, p.Hv);
  return cudaGetLastError();
}

}  // namespace gdn

// la_chunk.cu -- chunked linear attention with a decay for each head: the launches of the forward and of
// its gradients, and the gradient of the decays.
//
// Forward: the states entering the chunks (la_state.cu), then o (la_out.cu, role o).
// Backward: the states entering the chunks, the state gradients leaving them, then dq, dk, dv
// (la_out.cu, three roles), then dg, and with shared q/k heads the sums over their value heads.
//
// dg. o depends on g_t through every decay that spans token t: with (i < t <= j) all pairs of a chunk,
//   dg_t = sum_{i < t <= j} m_ji + sum_{j >= t} a_j + sum_{i < t} b_i + exp(gam_C) <S, dS>,
//   m_ji = scale D (q_j . k_i)(do_j . v_i),  a_j = q_j . (state part of dq_j),  b_i = k_i . (state part of dk_i),
// S entering and dS leaving the chunk. With r_j, c_i the row and column sums of m (i != j) the first
// sum is sum_{j >= t} (r_j - c_j). No term is larger than the decayed products themselves, where the
// usual suffix sum of q . dq - k . dk over the whole sequence subtracts undecayed ones.
#include <algorithm>

#include "kernels.h"
#include "la_chunk.cuh"

namespace gdn {
namespace la {
namespace {

struct DgParams {
  Seqs seqs;
  GateSrc gates;
  const float *rq, *rk, *aq, *bk;        // per (token, head): r and c in two parts, a, b
  int64_t th;                            // tokens x heads
  const float* edge;                     // exp(gam_C) <S, dS> per item, in parts; or null:
  int parts;
  const __nv_bfloat16 *S, *dS;           // then from the two terms of S and dS, per item
  int elems;                             // of a state
  float* dg;                             // [tokens, Hv], or per item with head_decay
};

// One CTA of 128 threads per (chunk slot, head): thread = token.
__global__ void __launch_bounds__(kC) la_dg_kernel(const DgParams p) {
  dependents_may_start();
  dependency_wait();
  const int64_t item = blockIdx.x;
  const int Hv = p.gates.Hv, h = (int)(item % Hv);
  const int64_t slot = item / Hv;
  int lo = 0, hi = p.seqs.N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.seqs.slot0(mid) <= slot) lo = mid;
    else hi = mid - 1;
  }
  const int64_t c = slot - p.seqs.slot0(lo), len = p.seqs.len(lo), tok = p.seqs.start(lo) + c * kC;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if (c < 0 || c * kC >= len) {
    if (p.gates.head_decay && t == 0) p.dg[item] = 0.f;
    return;
  }
  const int L = (int)(len - c * kC < kC ? len - c * kC : kC);
  __shared__ float red[3][4];
  // exp(gam_C) <S, dS>, from its parts (at most 32), or from S and dS
  float x = 0.f;
  if (p.edge) {
    if (t < p.parts) x = p.edge[item * p.parts + t];
  } else {
    float gx[4];
    Gates w;
    p.gates.load(gx, tok, h, L, lane);
    const uint4* S = reinterpret_cast<const uint4*>(p.S + 2 * item * p.elems);
    const uint4* dS = reinterpret_cast<const uint4*>(p.dS + 2 * item * p.elems);
    const int n = p.elems / 8;
    float2 s = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int i = t; i < n; i += kC) {
      const uint4 a = S[i], al = S[i + n], b = dS[i], bl = dS[i + n];
      const uint32_t au[4] = {a.x, a.y, a.z, a.w}, alu[4] = {al.x, al.y, al.z, al.w};
      const uint32_t bu[4] = {b.x, b.y, b.z, b.w}, blu[4] = {bl.x, bl.y, bl.z, bl.w};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        s = __ffma2_rn(__fadd2_rn(unpack_bf16(au[q]), unpack_bf16(alu[q])),
                       __fadd2_rn(unpack_bf16(bu[q]), unpack_bf16(blu[q])), s);
    }
    scan_gates(gx, w, lane);
    x = warp_sum(s.x + s.y) * expf((w.tot(0) + w.tot(1)) + (w.tot(2) + w.tot(3)));
  }
  const int64_t at = (tok + t) * Hv + h;
  float f = 0.f, b = 0.f;
  if (t < L) {
    f = ((p.rq[at] + p.rq[p.th + at]) - (p.rk[at] + p.rk[p.th + at])) + p.aq[at];
    b = p.bk[at];
  }
  float fs = f, bs = b;   // suffix sums of f, prefix sums of b, both with the own token
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const float yf = __shfl_down_sync(0xffffffffu, fs, off), yb = __shfl_up_sync(0xffffffffu, bs, off);
    if (lane + off < 32) fs += yf;
    if (lane >= off) bs += yb;
  }
  if (p.edge) x = warp_sum(x);
  if (lane == 0) {
    red[0][warp] = fs;
    red[2][warp] = x;
  }
  if (lane == 31) red[1][warp] = bs;
  __syncthreads();
  float v = fs + (bs - b);
  float before = 0.f, after = 0.f;
  for (int w = 0; w < 4; ++w) {
    if (w > warp) after += red[0][w];
    if (w < warp) before += red[1][w];
  }
  v = (v + (after + before)) + ((red[2][0] + red[2][1]) + (red[2][2] + red[2][3]));
  if (!p.gates.head_decay) {
    if (t < L) p.dg[at] = v;
    return;
  }
  v = warp_sum(t < L ? v : 0.f);
  __syncthreads();
  if (lane == 0) red[0][warp] = v;
  __syncthreads();
  if (t == 0) p.dg[item] = (red[0][0] + red[0][1]) + (red[0][2] + red[0][3]);
}

// dg of a fixed decay: the sum over all chunks, 256 threads in a fixed order, in 64 bits
__global__ void __launch_bounds__(256) la_dg_head_kernel(const float* part, float* dg, int64_t slots, int Hv) {
  __shared__ double red[256];
  dependents_may_start();
  dependency_wait();
  const int h = blockIdx.x, t = threadIdx.x;
  double s = 0.;
  for (int64_t i = t; i < slots; i += 256) s += part[i * Hv + h];
  red[t] = s;
  __syncthreads();
  for (int n = 128; n > 0; n >>= 1) {
    if (t < n) red[t] += red[t + n];
    __syncthreads();
  }
  if (t == 0) dg[h] = (float)red[0];
}

// The status word. Cleared by a kernel, the walk after it sets itself up meanwhile: a forward of 1 x 256 tokens, 2 heads
// 16.2 us with a memset in its place, 14.6 us with this; in a CUDA graph 15.8 and 12.9.
__global__ void la_clear_kernel(int* status) {
  dependents_may_start();
  *status = 0;
}

// Host values to device memory as launch parameters (4 KB hold 1000 of them). A copy would read the host's memory when
// the stream comes to it, if that is pinned, or at a replay: offsets of packed sequences have to be those that the call's
// sizes were made of.
struct Values {
  static constexpr int kMost = 1000;
  int32_t v[kMost];
};
__global__ void __launch_bounds__(128) upload_kernel(const __grid_constant__ Values x, int32_t* device, int n) {
  const int i = blockIdx.x * 128 + threadIdx.x;
  if (i < n) device[i] = x.v[i];
}

// dq and dk (blockIdx.y) of a shared head: the sum over its value heads, four channels a thread
__global__ void __launch_bounds__(256) la_group_sum_kernel(const float* x0, const float* x1, __nv_bfloat16* y0,
                                                           __nv_bfloat16* y1, int64_t quads, int G, int D4) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  dependency_wait();
  if (i >= quads) return;
  const float4* x = reinterpret_cast<const float4*>(blockIdx.y ? x1 : x0);
  const int64_t row = i / D4, d = i % D4;
  float4 s = x[row * G * D4 + d];
  for (int j = 1; j < G; ++j) {
    const float4 v = x[(row * G + j) * D4 + d];
    s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
  }
  reinterpret_cast<uint2*>(blockIdx.y ? y1 : y0)[i] = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
}

size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

// By sizes alone, so that a workspace serves every packing of the same sizes.
struct Layout {
  size_t S, dS, tot, dec, rq, rk, aq, bk, edge, pq, pk, item, total;
};
Layout layout_of(const LaProblem& p, bool bwd) {
  const size_t items = (size_t)la_slots(p) * p.Hv, elems = (size_t)p.dk * p.dv, th = (size_t)p.B * p.T * p.Hv;
  const int nseg = most_segments(p);
  Layout l{};
  size_t at = kStatusBytes;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += up(n);
    return here;
  };
  l.S = take(items * elems * 4);
  if (bwd) l.dS = take(items * elems * 4);
  if (nseg > 1) {
    l.tot = take((size_t)p.N * p.Hv * nseg * elems * 4);
    l.dec = take((size_t)p.N * p.Hv * nseg * 4);
  }
  if (bwd) {
    l.rq = take(th * 8);
    l.rk = take(th * 8);
    l.aq = take(th * 4);
    l.bk = take(th * 4);
    if (nseg > 1 || !walks_beside(p)) l.edge = take(items * edge_parts(p) * 4);
    if (p.Hv != p.Hqk) {
      l.pq = take(th * p.dk * 4);
      l.pk = take(th * p.dk * 4);
    }
    if (p.head_decay) l.item = take(items * 4);
  }
  l.total = at;
  return l;
}

}  // namespace
}  // namespace la

using namespace la;

cudaError_t launch_upload_i32(const int32_t* host, int32_t* device, int64_t n, cudaStream_t stream) {
  Values x;
  for (int64_t at = 0; at < n; at += Values::kMost) {
    const int m = (int)std::min<int64_t>(n - at, Values::kMost);
    std::copy(host + at, host + at + m, x.v);
    std::fill(x.v + m, x.v + Values::kMost, 0);
    const cudaError_t e = launch(false, upload_kernel, dim3((unsigned)((m + 127) / 128)), 128, 0, stream, x, device + at, m);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

size_t la_fwd_workspace(const LaProblem& p) { return layout_of(p, false).total; }
size_t la_bwd_workspace(const LaProblem& p) { return layout_of(p, true).total; }

cudaError_t launch_la_fwd(const LaProblem& p, void* ws, cudaStream_t stream) {
  unsigned char* const base = static_cast<unsigned char*>(ws);
  const Layout l = layout_of(p, false);
  int* const status = static_cast<int*>(ws);
  cudaError_t e = launch(false, la_clear_kernel, dim3(1), 1, 0, stream, status);
  if (e != cudaSuccess) return e;
  StateRun s{p.k, p.v, p.h0, p.hT, base + l.S, 0, 1.f, (float*)(base + l.tot), (float*)(base + l.dec),
             nullptr, nullptr, 0};
  // o reads h0 through the states alone, so hT may be h0
  if ((e = launch_states(p, s, status, true, stream)) != cudaSuccess) return e;
  // tiles k, q, v | S hi, lo
  OutRun o{{p.q, p.k, p.v, nullptr}, {base + l.S, nullptr}, 3, {1, 0, 2, 0}, 2, {0, 0}, {0, 1}, {}, 1};
  o.role[0] = {1, 0, 2, -1, 0, 0x37, 0, 0, p.scale, p.scale, p.o, 0, nullptr, nullptr};
  return launch_outputs(p, o, status, stream);
}

cudaError_t launch_la_bwd(const LaProblem& p, const LaGrads& gr, void* ws, cudaStream_t stream) {
  unsigned char* const base = static_cast<unsigned char*>(ws);
  const Layout l = layout_of(p, true);
  int* const status = static_cast<int*>(ws);
  const int64_t tokens = (int64_t)p.B * p.T, items = la_slots(p) * p.Hv;
  const int G = p.Hv / p.Hqk;
  float *tot = (float*)(base + l.tot), *dec = (float*)(base + l.dec);
  float *rq = (float*)(base + l.rq), *rk = (float*)(base + l.rk), *aq = (float*)(base + l.aq), *bk = (float*)(base + l.bk);
  float* const edge = (float*)(base + l.edge);
  float *pq = (float*)(base + l.pq), *pk = (float*)(base + l.pk);
  const bool beside = walks_beside(p);
  cudaError_t e = launch(false, la_clear_kernel, dim3(1), 1, 0, stream, status);
  if (e != cudaSuccess) return e;
  StateRun f{p.k, p.v, p.h0, nullptr, base + l.S, 0, 1.f, tot, dec, nullptr, nullptr, 0};
  // a walk that the next one may overtake starts when the status word is clear
  if ((e = launch_states(p, f, status, !beside, stream)) != cudaSuccess) return e;
  StateRun b{p.q, gr.dout, gr.dhT, gr.dh0, base + l.dS, 1, p.scale, tot, dec,
             beside ? nullptr : base + l.S, beside ? nullptr : edge, beside};
  if ((e = launch_states(p, b, status, true, stream)) != cudaSuccess) return e;
  if (tokens == 0 || items == 0)
    return p.head_decay ? cudaMemsetAsync(gr.dg, 0, (size_t)p.Hv * 4, stream) : cudaSuccess;
  // tiles v, q, k, do | S hi, lo, dS hi, lo
  OutRun o{{p.q, p.k, p.v, gr.dout}, {base + l.S, base + l.dS}, 4, {2, 0, 1, 3}, 4, {0, 0, 1, 1}, {0, 1, 0, 1}, {}, 3};
  o.role[0] = {3, 0, 2, 1, 0, 0x30, 1, 0, p.scale, p.scale, G > 1 ? (void*)pq : gr.dq, G > 1, rq, aq};
  o.role[1] = {0, 3, 1, 2, 2, 0x01, 1, 1, p.scale, 1.f, G > 1 ? (void*)pk : gr.dk, G > 1, rk, bk};
  o.role[2] = {2, 1, 3, -1, 2, 0x37, 0, 1, p.scale, 1.f, gr.dv, 0, nullptr, nullptr};
  if ((e = launch_outputs(p, o, status, stream)) != cudaSuccess) return e;
  DgParams d{{p.cu, p.T, p.N}, {p.g, p.Hv, p.head_decay}, rq, rk, aq, bk, tokens * p.Hv, beside ? nullptr : edge,
             edge_parts(p), (const __nv_bfloat16*)(base + l.S), (const __nv_bfloat16*)(base + l.dS), p.dk * p.dv,
             p.head_decay ? (float*)(base + l.item) : gr.dg};
  if ((e = launch(true, la_dg_kernel, dim3((unsigned)items), kC, 0, stream, d)) != cudaSuccess) return e;
  if (p.head_decay) {
    if ((e = launch(true, la_dg_head_kernel, dim3((unsigned)p.Hv), 256, 0, stream, (const float*)(base + l.item), gr.dg,
                    la_slots(p), p.Hv)) != cudaSuccess)
      return e;
  }
  if (G > 1) {
    const int64_t quads = tokens * p.Hqk * (p.dk / 4);
    e = launch(true, la_group_sum_kernel, dim3((unsigned)((quads + 255) / 256), 2), 256, 0, stream, (const float*)pq,
               (const float*)pk, (__nv_bfloat16*)gr.dq, (__nv_bfloat16*)gr.dk, quads, G, p.dk / 4);
  }
  return e;
}

}  // namespace gdn

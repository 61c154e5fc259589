// la_decode.cu -- one token per sequence of linear attention with a decay for each head.
//
//   S' = exp(g) S + k v^T,  o = scale S'^T q (from the updated, not yet quantized state),
//   state_out = QDQ(S') (E4M3: one scale per all key rows x 64 value columns, INT8: per key row x 32
//   value columns), or S'.
//
// Bound by HBM: the state is read once and written once, 8 dk dv bytes a head, against 4 dk dv
// flops. One CTA of 128 threads per (sequence, head, 64-column slab): a slab is a whole E4M3 tile
// (two INT8 blocks wide), so a CTA never waits for another, and few sequences still spread over
// dv / 64 times as many SMs. Warp w owns 16 columns; lane 4 rg + cg holds rows rg, rg + 8, ... of
// four columns in 16-byte accesses, and the sums over rows are xor shuffles in a fixed order. 512 sequences, 32
// heads, d 128, E4M3: 342 us, 6.32 TB/s (0.95 of the measured copy bandwidth); INT8: 449 us, 4.8 TB/s: a scale and
// a reciprocal a row lengthen the chain between a CTA's loads and stores, and four CTAs an SM do not cover it (issue
// slots 35 % used); one sequence, 16 heads: 5 us a call.
// The scale is amax times the rounded constant 1 / 448 (1 / 127), one multiply and at most an ulp from
// the quotient, 1 for an all-zero tile; the code is that of the correctly rounded quotient x / s, by paired fused
// multiply-adds (an IEEE divide an element took 425 us).
#include "common.cuh"
#include "la.h"

namespace gdn {
namespace {

// fl32(x / s) for two elements: paired fused multiply-adds with the rounded reciprocal (quotient2() in
// common.cuh) for a normal s, else the IEEE divide. `normal` is the same for a whole tile.
__device__ __forceinline__ float2 div2(float2 x, float s, float2 ns2, float2 r2, bool normal) {
  return normal ? quotient2(x, ns2, r2) : make_float2(__fdiv_rn(x.x, s), __fdiv_rn(x.y, s));
}

__device__ __forceinline__ float scale_of(float amax, float inv_max) {
  const float s = __fmul_rn(amax, inv_max);
  return s == 0.f ? 1.f : s;
}

template <int DK>
__global__ void __launch_bounds__(128)
la_decode_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                 const __nv_bfloat16* __restrict__ v, const float* __restrict__ g, const float* state,
                 float* state_out, __nv_bfloat16* __restrict__ o, int Hqk, int Hv, int dv, float scale,
                 int state_qdq) {
  constexpr int R = DK / 8;
  const int slabs = dv / 64;
  const int64_t unit = blockIdx.x / slabs;
  const int n = (int)(unit / Hv), h = (int)(unit % Hv), hq = h / (Hv / Hqk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rg = lane >> 2, cg = lane & 3;
  const int col = (int)(blockIdx.x % slabs) * 64 + warp * 16 + cg * 4;
  const int64_t base = unit * DK * dv + col;
  float4 s[R];
#pragma unroll
  for (int i = 0; i < R; ++i) s[i] = __ldcs(reinterpret_cast<const float4*>(state + base + (int64_t)(rg + 8 * i) * dv));
  const __nv_bfloat16* kp = k + ((int64_t)n * Hqk + hq) * DK;
  const __nv_bfloat16* qp = q + ((int64_t)n * Hqk + hq) * DK;
  const float a = expf(g[unit]);
  const __nv_bfloat162* vp = reinterpret_cast<const __nv_bfloat162*>(v + unit * dv + col);
  const float2 v01 = __bfloat1622float2(vp[0]), v23 = __bfloat1622float2(vp[1]);
  float4 ov = make_float4(0.f, 0.f, 0.f, 0.f);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float kr = bf16_to_f32(kp[rg + 8 * i]), qr = bf16_to_f32(qp[rg + 8 * i]);
    // a S is rounded, then the product k v, exact in fp32, is added: the two roundings of the formula
    s[i].x = fmaf(kr, v01.x, __fmul_rn(a, s[i].x)); s[i].y = fmaf(kr, v01.y, __fmul_rn(a, s[i].y));
    s[i].z = fmaf(kr, v23.x, __fmul_rn(a, s[i].z)); s[i].w = fmaf(kr, v23.y, __fmul_rn(a, s[i].w));
    ov.x = fmaf(s[i].x, qr, ov.x); ov.y = fmaf(s[i].y, qr, ov.y);
    ov.z = fmaf(s[i].z, qr, ov.z); ov.w = fmaf(s[i].w, qr, ov.w);
    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(s[i].x), fabsf(s[i].y)), fmaxf(fabsf(s[i].z), fabsf(s[i].w))));
  }
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    ov.x += __shfl_xor_sync(0xffffffffu, ov.x, off); ov.y += __shfl_xor_sync(0xffffffffu, ov.y, off);
    ov.z += __shfl_xor_sync(0xffffffffu, ov.z, off); ov.w += __shfl_xor_sync(0xffffffffu, ov.w, off);
  }
  if (rg == 0) {
    __nv_bfloat162 r[2] = {__floats2bfloat162_rn(scale * ov.x, scale * ov.y),
                           __floats2bfloat162_rn(scale * ov.z, scale * ov.w)};
    *reinterpret_cast<uint2*>(o + unit * dv + col) = *reinterpret_cast<const uint2*>(r);
  }
  if (state_qdq == 2) {   // INT8: a block is one key row x 32 columns = a row of warps 2 b and 2 b + 1
    __shared__ float rmax[4][DK];
    float m[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      m[i] = fmaxf(fmaxf(fabsf(s[i].x), fabsf(s[i].y)), fmaxf(fabsf(s[i].z), fabsf(s[i].w)));
      m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 1));
      m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 2));
      if (cg == 0) rmax[warp][rg + 8 * i] = m[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float sc = scale_of(fmaxf(m[i], rmax[warp ^ 1][rg + 8 * i]), 1.f / kInt8Max), rc = __frcp_rn(sc);
      const float2 ns2 = make_float2(-sc, -sc), r2 = make_float2(rc, rc);
      const float2 a = div2(make_float2(s[i].x, s[i].y), sc, ns2, r2, sc >= 1.0e-30f);
      const float2 b = div2(make_float2(s[i].z, s[i].w), sc, ns2, r2, sc >= 1.0e-30f);
      s[i] = make_float4(__fmul_rn(rintf(a.x), sc), __fmul_rn(rintf(a.y), sc), __fmul_rn(rintf(b.x), sc),
                         __fmul_rn(rintf(b.y), sc));
    }
  } else if (state_qdq) {
    __shared__ float wmax[4];
    amax = warp_max(amax);
    if (lane == 0) wmax[warp] = amax;
    __syncthreads();
    const float sc = scale_of(fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3])), 1.f / kE4M3Max);
    const float2 ns2 = make_float2(-sc, -sc), r2 = make_float2(__frcp_rn(sc), __frcp_rn(sc));
    auto qdq = [&](bool normal) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const __nv_fp8x2_e4m3 c01(div2(make_float2(s[i].x, s[i].y), sc, ns2, r2, normal));
        const __nv_fp8x2_e4m3 c23(div2(make_float2(s[i].z, s[i].w), sc, ns2, r2, normal));
        const float2 f01 = static_cast<float2>(c01), f23 = static_cast<float2>(c23);
        s[i] = make_float4(__fmul_rn(f01.x, sc), __fmul_rn(f01.y, sc), __fmul_rn(f23.x, sc), __fmul_rn(f23.y, sc));
      }
    };
    if (sc >= 1.0e-30f) qdq(true);
    else qdq(false);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) __stcs(reinterpret_cast<float4*>(state_out + base + (int64_t)(rg + 8 * i) * dv), s[i]);
}

}  // namespace

cudaError_t launch_la_decode(const void* q, const void* k, const void* v, const float* g, const float* state,
                             float* state_out, void* o, int N, int Hqk, int Hv, int dk, int dv, float scale,
                             int state_qdq, cudaStream_t stream) {
  const int64_t ctas = (int64_t)N * Hv * (dv / 64);
  if (ctas == 0) return cudaSuccess;
  const auto qb = static_cast<const __nv_bfloat16*>(q), kb = static_cast<const __nv_bfloat16*>(k);
  const auto vb = static_cast<const __nv_bfloat16*>(v);
  const auto ob = static_cast<__nv_bfloat16*>(o);
  if (dk == 64)
    la_decode_kernel<64><<<(unsigned)ctas, 128, 0, stream>>>(qb, kb, vb, g, state, state_out, ob, Hqk, Hv, dv, scale,
                                                            state_qdq);
  else
    la_decode_kernel<128><<<(unsigned)ctas, 128, 0, stream>>>(qb, kb, vb, g, state, state_out, ob, Hqk, Hv, dv, scale,
                                                             state_qdq);
  return cudaGetLastError();
}

}  // namespace gdn

// norm.cu -- RMS norms around a block, fused with the gate and the residual scale, and their gradients.
//
//   gated norm     y  = rms(x) w silu(z),                     rms(x) = x rsqrt(mean(x^2) + eps)
//   residual norm  h' = h + alpha n,  n = rms(y) w_post (or y without w_post);  x = rms(h') w_pre
//
// A row is held by TPR threads, 8 elements each, from its load to its store, so every tensor moves
// once: the kernels are bound by HBM (about 1 to 2 flops a byte). Statistics, sums and weight
// gradients are fp32; each output is rounded once. VEC: element e of thread t is column 8 t + e and
// moves in 16-byte accesses (D % 8 == 0, aligned pointers); otherwise column t + TPR e, one element
// at a time, so that a warp still reads whole lines of a row of any length and alignment.
// TPR is the power of two >= D / 8, at least 8: up to 32 threads a row reduces by shuffles alone and
// a CTA holds 256 / TPR rows; above that a CTA holds one row (two for TPR 64, 128) and adds one
// shared-memory step per reduction.
//
// The backward recomputes the statistics from the inputs it reads anyway (no tensor is saved for
// it). Weight gradients are sums over all rows: each thread sums its columns over the rows its CTA
// takes, a CTA adds its row groups in order, and a second launch adds the CTAs' partial rows in a
// fixed order -- no atomics, the same bits every run. That launch is set up while the first still runs (forward and
// backward of 16384 x 2048, fp32 stream: 172 -> 170 us; of 2000 x 2048: 34 -> 31).
//
// Each thread loads its next row before it works on the present one. Measured: gated norm of 262144 x 128 bf16, forward 33 us
// (6.1 TB/s of its inputs and outputs), backward 58 us (5.8); residual norm of 16384 x 2048, fp32 stream, forward
// 58 us (6.9), backward 90 us (6.7). At 33.5 M elements of other even widths the backwards reach 3.9 to 6.2 TB/s, 2.8 to 3.9 at
// 8192 columns; odd widths move 2 or 4 bytes a thread at a time and reach 2.0 to 5.7 TB/s.
#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace gdn {
namespace {

constexpr int E = 8;                  // elements a thread

__device__ __forceinline__ void store8f(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8f(__nv_bfloat16* p, const float* v) {
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
}
__device__ __forceinline__ float tof(float x) { return x; }
__device__ __forceinline__ float tof(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// The 8 elements of thread t of a row as they lie in memory, so that the next row's loads can be in flight
// while a row is worked on; columns past D and rows past the end are zero.
template <int TPR, bool VEC, class T>
struct Raw {
  __align__(16) T x[E];
  __device__ __forceinline__ void load(const T* row, bool live, int D, int t) {
    if (VEC) {
      constexpr int N = E * sizeof(T) / 16;
      uint4* r = reinterpret_cast<uint4*>(x);
      const uint4* p = reinterpret_cast<const uint4*>(row + 8 * t);
#pragma unroll
      for (int i = 0; i < N; ++i) r[i] = live && 8 * t < D ? p[i] : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = live && t + TPR * e < D ? row[t + TPR * e] : T(0.f);
    }
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = tof(x[e]);
  }
};
template <int TPR, bool VEC, class T>
__device__ __forceinline__ void load_row(const T* row, int D, int t, float* v) {
  Raw<TPR, VEC, T> r;
  r.load(row, true, D, t);
  r.get(v);
}
template <int TPR, bool VEC, class T>
__device__ __forceinline__ void store_row(T* row, int D, int t, const float* v) {
  if (VEC) {
    if (8 * t < D) store8f(row + 8 * t, v);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (t + TPR * e < D) put(row + t + TPR * e, v[e]);
  }
}
// A weight of either type (bf16 or fp32), by a flag that is the same for the whole launch.
template <int TPR, bool VEC>
__device__ __forceinline__ void load_w(const void* w, int w_bf16, int D, int t, float* v) {
  if (w_bf16) load_row<TPR, VEC>(static_cast<const __nv_bfloat16*>(w), D, t, v);
  else load_row<TPR, VEC>(static_cast<const float*>(w), D, t, v);
}

constexpr int kSums = 8;               // places for the values that one reduction sums
constexpr int threads_of(int tpr) { return tpr < 256 ? 256 : tpr; }
// Resident CTAs an SM that a backward's registers leave room for (and its launch asks for): its rows in flight
// need about 100 registers a thread.
constexpr int bwd_per_sm(int tpr) { return tpr <= 256 ? 2 : 1; }

// Sums of M values over the TPR threads of a row, the same in each of them. `slot` alternates
// between calls, so that one barrier a call is enough.
template <int TPR, int M>
struct RowSum {
  static constexpr int kWarps = threads_of(TPR) / 32;
  static __device__ __forceinline__ void run(float (&v)[M], float (*smem)[kWarps][kSums], int& slot) {
    if constexpr (M > 4) many(v, smem, slot);
    else each(v, smem, slot);
  }
  static __device__ __forceinline__ void each(float (&v)[M], float (*smem)[kWarps][kSums], int& slot) {
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
    if constexpr (TPR > 32) {
      const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
      if (lane == 0)
#pragma unroll
        for (int m = 0; m < M; ++m) smem[slot][warp][m] = v[m];
      meet();
      constexpr int PER = TPR / 32;         // warps a row
      const int w0 = warp / PER * PER;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        float s = lane < PER ? smem[slot][w0 + lane][m] : 0.f;
#pragma unroll
        for (int o = (PER < 32 ? PER : 32) / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        v[m] = __shfl_sync(0xffffffffu, s, 0);
      }
      slot ^= 1;
    }
  }
  // 5 to 8 values: the first three exchanges halve the values that a lane keeps, so that lane l ends with the sum of
  // value l / (W / 8) alone; then everyone reads all of them. 18 shuffles for 7 values of 8 warps, where a tree for each
  // value takes 63, and half of the time went to them (residual backward of 33.5 M elements, 1024 columns, bf16 103 ->
  // 78 us, fp32 141 -> 103; 2048 columns 103 -> 78, 110 -> 98).
  static __device__ __forceinline__ void many(float (&v)[M], float (*smem)[kWarps][kSums], int& slot) {
    constexpr int W = TPR < 32 ? TPR : 32, G = W / 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float a[8];
#pragma unroll
    for (int m = 0; m < 8; ++m) a[m] = m < M ? v[m] : 0.f;
#pragma unroll
    for (int n = 4; n > 0; n >>= 1) {   // lanes o apart share 2 n values, the upper one keeps the upper n
      const int o = n * G;
      const bool upper = lane & o;
#pragma unroll
      for (int m = 0; m < n; ++m) {
        const float other = __shfl_xor_sync(0xffffffffu, upper ? a[m] : a[m + n], o);
        a[m] = (upper ? a[m + n] : a[m]) + other;
      }
    }
    float s = a[0];
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if constexpr (TPR <= 32) {
#pragma unroll
      for (int m = 0; m < M; ++m) v[m] = __shfl_sync(0xffffffffu, s, m * G, W);
    } else {
      if (lane % G == 0) smem[slot][warp][lane / G] = s;
      meet();
      constexpr int PER = TPR / 32;
      const int w0 = warp / PER * PER, m = lane & 7;
      s = 0.f;
#pragma unroll
      for (int w = 0; w < PER; w += 4)
        if (w + (lane >> 3) < PER) s += smem[slot][w0 + w + (lane >> 3)][m];
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
#pragma unroll
      for (int j = 0; j < M; ++j) v[j] = __shfl_sync(0xffffffffu, s, j);
      slot ^= 1;
    }
  }
  // the row's own threads meet, not those of the CTA's other rows
  static __device__ __forceinline__ void meet() {
    if constexpr (TPR < 256) asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / TPR), "n"(TPR) : "memory");
    else __syncthreads();
  }
};

// 1 / (1 + exp(-z)) from the hardware's exponential and reciprocal: a few units in 2^-22 for |z| up to 10, far
// below the rounding of what it goes into; exp(-z) = inf gives 0. The IEEE forms made the kernel issue-bound.
__device__ __forceinline__ float sigmoidf(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

template <int TPR, bool VEC, class X>
__global__ void __launch_bounds__(threads_of(TPR))
gated_norm_fwd_kernel(const X* __restrict__ x, const __nv_bfloat16* __restrict__ z, const void* __restrict__ w,
                      int w_bf16, __nv_bfloat16* __restrict__ y, int64_t rows, int D, float eps) {
  constexpr int RPC = threads_of(TPR) / TPR;
  __shared__ float sm[2][threads_of(TPR) / 32][kSums];
  int slot = 0;
  const int t = threadIdx.x % TPR, rg = threadIdx.x / TPR;
  float wv[E];
  load_w<TPR, VEC>(w, w_bf16, D, t, wv);
  const float inv_d = 1.f / (float)D;
  Raw<TPR, VEC, X> nx;
  Raw<TPR, VEC, __nv_bfloat16> nz;
  const int64_t stride = (int64_t)gridDim.x * RPC;
  int64_t r = (int64_t)blockIdx.x * RPC + rg;
  nx.load(x + r * D, r < rows, D, t);
  nz.load(z + r * D, r < rows, D, t);
  for (int64_t r0 = (int64_t)blockIdx.x * RPC; r0 < rows; r0 += stride, r += stride) {
    const bool live = r < rows;
    float xv[E], zv[E];
    nx.get(xv);
    nz.get(zv);
    nx.load(x + (r + stride) * D, r + stride < rows, D, t);
    nz.load(z + (r + stride) * D, r + stride < rows, D, t);
    float s[1] = {0.f};
#pragma unroll
    for (int e = 0; e < E; ++e) s[0] = fmaf(xv[e], xv[e], s[0]);
    RowSum<TPR, 1>::run(s, sm, slot);
    const float rs = rsqrtf(fmaf(s[0], inv_d, eps));
    if (live) {
      float o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = xv[e] * rs * wv[e] * (zv[e] * sigmoidf(zv[e]));
      store_row<TPR, VEC>(y + r * D, D, t, o);
    }
  }
}

// One row group's column sums of M weight gradients -> the CTA's partial row: the groups added in order.
template <int TPR, bool VEC, int M>
__device__ __forceinline__ void write_partials(float (&acc)[M][E], float* red, float* const (&out)[M], int D) {
  constexpr int RPC = threads_of(TPR) / TPR;
  const int t = threadIdx.x % TPR, rg = threadIdx.x / TPR;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    if (!out[m]) continue;
    if (RPC > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e) red[(rg * E + e) * TPR + t] = acc[m][e];
      __syncthreads();
      if (rg == 0)
        for (int g = 1; g < RPC; ++g)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[m][e] += red[(g * E + e) * TPR + t];
    }
    if (rg == 0) store_row<TPR, VEC>(out[m] + (int64_t)blockIdx.x * D, D, t, acc[m]);
  }
}

// With n = rms(x), s = silu(z), d = dy w s (the gradient at n):
//   dx = r (d - n mean(d n)),  dz = dy n w silu'(z),  dw = sum over rows of dy n s
template <int TPR, bool VEC, class X>
__global__ void __launch_bounds__(threads_of(TPR), bwd_per_sm(TPR))
gated_norm_bwd_kernel(const __nv_bfloat16* __restrict__ dy, const X* __restrict__ x,
                      const __nv_bfloat16* __restrict__ z, const void* __restrict__ w, int w_bf16,
                      X* __restrict__ dx, __nv_bfloat16* __restrict__ dz, float* __restrict__ part, int64_t rows,
                      int D, float eps) {
  constexpr int RPC = threads_of(TPR) / TPR;
  __shared__ float sm[2][threads_of(TPR) / 32][kSums];
  __shared__ float red[RPC > 1 ? threads_of(TPR) * E : 1];
  int slot = 0;
  dependents_may_start();
  const int t = threadIdx.x % TPR, rg = threadIdx.x / TPR;
  float wv[E], acc[1][E] = {};
  load_w<TPR, VEC>(w, w_bf16, D, t, wv);
  const float inv_d = 1.f / (float)D;
  Raw<TPR, VEC, X> nx;
  Raw<TPR, VEC, __nv_bfloat16> nz, nd;
  const int64_t stride = (int64_t)gridDim.x * RPC;
  int64_t r = (int64_t)blockIdx.x * RPC + rg;
  nx.load(x + r * D, r < rows, D, t);
  nz.load(z + r * D, r < rows, D, t);
  nd.load(dy + r * D, r < rows, D, t);
  for (int64_t r0 = (int64_t)blockIdx.x * RPC; r0 < rows; r0 += stride, r += stride) {
    const bool live = r < rows;
    float xv[E], zv[E], dv[E];
    nx.get(xv);
    nz.get(zv);
    nd.get(dv);
    nx.load(x + (r + stride) * D, r + stride < rows, D, t);
    nz.load(z + (r + stride) * D, r + stride < rows, D, t);
    nd.load(dy + (r + stride) * D, r + stride < rows, D, t);
    float s[2] = {0.f, 0.f}, sg[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      sg[e] = sigmoidf(zv[e]);
      s[0] = fmaf(xv[e], xv[e], s[0]);
      s[1] = fmaf(dv[e] * wv[e] * (zv[e] * sg[e]), xv[e], s[1]);
    }
    RowSum<TPR, 2>::run(s, sm, slot);
    const float rs = rsqrtf(fmaf(s[0], inv_d, eps));
    const float c = s[1] * inv_d * rs * rs;      // mean(d n) r, the factor of x in n mean(d n)
    if (live) {
      float ox[E], oz[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float si = zv[e] * sg[e], n = xv[e] * rs, dn = dv[e] * n;
        ox[e] = rs * fmaf(-c, xv[e], dv[e] * wv[e] * si);
        oz[e] = dn * wv[e] * (sg[e] * (1.f + zv[e] * (1.f - sg[e])));
        acc[0][e] = fmaf(dn, si, acc[0][e]);
      }
      store_row<TPR, VEC>(dx + r * D, D, t, ox);
      store_row<TPR, VEC>(dz + r * D, D, t, oz);
    }
  }
  float* const out[1] = {part};
  write_partials<TPR, VEC, 1>(acc, red, out, D);
}

template <int TPR, bool VEC, bool POST, class H>
__global__ void __launch_bounds__(threads_of(TPR))
residual_norm_fwd_kernel(const __nv_bfloat16* __restrict__ y, const H* h, const void* __restrict__ w_post,
                         const void* __restrict__ w_pre, int w_bf16, H* h_out,
                         __nv_bfloat16* __restrict__ x, int64_t rows, int D, float alpha, float eps) {
  constexpr int RPC = threads_of(TPR) / TPR;
  __shared__ float sm[2][threads_of(TPR) / 32][kSums];
  int slot = 0;
  const int t = threadIdx.x % TPR, rg = threadIdx.x / TPR;
  float w1[E], w2[E];
  load_w<TPR, VEC>(w_pre, w_bf16, D, t, w1);
  if (POST) load_w<TPR, VEC>(w_post, w_bf16, D, t, w2);
  const float inv_d = 1.f / (float)D;
  Raw<TPR, VEC, __nv_bfloat16> ny;
  Raw<TPR, VEC, H> nh;
  const int64_t stride = (int64_t)gridDim.x * RPC;
  int64_t r = (int64_t)blockIdx.x * RPC + rg;
  ny.load(y + r * D, r < rows, D, t);
  nh.load(h + r * D, r < rows, D, t);
  for (int64_t r0 = (int64_t)blockIdx.x * RPC; r0 < rows; r0 += stride, r += stride) {
    const bool live = r < rows;
    float yv[E], hv[E];
    ny.get(yv);
    nh.get(hv);
    ny.load(y + (r + stride) * D, r + stride < rows, D, t);
    nh.load(h + (r + stride) * D, r + stride < rows, D, t);
    float ry = 1.f;
    if (POST) {
      float s[1] = {0.f};
#pragma unroll
      for (int e = 0; e < E; ++e) s[0] = fmaf(yv[e], yv[e], s[0]);
      RowSum<TPR, 1>::run(s, sm, slot);
      ry = rsqrtf(fmaf(s[0], inv_d, eps));
    }
    float s[1] = {0.f};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      hv[e] = fmaf(alpha, POST ? yv[e] * ry * w2[e] : yv[e], hv[e]);
      s[0] = fmaf(hv[e], hv[e], s[0]);
    }
    RowSum<TPR, 1>::run(s, sm, slot);
    const float rh = rsqrtf(fmaf(s[0], inv_d, eps));
    if (live) {
      store_row<TPR, VEC>(h_out + r * D, D, t, hv);
#pragma unroll
      for (int e = 0; e < E; ++e) yv[e] = hv[e] * rh * w1[e];
      store_row<TPR, VEC>(x + r * D, D, t, yv);
    }
  }
}

// With m = rms(h'), n = rms(y) (POST), p = dx w_pre:
//   dh = dh' + r_h (p - m mean(p m)),  e = alpha dh,  dw_pre = sum dx m
//   POST: dy = r_y (e w_post - n mean(e w_post n)), dw_post = sum e n;  else dy = e
template <int TPR, bool VEC, bool POST, class H>
__global__ void __launch_bounds__(threads_of(TPR), bwd_per_sm(TPR))
residual_norm_bwd_kernel(const __nv_bfloat16* __restrict__ dx, const H* dh_out,
                         const __nv_bfloat16* __restrict__ y, const H* __restrict__ h, const void* __restrict__ w_post,
                         const void* __restrict__ w_pre, int w_bf16, __nv_bfloat16* __restrict__ dy,
                         H* dh, float* __restrict__ part_pre, float* __restrict__ part_post, int64_t rows,
                         int D, float alpha, float eps) {
  constexpr int RPC = threads_of(TPR) / TPR;
  __shared__ float sm[2][threads_of(TPR) / 32][kSums];
  __shared__ float red[RPC > 1 ? threads_of(TPR) * E : 1];
  int slot = 0;
  dependents_may_start();
  const int t = threadIdx.x % TPR, rg = threadIdx.x / TPR;
  // 1024 threads have 64 registers each: the weights come from L1 for every row, and no row is fetched ahead (207 us
  // at 4096 x 8192, fp32; with both, in spills, 267 us)
  constexpr bool LEAN = TPR == 1024;
  float w1[E], w2[E], acc[2][E] = {};
  auto weights = [&] {
    load_w<TPR, VEC>(w_pre, w_bf16, D, t, w1);
    if (POST) load_w<TPR, VEC>(w_post, w_bf16, D, t, w2);
  };
  if (!LEAN) weights();
  const float inv_d = 1.f / (float)D;
  Raw<TPR, VEC, __nv_bfloat16> ny, nd;
  Raw<TPR, VEC, H> nh, ndh;
  const int64_t stride = (int64_t)gridDim.x * RPC;
  int64_t r = (int64_t)blockIdx.x * RPC + rg;
  auto load = [&](int64_t q) {
    const bool in = q < rows;
    ny.load(y + q * D, in, D, t);
    nh.load(h + q * D, in, D, t);
    nd.load(dx + q * D, in, D, t);
    ndh.load(dh_out + q * D, in && dh_out, D, t);
  };
  if (!LEAN) load(r);
  for (int64_t r0 = (int64_t)blockIdx.x * RPC; r0 < rows; r0 += stride, r += stride) {
    const bool live = r < rows;
    float yv[E], hv[E], dv[E], dhv[E];
    if (LEAN) {
      load(r);
      weights();
    }
    ny.get(yv);
    nh.get(hv);
    nd.get(dv);
    ndh.get(dhv);
    if (!LEAN) load(r + stride);
    // With u = y w_post, p = dx w_pre, a = alpha r_y, h' = h + a u, all sums of the row are polynomials in a of
    // seven sums that need no other first: one reduction instead of three in a row.
    float ry = 1.f, ss, sp, su = 0.f, gu = 0.f, pu = 0.f;   // sums of h' h', p h', h' u, dh' u, p u
    if (POST) {
      float s[7] = {};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float u = yv[e] * w2[e], q = dv[e] * w1[e];
        s[0] = fmaf(yv[e], yv[e], s[0]);
        s[1] = fmaf(hv[e], hv[e], s[1]);
        s[2] = fmaf(hv[e], u, s[2]);
        s[3] = fmaf(u, u, s[3]);
        s[4] = fmaf(q, hv[e], s[4]);
        s[5] = fmaf(q, u, s[5]);
        s[6] = fmaf(dhv[e], u, s[6]);
      }
      RowSum<TPR, 7>::run(s, sm, slot);
      // rows past the end, all zero, add to the weights' gradients too: without a factor of 1 / sqrt(0 + 0)
      ry = live ? rsqrtf(fmaf(s[0], inv_d, eps)) : 0.f;
      const float a = alpha * ry;
      ss = fmaf(a, fmaf(a, s[3], 2.f * s[2]), s[1]);
      sp = fmaf(a, s[5], s[4]);
      su = fmaf(a, s[3], s[2]);
      gu = s[6];
      pu = s[5];
      // where h and a u nearly cancel, h' h' is summed from h' itself. The rows of a warp sum together, and each
      // takes the sums if it is one of those, so that no row's result depends on its neighbours
      const bool small = !(ss >= 0.1f * fmaf(a * a, s[3], s[1])) && live;
#pragma unroll
      for (int e = 0; e < E; ++e) hv[e] = fmaf(a, yv[e] * w2[e], hv[e]);
      if (TPR <= 32 ? __any_sync(0xffffffffu, small) : small) {
        float x[3] = {};
#pragma unroll
        for (int e = 0; e < E; ++e) {
          x[0] = fmaf(hv[e], hv[e], x[0]);
          x[1] = fmaf(dv[e] * w1[e], hv[e], x[1]);
          x[2] = fmaf(hv[e], yv[e] * w2[e], x[2]);
        }
        RowSum<TPR, 3>::run(x, sm, slot);
        if (small) {
          ss = x[0];
          sp = x[1];
          su = x[2];
        }
      }
    } else {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        hv[e] = fmaf(alpha, yv[e], hv[e]);
        s[0] = fmaf(hv[e], hv[e], s[0]);
        s[1] = fmaf(dv[e] * w1[e], hv[e], s[1]);
      }
      RowSum<TPR, 2>::run(s, sm, slot);
      ss = s[0];
      sp = s[1];
    }
    const float rh = live ? rsqrtf(fmaf(ss, inv_d, eps)) : 0.f;
    const float c = sp * inv_d * rh * rh;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      acc[0][e] = fmaf(dv[e], hv[e] * rh, acc[0][e]);
      dhv[e] += rh * fmaf(-c, hv[e], dv[e] * w1[e]);
    }
    if (live) store_row<TPR, VEC>(dh + r * D, D, t, dhv);
    if (POST) {
      const float cy = alpha * (gu + rh * (pu - c * su)) * inv_d * ry * ry;   // mean(e w_post n) r_y
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float en = alpha * dhv[e];
        acc[1][e] = fmaf(en, yv[e] * ry, acc[1][e]);
        yv[e] = ry * fmaf(-cy, yv[e], en * w2[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) yv[e] = alpha * dhv[e];
    }
    if (live) store_row<TPR, VEC>(dy + r * D, D, t, yv);
  }
  float* const out[2] = {part_pre, POST ? part_post : nullptr};
  write_partials<TPR, VEC, 2>(acc, red, out, D);
}

// out[m][d] = the sum of the m-th array's `parts` partial rows, in a fixed order: 32 threads a column, each
// summing every 32nd row, and their sums added through shared memory by one thread, in four running sums.
__global__ void __launch_bounds__(256) sum_partials_kernel(const float* __restrict__ p0, const float* __restrict__ p1,
                                                           float* __restrict__ o0, float* __restrict__ o1, int parts,
                                                           int D) {
  dependency_wait();
  const float* p = blockIdx.y ? p1 : p0;
  float* o = blockIdx.y ? o1 : o0;
  const int cl = threadIdx.x & 7, pl = threadIdx.x >> 3;   // 8 columns x 32 row lanes
  const int d = blockIdx.x * 8 + cl;
  float s = 0.f;
  if (d < D)
    for (int i = pl; i < parts; i += 32) s += p[(int64_t)i * D + d];
  __shared__ float red[32][9];
  red[pl][cl] = s;
  __syncthreads();
  if (threadIdx.x < 8 && d < D) {
    float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 32; ++i) a[i & 3] += red[i][threadIdx.x];
    o[d] = (a[0] + a[1]) + (a[2] + a[3]);
  }
}

constexpr int kSMs = 152;
constexpr int kMaxD = 8192;

int tpr_of(int D) {
  int t = 8;
  while (t * E < D) t *= 2;
  return t;
}
// CTAs of a launch: enough for every row group, at most `per_sm` resident ones per SM.
int64_t grid_of(int64_t rows, int tpr, int per_sm) {
  const int64_t rpc = threads_of(tpr) / tpr;
  const int64_t need = (rows + rpc - 1) / rpc, most = (int64_t)kSMs * per_sm;
  return need < most ? need : most;
}
bool vec_ok(int D, std::initializer_list<const void*> ptrs) {
  if (D % 8) return false;
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 15) return false;
  return true;
}

// Calls f(tpr, vec) with both as compile-time constants.
template <class F>
void dispatch(int tpr, bool vec, F f) {
  auto go = [&](auto t) {
    if (vec) f(t, std::true_type());
    else f(t, std::false_type());
  };
  switch (tpr) {
    case 8: go(std::integral_constant<int, 8>()); break;
    case 16: go(std::integral_constant<int, 16>()); break;
    case 32: go(std::integral_constant<int, 32>()); break;
    case 64: go(std::integral_constant<int, 64>()); break;
    case 128: go(std::integral_constant<int, 128>()); break;
    case 256: go(std::integral_constant<int, 256>()); break;
    case 512: go(std::integral_constant<int, 512>()); break;
    default: go(std::integral_constant<int, 1024>()); break;
  }
}

}  // namespace

bool norm_dim_ok(int D) { return D >= 1 && D <= kMaxD; }

int64_t norm_bwd_parts(int64_t rows, int D) {
  const int tpr = tpr_of(D);
  return grid_of(rows, tpr, bwd_per_sm(tpr));
}

cudaError_t launch_gated_norm_fwd(const void* x, int x_f32, const void* z, const void* w, int w_bf16, void* y,
                                  int64_t rows, int D, float eps, cudaStream_t stream) {
  const int tpr = tpr_of(D);
  const unsigned grid = (unsigned)grid_of(rows, tpr, 2048 / threads_of(tpr));
  const bool vec = vec_ok(D, {x, z, w, y});
  dispatch(tpr, vec, [&](auto T, auto V) {
    constexpr int TPR = decltype(T)::value;
    constexpr bool VEC = decltype(V)::value;
    const auto zb = static_cast<const __nv_bfloat16*>(z);
    const auto yb = static_cast<__nv_bfloat16*>(y);
    if (x_f32)
      gated_norm_fwd_kernel<TPR, VEC, float><<<grid, threads_of(TPR), 0, stream>>>(
          static_cast<const float*>(x), zb, w, w_bf16, yb, rows, D, eps);
    else
      gated_norm_fwd_kernel<TPR, VEC, __nv_bfloat16><<<grid, threads_of(TPR), 0, stream>>>(
          static_cast<const __nv_bfloat16*>(x), zb, w, w_bf16, yb, rows, D, eps);
  });
  return cudaGetLastError();
}

cudaError_t launch_gated_norm_bwd(const void* dy, const void* x, int x_f32, const void* z, const void* w, int w_bf16,
                                  void* dx, void* dz, float* dw, int64_t rows, int D, float eps, float* part,
                                  cudaStream_t stream) {
  const int tpr = tpr_of(D);
  const unsigned grid = (unsigned)norm_bwd_parts(rows, D);
  if (grid == 1) part = dw;   // one CTA's sums are the gradient (10 x 128: the call takes 7.4 us of the host, not 9.6)
  const bool vec = vec_ok(D, {dy, x, z, w, dx, dz, part});
  dispatch(tpr, vec, [&](auto T, auto V) {
    constexpr int TPR = decltype(T)::value;
    constexpr bool VEC = decltype(V)::value;
    const auto dyb = static_cast<const __nv_bfloat16*>(dy), zb = static_cast<const __nv_bfloat16*>(z);
    const auto dzb = static_cast<__nv_bfloat16*>(dz);
    if (x_f32)
      gated_norm_bwd_kernel<TPR, VEC, float><<<grid, threads_of(TPR), 0, stream>>>(
          dyb, static_cast<const float*>(x), zb, w, w_bf16, static_cast<float*>(dx), dzb, part, rows, D, eps);
    else
      gated_norm_bwd_kernel<TPR, VEC, __nv_bfloat16><<<grid, threads_of(TPR), 0, stream>>>(
          dyb, static_cast<const __nv_bfloat16*>(x), zb, w, w_bf16, static_cast<__nv_bfloat16*>(dx), dzb, part, rows, D,
          eps);
  });
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (grid == 1) return cudaSuccess;
  return launch(true, sum_partials_kernel, dim3((D + 7) / 8, 1), 256, 0, stream, (const float*)part,
                (const float*)nullptr, dw, (float*)nullptr, (int)grid, D);
}

cudaError_t launch_residual_norm_fwd(const void* y, const void* h, int h_f32, const void* w_post, const void* w_pre,
                                     int w_bf16, void* h_out, void* x, int64_t rows, int D, float alpha, float eps,
                                     cudaStream_t stream) {
  const int tpr = tpr_of(D);
  const unsigned grid = (unsigned)grid_of(rows, tpr, 2048 / threads_of(tpr));
  const bool vec = vec_ok(D, {y, h, w_post, w_pre, h_out, x});
  dispatch(tpr, vec, [&](auto T, auto V) {
    constexpr int TPR = decltype(T)::value;
    constexpr bool VEC = decltype(V)::value;
    const auto yb = static_cast<const __nv_bfloat16*>(y);
    const auto xb = static_cast<__nv_bfloat16*>(x);
    auto go = [&](auto P, auto* tag) {
      using H = std::remove_pointer_t<decltype(tag)>;
      residual_norm_fwd_kernel<TPR, VEC, decltype(P)::value, H><<<grid, threads_of(TPR), 0, stream>>>(
          yb, static_cast<const H*>(h), w_post, w_pre, w_bf16, static_cast<H*>(h_out), xb, rows, D, alpha, eps);
    };
    if (h_f32) w_post ? go(std::true_type(), (float*)nullptr) : go(std::false_type(), (float*)nullptr);
    else w_post ? go(std::true_type(), (__nv_bfloat16*)nullptr) : go(std::false_type(), (__nv_bfloat16*)nullptr);
  });
  return cudaGetLastError();
}

cudaError_t launch_residual_norm_bwd(const void* dx, const void* dh_out, const void* y, const void* h, int h_f32,
                                     const void* w_post, const void* w_pre, int w_bf16, void* dy, void* dh,
                                     float* dw_post, float* dw_pre, int64_t rows, int D, float alpha, float eps,
                                     float* part, cudaStream_t stream) {
  const int tpr = tpr_of(D);
  const unsigned grid = (unsigned)norm_bwd_parts(rows, D);
  float* part2 = part + (int64_t)grid * D;
  if (grid == 1) {   // one CTA's sums are the gradients
    part = dw_pre;
    part2 = dw_post;
  }
  const bool vec = vec_ok(D, {dx, dh_out, y, h, w_post, w_pre, dy, dh, part, part2});
  dispatch(tpr, vec, [&](auto T, auto V) {
    constexpr int TPR = decltype(T)::value;
    constexpr bool VEC = decltype(V)::value;
    const auto dxb = static_cast<const __nv_bfloat16*>(dx), yb = static_cast<const __nv_bfloat16*>(y);
    const auto dyb = static_cast<__nv_bfloat16*>(dy);
    auto go = [&](auto P, auto* tag) {
      using H = std::remove_pointer_t<decltype(tag)>;
      residual_norm_bwd_kernel<TPR, VEC, decltype(P)::value, H><<<grid, threads_of(TPR), 0, stream>>>(
          dxb, static_cast<const H*>(dh_out), yb, static_cast<const H*>(h), w_post, w_pre, w_bf16, dyb,
          static_cast<H*>(dh), part, part2, rows, D, alpha, eps);
    };
    if (h_f32) w_post ? go(std::true_type(), (float*)nullptr) : go(std::false_type(), (float*)nullptr);
    else w_post ? go(std::true_type(), (__nv_bfloat16*)nullptr) : go(std::false_type(), (__nv_bfloat16*)nullptr);
  });
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (grid == 1) return cudaSuccess;
  return launch(true, sum_partials_kernel, dim3((D + 7) / 8, w_post ? 2 : 1), 256, 0, stream, (const float*)part,
                (const float*)part2, dw_pre, dw_post, (int)grid, D);
}

}  // namespace gdn

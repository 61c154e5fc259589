// la_state.cu -- the states at the chunk boundaries of linear attention with a decay for each head.
//
// Per sequence, value head and 64 (or 128) value columns, over 128-token chunks:
//   forwards  S <- Gam S + sum_i w_i k_i v_i^T,  w_i = exp(gam_C - gam_i),  Gam = exp(gam_C)
//   backwards dS <- Gam dS + sum_t w_t q_t do_t^T,  w_t = scale exp(gam_t),  chunks last to first
// and the state before each chunk's contribution is stored for the output kernel.
//
// The contributions do not depend on the state: each is one tcgen05 product [dk x 128] [128 x NV] into
// a fresh accumulator, and the walk itself is one fp32 multiply-add per state element, held in
// registers. The weights go to the K side, as the A operand in tensor memory: thread = key channel
// reads its column of the K tile, and w_i k_i (fp32) is written as three bf16 terms (24 bits, so the
// state has fp32 accuracy; two terms leave 2^-17 of it), A terms of chunk c + 1 being written while the
// products of chunk c run. V stays as TMA left it (MN-major B operand).
// Tail rows of a partial chunk belong to another sequence, so they are zeroed, not just weighted by zero.
//
// Few sequences and heads: each walk is cut into segments, a first launch computes every segment's
// contribution from a zero state, a scan joins them, and the second launch walks all segments at once
// from their true starting states.
#include <algorithm>

#include "la_chunk.cuh"
#include "kernels.h"

namespace gdn {
namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kStages = 3;
constexpr uint32_t TM_A = 0, TM_ACC = 384;   // two buffers of three 64-column A terms; the accumulator
constexpr uint32_t kTmemCols = 512;

struct Params {
  Seqs seqs;
  GateSrc gates;
  const float* s0;
  float* sT;
  __nv_bfloat16* states;
  float *seg_tot, *seg_dec;
  int* status;
  int Hqk, dk, dv, terms, reverse, nseg;
  int totals;       // this launch computes the segments' contributions
  float scale;
};

template <int NV>
constexpr uint32_t stage_bytes() { return kTile + NV / 64 * kBlk; }
template <int NV>
constexpr uint32_t smem_bytes() { return kStages * stage_bytes<NV>() + 8 * 64 * 4 + 1024; }

template <int NV>
__global__ void __launch_bounds__(kThreads, 1)
la_state_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap ty, const Params p) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[kStages + 1];
  __shared__ uint32_t tmem_slot;
  constexpr int HC = NV / 2;   // value columns a thread
  const uint32_t raw = tc::smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* sm = smem_raw + (sbase - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = warp & 3, half = warp >> 2;
  const uint32_t lane0 = 32u * quad;
  const int row = 32 * quad + lane;        // key channel
  const bool live = row < p.dk;            // dk 64: lanes 64-127 of the product are not used
  float* const ws = reinterpret_cast<float*>(sm + kStages * stage_bytes<NV>()) + warp * 64;

  const int tiles = p.dv / NV;
  int64_t u = blockIdx.x;
  const int vt = (int)(u % tiles);
  u /= tiles;
  const int seg = (int)(u % p.nseg);
  const int64_t unit = u / p.nseg;
  if (p.totals && seg == p.nseg - 1) return;   // nothing follows the last segment
  const int Hv = p.gates.Hv;
  const int n = (int)(unit / Hv), h = (int)(unit % Hv), hq = h / (Hv / p.Hqk);
  const int64_t t0 = p.seqs.start(n), len = p.seqs.len(n), slot0 = p.seqs.slot0(n);
  const int nch = (int)((len + kC - 1) / kC);
  const int per = (nch + p.nseg - 1) / p.nseg;
  const int first = min(seg * per, nch), last = min(first + per, nch);   // walk steps of this CTA
  const int steps = last - first;
  auto chunk_of = [&](int i) { return p.reverse ? nch - 1 - (first + i) : first + i; };
  auto rows_of = [&](int c) { return (int)min((int64_t)kC, len - (int64_t)c * kC); };

  const uint32_t bar_m = tc::smem_u32(&bars[kStages]);
  const uint32_t idesc = tc::make_idesc(tc::kKindBF16, 128, NV, false, true);
  auto load = [&](int i) {
    const uint32_t bar = tc::smem_u32(&bars[i % kStages]), dst = sbase + (i % kStages) * stage_bytes<NV>();
    const int tok = (int)(t0 + (int64_t)chunk_of(i) * kC);
    tc::mbar_expect_tx(bar, p.dk / 64 * kBlk + NV / 64 * kBlk);
    for (int b = 0; b < p.dk / 64; ++b) tc::tma_load_3d(dst + b * kBlk, &tx, bar, 64 * b, hq, tok);
    for (int b = 0; b < NV / 64; ++b) tc::tma_load_3d(dst + kTile + b * kBlk, &ty, bar, vt * NV + 64 * b, h, tok);
  };
  if (tid == 0) {
    for (int i = 0; i <= kStages; ++i) tc::mbar_init(tc::smem_u32(&bars[i]), 1);
    tc::mbar_fence_init();
    for (int i = 0; i < min(2, steps); ++i) load(i);
  }
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&tmem_slot), kTmemCols);
  float gx[4];
  if (steps) p.gates.load(gx, t0 + (int64_t)chunk_of(0) * kC, h, rows_of(chunk_of(0)), lane);

  // state elements (row, vt NV + half HC + j)
  float s[HC];
  const int64_t sbase_g = (unit * p.dk + row) * (int64_t)p.dv + vt * NV + half * HC;
  const int64_t seg_g = ((unit * p.nseg + seg) * p.dk + row) * (int64_t)p.dv + vt * NV + half * HC;
  {
    const float* src = p.totals ? nullptr : p.nseg > 1 ? p.seg_tot + seg_g : p.s0 ? p.s0 + sbase_g : nullptr;
#pragma unroll
    for (int j = 0; j < HC; j += 4) {
      const float4 v = src && live ? *reinterpret_cast<const float4*>(src + j) : make_float4(0.f, 0.f, 0.f, 0.f);
      s[j] = v.x; s[j + 1] = v.y; s[j + 2] = v.z; s[j + 3] = v.w;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // byte offsets of this channel within an 8-row group of the swizzled tile
  uint32_t off[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) off[r] = (row >> 6) * kBlk + tc::sw128(r, (row & 63) * 2);

  bool ok = true;
  int loaded = min(2, steps), waited = 0;   // TMA stages issued / seen complete (thread 0 drains the rest)
  int mma_issued = 0;
  float decay = 1.f;                        // Gam of the chunk whose product is in flight
  float log_decay = 0.f;                    // of the whole segment
  auto take = [&](int i) {                  // the product of step i -> the state
    ok = ok && tc::mbar_wait(bar_m, i & 1);
    tc::tc_fence_after();
    if (live || p.dk == 128) {
#pragma unroll
      for (int q = 0; q < HC / 32; ++q) {
        float v[32];
        ld32(tmem, lane0, TM_ACC + half * HC + 32 * q, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) s[32 * q + j] = fmaf(decay, s[32 * q + j], v[j]);
      }
    }
    tc::tc_fence_before();
  };

  for (int i = 0; i < steps; ++i) {
    const int c = chunk_of(i), L = rows_of(c);
    unsigned char* kt = sm + (i % kStages) * stage_bytes<NV>();
    Gates w;
    scan_gates(gx, w, lane);
    if (i + 1 < steps) {
      const int c1 = chunk_of(i + 1);
      p.gates.load(gx, t0 + (int64_t)c1 * kC, h, rows_of(c1), lane);
    }
    // this warp's 64 weights (tokens 64 half ..) to shared memory
    const float tt[4] = {w.tot(0), w.tot(1), w.tot(2), w.tot(3)};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if ((q >> 1) != half) continue;
      float e = p.reverse ? w.pre(q) : w.after(q);
#pragma unroll
      for (int m = 0; m < 4; ++m)
        if (p.reverse ? m < q : m > q) e += tt[m];
      __syncwarp();
      ws[32 * (q & 1) + lane] = 32 * q + lane < L ? p.scale * expf(e) : 0.f;
    }
    __syncwarp();
    ok = ok && tc::mbar_wait(tc::smem_u32(&bars[i % kStages]), (i / kStages) & 1);
    ++waited;
    if (L < kC) {   // uniform: the tail rows are another sequence's
      zero_tail_rows(kt, p.dk / 64, tid, L);
      zero_tail_rows(kt + kTile, NV / 64, tid, L);
      tc::fence_proxy_async_smem();
      __syncthreads();
    }
    if (live || p.dk == 128) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {   // 32 tokens each
        uint32_t t1[16], t2[16], t3[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const int r = 64 * half + 32 * b + 2 * q;   // (r & 7) is known at compile time: half and b move whole groups
          const unsigned char* g8 = kt + (r >> 3) * 1024;
          const float k0 = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(g8 + off[(2 * q) & 7]) << 16);
          const float k1 = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(g8 + off[(2 * q + 1) & 7]) << 16);
          const float2 wv = *reinterpret_cast<const float2*>(ws + 32 * b + 2 * q);
          const float x0 = k0 * wv.x, x1 = k1 * wv.y;
          t1[q] = pack_bf16(x0, x1);
          const float2 f1 = unpack_bf16(t1[q]);
          const float y0 = x0 - f1.x, y1 = x1 - f1.y;
          t2[q] = pack_bf16(y0, y1);
          const float2 f2 = unpack_bf16(t2[q]);
          t3[q] = pack_bf16(y0 - f2.x, y1 - f2.y);
        }
        const uint32_t at = TM_A + (i & 1) * 192 + 32 * half + 16 * b;
        tmem_st16u(tc::tmem_addr(tmem, lane0, at), t1);
        tmem_st16u(tc::tmem_addr(tmem, lane0, at + 64), t2);
        tmem_st16u(tc::tmem_addr(tmem, lane0, at + 128), t3);
      }
      tc::tmem_st_wait();
    }
    tc::tc_fence_before();
    if (i > 0) take(i - 1);
    decay = expf((tt[0] + tt[1]) + (tt[2] + tt[3]));
    log_decay += (tt[0] + tt[1]) + (tt[2] + tt[3]);
    if (p.states && live) {   // the state before this chunk
      const int64_t item = (slot0 + c) * Hv + h;
      const int64_t term = (int64_t)p.dk * p.dv;
      __nv_bfloat16* dst = p.states + item * p.terms * term +
                           ((int64_t)((vt * NV + half * HC) / 64) * p.dk + row) * 64 + (half * HC) % 64;
#pragma unroll
      for (int j = 0; j < HC; j += 8) {
        uint4 hi, lo;
        split8(s + j, hi, lo);
        const int64_t at = (int64_t)(j / 64) * p.dk * 64 + j % 64;
        *reinterpret_cast<uint4*>(dst + at) = hi;
        if (p.terms == 2) *reinterpret_cast<uint4*>(dst + term + at) = lo;
      }
    }
    if (__syncthreads_or(!ok)) {
      ok = false;
      break;
    }
    if (tid == 0) {
      tc::tc_fence_after();
      const uint64_t bd = tc::make_sdesc(sbase + (i % kStages) * stage_bytes<NV>() + kTile, kBlk, 1024);
#pragma unroll
      for (int t = 0; t < 3; ++t)
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_bf16_ta(tmem + TM_ACC, tmem + TM_A + (i & 1) * 192 + 64 * t + 8 * ks, dadv(bd, ks * 2048), idesc,
                      t + ks > 0);
      tc::mma_commit(bar_m);
      if (i + 2 < steps) {   // its stage held step i - 1, whose product is complete
        load(i + 2);
        ++loaded;
      }
    }
    mma_issued = i + 1;
  }
  if (ok && steps) take(steps - 1);
  if (tid == 0) {
    // nothing of this CTA is in flight when it ends
    for (int i = waited; i < loaded; ++i) tc::mbar_wait(tc::smem_u32(&bars[i % kStages]), (i / kStages) & 1, 1u << 22);
    if (!ok && mma_issued) tc::mbar_wait(bar_m, (mma_issued - 1) & 1, 1u << 22);
  }
  tc::tc_fence_before();
  const bool all_ok = !__syncthreads_or(!ok);
  tc::tc_fence_after();
  if (warp == 0) tc::tmem_dealloc(tmem, kTmemCols);
  if (!all_ok && tid == 0) atomicExch(p.status, 1);
  if (!all_ok || !live) return;
  float* dst = p.totals ? p.seg_tot + seg_g : p.sT && seg == p.nseg - 1 ? p.sT + sbase_g : nullptr;
  if (dst)
#pragma unroll
    for (int j = 0; j < HC; j += 4) *reinterpret_cast<float4*>(dst + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
  if (p.totals && tid == 0 && vt == 0) p.seg_dec[unit * p.nseg + seg] = expf(log_decay);
}

// Segment contributions -> the state that each segment starts from (in place), element by element.
__global__ void __launch_bounds__(256) la_join_kernel(float* seg_tot, const float* seg_dec, const float* s0, int nseg,
                                                      int64_t elems) {
  const int64_t unit = blockIdx.y;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;   // four state elements
  if (e * 4 >= elems) return;
  float4 s = s0 ? reinterpret_cast<const float4*>(s0 + unit * elems)[e] : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < nseg; ++i) {
    float4* at = reinterpret_cast<float4*>(seg_tot + (unit * nseg + i) * elems) + e;
    const float d = seg_dec[unit * nseg + i];
    const float4 x = i + 1 < nseg ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
    *at = s;
    s = make_float4(fmaf(d, s.x, x.x), fmaf(d, s.y, x.y), fmaf(d, s.z, x.z), fmaf(d, s.w, x.w));
  }
}

constexpr int kSMs = 152;

template <int NV>
cudaError_t run(const CUtensorMap& tx, const CUtensorMap& ty, const Params& p, int64_t units, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(la_state_kernel<NV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       smem_bytes<NV>());
  if (e != cudaSuccess) return e;
  la_state_kernel<NV><<<(unsigned)(units * p.nseg * (p.dv / NV)), kThreads, smem_bytes<NV>(), stream>>>(tx, ty, p);
  return cudaGetLastError();
}

}  // namespace

int64_t la_slots(const LaProblem& p) { return (int64_t)p.B * p.T / kC + p.N; }

// One CTA of a walk runs per SM. Splitting walks costs a second pass over K and V, so it is done only
// when half of the SMs or fewer have one, and then a segment keeps at least 4 chunks.
int state_segments(const LaProblem& p) {
  const int64_t walks = (int64_t)p.N * p.Hv * (p.dv / 64);
  if (walks == 0 || walks > kSMs / 2) return 1;
  int64_t longest = p.T;
  if (p.cu_host) {
    longest = 0;
    for (int n = 0; n < p.N; ++n) longest = std::max<int64_t>(longest, p.cu_host[n + 1] - p.cu_host[n]);
  }
  const int64_t chunks = (longest + kC - 1) / kC;
  return (int)std::max<int64_t>(1, std::min<int64_t>(kSMs / walks, chunks / 4));
}

cudaError_t launch_states(const LaProblem& p, const StateRun& r, int* status, cudaStream_t stream) {
  const int64_t units = (int64_t)p.N * p.Hv, tokens = (int64_t)p.B * p.T;
  if (units == 0) return cudaSuccess;
  const int64_t elems = (int64_t)p.dk * p.dv;
  if (tokens == 0) {   // no chunk anywhere: the final state is the first
    if (!r.sT || r.sT == r.s0) return cudaSuccess;
    return r.s0 ? cudaMemcpyAsync(r.sT, r.s0, units * elems * 4, cudaMemcpyDeviceToDevice, stream)
                : cudaMemsetAsync(r.sT, 0, units * elems * 4, stream);
  }
  CUtensorMap tx, ty;
  if (!make_bf16_map(&tx, r.x, p.dk, p.Hqk, tokens, kC) || !make_bf16_map(&ty, r.y, p.dv, p.Hv, tokens, kC))
    return cudaErrorNotSupported;
  Params s{{p.cu, p.T, p.N}, {p.g, p.Hv, p.head_decay}, r.s0, r.sT, (__nv_bfloat16*)r.states, r.seg_tot, r.seg_dec,
           status, p.Hqk, p.dk, p.dv, r.terms, r.reverse, state_segments(p), 0, r.scale};
  // a tile of 128 value columns weights K once for both halves, but has half as many CTAs
  const bool wide = p.dv == 128 && units * s.nseg >= kSMs;
  auto go = [&] { return wide ? run<128>(tx, ty, s, units, stream) : run<64>(tx, ty, s, units, stream); };
  if (s.nseg > 1) {
    s.totals = 1;
    s.states = nullptr;
    cudaError_t e = go();
    if (e != cudaSuccess) return e;
    la_join_kernel<<<dim3((unsigned)((elems / 4 + 255) / 256), (unsigned)units), 256, 0, stream>>>(
        r.seg_tot, r.seg_dec, r.s0, s.nseg, elems);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    s.totals = 0;
    s.states = (__nv_bfloat16*)r.states;
  }
  return go();
}

}  // namespace la
}  // namespace gdn

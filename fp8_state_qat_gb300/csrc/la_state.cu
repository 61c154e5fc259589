// la_state.cu -- the states at the chunk boundaries of linear attention with a decay for each head.
//
// Per sequence, value head and 64 value columns, over 128-token chunks:
//   forwards  S <- Gam S + sum_i w_i k_i v_i^T,  w_i = exp(gam_C - gam_i),  Gam = exp(gam_C)
//   backwards dS <- Gam dS + sum_t w_t q_t do_t^T,  w_t = scale exp(gam_t),  chunks last to first
// and the state before each chunk's contribution is stored for the output kernel.
//
// The contributions do not depend on the state: each is one tcgen05 product [dk x 128] [128 x 64] into a
// fresh accumulator, and the walk itself is one fp32 multiply-add per state element, held in registers.
// K stays as TMA left it (MN-major A operand). The weights go to the V side: w_i v_i (fp32) is written as
// three bf16 terms (24 bits, so the state has fp32 accuracy; two terms leave 2^-17 of it), in V's own
// swizzled places, so that a thread moves 16 bytes at a time and nothing is transposed. (Weighting K instead,
// through tensor memory, takes a 16-bit load an element and twice the elements: 64 us against 56.)
// The terms of chunk c + 1 are written while the products of chunk c run.
// Tail rows of a partial chunk belong to another sequence, so they are zeroed, not just weighted by zero.
//
// Few sequences and heads: each walk is cut into segments, a first launch computes every segment's
// contribution from a zero state, a scan joins them, and the second launch walks all segments at once
// from their true starting states.
//
// At 4 x 4096 tokens, 16 heads, d 128 (128 CTAs of 32 steps, cold): S 55 us, dS 76 us (with S read again for <S, dS>).
// Bound by the length of a step, a chain of hand-overs: 2.4 k cycles, of which the products take 1.0 k and V's
// conversion 1.4 k side by side. Not by traffic (48 KB in and 32 to 64 KB out or in again a step, 4 to 5 TB/s of DRAM): with K sent
// once to both value tiles' CTAs, a third of the loads less, it took longer, each step waiting for the slower of the two.
#include <algorithm>

#include "la_chunk.cuh"
#include "kernels.h"

namespace gdn {
namespace la {
namespace {

constexpr int kThreads = 640;                // warps 0-7 state, 8-15 V's terms, 16 products, 17, 18 weights, 19 states out
constexpr int kNV = 64;                      // value columns of a CTA
constexpr int kHC = kNV / 2;                 // of a thread of the state
constexpr uint32_t kTmemCols = 128;          // two accumulators
// shared memory: two K tiles, two V tiles, one or two sets of V's terms, the states on their way out, S
constexpr uint32_t kOffV = 2 * kTile, kOffTerm = kOffV + 2 * kBlk, kTermSet = 3 * kBlk;

struct Params {
  Seqs seqs;
  GateSrc gates;
  const float* s0;
  float* sT;
  float *seg_tot, *seg_dec;
  float* edge;
  int* status;
  int Hqk, dk, dv, reverse, nseg;
  int totals;       // this launch computes the segments' contributions
  int store, other; // the states are stored; <S, state> is computed
  int sets;         // of V's terms: 2, or 1 where S needs the room
  float scale;
  int beside;       // the kernel before this one need only be done when this one is
  int sorted;
  uint8_t order[64];   // the sequences, longest first
};
__host__ __device__ inline uint32_t off_out(const Params& p) { return kOffTerm + p.sets * kTermSet; }
__host__ __device__ inline uint32_t off_other(const Params& p) { return off_out(p) + (p.store ? 2 * kBlk : 0); }
inline uint32_t smem_bytes(const Params& p) { return off_other(p) + (p.other ? 2 * kBlk : 0) + 1024; }
constexpr uint32_t kMaxSmem = kOffTerm + 2 * kTermSet + 2 * kBlk + 1024;

constexpr int kW = 3;   // weights are computed up to three steps ahead
struct Shared {
  uint64_t kfull[2], vfull[2];   // a step's tiles have landed
  uint64_t wready[kW], wfree[kW];   // its weights are written; are read
  uint64_t aready[2];            // its terms are written (and V is read)
  uint64_t mma[2], accfree[2];   // its product is complete; is taken
  uint64_t sready, sfree;        // the state is laid out for its way out; has been read from there
  uint64_t ofull, oread;         // S of the step has landed; is read
  uint32_t tmem;
  int dead;
  float decay[kW], log_decay[2];   // Gam of a step; log Gam of the whole segment, in two parts
  __align__(16) float w[kW][kC];
};

// 8 values -> three bf16 terms each
__device__ __forceinline__ void split3(const float2 (&x)[4], uint4& t1, uint4& t2, uint4& t3) {
  const float2 neg = make_float2(-1.f, -1.f);
  uint32_t a[4], b[4], c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = pack_bf16(x[i].x, x[i].y);
    const float2 y = __ffma2_rn(unpack_bf16(a[i]), neg, x[i]);
    b[i] = pack_bf16(y.x, y.y);
    const float2 z = __ffma2_rn(unpack_bf16(b[i]), neg, y);
    c[i] = pack_bf16(z.x, z.y);
  }
  t1 = make_uint4(a[0], a[1], a[2], a[3]);
  t2 = make_uint4(b[0], b[1], b[2], b[3]);
  t3 = make_uint4(c[0], c[1], c[2], c[3]);
}

// Each group of warps walks the steps at its own pace: V's terms of a step are written while the products of
// the step before run and the state takes those of the step before that. Two warps compute the weights, of
// every other step each: the latency of a step's loads and sums is longer than the step.
__global__ void __launch_bounds__(kThreads, 1)
la_state_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap ty,
                const __grid_constant__ CUtensorMap ts, const __grid_constant__ CUtensorMap to,
                const __grid_constant__ Params p) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(16) Shared sh;
  const uint32_t raw = tc::smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* sm = smem_raw + (sbase - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = warp & 3, part = (warp >> 2) & 1;
  const uint32_t lane0 = 32u * quad;
  const int row = 32 * quad + lane;        // key channel
  const bool live = row < p.dk;            // dk 64: lanes 64-127 of the product are not used

  dependents_may_start();
  const int tiles = p.dv / kNV;
  int u = blockIdx.x;
  const int vt = u % tiles;
  u /= tiles;
  const int seg = u % p.nseg;
  u /= p.nseg;
  if (p.totals && seg == p.nseg - 1) {   // nothing follows the last segment
    dependency_wait();
    return;
  }
  const int Hv = p.gates.Hv;
  const int n = p.sorted ? p.order[u / Hv] : u / Hv, h = u % Hv, unit = n * Hv + h, hq = h / (Hv / p.Hqk);
  const int t0 = (int)p.seqs.start(n), len = (int)p.seqs.len(n), slot0 = (int)p.seqs.slot0(n);
  const int nch = len / kC + (len % kC != 0);
  const int per = (nch + p.nseg - 1) / p.nseg;
  const int first = min(seg * per, nch), last = min(first + per, nch);   // walk steps of this CTA
  const int steps = last - first;
  auto chunk_of = [&](int i) { return p.reverse ? nch - 1 - (first + i) : first + i; };
  auto rows_of = [&](int c) { return min(kC, len - c * kC); };

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tc::smem_u32(&sh.kfull[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh.vfull[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh.aready[i]), 8);
      tc::mbar_init(tc::smem_u32(&sh.mma[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh.accfree[i]), 8);
    }
    for (int i = 0; i < kW; ++i) {
      tc::mbar_init(tc::smem_u32(&sh.wready[i]), 32);
      tc::mbar_init(tc::smem_u32(&sh.wfree[i]), 16);
    }
    tc::mbar_init(tc::smem_u32(&sh.sready), 8);
    tc::mbar_init(tc::smem_u32(&sh.sfree), 1);
    tc::mbar_init(tc::smem_u32(&sh.ofull), 1);
    tc::mbar_init(tc::smem_u32(&sh.oread), 8);
    tc::mbar_fence_init();
    sh.dead = 0;
  }
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&sh.tmem), kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  bool ok = true;
  // inputs of the call are read above and below without waiting; what a kernel of this call wrote (the joined
  // segment states, S) and what it may still read (the workspace) only after
  if (!p.beside) dependency_wait();

  float s[kHC];   // state elements (row, vt kNV + part kHC + j)
  const int64_t sbase_g = ((int64_t)unit * p.dk + row) * p.dv + vt * kNV + part * kHC;
  const int64_t seg_g = (((int64_t)unit * p.nseg + seg) * p.dk + row) * p.dv + vt * kNV + part * kHC;

  auto token = [&](int i) { return t0 + chunk_of(i) * kC; };
  if (warp == 16) {
    // ---- token tiles and products ----
    constexpr uint32_t idesc = tc::make_idesc(tc::kKindBF16, 128, kNV, true, true);
    const uint32_t me = elect_one();
    const bool two = p.dk == 128;
    const uint32_t kbytes = two ? kTile : kBlk;
    auto load_k = [&](int i) {
      const uint32_t bar = tc::smem_u32(&sh.kfull[i & 1]), dst = sbase + (i & 1) * kTile;
      const int tok = token(i);
      mbar_expect_w(bar, kbytes, me);
      tma_load_3d_w(dst, &tx, bar, 0, hq, tok, me);
      if (two) tma_load_3d_w(dst + kBlk, &tx, bar, 64, hq, tok, me);
    };
    auto load_v = [&](int i) {
      const uint32_t bar = tc::smem_u32(&sh.vfull[i & 1]);
      mbar_expect_w(bar, kBlk, me);
      tma_load_3d_w(sbase + kOffV + (i & 1) * kBlk, &ty, bar, vt * kNV, h, token(i), me);
    };
    const int ks0 = min(2, steps);
    int ks = ks0, vs = ks0, issued = 0;   // loads and products issued
    for (int i = 0; i < ks0; ++i) {
      load_v(i);
      load_k(i);
    }
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      const uint32_t turn = (i >> 1) & 1;
      ok = wait(sh.dead, sh.aready[i & 1], turn);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      if (i + 2 < steps) {   // V of this step is weighted
        load_v(i + 2);
        ++vs;
      }
      ok = wait(sh.dead, sh.accfree[i & 1], turn ^ 1) && wait(sh.dead, sh.kfull[i & 1], turn);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      tc::tc_fence_after();
      const uint64_t ad = tc::make_sdesc(sbase + (i & 1) * kTile, kBlk, 1024);
      const uint64_t bd = tc::make_sdesc(sbase + kOffTerm + (p.sets == 2 ? (i & 1) * kTermSet : 0), kBlk, 1024);
#pragma unroll
      for (int t = 0; t < 3; ++t)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_bf16_w(tmem + (i & 1) * kNV, dadv(ad, k * 2048), dadv(bd, t * kBlk + k * 2048), idesc, t + k > 0, me);
      mma_commit_w(tc::smem_u32(&sh.mma[i & 1]), me);
      issued = i + 1;
      if (i + 2 < steps) {   // K is free when its product is complete
        ok = wait(sh.dead, sh.mma[i & 1], turn);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        load_k(i + 2);
        ++ks;
      }
    }
    if (lane == 0 && !ok) {   // nothing of this CTA is in flight when it ends
      for (int i = max(0, ks - 2); i < ks; ++i) tc::mbar_wait(tc::smem_u32(&sh.kfull[i & 1]), (i >> 1) & 1, 1u << 22);
      for (int i = max(0, vs - 2); i < vs; ++i) tc::mbar_wait(tc::smem_u32(&sh.vfull[i & 1]), (i >> 1) & 1, 1u << 22);
      if (issued) tc::mbar_wait(tc::smem_u32(&sh.mma[(issued - 1) & 1]), ((issued - 1) >> 1) & 1, 1u << 22);
    }
  } else if (warp == 19) {
    // ---- states out, S in ----
    auto state_row = [&](int i, int term) {   // of the stored states: this value tile's rows
      const int item = (slot0 + chunk_of(i)) * Hv + h;
      return ((item * 2 + term) * tiles + vt) * p.dk;
    };
    auto load_other = [&](int i) {
      tc::mbar_expect_tx(tc::smem_u32(&sh.ofull), 2 * p.dk * 128);
      for (int t = 0; t < 2; ++t)
        tc::tma_load_2d(sbase + off_other(p) + t * kBlk, &to, tc::smem_u32(&sh.ofull), 0, state_row(i, t));
    };
    int os = 0;
    if (p.other && steps) {
      if (lane == 0) load_other(0);
      os = 1;
    }
#pragma unroll 1
    for (int i = 0; i < steps && p.store; ++i) {
      ok = wait(sh.dead, sh.sready, i & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      if (lane == 0) {
        for (int t = 0; t < 2; ++t)
          tc::tma_store_2d(&ts, sbase + off_out(p) + t * kBlk, 0, state_row(i, t));
        tc::bulk_commit();
      }
      __syncwarp();
      if (p.other && i + 1 < steps) {
        ok = wait(sh.dead, sh.oread, i & 1);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (lane == 0) load_other(i + 1);
        ++os;
      }
      if (lane == 0) {
        tc::bulk_wait_read();
        tc::mbar_arrive(tc::smem_u32(&sh.sfree));
      }
      __syncwarp();
    }
    if (lane == 0 && !ok) {
      if (os) tc::mbar_wait(tc::smem_u32(&sh.ofull), (os - 1) & 1, 1u << 22);
      tc::bulk_wait_read();
    }
  } else if (warp > 16) {
    // ---- weights ----
    const int which = warp - 17;
    float gx[4], log_decay = 0.f;   // of this warp's steps
    auto gates = [&](int i) { p.gates.load(gx, t0 + (int64_t)chunk_of(i) * kC, h, rows_of(chunk_of(i)), lane); };
    if (which < steps) gates(which);
    for (int i = which; i < steps; i += 2) {
      ok = wait(sh.dead, sh.wfree[i % kW], ((i / kW) & 1) ^ 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const int L = rows_of(chunk_of(i));
      Gates w;
      scan_gates(gx, w, lane);
      if (i + 2 < steps) gates(i + 2);
      const float all = (w.tot(0) + w.tot(1)) + (w.tot(2) + w.tot(3));
      const float far = p.reverse ? w.blocks_before(lane) : w.blocks_after(lane);
      float v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        v[q] = 4 * lane + q < L ? p.scale * expf((p.reverse ? w.pre(q) : w.after(q)) + far) : 0.f;
      *reinterpret_cast<float4*>(&sh.w[i % kW][4 * lane]) = make_float4(v[0], v[1], v[2], v[3]);
      if (lane == 0) sh.decay[i % kW] = expf(all);
      log_decay += all;
      tc::mbar_arrive(tc::smem_u32(&sh.wready[i % kW]));
    }
    if (lane == 0) sh.log_decay[which] = log_decay;
  } else if (warp >= 8) {
    // ---- V's terms: this thread's 16-byte pieces, rows r, r + 32, .. of piece tid % 8 ----
    const int vrow = (tid - 256) >> 3;
    const uint32_t voff = tc::sw128(vrow, (tid & 7) * 16);
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      const int L = rows_of(chunk_of(i));
      ok = wait(sh.dead, sh.vfull[i & 1], (i >> 1) & 1) && wait(sh.dead, sh.wready[i % kW], (i / kW) & 1);
      // the products that read this set of terms before are complete
      if (i >= p.sets) ok = ok && wait(sh.dead, sh.mma[(i - p.sets) & 1], ((i - p.sets) >> 1) & 1);
      const unsigned char* v = sm + kOffV + (i & 1) * kBlk + voff;
      unsigned char* t = sm + kOffTerm + (p.sets == 2 ? (i & 1) * kTermSet : 0) + voff;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = sh.w[i % kW][vrow + 32 * e];
        uint4 q = *reinterpret_cast<const uint4*>(v + 4096 * e);
        if (vrow + 32 * e >= L) q = make_uint4(0, 0, 0, 0);   // another sequence's
        const float2 w2 = make_float2(w, w);
        const float2 x[4] = {__fmul2_rn(unpack_bf16(q.x), w2), __fmul2_rn(unpack_bf16(q.y), w2),
                             __fmul2_rn(unpack_bf16(q.z), w2), __fmul2_rn(unpack_bf16(q.w), w2)};
        uint4 t1, t2, t3;
        split3(x, t1, t2, t3);
        *reinterpret_cast<uint4*>(t + 4096 * e) = t1;
        *reinterpret_cast<uint4*>(t + 4096 * e + kBlk) = t2;
        *reinterpret_cast<uint4*>(t + 4096 * e + 2 * kBlk) = t3;
      }
      if (L < kC) {   // uniform: K's tail rows would meet zero weights, but not with a NaN
        ok = ok && wait(sh.dead, sh.kfull[i & 1], (i >> 1) & 1);
        zero_tail_rows(sm + (i & 1) * kTile, p.dk / 64, tid - 256, L);
      }
      tc::fence_proxy_async_smem();
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(tc::smem_u32(&sh.wfree[i % kW]));
        tc::mbar_arrive(tc::smem_u32(&sh.aready[i & 1]));
      }
    }
  } else {
    // ---- the state ----
    const float* src = p.totals ? nullptr : p.nseg > 1 ? p.seg_tot + seg_g : p.s0 ? p.s0 + sbase_g : nullptr;
#pragma unroll
    for (int j = 0; j < kHC; j += 4) {
      const float4 v = src && live ? *reinterpret_cast<const float4*>(src + j) : make_float4(0.f, 0.f, 0.f, 0.f);
      s[j] = v.x; s[j + 1] = v.y; s[j + 2] = v.z; s[j + 3] = v.w;
    }
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      const int c = chunk_of(i);
      if (p.store) {   // the state before this chunk, as 128-byte swizzled rows of 64 columns
        if (i > 0) ok = wait(sh.dead, sh.sfree, (i - 1) & 1);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (live) {
#pragma unroll
          for (int j = 0; j < kHC; j += 8) {
            unsigned char* at = sm + off_out(p) + tc::sw128(row, (part * kHC + j) * 2);
            uint4 hi, lo;
            split8(s + j, hi, lo);
            *reinterpret_cast<uint4*>(at) = hi;
            *reinterpret_cast<uint4*>(at + kBlk) = lo;
          }
          tc::fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.sready));
      }
      float2 x = make_float2(0.f, 0.f);
      if (p.other) {
        ok = wait(sh.dead, sh.ofull, i & 1);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (live) {
#pragma unroll
          for (int j = 0; j < kHC; j += 8) {
            const unsigned char* at = sm + off_other(p) + tc::sw128(row, (part * kHC + j) * 2);
            const uint4 hv = *reinterpret_cast<const uint4*>(at), lv = *reinterpret_cast<const uint4*>(at + kBlk);
            const uint32_t hu[4] = {hv.x, hv.y, hv.z, hv.w}, lu[4] = {lv.x, lv.y, lv.z, lv.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
              x = __ffma2_rn(__fadd2_rn(unpack_bf16(hu[q]), unpack_bf16(lu[q])),
                             make_float2(s[j + 2 * q], s[j + 2 * q + 1]), x);
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.oread));
      }
      ok = wait(sh.dead, sh.wready[i % kW], (i / kW) & 1);
      const float decay = sh.decay[i % kW];
      if (p.other) {
        const float sum = warp_sum(x.x + x.y);
        if (lane == 0) p.edge[(((int64_t)(slot0 + c) * Hv + h) * tiles + vt) * 8 + warp] = decay * sum;
      }
      ok = ok && wait(sh.dead, sh.mma[i & 1], (i >> 1) & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      tc::tc_fence_after();
      if (32 * quad < p.dk) {   // uniform in the warp
        float v[kHC];
        ld32(tmem, lane0, (i & 1) * kNV + part * kHC, v);
        const float2 d2 = make_float2(decay, decay);
#pragma unroll
        for (int j = 0; j < kHC; j += 2) {
          const float2 r = __ffma2_rn(d2, make_float2(s[j], s[j + 1]), make_float2(v[j], v[j + 1]));
          s[j] = r.x;
          s[j + 1] = r.y;
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(tc::smem_u32(&sh.wfree[i % kW]));
        tc::mbar_arrive(tc::smem_u32(&sh.accfree[i & 1]));
      }
    }
  }
  if (!ok) {
    *(volatile int*)&sh.dead = 1;
    atomicExch(p.status, 1);
  }
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 0) tc::tmem_dealloc(tmem, kTmemCols);
  if (p.beside) dependency_wait();   // what comes next waits for this kernel alone
  if (sh.dead) return;
  if (warp >= 8) {
    if (p.totals && tid == 256 && vt == 0) p.seg_dec[unit * p.nseg + seg] = expf(sh.log_decay[0] + sh.log_decay[1]);
    return;
  }
  float* dst = p.totals ? p.seg_tot + seg_g : p.sT && seg == p.nseg - 1 ? p.sT + sbase_g : nullptr;
  if (dst && live)
#pragma unroll
    for (int j = 0; j < kHC; j += 4) *reinterpret_cast<float4*>(dst + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
}

// Segment contributions -> the state that each segment starts from (in place), element by element; eight
// segments' loads are in flight at a time.
__global__ void __launch_bounds__(256) la_join_kernel(float* seg_tot, const float* seg_dec, const float* s0, int nseg,
                                                      int elems) {
  const int64_t unit = blockIdx.y;
  const int e = blockIdx.x * 256 + threadIdx.x;
  dependents_may_start();
  dependency_wait();
  if (e >= elems) return;
  float s = s0 ? s0[unit * elems + e] : 0.f;
  float* at = seg_tot + unit * nseg * elems + e;
  const float* dec = seg_dec + unit * nseg;
  for (int i0 = 0; i0 < nseg; i0 += 8) {
    float x[8], d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {   // the last segment's contribution is not computed, nor needed
      x[j] = i0 + j + 1 < nseg ? at[(int64_t)(i0 + j) * elems] : 0.f;
      d[j] = i0 + j + 1 < nseg ? dec[i0 + j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i0 + j < nseg) {
        at[(int64_t)(i0 + j) * elems] = s;
        s = fmaf(d[j], s, x[j]);
      }
  }
}

constexpr int kSMs = 152;

}  // namespace

int64_t la_slots(const LaProblem& p) { return (int64_t)p.B * p.T / kC + p.N; }

// One CTA of a walk runs per SM, and a split walk takes two passes over K and V and a join. Forward at one
// sequence, d 128, whole walks against split ones: T 16384, 16 walks, 9 segments 211 -> 91 us; 50 walks, 3
// segments 276 -> 236 us; 60 walks, 2 segments 295 -> 305 us; T 4096, 8 walks, 8 segments 56 -> 35 us; 50
// walks, 3 segments 83 -> 77 us; T 1024, 8 walks, 2 segments 26 -> 33 us. So a walk is split into three segments or more
// or not at all, and a segment keeps at least 4 chunks.
static int segments_of(const LaProblem& p, int64_t longest) {
  const int64_t walks = (int64_t)p.N * p.Hv * (p.dv / kNV);
  if (walks == 0 || walks > kSMs / 3) return 1;
  const int64_t chunks = (longest + kC - 1) / kC, most = std::min<int64_t>(kSMs / walks, chunks / 4);
  return most >= 3 ? (int)most : 1;
}
int state_segments(const LaProblem& p) {
  int64_t longest = p.T;
  if (p.cu_host) {
    longest = 0;
    for (int n = 0; n < p.N; ++n) longest = std::max<int64_t>(longest, p.cu_host[n + 1] - p.cu_host[n]);
  }
  return segments_of(p, longest);
}
int most_segments(const LaProblem& p) { return segments_of(p, p.T); }

// Few walks leave room for the backwards walk beside the forwards one: it then starts with it, and <S, dS>, which
// it would take from the stored S on its way, is left to the dg kernel. A training step at 5 packed sequences of 1 to
// 1000 tokens, 4 heads (40 CTAs): 82 -> 75 us; 3 x 1000 tokens, 8 heads, d 64 (24): 89 -> 78; 2 x 2048, 18 heads, d 128
// (72): 181 -> 180; at 4 x 1024, 16 heads (128, of which 24 find a free SM): 144 -> 171, so only where all have one.
bool walks_beside(const LaProblem& p) {
  return state_segments(p) == 1 && 2 * (int64_t)p.N * p.Hv * (p.dv / kNV) <= kSMs;
}

int edge_parts(const LaProblem& p) { return p.dv / kNV * 8; }

cudaError_t launch_states(const LaProblem& p, const StateRun& r, int* status, bool dependent, cudaStream_t stream) {
  const int64_t units = (int64_t)p.N * p.Hv, tokens = (int64_t)p.B * p.T;
  if (units == 0) return cudaSuccess;
  const int64_t elems = (int64_t)p.dk * p.dv;
  if (tokens == 0) {   // no chunk anywhere: the final state is the first
    if (!r.sT || r.sT == r.s0) return cudaSuccess;
    return r.s0 ? cudaMemcpyAsync(r.sT, r.s0, units * elems * 4, cudaMemcpyDeviceToDevice, stream)
                : cudaMemsetAsync(r.sT, 0, units * elems * 4, stream);
  }
  CUtensorMap m[4];
  if (!make_bf16_map(&m[0], r.x, p.dk, p.Hqk, tokens, kC) || !make_bf16_map(&m[1], r.y, p.dv, p.Hv, tokens, kC))
    return cudaErrorNotSupported;
  m[2] = m[3] = m[0];   // where not used
  const int64_t rows = la_slots(p) * p.Hv * p.dk * (p.dv / 64);   // of one term
  if (r.states && !make_bf16_rows_map(&m[2], r.states, rows * 2, p.dk)) return cudaErrorNotSupported;
  if (r.other && !make_bf16_rows_map(&m[3], r.other, rows * 2, p.dk)) return cudaErrorNotSupported;
  Params s{{p.cu, p.T, p.N}, {p.g, p.Hv, p.head_decay}, r.s0, r.sT, r.seg_tot, r.seg_dec, r.edge,
           status, p.Hqk, p.dk, p.dv, r.reverse, state_segments(p), 0, r.states != nullptr, r.other != nullptr,
           r.other ? 1 : 2, r.scale, r.beside};
  // Walks of unequal lengths: the longest first, so that the last ones to start are short (63 sequences of 128 tokens and
  // one of 16384 that comes last, 16 heads: 286 us, in the caller's order 367). The order of up to 64 fits the
  // launch's parameters; from 65 on it is the caller's, and a long one that comes last runs alone.
  if (p.cu_host && p.N <= 64) {
    s.sorted = 1;
    for (int i = 0; i < p.N; ++i) s.order[i] = (uint8_t)i;
    std::sort(s.order, s.order + p.N, [&](uint8_t a, uint8_t b) {
      const int32_t x = p.cu_host[a + 1] - p.cu_host[a], y = p.cu_host[b + 1] - p.cu_host[b];
      return x != y ? x > y : a < b;
    });
  }
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(la_state_kernel, kMaxSmem, allowed);
  if (e != cudaSuccess) return e;
  auto go = [&] {
    return launch(dependent, la_state_kernel, dim3((unsigned)(units * s.nseg * (p.dv / kNV))), kThreads, smem_bytes(s),
                  stream, m[0], m[1], m[2], m[3], s);
  };
  if (s.nseg > 1) {
    s.totals = 1;
    s.store = s.other = 0;
    if ((e = go()) != cudaSuccess) return e;
    e = launch(true, la_join_kernel, dim3((unsigned)((elems + 255) / 256), (unsigned)units), 256, 0, stream, r.seg_tot,
               (const float*)r.seg_dec, r.s0, s.nseg, (int)elems);
    if (e != cudaSuccess) return e;
    dependent = true;
    s.totals = 0;
    s.store = r.states != nullptr;
    s.other = r.other != nullptr;
  }
  return go();
}

}  // namespace la
}  // namespace gdn

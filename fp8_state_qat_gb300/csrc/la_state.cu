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
// state has fp32 accuracy; two terms leave 2^-17 of it), the A terms of chunk c + 1 while the products of
// chunk c run. That splitting is what the kernel spends its time on (about 7 instructions per K element and
// value tile), so 16 warps do it. V stays as TMA left it (MN-major B operand).
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

constexpr int kWorkers = 512, kThreads = kWorkers + 96;
constexpr int kStages = 3;
constexpr uint32_t TM_A = 0, TM_ACC = 384;   // two buffers of three 64-column A terms; the accumulator
constexpr uint32_t kTmemCols = 512;

struct Params {
  Seqs seqs;
  GateSrc gates;
  const float* s0;
  float* sT;
  float *seg_tot, *seg_dec;
  float* edge;
  int* status;
  int Hqk, dk, dv, terms, reverse, nseg;
  int totals;       // this launch computes the segments' contributions
  int store, other; // the states are stored; <S, state> is computed
  float scale;
  int sorted;
  uint8_t order[64];   // the sequences, longest first
};

template <int NV>
constexpr uint32_t stage_bytes() { return kTile + NV / 64 * kBlk; }
template <int NV>
constexpr uint32_t off_stage() { return kStages * stage_bytes<NV>(); }   // states on their way out: 32 KB
template <int NV>
constexpr uint32_t off_other() { return off_stage<NV>() + kTile; }         // S of the chunk, hi and lo (NV 64)
template <int NV>
constexpr uint32_t smem_bytes() { return off_other<NV>() + (NV == 64 ? kTile : 0) + 1024; }

struct Shared {
  uint64_t full[kStages];   // a step's tiles have landed
  uint64_t wready[2];       // its weights are written
  uint64_t wfree[2];        // and read
  uint64_t aready;          // its A terms are written and the accumulator of the step before is read
  uint64_t mma;             // its product is complete
  uint64_t sfree;           // the states written out are read from shared memory
  uint64_t ofull, oread;    // S of the step has landed; is read
  uint32_t tmem;
  int dead;
  float decay[2], log_decay[2];   // Gam of a step; log Gam of the whole segment, in two parts
  __align__(16) float w[2][kC];   // read and written 16 bytes at a time
};

// Warps 0-15 weight K and hold the state; warp 16 loads and issues the products; warps 17
// and 18 compute the weights, of every other step each: the latency of a step's loads and sums is longer than
// the step.
template <int NV>
__global__ void __launch_bounds__(kThreads, 1)
la_state_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap ty,
                const __grid_constant__ CUtensorMap ts, const __grid_constant__ CUtensorMap to, const Params p) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(16) Shared sh;
  constexpr int HC = NV / 4;   // value columns a thread
  const uint32_t raw = tc::smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* sm = smem_raw + (sbase - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = warp & 3, part = warp >> 2;
  const uint32_t lane0 = 32u * quad;
  const int row = 32 * quad + lane;        // key channel
  const bool live = row < p.dk;            // dk 64: lanes 64-127 of the product are not used

  dependents_may_start();
  const int tiles = p.dv / NV;
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
    for (int i = 0; i < kStages; ++i) tc::mbar_init(tc::smem_u32(&sh.full[i]), 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tc::smem_u32(&sh.wready[i]), 32);
      tc::mbar_init(tc::smem_u32(&sh.wfree[i]), kWorkers / 32);
    }
    tc::mbar_init(tc::smem_u32(&sh.aready), kWorkers / 32);
    tc::mbar_init(tc::smem_u32(&sh.mma), 1);
    tc::mbar_init(tc::smem_u32(&sh.sfree), 1);
    tc::mbar_init(tc::smem_u32(&sh.ofull), 1);
    tc::mbar_init(tc::smem_u32(&sh.oread), kWorkers / 32);
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
  dependency_wait();

  float s[HC];   // state elements (row, vt NV + part HC + j)
  const int64_t sbase_g = ((int64_t)unit * p.dk + row) * p.dv + vt * NV + part * HC;
  const int64_t seg_g = (((int64_t)unit * p.nseg + seg) * p.dk + row) * p.dv + vt * NV + part * HC;
  float log_decay = 0.f;   // of this warp's steps (warps 17, 18)

  if (warp == kWorkers / 32) {
    const uint32_t idesc = tc::make_idesc(tc::kKindBF16, 128, NV, false, true);
    int loaded = 0;
    auto load = [&](int i) {
      const uint32_t bar = tc::smem_u32(&sh.full[i % kStages]), dst = sbase + (i % kStages) * stage_bytes<NV>();
      const int tok = t0 + chunk_of(i) * kC;
      tc::mbar_expect_tx(bar, p.dk / 64 * kBlk + NV / 64 * kBlk);
      for (int b = 0; b < p.dk / 64; ++b) tc::tma_load_3d(dst + b * kBlk, &tx, bar, 64 * b, hq, tok);
      for (int b = 0; b < NV / 64; ++b) tc::tma_load_3d(dst + kTile + b * kBlk, &ty, bar, vt * NV + 64 * b, h, tok);
    };
    auto state_row = [&](int i, int terms, int term) {   // of the stored states: this value tile's rows
      const int item = (slot0 + chunk_of(i)) * Hv + h;
      return ((item * terms + term) * (p.dv / 64) + vt * (NV / 64)) * p.dk;
    };
    auto load_other = [&](int i) {
      tc::mbar_expect_tx(tc::smem_u32(&sh.ofull), 2 * p.dk * 128);
      for (int t = 0; t < 2; ++t)
        tc::tma_load_2d(sbase + off_other<NV>() + t * kBlk, &to, tc::smem_u32(&sh.ofull), 0, state_row(i, 2, t));
    };
    for (; loaded < min(2, steps); ++loaded)
      if (lane == 0) load(loaded);
    int others = 0;
    if (p.other && steps) {
      if (lane == 0) load_other(0);
      others = 1;
    }
    const uint32_t me = elect_one();
    int issued = 0;
    for (int i = 0; i < steps; ++i) {
      ok = wait(sh.dead, sh.aready, i & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      tc::tc_fence_after();
      const uint64_t bd = tc::make_sdesc(sbase + (i % kStages) * stage_bytes<NV>() + kTile, kBlk, 1024);
      const uint32_t a = tmem + TM_A + (i & 1) * 192;
#pragma unroll
      for (int t = 0; t < 3; ++t)
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_bf16_ta(tmem + TM_ACC, a + 64 * t + 8 * ks, dadv(bd, ks * 2048), idesc, t + ks > 0, me);
      mma_commit_w(tc::smem_u32(&sh.mma), me);
      issued = i + 1;
      if (i + 2 < steps) {   // its stage held step i - 1, whose product the workers have taken
        if (lane == 0) load(i + 2);
        ++loaded;
      }
      if (p.store) {
        if (lane == 0) {
          for (int b = 0; b < (NV == 64 ? p.terms : 2); ++b)
            tc::tma_store_2d(&ts, sbase + off_stage<NV>() + b * kBlk, 0,
                             NV == 64 ? state_row(i, p.terms, b) : state_row(i, 1, 0) + b * p.dk);
          tc::bulk_commit();
        }
        __syncwarp();
      }
      if (p.other && i + 1 < steps) {
        ok = wait(sh.dead, sh.oread, i & 1);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (lane == 0) load_other(i + 1);
        ++others;
      }
      if (p.store && lane == 0) {
        tc::bulk_wait_read();
        tc::mbar_arrive(tc::smem_u32(&sh.sfree));
      }
      __syncwarp();
    }
    if (lane == 0 && !ok) {   // nothing of this CTA is in flight when it ends
      for (int i = max(0, loaded - kStages); i < loaded; ++i)
        tc::mbar_wait(tc::smem_u32(&sh.full[i % kStages]), (i / kStages) & 1, 1u << 22);
      if (issued) tc::mbar_wait(tc::smem_u32(&sh.mma), (issued - 1) & 1, 1u << 22);
      if (others) tc::mbar_wait(tc::smem_u32(&sh.ofull), (others - 1) & 1, 1u << 22);
      tc::bulk_wait_read();
    }
  } else if (warp > kWorkers / 32) {
    const int which = warp - kWorkers / 32 - 1;
    float gx[4];
    auto gates = [&](int i) { p.gates.load(gx, t0 + (int64_t)chunk_of(i) * kC, h, rows_of(chunk_of(i)), lane); };
    if (which < steps) gates(which);
    for (int i = which; i < steps; i += 2) {
      ok = wait(sh.dead, sh.wfree[i & 1], ((i >> 1) & 1) ^ 1);
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
      *reinterpret_cast<float4*>(&sh.w[i & 1][4 * lane]) = make_float4(v[0], v[1], v[2], v[3]);
      if (lane == 0) sh.decay[i & 1] = expf(all);
      log_decay += all;
      tc::mbar_arrive(tc::smem_u32(&sh.wready[i & 1]));
    }
    if (lane == 0) sh.log_decay[which] = log_decay;
  } else {
    const float* src = p.totals ? nullptr : p.nseg > 1 ? p.seg_tot + seg_g : p.s0 ? p.s0 + sbase_g : nullptr;
#pragma unroll
    for (int j = 0; j < HC; j += 4) {
      const float4 v = src && live ? *reinterpret_cast<const float4*>(src + j) : make_float4(0.f, 0.f, 0.f, 0.f);
      s[j] = v.x; s[j + 1] = v.y; s[j + 2] = v.z; s[j + 3] = v.w;
    }
    // byte offsets of this channel within an 8-row group of the swizzled tile
    uint32_t off[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) off[r] = (row >> 6) * kBlk + part * 4096 + tc::sw128(r, (row & 63) * 2);
    const bool work = 32 * quad < p.dk;   // uniform in the warp
    float decay = 1.f;                    // Gam of the chunk whose product is in flight
    auto take = [&](int i) {              // the product of step i -> the state
      ok = wait(sh.dead, sh.mma, i & 1);
      ok = __all_sync(0xffffffffu, ok);
      tc::tc_fence_after();
      if (!work) return;
      float v[HC];
#pragma unroll
      for (int q = 0; q < HC; q += 16) tc::tmem_ld16(tc::tmem_addr(tmem, lane0, TM_ACC + part * HC + q), v + q);
      tc::tmem_ld_wait();
      const float2 d2 = make_float2(decay, decay);
#pragma unroll
      for (int j = 0; j < HC; j += 2) {
        const float2 r = __ffma2_rn(d2, make_float2(s[j], s[j + 1]), make_float2(v[j], v[j + 1]));
        s[j] = r.x;
        s[j + 1] = r.y;
      }
    };
    const float2 neg = make_float2(-1.f, -1.f);
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      const int c = chunk_of(i), L = rows_of(c);
      unsigned char* kt = sm + (i % kStages) * stage_bytes<NV>();
      ok = wait(sh.dead, sh.full[i % kStages], (i / kStages) & 1) && wait(sh.dead, sh.wready[i & 1], (i >> 1) & 1);
      if (L < kC) {   // uniform: the tail rows are another sequence's. K: what this warp reads; V: the product
        const int r = 32 * part + lane;
        if (r >= L) {
#pragma unroll
          for (int b = 0; b < 4; ++b)
            *reinterpret_cast<uint4*>(kt + (quad >> 1) * kBlk + tc::sw128(r, (quad & 1) * 64 + 16 * b)) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
        zero_tail_rows(kt + kTile, NV / 64, tid, L);
        tc::fence_proxy_async_smem();
      }
      const float decay_i = sh.decay[i & 1];
      if (work) {
        const float* ws = sh.w[i & 1] + 32 * part;
        uint32_t t1[16], t2[16], t3[16];
#pragma unroll
        for (int q = 0; q < 16; q += 2) {
          const unsigned char* g8 = kt + (q >> 2) * 1024;
          const float4 wv = *reinterpret_cast<const float4*>(ws + 2 * q);
          const float2 w2[2] = {make_float2(wv.x, wv.y), make_float2(wv.z, wv.w)};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int o = q + e;
            const uint32_t k0 = *reinterpret_cast<const uint16_t*>(g8 + off[(2 * o) & 7]);
            const uint32_t k1 = *reinterpret_cast<const uint16_t*>(g8 + off[(2 * o + 1) & 7]);
            const float2 x = __fmul2_rn(make_float2(__uint_as_float(k0 << 16), __uint_as_float(k1 << 16)), w2[e]);
            t1[o] = pack_bf16(x.x, x.y);
            const float2 y = __ffma2_rn(unpack_bf16(t1[o]), neg, x);
            t2[o] = pack_bf16(y.x, y.y);
            const float2 z = __ffma2_rn(unpack_bf16(t2[o]), neg, y);
            t3[o] = pack_bf16(z.x, z.y);
          }
        }
        const uint32_t at = TM_A + (i & 1) * 192 + 16 * part;
        tmem_st16u(tc::tmem_addr(tmem, lane0, at), t1);
        tmem_st16u(tc::tmem_addr(tmem, lane0, at + 64), t2);
        tmem_st16u(tc::tmem_addr(tmem, lane0, at + 128), t3);
        tc::tmem_st_wait();
      }
      if (i > 0) take(i - 1);
      if (p.store && i > 0) ok = ok && wait(sh.dead, sh.sfree, (i - 1) & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      if (p.store && live) {   // the state before this chunk, 128-byte swizzled rows of 64 columns
#pragma unroll
        for (int j = 0; j < HC; j += 8) {
          const int col = part * HC + j;
          unsigned char* at = sm + off_stage<NV>() + (col / 64) * kBlk + tc::sw128(row, (col % 64) * 2);
          if (NV == 64 && p.terms == 2) {
            uint4 hi, lo;
            split8(s + j, hi, lo);
            *reinterpret_cast<uint4*>(at) = hi;
            *reinterpret_cast<uint4*>(at + kBlk) = lo;
          } else {
            *reinterpret_cast<uint4*>(at) = pack8(s + j);
          }
        }
        tc::fence_proxy_async_smem();
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(tc::smem_u32(&sh.wfree[i & 1]));
        tc::mbar_arrive(tc::smem_u32(&sh.aready));
      }
      decay = decay_i;
      if (NV == 64 && p.other) {
        ok = wait(sh.dead, sh.ofull, i & 1);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        float2 x = make_float2(0.f, 0.f);
        if (live) {
#pragma unroll
          for (int j = 0; j < HC; j += 8) {
            const unsigned char* at = sm + off_other<NV>() + tc::sw128(row, (part * HC + j) * 2);
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
        const float sum = warp_sum(x.x + x.y);
        if (lane == 0)
          p.edge[(((int64_t)(slot0 + c) * Hv + h) * tiles + vt) * (kWorkers / 32) + warp] = decay_i * sum;
      }
    }
    if (ok && steps) take(steps - 1);
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
  if (sh.dead) return;
  if (warp >= kWorkers / 32) {
    if (p.totals && tid == kWorkers && vt == 0)
      p.seg_dec[unit * p.nseg + seg] = expf(sh.log_decay[0] + sh.log_decay[1]);
    return;
  }
  float* dst = p.totals ? p.seg_tot + seg_g : p.sT && seg == p.nseg - 1 ? p.sT + sbase_g : nullptr;
  if (dst && live)
#pragma unroll
    for (int j = 0; j < HC; j += 4) *reinterpret_cast<float4*>(dst + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
}

// Segment contributions -> the state that each segment starts from (in place), element by element.
__global__ void __launch_bounds__(256) la_join_kernel(float* seg_tot, const float* seg_dec, const float* s0, int nseg,
                                                      int64_t elems) {
  const int64_t unit = blockIdx.y;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;   // four state elements
  dependents_may_start();
  dependency_wait();
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
cudaError_t run(const CUtensorMap (&m)[4], const Params& p, int64_t units, bool dependent, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(la_state_kernel<NV>, smem_bytes<NV>(), allowed);
  if (e != cudaSuccess) return e;
  return launch(dependent, la_state_kernel<NV>, dim3((unsigned)(units * p.nseg * (p.dv / NV))), kThreads, smem_bytes<NV>(),
                stream, m[0], m[1], m[2], m[3], p);
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

// A tile of 128 value columns weights K once for both halves, but has half as many CTAs and no room in
// shared memory for second terms.
static bool wide_tiles(const LaProblem& p) {
  return p.dv == 128 && (int64_t)p.N * p.Hv * state_segments(p) >= kSMs;
}
int edge_parts(const LaProblem& p) { return p.dv / 64 * (kWorkers / 32); }

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
  if (r.states && !make_bf16_rows_map(&m[2], r.states, rows * r.terms, p.dk)) return cudaErrorNotSupported;
  if (r.other && !make_bf16_rows_map(&m[3], r.other, rows * 2, p.dk)) return cudaErrorNotSupported;
  Params s{{p.cu, p.T, p.N}, {p.g, p.Hv, p.head_decay}, r.s0, r.sT, r.seg_tot, r.seg_dec, r.edge,
           status, p.Hqk, p.dk, p.dv, r.terms, r.reverse, state_segments(p), 0, r.states != nullptr, r.other != nullptr,
           r.scale};
  // Walks of unequal lengths: the longest first, so that the last ones to start are short (b = 1, 8 packed
  // sequences of 1 to 8192 tokens, 32 heads: 200 -> 177 us). Many sequences even out by themselves.
  if (p.cu_host && p.N <= 64) {
    s.sorted = 1;
    for (int i = 0; i < p.N; ++i) s.order[i] = (uint8_t)i;
    std::stable_sort(s.order, s.order + p.N, [&](uint8_t a, uint8_t b) {
      return p.cu_host[a + 1] - p.cu_host[a] > p.cu_host[b + 1] - p.cu_host[b];
    });
  }
  const bool wide = wide_tiles(p) && r.terms == 1;
  auto go = [&] { return wide ? run<128>(m, s, units, dependent, stream) : run<64>(m, s, units, dependent, stream); };
  if (s.nseg > 1) {
    s.totals = 1;
    s.store = s.other = 0;
    cudaError_t e = go();
    if (e != cudaSuccess) return e;
    e = launch(true, la_join_kernel, dim3((unsigned)((elems / 4 + 255) / 256), (unsigned)units), 256, 0, stream, r.seg_tot,
               (const float*)r.seg_dec, r.s0, s.nseg, elems);
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

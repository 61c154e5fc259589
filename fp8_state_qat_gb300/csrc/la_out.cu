// la_out.cu -- outputs and gradients of linear attention with a decay for each head, chunk by chunk in
// parallel: with the states at the chunk boundaries (la_state.cu) no chunk waits for another.
//
// The forward's output and the gradients of q, k, v are one computation in four roles,
//   out_t = f_in sum_s D(t, s) (a_t . b_s) c_s + f_st E_t a_t^T St
//   o:  a = q,  b = k,  c = v,  St = S (entering the chunk)      s <= t, D = exp(gam_t - gam_s), E = exp(gam_t)
//   dq: a = do, b = v,  c = k,  St = S^T                         likewise
//   dv: a = k,  b = q,  c = do, St = dS (leaving the chunk)      s >= t, D = exp(gam_s - gam_t), E = exp(gam_C - gam_t)
//   dk: a = v,  b = do, c = q,  St = dS^T                        likewise
// and per item (chunk, value head, role) three tcgen05 products with M = 128 tokens:
//   scores a b^T -> weighted by D and the mask, rounded to bf16, back into tensor memory as an A operand;
//   a St into an accumulator of its own (its row weights E differ from the scores');  P c.
// The roles dq and dk also give the parts of dg, sums over pairs of tokens of
// D (a_t . b_s) (e_t . c_s) with e = q or k: those take a fourth product e c^T and fp32 sums before any
// rounding, and e_t . (a_t^T St) with the state in two bf16 terms.
//
// Roundings to bf16: the weighted scores and the state, each once, against outputs that are bf16
// themselves; everything else is fp32.
//
// What bounds it is the traffic: 3 or 4 token tiles and 1 or 2 state terms in (32 KB each at d = 128), one tile
// out, for about 1 us of tensor-core and exponential work. So one persistent CTA per SM keeps a ring of
// six 32 KB tiles filled ahead by one TMA thread, across items; one thread issues the products; four warps
// weight the scores; four others write the outputs of the same item while the first go on to
// the next. The roles of one chunk run next to each other and read the same tiles from L2.
#include <algorithm>

#include "la_chunk.cuh"
#include "kernels.h"

namespace gdn {
namespace la {
namespace {

constexpr int kThreads = 384;            // warps 0 TMA, 1 products, 4-7 scores, 8-11 outputs
constexpr int kRing = 6;
constexpr uint32_t TM_S = 0, TM_E = 128, TM_I = 256, TM_O = 384;   // scores (P in place), e c^T, state part, P c
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSmemBytes = kRing * kTile + 4 * 128 * 4 + 1024;
constexpr int kSMs = 152;

struct Params {
  Seqs seqs;
  GateSrc gates;
  Role role[3];
  int heads[4], width[4];   // of q, k, v, do
  int terms[2];
  int* status;
  int64_t slots;
  int roles, dk, dv;
};
struct Maps {
  CUtensorMap t[4];   // q, k, v, do
  CUtensorMap s[2];   // S, dS: rows of 64 value columns
};

struct Item {
  int n, h, L, tok, role;
  int64_t state;   // index among the states
};

// The item's chunk, or false where no chunk uses its slot.
__device__ __forceinline__ bool locate(const Params& p, int64_t i, Item& it) {
  it.role = (int)(i % p.roles);
  i /= p.roles;
  it.h = (int)(i % p.gates.Hv);
  const int64_t slot = i / p.gates.Hv;
  int lo = 0, hi = p.seqs.N - 1;   // the last sequence whose slots start at or before this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.seqs.slot0(mid) <= slot) lo = mid;
    else hi = mid - 1;
  }
  it.n = lo;
  const int64_t t0 = p.seqs.start(lo), len = p.seqs.len(lo), c = slot - p.seqs.slot0(lo);
  if (c < 0 || c * kC >= len) return false;
  it.L = (int)(len - c * kC < kC ? len - c * kC : kC);
  it.tok = (int)(t0 + c * kC);
  it.state = slot * p.gates.Hv + it.h;
  return true;
}

struct Shared {
  uint64_t full[kRing], empty[kRing];
  uint64_t sc, oi, oo, pr, ofree;   // scores done, state part done, P c done, P written, accumulators read
  uint64_t drain;
  uint32_t tmem;
  int dead;                          // a wait gave up: every role winds down
};

// Bounded wait that also ends when another role has given up.
__device__ __forceinline__ bool wait(Shared& sh, uint64_t& bar, uint32_t parity) {
  const uint32_t a = tc::smem_u32(&bar);
  for (uint32_t i = 0; i < GDN_WAIT_LIMIT; ++i) {
    if (tc::mbar_try_wait(a, parity)) return true;
    if (*(volatile int*)&sh.dead) return false;
  }
  *(volatile int*)&sh.dead = 1;
  return false;
}

__global__ void __launch_bounds__(kThreads, 1)
la_out_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) Shared sh;
  const uint32_t raw = tc::smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* const sm = smem_raw + (sbase - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t items = p.slots * p.gates.Hv * p.roles;

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      tc::mbar_init(tc::smem_u32(&sh.full[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh.empty[i]), 1);
    }
    tc::mbar_init(tc::smem_u32(&sh.sc), 1);
    tc::mbar_init(tc::smem_u32(&sh.oi), 1);
    tc::mbar_init(tc::smem_u32(&sh.oo), 1);
    tc::mbar_init(tc::smem_u32(&sh.drain), 1);
    tc::mbar_init(tc::smem_u32(&sh.pr), 128);
    tc::mbar_init(tc::smem_u32(&sh.ofree), 128);
    tc::mbar_fence_init();
    sh.dead = 0;
  }
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&sh.tmem), kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  bool ok = true;

  // Tiles of an item, in ring order: b, a, state (, c) -- with e: b, a, c, e, state hi, state lo.
  if (tid == 0) {
    uint32_t x = 0;   // tiles issued
    auto slot_of = [&](uint32_t bytes) {
      if (!ok) return sbase;
      ok = wait(sh, sh.empty[x % kRing], ((x / kRing) & 1) ^ 1);
      if (ok) tc::mbar_expect_tx(tc::smem_u32(&sh.full[x % kRing]), bytes);
      return sbase + (x % kRing) * kTile;
    };
    for (int64_t i = blockIdx.x; i < items && ok; i += gridDim.x) {
      Item it;
      if (!locate(p, i, it)) continue;
      const Role& r = p.role[it.role];
      auto tokens = [&](int m) {
        const int D = p.width[m], hh = it.h / (p.gates.Hv / p.heads[m]);
        const uint32_t dst = slot_of(D / 64 * kBlk);
        if (!ok) return;
        for (int b = 0; b < D / 64; ++b)
          tc::tma_load_3d(dst + b * kBlk, &maps.t[m], tc::smem_u32(&sh.full[x % kRing]), 64 * b, hh, it.tok);
        ++x;
      };
      auto state = [&](int term) {
        const uint32_t dst = slot_of(p.dk * p.dv * 2);
        if (!ok) return;
        const int64_t row = (it.state * p.terms[r.st] + term) * p.dk * (p.dv / 64);
        for (int b = 0; b < p.dv / 64; ++b)
          tc::tma_load_2d(dst + b * p.dk * 128, &maps.s[r.st], tc::smem_u32(&sh.full[x % kRing]), 0,
                          (int)(row + b * p.dk));
        ++x;
      };
      tokens(r.b);
      tokens(r.a);
      if (r.e >= 0) {
        tokens(r.c);
        tokens(r.e);
        state(0);
        state(1);
      } else {
        state(0);
        tokens(r.c);
      }
    }
    // no copy may be in flight when the CTA ends
    for (uint32_t y = x > kRing ? x - kRing : 0; y < x; ++y)
      tc::mbar_wait(tc::smem_u32(&sh.full[y % kRing]), (y / kRing) & 1, 1u << 22);
  } else if (tid == 32) {
    uint32_t x = 0;
    uint32_t k = 0;   // items done
    auto tile = [&](uint32_t y) { return sbase + (y % kRing) * kTile; };
    auto landed = [&](uint32_t y) { ok = ok && wait(sh, sh.full[y % kRing], (y / kRing) & 1); };
    auto release = [&](uint32_t y) { tc::mma_commit(tc::smem_u32(&sh.empty[y % kRing])); };
    for (int64_t i = blockIdx.x; i < items && ok; i += gridDim.x) {
      Item it;
      if (!locate(p, i, it)) continue;
      const Role& r = p.role[it.role];
      const bool dg = r.e >= 0;
      const int da = p.width[r.a], dc = p.width[r.c];
      const uint32_t xb = x, xa = x + 1, xc = dg ? x + 2 : x + 3, xe = x + 3, xs = dg ? x + 4 : x + 2;
      // [128 x D] [128 x D]^T, both K-major
      auto scores = [&](uint32_t d, uint32_t ta, uint32_t tb, int D) {
        const uint64_t ad = tc::make_sdesc(ta, 16, 1024), bd = tc::make_sdesc(tb, 16, 1024);
        constexpr uint32_t idesc = tc::make_idesc(tc::kKindBF16, 128, 128, false, false);
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t at = (ks >> 2) * kBlk + (ks & 3) * 32;
          tc::mma_bf16(tmem + d, dadv(ad, at), dadv(bd, at), idesc, ks > 0);
        }
      };
      landed(xb);
      landed(xa);
      if (k > 0) ok = ok && wait(sh, sh.oo, (k - 1) & 1);   // P of the item before is consumed
      if (!ok) break;
      tc::tc_fence_after();
      scores(TM_S, tile(xa), tile(xb), da);
      release(xb);
      if (dg) {
        landed(xc);
        landed(xe);
        if (!ok) break;
        scores(TM_E, tile(xe), tile(xc), dc);
      }
      tc::mma_commit(tc::smem_u32(&sh.sc));
      landed(xs);
      if (dg) landed(xs + 1);
      if (k > 0) ok = ok && wait(sh, sh.ofree, (k - 1) & 1);
      if (!ok) break;
      tc::tc_fence_after();
      // a St: St [da x dc] is stored as rows of the key channel, 64 value columns each
      for (int t = 0; t < (dg ? 2 : 1); ++t) {
        const uint64_t ad = tc::make_sdesc(tile(xa), 16, 1024);
        const uint32_t sblk = p.dk * 128;   // a block of 64 value columns
        if (r.st_transposed) {   // K = value columns (K-major), N = key channels
          const uint64_t bd = tc::make_sdesc(tile(xs + t), 16, 1024);
          const uint32_t idesc = tc::make_idesc(tc::kKindBF16, 128, p.dk, false, false);
          for (int ks = 0; ks < da / 16; ++ks)
            tc::mma_bf16(tmem + TM_I, dadv(ad, (ks >> 2) * kBlk + (ks & 3) * 32),
                         dadv(bd, (ks >> 2) * sblk + (ks & 3) * 32), idesc, t + ks > 0);
        } else {                 // K = key channels, N = value columns (MN-major)
          const uint64_t bd = tc::make_sdesc(tile(xs + t), sblk, 1024);
          const uint32_t idesc = tc::make_idesc(tc::kKindBF16, 128, p.dv, false, true);
          for (int ks = 0; ks < da / 16; ++ks)
            tc::mma_bf16(tmem + TM_I, dadv(ad, (ks >> 2) * kBlk + (ks & 3) * 32), dadv(bd, ks * 2048), idesc, t + ks > 0);
        }
      }
      release(xa);
      release(xs);
      if (dg) release(xs + 1);
      tc::mma_commit(tc::smem_u32(&sh.oi));
      landed(xc);
      ok = ok && wait(sh, sh.pr, k & 1);
      if (!ok) break;
      tc::tc_fence_after();
      {
        const uint64_t bd = tc::make_sdesc(tile(xc), kBlk, 1024);
        const uint32_t idesc = tc::make_idesc(tc::kKindBF16, 128, dc, false, true);
        for (int ks = 0; ks < 8; ++ks) mma_bf16_ta(tmem + TM_O, tmem + TM_S + 8 * ks, dadv(bd, ks * 2048), idesc, ks > 0);
      }
      release(xc);
      tc::mma_commit(tc::smem_u32(&sh.oo));
      x += dg ? 6 : 4;
      ++k;
    }
    // the products in flight end before the tensor memory goes
    if (!ok) {
      tc::mma_commit(tc::smem_u32(&sh.drain));
      tc::mbar_wait(tc::smem_u32(&sh.drain), 0, 1u << 22);
    } else if (k > 0) {
      ok = wait(sh, sh.oo, (k - 1) & 1);
    }
  } else if (warp >= 4 && warp < 8) {
    const int w = warp - 4;
    const uint32_t lane0 = 32u * w;
    const int row = 32 * w + lane;
    float* const col = reinterpret_cast<float*>(sm + kRing * kTile) + 128 * w;
    uint32_t x = 0, k = 0;
    for (int64_t i = blockIdx.x; i < items && ok; i += gridDim.x) {
      Item it;
      if (!locate(p, i, it)) continue;
      const Role& r = p.role[it.role];
      const bool dg = r.e >= 0, rev = r.reverse;
      const int dc = p.width[r.c];
      const uint32_t xc = dg ? x + 2 : x + 3;
      float gx[4];
      Gates g;
      p.gates.load(gx, it.tok, it.h, it.L, lane);
      scan_gates(gx, g, lane);
      // column factors: the decay from a token to the end of its block (or from the block's start to it)
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) col[32 * j + lane] = 32 * j + lane < it.L ? expf(rev ? g.pre(j) : g.after(j)) : 0.f;
      __syncwarp();
      float ghi = 0.f, glo = 0.f, edge = 0.f;   // this row's prefix; the decay between it and its block's edge
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j == w) {
          ghi = g.hi[j];
          glo = g.lo[j];
          edge = rev ? g.after(j) : g.pre(j);
        }
      ok = wait(sh, sh.sc, k & 1);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc::tc_fence_after();
      float sum = 0.f;
      uint32_t zero[16] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (rev ? j < w : j > w) {
          tmem_st16u(tc::tmem_addr(tmem, lane0, TM_S + 16 * j), zero);
          continue;
        }
        float v[32];
        ld32(tmem, lane0, TM_S + 32 * j, v);
        if (j == w) {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float ch = __shfl_sync(0xffffffffu, ghi, c), cl = __shfl_sync(0xffffffffu, glo, c);
            const float d = (ghi - ch) + (glo - cl);
            const bool in = rev ? (c >= lane && 32 * j + c < it.L) : c <= lane;
            v[c] = in ? v[c] * __expf(rev ? -d : d) : 0.f;
          }
        } else {
          float e = edge;
#pragma unroll
          for (int m = 0; m < 4; ++m)
            if (rev ? (m > w && m < j) : (m > j && m < w)) e += g.tot(m);
          const float f = expf(e);
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 cf = *reinterpret_cast<const float4*>(col + 32 * j + c);
            const float cc[4] = {cf.x, cf.y, cf.z, cf.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)   // tokens past the chunk's end may hold anything
              v[c + q] = !rev || 32 * j + c + q < it.L ? v[c + q] * (f * cc[q]) : 0.f;
          }
        }
        if (dg) {
          float ev[32];
          ld32(tmem, lane0, TM_E + 32 * j, ev);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const bool in = j == w ? (rev ? (c > lane && 32 * j + c < it.L) : c < lane) : (!rev || 32 * j + c < it.L);
            sum += in ? v[c] * ev[c] : 0.f;
          }
        }
        uint32_t u[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) u[c] = pack_bf16(v[2 * c], v[2 * c + 1]);
        // columns [16 j, 16 j + 16) hold scores of blocks <= j / 2, read before
        tmem_st16u(tc::tmem_addr(tmem, lane0, TM_S + 16 * j), u);
      }
      tc::tmem_st_wait();
      if (it.L < kC) {   // rows past the end of c would meet zero weights: not with a NaN
        ok = wait(sh, sh.full[xc % kRing], (xc / kRing) & 1);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        zero_tail_rows(sm + (xc % kRing) * kTile, dc / 64, tid - 128, it.L);
        tc::fence_proxy_async_smem();
      }
      tc::tc_fence_before();
      tc::mbar_arrive(tc::smem_u32(&sh.pr));
      if (dg && row < it.L) r.dot_in[(int64_t)(it.tok + row) * p.gates.Hv + it.h] = r.f_in * sum;
      x += dg ? 6 : 4;
      ++k;
    }
  } else if (warp >= 8) {
    const int w = warp - 8;
    const uint32_t lane0 = 32u * w;
    const int row = 32 * w + lane;
    uint32_t x = 0, k = 0;
    for (int64_t i = blockIdx.x; i < items && ok; i += gridDim.x) {
      Item it;
      if (!locate(p, i, it)) continue;
      const Role& r = p.role[it.role];
      const bool dg = r.e >= 0, rev = r.reverse;
      const int dc = p.width[r.c];
      float gx[4];
      Gates g;
      p.gates.load(gx, it.tok, it.h, it.L, lane);
      scan_gates(gx, g, lane);
      float e = 0.f;   // log of the decay between the state and this row
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j == w) e += rev ? g.after(j) : g.pre(j);
        if (rev ? j > w : j < w) e += g.tot(j);
      }
      const float fs = expf(e) * r.f_st, fi = r.f_in;
      const int64_t at = (int64_t)(it.tok + row) * p.gates.Hv + it.h;
      ok = wait(sh, sh.oi, k & 1);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc::tc_fence_after();
      if (dg) {
        const uint32_t xe = x + 3;
        ok = wait(sh, sh.full[xe % kRing], (xe / kRing) & 1);   // landed long ago; makes it visible here
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        const unsigned char* et = sm + (xe % kRing) * kTile;
        float dot = 0.f;
        for (int b = 0; b < dc / 32; ++b) {
          float v[32];
          ld32(tmem, lane0, TM_I + 32 * b, v);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float ev[8];
            load_bf16x8(reinterpret_cast<const __nv_bfloat16*>(et + (b >> 1) * kBlk + tc::sw128(row, 64 * (b & 1) + 16 * c)), ev);
#pragma unroll
            for (int q = 0; q < 8; ++q) dot = fmaf(ev[q], v[8 * c + q], dot);
          }
        }
        if (row < it.L) r.dot_st[at] = fs * dot;
      }
      ok = wait(sh, sh.oo, k & 1);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc::tc_fence_after();
      for (int b = 0; b < dc / 32; ++b) {
        float v[32], s[32];
        ld32(tmem, lane0, TM_O + 32 * b, v);
        ld32(tmem, lane0, TM_I + 32 * b, s);
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = fmaf(fs, s[c], fi * v[c]);
        if (row < it.L) {
          if (r.out_f32) {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(r.out) + at * dc + 32 * b);
#pragma unroll
            for (int c = 0; c < 8; ++c) dst[c] = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(r.out) + at * dc + 32 * b);
#pragma unroll
            for (int c = 0; c < 4; ++c) dst[c] = pack8(v + 8 * c);
          }
        }
      }
      tc::tc_fence_before();
      tc::mbar_arrive(tc::smem_u32(&sh.ofree));
      if (dg) {   // e is read by all four warps
        tc::named_bar_sync(1, 128);
        if (tid == 256) tc::mbar_arrive(tc::smem_u32(&sh.empty[(x + 3) % kRing]));
      }
      x += dg ? 6 : 4;
      ++k;
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
}

}  // namespace

cudaError_t launch_outputs(const LaProblem& p, const OutRun& r, int* status, cudaStream_t stream) {
  const int64_t tokens = (int64_t)p.B * p.T, slots = la_slots(p), items = slots * p.Hv * r.roles;
  if (tokens == 0 || items == 0) return cudaSuccess;
  Maps m;
  const void* base[4] = {r.q, r.k, r.v, r.dout};
  Params o{{p.cu, p.T, p.N}, {p.g, p.Hv, p.head_decay}, {}, {p.Hqk, p.Hqk, p.Hv, p.Hv}, {p.dk, p.dk, p.dv, p.dv},
           {r.terms[0], r.terms[1]}, status, slots, r.roles, p.dk, p.dv};
  for (int i = 0; i < r.roles; ++i) o.role[i] = r.role[i];
  for (int i = 0; i < 4; ++i)
    if (!make_bf16_map(&m.t[i], base[i] ? base[i] : r.q, o.width[i], o.heads[i], tokens, kC)) return cudaErrorNotSupported;
  for (int i = 0; i < 2; ++i) {
    const int j = r.states[i] ? i : 0;
    if (!make_bf16_rows_map(&m.s[i], r.states[j], slots * p.Hv * r.terms[j] * p.dk * (p.dv / 64), p.dk))
      return cudaErrorNotSupported;
  }
  cudaError_t e = cudaFuncSetAttribute(la_out_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  la_out_kernel<<<(unsigned)std::min<int64_t>(items, kSMs), kThreads, kSmemBytes, stream>>>(m, o);
  return cudaGetLastError();
}

}  // namespace la
}  // namespace gdn

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
//   scores a b^T -> weighted by D and the mask, in two bf16 terms back into tensor memory as A operands;
//   a St into an accumulator of its own (its row weights E differ from the scores');  P c.
// The roles dq and dk also give the parts of dg, sums over pairs of tokens of
// D (a_t . b_s) (e_t . c_s) with e = q or k: those take a fourth product e c^T and fp32 sums before any
// rounding, and e_t . (a_t^T St) with the state in two bf16 terms.
//
// The weighted scores and the states are each a sum of two bf16 terms (16 bits and a sign: 2^-18 of the value), so
// that the outputs' own rounding to bf16 is the only one that shows: o, dq, dk, dv are off by 1.7e-3 of 64 bits, as the
// rounded 64-bit result is; with one term of each it was 2.3e-3, in 55 instead of 65 us (o) and 162 instead of 185 (dq,
// dk, dv) at the size below. dg is fp32 and rests on the same states: 4e-7 to 3e-6 off, up to 6e-6 in sequences of a few
// tokens whose gradient is all of the given states'. A third term would bring that to 3e-7: 32 KB more a chunk and state
// here, and in the walk room for one set of V's terms instead of two, which alone costs 10 us a walk there (a
// training step 451 -> 472 us).
//
// What bounds it is the traffic: 3 or 4 token tiles and 2 or 4 state terms in (32 KB each at d = 128), one tile out a
// role. So one persistent CTA per SM keeps six 32 KB tiles filled ahead by TMA, across items; the three roles of a
// chunk follow each other on the same token tiles; one warp issues the products; one computes the decays an
// item ahead; eight weight the scores; four write the outputs of an item while the others go on to the next. The
// loop bodies are kept small and shared by all roles: unrolled per block and role, the code outgrew the instruction cache
// and the same work took 4 (o) to 10 times (gradients) as long.
//
// At 4 x 4096 tokens, 16 heads, d 128 (cold): o 65 us, 405 MB of tiles, 6.2 TB/s (0.93 of the measured copy bandwidth); dq, dk,
// dv 185 us, 743 MB, 4.0 TB/s: all four token tiles of a chunk are in use until its last role, and the next chunk's
// arrive 3 us after they fall free.
#include <algorithm>
#include <cstddef>

#include "la_chunk.cuh"
#include "kernels.h"

namespace gdn {
namespace la {
namespace {

constexpr int kThreads = 512;            // warps 0, 3 TMA, 1 products, 2 gates, 4-11 scores, 12-15 outputs
constexpr int kTok = 4, kSt = 2;          // rings of token and state tiles, 32 KB each
constexpr uint32_t TM_S = 0, TM_E = 128, TM_I = 256, TM_O = 384;   // scores (P in place), e c^T, state part, P c
constexpr uint32_t kTmemCols = 512;
constexpr int kSMs = 152;

struct Params {
  Seqs seqs;
  GateSrc gates;
  Role role[3];
  int heads[4], width[4];   // of q, k, v, do
  int ntok, tok[4], nst, st[4], term[4];
  int* status;
  int64_t dot_stride;       // between the two halves of dot_in
  int slots, roles, dk, dv;
};
struct Maps {
  CUtensorMap t[4];   // q, k, v, do
  CUtensorMap s[2];   // S, dS: rows of 64 value columns
};

// What the score and output warps need to know of an item, written by the gate warp.
struct __align__(16) Entry {
  int tok, L, h, role;         // L == 0: no more items
  int pairwise;                // bit j: block j's decays are formed pair by pair (their range is too wide to factor)
  int pad[3];
  float tot[4];                // log-decay of a block
  // per token of the chunk; "far" = towards the tokens that attend to it
  float off[kC];               // decay from the token to the far edge of its block
  float dcol[kC], drow[kC];    // factors of a block's own decays: exp(+-(gam - mid)), mid the middle of its range
  float edge[kC];              // log-decay from the near edge of its block to the token
  float st[kC];                // decay between the state and the token, times f_st
  float hi[kC], lo[kC];        // prefix sums, for the pairwise decays
};
static_assert(offsetof(Entry, off) % 16 == 0 && offsetof(Entry, tot) % 16 == 0, "moved as float4");
constexpr int kEntries = 2;
constexpr uint32_t kOffOut = (kTok + kSt) * kTile + kEntries * sizeof(Entry);   // 4 KB for each output warp
constexpr uint32_t kSmemBytes = kOffOut + 4 * 4096 + 1024;
static_assert(kSmemBytes <= 226 * 1024, "shared memory");

struct Item {
  int h, L, tok, state;   // state: index among the states
};

// The item's chunk, or false where no chunk uses its slot.
__device__ __forceinline__ bool locate(const Params& p, int i, Item& it) {
  it.state = i;
  const int slot = i / p.gates.Hv;
  it.h = i - slot * p.gates.Hv;
  int lo = 0, hi = p.seqs.N - 1;   // the last sequence whose slots start at or before this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int)p.seqs.slot0(mid) <= slot) lo = mid;
    else hi = mid - 1;
  }
  const int t0 = (int)p.seqs.start(lo), len = (int)p.seqs.len(lo), c = slot - (t0 / kC + lo);
  if (c < 0 || c > (len - 1) / kC || len == 0) return false;
  it.L = min(len - c * kC, kC);
  it.tok = t0 + c * kC;
  return true;
}

struct Shared {
  uint64_t tfull[kTok], tempty[kTok], sfull[kSt], sempty[kSt];
  uint64_t gfull[kEntries], gempty[kEntries];
  uint64_t sc, oi, oo, pr, ofree;   // scores done, state part done, P c done, P written, accumulators read
  uint64_t drain;
  uint32_t tmem;
  int dead;                          // a wait gave up: every role winds down
};

// Four K = 16 steps of a product from shared memory.
__device__ __forceinline__ void mma4(uint32_t d, uint64_t a, uint32_t astep, uint64_t b, uint32_t bstep, uint32_t idesc,
                                     bool first, uint32_t me) {
#pragma unroll
  for (int s = 0; s < 4; ++s) mma_bf16_w(d, dadv(a, s * astep), dadv(b, s * bstep), idesc, !first || s > 0, me);
}

__global__ void __launch_bounds__(kThreads, 1)
la_out_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) Shared sh;
  const uint32_t raw = tc::smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* const sm = smem_raw + (sbase - raw);
  Entry* const entries = reinterpret_cast<Entry*>(sm + (kTok + kSt) * kTile);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int items = p.slots * p.gates.Hv;
  const uint32_t sstate = sbase + kTok * kTile;

  if (tid == 0) {
    for (int i = 0; i < kTok; ++i) {
      tc::mbar_init(tc::smem_u32(&sh.tfull[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh.tempty[i]), 1);
    }
    for (int i = 0; i < kSt; ++i) {
      tc::mbar_init(tc::smem_u32(&sh.sfull[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh.sempty[i]), 1);
    }
    for (int i = 0; i < kEntries; ++i) {
      tc::mbar_init(tc::smem_u32(&sh.gfull[i]), 32);
      tc::mbar_init(tc::smem_u32(&sh.gempty[i]), 1 + 256 + 128);
    }
    tc::mbar_init(tc::smem_u32(&sh.sc), 1);
    tc::mbar_init(tc::smem_u32(&sh.oi), 1);
    tc::mbar_init(tc::smem_u32(&sh.oo), 1);
    tc::mbar_init(tc::smem_u32(&sh.drain), 1);
    tc::mbar_init(tc::smem_u32(&sh.pr), 256);
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
  dependents_may_start();
  // the token tiles and gates are the call's own inputs, so their first ones are fetched during the walks; the
  // states, all that is written, and every wait for another warp come after
  if (tid != 0 && warp != 2) dependency_wait();

  if (tid == 0 || tid == 96) {
    // ---- loads: thread 0 the token tiles, thread 96 the state tiles, each as its slot falls free ----
    const bool toks = tid == 0;
    const int ring = toks ? kTok : kSt, per = toks ? p.ntok : p.nst;
    uint64_t* const full = toks ? sh.tfull : sh.sfull;
    uint64_t* const empty = toks ? sh.tempty : sh.sempty;
    const uint32_t base = toks ? sbase : sstate;
    int x = 0, slot = 0, turn = 0;   // tiles issued, x % ring, (x / ring) & 1
    for (int i = blockIdx.x; i < items && ok; i += gridDim.x) {
      Item it;
      if (!locate(p, i, it)) continue;
#pragma unroll 1
      for (int j = 0; j < per; ++j) {
        if (toks && x == kTok) dependency_wait();
        if (!(ok = wait(sh.dead, empty[slot], turn ^ 1))) break;
        const uint32_t dst = base + slot * kTile, bar = tc::smem_u32(&full[slot]);
        if (toks) {
          const int m = p.tok[j], D = p.width[m], hh = it.h / (p.gates.Hv / p.heads[m]);
          tc::mbar_expect_tx(bar, D / 64 * kBlk);
          for (int b = 0; b < D / 64; ++b) tc::tma_load_3d(dst + b * kBlk, &maps.t[m], bar, 64 * b, hh, it.tok);
        } else {
          const int w = p.st[j], row = (it.state * 2 + p.term[j]) * p.dk * (p.dv / 64);
          tc::mbar_expect_tx(bar, p.dk * p.dv * 2);
          for (int b = 0; b < p.dv / 64; ++b) tc::tma_load_2d(dst + b * p.dk * 128, &maps.s[w], bar, 0, row + b * p.dk);
        }
        ++x;
        if (++slot == ring) {
          slot = 0;
          turn ^= 1;
        }
      }
    }
    // no copy may be in flight when the CTA ends
    for (int y = max(0, x - ring); y < x; ++y)
      tc::mbar_wait(tc::smem_u32(&full[y % ring]), (y / ring) & 1, 1u << 22);
  } else if (warp == 2) {
    // ---- gates: prefix sums and decay factors, one item ahead of the warps that use them ----
    uint32_t k = 0;
    int i = blockIdx.x, role = 0;
    Item it;
    auto advance = [&] {
      while (i < items && !locate(p, i, it)) i += gridDim.x;
    };
    advance();
    float gx[4];
    if (i < items) p.gates.load(gx, it.tok, it.h, it.L, lane);
    while (true) {
      const bool more = i < items;
      const uint32_t s = k % kEntries;
      if (k == kEntries) dependency_wait();
      ok = wait(sh.dead, sh.gempty[s], ((k / kEntries) & 1) ^ 1);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      Entry& e = entries[s];
      if (more) {
        const Role& r = p.role[role];
        const bool rev = r.reverse;
        Gates g;
        scan_gates(gx, g, lane);
        if (lane == 0) {
          e.tok = it.tok;
          e.L = it.L;
          e.h = it.h;
          e.role = role;
        }
        // a block's own decays in two factors, both within exp(+-32), their product as exact as the prefix
        // sums, while its range is at most 64; else pair by pair
        float mx = g.pre(0), mn = mx;
#pragma unroll
        for (int q = 1; q < 4; ++q) {
          mx = fmaxf(mx, g.pre(q));
          mn = fminf(mn, g.pre(q));
        }
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) {
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
          mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
        }
        const float mid = 0.5f * (mx + mn);
        const uint32_t wide = __ballot_sync(0xffffffffu, !(mx - mn <= 64.f));
        const float near = rev ? g.blocks_after(lane) : g.blocks_before(lane);   // from the state to this block
        float4 off4, dr, dcl, ed, st;
        float* const po = &off4.x;
        float* const pr = &dr.x;
        float* const pc = &dcl.x;
        float* const pe = &ed.x;
        float* const ps = &st.x;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float pre = g.pre(q), aft = g.after(q);
          const float d = (g.hi[q] - mid) + g.lo[q];
          const float up = expf(d), down = expf(-d);
          po[q] = 4 * lane + q < it.L ? expf(rev ? pre : aft) : 0.f;
          pr[q] = rev ? down : up;
          pc[q] = rev ? up : down;
          pe[q] = rev ? aft : pre;
          ps[q] = r.f_st * expf((rev ? aft : pre) + near);
        }
        *reinterpret_cast<float4*>(e.off + 4 * lane) = off4;
        *reinterpret_cast<float4*>(e.drow + 4 * lane) = dr;
        *reinterpret_cast<float4*>(e.dcol + 4 * lane) = dcl;
        *reinterpret_cast<float4*>(e.edge + 4 * lane) = ed;
        *reinterpret_cast<float4*>(e.st + 4 * lane) = st;
        *reinterpret_cast<float4*>(e.hi + 4 * lane) = make_float4(g.hi[0], g.hi[1], g.hi[2], g.hi[3]);
        *reinterpret_cast<float4*>(e.lo + 4 * lane) = make_float4(g.lo[0], g.lo[1], g.lo[2], g.lo[3]);
        if (lane == 0) {
          *reinterpret_cast<float4*>(e.tot) = make_float4(g.tot(0), g.tot(1), g.tot(2), g.tot(3));
          e.pairwise = (wide & 1) | (wide >> 8 & 1) << 1 | (wide >> 16 & 1) << 2 | (wide >> 24 & 1) << 3;
        }
        if (++role == p.roles) {
          role = 0;
          i += gridDim.x;
          advance();
          if (i < items) p.gates.load(gx, it.tok, it.h, it.L, lane);
        }
      } else if (lane == 0) {
        e.L = 0;
      }
      tc::mbar_arrive(tc::smem_u32(&sh.gfull[s]));
      ++k;
      if (!more) break;
    }
  } else if (warp == 1) {
    // ---- products: the warp stays converged, one lane issues ----
    uint32_t x = 0, y = 0, k = 0;   // tiles of the chunks before; roles done
    const uint32_t me = elect_one();
    auto ttile = [&](int j) { return sbase + ((x + j) % kTok) * kTile; };
    auto stile = [&](int j) { return sstate + ((y + j) % kSt) * kTile; };
    auto tlanded = [&](int j) { ok = ok && wait(sh.dead, sh.tfull[(x + j) % kTok], ((x + j) / kTok) & 1); };
    auto slanded = [&](int j) { ok = ok && wait(sh.dead, sh.sfull[(y + j) % kSt], ((y + j) / kSt) & 1); };
    auto trelease = [&](int j) { mma_commit_w(tc::smem_u32(&sh.tempty[(x + j) % kTok]), me); };
    auto srelease = [&](int j) { mma_commit_w(tc::smem_u32(&sh.sempty[(y + j) % kSt]), me); };
    auto good = [&] { return ok = __all_sync(0xffffffffu, ok); };
    while (true) {
      const uint32_t gs = k % kEntries;
      ok = wait(sh.dead, sh.gfull[gs], (k / kEntries) & 1);
      if (!good()) break;
      const int role = entries[gs].role;
      const bool more = entries[gs].L > 0;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.gempty[gs]));
      if (!more) break;
      const Role& r = p.role[role];
      const bool dg = r.e >= 0;
      const int na = p.width[p.tok[r.a]] / 64, nc = p.width[p.tok[r.c]] / 64;
      // [128 x D] [128 x D]^T, both K-major
      auto scores = [&](uint32_t d, uint32_t ta, uint32_t tb, int blocks) {
        const uint64_t ad = tc::make_sdesc(ta, 16, 1024), bd = tc::make_sdesc(tb, 16, 1024);
        constexpr uint32_t idesc = tc::make_idesc(tc::kKindBF16, 128, 128, false, false);
#pragma unroll 1
        for (int b = 0; b < blocks; ++b)
          mma4(tmem + d, dadv(ad, b * kBlk), 32, dadv(bd, b * kBlk), 32, idesc, b == 0, me);
      };
      tlanded(r.b);
      tlanded(r.a);
      if (k > 0) ok = ok && wait(sh.dead, sh.oo, (k - 1) & 1);   // P of the item before is consumed
      if (!good()) break;
      tc::tc_fence_after();
      scores(TM_S, ttile(r.a), ttile(r.b), na);
      if (r.done & 2) trelease(r.b);
      if (dg) {
        tlanded(r.c);
        tlanded(r.e);
        if (!good()) break;
        scores(TM_E, ttile(r.e), ttile(r.c), nc);
      }
      mma_commit_w(tc::smem_u32(&sh.sc), me);
      slanded(r.st);
      slanded(r.st + 1);
      if (k > 0) ok = ok && wait(sh.dead, sh.ofree, (k - 1) & 1);
      if (!good()) break;
      tc::tc_fence_after();
      // a St: St [da x dc] is stored as rows of the key channel, 64 value columns each
      const uint32_t sblk = p.dk * 128;   // a block of 64 value columns
      // transposed: K = value columns (K-major), N = key channels; else K = key channels, N = value columns (MN-major)
      const uint32_t idesc_s = r.st_transposed ? tc::make_idesc(tc::kKindBF16, 128, p.dk, false, false)
                                               : tc::make_idesc(tc::kKindBF16, 128, p.dv, false, true);
      const uint32_t lbo = r.st_transposed ? 16 : sblk, kstep = r.st_transposed ? 32 : 2048;
      const uint32_t kblk = r.st_transposed ? sblk : 8192;
      const uint64_t ad = tc::make_sdesc(ttile(r.a), 16, 1024);
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        const uint64_t bd = tc::make_sdesc(stile(r.st + t), lbo, 1024);
#pragma unroll 1
        for (int b = 0; b < na; ++b)
          mma4(tmem + TM_I, dadv(ad, b * kBlk), 32, dadv(bd, b * kblk), kstep, idesc_s, t + b == 0, me);
      }
      // tiles read by the output warps too (e) are released a role later, after the wait on ofree above
      if (r.done & 1) trelease(r.a);
      if (r.done & 16) srelease(r.st);
      if (r.done & 32) srelease(r.st + 1);
      mma_commit_w(tc::smem_u32(&sh.oi), me);
      tlanded(r.c);
      ok = ok && wait(sh.dead, sh.pr, k & 1);
      if (!good()) break;
      tc::tc_fence_after();
      {
        const uint64_t bd = tc::make_sdesc(ttile(r.c), kBlk, 1024);
        const uint32_t idesc = tc::make_idesc(tc::kKindBF16, 128, 64 * nc, false, true);
#pragma unroll 1
        for (int t = 0; t < 2; ++t)   // P's terms: 16 columns each of a block's 32
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_bf16_ta(tmem + TM_O, tmem + TM_S + 16 * t + 32 * (ks >> 1) + 8 * (ks & 1), dadv(bd, ks * 2048), idesc,
                        t + ks > 0, me);
        if (r.done & 4) trelease(r.c);
        mma_commit_w(tc::smem_u32(&sh.oo), me);
      }
      if (role == p.roles - 1) {
        x += p.ntok;
        y += p.nst;
      }
      ++k;
    }
    // the products in flight end before the tensor memory goes
    if (!ok) {
      __syncwarp();
      mma_commit_w(tc::smem_u32(&sh.drain), me);
      tc::mbar_wait(tc::smem_u32(&sh.drain), 0, 1u << 22);
    } else if (k > 0) {
      ok = wait(sh.dead, sh.oo, (k - 1) & 1);
    }
  } else if (warp >= 4 && warp < 12) {
    // ---- scores -> weighted, masked, bf16 P; with e the pair sums of dg. Two warps for 32 rows, 64 columns each ----
    const int w = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane0 = 32u * w;
    const int row = 32 * w + lane;
    uint32_t x = 0, k = 0;
    while (true) {
      const uint32_t gs = k % kEntries;
      ok = wait(sh.dead, sh.gfull[gs], (k / kEntries) & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const Entry& e = entries[gs];
      const int L = e.L;
      if (L == 0) break;
      const Role& r = p.role[e.role];
      const bool dg = r.e >= 0, rev = r.reverse;
      const float edge = e.edge[row], drow = e.drow[row];
      const int pairwise = (e.pairwise >> w) & 1;
      ok = wait(sh.dead, sh.sc, k & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      tc::tc_fence_after();
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int j = 2 * half; j < 2 * half + 2; ++j) {
        uint32_t u[16];
        const uint32_t pcol = tc::tmem_addr(tmem, lane0, TM_S + 32 * j);   // P's terms over the block's own scores
        if (rev ? j < w : j > w) {
#pragma unroll
          for (int c = 0; c < 16; ++c) u[c] = 0;
          tmem_st16u(pcol, u);
          tmem_st16u(pcol + 16, u);
          continue;
        }
        const bool diag = j == w;
        // columns of this block that the row takes: tokens past the chunk's end may hold anything
        uint32_t mask = 0xffffffffu;
        if (rev && L - 32 * j < 32) mask = L > 32 * j ? (1u << (L - 32 * j)) - 1u : 0u;
        if (diag) mask &= rev ? 0xffffffffu << lane : 0xffffffffu >> (31 - lane);
        float f = drow;
        if (!diag) {   // from this row to the block's near edge
          float z = edge;
#pragma unroll
          for (int m = 1; m < 3; ++m)
            if (rev ? (m > w && m < j) : (m > j && m < w)) z += e.tot[m];
          f = expf(z);
        }
        const float* cf = (diag ? e.dcol : e.off) + 32 * j;
        float v[32];
        ld32(tmem, lane0, TM_S + 32 * j, v);
        if (diag && pairwise) {
          const float hr = e.hi[row], lr = e.lo[row];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float d = (hr - e.hi[32 * j + c]) + (lr - e.lo[32 * j + c]);
            v[c] = (mask >> c) & 1 ? v[c] * __expf(rev ? -d : d) : 0.f;
          }
        } else {
          const float2 f2 = make_float2(f, f);
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 cc = *reinterpret_cast<const float4*>(cf + c);
            const float2 a = __fmul2_rn(make_float2(v[c], v[c + 1]), __fmul2_rn(f2, make_float2(cc.x, cc.y)));
            const float2 b = __fmul2_rn(make_float2(v[c + 2], v[c + 3]), __fmul2_rn(f2, make_float2(cc.z, cc.w)));
            v[c] = (mask >> c) & 1 ? a.x : 0.f;
            v[c + 1] = (mask >> (c + 1)) & 1 ? a.y : 0.f;
            v[c + 2] = (mask >> (c + 2)) & 1 ? b.x : 0.f;
            v[c + 3] = (mask >> (c + 3)) & 1 ? b.y : 0.f;
          }
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) u[c] = pack_bf16(v[2 * c], v[2 * c + 1]);
        tmem_st16u(pcol, u);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float2 low = __ffma2_rn(unpack_bf16(u[c]), make_float2(-1.f, -1.f), make_float2(v[2 * c], v[2 * c + 1]));
          u[c] = pack_bf16(low.x, low.y);
        }
        tmem_st16u(pcol + 16, u);
        if (dg) {
          if (diag) mask &= ~(1u << lane);   // pairs of different tokens
          float ev[32];
          ld32(tmem, lane0, TM_E + 32 * j, ev);
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            ev[c] = (mask >> c) & 1 ? ev[c] : 0.f;
            ev[c + 1] = (mask >> (c + 1)) & 1 ? ev[c + 1] : 0.f;
            sum = __ffma2_rn(make_float2(v[c], v[c + 1]), make_float2(ev[c], ev[c + 1]), sum);
          }
        }
      }
      tc::tmem_st_wait();
      const int64_t at = (int64_t)(e.tok + row) * p.gates.Hv + e.h;
      if (L < kC) {   // rows past the end of c would meet zero weights: not with a NaN
        const uint32_t xc = x + r.c;
        ok = wait(sh.dead, sh.tfull[xc % kTok], (xc / kTok) & 1);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (half == 0) zero_tail_rows(sm + (xc % kTok) * kTile, p.width[p.tok[r.c]] / 64, tid - 128, L);
        tc::fence_proxy_async_smem();
      }
      tc::tc_fence_before();
      tc::mbar_arrive(tc::smem_u32(&sh.pr));
      const int role = e.role;
      tc::mbar_arrive(tc::smem_u32(&sh.gempty[gs]));
      if (dg && row < L) r.dot_in[half * p.dot_stride + at] = r.f_in * (sum.x + sum.y);
      if (role == p.roles - 1) x += p.ntok;
      ++k;
    }
  } else if (warp >= 12) {
    // ---- outputs ----
    const int w = warp - 12;
    unsigned char* const stage = sm + kOffOut + 4096 * w;
    const uint32_t lane0 = 32u * w;
    const int row = 32 * w + lane;
    uint32_t x = 0, k = 0;
    while (true) {
      const uint32_t gs = k % kEntries;
      ok = wait(sh.dead, sh.gfull[gs], (k / kEntries) & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const Entry& e = entries[gs];
      const int L = e.L;
      if (L == 0) break;
      const int role = e.role;
      const Role& r = p.role[role];
      const bool dg = r.e >= 0;
      const int nb = p.width[p.tok[r.c]] / 32;
      const float fs = e.st[row], fi = r.f_in;
      const int64_t at = (int64_t)(e.tok + row) * p.gates.Hv + e.h;
      tc::mbar_arrive(tc::smem_u32(&sh.gempty[gs]));
      ok = wait(sh.dead, sh.oi, k & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      tc::tc_fence_after();
      if (dg) {
        const uint32_t xe = x + r.e;
        ok = wait(sh.dead, sh.tfull[xe % kTok], (xe / kTok) & 1);   // landed long ago; makes it visible here
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const unsigned char* et = sm + (xe % kTok) * kTile;
        float2 dot[2] = {};
#pragma unroll 1
        for (int b = 0; b < nb; ++b) {
          float v[32];
          ld32(tmem, lane0, TM_I + 32 * b, v);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 q = *reinterpret_cast<const uint4*>(et + (b >> 1) * kBlk + tc::sw128(row, 64 * (b & 1) + 16 * c));
            const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int h = 0; h < 4; ++h)
              dot[h & 1] = __ffma2_rn(unpack_bf16(u[h]), make_float2(v[8 * c + 2 * h], v[8 * c + 2 * h + 1]), dot[h & 1]);
          }
        }
        if (row < L) r.dot_st[at] = fs * ((dot[0].x + dot[0].y) + (dot[1].x + dot[1].y));
      }
      ok = wait(sh.dead, sh.oo, k & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      tc::tc_fence_after();
      const float2 fs2 = make_float2(fs, fs), fi2 = make_float2(fi, fi);
      // 128-byte pieces of the 32 rows go through shared memory, so that a store instruction covers whole
      // lines of 4 rows instead of 16 bytes in each of 32
      const int esz = r.out_f32 ? 4 : 2;
      const int64_t rstride = (int64_t)p.gates.Hv * 32 * nb * esz;
      unsigned char* dst = static_cast<unsigned char*>(r.out) + (at - (int64_t)(lane - (lane >> 3)) * p.gates.Hv) * (32 * nb * esz) +
                           (lane & 7) * 16;   // row 32 w + lane / 8, piece lane % 8
      auto flush = [&] {
        __syncwarp();
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const int q = 4 * m + (lane >> 3);
          const uint4 x16 = *reinterpret_cast<const uint4*>(stage + q * 128 + (((lane & 7) ^ (q & 7)) << 4));
          if (32 * w + q < L) *reinterpret_cast<uint4*>(dst + 4 * m * rstride) = x16;
        }
        dst += 128;
        __syncwarp();
      };
#pragma unroll 1
      for (int b = 0; b < nb; ++b) {
        float v[32], s[32];
        ld32(tmem, lane0, TM_O + 32 * b, v);
        ld32(tmem, lane0, TM_I + 32 * b, s);
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float2 o = __ffma2_rn(fs2, make_float2(s[c], s[c + 1]), __fmul2_rn(fi2, make_float2(v[c], v[c + 1])));
          v[c] = o.x;
          v[c + 1] = o.y;
        }
        if (r.out_f32) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<float4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) =
                make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
          flush();
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * (b & 1) + c) ^ (lane & 7)) << 4)) = pack8(v + 8 * c);
          if (b & 1) flush();
        }
      }
      tc::tc_fence_before();
      tc::mbar_arrive(tc::smem_u32(&sh.ofree));
      if (role == p.roles - 1) x += p.ntok;
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
  const int64_t tokens = (int64_t)p.B * p.T, slots = la_slots(p), items = slots * p.Hv;   // < 2^22
  if (tokens == 0 || items == 0) return cudaSuccess;
  Maps m;
  Params o{};
  o.seqs = {p.cu, p.T, p.N};
  o.gates = {p.g, p.Hv, p.head_decay};
  const int heads[4] = {p.Hqk, p.Hqk, p.Hv, p.Hv}, width[4] = {p.dk, p.dk, p.dv, p.dv};
  for (int i = 0; i < r.roles; ++i) o.role[i] = r.role[i];
  for (int i = 0; i < 4; ++i) {
    o.heads[i] = heads[i];
    o.width[i] = width[i];
    o.tok[i] = r.tok[i];
    o.st[i] = r.st[i];
    o.term[i] = r.term[i];
    if (!r.tensor[i]) m.t[i] = m.t[0];   // not used
    else if (!make_bf16_map(&m.t[i], r.tensor[i], width[i], heads[i], tokens, kC)) return cudaErrorNotSupported;
  }
  for (int i = 0; i < 2; ++i) {
    if (!r.states[i]) m.s[i] = m.s[0];   // not used
    else if (!make_bf16_rows_map(&m.s[i], r.states[i], slots * p.Hv * 2 * p.dk * (p.dv / 64), p.dk))
      return cudaErrorNotSupported;
  }
  o.dot_stride = tokens * p.Hv;
  o.ntok = r.ntok;
  o.nst = r.nst;
  o.status = status;
  o.slots = (int)slots;
  o.roles = r.roles;
  o.dk = p.dk;
  o.dv = p.dv;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(la_out_kernel, kSmemBytes, allowed);
  if (e != cudaSuccess) return e;
  return launch(true, la_out_kernel, dim3((unsigned)std::min<int64_t>(items, kSMs)), kThreads, kSmemBytes, stream, m, o);
}

}  // namespace la
}  // namespace gdn

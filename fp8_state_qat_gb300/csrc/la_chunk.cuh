// la_chunk.cuh -- pieces shared by the chunked linear-attention kernels (128-token chunks).
#pragma once

#include <atomic>

#include "common.cuh"
#include "la.h"
#include "pdl.cuh"
#include "tc_common.cuh"
#include "tc_epilogue.cuh"

namespace gdn {
namespace la {

constexpr int kC = 128;                      // tokens a chunk: the M of one full tcgen05 product
constexpr uint32_t kBlk = 16 * 1024;         // a [128 tokens][64 channels] bf16 block, 128-byte rows
constexpr uint32_t kTile = 2 * kBlk;

// The chunk slots of sequence n start at start(n) / 128 + n: unique, and known without a table.
struct Seqs {
  const int32_t* cu;   // device cu_seqlens, or null: N sequences of T tokens
  int T, N;
  __device__ __forceinline__ int64_t start(int n) const { return cu ? (int64_t)cu[n] : (int64_t)n * T; }
  __device__ __forceinline__ int64_t len(int n) const { return cu ? (int64_t)cu[n + 1] - cu[n] : (int64_t)T; }
  __device__ __forceinline__ int64_t slot0(int n) const { return start(n) / kC + n; }
};

// exp(g) below -110 is zero in fp32; the bound keeps prefix sums finite where g = -inf resets a state
// (a NaN stays one)
__device__ __forceinline__ float gate(float g) { return g < -110.f ? -110.f : g; }

// Prefix sums of a chunk's log-decays within its four 32-token blocks, by one warp: lane l holds the
// four tokens 4 l + q, so a block is eight lanes. Each sum is a pair hi + lo, so that a difference of two
// of them keeps its accuracy when a large |g| (a reset) lies before both; decays across blocks are
// products of exponentials of sums <= 0 of such differences, so nothing overflows and nothing cancels.
struct Gates {
  float hi[4], lo[4];   // inclusive prefix of the block
  float thi[4], tlo[4]; // the total of block j
  float bhi, blo;       // of this lane's block
  __device__ __forceinline__ float tot(int j) const { return thi[j] + tlo[j]; }
  // sum over the tokens after token q, up to its block's end
  __device__ __forceinline__ float after(int q) const { return (bhi - hi[q]) + (blo - lo[q]); }
  __device__ __forceinline__ float pre(int q) const { return hi[q] + lo[q]; }
  // sums over the blocks before / after this lane's
  __device__ __forceinline__ float blocks_before(int lane) const {
    const int j = lane >> 3;
    return j > 1 ? (j > 2 ? (tot(0) + tot(1)) + tot(2) : tot(0) + tot(1)) : (j ? tot(0) : 0.f);
  }
  __device__ __forceinline__ float blocks_after(int lane) const {
    const int j = lane >> 3;
    return j < 2 ? (j < 1 ? (tot(1) + tot(2)) + tot(3) : tot(2) + tot(3)) : (j < 3 ? tot(3) : 0.f);
  }
};

struct GateSrc {
  const float* g;
  int Hv, head_decay;
  __device__ __forceinline__ void load(float (&x)[4], int64_t tok, int h, int L, int lane) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t = 4 * lane + q;
      x[q] = t < L ? (head_decay ? g[h] : g[(tok + t) * Hv + h]) : 0.f;   // not touched here: still in flight
    }
  }
};

// (s, e) + (ys, ye) with s = fl(s + ys) and the rounding error carried in e
__device__ __forceinline__ void add_pair(float& s, float& e, float ys, float ye) {
  const float t = __fadd_rn(s, ys), b = __fsub_rn(t, s);
  e += ye + __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(ys, b));
  s = t;
}

__device__ __forceinline__ void scan_gates(const float (&x)[4], Gates& w, int lane) {
  w.hi[0] = gate(x[0]);
  w.lo[0] = 0.f;
#pragma unroll
  for (int q = 1; q < 4; ++q) {
    w.hi[q] = gate(x[q]);
    w.lo[q] = 0.f;
    add_pair(w.hi[q], w.lo[q], w.hi[q - 1], w.lo[q - 1]);
  }
  float s = w.hi[3], e = w.lo[3];   // of the lanes before, within the block
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) {
    const float ys = __shfl_up_sync(0xffffffffu, s, off, 8), ye = __shfl_up_sync(0xffffffffu, e, off, 8);
    if ((lane & 7) >= off) add_pair(s, e, ys, ye);
  }
  const float ps = __shfl_up_sync(0xffffffffu, s, 1, 8), pe = __shfl_up_sync(0xffffffffu, e, 1, 8);
  if (lane & 7) {
#pragma unroll
    for (int q = 0; q < 4; ++q) add_pair(w.hi[q], w.lo[q], ps, pe);
  }
  // the block's total as its last token's prefix, so that nothing is left after that token
  w.bhi = __shfl_sync(0xffffffffu, w.hi[3], lane | 7);
  w.blo = __shfl_sync(0xffffffffu, w.lo[3], lane | 7);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w.thi[j] = __shfl_sync(0xffffffffu, w.bhi, 8 * j);
    w.tlo[j] = __shfl_sync(0xffffffffu, w.blo, 8 * j);
  }
}

// tcgen05 products issued by the one lane of a converged warp whose `me` is set: the whole warp walks the
// issuing code, so that its descriptors stay in uniform registers (inside a one-lane branch every product
// moved them there anew and took about 130 cycles to issue).
__device__ __forceinline__ void mma_bf16_w(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate, uint32_t me) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0; "
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(me)
      : "memory");
}
// with A in tensor memory (lane = row of A, each 32-bit column two bf16 of K)
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate, uint32_t me) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0; "
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(me)
      : "memory");
}
__device__ __forceinline__ void mma_commit_w(uint32_t mbar, uint32_t me) {
  asm volatile(
      "{ .reg .pred q; setp.ne.b32 q, %1, 0; "
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(mbar), "r"(me)
      : "memory");
}
// copies likewise
__device__ __forceinline__ void mbar_expect_w(uint32_t addr, uint32_t bytes, uint32_t me) {
  asm volatile(
      "{ .reg .pred q; .reg .b64 st; setp.ne.b32 q, %2, 0; @q mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1; }" ::"r"(addr),
      "r"(bytes), "r"(me)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_w(uint32_t dst, const CUtensorMap* map, uint32_t mbar, int c0, int c1, int c2,
                                              uint32_t me) {
  asm volatile(
      "{ .reg .pred q; setp.ne.b32 q, %6, 0; @q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2]; }" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar), "r"(c0), "r"(c1), "r"(c2), "r"(me)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t me;
  asm volatile("{ .reg .pred q; elect.sync _|q, 0xffffffff; selp.u32 %0, 1, 0, q; }" : "=r"(me));
  return me;
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// rows [L, 128) of a tile of `blocks` [128][64] blocks become zero (thread t of 128: row t)
__device__ __forceinline__ void zero_tail_rows(unsigned char* tile, int blocks, int t, int L) {
  if (t >= L && t < kC) {
    for (int b = 0; b < blocks; ++b)
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(tile + b * kBlk + (t >> 3) * 1024 + (t & 7) * 128 + c * 16) = make_uint4(0, 0, 0, 0);
  }
}

// Bounded wait that also ends when another warp has given up (`dead`, in shared memory).
static __device__ __noinline__ bool wait_slow(int* dead, uint32_t a, uint32_t parity) {
  for (uint32_t i = 0; i < GDN_WAIT_LIMIT; ++i) {
    if (tc::mbar_try_wait(a, parity)) return true;
    if (*(volatile int*)dead) return false;
  }
  *(volatile int*)dead = 1;
  return false;
}
__device__ __forceinline__ bool wait(int& dead, uint64_t& bar, uint32_t parity) {
  const uint32_t a = tc::smem_u32(&bar);
  if (GDN_WAIT_LIMIT > 0 && tc::mbar_try_wait(a, parity)) return true;
  return wait_slow(&dead, a, parity);
}

// cudaFuncSetAttribute(MaxDynamicSharedMemorySize), once per kernel and device
template <class K>
inline cudaError_t allow_smem(K kernel, uint32_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// ---- launchers of the parts (la_state.cu, la_out.cu) ----
// States at chunk boundaries, two bf16 terms (hi, lo) per item = slot * Hv + h: [term][dv / 64][dk][64].
struct StateRun {
  const void* x;        // bf16 [tokens, Hqk, dk]: k forwards, q backwards
  const void* y;        // bf16 [tokens, Hv, dv]: v forwards, dout backwards
  const float* s0;      // [N, Hv, dk, dv] or null
  float* sT;            // [N, Hv, dk, dv] or null
  void* states;         // the state before each chunk's own contribution, or null
  int reverse;
  float scale;          // weight of every token's contribution
  float* seg_tot;       // split walks: [N Hv][nseg][dk][dv]
  float* seg_dec;       // [N Hv][nseg]
  const void* other;    // the states S of the chunks, or null: then exp(gam_C) <S, state before the chunk>
  float* edge;          // per item goes here, in edge_parts() parts
  int beside;           // the launch before it may still run: nothing that it writes is read
};
int edge_parts(const LaProblem& p);
int state_segments(const LaProblem& p);
int most_segments(const LaProblem& p);   // of any packing of these sizes
bool walks_beside(const LaProblem& p);
// dependent: the launch before it in the stream is one of these kernels
cudaError_t launch_states(const LaProblem& p, const StateRun& r, int* status, bool dependent, cudaStream_t stream);

// One family of outputs: out_t = f_in sum_s decay(t, s) (a_t . b_s) c_s + f_st decay_t a_t^T St,
// s <= t with the state before the chunk (reverse 0), or s >= t with the state after it (reverse 1).
// The operands are tiles of the chunk, by their places in OutRun's lists.
struct Role {
  int a, b, c, e;        // token tiles; e: rows dotted with the outputs, or -1
  int st;                // first of the two tiles of the state's terms
  int done;              // tiles that no later role of the chunk reads: bits 0-2 a, b, c; bits 4, 5 the state terms
  int st_transposed;     // St = S^T: the product is over the value columns
  int reverse;
  float f_in, f_st;
  void* out;             // bf16 [tokens, Hv, dc] (fp32 with out_f32)
  int out_f32;
  float* dot_in;         // with e: sum_{s != t} decay (a_t . b_s) (e_t . c_s) f_in per (token, head), in two parts
  float* dot_st;         // with e: e_t . (the state part of out_t)
};
struct OutRun {
  const void* tensor[4]; // q, k, v, dout
  const void* states[2]; // S, dS
  int ntok, tok[4];      // token tiles of a chunk, in the order of their release: which tensor
  int nst, st[4], term[4];   // state tiles: which states, which term
  Role role[3];
  int roles;
};
cudaError_t launch_outputs(const LaProblem& p, const OutRun& r, int* status, cudaStream_t stream);

int64_t la_slots(const LaProblem& p);

}  // namespace la
}  // namespace gdn

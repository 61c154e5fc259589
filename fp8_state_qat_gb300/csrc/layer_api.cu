// layer_api.cu -- the extern "C" surface of the linear-attention and norm operators: host-side
// validation, then the device probe, then the launches; a non-OK status means nothing was enqueued.
#include <initializer_list>

#include "common.cuh"
#include "kernels.h"
#include "la.h"

namespace {

using gdn::LaGrads;
using gdn::LaProblem;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
struct Span {
  const void* p;
  size_t n;
};
// Whether an output overlaps another output or an input.
bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (auto a = outs.begin(); a != outs.end(); ++a) {
    for (auto b = outs.begin(); b != a; ++b)
      if (overlaps(a->p, a->n, b->p, b->n)) return true;
    for (const Span& b : ins)
      if (overlaps(a->p, a->n, b.p, b.n)) return true;
  }
  return false;
}

struct LaSizes {
  size_t qk, vo, g, st;
};
LaSizes la_sizes(const la_chunk_args* a) {
  const size_t tokens = (size_t)a->B * a->T;
  return {tokens * a->Hqk * a->dk * 2, tokens * a->Hv * a->dv * 2,
          (a->flags & LA_FLAG_HEAD_DECAY ? 1 : tokens) * a->Hv * 4, (size_t)a->N * a->Hv * a->dk * a->dv * 4};
}

// sizes and flags only: what the workspace depends on
gdn_status validate_la_sizes(const la_chunk_args* a) {
  if (!a || a->B < 0 || a->T < 0 || a->N < 0 || a->Hqk <= 0 || a->Hv <= 0) return GDN_ERR_INVALID_ARG;
  if (a->Hv % a->Hqk || (a->flags & ~LA_FLAG_HEAD_DECAY)) return GDN_ERR_INVALID_ARG;
  if ((a->dk != 64 && a->dk != 128) || (a->dv != 64 && a->dv != 128)) return GDN_ERR_UNSUPPORTED_SHAPE;
  const int64_t tokens = (int64_t)a->B * a->T;
  // TMA coordinates are 32-bit: tokens, and the rows of the stored states (512 a chunk and head at most,
  // 64 KB: more would not fit the device either)
  if (tokens > 0x7fffffff - 256 || (tokens / 128 + a->N) * (int64_t)a->Hv > 0x3fffff) return GDN_ERR_INVALID_ARG;
  if (a->cu_seqlens) {
    if (a->B != 1 || a->N < 1 || !a->cu_seqlens_host) return GDN_ERR_INVALID_ARG;
    const int32_t* c = a->cu_seqlens_host;
    if (c[0] != 0 || c[a->N] != a->T) return GDN_ERR_INVALID_ARG;
    for (int n = 0; n < a->N; ++n)
      if (c[n + 1] < c[n]) return GDN_ERR_INVALID_ARG;
  } else if (a->N != a->B) {
    return GDN_ERR_INVALID_ARG;
  }
  return GDN_OK;
}

gdn_status validate_la(const la_chunk_args* a) {
  const gdn_status s = validate_la_sizes(a);
  if (s != GDN_OK) return s;
  if ((int64_t)a->B * a->T > 0) {
    if (!a->q || !a->k || !a->v || !a->g) return GDN_ERR_INVALID_ARG;
    if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->g, 4)) return GDN_ERR_INVALID_ARG;
  }
  if (!aligned(a->h0, 16) || !aligned(a->cu_seqlens, 4)) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

LaProblem problem_of(const la_chunk_args* a) {
  return {a->q, a->k, a->v, a->g, a->h0, a->cu_seqlens, a->o, a->hT, a->B, a->T, a->N, a->Hqk, a->Hv, a->dk, a->dv,
          a->scale, (a->flags & LA_FLAG_HEAD_DECAY) ? 1 : 0, a->cu_seqlens ? a->cu_seqlens_host : nullptr};
}

gdn_status done(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

bool dtype_ok(int32_t t) { return t == GDN_DTYPE_BF16 || t == GDN_DTYPE_F32; }
size_t size_of(int32_t t) { return t == GDN_DTYPE_F32 ? 4 : 2; }
gdn_status norm_sizes(int64_t rows, int32_t D, int32_t t, int32_t tw, float eps) {
  if (rows < 0 || D < 1 || !dtype_ok(t) || !dtype_ok(tw) || !(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  if (!gdn::norm_dim_ok(D)) return GDN_ERR_UNSUPPORTED_SHAPE;
  return rows > (int64_t)1 << 40 ? GDN_ERR_INVALID_ARG : GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_upload_i32(const int32_t* host, int32_t* device, int64_t n, gdn_stream_t stream) {
  if (n < 0 || (n > 0 && (!host || !device)) || !aligned(host, 4) || !aligned(device, 4)) return GDN_ERR_INVALID_ARG;
  const gdn_status s = gdn::check_device();
  return s != GDN_OK ? s : done(gdn::launch_upload_i32(host, device, n, (cudaStream_t)stream));
}

size_t la_chunk_fwd_workspace_size(const la_chunk_args* args) {
  return validate_la_sizes(args) == GDN_OK ? gdn::la_fwd_workspace(problem_of(args)) : 0;
}
size_t la_chunk_bwd_workspace_size(const la_chunk_args* args) {
  return validate_la_sizes(args) == GDN_OK ? gdn::la_bwd_workspace(problem_of(args)) : 0;
}

gdn_status la_chunk_fwd(const la_chunk_args* a, void* ws, size_t ws_bytes, gdn_stream_t stream) {
  gdn_status s = validate_la(a);
  if (s != GDN_OK) return s;
  const LaSizes z = la_sizes(a);
  if ((z.vo && !a->o) || !aligned(a->o, 16) || !aligned(a->hT, 16)) return GDN_ERR_INVALID_ARG;
  if (clash({{a->o, z.vo}}, {{a->q, z.qk}, {a->k, z.qk}, {a->v, z.vo}, {a->g, z.g}, {a->h0, z.st}, {a->hT, z.st}}) ||
      clash({{a->hT, z.st}}, {{a->q, z.qk}, {a->k, z.qk}, {a->v, z.vo}, {a->g, z.g},
                              {a->hT == a->h0 ? nullptr : a->h0, z.st}}))
    return GDN_ERR_INVALID_ARG;
  const LaProblem p = problem_of(a);
  if (!ws || ws_bytes < gdn::la_fwd_workspace(p)) return GDN_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(ws, 256)) return GDN_ERR_INVALID_ARG;
  if ((s = gdn::check_device()) != GDN_OK) return s;
  return done(gdn::launch_la_fwd(p, ws, (cudaStream_t)stream));
}

gdn_status la_chunk_bwd(const la_chunk_args* a, const la_chunk_grads* gr, void* ws, size_t ws_bytes,
                        gdn_stream_t stream) {
  gdn_status s = validate_la(a);
  if (s != GDN_OK) return s;
  if (!gr) return GDN_ERR_INVALID_ARG;
  const LaSizes z = la_sizes(a);
  if ((int64_t)a->B * a->T > 0 && (!gr->dout || !gr->dq || !gr->dk || !gr->dv)) return GDN_ERR_INVALID_ARG;
  if (z.g && !gr->dg) return GDN_ERR_INVALID_ARG;
  if (!aligned(gr->dout, 16) || !aligned(gr->dhT, 16) || !aligned(gr->dq, 16) || !aligned(gr->dk, 16) ||
      !aligned(gr->dv, 16) || !aligned(gr->dg, 4) || !aligned(gr->dh0, 16))
    return GDN_ERR_INVALID_ARG;
  if (clash({{gr->dq, z.qk}, {gr->dk, z.qk}, {gr->dv, z.vo}, {gr->dg, z.g}, {gr->dh0, z.st}},
            {{a->q, z.qk}, {a->k, z.qk}, {a->v, z.vo}, {a->g, z.g}, {a->h0, z.st}, {gr->dout, z.vo}, {gr->dhT, z.st}}))
    return GDN_ERR_INVALID_ARG;
  const LaProblem p = problem_of(a);
  if (!ws || ws_bytes < gdn::la_bwd_workspace(p)) return GDN_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(ws, 256)) return GDN_ERR_INVALID_ARG;
  if ((s = gdn::check_device()) != GDN_OK) return s;
  return done(gdn::launch_la_bwd(p, {gr->dout, gr->dhT, gr->dq, gr->dk, gr->dv, gr->dg, gr->dh0}, ws,
                                 (cudaStream_t)stream));
}

gdn_status la_decode_step(const void* q, const void* k, const void* v, const float* g, const float* state,
                          float* state_out, void* o, int32_t N, int32_t Hqk, int32_t Hv, int32_t dk, int32_t dv,
                          float scale, uint32_t flags, gdn_stream_t stream) {
  if (N < 0 || Hqk <= 0 || Hv <= 0 || Hv % Hqk) return GDN_ERR_INVALID_ARG;
  if (flags & ~(GDN_FLAG_STATE_QDQ | GDN_FLAG_STATE_INT8)) return GDN_ERR_INVALID_ARG;
  if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128 && dv != 256)) return GDN_ERR_UNSUPPORTED_SHAPE;
  if ((int64_t)N * Hv > 0x7fffffff / 4) return GDN_ERR_INVALID_ARG;
  if (N > 0) {
    if (!q || !k || !v || !g || !state || !state_out || !o) return GDN_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, 4) || !aligned(state, 16) ||
        !aligned(state_out, 16) || !aligned(o, 16))
      return GDN_ERR_INVALID_ARG;
    const size_t nq = (size_t)N * Hqk * dk * 2, nv = (size_t)N * Hv * dv * 2, ng = (size_t)N * Hv * 4,
                 ns = (size_t)N * Hv * dk * dv * 4;
    if (clash({{o, nv}}, {{q, nq}, {k, nq}, {v, nv}, {g, ng}, {state, ns}, {state_out, ns}}) ||
        clash({{state_out, ns}}, {{q, nq}, {k, nq}, {v, nv}, {g, ng}, {state_out == state ? nullptr : state, ns}}))
      return GDN_ERR_INVALID_ARG;
  }
  const gdn_status s = gdn::check_device();
  if (s != GDN_OK) return s;
  const int qdq = !(flags & GDN_FLAG_STATE_QDQ) ? 0 : (flags & GDN_FLAG_STATE_INT8) ? 2 : 1;
  return done(gdn::launch_la_decode(q, k, v, g, state, state_out, o, N, Hqk, Hv, dk, dv, scale, qdq,
                                    (cudaStream_t)stream));
}

gdn_status gated_norm_fwd(const void* x, int32_t x_dtype, const void* z, const void* w, int32_t w_dtype, void* y,
                          int64_t rows, int32_t D, float eps, gdn_stream_t stream) {
  gdn_status s = norm_sizes(rows, D, x_dtype, w_dtype, eps);
  if (s != GDN_OK) return s;
  if (rows > 0) {
    if (!x || !z || !w || !y || !aligned(x, size_of(x_dtype)) || !aligned(z, 2) || !aligned(w, size_of(w_dtype)) ||
        !aligned(y, 2))
      return GDN_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * D;
    if (clash({{y, n * 2}}, {{x, n * size_of(x_dtype)}, {z, n * 2}, {w, D * size_of(w_dtype)}})) return GDN_ERR_INVALID_ARG;
  }
  if ((s = gdn::check_device()) != GDN_OK) return s;
  if (rows == 0) return GDN_OK;
  return done(gdn::launch_gated_norm_fwd(x, x_dtype == GDN_DTYPE_F32, z, w, w_dtype == GDN_DTYPE_BF16, y, rows, D, eps,
                                         (cudaStream_t)stream));
}

size_t gated_norm_bwd_workspace_size(int64_t rows, int32_t D) {
  if (norm_sizes(rows, D, 0, 0, 0.f) != GDN_OK) return 0;
  return 256 + (size_t)gdn::norm_bwd_parts(rows, D) * D * 4;
}
size_t residual_norm_bwd_workspace_size(int64_t rows, int32_t D) {
  if (norm_sizes(rows, D, 0, 0, 0.f) != GDN_OK) return 0;
  return 256 + (size_t)gdn::norm_bwd_parts(rows, D) * D * 8;
}

gdn_status gated_norm_bwd(const void* dy, const void* x, int32_t x_dtype, const void* z, const void* w,
                          int32_t w_dtype, void* dx, void* dz, float* dw, int64_t rows, int32_t D, float eps,
                          void* ws, size_t ws_bytes, gdn_stream_t stream) {
  gdn_status s = norm_sizes(rows, D, x_dtype, w_dtype, eps);
  if (s != GDN_OK) return s;
  if (!dw || !w || !aligned(dw, 4) || !aligned(w, size_of(w_dtype))) return GDN_ERR_INVALID_ARG;
  const size_t n = (size_t)rows * D, nx = n * size_of(x_dtype), nw = D * size_of(w_dtype);
  if (rows > 0 && (!dy || !x || !z || !dx || !dz || !aligned(dy, 2) || !aligned(x, size_of(x_dtype)) ||
                   !aligned(z, 2) || !aligned(dx, size_of(x_dtype)) || !aligned(dz, 2)))
    return GDN_ERR_INVALID_ARG;
  if (clash({{dx, nx}, {dz, n * 2}, {dw, (size_t)D * 4}}, {{dy, n * 2}, {x, nx}, {z, n * 2}, {w, nw}}))
    return GDN_ERR_INVALID_ARG;
  if (!ws || ws_bytes < gated_norm_bwd_workspace_size(rows, D)) return GDN_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(ws, 16)) return GDN_ERR_INVALID_ARG;
  if ((s = gdn::check_device()) != GDN_OK) return s;
  if (rows == 0) return done(cudaMemsetAsync(dw, 0, (size_t)D * 4, (cudaStream_t)stream));
  return done(gdn::launch_gated_norm_bwd(dy, x, x_dtype == GDN_DTYPE_F32, z, w, w_dtype == GDN_DTYPE_BF16, dx, dz, dw,
                                         rows, D, eps, static_cast<float*>(ws), (cudaStream_t)stream));
}

gdn_status residual_norm_fwd(const void* y, const void* h, int32_t h_dtype, const void* w_post, const void* w_pre,
                             int32_t w_dtype, void* h_out, void* x, int64_t rows, int32_t D, float alpha, float eps,
                             gdn_stream_t stream) {
  gdn_status s = norm_sizes(rows, D, h_dtype, w_dtype, eps);
  if (s != GDN_OK) return s;
  if (rows > 0) {
    const size_t hs = size_of(h_dtype), n = (size_t)rows * D, nw = D * size_of(w_dtype);
    if (!y || !h || !w_pre || !h_out || !x || !aligned(y, 2) || !aligned(h, hs) || !aligned(h_out, hs) ||
        !aligned(x, 2) || !aligned(w_pre, size_of(w_dtype)) || !aligned(w_post, size_of(w_dtype)))
      return GDN_ERR_INVALID_ARG;
    if (clash({{h_out, n * hs}, {x, n * 2}},
              {{y, n * 2}, {h_out == h ? nullptr : h, n * hs}, {w_post, nw}, {w_pre, nw}}) ||
        overlaps(x, n * 2, h, n * hs))
      return GDN_ERR_INVALID_ARG;
  }
  if ((s = gdn::check_device()) != GDN_OK) return s;
  if (rows == 0) return GDN_OK;
  return done(gdn::launch_residual_norm_fwd(y, h, h_dtype == GDN_DTYPE_F32, w_post, w_pre, w_dtype == GDN_DTYPE_BF16,
                                            h_out, x, rows, D, alpha, eps, (cudaStream_t)stream));
}

gdn_status residual_norm_bwd(const void* dx, const void* dh_out, const void* y, const void* h, int32_t h_dtype,
                             const void* w_post, const void* w_pre, int32_t w_dtype, void* dy, void* dh,
                             float* dw_post, float* dw_pre, int64_t rows, int32_t D, float alpha, float eps, void* ws,
                             size_t ws_bytes, gdn_stream_t stream) {
  gdn_status s = norm_sizes(rows, D, h_dtype, w_dtype, eps);
  if (s != GDN_OK) return s;
  const size_t hs = size_of(h_dtype), wsz = size_of(w_dtype), n = (size_t)rows * D, nw = D * wsz;
  if (!w_pre || !dw_pre || !aligned(w_pre, wsz) || !aligned(w_post, wsz) || !aligned(dw_pre, 4) ||
      !aligned(dw_post, 4) || (w_post != nullptr) != (dw_post != nullptr))
    return GDN_ERR_INVALID_ARG;
  if (rows > 0 && (!dx || !y || !h || !dy || !dh || !aligned(dx, 2) || !aligned(y, 2) || !aligned(dy, 2) ||
                   !aligned(h, hs) || !aligned(dh, hs) || !aligned(dh_out, hs)))
    return GDN_ERR_INVALID_ARG;
  if (clash({{dy, n * 2}, {dh, n * hs}, {dw_post, (size_t)D * 4}, {dw_pre, (size_t)D * 4}},
            {{dx, n * 2}, {dh_out == dh ? nullptr : dh_out, n * hs}, {y, n * 2}, {h, n * hs}, {w_post, nw}, {w_pre, nw}}) ||
      clash({{dy, n * 2}, {dw_post, (size_t)D * 4}, {dw_pre, (size_t)D * 4}}, {{dh_out, n * hs}}))
    return GDN_ERR_INVALID_ARG;
  if (!ws || ws_bytes < residual_norm_bwd_workspace_size(rows, D)) return GDN_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(ws, 16)) return GDN_ERR_INVALID_ARG;
  if ((s = gdn::check_device()) != GDN_OK) return s;
  if (rows == 0) {
    if (dw_post && cudaMemsetAsync(dw_post, 0, (size_t)D * 4, (cudaStream_t)stream) != cudaSuccess) return GDN_ERR_CUDA;
    return done(cudaMemsetAsync(dw_pre, 0, (size_t)D * 4, (cudaStream_t)stream));
  }
  return done(gdn::launch_residual_norm_bwd(dx, dh_out, y, h, h_dtype == GDN_DTYPE_F32, w_post, w_pre,
                                            w_dtype == GDN_DTYPE_BF16, dy, dh, dw_post, dw_pre, rows, D, alpha, eps,
                                            static_cast<float*>(ws), (cudaStream_t)stream));
}

}  // extern "C"

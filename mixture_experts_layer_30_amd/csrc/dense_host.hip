// Host side of the dense feed-forward block and the MXFP4 calls of
// include/mok.h: argument checks, workspace layouts and launch sequences.
#include <string.h>

#include <algorithm>

#include "../../include/mok.h"
#include "dense_launch.h"
#include "host_common.h"

using namespace mok;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30, kMaxK = (int64_t)1 << 20, kMaxTiles = (int64_t)1 << 23;
constexpr int64_t kMaxPitch = (int64_t)1 << 22;  // row pitch of x, y, dy, dx in elements (copies: 32-bit offsets)

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// rows x cols in 128 x 128 tiles, of 256 threads each, within one launch (2^32 threads; tiles of
// 256 x 256 have 512 threads and are split into no more than 512)
bool tiles_fit(int64_t rows, int64_t cols) { return cdiv(rows, 128) * cdiv(cols, 128) <= kMaxTiles; }

struct Ffn {
  int64_t T, H, I, ldx, ldy;
  bool mx, fwd_only;
  int act;
};

mok_status resolve(const mok_ffn_problem* p, Ffn* r) {
  if (!p || p->T < 0 || p->H <= 0 || p->I <= 0) return MOK_ERR_INVALID_ARG;
  if (p->dtype != MOK_BF16 && p->dtype != MOK_MXFP8 && p->dtype != MOK_MXFP4) return MOK_ERR_INVALID_ARG;
  if (p->activation != MOK_ACT_SILU && p->activation != MOK_ACT_GELU_TANH) return MOK_ERR_INVALID_ARG;
  if (p->forward_only != 0 && p->forward_only != 1) return MOK_ERR_INVALID_ARG;
  r->T = p->T; r->H = p->H; r->I = p->I;
  r->fwd_only = p->forward_only != 0;
  if (p->dtype == MOK_MXFP8) return MOK_ERR_UNSUPPORTED;
  r->mx = p->dtype == MOK_MXFP4;
  r->act = p->activation;
  const int64_t unit = r->mx ? 128 : 8;
  if (p->H % unit || p->I % unit || p->H > kMaxK || p->I > kMaxK || p->T > kMaxRows) return MOK_ERR_UNSUPPORTED;
  r->ldx = p->ld_x ? p->ld_x : p->H;
  r->ldy = p->ld_y ? p->ld_y : p->H;
  if (r->ldx < p->H || r->ldy < p->H || r->ldx % 8 || r->ldy % 8) return MOK_ERR_INVALID_ARG;
  if (r->ldx > kMaxPitch || r->ldy > kMaxPitch) return MOK_ERR_UNSUPPORTED;
  if (!tiles_fit(p->T, std::max(p->H, 2 * p->I)) || !tiles_fit(p->H, 2 * p->I)) return MOK_ERR_UNSUPPORTED;
  return MOK_OK;
}

mok_ffn_args ffn_args(const Ffn& r) {
  mok_ffn_args a;
  memset(&a, 0, sizeof a);
  a.T = (int)r.T; a.H = (int)r.H; a.I = (int)r.I;
  a.Ip = (int)(cdiv(r.I, 64) * 64);
  a.ldx = r.ldx; a.ldy = r.ldy;
  return a;
}

// x . [Wg; Wu]^T and h . Wd^T of the block with 4-bit weights
mok_mx_args mx_up(const Ffn& r) {
  mok_mx_args a;
  memset(&a, 0, sizeof a);
  a.M = (int)r.T; a.N = (int)r.I; a.K = (int)r.H; a.a8 = true;
  return a;
}
mok_mx_args mx_down(const Ffn& r) {
  mok_mx_args a;
  memset(&a, 0, sizeof a);
  a.M = (int)r.T; a.N = (int)r.H; a.K = (int)r.I; a.a8 = true;
  a.ldd = r.ldy;
  return a;
}

// Workspace carve-up; forward and backward share the bytes.
struct FfnWs {
  size_t h, hf, hs, xq, xs, part, total;         // forward (hf, hs, xq, xs: MXFP4)
};
struct FfnBwdWs {
  size_t h, dab, part, total;
};
FfnWs fwd_ws(const Ffn& r) {
  FfnWs w;
  const size_t T = (size_t)r.T, H = (size_t)r.H, I = (size_t)r.I;
  size_t o = 0, part;
  w.h = o;    o = align_up(o + T * I * (r.mx ? 1 : 2));
  w.hf = o;   o = align_up(o + (r.mx && mok_mx_few((int)r.T) ? T * I * 4 : 0));
  w.hs = o;   o = align_up(o + (r.mx ? T * (I / 32) : 0));
  w.xq = o;   o = align_up(o + (r.mx ? T * H : 0));
  w.xs = o;   o = align_up(o + (r.mx ? T * (H / 32) : 0));
  if (r.mx) {
    part = std::max(mok_mx_part_bytes(mx_up(r), true), mok_mx_part_bytes(mx_down(r), false));
  } else {
    const mok_ffn_args a = ffn_args(r);
    part = std::max(mok_ffn_part_bytes(a, FFN_GATEUP), mok_ffn_part_bytes(a, FFN_DOWN));
  }
  w.part = o; o = align_up(o + part);
  w.total = o;
  return w;
}
FfnBwdWs bwd_ws(const Ffn& r) {
  FfnBwdWs w;
  const mok_ffn_args a = ffn_args(r);
  size_t o = 0, part;
  w.h = o;    o = align_up(o + (size_t)r.T * r.I * 2);
  w.dab = o;  o = align_up(o + (size_t)r.T * a.Ip * 4);
  part = std::max(mok_ffn_part_bytes(a, FFN_DH), mok_ffn_grads_part_bytes(a));
  w.part = o; o = align_up(o + part);
  w.total = o;
  return w;
}
// (a backward's is up to thousands of times a forward's: 22 MB against 4 KB for one token of 7168 x 2048)
size_t ffn_ws_bytes(const Ffn& r) {
  const size_t fwd = fwd_ws(r).total;
  return r.mx || r.fwd_only ? fwd : std::max(fwd, bwd_ws(r).total);
}
size_t ffn_ctx_bytes(const Ffn& r) { return r.mx ? 0 : (size_t)r.T * 2 * r.I * 2; }

// whether rows of H elements share memory: T rows at a of pitch lda, and at b of pitch ldb
// (rows of one pitch that lie side by side do not)
bool rows_overlap(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t T, int64_t H) {
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(a) - reinterpret_cast<uintptr_t>(b)) / 2;
  if (T <= 0 || d >= (T - 1) * ldb + H || -d >= (T - 1) * lda + H) return false;
  if (lda != ldb) return true;
  const int64_t m = (d % lda + lda) % lda;
  return m < H || m > lda - H;
}

struct Span {
  const void* p;
  size_t n;                                      // bytes (rows with a pitch: from the first to the last)
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.n && b.n && (x < y ? y - x < a.n : x - y < b.n);
}
Span rows_span(const void* p, int64_t T, int64_t H, int64_t ld) { return {p, (size_t)((T - 1) * ld + H) * 2}; }

// whether memory that a forward writes (y, ctx, the workspace) is also memory of another
// operand of it that it reads or writes; y over x or the residual is not looked at here
bool fwd_overlap(const Ffn& r, const void* x, const mok_weights& w, const void* res, const void* y, const void* ctx,
                 const void* ws, size_t ws_bytes) {
  const size_t m = (size_t)r.H * r.I, wb = r.mx ? m / 2 : m * 2, sb = r.mx ? m / 32 : 0;
  const Span sy = rows_span(y, r.T, r.H, r.ldy), sc = {ctx, ffn_ctx_bytes(r)}, sw = {ws, ws_bytes};
  for (const Span& o : {sy, sc, sw})
    for (const Span& i : {Span{w.w_gate, wb}, Span{w.w_up, wb}, Span{w.w_down, wb}, Span{sb ? w.s_gate : nullptr, sb},
                          Span{sb ? w.s_up : nullptr, sb}, Span{sb ? w.s_down : nullptr, sb}})
      if (overlap(o, i)) return true;
  const Span sx = rows_span(x, r.T, r.H, r.ldx), sr = rows_span(res, r.T, r.H, r.ldy);
  for (const Span& o : {sc, sw})
    for (const Span& i : {sx, sr, sy})
      if (overlap(o, i)) return true;
  return overlap(sc, sw);
}

// the same for what a backward writes: dx, the weight gradients and the workspace (dx over x or dy:
// rows_overlap)
bool bwd_overlap(const Ffn& r, const void* ctx, const void* x, const mok_weights& w, const void* dy, const void* dx,
                 const void* dwg, const void* dwu, const void* dwd, const void* ws, size_t ws_bytes) {
  const size_t m = (size_t)r.H * r.I * 2;
  const Span sdx = rows_span(dx, r.T, r.H, r.ldx), sx = rows_span(x, r.T, r.H, r.ldx), sc = {ctx, ffn_ctx_bytes(r)},
             sdy = rows_span(dy, r.T, r.H, r.ldy), sw = {ws, ws_bytes};
  const Span grads[3] = {{dwg, m}, {dwu, m}, {dwd, m}}, weights[3] = {{w.w_gate, m}, {w.w_up, m}, {w.w_down, m}};
  if (overlap(sdx, sc) || overlap(sw, sc) || overlap(sw, sx) || overlap(sw, sdy) || overlap(sw, sdx)) return true;
  for (int i = 0; i < 3; ++i) {
    if (overlap(sdx, weights[i]) || overlap(sw, weights[i])) return true;
    for (const Span& o : {sx, sdy, sc, sdx, sw})
      if (overlap(grads[i], o)) return true;
  }
  return false;
}

mok_status ffn_weights(const Ffn& r, const mok_weights* w) {
  if (!w || !w->w_gate || !w->w_up || !w->w_down) return MOK_ERR_INVALID_ARG;
  if (!aligned(w->w_gate, 16) || !aligned(w->w_up, 16) || !aligned(w->w_down, 16)) return MOK_ERR_INVALID_ARG;
  if (r.mx && (!w->s_gate || !w->s_up || !w->s_down || !aligned(w->s_gate, 4) || !aligned(w->s_up, 4) ||
               !aligned(w->s_down, 4)))
    return MOK_ERR_INVALID_ARG;
  return MOK_OK;
}

mok_status resolve(const mok_mx_problem* p, mok_mx_args* a) {
  if (!p || p->M < 0 || p->N < 0 || p->K <= 0) return MOK_ERR_INVALID_ARG;
  if (p->a_dtype != MOK_MXFP4 && p->a_dtype != MOK_MXFP8) return MOK_ERR_INVALID_ARG;
  if (p->ld_d != 0 && p->ld_d < p->N) return MOK_ERR_INVALID_ARG;
  if (p->K % 128 || p->K > kMaxK || p->M > kMaxRows || p->N > kMaxRows || p->ld_d > ((int64_t)1 << 40) ||
      !tiles_fit(p->M, p->N))
    return MOK_ERR_UNSUPPORTED;
  memset(a, 0, sizeof *a);
  a->M = (int)p->M; a->N = (int)p->N; a->K = (int)p->K;
  a->a8 = p->a_dtype == MOK_MXFP8;
  a->ldd = p->ld_d ? p->ld_d : p->N;
  return MOK_OK;
}

}  // namespace

extern "C" {

mok_status mok_ffn_buffer_sizes(const mok_ffn_problem* problem, size_t* workspace_bytes, size_t* ctx_bytes) {
  Ffn r;
  const mok_status s = resolve(problem, &r);
  if (s != MOK_OK) return s;
  if (workspace_bytes) *workspace_bytes = ffn_ws_bytes(r);
  if (ctx_bytes) *ctx_bytes = ffn_ctx_bytes(r);
  return MOK_OK;
}

mok_status mok_ffn_forward(const mok_ffn_problem* problem, const void* x, const mok_weights* weights,
                           const void* residual, void* y, void* ctx, void* workspace, size_t workspace_bytes,
                           void* stream) {
  TraceCall tc;
  Ffn r;
  mok_status s = resolve(problem, &r);
  if (s != MOK_OK) return s;
  if ((s = ffn_weights(r, weights)) != MOK_OK) return s;
  if (r.mx && ctx) return MOK_ERR_UNSUPPORTED;   // no backward through 4-bit weights
  if (r.T > 0 && (!x || !y)) return MOK_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(residual, 16) || !aligned(ctx, 16) || !aligned(workspace, 16))
    return MOK_ERR_INVALID_ARG;
  // (a workgroup reads the residual of its own part of y alone before it stores that)
  if (residual && residual != y && rows_overlap(y, r.ldy, residual, r.ldy, r.T, r.H)) return MOK_ERR_INVALID_ARG;
  const FfnWs W = fwd_ws(r);
  const size_t need = ffn_ws_bytes(r);
  if (r.T > 0 && (!workspace || workspace_bytes < need)) return MOK_ERR_BUFFER_TOO_SMALL;
  if (r.T > 0 && fwd_overlap(r, x, *weights, residual, y, ctx, workspace, need)) return MOK_ERR_INVALID_ARG;
  if ((s = check_device()) != MOK_OK) return s;
  if (r.T == 0) return MOK_OK;
  hipStream_t st = (hipStream_t)stream;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* part = reinterpret_cast<float*>(ws + W.part);
  if (r.mx) {
    mok_mx_args u = mx_up(r), d = mx_down(r);
    u.a = ws + W.xq; u.sa = ws + W.xs;
    u.b = static_cast<const uint8_t*>(weights->w_gate); u.sb = weights->s_gate;
    u.b2 = static_cast<const uint8_t*>(weights->w_up); u.sb2 = weights->s_up;
    u.hq = ws + W.h; u.hs = ws + W.hs; u.part = part;
    d.a = u.hq; d.sa = u.hs;
    d.b = static_cast<const uint8_t*>(weights->w_down); d.sb = weights->s_down;
    d.d = static_cast<bf16_t*>(y); d.res = static_cast<const bf16_t*>(residual); d.part = part;
    u.hf = reinterpret_cast<float*>(ws + W.hf);
    MOK_RUN("ffn_quantize_x", mok_launch_mxfp8_rows(x, false, r.ldx, r.T, r.H, ws + W.xq, ws + W.xs, st));
    MOK_RUN("ffn_gateup_mxfp4", mok_launch_mx(u, true, r.act, st));
    if (mok_mx_few((int)r.T))
      MOK_RUN("ffn_quantize_h", mok_launch_mxfp8_rows(u.hf, true, r.I, r.T, r.I, ws + W.h, ws + W.hs, st));
    MOK_RUN("ffn_down_mxfp4", mok_launch_mx(d, false, 0, st));
    return MOK_OK;
  }
  mok_ffn_args a = ffn_args(r);
  a.x = static_cast<const bf16_t*>(x);
  a.wg = static_cast<const bf16_t*>(weights->w_gate);
  a.wu = static_cast<const bf16_t*>(weights->w_up);
  a.wd = static_cast<const bf16_t*>(weights->w_down);
  a.res = static_cast<const bf16_t*>(residual);
  a.y = static_cast<bf16_t*>(y);
  a.h = reinterpret_cast<bf16_t*>(ws + W.h);
  a.ab = static_cast<bf16_t*>(ctx);
  a.part = part;
  MOK_RUN("ffn_gateup", mok_launch_ffn(a, FFN_GATEUP, r.act, st));
  MOK_RUN("ffn_down", mok_launch_ffn(a, FFN_DOWN, r.act, st));
  return MOK_OK;
}

mok_status mok_ffn_backward(const mok_ffn_problem* problem, const void* ctx, const void* x,
                            const mok_weights* weights, const void* dy, void* dx, void* dw_gate, void* dw_up,
                            void* dw_down, void* workspace, size_t workspace_bytes, void* stream) {
  TraceCall tc;
  Ffn r;
  mok_status s = resolve(problem, &r);
  if (s != MOK_OK) return s;
  if (r.mx) return MOK_ERR_UNSUPPORTED;
  if (r.fwd_only) return MOK_ERR_INVALID_ARG;
  if ((s = ffn_weights(r, weights)) != MOK_OK) return s;
  if (!dw_gate || !dw_up || !dw_down) return MOK_ERR_INVALID_ARG;
  if (r.T > 0 && (!ctx || !x || !dy || !dx)) return MOK_ERR_INVALID_ARG;
  for (const void* p : {ctx, x, dy, (const void*)dx, (const void*)dw_gate, (const void*)dw_up, (const void*)dw_down,
                        (const void*)workspace})
    if (!aligned(p, 16)) return MOK_ERR_INVALID_ARG;
  if (rows_overlap(dx, r.ldx, x, r.ldx, r.T, r.H) || rows_overlap(dx, r.ldx, dy, r.ldy, r.T, r.H))
    return MOK_ERR_INVALID_ARG;
  const void* mats[] = {dw_gate, dw_up, dw_down, weights->w_gate, weights->w_up, weights->w_down};
  for (int i = 0; i < 3; ++i)                    // no gradient over another, or over a weight
    for (int j = i + 1; j < 6; ++j)
      if (rows_overlap(mats[i], r.H, mats[j], r.H, r.I, r.H)) return MOK_ERR_INVALID_ARG;
  const FfnBwdWs W = bwd_ws(r);
  const size_t need = ffn_ws_bytes(r);
  if (r.T > 0 && (!workspace || workspace_bytes < need)) return MOK_ERR_BUFFER_TOO_SMALL;
  if (r.T > 0 && bwd_overlap(r, ctx, x, *weights, dy, dx, dw_gate, dw_up, dw_down, workspace, need))
    return MOK_ERR_INVALID_ARG;
  if ((s = check_device()) != MOK_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  mok_ffn_args a = ffn_args(r);
  a.x = static_cast<const bf16_t*>(x);
  a.wg = static_cast<const bf16_t*>(weights->w_gate);
  a.wu = static_cast<const bf16_t*>(weights->w_up);
  a.wd = static_cast<const bf16_t*>(weights->w_down);
  a.ab = static_cast<bf16_t*>(const_cast<void*>(ctx));
  a.dy = static_cast<const bf16_t*>(dy);
  a.dx = static_cast<bf16_t*>(dx);
  a.dwg = static_cast<bf16_t*>(dw_gate);
  a.dwu = static_cast<bf16_t*>(dw_up);
  a.dwd = static_cast<bf16_t*>(dw_down);
  if (r.T > 0) {
    a.h = reinterpret_cast<bf16_t*>(ws + W.h);
    a.dab = reinterpret_cast<bf16_t*>(ws + W.dab);
    a.part = reinterpret_cast<float*>(ws + W.part);
    MOK_RUN("ffn_bwd_dh", mok_launch_ffn(a, FFN_DH, r.act, st));
  }
  // (no tokens: the sums over them are empty, and the weight gradients zeros)
  MOK_RUN("ffn_bwd_grads", mok_launch_ffn_grads(a, st));
  return MOK_OK;
}

mok_status mok_mxfp4_quantize(const void* src, int64_t rows, int64_t K, uint8_t* q, uint8_t* scales, void* stream) {
  TraceCall tc;
  if (rows < 0 || K <= 0 || K % 32 != 0) return MOK_ERR_INVALID_ARG;
  if (rows > 0 && (!src || !q || !scales)) return MOK_ERR_INVALID_ARG;
  if (!aligned(src, 16) || !aligned(q, 4)) return MOK_ERR_INVALID_ARG;
  if (K > ((int64_t)1 << 38) || rows > ((int64_t)1 << 38) / K) return MOK_ERR_UNSUPPORTED;
  const size_t n = (size_t)rows * K;
  const Span v = {src, n * 2}, c = {q, n / 2}, e = {scales, n / 32};
  if (overlap(v, c) || overlap(v, e) || overlap(c, e)) return MOK_ERR_INVALID_ARG;
  mok_status s = check_device();
  if (s != MOK_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  MOK_RUN("mxfp4_quantize", mok_launch_mxfp4_quantize(static_cast<const bf16_t*>(src), rows, K, q, scales, st));
  return MOK_OK;
}

mok_status mok_mxfp4_dequantize(const uint8_t* q, const uint8_t* scales, int64_t rows, int64_t K, void* dst,
                                void* stream) {
  TraceCall tc;
  if (rows < 0 || K <= 0 || K % 32 != 0) return MOK_ERR_INVALID_ARG;
  if (rows > 0 && (!dst || !q || !scales)) return MOK_ERR_INVALID_ARG;
  if (!aligned(dst, 16) || !aligned(q, 4)) return MOK_ERR_INVALID_ARG;
  if (K > ((int64_t)1 << 38) || rows > ((int64_t)1 << 38) / K) return MOK_ERR_UNSUPPORTED;
  const size_t n = (size_t)rows * K;
  const Span v = {dst, n * 2}, c = {q, n / 2}, e = {scales, n / 32};
  if (overlap(v, c) || overlap(v, e)) return MOK_ERR_INVALID_ARG;
  mok_status s = check_device();
  if (s != MOK_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  MOK_RUN("mxfp4_dequantize", mok_launch_mxfp4_dequantize(q, scales, rows, K, static_cast<bf16_t*>(dst), st));
  return MOK_OK;
}

mok_status mok_mx_matmul_workspace(const mok_mx_problem* problem, size_t* workspace_bytes) {
  mok_mx_args a;
  const mok_status s = resolve(problem, &a);
  if (s != MOK_OK) return s;
  if (workspace_bytes) *workspace_bytes = mok_mx_part_bytes(a, false);
  return MOK_OK;
}

mok_status mok_mx_matmul(const mok_mx_problem* problem, const uint8_t* a, const uint8_t* a_scales, const uint8_t* b,
                         const uint8_t* b_scales, void* d, void* workspace, size_t workspace_bytes, void* stream) {
  TraceCall tc;
  mok_mx_args p;
  mok_status s = resolve(problem, &p);
  if (s != MOK_OK) return s;
  if (p.M > 0 && p.N > 0 && (!a || !a_scales || !b || !b_scales || !d)) return MOK_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_scales, 4) || !aligned(b_scales, 4) || !aligned(d, 2) ||
      !aligned(workspace, 16))
    return MOK_ERR_INVALID_ARG;
  const size_t need = mok_mx_part_bytes(p, false);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MOK_ERR_BUFFER_TOO_SMALL;
  if (p.M > 0 && p.N > 0) {
    const size_t K = (size_t)p.K;
    const Span sd = rows_span(d, p.M, p.N, p.ldd), sw = {workspace, need};
    for (const Span& i : {Span{a, p.M * (p.a8 ? K : K / 2)}, Span{a_scales, p.M * (K / 32)}, Span{b, p.N * (K / 2)},
                          Span{b_scales, p.N * (K / 32)}})
      if (overlap(sd, i) || overlap(sw, i)) return MOK_ERR_INVALID_ARG;
    if (overlap(sd, sw)) return MOK_ERR_INVALID_ARG;
  }
  if ((s = check_device()) != MOK_OK) return s;
  if (p.M == 0 || p.N == 0) return MOK_OK;
  p.a = a; p.sa = a_scales; p.b = b; p.sb = b_scales;
  p.d = static_cast<bf16_t*>(d);
  p.part = static_cast<float*>(workspace);
  hipStream_t st = (hipStream_t)stream;
  MOK_RUN("mx_matmul", mok_launch_mx(p, false, 0, st));
  return MOK_OK;
}

}  // extern "C"

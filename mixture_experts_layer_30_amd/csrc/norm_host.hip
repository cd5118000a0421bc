// Host side of the norm and the MXFP8 read-back of include/mok.h: argument
// checks and launch sequences.
#include <float.h>
#include <math.h>
#include <string.h>

#include "../../include/mok.h"
#include "host_common.h"
#include "norm_launch.h"

using namespace mok;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30, kMaxPitch = (int64_t)1 << 31;

mok_status resolve(const mok_norm_problem* p, mok_norm_args* a) {
  if (!p || p->T < 0 || p->H <= 0) return MOK_ERR_INVALID_ARG;
  if (p->weight_f32 != 0 && p->weight_f32 != 1) return MOK_ERR_INVALID_ARG;
  if (!(p->eps >= FLT_MIN) || !isfinite(p->eps)) return MOK_ERR_INVALID_ARG;
  if (p->H % 8 || p->H > kNormMaxH || p->T > kMaxRows) return MOK_ERR_UNSUPPORTED;
  memset(a, 0, sizeof *a);
  a->T = p->T;
  a->H = (int)p->H;
  a->eps = p->eps;
  const int64_t in[3] = {p->ld_x, p->ld_s, p->ld_y};
  int64_t* out[3] = {&a->ldx, &a->lds, &a->ldy};
  for (int i = 0; i < 3; ++i) {
    if (in[i] != 0 && (in[i] < p->H || in[i] % 8)) return MOK_ERR_INVALID_ARG;
    if (in[i] > kMaxPitch) return MOK_ERR_UNSUPPORTED;
    *out[i] = in[i] ? in[i] : p->H;
  }
  return MOK_OK;
}

struct Rows {
  const void* p;
  int64_t ld;
};
// whether output rows o lie on input rows i otherwise than exactly (`over`: that may be)
bool clash(const mok_norm_args& a, const Rows& o, const Rows& i, bool over) {
  if (!o.p || !i.p || (over && o.p == i.p && o.ld == i.ld)) return false;
  return rows_overlap(o.p, o.ld, i.p, i.ld, a.T, a.H);
}

Span weight_span(const mok_norm_args& a, const void* w) {
  return {w, w ? (size_t)a.H * (a.wf == 2 ? 4 : 2) : 0};
}

}  // namespace

extern "C" {

mok_status mok_norm_forward(const mok_norm_problem* problem, const void* x, const void* residual, const void* weight,
                            void* y, void* sum, float* rstd, uint8_t* q, uint8_t* scales, void* stream) {
  TraceCall tc;
  mok_norm_args a;
  mok_status s = resolve(problem, &a);
  if (s != MOK_OK) return s;
  if (q && a.H % 32) return MOK_ERR_UNSUPPORTED;
  if (!residual != !sum || !q != !scales) return MOK_ERR_INVALID_ARG;
  if (a.T > 0 && (!x || (!y && !q))) return MOK_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(y, 16) || !aligned(sum, 16) ||
      !aligned(rstd, 4) || !aligned(q, 16))
    return MOK_ERR_INVALID_ARG;
  a.wf = !weight ? 0 : problem->weight_f32 ? 2 : 1;
  if (a.T > 0) {
    // a thread stores a place of sum, and of y, after it has read that place of x and the residual itself
    const Rows rx = {x, a.ldx}, rr = {residual, a.lds}, ry = {y, a.ldy}, rs = {sum, a.lds};
    if (clash(a, rs, rx, true) || clash(a, rs, rr, true) || clash(a, ry, rx, true) || clash(a, ry, rr, true) ||
        clash(a, ry, rs, false))
      return MOK_ERR_INVALID_ARG;
    const size_t n = (size_t)a.T * a.H;
    const Span outs[3] = {{rstd, (size_t)a.T * 4}, {q, n}, {scales, n / 32}}, w = weight_span(a, weight);
    const Rows rows[4] = {rx, rr, ry, rs};
    for (int i = 0; i < 3; ++i) {
      if (overlap(outs[i], w)) return MOK_ERR_INVALID_ARG;
      for (int j = 0; j < i; ++j)
        if (overlap(outs[i], outs[j])) return MOK_ERR_INVALID_ARG;
      for (const Rows& r : rows)
        if (overlap(outs[i], rows_span(r.p, a.T, a.H, r.ld))) return MOK_ERR_INVALID_ARG;
    }
    if (overlap(w, rows_span(y, a.T, a.H, a.ldy)) || overlap(w, rows_span(sum, a.T, a.H, a.lds)))
      return MOK_ERR_INVALID_ARG;
  }
  if ((s = check_device()) != MOK_OK) return s;
  if (a.T == 0) return MOK_OK;
  a.w = weight;
  a.x = static_cast<const bf16_t*>(x);
  a.res = static_cast<const bf16_t*>(residual);
  a.y = static_cast<bf16_t*>(y);
  a.sum = static_cast<bf16_t*>(sum);
  a.rstd = rstd;
  a.q = q;
  a.scales = scales;
  hipStream_t st = (hipStream_t)stream;
  MOK_RUN("norm_forward", mok_launch_norm_forward(a, st));
  return MOK_OK;
}

mok_status mok_norm_workspace(const mok_norm_problem* problem, size_t* workspace_bytes) {
  mok_norm_args a;
  const mok_status s = resolve(problem, &a);
  if (s != MOK_OK) return s;
  const int groups = mok_norm_groups(a.T, a.H);
  if (workspace_bytes) *workspace_bytes = groups > 1 ? (size_t)groups * a.H * 4 : 0;
  return MOK_OK;
}

mok_status mok_norm_backward(const mok_norm_problem* problem, const void* dy, const void* z, int64_t ld_z,
                             const float* rstd, const void* weight, const void* d_sum, void* dx, void* d_weight,
                             void* workspace, size_t workspace_bytes, void* stream) {
  TraceCall tc;
  mok_norm_args a;
  mok_status s = resolve(problem, &a);
  if (s != MOK_OK) return s;
  if (ld_z != 0 && (ld_z < a.H || ld_z % 8)) return MOK_ERR_INVALID_ARG;
  if (ld_z > kMaxPitch) return MOK_ERR_UNSUPPORTED;
  a.ldx = ld_z ? ld_z : a.H;
  if (a.T > 0 && (!dy || !z || !rstd || !dx)) return MOK_ERR_INVALID_ARG;
  if (d_weight && !weight) return MOK_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(z, 16) || !aligned(rstd, 4) || !aligned(weight, 16) || !aligned(d_sum, 16) ||
      !aligned(dx, 16) || !aligned(d_weight, 16) || !aligned(workspace, 16))
    return MOK_ERR_INVALID_ARG;
  a.wf = !weight ? 0 : problem->weight_f32 ? 2 : 1;
  const int groups = mok_norm_groups(a.T, a.H);
  const size_t need = groups > 1 && d_weight ? (size_t)groups * a.H * 4 : 0;
  if (need && (!workspace || workspace_bytes < need)) return MOK_ERR_BUFFER_TOO_SMALL;
  const Span w = weight_span(a, weight), dw = weight_span(a, d_weight);
  if (overlap(w, dw)) return MOK_ERR_INVALID_ARG;
  if (a.T > 0) {
    const Rows rd = {dy, a.ldy}, rz = {z, a.ldx}, rs = {d_sum, a.lds}, ro = {dx, a.lds};
    if (clash(a, ro, rd, true) || clash(a, ro, rs, true) || clash(a, ro, rz, false)) return MOK_ERR_INVALID_ARG;
    const Span outs[2] = {dw, {workspace, need}}, r = {rstd, (size_t)a.T * 4};
    const Rows rows[4] = {rd, rz, rs, ro};
    for (const Span& o : outs) {
      if (overlap(o, r)) return MOK_ERR_INVALID_ARG;
      for (const Rows& i : rows)
        if (overlap(o, rows_span(i.p, a.T, a.H, i.ld))) return MOK_ERR_INVALID_ARG;
    }
    const Span so = rows_span(dx, a.T, a.H, a.lds);
    if (overlap(outs[0], outs[1]) || overlap(outs[1], w) || overlap(so, r) || overlap(so, w))
      return MOK_ERR_INVALID_ARG;
  }
  if ((s = check_device()) != MOK_OK) return s;
  if (a.T == 0 && !d_weight) return MOK_OK;
  a.w = weight;
  a.dy = static_cast<const bf16_t*>(dy);
  a.x = static_cast<const bf16_t*>(z);
  a.rstd = const_cast<float*>(rstd);
  a.res = static_cast<const bf16_t*>(d_sum);
  a.sum = static_cast<bf16_t*>(dx);
  a.dw = d_weight;
  a.part = static_cast<float*>(workspace);
  hipStream_t st = (hipStream_t)stream;
  // (no rows: one workgroup that writes the empty sums)
  MOK_RUN("norm_backward", mok_launch_norm_backward(a, st));
  return MOK_OK;
}

mok_status mok_mxfp8_dequantize(const uint8_t* q, const uint8_t* scales, int64_t rows, int64_t K, void* dst,
                                void* stream) {
  TraceCall tc;
  if (rows < 0 || K <= 0 || K % 32 != 0) return MOK_ERR_INVALID_ARG;
  if (rows > 0 && (!dst || !q || !scales)) return MOK_ERR_INVALID_ARG;
  if (!aligned(dst, 16) || !aligned(q, 16)) return MOK_ERR_INVALID_ARG;
  if (K > ((int64_t)1 << 38) || rows > ((int64_t)1 << 38) / K) return MOK_ERR_UNSUPPORTED;
  const size_t n = (size_t)rows * K;
  const Span v = {dst, n * 2};
  if (overlap(v, {q, n}) || overlap(v, {scales, n / 32})) return MOK_ERR_INVALID_ARG;
  mok_status s = check_device();
  if (s != MOK_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  MOK_RUN("mxfp8_dequantize", mok_launch_mxfp8_dequantize(q, scales, rows, K, static_cast<bf16_t*>(dst), st));
  return MOK_OK;
}

}  // extern "C"

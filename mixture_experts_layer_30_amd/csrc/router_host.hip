// Host side of the router's losses and its dense backward of include/mok.h:
// argument checks, workspace and launch sequences.
#include <string.h>

#include <algorithm>

#include "../../include/mok.h"
#include "host_common.h"
#include "router_launch.h"

using namespace mok;

namespace {

constexpr int64_t kMaxH = (int64_t)1 << 20, kMaxT = (int64_t)1 << 30;

mok_status resolve(const mok_problem* p) {
  const mok_status s = mok_buffer_sizes(p, nullptr, nullptr, nullptr, nullptr);
  if (s != MOK_OK) return s;
  return p->H > kMaxH || p->T > kMaxT ? MOK_ERR_UNSUPPORTED : MOK_OK;
}

bool any_overlap(const Span* outs, int no, const Span* ins, int ni) {
  for (int i = 0; i < no; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return true;
    for (int j = 0; j < ni; ++j)
      if (overlap(outs[i], ins[j])) return true;
  }
  return false;
}

// Alignment of [T][E] logits and their gradient. Where E is not a multiple of 4 their rows start at any value, so the
// losses' kernels go through them value by value, and the dense backward loads 16 bytes from any value on.
size_t row_align(size_t E) { return E % 4 == 0 ? 16 : 4; }

mok_losses_args losses_args(const mok_problem& p) {
  mok_losses_args a;
  memset(&a, 0, sizeof a);
  a.T = p.T;
  a.E = p.E;
  a.k = p.topk;
  return a;
}

}  // namespace

extern "C" {

mok_status mok_router_forward_logits(const mok_problem* problem, const void* x, const float* w_router,
                                     const float* bias, int32_t* topk_ids, float* topk_w, float* logits,
                                     void* stream) {
  TraceCall tc;
  mok_status s = resolve(problem);
  if (s != MOK_OK) return s;
  const int64_t T = problem->T, H = problem->H, E = problem->E, k = problem->topk;
  if (T > 0 && (!x || !w_router || !topk_ids || !topk_w || !logits)) return MOK_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w_router, 16) || !aligned(bias, 4) || !aligned(topk_ids, 4) ||
      !aligned(topk_w, 4) || !aligned(logits, 4))
    return MOK_ERR_INVALID_ARG;
  if (k > 64) return MOK_ERR_UNSUPPORTED;
  const Span outs[3] = {{topk_ids, (size_t)(T * k) * 4}, {topk_w, (size_t)(T * k) * 4}, {logits, (size_t)(T * E) * 4}};
  const Span ins[3] = {{x, (size_t)(T * H) * 2}, {w_router, (size_t)(E * H) * 4}, {bias, (size_t)E * 4}};
  if (any_overlap(outs, 3, ins, 3)) return MOK_ERR_INVALID_ARG;
  if ((s = check_device()) != MOK_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  MOK_RUN("router_forward", mok_launch_router_forward_logits(static_cast<const bf16_t*>(x), w_router, bias, T, (int)H,
                                                             (int)E, (int)k, topk_ids, topk_w, logits, st));
  return MOK_OK;
}

mok_status mok_router_workspace(const mok_problem* problem, size_t* workspace_bytes) {
  const mok_status s = resolve(problem);
  if (s != MOK_OK) return s;
  if (workspace_bytes)
    *workspace_bytes = std::max(mok_losses_part_bytes(problem->T, problem->E),
                                mok_logits_bwd_part_bytes(problem->T, (int)problem->H, problem->E));
  return MOK_OK;
}

mok_status mok_router_losses(const mok_problem* problem, const float* logits, const int32_t* topk_ids,
                             const uint8_t* token_mask, float* losses, int32_t* counts, float* prob_sum,
                             int32_t* n_tokens, void* workspace, size_t workspace_bytes, void* stream) {
  TraceCall tc;
  mok_status s = resolve(problem);
  if (s != MOK_OK) return s;
  const size_t T = (size_t)problem->T, E = (size_t)problem->E, k = (size_t)problem->topk;
  if (!losses || !counts || !prob_sum || !n_tokens || (T > 0 && (!logits || !topk_ids))) return MOK_ERR_INVALID_ARG;
  if (!aligned(logits, row_align(E)) || !aligned(topk_ids, 4) || !aligned(losses, 4) || !aligned(counts, 4) ||
      !aligned(prob_sum, 4) || !aligned(n_tokens, 4) || !aligned(workspace, 16))
    return MOK_ERR_INVALID_ARG;
  const size_t need = mok_losses_part_bytes(problem->T, problem->E);
  if (need && (!workspace || workspace_bytes < need)) return MOK_ERR_BUFFER_TOO_SMALL;
  const Span outs[5] = {{losses, 8}, {counts, E * 4}, {prob_sum, E * 4}, {n_tokens, 4}, {workspace, need}};
  const Span ins[3] = {{logits, T * E * 4}, {topk_ids, T * k * 4}, {token_mask, T}};
  if (any_overlap(outs, 5, ins, 3)) return MOK_ERR_INVALID_ARG;
  if ((s = check_device()) != MOK_OK) return s;
  mok_losses_args a = losses_args(*problem);
  a.logits = logits;
  a.ids = topk_ids;
  a.mask = token_mask;
  a.losses = losses;
  a.counts = counts;
  a.prob = prob_sum;
  a.n = n_tokens;
  a.part = static_cast<uint32_t*>(workspace);
  hipStream_t st = (hipStream_t)stream;
  MOK_RUN("router_losses", mok_launch_losses(a, st));
  return MOK_OK;
}

mok_status mok_router_losses_backward(const mok_problem* problem, const float* logits, const int32_t* topk_ids,
                                      const uint8_t* token_mask, const int32_t* counts, const int32_t* n_tokens,
                                      const float* d_losses, const float* topk_w, const float* d_topk_w,
                                      float* d_logits, void* stream) {
  TraceCall tc;
  mok_status s = resolve(problem);
  if (s != MOK_OK) return s;
  const size_t T = (size_t)problem->T, E = (size_t)problem->E, k = (size_t)problem->topk;
  if (!counts || !n_tokens || !d_losses) return MOK_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !topk_ids || !d_logits || !topk_w != !d_topk_w)) return MOK_ERR_INVALID_ARG;
  if (!aligned(logits, row_align(E)) || !aligned(topk_ids, 4) || !aligned(counts, 4) || !aligned(n_tokens, 4) ||
      !aligned(d_losses, 4) || !aligned(topk_w, 4) || !aligned(d_topk_w, 4) || !aligned(d_logits, row_align(E)))
    return MOK_ERR_INVALID_ARG;
  const Span out = {d_logits, T * E * 4};
  // (a row is read before the same lanes write it)
  const Span ins[8] = {{d_logits == logits ? nullptr : logits, T * E * 4}, {topk_ids, T * k * 4}, {token_mask, T},
                       {counts, E * 4}, {n_tokens, 4}, {d_losses, 8}, {topk_w, T * k * 4}, {d_topk_w, T * k * 4}};
  if (any_overlap(&out, 1, ins, 8)) return MOK_ERR_INVALID_ARG;
  if ((s = check_device()) != MOK_OK) return s;
  mok_losses_args a = losses_args(*problem);
  a.logits = logits;
  a.ids = topk_ids;
  a.mask = token_mask;
  a.counts = const_cast<int32_t*>(counts);
  a.n = const_cast<int32_t*>(n_tokens);
  a.d_losses = d_losses;
  a.w = topk_w;
  a.g = d_topk_w;
  a.d_logits = d_logits;
  hipStream_t st = (hipStream_t)stream;
  MOK_RUN("router_losses_backward", mok_launch_losses_backward(a, st));
  return MOK_OK;
}

mok_status mok_router_logits_backward(const mok_problem* problem, const void* x, const float* w_router,
                                      const float* d_logits, const void* residual, void* dx, float* d_w_router,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  TraceCall tc;
  mok_status s = resolve(problem);
  if (s != MOK_OK) return s;
  const size_t T = (size_t)problem->T, H = (size_t)problem->H, E = (size_t)problem->E;
  if (!d_w_router || (T > 0 && (!x || !w_router || !d_logits || !dx))) return MOK_ERR_INVALID_ARG;
  for (const void* p : {x, (const void*)w_router, residual, (const void*)dx, (const void*)d_w_router,
                        (const void*)workspace})
    if (!aligned(p, 16)) return MOK_ERR_INVALID_ARG;
  if (!aligned(d_logits, row_align(E))) return MOK_ERR_INVALID_ARG;
  const size_t need = mok_logits_bwd_part_bytes(problem->T, (int)H, (int)E);
  if (need && (!workspace || workspace_bytes < need)) return MOK_ERR_BUFFER_TOO_SMALL;
  const Span outs[3] = {{dx, T * H * 2}, {d_w_router, E * H * 4}, {workspace, need}};
  // (a thread reads its part of the residual before it writes that part of dx)
  const Span ins[4] = {{x, T * H * 2}, {w_router, E * H * 4}, {d_logits, T * E * 4},
                       {residual == dx ? nullptr : residual, T * H * 2}};
  if (any_overlap(outs, 3, ins, 4)) return MOK_ERR_INVALID_ARG;
  if ((s = check_device()) != MOK_OK) return s;
  mok_logits_bwd_args a;
  memset(&a, 0, sizeof a);
  a.T = problem->T;
  a.H = (int)H;
  a.E = (int)E;
  a.x = static_cast<const bf16_t*>(x);
  a.wr = w_router;
  a.dl = d_logits;
  a.res = static_cast<const bf16_t*>(residual);
  a.dx = static_cast<bf16_t*>(dx);
  a.dwr = d_w_router;
  a.part = static_cast<float*>(workspace);
  hipStream_t st = (hipStream_t)stream;
  // (no tokens: the sums over them are empty, and there is no dx)
  MOK_RUN("router_logits_backward", mok_launch_logits_bwd(a, st));
  return MOK_OK;
}

}  // extern "C"

// Host-side launch entry points of the router's losses and its dense backward
// (internal to libmok).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mok_device.h"

// as mok_launch_router_forward, keeping the logits [T][E]
hipError_t mok_launch_router_forward_logits(const bf16_t* x, const float* wr, const float* bias, int64_t T, int H,
                                            int E, int k, int32_t* ids, float* w, float* logits, hipStream_t st);

// ---------------------------------------------------------------- losses
struct mok_losses_args {
  int64_t T;
  int E, k;
  const float* logits;
  const int32_t* ids;
  const uint8_t* mask;                 // NULL: every token
  float* losses;
  int32_t* counts;                     // backward: in
  float* prob;
  int32_t* n;                          // backward: in
  uint32_t* part;                      // [groups][2E + 2]: prob, counts, z, n of each workgroup
  const float* d_losses;
  const float* w;                      // NULL with g: no gradient through the combine weights
  const float* g;
  float* d_logits;
};
size_t mok_losses_part_bytes(int64_t T, int E);
hipError_t mok_launch_losses(const mok_losses_args& a, hipStream_t st);
hipError_t mok_launch_losses_backward(const mok_losses_args& a, hipStream_t st);

// ---------------------------------------------------------------- dense backward
struct mok_logits_bwd_args {
  int64_t T;
  int H, E;
  const bf16_t* x;
  const float* wr;                     // [E][H]
  const float* dl;                     // [T][E]
  const bf16_t* res;
  bf16_t* dx;
  float* dwr;                          // [E][H]
  float* part;                         // [slices][E][H]
};
size_t mok_logits_bwd_part_bytes(int64_t T, int H, int E);
hipError_t mok_launch_logits_bwd(const mok_logits_bwd_args& a, hipStream_t st);   // with no tokens: dWr = 0 alone

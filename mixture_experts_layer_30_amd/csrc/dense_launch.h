// Host-side launch entry points of the dense feed-forward block and the MXFP4
// kernels (internal to libmok).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mok_device.h"

// ---------------------------------------------------------------- dense gated FFN, bf16
// Row pitches (ld*) are in elements. Ip = I rounded up to 64: the row pitch of
// each half of dab, whose columns I .. Ip-1 hold zeros, so that the contraction
// of dx over [da | db] never meets a slot of K that straddles the halves.
struct mok_ffn_args {
  int T, H, I, Ip;
  int64_t ldx, ldy;      // x, dx / y, residual, dy
  const bf16_t* x;
  const bf16_t* wg;      // [I][H]
  const bf16_t* wu;      // [I][H]
  const bf16_t* wd;      // [H][I]
  const bf16_t* res;     // added to y (NULL: nothing)
  bf16_t* y;
  bf16_t* h;             // [T][I] forward: h; backward: h from the saved a, b
  bf16_t* ab;            // [T][2I] pre-activations a | b (forward: written, NULL = not kept)
  const bf16_t* dy;
  bf16_t* dab;           // [T][2 Ip] da | db
  bf16_t* dx;
  bf16_t* dwg;
  bf16_t* dwu;
  bf16_t* dwd;
  float* part;           // partial tiles of products split along K
};

enum mok_ffn_op { FFN_GATEUP, FFN_DOWN, FFN_DH, FFN_DWD, FFN_DWGU, FFN_DX, FFN_OPS };

// bytes of partial tiles that `op` needs at this shape (0: not split)
size_t mok_ffn_part_bytes(const mok_ffn_args& a, mok_ffn_op op);
// the product `op` (not those of mok_launch_ffn_grads) with its epilogue (and, where it is split along K, the sum
// of its partial tiles); act: mok_activation, used by FFN_GATEUP and FFN_DH
hipError_t mok_launch_ffn(const mok_ffn_args& a, mok_ffn_op op, int act, hipStream_t st);

// dWd, dWg, dWu and dx together, once FFN_DH has made h and dab; with no tokens
// the weight gradients are zeros and there is no dx
size_t mok_ffn_grads_part_bytes(const mok_ffn_args& a);
hipError_t mok_launch_ffn_grads(const mok_ffn_args& a, hipStream_t st);

// ---------------------------------------------------------------- MX formats
hipError_t mok_launch_mxfp4_quantize(const bf16_t* src, int64_t rows, int64_t K, uint8_t* q, uint8_t* scales,
                                     hipStream_t st);
hipError_t mok_launch_mxfp4_dequantize(const uint8_t* q, const uint8_t* scales, int64_t rows, int64_t K,
                                       bf16_t* dst, hipStream_t st);
hipError_t mok_launch_mxfp8_rows(const void* src, bool f32, int64_t ld, int64_t rows, int64_t K, uint8_t* q,
                                 uint8_t* scales, hipStream_t st);

// d [M][N] (pitch ldd) = A . B^T (+ res), A in MXFP4 or MXFP8, B in MXFP4; with
// glu: B = [Wg; Wu] interleaved by the kernel, N = I, and act(a)*b is written
// as MXFP8 rows hq [M][N] with scales hs [M][N/32], or, with few rows (mok_mx_few),
// as fp32 rows hf [M][N].
struct mok_mx_args {
  int M, N, K;
  bool a8;               // A is E4M3 (else E2M1)
  const uint8_t* a;
  const uint8_t* sa;
  const uint8_t* b;      // B, or Wg
  const uint8_t* sb;
  const uint8_t* b2;     // Wu (glu)
  const uint8_t* sb2;
  bf16_t* d;
  int64_t ldd;
  const bf16_t* res;
  uint8_t* hq;
  uint8_t* hs;
  float* part;
  float* hf;
};
bool mok_mx_few(int M);
size_t mok_mx_part_bytes(const mok_mx_args& a, bool glu);
hipError_t mok_launch_mx(const mok_mx_args& a, bool glu, int act, hipStream_t st);
